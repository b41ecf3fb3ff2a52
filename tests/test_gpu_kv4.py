"""The 4-bit cache and the attention over it, on the GPU against the float64 oracle."""

import numpy as np
import pytest
import torch

import cache_gating_kv_b200 as fc
from oracle import kv4_oracle as O

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16, F32 = torch.bfloat16, torch.float32


def _randn(g, *shape):
    return torch.randn(*shape, generator=g)


def _bytes(t):
    return t.cpu().numpy()


# ---- store and load ---------------------------------------------------------------
def _store_case(N, H, L, d, cap, row0, dtype, e=0, B=0, layout="nhld", scale=1.0, seed=0):
    g = torch.Generator().manual_seed(seed)

    def make():
        t = _randn(g, N, H, L, d) * torch.exp(_randn(g, N, H, L, 1)) * scale
        t = t.to(dtype).to(DEV)
        return t.permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3) if layout == "nlhd" else t

    k, v = make(), make()
    cache = fc.fc_kv4_cache(N, H, cap, d, k_exp=e, v_exp=-e)
    for t in (cache.k_codes, cache.k_scales, cache.v_codes, cache.v_scales):
        t.fill_(0x5A)
    idx = None
    rows = B or L
    if B:
        idx = torch.randint(-1, L, (N, H, B), generator=g).to(torch.int32)
        idx[0, 0, 0] = L + 3  # outside: zeros
    first = row0 if isinstance(row0, list) else [row0] * N
    r0 = torch.tensor(row0, dtype=torch.int32, device=DEV) if isinstance(row0, list) else row0
    fc.fc_kv4_store(k, v, cache, row0=r0, idx=None if idx is None else idx.to(DEV))
    assert fc.fc_last_launches() == 1
    torch.cuda.synchronize()
    outs = [torch.full((N, H, rows, d), 9.0, dtype=dtype, device=DEV) for _ in range(2)]
    fc.fc_kv4_load(cache, outs[0], outs[1], row0=r0)
    torch.cuda.synchronize()
    for x, codes, scales, ex, out in ((k, cache.k_codes, cache.k_scales, e, outs[0]),
                                      (v, cache.v_codes, cache.v_scales, -e, outs[1])):
        xn = x.float().cpu().numpy()
        if B:
            src = np.zeros((N, H, B, d), np.float32)
            for n in range(N):
                for h in range(H):
                    for r in range(B):
                        j = int(idx[n, h, r])
                        if 0 <= j < L:
                            src[n, h, r] = xn[n, h, j]
            xn = src
        code, sc = O.kv4_quantise(xn, ex)
        packed = O.kv4_pack(code)
        want_c = np.full((N, H, cap, d // 2), 0x5A, np.uint8)
        want_s = np.full((N, H, cap, d // 16), 0x5A, np.uint8)
        want_o = np.zeros((N, H, rows, d))
        for n in range(N):
            for r in range(rows):
                at = first[n] + r
                if 0 <= at < cap:
                    want_c[n, :, at], want_s[n, :, at] = packed[n, :, r], sc[n, :, r]
                    want_o[n, :, r] = O.kv4_values(packed[n, :, r], sc[n, :, r], ex)
        assert np.array_equal(_bytes(scales), want_s)
        assert np.array_equal(_bytes(codes), want_c)
        assert np.array_equal(out.double().cpu().numpy(), want_o)
    return cache, outs


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("N,H,L,cap,row0,e", [
    (1, 1, 1, 16, 0, 0), (1, 3, 33, 48, 15, 0), (2, 2, 17, 32, 20, 3), (3, 5, 1, 64, [0, 63, 7], -4),
    (2, 1, 200, 208, 0, 0), (2, 3, 9, 16, [-4, 12], 1), (1, 2, 40, 32, 100, 0)])
def test_store_and_load_bitwise(N, H, L, cap, row0, e, d, dtype):
    _store_case(N, H, L, d, cap, row0, dtype, e)
    _store_case(N, H, L, d, cap, row0, dtype, e, layout="nlhd", seed=1)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_store_selected_rows(dtype):
    _store_case(2, 3, 70, 128, 64, 0, dtype, B=41)
    _store_case(1, 2, 5, 64, 32, 16, dtype, B=16, e=2)
    _store_case(1, 2, 3, 64, 32, 0, dtype, B=1)


@pytest.mark.parametrize("scale", [2.0 ** -12, 1e-30, 300.0, 1e30])
def test_store_ranges(scale):
    """Scales that are zero, subnormal, and saturated."""
    _store_case(1, 2, 64, 128, 64, 0, F32, scale=scale)


def test_store_ties_and_every_scale():
    """Numbers on and beside the borders between codes, under every scale byte."""
    s = O.E4M3[1:127]
    mid = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])
    t = np.zeros((1, 1, 126, 64), np.float32)
    t[0, 0, :, 0:64:16] = 6.0
    for i in range(7):
        t[0, 0, :, 1 + 2 * i] = mid[i]
        t[0, 0, :, 2 + 2 * i] = -mid[i]
        t[0, 0, :, 17 + 2 * i] = np.nextafter(np.float32(mid[i]), np.float32(9))
        t[0, 0, :, 18 + 2 * i] = -np.nextafter(np.float32(mid[i]), np.float32(0))
    x = (t * s[None, None, :, None]).astype(np.float32)
    k = torch.from_numpy(x).to(DEV)
    cache = fc.fc_kv4_cache(1, 1, 128, 64)
    fc.fc_kv4_store(k, -k, cache)
    code, sc = O.kv4_quantise(x)
    assert np.array_equal(sc[0, 0, :, 0], np.arange(1, 127))  # the scale each row was made for
    assert np.array_equal(_bytes(cache.k_scales)[0, 0, :126], sc[0, 0])
    assert np.array_equal(_bytes(cache.k_codes)[0, 0, :126], O.kv4_pack(code)[0, 0])
    assert np.array_equal(_bytes(cache.v_codes)[0, 0, :126], O.kv4_pack(O.kv4_quantise(-x)[0])[0, 0])


def test_store_special_values():
    x = torch.randn(1, 1, 4, 64, device=DEV)
    x[0, 0, 0, 3] = float("nan")
    x[0, 0, 1, 20] = float("inf")
    x[0, 0, 1, 21] = -float("inf")
    x[0, 0, 2] = 0.0
    for t in (x, x.bfloat16()):
        cache = fc.fc_kv4_cache(1, 1, 16, 64)
        fc.fc_kv4_store(t, t, cache)
        o = [torch.empty(1, 1, 4, 64, dtype=t.dtype, device=DEV) for _ in range(2)]
        fc.fc_kv4_load(cache, *o)
        y = o[0][0, 0].float()
        assert torch.isnan(y[0, :16]).all() and torch.isfinite(y[0, 16:]).all()
        assert y[1, 20] == 2688 and y[1, 21] == -2688 and torch.isfinite(y[1]).all()
        assert (y[2] == 0).all()
        assert torch.equal(o[0].isnan(), o[1].isnan())


def test_storing_loaded_rows_changes_nothing():
    cache, outs = _store_case(2, 3, 90, 128, 96, 0, BF16, seed=7)
    again = fc.fc_kv4_cache(2, 3, 96, 128)
    fc.fc_kv4_store(outs[0], outs[1], again)
    for a, b, s, t in ((again.k_codes, cache.k_codes, again.k_scales, cache.k_scales),
                       (again.v_codes, cache.v_codes, again.v_scales, cache.v_scales)):
        normal = t[:, :, :90] >= 0x08  # of each group
        assert normal.float().mean() > 0.9
        assert torch.equal(s[:, :, :90][normal], t[:, :, :90][normal])
        of_byte = normal.repeat_interleave(8, -1)
        assert torch.equal(a[:, :, :90][of_byte], b[:, :, :90][of_byte])


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("d,rot,sections", [(128, 128, None), (128, 64, [10, 10, 12]), (64, 24, None), (64, 32, None),
                                            (64, 6, [1, 1, 1])])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_store_rotates_as_fc_rope(dtype, d, rot, sections, interleaved):
    """Rotating on the way gives the bits of fc_rope in float32 and a plain store."""
    g = torch.Generator().manual_seed(11)
    N, H, L = 2, 3, 37
    k = _randn(g, N, L, H, d).to(dtype).to(DEV).permute(0, 2, 1, 3)
    v = _randn(g, N, H, L, d).to(dtype).to(DEV)
    plan = fc.fc_rope_init(rot, int(interleaved), sections=sections, scaling=fc.FC_ROPE_YARN, factor=4.0,
                           orig_len=100)
    pos = torch.randint(0, 5000, (plan.n_axes, N, L), generator=g).to(torch.int32).to(DEV)
    a, b = fc.fc_kv4_cache(N, H, 48, d, 1, 0), fc.fc_kv4_cache(N, H, 48, d, 1, 0)
    fc.fc_kv4_store(k, v, a, row0=3, rope=plan, pos=pos)
    k32 = torch.empty(N, H, L, d, device=DEV)
    fc.fc_rope(k.float(), k32, pos, plan)
    fc.fc_kv4_store(k32, v.float(), b, row0=3)
    for n in ("k_codes", "k_scales", "v_codes", "v_scales"):
        assert torch.equal(getattr(a, n), getattr(b, n)), n


def test_store_and_load_refusals():
    k = torch.zeros(1, 2, 4, 64, device=DEV)
    c = fc.fc_kv4_cache(1, 2, 16, 64)
    o = torch.empty_like(k)
    idx = torch.zeros(1, 2, 3, dtype=torch.int32, device=DEV)
    plan, pos = fc.fc_rope_init(64), torch.zeros(4, dtype=torch.int32, device=DEV)
    for call in [lambda: fc.fc_kv4_store(k.cpu(), k, c), lambda: fc.fc_kv4_store(k, k.bfloat16(), c),
                 lambda: fc.fc_kv4_store(k[:, :1], k[:, :1], c), lambda: fc.fc_kv4_store(k, k, c, row0=-1),
                 lambda: fc.fc_kv4_store(k.half(), k.half(), c), lambda: fc.fc_kv4_store(k, k, c, idx=idx.long()),
                 lambda: fc.fc_kv4_store(k, k, c, idx=idx[:, :1]), lambda: fc.fc_kv4_store(k, k, c, rope=plan),
                 lambda: fc.fc_kv4_store(k, k, c, rope=fc.fc_rope_init(128), pos=pos),
                 lambda: fc.fc_kv4_store(k[..., :32], k[..., :32], c),
                 lambda: fc.fc_kv4_store(k, k, c, row0=torch.zeros(2, dtype=torch.int32, device=DEV)),
                 lambda: fc.fc_kv4_load(c, o, o), lambda: fc.fc_kv4_load(c, o, o.clone(), row0=-2),
                 lambda: fc.fc_kv4_load(c, o.half(), o.half()), lambda: fc.fc_kv4_load(c, o[:, :1], o[:, 1:]),
                 lambda: fc.fc_kv4_load(c, o, o[:, :1].expand(1, 2, 4, 64)),
                 lambda: fc.Kv4Cache(c.k_codes, c.v_codes, c.v_codes, c.v_scales)]:
        with pytest.raises(fc.FlowCacheError):
            call()
    with pytest.raises(fc.FlowCacheError, match="UNSUPPORTED"):
        fc.fc_kv4_store(k, k, c, idx=idx, rope=plan, pos=pos)
    with pytest.raises(fc.FlowCacheError, match="UNSUPPORTED"):
        c96 = fc.fc_kv4_cache(1, 1, 16, 96)
        fc.fc_kv4_load(c96, torch.empty(1, 1, 4, 96, device=DEV), torch.empty(1, 1, 4, 96, device=DEV))
    with pytest.raises(fc.FlowCacheError, match="cap"):
        c20 = fc.fc_kv4_cache(1, 1, 20, 64)
        fc.fc_kv4_load(c20, torch.empty(1, 1, 4, 64, device=DEV), torch.empty(1, 1, 4, 64, device=DEV))
    assert (c.k_codes == 0).all() and (c.v_scales == 0).all()


# ---- attention ----------------------------------------------------------------------
def _cache(g, N, H, cap, d, ek=0, ev=0, spread=0.5):
    c = fc.fc_kv4_cache(N, H, cap, d, ek, ev)
    k = (_randn(g, N, H, cap, d) * torch.exp(spread * _randn(g, 1, H, 1, d))).to(DEV)
    fc.fc_kv4_store(k, _randn(g, N, H, cap, d).to(DEV), c)
    return c


def _numbers(c, n_rows):
    return [O.kv4_values(_bytes(a)[:, :, :n_rows], _bytes(s)[:, :, :n_rows], e)
            for a, s, e in ((c.k_codes, c.k_scales, c.struct.k_exp), (c.v_codes, c.v_scales, c.struct.v_exp))]


def _attend(q, c, lens, max_len=None, causal=False, scale=0.0, out=None, want_lse=True):
    N, Hq, Lq, d = q.shape
    code = fc.FC_BF16 if q.dtype == BF16 else fc.FC_F32
    m = c.cap if max_len is None else max_len
    ws = fc.workspace(fc.fc_kv4_attention_workspace_size(code, N, Hq, c.H, Lq, m, d))
    ws[4:].fill_(0xFF)  # nothing but the error word is carried
    out = torch.full((N, Hq, Lq, d), 7.0, dtype=q.dtype, device=DEV) if out is None else out
    lse = torch.full((N, Hq, Lq), 7.0, device=DEV) if want_lse else None
    fc.fc_kv4_attention(q, c, lens, out, ws, max_len=max_len, causal=causal, scale=scale, lse=lse)
    _attend.launches = fc.fc_last_launches()
    torch.cuda.synchronize()
    assert fc.fc_check_workspace(fc.FC_WS_IMPORTANCE, ws)
    return out, lse


def _check(q, c, lens, out, lse, causal=False, scale=None):
    """Bounds: a logit sums d products, each addition at most 2^-23 of the reach
    (tensor cores may cut), and its float32 multiply-add and base-2 exponential add
    2^-22 of the logit's size and of one; a probability rounds to float16 (bf16
    queries: half a step 2^-11) or to two of them (2^-21, the smaller term subnormal at
    times); numerator and denominator carry each once; the sums over keys, at most 2^-23
    per step of 32 keys and warp; the result rounds once.  float16 ends at 2^-24, so a
    probability is also off by up to 2^-25; the largest enters as 2^5 at least (float32:
    as 2^14), so that is 2^-30 (2^-39) of it for every key, however small its
    probability: over the keys, flat times that (denominators are float32 sums)."""
    N, Hq, Lq, d = q.shape
    top = max(max(lens), 1)
    k, v = _numbers(c, top)
    o, l, spread, reach, flat = O.kv4_attention(q.double().cpu().numpy(), k, v, lens, causal, scale)
    assert np.isfinite(l).any() or max(lens) <= 0 or causal
    with np.errstate(invalid="ignore"):
        dx = (d + 8) * 2.0 ** -23 * reach + 2.0 ** -22
        keys = 2.0 ** -23 * (top / 32 + 64)
        p = (2.0 ** -11 if q.dtype == BF16 else 2.0 ** -21) + 2 * dx + 2 * keys
        tol = torch.finfo(q.dtype).eps / 2 * np.abs(o) + (p[..., None] + 2.0 ** -22) * spread
        tol += (2.0 ** -30 if q.dtype == BF16 else 2.0 ** -39) * flat
        got = out.double().cpu().numpy()
        assert np.isfinite(got).all()
        worst = (np.abs(got - o) - tol).max()
        assert worst <= 0, f"off by {worst} over the bound"
        if lse is not None:
            gl = lse.double().cpu().numpy()
            assert np.array_equal(np.isneginf(gl), np.isneginf(l))
            f = np.isfinite(l)
            assert (np.abs(gl - l)[f] <= (dx + keys + 2.0 ** -22 * (1 + np.abs(l)))[f]).all()
    empty = np.isneginf(l)
    assert (got[empty] == 0).all()


SHAPES = [  # N, Hq, Hkv, Lq, lens, cap, causal
    (1, 1, 1, 1, [1], 16, False), (1, 2, 1, 1, [0], 16, False), (2, 4, 2, 1, [15, 16], 16, True),
    (3, 5, 1, 1, [17, 31, 33], 48, False), (2, 8, 8, 1, [127, 300], 304, True),
    (2, 40, 8, 1, [513, 2000], 2000, True), (1, 8, 2, 1, [5000], 5008, False),
    (1, 16, 1, 1, [640], 640, False), (1, 17, 1, 1, [700], 704, False), (1, 20, 1, 2, [90], 96, True),
    (2, 6, 2, 5, [3, 600], 608, True), (1, 2, 2, 16, [40], 48, True), (1, 2, 2, 17, [1000], 1008, True),
    (2, 3, 1, 33, [70, 0], 80, True), (1, 2, 1, 64, [64], 64, True), (1, 1, 1, 129, [500], 512, False),
    (2, 2, 1, 70, [300, 20], 304, True), (1, 2, 2, 257, [257], 272, True), (1, 3, 3, 200, [1111], 1120, False),
    (2, 1, 1, 130, [129, 4], 144, True), (1, 4, 1, 100, [777], 784, True), (1, 1, 1, 300, [40], 48, True),
]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("N,Hq,Hkv,Lq,lens,cap,causal", SHAPES)
def test_attention_shapes(N, Hq, Hkv, Lq, lens, cap, causal, d, dtype):
    g = torch.Generator().manual_seed(Lq * 1000 + cap)
    c = _cache(g, N, Hkv, cap, d)
    q = _randn(g, N, Hq, Lq, d).to(dtype).to(DEV)
    dl = torch.tensor(lens, dtype=torch.int32, device=DEV)
    out, lse = _attend(q, c, dl, causal=causal)
    _check(q, c, lens, out, lse, causal)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("Lq", [1, 40, 200])
def test_attention_strides_exponents_and_scale(Lq, dtype):
    g = torch.Generator().manual_seed(21)
    N, Hq, Hkv, d = 2, 6, 3, 128
    c = _cache(g, N, Hkv, 416, d, ek=3, ev=-2)
    q = _randn(g, N, Lq, 2, Hq, d).to(dtype).to(DEV)[:, :, 1].permute(0, 2, 1, 3)
    buf = torch.full((N, Lq, Hq + 1, d), 5.0, dtype=dtype, device=DEV)
    out, lse = _attend(q, c, torch.tensor([400, 201], dtype=torch.int32, device=DEV), causal=True, scale=0.05,
                       out=buf[:, :, :Hq].permute(0, 2, 1, 3))
    _check(q, c, [400, 201], out, lse, True, 0.05)
    assert (buf[:, :, Hq] == 5.0).all()
    out2, _ = _attend(q, c, torch.tensor([400, 201], dtype=torch.int32, device=DEV), causal=True, scale=0.05,
                      want_lse=False)
    assert torch.equal(out2, out)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("Lq", [1, 24, 150])
@pytest.mark.parametrize("kind", ["rising", "falling", "spike", "tiny", "zero", "wide"])
def test_attention_logit_ranges(kind, Lq, dtype):
    """Running maxima that move at every step, once, or late; queries of zeros, of tiny
    numbers and of numbers 2^20 apart in a row."""
    g = torch.Generator().manual_seed(31)
    N, H, d, cap = 1, 2, 64, 1200
    k = _randn(g, N, H, cap, d) * 0.1
    q = _randn(g, N, H, Lq, d) * 0.1
    ramp = torch.linspace(0, 1, cap)
    if kind in ("rising", "falling"):
        k[..., 0] += 40 * (ramp if kind == "rising" else 1 - ramp)
        q[..., 0] = 4.0
    elif kind == "spike":
        k[:, :, 1111, 0] = 60.0
        q[..., 0] = 5.0
    elif kind == "tiny":
        q *= 1e-30
    elif kind == "zero":
        q.zero_()
    else:
        q[..., ::2] *= 2.0 ** 10
        q[..., 1::2] *= 2.0 ** -10
        k[..., ::2] *= 2.0 ** -6
    c = fc.fc_kv4_cache(N, H, cap, d)
    fc.fc_kv4_store(k.to(DEV), _randn(g, N, H, cap, d).to(DEV), c)
    q = q.to(dtype).to(DEV)
    out, lse = _attend(q, c, [cap][0])
    _check(q, c, [cap], out, lse)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("Lq", [1, 3, 20, 140])
def test_attention_nan_that_nobody_sees(Lq, dtype):
    """NaN scales behind the sequences, and in keys that only later queries see."""
    g = torch.Generator().manual_seed(41)
    N, Hq, Hkv, d, cap = 2, 4, 2, 128, 464
    c = _cache(g, N, Hkv, cap, d)
    lens = [450, 170]
    q = _randn(g, N, Hq, Lq, d).to(dtype).to(DEV)
    dl = torch.tensor(lens, dtype=torch.int32, device=DEV)
    want, want_l = _attend(q, c, dl, causal=True)
    _check(q, c, lens, want, want_l, True)
    for n in range(N):
        c.k_scales[n, :, lens[n]:] = 0x7F
        c.v_scales[n, :, lens[n]:] = 0xFF
        c.k_codes[n, :, lens[n]:] = 0x77
    out, lse = _attend(q, c, dl, causal=True)
    assert torch.equal(out, want) and torch.equal(lse, want_l)
    # the last key: of all queries only the last one sees it
    for part in (c.v_scales, c.k_scales):
        kept = part.clone()
        part[0, 1, lens[0] - 1, 2] = 0x7F
        out, lse = _attend(q, c, dl, causal=True)
        G = Hq // Hkv
        assert torch.isnan(out[0, G:, -1]).all()
        seen = torch.ones(N, Hq, Lq, dtype=torch.bool, device=DEV)
        seen[0, G:, -1] = False
        assert torch.equal(out[seen], want[seen]) and torch.equal(lse[seen], want_l[seen])
        part.copy_(kept)


def test_attention_lengths_are_clamped_and_may_be_host_side():
    g = torch.Generator().manual_seed(51)
    c = _cache(g, 3, 2, 208, 64)
    q = _randn(g, 3, 4, 1, 64).to(BF16).to(DEV)
    a = _attend(q, c, torch.tensor([-5, 1000, 100], dtype=torch.int32, device=DEV), max_len=200)
    b = _attend(q, c, torch.tensor([0, 200, 100], dtype=torch.int32, device=DEV), max_len=200)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    a = _attend(q, c, 130)
    b = _attend(q, c, torch.full((3,), 130, dtype=torch.int32, device=DEV))
    assert torch.equal(a[0], b[0])
    for n in (0, 0.0):
        o, l = _attend(q, c, int(n))
        assert (o == 0).all() and torch.isneginf(l).all()
    code = fc.FC_BF16
    ws = fc.workspace(fc.fc_kv4_attention_workspace_size(code, 3, 4, 2, 1, 208, 64))
    o2 = torch.empty_like(q)
    fc.fc_kv4_attention(q, c, 130, o2, ws)  # a workspace made for the longest length
    assert torch.equal(o2, a[0])


@pytest.mark.parametrize("Lq", [1, 200])
def test_attention_far_offsets(Lq):
    """Rows whose bytes lie beyond 2^32 from the start of the cache."""
    g = torch.Generator().manual_seed(61)
    N, H, d, cap = 3, 2, 128, 1 << 24  # codes of a head: 2^30 bytes
    c = fc.Kv4Cache(*[torch.empty(N, H, cap, w, dtype=torch.uint8, device=DEV) for w in (64, 8, 64, 8)])
    k, v = _randn(g, 1, H, 300, d).to(DEV), _randn(g, 1, H, 300, d).to(DEV)
    last = fc.Kv4Cache(c.k_codes[2:], c.k_scales[2:], c.v_codes[2:], c.v_scales[2:])
    fc.fc_kv4_store(k, v, last, row0=0)
    q = _randn(g, N, H, Lq, d).to(BF16).to(DEV)
    lens = [0, 0, 300]
    out, lse = _attend(q, c, torch.tensor(lens, dtype=torch.int32, device=DEV), max_len=512)
    small = fc.Kv4Cache(*[t[2:, :, :304].contiguous() for t in (c.k_codes, c.k_scales, c.v_codes, c.v_scales)])
    _check(q[2:], small, [300], out[2:], lse[2:])
    # the far end of the last head
    fc.fc_kv4_store(k, v, c.__class__(c.k_codes[2:], c.k_scales[2:], c.v_codes[2:], c.v_scales[2:]), row0=cap - 300)
    ko, vo = torch.empty(1, H, 300, d, device=DEV), torch.empty(1, H, 300, d, device=DEV)
    fc.fc_kv4_load(last, ko, vo, row0=cap - 300)
    k0, v0 = torch.empty_like(ko), torch.empty_like(vo)
    fc.fc_kv4_load(last, k0, v0, row0=0)
    assert torch.equal(ko, k0) and torch.equal(vo, v0)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype,N,Hq,Hkv,Lq,lens,causal", [
    (BF16, 3, 2, 2, 150, [2600, 130, 0], False), (BF16, 2, 4, 1, 40, [4090, 1700], True),
    (BF16, 1, 3, 3, 300, [5000], True), (BF16, 2, 2, 1, 9, [6000, 3001], True),
    (F32, 2, 2, 2, 70, [1500, 40], True), (F32, 1, 12, 1, 1, [3000], False)])
def test_attention_long_axes_are_joined(dtype, N, Hq, Hkv, Lq, lens, causal, d):
    """Units that several blocks share, in both kernels, beside short and empty ones."""
    g = torch.Generator().manual_seed(57)
    cap = (max(lens) + 15) // 16 * 16
    c = _cache(g, N, Hkv, cap, d)
    q = _randn(g, N, Hq, Lq, d).to(dtype).to(DEV)
    out, lse = _attend(q, c, torch.tensor(lens, dtype=torch.int32, device=DEV), causal=causal)
    assert _attend.launches == 2
    _check(q, c, lens, out, lse, causal)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("N,Hkv", [(70, 3), (700, 8)])
def test_attention_of_many_sequences(N, Hkv, dtype):
    """More units than a block's threads add up at once, and more than are shared out."""
    g = torch.Generator().manual_seed(59)
    cap, d = 528, 64
    c = fc.fc_kv4_cache(N, Hkv, cap, d)
    for t in (c.k_codes, c.v_codes):
        t.random_(0, 256)
    for t in (c.k_scales, c.v_scales):
        t.random_(0x28, 0x40)  # about a tenth to two
    lens = torch.randint(0, cap + 1, (N,), generator=g, dtype=torch.int32)
    lens[3], lens[5], lens[-1] = 0, cap, 1
    q = _randn(g, N, 2 * Hkv, 1, d).to(dtype).to(DEV)
    out, lse = _attend(q, c, lens.to(DEV))
    some = [0, 3, 5, 41, N - 1]
    few = fc.Kv4Cache(*[t[some].contiguous() for t in (c.k_codes, c.k_scales, c.v_codes, c.v_scales)])
    _check(q[some], few, [int(lens[n]) for n in some], out[some], lse[some])


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("tail", [1, 33, 65, 96])
def test_attention_short_last_stages(tail, d, dtype):
    """Pieces of 7 to 20 stages of 128 keys whose last has keys for one to three of its four
    warps, with a late maximum among one warp's keys: 256 units of the same numbers, ten
    calls, all bitwise the same."""
    g = torch.Generator().manual_seed(53 + tail)
    N, H = 32, 8
    for stages in (7, 8, 9, 13, 20):
        keys = (stages - 1) * 128 + tail
        cap = (keys + 15) // 16 * 16
        k, v = _randn(g, 1, 1, cap, d), _randn(g, 1, 1, cap, d)
        q = _randn(g, 1, 1, 1, d)
        k[0, 0, keys - 128 + 40] = 3 * q[0, 0, 0]
        one = fc.fc_kv4_cache(1, 1, cap, d)
        fc.fc_kv4_store(k.to(DEV), v.to(DEV), one)
        c = fc.Kv4Cache(*[t.expand(N, H, -1, -1).contiguous()
                          for t in (one.k_codes, one.k_scales, one.v_codes, one.v_scales)])
        q = q.to(dtype).to(DEV).expand(N, H, 1, d)
        out, lse = _attend(q, c, keys)
        assert _attend.launches == 1  # a block for each unit
        _check(q[:1, :1], one, [keys], out[:1, :1], lse[:1, :1])
        for _ in range(10):
            assert torch.equal(out, out[:1, :1].expand_as(out)) and torch.equal(lse, lse[:1, :1].expand_as(lse))
            out, lse = _attend(q, c, keys)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("keys", [49, 1000, 2900])
def test_attention_f32_divides_exactly(keys, d):
    """Equal keys and equal values, float32: every probability is the same power of two, so
    numerator (n v 2^k, v of six bits) and denominator are exact and so is the quotient."""
    g = torch.Generator().manual_seed(keys)
    for n in range(keys - 8, keys + 1):
        c = fc.fc_kv4_cache(1, 2, 2912, d, v_exp=3)
        v = _randn(g, 1, 2, 1, d).to(DEV).expand(1, 2, n, d)
        fc.fc_kv4_store(torch.zeros(1, 2, n, d, device=DEV), v, c)
        got = [torch.empty(1, 2, n, d, device=DEV) for _ in range(2)]
        fc.fc_kv4_load(c, *got)
        q = _randn(g, 1, 4, 3, d).to(DEV)
        out, _ = _attend(q, c, n, max_len=n)
        assert torch.equal(out, got[1][:, :, :1].repeat_interleave(2, 1).expand_as(out)), n


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G", [1, 12])
def test_attention_f32_sums_are_not_biased(G, d):
    """Values of six (code 6, scale 1), float32: the result is six times the sum of the probabilities over itself,
    by the two ways in which the kernel adds them, over 256 x G rows of 8192 keys each, so its mean over the rows
    shows whether one of them leans to a side.

    Roundings to nearest have no mean: 64 steps of a warp and the join of eight warps, in
    numerator and denominator, each at most 2^-24, are 2^-24 sqrt(2 x 72 / 3) = 7 x 2^-24 a
    row in the root mean square, 6 deviations of the mean over 256 rows 2.6 x 2^-24.  One
    product on the tensor cores may cut what it adds: 16 products of a step and the two
    terms of the probabilities, half of 2^-24 each at most of their largest and on average
    half of that, below 2^-24 of their sum.  The quotient and its result round to nearest.
    2^-22 in all.  (128 sums one behind the other, cut at 2^-23 of what they have reached,
    would lean by some 128 / 4 x 2^-23 = 2^-18.)"""
    g = torch.Generator().manual_seed(67)
    N, H, keys = 64, 4, 8192
    one = fc.fc_kv4_cache(1, 1, keys, d)
    fc.fc_kv4_store(_randn(g, 1, 1, keys, d).to(DEV), torch.full((1, 1, keys, d), 6.0, device=DEV), one)
    c = fc.Kv4Cache(*[t.expand(N, H, -1, -1).contiguous()
                      for t in (one.k_codes, one.k_scales, one.v_codes, one.v_scales)])
    q = _randn(g, N, H * G, 1, d).to(DEV)
    out, _ = _attend(q, c, keys)
    off = out.double()[..., 0].mean().item() / 6 - 1
    assert abs(off) <= 2.0 ** -22, f"{off * 2 ** 24:.2f} x 2^-24"


def test_attention_refusals():
    c = fc.fc_kv4_cache(2, 2, 32, 64)
    q = torch.zeros(2, 4, 3, 64, device=DEV, dtype=BF16)
    o = torch.empty_like(q)
    ws = fc.workspace(1 << 16)
    lens = torch.zeros(2, dtype=torch.int32, device=DEV)
    for call in [lambda: fc.fc_kv4_attention(q[:, :3], c, lens, o[:, :3], ws),
                 lambda: fc.fc_kv4_attention(q[:1], c, lens, o[:1], ws),
                 lambda: fc.fc_kv4_attention(q, c, lens[:1], o, ws), lambda: fc.fc_kv4_attention(q, c, lens.long(), o, ws),
                 lambda: fc.fc_kv4_attention(q, c, lens, o, ws, max_len=33),
                 lambda: fc.fc_kv4_attention(q, c, -1, o, ws), lambda: fc.fc_kv4_attention(q, c, lens, q, ws),
                 lambda: fc.fc_kv4_attention(q, c, lens, o.float(), ws), lambda: fc.fc_kv4_attention(q.half(), c, lens, o.half(), ws),
                 lambda: fc.fc_kv4_attention(q, c, lens, o, ws[:100]),
                 lambda: fc.fc_kv4_attention(q, c, lens, o, ws, lse=torch.empty(2, 4, 3, device=DEV, dtype=BF16)),
                 lambda: fc.fc_kv4_attention(q.cpu(), c, lens, o, ws)]:
        with pytest.raises(fc.FlowCacheError):
            call()
    with pytest.raises(fc.FlowCacheError, match="WORKSPACE"):
        fc.fc_kv4_attention(q, c, lens, o, ws[:16])


def test_attention_is_deterministic_and_captures():
    """Bitwise the same again, on another stream, in a graph, and in two graphs that share
    one workspace and follow one another."""
    g = torch.Generator().manual_seed(71)
    c = _cache(g, 2, 2, 2000, 128)
    for Lq in (1, 180):
        q = _randn(g, 2, 4, Lq, 128).to(BF16).to(DEV)
        lens = torch.tensor([1999, 700], dtype=torch.int32, device=DEV)
        want, lse = _attend(q, c, lens, causal=True)
        ws = fc.workspace(fc.fc_kv4_attention_workspace_size(fc.FC_BF16, 2, 4, 2, Lq, 2000, 128))
        o = torch.empty_like(q)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            for _ in range(5):
                fc.fc_kv4_attention(q, c, lens, o, ws, causal=True)
        torch.cuda.synchronize()
        assert torch.equal(o, want)
        graphs, outs = [], []
        for _ in range(2):
            gr, o = torch.cuda.CUDAGraph(), torch.zeros_like(q)
            with torch.cuda.graph(gr):
                fc.fc_kv4_attention(q, c, lens, o, ws, causal=True)
            graphs.append(gr)
            outs.append(o)
        for gr in graphs + graphs:
            gr.replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[0], want) and torch.equal(outs[1], want)
        lens.copy_(torch.tensor([1500, 3], dtype=torch.int32))  # a replay follows the lengths
        graphs[0].replay()
        want2, _ = _attend(q, c, lens, causal=True)
        assert torch.equal(outs[0], want2)


# ---- together -----------------------------------------------------------------------
def test_decode_steps_together():
    """A prompt and eight tokens of two sequences: rotated queries over keys that are
    rotated into the cache, one row at a time; captured once, replayed per token."""
    g = torch.Generator().manual_seed(81)
    N, Hq, Hkv, d, P, cap, steps = 2, 4, 2, 64, 50, 64, 8
    plan = fc.fc_rope_init(d)
    cache = fc.fc_kv4_cache(N, Hkv, cap, d)
    k0, v0 = _randn(g, N, P, Hkv, d).to(BF16).to(DEV), _randn(g, N, P, Hkv, d).to(BF16).to(DEV)
    pos = torch.arange(P, dtype=torch.int32, device=DEV).repeat(N, 1)
    fc.fc_kv4_store(k0.permute(0, 2, 1, 3), v0.permute(0, 2, 1, 3), cache, rope=plan, pos=pos)
    lens = torch.tensor([P, 20], dtype=torch.int32, device=DEV)  # the second prompt is padded
    q, k, v = (torch.empty(N, h, 1, d, dtype=BF16, device=DEV) for h in (Hq, Hkv, Hkv))
    at = lens.clone()
    qr, out = torch.empty_like(q), torch.empty_like(q)
    ws = fc.workspace(fc.fc_kv4_attention_workspace_size(fc.FC_BF16, N, Hq, Hkv, 1, cap, d))

    def step():
        fc.fc_rope(q, qr, at, plan)
        fc.fc_kv4_store(k, v, cache, row0=at, rope=plan, pos=at)
        lens.copy_(at + 1)
        fc.fc_kv4_attention(qr, cache, lens, out, ws, causal=True)
        at.add_(1)

    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        step()
    ks = [[k0[n, i].float().cpu().numpy() for i in range([P, 20][n])] for n in range(N)]
    vs = [[v0[n, i].float().cpu().numpy() for i in range([P, 20][n])] for n in range(N)]
    w = np.array(plan.turns[: d // 2])
    for t in range(steps):
        new = [_randn(g, *x.shape).to(BF16) for x in (q, k, v)]
        for x, y in zip((q, k, v), new):
            x.copy_(y)
        gr.replay()
        torch.cuda.synchronize()
        for n in range(N):
            ks[n].append(new[1][n, :, 0].float().numpy())
            vs[n].append(new[2][n, :, 0].float().numpy())
            L = len(ks[n])
            assert int(lens[n]) == L
            kk, vv = _numbers(cache, L)
            # the cache holds the rotated keys to the format's half step: |y| / 12 of a
            # group's largest for the scale's rounding and the widest code gap
            rot = O.rope(np.stack(ks[n], 1)[None], np.arange(L)[None, None], w)
            big = np.abs(rot).reshape(1, Hkv, L, -1, 16).max(-1).repeat(16, -1)
            assert (np.abs(kk[n:n + 1] - rot) <= big * (1 / 6 + 1 / 16) + 1e-6).all()
            qn = O.rope(new[0][n:n + 1].double().numpy(), [[[L - 1]]], w)
            o, _, spread, _, _ = O.kv4_attention(qn, kk[n:n + 1], vv[n:n + 1], [L], True)
            # the rotated query rounds to bf16: 2^-8 of every logit's reach (below 8 here)
            tol = 2.0 ** -8 * np.abs(o) + (2.0 ** -11 + 2 * 8 * 2.0 ** -8) * spread
            assert (np.abs(out[n:n + 1].double().cpu().numpy() - o) <= tol).all()


def test_compression_into_the_cache_together():
    """A finished chunk: load the cache for scoring, select, store the kept rows into the
    other cache, and attend over it."""
    g = torch.Generator().manual_seed(91)
    H, Lq, L, B, d = 3, 130, 400, 200, 128
    c = _cache(g, 1, H, L, d)
    k, v = (torch.empty(1, H, L, d, dtype=BF16, device=DEV) for _ in range(2))
    fc.fc_kv4_load(c, k, v)
    q = _randn(g, H, Lq, d).to(BF16).to(DEV)
    imp, red = torch.empty(H, L, device=DEV), torch.empty(H, L, device=DEV)
    idx = torch.empty(H, B, dtype=torch.int32, device=DEV)
    fc.fc_kv_importance(q, k[0], imp, fc.workspace(fc.fc_importance_workspace_size(fc.FC_BF16, H, Lq, L, d)))
    fc.fc_kv_redundancy(k[0], red, fc.workspace(fc.fc_redundancy_workspace_size(fc.FC_BF16, H, L, d)))
    fc.fc_kv_score_topb(imp, red, 7, 0.5, B, idx, fc.workspace(fc.fc_score_topb_workspace_size(H, L, B)))
    nxt = fc.fc_kv4_cache(1, H, B + 8, d)
    fc.fc_kv4_store(k, v, nxt, idx=idx)
    # kept rows keep their bits
    for h in range(H):
        i = idx[h].long()
        assert torch.equal(nxt.k_codes[0, h, :B], c.k_codes[0, h, i])
        assert torch.equal(nxt.v_scales[0, h, :B], c.v_scales[0, h, i])
    out, lse = _attend(q[None], nxt, B)
    _check(q[None], nxt, [B], out, lse)


def test_keys_that_are_the_values():
    """A cache may be read with one set of buffers for keys and values; writing it is refused."""
    g = torch.Generator().manual_seed(97)
    c = _cache(g, 1, 2, 80, 64)
    same = fc.Kv4Cache(c.k_codes, c.k_scales, c.k_codes, c.k_scales)
    for Lq in (1, 130):
        q = _randn(g, 1, 4, Lq, 64).to(BF16).to(DEV)
        out, lse = _attend(q, same, 77)
        _check(q, same, [77], out, lse)
    x = torch.zeros(1, 2, 3, 64, device=DEV)
    with pytest.raises(fc.FlowCacheError, match="overlap"):
        fc.fc_kv4_store(x, x, same)


def test_attention_host_length_over_the_limit_is_refused():
    c = fc.fc_kv4_cache(2, 2, 32, 64)
    q = torch.zeros(2, 4, 3, 64, device=DEV, dtype=BF16)
    o, ws = torch.empty_like(q), fc.workspace(1 << 16)
    fc.fc_kv4_attention(q, c, 32, o, ws)
    fc.fc_kv4_attention(q, c, 20, o, ws, max_len=20)
    for lens, max_len in ((33, None), (21, 20), (33, 40)):
        with pytest.raises(fc.FlowCacheError, match="INVALID_ARG"):
            fc.fc_kv4_attention(q, c, lens, o, ws, max_len=max_len)


# ---- signs of zeros ---------------------------------------------------------------
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("d,rot", [(128, 128), (64, 32), (64, 24), (64, 6)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_store_rotates_zeros_as_fc_rope(dtype, d, rot, interleaved):
    """Zeros of both signs, pairs that cancel, whole rows of zeros (a padded row): the bits
    of fc_rope in float32 and a plain store, signs of zeros among them."""
    g = torch.Generator().manual_seed(13)
    N, H, L = 2, 3, 24
    k = _randn(g, N, H, L, d).to(dtype)
    k[:, :, 0] = 0.0
    k[:, :, 1] = -0.0
    k[:, :, 2, ::2], k[:, :, 2, 1::2] = 0.0, -0.0
    k[:, :, 3, : rot // 2], k[:, :, 3, rot // 2: rot] = 0.0, -0.0
    k[torch.rand(N, H, L, d, generator=g) < 0.3] = 0.0
    k[torch.rand(N, H, L, d, generator=g) < 0.2] = -0.0
    k = k.to(DEV)
    plan = fc.fc_rope_init(rot, int(interleaved))
    pos = torch.randint(-50, 50, (N, L), generator=g).to(torch.int32)
    pos[:, 4:8] = 0  # no turn: cos 1, sin 0
    pos = pos.to(DEV)
    a, b = fc.fc_kv4_cache(N, H, 32, d), fc.fc_kv4_cache(N, H, 32, d)
    fc.fc_kv4_store(k, k, a, rope=plan, pos=pos)
    k32 = torch.empty(N, H, L, d, device=DEV)
    fc.fc_rope(k.float(), k32, pos, plan)
    fc.fc_kv4_store(k32, k.float(), b)
    for n in ("k_codes", "k_scales", "v_codes", "v_scales"):
        assert torch.equal(getattr(a, n), getattr(b, n)), n
    code, sc = O.kv4_quantise(k32.cpu().numpy())
    assert np.array_equal(_bytes(b.k_codes)[:, :, :L], O.kv4_pack(code))
