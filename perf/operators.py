"""Measurement cases of the quantised-cache operators, with their plain forms.

Three operators stand behind one another in a denoising or decoding step:

  rope       rotary positions of queries or keys (``fc_rope``)
  store      keys (rotated on the way, or gathered by a selection) and values
             written as 4-bit floating point into the cache and read back as
             numbers for the scoring calls (``fc_kv4_store``, ``fc_kv4_load``)
  attention  grouped-query attention over that cache (``fc_kv4_attention``)

With ``own`` false ``run`` computes them from elementary torch operations in
float32 (angles in float64), rounded once at the end; with ``own`` true it makes
the library calls.  ``exact`` computes the definitions in float64.

The 4-bit format.  A row of d numbers is d codes of e2m1 (0, .5, 1, 1.5, 2, 3,
4, 6 and their negatives; two to a byte, the even element in the low half) and
d/16 scales of e4m3, one for 16 consecutive elements.  With y the number as
float32 times 2^-e (e given for the tensor) and a the largest |y| of the 16:
scale = e4m3(min(a/6, 448)), code = e2m1(y/scale), both to nearest, ties to
even, both divisions rounded to float32; a zero scale has zero codes.  It stands
for code * scale * 2^e, exactly.

Rotation.  For the pair (a, b) of frequency i at position p:
(a, b) -> (a c - b s, b c + a s), each product and each sum rounded once to
float32, c and s the float32 values of m cos and m sin of 2 pi frac(p t_i), t_i
the frequency in turns per position in float64; the inverse takes -s.  The keys
of a store are rotated the same way and quantised without another rounding.
"""

import math

import torch

own = False

DEV = "cuda"
HALF, INTERLEAVED = 0, 1
PLAIN, LINEAR, NTK, YARN = 0, 1, 2, 3
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---- cases -------------------------------------------------------------------
def listed():
    return [
        # the queries of one new token in each of 32 sequences, far positions,
        # frequencies scaled by parts for a context 8 times the trained one
        dict(name="rope_tokens", op="rope", dtype="bf16", N=32, H=40, L=1, d=128, rot=128, layout=HALF,
             scaling=YARN, factor=8.0, orig=16384, axes=1, far=131072, inverse=False),
        # the queries of a video chunk of 21 x 39 x 10 tokens, three axes, 40 heads
        dict(name="rope_chunk", op="rope", dtype="bf16", N=1, H=40, L=8190, d=128, rot=128,
             layout=INTERLEAVED, scaling=PLAIN, factor=1.0, orig=0, axes=3, far=64, inverse=False),
        # the gradient of a partial rotation at an odd length, float32
        dict(name="rope_partial_grad", op="rope", dtype="f32", N=2, H=6, L=1021, d=64, rot=32,
             layout=HALF, scaling=NTK, factor=4.0, orig=0, axes=1, far=65536, inverse=True),
        # decoding: the keys and values of one token of 64 sequences, each to its own row
        dict(name="store_tokens", op="store", dtype="bf16", N=64, H=8, L=1, d=128, rot=128,
             layout=HALF, scaling=LINEAR, factor=4.0, orig=0, axes=1, far=8192, cap=1024, row0=-1,
             B=0, e=0),
        # a finished video chunk of 24 heads enters behind 16384 clean rows
        dict(name="store_chunk", op="store", dtype="bf16", N=1, H=24, L=4096, d=128, rot=128,
             layout=INTERLEAVED, scaling=PLAIN, factor=1.0, orig=0, axes=3, far=64, cap=20480,
             row0=16384, B=0, e=0),
        # the kept half of 32760 candidate rows of 40 heads, gathered into a fresh cache
        dict(name="store_selected", op="store", dtype="bf16", N=1, H=40, L=32760, d=128, rot=0,
             layout=HALF, scaling=PLAIN, factor=1.0, orig=0, axes=1, far=1, cap=16384, row0=0,
             B=16380, e=2),
        # one query of a short history: latency
        dict(name="attn_small", op="attn", dtype="bf16", N=1, Hq=8, Hkv=2, Lq=1, d=128, cap=320,
             longest=301, ragged=False, causal=False, ek=0, ev=0),
        # the parity configuration: 2 heads of 64, 256 queries, 1024 keys, float32
        dict(name="attn_f32", op="attn", dtype="f32", N=1, Hq=2, Hkv=2, Lq=256, d=64, cap=1024,
             longest=1024, ragged=False, causal=False, ek=0, ev=0),
        # decoding a batch of 32 sequences of unlike lengths, 5 query heads to a key head
        dict(name="attn_decode", op="attn", dtype="bf16", N=32, Hq=40, Hkv=8, Lq=1, d=128,
             cap=16384, longest=16384, ragged=True, causal=True, ek=0, ev=0),
        # one token over the long history of a single sequence
        dict(name="attn_history", op="attn", dtype="bf16", N=1, Hq=40, Hkv=8, Lq=1, d=128,
             cap=131072, longest=131072, ragged=False, causal=True, ek=1, ev=-1),
        # causal prompts of unlike lengths, some shorter than the padded queries, heads of 64
        dict(name="attn_prompt", op="attn", dtype="bf16", N=4, Hq=12, Hkv=4, Lq=1021, d=64,
             cap=2048, longest=2040, ragged=True, causal=True, ek=0, ev=0),
        # a denoising chunk of 4096 queries over 4 clean chunks and itself
        dict(name="attn_chunk", op="attn", dtype="bf16", N=1, Hq=24, Hkv=24, Lq=4096, d=128,
             cap=20480, longest=20480, ragged=False, causal=False, ek=0, ev=0),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "store", "attn", "attn"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    d = rng.choice([64, 128, 128])
    if op in ("rope", "store"):
        H = rng.choice([1, 2, 5, 8, 12, 24, 40])
        L = _log_int(rng, 1, 8192)
        N = _log_int(rng, 1, max(1, min(64, 8192 // L)))
        rot = rng.choice([d, d, d // 2, 24, 6])
        axes = rng.choice([1, 1, 3])
        c = dict(op=op, dtype=dtype, N=N, H=H, L=L, d=d, rot=rot,
                 layout=rng.choice([HALF, INTERLEAVED]),
                 scaling=rng.choice([PLAIN, LINEAR, NTK, YARN]),
                 factor=rng.choice([2.0, 4.0, 8.0, 10.5]), orig=rng.choice([4096, 8192, 16384]),
                 axes=axes, far=rng.choice([64, 4096, 131072]))
        if op == "rope":
            return dict(c, inverse=rng.random() < 0.4)
        B = 0
        if rng.random() < 0.4:  # a selection takes rows that are rotated already
            c["rot"], B = 0, rng.randint(1, L)
        rows = B or L
        row0 = rng.choice([-1, 0, rng.randint(0, 1000)])
        cap = (rows + max(row0, 64) + rng.randint(0, 200) + 15) // 16 * 16
        return dict(c, cap=cap, row0=row0, B=B, e=rng.choice([0, 0, 3, -2]))
    Hkv = rng.choice([1, 2, 4, 8, 24])
    G = rng.choice([1, 1, 2, 4, 5, 8])
    while Hkv * G > 64:
        G = max(1, G // 2)
    Lq = 1 if rng.random() < 0.4 else _log_int(rng, 2, 4096)
    N = _log_int(rng, 1, 32)
    longest = _log_int(rng, 1, 65536)
    while N > 1 and (N * Hkv * longest > 32 * 8 * 16384 or N * Hkv * G * Lq * longest > 1.5e9):
        N //= 2
    while N * Hkv * G * Lq * longest > 1.5e9 or Hkv * longest > 32 * 8 * 16384:
        longest = longest // 2 + 1
    if dtype == "f32" and Lq * G * Hkv * N * longest > 3e8:
        dtype = "bf16"
    cap = (longest + rng.randint(0, 100) + 15) // 16 * 16
    return dict(op="attn", dtype=dtype, N=N, Hq=Hkv * G, Hkv=Hkv, Lq=Lq, d=d, cap=cap,
                longest=longest, ragged=rng.random() < 0.5, causal=rng.random() < 0.5,
                ek=rng.choice([0, 0, 2, -1]), ev=rng.choice([0, 0, 1, -2]))


# ---- inputs -------------------------------------------------------------------
def _sections(case):
    half = case["rot"] // 2
    if case["axes"] == 1:
        return [half]
    a = half // 3
    return [half - 2 * a, a, a]


def _positions(case, g):
    """int32 [axes][N][L]: a run of positions for one axis, the frame, row and
    column of a token grid for three."""
    N, L, A = case["N"], case["L"], case["axes"]
    t = torch.arange(L, device=DEV, dtype=torch.int64)
    start = torch.randint(0, case["far"], (N, 1), generator=g, device=DEV)
    if A == 1:
        p = (start + t)[None]
    else:
        p = torch.stack([start + t // 390, (t // 10 % 39).expand(N, L), (t % 10).expand(N, L)])
    return p.to(torch.int32).contiguous()


def _turns(case):
    """Turns per position of each frequency, float64, and the factor m."""
    base, rot, f = 10000.0, case["rot"], case["factor"]
    m = 1.0
    if case["scaling"] == NTK and rot > 2:
        base = base * math.pow(f, rot / (rot - 2.0))
    w = [math.pow(base, -2.0 * i / rot) / (2.0 * math.pi) for i in range(rot // 2)]
    if case["scaling"] == LINEAR:
        w = [x / f for x in w]
    if case["scaling"] == YARN:
        keep = [min(1.0, max(0.0, (case["orig"] * x - 1.0) / 31.0)) for x in w]
        w = [(1.0 - k) * (x / f) + k * x for x, k in zip(w, keep)]
        m = 0.1 * math.log(f) + 1.0
    return w, m


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    s = dict(case=dict(case))

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=DEV)

    d = case["d"]
    if case["op"] == "attn":
        N, Hkv, cap = case["N"], case["Hkv"], case["cap"]
        if case["ragged"]:
            lens = torch.randint(0, case["longest"] + 1, (N,), generator=g, device=DEV)
            lens[0] = case["longest"]
        else:
            lens = torch.full((N,), case["longest"], device=DEV)
        s["lens"] = lens.to(torch.int32)
        s["q"] = normal(N, case["Hq"], case["Lq"], d).to(dt)
        # a few channels of the keys are several times the others, as keys have them
        chan = torch.exp(0.5 * normal(1, Hkv, 1, d))
        past = torch.arange(cap, device=DEV) >= s["lens"][:, None, None]
        for name, scale, e in (("k", chan, case["ek"]), ("v", 1.0, case["ev"])):
            codes, scales = _quantise(normal(N, Hkv, cap, d) * scale, e)
            # what stands behind a sequence is whatever was there before
            codes.masked_fill_(past[..., None], 0x7B)
            scales.masked_fill_(past[..., None], 0x7F)
            s[name + "_codes"], s[name + "_scales"] = codes, scales
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty(N, case["Hq"], case["Lq"], device=DEV)
        return s
    N, H, L = case["N"], case["H"], case["L"]
    s["pos"] = _positions(case, g)
    turns, s["m"] = _turns(case) if case["rot"] else ([0.0], 1.0)
    s["turns"] = torch.tensor(turns, dtype=torch.float64, device=DEV)
    s["axis"] = torch.repeat_interleave(torch.arange(case["axes"]), torch.tensor(
        _sections(case) if case["rot"] else [1] + [0] * (case["axes"] - 1))).to(DEV)
    if case["op"] == "rope":
        s["x"] = normal(N, L, H, d).to(dt).permute(0, 2, 1, 3)  # as a projection leaves it
        s["y"] = torch.empty(N, H, L, d, dtype=dt, device=DEV)
        return s
    chan = torch.exp(0.5 * normal(1, 1, H, d))
    k = (normal(N, L, H, d) * chan).to(dt)
    v = normal(N, L, H, d).to(dt)
    s["k"], s["v"] = k.permute(0, 2, 1, 3), v.permute(0, 2, 1, 3)
    if case["B"]:  # a selection reads the head-major buffer
        s["k"], s["v"] = s["k"].contiguous(), s["v"].contiguous()
        order = torch.rand(N, H, L, generator=g, device=DEV).argsort(-1)[..., : case["B"]]
        s["idx"] = order.sort(-1).values.to(torch.int32).contiguous()
    rows = case["B"] or L
    cap = case["cap"]
    if case["row0"] < 0:
        s["row0"] = torch.randint(0, cap - rows + 1, (N,), generator=g, device=DEV).to(torch.int32)
    else:
        s["row0"] = case["row0"]
    for n in ("k", "v"):
        s[n + "_codes"] = torch.zeros(N, H, cap, d // 2, dtype=torch.uint8, device=DEV)
        s[n + "_scales"] = torch.zeros(N, H, cap, d // 16, dtype=torch.uint8, device=DEV)
        s[n + "_out"] = torch.empty(N, H, rows, d, dtype=dt, device=DEV)
    return s


# ---- plain forms -----------------------------------------------------------------
def _scale_code(x, e):
    """float32 x [..., d] -> (signed e2m1 values [..., d/16, 16], e4m3 scales)."""
    y = (x * 2.0 ** -e).unflatten(-1, (-1, 16))
    scale = (y.abs().amax(-1) / 6.0).clamp(max=448.0).to(torch.float8_e4m3fn)
    sf = scale.float()[..., None]
    t = torch.where(sf > 0, y.abs() / sf, torch.zeros_like(y))
    c = torch.where(t < 2, torch.round(t * 2) * 0.5, torch.where(t < 4, torch.round(t), torch.round(t * 0.5) * 2))
    return torch.copysign(c.clamp_(max=6.0), y), scale


def _quantise(x, e):
    """The packed form of float32 x [..., d]: codes [..., d/2], scales [..., d/16]."""
    c, scale = _scale_code(x, e)
    a = c.abs()
    n = torch.where(a < 2, a * 2, torch.where(a < 4, a + 2, a * 0.5 + 4)).to(torch.uint8)
    n = (n | (torch.signbit(c).to(torch.uint8) << 3)).flatten(-2)
    return n[..., 0::2] | (n[..., 1::2] << 4), scale.view(torch.uint8)


def _values(codes, scales, e):
    """float32 numbers that packed rows stand for."""
    n = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).unflatten(-1, (-1, 16))
    table = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0.0, -.5, -1, -1.5, -2, -3, -4, -6], device=codes.device)
    return (table[n.int()] * (scales.view(torch.float8_e4m3fn).float() * 2.0 ** e)[..., None]).flatten(-2)


def _rotate(x, state, inverse):
    """float32 x [N, H, L, d] rotated in its first ``rot`` elements."""
    case = state["case"]
    rot = case["rot"]
    if rot == 0:
        return x
    p = state["pos"].double().permute(1, 2, 0)[..., state["axis"]]  # [N, L, rot/2]
    t = p * state["turns"]
    t = (t - torch.round(t)) * (2.0 * math.pi)
    c = (torch.cos(t) * state["m"]).float()[:, None]
    s = (torch.sin(t) * state["m"]).float()[:, None]
    if inverse:
        s = -s
    r = x[..., :rot]
    a, b = (r[..., : rot // 2], r[..., rot // 2:]) if case["layout"] == HALF else (r[..., 0::2], r[..., 1::2])
    u, w = a * c - b * s, b * c + a * s
    r = torch.cat([u, w], -1) if case["layout"] == HALF else torch.stack([u, w], -1).flatten(-2)
    return torch.cat([r, x[..., rot:]], -1)


def _plain_store(state):
    case = state["case"]
    k, v = _rotate(state["k"].float(), state, False), state["v"].float()
    if case["B"]:
        at = state["idx"].long()[..., None].expand(-1, -1, -1, case["d"])
        k, v = k.gather(2, at), v.gather(2, at)
    ck, sk = _scale_code(k, case["e"])
    cv, sv = _scale_code(v, case["e"])
    up, dt = 2.0 ** case["e"], state["k"].dtype
    return [(ck * (sk.float() * up)[..., None]).flatten(-2).to(dt),
            (cv * (sv.float() * up)[..., None]).flatten(-2).to(dt)]


def _plain_attention(state):
    case = state["case"]
    N, Hq, Hkv, Lq, d, M = (case[n] for n in ("N", "Hq", "Hkv", "Lq", "d", "longest"))
    lens = state["lens"].long()
    j = torch.arange(M, device=DEV)
    dead = (j >= lens[:, None])[:, None, :, None]
    k = _values(state["k_codes"][:, :, :M], state["k_scales"][:, :, :M], case["ek"]).masked_fill_(dead, 0.0)
    v = _values(state["v_codes"][:, :, :M], state["v_scales"][:, :, :M], case["ev"]).masked_fill_(dead, 0.0)
    q = state["q"].float().view(N, Hkv, Hq // Hkv * Lq, d)
    s = torch.matmul(q, k.transpose(-1, -2)).mul_(1.0 / math.sqrt(d))
    del k
    last = lens[:, None] - 1
    if case["causal"]:
        last = lens[:, None] - Lq + torch.arange(Lq, device=DEV)
    hidden = j > last[..., None]  # [N, Lq or 1, M]
    s5 = s.view(N, Hkv, Hq // Hkv, Lq, M)
    s5.masked_fill_(hidden[:, None, None], float("-inf"))
    m = s.amax(-1, keepdim=True)
    m = torch.where(m == float("-inf"), torch.zeros_like(m), m)
    p = s.sub_(m).exp_()
    z = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v) / torch.where(z > 0, z, torch.ones_like(z))
    return o.view(N, Hq, Lq, d).to(state["q"].dtype), (m + torch.log(z)).view(N, Hq, Lq)


# ---- the library's calls -----------------------------------------------------------
def _plan(state):
    import cache_gating_kv_b200 as fc

    c = state["case"]
    if "plan" not in state:
        state["plan"] = fc.fc_rope_init(c["rot"], c["layout"], scaling=c["scaling"], factor=c["factor"],
                                        orig_len=c["orig"], sections=_sections(c))
    return state["plan"]


def _cache(state, ek, ev):
    import cache_gating_kv_b200 as fc

    if "cache" not in state:
        state["cache"] = fc.Kv4Cache(state["k_codes"], state["k_scales"], state["v_codes"],
                                     state["v_scales"], ek, ev)
    return state["cache"]


def _own_rope(state):
    import cache_gating_kv_b200 as fc

    fc.fc_rope(state["x"], state["y"], state["pos"], _plan(state), inverse=state["case"]["inverse"])
    return state["y"]


def _own_store(state):
    import cache_gating_kv_b200 as fc

    c = state["case"]
    cache = _cache(state, c["e"], c["e"])
    rope = dict(rope=_plan(state), pos=state["pos"]) if c["rot"] else {}
    fc.fc_kv4_store(state["k"], state["v"], cache, row0=state["row0"], idx=state.get("idx"), **rope)
    fc.fc_kv4_load(cache, state["k_out"], state["v_out"], row0=state["row0"])
    return [state["k_out"], state["v_out"]]


def _own_attention(state):
    import cache_gating_kv_b200 as fc

    c = state["case"]
    cache = _cache(state, c["ek"], c["ev"])
    if "ws" not in state:
        code = fc.FC_BF16 if c["dtype"] == "bf16" else fc.FC_F32
        state["ws"] = fc.workspace(fc.fc_kv4_attention_workspace_size(
            code, c["N"], c["Hq"], c["Hkv"], c["Lq"], c["longest"], c["d"]))
    fc.fc_kv4_attention(state["q"], cache, state["lens"], state["out"], state["ws"], max_len=c["longest"],
                        causal=c["causal"], lse=state["lse"])
    return state["out"], state["lse"]


def run(state):
    op = state["case"]["op"]
    if op == "rope":
        if own:
            return _own_rope(state)
        return _rotate(state["x"].float(), state, state["case"]["inverse"]).to(state["x"].dtype)
    if op == "store":
        return _own_store(state) if own else _plain_store(state)
    return _own_attention(state) if own else _plain_attention(state)


# ---- what a pass cannot do without -----------------------------------------------
def work(case):
    d, el = case["d"], 2 if case["dtype"] == "bf16" else 4
    packed = d // 2 + d // 16
    if case["op"] == "rope":
        n = case["N"] * case["L"]
        return {"bytes": 2 * n * case["H"] * d * el + 4 * n * case["axes"], "flops": 3 * n * case["H"] * case["rot"]}
    if case["op"] == "store":
        n = case["N"] * case["H"] * (case["B"] or case["L"])
        # read K and V, write the packed rows and the numbers that are read back
        return {"bytes": 2 * n * (2 * d * el + packed) + (4 * n if case["B"] else 4 * case["N"] * case["L"] * case["axes"]),
                "flops": 2 * n * d * 3}
    N, Lq, top = case["N"], case["Lq"], case["longest"]
    mean = (top + (N - 1) * top / 2) / N if case["ragged"] else top  # lengths are uniform up to the longest
    pairs = N * case["Hq"] * Lq * mean
    if case["causal"]:
        pairs = N * case["Hq"] * max(Lq * mean - Lq * (Lq - 1) / 2, min(mean, Lq) * (mean + 1) / 2)
    return {"bytes": 2 * N * case["Hkv"] * mean * packed + N * case["Hq"] * Lq * (2 * d * el + 4),
            "flops": 4 * pairs * d}


# ---- the definitions in 64 bits ------------------------------------------------------
def _number64(codes, scales, e):
    """Packed rows as float64 numbers, from the bits of the two formats."""
    c = torch.empty(*codes.shape[:-1], codes.shape[-1] * 2, dtype=torch.int64, device=codes.device)
    c[..., 0::2] = codes & 15
    c[..., 1::2] = codes >> 4
    ex, ma = (c >> 1) & 3, c & 1
    num = torch.where(ex > 0, (2 + ma).double() * 2.0 ** (ex - 2).double(), ma.double() * 0.5)
    num = torch.where(c >= 8, -num, num)
    b = scales.long()
    ex, ma = (b >> 3) & 15, b & 7
    sc = torch.where(ex > 0, (8 + ma).double() * 2.0 ** (ex - 10).double(), ma.double() * 2.0 ** -9)
    return num * sc.repeat_interleave(16, -1) * 2.0 ** e


def _round32(x):
    return x.float().double()


def _exact_rotation(x, state, inverse):
    """float64 x [N, H, L, d]; the rotation as complex multiplication by hand."""
    case = state["case"]
    half = case["rot"] // 2
    ang = state["pos"].double()[state["axis"]].permute(1, 2, 0) * state["turns"] * (2 * math.pi)
    c, s = (torch.cos(ang) * state["m"])[:, None], (torch.sin(ang) * state["m"])[:, None]
    s = -s if inverse else s
    i = torch.arange(half, device=DEV)
    ia, ib = (i, i + half) if case["layout"] == HALF else (2 * i, 2 * i + 1)
    return c, s, ia, ib


def _exact_store(state):
    case = state["case"]
    k, v = state["k"].double(), state["v"].double()
    if case["rot"]:  # the definition rounds the angle's functions, the products and the sums to float32
        c, s, ia, ib = _exact_rotation(k, state, False)
        c, s = _round32(c), _round32(s)
        a, b = k[..., ia].clone(), k[..., ib].clone()
        k[..., ia] = _round32(_round32(a * c) - _round32(b * s))
        k[..., ib] = _round32(_round32(b * c) + _round32(a * s))
    grid = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=DEV)
    mid = (grid[1:] + grid[:-1]) / 2
    up = torch.tensor([False, True] * 3 + [False], device=DEV)  # a tie goes to the even code
    out = []
    for x in (k, v):
        if case["B"]:
            x = torch.stack([torch.stack([x[n, h][state["idx"][n, h].long()] for h in range(case["H"])])
                             for n in range(case["N"])])
        y = x * 2.0 ** -case["e"]
        y = y.reshape(*y.shape[:-1], -1, 16)
        sc = torch.clamp(_round32(y.abs().max(-1).values / 6.0), max=448.0).to(torch.float8_e4m3fn).double()[..., None]
        t = _round32(torch.where(sc > 0, y.abs() / torch.where(sc > 0, sc, torch.ones_like(sc)), torch.zeros_like(y)))
        code = torch.zeros(t.shape, dtype=torch.int64, device=DEV)
        for m, tie in zip(mid.tolist(), up.tolist()):
            code += (t >= m) if tie else (t > m)
        num = torch.where(y < 0, -grid[code], grid[code]) * sc * 2.0 ** case["e"]
        out.append(num.reshape(*x.shape))
    return out


def _exact_attention(state):
    case = state["case"]
    N, Hq, Hkv, Lq, d = (case[n] for n in ("N", "Hq", "Hkv", "Lq", "d"))
    G = Hq // Hkv
    out = torch.zeros(N, Hq, Lq, d, dtype=torch.float64, device=DEV)
    lse = torch.full((N, Hq, Lq), float("-inf"), dtype=torch.float64, device=DEV)
    for n, length in enumerate(state["lens"].tolist()):
        if length == 0:
            continue
        first = max(0, Lq - length) if case["causal"] else 0  # queries before this one see nothing
        if first >= Lq:
            continue
        for h in range(Hkv):
            kk = _number64(state["k_codes"][n, h, :length], state["k_scales"][n, h, :length], case["ek"])
            vv = _number64(state["v_codes"][n, h, :length], state["v_scales"][n, h, :length], case["ev"])
            for r in range(h * G, h * G + G):
                x = state["q"][n, r, first:].double() @ kk.T / math.sqrt(d)
                if case["causal"]:
                    i = torch.arange(first, Lq, device=DEV)[:, None]
                    x[torch.arange(length, device=DEV)[None, :] - i > length - Lq] = float("-inf")
                z = torch.logsumexp(x, -1)
                lse[n, r, first:] = z
                out[n, r, first:] = x.sub_(z[:, None]).exp_() @ vv
    return out, lse


def exact(case, seed):
    state = prepare(case, seed)
    if case["op"] == "store":
        return _exact_store(state)
    if case["op"] == "attn":
        if work(case)["flops"] > 4e12:
            return None
        return _exact_attention(state)
    x = state["x"].double()
    c, s, ia, ib = _exact_rotation(x, state, case["inverse"])
    y = x.clone()
    y[..., ia] = x[..., ia] * c - x[..., ib] * s
    y[..., ib] = x[..., ib] * c + x[..., ia] * s
    return y
