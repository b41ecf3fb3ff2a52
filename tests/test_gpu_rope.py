"""Rotary positions on the GPU against the float64 oracle."""

import numpy as np
import pytest
import torch

import cache_gating_kv_b200 as fc
from oracle import kv4_oracle as O
from tests.test_kv4_host import axis_ladders

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _bound(x, y, m, dtype):
    """c and s are half a float32 ulp off, products and the sum round once each: three
    roundings of 2^-24 on at most m (|a| + |b|); the result rounds once to its type."""
    t = 3 * 2.0 ** -24 * m * 2 * np.abs(x).max(-1, keepdims=True)
    return t + np.abs(y) * torch.finfo(dtype).eps / 2 + 1e-40


def _run(N, H, L, d, rot, dtype, interleaved=False, scaling="plain", factor=1.0, orig=1,
         sections=None, far=1000, inverse=False, inplace=False, layout="nhld", seed=0):
    g = torch.Generator().manual_seed(seed)
    if layout == "nhld":
        x = torch.randn(N, H, L, d, generator=g).to(dtype).to(DEV)
    elif layout == "nlhd":
        x = torch.randn(N, L, H, d, generator=g).to(dtype).to(DEV).permute(0, 2, 1, 3)
    else:  # a slice of a packed projection
        x = torch.randn(N, L, 3, H, d, generator=g).to(dtype).to(DEV)[:, :, 1].permute(0, 2, 1, 3)
    axes = 1 if sections is None else len(sections)
    pos = torch.randint(-far, far, (axes, N, L), generator=g).to(torch.int32)
    plan = fc.fc_rope_init(rot, int(interleaved), scaling={"plain": 0, "linear": 1, "ntk": 2, "yarn": 3}[scaling],
                           factor=factor, orig_len=orig, sections=sections)
    xn = x.double().cpu().numpy()
    y = x if inplace else torch.full((N, H, L, d), 7.0, dtype=dtype, device=DEV)
    fc.fc_rope(x, y, pos.to(DEV), plan, inverse=inverse)
    torch.cuda.synchronize()
    w = np.array(plan.turns[: rot // 2])
    ax = np.repeat(np.arange(axes), [rot // 2] if sections is None else sections)
    want = O.rope(xn, pos.numpy(), w, plan.m, interleaved, ax, inverse)
    got = y.double().cpu().numpy()
    assert (np.abs(got - want) <= _bound(xn, want, plan.m, dtype)).all()
    assert np.array_equal(got[..., rot:], xn[..., rot:])  # copied


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("N,H,L,d,rot", [
    (1, 1, 1, 64, 64), (1, 3, 17, 128, 128), (2, 5, 33, 128, 64), (3, 2, 15, 64, 24),
    (1, 2, 7, 64, 6), (2, 1, 16, 8, 8), (1, 2, 5, 256, 256), (1, 7, 9, 72, 40), (1, 1, 3, 16, 2),
    (1, 40, 100, 128, 128), (5, 1, 1, 128, 16)])
def test_rope_shapes(N, H, L, d, rot, interleaved, dtype):
    _run(N, H, L, d, rot, dtype, interleaved)
    _run(N, H, L, d, rot, dtype, interleaved, inverse=True, layout="nlhd", seed=1)


@pytest.mark.parametrize("scaling", ["linear", "ntk", "yarn"])
def test_rope_scalings(scaling):
    _run(2, 3, 40, 128, 128, torch.float32, scaling=scaling, factor=8.0, orig=4096, far=100000)
    _run(1, 2, 9, 64, 32, torch.bfloat16, True, scaling=scaling, factor=4.0, orig=8192)


def test_rope_axes_layouts_and_in_place():
    _run(2, 4, 390, 128, 128, torch.bfloat16, True, sections=[22, 21, 21], layout="packed")
    _run(1, 4, 50, 128, 96, torch.float32, False, sections=[16, 0, 32], inplace=True)
    _run(1, 4, 50, 64, 64, torch.bfloat16, False, inplace=True, layout="packed")
    _run(2, 3, 21, 64, 20, torch.float32, True, inplace=True, layout="nlhd")


def test_rope_far_positions():
    """The whole int32 range: the turn p w rounds once in float64 on both sides."""
    _run(1, 2, 64, 128, 128, torch.float32, far=2 ** 31 - 1, seed=3)
    _run(1, 2, 64, 128, 128, torch.float32, True, far=2 ** 31 - 1, scaling="linear", factor=3.0, seed=4)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_gradient(interleaved):
    """`inverse` maps the gradient of y to that of x: against the formula's transpose and
    against differences of the forward call."""
    g = torch.Generator().manual_seed(5)
    N, H, L, d, rot = 1, 2, 6, 32, 24
    x = torch.randn(N, H, L, d, generator=g).to(DEV)
    dy = torch.randn(N, H, L, d, generator=g).to(DEV)
    pos = torch.arange(L, dtype=torch.int32, device=DEV) * 3
    plan = fc.fc_rope_init(rot, int(interleaved), scaling=fc.FC_ROPE_YARN, factor=4.0, orig_len=64)
    dx, y = torch.empty_like(x), torch.empty_like(x)
    fc.fc_rope(dy, dx, pos, plan, inverse=True)
    fc.fc_rope(x, y, pos, plan)
    # <dy, R x> = <R^T dy, x>, each element off by the bound of _bound
    lhs, rhs = (dy.double() * y.double()).sum().item(), (dx.double() * x.double()).sum().item()
    n = x.numel()
    assert abs(lhs - rhs) <= n * 2 * 6 * 2.0 ** -24 * plan.m * 4.0 * 4.0
    # the map is linear, so a difference of step 1 is exact up to rounding
    for e in (0, 5, 11, 23, 24, 31):
        x2 = x.clone()
        x2[0, 1, 4, e] += 1.0
        y2 = torch.empty_like(x)
        fc.fc_rope(x2, y2, pos, plan)
        diff = ((y2.double() - y.double()) * dy.double()).sum().item()
        # four roundings of numbers below m (4 + 1) in each of two outputs of two calls
        assert abs(diff - dx[0, 1, 4, e].item()) <= 16 * 2.0 ** -24 * plan.m * 5.0 * 8.0


def test_rope_special_values():
    """Infinities and NaN stay in their pair; zeros stay zero."""
    x = torch.zeros(1, 1, 2, 64, device=DEV)
    x[0, 0, 0, 3] = float("nan")
    x[0, 0, 1, 5] = float("inf")
    y = torch.empty_like(x)
    fc.fc_rope(x, y, torch.tensor([1, 2], dtype=torch.int32, device=DEV), fc.fc_rope_init(64))
    bad = (~torch.isfinite(y)).nonzero().tolist()
    assert bad == [[0, 0, 0, 3], [0, 0, 0, 35], [0, 0, 1, 5], [0, 0, 1, 37]]
    assert (y[torch.isfinite(y)] == 0).all()


def test_rope_refusals():
    x = torch.zeros(1, 2, 4, 64, device=DEV)
    pos = torch.zeros(4, dtype=torch.int32, device=DEV)
    plan = fc.fc_rope_init(64)
    y = torch.empty_like(x)
    for bad in [dict(x=x.cpu()), dict(y=torch.empty(1, 2, 4, 64)), dict(pos=pos.long()),
                dict(pos=pos[:3]), dict(y=y[:, :1]), dict(y=y.bfloat16()), dict(x=x.half(), y=y.half()),
                dict(x=x[0, 0], y=y[0, 0]), dict(x=x.transpose(2, 3), y=y.transpose(2, 3)),
                dict(plan=fc.fc_rope_init(128)), dict(x=x[..., :60], y=y[..., :60])]:
        a = dict(x=x, y=y, pos=pos, plan=plan) | bad
        with pytest.raises(fc.FlowCacheError):
            fc.fc_rope(a["x"], a["y"], a["pos"], a["plan"])
    buf = torch.zeros(1, 2, 8, 64, device=DEV)
    with pytest.raises(fc.FlowCacheError, match="overlap"):  # shifted by a row
        fc.fc_rope(buf[:, :, :4], buf[:, :, 1:5], pos, plan)
    with pytest.raises(fc.FlowCacheError, match="overlap"):  # in place with other strides
        fc.fc_rope(buf[:, :, :4], buf.view(1, 2, 2, 4, 64)[:, 0], pos, plan)
    with pytest.raises(fc.FlowCacheError, match="overlap"):
        fc.fc_rope(x, torch.empty(1, 1, 4, 64, device=DEV).expand(1, 2, 4, 64), pos, plan)
    fc.fc_rope(x[:, :1].expand(1, 2, 4, 64), y, pos, plan)  # a broadcast input is fine


def test_rope_on_a_stream_and_in_a_graph():
    g = torch.Generator().manual_seed(6)
    x = torch.randn(2, 3, 65, 64, generator=g).to(DEV)
    pos = torch.arange(130, dtype=torch.int32, device=DEV).view(1, 2, 65)
    plan = fc.fc_rope_init(64)
    want, y = torch.empty_like(x), torch.empty_like(x)
    fc.fc_rope(x, want, pos, plan)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    fc.fc_rope(x, y, pos, plan, stream=s)
    assert fc.fc_last_launches() == 1
    torch.cuda.synchronize()
    assert torch.equal(y, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fc.fc_rope(x, y, pos, plan)
    x.copy_(torch.randn(2, 3, 65, 64, generator=g))
    graph.replay()
    fc.fc_rope(x, want, pos, plan)
    torch.cuda.synchronize()
    assert torch.equal(y, want)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("sections", [[22, 21, 21], [8, 12, 12], [5, 0, 3]])
def test_rope_with_a_ladder_for_each_axis(sections, dtype):
    """Frame, row and column parts of a video token's heads, each rotated as by itself."""
    g = torch.Generator().manual_seed(9)
    N, H, F, R, C = 2, 3, 3, 5, 4
    L, d = F * R * C, 2 * sum(sections)
    plan = axis_ladders(sections)
    t = torch.arange(L)
    pos = torch.stack([t // (R * C) + 7, t // C % R, t % C]).to(torch.int32)[:, None].repeat(1, N, 1)
    x = torch.randn(N, H, L, d, generator=g).to(dtype)
    y = torch.empty(N, H, L, d, dtype=dtype, device=DEV)
    fc.fc_rope(x.to(DEV), y, pos.to(DEV), plan)
    got, xn = y.double().cpu().numpy(), x.double().numpy()
    at = 0
    for a, n in enumerate(sections):
        if n:
            w, _ = O.rope_turns(2 * n)
            part = xn[..., at:at + 2 * n]
            want = O.rope(part, pos[a:a + 1].numpy(), w, interleaved=True)
            # (the turns agree to 1e-14: at positions below 16 that is nothing to float32)
            assert (np.abs(got[..., at:at + 2 * n] - want) <= _bound(part, want, 1.0, dtype)).all()
        at += 2 * n
