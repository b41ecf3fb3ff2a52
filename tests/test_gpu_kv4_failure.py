"""Waits of the attention over the 4-bit cache that run out: a slot of the ring whose barrier
wants an arrival that nobody makes (a self-test), after which the kernels return, the error
word is set and the workspace, whatever it held, serves the next call."""

import ctypes

import pytest
import torch

import cache_gating_kv_b200 as fc

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture
def stick():
    f = fc.library().fc_selftest_kv4_stuck_slot
    f.restype, f.argtypes = ctypes.c_int, [ctypes.c_int, ctypes.c_longlong]

    def set_slot(slot):
        assert f(slot, 20_000_000) == 0  # some 10 ms

    yield set_slot
    set_slot(-1)


def _random_cache(N, H, cap, d):
    c = fc.fc_kv4_cache(N, H, cap, d)
    for t in (c.k_codes, c.v_codes):
        t.random_(0, 256)
    for t in (c.k_scales, c.v_scales):
        t.random_(0x28, 0x40)  # about a tenth to two
    return c


# A unit that several blocks share; shares that hold several units; a block for each unit,
# with stages behind the ring; the same of float32 and 16 rows; many rows, whole units and
# units split along the keys.  `most`: the slots that a block uses at most.  The first case
# has 4 x (47 + 3 + 40 + 3) = 372 of work for 148 x 2 blocks, which get two stages at least.
CASES = [(BF16, 2, 4, 4, 1, 128, [6000, 5000], 2, 2), (BF16, 100, 2, 2, 1, 64, [4400, 130] * 50, 2, 8),
         (BF16, 8, 32, 32, 1, 128, [1100] * 8, 1, 6), (F32, 20, 8, 4, 8, 64, [1400] * 20, 1, 8),
         (BF16, 2, 2, 2, 200, 128, [500, 470], 1, 3), (BF16, 1, 2, 2, 300, 64, [6000], 2, 3)]


@pytest.mark.parametrize("slot", [0, 1, 2])
@pytest.mark.parametrize("dtype,N,Hq,Hkv,Lq,d,lens,launches,most", CASES)
def test_stuck_slot_is_reported_and_nothing_lasts(stick, dtype, N, Hq, Hkv, Lq, d, lens, launches, most, slot):
    cap = (max(lens) + 15) // 16 * 16
    c = _random_cache(N, Hkv, cap, d)
    q = torch.randn(N, Hq, Lq, d, device=DEV).to(dtype)
    dl = torch.tensor(lens, dtype=torch.int32, device=DEV)
    code = fc.FC_BF16 if dtype == BF16 else fc.FC_F32
    ws = fc.workspace(fc.fc_kv4_attention_workspace_size(code, N, Hq, Hkv, Lq, cap, d))
    want, out = torch.empty_like(q), torch.empty_like(q)
    lse = torch.empty(N, Hq, Lq, device=DEV)
    fc.fc_kv4_attention(q, c, dl, want, ws)
    assert fc.fc_last_launches() == launches
    assert fc.fc_check_workspace(fc.FC_WS_IMPORTANCE, ws)
    for junk in (0x7F, 0xFF, 0x01):  # large, negative and large again as slots and counts
        ws[4:].fill_(junk)
        stick(slot)
        fc.fc_kv4_attention(q, c, dl, out, ws, lse=lse)
        assert fc.fc_check_workspace(fc.FC_WS_IMPORTANCE, ws, clear=True) == (slot >= most)
        stick(-1)
        fc.fc_kv4_attention(q, c, dl, out, ws)
        assert fc.fc_check_workspace(fc.FC_WS_IMPORTANCE, ws)
        assert torch.equal(out, want)


def test_slot_that_no_block_reaches_is_not_missed(stick):
    c = _random_cache(2, 2, 256, 64)
    q = torch.randn(2, 2, 1, 64, device=DEV).to(BF16)
    ws = fc.workspace(fc.fc_kv4_attention_workspace_size(fc.FC_BF16, 2, 2, 2, 1, 256, 64))
    want, out = torch.empty_like(q), torch.empty_like(q)
    fc.fc_kv4_attention(q, c, None, want, ws)
    stick(2)
    fc.fc_kv4_attention(q, c, None, out, ws)
    assert fc.fc_check_workspace(fc.FC_WS_IMPORTANCE, ws) and torch.equal(out, want)


def test_refused_launch_leaves_no_error_behind():
    """A launch that the driver refuses (into a capture that is broken already) is reported by
    its own call and not again by the next one, which is in order."""
    cu = ctypes.CDLL("libcuda.so.1")
    vp = ctypes.c_void_p
    x = torch.randn(1, 2, 8, 64, device=DEV)
    pos = torch.arange(8, dtype=torch.int32, device=DEV)
    plan = fc.fc_rope_init(64)
    want, y = torch.empty_like(x), torch.empty_like(x)
    fc.fc_rope(x, want, pos, plan)
    torch.cuda.synchronize()
    s = vp()
    assert cu.cuStreamCreate(ctypes.byref(s), 1) == 0
    assert cu.cuStreamBeginCapture_v2(s, 2) == 0  # relaxed: no other call is concerned
    assert cu.cuStreamSynchronize(s) != 0  # not allowed in a capture: it is broken now
    with pytest.raises(fc.FlowCacheError, match="launch failed"):
        fc.fc_rope(x, y, pos, plan, stream=s.value)
    fc.fc_rope(x, y, pos, plan)
    with pytest.raises(fc.FlowCacheError, match="error word"):
        fc.fc_check_workspace(fc.FC_WS_IMPORTANCE, fc.workspace(256), stream=s.value)
    g = vp()
    assert cu.cuStreamEndCapture(s, ctypes.byref(g)) != 0
    fc.fc_rope(x, y, pos, plan)
    torch.cuda.synchronize()
    assert torch.equal(y, want)
    assert cu.cuStreamDestroy_v2(s) == 0
