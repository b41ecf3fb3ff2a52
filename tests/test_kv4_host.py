"""Rotary plans, the 4-bit format and the refusals of the cache calls, on the host."""

import ctypes

import numpy as np
import pytest

import cache_gating_kv_b200 as fc
from oracle import kv4_oracle as O

SCALINGS = {"plain": fc.FC_ROPE_PLAIN, "linear": fc.FC_ROPE_LINEAR, "ntk": fc.FC_ROPE_NTK,
            "yarn": fc.FC_ROPE_YARN}


@pytest.mark.parametrize("scaling", list(SCALINGS))
@pytest.mark.parametrize("rot,base,factor,orig", [(128, 10000.0, 8.0, 16384), (64, 500000.0, 1.0, 1),
                                                  (2, 10000.0, 4.0, 4096), (256, 100.0, 32.0, 8192)])
def test_plan_matches_the_formulas(scaling, rot, base, factor, orig):
    p = fc.fc_rope_init(rot, fc.FC_ROPE_INTERLEAVED, base=base, scaling=SCALINGS[scaling],
                        factor=factor, orig_len=orig)
    w, m = O.rope_turns(rot, base, scaling, factor, orig)
    # a few float64 operations on each side
    np.testing.assert_allclose(np.array(p.turns[: rot // 2]), w, rtol=1e-14)
    assert abs(p.m - m) <= 1e-15 * m
    assert (p.rot_dim, p.layout, p.n_axes) == (rot, 1, 1) and not any(p.axis[:])


def test_plan_sections():
    p = fc.fc_rope_init(128, sections=[22, 21, 21])
    assert list(p.axis[:64]) == [0] * 22 + [1] * 21 + [2] * 21
    p = fc.fc_rope_init(8, sections=[0, 4, 0])
    assert list(p.axis[:4]) == [1] * 4 and p.n_axes == 3


@pytest.mark.parametrize("kw", [
    dict(rot_dim=0), dict(rot_dim=7), dict(rot_dim=258), dict(rot_dim=-2),
    dict(rot_dim=64, layout=2), dict(rot_dim=64, base=1.0), dict(rot_dim=64, base=float("nan")),
    dict(rot_dim=64, base=float("inf")), dict(rot_dim=64, scaling=4), dict(rot_dim=64, scaling=-1),
    dict(rot_dim=64, scaling=fc.FC_ROPE_LINEAR, factor=0.5),
    dict(rot_dim=64, scaling=fc.FC_ROPE_NTK, factor=float("nan")),
    dict(rot_dim=64, scaling=fc.FC_ROPE_YARN, factor=2.0, orig_len=0),
    dict(rot_dim=64, scaling=fc.FC_ROPE_YARN, factor=2.0, orig_len=10, beta_fast=1.0, beta_slow=1.0),
    dict(rot_dim=64, sections=[16, 15]), dict(rot_dim=64, sections=[40, -8]),
    dict(rot_dim=64, sections=[8, 8, 8, 8]), dict(rot_dim=64, sections=[]),
])
def test_plan_refusals(kw):
    with pytest.raises(fc.FlowCacheError, match="FC_ERR_INVALID_ARG"):
        fc.fc_rope_init(**kw)


def test_plan_is_untouched_by_a_refusal():
    p = fc.RopePlan()
    p.rot_dim = 77
    assert fc.library().fc_rope_init(ctypes.byref(p), 3, 0, 10000.0, 0, 1.0, 0, 32.0, 1.0, 1, None) == 1
    assert p.rot_dim == 77
    assert fc.library().fc_rope_init(None, 4, 0, 10000.0, 0, 1.0, 0, 32.0, 1.0, 1, None) == 1


def test_struct_sizes_match_the_header():
    # 4 int32, a double, 128 doubles, 128 bytes; 4 pointers, 6 int32
    assert ctypes.sizeof(fc.RopePlan) == 16 + 8 + 1024 + 128
    assert ctypes.sizeof(fc._Kv4) == 32 + 24


def test_workspace_sizes():
    f = fc.fc_kv4_attention_workspace_size
    assert f(fc.FC_BF16, 1, 8, 2, 1, 300, 128) >= 256
    for bad in [(9, 1, 8, 2, 1, 300, 128), (1, 0, 8, 2, 1, 300, 128), (1, 1, 7, 2, 1, 300, 128),
                (1, 1, 8, 2, 0, 300, 128), (1, 1, 8, 2, 1, -1, 128), (1, 1, 8, 2, 1, 300, 96),
                (1, 1, 0, 0, 1, 300, 64), (1, 1 << 18, 8, 2, 1, 300, 64)]:
        assert f(*bad) == 0, bad


@pytest.mark.parametrize("dtype", [fc.FC_BF16, fc.FC_F32])
@pytest.mark.parametrize("N,Hq,Hkv,Lq,d", [(1, 40, 8, 1, 128), (3, 8, 8, 1, 64), (1, 4, 1, 9, 128),
                                           (1, 1, 1, 200, 128), (2, 24, 24, 700, 128)])
def test_workspace_for_a_length_serves_shorter_ones(dtype, N, Hq, Hkv, Lq, d):
    sizes = [fc.fc_kv4_attention_workspace_size(dtype, N, Hq, Hkv, Lq, m, d)
             for m in list(range(0, 3000, 37)) + list(range(3000, 140000, 1111))]
    assert sizes == sorted(sizes)


def test_size_refusals_come_before_pointers():
    lib = fc.library()
    p = fc.fc_rope_init(64)
    c = fc._Kv4(0, 0, 0, 0, 1, 1, 16, 64, 0, 0)
    r = ctypes.byref
    assert lib.fc_rope(None, None, 9, 1, 1, 1, 64, None, None, None, r(p), 0, None) == 1
    assert lib.fc_rope(None, None, 1, 0, 1, 1, 64, None, None, None, r(p), 0, None) == 1
    assert lib.fc_rope(None, None, 1, 1, 1, 1, 32, None, None, None, r(p), 0, None) == 1
    assert lib.fc_rope(None, None, 1, 1, 1, 1, 68, None, None, None, r(p), 0, None) == 1
    assert lib.fc_rope(None, None, 1, 1, 1, 1, 64, None, None, None, None, 0, None) == 1
    assert lib.fc_rope(None, None, 1, 1, 1, 1, 64, None, None, None, r(fc.RopePlan()), 0, None) == 1
    bad = (ctypes.c_int64 * 3)(64, 64, -64)
    assert lib.fc_rope(None, None, 1, 2, 2, 2, 64, bad, None, None, r(p), 0, None) == 1
    odd = (ctypes.c_int64 * 3)(256, 128, 65)
    assert lib.fc_rope(None, None, 1, 2, 2, 2, 64, odd, None, None, r(p), 0, None) == 1
    same = (ctypes.c_int64 * 3)(0, 128, 64)
    assert lib.fc_rope(None, None, 1, 2, 2, 2, 64, None, same, None, r(p), 0, None) == 1
    assert b"overlap" in lib.fc_last_error()
    assert lib.fc_kv4_load(None, None, None, 1, 1, None, None, 0, None, None) == 1
    for field, value, want in [("N", 0, 1), ("H", 0, 1), ("d", 96, 2), ("cap", 20, 1), ("cap", 0, 1),
                               ("cap", (1 << 30) + 16, 1),
                               ("k_exp", 65, 1), ("v_exp", -65, 1)]:
        x = fc._Kv4(0, 0, 0, 0, 1, 1, 16, 64, 0, 0)
        setattr(x, field, value)
        assert lib.fc_kv4_load(r(x), None, None, 1, 1, None, None, 0, None, None) == want, field
    assert lib.fc_kv4_load(r(c), None, None, 1, 1, None, None, 0, None, None) == 1  # NULL codes
    assert b"NULL" in lib.fc_last_error()


def test_oracle_format_round_trip():
    """Every number of the format is its own nearest number, ties go to even codes, and
    storing stored rows changes nothing while the scales are normal."""
    rng = np.random.default_rng(0)
    x = (rng.standard_normal((50, 64)) * np.exp(2 * rng.standard_normal((50, 1)))).astype(np.float32)
    for e in (0, 3, -5):
        code, s = O.kv4_quantise(x, e)
        v = O.kv4_values(O.kv4_pack(code), s, e)
        code2, s2 = O.kv4_quantise(v.astype(np.float32), e)
        ok = np.repeat(O.E4M3[s] >= 2.0 ** -6, 16, -1)
        assert np.array_equal(s2[O.E4M3[s] >= 2.0 ** -6], s[O.E4M3[s] >= 2.0 ** -6])
        assert np.array_equal(O.kv4_values(O.kv4_pack(code2), s2, e)[ok], v[ok])
    t = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0] * 2, np.float32)[None]
    code, s = O.kv4_quantise(t)
    assert O.E4M3[s[0, 0]] == 1.0
    assert list(code[0, :8]) == [0, 2, 2, 4, 4, 6, 6, 7]


def test_oracle_rotation_keeps_norms_and_relative_positions():
    rng = np.random.default_rng(1)
    w, _ = O.rope_turns(32)
    q, k = rng.standard_normal((2, 1, 1, 1, 32))
    dots = []
    for shift in (0, 5, 1000):
        a = O.rope(q, [[[7 + shift]]], w)
        b = O.rope(k, [[[3 + shift]]], w)
        assert abs(np.linalg.norm(a) - np.linalg.norm(q)) < 1e-12
        dots.append(float((a * b).sum()))
    assert max(dots) - min(dots) < 1e-10
    y = O.rope(q, [[[11]]], w)
    np.testing.assert_allclose(O.rope(y, [[[11]]], w, inverse=True), q, atol=1e-14)


def test_stuck_slot_selftest_validates():
    f = fc.library().fc_selftest_kv4_stuck_slot
    f.restype, f.argtypes = ctypes.c_int, [ctypes.c_int, ctypes.c_longlong]
    assert f(0, -1) == 1 and f(0, 4_000_000_001) == 1 and f(3, 0) == 1
    assert f(2, 1000) == 0 and f(-1, 0) == 0


def _fake(n):
    """An aligned address per n; overlap is refused before a pointer is asked about."""
    return 0x7F00_0000_0000 + n * (1 << 24)


def _refused(status):
    return status == 1 and b"overlap" in fc.library().fc_last_error()


def test_buffers_of_a_cache_that_is_written_must_be_apart():
    lib, r = fc.library(), ctypes.byref
    size = {0: 16 * 32, 1: 16 * 4, 2: 16 * 32, 3: 16 * 4}  # k codes, k scales, v codes, v scales
    for i in range(4):
        for j in range(4):
            if i == j:
                continue
            at = [_fake(n) for n in range(4)]
            at[j] = at[i] + size[i] - 16  # the last 16 bytes
            c = fc._Kv4(*at, 1, 1, 16, 64, 0, 0)
            store = lambda: lib.fc_kv4_store(_fake(8), _fake(9), 1, 1, 1, 4, 64, None, None, None, 0, 0, None,  # noqa: E731
                                             None, None, r(c), None)
            assert _refused(store())
            # who only reads may share them (keys that are the values)
            assert not _refused(lib.fc_kv4_load(r(c), _fake(8), _fake(9), 1, 4, None, None, 0, None, None))
            assert not _refused(lib.fc_kv4_attention(_fake(8), r(c), None, 16, 1, 1, 1, 1, 64, None, 0, 0.0, _fake(9),
                                                     None, None, _fake(10), 1 << 20, None))
            at[j] = at[i] + size[i]  # behind it; the addresses are nobody's
            c = fc._Kv4(*at, 1, 1, 16, 64, 0, 0)
            assert not _refused(store()) and b"overlap" not in fc.library().fc_last_error()


def test_arrays_that_are_read_must_be_apart_from_what_is_written():
    lib, r = fc.library(), ctypes.byref
    c = fc._Kv4(*[_fake(n) for n in range(4)], 2, 2, 16, 64, 0, 0)
    size = [64 * 32, 64 * 4, 64 * 32, 64 * 4]
    p = fc.fc_rope_init(64, sections=[16, 16])
    for n in range(4):
        end = _fake(n) + size[n] - 16
        store = lambda **a: lib.fc_kv4_store(  # noqa: E731
            _fake(8), _fake(9), 1, 2, 2, 4, 64, None, None, a.get("idx"), 3 if "idx" in a else 0, 0, a.get("row0"),
            r(p) if "pos" in a else None, a.get("pos"), r(c), None)
        for name, nbytes in (("idx", 2 * 2 * 3 * 4), ("row0", 8), ("pos", 2 * 2 * 4 * 4)):
            assert _refused(store(**{name: end})), name
            assert nbytes <= 16 or _refused(store(**{name: _fake(n) - 16})), name  # its end in the buffer
            store(**{name: end + 16})
            assert b"overlap" not in lib.fc_last_error()
    for out in (8, 9):
        assert _refused(lib.fc_kv4_load(r(c), _fake(8), _fake(9), 1, 4, None, None, 0, _fake(out) + 16, None))
    attend = lambda lens=_fake(11), lse=_fake(12): lib.fc_kv4_attention(  # noqa: E731
        _fake(8), r(c), lens, 16, 1, 2, 2, 1, 64, None, 0, 0.0, _fake(9), None, lse, _fake(10), 1 << 20, None)
    assert not _refused(attend())
    assert _refused(attend(lens=_fake(9)))
    assert _refused(attend(lens=_fake(12)))
    assert _refused(attend(lens=_fake(10) + 16))
    assert _refused(attend(lse=_fake(8))) and _refused(attend(lse=_fake(9))) and _refused(attend(lse=_fake(10)))
    assert _refused(attend(lse=_fake(3)))


def axis_ladders(sections, layout=fc.FC_ROPE_INTERLEAVED):
    """A plan whose axes have a ladder of frequencies each, made as documented."""
    plan = fc.fc_rope_init(2 * sum(sections), layout, sections=sections)
    at = 0
    for n in sections:
        plan.turns[at:at + n] = fc.fc_rope_init(2 * n).turns[:n] if n else []
        at += n
    return plan


def test_plan_with_a_ladder_for_each_axis():
    sections = [22, 21, 21]
    p = axis_ladders(sections)
    want = np.concatenate([10000.0 ** (-2.0 * np.arange(n) / (2 * n)) / (2 * np.pi) for n in sections])
    np.testing.assert_allclose(np.array(p.turns[:64]), want, rtol=1e-14)
    assert list(p.axis[:64]) == [0] * 22 + [1] * 21 + [2] * 21 and p.m == 1.0
