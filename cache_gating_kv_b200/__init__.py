"""FlowCache hot path on B200: thin Python binding of ``libflowcache.so``.

Every function here marshals torch CUDA tensors into the C-ABI call of the
same name declared in ``include/flowcache.h``; all arithmetic runs in the
library's CUDA kernels.  There is no CPU fallback: if the shared library is
missing or fails to load, every call raises :class:`FlowCacheError`.

Method: "Flow Caching for Autoregressive Video Generation" (papernotes.org),
方法详解 / 关键设计 1-3 (chunkwise relative-L1 cache gate; joint
importance-redundancy KV-cache compression).
"""

import ctypes
import os

import torch

__all__ = [
    "FlowCacheError",
    "FC_F32",
    "FC_BF16",
    "library",
    "library_path",
    "fc_version",
    "fc_last_launches",
    "fc_chunk_l1_gate",
    "fc_chunk_l1_gate_noalloc",
    "fc_history_l1_gate",
    "fc_gather_recompute",
    "fc_scatter_velocity",
    "fc_kv_cache_workspace_size",
    "fc_check_workspace",
    "FC_WS_GATE",
    "FC_WS_GATE_NOALLOC",
    "FC_WS_IMPORTANCE",
    "FC_WS_CACHE",
    "fc_kv_cache_commit",
    "fc_kv_importance",
    "fc_kv_redundancy",
    "fc_kv_score_topb",
    "fc_kv_compact",
    "FC_ROPE_HALF",
    "FC_ROPE_INTERLEAVED",
    "FC_ROPE_PLAIN",
    "FC_ROPE_LINEAR",
    "FC_ROPE_NTK",
    "FC_ROPE_YARN",
    "RopePlan",
    "fc_rope_init",
    "fc_rope",
    "Kv4Cache",
    "fc_kv4_cache",
    "fc_kv4_store",
    "fc_kv4_load",
    "fc_kv4_attention",
    "fc_kv4_attention_workspace_size",
    "fc_gate_workspace_size",
    "fc_importance_workspace_size",
    "fc_redundancy_workspace_size",
    "fc_score_topb_workspace_size",
    "workspace",
]

FC_F32, FC_BF16 = 0, 1
_STATUS = {0: "FC_OK", 1: "FC_ERR_INVALID_ARG", 2: "FC_ERR_UNSUPPORTED", 3: "FC_ERR_WORKSPACE",
           4: "FC_ERR_CUDA", 5: "FC_ERR_TIMEOUT"}

library_path = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libflowcache.so")
_lib = None


class FlowCacheError(RuntimeError):
    """A libflowcache call returned an error status, or the library is missing."""

    def __init__(self, msg, status=None):
        super().__init__(msg)
        self.status = status


class RopePlan(ctypes.Structure):
    """``fc_rope_plan``: what :func:`fc_rope_init` fills and the calls read."""

    _fields_ = [("rot_dim", ctypes.c_int32), ("layout", ctypes.c_int32),
                ("n_axes", ctypes.c_int32), ("reserved", ctypes.c_int32), ("m", ctypes.c_double),
                ("turns", ctypes.c_double * 128), ("axis", ctypes.c_uint8 * 128)]


class _Kv4(ctypes.Structure):
    _fields_ = [("k_codes", ctypes.c_void_p), ("k_scales", ctypes.c_void_p),
                ("v_codes", ctypes.c_void_p), ("v_scales", ctypes.c_void_p),
                ("N", ctypes.c_int32), ("H", ctypes.c_int32), ("cap", ctypes.c_int32),
                ("d", ctypes.c_int32), ("k_exp", ctypes.c_int32), ("v_exp", ctypes.c_int32)]


def _declare(lib):
    c_int, c_i64, c_f, c_sz, c_p = (ctypes.c_int, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t,
                                     ctypes.c_void_p)
    sig = {
        "fc_last_error": (ctypes.c_char_p, []),
        "fc_version": (c_int, []),
        "fc_last_launches": (c_int, []),
        "fc_gate_workspace_size": (c_sz, [c_int, c_i64]),
        "fc_chunk_l1_gate": (c_int, [c_p, c_p, c_int, c_i64, c_p, c_p, ctypes.c_int32, c_f, c_p,
                                     c_p, c_p, c_p, c_sz, c_p]),
        "fc_chunk_l1_gate_noalloc": (c_int, [c_p, c_p, c_int, c_i64, c_p, c_p, ctypes.c_int32,
                                             c_f, c_p, c_p, c_p, c_p]),
        "fc_history_l1_gate": (c_int, [c_p, c_p, c_int, c_i64, c_p, ctypes.c_int32, c_f, c_p, c_p,
                                       c_p, c_p, c_sz, c_p]),
        "fc_gather_recompute": (c_int, [c_p, c_p, c_int, c_i64, c_p, c_p, c_p, c_p]),
        "fc_scatter_velocity": (c_int, [c_p, c_p, c_p, c_int, c_i64, c_p, c_p]),
        "fc_importance_workspace_size": (c_sz, [c_int, c_int, c_int, c_int, c_int]),
        "fc_kv_importance": (c_int, [c_p, c_p, c_int, c_int, c_int, c_int, c_int, c_f, c_p, c_p,
                                     c_sz, c_p]),
        "fc_redundancy_workspace_size": (c_sz, [c_int, c_int, c_int, c_int]),
        "fc_kv_redundancy": (c_int, [c_p, c_int, c_int, c_int, c_int, c_p, c_p, c_sz, c_p]),
        "fc_score_topb_workspace_size": (c_sz, [c_int, c_int, c_int]),
        "fc_kv_score_topb": (c_int, [c_p, c_p, c_int, c_int, c_int, c_f, c_int, c_p, c_p, c_p,
                                     c_sz, c_p]),
        "fc_kv_compact": (c_int, [c_p, c_p, c_int, c_int, c_int, c_int, c_p, c_int, c_p, c_p,
                                  c_p]),
        "fc_kv_cache_workspace_size": (c_sz, [c_int, c_int, c_int, c_int, c_int, c_int]),
        "fc_check_workspace": (c_int, [c_int, c_p, c_int, c_int, c_p]),
        "fc_kv_cache_commit": (c_int, [c_p, c_p, c_p, c_p, c_p, c_int, c_int, c_int, c_int, c_int,
                                       c_int, c_int, c_f, c_int, c_f, c_p, c_p, c_sz,
                                       ctypes.POINTER(c_int), ctypes.POINTER(c_int), c_p]),
        "fc_rope_init": (c_int, [c_p, c_int, c_int, ctypes.c_double, c_int, ctypes.c_double, c_i64,
                                 ctypes.c_double, ctypes.c_double, c_int, c_p]),
        "fc_rope": (c_int, [c_p, c_p, c_int, c_int, c_int, c_int, c_int, c_p, c_p, c_p, c_p, c_int,
                            c_p]),
        "fc_kv4_store": (c_int, [c_p, c_p, c_int, c_int, c_int, c_int, c_int, c_p, c_p, c_p, c_int,
                                 c_int, c_p, c_p, c_p, c_p, c_p]),
        "fc_kv4_load": (c_int, [c_p, c_p, c_p, c_int, c_int, c_p, c_p, c_int, c_p, c_p]),
        "fc_kv4_attention_workspace_size": (c_sz, [c_int, c_int, c_int, c_int, c_int, c_int, c_int]),
        "fc_kv4_attention": (c_int, [c_p, c_p, c_p, c_int, c_int, c_int, c_int, c_int, c_int, c_p,
                                     c_int, c_f, c_p, c_p, c_p, c_p, c_sz, c_p]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    return lib


def library():
    """The loaded ``ctypes.CDLL`` (loaded on first use)."""
    global _lib
    if _lib is None:
        if not os.path.exists(library_path):
            raise FlowCacheError(
                f"{library_path} is not built; run `python -m cache_gating_kv_b200.build`")
        try:
            _lib = _declare(ctypes.CDLL(library_path))
        except OSError as e:
            raise FlowCacheError(f"cannot load {library_path}: {e}") from e
    return _lib


def _check(name, st):
    if st != 0:
        msg = library().fc_last_error().decode(errors="replace")
        raise FlowCacheError(f"{name}: {_STATUS.get(st, st)}: {msg}", st)


def _p(t):
    if t is None:
        return None
    if not t.is_cuda:
        raise FlowCacheError("tensor arguments must be CUDA tensors")
    if not t.is_contiguous():
        raise FlowCacheError("tensor arguments must be contiguous")
    return t.data_ptr()


# The current stream's handle without building a Stream object (4 us of a call that
# is 9 us in all); the Stream object where torch does not have the short way.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_raw_device = getattr(torch._C, "_cuda_getDevice", None)


def _s(stream):
    if stream is None:
        if _raw_stream is not None and _raw_device is not None and torch.cuda.is_initialized():
            return _raw_stream(_raw_device())
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _dtype_code(t):
    if t.dtype == torch.bfloat16:
        return FC_BF16
    if t.dtype == torch.float32:
        return FC_F32
    raise FlowCacheError(f"unsupported dtype {t.dtype}")


def fc_version():
    return library().fc_version()


def fc_last_launches():
    """Kernel launches (memsets included) the last compute call on this thread
    enqueued."""
    return library().fc_last_launches()


# ---- workspace sizes and allocation ----------------------------------------
def fc_gate_workspace_size(n_chunks, n_per_chunk):
    return library().fc_gate_workspace_size(n_chunks, n_per_chunk)


def fc_importance_workspace_size(dtype, H, Lq, Lk, d):
    return library().fc_importance_workspace_size(dtype, H, Lq, Lk, d)


def fc_redundancy_workspace_size(dtype, H, Lk, d):
    return library().fc_redundancy_workspace_size(dtype, H, Lk, d)


def fc_score_topb_workspace_size(H, Lk, B):
    return library().fc_score_topb_workspace_size(H, Lk, B)


def fc_kv_cache_workspace_size(dtype, H, Lq, B_budget, C, d):
    return library().fc_kv_cache_workspace_size(dtype, H, Lq, B_budget, C, d)


FC_WS_GATE, FC_WS_GATE_NOALLOC, FC_WS_IMPORTANCE, FC_WS_CACHE = 0, 1, 2, 3


def fc_check_workspace(kind, ws=None, n_chunks=0, clear=False, stream=None):
    """True if no bounded device-side wait of the calls that used ``ws`` gave
    up (synchronises the stream); False if one did (their outputs are not
    valid).  ``clear`` resets the error word after reading it."""
    st = library().fc_check_workspace(int(kind), _p(ws), int(n_chunks), 1 if clear else 0,
                                      _s(stream))
    if st == 5:
        return False
    _check("fc_check_workspace", st)
    return True


def workspace(nbytes, device=None):
    """A zero-filled device byte buffer of ``nbytes`` (at least 256) bytes."""
    return torch.zeros(max(int(nbytes), 256), dtype=torch.uint8, device=device or "cuda")


# ---- the five calls -----------------------------------------------------------
def fc_chunk_l1_gate(x, v, dt, step, m, eps, f, l1_rel, recompute, ws, stream=None):
    """Chunkwise cache gate step (in place on ``x`` and ``f``).  x, v: [n_c, N]
    float32; dt: [n_c] float32; step: [n_c] int32; f, l1_rel: [n_c] float32;
    recompute: [n_c] uint8; ws from :func:`fc_gate_workspace_size` (zeroed once)."""
    n_c, N = x.shape
    st = library().fc_chunk_l1_gate(_p(x), _p(v), n_c, N, _p(dt), _p(step), int(m), float(eps),
                                     _p(f), _p(l1_rel), _p(recompute), _p(ws), ws.numel(),
                                     _s(stream))
    _check("fc_chunk_l1_gate", st)


def fc_history_l1_gate(h_old, h_new, step, m, delta, f, d_rel, refresh, ws, stream=None):
    """History-guided gate step (in place on ``h_old`` and ``f``): h_old is
    h_{t+1} in and h_t out.  [n, N] float32 snapshots; step [n] int32; f, d_rel
    [n] float32; refresh [n] uint8; ws from :func:`fc_gate_workspace_size`."""
    n, N = h_old.shape
    st = library().fc_history_l1_gate(_p(h_old), _p(h_new), n, N, _p(step), int(m), float(delta),
                                       _p(f), _p(d_rel), _p(refresh), _p(ws), ws.numel(),
                                       _s(stream))
    _check("fc_history_l1_gate", st)


def fc_chunk_l1_gate_noalloc(x, v, dt, step, m, eps, f, l1_rel, recompute, stream=None):
    """The gate step without a workspace, for callers that cannot allocate
    device memory while they run it (the library keeps a fixed static scratch
    array instead).  At most 32 chunks per call; calls must not overlap on the
    GPU; the first call on a device should precede any stream capture."""
    n_c, N = x.shape
    st = library().fc_chunk_l1_gate_noalloc(_p(x), _p(v), n_c, N, _p(dt), _p(step), int(m),
                                             float(eps), _p(f), _p(l1_rel), _p(recompute),
                                             _s(stream))
    _check("fc_chunk_l1_gate_noalloc", st)


def fc_gather_recompute(x, recompute, dense, ids, count, stream=None):
    """Gather the recompute chunks' rows of x [n_c, N] into dense [n_c, N];
    ids [n_c] int32 and count [1] int32 are written on the device."""
    n_c, N = x.shape
    st = library().fc_gather_recompute(_p(x), _p(recompute), n_c, N, _p(dense), _p(ids),
                                        _p(count), _s(stream))
    _check("fc_gather_recompute", st)


def fc_scatter_velocity(v_dense, ids, count, v_cache, stream=None):
    """v_cache[ids[i]] = v_dense[i] for i < count (device-side count)."""
    n_c, N = v_cache.shape
    st = library().fc_scatter_velocity(_p(v_dense), _p(ids), _p(count), n_c, N, _p(v_cache),
                                        _s(stream))
    _check("fc_scatter_velocity", st)


def fc_kv_importance(q, k, imp, ws, scale=0.0, stream=None):
    """Pre-pooling importance.  q [H, Lq, d], k [H, Lk, d] (bf16 or float32);
    imp [H, Lk] float32 out."""
    H, Lq, d = q.shape
    Lk = k.shape[1]
    st = library().fc_kv_importance(_p(q), _p(k), _dtype_code(q), H, Lq, Lk, d, float(scale),
                                     _p(imp), _p(ws), ws.numel(), _s(stream))
    _check("fc_kv_importance", st)


def fc_kv_redundancy(k, red, ws, stream=None):
    """Redundancy.  k [H, Lk, d]; red [H, Lk] float32 out."""
    H, Lk, d = k.shape
    st = library().fc_kv_redundancy(_p(k), _dtype_code(k), H, Lk, d, _p(red), _p(ws), ws.numel(),
                                     _s(stream))
    _check("fc_kv_redundancy", st)


def fc_kv_score_topb(imp, red, pool_window, lam, B, idx, ws, score=None, stream=None):
    """Pooled joint score and per-head top-B.  imp, red [H, Lk] float32;
    idx [H, B] int32 out (ascending); score [H, Lk] float32 out or None."""
    H, Lk = imp.shape
    st = library().fc_kv_score_topb(_p(imp), _p(red), H, Lk, int(pool_window), float(lam), int(B),
                                     _p(score), _p(idx), _p(ws), ws.numel(), _s(stream))
    _check("fc_kv_score_topb", st)


def fc_kv_cache_commit(q, k_buf, v_buf, k_next, v_next, n_clean, C, ws, pool_window, lam,
                       scale=0.0, idx=None, stream=None):
    """One finished chunk enters the cache buffer [H, B_budget + C, d]; returns
    (n_next, compressed).  When compressed, the kept rows are in rows
    [0, B_budget) of k_next / v_next and the caller swaps the buffers."""
    H, cap, d = k_buf.shape
    Lq = q.shape[1]
    n_next, comp = ctypes.c_int(-1), ctypes.c_int(-1)
    st = library().fc_kv_cache_commit(
        _p(q), _p(k_buf), _p(v_buf), _p(k_next), _p(v_next), _dtype_code(k_buf), H, Lq, d,
        cap - C, C, n_clean, float(scale), int(pool_window), float(lam), _p(idx), _p(ws),
        0 if ws is None else ws.numel() * ws.element_size(), ctypes.byref(n_next), ctypes.byref(comp), _s(stream))
    _check("fc_kv_cache_commit", st)
    return n_next.value, bool(comp.value)


def fc_kv_compact(k, v, idx, k_out, v_out, stream=None):
    """Gather the kept rows: k_out[h, r] = k[h, idx[h, r]] (and V)."""
    H, Lk, d = k.shape
    B = idx.shape[1]
    st = library().fc_kv_compact(_p(k), _p(v), _dtype_code(k), H, Lk, d, _p(idx), B, _p(k_out),
                                  _p(v_out), _s(stream))
    _check("fc_kv_compact", st)


# ---- rotary positions and the 4-bit cache ---------------------------------------
FC_ROPE_HALF, FC_ROPE_INTERLEAVED = 0, 1
FC_ROPE_PLAIN, FC_ROPE_LINEAR, FC_ROPE_NTK, FC_ROPE_YARN = 0, 1, 2, 3
_I64x3 = ctypes.c_int64 * 3


def _rows(t, name):
    """(pointer, (N, H, L, d), strides) of a [N, H, L, d] or [H, L, d] tensor whose
    rows are contiguous; the other strides are free (None: dense)."""
    if not t.is_cuda:
        raise FlowCacheError("tensor arguments must be CUDA tensors")
    shape = t.shape
    n = len(shape)
    if n != 4:
        if n != 3:
            raise FlowCacheError(f"{name} must be [N, H, L, d] or [H, L, d]")
        shape = (1,) + tuple(shape)
    if t.is_contiguous():
        return t.data_ptr(), shape, None
    st = t.stride()
    if st[-1] != 1 and shape[-1] > 1:
        raise FlowCacheError(f"the rows of {name} must be contiguous")
    return t.data_ptr(), shape, _I64x3(st[0] if n == 4 else 0, st[-3], st[-2])


def _ints(t, n, name):
    """Pointer of a contiguous int32 CUDA tensor of n elements."""
    if t.dtype is not torch.int32:
        raise FlowCacheError(f"{name} must be int32")
    if t.numel() != n:
        raise FlowCacheError(f"{name} has {t.numel()} elements, not {n}")
    return _p(t)


def _first_row(row0, N):
    """(host row, device rows) of a ``row0`` argument."""
    if isinstance(row0, torch.Tensor):
        return 0, _ints(row0, N, "row0")
    return int(row0), None


def _plan_args(rope, pos, N, L):
    if rope is None:
        return None, None
    if pos is None:
        raise FlowCacheError("a rotation needs pos")
    return ctypes.byref(rope), _ints(pos, rope.n_axes * N * L, "pos")


def fc_rope_init(rot_dim, layout=FC_ROPE_HALF, base=10000.0, scaling=FC_ROPE_PLAIN, factor=1.0,
                 orig_len=0, beta_fast=32.0, beta_slow=1.0, sections=None):
    """A :class:`RopePlan` for rows whose first ``rot_dim`` elements are rotated.
    ``sections``: the number of frequencies that follow each position axis (up to
    three, summing to rot_dim / 2); None for one axis."""
    plan = RopePlan()
    axes = 1 if sections is None else len(sections)
    sec = None if sections is None else (ctypes.c_int * axes)(*[int(s) for s in sections])
    st = library().fc_rope_init(ctypes.byref(plan), int(rot_dim), int(layout), float(base),
                                int(scaling), float(factor), int(orig_len), float(beta_fast),
                                float(beta_slow), axes, sec)
    _check("fc_rope_init", st)
    return plan


def fc_rope(x, y, pos, plan, inverse=False, stream=None):
    """Rotary positions.  x, y [N, H, L, d] (or [H, L, d]), strided, y may be x;
    pos [axes, N, L] int32.  ``inverse`` applies the transpose, which maps the
    gradient of y to the gradient of x."""
    xp, (N, H, L, d), xs = _rows(x, "x")
    yp, yshape, ys = _rows(y, "y")
    if yshape != (N, H, L, d) or y.dtype != x.dtype:
        raise FlowCacheError("x and y must have the same shape and type")
    rope, p = _plan_args(plan, pos, N, L)
    st = library().fc_rope(xp, yp, _dtype_code(x), N, H, L, d, xs, ys, p, rope, 1 if inverse else 0,
                            _s(stream))
    _check("fc_rope", st)


class Kv4Cache:
    """A cache in 4 bits: codes [N, H, cap, d/2] and scales [N, H, cap, d/16], uint8,
    for keys and for values.  Keeps the tensors alive; ``struct`` is the
    ``fc_kv4_cache`` that the calls take."""

    def __init__(self, k_codes, k_scales, v_codes, v_scales, k_exp=0, v_exp=0):
        N, H, cap, half = k_codes.shape
        for t, last in ((k_codes, half), (v_codes, half), (k_scales, half // 8), (v_scales, half // 8)):
            if t.dtype != torch.uint8 or tuple(t.shape) != (N, H, cap, last):
                raise FlowCacheError("a cache has uint8 codes [N, H, cap, d/2] and scales [N, H, cap, d/16]")
        self.k_codes, self.k_scales, self.v_codes, self.v_scales = k_codes, k_scales, v_codes, v_scales
        self.N, self.H, self.cap, self.d = N, H, cap, 2 * half
        self.struct = _Kv4(_p(k_codes), _p(k_scales), _p(v_codes), _p(v_scales), N, H, cap, 2 * half,
                           int(k_exp), int(v_exp))
        self._ref = ctypes.byref(self.struct)


def fc_kv4_cache(N, H, cap, d, k_exp=0, v_exp=0, device=None):
    """A zeroed :class:`Kv4Cache` of N sequences, H heads and cap rows (a multiple
    of 16) of d elements."""
    z = lambda last: torch.zeros(N, H, cap, last, dtype=torch.uint8, device=device or "cuda")  # noqa: E731
    return Kv4Cache(z(d // 2), z(d // 16), z(d // 2), z(d // 16), k_exp, v_exp)


def fc_kv4_store(k, v, cache, row0=0, idx=None, rope=None, pos=None, stream=None):
    """Write k, v [N, H, L, d] (or [H, L, d]) as 4-bit rows from ``row0`` on (an int,
    or [N] int32 on the device).  ``idx`` [N, H, B] int32 selects the rows written;
    ``rope`` and ``pos`` rotate the keys on the way."""
    kp, (N, H, L, d), ks = _rows(k, "k")
    vp, vshape, vs = _rows(v, "v")
    if vshape != (N, H, L, d) or v.dtype != k.dtype:
        raise FlowCacheError("k and v must have the same shape and type")
    host, dev = _first_row(row0, N)
    B = 0 if idx is None else idx.shape[-1]
    plan, p = _plan_args(rope, pos, N, L)
    st = library().fc_kv4_store(kp, vp, _dtype_code(k), N, H, L, d, ks, vs,
                                 None if idx is None else _ints(idx, N * H * B, "idx"), B, host, dev,
                                 plan, p, cache._ref, _s(stream))
    _check("fc_kv4_store", st)


def fc_kv4_load(cache, k_out, v_out, row0=0, stream=None):
    """The numbers of rows row0 .. row0 + L of the cache into k_out, v_out
    [N, H, L, d] (or [H, L, d])."""
    kp, (N, H, L, d), ks = _rows(k_out, "k_out")
    vp, vshape, vs = _rows(v_out, "v_out")
    if vshape != (N, H, L, d) or v_out.dtype != k_out.dtype or (N, H, d) != (cache.N, cache.H, cache.d):
        raise FlowCacheError("k_out and v_out must be [N, H, L, d] of the cache, of one type")
    host, dev = _first_row(row0, N)
    st = library().fc_kv4_load(cache._ref, kp, vp, _dtype_code(k_out), L, ks, vs, host,
                                dev, _s(stream))
    _check("fc_kv4_load", st)


def fc_kv4_attention_workspace_size(dtype, N, Hq, Hkv, Lq, max_len, d):
    return library().fc_kv4_attention_workspace_size(dtype, N, Hq, Hkv, Lq, max_len, d)


def fc_kv4_attention(q, cache, lens, out, ws, max_len=None, causal=False, scale=0.0, lse=None,
                     stream=None):
    """Attention of q [N, Hq, Lq, d] (or [Hq, Lq, d]) over the cache.  lens: [N] int32
    on the device, an int (at most max_len) for all sequences, or None (max_len of
    each); max_len bounds the lengths (cap if None; those on the device are clamped).
    out like q; lse [N, Hq, Lq] float32 or None; ws from :func:`fc_kv4_attention_workspace_size`."""
    qp, (N, Hq, Lq, d), qs = _rows(q, "q")
    op, oshape, os_ = _rows(out, "out")
    if oshape != (N, Hq, Lq, d) or out.dtype != q.dtype:
        raise FlowCacheError("q and out must have the same shape and type")
    if max_len is None:
        max_len = cache.cap
    lp = None
    if isinstance(lens, torch.Tensor):
        lp = _ints(lens, N, "lens")
    elif lens is not None:
        if int(lens) > int(max_len):
            raise FlowCacheError(f"FC_ERR_INVALID_ARG: lens {int(lens)} is over max_len {int(max_len)}", 1)
        max_len = int(lens)
    if lse is not None and (lse.dtype != torch.float32 or lse.numel() != N * Hq * Lq):
        raise FlowCacheError("lse must be [N, Hq, Lq] float32")
    st = library().fc_kv4_attention(qp, cache._ref, lp, int(max_len), _dtype_code(q),
                                     N, Hq, Lq, d, qs, 1 if causal else 0, float(scale), op, os_,
                                     _p(lse), _p(ws), ws.numel() * ws.element_size(), _s(stream))
    _check("fc_kv4_attention", st)
