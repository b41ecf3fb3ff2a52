"""Plain CPU oracle of the rotary positions, the 4-bit cache and its attention.

TEST INFRASTRUCTURE, NOT PRODUCT CODE, like the rest of this folder: numpy, one
definition after the other, float64 except where a definition rounds to a
narrower type (those roundings are written out).
"""

import numpy as np

__all__ = ["rope_turns", "rope", "kv4_quantise", "kv4_values", "kv4_pack", "kv4_unpack",
           "kv4_attention"]

E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])


def _e4m3(b):
    """The number of an e4m3 byte."""
    e, m = (b >> 3) & 15, b & 7
    if e == 15 and m == 7:
        return np.nan
    return (m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)) * (-1 if b & 128 else 1)


E4M3 = np.array([_e4m3(b) for b in range(256)])


def rope_turns(rot_dim, base=10000.0, scaling="plain", factor=1.0, orig_len=0, beta_fast=32.0,
               beta_slow=1.0):
    """(turns per position of every frequency, the factor m)."""
    i = np.arange(rot_dim // 2)
    if scaling == "ntk" and rot_dim > 2:
        base = base * factor ** (rot_dim / (rot_dim - 2))
    w = base ** (-2.0 * i / rot_dim) / (2 * np.pi)
    if scaling == "linear":
        return w / factor, 1.0
    if scaling == "yarn":
        keep = np.clip((orig_len * w - beta_slow) / (beta_fast - beta_slow), 0, 1)
        return (1 - keep) * w / factor + keep * w, 0.1 * np.log(factor) + 1
    return w, 1.0


def rope(x, pos, turns, m=1.0, interleaved=False, axis=None, inverse=False):
    """x [N, H, L, d] rotated in its first 2*len(turns) elements; pos [A, N, L]."""
    x = np.array(x, np.float64)
    half = len(turns)
    axis = np.zeros(half, int) if axis is None else np.asarray(axis)
    u = np.moveaxis(np.asarray(pos, np.float64)[axis], 0, -1) * turns  # [N, L, half]
    u = (u - np.rint(u)) * 2 * np.pi
    c, s = (m * np.cos(u))[:, None], (m * np.sin(u))[:, None]
    if inverse:
        s = -s
    i = np.arange(half)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    y = x.copy()
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    return y


def kv4_quantise(x, exp=0):
    """x [..., d] (float32 values) -> (codes 0..15 [..., d], scale bytes [..., d/16])."""
    with np.errstate(all="ignore"):
        y = (np.asarray(x, np.float32) * np.float32(2.0 ** -exp)).reshape(*x.shape[:-1], -1, 16)
        a = np.abs(y).max(-1)  # NaN stays
        q = np.minimum(a / np.float32(6), np.float32(448)).astype(np.float64)
        # nearest of the 127 non-negative numbers, the even mantissa on a tie
        grid = E4M3[:127]
        hi = np.clip(np.searchsorted(grid, q), 1, 126)
        lo = hi - 1
        dl, dh = q - grid[lo], grid[hi] - q
        b = np.where((dh < dl) | ((dh == dl) & (hi % 2 == 0)), hi, lo)
        b = np.where(np.isnan(q), 0x7F, b)
        s = E4M3[b].astype(np.float32)[..., None]
        t = np.where(s > 0, np.abs(y) / s, np.float32(0)).astype(np.float64)
    mid = (E2M1[1:] + E2M1[:-1]) / 2
    code = np.zeros(y.shape, np.int64)
    for k, mv in enumerate(mid):  # a tie goes to the even code
        code += (t >= mv) if k % 2 else (t > mv)
    code = np.where(np.isnan(s), 0, code | (np.signbit(y).astype(np.int64) << 3))
    return code.reshape(x.shape).astype(np.uint8), b.astype(np.uint8)


def kv4_pack(code):
    return (code[..., 0::2] | (code[..., 1::2] << 4)).astype(np.uint8)


def kv4_unpack(packed):
    out = np.empty(packed.shape[:-1] + (packed.shape[-1] * 2,), np.uint8)
    out[..., 0::2] = packed & 15
    out[..., 1::2] = packed >> 4
    return out


def kv4_values(packed, scales, exp=0):
    """float64 numbers of packed rows."""
    c = kv4_unpack(packed)
    v = E2M1[c & 7] * np.where(c & 8, -1.0, 1.0)
    return v * np.repeat(E4M3[scales], 16, axis=-1) * 2.0 ** exp


def kv4_attention(q, k, v, lens, causal=False, scale=None):
    """q [N, Hq, Lq, d]; k, v [N, Hkv, cap, d] numbers; lens [N].  Returns (out, lse,
    spread, reach, flat): spread_i = sum p |v| / sum p and flat_i = max p sum |v| /
    sum p per element, and reach_i = max_j scale sum_d |q_d k_jd|: what the error
    bounds of a test go by."""
    N, Hq, Lq, d = q.shape
    G = Hq // k.shape[1]
    scale = 1 / np.sqrt(d) if scale is None else scale
    out = np.zeros(q.shape)
    spread, flat = np.zeros(q.shape), np.zeros(q.shape)
    lse = np.full((N, Hq, Lq), -np.inf)
    reach = np.zeros((N, Hq, Lq))
    for n in range(N):
        for h in range(Hq):
            kk, vv = k[n, h // G], v[n, h // G]
            for i in range(Lq):
                top = min(lens[n], lens[n] - Lq + i + 1) if causal else lens[n]
                if top <= 0:
                    continue
                x = kk[:top] @ q[n, h, i] * scale
                p = np.exp(x - x.max())
                z = p.sum()
                out[n, h, i] = p @ vv[:top] / z
                spread[n, h, i] = p @ np.abs(vv[:top]) / z
                flat[n, h, i] = np.abs(vv[:top]).sum(0) / z
                lse[n, h, i] = np.log(z) + x.max()
                reach[n, h, i] = scale * (np.abs(kk[:top]) @ np.abs(q[n, h, i])).max()
    return out, lse, spread, reach, flat
