"""fp64 numpy oracle of the operators around the attention: the per-head norm
and rotation of queries and keys with its gradient, the append to a paged
cache, decode attention over such a cache, and what a cache in 4 bits holds.
Written row by row from the definitions; shares no code with the CUDA library."""
from __future__ import annotations

import numpy as np


def angles(positions, inv_freq):
    """positions [...] x inv_freq [r] -> angles [..., r], reduced modulo a turn in extended
    precision where the platform has it."""
    p = np.asarray(positions, dtype=np.longdouble)[..., None]
    f = np.asarray(inv_freq, dtype=np.float32).astype(np.longdouble)
    turn = 2 * np.longdouble("3.14159265358979323846264338327950288")
    return np.fmod(p * f, turn).astype(np.float64)


def rotate(x, angle, interleaved):
    """x [..., d]: pairs of its first 2 * angle.shape[-1] entries turned by angle [..., r]."""
    y = np.array(x, dtype=np.float64)
    r = angle.shape[-1]
    a_at = np.arange(r) * 2 if interleaved else np.arange(r)
    b_at = a_at + (1 if interleaved else r)
    a, b = x[..., a_at], x[..., b_at]
    y[..., a_at] = a * np.cos(angle) - b * np.sin(angle)
    y[..., b_at] = b * np.cos(angle) + a * np.sin(angle)
    return y


def norm_rope(x, weight, eps, inv_freq, positions, interleaved=False):
    """x [B, S, H, d], positions [B, S] -> (y, x's norms' reciprocals [B, S, H, 1])."""
    x = np.asarray(x, dtype=np.float64)
    r = np.ones(x.shape[:-1] + (1,))
    y = x
    if weight is not None:
        r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
        y = x * r * np.asarray(weight, dtype=np.float64)
    if inv_freq is not None and len(inv_freq):
        y = rotate(y, angles(positions, inv_freq)[:, :, None, :], interleaved)
    return y, r


def norm_rope_bwd(dy, x, weight, eps, inv_freq, positions, interleaved=False):
    """Gradients (dx, dweight or None) of sum(norm_rope(x) * dy)."""
    g = np.asarray(dy, dtype=np.float64)
    x = np.asarray(x, dtype=np.float64)
    if inv_freq is not None and len(inv_freq):
        g = rotate(g, -angles(positions, inv_freq)[:, :, None, :], interleaved)
    if weight is None:
        return g, None
    w = np.asarray(weight, dtype=np.float64)
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    u = x * r
    gw = g * w
    return r * (gw - u * (gw * u).mean(-1, keepdims=True)), (g * u).sum((0, 1, 2))


def paged_decode(q, k_cache, v_cache, table, seq_lens, prefix_pages=(), prefix_len=0):
    """q [B, n, Hq, d]; caches [pages, page_size, Hk, d] (values); one softmax per row over the keys
    it sees, gathered one by one.  Returns out [B, n, Hq, d] and lse [B, Hq, n]."""
    q = np.asarray(q, dtype=np.float64)
    B, n, Hq, d = q.shape
    ps, Hk = k_cache.shape[1], k_cache.shape[2]
    out = np.zeros((B, n, Hq, d))
    lse = np.full((B, Hq, n), -np.inf)
    for b in range(B):
        L = int(seq_lens[b])
        if L == 0:
            continue
        for i in range(n):
            seen = [(int(prefix_pages[p // ps]), p % ps) for p in range(prefix_len)]
            seen += [(int(table[b][p // ps]), p % ps)
                     for p in range(prefix_len, L - n + i + 1)]
            if not seen:
                continue
            pg, sl = (np.array(x) for x in zip(*seen))
            for h in range(Hq):
                hk = h // (Hq // Hk)
                s = k_cache[pg, sl, hk].astype(np.float64) @ q[b, i, h] / np.sqrt(d)
                m = s.max()
                e = np.exp(s - m)
                out[b, i, h] = (e / e.sum()) @ v_cache[pg, sl, hk].astype(np.float64)
                lse[b, h, i] = m + np.log(e.sum())
    return out, lse


def e4m3_values():
    """The values of the E4M3 codes 0 .. 0x7E (a sign bit of 0; 0x7F is NaN), ascending."""
    return np.array([(m / 8 * 2.0 ** -6) if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
                     for e in range(16) for m in range(8)][:127])


def e4m3_codes(x):
    """Codes of the nearest E4M3 values of x >= 0, ties to the even code, saturated at 448."""
    v = e4m3_values()
    up = np.clip(np.searchsorted(v, x), 1, 126)
    lo, hi = v[up - 1], v[up]
    even = np.where(up % 2 == 0, up, up - 1)
    code = np.where(x - lo < hi - x, up - 1, np.where(x - lo > hi - x, up, even))
    return np.where(x >= 448, 126, code).astype(np.uint8)


def quantise4(x, descale=None):
    """Rows x [..., Hk, d] as a cache in 4 bits holds them: codes [..., Hk, d / 2] (two to a byte,
    the low half first) and E4M3 scale codes [..., Hk, d / 16].  The products with 1 / descale and
    1 / 7 are fp32 operations by definition; the quotient's rounding is the same from fp32 and
    from fp64 but for ties that fp32 makes, which no bf16 row without a descale has."""
    f = np.float32
    y = np.asarray(x, dtype=f)
    if descale is not None:
        y = y * (f(1) / np.asarray(descale, dtype=f))[:, None]
    y = y.reshape(*y.shape[:-1], -1, 16)
    scales = e4m3_codes((np.abs(y).max(-1) * (f(1) / f(7))).astype(np.float64))
    s = e4m3_values()[scales][..., None]
    q = np.divide(y, s.astype(f), out=np.zeros_like(y), where=s > 0)
    n = np.clip(np.rint(np.nan_to_num(q, nan=0.0, posinf=7, neginf=-7)), -7, 7) + 8
    n = n.astype(np.uint8).reshape(*y.shape[:-2], -1)
    return n[..., ::2] | n[..., 1::2] << 4, scales


def values4(codes, scales, descale=None):
    """What codes [..., Hk, d / 2] with scale codes [..., Hk, d / 16] stand for, in 64 bits."""
    n = np.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-1], -1).astype(np.float64) - 8
    s = np.append(e4m3_values(), np.nan)[scales & 0x7F] * np.where(scales >> 7, -1.0, 1.0)
    v = (n.reshape(*n.shape[:-1], -1, 16) * s[..., None]).reshape(n.shape)
    return v if descale is None else v * np.asarray(descale, dtype=np.float64)[:, None]
