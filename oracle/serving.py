"""fp64 numpy oracle of the operators around the attention: the per-head norm
and rotation of queries and keys with its gradient, the append to a paged
cache, and decode attention over such a cache.  Written row by row from the
definitions; shares no code with the CUDA library."""
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
