"""fp64 numpy oracle of attention over packed prompts with grouped heads, and of its gradients,
sequence by sequence and head by head from the definition.  Shares no code with the CUDA
library."""
from __future__ import annotations

import numpy as np


def _spans(offsets):
    return [(int(a), int(z)) for a, z in zip(offsets, offsets[1:]) if z > a]


def _scores(q, k, causal):
    s = q @ k.T / np.sqrt(q.shape[-1])
    if causal:
        s[np.triu_indices(len(s), 1)] = -np.inf
    return s


def attention(q, k, v, offsets, causal):
    """q [T, Hq, d], k, v [T, Hk, d]: out [T, Hq, d] and lse [Hq, T], NaN in rows of no sequence;
    then, row by row, the largest sum |q k| / sqrt(d) [T, Hq] and sum p |v| [T, Hq, d], which
    errors are measured in."""
    T, Hq, d = q.shape
    G = Hq // k.shape[1]
    out, lse = np.full((T, Hq, d), np.nan), np.full((Hq, T), np.nan)
    size, spread = np.zeros((T, Hq)), np.zeros((T, Hq, d))
    for a, z in _spans(offsets):
        for h in range(Hq):
            kh, vh = k[a:z, h // G], v[a:z, h // G]
            s = _scores(q[a:z, h], kh, causal)
            m = s.max(-1, keepdims=True)
            e = np.exp(s - m)
            total = e.sum(-1, keepdims=True)
            out[a:z, h] = e / total @ vh
            lse[h, a:z] = (m + np.log(total))[:, 0]
            size[a:z, h] = _scores(np.abs(q[a:z, h]), np.abs(kh), causal).max(-1)
            spread[a:z, h] = e / total @ np.abs(vh)
    return out, lse, size, spread


def attention_bwd(q, k, v, out, lse, dout, offsets, causal):
    """The gradients of sum(out * dout) from the forward's out and lse: dq, dk, dv (NaN in rows of
    no sequence), and the sums of their terms' magnitudes: for each gradient the sum of |dS| (P
    for dv) times the other factor, and that of P (sum |dO v| + sum |dO O|) for dq and dk."""
    Hq, Hk, d = q.shape[1], k.shape[1], q.shape[2]
    G = Hq // Hk
    dq = np.full(q.shape, np.nan)
    dk, dv = np.full(k.shape, np.nan), np.full(v.shape, np.nan)
    terms = [np.zeros(q.shape), np.zeros(k.shape), np.zeros(v.shape)]
    fine = [np.zeros(q.shape), np.zeros(k.shape)]
    for a, z in _spans(offsets):
        dk[a:z] = dv[a:z] = 0
        for h in range(Hq):
            g, kv = dout[a:z, h], h // G
            qh, kh, vh = q[a:z, h], k[a:z, kv], v[a:z, kv]
            p = np.exp(_scores(qh, kh, causal) - lse[h, a:z, None])
            ds = p * (g @ vh.T - (g * out[a:z, h]).sum(-1, keepdims=True)) / np.sqrt(d)
            rough = p * (np.abs(g) @ np.abs(vh).T
                         + np.abs(g * out[a:z, h]).sum(-1, keepdims=True)) / np.sqrt(d)
            dv[a:z, kv] += p.T @ g
            dk[a:z, kv] += ds.T @ qh
            dq[a:z, h] = ds @ kh
            terms[2][a:z, kv] += p.T @ np.abs(g)
            terms[1][a:z, kv] += np.abs(ds).T @ np.abs(qh)
            terms[0][a:z, h] = np.abs(ds) @ np.abs(kh)
            fine[1][a:z, kv] += rough.T @ np.abs(qh)
            fine[0][a:z, h] = rough @ np.abs(kh)
    return (dq, dk, dv), terms, fine
