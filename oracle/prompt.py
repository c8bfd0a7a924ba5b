"""Causal attention of packed prompts in 64 bits, row by row over the keys that the row sees."""
from __future__ import annotations

import numpy as np


def attention(q, k, v, cu_q, cu_k, heads_per_group, softmax_scale):
    """q [Nq, H, D], k, v [Nk, G, D] float64 -> out [Nq, H, D], lse [Nq, H] (rows of no sequence: 0,
    -inf), and what error bounds need: spread = sum p |v|, logit = max over the row's keys of sum |q k|,
    keys = how many a row sees."""
    Nq, H, D = q.shape
    out, lse = np.zeros((Nq, H, D)), np.full((Nq, H), -np.inf)
    spread, logit, keys = np.zeros((Nq, H, D)), np.zeros((Nq, H)), np.zeros((Nq, H))
    for b in range(len(cu_q) - 1):
        Lq, Lk = int(cu_q[b + 1] - cu_q[b]), int(cu_k[b + 1] - cu_k[b])
        for g in range(k.shape[1]):
            K, V = k[cu_k[b]:cu_k[b + 1], g], v[cu_k[b]:cu_k[b + 1], g]
            for t in range(Lq):
                n = Lk - Lq + t + 1
                if n <= 0:
                    continue
                rows = slice(g * heads_per_group, (g + 1) * heads_per_group)
                x = q[cu_q[b] + t, rows]
                z = (x @ K[:n].T) * softmax_scale
                m = z.max(axis=1, keepdims=True)
                p = np.exp(z - m)
                total = p.sum(axis=1, keepdims=True)
                p /= total
                i = (cu_q[b] + t, rows)
                out[i] = p @ V[:n]
                lse[i] = (m + np.log(total))[:, 0]
                spread[i] = p @ np.abs(V[:n])
                logit[i] = (np.abs(x) @ np.abs(K[:n]).T).max(axis=1)
                keys[i] = n
    return dict(out=out, lse=lse, spread=spread, logit=logit, keys=keys)
