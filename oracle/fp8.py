"""Plain CPU oracle of the FP8 page cache: the cache write, attention over the pages (dense or
over selected blocks) with the weight each block collects, and eviction by that weight.

TEST INFRASTRUCTURE ONLY, like the rest of this package: float64 numpy from the exact values
of the cache bytes, sharing no code with the CUDA path.  The definitions are those of
include/msa.h (msa_fp8_append, msa_fp8_attn, msa_evict_blocks).

attention() also returns what bounds a float32 computation of the same formula, so that tests
state their tolerances from the inputs instead of fitting them:
  spread  A = sum_j p_j |v_j| per output element: an error of relative size r in every p_j moves
          the output by at most r A
  logit   the largest sum_d |q_d k_jd| over the row's visible keys: float32 accumulation of the 128
          products is off by at most 128 * 2^-24 times it
  k_abs   the largest sum_d |k_jd|, for errors of the query elements
  v_abs   the largest |v_jd| per output element;  p_max  the largest p_j
"""
from __future__ import annotations

import math

import numpy as np

from .formats import E4M3_TABLE, e4m3_encode

BLOCK, DIM = 128, 128
E8M0_ONE, E8M0_MIN, E8M0_MAX = 127, 87, 167


def page_exponent(amax: float) -> int:
    """Smallest e in -40..40 with amax <= 448 * 2^e (40 if there is none)."""
    for e in range(E8M0_MIN - E8M0_ONE, E8M0_MAX - E8M0_ONE):
        if amax <= math.ldexp(448.0, e):
            return e
    return E8M0_MAX - E8M0_ONE


def _encode(x: np.ndarray) -> np.ndarray:
    return np.where(np.isnan(x), 0x7F, e4m3_encode(np.where(np.isnan(x), 0.0, x))).astype(np.uint8)


def append(data, scale, x, table, lens):
    """One pool (K or V): data uint8 [P, G, 128, 128], scale uint8 [P, G], x float [B, T, G, 128]
    at positions lens[b] - T .. lens[b] - 1.  Returns the pool's new contents."""
    data, scale = data.copy(), scale.copy()
    B, T, G, _ = x.shape
    for b in range(B):
        L = int(lens[b])
        if L < T or L > table.shape[1] * BLOCK:
            continue
        for n in range((L - T) // BLOCK, (L - 1) // BLOCK + 1):
            page = int(table[b, n])
            if not 0 <= page < data.shape[0]:
                continue
            lo, hi = max(L - T - n * BLOCK, 0), min(L - n * BLOCK, BLOCK)
            for g in range(G):
                rows = x[b, n * BLOCK + lo - (L - T):n * BLOCK + hi - (L - T), g].astype(np.float64)
                real = np.abs(rows[~np.isnan(rows)])
                e = page_exponent(float(real.max()) if real.size else 0.0)
                if lo > 0:
                    if not E8M0_MIN <= scale[page, g] <= E8M0_MAX:
                        continue
                    old = int(scale[page, g]) - E8M0_ONE
                    e = max(e, old)
                    if e > old:
                        data[page, g, :lo] = _encode(E4M3_TABLE[data[page, g, :lo]] * 2.0 ** (old - e))
                data[page, g, lo:hi] = _encode(rows * 2.0 ** -e)
                scale[page, g] = e + E8M0_ONE
    return data, scale


def values(codes, scale):
    """Exact values of code pages [..., 128, 128] under E8M0 scales [...]."""
    return E4M3_TABLE[codes] * np.exp2(scale.astype(np.float64) - E8M0_ONE)[..., None, None]


def attention(q, cache, table, lens, heads_per_group, selection=None, weight_in=None, decay=1.0,
              softmax_scale=1.0 / math.sqrt(DIM)):
    """q float64 [B, T, H, 128]; cache (k_data, k_scale, v_data, v_scale); selection [B, T, G, 16] or
    None (dense).  Returns a dict: out, lse, weight, and the error scales above."""
    k_data, k_scale, v_data, v_scale = cache
    B, T, H, _ = q.shape
    Hg, MB = heads_per_group, table.shape[1]
    got = dict(out=np.zeros((B, T, H, DIM)), lse=np.full((B, T, H), -np.inf), spread=np.zeros((B, T, H, DIM)),
               logit=np.zeros((B, T, H)), k_abs=np.zeros((B, T, H)), v_abs=np.zeros((B, T, H, DIM)),
               p_max=np.zeros((B, T, H)), keys=np.zeros((B, T, H), np.int64))
    weight = np.zeros((B, MB)) if weight_in is None else decay * weight_in.astype(np.float64)
    ok_scale = lambda s: E8M0_MIN <= s <= E8M0_MAX  # noqa: E731
    for b in range(B):
        L = int(lens[b])
        if L < T or L <= 0 or L > MB * BLOCK:
            continue
        for t in range(T):
            pos = L - T + t
            for g in range(H // Hg):
                blocks = range(pos // BLOCK + 1) if selection is None else [
                    int(n) for n in selection[b, t, g] if 0 <= n <= pos // BLOCK]
                blocks = [n for n in blocks if 0 <= table[b, n] < k_data.shape[0]
                          and ok_scale(k_scale[table[b, n], g]) and ok_scale(v_scale[table[b, n], g])]
                if not blocks:
                    continue
                pages = table[b, blocks]
                seen = (np.array(blocks)[:, None] * BLOCK + np.arange(BLOCK) <= pos).reshape(-1)
                K = values(k_data[pages, g], k_scale[pages, g]).reshape(-1, DIM)[seen]
                V = values(v_data[pages, g], v_scale[pages, g]).reshape(-1, DIM)[seen]
                owner = np.repeat(np.array(blocks), BLOCK)[seen]
                for h in range(g * Hg, (g + 1) * Hg):
                    z = K @ q[b, t, h] * softmax_scale
                    top = z.max()
                    p = np.exp(z - top)
                    total = p.sum()
                    p /= total
                    got["lse"][b, t, h] = top + math.log(total) if total > 0 else np.nan
                    got["out"][b, t, h] = p @ V
                    got["spread"][b, t, h] = p @ np.abs(V)
                    got["logit"][b, t, h] = (np.abs(K) @ np.abs(q[b, t, h])).max()
                    got["k_abs"][b, t, h] = np.abs(K).sum(1).max()
                    got["v_abs"][b, t, h] = np.abs(V).max(0)
                    got["p_max"][b, t, h] = p.max()
                    got["keys"][b, t, h] = len(z)
                    np.add.at(weight[b], owner, p)
    got["weight"] = weight
    return got


def evict(table, lens, weight, budget, keep_first, keep_last):
    """(table, lens, weight, freed, freed count) after the cut."""
    B, MB = table.shape
    out = (np.full((B, MB), -1, np.int32), lens.copy(), np.zeros((B, MB), weight.dtype),
           np.full((B, MB), -1, np.int32), np.zeros(B, np.int32))
    for b in range(B):
        L = int(lens[b])
        bad = L < 0 or L > MB * BLOCK
        nb = MB if bad else -(-L // BLOCK)
        stay = list(range(nb))
        if not bad and nb > budget:
            forced = [n for n in stay if n < keep_first or n >= nb - keep_last]
            # NaN below -inf: (is a number, value)
            rest = sorted((n for n in stay if n not in set(forced)),
                          key=lambda n: (not math.isnan(weight[b, n]), 0.0 if math.isnan(weight[b, n]) else weight[b, n]),
                          reverse=True)  # stable: the lower block first among equals
            stay = sorted(forced + rest[:budget - len(forced)])
        gone = sorted(set(range(nb)) - set(stay))
        out[0][b, :len(stay)], out[2][b, :len(stay)] = table[b, stay], weight[b, stay]
        out[3][b, :len(gone)], out[4][b] = table[b, gone], len(gone)
        if not bad:
            out[1][b] = L - BLOCK * len(gone)
    return out
