"""Inputs and tolerances shared by the tests of the packed prompt attention."""
from __future__ import annotations

import numpy as np

from oracle import prompt as OP


class Prompts:
    """Packed prompts on both sides.  Tokens of no sequence (gaps before the first one, behind the last one) are NaN.
    fused: q, k and v are slices of one projection's rows (needs equal lengths)."""

    def __init__(self, seed, lens_q, lens_k=None, G=2, Hg=8, before=0, behind=0, fused=False, scale=0.0, dev=1.5):
        import torch
        rng = self.rng = np.random.default_rng(seed)
        lens_k = list(lens_q) if lens_k is None else list(lens_k)
        self.G, self.Hg, self.H, self.scale, self.B = G, Hg, G * Hg, scale, len(lens_q)
        self.cu_q = (before + np.concatenate([[0], np.cumsum(lens_q)])).astype(np.int32)
        self.cu_k = (before + np.concatenate([[0], np.cumsum(lens_k)])).astype(np.int32)
        self.Nq, self.Nk = int(self.cu_q[-1]) + behind, int(self.cu_k[-1]) + behind
        self.used_q = np.zeros(self.Nq, bool)
        self.used_q[before:self.cu_q[-1]] = True

        def rows(n, heads, used, dev):
            x = torch.from_numpy(rng.normal(0, dev, (n, heads, 128)).astype(np.float32)).to(torch.bfloat16)
            x[~torch.from_numpy(used)] = float("nan")
            return x

        used_k = np.zeros(self.Nk, bool)
        used_k[before:self.cu_k[-1]] = True
        self.q, self.k, self.v = rows(self.Nq, self.H, self.used_q, dev), rows(self.Nk, G, used_k, dev), rows(self.Nk, G, used_k, 1.0)
        self.fused = fused

    def oracle(self):
        scale = self.scale or 1.0 / np.sqrt(128.0)
        with np.errstate(invalid="ignore", over="ignore", divide="ignore"):
            return OP.attention(self.q.double().numpy(), self.k.double().numpy(), self.v.double().numpy(), self.cu_q, self.cu_k,
                                self.Hg, scale)

    def upload(self):
        import torch
        import block_sparse_attention_indexer_gb300 as msa
        self.cfg = msa.Config(num_kv_groups=self.G, heads_per_group=self.Hg, softmax_scale=self.scale)
        self.packed = msa.Packed(torch.from_numpy(self.cu_q).cuda(), torch.from_numpy(self.cu_k).cuda(), self.Nq, self.Nk)
        if self.fused:
            self.d = torch.cat([self.q, self.k, self.v], dim=1).cuda().split((self.H, self.G, self.G), dim=1)
        else:
            self.d = [x.cuda() for x in (self.q, self.k, self.v)]
        self.out = torch.full((self.Nq, self.H, 128), 7.0, dtype=torch.bfloat16, device="cuda")
        self.lse = torch.full((self.Nq, self.H), 7.0, device="cuda")
        self.ws = msa.alloc_workspace(msa.MSA_OP_PROMPT_ATTN, self.cfg, self.packed)
        return self

    def call(self, lse=True, stream=None):
        import block_sparse_attention_indexer_gb300 as msa
        msa.msa_prompt_attn(self.cfg, self.packed, *self.d, self.out, self.lse if lse else None, self.ws, stream=stream)

    def results(self):
        import torch
        import block_sparse_attention_indexer_gb300 as msa
        torch.cuda.synchronize()
        return self.out.double().cpu().numpy(), self.lse.double().cpu().numpy(), msa.msa_read_device_error(self.ws)

    def check(self, got, ref=None):
        """Against the 64-bit definition, element by element:
          * a logit: 128 exact products summed in float32 in any order, and the products with the scale and the
            subtraction of the reference: (128 + 4) * 2^-24 of sum |q k|;
          * a probability: the logit's error twice (in it and in the sum), 2^-20 for exp2 and the sums;
          * it is rounded to bfloat16, p (1 + d_j) with |d_j| <= 2^-8 (half a step), and the output divided by the sum of what
            was rounded: sum p_j (1 + d_j) v_j / (1 + D) with D = sum p_j d_j is off by
            sum p_j (d_j - D) v_j / (1 + D), at most 2 * 2^-8 / (1 - 2^-8) < 2^-7 + 2^-14 of sum p |v|;
          * the sum over keys in float32: one rounding for each key, 2^-24 of sum p |v|;
          * the output rounded to bfloat16: 2^-8 of it.
        Rows of no sequence keep what they held."""
        out, lse, err = got
        ref = self.oracle() if ref is None else ref
        scale = self.scale or 1.0 / np.sqrt(128.0)
        assert err == 0, err
        assert (out[~self.used_q] == 7.0).all() and (lse[~self.used_q] == 7.0).all(), "rows of no sequence"
        u = self.used_q
        dz = scale * ref["logit"] * (128 + 4) * 2.0 ** -24
        rel = 2 * dz + 2.0 ** -20 + ref["keys"] * 2.0 ** -24 + 2.0 ** -7 + 2.0 ** -14
        close("out", out[u], ref["out"][u], (2.0 ** -8 * np.abs(ref["out"]) + rel[..., None] * ref["spread"] + 1e-30)[u])
        at = np.where(np.isfinite(ref["lse"]), ref["lse"], 0.0)
        close("lse", lse[u], ref["lse"][u], (dz + 2.0 ** -20 + ref["keys"] * 2.0 ** -24 + 2.0 ** -22 * np.abs(at))[u])


def close(name, got, want, bound):
    special = ~np.isfinite(want)
    assert np.array_equal(np.isnan(got), np.isnan(want)), (name, "NaN at other places", np.argwhere(
        np.isnan(got) != np.isnan(want))[:4])
    assert np.array_equal(got[special & ~np.isnan(want)], want[special & ~np.isnan(want)]), (name, "infinities")
    err = np.where(special, 0.0, np.abs(np.where(special, 0, got) - np.where(special, 0, want)))
    bad = err > np.where(special, 0.0, bound)
    assert not bad.any(), (name, int(bad.sum()), np.argwhere(bad)[:4].tolist(), float(np.nanmax(err / np.where(special, 1, bound))))
