"""Inputs and tolerances shared by the tests of the FP8 page cache."""
from __future__ import annotations

import numpy as np

from oracle import fp8 as OF8
from oracle.formats import E4M3_TABLE, e4m3_encode


def random_codes(rng, *shape, dev=64.0):
    return e4m3_encode(rng.normal(0, dev, shape).clip(-448, 448)).astype(np.uint8)


class Case:
    """A paged cache on both sides.  Everything that no row may use is poison: NaN codes behind
    each sequence's end and in pages of no sequence, whose scales are invalid too."""

    def __init__(self, seed, lens, T, G, Hg, q_type="e4m3", max_blocks=None, spare=2, scales=(119, 124), q_dev=1.5,
                 softmax_scale=0.0, q_scale=1.0):
        rng = self.rng = np.random.default_rng(seed)
        self.T, self.G, self.Hg, self.B = T, G, Hg, len(lens)
        self.lens = np.array(lens, np.int32)
        nb = [-(-int(n) // 128) for n in lens]
        self.max_blocks = max_blocks or max(1, max(nb))
        P = sum(nb) + spare
        order = rng.permutation(P)
        self.table = np.full((self.B, self.max_blocks), -1, np.int32)
        self.k, self.v = random_codes(rng, P, G, 128, 128), random_codes(rng, P, G, 128, 128)
        self.ks = rng.integers(scales[0], scales[1], (P, G)).astype(np.uint8)
        self.vs = rng.integers(scales[0], scales[1], (P, G)).astype(np.uint8)
        at = 0
        for b, n in enumerate(nb):
            self.table[b, :n] = order[at:at + n]
            at += n
            if lens[b] % 128:
                last = self.table[b, n - 1]
                self.k[last, :, lens[b] % 128:] = 0x7F
                self.v[last, :, lens[b] % 128:] = 0xFF
        for p in order[at:]:
            self.k[p], self.v[p], self.ks[p], self.vs[p] = 0x7F, 0x7F, 255, 0
        q = rng.normal(0, q_dev, (self.B, T, G * Hg, 128)) * q_scale
        self.q_type, self.softmax_scale = q_type, softmax_scale
        if q_type == "e4m3":
            self.q_codes = e4m3_encode(q.clip(-448, 448)).astype(np.uint8)
            self.q = E4M3_TABLE[self.q_codes]
        else:
            import torch
            self.q_bf16 = torch.from_numpy(q).to(torch.bfloat16)
            self.q = self.q_bf16.double().numpy()

    def selection(self, most=16, empty=()):
        """The recent block and random ones before it, ascending, -1 behind; rows (b, t, g) in
        `empty` select nothing."""
        sel = np.full((self.B, self.T, self.G, 16), -1, np.int32)
        for b in range(self.B):
            for t in range(self.T):
                r = (int(self.lens[b]) - self.T + t) // 128
                if self.lens[b] < self.T:
                    continue
                for g in range(self.G):
                    if (b, t, g) in empty:
                        continue
                    k = min(most, r + 1)
                    got = sorted([r] + self.rng.choice(r, k - 1, replace=False).tolist()) if k > 1 else [r]
                    sel[b, t, g, :k] = got
        return sel

    def cache_arrays(self):
        return self.k, self.ks, self.v, self.vs

    def oracle(self, **kw):
        scale = self.softmax_scale or 1.0 / np.sqrt(128.0)
        with np.errstate(invalid="ignore"):
            return OF8.attention(self.q, self.cache_arrays(), self.table, self.lens, self.Hg, softmax_scale=scale, **kw)

    # ---- device side
    def upload(self):
        import torch
        import block_sparse_attention_indexer_gb300 as msa
        dev = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()  # noqa: E731
        self.cfg = msa.Config(num_kv_groups=self.G, heads_per_group=self.Hg, softmax_scale=self.softmax_scale)
        self.cache = msa.Fp8Cache.from_tensors(dev(self.k), dev(self.ks), dev(self.v), dev(self.vs))
        self.batch = msa.Batch(dev(self.table), dev(self.lens), q_len=self.T)
        self.dq = dev(self.q_codes) if self.q_type == "e4m3" else self.q_bf16.cuda()
        return self

    def buffers(self):
        import torch
        out = torch.full((self.B, self.T, self.G * self.Hg, 128), 7.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((self.B, self.T, self.G * self.Hg), 7.0, device="cuda")
        return out, lse

    def run(self, selection=None, weight_in=None, weights=False, decay=1.0, ws=None):
        """(out, lse, weight or None, error word) of one call, as numpy float64."""
        import torch
        import block_sparse_attention_indexer_gb300 as msa
        out, lse = self.buffers()
        sel = None if selection is None else torch.from_numpy(selection).cuda()
        w_in = None if weight_in is None else torch.from_numpy(weight_in).cuda()
        w_out = torch.full((self.B, self.max_blocks), 7.0, device="cuda") if weights else None
        if ws is None:
            ws = msa.alloc_workspace(msa.MSA_OP_FP8_ATTN_WEIGHTS if weights else msa.MSA_OP_FP8_ATTN, self.cfg, self.batch)
        msa.msa_fp8_attn(self.cfg, self.cache, self.batch, self.dq, out, lse, ws, selection=sel, weight_in=w_in,
                         weight_out=w_out, weight_decay=decay)
        torch.cuda.synchronize()
        return (out.double().cpu().numpy(), lse.double().cpu().numpy(),
                None if w_out is None else w_out.double().cpu().numpy(), msa.msa_read_device_error(ws))


def attention_bounds(case, ref):
    """(out, lse, weight) tolerances from the arithmetic of a float32 kernel with fp16
    probabilities, element by element:
      * a logit: 128 products accumulated in float32 in any order, 128 * 2^-24 of sum |q k| (and
        the products with the scale and the reference's subtraction, 4 * 2^-24 of its size); a bf16
        query element may be off by 2^-21 of its row's largest;
      * a probability: the logit's error twice (in it and in the sum), 2^-11 for its rounding to
        fp16, 2^-20 for exp2, the sums and the merges; below fp16's normal range 2^-24 of the largest
        probability, for each key;
      * the output is rounded to bf16 (half a step: 2^-8), lse and weights to float32.
    """
    scale = case.softmax_scale or 1.0 / np.sqrt(128.0)
    dz = scale * ref["logit"] * (128 + 4) * 2.0 ** -24
    if case.q_type != "e4m3":
        dz = dz + scale * 2.0 ** -21 * np.abs(case.q).max(-1) * ref["k_abs"]
    rel = 2 * dz + 2.0 ** -20
    flush = (ref["keys"] * 2.0 ** -24 * ref["p_max"])[..., None] * ref["v_abs"]
    out = 2.0 ** -8 * np.abs(ref["out"]) + (rel + 2.0 ** -11)[..., None] * ref["spread"] + flush + 1e-30
    lse = dz + 2.0 ** -20 + 2.0 ** -22 * np.abs(np.where(np.isfinite(ref["lse"]), ref["lse"], 0.0))
    # a row's probabilities are off by rel each; the row's share of a block is at most 1
    T, H = case.T, case.G * case.Hg
    weight = np.abs(ref["weight"]) * 2.0 ** -22 + rel.max(axis=(1, 2))[:, None] * np.maximum(ref["weight"], 2.0 ** -20) \
        + T * H * 2.0 ** -41
    return out, lse, weight


def assert_attention(case, got, ref, weights=False):
    out, lse, w, err = got
    b_out, b_lse, b_w = attention_bounds(case, ref)
    assert err == 0, err
    _close("out", out, ref["out"], b_out)
    _close("lse", lse, ref["lse"], b_lse)
    if weights:
        _close("weight", w, ref["weight"], b_w)


def _close(name, got, want, bound):
    special = ~np.isfinite(want)
    assert np.array_equal(np.isnan(got), np.isnan(want)), (name, "NaN at other places", np.argwhere(
        np.isnan(got) != np.isnan(want))[:4])
    assert np.array_equal(got[special & ~np.isnan(want)], want[special & ~np.isnan(want)]), (name, "infinities")
    err = np.where(special, 0.0, np.abs(np.where(special, 0, got) - np.where(special, 0, want)))
    bad = err > np.where(special, 0.0, bound)
    assert not bad.any(), (name, int(bad.sum()), np.argwhere(bad)[:4].tolist(),
                           float((err / np.maximum(np.where(special, 1, bound), 1e-300)).max()))


def run_repeated(c, n, selection=None):
    """c.run with c's sequences n times over, on the same pages (so many units that a CTA or team has all pages of
    one): the results of the first copy and of the last."""
    queries = "q_codes" if c.q_type == "e4m3" else "q_bf16"
    was = {name: getattr(c, name) for name in ("B", "table", "lens", queries)}
    c.B, c.table, c.lens = n * c.B, np.tile(c.table, (n, 1)), np.tile(c.lens, n)
    setattr(c, queries, was[queries].repeat(n, 1, 1, 1) if queries == "q_bf16" else np.tile(was[queries], (n, 1, 1, 1)))
    out, lse, w, err = c.upload().run(selection=None if selection is None else np.tile(selection, (n, 1, 1, 1)), weights=True)
    for name, value in was.items():
        setattr(c, name, value)
    c.upload()
    return [(out[s], lse[s], w[s], err) for s in (slice(0, c.B), slice(-c.B, None))]
