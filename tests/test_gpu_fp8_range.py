"""GPU: msa_fp8_attn where the probabilities or the V scales of one row are far apart, against the float64
oracle.  The output's allowance here follows from one rule of the kernels: a key's probability is held in fp16
in units in which the probabilities so far, at the scale of its page, sum to 2^8 at least (2^4 in the form with
128-row tiles; 2^6 where all pages have one V scale).  Below fp16's normal range it is then off by 2^-25 / 2^8 of
that sum, so that all keys of a row together move the output by keys * 2^-33 (2^-29, 2^-31) of the largest value in
its dim, whatever the other pages' scales are."""
import numpy as np
import pytest

from fp8_util import Case, _close, attention_bounds, run_repeated
from gpu_util import need_gpu

pytestmark = pytest.mark.gpu

# rows per (sequence, group): both forms of the streaming kernel, one and two tiles of the other
FORMS = [(1, 8), (2, 8), (40, 3), (100, 3)]


def _bounds(case, ref, one_scale=False):
    _, lse, weight = attention_bounds(case, ref)
    dz = lse - 2.0 ** -20 - 2.0 ** -22 * np.abs(np.where(np.isfinite(ref["lse"]), ref["lse"], 0.0))
    rel = 2 * dz + 2.0 ** -20 + 2.0 ** -11
    tiles = case.T * case.Hg > 16 and not ref.get("sparse")
    flush = 2.0 ** -33 if not tiles else 2.0 ** -31 if one_scale else 2.0 ** -29
    out = 2.0 ** -8 * np.abs(ref["out"]) + rel[..., None] * ref["spread"] \
        + flush * ref["keys"][..., None] * ref["v_abs"] + 1e-30
    return out, lse, weight


def _check(case, got, ref, one_scale=False):
    out, lse, w, err = got
    b_out, b_lse, b_w = _bounds(case, ref, one_scale)
    assert err == 0, err
    _close("lse", lse, ref["lse"], b_lse)
    _close("out", out, ref["out"], b_out)
    _close("weight", w, ref["weight"], b_w)


def _write(c, k, v):
    """The rows k, v (lists of [L, G, 128], one of each sequence) through msa_fp8_append; the pools read back."""
    import torch
    import block_sparse_attention_indexer_gb300 as msa
    c.upload()
    for b, n in enumerate(c.lens):
        batch = msa.Batch(c.batch.block_table[b:b + 1], c.batch.seq_lens[b:b + 1], q_len=int(n))
        ws = msa.alloc_workspace(msa.MSA_OP_FP8_APPEND, c.cfg, batch)
        rows = [torch.from_numpy(x[b][None]).float().cuda() for x in (k, v)]
        msa.msa_fp8_append(c.cfg, c.cache, batch, *rows, ws)
        assert msa.msa_read_device_error(ws) == 0
    c.k, c.ks, c.v, c.vs = (t.cpu().numpy() for t in c.cache.tensors())


def _check_repeated(c, n, selection=None, one_scale=False):
    """The call, and one of c's sequences n times over: units cut between CTAs and whole ones."""
    ref = c.oracle(selection=selection) | {"sparse": selection is not None}
    c.upload()
    _check(c, c.run(selection=selection, weights=True), ref, one_scale)
    for part in run_repeated(c, n, selection):
        _check(c, part, ref, one_scale)


@pytest.mark.parametrize("size", [1e5, 1e8, float("inf")])
@pytest.mark.parametrize("T,Hg", FORMS)
def test_one_large_value_leaves_the_other_dims_of_v(T, Hg, size):
    need_gpu()
    c = Case(700 + T, [900, 500, 1300], T, 2, Hg)
    k, v = ([c.rng.normal(0, 1, (n, 2, 128)) for n in c.lens] for _ in range(2))
    v[0][200, 0, 0] = v[0][700, 1, 5] = size     # between other pages
    v[1][3, :, 7] = -size                        # in the first page
    v[2][1299, 0, 9] = size                      # in the last
    _write(c, k, v)
    _check_repeated(c, 80)
    sel = c.selection(most=7)
    sel[0, :, :, 7] = 1                          # (so that the large values are among them; twice counts twice)
    _check_repeated(c, 80 // min(T, 8), sel)


@pytest.mark.parametrize("first", [False, True])
@pytest.mark.parametrize("T,Hg", FORMS)
def test_v_scales_at_both_ends_with_empty_dims(T, Hg, first):
    need_gpu()
    # one page at 2^40 with zeros in half of its dims, the others at 2^-40: 80 powers of two in one row's sum
    c = Case(710 + T, [1000, 700], T, 2, Hg)
    for b in range(2):
        c.vs[c.table[b][c.table[b] >= 0]] = 87
        page = c.table[b, 0 if first else 3]
        c.vs[page] = 167
        c.v[page, :, :, :64] = 0
    _check_repeated(c, 120)
    sel = c.selection(most=7)
    sel[:, :, :, 7] = 0 if first else 3
    _check_repeated(c, 120 // min(T, 8), sel)


@pytest.mark.parametrize("gap", [18, 22, 25, 28, 34])
@pytest.mark.parametrize("T,Hg,q_type", [(1, 8, "e4m3"), (2, 8, "bf16"), (20, 1, "e4m3"), (100, 3, "bf16")])
def test_many_small_probabilities_beside_one_large(T, Hg, q_type, gap):
    need_gpu()
    # a first key `gap` powers of two above all others, its values zero: the output is what the others add
    c = Case(720 + T, [1500], T, 8, Hg, q_type, softmax_scale=float(np.float32(gap * np.log(2) / 64)))
    pages = c.table[0]
    c.ks[pages] = c.vs[pages] = 127
    c.k[pages] = 0
    c.k[pages[0], :, 0, 0] = 0x68                # 64
    c.v[pages] &= 0x7F
    c.v[pages[0], :, 0] = 0
    c.q[:] = 0.0
    c.q[..., 0] = 1.0
    if q_type == "e4m3":
        c.q_codes[:] = 0
        c.q_codes[..., 0] = 0x38
    else:
        c.q_bf16.zero_()
        c.q_bf16[..., 0] = 1.0
    _check_repeated(c, 70, one_scale=True)


@pytest.mark.parametrize("T,Hg", FORMS)
def test_zero_keys_under_the_largest_scale(T, Hg):
    need_gpu()
    # every logit is 0, whatever the factors before it
    c = Case(750 + T, [600, 260], T, 1, Hg, "bf16", q_scale=1e36)
    c.k[c.k != 0x7F] = 0
    c.ks[c.ks != 255] = 167
    c.upload()
    _check(c, c.run(weights=True), c.oracle())


@pytest.mark.parametrize("T,Hg", FORMS)
@pytest.mark.parametrize("size,scales", [(4e37, (99, 104)), (3e-37, (139, 144))])
def test_bf16_queries_at_the_ends_of_their_range(T, Hg, size, scales):
    need_gpu()
    a = 2.0 ** (121.5 - np.mean(scales))         # K's values times this are those of the other tests
    c = Case(760 + T, [600, 260], T, 1, Hg, "bf16", scales=scales, q_scale=size, softmax_scale=float(np.float32(0.05 / size * a)))
    c.upload()
    _check(c, c.run(weights=True), c.oracle())


@pytest.mark.parametrize("byte", [87, 107, 147, 167])
@pytest.mark.parametrize("T,Hg", FORMS)
def test_lse_of_few_keys_under_any_v_scale(T, Hg, byte):
    need_gpu()
    # rows of 1 to some keys with logits near 0: the V scale must not show in the sum's logarithm
    c = Case(770 + T, [T, T + 2, T + 7, T + 40], T, 4, Hg, "bf16", softmax_scale=1e-6)
    c.vs[c.vs <= 167] = byte
    c.upload()
    _check(c, c.run(weights=True), c.oracle())
