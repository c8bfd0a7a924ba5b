"""GPU: msa_fp8_attn against the float64 oracle, with tolerances from the arithmetic
(fp8_util.attention_bounds).  Codes that no row may use are NaN in every case."""
import numpy as np
import pytest

from fp8_util import Case, assert_attention
from gpu_util import need_gpu

pytestmark = pytest.mark.gpu

# (lens, T, G, Hg): from one token to several pages, around page ends, padding rows, rows per
# (sequence, group) from 1 to more than one tile of 128 and more than two
SHAPES = [
    ([1], 1, 1, 1), ([127, 128, 129, 0, 2], 1, 4, 8), ([1000, 64, 257], 1, 2, 5), ([5000], 1, 1, 8),
    ([300, 7, 0, 129], 2, 2, 8), ([256, 20], 16, 1, 1), ([130, 3], 3, 4, 5),
    ([300, 17, 0], 17, 2, 1), ([700, 130], 8, 2, 8), ([1500, 11, 600], 11, 1, 8), ([260, 128], 128, 1, 1),
    ([129, 140], 129, 2, 1), ([500], 40, 2, 7), ([400, 300], 300, 1, 1), ([300], 100, 1, 4), ([390], 129, 1, 8),
    ([2100], 70, 1, 8), ([300, 500], 17, 8, 8), ([20000], 1, 1, 3), ([9000], 20, 1, 1), ([1300, 900], 700, 1, 1),
]


@pytest.mark.parametrize("q_type", ["e4m3", "bf16"])
@pytest.mark.parametrize("lens,T,G,Hg", SHAPES)
def test_dense_matches_the_oracle(lens, T, G, Hg, q_type):
    need_gpu()
    c = Case(100 + T + len(lens), lens, T, G, Hg, q_type).upload()
    w_in = c.rng.random((c.B, c.max_blocks)).astype(np.float32)
    ref = c.oracle(weight_in=w_in, decay=0.5)
    assert_attention(c, c.run(weight_in=w_in, weights=True, decay=0.5), ref, weights=True)


@pytest.mark.parametrize("q_type", ["e4m3", "bf16"])
@pytest.mark.parametrize("lens,T,G,Hg", [
    ([1], 1, 1, 1), ([5000, 129, 0, 2100], 1, 4, 8), ([3000, 40], 5, 2, 5), ([2500], 70, 1, 3), ([4000, 200], 3, 8, 8),
    ([900, 3000], 40, 4, 2)])
def test_sparse_matches_the_oracle(lens, T, G, Hg, q_type):
    need_gpu()
    c = Case(300 + T, lens, T, G, Hg, q_type).upload()
    sel = c.selection(empty={(0, T - 1, G - 1)} if len(lens) > 1 else ())
    w_in = c.rng.random((c.B, c.max_blocks)).astype(np.float32)
    ref = c.oracle(selection=sel, weight_in=w_in, decay=0.25)
    assert_attention(c, c.run(selection=sel, weight_in=w_in, weights=True, decay=0.25), ref, weights=True)


@pytest.mark.parametrize("B,T,G,Hg,most", [(33, 1, 2, 4, 400), (200, 1, 1, 8, 300), (2048, 1, 1, 1, 200), (70, 5, 1, 8, 200),
                                           (40, 2, 1, 3, 500), (600, 17, 1, 1, 150), (1100, 17, 1, 1, 60)])
def test_many_sequences(B, T, G, Hg, most):
    need_gpu()
    rng = np.random.default_rng(B)
    lens = rng.integers(T, most, B)
    lens[rng.integers(0, B, B // 8)] = 0
    c = Case(400 + B, lens.tolist(), T, G, Hg).upload()
    assert_attention(c, c.run(weights=True), c.oracle(), weights=True)


@pytest.mark.parametrize("B,T,G,Hg,q_type", [(40, 17, 4, 8, "e4m3"), (39, 17, 4, 8, "bf16"), (50, 9, 4, 4, "bf16"), (20, 150, 8, 1, "e4m3")])
def test_long_units_cut_beside_short_whole_ones(B, T, G, Hg, q_type):
    # the split of the work leaves short units to one CTA each: one and two tiles of rows, a row of long
    # sequences between short ones, empty sequences at cuts
    need_gpu()
    rng = np.random.default_rng(B)
    lens = rng.integers(T, 600, B)
    lens[[0, B // 2, B - 1]] = [4000, 3001, 4097]
    lens[rng.integers(1, B // 2, 3)] = 0
    c = Case(500 + B, lens.tolist(), T, G, Hg, q_type).upload()
    w_in = c.rng.random((B, c.max_blocks)).astype(np.float32)
    assert_attention(c, c.run(weight_in=w_in, weights=True, decay=0.5), c.oracle(weight_in=w_in, decay=0.5), weights=True)


@pytest.mark.parametrize("B,T,Hg", [(225, 1, 2), (75, 9, 1)])
def test_few_rows_of_long_sequences_beside_short_ones(B, T, Hg):
    need_gpu()
    rng = np.random.default_rng(B)
    lens = rng.integers(T, 400, B)
    lens[[0, B // 3, B - 1]] = [5000, 4737, 4224]
    lens[rng.integers(1, B // 3, 3)] = 0
    c = Case(550 + B, lens.tolist(), T, 4, Hg, "bf16").upload()
    assert_attention(c, c.run(weights=True), c.oracle(), weights=True)
    sel = c.selection()
    assert_attention(c, c.run(selection=sel, weights=True), c.oracle(selection=sel), weights=True)


def test_tables_far_wider_than_the_sequences():
    need_gpu()
    for T in (1, 30):
        c = Case(31 + T, [300, 0, 129, 64], T, 1, 2, max_blocks=5000).upload()
        w_in = c.rng.random((4, 5000)).astype(np.float32)
        ref = c.oracle(weight_in=w_in, decay=1.0)
        assert_attention(c, c.run(weight_in=w_in, weights=True), ref, weights=True)
        if T == 1:
            sel = c.selection()
            ref = c.oracle(selection=sel, weight_in=w_in, decay=0.0)
            assert_attention(c, c.run(selection=sel, weight_in=w_in, weights=True, decay=0.0), ref, weights=True)


@pytest.mark.parametrize("T,Hg", [(1, 8), (2, 8), (40, 4)])
def test_an_infinite_or_nan_query_makes_its_row_nan(T, Hg):
    need_gpu()
    c = Case(32, [300, 200], T, 1, Hg, "bf16").upload()
    want = c.run()
    for h, value in ((0, float("inf")), (Hg - 1, float("-inf")), (1, float("nan"))):
        c.dq[1, T - 1, h, 77] = value
    out, lse, _, err = c.run()
    hit = np.zeros(lse.shape, bool)
    hit[1, T - 1, [0, Hg - 1, 1]] = True
    assert err == 0 and np.isnan(out[hit]).all() and np.isnan(lse[hit]).all()
    assert np.array_equal(out[~hit], want[0][~hit]) and np.array_equal(lse[~hit], want[1][~hit])


def test_a_selection_in_any_order_with_gaps():
    need_gpu()
    c = Case(17, [3000, 700], 2, 2, 4).upload()
    sel = c.selection(most=9)
    sel = c.rng.permuted(sel, axis=-1)
    sel[0, 1, 0, 3] = 9999  # beyond the table: no block of this row
    ref = c.oracle(selection=sel)
    assert_attention(c, c.run(selection=sel, weights=True), ref, weights=True)


@pytest.mark.parametrize("T,Hg", [(1, 8), (4, 8), (40, 4), (200, 2)])
def test_scales_over_their_whole_range(T, Hg):
    need_gpu()
    # K scales that keep the logits moderate, V scales over all of 2^-40..2^40
    c = Case(21, [900, 333], T, 1, Hg, scales=(87, 168))
    c.ks[:] = np.where(c.ks <= 167, c.rng.integers(115, 125, c.ks.shape), c.ks).astype(np.uint8)
    c.upload()
    assert_attention(c, c.run(weights=True), c.oracle(), weights=True)


@pytest.mark.parametrize("T,Hg", [(1, 8), (4, 8), (40, 4), (200, 2)])
def test_sharp_and_flat_softmax(T, Hg):
    need_gpu()
    for scale in (4.0, 1e-6):
        c = Case(22, [1200, 260], T, 1, Hg, softmax_scale=scale).upload()
        assert_attention(c, c.run(weights=True), c.oracle(), weights=True)


@pytest.mark.parametrize("T,Hg", [(1, 8), (4, 8), (40, 4), (200, 2)])
def test_bf16_queries_of_any_size(T, Hg):
    need_gpu()
    for size in (1e-30, 1e-4, 1e6):
        c = Case(23, [600, 260], T, 1, Hg, "bf16", q_scale=size, softmax_scale=0.05 / size if size > 1e-20 else 0.0).upload()
        assert_attention(c, c.run(), c.oracle())


@pytest.mark.parametrize("T,Hg", [(2, 8), (4, 8), (40, 4), (200, 2)])
@pytest.mark.parametrize("what", ["k", "v"])
def test_nan_reaches_only_rows_that_see_it(T, Hg, what):
    need_gpu()
    L = 390 + T // 2
    c = Case(24, [L, 450], T, 1, Hg)
    at = L - T + T // 2                       # seen by the later half of the tokens
    getattr(c, what)[c.table[0, at // 128], 0, at % 128, 5:9] = 0x7F
    c.upload()
    got, ref = c.run(weights=True), c.oracle()
    assert np.isnan(ref["out"][0, T // 2:]).any() and not np.isnan(ref["out"][0, :T // 2]).any()
    with np.errstate(invalid="ignore"):
        out, lse, _, err = got
        assert err == 0
        for b in range(2):
            for t in range(T):
                assert np.array_equal(np.isnan(out[b, t]), np.isnan(ref["out"][b, t])), (b, t)
        fine = ~np.isnan(ref["out"])
        assert (np.abs(out - ref["out"])[fine] <= 2.0 ** -7 * (1 + np.abs(ref["out"][fine]))).all()
        assert np.array_equal(np.isnan(lse), np.isnan(ref["lse"]))


def test_an_older_nan_reaches_every_row():
    need_gpu()
    for T, Hg in ((1, 8), (40, 4), (200, 2)):
        c = Case(25, [500], T, 1, Hg)
        c.v[c.table[0, 0], 0, 3, 100] = 0x7F
        c.upload()
        out, lse, _, err = c.run()
        assert err == 0 and np.isnan(out[..., 100]).all() and not np.isnan(np.delete(out, 100, -1)).any()
        assert np.isfinite(lse).all()


@pytest.mark.parametrize("T,Hg", [(1, 8), (8, 8), (150, 4)])
@pytest.mark.parametrize("sparse", [False, True])
def test_bad_pages_scales_and_lengths(T, Hg, sparse):
    need_gpu()
    import block_sparse_attention_indexer_gb300 as msa
    c = Case(26, [900, 800, 700, 600, T], T, 2, Hg)
    c.table[0, 2] = -5
    c.table[1, 1] = len(c.k)
    c.ks[c.table[2, 0], 1] = 86
    c.vs[c.table[3, 1], 0] = 168
    c.table[4] = 1 << 30                    # every page of the sequence: empty rows
    sel = c.selection() if sparse else None
    c.upload()
    ref = c.oracle(selection=sel)
    got = c.run(selection=sel, weights=True)
    assert got[3] == msa.MSA_DEVERR_BAD_PAGE | msa.MSA_DEVERR_BAD_SCALE
    assert not got[0][4].any() and np.isneginf(got[1][4]).all()
    assert_attention(c, (*got[:3], 0), ref, weights=True)
    c.lens[0], c.lens[1] = T - 1 or -1, c.max_blocks * 128 + 1
    c.upload()
    got = c.run(selection=sel, weights=True)
    assert got[3] & msa.MSA_DEVERR_BAD_SEQLEN
    assert_attention(c, (*got[:3], 0), c.oracle(selection=sel), weights=True)


@pytest.mark.parametrize("T,G,Hg,q_type", [(1, 4, 8, "e4m3"), (1, 2, 3, "bf16"), (9, 2, 4, "bf16"), (70, 2, 4, "e4m3")])
def test_strided_queries_equal_contiguous_ones(T, G, Hg, q_type):
    need_gpu()
    import torch
    c = Case(27, [300, 150], T, G, Hg, q_type).upload()
    want = c.run()
    H = G * Hg
    wide = torch.full((c.B, T, H + 2 * G, 128), 0x7F if q_type == "e4m3" else float("nan"), dtype=c.dq.dtype, device="cuda")
    wide[:, :, :H] = c.dq
    c.dq = wide[:, :, :H]
    got = c.run()
    assert np.array_equal(got[0], want[0]) and np.array_equal(got[1], want[1])


def test_lse_and_weights_are_optional_and_change_nothing():
    need_gpu()
    import torch
    import block_sparse_attention_indexer_gb300 as msa
    for T, Hg in ((1, 8), (9, 8), (150, 2)):
        c = Case(28, [700, 200], T, 2, Hg).upload()
        out, lse, w, err = c.run(weights=True)
        bare, _ = c.buffers()
        ws = msa.alloc_workspace(msa.MSA_OP_FP8_ATTN, c.cfg, c.batch)
        msa.msa_fp8_attn(c.cfg, c.cache, c.batch, c.dq, bare, None, ws)
        assert err == 0 and np.array_equal(bare.double().cpu().numpy(), out)
        # in place: decay 1, a second call doubles what the first collected
        wb = torch.zeros(c.B, c.max_blocks, device="cuda")
        ws = msa.alloc_workspace(msa.MSA_OP_FP8_ATTN_WEIGHTS, c.cfg, c.batch)
        for _ in range(2):
            msa.msa_fp8_attn(c.cfg, c.cache, c.batch, c.dq, bare, None, ws, weight_in=wb, weight_out=wb)
        assert np.array_equal(wb.double().cpu().numpy(), 2 * w)


@pytest.mark.parametrize("T,Hg,sparse", [(1, 8, False), (1, 8, True), (8, 8, False), (150, 4, False), (30, 4, True)])
def test_repeated_overlapping_and_captured_calls_give_the_same_bits(T, Hg, sparse):
    need_gpu()
    import torch
    import block_sparse_attention_indexer_gb300 as msa
    c = Case(29, [2000, 900, 0, 300], T, 2, Hg).upload()
    d = Case(30, [1500, 1300, 260, 0], T, 2, Hg).upload()
    sel = {x: torch.from_numpy(x.selection()).cuda() if sparse else None for x in (c, d)}
    want = {x: x.run(selection=None if sel[x] is None else sel[x].cpu().numpy(), weights=True) for x in (c, d)}
    streams = {c: torch.cuda.Stream(), d: torch.cuda.Stream()}
    res = {}
    for x in (c, d):
        ws = msa.alloc_workspace(msa.MSA_OP_FP8_ATTN_WEIGHTS, x.cfg, x.batch)
        out, lse = x.buffers()
        res[x] = (out, lse, torch.zeros(x.B, x.max_blocks, device="cuda"), ws)
    torch.cuda.synchronize()

    def call(x, stream=None):
        out, lse, w, ws = res[x]
        msa.msa_fp8_attn(x.cfg, x.cache, x.batch, x.dq, out, lse, ws, selection=sel[x], weight_out=w, stream=stream)

    def check():
        torch.cuda.synchronize()
        for x in (c, d):
            for got, ref in zip(res[x], want[x][:3]):
                assert np.array_equal(got.double().cpu().numpy(), ref)
            for t in res[x][:3]:
                t.fill_(3.0)
        torch.cuda.synchronize()

    for _ in range(5):                      # two calls in flight at once, a workspace each
        for x in (c, d):
            call(x, streams[x])
    check()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(c)
        call(d)
    for _ in range(3):
        graph.replay()
    check()
