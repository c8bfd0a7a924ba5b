"""GPU: the block weights that msa_fp8_attn collects from rows with a NaN (in the query, a key or a value), dense
and over selections of few and of many entries a sequence, against the float64 oracle."""
import numpy as np
import pytest

from fp8_util import Case, _close, attention_bounds, run_repeated
from gpu_util import need_gpu

pytestmark = pytest.mark.gpu

# rows of a group in both kernels' forms; for selections, up to 2,048 entries a sequence and more
FORMS = [(1, 8), (2, 8), (40, 3), (100, 3)]


def _compare(c, sel):
    """out, lse and weights, NaN for NaN."""
    with np.errstate(invalid="ignore"):
        ref = c.oracle(selection=sel)
        got = c.run(selection=sel, weights=True)
        more = run_repeated(c, max(1, 240 // (c.B * c.G * (min(c.T, 20) if sel is not None else 1))), sel)
        ok = {n: np.where(np.isnan(x), 0.0, x) if x.dtype == np.float64 else x for n, x in ref.items()}
        bounds = attention_bounds(c, ok)
        for part in (got, *more):
            assert part[3] == 0
            for name, a, b, bound in zip(("out", "lse", "weight"), part, (ref["out"], ref["lse"], ref["weight"]), bounds):
                _close(name, a, b, bound)
    return ref["weight"]


def _selection(c, sparse, with_block, rows):
    """A selection in which the given rows (b, t, g) have block `with_block` and no other row has."""
    if not sparse:
        return None
    sel = c.selection(most=9)
    sel[sel == with_block] = -1
    for r in rows:
        sel[r][9] = with_block
    return sel


@pytest.mark.parametrize("sparse", [False, True])
@pytest.mark.parametrize("T,Hg", FORMS)
@pytest.mark.parametrize("what", ["q", "k", "v"])
def test_weights_of_rows_with_a_nan(what, T, Hg, sparse):
    need_gpu()
    if T == 100 and not sparse:
        T = 150                                  # (two tiles)
    c = Case(800 + T, [1700, 900, 300], T, 2, Hg, "bf16")
    page = c.table[0, 2]
    if what != "q":
        getattr(c, what)[page, 1, 77, 5] = 0x7F
    sel = _selection(c, sparse, 2, [(0, T - 1, 1), (0, 0, 1)])
    if what == "q":
        c.q_bf16[0, T - 1, 2 * Hg - 1, 3] = float("nan")
        c.q = c.q_bf16.double().numpy()
    c.upload()
    w = _compare(c, sel)
    assert np.isnan(w[0]).any() == (what != "v") and np.isfinite(w[1:]).all()


@pytest.mark.parametrize("sparse", [False, True])
@pytest.mark.parametrize("T,Hg", FORMS)
def test_blocks_that_underflow_collect_nan_too(T, Hg, sparse):
    need_gpu()
    # a NaN key in block 1; block 3 is e^-256 of the sum, which float32 does not hold
    c = Case(810 + T, [700, 500], T, 1, Hg, softmax_scale=4.0)
    c.q_codes[:] = 0
    c.q_codes[..., 0] = 0x38                     # 1
    c.q[:] = 0.0
    c.q[..., 0] = 1.0
    for n in range(6):
        p = c.table[0, n]
        c.ks[p] = 127
        real = c.k[p, 0] != 0x7F
        c.k[p, 0] = np.where(real, 0, c.k[p, 0])
        c.k[p, 0, :, 0] = np.where(real[:, 0], 0xE8 if n == 3 else 0, c.k[p, 0, :, 0])  # -64 in block 3
    c.k[c.table[0, 1], 0, 5, 0] = 0x7F
    sel = None
    if sparse:
        sel = np.full((2, T, 1, 16), -1, np.int32)
        sel[:, :, :, :3] = [0, 1, 3]
    c.upload()
    w = _compare(c, sel)
    assert np.isnan(w[0, [0, 1, 3]]).all() and np.isfinite(w[1]).all()
    # ... and not where its scale is out of range
    import block_sparse_attention_indexer_gb300 as msa
    c.ks[c.table[0, 3]] = 200
    want = c.oracle(selection=sel)["weight"]
    assert want[0, 3] == 0
    for n in (1, 200 // (min(T, 20) if sparse else 1)):
        for _, _, part, err in run_repeated(c, n, sel):
            assert err == msa.MSA_DEVERR_BAD_SCALE
            assert np.array_equal(np.isnan(part), np.isnan(want)) and part[0, 3] == 0


@pytest.mark.parametrize("T,Hg", [(3, 2), (4, 4), (40, 3), (100, 3)])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
def test_a_nan_query_that_sees_only_a_skipped_page_is_an_empty_row(value, T, Hg):
    need_gpu()
    import block_sparse_attention_indexer_gb300 as msa
    c = Case(820 + T, [129 + T // 2], T, 1, Hg, "bf16")  # the first half of the tokens sees page 0 alone
    c.table[0, 0] = -1
    c.q_bf16[0, 0, 0, 5] = value
    c.q_bf16[0, T - 1, Hg - 1, 5] = value
    c.q = c.q_bf16.double().numpy()
    c.upload()
    out, lse, w, err = c.run(weights=True)
    assert err == msa.MSA_DEVERR_BAD_PAGE
    assert not out[0, 0].any() and np.isneginf(lse[0, 0]).all()
    assert np.isnan(out[0, T - 1, Hg - 1]).all() and np.isnan(lse[0, T - 1, Hg - 1]) and np.isnan(w[0, 1]) and w[0, 0] == 0
    hit = np.zeros((T, Hg), bool)
    hit[T - 1, Hg - 1] = True
    assert np.isfinite(out[0][~hit]).all()
