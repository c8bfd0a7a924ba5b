"""GPU: msa_evict_blocks against the oracle, value for value."""
import numpy as np
import pytest

from gpu_util import need_gpu
from oracle import fp8 as OF8

pytestmark = pytest.mark.gpu


def _run(table, lens, weight, budget, first, last, in_place=False):
    import torch
    import block_sparse_attention_indexer_gb300 as msa
    B, MB = table.shape
    t, n, w = (torch.from_numpy(x.copy()).cuda() for x in (table, lens, weight))
    batch = msa.Batch(t, n)
    to, no, wo = (t, n, w) if in_place else (torch.full_like(t, 77), torch.full_like(n, 77), torch.full_like(w, 77))
    freed, count = torch.full_like(t, 77), torch.full_like(n, 77)
    ws = msa.alloc_workspace(msa.MSA_OP_EVICT, msa.Config(), batch)
    msa.msa_evict_blocks(batch, w, budget, first, last, to, no, wo, freed, count, ws)
    torch.cuda.synchronize()
    return [x.cpu().numpy() for x in (to, no, wo, freed, count)], msa.msa_read_device_error(ws)


def _inputs(seed, B, MB, kind):
    rng = np.random.default_rng(seed)
    table = rng.permutation(B * MB).reshape(B, MB).astype(np.int32)
    lens = rng.integers(0, MB * 128 + 1, B).astype(np.int32)
    lens[0] = MB * 128
    if B > 2:
        lens[1], lens[2] = 0, 1
    w = {"ties": rng.integers(0, 3, (B, MB)), "equal": np.full((B, MB), 0.25), "spread": np.exp(rng.normal(0, 20, (B, MB))),
         "signed": rng.normal(0, 1, (B, MB)), "special": rng.choice([np.nan, -np.inf, np.inf, 0.0, -0.0, 1e-45, 1.0], (B, MB))
         }[kind].astype(np.float32)
    return table, lens, w


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("kind", ["ties", "equal", "spread", "signed", "special"])
@pytest.mark.parametrize("B,MB,budget,first,last", [
    (1, 1, 1, 0, 1), (3, 7, 3, 1, 2), (4, 129, 40, 1, 2), (5, 1000, 1000, 3, 5), (2, 1025, 512, 0, 1), (3, 9000, 4000, 4, 8),
    (2, 20000, 16500, 4, 8), (64, 33, 17, 16, 1)])
def test_evict_matches_the_oracle(B, MB, budget, first, last, kind, in_place):
    need_gpu()
    table, lens, w = _inputs(B * MB + budget, B, MB, kind)
    got, err = _run(table, lens, w, budget, first, last, in_place)
    assert err == 0
    for name, a, b in zip(("table", "lens", "weight", "freed", "count"), got, OF8.evict(table, lens, w, budget, first, last)):
        assert np.array_equal(a, b, equal_nan=(name == "weight")), name


def test_a_bad_length_is_flagged_and_the_row_stays():
    need_gpu()
    import block_sparse_attention_indexer_gb300 as msa
    table, lens, w = _inputs(4, 4, 50, "signed")
    lens[:] = [-3, 50 * 128 + 1, 3000, 6400]
    got, err = _run(table, lens, w, 10, 1, 1)
    assert err == msa.MSA_DEVERR_BAD_SEQLEN
    for a, b in zip(got, OF8.evict(table, lens, w, 10, 1, 1)):
        assert np.array_equal(a, b)
