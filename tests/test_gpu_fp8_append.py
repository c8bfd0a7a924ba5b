"""GPU: msa_fp8_append against the oracle, byte for byte."""
import numpy as np
import pytest

from fp8_util import Case
from gpu_util import need_gpu
from oracle import fp8 as OF8

pytestmark = pytest.mark.gpu


def _append(c, x, y, **kw):
    """x, y: device K and V rows.  Returns the four pools and the error word."""
    import torch
    import block_sparse_attention_indexer_gb300 as msa
    ws = msa.alloc_workspace(msa.MSA_OP_FP8_APPEND, c.cfg, c.batch)
    msa.msa_fp8_append(c.cfg, c.cache, c.batch, x, y, ws, **kw)
    torch.cuda.synchronize()
    return [t.cpu().numpy() for t in c.cache.tensors()], msa.msa_read_device_error(ws)


def _rows(c, dtype, dev=1.0, edges=True):
    """Fused rows [B, T, 2 G, 128] of the type, and their values."""
    import torch
    x = c.rng.normal(0, dev, (c.B, c.T, 2 * c.G, 128)) * np.exp(c.rng.normal(0, 1, (c.B, c.T, 2 * c.G, 1)))
    if edges and c.T > 1:
        x[0, 0, 0, :6] = [np.nan, -0.0, 0.0, 1e-30, -1e-30, 1e-9]
    t = torch.from_numpy(x).to(dtype)
    return t.cuda(), t.double().numpy()


def _check(c, kv, x, **kw):
    G = c.G
    got, err = _append(c, kv[:, :, :G], kv[:, :, G:], **kw)
    assert err == 0
    k, ks = OF8.append(c.k, c.ks, x[:, :, :G], c.table, c.lens)
    v, vs = OF8.append(c.v, c.vs, x[:, :, G:], c.table, c.lens)
    for name, a, b in (("k_scale", got[1], ks), ("v_scale", got[3], vs), ("k", got[0], k), ("v", got[2], v)):
        assert np.array_equal(a, b), (name, np.argwhere(a != b)[:4])


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("lens,T,G", [
    ([1], 1, 1), ([128, 129, 5, 0, 300], 1, 4), ([130, 128, 257, 0, 4], 3, 2), ([300], 300, 1), ([301, 700], 257, 2),
    ([1000, 129, 256], 129, 8), ([128, 256], 128, 3), ([1025], 1, 8)])
def test_append_matches_the_oracle(lens, T, G, dtype):
    need_gpu()
    import torch
    c = Case(11 + T, lens, T, G, 2).upload()
    kv, x = _rows(c, getattr(torch, dtype))
    _check(c, kv, x)


def test_scale_grows_and_older_rows_are_encoded_again():
    need_gpu()
    import torch
    c = Case(5, [100, 200, 77], 2, 2, 1, scales=(112, 118)).upload()   # old scales far below what the new rows need
    kv, x = _rows(c, torch.float32, dev=4.0)
    _check(c, kv, x)


@pytest.mark.parametrize("size", [0.0, 1e-20, 1e20, float("inf"), 448.0, float(np.nextafter(np.float32(448), np.float32(500)))])
def test_extreme_values(size):
    need_gpu()
    import torch
    c = Case(6, [140, 5], 3, 1, 1).upload()
    x = np.zeros((2, 3, 2, 128))
    x[:, 1, :, 3], x[:, 2, :, 5] = size, -size
    x[1, 0, 0, 0] = 1e-30
    t = torch.from_numpy(x).to(torch.float32)
    _check(c, t.cuda(), t.double().numpy())


def test_all_nan_rows():
    need_gpu()
    import torch
    c = Case(7, [140], 1, 1, 1).upload()
    t = torch.full((1, 1, 2, 128), float("nan"))
    _check(c, t.cuda(), t.double().numpy())


def test_contiguous_rows_and_repeated_writes():
    need_gpu()
    import torch
    c = Case(8, [140, 260], 5, 2, 1).upload()
    kv, x = _rows(c, torch.bfloat16)
    k, v = kv[:, :, :2].contiguous(), kv[:, :, 2:].contiguous()
    first, err = _append(c, k, v)
    again, err2 = _append(c, kv[:, :, :2], kv[:, :, 2:])
    assert err == err2 == 0 and all(np.array_equal(a, b) for a, b in zip(first, again))


def test_token_by_token_equals_the_oracle_step_by_step():
    """200 decode steps over one sequence, crossing pages."""
    need_gpu()
    import torch
    import block_sparse_attention_indexer_gb300 as msa
    c = Case(9, [200], 1, 2, 1).upload()
    x = c.rng.normal(0, 1, (1, 200, 4, 128)) * np.exp(c.rng.normal(0, 1, (1, 200, 1, 1)))
    t = torch.from_numpy(x).float().cuda()
    x = t.double().cpu().numpy()
    ws = msa.alloc_workspace(msa.MSA_OP_FP8_APPEND, c.cfg, c.batch)
    k, ks, v, vs = c.cache_arrays()
    for i in range(200):
        c.batch.seq_lens.fill_(i + 1)
        msa.msa_fp8_append(c.cfg, c.cache, c.batch, t[:, i:i + 1, :2], t[:, i:i + 1, 2:], ws)
        k, ks = OF8.append(k, ks, x[:, i:i + 1, :2], c.table, [i + 1])
        v, vs = OF8.append(v, vs, x[:, i:i + 1, 2:], c.table, [i + 1])
    torch.cuda.synchronize()
    assert msa.msa_read_device_error(ws) == 0
    for a, b in zip(c.cache.tensors(), (k, ks, v, vs)):
        assert np.array_equal(a.cpu().numpy(), b)


def test_bad_pages_lengths_and_scales_are_flagged_and_left_alone():
    need_gpu()
    import torch
    import block_sparse_attention_indexer_gb300 as msa
    c = Case(10, [140, 260, 300, 50], 5, 2, 1)
    c.table[0, 1] = len(c.k)             # a page past the pool
    c.lens[2] = 3                        # fewer tokens than the call writes
    c.ks[c.table[1, 2], 1] = 3           # an invalid scale on a page with older rows
    c.lens[1] = 262
    c.upload()
    kv, x = _rows(c, torch.float32, edges=False)
    got, err = _append(c, kv[:, :, :2], kv[:, :, 2:])
    assert err == msa.MSA_DEVERR_BAD_PAGE | msa.MSA_DEVERR_BAD_SEQLEN | msa.MSA_DEVERR_BAD_SCALE
    k, ks = OF8.append(c.k, c.ks, x[:, :, :2], c.table, c.lens)
    v, vs = OF8.append(c.v, c.vs, x[:, :, 2:], c.table, c.lens)
    for a, b in zip(got, (k, ks, v, vs)):
        assert np.array_equal(a, b)
