"""GPU: the FP8 operators together, as a decoding program uses them: append, attend while the
weights accumulate, evict, go on with the shorter table; every step against the oracle."""
import numpy as np
import pytest

from fp8_util import Case, assert_attention
from gpu_util import need_gpu
from oracle import fp8 as OF8

pytestmark = pytest.mark.gpu


def test_prompt_decode_evict_decode():
    need_gpu()
    import torch
    import block_sparse_attention_indexer_gb300 as msa
    G, Hg, B, MB, P = 2, 4, 3, 8, 24
    rng = np.random.default_rng(77)
    cfg = msa.Config(num_kv_groups=G, heads_per_group=Hg)
    cache = msa.Fp8Cache(P, groups=G)
    pools = [t.cpu().numpy() for t in cache.tensors()]
    table_h = rng.permutation(P).reshape(B, MB).astype(np.int32)
    table, lens = torch.from_numpy(table_h.copy()).cuda(), torch.zeros(B, dtype=torch.int32, device="cuda")
    lens_h = np.zeros(B, np.int32)
    weight = torch.zeros(B, MB, device="cuda")
    freed, count = torch.empty_like(table), torch.empty_like(lens)
    batch = msa.Batch(table, lens)
    ws_e = msa.alloc_workspace(msa.MSA_OP_EVICT, cfg, batch)
    checker = Case(1, [128], 1, G, Hg, "bf16")

    for step, T in enumerate([300, 1, 1, 90, 1, 20, 260, 1]):
        lens += T
        lens_h = lens_h + T
        batch.q_len = T
        ws_a = msa.alloc_workspace(msa.MSA_OP_FP8_APPEND, cfg, batch)
        ws_t = msa.alloc_workspace(msa.MSA_OP_FP8_ATTN_WEIGHTS, cfg, batch)
        qkv = torch.from_numpy(rng.normal(0, 1, (B, T, G * Hg + 2 * G, 128))).to(torch.bfloat16).cuda()
        q, k, v = qkv.split([G * Hg, G, G], dim=2)
        msa.msa_fp8_append(cfg, cache, batch, k, v, ws_a)
        out = torch.empty(B, T, G * Hg, 128, dtype=torch.bfloat16, device="cuda")
        lse = torch.empty(B, T, G * Hg, device="cuda")
        w_before = weight.double().cpu().numpy()
        msa.msa_fp8_attn(cfg, cache, batch, q, out, lse, ws_t, weight_in=weight, weight_out=weight, weight_decay=0.75)
        torch.cuda.synchronize()
        kn, vn = k.double().cpu().numpy(), v.double().cpu().numpy()
        pools[0], pools[1] = OF8.append(pools[0], pools[1], kn, table_h, lens_h)
        pools[2], pools[3] = OF8.append(pools[2], pools[3], vn, table_h, lens_h)
        for a, b in zip(cache.tensors(), pools):
            assert np.array_equal(a.cpu().numpy(), b), step
        checker.T, checker.q = T, q.double().cpu().numpy()
        ref = OF8.attention(checker.q, pools, table_h, lens_h, Hg, weight_in=w_before, decay=0.75)
        got = (out.double().cpu().numpy(), lse.double().cpu().numpy(), weight.double().cpu().numpy(),
               msa.msa_read_device_error(ws_t))
        assert msa.msa_read_device_error(ws_a) == 0
        assert_attention(checker, got, ref, weights=True)
        if step in (3, 6):
            w_h = weight.cpu().numpy()
            msa.msa_evict_blocks(batch, weight, 2, 1, 1, table, lens, weight, freed, count, ws_e)
            torch.cuda.synchronize()
            want = OF8.evict(table_h, lens_h, w_h, 2, 1, 1)
            assert all(np.array_equal(a.cpu().numpy(), b) for a, b in zip((table, lens, weight, freed, count), want))
            table_h, lens_h = want[0].copy(), want[1]
            gone = want[3][want[3] >= 0]
            assert len(gone) == want[4].sum() > 0
            # the freed pages go to the ends of the tables again
            for b in range(B):
                n = int(want[4][b])
                table_h[b, 2:2 + n] = want[3][b, :n]
            rest = sorted(set(range(P)) - set(table_h[table_h >= 0].tolist()))
            for b in range(B):
                for j in range(MB):
                    if table_h[b, j] < 0:
                        table_h[b, j] = rest.pop()
            table.copy_(torch.from_numpy(table_h))
    assert msa.msa_read_device_error(ws_e) == 0


def test_selection_from_the_indexer_drives_the_fp8_attention():
    """A sparse layer with an NVFP4 index-key cache and FP8 K/V: scores, selection, attention."""
    need_gpu()
    import torch
    import block_sparse_attention_indexer_gb300 as msa
    c = Case(41, [4000, 900, 0], 2, 4, 8).upload()
    pages = c.cache.num_pages
    nv = msa.PagedCache(pages)
    slots = torch.arange(pages * 128, device="cuda")
    idx = torch.from_numpy(c.rng.normal(0, 1, (pages * 128, 1, 128))).float().cuda()
    msa.msa_nvfp4_insert(idx, slots, nv.idx_data.view(pages, 1, 128, 64), nv.idx_scale.view(pages, 1, 128, 8))
    qi = torch.empty(c.B, c.T, 4, 128, dtype=torch.uint8, device="cuda")
    msa.msa_fp8_quantize(torch.from_numpy(c.rng.normal(0, 1, (c.B, c.T, 4, 128))).float().cuda(), qi)
    scores = torch.empty(c.B, c.T, 4, c.max_blocks, device="cuda")
    msa.msa_indexer_scores(c.cfg, nv, c.batch, qi, scores, msa.alloc_workspace(msa.MSA_OP_INDEXER_SCORES, c.cfg, c.batch))
    sel = torch.empty(c.B, c.T, 4, 16, dtype=torch.int32, device="cuda")
    msa.msa_select_blocks(c.cfg, c.batch, scores, sel)
    torch.cuda.synchronize()
    sel = sel.cpu().numpy()
    assert_attention(c, c.run(selection=sel, weights=True), c.oracle(selection=sel), weights=True)
