"""GPU: packed prompts, the FP8 pages and the page pool together, as a serving program uses them; tables, lengths,
counts, pages and outputs of every step against the plain definitions."""
import numpy as np
import pytest

from fp8_util import Case, assert_attention
from gpu_util import need_gpu
from oracle import fp8 as OF8
from oracle import pages as OP
from prompt_util import Prompts

pytestmark = pytest.mark.gpu


def test_prompts_samples_decode_evict_compact():
    need_gpu()
    import torch
    import block_sparse_attention_indexer_gb300 as msa
    G, Hg, P, MB = 2, 3, 40, 9
    rng = np.random.default_rng(5)
    cfg = msa.Config(num_kv_groups=G, heads_per_group=Hg)
    cache = msa.Fp8Cache(P, groups=G)
    pools = [t.cpu().numpy() for t in cache.tensors()]
    buffers = lambda: [(x, None if x.ndim == 2 else 2) for x in pools]  # noqa: E731
    pool = msa.PagePool([cache])
    refs = np.zeros(P, np.int32)
    ws_p = msa.alloc_page_workspace(pool, 16)
    dev = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()  # noqa: E731

    def same(batch, table, lens):
        assert np.array_equal(batch.block_table.cpu().numpy(), table) and np.array_equal(batch.seq_lens.cpu().numpy(), lens)
        assert np.array_equal(pool.refs.cpu().numpy(), refs) and msa.msa_read_device_error(ws_p) == 0
        for a, b in zip(cache.tensors(), pools):
            assert np.array_equal(a.cpu().numpy(), b)

    # three prompts: pages, attention over their own K and V, K and V into the pages
    prompts = [300, 5, 256]
    table, lens = np.full((3, MB), -1, np.int32), np.zeros(3, np.int32)
    batch = msa.Batch(dev(table), dev(lens))
    msa.msa_extend_pages(pool, batch, ws_p, new_tokens=dev(np.array(prompts, np.int32)))
    refs, table, lens, err = OP.extend(refs, table, lens, prompts)
    assert err == 0
    same(batch, table, lens)
    pr = Prompts(6, prompts, G=G, Hg=Hg, fused=True, dev=1.0).upload()
    pr.call()
    pr.check(pr.results())
    for b, n in enumerate(prompts):
        rows = slice(int(pr.cu_q[b]), int(pr.cu_q[b + 1]))
        one = msa.Batch(batch.block_table[b:b + 1], batch.seq_lens[b:b + 1], q_len=n)
        k, v = pr.d[1][None, rows], pr.d[2][None, rows]
        msa.msa_fp8_append(cfg, cache, one, k, v, msa.alloc_workspace(msa.MSA_OP_FP8_APPEND, cfg, one))
        for i, x in ((0, k), (2, v)):
            pools[i], pools[i + 1] = OF8.append(pools[i], pools[i + 1], x.double().cpu().numpy(), table[b:b + 1], lens[b:b + 1])
    same(batch, table, lens)

    # samples of them; the prompts' rows go
    parents = np.array([0, 0, 2, 1, 0], np.int32)
    kids, kid_lens = torch.empty(5, MB, dtype=torch.int32, device="cuda"), torch.empty(5, dtype=torch.int32, device="cuda")
    msa.msa_fork_pages(pool, batch, dev(parents), kids, kid_lens, ws_p)
    msa.msa_free_pages(pool, batch.block_table, ws_p)
    old = table
    refs, table, lens, err = OP.fork(refs, table, lens, parents, buffers())
    refs, err2 = OP.free(refs, old)
    assert err == err2 == 0
    batch = msa.Batch(kids, kid_lens)
    same(batch, table, lens)

    # steps of 100, 1 and 60 tokens, over the pages' ends, with collected weights; the last ones after a compaction
    case = Case(1, [128], 1, G, Hg, "bf16")
    weight = torch.zeros(5, MB, device="cuda")
    for step, T in enumerate([100, 1, 60, 1]):
        if step == 2:
            freed, count = torch.empty_like(kids), torch.empty_like(kid_lens)
            msa.msa_evict_blocks(batch, weight, 3, 1, 1, kids, kid_lens, weight, freed, count,
                                 msa.alloc_workspace(msa.MSA_OP_EVICT, cfg, batch))
            msa.msa_free_pages(pool, freed, ws_p, counts=count)
            table, lens, _, gone, counts = OF8.evict(table, lens, w_after.astype(np.float32), 3, 1, 1)
            refs, err = OP.free(refs, gone, counts)
            assert err == 0
            same(batch, table, lens)
            page_map, live = torch.empty(P, dtype=torch.int32, device="cuda"), torch.empty(1, dtype=torch.int32, device="cuda")
            msa.msa_compact_pages(pool, batch, page_map, live, ws_p)
            refs, table, want_map, n, err = OP.compact(refs, table, lens, buffers())
            assert err == 0 and live.tolist() == [n] and np.array_equal(page_map.cpu().numpy(), want_map)
            same(batch, table, lens)
        batch.q_len = T
        msa.msa_extend_pages(pool, batch, ws_p)
        refs, table, lens, err = OP.extend(refs, table, lens, [T] * 5)
        assert err == 0
        same(batch, table, lens)
        qkv = torch.from_numpy(rng.normal(0, 1, (5, T, G * Hg + 2 * G, 128))).to(torch.bfloat16).cuda()
        q, k, v = qkv.split([G * Hg, G, G], dim=2)
        msa.msa_fp8_append(cfg, cache, batch, k, v, msa.alloc_workspace(msa.MSA_OP_FP8_APPEND, cfg, batch))
        for i, x in ((0, k), (2, v)):
            pools[i], pools[i + 1] = OF8.append(pools[i], pools[i + 1], x.double().cpu().numpy(), table, lens)
        same(batch, table, lens)
        out = torch.empty(5, T, G * Hg, 128, dtype=torch.bfloat16, device="cuda")
        lse = torch.empty(5, T, G * Hg, device="cuda")
        ws = msa.alloc_workspace(msa.MSA_OP_FP8_ATTN_WEIGHTS, cfg, batch)
        w_before = weight.double().cpu().numpy()
        msa.msa_fp8_attn(cfg, cache, batch, q, out, lse, ws, weight_in=weight, weight_out=weight)
        torch.cuda.synchronize()
        case.T, case.q = T, q.double().cpu().numpy()
        ref = OF8.attention(case.q, pools, table, lens, Hg, weight_in=w_before, decay=1.0)
        w_after = weight.double().cpu().numpy()
        assert_attention(case, (out.double().cpu().numpy(), lse.double().cpu().numpy(), w_after,
                                   msa.msa_read_device_error(ws)), ref, weights=True)
