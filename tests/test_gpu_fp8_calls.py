"""GPU: calls of the FP8 page cache that its documentation allows beside the ordinary ones: pages that
several table entries name, a block selected twice, pools past 4 GB, the whole loop in a graph."""
import numpy as np
import pytest

from fp8_util import Case, assert_attention
from gpu_util import need_gpu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,Hg", [(1, 8), (2, 8), (30, 4), (150, 2)])
def test_pages_that_several_table_entries_name(T, Hg):
    need_gpu()
    c = Case(600 + T, [900, 700, 300], T, 2, Hg)
    c.table[1, :3] = c.table[0, :3]      # a shared prefix
    c.table[2, 1] = c.table[2, 0]        # the same page twice in one sequence
    c.upload()
    assert_attention(c, c.run(weights=True), c.oracle(), weights=True)
    sel = c.selection()
    assert_attention(c, c.run(selection=sel, weights=True), c.oracle(selection=sel), weights=True)


@pytest.mark.parametrize("T,Hg", [(1, 8), (40, 3)])
def test_a_block_selected_twice_counts_twice(T, Hg):
    need_gpu()
    c = Case(610 + T, [900, 400], T, 2, Hg).upload()
    sel = c.selection(most=3)
    sel[:, :, :, 5] = sel[:, :, :, 0]
    sel[0, 0, 1] = 0                     # one block sixteen times
    assert_attention(c, c.run(selection=sel, weights=True), c.oracle(selection=sel), weights=True)


def test_pools_past_four_gigabytes():
    # 70,000 pages of 4 heads: 4.6 GB of codes a pool; the sequences' pages are the first and the last ones
    need_gpu()
    import torch
    import block_sparse_attention_indexer_gb300 as msa
    P = 70000
    pool = lambda *s: torch.empty(P, 4, *s, dtype=torch.uint8, device="cuda")  # noqa: E731
    big = msa.Fp8Cache.from_tensors(pool(128, 128), pool(), pool(128, 128), pool())
    for T in (1, 30):
        c = Case(620 + T, [700, 300], T, 4, 8).upload()
        small = c.cache
        n = small.num_pages
        where = torch.tensor([(P - 1 - i if i % 2 else i) for i in range(n)], device="cuda")
        for x, y in zip(big.tensors(), small.tensors()):
            x[where] = y
        table = c.batch.block_table
        far = msa.Batch(torch.where(table >= 0, where[table.clamp(min=0).long()].int(), table), c.batch.seq_lens, q_len=T)
        sel = torch.from_numpy(c.selection()).cuda()
        kv = torch.randn(c.B, T, 8, 128, device="cuda")
        got = []
        for cache, batch in ((small, c.batch), (big, far)):
            for s in (None, sel):
                ws = msa.alloc_workspace(msa.MSA_OP_FP8_ATTN, c.cfg, batch)
                out, lse = c.buffers()
                msa.msa_fp8_attn(c.cfg, cache, batch, c.dq, out, lse, ws, selection=s)
                got += [out, lse]
            ws = msa.alloc_workspace(msa.MSA_OP_FP8_APPEND, c.cfg, batch)
            msa.msa_fp8_append(c.cfg, cache, batch, kv[:, :, :4], kv[:, :, 4:], ws)
            assert msa.msa_read_device_error(ws) == 0
        torch.cuda.synchronize()
        for x, y in zip(got[:4], got[4:]):
            assert torch.equal(x, y)
        for x, y in zip(big.tensors(), small.tensors()):
            assert torch.equal(x[where], y)


@pytest.mark.parametrize("T,Hg", [(1, 8), (3, 8)])
def test_append_attend_and_evict_in_one_graph(T, Hg):
    need_gpu()
    import torch
    import block_sparse_attention_indexer_gb300 as msa
    c = Case(630 + T, [1300, 640, 0, 200], T, 2, Hg).upload()
    d = Case(630 + T, [1300, 640, 0, 200], T, 2, Hg).upload()       # the same again
    kv = torch.randn(c.B, T, 4, 128, dtype=torch.bfloat16, device="cuda")

    def state(x):
        i32 = dict(dtype=torch.int32, device="cuda")
        out, lse = x.buffers()
        ops = (msa.MSA_OP_FP8_APPEND, msa.MSA_OP_FP8_ATTN_WEIGHTS, msa.MSA_OP_EVICT)
        return dict(ws=[msa.alloc_workspace(o, x.cfg, x.batch) for o in ops], out=out, lse=lse,
                    w=torch.zeros(x.B, x.max_blocks, device="cuda"), table=torch.zeros(x.B, x.max_blocks, **i32),
                    lens=torch.zeros(x.B, **i32), w2=torch.zeros(x.B, x.max_blocks, device="cuda"),
                    freed=torch.zeros(x.B, x.max_blocks, **i32), count=torch.zeros(x.B, **i32))

    def loop(x, s):
        msa.msa_fp8_append(x.cfg, x.cache, x.batch, kv[:, :, :2], kv[:, :, 2:], s["ws"][0])
        msa.msa_fp8_attn(x.cfg, x.cache, x.batch, x.dq, s["out"], s["lse"], s["ws"][1], weight_out=s["w"])
        msa.msa_evict_blocks(x.batch, s["w"], 4, 1, 1, s["table"], s["lens"], s["w2"], s["freed"], s["count"], s["ws"][2])

    sc, sd = state(c), state(d)
    loop(c, sc)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        loop(d, sd)
    for _ in range(3):                   # (writing the same rows again changes nothing)
        graph.replay()
    torch.cuda.synchronize()
    for n in ("out", "lse", "w", "table", "lens", "w2", "freed", "count"):
        assert torch.equal(sc[n], sd[n]), n
    for x, y in zip(c.cache.tensors(), d.cache.tensors()):
        assert torch.equal(x, y)
    assert sc["count"].tolist() == [7, 1, 0, 0]
    assert all(msa.msa_read_device_error(w) == 0 for w in sc["ws"] + sd["ws"])


@pytest.mark.parametrize("T", [40, 100])
def test_a_long_selection_with_weights_in_a_graph(T):
    # 1,280 and 3,200 entries a sequence: the weights in one launch, and in three behind a memset
    need_gpu()
    import torch
    import block_sparse_attention_indexer_gb300 as msa
    c = Case(640 + T, [2000, 900, 0, 300], T, 2, 8).upload()
    sel = c.selection()
    want = c.run(selection=sel, weights=True)
    assert_attention(c, want, c.oracle(selection=sel), weights=True)
    sel = torch.from_numpy(sel).cuda()
    ws = msa.alloc_workspace(msa.MSA_OP_FP8_ATTN_WEIGHTS, c.cfg, c.batch)
    out, lse = c.buffers()
    w = torch.zeros(c.B, c.max_blocks, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(2):               # (one call behind the other: the second clears what the first has read)
            msa.msa_fp8_attn(c.cfg, c.cache, c.batch, c.dq, out, lse, ws, selection=sel, weight_out=w)
    for _ in range(3):
        for t in (out, lse, w):
            t.fill_(3.0)
        graph.replay()
        torch.cuda.synchronize()
        for got, ref in zip((out, lse, w), want):
            assert np.array_equal(got.double().cpu().numpy(), ref)
    assert msa.msa_read_device_error(ws) == 0
