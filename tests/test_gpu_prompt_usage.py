"""The README's example of packed prompts and the page pool, run as written; the prompts' attention, the last decode step
and the pool's counts are checked afterwards."""
import pytest

from gpu_util import need_gpu

pytestmark = pytest.mark.gpu


def test_readme_prompt_and_pool_example_runs():
    need_gpu()
    # ---- begin README example
    import torch
    import block_sparse_attention_indexer_gb300 as msa

    cfg = msa.Config(num_kv_groups=4, heads_per_group=8)
    cache = msa.Fp8Cache(64, groups=4)                         # E4M3 pages; a model has one cache a layer
    pool = msa.PagePool([cache])                               # how many references each page has: all free
    prompts, blocks = [700, 1, 300], 8                         # tokens of each prompt, table width
    table = torch.full((3, blocks), -1, dtype=torch.int32, device="cuda")
    lens = torch.zeros(3, dtype=torch.int32, device="cuda")
    batch = msa.Batch(table, lens)
    pages_ws = msa.alloc_page_workspace(pool, 6)
    # pages for the prompts, straight into the tables
    msa.msa_extend_pages(pool, batch, pages_ws, new_tokens=torch.tensor(prompts, dtype=torch.int32, device="cuda"))
    # the prompts packed one after another: causal attention over their own bf16 K and V (a fused projection's rows)
    N = sum(prompts)
    q, k, v = torch.randn(N, 32 + 2 * 4, 128, device="cuda").bfloat16().split((32, 4, 4), dim=1)
    starts = torch.tensor([0, 700, 701, 1001], dtype=torch.int32, device="cuda")
    packed = msa.Packed(starts, starts, N, N)
    out = torch.empty(N, 32, 128, dtype=torch.bfloat16, device="cuda")
    ws = msa.alloc_workspace(msa.MSA_OP_PROMPT_ATTN, cfg, packed)
    msa.msa_prompt_attn(cfg, packed, q, k, v, out, None, ws)
    assert msa.msa_read_device_error(ws) == 0
    # their K and V into the pages
    for b, (n, at) in enumerate(zip(prompts, (0, 700, 701))):
        one = msa.Batch(table[b:b + 1], lens[b:b + 1], q_len=n)
        msa.msa_fp8_append(cfg, cache, one, k[None, at:at + n], v[None, at:at + n],
                           msa.alloc_workspace(msa.MSA_OP_FP8_APPEND, cfg, one))
    # four samples of the first prompt, one of each other; the prompts' own rows are given back
    samples = torch.empty(6, blocks, dtype=torch.int32, device="cuda")
    sample_lens = torch.empty(6, dtype=torch.int32, device="cuda")
    parents = torch.tensor([0, 0, 0, 0, 1, 2], dtype=torch.int32, device="cuda")
    msa.msa_fork_pages(pool, batch, parents, samples, sample_lens, pages_ws)
    msa.msa_free_pages(pool, table, pages_ws)
    # decode steps: a page where a sequence needs one, the new K and V, attention over the pages
    step = msa.Batch(samples, sample_lens, q_len=1)
    append_ws = msa.alloc_workspace(msa.MSA_OP_FP8_APPEND, cfg, step)
    ws = msa.alloc_workspace(msa.MSA_OP_FP8_ATTN, cfg, step)
    out1 = torch.empty(6, 1, 32, 128, dtype=torch.bfloat16, device="cuda")
    for _ in range(3):
        q1, k1, v1 = torch.randn(6, 1, 32 + 2 * 4, 128, device="cuda").bfloat16().split((32, 4, 4), dim=2)
        msa.msa_extend_pages(pool, step, pages_ws)
        msa.msa_fp8_append(cfg, cache, step, k1, v1, append_ws)
        msa.msa_fp8_attn(cfg, cache, step, q1, out1, None, ws)
    # three samples are finished; what is left moves to the front of the pool
    msa.msa_free_pages(pool, samples[:3], pages_ws)
    left = msa.Batch(samples[3:], sample_lens[3:])
    new_number = torch.empty(64, dtype=torch.int32, device="cuda")
    in_use = torch.empty(1, dtype=torch.int32, device="cuda")
    msa.msa_compact_pages(pool, left, new_number, in_use, pages_ws)
    assert msa.msa_read_device_error(pages_ws) == 0
    # ---- end README example
    for b, (n, at) in enumerate(zip(prompts, (0, 700, 701))):
        kd, vd, qd = (x[at:at + n].double() for x in (k, v, q))
        z = torch.einsum("tghd,jgd->ghtj", qd.view(n, 4, 8, 128), kd) * 128 ** -0.5
        z.masked_fill_(torch.ones(n, n, dtype=torch.bool, device="cuda").triu(1), float("-inf"))
        p = torch.softmax(z, -1)
        want = torch.einsum("ghtj,jgd->tghd", p, vd).reshape(n, 32, 128)
        # P in bf16 is off by 2^-8 of each term and so is the sum that divides it; the output by 2^-8 of itself
        bound = 2.0 ** -8 * want.abs() + 2.0 ** -6.9 * torch.einsum("ghtj,jgd->tghd", p, vd.abs()).reshape(n, 32, 128) + 1e-6
        assert ((out[at:at + n].double() - want).abs() <= bound).all()
    # six full pages of the first prompt, one sample's last page, the other prompts' pages: all of them at the front
    assert sample_lens.tolist() == [703] * 4 + [4, 303]
    assert in_use.tolist() == [6 + 1 + 3] and pool.refs.tolist() == [1] * 10 + [0] * 54
    assert sorted(x for row in samples[3:].tolist() for x in row if x >= 0) == list(range(10))
    assert sorted(x for x in new_number.tolist() if x >= 0) == list(range(10))

    def rows(data, scale, b, n):
        page = samples[b, :-(-n // 128)].long()
        power = torch.exp2(scale[page].double() - 127)[:, :, None, None]
        return (data[page].view(torch.float8_e4m3fn).double() * power).transpose(1, 2).reshape(-1, 4, 128)[:n]

    for b in (3, 4, 5):
        n = int(sample_lens[b])
        kd, vd = rows(cache.k_data, cache.k_scale, b, n), rows(cache.v_data, cache.v_scale, b, n)
        p = torch.softmax(torch.einsum("ghd,ngd->ghn", q1[b, 0].double().view(4, 8, 128), kd) * 128 ** -0.5, -1)
        want = torch.einsum("ghn,ngd->ghd", p, vd).reshape(32, 128)
        # P in fp16 is off by 2^-11 of each term, the bf16 output by 2^-8 of itself; float32 sums far less
        bound = 2.0 ** -8 * want.abs() + 2.0 ** -10 * torch.einsum("ghn,ngd->ghd", p, vd.abs()).reshape(32, 128) + 1e-6
        assert ((out1[b, 0].double() - want).abs() <= bound).all()
