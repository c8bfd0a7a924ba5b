"""The README's example of the FP8 page cache, run as written: a prompt written and attended to with its
weights collected, the tables cut, one decode step.  Its last output must agree with a float64
softmax over the dequantised pages that are left."""
import pytest

from gpu_util import need_gpu

pytestmark = pytest.mark.gpu


def test_readme_fp8_example_runs():
    need_gpu()
    # ---- begin README example
    import torch
    import block_sparse_attention_indexer_gb300 as msa

    cfg = msa.Config(num_kv_groups=4, heads_per_group=8)
    B, L, blocks = 2, 5000, 48                                 # sequences, prompt tokens, table width
    cache = msa.Fp8Cache(B * blocks, groups=4)                 # E4M3 pages, a power-of-two scale per (page, KV head)
    table = torch.arange(B * blocks, dtype=torch.int32, device="cuda").view(B, blocks)  # block -> page
    lens = torch.full((B,), L, dtype=torch.int32, device="cuda")
    weight = torch.zeros(B, blocks, device="cuda")             # attention weight that each block has collected
    # the prompt: write K and V (a fused projection's heads, no copy), attend, collect the weights
    prompt = msa.Batch(table, lens, q_len=L)
    k, v = torch.randn(B, L, 8, 128, dtype=torch.bfloat16, device="cuda").chunk(2, dim=2)
    q = torch.randn(B, L, 32, 128, dtype=torch.bfloat16, device="cuda")
    out = torch.empty_like(q)
    msa.msa_fp8_append(cfg, cache, prompt, k, v, msa.alloc_workspace(msa.MSA_OP_FP8_APPEND, cfg, prompt))
    ws = msa.alloc_workspace(msa.MSA_OP_FP8_ATTN_WEIGHTS, cfg, prompt)
    msa.msa_fp8_attn(cfg, cache, prompt, q, out, None, ws, weight_in=weight, weight_out=weight)
    assert msa.msa_read_device_error(ws) == 0
    # cut every sequence to 24 blocks: the first, the last two and the 21 heaviest of the others
    freed, count = torch.empty_like(table), torch.empty_like(lens)
    msa.msa_evict_blocks(prompt, weight, 24, 1, 2, table, lens, weight, freed, count,
                         msa.alloc_workspace(msa.MSA_OP_EVICT, cfg, prompt))
    # one decode step on what is left (its last block still has room; else a page goes into the table first)
    lens += 1
    step = msa.Batch(table, lens, q_len=1)
    k1, v1 = torch.randn(B, 1, 8, 128, dtype=torch.bfloat16, device="cuda").chunk(2, dim=2)
    q1 = torch.randn(B, 1, 32, 128, dtype=torch.bfloat16, device="cuda")
    out1 = torch.empty_like(q1)
    msa.msa_fp8_append(cfg, cache, step, k1, v1, msa.alloc_workspace(msa.MSA_OP_FP8_APPEND, cfg, step))
    ws = msa.alloc_workspace(msa.MSA_OP_FP8_ATTN_WEIGHTS, cfg, step)
    msa.msa_fp8_attn(cfg, cache, step, q1, out1, None, ws, weight_in=weight, weight_out=weight, weight_decay=0.99)
    assert msa.msa_read_device_error(ws) == 0
    # ---- end README example
    # of 40 blocks 24 stay, in order
    assert count.tolist() == [16, 16] and lens.tolist() == [L - 16 * 128 + 1] * 2
    assert (table[:, :24] >= 0).all() and (table[:, 1:24] > table[:, :23]).all() and (table[:, 24:] == -1).all() and (weight[:, 24:] == 0).all()
    assert sorted(set(table[0, :24].tolist()) | set(freed[0, :16].tolist())) == list(range(40))
    assert torch.isfinite(out.float()).all()
    n = int(lens[0])

    def rows(data, scale, b):
        codes = data[table[b, :24].long()].view(torch.float8_e4m3fn).double()         # [24, 4, 128, 128]
        power = torch.exp2(scale[table[b, :24].long()].double() - 127)[:, :, None, None]
        return (codes * power).transpose(1, 2).reshape(24 * 128, 4, 128)[:n]

    for b in range(B):
        kd, vd = rows(cache.k_data, cache.k_scale, b), rows(cache.v_data, cache.v_scale, b)
        z = torch.einsum("ghd,ngd->ghn", q1[b, 0].double().view(4, 8, 128), kd) * 128 ** -0.5
        want = torch.einsum("ghn,ngd->ghd", torch.softmax(z, -1), vd).reshape(32, 128)
        # P in fp16 is off by 2^-11 of each term, the bf16 output by 2^-8 of itself; float32 sums far less
        bound = 2.0 ** -8 * want.abs() + 2.0 ** -10 * torch.einsum(
            "ghn,ngd->ghd", torch.softmax(z, -1), vd.abs()).reshape(32, 128) + 1e-6
        assert ((out1[b, 0].double() - want).abs() <= bound).all()
