"""Operators around the page caches, as cases to be measured: what each computes in plain torch operations, and the calls
that a program makes of the library.

  prompt   msa_prompt_attn: causal attention of packed prompts of different lengths over their own bf16 K and V
  extend   msa_extend_pages: pages for the new tokens of every sequence
  fork     msa_fork_pages: sequences that go on from others: full pages shared, the last one's tokens copied
  free     msa_free_pages: references to listed pages given back
  compact  msa_compact_pages: live pages moved to the lowest numbers, block tables renamed

A page holds 128 tokens of every KV head.  Reference counts, tables and lengths are written to tensors of their own here, so
that a pass can be repeated; the pages' data is changed in place.
"""
import math
import random

import torch

own = False

BLOCK, DIM = 128, 128
DEV = "cuda"


# ------------------------------------------------------------------------------------------------ cases
def listed():
    return [
        # a handful of short questions in one call: the smallest prompts, all latency
        dict(name="prompt_short8", op="prompt", batch=8, tokens=75, prefix=0, groups=4, heads=8),
        # a batch of prompts of different lengths as a scheduler packs them, the last row padding
        dict(name="prompt_ragged32", op="prompt", batch=32, tokens=2000, prefix=0, groups=4, heads=8),
        # the next chunk of long prompts: new queries over the keys so far as well
        dict(name="prompt_chunk4_on_16k", op="prompt", batch=4, tokens=1003, prefix=16384, groups=2, heads=5),
        # one long prompt: bound by the tensor cores
        dict(name="prompt_16k", op="prompt", batch=1, tokens=16384, prefix=0, groups=4, heads=8),
        # the pages of one decode step of a serving batch: few sequences reach a new page
        dict(name="extend_decode64", op="extend", batch=64, longest=131072, tokens=1, spare=512),
        # a large batch of long sequences, half of them new prompts: many pages out of a large pool
        dict(name="extend_b512_512k", op="extend", batch=512, longest=524288, tokens=65536, spare=300_000),
        # four samples of one chat: a small fork
        dict(name="fork_1_to_4", op="fork", batch=1, longest=4000, children=4, layers=2, groups=4),
        # a beam step over a batch: 64 sequences go on from 16, in the caches of twelve layers
        dict(name="fork_16_to_64", op="fork", batch=16, longest=3000, children=64, layers=12, groups=4),
        # what one eviction pass of a serving batch gave up
        dict(name="free_b64", op="free", batch=64, longest=131072, pages=70_000),
        # finished sequences of a large batch, pages shared among several
        dict(name="free_b512_shared", op="free", batch=512, longest=524288, pages=400_000),
        # a small pool after some chats have left
        dict(name="compact_200", op="compact", batch=8, longest=2500, pages=200, layers=2, groups=4),
        # half of a pool's pages in use: the move of a quarter of it in the caches of four layers
        dict(name="compact_2k_half", op="compact", batch=32, longest=6000, pages=2048, layers=4, groups=4),
    ]


def _spread(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["prompt"] * 4 + ["extend", "fork", "free", "compact"])
    groups = rng.choice([1, 2, 4, 8])
    if op == "prompt":
        heads = rng.choice([1, 2, 3, 4, 5, 6, 7, 8])
        tokens = _spread(rng, 1, 8192)
        prefix = 0 if rng.random() < 0.6 else _spread(rng, 1, 16384)
        # twice the pairs of queries and keys of the largest listed case (of the longest sequence here, all heads)
        pairs = 8_500_000_000 // (groups * heads)
        while tokens * (tokens + 2 * prefix) > pairs:
            tokens, prefix = tokens * 3 // 4, prefix * 3 // 4
        most = pairs // (tokens * (tokens + 2 * prefix))
        batch = _spread(rng, 1, max(1, min(64, most, 32768 // tokens, 65536 // (tokens + prefix))))
        return dict(op=op, batch=batch, tokens=tokens, prefix=prefix, groups=groups, heads=heads)
    if op == "extend":
        batch = _spread(rng, 1, 512)
        longest = _spread(rng, 200, 524288)
        return dict(op=op, batch=batch, longest=longest, tokens=_spread(rng, 1, max(1, longest // 8)),
                    spare=_spread(rng, 600, 300_000) + batch * (-(-longest // 8 // BLOCK) + 1))
    if op == "free":
        longest = _spread(rng, 200, 524288)
        return dict(op=op, batch=_spread(rng, 1, 512), longest=longest, pages=_spread(rng, 600, 400_000))
    layers = rng.randint(1, 8)
    if op == "fork":
        longest = _spread(rng, 5, 4000)
        batch = _spread(rng, 1, 16)
        return dict(op=op, batch=batch, longest=longest, children=_spread(rng, 1, 64), layers=layers, groups=groups)
    pages = _spread(rng, 16, 8192 // (layers * groups))
    blocks = max(1, int(pages * rng.uniform(0.05, 0.9)))
    batch = _spread(rng, 1, max(1, min(64, blocks)))
    return dict(op=op, batch=batch, longest=max(1, blocks // batch * BLOCK - rng.randint(0, 127)), pages=pages,
                layers=layers, groups=groups)


def _lengths(case):
    """Tokens of each sequence: one has the most, the others lie between an eighth of it and all of it; in a batch of 16
    or more the last row is padding."""
    B, most = case["batch"], case["tokens"] if case["op"] == "prompt" else case["longest"]
    least = max(1, most // 8)
    got = [most] + [least + int((most - least) * ((b * 0.6180339887498949) % 1.0)) for b in range(1, B)]
    if B >= 16:
        got[-1] = 0
    return got


def _prefixes(case):
    """Keys before each sequence's first query."""
    most = case["prefix"]
    return [int(most * (1.0 - (b * 0.7548776662466927) % 1.0)) if n else 0 for b, n in enumerate(_lengths(case))]


def _new_tokens(case):
    """(length before, new tokens) of each sequence of an `extend` case.  One token each, or: every other sequence is new."""
    lens = _lengths(case)
    if case["tokens"] == 1:
        return [(max(0, n - 1), 1 if n else 0) for n in lens]
    return [(0, min(n, case["tokens"])) if b % 2 else (max(0, n - 1 - b % 300), min(n, 1 + b % 300)) for b, n in enumerate(lens)]


def _blocks(n):
    return -(-n // BLOCK)


# ------------------------------------------------------------------------------------------------ inputs
def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _cumulative(lens):
    return _i32([sum(lens[:i]) for i in range(len(lens) + 1)])


def _codes(gen, *shape):
    """E4M3 codes of normal values with deviation 64."""
    out = torch.empty(shape, dtype=torch.uint8, device=DEV)
    flat = out.view(-1)
    for at in range(0, flat.numel(), 1 << 28):
        part = flat[at:at + (1 << 28)]
        part.copy_(torch.randn(part.numel(), generator=gen, device=DEV).mul_(64).clamp_(-448, 448)
                   .to(torch.float8_e4m3fn).view(torch.uint8))
    return out


def _table(blocks, width, pages, gen, order=None):
    """A block table whose rows' first blocks are pages of `order` (a random one) one after another, round and round."""
    if order is None:
        order = torch.randperm(pages, generator=gen, device=DEV).to(torch.int32)
    nb = torch.tensor(blocks, device=DEV)
    n = torch.arange(width, device=DEV)
    at = (nb.cumsum(0) - nb)[:, None] + n
    return torch.where(n < nb[:, None], order[at % order.numel()], -1).to(torch.int32)


def _references(table, pages):
    used = table[table >= 0].long()
    return torch.zeros(pages, dtype=torch.int32, device=DEV).index_add_(0, used, torch.ones_like(used, dtype=torch.int32))


def prepare(case, seed):
    gen = torch.Generator(DEV).manual_seed(seed)
    s = dict(case=case)
    op = case["op"]
    if op == "prompt":
        G, H = case["groups"], case["groups"] * case["heads"]
        s["lq"] = _lengths(case)
        s["lk"] = [n + p for n, p in zip(s["lq"], _prefixes(case))]
        Nq, Nk = sum(s["lq"]), sum(s["lk"])
        s["cu_q"], s["cu_k"] = _cumulative(s["lq"]), _cumulative(s["lk"])
        s["tokens"] = (Nq, Nk)
        if case["prefix"] == 0:  # rows as a fused projection leaves them
            qkv = torch.randn(Nq, H + 2 * G, DIM, generator=gen, device=DEV)
            qkv[:, :H + G] *= 1.5
            s["q"], s["k"], s["v"] = qkv.to(torch.bfloat16).split((H, G, G), dim=1)
        else:
            s["q"] = (1.5 * torch.randn(Nq, H, DIM, generator=gen, device=DEV)).to(torch.bfloat16)
            s["k"] = (1.5 * torch.randn(Nk, G, DIM, generator=gen, device=DEV)).to(torch.bfloat16)
            s["v"] = torch.randn(Nk, G, DIM, generator=gen, device=DEV).to(torch.bfloat16)
        s["out"] = torch.empty(Nq, H, DIM, dtype=torch.bfloat16, device=DEV)
        s["lse"] = torch.empty(Nq, H, device=DEV)
    else:
        _prepare_pages(s, gen)
    if own:
        _library(s)
    return s


def _prepare_pages(s, gen):
    case = s["case"]
    op = case["op"]
    lens = _lengths(case)
    nb = [_blocks(n) for n in lens]
    width = max(1, max(nb))
    if op == "extend":
        was = _new_tokens(case)
        held = [_blocks(a) for a, _ in was]
        pages = sum(held) + case["spare"]
        s["new"] = _i32([n for _, n in was]) if case["tokens"] > 1 else None
        lens = [a for a, _ in was]
        s["table"] = _table(held, width, pages, gen)
        s["refs"] = _references(s["table"], pages)
    elif op == "free":
        # sequences share pages where the pool is smaller than what they hold
        pages = case["pages"]
        s["table"] = _table(nb, width, pages, gen)
        s["refs"] = _references(s["table"], pages)
        s["counts"] = (torch.rand(len(nb), generator=gen, device=DEV) * (_i32(nb) + 1)).to(torch.int32)
    elif op == "fork":
        n = case["children"]
        pages = sum(nb) + n + 16
        s["table"] = _table(nb, width, pages, gen)
        s["refs"] = _references(s["table"], pages)
        s["parents"] = torch.randint(len(nb) - (len(nb) >= 16), (n,), generator=gen, device=DEV, dtype=torch.int32)
    else:
        pages = case["pages"]
        s["table"] = _table(nb, width, pages, gen)
        s["refs"] = _references(s["table"], pages)
        s["page_map"] = torch.empty(pages, dtype=torch.int32, device=DEV)
        s["live"] = torch.empty(1, dtype=torch.int32, device=DEV)
    s["lens"] = _i32(lens)
    s["refs_out"] = torch.empty_like(s["refs"])
    rows = case["children"] if op == "fork" else len(lens)
    s["table_out"] = torch.empty(rows, width, dtype=torch.int32, device=DEV)
    s["lens_out"] = torch.empty(rows, dtype=torch.int32, device=DEV)
    G = case.get("groups")
    s["layers"] = []
    for _ in range(case.get("layers", 0)):
        pool, heads = (pages, G, BLOCK, DIM), (pages, G)
        s["layers"].append((_codes(gen, *pool), torch.randint(100, 140, heads, generator=gen, device=DEV, dtype=torch.uint8),
                            _codes(gen, *pool), torch.randint(100, 140, heads, generator=gen, device=DEV, dtype=torch.uint8)))


def _library(s):
    """The handles and the workspace that a program keeps."""
    import block_sparse_attention_indexer_gb300 as msa
    case = s["case"]
    s["msa"] = msa
    if case["op"] == "prompt":
        s["cfg"] = msa.Config(num_kv_groups=case["groups"], heads_per_group=case["heads"])
        s["packed"] = msa.Packed(s["cu_q"], s["cu_k"], *s["tokens"])
        s["ws"] = msa.alloc_workspace(msa.MSA_OP_PROMPT_ATTN, s["cfg"], s["packed"])
        return
    s["pool"] = msa.PagePool([msa.Fp8Cache.from_tensors(*t) for t in s["layers"]], refs=s["refs"])
    s["batch"] = msa.Batch(s["table"], s["lens"], q_len=1)
    s["ws"] = msa.alloc_page_workspace(s["pool"], s["table_out"].shape[0])


# ------------------------------------------------------------------------------------------------ one pass
_OUTPUTS = {"extend": ("table_out", "lens_out", "refs_out"), "fork": ("table_out", "lens_out", "refs_out"),
            "free": ("refs_out",), "compact": ("table_out", "refs_out", "page_map", "live")}


def run(s):
    op = s["case"]["op"]
    if op == "prompt":
        if own:
            s["msa"].msa_prompt_attn(s["cfg"], s["packed"], s["q"], s["k"], s["v"], s["out"], s["lse"], s["ws"])
        else:
            _plain_prompt(s)
        return {"out": s["out"], "lse": s["lse"]}
    if own:
        msa, pool, out = s["msa"], s["pool"], dict(refs_out=s["refs_out"])
        if op == "extend":
            msa.msa_extend_pages(pool, s["batch"], s["ws"], new_tokens=s["new"], table_out=s["table_out"],
                                 seq_lens_out=s["lens_out"], **out)
        elif op == "fork":
            msa.msa_fork_pages(pool, s["batch"], s["parents"], s["table_out"], s["lens_out"], s["ws"], **out)
        elif op == "free":
            msa.msa_free_pages(pool, s["table"], s["ws"], counts=s["counts"], **out)
        else:
            msa.msa_compact_pages(pool, s["batch"], s["page_map"], s["live"], s["ws"], table_out=s["table_out"], **out)
    else:
        {"extend": _plain_extend, "fork": _plain_fork, "free": _plain_free, "compact": _plain_compact}[op](s)
    got = {n: s[n] for n in _OUTPUTS[op]}
    for i, (k, ks, v, vs) in enumerate(s["layers"]):
        # codes as the values that they stand for in units of their page's scale, and the scales' exponents
        got.update({f"k{i}": k.view(torch.float8_e4m3fn), f"k_scale{i}": ks, f"v{i}": v.view(torch.float8_e4m3fn), f"v_scale{i}": vs})
    return got


def _plain_prompt(s):
    case = s["case"]
    G, Hg = case["groups"], case["heads"]
    q0 = k0 = 0
    for nq, nk in zip(s["lq"], s["lk"]):
        pos = nk - nq + torch.arange(nq, device=DEV)
        at = torch.arange(nk, device=DEV)
        heads = max(1, min(Hg, 600_000_000 // max(1, nq * nk)))
        for g in range(G if nq else 0):
            K, V = s["k"][k0:k0 + nk, g].float(), s["v"][k0:k0 + nk, g].float()
            for h in range(g * Hg, (g + 1) * Hg, heads):
                h1 = min(h + heads, (g + 1) * Hg)
                p = s["q"][q0:q0 + nq, h:h1].float().transpose(0, 1).mul(1.0 / math.sqrt(DIM)) @ K.T     # [heads, nq, nk]
                p.masked_fill_(at > pos[:, None], -math.inf)
                top = p.amax(-1, keepdim=True)
                p.sub_(top).exp_()
                total = p.sum(-1, keepdim=True)
                s["out"][q0:q0 + nq, h:h1] = ((p @ V) / total).transpose(0, 1).to(torch.bfloat16)
                s["lse"][q0:q0 + nq, h:h1] = (top + total.log()).squeeze(-1).T
        q0, k0 = q0 + nq, k0 + nk


def _plain_extend(s):
    lens, table, refs = s["lens"].long(), s["table"], s["refs"]
    new = s["new"].long() if s["new"] is not None else (lens > 0).long()
    first = (lens + BLOCK - 1) // BLOCK
    need = (lens + new + BLOCK - 1) // BLOCK - first
    upto = need.cumsum(0)
    free = torch.nonzero(refs == 0).squeeze(1)
    ok = (need == 0) | (upto <= free.numel())
    n = torch.arange(table.shape[1], device=DEV)
    fresh = ok[:, None] & (n >= first[:, None]) & (n < (first + need)[:, None])
    rank = ((upto - need - first)[:, None] + n)[fresh]
    pages = free[rank]
    s["table_out"].copy_(table)
    s["table_out"][fresh] = pages.to(torch.int32)
    s["refs_out"].copy_(refs)
    s["refs_out"][pages] = 1
    s["lens_out"].copy_(lens + torch.where(ok, new, 0))


def _plain_fork(s):
    parents, refs, table = s["parents"].long(), s["refs"], s["table"]
    lens = s["lens"].long()[parents]
    full, tail = lens // BLOCK, lens % BLOCK
    n = torch.arange(table.shape[1], device=DEV)
    rows = torch.where(n < full[:, None], table[parents], -1)
    s["refs_out"].copy_(refs)
    shared = rows[rows >= 0].long()
    s["refs_out"].index_add_(0, shared, torch.ones_like(shared, dtype=torch.int32))
    child = torch.nonzero(tail).squeeze(1)
    page = torch.nonzero(refs == 0).squeeze(1)[:child.numel()]
    old = table[parents[child], full[child]].long()
    s["refs_out"][page] = 1
    rows[child, full[child]] = page.to(torch.int32)
    s["table_out"].copy_(rows)
    s["lens_out"].copy_(lens)
    here = (torch.arange(BLOCK, device=DEV) < tail[child][:, None])[:, None, :, None]
    for k, ks, v, vs in s["layers"]:
        for data in (k, v):
            data[page] = torch.where(here, data[old], data[page])
        ks[page], vs[page] = ks[old], vs[old]


def _plain_free(s):
    table, refs = s["table"], s["refs"]
    listed_ = torch.arange(table.shape[1], device=DEV) < s["counts"][:, None]
    gone = table[listed_ & (table >= 0)].long()
    s["refs_out"].copy_(refs)
    s["refs_out"].index_add_(0, gone, torch.full_like(gone, -1, dtype=torch.int32))
    s["refs_out"].clamp_(min=0)


def _plain_compact(s):
    refs, table = s["refs"], s["table"]
    number = torch.arange(refs.numel(), device=DEV)
    live = refs != 0
    n = live.sum()
    hole = torch.nonzero(~live & (number < n)).squeeze(1)
    mover = torch.nonzero(live & (number >= n)).squeeze(1)
    to = torch.where(live, number, -1)
    to[mover] = hole
    s["page_map"].copy_(to)
    s["live"].copy_(n)
    s["refs_out"].copy_(refs)
    s["refs_out"][hole] = refs[mover]
    s["refs_out"][mover] = 0
    nb = (s["lens"].long() + BLOCK - 1) // BLOCK
    held = (torch.arange(table.shape[1], device=DEV) < nb[:, None]) & (table >= 0)
    s["table_out"].copy_(torch.where(held, to[table.clamp(min=0).long()], -1))
    for data in (t for layer in s["layers"] for t in layer):
        data[hole] = data[mover]


# ------------------------------------------------------------------------------------------------ what it costs
def work(case):
    op = case["op"]
    lens = _lengths(case)
    if op == "prompt":
        G, H = case["groups"], case["groups"] * case["heads"]
        keys = [n + p for n, p in zip(lens, _prefixes(case))]
        seen = sum(n * (k - n) + n * (n + 1) // 2 for n, k in zip(lens, keys))
        return {"bytes": float(sum(lens) * H * (4 * DIM + 4) + sum(keys) * 4 * G * DIM), "flops": float(4 * DIM * H * seen)}
    nb = [_blocks(n) for n in lens]
    width = max(1, max(nb))
    if op == "extend":
        was = _new_tokens(case)
        pages = sum(_blocks(a) for a, _ in was) + case["spare"]
        return {"bytes": float(8 * pages + 8 * width * len(lens) + 12 * len(lens)), "flops": float(pages + width * len(lens))}
    if op == "free":
        return {"bytes": float(8 * case["pages"] + 4 * len(lens) + 2 * sum(nb)), "flops": float(sum(nb) / 2)}
    page = case["groups"] * case["layers"] * 2 * (BLOCK * DIM + 1)  # bytes of a page in every buffer
    if op == "fork":
        pages, n = sum(nb) + case["children"] + 16, case["children"]
        parents = lens[:-1] if len(lens) >= 16 else lens
        tail = n * sum(x % BLOCK for x in parents) / len(parents)
        return {"bytes": float(8 * pages + 4 * sum(nb) + 4 * n * width + 2 * tail / BLOCK * page), "flops": float(n * width)}
    live = min(sum(nb), case["pages"])
    moved = live * (case["pages"] - live) / case["pages"]
    return {"bytes": float(12 * case["pages"] + 4 * sum(nb) + 4 * width * len(lens) + 2 * moved * page),
            "flops": float(case["pages"] + sum(nb))}


# ------------------------------------------------------------------------------------------------ in 64 bits
def exact(case, seed):
    """The attention by blocks of queries, every block against all keys before its last position.  The page operators
    give whole numbers and copies: none."""
    if case["op"] != "prompt" or work(case)["flops"] > 3e12:
        return None
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device=DEV)
    lse = torch.full(s["lse"].shape, -math.inf, dtype=torch.float64, device=DEV)
    cq, ck = s["cu_q"].tolist(), s["cu_k"].tolist()
    for b in range(case["batch"]):
        before = (ck[b + 1] - ck[b]) - (cq[b + 1] - cq[b])
        for t0 in range(cq[b], cq[b + 1], 1024):
            t1 = min(t0 + 1024, cq[b + 1])
            end = ck[b] + before + (t1 - cq[b])
            if end <= ck[b]:
                continue
            late = torch.arange(end - ck[b], device=DEV)[None, :] - torch.arange(t0 - cq[b], t1 - cq[b], device=DEV)[:, None] > before
            for h in range(s["q"].shape[1]):
                g = h // case["heads"]
                z = torch.einsum("td,jd->tj", s["q"][t0:t1, h].double(), s["k"][ck[b]:end, g].double()) / DIM ** 0.5
                z[late] = -math.inf
                norm = torch.logsumexp(z, dim=1)
                lse[t0:t1, h] = norm
                out[t0:t1, h] = torch.exp(z - norm[:, None]) @ s["v"][ck[b]:end, g].double()
    return {"out": out, "lse": lse}
