"""The page pool on the GPU against the plain definition, bit for bit: pages handed out, shared, given
back and moved, in the pools of FP8 and NVFP4 caches."""
import numpy as np
import pytest

from gpu_util import need_gpu
from oracle import pages as OP

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    need_gpu()


def dev(x):
    import torch
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


def host(t):
    return t.cpu().numpy()


class Pool:
    """Sequences that hold pages (some shared), a pool with its buffers on both sides."""

    def __init__(self, seed, lens, P, width=None, shared=0.0, caches=()):
        import torch
        import block_sparse_attention_indexer_gb300 as msa
        rng = self.rng = np.random.default_rng(seed)
        self.lens = np.array(lens, np.int32)
        nb = [OP.blocks(n) if n > 0 else 0 for n in lens]
        width = width or max(1, max(nb, default=1))
        self.table, self.refs = np.full((len(lens), width), -1, np.int32), np.zeros(P, np.int32)
        fresh = rng.permutation(P).tolist()
        for b, n in enumerate(nb):
            for j in range(n):
                used = np.flatnonzero(self.refs)
                page = int(rng.choice(used)) if len(used) and rng.random() < shared else fresh.pop()
                self.table[b, j] = page
                self.refs[page] += 1
        self.caches = []
        for kind, G in caches:
            c = msa.Fp8Cache(P, groups=G) if kind == "fp8" else msa.PagedCache(P, groups=G)
            for t in c.tensors():
                t.copy_(torch.from_numpy(rng.integers(0, 256, tuple(t.shape), dtype=np.uint8)))
            self.caches.append(c)
        self.buffers = [(host(t), None if t.dim() == 2 else t.dim() - 2) for c in self.caches for t in c.tensors()]
        self.d_refs, self.d_table, self.d_lens = dev(self.refs), dev(self.table), dev(self.lens)
        self.pool = msa.PagePool(self.caches, refs=self.d_refs)
        self.batch = msa.Batch(self.d_table, self.d_lens)
        self.ws = msa.alloc_page_workspace(self.pool, 2048)

    def err(self):
        import block_sparse_attention_indexer_gb300 as msa
        e = msa.msa_read_device_error(self.ws)
        msa.msa_clear_device_error(self.ws)
        return e

    def same_buffers(self):
        for t, (want, _) in zip([t for c in self.caches for t in c.tensors()], self.buffers, strict=True):
            assert np.array_equal(host(t), want)


def outs(p, rows, in_place):
    import torch
    if in_place:
        return dict()
    return dict(table_out=torch.full((rows, p.table.shape[1]), 77, dtype=torch.int32, device="cuda"),
                refs_out=torch.full((len(p.refs),), 77, dtype=torch.int32, device="cuda"))


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("lens,new,P,width", [
    ([0, 1, 127, 128, 129], [1, 1, 1, 1, 1], 10, 3),
    ([0, 0, 300, 5], [0, 1000, 84, 0], 30, 16),
    ([200] * 9, [3000] * 9, 160, 40),                     # the later ones find too few pages
    ([200, 10, 50, 70], [5000, 1, 5000, 118], 50, 64),    # a short need fits no more behind a long one
    ([100, -5, 900, 100], [29, 5, 500, -1], 40, 10),      # lengths and counts that cannot be
    ([0] * 2048, [1] * 2048, 5000, 2),
    ([100] * 1500, [200] * 1500, 4097, 3),
])
def test_extend(lens, new, P, width, in_place):
    import torch
    import block_sparse_attention_indexer_gb300 as msa
    p = Pool(len(lens) + P, lens, P, width)
    refs, table, out_lens, err = OP.extend(p.refs, p.table, p.lens, new)
    kw = outs(p, len(lens), in_place)
    if not in_place:
        kw["seq_lens_out"] = torch.full((len(lens),), 77, dtype=torch.int32, device="cuda")
    msa.msa_extend_pages(p.pool, p.batch, p.ws, new_tokens=dev(np.array(new, np.int32)), **kw)
    assert np.array_equal(host(kw.get("refs_out", p.d_refs)), refs)
    assert np.array_equal(host(kw.get("table_out", p.d_table)), table)
    assert np.array_equal(host(kw.get("seq_lens_out", p.d_lens)), out_lens)
    assert p.err() == err
    if not in_place:  # and the inputs as they were
        assert np.array_equal(host(p.d_refs), p.refs) and np.array_equal(host(p.d_table), p.table)


@pytest.mark.parametrize("P", [1, 3, 4, 5, 127, 128, 129, 1023, 32768, 32769, 524287, 524288, 524289, 1_200_003])
def test_extend_pool_sizes(P):
    """Pools of one round of the scan and of several, with free pages spread over all of it."""
    import block_sparse_attention_indexer_gb300 as msa
    p = Pool(P, [0, 0, 0], P, 1000)
    refs = p.rng.integers(0, 2, P).astype(np.int32) if P > 5 else np.zeros(P, np.int32)
    refs[-1] = 0
    # the last free page is handed out as well, but for the large pools
    free = int((refs == 0).sum())
    most = min(free, 3 * 1000)
    new = np.array([128 * min(most, 1000), 128 * min(max(most - 1000, 0), 1000), 128 * max(most - 2000, 0)], np.int32)
    if free > 3000:
        refs[np.flatnonzero(refs == 0)[:free - 3000]] = 1     # the free ones lie at the end
    p.d_refs.copy_(dev(refs))
    want = OP.extend(refs, p.table, p.lens, new)
    msa.msa_extend_pages(p.pool, p.batch, p.ws, new_tokens=dev(new))
    for got, x in zip((p.d_refs, p.d_table, p.d_lens), want):
        assert np.array_equal(host(got), x)
    assert p.err() == want[3] == 0


def test_extend_by_the_batch_length():
    import block_sparse_attention_indexer_gb300 as msa
    p = Pool(5, [0, 127, 500, 126], 40, 8)
    p.batch.q_len = 3
    want = OP.extend(p.refs, p.table, p.lens, [0, 3, 3, 3])
    msa.msa_extend_pages(p.pool, p.batch, p.ws)
    for got, x in zip((p.d_refs, p.d_table, p.d_lens), want):
        assert np.array_equal(host(got), x)


CACHES = [("fp8", 4)], [("nvfp4", 4)], [("fp8", 3), ("nvfp4", 1), ("fp8", 1)], []


@pytest.mark.parametrize("caches", CACHES)
@pytest.mark.parametrize("in_place", [True, False])
def test_fork(caches, in_place):
    import torch
    import block_sparse_attention_indexer_gb300 as msa
    p = Pool(21, [1, 128, 700, 0, 383, 127, 512], 48, 6, caches=caches)
    parents = np.array([2, 2, 0, 1, -1, 4, 3, 5, 6, 2, 0], np.int32)
    refs, table, lens, err = OP.fork(p.refs, p.table, p.lens, parents, p.buffers)
    kw = outs(p, len(parents), in_place)
    to = kw.pop("table_out", torch.full((len(parents), 6), 77, dtype=torch.int32, device="cuda"))
    out_lens = torch.full((len(parents),), 77, dtype=torch.int32, device="cuda")
    msa.msa_fork_pages(p.pool, p.batch, dev(parents), to, out_lens, p.ws, **kw)
    assert np.array_equal(host(kw.get("refs_out", p.d_refs)), refs)
    assert np.array_equal(host(to), table) and np.array_equal(host(out_lens), lens)
    assert p.err() == err == 0
    p.same_buffers()


def test_fork_refusals_on_the_device():
    """Parents and lengths out of range, bad entries, too few free pages."""
    import torch
    import block_sparse_attention_indexer_gb300 as msa
    p = Pool(22, [130, 300, 50, 260, 200, 20], 13, 3, caches=[("fp8", 2)])
    p.table[1, 1], p.table[2, 0], p.table[4, 1] = 13, -1, 1 << 30
    p.lens[3] = 385
    p.d_table.copy_(dev(p.table))
    p.d_lens.copy_(dev(p.lens))
    parents = np.array([0, 6, -2, 1, 2, 3, 4, 5, 0, 0, 5, 1 << 30], np.int32)
    refs, table, lens, err = OP.fork(p.refs, p.table, p.lens, parents, p.buffers)
    assert err == 0x33
    to = torch.full((len(parents), 3), 77, dtype=torch.int32, device="cuda")
    out_lens = torch.full((len(parents),), 77, dtype=torch.int32, device="cuda")
    msa.msa_fork_pages(p.pool, p.batch, dev(parents), to, out_lens, p.ws)
    assert p.err() == err
    assert np.array_equal(host(p.d_refs), refs) and np.array_equal(host(to), table) and np.array_equal(host(out_lens), lens)
    p.same_buffers()


def test_fork_many_buffers():
    """More buffers than one launch takes, and many children of one parent."""
    import torch
    import block_sparse_attention_indexer_gb300 as msa
    p = Pool(23, [200], 40, 2, caches=[("fp8", 1)] * 13 + [("nvfp4", 1)] * 4)
    assert len(p.buffers) == 76
    parents = np.zeros(30, np.int32)
    refs, table, lens, err = OP.fork(p.refs, p.table, p.lens, parents, p.buffers)
    to, out_lens = torch.empty(30, 2, dtype=torch.int32, device="cuda"), torch.empty(30, dtype=torch.int32, device="cuda")
    msa.msa_fork_pages(p.pool, p.batch, dev(parents), to, out_lens, p.ws)
    assert np.array_equal(host(p.d_refs), refs) and np.array_equal(host(to), table) and p.err() == 0
    p.same_buffers()


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("case", ["counts", "all", "twice", "bad", "empty"])
def test_free(case, in_place):
    import torch
    import block_sparse_attention_indexer_gb300 as msa
    p = Pool(31, [1000, 0, 300, 5000, 128], 60, 50, shared=0.4)
    pages, counts = p.table, np.array([8, 0, 3, 40, 1], np.int32)
    if case == "all":
        counts = None
    elif case == "twice":            # more references than there are, many of them at once
        pages = np.repeat(p.table, 3, axis=0)
        counts = None
    elif case == "bad":
        pages = pages.copy()
        pages[0, :3] = [60, -2, 1 << 30]
        counts = np.array([5, -1, 51, 2, 0], np.int32)
    elif case == "empty":
        pages, counts = np.zeros((0, 4), np.int32), None
    refs, err = OP.free(p.refs, pages, counts)
    out = None if in_place else torch.full((60,), 77, dtype=torch.int32, device="cuda")
    msa.msa_free_pages(p.pool, dev(pages), p.ws, counts=None if counts is None else dev(counts), refs_out=out)
    assert np.array_equal(host(p.d_refs if in_place else out), refs)
    assert p.err() == err == {"twice": 1, "bad": 3}.get(case, 0)


def test_free_hammered():
    """One page given back by every thread of a grid."""
    import torch
    import block_sparse_attention_indexer_gb300 as msa
    p = Pool(32, [1], 7, 1)
    p.d_refs.copy_(dev(np.array([5, 100_000, 0, 1, 1, 1, 1], np.int32)))
    pages = torch.ones(500, 333, dtype=torch.int32, device="cuda")
    pages[:, 0] = 2
    msa.msa_free_pages(p.pool, pages, p.ws)
    assert host(p.d_refs).tolist() == [5, 0, 0, 1, 1, 1, 1] and p.err() == 1


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("P,lens,shared,caches", [
    (64, [1000, 0, 300, 128, 2000], 0.0, [("fp8", 4)]),
    (64, [1000, 0, 300, 128, 2000], 0.5, [("nvfp4", 2), ("fp8", 3)]),
    (25, [3000, 20], 0.0, [("fp8", 1)]),               # full
    (9, [0, 0], 0.0, [("fp8", 1)]),                    # empty
    (5000, [128 * 40] * 50, 0.1, []),
    (1, [5], 0.0, [("nvfp4", 8)]),
])
def test_compact(P, lens, shared, caches, in_place):
    import torch
    import block_sparse_attention_indexer_gb300 as msa
    p = Pool(41 + P, lens, P, shared=shared, caches=caches)
    refs, table, page_map, n, err = OP.compact(p.refs, p.table, p.lens, p.buffers)
    kw = outs(p, len(lens), in_place)
    d_map, live = torch.full((P,), 77, dtype=torch.int32, device="cuda"), torch.full((1,), 77, dtype=torch.int32, device="cuda")
    msa.msa_compact_pages(p.pool, p.batch, d_map, live, p.ws, **kw)
    assert host(live)[0] == n and np.array_equal(host(d_map), page_map)
    assert np.array_equal(host(kw.get("refs_out", p.d_refs)), refs)
    assert np.array_equal(host(kw.get("table_out", p.d_table)), table)
    assert p.err() == err == 0
    p.same_buffers()


@pytest.mark.parametrize("P,density", [(524288, 0.5), (524289, 0.9), (1_300_001, 0.3), (600_000, 0.999)])
def test_compact_large_pools(P, density):
    import torch
    import block_sparse_attention_indexer_gb300 as msa
    p = Pool(P, [0], P, 1)
    refs = (p.rng.random(P) < density).astype(np.int32) * p.rng.integers(1, 4, P).astype(np.int32)
    used = np.flatnonzero(refs)
    p.d_refs.copy_(dev(refs))
    table = p.rng.choice(used, (64, 1000)).astype(np.int32)
    lens = np.full(64, 128 * 1000 - 5, np.int32)
    d_table = dev(table)
    d_map, live = torch.empty(P, dtype=torch.int32, device="cuda"), torch.empty(1, dtype=torch.int32, device="cuda")
    want = OP.compact(refs, table, lens)
    msa.msa_compact_pages(p.pool, msa.Batch(d_table, dev(lens)), d_map, live, p.ws)
    assert np.array_equal(host(p.d_refs), want[0]) and np.array_equal(host(d_table), want[1])
    assert np.array_equal(host(d_map), want[2]) and host(live)[0] == want[3] and p.err() == 0


def test_compact_bad_entries():
    import torch
    import block_sparse_attention_indexer_gb300 as msa
    p = Pool(51, [600, 300, 128, 40], 30, 5)
    p.table[0, 1], p.table[0, 2], p.table[1, 0] = -1, 30, int(np.flatnonzero(p.refs == 0)[0])
    p.table[3, 1:] = [5, 6, 7, 8]                   # behind the row's end
    p.lens[2] = -1
    p.d_table.copy_(dev(p.table))
    p.d_lens.copy_(dev(p.lens))
    want = OP.compact(p.refs, p.table, p.lens)
    d_map, live = torch.empty(30, dtype=torch.int32, device="cuda"), torch.empty(1, dtype=torch.int32, device="cuda")
    msa.msa_compact_pages(p.pool, p.batch, d_map, live, p.ws)
    assert np.array_equal(host(p.d_table), want[1]) and np.array_equal(host(p.d_refs), want[0])
    assert p.err() == want[4] == 3


def test_buffers_of_any_alignment():
    """FP8 scales of three heads at an odd address: pages of three bytes."""
    import torch
    import block_sparse_attention_indexer_gb300 as msa
    p = Pool(61, [200, 70, 128 * 9, 5], 40, 9, caches=[("fp8", 3)])
    c = p.caches[0]
    odd = [torch.empty(40 * 3 + 1, dtype=torch.uint8, device="cuda")[1:].view(40, 3) for _ in range(2)]
    for o, s in zip(odd, (c.k_scale, c.v_scale)):
        o.copy_(s)
    p.caches[0] = msa.Fp8Cache.from_tensors(c.k_data, odd[0], c.v_data, odd[1])
    pool = msa.PagePool(p.caches, refs=p.d_refs)
    refs, table, page_map, n, err = OP.compact(p.refs, p.table, p.lens, p.buffers)
    d_map, live = torch.empty(40, dtype=torch.int32, device="cuda"), torch.empty(1, dtype=torch.int32, device="cuda")
    msa.msa_compact_pages(pool, p.batch, d_map, live, p.ws)
    p.same_buffers()
    refs, table, lens, err = OP.fork(refs, table, p.lens, [0, 1, 3], p.buffers)
    to, out_lens = torch.empty(3, 9, dtype=torch.int32, device="cuda"), torch.empty(3, dtype=torch.int32, device="cuda")
    msa.msa_fork_pages(pool, p.batch, dev(np.array([0, 1, 3], np.int32)), to, out_lens, p.ws)
    p.same_buffers()
    assert np.array_equal(host(to), table) and np.array_equal(host(p.d_refs), refs)


def test_captured_life_of_a_pool():
    """Extend, fork, free and compact in one graph, replayed: every replay goes on from the last one's state."""
    import torch
    import block_sparse_attention_indexer_gb300 as msa
    p = Pool(71, [100, 250, 128], 64, 8, caches=[("fp8", 2)])
    parents = dev(np.array([1, 0, 1], np.int32))
    to, out_lens = torch.empty(3, 8, dtype=torch.int32, device="cuda"), torch.empty(3, dtype=torch.int32, device="cuda")
    d_map, live = torch.empty(64, dtype=torch.int32, device="cuda"), torch.empty(1, dtype=torch.int32, device="cuda")
    new = dev(np.array([60, 60, 60], np.int32))

    def step():
        msa.msa_extend_pages(p.pool, p.batch, p.ws, new_tokens=new)
        msa.msa_fork_pages(p.pool, p.batch, parents, to, out_lens, p.ws)
        msa.msa_free_pages(p.pool, p.d_table, p.ws)
        p.d_table.copy_(to)
        p.d_lens.copy_(out_lens)
        msa.msa_compact_pages(p.pool, p.batch, d_map, live, p.ws)

    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    refs, table, lens = p.refs, p.table, p.lens
    for _ in range(5):
        refs, table, lens, e = OP.extend(refs, table, lens, [60, 60, 60])
        refs, kids, kid_lens, f = OP.fork(refs, table, lens, [1, 0, 1], p.buffers)
        refs, h = OP.free(refs, table)
        refs, table, page_map, n, c = OP.compact(refs, kids, kid_lens, p.buffers)
        lens = kid_lens
        assert e == f == h == c == 0
        g.replay()
        assert np.array_equal(host(p.d_refs), refs) and np.array_equal(host(p.d_table), table)
        assert np.array_equal(host(p.d_lens), lens) and host(live)[0] == n and np.array_equal(host(d_map), page_map)
        p.same_buffers()
    assert p.err() == 0


def test_calls_with_nothing_in_them():
    """No sequences, no children, lists without columns: counts and maps are still what they should be."""
    import torch
    import block_sparse_attention_indexer_gb300 as msa
    p = Pool(81, [], 9, 4, caches=[("fp8", 1)])
    refs = np.array([0, 2, 0, 0, 1, 1, 0, 0, 3], np.int32)
    p.d_refs.copy_(dev(refs))
    i32 = dict(dtype=torch.int32, device="cuda")
    out = torch.full((9,), 77, **i32)
    msa.msa_extend_pages(p.pool, p.batch, p.ws, new_tokens=torch.empty(0, **i32), refs_out=out)
    assert np.array_equal(host(out), refs)
    q = Pool(82, [300, 5], 9, 4, caches=[("fp8", 1)])
    out.fill_(77)
    msa.msa_fork_pages(q.pool, q.batch, torch.empty(0, **i32), torch.empty(0, 4, **i32), torch.empty(0, **i32), q.ws, refs_out=out)
    assert np.array_equal(host(out), q.refs)
    out.fill_(77)
    msa.msa_free_pages(p.pool, torch.empty(3, 0, **i32), p.ws, refs_out=out)
    assert np.array_equal(host(out), refs)
    want = OP.compact(refs, p.table, p.lens, p.buffers)
    d_map, live = torch.empty(9, **i32), torch.empty(1, **i32)
    msa.msa_compact_pages(p.pool, p.batch, d_map, live, p.ws)
    assert np.array_equal(host(p.d_refs), want[0]) and np.array_equal(host(d_map), want[2]) and host(live)[0] == want[3] == 4
    p.same_buffers()
    assert p.err() == q.err() == 0


@pytest.mark.parametrize("P", [1, 2, 2047, 2048, 2049, 4096])
@pytest.mark.parametrize("used", ["none", "all", "last"])
def test_compact_pools_at_the_ends(P, used):
    import torch
    import block_sparse_attention_indexer_gb300 as msa
    p = Pool(83, [128, 0], P, 2)
    refs = np.full(P, 2 if used == "all" else 0, np.int32)
    refs[-1] = 0 if used == "none" else 5
    p.table[0, 0] = P - 1
    if used == "none":
        p.lens[0] = 0
    p.d_refs.copy_(dev(refs))
    p.d_table.copy_(dev(p.table))
    p.d_lens.copy_(dev(p.lens))
    want = OP.compact(refs, p.table, p.lens)
    d_map, live = torch.empty(P, dtype=torch.int32, device="cuda"), torch.empty(1, dtype=torch.int32, device="cuda")
    msa.msa_compact_pages(p.pool, p.batch, d_map, live, p.ws)
    for got, x in zip((p.d_refs, p.d_table, d_map), want):
        assert np.array_equal(host(got), x)
    assert host(live)[0] == want[3] and p.err() == want[4] == 0


def test_two_pools_at_once_on_their_own_streams():
    import torch
    import block_sparse_attention_indexer_gb300 as msa
    pools = [Pool(84 + i, [700, 90, 1000, 3], n, 32, shared=0.2, caches=[("fp8", 2)]) for i, n in enumerate((60, 4100))]
    streams = [torch.cuda.Stream() for _ in pools]
    new, parents = np.array([300, 300, 1, 500], np.int32), np.array([2, 1, 1, 0, 3], np.int32)
    space = [dict(to=torch.empty(5, 32, dtype=torch.int32, device="cuda"), lens=torch.empty(5, dtype=torch.int32, device="cuda"),
                  map=torch.empty(len(p.refs), dtype=torch.int32, device="cuda"), live=torch.empty(1, dtype=torch.int32, device="cuda"),
                  new=dev(new), parents=dev(parents)) for p in pools]
    torch.cuda.synchronize()
    for step in range(4):
        for p, x, s in zip(pools, space, streams):
            if step == 0:
                msa.msa_extend_pages(p.pool, p.batch, p.ws, new_tokens=x["new"], stream=s)
            elif step == 1:
                msa.msa_fork_pages(p.pool, p.batch, x["parents"], x["to"], x["lens"], p.ws, stream=s)
            elif step == 2:
                msa.msa_free_pages(p.pool, p.d_table, p.ws, stream=s)
            else:
                msa.msa_compact_pages(p.pool, msa.Batch(x["to"], x["lens"]), x["map"], x["live"], p.ws, stream=s)
    torch.cuda.synchronize()
    for p, x in zip(pools, space):
        refs, table, lens, e = OP.extend(p.refs, p.table, p.lens, new)
        refs, kids, kid_lens, f = OP.fork(refs, table, lens, parents, p.buffers)
        refs, g = OP.free(refs, table)
        refs, kids, page_map, n, h = OP.compact(refs, kids, kid_lens, p.buffers)
        assert e == f == g == h == p.err() == 0
        assert np.array_equal(host(p.d_refs), refs) and np.array_equal(host(x["to"]), kids)
        assert np.array_equal(host(x["lens"]), kid_lens) and np.array_equal(host(x["map"]), page_map) and host(x["live"])[0] == n
        p.same_buffers()


@pytest.mark.parametrize("width", [1_200_000_000, 2 ** 31 - 1])
def test_free_of_long_rows(width):
    """Rows of more than 2^30 entries: the place behind the last one and the grid's step together pass 2^31."""
    import torch
    import block_sparse_attention_indexer_gb300 as msa
    p = Pool(91, [128 * 20], 30, 20)
    p.d_refs.copy_(dev(np.full(30, 9, np.int32)))
    pages = torch.full((1, width), -1, dtype=torch.int32, device="cuda")
    want = np.full(30, 9, np.int32)
    for at in (0, 255, 1023, 1024, 2 ** 30 - 1, 2 ** 30, width - 1025, width - 257, width - 2):
        pages[0, at] = at % 30
        want[at % 30] -= 1
    pages[0, width - 1] = 30                                   # behind the row's count
    msa.msa_free_pages(p.pool, pages, p.ws, counts=dev(np.array([width - 1], np.int32)))
    assert np.array_equal(host(p.d_refs), want) and p.err() == 0
    msa.msa_free_pages(p.pool, pages, p.ws)
    for at in (0, 255, 1023, 1024, 2 ** 30 - 1, 2 ** 30, width - 1025, width - 257, width - 2):
        want[at % 30] -= 1
    assert np.array_equal(host(p.d_refs), want) and p.err() == 1


@pytest.mark.parametrize("page", [2 ** 31 - 1, 2 ** 31 - 16384, 2 ** 31 - 16383])
def test_pages_of_two_gigabytes(page):
    """Pages whose bytes and a copy's piece together pass 2^31, moved by a compaction and copied by a fork."""
    import torch
    import block_sparse_attention_indexer_gb300 as msa

    class Pages:                                               # what a pool asks of a cache
        num_pages = 3
        data = torch.zeros(3, page, dtype=torch.uint8, device="cuda")

        def tensors(self):
            return (self.data,)

    cache = Pages()
    data, marks = cache.data, [0, 16383, 16384, 2 ** 30, page - 16384, page - 2, page - 1]
    data[2, :] = 9
    data[2, marks] = torch.arange(1, 8, dtype=torch.uint8, device="cuda")
    want = data[2].clone()
    pool = msa.PagePool([cache], refs=dev(np.array([0, 0, 1], np.int32)))
    table, lens = dev(np.array([[2]], np.int32)), dev(np.array([5], np.int32))
    batch, ws = msa.Batch(table, lens), msa.alloc_page_workspace(pool, 1)
    page_map, live = torch.empty(3, dtype=torch.int32, device="cuda"), torch.empty(1, dtype=torch.int32, device="cuda")
    msa.msa_compact_pages(pool, batch, page_map, live, ws)
    assert host(page_map).tolist() == [-1, -1, 0] and host(table).tolist() == [[0]] and host(live).tolist() == [1]
    assert torch.equal(data[0], want)
    kids, kid_lens = torch.empty(1, 1, dtype=torch.int32, device="cuda"), torch.empty(1, dtype=torch.int32, device="cuda")
    msa.msa_fork_pages(pool, batch, dev(np.array([0], np.int32)), kids, kid_lens, ws)
    assert host(kids).tolist() == [[1]] and host(pool.refs).tolist() == [1, 1, 0]
    assert torch.equal(data[1], want) and msa.msa_read_device_error(ws) == 0


def test_counts_and_tensors_replaced_between_calls():
    """A program that goes on from a call's refs_out as the pool's counts, and with other tensors in a cache."""
    import torch
    import block_sparse_attention_indexer_gb300 as msa
    p = Pool(92, [700, 90, 300], 40, 8, caches=[("nvfp4", 2), ("fp8", 1)])
    new, out = np.array([200, 60, 1], np.int32), torch.empty(40, dtype=torch.int32, device="cuda")
    msa.msa_extend_pages(p.pool, p.batch, p.ws, new_tokens=dev(new), refs_out=out)
    refs, table, lens, err = OP.extend(p.refs, p.table, p.lens, new)
    assert np.array_equal(host(out), refs) and np.array_equal(host(p.d_refs), p.refs)
    p.pool.refs = out
    msa.msa_extend_pages(p.pool, p.batch, p.ws, new_tokens=dev(new))
    refs, table, lens, err2 = OP.extend(refs, table, lens, new)
    assert np.array_equal(host(out), refs) and np.array_equal(host(p.d_table), table)
    assert np.array_equal(host(p.d_refs), p.refs)                               # the first counts are left alone
    old, p.caches[0].k_data = p.caches[0].k_data, p.caches[0].k_data.clone()
    before = old.clone()
    parents = np.array([1, 1, 0, 2], np.int32)
    refs, kids, kid_lens, err3 = OP.fork(refs, table, lens, parents, p.buffers)
    to, to_lens = torch.empty(4, 8, dtype=torch.int32, device="cuda"), torch.empty(4, dtype=torch.int32, device="cuda")
    msa.msa_fork_pages(p.pool, p.batch, dev(parents), to, to_lens, p.ws)
    assert np.array_equal(host(out), refs) and np.array_equal(host(to), kids) and err == err3 == 0
    assert p.err() == err2 == OP.BAD_SEQLEN                                     # (the first one has no room for 200 more)
    p.same_buffers()
    assert torch.equal(old, before)


# One launch up to 2,048 pages and 8,192 copied entries of a table, two beyond.
@pytest.mark.parametrize("P", [2047, 2048, 2049, 4096, 4097])
@pytest.mark.parametrize("rows,width", [(64, 128), (3, 2731), (129, 64), (1, 1)])
@pytest.mark.parametrize("in_place", [True, False])
def test_extend_and_fork_around_one_launch(P, rows, width, in_place):
    import torch
    import block_sparse_attention_indexer_gb300 as msa
    p = Pool(P + rows, [0] * rows, P, width, caches=[("fp8", 1)])
    refs = p.rng.integers(0, 3, P).astype(np.int32)
    refs[-2:] = 0                                               # the last free pages are handed out as well
    lens = p.rng.integers(0, width * 64, rows).astype(np.int32)
    table = p.rng.integers(0, P, (rows, width)).astype(np.int32)
    free, new = int((refs == 0).sum()), np.zeros(rows, np.int32)
    for b in range(rows):                                       # as many tokens as there are pages for, the first row the most
        blocks = min(free, width - OP.blocks(lens[b]), free if b == 0 else 7)
        new[b] = blocks * 128
        free -= blocks
    p.d_refs.copy_(dev(refs))
    p.d_table.copy_(dev(table))
    p.d_lens.copy_(dev(lens))
    want = OP.extend(refs, table, lens, new)
    kw = outs(p, rows, in_place)
    if not in_place:
        kw["seq_lens_out"] = torch.full((rows,), 77, dtype=torch.int32, device="cuda")
    msa.msa_extend_pages(p.pool, p.batch, p.ws, new_tokens=dev(new), **kw)
    for got, x in zip((kw.get("refs_out", p.d_refs), kw.get("table_out", p.d_table), kw.get("seq_lens_out", p.d_lens)), want):
        assert np.array_equal(host(got), x)
    assert p.err() == want[3] == 0
    # children of the rows as they were, every row once and the first ones again; the counts as they were
    parents = (np.arange(rows + 5) % rows).astype(np.int32)
    refs[:] = np.where(p.rng.random(P) < 0.9, np.maximum(refs, 1), 0)
    refs[-2:] = 0
    table = p.rng.choice(np.flatnonzero(refs), (rows, width)).astype(np.int32)
    p.d_refs.copy_(dev(refs))
    p.d_table.copy_(dev(table))
    p.d_lens.copy_(dev(lens))
    refs, kids, kid_lens, err = OP.fork(refs, table, lens, parents, p.buffers)
    to, out_lens = torch.empty(rows + 5, width, dtype=torch.int32, device="cuda"), torch.empty(rows + 5, dtype=torch.int32, device="cuda")
    kw = {k: v for k, v in outs(p, rows, in_place).items() if k == "refs_out"}
    msa.msa_fork_pages(p.pool, p.batch, dev(parents), to, out_lens, p.ws, **kw)
    assert np.array_equal(host(kw.get("refs_out", p.d_refs)), refs) and p.err() == err
    assert np.array_equal(host(to), kids) and np.array_equal(host(out_lens), kid_lens)
    p.same_buffers()
