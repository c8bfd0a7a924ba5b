"""The packed prompt attention and the page pool without a GPU: workspace sizes, refusals before any
CUDA call, the binding's checks, and small pins of the plain definitions."""
import ctypes

import numpy as np
import pytest

from oracle import pages as OP
from oracle import prompt as OQ


@pytest.fixture(scope="module")
def msa():
    import __graft_entry__
    __graft_entry__.build()
    import block_sparse_attention_indexer_gb300 as msa
    return msa


P = 1 << 30  # stands for a device address: never followed, every call below is refused before a launch
r = ctypes.byref


def test_prompt_workspace(msa):
    b = msa.binding
    cfg = b._Config(4, 8, 128, 128, 128, 16, 0, 1, 0.0)
    f = lambda c, p: b._lib.msa_prompt_workspace_bytes(r(c), p and r(p))  # noqa: E731
    assert f(cfg, b._Packed(P, P, 3, 1000, 1000)) >= 256
    assert f(cfg, b._Packed(P, P, 3, 200_000, 200_000)) >= f(cfg, b._Packed(P, P, 3, 1000, 1000))
    assert f(cfg, None) == f(cfg, b._Packed(None, P, 3, 5, 5)) == f(cfg, b._Packed(P, P, -1, 5, 5)) == 0
    assert f(b._Config(4, 9, 128, 128, 128, 16, 0, 1, 0.0), b._Packed(P, P, 3, 5, 5)) == 0
    assert f(cfg, b._Packed(P, P, 2049, 5, 5)) == f(cfg, b._Packed(P, P, 1, 1 << 29, 5)) == 0


def test_prompt_refusals(msa):
    b = msa.binding
    L = b._lib
    cfg = b._Config(4, 8, 128, 128, 128, 16, 0, 1, 0.0)
    pk = b._Packed(P, P, 2, 100, 200)
    far = 1 << 40

    def call(cfg=cfg, pk=pk, q=P, qs=4096, k=2 * P, ks=512, v=3 * P, vs=512, out=far, lse=None, ws=P, n=1 << 40):
        return L.msa_prompt_attn(cfg and r(cfg), pk and r(pk), q, qs, k, ks, v, vs, out, lse, ws, n, None)

    assert call(cfg=None) == call(pk=None) == 1
    assert call(cfg=b._Config(9, 8, 128, 128, 128, 16, 0, 1, 0.0)) == call(cfg=b._Config(4, 8, 64, 128, 128, 16, 0, 1, 0.0)) == 2
    assert call(pk=b._Packed(None, P, 2, 100, 200)) == call(pk=b._Packed(P, None, 2, 100, 200)) == 1
    assert call(pk=b._Packed(P, P, 2, -1, 200)) == call(pk=b._Packed(P, P, 2, 100, -200)) == 1
    assert call(pk=b._Packed(P, P, 2049, 100, 200)) == call(pk=b._Packed(P, P, 2, 1 << 29, 200)) == 2
    assert call(pk=b._Packed(P, P, 2, 1 << 23, 1 << 23)) == 2          # more steps than 31 bits count
    assert call(q=None) == call(k=None) == call(v=None) == call(out=None) == 1
    assert call(q=P + 8) == call(k=P + 2) == call(v=P + 4) == call(out=far + 8) == 1
    assert call(qs=4088) == call(qs=4100) == call(ks=504) == call(vs=0) == call(vs=-512) == call(ks=516) == 1
    assert call(out=P) == call(out=P + 99 * 4096 * 2) == call(out=2 * P) == call(out=3 * P + 4096) == 1      # over an input
    assert call(lse=P) == call(lse=far + 4096) == 1
    assert call(ws=None) == call(n=255) == call(ws=P + 8) == 3
    # nothing to do
    assert call(pk=b._Packed(None, None, 0, 100, 200)) == call(pk=b._Packed(P, P, 2, 0, 200), q=None, out=None, ws=None) == 0


def _pool(b, buffers=(), refs=P, out=None, pages=1000):
    arr = (b._PageBuffer * max(1, len(buffers)))(*buffers)
    return b._PagePool(refs, refs if out is None else out, pages, arr, len(buffers))


def test_pool_refusals(msa):
    b = msa.binding
    f = lambda p, rows=8: b._lib.msa_page_workspace_bytes(p and r(p), rows)  # noqa: E731
    B = b._PageBuffer
    assert f(_pool(b)) >= 256 and f(_pool(b, [B(P, 512, 4), B(P + 1, 3, 0)])) >= 256
    assert f(_pool(b, pages=100_000)) > f(_pool(b)) and f(_pool(b), 2000) > f(_pool(b), 2)
    assert f(None) == f(_pool(b), -1) == f(_pool(b, pages=0)) == f(_pool(b, pages=(1 << 27) + 1)) == 0
    assert f(_pool(b, refs=None)) == f(_pool(b, refs=P + 4)) == f(_pool(b, out=P + 8)) == 0
    assert f(_pool(b, [B(None, 512, 4)])) == f(_pool(b, [B(P, 0, 0)])) == f(_pool(b, [B(P, 512, -1)])) == 0
    assert f(_pool(b, [B(P, 1 << 31, 0)])) == f(_pool(b, [B(P, 512, 3)])) == f(_pool(b, [B(P, 100, 4)])) == 0
    bad = b._PagePool(P, P, 10, None, 1)
    assert f(bad) == 0 and f(b._PagePool(P, P, 10, None, -1)) == 0 and f(b._PagePool(P, P, 10, None, 0)) >= 256


def test_extend_fork_refusals(msa):
    b = msa.binding
    L = b._lib
    pool, bt = _pool(b), b._Batch(2 * P, 3 * P, 4, 100, 1)
    n = 1 << 40

    def extend(pool=pool, bt=bt, new=4 * P, to=5 * P, lens=6 * P, ws=P, n=n):
        return L.msa_extend_pages(pool and r(pool), bt and r(bt), new, to, lens, ws, n, None)

    assert extend(pool=None) == extend(bt=None) == extend(to=None) == extend(lens=None) == 1
    assert extend(bt=b._Batch(2 * P, 3 * P, 2049, 100, 1)) == extend(bt=b._Batch(2 * P, 3 * P, 2048, 1 << 21, 1)) == 2
    assert extend(to=3 * P) == extend(lens=2 * P) == extend(to=4 * P) == extend(to=6 * P) == extend(lens=4 * P) == 1
    assert extend(to=2 * P + 4) == extend(to=P + 64) == extend(pool=_pool(b, out=P + 16)) == extend(pool=_pool(b, out=2 * P)) == 1
    assert extend(ws=None) == extend(n=300) == extend(ws=P + 8) == 3

    def fork(pool=pool, bt=bt, parents=4 * P, n_kids=8, to=5 * P, lens=6 * P, ws=P, n=n):
        return L.msa_fork_pages(pool and r(pool), bt and r(bt), parents, n_kids, to, lens, ws, n, None)

    assert fork(pool=None) == fork(bt=None) == fork(parents=None) == fork(to=None) == fork(lens=None) == fork(n_kids=-1) == 1
    assert fork(n_kids=2049) == 2
    assert fork(to=2 * P) == fork(lens=3 * P) == fork(to=4 * P) == fork(lens=5 * P + 400) == fork(pool=_pool(b, out=6 * P)) == 1
    assert fork(ws=None) == fork(n=300) == 3


def test_free_compact_refusals(msa):
    b = msa.binding
    L = b._lib
    pool, n = _pool(b), 1 << 40

    def free(pool=pool, pages=2 * P, counts=3 * P, rows=4, width=100, ws=P, n=n):
        return L.msa_free_pages(pool and r(pool), pages, counts, rows, width, ws, n, None)

    assert free(pool=None) == free(pages=None) == free(rows=-1) == free(width=-1) == 1
    assert free(rows=1 << 16, width=1 << 16) == 2
    assert free(pages=P) == free(counts=P + 3996) == free(pool=_pool(b, out=2 * P)) == 1
    assert free(ws=None) == free(n=300) == 3
    bt = b._Batch(2 * P, 3 * P, 4, 100, 1)

    def compact(pool=pool, bt=bt, to=2 * P, page_map=4 * P, live=5 * P, ws=P, n=n):
        return L.msa_compact_pages(pool and r(pool), bt and r(bt), to, page_map, live, ws, n, None)

    assert compact(pool=None) == compact(bt=None) == compact(to=None) == compact(page_map=None) == compact(live=None) == 1
    assert compact(to=3 * P) == compact(to=2 * P + 4) == compact(page_map=2 * P) == compact(page_map=P) == compact(live=4 * P) == 1
    assert compact(ws=None) == compact(n=300) == 3


def test_binding_checks(msa):
    import torch
    cpu = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError):
        msa.PagePool(refs=cpu)
    with pytest.raises(ValueError):
        msa.Packed(cpu, cpu, 3, 3).c()
    with pytest.raises(ValueError):
        msa.PagePool()
    x = torch.zeros(4, 16, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        msa.msa_prompt_attn(msa.Config(), msa.Packed(cpu, cpu, 4, 4), x, x, x, x, None, cpu)


def test_oracle_prompt_pins():
    rng = np.random.default_rng(0)
    q, k, v = rng.normal(size=(5, 2, 128)), rng.normal(size=(7, 1, 128)), rng.normal(size=(7, 1, 128))
    got = OQ.attention(q, k, v, [0, 2, 5], [0, 1, 7], 2, 0.1)
    assert (got["out"][0] == 0).all() and np.isneginf(got["lse"][0]).all()      # two queries, one key
    assert np.allclose(got["out"][1], v[0, 0])
    z = 0.1 * q[2, 1] @ k[1:5, 0].T                                             # first of three queries over six keys
    p = np.exp(z) / np.exp(z).sum()
    assert np.allclose(got["out"][2, 1], p @ v[1:5, 0]) and np.allclose(got["lse"][2, 1], np.log(np.exp(z).sum()))


def test_oracle_pages_pins():
    refs = np.array([1, 0, 2, 0, 1, 0], np.int32)
    table, lens = np.array([[2, 0, -1], [2, 4, -1]], np.int32), np.array([200, 256], np.int32)
    got = OP.extend(refs, table, lens, [56, 1])
    assert got[0].tolist() == [1, 1, 2, 0, 1, 0] and got[1].tolist() == [[2, 0, -1], [2, 4, 1]]
    assert got[2].tolist() == [256, 257] and got[3] == 0
    assert OP.extend(refs, table, lens, [57, 128])[1].tolist() == [[2, 0, 1], [2, 4, 3]]
    data = np.arange(6 * 128).reshape(6, 128, 1)
    got = OP.fork(refs, table, lens, [0, 1, 0], [(data, 1)])
    assert got[0].tolist() == [1, 1, 5, 1, 2, 0] and got[1].tolist() == [[2, 1, -1], [2, 4, -1], [2, 3, -1]]
    assert (data[1, :72, 0] == np.arange(72)).all() and data[1, 72, 0] == 128 + 72
    assert OP.free(refs, np.array([[2, 2, 2, 0]], np.int32)) [0].tolist() == [0, 0, 0, 0, 1, 0]
    got = OP.compact(refs, table, lens)
    assert got[0].tolist() == [1, 1, 2, 0, 0, 0] and got[1].tolist() == [[2, 0, -1], [2, 1, -1]] and got[3] == 3


def test_pool_goes_by_its_present_tensors(msa, monkeypatch):
    """Counts and caches' tensors that were replaced after the pool was made: the next call's struct has the new ones, and
    what the struct points to stays alive."""
    import gc
    import weakref

    import torch
    monkeypatch.setattr(msa.binding, "_on", lambda t, name: t.get_device())     # tensors of the host stand for the device's
    cache, other = msa.PagedCache(5, groups=2, device="cpu"), msa.PagedCache(5, groups=1, device="cpu")
    pool = msa.PagePool([cache, other], refs=torch.zeros(5, dtype=torch.int32))
    new = torch.ones(5, dtype=torch.int32)
    pool.refs = new
    c = pool.c()._obj
    assert pool.refs is new and c.refs == c.refs_out == new.data_ptr()
    out = torch.empty(5, dtype=torch.int32)
    c = pool.c(out, True)._obj
    assert c.refs == new.data_ptr() and c.refs_out == out.data_ptr()
    for bad, error in ((torch.ones(4, dtype=torch.int32), ValueError), (torch.ones(5), TypeError),
                       (torch.ones(10, dtype=torch.int32)[::2], ValueError)):
        with pytest.raises(error):
            pool.refs = bad
    assert pool.refs is new and pool.c()._obj.refs == new.data_ptr()

    at = lambda: [(b.data, b.page_bytes, b.token_bytes) for b in (pool.c(None, True)._obj.buffers[i] for i in range(12))]  # noqa: E731
    want = lambda: [(t.data_ptr(), t.numel() // 5, t.shape[-1]) for k in (cache, other) for t in k.tensors()]  # noqa: E731
    assert at() == want()
    old = weakref.ref(cache.v_data)
    cache.v_data = cache.v_data.clone()
    gc.collect()
    assert old() is not None                                                    # the pool's struct still has it
    assert at() == want() and pool.c(out, True)._obj.buffers[2].data == cache.v_data.data_ptr()
    gc.collect()
    assert old() is None
    cache.k_scale = torch.zeros(4, 2, 128, 8, dtype=torch.uint8)
    with pytest.raises(ValueError):
        pool.c(None, True)


@pytest.mark.parametrize("G,Hg,batch", [(4, 8, 1), (8, 4, 1), (8, 8, 3), (1, 1, 1), (2, 3, 700)])
def test_prompt_limit(msa, G, Hg, batch):
    """Tokens that a call may have, from the formula in msa.h: the last number that is taken and the first that is not."""
    b = msa.binding
    cfg = b._Config(G, Hg, 128, 128, 128, 16, 0, 1, 0.0)
    taken = lambda q, k: b._lib.msa_prompt_workspace_bytes(r(cfg), r(b._Packed(P, P, batch, q, k))) > 0  # noqa: E731
    fits = lambda q, k: G * (q // (2 * (128 // Hg)) + batch) * (2 * max(1, -(-k // 128)) + 4) <= 2 ** 31 - 1  # noqa: E731
    for both in (True, False):               # as many keys as queries; no keys
        lo, hi = 1, 1 << 28
        while lo < hi:
            mid = (lo + hi + 1) // 2
            lo, hi = (mid, hi) if fits(mid, mid if both else 0) else (lo, mid - 1)
        assert taken(lo, lo if both else 0) and not taken(lo + 1, lo + 1 if both else 0)
        if both and G * Hg == 32:
            assert 1_045_000 < lo < 1_050_000
