"""The FP8 entry points without a GPU: workspace sizes, refusals before any CUDA call, and the
binding's checks of shapes, types and strides."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def msa():
    import __graft_entry__
    __graft_entry__.build()
    import block_sparse_attention_indexer_gb300 as msa
    return msa


P = 1 << 20  # stands for a device address: never followed, every call below is refused before a launch


def _parts(msa):
    b = msa.binding
    cfg = b._Config(4, 8, 128, 128, 128, 16, 0, 1, 0.0)
    return b, b._lib, cfg, b._Fp8Cache(P, P, P, P, 10), b._Batch(P, P, 2, 8, 3)


def test_workspace_sizes(msa):
    b, L, cfg, _, bt = _parts(msa)
    f = lambda op, c=cfg, t=bt: L.msa_workspace_bytes(op, ctypes.byref(c), ctypes.byref(t))  # noqa: E731
    assert f(msa.MSA_OP_FP8_APPEND) == f(msa.MSA_OP_EVICT) == 256
    plain, more = f(msa.MSA_OP_FP8_ATTN), f(msa.MSA_OP_FP8_ATTN_WEIGHTS)
    assert 256 <= plain < more
    longer = b._Batch(P, P, 2, 4000, 3)
    assert f(msa.MSA_OP_FP8_ATTN, t=longer) == plain and f(msa.MSA_OP_FP8_ATTN_WEIGHTS, t=longer) > more
    bad = b._Config(4, 9, 128, 128, 128, 16, 0, 1, 0.0)
    assert all(f(op, bad) == 0 for op in range(4, 8)) and f(8) == 0


def test_append_refusals(msa):
    b, L, cfg, ca, bt = _parts(msa)
    r = ctypes.byref

    def call(cfg=cfg, ca=ca, bt=bt, k=P, v=P, t=0, ks=512, vs=512, ws=P, n=256):
        return L.msa_fp8_append(cfg and r(cfg), ca and r(ca), bt and r(bt), k, v, t, ks, vs, ws, n, None)

    assert call(cfg=None) == call(ca=None) == call(bt=None) == 1
    assert call(cfg=b._Config(4, 8, 64, 128, 128, 16, 0, 1, 0.0)) == 2
    assert call(t=2) == call(t=-1) == 2
    assert call(k=None) == call(v=None) == call(k=P + 8) == call(v=P + 4) == 1
    assert call(ks=511) == call(ks=514) == call(vs=0) == call(vs=-512) == 1
    assert call(t=1, ks=516) == 1 and call(t=1, vs=516) == 1          # 1032 bytes: not a multiple of 16
    assert call(ca=b._Fp8Cache(P, P, P, P, 0)) == call(ca=b._Fp8Cache(P + 1, P, P, P, 10)) == 1
    assert call(ca=b._Fp8Cache(P, None, P, P, 10)) == call(ca=b._Fp8Cache(P, P, P, P, 1 << 31)) == 1
    assert call(bt=b._Batch(P, P, 2, 8, 0)) == call(bt=b._Batch(None, P, 2, 8, 1)) == 1
    assert call(bt=b._Batch(P, P, 2049, 8, 1)) == call(bt=b._Batch(P, P, 2, 8, 32768)) == 2
    assert call(ws=None) == call(n=255) == call(ws=P + 8) == 3
    assert call(bt=b._Batch(None, None, 0, 8, 1), k=None, v=None, ws=None) == 0   # nothing to do


def test_attention_refusals(msa):
    b, L, cfg, ca, bt = _parts(msa)
    r = ctypes.byref
    need = L.msa_workspace_bytes(msa.MSA_OP_FP8_ATTN, r(cfg), r(bt))
    need_w = L.msa_workspace_bytes(msa.MSA_OP_FP8_ATTN_WEIGHTS, r(cfg), r(bt))

    def call(cfg=cfg, ca=ca, bt=bt, q=P, t=2, qs=4096, sel=None, out=P, win=None, decay=1.0, wout=None, ws=P, n=1 << 40):
        return L.msa_fp8_attn(cfg and r(cfg), ca and r(ca), bt and r(bt), q, t, qs, sel, out, None, win, decay, wout, ws,
                              n, None)

    assert call(cfg=None) == call(ca=None) == call(bt=None) == call(q=None) == call(out=None) == 1
    assert call(t=0) == call(t=3) == 2
    assert call(q=P + 8) == call(qs=4095) == call(qs=4104) == call(out=P + 2) == 1
    assert call(t=1, qs=4100) == 1
    assert call(ca=b._Fp8Cache(P, P, P, P, (1 << 22) + 1)) == 2       # 4 heads: past 2^24 page heads
    assert call(decay=-0.1, wout=P) == call(decay=1.5, wout=P) == call(decay=float("nan"), wout=P) == 1
    assert call(win=P) == 1                                           # weights in, nowhere to put them
    assert call(win=P, wout=P + 32) == 1                              # overlapping by half
    assert call(n=need - 1) == call(ws=None) == call(ws=P + 4) == call(wout=P, n=need_w - 1) == 3
    assert call(bt=b._Batch(None, None, 0, 8, 1), q=None, out=None, ws=None) == 0


def test_evict_refusals(msa):
    b, L, _, _, bt = _parts(msa)
    r = ctypes.byref
    step = 1 << 12
    names = ["weight", "table_out", "lens_out", "weight_out", "freed", "count"]

    def call(bt=b._Batch(P, P + step, 2, 8, 1), budget=4, first=1, last=1, ws=P - 1024, n=256, **at):
        p = {m: P + step * (2 + i) for i, m in enumerate(names)} | at
        return L.msa_evict_blocks(r(bt), p["weight"], budget, first, last, *(p[m] for m in names[1:]), ws, n, None)

    assert call(first=-1) == call(last=0) == call(budget=1) == call(first=2 ** 31 - 1, last=2 ** 31 - 1) == 1
    for m in names:
        assert call(**{m: None}) == 1
    assert call(table_out=P + 4) == call(table_out=P + step) == call(weight_out=P) == 1
    assert call(freed=P) == call(freed=P + 2 * step) == call(count=P + step) == call(lens_out=P + 2 * step + 4) == 1
    assert call(freed=P + 3 * step) == 1                              # the same place as table_out
    assert call(ws=None) == call(n=8) == call(ws=P + 4) == 3
    assert call(bt=b._Batch(P, P, 5000, 8, 1)) == 2
    assert call(bt=b._Batch(None, None, 0, 8, 1)) == 0


class _Dev:
    """A tensor's shape, type and strides as if it were on a device (nothing is followed)."""

    is_cuda = True

    def __init__(self, t, dev=0):
        self.t, self.shape, self.dtype, self.dev, self.device = t, t.shape, t.dtype, dev, f"cuda:{dev}"

    def __getattr__(self, name):
        return getattr(self.t, name)

    def get_device(self):
        return self.dev

    def data_ptr(self):
        return 64


def test_binding_checks_strides(msa):
    import torch
    f = msa.binding._token_rows
    with pytest.raises(ValueError, match="device"):
        f(torch.zeros(2, 3, 4, 128), (2, 3, 4, 128), 0, "k")
    with pytest.raises(ValueError, match="device 0"):
        f(_Dev(torch.zeros(2, 3, 4, 128), 1), (2, 3, 4, 128), 0, "k")
    wide = torch.zeros(2, 5, 8, 128)
    assert f(_Dev(wide), (2, 5, 8, 128), 0, "k") == (64, 1024)
    assert f(_Dev(wide[:, :, 4:]), (2, 5, 4, 128), 0, "k") == (64, 1024)
    assert f(_Dev(wide[:, :1]), (2, 1, 8, 128), 0, "k") == (64, 5120)
    assert f(_Dev(wide[:1, :1]), (1, 1, 8, 128), 0, "k") == (64, 1024)
    assert f(_Dev(wide[:, :, 3:4]), (2, 5, 1, 128), 0, "k") == (64, 1024)
    for bad in (wide.transpose(0, 1), wide[:, :, ::2], wide[..., ::2], wide[:, ::2], wide[:, :2]):
        with pytest.raises(ValueError):
            f(_Dev(bad), tuple(bad.shape), 0, "k")
    with pytest.raises(ValueError, match="shape"):
        f(_Dev(wide), (2, 5, 4, 128), 0, "k")


def test_binding_checks_tensors(msa):
    import torch
    u8 = torch.uint8

    def cache(k=(3, 4, 128, 128), ks=(3, 4), v=(3, 4, 128, 128), vs=(3, 4), dtype=u8, dev=0):
        return msa.Fp8Cache.from_tensors(_Dev(torch.zeros(k, dtype=u8)), _Dev(torch.zeros(ks, dtype=u8)),
                                         _Dev(torch.zeros(v, dtype=dtype)), _Dev(torch.zeros(vs, dtype=u8), dev))

    ca = cache()
    assert (ca.num_pages, ca.groups) == (3, 4) and ca.nbytes == 2 * 3 * 4 * (128 * 128 + 1)
    for bad in (dict(ks=(4, 3)), dict(v=(2, 4, 128, 128)), dict(vs=(3,)), dict(dev=1)):
        with pytest.raises(ValueError):
            cache(**bad)
    with pytest.raises(TypeError):
        cache(dtype=torch.int8)
    with pytest.raises(AttributeError):
        ca.k_data = None
    with pytest.raises(ValueError, match="CUDA"):
        msa.Fp8Cache.from_tensors(*(torch.zeros(3, 4, 128, 128, dtype=u8) for _ in range(4)))

    i32 = torch.int32
    table, lens = _Dev(torch.zeros(2, 8, dtype=i32)), _Dev(torch.zeros(2, dtype=i32))
    batch, ws = msa.Batch(table, lens, 3), _Dev(torch.zeros(1 << 10, dtype=u8))
    x = _Dev(torch.zeros(2, 3, 4, 128))
    with pytest.raises(ValueError, match="pages"):
        msa.msa_fp8_append(msa.Config(num_kv_groups=2), ca, batch, x, x, ws)
    with pytest.raises(TypeError, match="float32"):
        msa.msa_fp8_append(msa.Config(), ca, batch, _Dev(torch.zeros(2, 3, 4, 128, dtype=torch.float16)), x, ws)
    with pytest.raises(TypeError, match="float32"):
        msa.msa_fp8_append(msa.Config(), ca, batch, x, _Dev(torch.zeros(2, 3, 4, 128, dtype=torch.bfloat16)), ws)
    with pytest.raises(ValueError, match="seq_lens"):
        msa.msa_fp8_append(msa.Config(), ca, msa.Batch(table, _Dev(torch.zeros(3, dtype=i32)), 3), x, x, ws)
    q, out = _Dev(torch.zeros(2, 3, 32, 128, dtype=u8)), _Dev(torch.zeros(2, 3, 32, 128, dtype=torch.bfloat16))
    cfg = msa.Config()
    with pytest.raises(TypeError, match="q must"):
        msa.msa_fp8_attn(cfg, ca, batch, _Dev(torch.zeros(2, 3, 32, 128)), out, None, ws)
    for kw, what in ((dict(selection=_Dev(torch.zeros(2, 3, 4, 15, dtype=i32))), "selection"),
                     (dict(weight_out=_Dev(torch.zeros(2, 9))), "weight_out"),
                     (dict(weight_in=_Dev(torch.zeros(8, 2).t())), "weight_in")):
        with pytest.raises(ValueError, match=what):
            msa.msa_fp8_attn(cfg, ca, batch, q, out, None, ws, **kw)
    with pytest.raises(TypeError, match="out"):
        msa.msa_fp8_attn(cfg, ca, batch, q, q, None, ws)
    w, ints, row = (_Dev(torch.zeros(2, 8)), _Dev(torch.zeros(2, 8, dtype=i32)), _Dev(torch.zeros(2, dtype=i32)))
    with pytest.raises(ValueError, match="freed_count"):
        msa.msa_evict_blocks(batch, w, 4, 1, 1, ints, row, w, ints, ints, ws)
    with pytest.raises(ValueError, match="workspace"):
        msa.msa_evict_blocks(batch, w, 4, 1, 1, ints, row, w, ints, row, _Dev(torch.zeros(256, dtype=u8), 1))
