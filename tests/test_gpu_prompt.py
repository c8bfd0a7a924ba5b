"""msa_prompt_attn against its definition in 64 bits: lengths around the tiles' edges, every number of heads,
empty rows and sequences, strides, what masked places hold, captured calls."""
import numpy as np
import pytest

from gpu_util import need_gpu
from prompt_util import Prompts, close

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    need_gpu()


def run(p):
    p.upload().call()
    return p.results()


@pytest.mark.parametrize("Hg", [1, 2, 3, 4, 5, 6, 7, 8])
def test_heads(Hg):
    p = Prompts(10 + Hg, [1, 37, 200, 0, 129], G=2, Hg=Hg, before=3, behind=5, fused=Hg % 2 == 1)
    p.check(run(p))


@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 300])
def test_lengths(n):
    p = Prompts(n, [n], G=1, Hg=8)
    p.check(run(p))
    p = Prompts(n + 1, [n, n], G=1, Hg=1, fused=True)
    p.check(run(p))


@pytest.mark.parametrize("Lq,Lk", [(1, 1000), (1, 128), (1, 129), (5, 640), (40, 41), (100, 513), (130, 1029), (257, 700)])
def test_keys_before_the_queries(Lq, Lk):
    p = Prompts(Lq * 7 + Lk, [Lq, 3, Lq], [Lk, 3, Lk + 1], G=2, Hg=4)
    p.check(run(p))


@pytest.mark.parametrize("Hg", [1, 5, 8])
def test_rows_without_keys(Hg):
    # more queries than keys: the first ones see nothing; sequences without keys; without queries
    p = Prompts(77, [200, 10, 300, 5, 0, 1], [150, 0, 1, 0, 40, 0], G=2, Hg=Hg, behind=2)
    got = run(p)
    p.check(got)
    assert (got[0][:50] == 0).all() and (got[1][:50] == -np.inf).all()


def test_no_keys_at_all():
    p = Prompts(78, [20, 5], [0, 0], G=2, Hg=3)
    assert p.Nk == 0
    got = run(p)
    assert (got[0] == 0).all() and (got[1] == -np.inf).all() and got[2] == 0


def test_nothing_to_do():
    p = Prompts(79, [0, 0], [4, 0], G=1, Hg=2, behind=3)
    p.check(run(p))
    p = Prompts(80, [], G=1, Hg=2, behind=3)
    p.check(run(p))


def test_many_sequences():
    rng = np.random.default_rng(5)
    lens = rng.integers(0, 20, 700).tolist()
    p = Prompts(81, lens, G=1, Hg=2, before=1)
    p.check(run(p))
    p = Prompts(82, [1] * 2048, G=1, Hg=1)
    p.check(run(p))


def test_ragged_batch():
    p = Prompts(83, [400, 1, 77, 513, 128, 250], G=2, Hg=4, fused=True)
    p.check(run(p))


def test_one_long_prompt():
    p = Prompts(84, [2500], G=1, Hg=2)
    p.check(run(p))


@pytest.mark.parametrize("scale,dev", [(0.5, 1.5), (1e-3, 1.5), (1.0, 20.0), (1e-30, 1.0), (0.08, 1e-20)])
def test_scales(scale, dev):
    p = Prompts(85, [150, 33], G=1, Hg=4, scale=scale, dev=dev)
    p.check(run(p))


def test_rising_and_falling_logits():
    # the running maximum moves at nearly every key, or never again after the first
    for sign in (1.0, -1.0):
        p = Prompts(86, [700], G=1, Hg=2)
        ramp = (np.arange(700) * 0.25 * sign).astype(np.float32)
        p.q[:], p.k[:] = 0.0, 0.0
        p.q[:, :, 0] = 11.3125
        import torch
        p.k[:, :, 0] = torch.from_numpy(ramp)[:, None].to(torch.bfloat16)
        p.check(run(p))


@pytest.mark.parametrize("what", [np.nan, np.inf, -np.inf])
@pytest.mark.parametrize("Hg", [2, 8])
def test_values_of_later_keys(what, Hg):
    """A special value in one dim of v at a key touches the rows that see the key, in that dim, and no others; in k,
    rows that do not see it stay as they are."""
    p = Prompts(87, [300, 150], G=2, Hg=Hg)
    for key, dim in ((130, 5), (140, 127), (299, 64), (300, 0), (449, 1)):
        p.v[key, 0, dim] = what
    p.v[135, 0, 5] = np.inf        # meets -inf or NaN of key 130
    p.v[128, 1, 7], p.v[129, 1, 7] = -np.inf, what
    ref = p.oracle()
    # the definition over infinities: numpy's 0 weights do not occur here (every probability is above 0)
    got = run(p)
    special = ~np.isfinite(ref["out"])
    assert special.any()
    ref["spread"] = np.where(special, 0.0, ref["spread"])
    p.check(got, ref)


def test_special_values_in_keys_and_queries():
    p = Prompts(88, [300], G=1, Hg=4)
    p.k[200, 0, 3] = np.nan
    p.k[290, 0, 3] = np.inf
    p.q[20, 1, 0] = np.nan
    got = run(p)
    ref = p.oracle()
    clean = np.isfinite(ref["lse"])
    assert not clean[200:].any() and not clean[20, 1] and clean[:200].sum() == 200 * 4 - 1
    assert np.isnan(got[0][200:]).all() and np.isnan(got[0][20, 1]).all()
    for r in (ref, ):
        r["out"][~clean], r["lse"][~clean] = 0, 0
        r["spread"][~clean], r["logit"][~clean] = 0, 0
    got[0][~clean], got[1][~clean] = 0, 0
    p.check(got, ref)


@pytest.mark.parametrize("cu_q,cu_k", [([0, 50, 40, 80], [0, 50, 60, 80]), ([0, 50, 60, 80], [0, 50, 60, 81]),
                                       ([-1, 50, 60, 80], [0, 50, 60, 80]), ([0, 50, 60, 80], [0, 20, 10, 80])])
def test_bad_offsets(cu_q, cu_k):
    import block_sparse_attention_indexer_gb300 as msa
    p = Prompts(89, [50, 10, 20], G=1, Hg=2)
    p.cu_q, p.cu_k = np.array(cu_q, np.int32), np.array(cu_k, np.int32)
    out, lse, err = run(p)
    assert err == msa.MSA_DEVERR_BAD_SEQLEN and (out == 7).all() and (lse == 7).all()


@pytest.mark.parametrize("lens,at", [([900, 500, 600], 2), ([5] * 600, 599), ([4] * 70, 66)])
@pytest.mark.parametrize("which", ["cu_q", "cu_k"])
def test_bad_offsets_of_longer_lists(lens, at, which):
    """The same where the plan is made by every block, by a launch before, and for more than 64 sequences."""
    import block_sparse_attention_indexer_gb300 as msa
    p = Prompts(99, lens, G=1, Hg=2)
    cu = getattr(p, which).copy()
    cu[at] = cu[at - 1] - 1
    setattr(p, which, cu)
    out, lse, err = run(p)
    assert err == msa.MSA_DEVERR_BAD_SEQLEN and (out == 7).all() and (lse == 7).all()


def test_without_lse_same_bits():
    p = Prompts(90, [513, 64, 900], G=2, Hg=5)
    first = run(p)
    for _ in range(3):
        p.out.fill_(7.0)
        p.call(lse=False)
        again = p.results()
        assert np.array_equal(first[0], again[0]) and np.array_equal(first[1], again[1])


def test_captured_and_on_another_stream():
    import torch
    p = Prompts(91, [300, 20, 1], G=2, Hg=8)
    ref = p.oracle()
    p.upload()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    p.call(stream=s)
    s.synchronize()
    p.check(p.results(), ref)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        p.call()
    for lens in ([300, 20, 1], [1, 319, 1], [0, 0, 321]):     # new lengths under the same graph
        cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
        p.packed.cu_q.copy_(torch.from_numpy(cu))
        p.packed.cu_k.copy_(torch.from_numpy(cu))
        p.cu_q = p.cu_k = cu
        p.out.fill_(7.0)
        p.lse.fill_(7.0)
        g.replay()
        p.check(p.results())


@pytest.mark.parametrize("room,batch,G,Hg", [(2100, 1, 8, 3), (3000, 3, 2, 8), (3000, 600, 1, 2)])
def test_captured_with_room_for_more(room, batch, G, Hg):
    """A graph whose lists have room for more tokens than a replay's sequences take: how the work is split is chosen by the
    room, the rows behind the last sequence stay as they were."""
    import torch
    p = Prompts(100, [room] + [0] * (batch - 1), G=G, Hg=Hg).upload()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        p.call()
    for lens_q, lens_k in (([1], [900]), ([0, 130], [7, 140]), ([200, 3, 40], [200, 800, 41])):
        n = min(batch, len(lens_q))
        p.cu_q, p.cu_k = (np.cumsum([0] + list(x[:n]) + [0] * (batch - n)).astype(np.int32) for x in (lens_q, lens_k))
        p.packed.cu_q.copy_(torch.from_numpy(p.cu_q))
        p.packed.cu_k.copy_(torch.from_numpy(p.cu_k))
        p.used_q = np.arange(p.Nq) < p.cu_q[-1]
        p.out.fill_(7.0)
        p.lse.fill_(7.0)
        g.replay()
        p.check(p.results())


def test_single_token_agrees_with_the_prompt():
    """The last row of a prompt is the single-token call over the same keys."""
    p = Prompts(92, [700], G=2, Hg=4)
    out, lse, _ = run(p)
    one = Prompts(92, [700], G=2, Hg=4)
    one.cu_q, one.Nq, one.q = np.array([0, 1], np.int32), 1, p.q[-1:]
    one.used_q = np.ones(1, bool)
    o1, l1, err = run(one)
    assert err == 0
    close("out", o1[0], out[-1], np.abs(out[-1]) * 2.0 ** -7 + 2.0 ** -8)
    close("lse", l1[0], lse[-1], np.full(l1[0].shape, 1e-4))


# How the work is split: units that stay whole and are dealt out by cost, cut units, plans made by the attention's blocks
# themselves (up to 512 sequences) or by a launch before them, more units than are put in order.
@pytest.mark.parametrize("lens_q,lens_k,G,Hg", [
    ([1100], None, 2, 8),                                        # whole: a unit for nearly every block of the grid
    ([2100, 3, 700], None, 2, 8),                                # whole, two a block
    ([1000] + [37 * i % 500 for i in range(1, 32)], None, 2, 8),  # whole, many units of the same cost
    ([2100], None, 8, 3),                                        # no plan: one prompt, more units than blocks
    ([0, 90, 1, 0, 33] * 11 + [200], None, 3, 5),                # no plan: short ones, some of them empty, over 32 of them
    ([40, 0, 7], [600, 500, 20], 8, 1),                          # no plan: chunks
    ([40], [5000], 2, 8),                                        # cut, few units
    ([1], [6000], 1, 8),                                         # one row tile cut into nearly as many parts as pages
    ([1, 1, 1], [3000, 20, 2000], 1, 1),
    ([20] * 599 + [900], None, 1, 2),                            # planned by a launch: one much longer than the rest
    ([300] * 8 + [9] * 592, None, 1, 4),                         # planned by a launch, whole
    ([70] + [1] * 519, [4000] + [2] * 519, 1, 4),                # planned by a launch, cut
    ([33] * 1029 + [300], None, 1, 8),                           # more units than are put in order
])
def test_split_of_the_work(lens_q, lens_k, G, Hg):
    p = Prompts(len(lens_q) + sum(lens_q), lens_q, lens_k, G=G, Hg=Hg, before=2, behind=3)
    first = run(p)
    p.check(first)
    p.out.fill_(7.0)
    p.lse.fill_(7.0)
    p.call()
    again = p.results()
    assert np.array_equal(first[0], again[0]) and np.array_equal(first[1], again[1])


@pytest.mark.parametrize("lens_q,lens_k", [([40, 3], [5000, 700]), ([1], [4000]), ([130, 1], [2000, 3000])])
def test_values_of_later_keys_in_cut_units(lens_q, lens_k):
    p = Prompts(93, lens_q, lens_k, G=1, Hg=8)
    for b in range(p.B):
        end = int(p.cu_k[b + 1])
        for back, dim, what in ((1, 5, np.nan), (2, 127, np.inf), (17, 64, -np.inf), (33, 64, np.inf), (39, 0, np.inf),
                                (129, 9, np.nan), (600, 11, np.inf)):
            p.v[end - back, 0, dim] = what
    ref = p.oracle()
    got = run(p)
    special = ~np.isfinite(ref["out"])
    assert special.any()
    ref["spread"] = np.where(special, 0.0, ref["spread"])
    p.check(got, ref)


@pytest.mark.parametrize("G,Hg,most", [(8, 3, 4), (4, 2, 200), (3, 1, 300)])
def test_values_of_later_keys_in_short_units(G, Hg, most):
    """Several short units a block of the grid, some with special values: what one holds stays out of the others."""
    rng = np.random.default_rng(most)
    lens = rng.integers(0, most + 1, 60).tolist()
    p = Prompts(98, lens, G=G, Hg=Hg, behind=2)
    for i in range(0, p.B, 3):
        if lens[i]:
            key, g = int(p.cu_k[i]) + int(rng.integers(lens[i])), int(rng.integers(G))
            p.v[key, g, int(rng.integers(128))] = (np.nan, np.inf, -np.inf)[i % 3 if i % 2 else (i + 1) % 3]
    ref = p.oracle()
    got = run(p)
    special = ~np.isfinite(ref["out"])
    assert special.any()
    ref["spread"] = np.where(special, 0.0, ref["spread"])
    p.check(got, ref)


def test_two_calls_at_once():
    import torch
    a, b = Prompts(94, [900, 50], G=2, Hg=4).upload(), Prompts(95, [30, 5], [4000, 3000], G=2, Hg=4).upload()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(20):
        for p, s in zip((a, b), streams):
            p.call(stream=s)
    for p in (a, b):
        p.check(p.results())


def test_tokens_far_apart():
    """Rows 2^27 elements apart: the last ones lie beyond 2^31 elements and 2^32 bytes."""
    import torch
    p = Prompts(96, [18], G=2, Hg=4)
    ref = p.oracle()
    p.upload()
    wide = torch.empty(17 * 2 ** 27 + 4096, dtype=torch.bfloat16, device="cuda")
    far = []
    for i, x in enumerate(p.d):
        v = wide[1024 * i:].as_strided((18,) + tuple(x.shape[1:]), (2 ** 27, 128, 1))
        v.copy_(x)
        far.append(v)
    p.d = far
    p.call()
    p.check(p.results(), ref)


def test_scores_that_are_all_minus_infinity():
    # such a row is one without keys
    p = Prompts(97, [40], G=1, Hg=2)
    p.q[:, :, :] = 0.0
    p.q[:, 0, 0], p.k[:, 0, 0] = 1.0, -np.inf
    p.q[:, 1, 1] = 1.0
    p.k[:, 0, 1:] = 0.0
    p.q[:, 1, 0] = 1.0
    got = run(p)
    assert (got[0] == 0).all() and (got[1] == -np.inf).all() and got[2] == 0


@pytest.mark.parametrize("lens_q,lens_k,G,Hg", [([40, 90], [5000, 700], 2, 8), ([1], [4000], 1, 8), ([1100], None, 2, 8)])
def test_the_plan_is_read_before_keys_are_copied_over_it(lens_q, lens_k, G, Hg):
    """The plan that every block makes for itself lies where the first keys are copied to: a lane that read it late would find
    keys there.  Cut and whole units, many calls one after another, the same bits in all of them."""
    import torch
    p = Prompts(101, lens_q, lens_k, G=G, Hg=Hg)
    first = run(p)
    p.check(first)
    out, lse = p.out.clone(), p.lse.clone()
    different = torch.zeros((), dtype=torch.int64, device="cuda")
    for _ in range(300):
        p.out.fill_(7.0)
        p.lse.fill_(7.0)
        p.call()
        different += (p.out != out).sum() + (p.lse != lse).sum()
    assert int(different) == 0 and p.results()[2] == 0


# Scores from small ones to where float32 numbers lie 2^80 apart.
@pytest.mark.parametrize("scale", [0.0, 1.0, 100.0, 2.0 ** 70])
@pytest.mark.parametrize("lens_q,lens_k,G,Hg", [
    ([1], [1], 1, 1), ([1, 2, 5], None, 1, 8), ([300, 40], None, 2, 5),     # dealt out as they come
    ([1100], None, 2, 8),                                                    # planned, whole
    ([40], [5000], 2, 8), ([1], [6000], 1, 8), ([130, 1], [2000, 3000], 1, 4),   # cut
])
def test_large_logits(scale, lens_q, lens_k, G, Hg):
    """Finite scores of any size.  Every element of a query is x and of a key 24,576 s, x and s powers of two or 3 or 9 times
    one: 128 equal products, whose sums are exact in float32 in any order.  So equal scores stay equal, others are apart by far more than
    the softmax can tell, and a row is the mean of V over its keys with the largest score: the tolerance of out has no term
    for the logits.  lse is off by the factor's three roundings, one of the product, two of the sum with log2 l, two of ln 2:
    8 * 2^-24 of it."""
    import torch
    p = Prompts(102, lens_q, lens_k, G=G, Hg=Hg, scale=scale)
    x = torch.tensor([24576.0, -24576.0, 18432.0, 1.0, 98304.0, -98304.0, 2.0 ** -6, 49152.0]).to(torch.bfloat16)
    p.q[:] = x[:p.Hg].repeat(p.G)[None, :, None]
    for b in range(p.B):
        n = int(p.cu_k[b + 1] - p.cu_k[b])
        j = torch.arange(n)
        # signs by turns; all positive; rising, from a size that is not large
        s = (torch.tensor([1.0, -1.0, 1.0, 0.5])[j % 4], torch.tensor([0.5, 1.0, 0.25, 1.0])[j % 4],
             torch.exp2(torch.floor(24.0 * j / n) - 23))[(b + len(lens_q) + G) % 3]
        p.k[int(p.cu_k[b]):int(p.cu_k[b + 1])] = (24576.0 * s).to(torch.bfloat16)[:, None, None]
    ref = p.oracle()
    assert np.isfinite(ref["lse"]).all()
    out, lse, err = run(p)
    assert err == 0 and np.isfinite(out).all()
    rel = 2.0 ** -20 + ref["keys"] * 2.0 ** -24 + 2.0 ** -7 + 2.0 ** -14
    close("out", out, ref["out"], 2.0 ** -8 * np.abs(ref["out"]) + rel[..., None] * ref["spread"] + 1e-30)
    close("lse", lse, ref["lse"], 2.0 ** -20 + ref["keys"] * 2.0 ** -24 + 2.0 ** -21 * np.abs(ref["lse"]))


@pytest.mark.parametrize("what", ["minus infinity", "far below"])
@pytest.mark.parametrize("lens_q,lens_k,G,Hg", [
    ([300, 40, 6], None, 2, 8), ([150, 10], None, 1, 3),                     # dealt out as they come
    ([1100], None, 2, 8),                                                    # planned, whole
    ([40], [5000], 2, 8), ([1], [6000], 1, 8), ([130, 1], [2000, 3000], 1, 4),   # cut
])
def test_special_values_of_no_probability(lens_q, lens_k, G, Hg, what):
    """Infinities and NaN in v at keys whose probability is 0: what 0 times them gives, wherever the key lies in a unit."""
    p = Prompts(104, lens_q, lens_k, G=G, Hg=Hg)
    p.q[:, :, 0] = 64.0
    low = []
    for b in range(p.B):
        a, n = int(p.cu_k[b]), int(p.cu_k[b + 1] - p.cu_k[b])
        low += [a + x for x in {1, 5, n // 3, n // 2, n - 129, n - 33, n - 18, n - 2, n - 1} if 0 < x < n]
    for i, key in enumerate(sorted(low)):
        p.v[key, :, 3 + 5 * i % 120] = np.inf
        p.v[key, :, 4 + 5 * i % 120] = -np.inf
        p.v[key, :, 5 + 5 * i % 120] = np.nan
        p.v[key - 1, 0, 3 + 5 * i % 120] = np.inf                            # and one that has a probability beside it
    k = p.k.clone()
    k[low] = 0.0
    p.k[low, :, 0] = -np.inf if what == "minus infinity" else -4096.0        # e^-23,000
    ref = p.oracle()
    special = ~np.isfinite(ref["out"])
    assert np.isnan(ref["out"]).any() and np.isfinite(ref["lse"]).all()
    ref["spread"] = np.where(special, 0.0, ref["spread"])
    got = run(p)
    p.k = k                                                                  # the other keys' logits are what has an error
    ref["logit"] = p.oracle()["logit"]
    p.check(got, ref)


@pytest.mark.parametrize("lens_q,lens_k,Hg", [([40], None, 2), ([300], None, 8), ([30], [5000], 8), ([1], [4000], 8)])
def test_special_values_in_rows_of_minus_infinity(lens_q, lens_k, Hg):
    """Rows whose logits are all -inf: 0, and NaN in the dims where what they see of v is not finite."""
    p = Prompts(105, lens_q, lens_k, G=1, Hg=Hg)
    p.q[:], p.k[:] = 0.0, 0.0
    p.q[:, :, 0], p.k[:, :, 0] = 1.0, -np.inf
    want = np.zeros((p.Nq, p.H, 128))
    for back, dim, what in ((p.Nk - 3, 7, np.inf), (20, 1, np.nan), (7, 9, -np.inf), (1, 100, np.inf), (min(p.Nk, 250), 50, np.inf)):
        p.v[p.Nk - back, 0, dim] = what
        want[max(0, p.Nq - back):, :, dim] = np.nan
    got = run(p)
    close("out", got[0], want, np.zeros_like(want))
    assert (got[1] == -np.inf).all() and got[2] == 0
