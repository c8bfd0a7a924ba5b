"""Pins of the FP8 page cache's oracle (oracle/fp8.py): against torch's own E4M3 rounding and
float64 softmax, brute force over subsets, and identities of the formulas."""
import itertools
import math

import numpy as np
import pytest

from oracle import fp8 as OF8
from oracle.formats import E4M3_TABLE

torch = pytest.importorskip("torch")


def _pool(rng, pages, G):
    codes = np.ascontiguousarray(torch.from_numpy(rng.normal(0, 64, (pages, G, 128, 128))).clamp(-448, 448)
                                 .to(torch.float8_e4m3fn).view(torch.uint8).numpy())
    return codes, rng.integers(119, 124, (pages, G)).astype(np.uint8)


def test_page_exponent_is_the_smallest_that_holds_the_maximum():
    for e in (-40, -9, -1, 0, 3, 39, 40):
        top = math.ldexp(448.0, e)
        assert OF8.page_exponent(top) == e
        assert OF8.page_exponent(float(np.nextafter(np.float32(top), np.float32(np.inf)))) == min(e + 1, 40)
    assert OF8.page_exponent(0.0) == -40 and OF8.page_exponent(math.inf) == 40


@pytest.mark.parametrize("L,T", [(1, 1), (128, 1), (129, 1), (200, 73), (260, 259), (384, 256)])
def test_append_against_torchs_rounding(L, T):
    rng = np.random.default_rng(L * 1000 + T)
    data, scale = _pool(rng, 5, 2)
    x = rng.normal(0, 1, (1, T, 2, 128)).astype(np.float32) * np.float32(3.0)
    table = np.array([[4, 1, 3]], np.int32)
    got, sc = OF8.append(data, scale, x, table, np.array([L]))
    touched = np.zeros((5, 128), bool)
    for pos in range(L - T, L):
        page, row = table[0, pos // 128], pos % 128
        touched[page, row] = True
        for g in range(2):
            unit = math.ldexp(1.0, int(sc[page, g]) - 127)
            want = (torch.from_numpy(x[0, pos - (L - T), g]) / unit).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
            assert np.array_equal(got[page, g, row], want)
            # half a step of 2^-3 in a binade, half the smallest step below
            v = E4M3_TABLE[got[page, g, row]] * unit
            assert (np.abs(v - x[0, pos - (L - T), g]) <= np.maximum(np.abs(x[0, pos - (L - T), g]) * 2.0 ** -4,
                                                                   2.0 ** -10 * unit)).all()
    first = L - T
    for page in range(5):
        for row in range(128):
            if touched[page, row]:
                continue
            older = page in table[0] and int(np.where(table[0] == page)[0][0]) * 128 + row < first
            grown = older and page == table[0, first // 128]
            for g in range(2):
                if not grown or sc[page, g] == scale[page, g]:
                    assert np.array_equal(got[page, g, row], data[page, g, row])
                else:
                    v = torch.from_numpy(E4M3_TABLE[data[page, g, row]] * 2.0 ** (int(scale[page, g]) - int(sc[page, g])))
                    assert np.array_equal(got[page, g, row], v.to(torch.float8_e4m3fn).view(torch.uint8).numpy())
    # the same write again changes nothing
    again, sc2 = OF8.append(got, sc, x, table, np.array([L]))
    assert np.array_equal(again, got) and np.array_equal(sc2, sc)


@pytest.mark.parametrize("sparse", [False, True])
def test_attention_against_torch_softmax(sparse):
    rng = np.random.default_rng(7)
    G, Hg, T, MB = 2, 3, 3, 4
    k, ks = _pool(rng, 9, G)
    v, vs = _pool(rng, 9, G)
    table = rng.permutation(9)[:MB * 2].reshape(2, MB).astype(np.int32)
    lens = np.array([400, 0])
    q = rng.normal(0, 1, (2, T, G * Hg, 128))
    sel = np.full((2, T, G, 16), -1, np.int32)
    sel[0, :, 0, :2], sel[0, :, 1, :3] = [1, 3], [0, 2, 3]
    w_in = rng.random((2, MB)).astype(np.float32)
    got = OF8.attention(q, (k, ks, v, vs), table, lens, Hg, sel if sparse else None, w_in, 0.5)
    mass = 0.5 * torch.from_numpy(w_in.astype(np.float64))
    for t in range(T):
        for h in range(G * Hg):
            g = h // Hg
            K = torch.from_numpy(OF8.values(k[table[0], g], ks[table[0], g]).reshape(-1, 128))
            V = torch.from_numpy(OF8.values(v[table[0], g], vs[table[0], g]).reshape(-1, 128))
            z = K @ torch.from_numpy(q[0, t, h]) / math.sqrt(128)
            key = torch.arange(MB * 128)
            hide = key > 400 - T + t
            if sparse:
                hide |= ~torch.isin(key // 128, torch.from_numpy(sel[0, t, g].astype(np.int64)))
            z = z.masked_fill(hide, -math.inf)
            p = torch.softmax(z, 0)
            assert np.allclose(got["out"][0, t, h], (p @ V).numpy(), rtol=1e-12, atol=1e-12)
            assert np.isclose(got["lse"][0, t, h], torch.logsumexp(z, 0).item(), rtol=1e-12)
            mass[0] += p.view(MB, 128).sum(1)
    assert np.allclose(got["weight"], mass.numpy(), rtol=1e-12)
    # a row's weights sum to one: the sequence collects T * H
    assert np.isclose((got["weight"] - 0.5 * w_in)[0].sum(), T * G * Hg) and not (got["weight"] - 0.5 * w_in)[1].any()
    assert not got["out"][1].any() and np.isneginf(got["lse"][1]).all()


def test_evict_keeps_the_subset_of_largest_weight():
    rng = np.random.default_rng(3)
    for trial in range(60):
        nb = int(rng.integers(1, 9))
        first, last = int(rng.integers(0, 3)), int(rng.integers(1, 3))
        budget = first + last + int(rng.integers(0, 4))
        w = rng.integers(0, 4, (1, 9)).astype(np.float32)
        table = rng.permutation(20)[:9].reshape(1, 9).astype(np.int32)
        L = nb * 128 - int(rng.integers(0, 128))
        tab, ln, wt, freed, count = OF8.evict(table, np.array([L], np.int32), w, budget, first, last)
        keep = min(nb, budget)
        best = None
        for sub in itertools.combinations(range(nb), keep):  # lexicographic: lower blocks first on ties
            if any((n < first or n >= nb - last) and n not in sub for n in range(nb)):
                continue
            key = sum(float(w[0, n]) for n in sub)
            if best is None or key > best[0]:
                best = (key, sub)
        sub = list(best[1])
        assert tab[0, :keep].tolist() == table[0, sub].tolist() and (tab[0, keep:] == -1).all()
        assert wt[0, :keep].tolist() == w[0, sub].tolist() and not wt[0, keep:].any()
        gone = [n for n in range(nb) if n not in sub]
        assert count[0] == len(gone) and freed[0, :len(gone)].tolist() == table[0, gone].tolist()
        assert ln[0] == L - 128 * len(gone)


def test_evict_ranks_nan_below_minus_infinity():
    w = np.array([[np.nan, -np.inf, np.nan, 5.0]], np.float32)
    tab = OF8.evict(np.arange(4, dtype=np.int32)[None], np.array([512], np.int32), w, 2, 0, 1)[0]
    assert tab[0].tolist() == [1, 3, -1, -1]
