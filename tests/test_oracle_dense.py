"""Pins of the dense layers' oracle (CPU only): the generator's published known answers, the
numbers' layout, gradients against central differences."""
import numpy as np
import pytest

from oracle import dense as D


@pytest.mark.parametrize("counter,key,words", [
    ((0, 0, 0, 0), (0, 0), (0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8)),
    ((0xFFFFFFFF,) * 4, (0xFFFFFFFF,) * 2, (0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD)),
    ((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0),
     (0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1))])
def test_philox_known_answers(counter, key, words):
    assert D.philox(counter, key) == words


def test_numbers_come_from_the_generator_in_order():
    seed, offset = 0x0123456789ABCDEF, 0xFEDCBA9876543210
    for first in (0, 5, (1 << 35) + 3):
        got = D.uniform(first, 40, seed, offset)
        for n, i in enumerate(range(first, first + 40)):
            b, j = i >> 3, i & 7
            hi, lo = (D.philox((b & 0xFFFFFFFF, (b >> 32) | h << 31, offset & 0xFFFFFFFF, offset >> 32),
                               (seed & 0xFFFFFFFF, seed >> 32))[j >> 1] >> 16 * (j & 1) & 0xFFFF for h in (0, 1))
            assert got[n] == hi << 16 | lo


def test_dropout_keeps_its_share_and_its_mean():
    n = 200_000
    for p in (0.0, 0.1, 0.5, 0.999, 1.0):
        k = D.kept((n,), p, 7, 3) if p else np.ones(n, bool)
        assert abs(k.mean() - (1 - p)) <= 5 * (p * (1 - p) / n) ** 0.5
        y = D.dropout(np.ones(n), p, 7, 3)
        assert set(np.unique(y)) <= {0.0, 1.0 / (1.0 - p) if p < 1 else 0.0}
    assert (D.kept((n,), 0.5, 7, 3) != D.kept((n,), 0.5, 7, 4)).mean() > 0.49
    assert (D.kept((n,), 0.5, 7, 3) != D.kept((n,), 0.5, 8, 3)).mean() > 0.49


def _differences(f, x, h=1e-6):
    g = np.zeros_like(x)
    for i in np.ndindex(*x.shape):
        a, b = x.copy(), x.copy()
        a[i] += h
        b[i] -= h
        g[i] = (f(a) - f(b)) / (2 * h)
    return g


@pytest.mark.parametrize("kind,p", [("none", 0.0), ("relu", 0.3), ("silu", 0.5), ("gelu", 0.1)])
def test_linear_gradients(kind, p):
    rng = np.random.default_rng(4)
    x, w, b = rng.standard_normal((2, 3, 5)), rng.standard_normal((5, 7)), rng.standard_normal(7)
    dy, res = rng.standard_normal((2, 3, 7)), rng.standard_normal((2, 3, 7))
    loss = lambda x, w, b: float((D.linear(x, w, b, kind, res, p, 11, 5)["y"] * dy).sum())
    g = D.linear_backward(dy, x, w, b, kind, p, 11, 5)
    np.testing.assert_allclose(g["dx"], _differences(lambda t: loss(t, w, b), x), rtol=1e-6, atol=1e-7)
    np.testing.assert_allclose(g["dw"], _differences(lambda t: loss(x, t, b), w), rtol=1e-6, atol=1e-7)
    np.testing.assert_allclose(g["db"], _differences(lambda t: loss(x, w, t), b), rtol=1e-6, atol=1e-7)
    y = D.linear(x, w, b, kind, res, p, 11, 5)["y"]
    np.testing.assert_array_equal(y, D.dropout(D.act(x @ w + b, kind), p, 11, 5) + res)
