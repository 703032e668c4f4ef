"""Pins of the appearance oracle (CPU only): gradients against central differences, the
table gradient as the transpose of the lookup, the singular-value form of the
orthogonalised update against its products."""
import numpy as np
import pytest

from oracle import appearance as A


def _differences(f, x, h=1e-6):
    g = np.zeros_like(x)
    it = np.nditer(x, flags=["multi_index"])
    for _ in it:
        i = it.multi_index
        a, b = x.copy(), x.copy()
        a[i] += h
        b[i] -= h
        g[i] = (f(a) - f(b)) / (2 * h)
    return g


def test_lookup_and_its_gradient():
    rng = np.random.default_rng(1)
    table = rng.standard_normal((5, 3))
    ids = np.array([4, 0, -1, 4, 5, 2, 4, 1 << 40])
    y = A.lookup(table, ids, 0.5)
    np.testing.assert_array_equal(y[[0, 3, 6]], 0.5 * table[[4, 4, 4]])
    np.testing.assert_array_equal(y[[2, 4, 7]], 0.0)
    dy = rng.standard_normal(y.shape)
    d = A.lookup_backward(dy, ids, 5, 0.5)
    np.testing.assert_allclose(d, _differences(lambda t: float((A.lookup(t, ids, 0.5) * dy).sum()), table), atol=1e-8)
    np.testing.assert_array_equal(d[3], 0.0)


@pytest.mark.parametrize("kind", ["none", "relu", "silu", "gelu"])
def test_group_norm_gradients(kind):
    rng = np.random.default_rng(2)
    x = rng.standard_normal((2, 2, 3, 6)) + 0.5
    w, b, dy = rng.standard_normal(6), rng.standard_normal(6), rng.standard_normal(x.shape)
    f = A.group_norm(x, 3, w, b, 1e-3, kind)
    v = x.reshape(2, 6, 3, 2)
    np.testing.assert_allclose(f["mean"], v.mean(axis=(1, 3)), rtol=1e-12)
    np.testing.assert_allclose(f["rstd"], (v.var(axis=(1, 3)) + 1e-3) ** -0.5, rtol=1e-12)
    g = A.group_norm_backward(dy, x, 3, w, b, 1e-3, kind)
    loss = lambda x, w, b: float((A.group_norm(x, 3, w, b, 1e-3, kind)["y"] * dy).sum())
    np.testing.assert_allclose(g["dx"], _differences(lambda t: loss(t, w, b), x), rtol=1e-6, atol=1e-7)
    np.testing.assert_allclose(g["dw"], _differences(lambda t: loss(x, t, b), w), rtol=1e-6, atol=1e-7)
    np.testing.assert_allclose(g["db"], _differences(lambda t: loss(x, w, t), b), rtol=1e-6, atol=1e-7)


@pytest.mark.parametrize("shape", [(7, 7), (4, 9), (9, 4), (1, 5), (2, 6, 5)])
def test_orthogonalize_is_the_products(shape):
    rng = np.random.default_rng(3)
    g = rng.standard_normal(shape)
    x = g / (np.sqrt((g * g).sum((-2, -1), keepdims=True)) + 1e-7)
    a, b, c = 3.4445, -4.7750, 2.0315
    for _ in range(5):
        s = np.matmul(x, np.swapaxes(x, -1, -2))
        x = a * x + np.matmul(b * s + c * np.matmul(s, s), x)
    np.testing.assert_allclose(A.orthogonalize(g), x, rtol=1e-9, atol=1e-10)
    # singular values of a full-rank matrix end near one
    sv = np.linalg.svd(A.orthogonalize(rng.standard_normal((6, 6))), compute_uv=False)
    assert sv.max() < 1.3


@pytest.mark.parametrize("shape", [(1, 7), (8, 8), (64, 32), (65, 130), (257, 70), (96, 96), (40, 700), (90, 1500), (200, 250)])
def test_the_bound_tells_both_parts_of_a_factor_from_one(shape):
    """Two parts per factor stay below the bound; any cross product left out does not."""
    from tests import ortho_parts as H
    g = np.random.default_rng(shape[0] * 7 + shape[1]).standard_normal(shape).astype(np.float32)
    ref = A.orthogonalize(g)
    assert H.error(H.orthogonalize(g), ref) <= H.BOUND / 4
    for product in H.PRODUCTS:
        for lost in (H.CROSS[:1], H.CROSS[1:], H.CROSS):
            assert H.error(H.orthogonalize(g, {product: lost}), ref) > 2 * H.BOUND, (product, lost)
