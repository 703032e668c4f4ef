"""Gradients of dense layers over the whole range of their types, on every kernel that serves
them, against the fp64 oracle (oracle/dense.py).

Tolerances count roundings, value by value. U is fp32's unit roundoff, RO the type's, TINY half
of fp16's smallest step. Sums of k products in fp32 are off by at most 2 U k times the sum of
the terms' magnitudes. The slopes of silu and gelu change by less than 1 per unit of z and
are constant to 1e-11 beyond |z| = 30, so that neither z's own error nor the rounding with which
it is read back counts there."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from oracle import dense as D

U = 2.0 ** -24
RO = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}
TINY = {"f32": 0.0, "f16": 2.0 ** -25, "bf16": 0.0}
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
# rows, in, out: rows kernels of whole and of odd chunks, one and two blocks of 32; tiles from
# registers and straight to LDS; few rows
LAYERS = [(300, 24, 32), (300, 64, 64), (301, 33, 45), (300, 32, 3), (150, 200, 130), (150, 203, 131), (300, 256, 264),
          (3, 304, 72), (2, 2048, 72), (9, 77, 500)]


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda:0")


@pytest.fixture(autouse=True)
def _say(request):
    print(f"[case] {request.node.name}", flush=True)
    yield


def _put(a, dt, dev):
    return torch.from_numpy(np.asarray(a, np.float32)).to(DT[dt]).to(dev)


def _np(t):
    return t.detach().double().cpu().numpy()


def _check(got, ref, tol, what):
    got = _np(got)
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} off, worst {np.nanmax(np.abs(got - ref)):.3e}, {np.isnan(got).sum()} NaN"


def _gradients(dt, act, p, x, w, b, dy, e_dz, what):
    """Checks linear_backward with and without what the forward kept. e_dz(g): how far dz may be
    off besides z's error, as a multiple of |dy| times the slope's bound and in absolute terms."""
    from sphere_rasterization_amd import appearance as A
    more = dict(act=act, p=p, rng=(5, 6) if p else None)
    xn, wn, bn, dn = (_np(t) for t in (x, w, b, dy))
    m, k = xn.shape
    n = wn.shape[1]
    with np.errstate(over="ignore"):                         # exp(-z) of the oracle's slopes, whose limit is right
        g = D.linear_backward(dn, xn, wn, bn, act, p, 5, 6)
    z = g["z"]
    s = 1.0 / (1.0 - p)
    keep = D.kept(z.shape, p, 5, 6) if p else np.ones(z.shape, bool)
    e_z = 2 * (k + 8) * U * (np.abs(xn) @ np.abs(wn) + np.abs(bn)) + RO[dt] * np.abs(z) + TINY[dt]
    if act == "none":
        e_slope = 0.0 * z
    elif act == "relu":
        e_slope = (np.abs(z) <= e_z) * 1.0
    else:
        e_slope = np.where(np.abs(z) > 30.0, 1e-10, np.minimum(e_z, 1.2)) + 2e-7 + 8 * U
    rel, least = e_dz
    d = s * keep * np.abs(dn)
    e = d * e_slope + (rel + 4 * U) * np.abs(g["dz"]) + s * keep * least * (dn != 0)
    a = np.abs(g["dz"]) + e
    parts = 2                                                # of dz: twice as many terms
    top = lambda v, t=dt: RO[t] * np.abs(v) + TINY[t]
    _, pre = A.linear_forward(x, w, b, **more)
    for kept in (pre, None):
        dx, dw, db = A.linear_backward(dy, x, w, b, pre=kept, **more)
        _check(dx, g["dx"], e @ np.abs(wn).T + 2 * (parts * n + 8) * U * (a @ np.abs(wn).T) + top(g["dx"]), f"dx {what}")
        _check(dw, g["dw"], np.abs(xn).T @ e + 2 * (parts * m + 8) * U * (np.abs(xn).T @ a) + top(g["dw"]), f"dw {what}")
        bt = "f32" if db.dtype == torch.float32 else dt
        _check(db, g["db"], e.sum(0) + 2 * (m + 8) * U * a.sum(0) + top(g["db"], bt), f"db {what}")


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("act", ["relu", "silu", "gelu"])
@pytest.mark.parametrize("m,k,n", LAYERS + [(65536, 16, 72)])
def test_z_beyond_the_range_of_16_bits(dev, m, k, n, act, dt):
    """Finite inputs whose z passes fp16's largest value, 65504, on either side: the slope there is
    0 or 1. dz may be rounded once."""
    from sphere_rasterization_amd import appearance as A
    rng = np.random.default_rng(m + k + n)
    xn, wn = rng.standard_normal((m, k)), rng.standard_normal((k, n)) * k ** -0.5
    row = min(m - 1, 5)
    xn[row, 0] = 400.0
    wn[0] = np.where(rng.random(n) < 0.5, 250.0, -250.0)
    xn[np.arange(m) != row, 0] = 0.0
    x, w, b = _put(xn, dt, dev), _put(wn, dt, dev), _put(0.3 * rng.standard_normal(n), dt, dev)
    dy = _put(rng.standard_normal((m, n)), dt, dev)
    z = _np(x)[row] @ _np(w) + _np(b)
    assert z.max() > 70000 and (z.min() < -70000 or n < 8)
    if dt == "f16":
        y = A.linear(x, w, b, act=act)[row]
        assert bool((y[torch.from_numpy(z < -70000).to(dev)] == 0).all()) and bool(torch.isinf(y[torch.from_numpy(z > 70000).to(dev)]).all())
    _gradients(dt, act, 0.0, x, w, b, dy, (RO[dt], TINY[dt]), act)


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu"])
@pytest.mark.parametrize("m,k,n", LAYERS)
def test_large_gradients(dev, m, k, n, act, dt):
    """dz beyond fp16's range, by dropout's factor and by slopes past 1, under gradients that are
    inside it. dz is exact where the slope is 0 or 1, and held in two parts otherwise."""
    rng = np.random.default_rng(m + k + n)
    x, w = (_put(0.005 * rng.standard_normal(s), dt, dev) for s in ((m, k), (k, n)))
    b = _put(1.5 * rng.standard_normal(n), "f32", dev)
    dy = _put(rng.uniform(40000.0, 60000.0, (m, n)) * np.where(rng.random((m, n)) < 0.5, 1.0, -1.0), dt, dev)
    rel = 0.0 if act in ("none", "relu") else RO[dt] ** 2
    for p in (0.0, 0.5):
        _gradients(dt, act, p, x, w, b, dy, (rel, TINY[dt]), f"{act} p {p}")


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("m,k,n", LAYERS)
def test_gradients_of_nothing_kept(dev, m, k, n, dt):
    from sphere_rasterization_amd import appearance as A
    x, w, dy = (torch.randn(*s, device=dev).to(DT[dt]) for s in ((m, k), (k, n), (m, n)))
    for act in ("none", "gelu"):
        for g in A.linear_backward(dy, x, w, act=act, p=1.0, rng=(1, 2)):
            assert torch.equal(g, torch.zeros_like(g))
