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
from tests.dense_layers import LARGE

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


@pytest.mark.parametrize("large", ["x", "w"])
@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("m,k,n", LAYERS)
def test_small_gradients_of_fp16(dev, m, k, n, act, large):
    """d_y down to fp16's smallest step: dz is held to 2^-22 of itself and to 2^-35, whatever the
    others' size. x or W is large, so that the gradients' own steps do not hide it."""
    rng = np.random.default_rng(m + k + n)
    xn, wn = rng.standard_normal((m, k)), rng.standard_normal((k, n)) * k ** -0.5
    xn, wn = (4.0 * xn, wn / 4.0) if large == "x" else (xn * k ** -0.5 / 4.0, 4.0 * wn * k ** 0.5)
    x, w, b = _put(xn, "f16", dev), _put(wn, "f16", dev), _put(0.3 * rng.standard_normal(n), "f32", dev)
    for scale in (2.0 ** -16, 2.0 ** -20, 2.0 ** -22, 2.0 ** -24, 0.0):
        # 0: every row has a size of its own, from the smallest step to a hundred
        by = scale if scale else 2.0 ** rng.integers(-24, 8, (m, 1))
        dy = _put(by * rng.standard_normal((m, n)), "f16", dev)
        for p in (0.0, 0.25):
            _gradients("f16", act, p, x, w, b, dy, (2.0 ** -22, 2.0 ** -35), f"{act} {scale} p {p}")


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("order", ["io", "oi"])
@pytest.mark.parametrize("m,k,n", LARGE)
def test_large_layers(dev, m, k, n, order, dt):
    """Every tile of the products, whole and split, at ends inside tiles and stages, with all that
    goes with the forward, value by value against torch in 64 bits. dz of bf16 may be rounded once."""
    from sphere_rasterization_amd import appearance as A
    gen = torch.Generator(device=dev).manual_seed(m + k + n)
    randn = lambda *s: torch.randn(*s, generator=gen, device=dev)
    x, r, dy = (randn(*s).to(DT[dt]) for s in ((m, k), (m, n), (m, n)))
    w = (randn(k, n) * k ** -0.5).to(DT[dt]) if order == "io" else (randn(n, k) * k ** -0.5).to(DT[dt]).t()
    b, p = randn(n).to(DT[dt]), 0.1
    more = dict(act="gelu", p=p, rng=(5, 6))
    y, pre = A.linear_forward(x, w, b, residual=r, **more)
    dx, dw, db = A.linear_backward(dy, x, w, b, pre=pre, **more)
    keep = A.dropout(torch.ones_like(y), p, (5, 6)) != 0
    wide = lambda t: t.double().contiguous()
    x, w, b, r, dy = (wide(t) for t in (x, w, b, r, dy))
    mm = lambda a, c: a @ c.contiguous()
    s = keep / (1.0 - p)
    z = mm(x, w) + b
    e_z = 2 * (k + 8) * U * (mm(x.abs(), w.abs()) + b.abs())
    cdf, density = torch.special.ndtr(z), torch.exp(-0.5 * z * z) * 0.3989422804014327
    want = r + s * z * cdf
    # gelu of 16-bit results is off by 1.9e-6 and a fifth of a rounding more
    e_y = s * (1.13 * e_z + 2e-6 + 8 * U * z.abs()) + 4 * U * (want.abs() + r.abs()) + 1.2 * RO[dt] * want.abs() + TINY[dt]
    e_pre = RO[dt] * z.abs() + TINY[dt]

    def check(got, ref, tol, what):
        bad = ~((got.double() - ref).abs() <= tol)
        assert not bool(bad.any()), f"{what}: {int(bad.sum())} of {bad.numel()} off, worst {float((got.double() - ref).abs().max()):.3e}"

    check(y, want, e_y, "y")
    check(pre, z, e_z + e_pre, "pre")
    dz = s * dy * (cdf + z * density)
    rel = dict(f32=0.0, f16=RO["f16"] ** 2, bf16=RO["bf16"])[dt]
    e_dz = s * dy.abs() * (e_z + e_pre + 2e-7 + 8 * U) + (rel + 4 * U) * dz.abs() + TINY[dt] ** 2
    a = dz.abs() + e_dz
    top = lambda v: RO[dt] * v.abs() + TINY[dt]
    ref = mm(dz, w.t())
    check(dx, ref, mm(e_dz, w.abs().t()) + 2 * (2 * n + 8) * U * mm(a, w.abs().t()) + top(ref), "d_x")
    ref = mm(x.t(), dz)
    check(dw, ref, mm(x.abs().t(), e_dz) + 2 * (2 * m + 8) * U * mm(x.abs().t(), a) + top(ref), "d_W")
    ref = dz.sum(0)
    check(db, ref, e_dz.sum(0) + 2 * (m + 8) * U * a.sum(0) + top(ref), "d_b")
    # and in the norm, where the roundings' signs cancel: those of z, of dz and of the result, at most RO each
    for got, ref in ((dx, mm(dz, w.t())), (dw, mm(x.t(), dz))):
        assert float((got.double() - ref).norm() / ref.norm()) <= 3 * RO[dt] + 2e-6


@pytest.mark.parametrize("m,k,n", LARGE)
def test_small_gradients_of_large_fp16_layers(dev, m, k, n):
    """d_y of a few of fp16's smallest steps: dz is held to 2^-35 on every tile and across splits
    that hold parts of both of its parts. x is large and z exact, so that nothing else counts."""
    from sphere_rasterization_amd import appearance as A
    gen = torch.Generator(device=dev).manual_seed(m + k + n)
    randn = lambda *s: torch.randn(*s, generator=gen, device=dev)
    x, dy = (8.0 * torch.sign(randn(m, k))).half(), (2.0 ** -23 * randn(m, n)).half()
    w = torch.zeros(k, n, device=dev)
    w[torch.randint(0, k, (n,), generator=gen, device=dev), torch.arange(n, device=dev)] = 0.0625 * torch.sign(randn(n))
    w = w.half()
    dx, dw, db = A.linear_backward(dy, x, w, act="silu", pre=A.linear_forward(x, w, act="silu")[1])
    x, w, dy = x.double(), w.double(), dy.double()
    z = x @ w
    assert bool(((z.abs() == 0.5) | (z == 0.0)).all())        # a normal number may be 0, and its sign then
    dz = dy * (torch.sigmoid(z) + z * torch.sigmoid(z) * torch.sigmoid(-z))
    e_dz = (2e-7 + 8 * U) * dy.abs() + 2.0 ** -22 * dz.abs() + 2.0 ** -35
    for got, ref, e, size in ((dx, dz @ w.t().contiguous(), e_dz @ w.abs().t().contiguous(), dz.abs() @ w.abs().t().contiguous()),
                              (dw, x.t().contiguous() @ dz, x.abs().t().contiguous() @ e_dz, x.abs().t().contiguous() @ dz.abs())):
        bad = ~((got.double() - ref).abs() <= e + 2 * (2 * max(m, n) + 8) * U * size + RO["f16"] * ref.abs() + TINY["f16"])
        assert not bool(bad.any()), (int(bad.sum()), float((got.double() - ref).abs().max()))
        # in the norm: errors of dz of 2^-35 at most add up as independent ones, beside one rounding
        err, most = float((got.double() - ref).norm()), float((ref.half().double() - ref).norm())
        count = float(n if got is dx else m)
        assert err <= 1.1 * most + 2.0 ** -35 * (8.0 if got is dw else 0.0625) * (count * got.numel()) ** 0.5 + 4e-6 * float(ref.norm())


TWO_PARTS = [("bf16", *s) for s in ((2000, 24, 32), (2000, 64, 64), (2001, 33, 45), (1000, 264, 392), (1001, 203, 131), (16, 2048, 520),
                                    (9, 304, 264), (4100, 504, 1032), (70_000, 160, 200))]
TWO_PARTS += [("f16", *s) for s in ((2000, 24, 32), (2001, 33, 45), (1001, 203, 131), (9, 304, 264), (4200, 520, 1000), (8191, 1024, 2056))]
ONE_PART = [("bf16", *s) for s in ((4200, 520, 1000), (65_536, 160, 208), (4199, 521, 1001), (600, 1024, 4096))]


@pytest.mark.parametrize("act", ["silu", "gelu", "relu", "none"])
@pytest.mark.parametrize("dt,m,k,n", TWO_PARTS + ONE_PART)
def test_parts_of_dz(dev, dt, m, k, n, act):
    """How dz is held, by the error of the gradients over that of rounding them once: 1 where dz is
    exact or in two parts, and the square root of 2 where one more rounding of the same size goes in.
    z is exact in the type (sums of 1/16), so that only dz counts. Both errors are norms over more than
    2000 values of one distribution, steady to a few in a hundred."""
    from sphere_rasterization_amd import appearance as A
    gen = torch.Generator(device=dev).manual_seed(m + k + n)
    sign = lambda *s: torch.where(torch.rand(*s, generator=gen, device=dev) < 0.5, 1.0, -1.0)
    x, w = sign(m, k).to(DT[dt]), (sign(k, n) / 16).to(DT[dt])
    dy = torch.randn(m, n, generator=gen, device=dev).to(DT[dt])
    _, pre = A.linear_forward(x, w, act=act)
    got = A.linear_backward(dy, x, w, act=act, pre=pre, p=0.25, rng=(5, 6))
    keep = A.dropout(torch.ones_like(dy), 0.25, (5, 6)) != 0
    x, w, dz = x.double(), w.double(), dy.double() * keep / 0.75
    z = x @ w
    if act == "silu":
        dz = dz * (torch.sigmoid(z) + z * torch.sigmoid(z) * torch.sigmoid(-z))
    elif act == "gelu":
        dz = dz * (torch.special.ndtr(z) + z * torch.exp(-0.5 * z * z) * 0.3989422804014327)
    elif act == "relu":
        dz = dz * (z > 0)
    one = (dt, m, k, n) in ONE_PART and act in ("silu", "gelu")
    for what, g, ref in (("d_x", got[0], dz @ w.t().contiguous()), ("d_W", got[1], x.t().contiguous() @ dz)):
        once = float((ref.to(DT[dt]).double() - ref).norm())
        ratio = float((g.double() - ref).norm()) / once
        assert (1.2 <= ratio <= 1.6) if one else ratio <= 1.1, (what, ratio)
