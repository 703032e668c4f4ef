"""Dense layers and dropout on the GPU against the fp64 oracle (oracle/dense.py).

Tolerances count roundings. U is fp32's unit roundoff, RO the type's, TINY half of fp16's
smallest step. A sum of k products in fp32, in any order, is off by at most k roundings of
the running sum, each at most U (2 U where the matrix cores cut instead of rounding) times
the sum of the terms' magnitudes. Where dz is rounded to the arrays' type before it is
multiplied, each of its terms carries RO; where z is read back rounded, RO of z more."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from oracle import dense as D

U = 2.0 ** -24
RO = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}
TINY = {"f32": 0.0, "f16": 2.0 ** -25, "bf16": 0.0}
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SEED, OFFSET = 0x9E3779B97F4A7C15, (5 << 40) + 3


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
    assert got.shape == ref.shape, what
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} off, worst {np.nanmax(np.abs(got - ref)):.3e}"


# ---- dropout -------------------------------------------------------------------------

@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("shape", [(1,), (7,), (8,), (9,), (3, 5), (33, 47, 64), (1000, 3), (1, 100_001), (4096, 520)])
def test_dropout(dev, shape, dt):
    from sphere_rasterization_amd import appearance as A
    rng = np.random.default_rng(len(shape) + shape[-1])
    x, r = _put(rng.standard_normal(shape), dt, dev), _put(rng.standard_normal(shape), dt, dev)
    for p in (0.1, 0.5, 0.75):
        scale = float(np.float32(1.0 / (1.0 - p)))
        keep = D.kept(shape, p, SEED, OFFSET)
        for res in (None, r):
            got = A.dropout(x, p, (SEED, OFFSET), residual=res)
            want = np.where(keep, _np(x) * scale, 0.0) + (0.0 if res is None else _np(res))
            tol = RO[dt] * np.abs(want) + 2 * U * (np.abs(want) + np.abs(_np(x)) * scale) + TINY[dt]
            _check(got, want, tol, f"p {p}")
            if res is None:
                assert np.array_equal(_np(got) == 0.0, ~keep | (_np(x) == 0.0))
        assert torch.equal(A.dropout_backward(x, p, (SEED, OFFSET)), A.dropout(x, p, (SEED, OFFSET)))
    assert torch.equal(A.dropout(x, 0.0, None), x) and torch.equal(A.dropout(x, 0.0, None, residual=r), (x.float() + r.float()).to(x.dtype))
    assert torch.equal(A.dropout(x, 1.0, (1, 2)), torch.zeros_like(x)) and torch.equal(A.dropout(x, 1.0, (1, 2), r), r)


@pytest.mark.parametrize("p", [2.0 ** -33, 2.0 ** -32, 1e-5, 1 / 3, 1 - 2.0 ** -20, 1 - 2.0 ** -32])
def test_dropout_of_any_probability(dev, p):
    """The threshold has 32 bits: the second draw decides where the first ties."""
    from sphere_rasterization_amd import appearance as A
    n = 1_000_003
    got = A.dropout(torch.ones(n, device=dev), p, (3, 4))
    keep = D.kept((n,), p, 3, 4)
    assert np.array_equal(got.cpu().numpy() != 0.0, keep)
    # the first 16 bits tie for some of a million elements, so both outcomes of a tie are seen
    tie = D.uniform(0, n, 3, 4) >> 16 == round(p * 2.0 ** 32) >> 16
    if round(p * 2.0 ** 32) >> 16 < 65536:
        assert tie.any()


def test_dropout_strides_alignment_and_nonfinite(dev):
    from sphere_rasterization_amd import appearance as A
    rng = np.random.default_rng(9)
    for dt in ("f32", "bf16"):
        for cols in (5, 8, 64, 100):
            big = _put(rng.standard_normal((50, cols + 7)), dt, dev)
            x = big[:, 3:3 + cols]
            want = A.dropout(x.contiguous(), 0.3, (1, 2))
            assert torch.equal(A.dropout(x, 0.3, (1, 2)), want)
            assert torch.equal(A.dropout(x, 0.3, (1, 2), residual=x), A.dropout(x.contiguous(), 0.3, (1, 2), x.contiguous()))
            assert torch.equal(A.dropout(x.t(), 0.3, (1, 2)), A.dropout(x.t().contiguous(), 0.3, (1, 2)))
            one = big.reshape(-1)[1:1 + 50 * cols]
            assert torch.equal(A.dropout(one, 0.3, (1, 2)), A.dropout(one.clone(), 0.3, (1, 2)))
        x = _put(np.full(4096, np.inf), dt, dev)
        x[1::2] = float("nan")
        y, keep = A.dropout(x, 0.5, (1, 2)).float().cpu().numpy(), D.kept((4096,), 0.5, 1, 2)
        assert np.array_equal(y == 0.0, ~keep)              # what is dropped is zero, whatever it was
        assert np.isnan(y[1::2][keep[1::2]]).all() and np.isinf(y[::2][keep[::2]]).all()
    assert A.dropout(torch.empty(0, 4, device=dev), 0.5, (1, 2)).shape == (0, 4)
    assert A.dropout(torch.empty(3, 0, device=dev).t(), 0.5, (1, 2)).shape == (0, 3)
    assert A.dropout(torch.tensor(2.0, device=dev), 0.0, None).shape == ()


def test_dropout_past_32_bits(dev):
    from sphere_rasterization_amd import appearance as A
    n = (1 << 32) + 1003
    x = torch.ones(n, dtype=torch.bfloat16, device=dev)
    y = A.dropout(x, 0.5, (1, 2))
    for first in (0, (1 << 31) - 500, (1 << 32) - 500, n - 1000):
        keep = D.kept((1000,), 0.5, 1, 2, first)
        assert np.array_equal(y[first:first + 1000].float().cpu().numpy(), np.where(keep, 2.0, 0.0))


def test_state_on_the_device(dev):
    """A state's words are the seed and what is added to the offset, modulo 2^64."""
    from sphere_rasterization_amd import appearance as A
    x = torch.randn(1000, 24, device=dev)
    w = torch.randn(24, 40, device=dev)
    for seed, word, offset in ((5, 7, 11), (SEED, OFFSET, 0), ((1 << 64) - 1, (1 << 64) - 2, 5)):
        state = torch.from_numpy(np.array([seed, word], np.uint64).view(np.int64)).to(dev)
        total = (word + offset) % (1 << 64)
        assert torch.equal(A.dropout(x, 0.4, (state, offset)), A.dropout(x, 0.4, (seed, total)))
        assert torch.equal(A.linear(x, w, act="silu", p=0.4, rng=(state, offset)),
                           A.linear(x, w, act="silu", p=0.4, rng=(seed, total)))
        for a, b in zip(A.linear_backward(A.linear(x, w), x, w, act="silu", p=0.4, rng=(state, offset)),
                        A.linear_backward(A.linear(x, w), x, w, act="silu", p=0.4, rng=(seed, total))):
            assert torch.equal(a, b)


# ---- dense layers ----------------------------------------------------------------------

SHAPES = [  # rows, in, out
    (1, 1, 1), (1, 64, 32), (3, 5, 7), (2, 7, 3), (17, 8, 8), (33, 24, 32), (64, 64, 64), (65, 63, 66), (129, 130, 31),
    (300, 32, 64), (1000, 3, 5), (5, 1000, 9), (1, 2048, 257), (2, 600, 1030), (16, 300, 500), (31, 129, 72), (70, 257, 129),
    (5000, 24, 32), (4097, 33, 1), (3000, 64, 48), (257, 512, 640), (300, 264, 520), (40000, 16, 3), (20001, 65, 70)]
KINDS = [  # act, bias, residual, p, order
    ("none", None, False, 0.0, "io"), ("silu", "same", True, 0.1, "oi"), ("gelu", "f32", False, 0.5, "io"),
    ("relu", "same", True, 0.0, "oi"), ("none", "f32", True, 0.25, "oi"), ("gelu", "same", True, 0.0, "io"),
    ("silu", None, False, 0.0, "io")]


def _layer(rng, m, k, n, dt, bias, residual, order, dev):
    x = _put(rng.standard_normal((m, k)) * rng.uniform(0.5, 1.5, k), dt, dev)
    w = rng.standard_normal((k, n)) * k ** -0.5
    w = _put(w, dt, dev) if order == "io" else _put(w.T.copy(), dt, dev).t()
    b = None if bias is None else _put(0.3 * rng.standard_normal(n), "f32" if bias == "f32" else dt, dev)
    r = _put(rng.standard_normal((m, n)), dt, dev) if residual else None
    return x, w, b, r, _put(rng.standard_normal((m, n)), dt, dev)


def _e_act(z, kind, dt):
    """Error of the activation itself: fp32's roundings of z, gelu's fit (its 16-bit form's is
    counted in tenths of a rounding of the result, below)."""
    if kind in ("none", "relu"):
        return 0.0 * z
    return 8 * U * (1 + np.abs(z)) + (1.6e-7 * np.abs(z) + (1.9e-6 if dt != "f32" else 0.0) if kind == "gelu" else 0.0)


def _bounds(x, w, b, z, dt):
    """Bound on the computed z."""
    k = x.shape[1]
    return 2 * (k + 8) * U * (np.abs(x) @ np.abs(w) + (0.0 if b is None else np.abs(b)))


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("at", range(len(SHAPES)))
def test_linear(dev, at, dt):
    from sphere_rasterization_amd import appearance as A
    m, k, n = SHAPES[at]
    for which in (at % len(KINDS), (at + 3) % len(KINDS)):
        kind, bias, residual, p, order = KINDS[which]
        rng = np.random.default_rng(100 * at + which)
        x, w, b, r, dy = _layer(rng, m, k, n, dt, bias, residual, order, dev)
        more = dict(act=kind, p=p, rng=(SEED, OFFSET) if p else None)
        xn, wn, bn, rn, dn = (None if t is None else _np(t) for t in (x, w, b, r, dy))
        f = D.linear(xn, wn, bn, kind, rn, p, SEED, OFFSET)
        z = f["z"]
        e_z = _bounds(xn, wn, bn, z, dt)
        s = float(np.float32(1 / (1 - p)))
        keep = D.kept(z.shape, p, SEED, OFFSET) if p else np.ones(z.shape, bool)
        y = A.linear(x, w, b, residual=r, **more)
        e_y = s * keep * (1.13 * e_z + _e_act(z, kind, dt) + 2 * U * np.abs(D.act(z, kind)))
        _check(y, f["y"], e_y + (RO[dt] * 1.2 + 2 * U) * np.abs(f["y"]) + 2 * U * np.abs(rn if residual else 0.0) + TINY[dt],
               f"y {kind}")
        if dt != "f32":
            # a rounding is at most RO of each value: so in the norm, with a tenth for the sums
            assert np.linalg.norm(_np(y) - f["y"]) <= 1.1 * RO[dt] * np.linalg.norm(f["y"]) + TINY[dt] * z.size ** 0.5
        y2, pre = A.linear_forward(x, w, b, residual=r, **more)
        assert torch.equal(y, y2)
        e_pre = np.zeros_like(z)
        if pre is not None:
            _check(pre, z, e_z + RO[dt] * np.abs(z) + TINY[dt], "pre")
            e_pre = RO[dt] * np.abs(z) + TINY[dt]
        g = D.linear_backward(dn, xn, wn, bn, kind, p, SEED, OFFSET)
        d = s * keep * np.abs(dn)
        e_dz = d * ((e_z + e_pre + 8 * U + 1.6e-7) if kind in ("silu", "gelu") else 0.0) + 2 * U * np.abs(g["dz"])
        if kind == "relu":
            e_dz = e_dz + d * (np.abs(z) <= e_z + e_pre)
        shaped = kind != "none" or p > 0
        e_in = e_dz + (RO[dt] * (np.abs(g["dz"]) + e_dz) + TINY[dt] if shaped and dt != "f32" else 0.0)
        a_dz = np.abs(g["dz"]) + e_in
        dx, dw, db = A.linear_backward(dy, x, w, b, pre=pre, **more)
        top = lambda v: RO[dt] * np.abs(v) + TINY[dt]
        _check(dx, g["dx"], e_in @ np.abs(wn).T + 2 * (n + 8) * U * (a_dz @ np.abs(wn).T) + top(g["dx"]), f"dx {kind}")
        _check(dw, g["dw"], np.abs(xn).T @ e_in + 2 * (m + 8) * U * (np.abs(xn).T @ a_dz) + top(g["dw"]), f"dw {kind}")
        bt = "f32" if bias == "f32" else dt
        _check(db, g["db"], e_in.sum(0) + (m + 8) * U * a_dz.sum(0) + RO[bt] * np.abs(g["db"]) + TINY[bt], f"db {kind}")
        assert dw.stride() == w.stride() or 1 in w.shape
        again = A.linear_backward(dy, x, w, b, pre=pre, **more)
        assert all(torch.equal(u, v) for u, v in zip((dx, dw, db), again)), "not the same bits twice"
        # z computed anew is the z that the forward rounded
        for u, v in zip(A.linear_backward(dy, x, w, b, **more), (dx, dw, db)):
            assert torch.equal(u, v)
        one = A.linear_backward(dy, x, w, b, pre=pre, want=("weight",), **more)
        assert one[0] is None and one[2] is None and torch.equal(one[1], dw)


@pytest.mark.parametrize("dt,m,k,n", [("bf16", 3000, 520, 1030), ("f16", 2050, 1030, 264), ("f32", 1500, 300, 700),
                                      ("bf16", 120_000, 96, 40), ("f32", 300_000, 24, 32), ("bf16", 4, 8192, 1000),
                                      ("f16", 9, 777, 4097), ("bf16", 1000, 2000, 1999)])
def test_linear_larger(dev, dt, m, k, n):
    """Larger layers against torch in 64 bits: the error in the norm. Each output is rounded once
    (at most RO, in the norm too) after sums whose error is far below; a product with dz, itself
    rounded and computed from a rounded z, adds at most 2 RO in the norm of the terms, which for
    independent terms is the norm of the result."""
    from sphere_rasterization_amd import appearance as A
    gen = torch.Generator(device=dev).manual_seed(m + n)
    randn = lambda *s: torch.randn(*s, generator=gen, device=dev)
    for order in ("io", "oi"):
        x, dy = randn(m, k).to(DT[dt]), randn(m, n).to(DT[dt])
        w = (randn(k, n) * k ** -0.5).to(DT[dt]) if order == "io" else (randn(n, k) * k ** -0.5).to(DT[dt]).t()
        b = randn(n).to(DT[dt])
        z = x.double() @ w.double().contiguous() + b.double()
        y, pre = A.linear_forward(x, w, b, act="gelu")
        dx, dw, db = A.linear_backward(dy, x, w, b, act="gelu", pre=pre)
        ref = z * torch.special.ndtr(z)
        dz = dy.double() * (torch.special.ndtr(z) + z * torch.exp(-0.5 * z * z) * 0.3989422804014327)
        most = max(RO[dt], 2e-6)
        for what, got, want, times in (("y", y, ref, 1.0), ("dx", dx, dz @ w.double().t().contiguous(), 3.0),
                                       ("dw", dw, x.double().t().contiguous() @ dz, 3.0), ("db", db, dz.sum(0), 3.0)):
            err = float((got.double() - want).norm() / want.norm())
            assert err <= times * most, (what, order, err)


def test_linear_drops_what_dropout_drops(dev):
    """The epilogue's mask is that of dropout over the layer's result, and so is its arithmetic."""
    from sphere_rasterization_amd import appearance as A
    for m, k, n in ((1, 64, 7), (100, 24, 33), (513, 130, 64), (40, 300, 515), (7, 500, 1001)):
        x, w, b, r = (torch.randn(*s, device=dev) for s in ((m, k), (k, n), (n,), (m, n)))
        for act in ("none", "silu"):
            plain = A.linear(x, w, b, act=act)
            assert torch.equal(A.linear(x, w, b, act=act, p=0.3, rng=(8, 9)), A.dropout(plain, 0.3, (8, 9)))
            assert torch.equal(A.linear(x, w, b, act=act, residual=r, p=0.3, rng=(8, 9)), A.dropout(plain, 0.3, (8, 9), r))


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
def test_linear_strides_and_alignment(dev, dt):
    """Rows apart, arrays at any element, W of either order and of rows apart: the same bits."""
    from sphere_rasterization_amd import appearance as A
    rng = np.random.default_rng(5)
    for m, k, n in ((5, 32, 24), (70, 24, 40), (130, 136, 72), (300, 61, 45), (3, 520, 100), (600, 200, 128)):
        for order in ("io", "oi"):
            x, w, b, r, dy = _layer(rng, m, k, n, dt, "same", True, order, dev)

            def apart(t, by, at):
                rows, cols = t.shape
                big = torch.full((rows * (cols + by) + at,), float("nan"), dtype=t.dtype, device=dev)
                v = big[at:].view(rows, cols + by)[:, :cols]
                return v.copy_(t)

            more = dict(act="gelu", p=0.2, rng=(1, 2))
            y, pre = A.linear_forward(x, w, b, residual=r, **more)
            grads = A.linear_backward(dy, x, w, b, pre=pre, **more)
            for by, at in ((1, 0), (8, 0), (3, 1), (0, 1), (16, 8)):
                v = [apart(t, by, at) for t in (x, r, dy)]
                wv = apart(w, by, at) if order == "io" else apart(w.t(), by, at).t()
                bv = apart(b[None], 0, at)[0]
                y2, pre2 = A.linear_forward(v[0], wv, bv, residual=v[1], **more)
                tol = 4 * RO[dt] * y.float().norm() + 1e-6
                assert float((y2.float() - y.float()).norm()) <= tol
                for g, h in zip(A.linear_backward(v[2], v[0], wv, bv, pre=pre2, **more), grads):
                    assert float((g.float() - h.float()).norm()) <= 4 * RO[dt] * float(h.float().norm()) + 1e-6
    x3 = torch.randn(4, 3, 5, 16, device=dev).to(DT[dt])
    w = torch.randn(16, 6, device=dev).to(DT[dt])
    for t in (x3, x3.transpose(0, 2), x3[:, 1:2], x3[..., ::2, :]):
        got = A.linear(t, w)
        assert got.shape == t.shape[:-1] + (6,)
        assert torch.equal(got.reshape(-1, 6), A.linear(t.contiguous().reshape(-1, 16), w))
    assert A.linear(x3[0, 0, 0], w).shape == (6,)
    assert torch.equal(A.linear(x3[0, 0, :1].expand(5, 16), w), A.linear(x3[0, 0, :1].repeat(5, 1), w))


def test_linear_of_nothing(dev):
    from sphere_rasterization_amd import appearance as A
    for dt in (torch.float32, torch.bfloat16):
        z = lambda *s: torch.zeros(*s, dtype=dt, device=dev)
        assert A.linear(z(0, 8), z(8, 4)).shape == (0, 4)
        assert A.linear(z(3, 8), z(8, 0)).shape == (3, 0)
        dx, dw, db = A.linear_backward(z(0, 4), z(0, 8), z(8, 4), z(4), act="silu")
        assert dx.shape == (0, 8) and torch.equal(dw, z(8, 4)) and torch.equal(db, z(4))
        dx, dw, db = A.linear_backward(z(3, 0), z(3, 8), z(8, 0))
        assert torch.equal(dx, z(3, 8)) and dw.shape == (8, 0) and db.shape == (0,)
        # no inputs: the bias alone
        b, r, dy = torch.randn(4, device=dev).to(dt), torch.randn(3, 4, device=dev).to(dt), torch.randn(3, 4, device=dev).to(dt)
        assert torch.equal(A.linear(z(3, 0), z(0, 4), b), b.expand(3, 4))
        assert torch.equal(A.linear(z(3, 0), z(0, 4)), z(3, 4))
        dx, dw, db = A.linear_backward(dy, z(3, 0), z(0, 4), b)
        assert dx.shape == (3, 0) and dw.shape == (0, 4)
        assert torch.allclose(db.float(), dy.float().sum(0), rtol=1e-2, atol=1e-6)


def test_linear_nonfinite(dev):
    """Infinities and NaN go where the formula takes them, and no further."""
    from sphere_rasterization_amd import appearance as A
    for dt in ("f32", "f16", "bf16"):
        for m, k, n in ((20, 40, 24), (3, 300, 70), (150, 200, 130)):
            rng = np.random.default_rng(m)
            x, w, b, r, dy = _layer(rng, m, k, n, dt, "same", True, "io", dev)
            clean = A.linear(x, w, b, residual=r)
            x2 = x.clone()
            x2[1, 3] = float("inf")
            x2[2, 5] = float("nan")
            y = A.linear(x2, w, b, residual=r)
            assert torch.isnan(y[2]).all()
            sign = torch.sign(w[3].float())
            assert torch.equal(y[1].float(), torch.where(sign == 0, torch.nan, sign * float("inf")).to(y.dtype).float()) or bool((sign == 0).any())
            others = [i for i in range(m) if i not in (1, 2)]
            assert torch.equal(y[others], clean[others])
            w2 = w.clone()
            w2[0, 7] = float("nan")
            y = A.linear(x, w2, b)
            assert torch.isnan(y[:, 7]).all() and not torch.isnan(y[:, :7]).any() and not torch.isnan(y[:, 8:]).any()
            dy2 = dy.clone()
            dy2[1, 2] = float("inf")
            dx, dw, db = A.linear_backward(dy2, x, w, b)
            assert not torch.isfinite(db[2]) and torch.isfinite(db[:2]).all() and torch.isfinite(db[3:]).all()
            assert torch.isfinite(dx[others[:1]]).all() and not torch.isfinite(dx[1]).any()
            assert torch.isfinite(dw[:, 3:]).all() and not torch.isfinite(dw[:, 2]).any()


def test_linear_past_32_bits(dev):
    """More than 2^32 elements of x and of y, checked at both ends and around the seams."""
    from sphere_rasterization_amd import appearance as A
    m = (1 << 26) + 77
    x = torch.zeros(m, 64, dtype=torch.bfloat16, device=dev)
    w = torch.randn(64, 64, device=dev).to(torch.bfloat16)
    b = torch.randn(64, device=dev).to(torch.bfloat16)
    spots = [0, (1 << 25) - 40, (1 << 26) - 40, m - 60]
    for s in spots:
        x[s:s + 60] = torch.randn(60, 64, device=dev).to(torch.bfloat16)
    y = A.linear(x, w, b, act="silu")
    small = [A.linear(x[s:s + 60].clone(), w, b, act="silu") for s in spots]
    for s, ref in zip(spots, small):
        assert float((y[s:s + 60].float() - ref.float()).norm()) <= 2 * RO["bf16"] * float(ref.float().norm())
    dx, dw, db = A.linear_backward(x, x, w, b, act="silu", pre=A.linear_forward(x, w, b, act="silu")[1])
    for s in spots:
        v = x[s:s + 60].clone()
        gx = A.linear_backward(v, v, w, b, act="silu")[0]
        assert float((dx[s:s + 60].float() - gx.float()).norm()) <= 3 * RO["bf16"] * float(gx.float().norm())
    # the last two stretches overlap: each row counts once
    v = x[torch.unique(torch.cat([torch.arange(s, s + 60) for s in spots])).to(dev)]
    want = A.linear_backward(v, v, w, b, act="silu")[1].double()
    # both are rounded once, and so are their terms
    assert float((dw.double() - want).norm()) <= 4 * RO["bf16"] * float(want.norm())


def test_autograd(dev):
    """One layer after another with everything on, against torch's own gradients in 64 bits."""
    from sphere_rasterization_amd import appearance as A
    torch.manual_seed(3)
    x = torch.randn(6, 50, 24, device=dev, requires_grad=True)
    w1, b1 = torch.randn(24, 40, device=dev, requires_grad=True), torch.randn(40, device=dev, requires_grad=True)
    w2 = torch.randn(24, 40, device=dev, requires_grad=True)              # [out, in], handed over transposed
    row = torch.randn(24, device=dev, requires_grad=True)                 # broadcast over all rows
    state = torch.tensor([5, 6], device=dev)

    def net(x, w1, b1, w2, row):
        h = A.linear(x, w1, b1, act="silu", p=0.2, rng=(1, 2))
        h = A.linear(h, w2.t(), residual=x + row, act="gelu", p=0.1, rng=(state, 1))
        return A.dropout(h, 0.3, (state, 2), residual=x)

    def ref(x, w1, b1, w2, row):
        drop = lambda v, p, s, o: v * torch.from_numpy(D.kept(tuple(v.shape), p, s, o)).to(dev) / (1 - p)
        h = drop(torch.nn.functional.silu(x @ w1 + b1), 0.2, 1, 2)
        h = drop(torch.nn.functional.gelu(h @ w2.t()), 0.1, 5, 7) + x + row
        return drop(h, 0.3, 5, 8) + x

    leaves = (x, w1, b1, w2, row)
    wide = [t.detach().double().requires_grad_() for t in leaves]
    dy = torch.randn(6, 50, 24, device=dev)
    y, yd = net(*leaves), ref(*wide)
    assert float((y.double() - yd).norm() / yd.norm()) <= 1e-6
    y.backward(dy)
    yd.backward(dy.double())
    for t, u in zip(leaves, wide):
        assert float((t.grad.double() - u.grad).norm() / u.grad.norm()) <= 2e-6
    # gradients of what is wanted alone
    (gb,) = torch.autograd.grad(net(x.detach(), w1.detach(), b1, w2.detach(), row.detach()), b1, dy)
    assert torch.allclose(gb, b1.grad, rtol=1e-5, atol=1e-5)
    (gr,) = torch.autograd.grad(A.linear(x.detach(), w1.detach(), residual=(r := torch.zeros(6, 50, 40, device=dev, requires_grad=True))), r,
                                torch.ones(6, 50, 40, device=dev))
    assert torch.equal(gr, torch.ones_like(gr))


def test_a_changed_state_is_seen_by_autograd(dev):
    from sphere_rasterization_amd import appearance as A
    state, x = torch.tensor([5, 6], device=dev), torch.randn(8, 8, device=dev, requires_grad=True)
    for call in (lambda: A.dropout(x, 0.5, (state, 0)), lambda: A.linear(x, torch.randn(8, 8, device=dev), p=0.5, rng=(state, 0))):
        y = call()
        state.add_(1)
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            y.sum().backward()


def test_gradients_against_differences(dev):
    """Along random directions, in fp32: (f(t + h v) - f(t - h v)) / 2 h. The loss is a sum of
    about 2000 values of order one in fp64, so the difference is off by its outputs' fp32
    roundings, U |f| / h, and h^2 times a third derivative of order one."""
    from sphere_rasterization_amd import appearance as A
    torch.manual_seed(4)
    t = [torch.randn(*s, device=dev) for s in ((50, 30), (30, 40), (40,), (50, 40))]
    dy, h = torch.randn(50, 40, device=dev), 2.0 ** -8
    f = lambda x, w, b, r: float((A.linear(x, w * 30 ** -0.5, b, act="gelu", residual=r, p=0.25, rng=(3, 4)).double() * dy).sum())
    leaves = [v.clone().requires_grad_() for v in t]
    y = A.linear(leaves[0], leaves[1] * 30 ** -0.5, leaves[2], act="gelu", residual=leaves[3], p=0.25, rng=(3, 4))
    y.backward(dy)
    for i, leaf in enumerate(leaves):
        v = torch.randn_like(t[i])
        v /= v.norm()
        up, down = ([u + s * h * v if j == i else u for j, u in enumerate(t)] for s in (1, -1))
        got, want = (f(*up) - f(*down)) / (2 * h), float((leaf.grad * v).sum())
        assert abs(got - want) <= 2000 ** 0.5 * 8 * U / h + 4 * h * h * float(dy.norm()), (i, got, want)


def test_other_stream_and_graph(dev):
    """A training step on its own stream, captured, replayed with a state that moves on, two
    captured graphs side by side: each replay equals the eager step of its state."""
    from sphere_rasterization_amd import appearance as A
    torch.manual_seed(5)

    def make(m, k, n, dt):
        return [torch.randn(*s, device=dev).to(dt) for s in ((m, k), (k, n), (n,), (m, n), (m, n))]

    def step(t, rng):
        x, w, b, r, dy = t
        y, pre = A.linear_forward(x, w, b, act="silu", residual=r, p=0.3, rng=rng)
        grads = A.linear_backward(dy, x, w, b, act="silu", pre=pre, p=0.3, rng=rng)
        return (y, A.dropout(y, 0.2, (rng[0], rng[1] + 1), residual=r)) + grads

    side = torch.cuda.Stream()
    sets = [make(700, 24, 32, torch.bfloat16), make(300, 200, 130, torch.float32), make(2, 900, 500, torch.float16)]
    states = [torch.tensor([7, 100 * i], device=dev) for i in range(len(sets))]
    want = [step(t, (7, 100 * i)) for i, t in enumerate(sets)]
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        outs = [step(t, (s, 0)) for t, s in zip(sets, states)]
    side.synchronize()
    assert all(torch.equal(p, q) for a, b in zip(want, outs) for p, q in zip(a, b))
    graphs, held = [], []
    for t, s in zip(sets, states):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            held.append(step(t, (s, 0)))
            s[1:].add_(1)
        graphs.append(g)
    for k in range(4):
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for i, t in enumerate(sets):
            eager = step(t, (7, 100 * i + k))
            assert all(torch.equal(p, q) for p, q in zip(eager, held[i])), f"replay {k} of graph {i}"
            assert int(states[i][1]) == 100 * i + k + 1


def test_captured_backward(dev):
    """A whole training step through autograd captured, and replayed with other inputs."""
    from sphere_rasterization_amd import appearance as A
    torch.manual_seed(6)
    x, dy = torch.randn(500, 24, device=dev), torch.randn(500, 3, device=dev)
    w1, w2 = (torch.randn(*s, device=dev, requires_grad=True) for s in ((24, 32), (32, 3)))
    state = torch.tensor([1, 0], device=dev)

    def step(x, w1, w2, rng):
        h = A.linear(x, w1, act="gelu", p=0.1, rng=rng)
        return torch.autograd.grad(A.linear(h, w2), (w1, w2), dy)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(x, w1, w2, (state, 0))
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        held = step(x, w1, w2, (state, 0))
        state[1:].add_(1)
    for k in range(3):
        x.copy_(torch.randn(500, 24, device=dev))
        g.replay()
        torch.cuda.synchronize()
        fresh = [t.detach().clone().requires_grad_() for t in (w1, w2)]
        assert all(torch.equal(p, q) for p, q in zip(step(x, *fresh, (1, k)), held))


def test_refusals(dev):
    from sphere_rasterization_amd import _lib as L
    from sphere_rasterization_amd import appearance as A
    x, w, b, y = (torch.zeros(*s, device=dev) for s in ((4, 8), (8, 3), (3,), (4, 3)))
    state = torch.zeros(2, dtype=torch.int64, device=dev)
    for call in (lambda: A.linear(x, w.cpu()), lambda: A.linear(x, w.half()), lambda: A.linear(x, w.t()),
                 lambda: A.linear(x, w, b[:2]), lambda: A.linear(x, w, b.half()), lambda: A.linear(x.half(), w.half(), b.bfloat16()),
                 lambda: A.linear(x, w, b.cpu()), lambda: A.linear(x, w, residual=y[:3]), lambda: A.linear(x, w, residual=y.half()),
                 lambda: A.linear(x, w, residual=b), lambda: A.linear(x, w, p=0.5), lambda: A.linear(x, w, p=0.5, rng=(state.cpu(), 0)),
                 lambda: A.linear(x, w, p=0.5, rng=(state.int(), 0)), lambda: A.linear(x, w, p=0.5, rng=(state[:1], 0)),
                 lambda: A.linear(x, w, p=0.5, rng=(torch.zeros(4, dtype=torch.int64, device=dev)[::2], 0)),
                 lambda: A.linear_backward(y[:3], x, w), lambda: A.linear_backward(y.half(), x, w),
                 lambda: A.linear_backward(y, x, w, pre=y[:2]), lambda: A.linear_backward(y, x, w, pre=y.half()),
                 lambda: A.dropout(x, 0.5, (1, 2), residual=x[:2]), lambda: A.dropout(x, 0.5, (1, 2), residual=x.half()),
                 lambda: A.dropout(x, 2.0, (1, 2)), lambda: A.dropout(x, 0.5, None)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(L.SplatError):
        A.linear(torch.zeros(1, (1 << 20) + 1, device=dev), torch.zeros((1 << 20) + 1, 1, device=dev))


def test_the_example_runs_and_its_gradients_fit(dev):
    """The example's shading network: dense layers, normalisation and dropout together, against
    torch's operations and gradients in 64 bits. And its loop, with dropout, for running."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "train_appearance.py")
    spec = importlib.util.spec_from_file_location("train_appearance", path)
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    torch.manual_seed(8)
    leaves = [torch.randn(*s, device=dev) for s in ((1, 777, 16), (16, 32), (32,), (32,), (32, 32), (32,), (32, 3), (3,))]
    wide = [t.double().requires_grad_() for t in leaves]
    leaves = [t.requires_grad_() for t in leaves]
    dy = torch.randn(1, 777, 3, device=dev)
    got = ex.shade(*leaves, 0.25, (5, 6))

    def ref(img, w1, gain, bias, wh, bh, w2, bias2):
        h = torch.nn.functional.group_norm((img @ w1).transpose(1, 2), ex.GROUPS, gain, bias).transpose(1, 2)
        h = torch.nn.functional.silu(h)
        keep = torch.from_numpy(D.kept((1, 777, 32), 0.25, 5, 6)).to(dev)
        h = h + torch.nn.functional.silu(h @ wh + bh) * keep / 0.75
        return h @ w2 + bias2

    want = ref(*wide)
    # some ten products and sums in fp32, each within a few tens of roundings in the norm
    assert float((got.double() - want).norm() / want.norm()) <= 1e-5
    got.backward(dy)
    want.backward(dy.double())
    for t, u in zip(leaves, wide):
        assert float((t.grad.double() - u.grad).norm() / u.grad.norm()) <= 2e-5
    assert all(np.isfinite(ex.train(steps=3, n=2000, width=64, height=48, dropout=0.1)))


EDGES = [  # rows, in, out: around the kernels' own sizes
    (16, 64, 64), (15, 65, 64), (17, 64, 65), (16, 72, 136), (1, 32, 8), (1, 8, 8), (2, 4, 4), (3, 3, 3), (1, 3, 2),
    (8, 64, 1), (9, 1, 64), (64, 33, 33), (16, 4096, 40), (3, 2056, 24), (16, 520, 8200), (255, 128, 256), (256, 32, 256),
    (257, 40, 264), (128, 1000, 128), (129, 96, 384), (513, 72, 72), (2048, 80, 80), (300, 65, 4), (1000, 5000, 70), (70, 67, 3001)]


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("order", ["io", "oi"])
@pytest.mark.parametrize("m,k,n", EDGES)
def test_linear_at_its_kernels_edges(dev, m, k, n, order, dt):
    """Layers around the sizes at which another kernel, tile or split takes over. The activation is
    none, so that every bound is one of sums and of one rounding."""
    from sphere_rasterization_amd import appearance as A
    rng = np.random.default_rng(m + k + n)
    x, w, b, r, dy = _layer(rng, m, k, n, dt, "same", True, order, dev)
    xn, wn, bn, rn, dn = (_np(t) for t in (x, w, b, r, dy))
    f = D.linear(xn, wn, bn, "none", rn)
    y, pre = A.linear_forward(x, w, b, residual=r)
    assert pre is None
    top = lambda v: RO[dt] * np.abs(v) + TINY[dt]
    _check(y, f["y"], _bounds(xn, wn, bn, f["z"], dt) + 2 * U * (np.abs(f["y"]) + np.abs(rn)) + top(f["y"]), "y")
    dx, dw, db = A.linear_backward(dy, x, w, b)
    g = D.linear_backward(dn, xn, wn, bn)
    _check(dx, g["dx"], 2 * (n + 8) * U * (np.abs(dn) @ np.abs(wn).T) + top(g["dx"]), "dx")
    _check(dw, g["dw"], 2 * (m + 8) * U * (np.abs(xn).T @ np.abs(dn)) + top(g["dw"]), "dw")
    _check(db, g["db"], (m + 8) * U * np.abs(dn).sum(0) + top(g["db"]), "db")
    # with the activation, its gradient against the same formula on the kernels' own z in 64 bits
    y2, pre = A.linear_forward(x, w, b, act="silu", p=0.3, rng=(1, 2))
    grads = A.linear_backward(dy, x, w, b, act="silu", pre=pre, p=0.3, rng=(1, 2))
    g = D.linear_backward(dn, xn, wn, bn, "silu", 0.3, 1, 2)
    for got, want, what in zip(grads, (g["dx"], g["dw"], g["db"]), ("dx", "dw", "db")):
        size = np.linalg.norm(want)
        # rounded once, from terms that carry at most one rounding of z and one of dz (each below RO
        # of the terms, whose norm is at most the square root of their number times that of the sum's)
        assert np.linalg.norm(_np(got) - want) <= (2.5 * RO[dt] + 2e-5) * max(size, np.linalg.norm(g["dz"])) + TINY[dt] * want.size ** 0.5, what


def test_two_calls_of_one_layer_at_once(dev):
    """Forward and backward of the same arrays on two streams: each has a workspace of its own."""
    from sphere_rasterization_amd import appearance as A
    torch.manual_seed(9)
    for m, k, n in ((4000, 32, 32), (500, 400, 300), (3, 1000, 600)):
        x, w, b, dy = (torch.randn(*s, device=dev) for s in ((m, k), (k, n), (n,), (m, n)))
        run = lambda: (A.linear(x, w, b, act="gelu"),) + A.linear_backward(dy, x, w, b, act="gelu")
        want = run()
        streams = [torch.cuda.Stream() for _ in range(2)]
        torch.cuda.synchronize()
        outs = []
        for _ in range(5):
            for s in streams:
                with torch.cuda.stream(s):
                    outs.append(run())
        torch.cuda.synchronize()
        for o in outs:
            assert all(torch.equal(p, q) for p, q in zip(o, want))


def test_c_calls_with_strides_and_given_outputs(dev):
    """Outputs a stride apart, gradients of W in the other order than W, and the elements between
    rows left as they were."""
    import ctypes as C
    from sphere_rasterization_amd import _lib as L
    from sphere_rasterization_amd import appearance as A
    torch.manual_seed(10)
    stream = torch.cuda.current_stream().cuda_stream
    for m, k, n in ((300, 24, 40), (200, 136, 264), (100, 65, 77), (5, 320, 96)):
        x, w, b, dy = (torch.randn(*s, device=dev) for s in ((m, k), (k, n), (n,), (m, n)))
        y = torch.full((m, n + 5), -7.0, device=dev)
        dx = torch.full((m, k + 3), -7.0, device=dev)
        dw = torch.full((n, k + 2), -7.0, device=dev)                  # by outputs
        db = torch.empty(n, device=dev)
        d = L.splat_dense(0, 0, L.SPLAT_ACT_SILU, k, n, m, k, n, 1, n, n + 5, k + 3, 1, k + 2, L.splat_drop())
        nbytes = max(L.splat_linear_workspace_bytes(d, False), L.splat_linear_workspace_bytes(d, True), 16)
        ws = torch.empty(nbytes, dtype=torch.uint8, device=dev)
        L.splat_linear(d, x.data_ptr(), w.data_ptr(), b.data_ptr(), None, y.data_ptr(), None, ws.data_ptr(), nbytes, stream)
        ref = A.linear(x, w, b, act="silu")
        assert torch.equal(y[:, :n], ref) and bool((y[:, n:] == -7.0).all())
        d.y_stride = n
        nbytes = max(L.splat_linear_workspace_bytes(d, True), 16)
        ws = torch.empty(nbytes, dtype=torch.uint8, device=dev)
        L.splat_linear_bwd(d, dy.data_ptr(), x.data_ptr(), w.data_ptr(), b.data_ptr(), None, dx.data_ptr(), dw.data_ptr(),
                           db.data_ptr(), ws.data_ptr(), nbytes, stream)
        gx, gw, gb = A.linear_backward(dy, x, w, b, act="silu")
        assert torch.equal(dx[:, :k], gx) and bool((dx[:, k:] == -7.0).all()) and torch.equal(db, gb)
        assert float((dw[:, :k].t() - gw).norm() / gw.norm()) <= 1e-5 and bool((dw[:, k:] == -7.0).all())


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("m,k,n", [(65536, 24, 72), (70000, 33, 100), (66001, 64, 256), (66500, 7, 129), (65535, 48, 65)])
def test_many_rows_of_more_outputs(dev, m, k, n, dt):
    """Many rows of few inputs and 65 to 256 outputs, which are taken in slices of them, with and
    without what goes with the product; dropout over them is that of dropout alone."""
    from sphere_rasterization_amd import appearance as A
    rng = np.random.default_rng(n)
    x, w, b, r, dy = _layer(rng, m, k, n, dt, "same", True, "io", dev)
    y, pre = A.linear_forward(x, w, b, act="gelu", residual=r)
    xn, wn, bn, rn = _np(x), _np(w), _np(b), _np(r)
    f = D.linear(xn, wn, bn, "gelu", rn)
    e_z = _bounds(xn, wn, bn, f["z"], dt)
    _check(pre, f["z"], e_z + RO[dt] * np.abs(f["z"]) + TINY[dt], "pre")
    e_y = 1.13 * e_z + _e_act(f["z"], "gelu", dt) + 4 * U * np.abs(f["z"]) + 2 * U * np.abs(rn) + 0.2 * RO[dt] * np.abs(f["y"] - rn)
    _check(y, f["y"], e_y + (RO[dt] + 2 * U) * np.abs(f["y"]) + TINY[dt], "y")
    assert torch.equal(y, A.linear(x, w, b, act="gelu", residual=r))
    assert torch.equal(y, A.linear(x, w.t().contiguous().t(), b, act="gelu", residual=r))
    plain = A.linear(x, w)
    _check(plain, xn @ wn, _bounds(xn, wn, None, None, dt) + RO[dt] * np.abs(xn @ wn) + TINY[dt], "product")
    got = A.linear(x, w, p=0.2, rng=(SEED, OFFSET))
    # another kernel's sums, so that a kept value may round to zero in one and not in the other
    keep = A.dropout(torch.ones_like(plain), 0.2, (SEED, OFFSET)) != 0
    assert bool((got[~keep] == 0).all())
    want = plain.float()[keep] * 1.25
    assert float((got.float()[keep] - want).norm()) <= (3 * RO[dt] + 1e-6) * float(want.norm())
    dx, dw, db = A.linear_backward(dy, x, w, b, act="gelu", pre=pre)
    wide = [t.double().requires_grad_() for t in (x, w, b)]
    torch.nn.functional.gelu(wide[0] @ wide[1] + wide[2]).backward(dy.double())
    # rounded once, with z and dz each rounded once below it; fp32: sums of m terms in parts
    for g, t, what in zip((dx, dw, db), wide, ("dx", "dw", "db")):
        assert float((g.double() - t.grad).norm() / t.grad.norm()) <= 3 * RO[dt] + 1e-5, what
