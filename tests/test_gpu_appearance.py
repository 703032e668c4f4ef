"""The appearance operators on the GPU against the fp64 oracle (oracle/appearance.py).

Tolerances are bounds on an fp32 evaluation of each formula followed by one rounding to
the array's type. U is fp32's unit roundoff, RO the type's; sums of k terms in the
kernels' order have a depth of at most 8 + 64 x 4 + n / 4096 (table gradient) and DEPTH
(group norm: batches of 8, at most 16 to a few hundred batches per thread, then trees)."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from oracle import appearance as O

U = 2.0 ** -24
RO = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}
TINY = {"f32": 0.0, "f16": 2.0 ** -25, "bf16": 0.0}       # half of f16's smallest step
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
COEFFS = (3.4445, -4.7750, 2.0315)


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


# ---- lookup -------------------------------------------------------------------------

def _ids(rng, n, rows, skew, kind):
    ids = (np.exp(rng.uniform(0, np.log(rows + 1.0), n)) - 1).astype(np.int64) if skew else rng.integers(0, rows, n)
    ids = np.minimum(ids, rows - 1)
    out = rng.random(n) < 0.05
    ids[out] = rng.choice([-1, rows, rows + 7, -(1 << 31), (1 << 31) - 1], size=int(out.sum()))
    return ids.astype(kind)


LOOKUPS = [  # n, rows, dim
    (1, 1, 1), (1, 70000, 64), (7, 3, 5), (63, 256, 3), (64, 1, 16), (257, 1000, 33), (4096, 256, 3), (4097, 511, 12),
    (5000, 512, 64), (20000, 7, 24), (9000, 1, 8), (3000, 70000, 6), (50, 40, 1031), (700, 90, 2048), (33000, 3, 130)]


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("n,rows,dim", LOOKUPS)
def test_lookup(dev, n, rows, dim, dt):
    rng = np.random.default_rng(n + rows + dim)
    from sphere_rasterization_amd import appearance as A
    for kind, scale in ((np.int32, 1.0), (np.int64, -0.37)):
        ids = _ids(rng, n, rows, False, kind)
        table = _put(rng.standard_normal((rows, dim)), dt, dev)
        got = A.lookup(table, torch.from_numpy(ids).to(dev), scale)
        s = float(np.float32(scale))
        ref = O.lookup(_np(table), ids, s)
        _check(got, ref, np.abs(ref) * (U + RO[dt]) * 1.01 + TINY[dt], "lookup")


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("n,rows,dim", LOOKUPS)
def test_lookup_backward(dev, n, rows, dim, dt):
    rng = np.random.default_rng(n * 3 + rows + dim)
    from sphere_rasterization_amd import appearance as A
    depth = 8 + 64 * 4 + n / 4096
    for kind, skew, scale in ((np.int64, False, 1.0), (np.int32, True, 0.37)):
        ids = _ids(rng, n, rows, skew, kind)
        dy = _put(rng.standard_normal((n, dim)), dt, dev)
        dev_ids = torch.from_numpy(ids).to(dev)
        s = float(np.float32(scale))
        got = A.lookup_backward(dy, dev_ids, rows, scale)
        ref, mag = O.lookup_backward(_np(dy), ids, rows, s), O.lookup_backward(np.abs(_np(dy)), ids, rows, s)
        tol = (min(depth, n) + 2) * U * mag + RO[dt] * np.abs(ref) * 1.01 + TINY[dt]
        _check(got, ref, tol, "table gradient")
        assert torch.equal(got, A.lookup_backward(dy, dev_ids, rows, scale)), "not the same bits twice"
        old = _put(rng.standard_normal((rows, dim)), dt, dev)
        acc = old.clone()
        assert A.lookup_backward(dy, dev_ids, rows, scale, out=acc, accumulate=True) is acc
        full = _np(old) + ref
        _check(acc, full, tol + 2 * (U + RO[dt]) * (np.abs(full) + np.abs(_np(old))), "accumulated gradient")


@pytest.mark.parametrize("n,rows,dim", [(4096, 12288, 5), (4096, 12289, 5), (4096, 200000, 3), (40, 70001, 8), (12, 70001, 8),
                                        (8192, 3000, 5), (8193, 3000, 5), (5000, 300000, 2), (262145, 511, 3)])
def test_lookup_backward_around_its_rules(dev, n, rows, dim):
    """Sizes on both sides of where the gradient goes over to sorting, to sorting with
    counts of its own, and to larger tiles."""
    test_lookup_backward(dev, n, rows, dim, "f32")


def test_lookup_large_and_skewed(dev):
    """Many tokens: several sort passes, both chunk levels, one row with a third of all."""
    from sphere_rasterization_amd import appearance as A
    rng = np.random.default_rng(11)
    n, rows, dim = 300_001, 300_000, 6
    ids = _ids(rng, n, rows, True, np.int32)
    ids[rng.random(n) < 0.33] = 12345
    dy = _put(rng.standard_normal((n, dim)), "f32", dev)
    got = A.lookup_backward(dy, torch.from_numpy(ids).to(dev), rows)
    ref, mag = O.lookup_backward(_np(dy), ids, rows), O.lookup_backward(np.abs(_np(dy)), ids, rows)
    _check(got, ref, (8 + 256 + n / 4096) * U * mag + U * np.abs(ref), "table gradient")


def test_lookup_few_tokens_in_one_row(dev):
    """The one-launch form with most of its tokens in one row, at the ends of its range."""
    from sphere_rasterization_amd import appearance as A
    rng = np.random.default_rng(13)
    for n, rows, dim in ((4096, 5, 3), (4096, 3000, 70), (4095, 100_000, 1), (300, 1, 600), (257, 2, 33), (4097, 9, 20)):
        ids = np.where(rng.random(n) < 0.9, rows // 2, rng.integers(0, rows, n)).astype(np.int32)
        dy = _put(rng.standard_normal((n, dim)), "f32", dev)
        t = torch.from_numpy(ids).to(dev)
        got = A.lookup_backward(dy, t, rows)
        ref, mag = O.lookup_backward(_np(dy), ids, rows), O.lookup_backward(np.abs(_np(dy)), ids, rows)
        # depth: eight waves' chains of at most 512 / 1 adds, eight in flight, then joins
        _check(got, ref, (520 + 16) * U * mag + U * np.abs(ref), "table gradient")
        acc = got.clone()
        A.lookup_backward(dy, t, rows, out=acc, accumulate=True)
        _check(acc, 2 * ref, (520 + 16) * 3 * U * mag + 4 * U * np.abs(ref), "accumulated gradient")
        assert torch.equal(got, A.lookup_backward(dy, t, rows)), "not the same bits twice"


def test_lookup_no_valid_ids_nan_and_strides(dev):
    from sphere_rasterization_amd import appearance as A
    rng = np.random.default_rng(12)
    base = torch.full((40, 11), float("nan"), device=dev)
    table = base[::2, 1:6]                                    # strided, 4-byte aligned rows
    table.copy_(_put(rng.standard_normal((20, 5)), "f32", dev))
    ids = torch.tensor([[3, 19], [-1, 20]], device=dev)
    got = A.lookup(table, ids)
    assert got.shape == (2, 2, 5)
    assert torch.equal(got[0], table[ids[0]]) and torch.equal(got[1], torch.zeros(2, 5, device=dev))
    # a NaN row of the table or of d_out stays in its own row
    t2 = table.clone()
    t2[3] = float("nan")
    y = A.lookup(t2, ids, 0.0)
    assert torch.isnan(y[0, 0]).all() and (y[0, 1] == 0).all()
    dy = torch.ones(100, 5, device=dev)
    dy[7] = float("nan")
    dy[8] = float("inf")
    i = torch.arange(100, device=dev) % 10
    i[7], i[8] = -5, 4                                        # the NaN token has no entry
    d = A.lookup_backward(dy, i, 10)
    assert torch.isinf(d[4]).all() and torch.isfinite(d[torch.arange(10, device=dev) != 4]).all()
    none = torch.full((100,), -1, device=dev)
    assert (A.lookup_backward(dy, none, 10) == 0).all()
    # strided gradients and outputs
    wide = torch.randn(100, 9, device=dev)
    out = torch.full((10, 8), 3.0, device=dev)
    A.lookup_backward(wide[:, 2:7], i, 10, out=out[:, 1:6])
    keep = i >= 0
    ref = torch.zeros(10, 5, device=dev, dtype=torch.float64).index_add_(0, i[keep], wide[keep, 2:7].double())
    assert (out[:, 1:6].double() - ref).abs().max() <= 40 * U * 10 * 4
    assert (out[:, 0] == 3).all() and (out[:, 6:] == 3).all()
    # transposed table: last axis not contiguous
    tt = torch.randn(5, 20, device=dev).t()
    assert torch.equal(A.lookup(tt, ids[0]), tt[ids[0]])
    # no tokens
    empty = torch.empty(0, dtype=torch.int32, device=dev)
    assert A.lookup(table, empty).shape == (0, 5)
    assert (A.lookup_backward(torch.empty(0, 5, device=dev), empty, 10) == 0).all()
    assert A.lookup_backward(torch.empty(3, 0, device=dev), i[:3], 10).shape == (10, 0)


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("n,rows", [(300, 40), (6000, 9), (9000, 5000)])
def test_lookup_rows_at_any_element(dev, n, rows, dt):
    """Rows of 1 to 33 elements that start anywhere in wider arrays: the same as of their
    contiguous copies, and nothing beside them is written."""
    from sphere_rasterization_amd import appearance as A
    rng = np.random.default_rng(n + rows)
    ids = torch.from_numpy(_ids(rng, n, rows, True, np.int64)).to(dev)
    for dim in (1, 2, 3, 4, 7, 8, 9, 15, 16, 17, 31, 33):
        for left, right in ((1, 0), (3, 2), (0, 1)):
            def wide(k):
                a = _put(rng.standard_normal((k, left + dim + right)), dt, dev)
                return a, a[:, left:left + dim]
            table, dy = wide(rows)[1], wide(n)[1]
            ref = torch.where(((ids >= 0) & (ids < rows))[:, None], table[ids.clamp(0, rows - 1)], torch.zeros_like(dy))
            assert torch.equal(A.lookup(table, ids), ref)
            whole = A.lookup_backward(dy.contiguous(), ids, rows, 0.37)
            for accumulate in (False, True):
                a, out = wide(rows)
                old = a.clone()
                A.lookup_backward(dy, ids, rows, 0.37, out=out, accumulate=accumulate)
                if accumulate:
                    packed = old[:, left:left + dim].contiguous()
                    A.lookup_backward(dy.contiguous(), ids, rows, 0.37, out=packed, accumulate=True)
                    assert torch.equal(out, packed)
                else:
                    assert torch.equal(out, whole)
                assert torch.equal(a[:, :left], old[:, :left])
                assert torch.equal(a[:, left + dim:], old[:, left + dim:])


def test_lookup_past_32_bits(dev):
    """A table whose offsets in bytes and in elements pass 2^31."""
    from sphere_rasterization_amd import appearance as A
    rows, dim = 40_000_001, 64
    table = torch.zeros(rows, dim, dtype=torch.float16, device=dev)
    ids = torch.tensor([rows - 1, 0, rows - 2, 33_554_432, rows], device=dev)
    table[ids[:4]] = torch.arange(1, 5, device=dev, dtype=torch.float16)[:, None]
    got = A.lookup(table, ids, 2.0)
    assert got[:, 0].tolist() == [2.0, 4.0, 6.0, 8.0, 0.0] and torch.equal(got[:, :1].expand(-1, dim), got)
    A.lookup_backward(got, ids, rows, 0.5, out=table)
    assert table[ids[:4], 5].tolist() == [1.0, 2.0, 3.0, 4.0]
    assert int((table != 0).any(dim=1).sum()) == 4


def test_lookup_backward_into_a_tensor_is_seen_by_autograd(dev):
    """A tensor that a graph has saved may not change unnoticed."""
    from sphere_rasterization_amd import appearance as A
    dy, ids = torch.ones(3, 8, device=dev), torch.tensor([0, 2, 2], device=dev)
    out, w = torch.zeros(4, 8, device=dev), torch.ones(4, 8, device=dev, requires_grad=True)
    loss = (w * out).sum()                                    # saves out
    A.lookup_backward(dy, ids, 4, out=out)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()
    with torch.inference_mode():                              # tensors without versions
        held = torch.zeros(4, 8, device=dev)
        assert torch.equal(A.lookup_backward(dy, ids, 4, out=held, accumulate=True), out)


# ---- group norm ------------------------------------------------------------------------

DEPTH = 64
NORMS = [  # images, pixels (as a shape), channels, groups
    (1, (1,), 8, 2), (2, (1, 1), 4, 4), (1, (3, 5), 1, 1), (3, (7, 11), 6, 2), (2, (33, 47), 64, 8), (1, (130, 129), 24, 4),
    (5, (17,), 40, 1), (2, (64, 3), 96, 32), (1, (9, 10), 1000, 5), (1, (40, 25), 2056, 4), (70, (4, 4), 16, 8),
    (1, (4, 5), 4096, 1), (1, (300, 200), 32, 8), (1, (500,), 9, 3)]


def _norm_inputs(rng, images, shape, c, dt, dev):
    full = (images,) + shape + (c,)
    x = _put(rng.standard_normal(full) * rng.uniform(0.5, 2, c) + rng.standard_normal(c) * 3, dt, dev)
    return x, _put(1 + 0.3 * rng.standard_normal(c), dt, dev), _put(0.3 * rng.standard_normal(c), dt, dev), full


def _norm_errors(f, x, groups):
    """Bounds on the computed xh and z, from the mean's, the variance's and the centring's
    roundings: each at most DEPTH U of the values' magnitude in the group."""
    n, c = x.shape[0], x.shape[-1]
    top = np.abs(x.reshape(n, -1, groups, c // groups)).max(axis=(1, 3)) * f["rstd"]
    top = np.broadcast_to(top[:, None, :, None], (n, x[0].size // c, groups, c // groups)).reshape(x.shape)
    e_h = DEPTH * U * (1 + np.abs(f["xh"])) * (1 + top)
    return e_h, np.abs(f["w"]) * e_h + 4 * U * (np.abs(f["z"]) + 1)


@pytest.mark.parametrize("dt,kind", [("f32", "none"), ("f32", "silu"), ("f32", "gelu"), ("f32", "relu"), ("f16", "silu"),
                                     ("bf16", "gelu"), ("bf16", "none")])
@pytest.mark.parametrize("images,shape,c,groups", NORMS)
def test_group_norm(dev, images, shape, c, groups, dt, kind):
    rng = np.random.default_rng(c + groups + images)
    from sphere_rasterization_amd import appearance as A
    x, w, b, full = _norm_inputs(rng, images, shape, c, dt, dev)
    dy = _put(rng.standard_normal(full), dt, dev)
    y, mean, rstd = A.group_norm_forward(x, groups, w, b, 1e-5, kind)
    f = O.group_norm_backward(_np(dy), _np(x), groups, _np(w), _np(b), float(np.float32(1e-5)), kind)
    e_h, e_z = _norm_errors(f, _np(x), groups)
    e_act = 8 * U * (1 + np.abs(f["z"])) + (1.6e-7 * np.abs(f["z"]) if kind == "gelu" else 0.0)
    _check(y, f["y"], 1.13 * e_z + e_act + 1.01 * RO[dt] * np.abs(f["y"]) + TINY[dt], "y")
    assert torch.equal(y, A.group_norm(x, groups, w, b, 1e-5, kind))
    dx, dw, db = A.group_norm_backward(dy, x, mean, rstd, w, b, kind)
    # dz: the slope is Lipschitz with constant at most 1 (silu 1/2, gelu 0.8); relu's jumps at 0
    d = np.abs(_np(dy))
    e_dz = d * (e_z + 8 * U + (1.6e-7 if kind == "gelu" else 0.0))
    if kind == "none":
        e_dz = np.zeros_like(d)
    if kind == "relu":
        e_dz = d * (np.abs(f["z"]) <= e_z)
    wz = np.abs(f["w"] * f["dz"])
    n, k = images, c // groups
    grp = lambda v: np.broadcast_to(v.reshape(n, -1, groups, k).mean(axis=(1, 3), keepdims=True),
                                    (n, x[0].numel() // c, groups, k)).reshape(full)
    h = np.abs(f["xh"])
    e_t1 = grp(np.abs(f["w"]) * e_dz) + DEPTH * U * grp(wz)
    e_t2 = grp(np.abs(f["w"]) * (e_dz * h + np.abs(f["dz"]) * e_h)) + DEPTH * U * grp(wz * h)
    t2 = np.abs(grp(f["w"] * f["dz"] * f["xh"]))
    r = np.broadcast_to(np.repeat(f["rstd"], k, axis=1).reshape((n,) + (1,) * len(shape) + (c,)), full)
    top = e_h / (1 + h)                                       # relative error of rstd
    tol = r * (np.abs(f["w"]) * e_dz + e_t1 + h * e_t2 + e_h * t2 + (8 * U + top) * (wz + grp(wz) + h * t2))
    _check(dx, f["dx"], tol + 1.01 * RO[dt] * np.abs(f["dx"]) + TINY[dt], "dx")
    flat = lambda v: v.reshape(-1, c).sum(0)
    _check(dw, f["dw"], flat(e_dz * h + np.abs(f["dz"]) * e_h) + DEPTH * U * flat(np.abs(f["dz"]) * h)
           + 1.01 * RO[dt] * np.abs(f["dw"]) + TINY[dt], "dw")
    _check(db, f["db"], flat(e_dz) + DEPTH * U * flat(np.abs(f["dz"])) + 1.01 * RO[dt] * np.abs(f["db"]) + TINY[dt], "db")
    again = A.group_norm_backward(dy, x, mean, rstd, w, b, kind)
    assert all(torch.equal(p, q) for p, q in zip((dx, dw, db), again)), "not the same bits twice"


def test_group_norm_far_from_zero(dev):
    """Values of mean 1000 and deviation 0.01: a variance from E[x^2] - mean^2 would be lost.
    fp32 holds such values to 2^-14, so the input itself is what the oracle reads."""
    from sphere_rasterization_amd import appearance as A
    rng = np.random.default_rng(21)
    x = _put(1000 + 0.01 * rng.standard_normal((1, 300, 8)), "f32", dev)
    x[0, 0] = 0.0                                             # a background pixel first
    x2 = x[:, 1:].contiguous()
    for v in (x, x2):
        y, mean, rstd = A.group_norm_forward(v, 2, eps=1e-12)
        f = O.group_norm(_np(v), 2, eps=float(np.float32(1e-12)))
        # centring: mean to DEPTH U relative to itself, seen in units of the deviation
        rel = DEPTH * U * 1000 * f["rstd"].max()
        _check(rstd, f["rstd"], (2 * DEPTH * U + 2 * rel * rel) * f["rstd"], "rstd")
        _check(y, f["y"], (rel + 2 * rel * rel + DEPTH * U) * (1 + np.abs(f["y"])), "y")


@pytest.mark.parametrize("images,shape,c,groups,dt,sd", [
    (1, (300, 200), 32, 8, "f32", 1e16), (1, (130, 129), 24, 4, "f32", 1e16), (2, (33, 47), 64, 8, "f32", 1e16),
    (1, (9000,), 1, 1, "f32", 1e16), (200, (3, 5), 16, 8, "f32", 1e18), (200, (3, 5), 16, 8, "bf16", 1e18)])
def test_group_norm_of_values_whose_squares_overflow(dev, images, shape, c, groups, dt, sd):
    """1e20 +- sd: the values' squares are beyond fp32, their deviations' are not, nor the
    sum of a group's (n sd^2 < 2^125), which any fp32 evaluation has to hold."""
    from sphere_rasterization_amd import appearance as A
    rng = np.random.default_rng(22)
    x = _put(1e20 + sd * rng.standard_normal((images,) + shape + (c,)), dt, dev)
    dy = _put(rng.standard_normal(x.shape), dt, dev)
    y, mean, rstd = A.group_norm_forward(x, groups)
    f = O.group_norm_backward(_np(dy), _np(x), groups)
    # a mean off by DEPTH U of itself, in units of the deviation
    rel = DEPTH * U * 1.1e20 * f["rstd"].max()
    _check(mean, f["mean"], DEPTH * U * np.abs(f["mean"]) * 1.1, "mean")
    _check(rstd, f["rstd"], (2 * DEPTH * U + 2 * rel * rel) * f["rstd"], "rstd")
    _check(y, f["y"], (rel + 2 * rel * rel + DEPTH * U) * (1 + np.abs(f["y"])) + 1.01 * RO[dt] * np.abs(f["y"]), "y")
    dx, dw, db = A.group_norm_backward(dy, x, mean, rstd)
    assert all(torch.isfinite(t).all() for t in (dx, dw, db))


def test_group_norm_constant_nonfinite_and_params(dev):
    from sphere_rasterization_amd import appearance as A
    x = torch.full((2, 5, 4), 7.0, device=dev)
    b = torch.tensor([1.0, 2.0, 3.0, 4.0], device=dev)
    y, mean, rstd = A.group_norm_forward(x, 2, None, b)
    assert torch.equal(y, b.expand(2, 5, 4)) and (mean == 7).all()
    dx, dw, db = A.group_norm_backward(torch.ones_like(x), x, mean, rstd, None, b)
    assert (dx == 0).all() and (dw == 0).all() and (db == 10).all()
    # a NaN spoils its own image and group only
    x = torch.randn(2, 50, 8, device=dev)
    clean = A.group_norm(x, 4, act="silu")
    x[1, 3, 2] = float("nan")
    y = A.group_norm(x, 4, act="silu")
    assert torch.isnan(y[1, :, 2:4]).all() and torch.equal(y[0], clean[0])
    assert torch.equal(y[1, :, :2], clean[1, :, :2]) and torch.equal(y[1, :, 4:], clean[1, :, 4:])
    # float32 parameters with bf16 images; only some gradients wanted
    xb = torch.randn(1, 30, 16, device=dev).to(torch.bfloat16)
    w = torch.randn(16, device=dev)
    y, mean, rstd = A.group_norm_forward(xb, 4, w)
    dx, dw, db = A.group_norm_backward(torch.randn_like(xb), xb, mean, rstd, w, want=("weight",))
    assert dx is None and db is None and dw.dtype == torch.float32
    # nothing to normalise
    e = torch.empty(0, 4, 8, device=dev)
    y, mean, rstd = A.group_norm_forward(e, 2)
    dx, dw, db = A.group_norm_backward(e, e, mean, rstd)
    assert y.shape == e.shape and (dw == 0).all() and (db == 0).all() and dw.shape == (8,)


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("shape", [(2, 0, 8), (0, 0, 8), (3, 4, 0, 8), (0, 5, 8), (600, 0, 8)])
def test_group_norm_of_no_values(dev, shape, dt):
    """No pixels or no images: statistics of nothing are 0 and 1 / sqrt(eps), gradients zero."""
    from sphere_rasterization_amd import appearance as A
    eps, n = 1e-3, shape[0]
    x = torch.empty(shape, dtype=DT[dt], device=dev)
    w = torch.randn(8, device=dev, requires_grad=True)
    b = torch.randn(8, device=dev, requires_grad=True)
    for _ in range(2):                                        # the second time on used memory
        held = torch.full((2, n, 2), 7.0, device=dev)
        del held
        y, mean, rstd = A.group_norm_forward(x, 2, w.detach(), b.detach(), eps, "silu")
        assert y.shape == x.shape and y.dtype == x.dtype and mean.shape == rstd.shape == (n, 2)
        assert (mean == 0).all()
        ref = np.float32(eps) ** np.float64(-0.5)
        assert ((rstd.double() - ref).abs() <= 4 * U * ref).all()
    dx, dw, db = A.group_norm_backward(x, x, mean, rstd, w.detach(), b.detach(), "silu")
    assert dx.shape == x.shape and (dw == 0).all() and (db == 0).all() and dw.shape == db.shape == (8,)
    with torch.no_grad():
        assert A.group_norm(x, 2, w, b, act="gelu").shape == x.shape
    A.group_norm(x.requires_grad_(), 2, w, b, act="gelu").sum().backward()
    assert x.grad.shape == x.shape and (w.grad == 0).all() and (b.grad == 0).all()


def test_group_norm_strides(dev):
    """Images inside wider ones, channels_last tensors, transposed pixels, odd alignment,
    repeated gradients: the same bits as on packed copies."""
    from sphere_rasterization_amd import appearance as A
    torch.manual_seed(5)
    wide = torch.randn(2, 9, 7, 30, device=dev)
    nchw = torch.randn(2, 16, 9, 7, device=dev).contiguous(memory_format=torch.channels_last)
    odd = torch.randn(2 * 9 * 7 * 16 + 1, device=dev)[1:].view(2, 9, 7, 16)
    for x in (wide[..., 3:19], nchw.permute(0, 2, 3, 1), wide[:, :, 2:5, 4:20], wide[..., :16].transpose(1, 2), odd,
              torch.randn(2, 9, 16, 7, device=dev).transpose(2, 3), wide[:, ::2, :, 5:21]):
        dense = x.clone(memory_format=torch.contiguous_format)
        g = torch.ones(1, device=dev).expand(x.shape)
        a, b = A.group_norm_forward(x, 4, act="silu"), A.group_norm_forward(dense, 4, act="silu")
        for p, q in zip(a, b):
            assert (p - q).abs().max() <= 1e-5            # other vector widths sum in another order
        da = A.group_norm_backward(g, x, *a[1:], act="silu")
        db = A.group_norm_backward(torch.ones_like(dense), dense, *b[1:], act="silu")
        for p, q in zip(da, db):
            assert (p - q).abs().max() <= 1e-4 * max(1.0, float(q.abs().max()))


def _act_and_slope(dev, z, kind, groups):
    """The fp32 kernels' activation and slope at exactly z: a weight of zero leaves the bias."""
    from sphere_rasterization_amd import appearance as A
    b = torch.from_numpy(z).to(dev)
    x, w = torch.randn(1, 1, len(z), device=dev), torch.zeros(len(z), device=dev)
    y, mean, rstd = A.group_norm_forward(x, groups, w, b, 1e-5, kind)
    db = A.group_norm_backward(torch.ones_like(x), x, mean, rstd, w, b, kind)[2]      # one pixel: db is the slope
    return _np(y).reshape(-1), _np(db)


@pytest.mark.parametrize("groups", [1, 32])                   # three launches; one
def test_gelu_in_fp32_holds_its_tail(dev, groups):
    """Roundings counted, in units of U. The exponential: 3 of its argument, each of which
    moves it by z^2 / 2 of its value, and 2 of its own. The tail beyond 1.25: reciprocal 4,
    polynomial 3, products 2, fit 0.4, and the exponential's. Within: 4 of F - 1/2 and the
    half's sum. Then the activation's product, or the slope's."""
    z = np.concatenate([np.linspace(-9, 9, 65536 - 512), -np.geomspace(1e-8, 12, 256),
                        np.geomspace(1e-8, 30, 256)]).astype(np.float32)
    y, slope = _act_and_slope(dev, z, "gelu", groups)
    import scipy.special as sp
    zd = z.astype(np.float64)
    a, tail = np.abs(zd), 0.5 * sp.erfc(np.abs(zd) / np.sqrt(2.0))
    whole, density = np.where(zd < 0, tail, 1.0 - tail), np.exp(-0.5 * zd * zd) / np.sqrt(2.0 * np.pi)
    e_exp = 2 + 1.5 * zd * zd
    e_far = (10 + e_exp) * tail + np.where(zd < 0, 0.0, 1.0)
    e_int = U * np.where(a < 1.25, 1 + 4 * (0.5 - tail), e_far) * 1.01
    tiny = 2.0 ** -126 * (1 + a)                              # below fp32's normal range nothing is promised
    assert (np.abs(y - zd * whole) <= a * e_int + U * a * whole + tiny).all()
    e_slope = e_int + U * (a * density * (3 + e_exp) + np.abs(whole + zd * density))
    assert (np.abs(slope - (whole + zd * density)) <= e_slope * 1.01 + tiny).all()


@pytest.mark.parametrize("groups", [1, 32])
@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_gelu_in_16_bits_is_rounded_once(dev, dt, groups):
    """Every value of the type from -12 to 12: half a step of the result, and the part before
    the rounding, for which a tenth of a step is allowed."""
    from sphere_rasterization_amd import appearance as A
    import scipy.special as sp
    bits = torch.arange(65536, dtype=torch.int32).to(torch.int16)
    v = bits.view(DT[dt]).float()
    v = v[torch.isfinite(v) & (v.abs() <= 12)]
    v = torch.cat([v, torch.zeros(-len(v) % 32)])
    b = v.to(DT[dt]).to(dev)
    x, w = torch.randn(1, 1, len(v), device=dev).to(DT[dt]), torch.zeros(len(v), device=dev, dtype=DT[dt])
    y = _np(A.group_norm(x, groups, w, b, act="gelu")).reshape(-1)
    z = v.double().numpy()
    ref = z * 0.5 * sp.erfc(-z / np.sqrt(2.0))
    least = {"f16": 2.0 ** -24, "bf16": 2.0 ** -133}[dt]
    step = np.maximum(2.0 ** (np.floor(np.log2(np.maximum(np.abs(ref), 1e-300)))) * 2 * RO[dt], least)
    assert (np.abs(y - ref) <= 0.6 * step + 2.0 ** -126).all()


@pytest.mark.parametrize("groups", [1, 32])
def test_silu_in_fp32_holds_its_tail(dev, groups):
    """At most 8 roundings of the result at any z: exponential 2, its argument's remainder 1,
    sum 1, reciprocal 2, products 2."""
    z = np.concatenate([np.linspace(-85, 85, 65536 - 512), -np.geomspace(1e-8, 9, 256),
                        np.geomspace(1e-8, 9, 256)]).astype(np.float32)
    y, slope = _act_and_slope(dev, z, "silu", groups)
    zd = z.astype(np.float64)
    s, q = 1.0 / (1.0 + np.exp(-zd)), 1.0 / (1.0 + np.exp(zd))
    assert (np.abs(y - zd * s) <= 8 * U * 1.01 * np.abs(zd * s)).all()
    assert (np.abs(slope - s * (1 + zd * q)) <= 8 * U * 1.01 * s * (1 + np.abs(zd) * q)).all()
    ends = np.array([np.inf, 1e30, 200.0, -200.0, -1e30, 0.0, -0.0, 3.0] * 8, np.float32)
    y, slope = _act_and_slope(dev, ends, "silu", 1)
    assert np.array_equal(y[:7], [np.inf, np.float32(1e30), 200.0, 0.0, 0.0, 0.0, 0.0])
    assert np.array_equal(slope[1:7], [1.0, 1.0, 0.0, 0.0, 0.5, 0.5])


# ---- orthogonalize ----------------------------------------------------------------------

def _ortho_tol(ref, dt, steps=5, a=3.4445):
    """Frobenius: each factor is held to 2^-22 and each step's three products and sums add
    at most four such errors of the factor; a step lets an error grow at most a-fold, so
    each of them (relative to X0's norm of one) ends below a^steps. Then one rounding."""
    return 4 * (steps + 1) * 2.0 ** -21 * a ** steps + 1.01 * RO[dt] * np.linalg.norm(ref)


ORTHOS = [(1, 1), (1, 7), (5, 1), (8, 8), (16, 40), (64, 32), (31, 33), (65, 130), (128, 128), (129, 127), (100, 300),
          (257, 70), (96, 96), (200, 513), (40, 2100), (384, 260)]


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows,cols", ORTHOS)
def test_orthogonalize(dev, rows, cols, dt):
    from sphere_rasterization_amd import appearance as A
    rng = np.random.default_rng(rows * 7 + cols)
    g = _put(rng.standard_normal((rows, cols)), dt, dev)
    got = A.orthogonalize(g)
    ref = O.orthogonalize(_np(g))
    assert np.linalg.norm(_np(got) - ref) <= _ortho_tol(ref, dt)
    assert torch.equal(got, A.orthogonalize(g)), "not the same bits twice"


def test_orthogonalize_batches_strides_and_scale(dev):
    from sphere_rasterization_amd import appearance as A
    rng = np.random.default_rng(31)
    for shape in ((5, 24, 40), (3, 130, 50), (2, 3, 60, 20)):
        g = _put(rng.standard_normal(shape) * np.exp(rng.uniform(-20, 20, shape[:-2] + (1, 1))), "f32", dev)
        got = A.orthogonalize(g, scale=0.2)
        ref = O.orthogonalize(_np(g), scale=0.2)
        for p, q in zip(_np(got).reshape((-1,) + shape[-2:]), ref.reshape((-1,) + shape[-2:])):
            assert np.linalg.norm(p - q) <= _ortho_tol(q, "f32")
    wide = _put(rng.standard_normal((4, 50, 90)), "f32", dev)
    for v in (wide[1:, 3:40, 5:80], wide.transpose(1, 2), wide[::2], wide[0, :, ::3], wide[:1].expand(3, 50, 90)):
        assert torch.equal(A.orthogonalize(v), A.orthogonalize(v.clone(memory_format=torch.contiguous_format)))
    g = _put(rng.standard_normal((70, 90)), "f32", dev)
    for steps, coeffs in ((1, COEFFS), (8, (1.5, -0.5, 0.0)), (3, (2.0, -1.5, 0.5)), (2, (0.0, 0.0, 0.0))):
        ref = O.orthogonalize(_np(g), steps, coeffs)
        assert np.linalg.norm(_np(A.orthogonalize(g, steps, coeffs)) - ref) <= _ortho_tol(ref, "f32", steps, max(1.0, coeffs[0]))


@pytest.mark.parametrize("shape", [(130, 2500), (300, 4100), (3, 70, 2049), (513, 16400), (130, 200, 250), (2300, 60),
                                   (3, 33, 1025), (96, 8192), (8192, 65), (9, 8193), (1, 4000), (97, 1500), (40, 64, 500),
                                   (90, 1537), (90, 1536)])
def test_orthogonalize_tiles(dev, shape):
    """Long summed axes (a product's steps shared out over all workgroups) and many tiles."""
    from sphere_rasterization_amd import appearance as A
    g = _put(np.random.default_rng(33).standard_normal(shape), "f32", dev)
    got, ref = A.orthogonalize(g), O.orthogonalize(_np(g))
    for p, q in zip(_np(got).reshape((-1,) + shape[-2:]), ref.reshape((-1,) + shape[-2:])):
        assert np.linalg.norm(p - q) <= _ortho_tol(q, "f32")
    assert torch.equal(got, A.orthogonalize(g)), "not the same bits twice"


def test_orthogonalize_zero_tiny_huge_and_low_rank(dev):
    from sphere_rasterization_amd import appearance as A
    assert (A.orthogonalize(torch.zeros(2, 40, 30, device=dev)) == 0).all()
    rng = np.random.default_rng(32)
    g = rng.standard_normal((40, 60))
    for s in (1e-30, 1e30):                                   # squares outside fp32's range
        t = _put(g * s, "f32", dev)
        ref = O.orthogonalize(_np(t), eps=float(np.float32(1e-7)))
        assert np.linalg.norm(_np(A.orthogonalize(t)) - ref) <= _ortho_tol(ref, "f32")
    low = _put(np.outer(rng.standard_normal(150), rng.standard_normal(90)), "f32", dev)
    ref = O.orthogonalize(_np(low))
    assert np.linalg.norm(_np(A.orthogonalize(low)) - ref) <= _ortho_tol(ref, "f32")
    bad = _put(g, "f32", dev)
    bad[3, 5] = float("nan")
    assert torch.isnan(A.orthogonalize(bad)).any()
    pair = torch.stack([bad, _put(g, "f32", dev)])            # a NaN stays in its own matrix
    assert torch.equal(A.orthogonalize(pair)[1], A.orthogonalize(pair[1]))
    assert A.orthogonalize(torch.empty(0, 3, 4, device=dev)).shape == (0, 3, 4)
    assert A.orthogonalize(torch.empty(2, 0, 4, device=dev)).shape == (2, 0, 4)


@pytest.mark.parametrize("shape", [(40, 60), (70, 400), (150, 260), (2, 33, 45)])
def test_orthogonalize_without_eps(dev, shape):
    """eps = 0, matrices of any size of value (one workgroup, narrow, tiles): the result does
    not depend on it, down to where fp32 itself runs out."""
    from sphere_rasterization_amd import appearance as A
    g = np.random.default_rng(34).standard_normal(shape)
    for s in (1e-43, 1e-39, 1e-36, 1e-33, 1e-20, 1.0, 1e20, 6e37):
        t = _put(g * s, "f32", dev)
        ref = O.orthogonalize(_np(t), eps=0.0)
        got = A.orthogonalize(t, eps=0.0)
        for p, q in zip(_np(got).reshape((-1,) + shape[-2:]), ref.reshape((-1,) + shape[-2:])):
            assert np.linalg.norm(p - q) <= _ortho_tol(q, "f32"), s
    whole = A.orthogonalize(_put(g, "f32", dev), eps=0.0)     # powers of two: the same bits
    for k in (-100, -60, 60, 100):
        assert torch.equal(A.orthogonalize(torch.ldexp(_put(g, "f32", dev), torch.tensor(k, device=dev)), eps=0.0), whole), k


@pytest.mark.parametrize("shape", [
    (1, 7), (8, 8), (64, 32), (65, 32), (96, 96), (3, 64, 128),                        # one workgroup, both LDS sizes
    (128, 96), (257, 70), (40, 700), (64, 1024), (64, 2500), (90, 1500), (1025, 9),               # narrow, 64 and 128 columns a slice
    (200, 250), (300, 400), (700, 129), (2, 130, 300),                                 # 64 x 64 tiles
    (130, 2500), (97, 4096),                                                           # and shared out
    (130, 200, 250), (520, 97, 120), (6, 1024, 1300), (513, 16400)])                   # 128 x 128 tiles, and shared out
def test_orthogonalize_holds_both_parts(dev, shape):
    """The error of every form is that of two-part factors, far below one with a part lost."""
    from tests import ortho_parts as H
    from sphere_rasterization_amd import appearance as A
    g = _put(np.random.default_rng(shape[-2] * 7 + shape[-1]).standard_normal(shape), "f32", dev)
    flat = (-1,) + shape[-2:]
    got, src = _np(A.orthogonalize(g)).reshape(flat), _np(g).reshape(flat)
    some = range(len(src)) if len(src) < 8 else (0, 1, len(src) // 2, len(src) - 1)
    for k in some:
        assert H.error(got[k], O.orthogonalize(src[k])) <= H.BOUND, k


def test_interleaved_outputs_of_the_c_calls(dev):
    """Matrices interleaved by rows and images interleaved by pixels do not overlap."""
    from sphere_rasterization_amd import _lib as L
    from sphere_rasterization_amd import appearance as A
    s = torch.cuda.current_stream().cuda_stream
    g, out = torch.randn(2, 40, 60, device=dev), torch.zeros(40, 2, 60, device=dev)
    L.splat_orthogonalize(g.data_ptr(), L.SPLAT_F32, 2, 40, 60, 2400, 60, 5, *COEFFS, 1e-7, 1.0, out.data_ptr(), 60, 120,
                          None, 0, s)
    assert torch.equal(out.transpose(0, 1), A.orthogonalize(g))
    x, y, st = torch.randn(3, 50, 8, device=dev), torch.zeros(50, 3, 8, device=dev), torch.zeros(2, 3, 2, device=dev)
    d = L.splat_norm()
    d.channels, d.groups, d.eps, d.images, d.pixels = 8, 2, 1e-5, 3, 50
    d.x_image_stride, d.x_pixel_stride, d.y_image_stride, d.y_pixel_stride = 400, 8, 8, 24
    L.splat_group_norm(d, x.data_ptr(), None, None, y.data_ptr(), st.data_ptr(), st[1].data_ptr(), None, 0, s)
    assert torch.equal(y.transpose(0, 1), A.group_norm(x, 2))


# ---- together ------------------------------------------------------------------------------

def test_autograd(dev):
    from sphere_rasterization_amd import appearance as A
    torch.manual_seed(7)
    table = torch.randn(30, 16, device=dev, requires_grad=True)
    ids = torch.randint(-1, 30, (2, 9, 5), device=dev)
    w = torch.randn(16, device=dev, requires_grad=True)
    b = torch.randn(16, device=dev, requires_grad=True)
    y = A.group_norm(A.lookup(table, ids, 3.0), 4, w, b, act="gelu")
    up = torch.randn_like(y)
    y.backward(up)
    feat = O.lookup(_np(table), ids.cpu().numpy(), 3.0)
    f = O.group_norm_backward(_np(up), feat, 4, _np(w), _np(b), 1e-5, "gelu")
    d = O.lookup_backward(f["dx"], ids.cpu().numpy(), 30, 3.0)
    # 90 values per sum, each an fp32 chain of a few dozen roundings
    for got, ref in ((y, f["y"]), (w.grad, f["dw"]), (b.grad, f["db"]), (table.grad, d)):
        assert np.abs(_np(got) - ref).max() <= 256 * 16 * U * max(1.0, np.abs(ref).max())
    with torch.no_grad():
        assert not A.lookup(table, ids).requires_grad
    # frozen inputs get no gradient
    z = A.group_norm(torch.randn(1, 4, 16, device=dev), 4, w)
    w.grad = None
    z.sum().backward()
    assert w.grad is not None


def test_other_stream_and_graph(dev):
    """On a side stream, and replayed from a graph with other work and synchronisation in
    between: the same bits as eager calls on the current stream."""
    from sphere_rasterization_amd import appearance as A
    torch.manual_seed(8)
    n, rows, c = 20000, 600, 16
    table, dy = torch.randn(rows, c, device=dev), torch.randn(n, c, device=dev)
    ids = torch.randint(0, rows, (n,), device=dev)
    x, g = torch.randn(2, 700, c, device=dev), torch.randn(140, 90, device=dev)

    def work():
        f = A.lookup(table, ids)
        d = A.lookup_backward(dy, ids, rows)
        y, m, r = A.group_norm_forward(x, 4, act="silu")
        return (f, d, y) + A.group_norm_backward(x, x, m, r, act="silu") + (A.orthogonalize(g),)

    ref = [t.clone() for t in work()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = work()
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(p, q) for p, q in zip(ref, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = work()
    for k in range(4):
        for t in (table, dy, x, g):
            t.mul_(-1.25 if k % 2 else 0.8)
        ids.copy_(torch.randint(0, rows, (n,), device=dev))
        graph.replay()
        torch.cuda.synchronize()
        want = work()
        assert all(torch.equal(p, q) for p, q in zip(want, out)), f"replay {k}"
        torch.cuda.synchronize()


def test_refusals(dev):
    from sphere_rasterization_amd import _lib as L
    from sphere_rasterization_amd import appearance as A
    t, ids = torch.zeros(4, 8, device=dev), torch.zeros(3, dtype=torch.int64, device=dev)
    for call in (lambda: A.lookup(t, ids.float()), lambda: A.lookup(t, ids.cpu()), lambda: A.lookup(t.double(), ids),
                 lambda: A.lookup_backward(t, ids, 4), lambda: A.lookup_backward(t[:3], ids, 4, accumulate=True),
                 lambda: A.lookup_backward(t[:3], ids, 4, out=torch.zeros(4, 7, device=dev)),
                 lambda: A.lookup_backward(t[:3], ids, 4, out=torch.zeros(8, 4, device=dev).t()),
                 lambda: A.group_norm(t, 2, weight=torch.ones(7, device=dev)),
                 lambda: A.group_norm(t, 2, weight=torch.ones(8)),
                 lambda: A.group_norm(t, 2, torch.ones(8, device=dev), torch.ones(8, device=dev).half()),
                 lambda: A.group_norm_backward(t[:2], t, torch.zeros(4, 2, device=dev), torch.zeros(4, 2, device=dev)),
                 lambda: A.group_norm_backward(t, t, torch.zeros(4, 2, device=dev), torch.zeros(4, 1, device=dev)),
                 lambda: A.orthogonalize(t, coeffs=(1.0, 2.0))):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: A.group_norm(t, 3), lambda: A.group_norm(t, 2, eps=-1.0), lambda: A.lookup(t, ids, float("inf")),
                 lambda: A.orthogonalize(t, steps=0), lambda: A.orthogonalize(t, coeffs=(30.0, 0.0, 0.0)),
                 lambda: A.orthogonalize(torch.zeros(70000, 2, device=dev))):
        with pytest.raises(L.SplatError):
            call()


def test_training_example(dev):
    """The example's loop: table, renderer, shading and orthogonalised updates together."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "train_appearance.py")
    spec = importlib.util.spec_from_file_location("train_appearance", path)
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    losses = ex.train(steps=25, n=5000, width=160, height=96)
    assert all(np.isfinite(losses)) and losses[-1] < 0.5 * losses[0]
