"""Host checks of the dense layers and of dropout (no GPU): size queries, refusals before any
launch, sizes of zero."""
import ctypes as C

import pytest
import torch

from sphere_rasterization_amd import _lib as L

P = C.c_void_p(256)          # an aligned address that no refused call may touch


def _drop(p=0.0, seed=1, offset=2, state=None):
    return L.splat_drop(p, seed, offset, state)


def _dense(**kw):
    d = L.splat_dense()
    d.dtype, d.bias_dtype, d.act, d.inputs, d.outputs, d.rows = 0, 0, 2, 24, 40, 100
    d.x_stride = d.dx_stride = 24
    d.residual_stride = d.y_stride = 40
    d.w_in_stride = d.dw_in_stride = 40
    d.w_out_stride = d.dw_out_stride = 1
    drop = {k: kw.pop(k) for k in ("p", "seed", "offset", "state") if k in kw}
    d.drop = _drop(**drop)
    for k, v in kw.items():
        setattr(d, k, v)
    return d


def _fwd(d, x=P, w=P, bias=P, res=P, y=P, pre=P, ws=P, nbytes=1 << 40):
    return L.lib().splat_linear(C.byref(d), x, w, bias, res, y, pre, ws, nbytes, None)


def _bwd(d, dy=P, x=P, w=P, bias=P, pre=P, dx=P, dw=P, db=P, ws=P, nbytes=1 << 40):
    return L.lib().splat_linear_bwd(C.byref(d), dy, x, w, bias, pre, dx, dw, db, ws, nbytes, None)


@pytest.mark.parametrize("change", [
    dict(dtype=3), dict(dtype=1, bias_dtype=2), dict(act=4), dict(act=-1), dict(rows=-1), dict(rows=1 << 31), dict(inputs=-1),
    dict(outputs=(1 << 20) + 1), dict(inputs=(1 << 20) + 1), dict(w_in_stride=39), dict(w_out_stride=2), dict(w_in_stride=1),
    dict(w_in_stride=-40), dict(w_in_stride=0), dict(p=-0.1), dict(p=1.5), dict(p=float("nan")),
    dict(p=0.5, state=260), dict(x_stride=23), dict(x_stride=-24), dict(y_stride=39), dict(x_stride=1 << 61)])
def test_linear_descriptor_refusals(change):
    d = _dense(**change)
    assert _fwd(d) == L.SPLAT_ERR_INVALID_ARG
    assert _bwd(d) == L.SPLAT_ERR_INVALID_ARG
    strides = ("x_stride", "y_stride")
    if not any(k in strides for k in change):
        assert L.splat_linear_workspace_bytes(d, False) == 0 and L.splat_linear_workspace_bytes(d, True) == 0


def test_linear_refusals_of_one_direction():
    assert _fwd(_dense(residual_stride=39)) == L.SPLAT_ERR_INVALID_ARG
    for change in (dict(dx_stride=23), dict(dw_in_stride=39), dict(dw_out_stride=2), dict(dw_in_stride=0)):
        assert _bwd(_dense(**change)) == L.SPLAT_ERR_INVALID_ARG


def test_linear_pointer_refusals():
    d = _dense()
    for k in ("x", "w", "y"):
        assert _fwd(d, **{k: None}) == L.SPLAT_ERR_INVALID_ARG
    for k in ("dy", "x", "w"):
        assert _bwd(d, **{k: None}) == L.SPLAT_ERR_INVALID_ARG
    for k in ("x", "w", "bias", "res", "y", "pre"):
        assert _fwd(d, **{k: C.c_void_p(258)}) == L.SPLAT_ERR_INVALID_ARG
    for k in ("dy", "x", "w", "bias", "pre", "dx", "dw", "db"):
        assert _bwd(d, **{k: C.c_void_p(258)}) == L.SPLAT_ERR_INVALID_ARG
    need = L.splat_linear_workspace_bytes(_dense(rows=100_000, outputs=300, y_stride=300, w_in_stride=300,
                                                 dw_in_stride=300), True)
    assert need > 0
    big = _dense(rows=100_000, outputs=300, y_stride=300, w_in_stride=300, dw_in_stride=300)
    assert _bwd(big, ws=None) == L.SPLAT_ERR_INVALID_ARG
    assert _bwd(big, ws=C.c_void_p(264)) == L.SPLAT_ERR_INVALID_ARG
    assert _bwd(big, nbytes=need - 1) == L.SPLAT_ERR_CAPACITY
    # nothing asked for: nothing done
    assert _bwd(d, dx=None, dw=None, db=None) == L.SPLAT_OK


def test_sizes_of_zero_touch_nothing():
    none = {k: None for k in ("x", "w", "bias", "res", "y", "pre", "ws")}
    assert _fwd(_dense(rows=0), **none) == L.SPLAT_OK
    assert _fwd(_dense(outputs=0, w_in_stride=1), **none) == L.SPLAT_OK
    assert L.lib().splat_dropout(C.byref(_drop(0.5)), 0, 0, 8, None, 8, None, 8, None, 8, None) == L.SPLAT_OK
    assert L.lib().splat_dropout(C.byref(_drop(0.5)), 0, 8, 0, None, 0, None, 0, None, 0, None) == L.SPLAT_OK


def test_saves_and_workspace_queries():
    for dtype in (L.SPLAT_F32, L.SPLAT_F16, L.SPLAT_BF16):
        for rows in (0, 1, 5, 1000, 2_000_000):
            for k, n in ((1, 1), (32, 64), (65, 130), (1024, 4096), (0, 8), (8, 0)):
                for by_out in (True, False):
                    s = dict(w_in_stride=n, w_out_stride=1) if by_out else dict(w_in_stride=1, w_out_stride=k)
                    s.update({"d" + a: b for a, b in s.items()})
                    if k <= 1 or n <= 1:
                        s = dict.fromkeys(s, 1)
                    d = _dense(dtype=dtype, bias_dtype=dtype, rows=rows, inputs=k, outputs=n, p=0.5, **s)
                    assert L.splat_linear_saves(d) in (False, True)
                    fwd, bwd = L.splat_linear_workspace_bytes(d, False), L.splat_linear_workspace_bytes(d, True)
                    assert fwd <= 1 << 32 and bwd <= 1 << 36
                    if rows == 0 or n == 0:
                        assert fwd == 0 and bwd == 0
                    d.act = 0
                    assert not L.splat_linear_saves(d)


@pytest.mark.parametrize("change", [
    dict(dtype=3), dict(rows=-1), dict(cols=-1), dict(rows=1 << 40, cols=1 << 30), dict(x=None), dict(y=None), dict(xs=7),
    dict(rs=7), dict(ys=7), dict(xs=-8), dict(x=C.c_void_p(258)), dict(y=C.c_void_p(258)), dict(res=C.c_void_p(257)),
    dict(drop=_drop(-1.0)), dict(drop=_drop(1.01)), dict(drop=_drop(float("nan"))), dict(drop=_drop(0.5, state=100))])
def test_dropout_refusals(change):
    a = dict(drop=_drop(0.5), dtype=0, rows=100, cols=8, x=P, xs=8, res=P, rs=8, y=P, ys=8)
    a.update(change)
    a["drop"] = C.byref(a["drop"])
    assert L.lib().splat_dropout(*a.values(), None) == L.SPLAT_ERR_INVALID_ARG


def test_python_refusals_without_a_gpu():
    from sphere_rasterization_amd import appearance as A
    x, w = torch.zeros(4, 8), torch.zeros(8, 3)
    for call, match in ((lambda: A.linear(x, w), "GPU tensor"), (lambda: A.linear(x.double(), w.double()), "float32"),
                        (lambda: A.linear(x, w.t()), "weight"), (lambda: A.linear(x, w[0]), "weight"),
                        (lambda: A.linear(x, w, act="tanh"), "act"), (lambda: A.linear_backward(x, x, w.t()), "weight"),
                        (lambda: A.dropout(x, 0.5, (1, 2)), "GPU tensor"), (lambda: A.dropout(x.long(), 0.5, (1, 2)), "float32")):
        with pytest.raises(ValueError, match=match):
            call()


class _OnGpu:
    """A tensor's face alone."""

    def __init__(self, *shape):
        self.shape, self.dtype, self.is_cuda, self.device = torch.Size(shape), torch.float16, True, torch.device("cuda:0")
        self.requires_grad = False

    def dim(self):
        return len(self.shape)


def test_refused_numbers():
    from sphere_rasterization_amd import appearance as A
    x = _OnGpu(4, 8)
    for p, rng, match in ((0.5, None, "rng"), (1.5, (1, 2), "p:"), (-0.5, (1, 2), "p:"), (float("nan"), (1, 2), "p:"),
                          (0.5, 7, "rng"), (0.5, (1, 2, 3), "rng"), (0.5, (-1, 2), "seed"), (0.5, (1 << 64, 2), "seed"),
                          (0.5, (1, -2), "offset"), (0.5, (1, 1 << 64), "offset"), (0.5, (1.5, 2), "seed"),
                          (0.5, (torch.zeros(2, dtype=torch.int64), 0), "state")):
        with pytest.raises(ValueError, match=match):
            A.dropout(x, p, rng)
    with pytest.raises(ValueError, match="2\\^31"):
        A.linear(_OnGpu(4, (1 << 32) + 8), _OnGpu((1 << 32) + 8, 3))


def test_forward_mode_is_refused():
    import torch.autograd.forward_ad as fwd
    from sphere_rasterization_amd import appearance as A
    x, w, b, y = torch.zeros(4, 8), torch.zeros(8, 3), torch.zeros(3), torch.zeros(4, 3)
    with fwd.dual_level():
        dual = lambda t: fwd.make_dual(t, torch.ones_like(t))
        for call in (lambda: A.linear(dual(x), w), lambda: A.linear(x, dual(w)), lambda: A.linear(x, w, dual(b)),
                     lambda: A.linear(x, w, residual=dual(y)), lambda: A.linear_forward(dual(x), w),
                     lambda: A.linear_backward(dual(y), x, w), lambda: A.linear_backward(y, dual(x), w),
                     lambda: A.dropout(dual(x), 0.5, (1, 2)), lambda: A.dropout(x, 0.5, (1, 2), dual(x)),
                     lambda: A.dropout_backward(dual(x), 0.5, (1, 2))):
            with pytest.raises(NotImplementedError, match="forward-mode"):
                call()


def test_the_large_layers_reach_every_tile():
    """The layers that the GPU tests hold value by value are cut in every way that there is."""
    from tests.dense_layers import LARGE, cut
    products = dict(y=lambda m, k, n: [(m, n, k)], d_x=lambda m, k, n: [(m, k, n)], d_W=lambda m, k, n: [(k, n, m), (n, k, m)])
    for f32, parts, tiles in ((False, 1, {0, 1, 2}), (False, 2, {0, 1, 2}), (True, 1, {1, 2})):
        got = {name: {cut(*size, parts, f32) for c in LARGE for size in sizes(*c)} for name, sizes in products.items()
               if name != "y" or parts == 1}
        for name, cuts in got.items():
            assert {t for t, _ in cuts} == tiles, (name, f32, parts)
        whole, split = ({t for cuts in got.values() for t, s in cuts if (s > 1) == k} for k in (False, True))
        assert whole == tiles and split == tiles, (f32, parts)
