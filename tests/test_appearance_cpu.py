"""Host checks of the appearance operators (no GPU): size queries, refusals before any
launch, sizes of zero."""
import ctypes as C
import os
import re

import pytest
import torch

from sphere_rasterization_amd import _lib as L

P = C.c_void_p(256)          # an aligned address that no refused call may touch
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _norm(**kw):
    d = L.splat_norm()
    d.dtype, d.param_dtype, d.act, d.channels, d.groups, d.eps = 0, 0, 0, 8, 2, 1e-5
    d.images, d.pixels = 2, 16
    for k in ("x", "y", "dx"):
        setattr(d, k + "_image_stride", 128)
        setattr(d, k + "_pixel_stride", 8)
    for k, v in kw.items():
        setattr(d, k, v)
    return d


def test_enums_match_the_header():
    src = open(os.path.join(ROOT, "include", "splat.h")).read()
    for name in ("SPLAT_F32", "SPLAT_F16", "SPLAT_BF16", "SPLAT_I32", "SPLAT_I64", "SPLAT_ACT_NONE", "SPLAT_ACT_RELU",
                 "SPLAT_ACT_SILU", "SPLAT_ACT_GELU"):
        assert int(re.search(name + r" = (\d+)", src).group(1)) == getattr(L, name)


def test_size_queries():
    n, rows, dim = 100_000, 5000, 32
    need = L.splat_lookup_bwd_workspace_bytes(n, rows, dim)
    assert need >= 16 * n + 8 * rows + 4 * dim * (n // 64)
    assert L.splat_lookup_bwd_workspace_bytes(-1, rows, dim) == 0
    assert L.splat_lookup_bwd_workspace_bytes(1000, rows, dim) == 0       # one launch, no workspace
    assert L.splat_group_norm_workspace_bytes(_norm(pixels=1 << 20), False) >= 2 * 2 * 8
    assert L.splat_group_norm_workspace_bytes(_norm(pixels=1 << 20), True) >= 2 * 8 * 8
    assert L.splat_group_norm_workspace_bytes(_norm(groups=3, pixels=1 << 20), False) == 0
    assert L.splat_orthogonalize_workspace_bytes(2, 200, 300) >= 2 * 200 * 300 * 4 * 2
    assert L.splat_orthogonalize_workspace_bytes(1, 100_000, 3) == 0
    assert L.splat_orthogonalize_workspace_bytes(100, 64, 96) == 0        # held in LDS


@pytest.mark.parametrize("change", [
    dict(dtype=7), dict(itype=2), dict(rows=-1), dict(n=-1), dict(n=1 << 31), dict(dim=70000), dict(scale=float("nan")),
    dict(table=None), dict(ids=None), dict(out=None), dict(ldt=7), dict(ldo=7), dict(ldt=-8), dict(ldt=1 << 61),
    dict(table=C.c_void_p(258)), dict(ids=C.c_void_p(260))])
def test_lookup_refusals(change):
    a = dict(table=P, dtype=0, rows=100, dim=8, ldt=8, ids=P, itype=1, n=10, scale=1.0, out=P, ldo=8)
    a.update(change)
    assert L.lib().splat_lookup(*a.values(), None) == L.SPLAT_ERR_INVALID_ARG


@pytest.mark.parametrize("change,code", [
    (dict(dtype=3), -1), (dict(itype=-1), -1), (dict(n=1 << 31), -1), (dict(rows=(1 << 31) - 1), -1),
    (dict(scale=float("inf")), -1), (dict(accumulate=2), -1), (dict(d_out=None), -1), (dict(ids=None), -1),
    (dict(d_table=None), -1), (dict(ldy=7), -1), (dict(ldg=7), -1), (dict(ws=None), -1), (dict(ws=C.c_void_p(264)), -1),
    (dict(nbytes=100), -2)])
def test_lookup_bwd_refusals(change, code):
    a = dict(d_out=P, dtype=0, ldy=8, ids=P, itype=0, n=10_000, rows=100, dim=8, scale=1.0, d_table=P, ldg=8, accumulate=0,
             ws=P, nbytes=1 << 30)
    a.update(change)
    assert L.lib().splat_lookup_bwd(*a.values(), None) == code


@pytest.mark.parametrize("change", [
    dict(dtype=3), dict(param_dtype=1), dict(act=4), dict(channels=0), dict(groups=0), dict(groups=3), dict(eps=-1.0),
    dict(eps=float("nan")), dict(images=-1), dict(pixels=-1), dict(images=1 << 30, pixels=1 << 30),
    dict(x_pixel_stride=-8), dict(x_image_stride=1 << 60), dict(y_pixel_stride=7), dict(y_image_stride=0)])
def test_group_norm_descriptor_refusals(change):
    d = _norm(**change)
    assert L.lib().splat_group_norm(C.byref(d), P, P, P, P, P, P, P, 1 << 30, None) == L.SPLAT_ERR_INVALID_ARG
    if not any(k.startswith("y_") for k in change):
        assert L.lib().splat_group_norm_bwd(C.byref(d), P, P, P, P, P, P, P, P, P, P, 1 << 30,
                                            None) == L.SPLAT_ERR_INVALID_ARG


def test_group_norm_pointer_refusals():
    f, b, d = L.lib().splat_group_norm, L.lib().splat_group_norm_bwd, _norm(pixels=1 << 20)
    bad = [P] * 7
    for k in (0, 3, 4, 5, 6):                # x, y, mean, rstd, workspace
        args = list(bad)
        args[k] = None
        assert f(C.byref(d), *args, 1 << 30, None) == L.SPLAT_ERR_INVALID_ARG
    assert f(C.byref(d), *bad, 8, None) == L.SPLAT_ERR_CAPACITY
    assert f(C.byref(d), C.c_void_p(258), *bad[1:], 1 << 30, None) == L.SPLAT_ERR_INVALID_ARG
    for k in (0, 1, 2, 3, 9):                # d_y, x, mean, rstd, workspace
        args = [P] * 10
        args[k] = None
        assert b(C.byref(d), *args, 1 << 30, None) == L.SPLAT_ERR_INVALID_ARG
    assert b(C.byref(d), *[P] * 10, 8, None) == L.SPLAT_ERR_CAPACITY
    overlap = _norm(pixels=1 << 20, dx_pixel_stride=4)
    assert b(C.byref(overlap), *[P] * 10, 1 << 30, None) == L.SPLAT_ERR_INVALID_ARG
    # nothing asked for: nothing done
    assert b(C.byref(d), P, P, P, P, P, P, None, None, None, P, 1 << 30, None) == L.SPLAT_OK


@pytest.mark.parametrize("change,code", [
    (dict(dtype=3), -1), (dict(batch=-1), -1), (dict(batch=65536), -1), (dict(rows=70000), -1), (dict(cols=-1), -1),
    (dict(steps=0), -1), (dict(steps=65), -1), (dict(a=float("nan")), -1), (dict(eps=-1e-7), -1),
    (dict(scale=float("inf")), -1), (dict(a=20.0), -4), (dict(g=None), -1), (dict(out=None), -1), (dict(gr=9), -1),
    (dict(orow=9), -1), (dict(gb=-1), -1), (dict(ws=None), -1), (dict(nbytes=64), -2)])
def test_orthogonalize_refusals(change, code):
    a = dict(g=P, dtype=0, batch=2, rows=300, cols=400, gb=120000, gr=400, steps=5, a=3.4445, b=-4.775, c=2.0315,
             eps=1e-7, scale=1.0, out=P, ob=120000, orow=400, ws=P, nbytes=1 << 30)
    a.update(change)
    assert L.lib().splat_orthogonalize(*a.values(), None) == code


def test_sizes_of_zero_touch_nothing():
    lib = L.lib()
    assert lib.splat_lookup(None, 0, 0, 8, 8, None, 0, 0, 1.0, None, 8, None) == L.SPLAT_OK
    assert lib.splat_lookup_bwd(None, 0, 8, None, 0, 0, 0, 8, 1.0, None, 8, 0, None, 0, None) == L.SPLAT_OK
    assert lib.splat_lookup_bwd(P, 0, 8, P, 0, 0, 4, 8, 1.0, P, 8, 1, None, 0, None) == L.SPLAT_OK
    d = _norm(images=0)
    assert lib.splat_group_norm(C.byref(d), None, None, None, None, None, None, None, 0, None) == L.SPLAT_OK
    assert lib.splat_orthogonalize(None, 0, 0, 8, 8, 64, 8, 5, 3.4445, -4.775, 2.0315, 1e-7, 1.0, None, 64, 8, None, 0,
                                   None) == L.SPLAT_OK


@pytest.mark.parametrize("images", [0, 1, 2, 600])
@pytest.mark.parametrize("channels,groups", [(8, 2), (9, 3), (1, 1), (4096, 1)])
def test_group_norm_of_no_pixels(images, channels, groups):
    """Neither query divides by the pixels, and the backward wants nothing for them."""
    for dtype in (L.SPLAT_F32, L.SPLAT_F16, L.SPLAT_BF16):
        d = _norm(images=images, pixels=0, channels=channels, groups=groups, dtype=dtype, param_dtype=dtype,
                  x_pixel_stride=channels, y_pixel_stride=channels, dx_pixel_stride=channels, x_image_stride=channels,
                  y_image_stride=channels, dx_image_stride=channels)
        assert L.splat_group_norm_workspace_bytes(d, False) == 0
        assert L.splat_group_norm_workspace_bytes(d, True) == 0
        assert L.lib().splat_group_norm_bwd(C.byref(d), None, None, None, None, None, None, None, None, None, None, 0,
                                            None) == L.SPLAT_OK


def test_packed_images_of_no_pixels_do_not_overlap():
    """Packed images of no pixels lie zero elements apart, as a contiguous tensor's do."""
    d = _norm(images=3, pixels=0, x_image_stride=0, y_image_stride=0, dx_image_stride=0)
    assert L.lib().splat_group_norm_bwd(C.byref(d), None, None, P, P, None, None, P, None, None, None, 0,
                                        None) == L.SPLAT_OK
    d.pixels = 1
    assert L.lib().splat_group_norm_bwd(C.byref(d), P, P, P, P, None, None, P, None, None, P, 1 << 20,
                                        None) == L.SPLAT_ERR_INVALID_ARG


def test_group_norm_of_no_pixels_still_has_statistics_to_write():
    f, d = L.lib().splat_group_norm, _norm(pixels=0)
    for mean, rstd in ((None, P), (P, None), (C.c_void_p(258), P)):
        assert f(C.byref(d), None, None, None, None, mean, rstd, None, 0, None) == L.SPLAT_ERR_INVALID_ARG


@pytest.mark.parametrize("ob,orow,code", [
    (0, 400, -1), (400, 400, -1), (119_999, 400, -1), (120_000, 400, -2), (120_000, 399, -1), (400, 800, -2),
    (399, 800, -1), (400, 799, -1), (119_600 + 400, 400, -2), (299 * 500 + 400, 500, -2), (299 * 500 + 399, 500, -1)])
def test_output_matrices_that_overlap_are_refused(ob, orow, code):
    """Two 300 x 400 results one after the other or interleaved by rows; nothing between. The
    accepted ones stop at their workspace (-2)."""
    a = dict(g=P, dtype=0, batch=2, rows=300, cols=400, gb=120000, gr=400, steps=5, a=3.4445, b=-4.775, c=2.0315,
             eps=1e-7, scale=1.0, out=P, ob=ob, orow=orow, ws=P, nbytes=64)
    assert L.lib().splat_orthogonalize(*a.values(), None) == code


@pytest.mark.parametrize("image,pixel", [((8 << 20) - 1, 8), (8, 8), (8, 15), (9, 16), (0, 8), (1 << 20, 9)])
def test_output_images_that_overlap_are_refused(image, pixel):
    """Two images of 2^20 pixels of 8 channels are written apart or interleaved by pixels."""
    d = _norm(pixels=1 << 20, y_image_stride=image, y_pixel_stride=pixel)
    assert L.lib().splat_group_norm(C.byref(d), *[P] * 7, 1 << 40, None) == L.SPLAT_ERR_INVALID_ARG
    d = _norm(pixels=1 << 20, x_image_stride=8 << 20, y_image_stride=8 << 20, dx_image_stride=image, dx_pixel_stride=pixel)
    assert L.lib().splat_group_norm_bwd(C.byref(d), *[P] * 10, 1 << 40, None) == L.SPLAT_ERR_INVALID_ARG


def test_python_refusals_without_a_gpu():
    from sphere_rasterization_amd import appearance as A
    t = torch.zeros(4, 8)
    ids = torch.zeros(3, dtype=torch.int64)
    with pytest.raises(ValueError, match="GPU tensor"):
        A.lookup(t, ids)
    with pytest.raises(ValueError, match="float32, float16 or bfloat16"):
        A.lookup(t.double(), ids)
    with pytest.raises(ValueError, match="rows, dim"):
        A.lookup(t[0], ids)
    with pytest.raises(ValueError, match="act"):
        A.group_norm(t, 2, act="tanh")
    with pytest.raises(ValueError, match="images"):
        A.group_norm(t[0], 2)
    with pytest.raises(ValueError, match="rows, cols"):
        A.orthogonalize(t[0])


def test_forward_mode_is_refused():
    """A tangent can not be followed through the kernels: it is refused, not dropped."""
    import torch.autograd.forward_ad as fwd
    from sphere_rasterization_amd import appearance as A
    t, ids, w = torch.zeros(4, 8), torch.zeros(3, dtype=torch.int64), torch.ones(8)
    with fwd.dual_level():
        dual, dual_w = fwd.make_dual(t, torch.ones_like(t)), fwd.make_dual(w, torch.ones_like(w))
        for call in (lambda: A.lookup(dual, ids), lambda: A.group_norm(dual, 2), lambda: A.group_norm(t, 2, dual_w),
                     lambda: A.group_norm(t, 2, w, dual_w), lambda: A.orthogonalize(dual),
                     lambda: A.lookup_backward(dual[:3], ids, 4), lambda: A.group_norm_forward(dual, 2),
                     lambda: A.group_norm_backward(dual, t, torch.zeros(4, 2), torch.zeros(4, 2)),
                     lambda: A.lookup(dual.requires_grad_(), ids)):
            with pytest.raises(NotImplementedError, match="forward-mode"):
                call()
        with pytest.raises(ValueError, match="GPU tensor"):   # no tangent: as ever
            A.lookup(t, ids)


class _Huge:
    """A tensor's face alone: sizes past 31 bits without their memory."""

    def __init__(self, *shape, dtype=torch.float16):
        self.shape, self.dtype, self.is_cuda, self.device = shape, dtype, True, torch.device("cuda:0")
        self.requires_grad = False

    def dim(self):
        return len(self.shape)

    def numel(self):
        n = 1
        for k in self.shape:
            n *= k
        return n


def test_sizes_past_31_bits_do_not_wrap():
    """A size or count that C's int does not hold is refused, not taken modulo 2^32."""
    from sphere_rasterization_amd import appearance as A
    big, t = (1 << 32) + 8, torch.zeros(4, 8)
    ids = _Huge(3, dtype=torch.int64)
    gpu = _Huge(4, 8)
    for call in (lambda: A.lookup(_Huge(1, big), ids), lambda: A.lookup_backward(_Huge(3, big), ids, 1),
                 lambda: A.group_norm(gpu, (1 << 32) + 2), lambda: A.group_norm(gpu, -(1 << 32) + 2),
                 lambda: A.group_norm(_Huge(2, big), 2), lambda: A.orthogonalize(_Huge(big, 1)),
                 lambda: A.orthogonalize(_Huge(1, big)), lambda: A.orthogonalize(gpu, steps=(1 << 32) + 5)):
        with pytest.raises(ValueError, match="2\\^31"):
            call()
    for call in (lambda: A.group_norm(gpu, 2.7), lambda: A.orthogonalize(gpu, steps=2.5)):
        with pytest.raises(ValueError, match="whole number"):
            call()
