"""Learned appearance on either side of the renderer: shared features, shading, updates.

    feat = lookup(table, ids)                          # features of n primitives from one table
    img = autograd.render(rz, feat=feat)               # rendered feature image
    h = linear(img, w, b, act="silu", residual=r,      # a dense layer of a channels-last
               p=0.1, rng=(seed, step))                # shading network, with dropout
    y = group_norm(h, 8, weight, bias, act="silu")     # its normalisation
    y = dropout(y, 0.1, (seed, step), residual=r)
    step = orthogonalize(momentum)                     # update of the network's matrices

`lookup`, `linear`, `group_norm` and `dropout` carry autograd; `lookup_backward`,
`linear_forward`, `linear_backward`, `group_norm_forward`, `group_norm_backward` and
`dropout_backward` are the same kernels without it. Forward-mode derivatives are refused:
a tensor with a tangent raises NotImplementedError. Every step runs in libsplat's HIP
kernels (csrc/lookup.hip, csrc/linear.hip, csrc/dropout.hip, csrc/group_norm.hip,
csrc/orthogonalize.hip); torch provides device memory and the stream. Tensors are float32,
float16 or bfloat16 on one GPU, and work is enqueued on that GPU's current stream. Arithmetic
is fp32 with one rounding at the end (`linear_backward` says what else is rounded there), sums
run in a fixed order (equal inputs give equal bits), and no call waits for the device. Tensors
whose last axis is not contiguous, or whose pixels are not evenly spaced, are copied first;
everything else is read in place.
"""
from __future__ import annotations

import math
from typing import Optional, Sequence, Tuple

import torch
from torch.autograd import forward_ad
from torch.autograd.function import once_differentiable

from . import _lib as L

_DTYPES = {torch.float32: L.SPLAT_F32, torch.float16: L.SPLAT_F16, torch.bfloat16: L.SPLAT_BF16}
_ITYPES = {torch.int32: L.SPLAT_I32, torch.int64: L.SPLAT_I64}
ACTS = {"none": L.SPLAT_ACT_NONE, "relu": L.SPLAT_ACT_RELU, "silu": L.SPLAT_ACT_SILU, "gelu": L.SPLAT_ACT_GELU}


def _dtype(name: str, t: torch.Tensor) -> int:
    code = _DTYPES.get(t.dtype)
    if code is None:
        raise ValueError(f"{name}: expected float32, float16 or bfloat16, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name}: expected a GPU tensor, got one on {t.device}")
    return code


def _int32(name: str, v) -> int:
    """v as the C calls take it: ctypes would keep the low 32 bits of a larger number."""
    k = int(v)
    if k != v:
        raise ValueError(f"{name}: expected a whole number, got {v!r}")
    if not -(1 << 31) <= k < 1 << 31:
        raise ValueError(f"{name}: expected less than 2^31, got {k}")
    return k


def _like(name: str, t: torch.Tensor, ref: torch.Tensor, shape, dtypes):
    if t.device != ref.device or t.dtype not in dtypes or tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: expected {tuple(shape)} of {' or '.join(str(d) for d in dtypes)} on {ref.device}, "
                         f"got {tuple(t.shape)} of {t.dtype} on {t.device}")


def _no_tangents(*tensors: Optional[torch.Tensor]):
    """Refuses dual tensors: the kernels see no tangents, and would drop them in silence."""
    if forward_ad._current_level < 0:        # outside every dual level
        return
    for t in tensors:
        if isinstance(t, torch.Tensor) and forward_ad.unpack_dual(t).tangent is not None:
            raise NotImplementedError("forward-mode derivatives of the appearance operators are not available")


def _launch(t: torch.Tensor, fn, *args):
    """fn(*args, stream) on the current stream of t's GPU, with that GPU current."""
    dev = t.get_device()
    if dev == torch.cuda.current_device():
        return fn(*args, torch._C._cuda_getCurrentRawStream(dev))
    with torch.cuda.device(dev):
        return fn(*args, torch._C._cuda_getCurrentRawStream(dev))


def _workspace(nbytes: int, ref: torch.Tensor) -> Tuple[Optional[torch.Tensor], Optional[int], int]:
    """(memory to keep until the call returns, its address, its bytes)."""
    if nbytes == 0:
        return None, None, 0
    ws = torch.empty(nbytes, dtype=torch.uint8, device=ref.device)
    return ws, ws.data_ptr(), nbytes


def _packed_like(t: torch.Tensor) -> torch.Tensor:
    """An uninitialised contiguous tensor of t's shape, type and device (1 us less than
    torch.empty of the three)."""
    return torch.empty_like(t, requires_grad=False, memory_format=torch.contiguous_format)


def _rows(t: torch.Tensor) -> torch.Tensor:
    """A 2-D tensor whose rows are contiguous and do not overlap."""
    ok = (t.shape[1] <= 1 or t.stride(1) == 1) and (t.shape[0] <= 1 or t.stride(0) >= t.shape[1])
    return t if ok else t.contiguous()


# ---- shared feature table ---------------------------------------------------------

def _check_ids(ids: torch.Tensor, ref: torch.Tensor) -> int:
    code = _ITYPES.get(ids.dtype)
    if code is None or ids.device != ref.device:
        raise ValueError(f"ids: expected int32 or int64 on {ref.device}, got {ids.dtype} on {ids.device}")
    return code


def _lookup(table: torch.Tensor, ids: torch.Tensor, scale: float) -> torch.Tensor:
    if table.dim() != 2:
        raise ValueError(f"table: expected [rows, dim], got {tuple(table.shape)}")
    dt = _dtype("table", table)
    it = _check_ids(ids, table)
    rows, dim = table.shape[0], _int32("dim", table.shape[1])
    table, flat = _rows(table), ids.contiguous()
    out = torch.empty(tuple(ids.shape) + (dim,), dtype=table.dtype, device=table.device)
    _launch(table, L.splat_lookup, table.data_ptr(), dt, rows, dim, table.stride(0), flat.data_ptr(), it, flat.numel(),
            scale, out.data_ptr(), dim)
    return out


def lookup_backward(d_out: torch.Tensor, ids: torch.Tensor, rows: int, scale: float = 1.0,
                    out: Optional[torch.Tensor] = None, accumulate: bool = False) -> torch.Tensor:
    """Gradient of `lookup` w.r.t. its table of `rows` rows: d_table[v] = scale * (sum of
    d_out over the tokens whose id is v). `out` [rows, dim] receives it (added to what it
    holds with accumulate=True); a new tensor of d_out's type otherwise."""
    _no_tangents(d_out, out)
    dt = _dtype("d_out", d_out)
    it = _check_ids(ids, d_out)
    if d_out.dim() < 1 or tuple(d_out.shape[:-1]) != tuple(ids.shape):
        raise ValueError(f"d_out: expected {tuple(ids.shape)} + (dim,), got {tuple(d_out.shape)}")
    dim = _int32("dim", d_out.shape[-1])
    if accumulate and out is None:
        raise ValueError("accumulate needs out")
    given = out is not None
    if not given:
        out = torch.empty((rows, dim), dtype=d_out.dtype, device=d_out.device)
    else:
        _like("out", out, d_out, (rows, dim), (d_out.dtype,))
        if _rows(out) is not out:
            raise ValueError("out: rows must be contiguous and must not overlap")
    n = ids.numel()
    dy, flat = _rows(d_out.reshape(n, dim)), ids.contiguous()
    _keep, ws, nbytes = _workspace(L.splat_lookup_bwd_workspace_bytes(n, rows, dim), d_out)
    _launch(d_out, L.splat_lookup_bwd, dy.data_ptr(), dt, dy.stride(0), flat.data_ptr(), it, n, rows, dim, scale,
            out.data_ptr(), out.stride(0), 1 if accumulate else 0, ws, nbytes)
    if given:                                # a graph that has saved it has to know
        torch.autograd.graph.increment_version(out)
    return out


class _Lookup(torch.autograd.Function):
    @staticmethod
    def forward(ctx, table, ids, scale):
        ctx.save_for_backward(ids)
        ctx.rows, ctx.scale = table.shape[0], scale
        return _lookup(table, ids, scale)

    @staticmethod
    @once_differentiable
    def backward(ctx, d_out):
        (ids,) = ctx.saved_tensors
        return lookup_backward(d_out, ids, ctx.rows, ctx.scale), None, None


def lookup(table: torch.Tensor, ids: torch.Tensor, scale: float = 1.0) -> torch.Tensor:
    """scale * table[ids]: rows of a feature table that primitives share, [*ids.shape, dim].
    Ids outside [0, rows) (primitives without an entry, -1 say) give zeros and receive no
    gradient. The gradient is dense, [rows, dim]."""
    _no_tangents(table)
    if torch.is_grad_enabled() and table.requires_grad:
        return _Lookup.apply(table, ids, float(scale))
    return _lookup(table, ids, float(scale))


# ---- group norm with an activation --------------------------------------------------

def _pixels(t: torch.Tensor) -> Tuple[torch.Tensor, int, int]:
    """(tensor, image stride, pixel stride) of [N, ..., C] read as [N][pixels][C]; a copy
    where the pixels are not evenly spaced."""
    if t.is_contiguous():
        n, c = t.shape[0], t.shape[-1]
        return t, t.numel() // n if n else 0, c
    if t.shape[-1] <= 1 or t.stride(-1) == 1:
        dims = [(t.shape[i], t.stride(i)) for i in range(1, t.dim() - 1) if t.shape[i] != 1]
        if all(dims[i][1] == dims[i + 1][1] * dims[i + 1][0] for i in range(len(dims) - 1)):
            return t, t.stride(0), dims[-1][1] if dims else t.shape[-1]
    return _pixels(t.contiguous())


def _norm_desc(x, weight, bias, groups: int, act: str, eps: float) -> L.splat_norm:
    if x.dim() < 2:
        raise ValueError(f"x: expected [images, ..., channels], got {tuple(x.shape)}")
    if act not in ACTS:
        raise ValueError(f"act: expected one of {', '.join(ACTS)}, got {act!r}")
    d = L.splat_norm()
    d.dtype = _dtype("x", x)
    shape = x.shape
    d.images, d.pixels, d.channels = shape[0], math.prod(shape[1:-1]), _int32("channels", shape[-1])
    d.groups, d.act, d.eps = _int32("groups", groups), ACTS[act], float(eps)
    kind = None
    for name, p in (("weight", weight), ("bias", bias)):
        if p is not None:
            _like(name, p, x, (x.shape[-1],), (torch.float32, x.dtype) if kind is None else (kind,))
            kind = p.dtype
    d.param_dtype = _DTYPES[kind if kind is not None else x.dtype]
    return d


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _flat(t: Optional[torch.Tensor]):
    return t if t is None or t.is_contiguous() else t.contiguous()


def _group_norm(x, groups, weight, bias, eps, act, keep: bool):
    """y and, if kept, the statistics [2, images, groups] (mean, rstd)."""
    d = _norm_desc(x, weight, bias, groups, act, eps)
    x, d.x_image_stride, d.x_pixel_stride = _pixels(x)
    weight, bias = _flat(weight), _flat(bias)
    y = _packed_like(x)
    d.y_image_stride, d.y_pixel_stride = d.pixels * d.channels, d.channels
    one, nbytes = 4 * d.images * d.groups, L.splat_group_norm_workspace_bytes(d, False)
    if keep:
        stats = torch.empty((2, d.images, d.groups), dtype=torch.float32, device=x.device)
        mean = stats.data_ptr()
        _ws, ws, nbytes = _workspace(nbytes, x)
    else:                                    # one allocation: the workspace, then the statistics
        stats, ws, _n = _workspace(nbytes + 2 * one, x)
        mean = (ws or 0) + nbytes
    _launch(x, L.splat_group_norm, d, x.data_ptr(), _ptr(weight), _ptr(bias), y.data_ptr(), mean, mean + one, ws, nbytes)
    return y, stats


def group_norm_forward(x: torch.Tensor, groups: int, weight: Optional[torch.Tensor] = None,
                       bias: Optional[torch.Tensor] = None, eps: float = 1e-5, act: str = "none"):
    """(y, mean, rstd) of `group_norm`: mean and rstd [images, groups] are what the
    backward needs besides x."""
    _no_tangents(x, weight, bias)
    y, stats = _group_norm(x, groups, weight, bias, eps, act, True)
    return y, stats[0], stats[1]


def group_norm_backward(d_y: torch.Tensor, x: torch.Tensor, mean: torch.Tensor, rstd: torch.Tensor,
                        weight: Optional[torch.Tensor] = None, bias: Optional[torch.Tensor] = None, act: str = "none",
                        want: Sequence[str] = ("x", "weight", "bias")):
    """(d_x, d_weight, d_bias) given d_y and the forward's x, mean and rstd; None for what
    `want` leaves out. d_weight and d_bias have the type of weight and bias (of x without
    either)."""
    _no_tangents(d_y, x, mean, rstd, weight, bias)
    if mean.dim() != 2:
        raise ValueError(f"mean: expected [images, groups], got {tuple(mean.shape)}")
    d = _norm_desc(x, weight, bias, mean.shape[1], act, 0.0)
    _like("d_y", d_y, x, x.shape, (x.dtype,))
    for name, s in (("mean", mean), ("rstd", rstd)):
        _like(name, s, x, (d.images, d.groups), (torch.float32,))
    x, d.x_image_stride, d.x_pixel_stride = _pixels(x)
    d_y, d.y_image_stride, d.y_pixel_stride = _pixels(d_y)
    weight, bias, mean, rstd = _flat(weight), _flat(bias), _flat(mean), _flat(rstd)
    kind = weight.dtype if weight is not None else bias.dtype if bias is not None else x.dtype
    dx = _packed_like(x) if "x" in want else None
    dw = torch.empty(d.channels, dtype=kind, device=x.device) if "weight" in want else None
    db = torch.empty(d.channels, dtype=kind, device=x.device) if "bias" in want else None
    d.dx_image_stride, d.dx_pixel_stride = d.pixels * d.channels, d.channels
    _keep, ws, nbytes = _workspace(L.splat_group_norm_workspace_bytes(d, True), x)
    _launch(x, L.splat_group_norm_bwd, d, d_y.data_ptr(), x.data_ptr(), mean.data_ptr(), rstd.data_ptr(), _ptr(weight),
            _ptr(bias), _ptr(dx), _ptr(dw), _ptr(db), ws, nbytes)
    return dx, dw, db


class _GroupNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, groups, weight, bias, eps, act):
        y, mean, rstd = group_norm_forward(x, groups, weight, bias, eps, act)
        ctx.save_for_backward(x, mean, rstd, weight, bias)
        ctx.act = act
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, d_y):
        x, mean, rstd, weight, bias = ctx.saved_tensors
        need = ctx.needs_input_grad
        want = [n for n, k in (("x", need[0]), ("weight", need[2]), ("bias", need[3])) if k]
        dx, dw, db = group_norm_backward(d_y, x, mean, rstd, weight, bias, ctx.act, want)
        return dx, None, dw, db, None, None


def group_norm(x: torch.Tensor, groups: int, weight: Optional[torch.Tensor] = None,
               bias: Optional[torch.Tensor] = None, eps: float = 1e-5, act: str = "none") -> torch.Tensor:
    """act(weight * (x - mean) / sqrt(var + eps) + bias) over channels-last images
    [images, ..., channels], mean and variance over each image's pixels and the
    channels / groups channels of a group. act: none, relu, silu or gelu (with erf).
    weight and bias [channels], float32 or x's type. An NCHW tensor in torch's
    channels_last memory format is read in place as x.permute(0, 2, 3, 1)."""
    _no_tangents(x, weight, bias)
    if torch.is_grad_enabled() and (x.requires_grad or (weight is not None and weight.requires_grad)
                                    or (bias is not None and bias.requires_grad)):
        return _GroupNorm.apply(x, groups, weight, bias, eps, act)
    return _group_norm(x, groups, weight, bias, eps, act, False)[0]


# ---- dense layers and dropout --------------------------------------------------------

def _word(name: str, v) -> int:
    k = int(v)
    if k != v or not 0 <= k < 1 << 64:
        raise ValueError(f"{name}: expected a whole number from 0 to 2^64 - 1, got {v!r}")
    return k


_NO_DROP = L.splat_drop()


def _drop(p: float, rng, ref: torch.Tensor) -> L.splat_drop:
    """The descriptor of dropout for tensors on ref's device."""
    p = float(p)
    if not 0.0 <= p <= 1.0:
        raise ValueError(f"p: expected a number from 0 to 1, got {p!r}")
    if rng is None:
        if p > 0.0:
            raise ValueError("rng: dropout needs (seed, offset) or (state, offset)")
        return _NO_DROP
    if not isinstance(rng, (tuple, list)) or len(rng) != 2:
        raise ValueError("rng: expected (seed, offset) or (state, offset)")
    seed, offset = rng[0], _word("offset", rng[1])
    if not isinstance(seed, torch.Tensor):
        return L.splat_drop(p, _word("seed", seed), offset, None)
    _like("state", seed, ref, (2,), (torch.int64,))
    if seed.stride(0) != 1:
        raise ValueError("state: expected two neighbouring words")
    return L.splat_drop(p, 0, offset, seed.data_ptr())


def _by_rows(t: torch.Tensor, width: int) -> Tuple[torch.Tensor, int]:
    """(tensor, row stride) of t [..., width] read as rows that are contiguous and do not overlap;
    a copy where the rows are not evenly spaced."""
    if t.is_contiguous():
        return t, width
    t = _rows(t.reshape(-1, width) if width else t.reshape(t.shape[:-1].numel(), 0))
    return t, t.stride(0)


def _by_strides(t: torch.Tensor) -> Tuple[torch.Tensor, int, int]:
    """(tensor, strides) of a matrix of which one axis is contiguous and whose rows (or columns)
    do not overlap; a copy of others."""
    r, c = t.shape
    si, so = t.stride()
    if r > 1 and c > 1 and ((so == 1 and si >= c) or (si == 1 and so >= r)):
        return t, si, so
    return t.contiguous(), c, 1


def _check_layer(x, weight, bias, act: str) -> Tuple[int, int, int]:
    """(dtype, inputs, outputs) of a layer whose arguments fit together."""
    if x.dim() < 1 or weight.dim() != 2 or x.shape[-1] != weight.shape[0]:
        raise ValueError(f"expected x [..., in] and weight [in, out], got {tuple(x.shape)} and {tuple(weight.shape)}")
    if act not in ACTS:
        raise ValueError(f"act: expected one of {', '.join(ACTS)}, got {act!r}")
    k, n = weight.shape
    k, n = _int32("in", k), _int32("out", n)
    dt = _dtype("x", x)
    if weight.dtype != x.dtype or weight.device != x.device:
        _like("weight", weight, x, weight.shape, (x.dtype,))
    if bias is not None:
        _like("bias", bias, x, (n,), (torch.float32, x.dtype))
    return dt, k, n


def _linear(x, weight, bias, act, residual, p, rng, keep: bool):
    """y and, where the backward is faster with it and `keep`, z."""
    dt, k, n = _check_layer(x, weight, bias, act)
    drop = _drop(p, rng, x)
    shape = x.shape[:-1] + (n,)
    rs = 0
    if residual is not None:
        _like("residual", residual, x, shape, (x.dtype,))
        residual, rs = _by_rows(residual, n)
    x, xs = _by_rows(x, k)
    weight, wi, wo = _by_strides(weight)
    bdt = dt
    if bias is not None:
        bdt, bias = _DTYPES[bias.dtype], _flat(bias)
    y = torch.empty(shape, dtype=x.dtype, device=x.device)
    d = L.splat_dense(dt, bdt, ACTS[act], k, n, math.prod(shape[:-1]), xs, wi, wo, rs, n, 0, 0, 0, drop)
    pre = _packed_like(y) if keep and L.splat_linear_saves(d) else None
    _keep, ws, nbytes = _workspace(L.splat_linear_workspace_bytes(d, False), x)
    _launch(x, L.splat_linear, d, x.data_ptr(), weight.data_ptr(), _ptr(bias), _ptr(residual), y.data_ptr(), _ptr(pre),
            ws, nbytes)
    return y, pre


def linear_forward(x: torch.Tensor, weight: torch.Tensor, bias: Optional[torch.Tensor] = None, act: str = "none",
                   residual: Optional[torch.Tensor] = None, p: float = 0.0, rng=None):
    """(y, pre) of `linear`: pre is x @ weight + bias, rounded to x's type, where the backward
    is faster when it reads it, and None where it computes it anew."""
    _no_tangents(x, weight, bias, residual)
    return _linear(x, weight, bias, act, residual, p, rng, True)


def linear_backward(d_y: torch.Tensor, x: torch.Tensor, weight: torch.Tensor, bias: Optional[torch.Tensor] = None,
                    act: str = "none", pre: Optional[torch.Tensor] = None, p: float = 0.0, rng=None,
                    want: Sequence[str] = ("x", "weight", "bias")):
    """(d_x, d_weight, d_bias) given d_y and the forward's inputs; None for what `want` leaves
    out. The residual's gradient is d_y. pre: what `linear_forward` returned, or None (it is
    then computed anew). rng has to draw what the forward's drew: a state's words are read
    again. d_weight is laid out as weight is; d_bias has the type of bias (of x without one).
    With 16-bit types and silu or gelu, the gradient at z is multiplied in two parts of that
    type, or, of bfloat16 with in * out >= 2^15 and rows * in * out >= 2^31, rounded to it; an
    infinite x or weight may then give NaN where the formula has an infinity."""
    _no_tangents(d_y, x, weight, bias, pre)
    dt, k, n = _check_layer(x, weight, bias, act)
    drop = _drop(p, rng, x)
    shape = x.shape
    _like("d_y", d_y, x, shape[:-1] + (n,), (x.dtype,))
    if pre is not None:
        _like("pre", pre, x, d_y.shape, (x.dtype,))
        pre = _flat(pre)
    x, xs = _by_rows(x, k)
    d_y, ys = _by_rows(d_y, n)
    weight, wi, wo = _by_strides(weight)
    bdt = dt
    if bias is not None:
        bdt, bias = _DTYPES[bias.dtype], _flat(bias)
    dx = torch.empty(shape, dtype=x.dtype, device=x.device) if "x" in want else None
    dw = None
    if "weight" in want:
        dw = torch.empty((k, n), dtype=x.dtype, device=x.device) if wo == 1 else \
            torch.empty((n, k), dtype=x.dtype, device=x.device).t()
    db = None
    if "bias" in want:
        db = torch.empty(n, dtype=x.dtype if bias is None else bias.dtype, device=x.device)
    dwi, dwo = (n, 1) if wo == 1 else (1, k)
    d = L.splat_dense(dt, bdt, ACTS[act], k, n, math.prod(shape[:-1]), xs, wi, wo, 0, ys, k, dwi, dwo, drop)
    _keep, ws, nbytes = _workspace(L.splat_linear_workspace_bytes(d, True), x)
    _launch(x, L.splat_linear_bwd, d, d_y.data_ptr(), x.data_ptr(), weight.data_ptr(), _ptr(bias), _ptr(pre), _ptr(dx),
            _ptr(dw), _ptr(db), ws, nbytes)
    return dx, dw, db


class _Linear(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, act, residual, p, rng):
        y, pre = _linear(x, weight, bias, act, residual, p, rng, True)
        state = rng[0] if rng is not None and isinstance(rng[0], torch.Tensor) else None
        ctx.save_for_backward(x, weight, bias, pre, state)
        ctx.act, ctx.p, ctx.rng = act, p, None if rng is None else (None if state is not None else rng[0], rng[1])
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, d_y):
        x, weight, bias, pre, state = ctx.saved_tensors
        need = ctx.needs_input_grad
        rng = ctx.rng if state is None else (state, ctx.rng[1])
        dx = dw = db = None
        if need[0] or need[1] or need[2]:
            want = [n for n, k in (("x", need[0]), ("weight", need[1]), ("bias", need[2])) if k]
            dx, dw, db = linear_backward(d_y, x, weight, bias, ctx.act, pre, ctx.p, rng, want)
        return dx, dw, db, None, d_y if need[4] else None, None, None


def linear(x: torch.Tensor, weight: torch.Tensor, bias: Optional[torch.Tensor] = None, act: str = "none",
           residual: Optional[torch.Tensor] = None, p: float = 0.0, rng=None) -> torch.Tensor:
    """residual + drop(act(x @ weight + bias)) in one pass: x [..., in], weight [in, out] of
    x's type with either axis contiguous (the transpose of an [out, in] matrix is read in
    place), bias [out] in float32 or x's type, residual [..., out]. act: none, relu, silu or
    gelu (with erf). p and rng: as in `dropout`, over the elements of the result in order.
    Products of 16-bit values are summed in fp32; the result is rounded once. in and out up
    to 2^20, fewer than 2^31 rows."""
    _no_tangents(x, weight, bias, residual)
    if torch.is_grad_enabled() and (x.requires_grad or weight.requires_grad or (bias is not None and bias.requires_grad)
                                    or (residual is not None and residual.requires_grad)):
        return _Linear.apply(x, weight, bias, act, residual, p, rng)
    return _linear(x, weight, bias, act, residual, p, rng, False)[0]


def _dropout(x, p, rng, residual):
    dt = _dtype("x", x)
    drop = _drop(p, rng, x)
    if residual is not None:
        _like("residual", residual, x, x.shape, (x.dtype,))
    y = _packed_like(x)
    if x.is_contiguous() and (residual is None or residual.is_contiguous()):
        rows, cols, xs, rs = 1, x.numel(), 0, 0
    else:
        cols, rs = x.shape[-1], 0
        rows = x.numel() // cols if cols else 0
        x, xs = _by_rows(x, cols)
        if residual is not None:
            residual, rs = _by_rows(residual, cols)
    _launch(x, L.splat_dropout, drop, dt, rows, cols, x.data_ptr(), xs, _ptr(residual), rs, y.data_ptr(), cols)
    return y


def dropout_backward(d_y: torch.Tensor, p: float, rng) -> torch.Tensor:
    """Gradient of `dropout` w.r.t. x: the same elements of d_y, multiplied by 1 / (1 - p).
    The residual's gradient is d_y."""
    _no_tangents(d_y)
    return _dropout(d_y, p, rng, None)


class _Dropout(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, p, rng, residual):
        state = rng[0] if rng is not None and isinstance(rng[0], torch.Tensor) else None
        y = _dropout(x, p, rng, residual)
        ctx.save_for_backward(state)
        ctx.p, ctx.rng = p, None if rng is None else (None if state is not None else rng[0], rng[1])
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, d_y):
        (state,) = ctx.saved_tensors
        rng = ctx.rng if state is None else (state, ctx.rng[1])
        need = ctx.needs_input_grad
        return (dropout_backward(d_y, ctx.p, rng) if need[0] else None), None, None, d_y if need[3] else None


def dropout(x: torch.Tensor, p: float, rng, residual: Optional[torch.Tensor] = None) -> torch.Tensor:
    """residual + drop(x): each element is set to zero with probability p and multiplied by
    1 / (1 - p) otherwise. The choice is drawn from Philox4x32-10 by the element's place in x
    (in order, whatever the strides) and never stored: the backward draws it again.

    rng: (seed, offset), whole numbers from 0 to 2^64 - 1; the same pair draws the same
    elements, another offset (a number for each step and layer) others. Or (state, offset):
    an int64 tensor of two words on x's GPU, the seed and a number that is added to offset,
    read when the kernels run, so that a captured step that adds to state[1] at its end
    draws anew on every replay. p = 0 leaves every element."""
    _no_tangents(x, residual)
    if torch.is_grad_enabled() and (x.requires_grad or (residual is not None and residual.requires_grad)):
        return _Dropout.apply(x, p, rng, residual)
    return _dropout(x, p, rng, residual)


# ---- orthogonalised updates ----------------------------------------------------------

def orthogonalize(g: torch.Tensor, steps: int = 5, coeffs: Sequence[float] = (3.4445, -4.7750, 2.0315),
                  eps: float = 1e-7, scale: float = 1.0) -> torch.Tensor:
    """scale * (the matrices g [..., rows, cols] with their singular values brought towards
    one): X = g / (|g| + eps), then `steps` times X <- (a I + b A + c A A) X with A = X X^T
    (X transposed if rows > cols). For updates: no autograd. At most 65536 rows and
    columns and 65535 matrices."""
    _no_tangents(g)
    if g.dim() < 2:
        raise ValueError(f"g: expected [..., rows, cols], got {tuple(g.shape)}")
    dt = _dtype("g", g)
    if len(coeffs) != 3:
        raise ValueError("coeffs: expected three numbers")
    rows, cols, steps = _int32("rows", g.shape[-2]), _int32("cols", g.shape[-1]), _int32("steps", steps)
    out = _packed_like(g)
    m = g.detach().reshape((-1, rows, cols)) if g.numel() else g.detach().new_empty((0, rows, cols))
    if (cols > 1 and m.stride(2) != 1) or (rows > 1 and m.stride(1) < cols):
        m = m.contiguous()
    batch = m.shape[0]
    _keep, ws, nbytes = _workspace(L.splat_orthogonalize_workspace_bytes(batch, rows, cols), g)
    _launch(g, L.splat_orthogonalize, m.data_ptr(), dt, batch, rows, cols, m.stride(0), m.stride(1), steps,
            *map(float, coeffs), float(eps), float(scale), out.data_ptr(), rows * cols, cols, ws, nbytes)
    return out
