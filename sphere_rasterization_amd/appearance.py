"""Learned appearance on either side of the renderer: shared features, shading, updates.

    feat = lookup(table, ids)                          # features of n primitives from one table
    img = autograd.render(rz, feat=feat)               # rendered feature image
    y = group_norm(h, 8, weight, bias, act="silu")     # inside a channels-last shading network
    step = orthogonalize(momentum)                     # update of the network's matrices

`lookup` and `group_norm` carry autograd; `lookup_backward`, `group_norm_forward` and
`group_norm_backward` are the same kernels without it. Forward-mode derivatives are refused:
a tensor with a tangent raises NotImplementedError. Every step runs in libsplat's HIP
kernels (csrc/lookup.hip, csrc/group_norm.hip, csrc/orthogonalize.hip); torch provides
device memory and the stream. Tensors are float32, float16 or bfloat16 on one GPU, and
work is enqueued on that GPU's current stream. Arithmetic is fp32 with one rounding at
the end, sums run in a fixed order (equal inputs give equal bits), and no call waits for
the device. Tensors whose last axis is not contiguous, or whose pixels are not evenly
spaced, are copied first; everything else is read in place.
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
