"""CPU oracle of the appearance operators (numpy, fp64), written from the formulas.

It shares no code with the HIP path (csrc/lookup.hip, csrc/group_norm.hip,
csrc/orthogonalize.hip). Beside each result it can give the magnitude of the terms
behind it, from which the tests derive the error an fp32 evaluation may have.
"""
from __future__ import annotations

import math

import numpy as np

try:
    from scipy.special import erf as _erf
except ImportError:                                   # element by element, the same function
    _erf = np.vectorize(math.erf, otypes=[np.float64])


def lookup(table, ids, scale=1.0):
    table, ids = np.asarray(table, np.float64), np.asarray(ids)
    out = np.zeros(ids.shape + (table.shape[1],))
    ok = (ids >= 0) & (ids < table.shape[0])
    out[ok] = scale * table[ids[ok]]
    return out


def lookup_backward(d_out, ids, rows, scale=1.0):
    d_out, ids = np.asarray(d_out, np.float64), np.asarray(ids).reshape(-1)
    d = np.zeros((rows, d_out.shape[-1]))
    ok = (ids >= 0) & (ids < rows)
    np.add.at(d, ids[ok], scale * d_out.reshape(ids.size, -1)[ok])
    return d


def act(z, kind):
    if kind == "relu":
        return np.maximum(z, 0.0)
    if kind == "silu":
        return z / (1.0 + np.exp(-z))
    if kind == "gelu":
        return 0.5 * z * (1.0 + _erf(z / math.sqrt(2.0)))
    return z


def act_slope(z, kind):
    if kind == "relu":
        return (z > 0.0).astype(np.float64)
    if kind == "silu":
        s = 1.0 / (1.0 + np.exp(-z))
        return s + z * s * (1.0 - s)
    if kind == "gelu":
        return 0.5 * (1.0 + _erf(z / math.sqrt(2.0))) + z * np.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
    return np.ones_like(z)


def group_norm(x, groups, weight=None, bias=None, eps=1e-5, kind="none"):
    """dict of y, mean, rstd [N, G] and, per value, xh and z (x's shape)."""
    x = np.asarray(x, np.float64)
    n, c = x.shape[0], x.shape[-1]
    w = np.ones(c) if weight is None else np.asarray(weight, np.float64)
    b = np.zeros(c) if bias is None else np.asarray(bias, np.float64)
    v = x.reshape(n, -1, groups, c // groups)
    mean = v.mean(axis=(1, 3))
    var = ((v - mean[:, None, :, None]) ** 2).mean(axis=(1, 3))
    rstd = 1.0 / np.sqrt(var + eps)
    xh = ((v - mean[:, None, :, None]) * rstd[:, None, :, None]).reshape(x.shape)
    z = xh * w + b
    return dict(y=act(z, kind), mean=mean, rstd=rstd, xh=xh, z=z, w=w)


def group_norm_backward(d_y, x, groups, weight=None, bias=None, eps=1e-5, kind="none"):
    """dict of dx, dw, db and the per-value dz, given the forward's inputs."""
    f = group_norm(x, groups, weight, bias, eps, kind)
    d_y = np.asarray(d_y, np.float64)
    n, c = d_y.shape[0], d_y.shape[-1]
    dz = d_y * act_slope(f["z"], kind)
    shape = (n, -1, groups, c // groups)
    g = (dz * f["w"]).reshape(shape)
    h = f["xh"].reshape(shape)
    m1 = g.mean(axis=(1, 3), keepdims=True)
    m2 = (g * h).mean(axis=(1, 3), keepdims=True)
    dx = (f["rstd"][:, None, :, None] * (g - m1 - h * m2)).reshape(d_y.shape)
    return dict(f, dx=dx, dw=(dz * f["xh"]).reshape(-1, c).sum(0), db=dz.reshape(-1, c).sum(0), dz=dz)


def orthogonalize(g, steps=5, coeffs=(3.4445, -4.7750, 2.0315), eps=1e-7, scale=1.0):
    """The quintic applied to the singular values."""
    a, b, c = coeffs
    u, s, vt = np.linalg.svd(np.asarray(g, np.float64), full_matrices=False)
    s = s / (np.sqrt((s * s).sum(-1, keepdims=True)) + eps)
    for _ in range(steps):
        s = a * s + b * s ** 3 + c * s ** 5
    return scale * np.matmul(u * s[..., None, :], vt)
