"""CPU oracle of the dense layers and of dropout (numpy, fp64), written from the formulas.

It shares no code with the HIP path (csrc/linear.hip, csrc/dropout.hip, csrc/random.h). The
random numbers are Philox4x32-10 of Salmon, Moraes, Dror and Shaw (2011), in Python's own
integers and in numpy's for arrays.
"""
from __future__ import annotations

import numpy as np

from oracle.appearance import act, act_slope

M0, M1, W0, W1 = 0xD2511F53, 0xCD9E8D57, 0x9E3779B9, 0xBB67AE85


def philox(counter, key):
    """Four words from four words and two, as Python integers."""
    a, b, c, d = counter
    k0, k1 = key
    for _ in range(10):
        p, q = a * M0, c * M1
        a, b, c, d = (q >> 32) ^ b ^ k0, q & 0xFFFFFFFF, (p >> 32) ^ d ^ k1, p & 0xFFFFFFFF
        k0, k1 = (k0 + W0) & 0xFFFFFFFF, (k1 + W1) & 0xFFFFFFFF
    return a, b, c, d


def _philox_blocks(block, half, seed, offset):
    m, s = np.uint64(0xFFFFFFFF), np.uint64(32)
    a, b = block & m, (block >> s) + np.uint64(half << 31)
    c, d = np.full_like(block, offset & 0xFFFFFFFF), np.full_like(block, offset >> 32)
    k0, k1 = seed & 0xFFFFFFFF, seed >> 32
    for _ in range(10):
        p, q = a * np.uint64(M0), c * np.uint64(M1)
        a, b, c, d = (q >> s) ^ b ^ np.uint64(k0), q & m, (p >> s) ^ d ^ np.uint64(k1), p & m
        k0, k1 = (k0 + W0) & 0xFFFFFFFF, (k1 + W1) & 0xFFFFFFFF
    return np.stack([a, b, c, d], axis=-1)


def uniform(first, count, seed, offset):
    """The 32-bit numbers u_i of elements first .. first + count - 1."""
    i = np.arange(first, first + count, dtype=np.uint64)
    block, at = np.unique(i >> np.uint64(3), return_inverse=True)
    u = np.zeros(count, np.int64)
    for half in (0, 1):
        w = _philox_blocks(block, half, seed, offset)[at, (i & np.uint64(7)).astype(np.int64) >> 1]
        piece = (w >> (np.uint64(16) * (i & np.uint64(1)))) & np.uint64(0xFFFF)
        u = (u << 16) | piece.astype(np.int64)
    return u


def kept(shape, p, seed, offset, first=0):
    n = int(np.prod(shape, dtype=np.int64))
    return (uniform(first, n, seed, offset) >= round(p * 2.0 ** 32)).reshape(shape)


def dropout(x, p, seed, offset, residual=None):
    x = np.asarray(x, np.float64)
    if p > 0:
        x = np.where(kept(x.shape, p, seed, offset), x / (1.0 - p) if p < 1 else 0.0, 0.0)
    return x if residual is None else x + np.asarray(residual, np.float64)


def linear(x, w, b=None, kind="none", residual=None, p=0.0, seed=0, offset=0):
    """dict of y and z."""
    z = np.asarray(x, np.float64) @ np.asarray(w, np.float64)
    if b is not None:
        z = z + np.asarray(b, np.float64)
    return dict(z=z, y=dropout(act(z, kind), p, seed, offset, residual))


def linear_backward(d_y, x, w, b=None, kind="none", p=0.0, seed=0, offset=0):
    """dict of dx, dw, db and the per-value dz and z."""
    x, w = np.asarray(x, np.float64), np.asarray(w, np.float64)
    z = linear(x, w, b)["z"]
    dz = dropout(d_y, p, seed, offset) * act_slope(z, kind)
    flat = dz.reshape(-1, w.shape[1])
    return dict(z=z, dz=dz, dx=dz @ w.T, dw=x.reshape(-1, w.shape[0]).T @ flat, db=flat.sum(0))
