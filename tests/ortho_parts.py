"""The orthogonalised update with its factors held in two fp16 parts, on the CPU, and the
error that tells both parts from one.

BOUND is on the Frobenius error relative to the result, for fp32 matrices of independent
values and the usual five steps. Two parts hold 22 bits and give at most 2e-6 (shapes from
1x7 to 513x9000); a product that misses a lo part of either factor, 12 bits or less, gives
at least 1.4e-4. BOUND lies between, fifteen times the one and a quarter of the other;
test_oracle_appearance.py holds both sides to it.
"""
import numpy as np

BOUND = 2.0 ** -15
A, B, C = 3.4445, -4.7750, 2.0315
PRODUCTS = ("gram", "poly", "next")           # X X^T, A A and B X
CROSS = ("hi lo", "lo hi")


def _exponent(bound):
    """Of the largest power of two S with 1.02 bound S in fp16's range."""
    return int(np.frexp(65504.0 / (1.02 * bound))[1]) - 1


def _parts(v):
    v = v.astype(np.float32)
    hi = v.astype(np.float16)
    return hi.astype(np.float32), (v - hi.astype(np.float32)).astype(np.float16).astype(np.float32)


def _product(p, q, lost):
    """P Q^T of factors in parts, without the cross products in `lost`."""
    r = p[0] @ q[0].T
    if "hi lo" not in lost:
        r = r + p[0] @ q[1].T
    if "lo hi" not in lost:
        r = r + p[1] @ q[0].T
    return r


def orthogonalize(g, lost=None, steps=5):
    """`lost`: cross products left out, by product."""
    lost = lost or {}
    x = np.asarray(g, np.float64)
    tall = x.shape[0] > x.shape[1]
    x = x.T if tall else x
    u, grid = 1.0, np.linspace(0.0, 1.0, 4097)
    ex = _exponent(u)
    x = _parts(x / (np.sqrt((x * x).sum()) + 1e-7) * 2.0 ** ex)
    for k in range(steps):
        s = grid * u
        ea, eb = _exponent(u * u), _exponent(np.abs(A + s * s * (B + C * s * s)).max())
        u = np.abs(s * (A + s * s * (B + C * s * s))).max()
        en = _exponent(u)
        a = _parts(_product(x, x, lost.get("gram", ())) * np.float32(2.0 ** (ea - 2 * ex)))
        b = _product(a, a, lost.get("poly", ())) * np.float32(C * 2.0 ** (eb - 2 * ea))
        b = b + np.float32(B * 2.0 ** (eb - ea)) * (a[0] + a[1])
        b[np.diag_indices(len(b))] += np.float32(A * 2.0 ** eb)
        n = _product(_parts(b), (x[0].T, x[1].T), lost.get("next", ()))
        last = k + 1 == steps
        n = n * np.float32(2.0 ** (-(eb + ex) if last else en - eb - ex))
        x, ex = (n if last else _parts(n)), en
    return x.T if tall else x


def error(got, ref):
    return float(np.linalg.norm(got - ref) / np.linalg.norm(ref))
