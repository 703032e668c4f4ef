"""Larger layers that between them reach every tile of the dense layers' products, whole and with
the summed axis split, and the rule that chooses."""
import ctypes as C

from sphere_rasterization_amd import _lib as L

# rows, in, out: whole 16-byte chunks both ways, ends inside tiles and stages
LARGE = [(3003, 392, 4104), (2051, 16392, 392), (2563, 264, 2312), (2051, 6152, 264), (3003, 4104, 392), (2051, 392, 8200),
         (2563, 2312, 264), (2051, 264, 3080), (515, 5128, 2312), (5003, 3080, 392), (3003, 2056, 264), (515, 16392, 264),
         (12001, 392, 264)]


class Cut(C.Structure):
    _fields_ = [("tile", C.c_int), ("splits", C.c_int)]


def cut(i, j, k, parts, f32):
    """(tile, splits) of a product with i x j sums of k products."""
    rule = L.lib()._Z11product_cutlllii                     # product_cut of csrc/linear.hip
    rule.restype, rule.argtypes = Cut, [C.c_int64] * 3 + [C.c_int] * 2
    c = rule(i, j, k, parts, L.SPLAT_F32 if f32 else L.SPLAT_F16)
    return c.tile, c.splits
