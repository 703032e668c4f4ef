"""ctypes binding of libsplat's C ABI (include/splat.h).

Argument marshalling only: each function here has the name of the C entry
point it calls and passes device pointers (ints) straight through. The
library must be built (see build.py); nothing here computes any part of the
rasterizer, and there is no fallback when the library is missing.
"""
from __future__ import annotations

import ctypes as C
import os

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libsplat.so")

SPLAT_OK, SPLAT_ERR_INVALID_ARG, SPLAT_ERR_CAPACITY, SPLAT_ERR_HIP, SPLAT_ERR_UNSUPPORTED = 0, -1, -2, -3, -4
SPLAT_PRIM_GAUSS2D, SPLAT_PRIM_GAUSS3D, SPLAT_PRIM_SPHERE = 0, 1, 2
SPLAT_CAM_PINHOLE, SPLAT_CAM_SPHERICAL = 0, 1
SPLAT_MAX_VIEWS, SPLAT_MAX_CHANNELS = 16, 64
SPLAT_F32, SPLAT_F16, SPLAT_BF16 = 0, 1, 2
SPLAT_I32, SPLAT_I64 = 0, 1
SPLAT_ACT_NONE, SPLAT_ACT_RELU, SPLAT_ACT_SILU, SPLAT_ACT_GELU = 0, 1, 2, 3

# include/splat.h: size of the fixed device array splat_bin_sort_noalloc sorts in
SPLAT_NOALLOC_SCRATCH_BYTES = 64 << 20

EXPORTS = ["splat_projected_bytes", "splat_total_tiles", "splat_sort_workspace_bytes",
           "splat_bwd_workspace_bytes", "splat_project", "splat_bin_sort", "splat_bin_sort_noalloc", "splat_render_fwd",
           "splat_render_bwd", "splat_interpolate", "splat_interpolate_bwd", "splat_lookup",
           "splat_lookup_bwd_workspace_bytes", "splat_lookup_bwd", "splat_group_norm_workspace_bytes",
           "splat_group_norm", "splat_group_norm_bwd", "splat_orthogonalize_workspace_bytes",
           "splat_orthogonalize", "splat_status_string"]


class splat_camera(C.Structure):
    _fields_ = [("kind", C.c_int32), ("width", C.c_int32), ("height", C.c_int32),
                ("R", C.c_float * 9), ("t", C.c_float * 3),
                ("fx", C.c_float), ("fy", C.c_float), ("cx", C.c_float), ("cy", C.c_float),
                ("el_min_deg", C.c_float), ("el_max_deg", C.c_float),
                ("znear", C.c_float), ("zfar", C.c_float)]


class splat_prims(C.Structure):
    _fields_ = [("kind", C.c_int32), ("n", C.c_int32), ("channels", C.c_int32),
                ("pos", C.c_void_p), ("scale", C.c_void_p), ("rot", C.c_void_p),
                ("opacity", C.c_void_p), ("depth", C.c_void_p), ("feat", C.c_void_p)]


class splat_params(C.Structure):
    _fields_ = [("alpha_min", C.c_float), ("alpha_max", C.c_float), ("T_min", C.c_float),
                ("gamma", C.c_float), ("bg_weight", C.c_float), ("tau", C.c_float),
                ("top_k", C.c_int32), ("background", C.POINTER(C.c_float)), ("top_by_depth", C.c_int32),
                ("max_shift", C.c_int32), ("serial_views", C.c_int32)]


class splat_grads(C.Structure):
    _fields_ = [("pos", C.c_void_p), ("scale", C.c_void_p), ("rot", C.c_void_p),
                ("opacity", C.c_void_p), ("feat", C.c_void_p), ("cam_R", C.c_void_p),
                ("cam_t", C.c_void_p), ("cam_K", C.c_void_p), ("accumulate", C.c_int32),
                ("normalize", C.c_int32), ("sums_cleared", C.c_int32),
                ("atomic_direct_max", C.c_int32)]


class splat_norm(C.Structure):
    _fields_ = [("dtype", C.c_int32), ("param_dtype", C.c_int32), ("act", C.c_int32), ("channels", C.c_int32),
                ("groups", C.c_int32), ("eps", C.c_float), ("images", C.c_int64), ("pixels", C.c_int64),
                ("x_image_stride", C.c_int64), ("x_pixel_stride", C.c_int64),
                ("y_image_stride", C.c_int64), ("y_pixel_stride", C.c_int64),
                ("dx_image_stride", C.c_int64), ("dx_pixel_stride", C.c_int64)]


class SplatError(RuntimeError):
    def __init__(self, fn, status):
        super().__init__(f"{fn} failed: {status_string(status)} ({status})")
        self.status = status


_L = None


def lib():
    """Load libsplat.so (raises if it has not been built)."""
    global _L
    if _L is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it first (sphere_rasterization_amd.build)")
        L = C.CDLL(LIB_PATH)
        vp, i32, i64, sz = C.c_void_p, C.c_int, C.c_int64, C.c_size_t
        cam_p = C.POINTER(splat_camera)
        L.splat_projected_bytes.restype = sz
        L.splat_projected_bytes.argtypes = [i32, i32]
        L.splat_total_tiles.restype = i64
        L.splat_total_tiles.argtypes = [cam_p, i32]
        L.splat_sort_workspace_bytes.restype = sz
        L.splat_sort_workspace_bytes.argtypes = [cam_p, i32, i32, i64]
        L.splat_bwd_workspace_bytes.restype = sz
        L.splat_bwd_workspace_bytes.argtypes = [i32, i32, i32]
        L.splat_project.restype = i32
        L.splat_project.argtypes = [cam_p, i32, C.POINTER(splat_prims), C.POINTER(splat_params), vp, vp, vp]
        L.splat_bin_sort.restype = i32
        L.splat_bin_sort.argtypes = [cam_p, i32, i32, vp, vp, i64, vp, vp, vp, vp, vp, vp, sz, vp]
        L.splat_bin_sort_noalloc.restype = i32
        L.splat_bin_sort_noalloc.argtypes = [cam_p, i32, i32, vp, vp, i64, vp, vp, vp, vp, vp, vp]
        L.splat_render_fwd.restype = i32
        L.splat_render_fwd.argtypes = [cam_p, i32, C.POINTER(splat_prims), C.POINTER(splat_params), vp, vp, vp,
                                       vp, vp, vp, vp, vp, vp, vp, sz, vp]
        L.splat_render_bwd.restype = i32
        L.splat_render_bwd.argtypes = [cam_p, i32, i32, i32, C.POINTER(splat_prims), C.POINTER(splat_params),
                                       vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, C.POINTER(splat_grads), vp, sz, vp]
        fp = C.POINTER(C.c_float)
        L.splat_interpolate.restype = i32
        L.splat_interpolate.argtypes = [fp, i32, C.c_float, i32, vp, vp, vp, vp, vp]
        L.splat_interpolate_bwd.restype = i32
        L.splat_interpolate_bwd.argtypes = [fp, i32, C.c_float, i32, vp, vp, vp, vp, vp, vp]
        f32, norm_p = C.c_float, C.POINTER(splat_norm)
        L.splat_lookup.restype = i32
        L.splat_lookup.argtypes = [vp, i32, i64, i32, i64, vp, i32, i64, f32, vp, i64, vp]
        L.splat_lookup_bwd_workspace_bytes.restype = sz
        L.splat_lookup_bwd_workspace_bytes.argtypes = [i64, i64, i32]
        L.splat_lookup_bwd.restype = i32
        L.splat_lookup_bwd.argtypes = [vp, i32, i64, vp, i32, i64, i64, i32, f32, vp, i64, i32, vp, sz, vp]
        L.splat_group_norm_workspace_bytes.restype = sz
        L.splat_group_norm_workspace_bytes.argtypes = [norm_p, i32]
        L.splat_group_norm.restype = i32
        L.splat_group_norm.argtypes = [norm_p, vp, vp, vp, vp, vp, vp, vp, sz, vp]
        L.splat_group_norm_bwd.restype = i32
        L.splat_group_norm_bwd.argtypes = [norm_p, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
        L.splat_orthogonalize_workspace_bytes.restype = sz
        L.splat_orthogonalize_workspace_bytes.argtypes = [i64, i32, i32]
        L.splat_orthogonalize.restype = i32
        L.splat_orthogonalize.argtypes = [vp, i32, i64, i32, i32, i64, i64, i32, f32, f32, f32, f32, f32, vp, i64,
                                          i64, vp, sz, vp]
        L.splat_status_string.restype = C.c_char_p
        L.splat_status_string.argtypes = [i32]
        _L = L
    return _L


def status_string(status: int) -> str:
    return lib().splat_status_string(int(status)).decode()


def _check(fn, st):
    if st != SPLAT_OK:
        raise SplatError(fn, st)
    return st


# ---- same names as the C entry points ---------------------------------------

def splat_projected_bytes(n_views, n):
    return lib().splat_projected_bytes(n_views, n)


def splat_total_tiles(cams, n_views):
    return lib().splat_total_tiles(cams, n_views)


def splat_sort_workspace_bytes(cams, n_views, n, capacity):
    return lib().splat_sort_workspace_bytes(cams, n_views, n, capacity)


def splat_bwd_workspace_bytes(n_views, n, channels):
    return lib().splat_bwd_workspace_bytes(n_views, n, channels)


def splat_project(cams, n_views, prims, params, proj, pair_counts, stream):
    return _check("splat_project", lib().splat_project(cams, n_views, C.byref(prims), C.byref(params), proj,
                                                       pair_counts, stream))


def splat_bin_sort(cams, n_views, n, proj, pair_counts, capacity, keys, vals, tile_ranges, num_pairs, overflow,
                   workspace, ws_bytes, stream):
    return _check("splat_bin_sort", lib().splat_bin_sort(cams, n_views, n, proj, pair_counts, capacity, keys, vals,
                                                         tile_ranges, num_pairs, overflow, workspace, ws_bytes,
                                                         stream))


def splat_bin_sort_noalloc(cams, n_views, n, proj, pair_counts, capacity, keys, vals, tile_ranges, num_pairs,
                           overflow, stream):
    return _check("splat_bin_sort_noalloc", lib().splat_bin_sort_noalloc(cams, n_views, n, proj, pair_counts,
                                                                         capacity, keys, vals, tile_ranges,
                                                                         num_pairs, overflow, stream))


def splat_render_fwd(cams, n_views, prims, params, proj, vals, tile_ranges, overflow, img, T_final, last, norm, topk,
                     bwd_workspace, bwd_ws_bytes, stream):
    return _check("splat_render_fwd", lib().splat_render_fwd(cams, n_views, C.byref(prims), C.byref(params), proj,
                                                             vals, tile_ranges, overflow, img, T_final, last, norm,
                                                             topk, bwd_workspace, bwd_ws_bytes, stream))


def splat_render_bwd(cams, n_views, view_begin, view_count, prims, params, proj, vals, tile_ranges, overflow, img,
                     T_final, last, norm, topk, dL_dimg, grads, workspace, ws_bytes, stream):
    return _check("splat_render_bwd", lib().splat_render_bwd(cams, n_views, view_begin, view_count, C.byref(prims),
                                                             C.byref(params), proj, vals, tile_ranges, overflow, img,
                                                             T_final, last, norm, topk, dL_dimg, C.byref(grads),
                                                             workspace, ws_bytes, stream))


def _times(key_times):
    kt = (C.c_float * len(key_times))(*[float(x) for x in key_times])
    return kt, len(key_times)


def splat_interpolate(key_times, t, n, key_pos, key_rot, pos, rot, stream):
    kt, nk = _times(key_times)
    return _check("splat_interpolate", lib().splat_interpolate(kt, nk, float(t), n, key_pos, key_rot, pos, rot,
                                                               stream))


def splat_interpolate_bwd(key_times, t, n, key_rot, d_pos, d_rot, d_key_pos, d_key_rot, stream):
    kt, nk = _times(key_times)
    return _check("splat_interpolate_bwd", lib().splat_interpolate_bwd(kt, nk, float(t), n, key_rot, d_pos, d_rot,
                                                                       d_key_pos, d_key_rot, stream))


def splat_lookup(table, dtype, rows, dim, table_stride, ids, itype, n, scale, out, out_stride, stream):
    return _check("splat_lookup", lib().splat_lookup(table, dtype, rows, dim, table_stride, ids, itype, n, scale, out,
                                                     out_stride, stream))


def splat_lookup_bwd_workspace_bytes(n, rows, dim):
    return lib().splat_lookup_bwd_workspace_bytes(n, rows, dim)


def splat_lookup_bwd(d_out, dtype, d_out_stride, ids, itype, n, rows, dim, scale, d_table, d_table_stride, accumulate,
                     workspace, ws_bytes, stream):
    return _check("splat_lookup_bwd", lib().splat_lookup_bwd(d_out, dtype, d_out_stride, ids, itype, n, rows, dim,
                                                             scale, d_table, d_table_stride, accumulate, workspace,
                                                             ws_bytes, stream))


def splat_group_norm_workspace_bytes(norm, backward):
    return lib().splat_group_norm_workspace_bytes(C.byref(norm), 1 if backward else 0)


def splat_group_norm(norm, x, weight, bias, y, mean, rstd, workspace, ws_bytes, stream):
    return _check("splat_group_norm", lib().splat_group_norm(C.byref(norm), x, weight, bias, y, mean, rstd, workspace,
                                                             ws_bytes, stream))


def splat_group_norm_bwd(norm, d_y, x, mean, rstd, weight, bias, d_x, d_weight, d_bias, workspace, ws_bytes, stream):
    return _check("splat_group_norm_bwd", lib().splat_group_norm_bwd(C.byref(norm), d_y, x, mean, rstd, weight, bias,
                                                                     d_x, d_weight, d_bias, workspace, ws_bytes,
                                                                     stream))


def splat_orthogonalize_workspace_bytes(batch, rows, cols):
    return lib().splat_orthogonalize_workspace_bytes(batch, rows, cols)


def splat_orthogonalize(g, dtype, batch, rows, cols, g_batch_stride, g_row_stride, steps, a, b, c, eps, scale, out,
                        out_batch_stride, out_row_stride, workspace, ws_bytes, stream):
    return _check("splat_orthogonalize", lib().splat_orthogonalize(g, dtype, batch, rows, cols, g_batch_stride,
                                                                   g_row_stride, steps, a, b, c, eps, scale, out,
                                                                   out_batch_stride, out_row_stride, workspace,
                                                                   ws_bytes, stream))
