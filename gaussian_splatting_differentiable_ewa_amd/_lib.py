"""Thin ctypes binding of the C ABI in ``include/gs.h`` (same names).

Argument marshalling only: tensors become device pointers, cameras become
``gs_camera`` structs, the current HIP stream is passed through. Every step of
the computation runs in the HIP library; if that library is not built, every
call raises.
"""

from __future__ import annotations

import ctypes
import os
import struct
from typing import Optional, Sequence

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libgs_hip.so")

GS_OK, GS_ERR_INVALID_ARGUMENT, GS_ERR_CAPACITY, GS_ERR_HIP, GS_ERR_UNSUPPORTED = range(5)
GS_TILE = 16
GS_MAX_VIEWS = 16
GS_REC_FLOATS = 12
GS_GRAD2D_ROWS = 9
GS_ACCUMULATE_LOSS, GS_ACCUMULATE_GRAD2D = 1, 2
ABI_VERSION = 2
(REC_U, REC_V, REC_A, REC_B, REC_C, REC_OPACITY, REC_R, REC_G, REC_BLUE,
 REC_EXT_X, REC_EXT_Y, REC_DEPTH) = range(12)

# every function the header declares, for the export check
EXPORTS = (
    "gs_abi_version", "gs_status_string", "gs_param_rows", "gs_tiles_x", "gs_tiles_y",
    "gs_sort_end_bit", "gs_preprocess_workspace_bytes", "gs_sort_workspace_bytes",
    "gs_tile_lists_workspace_bytes", "gs_rasterize_fwd_l1_workspace_bytes", "gs_rasterize_fwd_bwd_l1_workspace_bytes",
    "gs_preprocess", "gs_emit_intersections", "gs_sort_keys", "gs_tile_lists", "gs_tile_ranges", "gs_tile_masks",
    "gs_tile_masks_workspace_bytes",
    "gs_rasterize_fwd", "gs_rasterize_fwd_l1", "gs_loss_l1", "gs_rasterize_bwd", "gs_rasterize_fwd_bwd_l1",
    "gs_preprocess_bwd", "gs_adam_step", "gs_adam_step_unless", "gs_preprocess_bwd_adam",
    "gs_raster_exp", "gs_stream_copy",
    "gs_rasterize_fwd_bwd_l1_noalloc", "gs_rasterize_fwd_bwd_l1_noalloc_max_bytes",
    "gs_window_gaussians", "gs_window_gaussians_workspace_bytes", "gs_adam_step_visible",
    "gs_seen_gaussians", "gs_seen_gaussians_workspace_bytes", "gs_preprocess_bwd_compact", "gs_adam_step_compact",
    "gs_rope_axes", "gs_norm_gate_fwd", "gs_norm_gate_bwd", "gs_norm_gate_bwd_workspace_bytes",
    "gs_block_summary", "gs_block_select", "gs_block_attn_fwd", "gs_block_attn_fwd_workspace_bytes",
    "gs_block_attn_bwd", "gs_block_attn_bwd_workspace_bytes",
    "gs_layer_norm_fwd", "gs_layer_norm_bwd", "gs_layer_norm_bwd_workspace_bytes",
    "gs_gated_ff_fwd", "gs_gated_ff_kept_bytes", "gs_gated_ff_fwd_workspace_bytes", "gs_gated_ff_bwd",
    "gs_gated_ff_bwd_workspace_bytes",
    "gs_quantise_fp4", "gs_dequantise_fp4", "gs_linear_fp4", "gs_linear_fp4_workspace_bytes",
)
GS_F32, GS_F16, GS_BF16 = range(3)
GS_QUERY_GROUP, GS_KEY_BLOCK = 128, 64
GS_MAX_SELECT_TOKENS = 2097152
GS_SILU, GS_GELU = range(2)


class GsError(RuntimeError):
    pass


class GsCamera(ctypes.Structure):
    _fields_ = [
        ("width", ctypes.c_int32), ("height", ctypes.c_int32),
        ("fx", ctypes.c_float), ("fy", ctypes.c_float),
        ("cx", ctypes.c_float), ("cy", ctypes.c_float),
        ("R", ctypes.c_float * 9), ("t", ctypes.c_float * 3),
        ("near_plane", ctypes.c_float), ("far_plane", ctypes.c_float),
    ]


class GsTokens(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("stride_b", ctypes.c_int64), ("stride_t", ctypes.c_int64),
                ("stride_h", ctypes.c_int64)]


class GsMatrix(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("stride", ctypes.c_int64)]


_P = ctypes.c_void_p
_I32, _I64, _U64 = ctypes.c_int32, ctypes.c_int64, ctypes.c_uint64
_F32, _F64, _SZ = ctypes.c_float, ctypes.c_double, ctypes.c_size_t
_LIB = None


def lib():
    """Load the HIP library (raises when it is not built)."""
    global _LIB
    if _LIB is None:
        if not os.path.exists(LIB_PATH):
            raise GsError(f"HIP library {LIB_PATH} is not built (run __graft_entry__.build())")
        L = ctypes.CDLL(LIB_PATH)
        sig = {
            "gs_abi_version": ([], ctypes.c_int),
            "gs_status_string": ([ctypes.c_int], ctypes.c_char_p),
            "gs_param_rows": ([_I32], ctypes.c_int),
            "gs_tiles_x": ([_I32], _I32),
            "gs_tiles_y": ([_I32], _I32),
            "gs_sort_end_bit": ([_I32, _I64], _I32),
            "gs_preprocess_workspace_bytes": ([_I64, _I32], _SZ),
            "gs_sort_workspace_bytes": ([_U64], _SZ),
            "gs_tile_lists_workspace_bytes": ([_I64, _I32, _I32, _I32, _U64], _SZ),
            "gs_rasterize_fwd_l1_workspace_bytes": ([_I32, _I32, _I32], _SZ),
            "gs_rasterize_fwd_bwd_l1_workspace_bytes": ([_I32, _I32, _I32], _SZ),
            "gs_preprocess": ([_P, _I64, _I32, _P, _I32, _P, _P, _P, _P, _P, _P, _P, _SZ, _P], ctypes.c_int),
            "gs_emit_intersections": ([_P, _P, _P, _I64, _I32, _I32, _I32, _P, _P, _U64, _P, _P], ctypes.c_int),
            "gs_sort_keys": ([_P, _P, _P, _P, _U64, _I32, _P, _SZ, _P, _P], ctypes.c_int),
            "gs_tile_ranges": ([_P, _U64, _I64, _P, _P], ctypes.c_int),
            "gs_tile_lists": ([_P, _P, _P, _P, _P, _I64, _I64, _I32, _I32, _I32, _I32, _I32, _P, _P, _U64, _P, _P, _P,
                               _P, _SZ, _P], ctypes.c_int),
            "gs_window_gaussians_workspace_bytes": ([_I64, _I32], _SZ),
            "gs_window_gaussians": ([_P, _I64, _I32, _I32, _I32, _I32, _P, _P, _P, _SZ, _P], ctypes.c_int),
            "gs_tile_masks_workspace_bytes": ([_U64], _SZ),
            "gs_tile_masks": ([_P, _I64, _P, _P, _U64, _P, _I32, _P, _P, _SZ, _P], ctypes.c_int),
            "gs_rasterize_fwd": ([_P, _I64, _P, _P, _P, _U64, _P, _I32, _I32, _I32, _P, _P, _P, _P, _P],
                                 ctypes.c_int),
            "gs_rasterize_fwd_l1": ([_P, _I64, _P, _P, _P, _U64, _P, _I32, _I32, _I32, _P, _P, _F32, _P, _P, _P, _P,
                                     _P, _I32, _P, _SZ, _P], ctypes.c_int),
            "gs_loss_l1": ([_P, _P, _I64, _F32, _P, _P, _I32, _P], ctypes.c_int),
            "gs_rasterize_fwd_bwd_l1": ([_P, _I64, _P, _P, _P, _U64, _P, _I32, _I32, _I32, _P, _P, _F32, _P, _P,
                                         _P, _P, _P, _P, _I32, _P, _SZ, _P], ctypes.c_int),
            "gs_rasterize_bwd": ([_P, _I64, _P, _P, _P, _U64, _P, _I32, _I32, _I32, _P, _P, _P, _P, _P, _I32, _P],
                                 ctypes.c_int),
            "gs_preprocess_bwd": ([_P, _I64, _I32, _P, _I32, _P, _P, _P, _P, _P], ctypes.c_int),
            "gs_adam_step_visible": ([_P, _P, _P, _P, _I64, _I32, _P, _P, _F64, _F64, _F64, _F64, _I64, _P, _P],
                                     ctypes.c_int),
            "gs_seen_gaussians_workspace_bytes": ([_I64], _SZ),
            "gs_seen_gaussians": ([_P, _I64, _I32, _P, _P, _P, _SZ, _P], ctypes.c_int),
            "gs_preprocess_bwd_compact": ([_P, _I64, _I32, _P, _I32, _P, _P, _P, _P, _I64, _P, _P, _P], ctypes.c_int),
            "gs_adam_step_compact": ([_P, _P, _I64, _P, _P, _P, _P, _I64, _I32, _P, _I32, _P, _F64, _F64, _F64, _F64,
                                      _I64, _P, _P], ctypes.c_int),
            "gs_adam_step": ([_P, _P, _P, _P, _I64, _F64, _F64, _F64, _F64, _I64, _P], ctypes.c_int),
            "gs_adam_step_unless": ([_P, _P, _P, _P, _I64, _F64, _F64, _F64, _F64, _I64, _P, _P], ctypes.c_int),
            "gs_preprocess_bwd_adam": ([_P, _I64, _I32, _P, _I32, _P, _P, _P, _P, _F64, _F64, _F64, _F64, _I64, _P,
                                        _P, _P, _P], ctypes.c_int),
            "gs_rasterize_fwd_bwd_l1_noalloc": ([_P, _I64, _P, _P, _P, _U64, _P, _I32, _I32, _I32, _P, _P, _F32, _P,
                                                 _P, _P, _P, _P, _P, _I32, _P], ctypes.c_int),
            "gs_rasterize_fwd_bwd_l1_noalloc_max_bytes": ([], _SZ),
            "gs_raster_exp": ([_P, _P, _I64, _P], ctypes.c_int),
            "gs_stream_copy": ([_P, _P, _U64, _P], ctypes.c_int),
            "gs_rope_axes": ([_P, _P, _P, _P, _I64, _I64, _I32, _I32, _I32, _I32, _P, _I64, _P, _P, _I32, _I32, _P],
                             ctypes.c_int),
            "gs_norm_gate_fwd": ([_P, _P, _P, _P, _P, _P, _P, _P, _I64, _I32, _I64, _F32, _F32, _I32, _P], ctypes.c_int),
            "gs_norm_gate_bwd_workspace_bytes": ([_I64, _I32, _I64], _SZ),
            "gs_norm_gate_bwd": ([_P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _I64, _I32, _I64, _F32, _I32, _P,
                                  _SZ, _P], ctypes.c_int),
            "gs_block_summary": ([_P, _I64, _I64, _I32, _I32, _I32, _P, _I64, _I64, _P, _P, _P], ctypes.c_int),
            "gs_block_select": ([_P, _P, _P, _I64, _I64, _I64, _I32, _I32, _I32, _I32, _P, _I32, _I32, _P, _P],
                                ctypes.c_int),
            "gs_block_attn_fwd_workspace_bytes": ([_I64, _I64, _I32, _I32, _I32], _SZ),
            "gs_block_attn_fwd": ([_P, _P, _P, _P, _I64, _I64, _I64, _I32, _I32, _I32, _I32, _P, _I32, _I32, _F32, _P,
                                   _P, _P, _SZ, _P], ctypes.c_int),
            "gs_block_attn_bwd_workspace_bytes": ([_I64, _I64, _I64, _I32, _I32, _I32], _SZ),
            "gs_block_attn_bwd": ([_P, _P, _P, _P, _P, _P, _P, _I64, _I64, _I64, _I32, _I32, _I32, _I32, _P, _I32, _I32,
                                   _F32, _P, _P, _P, _P, _SZ, _P], ctypes.c_int),
            "gs_layer_norm_fwd": ([_P, _P, _P, _P, _P, _I64, _I32, _F32, _I32, _P], ctypes.c_int),
            "gs_layer_norm_bwd_workspace_bytes": ([_I64, _I32], _SZ),
            "gs_layer_norm_bwd": ([_P, _P, _P, _P, _P, _P, _P, _I64, _I32, _I32, _P, _SZ, _P], ctypes.c_int),
            "gs_gated_ff_kept_bytes": ([_I64, _I32, _I32], _SZ),
            "gs_gated_ff_fwd_workspace_bytes": ([_I64, _I32, _I32, _I32], _SZ),
            "gs_gated_ff_fwd": ([_P, _P, _P, _P, _I64, _I32, _I32, _I32, _I32, _I32, _P, _P, _P, _P, _SZ, _P],
                                ctypes.c_int),
            "gs_gated_ff_bwd_workspace_bytes": ([_I64, _I32, _I32, _I32], _SZ),
            "gs_quantise_fp4": ([_P, _I64, _I32, _I32, _P, _P, _P], ctypes.c_int),
            "gs_dequantise_fp4": ([_P, _P, _I64, _I32, _I32, _P, _P], ctypes.c_int),
            "gs_linear_fp4_workspace_bytes": ([_I64, _I32, _I32], _SZ),
            "gs_linear_fp4": ([_P, _P, _P, _I64, _I32, _I32, _I32, _P, _P, _SZ, _P], ctypes.c_int),
            "gs_gated_ff_bwd": ([_P, _P, _P, _P, _P, _P, _P, _I64, _I32, _I32, _I32, _I32, _I32, _P, _P, _P, _P, _P, _SZ,
                                 _P], ctypes.c_int),
        }
        for name, (args, res) in sig.items():
            f = getattr(L, name)
            f.argtypes = args
            f.restype = res
        _LIB = L
    return _LIB


def status_string(status: int) -> str:
    return lib().gs_status_string(status).decode()


def _check(status: int, name: str):
    if status != GS_OK:
        raise GsError(f"{name} failed: {status_string(status)} ({status})")


def _ptr(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _stream(stream=None):
    import torch
    s = torch.cuda.current_stream() if stream is None else stream
    return s.cuda_stream


def cameras(cams: Sequence):
    arr = (GsCamera * len(cams))()
    for k, c in enumerate(cams):
        o = arr[k]
        o.width, o.height = int(c.width), int(c.height)
        o.fx, o.fy, o.cx, o.cy = c.fx, c.fy, c.cx, c.cy
        for i in range(9):
            o.R[i] = c.R[i]
        for i in range(3):
            o.t[i] = c.t[i]
        o.near_plane, o.far_plane = c.near, c.far
    return arr


# ---- queries (host only) ----------------------------------------------------
def abi_version() -> int:
    return lib().gs_abi_version()


def param_rows(sh_degree: int) -> int:
    return lib().gs_param_rows(sh_degree)


def sort_end_bit(n_views: int, tiles_per_view: int) -> int:
    return lib().gs_sort_end_bit(n_views, tiles_per_view)


def preprocess_workspace_bytes(n: int, n_views: int) -> int:
    return lib().gs_preprocess_workspace_bytes(n, n_views)


def sort_workspace_bytes(n_keys: int) -> int:
    return lib().gs_sort_workspace_bytes(n_keys)


def rasterize_fwd_l1_workspace_bytes(n_views: int, width: int, height: int) -> int:
    return lib().gs_rasterize_fwd_l1_workspace_bytes(n_views, width, height)


def rasterize_fwd_bwd_l1_workspace_bytes(n_views: int, width: int, height: int) -> int:
    return lib().gs_rasterize_fwd_bwd_l1_workspace_bytes(n_views, width, height)


def tile_lists_workspace_bytes(n: int, n_views: int, width: int, height: int, capacity: int) -> int:
    return lib().gs_tile_lists_workspace_bytes(n, n_views, width, height, capacity)


# ---- the step ----------------------------------------------------------------
def gs_preprocess(params, n, sh_degree, cams, rec, rect, offsets, total, ws, stream=None, depth=None, grad2d=None):
    """depth (optional): the compact depth copy; grad2d (optional): 2D-gradient
    records zeroed for every visible (view, Gaussian)."""
    cc = cameras(cams)
    _check(lib().gs_preprocess(_ptr(params), n, sh_degree, cc, len(cams), _ptr(rec), _ptr(rect), _ptr(depth),
                               _ptr(grad2d), _ptr(offsets), _ptr(total), _ptr(ws), ws.numel() * ws.element_size(),
                               _stream(stream)), "gs_preprocess")


def gs_emit_intersections(rec, rect, offsets, n, n_views, width, height, keys, vals, capacity,
                          overflow, stream=None):
    _check(lib().gs_emit_intersections(_ptr(rec), _ptr(rect), _ptr(offsets), n, n_views, width, height,
                                       _ptr(keys), _ptr(vals), capacity, _ptr(overflow),
                                       _stream(stream)), "gs_emit_intersections")


def tiles_y(height: int) -> int:
    return int(lib().gs_tiles_y(height))


def _window(height, rows):
    return tiles_y(height) if rows is None else rows


def gs_tile_lists(rec, rect, n, n_views, width, height, vals, capacity, ranges, overflow, ws, masks=None,
                  row0=0, rows=None, stream=None, depth=None, sticky=None, gauss=None, gauss_off=None, set_max=0):
    """masks (optional): the entries' sub-block masks, as gs_tile_masks;
    row0, rows: the window of tile rows (the whole image by default);
    depth (optional): gs_preprocess's compact depths; sticky (optional): a
    device flag set with the overflow and never cleared; gauss, gauss_off
    (optional): gs_window_gaussians' per-view sets to bin; set_max: the
    largest set expected (sizes the binning grid; 0 for all n)."""
    _check(lib().gs_tile_lists(_ptr(rec), _ptr(rect), _ptr(depth), _ptr(gauss), _ptr(gauss_off), set_max, n,
                               n_views, width,
                               height, row0, _window(height, rows),
                               _ptr(vals), _ptr(masks), capacity,
                               _ptr(ranges), _ptr(overflow), _ptr(sticky), _ptr(ws), ws.numel() * ws.element_size(),
                               _stream(stream)), "gs_tile_lists")


def window_gaussians_workspace_bytes(n: int, n_views: int) -> int:
    return lib().gs_window_gaussians_workspace_bytes(n, n_views)


def gs_window_gaussians(rect, n, n_views, height, row0, rows, gauss, gauss_off, ws, stream=None):
    _check(lib().gs_window_gaussians(_ptr(rect), n, n_views, height, row0, rows, _ptr(gauss), _ptr(gauss_off),
                                     _ptr(ws), ws.numel() * ws.element_size(), _stream(stream)), "gs_window_gaussians")


def gs_sort_keys(keys, vals, keys_alt, vals_alt, n_keys, end_bit, ws, stream=None) -> bool:
    """Returns True when the sorted data ended in the alt pair."""
    alt = ctypes.c_int32(0)
    _check(lib().gs_sort_keys(_ptr(keys), _ptr(vals), _ptr(keys_alt), _ptr(vals_alt), n_keys, end_bit,
                              _ptr(ws), ws.numel() * ws.element_size(), ctypes.byref(alt),
                              _stream(stream)), "gs_sort_keys")
    return bool(alt.value)


def gs_tile_ranges(keys, n_keys, n_tiles_total, ranges, stream=None):
    _check(lib().gs_tile_ranges(_ptr(keys), n_keys, n_tiles_total, _ptr(ranges), _stream(stream)),
           "gs_tile_ranges")


def tile_masks_workspace_bytes(capacity: int) -> int:
    return lib().gs_tile_masks_workspace_bytes(capacity)


def gs_tile_masks(rec, n, ranges, vals, capacity, cams, masks, ws, stream=None):
    _check(lib().gs_tile_masks(_ptr(rec), n, _ptr(ranges), _ptr(vals), capacity, cameras(cams), len(cams),
                               _ptr(masks), _ptr(ws), ws.numel() * ws.element_size(), _stream(stream)),
           "gs_tile_masks")


def _capacity(vals, masks, capacity):
    """List slots the raster calls may read: the given capacity, else the
    smaller of the two list buffers."""
    if capacity is not None:
        return int(capacity)
    return min(vals.numel(), masks.numel()) if vals is not None and masks is not None else 0


def gs_rasterize_fwd(rec, n, ranges, vals, masks, cams, bg, image, T_final, n_contrib, row0=0, rows=None, stream=None,
                     capacity=None):
    bgv = (ctypes.c_float * 3)(*bg)
    _check(lib().gs_rasterize_fwd(_ptr(rec), n, _ptr(ranges), _ptr(vals), _ptr(masks), _capacity(vals, masks, capacity),
                                  cameras(cams), len(cams), row0,
                                  _window(cams[0].height, rows), bgv,
                                  _ptr(image), _ptr(T_final), _ptr(n_contrib), _stream(stream)),
           "gs_rasterize_fwd")


def gs_rasterize_fwd_l1(rec, n, ranges, vals, masks, cams, bg, target, scale, image, T_final, n_contrib, dL_dimage, loss,
                        ws, accumulate=False, row0=0, rows=None, stream=None, capacity=None):
    """image may be None (not written)."""
    bgv = (ctypes.c_float * 3)(*bg)
    _check(lib().gs_rasterize_fwd_l1(_ptr(rec), n, _ptr(ranges), _ptr(vals), _ptr(masks),
                                     _capacity(vals, masks, capacity), cameras(cams), len(cams),
                                     row0, _window(cams[0].height, rows), bgv,
                                     _ptr(target), scale, _ptr(image), _ptr(T_final), _ptr(n_contrib),
                                     _ptr(dL_dimage), _ptr(loss), int(bool(accumulate)), _ptr(ws),
                                     ws.numel() * ws.element_size(), _stream(stream)), "gs_rasterize_fwd_l1")


def gs_loss_l1(image, target, count, scale, dL_dimage, loss, accumulate=False, stream=None):
    _check(lib().gs_loss_l1(_ptr(image), _ptr(target), count, scale, _ptr(dL_dimage), _ptr(loss),
                            int(bool(accumulate)), _stream(stream)), "gs_loss_l1")


def gs_rasterize_bwd(rec, n, ranges, vals, masks, cams, bg, T_final, n_contrib, dL_dimage, grad2d,
                     accumulate=False, row0=0, rows=None, stream=None, capacity=None):
    bgv = (ctypes.c_float * 3)(*bg)
    _check(lib().gs_rasterize_bwd(_ptr(rec), n, _ptr(ranges), _ptr(vals), _ptr(masks), _capacity(vals, masks, capacity),
                                  cameras(cams), len(cams), row0,
                                  _window(cams[0].height, rows), bgv,
                                  _ptr(T_final), _ptr(n_contrib), _ptr(dL_dimage), _ptr(grad2d),
                                  int(bool(accumulate)), _stream(stream)), "gs_rasterize_bwd")


def gs_rasterize_fwd_bwd_l1(rec, n, ranges, vals, masks, cams, bg, target, scale, loss, grad2d, ws, image=None,
                            T_final=None, n_contrib=None, dL_dimage=None, accumulate=False, row0=0, rows=None,
                            stream=None, capacity=None, accumulate_grad2d=None):
    """image, T_final, n_contrib and dL_dimage are optional outputs.
    `accumulate` adds to the loss and the 2D gradients; `accumulate_grad2d`,
    when given, decides for the 2D gradients alone (e.g. records zeroed by
    gs_preprocess, with the loss overwritten)."""
    bgv = (ctypes.c_float * 3)(*bg)
    acc_g = accumulate if accumulate_grad2d is None else accumulate_grad2d
    flags = (GS_ACCUMULATE_LOSS if accumulate else 0) | (GS_ACCUMULATE_GRAD2D if acc_g else 0)
    _check(lib().gs_rasterize_fwd_bwd_l1(_ptr(rec), n, _ptr(ranges), _ptr(vals), _ptr(masks),
                                         _capacity(vals, masks, capacity), cameras(cams),
                                         len(cams), row0, _window(cams[0].height, rows), bgv, _ptr(target), scale,
                                         _ptr(image), _ptr(T_final), _ptr(n_contrib), _ptr(dL_dimage), _ptr(loss),
                                         _ptr(grad2d), flags, _ptr(ws),
                                         ws.numel() * ws.element_size(), _stream(stream)), "gs_rasterize_fwd_bwd_l1")


def gs_rasterize_fwd_bwd_l1_noalloc(rec, n, ranges, vals, masks, cams, bg, target, scale, loss, grad2d, image=None,
                                    T_final=None, n_contrib=None, dL_dimage=None, accumulate=False, row0=0, rows=None,
                                    stream=None, capacity=None, accumulate_grad2d=None):
    """gs_rasterize_fwd_bwd_l1 with the library's fixed per-device workspace
    (no workspace argument, nothing allocated)."""
    bgv = (ctypes.c_float * 3)(*bg)
    acc_g = accumulate if accumulate_grad2d is None else accumulate_grad2d
    flags = (GS_ACCUMULATE_LOSS if accumulate else 0) | (GS_ACCUMULATE_GRAD2D if acc_g else 0)
    _check(lib().gs_rasterize_fwd_bwd_l1_noalloc(_ptr(rec), n, _ptr(ranges), _ptr(vals), _ptr(masks),
                                                 _capacity(vals, masks, capacity), cameras(cams), len(cams), row0,
                                                 _window(cams[0].height, rows), bgv, _ptr(target), scale, _ptr(image),
                                                 _ptr(T_final), _ptr(n_contrib), _ptr(dL_dimage), _ptr(loss),
                                                 _ptr(grad2d), flags, _stream(stream)),
           "gs_rasterize_fwd_bwd_l1_noalloc")


def gs_preprocess_bwd(params, n, sh_degree, cams, rect, grad2d, grad_params, stream=None, visible=None):
    """visible (optional, uint8 [n]): sparse output, rows written only for
    Gaussians visible in some view (see the header)."""
    _check(lib().gs_preprocess_bwd(_ptr(params), n, sh_degree, cameras(cams), len(cams), _ptr(rect),
                                   _ptr(grad2d), _ptr(grad_params), _ptr(visible), _stream(stream)),
           "gs_preprocess_bwd")


def gs_adam_step_visible(params, grad, m, v, n, rows, visible, lr, beta1, beta2, eps, step, state=None, skip=None,
                         stream=None):
    _check(lib().gs_adam_step_visible(_ptr(params), _ptr(grad), _ptr(m), _ptr(v), n, rows, _ptr(visible),
                                      _ptr(state), lr, beta1, beta2, eps, step, _ptr(skip), _stream(stream)),
           "gs_adam_step_visible")


def seen_gaussians_workspace_bytes(n: int) -> int:
    return lib().gs_seen_gaussians_workspace_bytes(n)


def gs_seen_gaussians(rect, n, n_views, gauss, count, ws, stream=None):
    _check(lib().gs_seen_gaussians(_ptr(rect), n, n_views, _ptr(gauss), _ptr(count), _ptr(ws),
                                   ws.numel() * ws.element_size(), _stream(stream)), "gs_seen_gaussians")


def gs_preprocess_bwd_compact(params, n, sh_degree, cams, rect, grad2d, gauss, count, stride, grad_compact, overflow,
                              stream=None):
    _check(lib().gs_preprocess_bwd_compact(_ptr(params), n, sh_degree, cameras(cams), len(cams), _ptr(rect),
                                           _ptr(grad2d), _ptr(gauss), _ptr(count), stride, _ptr(grad_compact),
                                           _ptr(overflow), _stream(stream)), "gs_preprocess_bwd_compact")


def gs_adam_step_compact(params, grad_compact, stride, gauss, count, m, v, n, rows, rect, n_views, lr, beta1, beta2,
                         eps, step, state=None, skip=None, stream=None):
    _check(lib().gs_adam_step_compact(_ptr(params), _ptr(grad_compact), stride, _ptr(gauss), _ptr(count), _ptr(m),
                                      _ptr(v), n, rows, _ptr(rect), n_views, _ptr(state), lr, beta1, beta2, eps, step,
                                      _ptr(skip), _stream(stream)), "gs_adam_step_compact")


def gs_adam_step(params, grad, m, v, count, lr, beta1, beta2, eps, step, stream=None):
    _check(lib().gs_adam_step(_ptr(params), _ptr(grad), _ptr(m), _ptr(v), count, lr, beta1, beta2, eps,
                              step, _stream(stream)), "gs_adam_step")


def gs_preprocess_bwd_adam(params, n, sh_degree, cams, rect, grad2d, m, v, lr, beta1, beta2, eps, step, skip=None,
                           grad_params=None, state=None, stream=None):
    """state (optional): uint8 [n], 0 where the Gaussian's moments are zero
    (see the header); never-seen Gaussians are then skipped."""
    _check(lib().gs_preprocess_bwd_adam(_ptr(params), n, sh_degree, cameras(cams), len(cams), _ptr(rect), _ptr(grad2d),
                                        _ptr(m), _ptr(v), lr, beta1, beta2, eps, step, _ptr(skip), _ptr(state),
                                        _ptr(grad_params), _stream(stream)), "gs_preprocess_bwd_adam")


def gs_adam_step_unless(params, grad, m, v, count, lr, beta1, beta2, eps, step, skip, stream=None):
    _check(lib().gs_adam_step_unless(_ptr(params), _ptr(grad), _ptr(m), _ptr(v), count, lr, beta1, beta2, eps,
                                     step, _ptr(skip), _stream(stream)), "gs_adam_step_unless")


def gs_raster_exp(x, y, stream=None):
    """y = the raster passes' exp of x (device fp32 tensors)."""
    _check(lib().gs_raster_exp(_ptr(x), _ptr(y), x.numel(), _stream(stream)), "gs_raster_exp")


def gs_stream_copy(dst, src, nbytes=None, stream=None):
    """Plain device copy of nbytes (default: all of src) from src to dst."""
    nb = src.numel() * src.element_size() if nbytes is None else int(nbytes)
    _check(lib().gs_stream_copy(_ptr(dst), _ptr(src), nb, _stream(stream)), "gs_stream_copy")


# ---- token operators -----------------------------------------------------------
# Token tensors are [batch][tokens][heads][dim] (any strides, dim contiguous).
def _current(t, stream):
    """The given stream's handle, or that of the tensor's device's current one
    (looked up once by name: torch.cuda.current_stream builds an object)."""
    global _RAW_STREAM
    if stream is not None:
        return stream.cuda_stream
    if _RAW_STREAM is None:
        import torch
        _RAW_STREAM = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
            lambda device: torch.cuda.current_stream(device).cuda_stream)
    return _RAW_STREAM(t.get_device())


class _Elsewhere:
    """The library with another device made current around each call."""

    def __init__(self, device):
        self.device = device

    def __getattr__(self, name):
        def call(*args):
            import torch
            with torch.cuda.device(self.device):
                return getattr(lib(), name)(*args)
        return call


def _at(t):
    """The library for a call on tensor t's device: a launch on a default stream
    goes to the device that is current, whatever its arguments."""
    global _DEVICE
    if _DEVICE is None:
        import torch
        _DEVICE = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
    device = t.get_device()
    return lib() if device == _DEVICE() else _Elsewhere(device)


_RAW_STREAM = _DEVICE = None
_DTYPES = {}
_Pairs = ctypes.c_int32 * 3


def dtype_of(t) -> int:
    """gs_dtype of a tensor (raises for other types)."""
    if not _DTYPES:
        import torch
        _DTYPES.update({torch.float32: GS_F32, torch.float16: GS_F16, torch.bfloat16: GS_BF16})
    try:
        return _DTYPES[t.dtype]
    except KeyError:
        raise GsError(f"unsupported element type {t.dtype}") from None


# gs_tokens as bytes: a third of the time of a ctypes structure, and small
# calls are bound by the host
_pack_tokens = struct.Struct("@Pqqq").pack


def _tok(t):
    if t is None:
        return None
    sb, st, sh, sd = t.stride()
    if sd != 1 and t.shape[3] > 1:
        raise GsError("the last dimension of a token tensor must be contiguous")
    return _pack_tokens(t.data_ptr(), sb, st, sh)


def _blk(t):
    """A summary [batch][heads][blocks](dim) as a token tensor of blocks."""
    if t.dim() == 4 and t.stride(3) != 1 and t.shape[3] > 1:
        raise GsError("the last dimension of a summary must be contiguous")
    st = t.stride()
    return _pack_tokens(t.data_ptr(), st[0], st[2], st[1])


def _ws(ws):
    return (None, 0) if ws is None else (ws.data_ptr(), ws.numel() * ws.element_size())


def gs_rope_axes(q, k, q_out, k_out, pos, freq, pairs, interleaved=False, inverse=False, stream=None):
    """pos int32 [batch or 1][tokens][3] contiguous; k and k_out may be None."""
    b, n, hq, d = q.shape
    _check(_at(q).gs_rope_axes(_tok(q), _tok(k), _tok(q_out), _tok(k_out), b, n, hq, 0 if k is None else k.shape[2], d,
                              dtype_of(q), _ptr(pos), 0 if pos.shape[0] == 1 else pos.stride(0), _ptr(freq),
                              _Pairs(*pairs), int(bool(interleaved)), int(bool(inverse)),
                              _current(q, stream)), "gs_rope_axes")


def gs_norm_gate_fwd(x, f, gate, w_post, w_pre, y, h, stats, rows_per_gate, scale=1.0, eps=1e-6, stream=None):
    """x, f, y, h [rows][channels] contiguous; f, gate, w_post, w_pre may be None."""
    rows, c = x.shape
    _check(_at(x).gs_norm_gate_fwd(_ptr(x), _ptr(f), _ptr(gate), _ptr(w_post), _ptr(w_pre), _ptr(y), _ptr(h), _ptr(stats),
                                  rows, c, rows_per_gate, scale, eps, dtype_of(x), _current(x, stream)), "gs_norm_gate_fwd")


def norm_gate_bwd_workspace_bytes(rows: int, channels: int, rows_per_gate: int) -> int:
    return lib().gs_norm_gate_bwd_workspace_bytes(rows, channels, rows_per_gate)


def gs_norm_gate_bwd(gy, gh, x, f, gate, w_post, w_pre, stats, gx, gf, ggate, gw_post, gw_pre, rows_per_gate, ws,
                     scale=1.0, stream=None):
    """gy, f, gate, w_post, w_pre and the fp32 outputs may be None."""
    rows, c = x.shape
    _check(_at(x).gs_norm_gate_bwd(_ptr(gy), _ptr(gh), _ptr(x), _ptr(f), _ptr(gate), _ptr(w_post), _ptr(w_pre),
                                  _ptr(stats), _ptr(gx), _ptr(gf), _ptr(ggate), _ptr(gw_post), _ptr(gw_pre), rows, c,
                                  rows_per_gate, scale, dtype_of(x), *_ws(ws), _current(x, stream)), "gs_norm_gate_bwd")


def gs_block_summary(k, sum8, scale, kv_len=None, block0=0, blocks=None, stream=None):
    """sum8 int8 [batch][heads][ceil(tokens / 64)][dim], scale fp32 without dim;
    any strides, dim contiguous."""
    b, n, h, d = k.shape
    every = (n + GS_KEY_BLOCK - 1) // GS_KEY_BLOCK
    _check(_at(k).gs_block_summary(_tok(k), b, n, h, d, dtype_of(k), _ptr(kv_len), block0,
                                  every - block0 if blocks is None else blocks, _blk(sum8), _blk(scale),
                                  _current(k, stream)), "gs_block_summary")


def gs_block_select(q, sum8, scale, tokens_k, heads_k, lists, kv_len=None, causal=False, stream=None):
    """lists int32 [batch][heads_q][ceil(tokens_q / 128)][top]."""
    b, n, h, d = q.shape
    _check(_at(q).gs_block_select(_tok(q), _blk(sum8), _blk(scale), b, n, tokens_k, h, heads_k, d, dtype_of(q),
                                 _ptr(kv_len), int(bool(causal)), lists.shape[3], _ptr(lists), _current(q, stream)),
           "gs_block_select")


def block_attn_fwd_workspace_bytes(batch: int, tokens_q: int, heads_q: int, dim: int, top: int) -> int:
    return lib().gs_block_attn_fwd_workspace_bytes(batch, tokens_q, heads_q, dim, top)


def gs_block_attn_fwd(q, k, v, lists, out, lse, ws=None, kv_len=None, causal=False, sm_scale=None, stream=None):
    """sm_scale: dim ** -0.5 by default."""
    b, n, h, d = q.shape
    _check(_at(q).gs_block_attn_fwd(_tok(q), _tok(k), _tok(v), _ptr(lists), b, n, k.shape[1], h, k.shape[2], d,
                                   dtype_of(q), _ptr(kv_len), int(bool(causal)), lists.shape[3],
                                   d ** -0.5 if sm_scale is None else sm_scale, _tok(out), _ptr(lse), *_ws(ws),
                                   _current(q, stream)), "gs_block_attn_fwd")


def block_attn_bwd_workspace_bytes(batch: int, tokens_q: int, tokens_k: int, heads_q: int, heads_k: int, dim: int) -> int:
    return lib().gs_block_attn_bwd_workspace_bytes(batch, tokens_q, tokens_k, heads_q, heads_k, dim)


def gs_block_attn_bwd(gout, q, k, v, out, lse, lists, gq, gk, gv, ws, kv_len=None, causal=False, sm_scale=None,
                      stream=None):
    b, n, h, d = q.shape
    _check(_at(q).gs_block_attn_bwd(_tok(gout), _tok(q), _tok(k), _tok(v), _tok(out), _ptr(lse), _ptr(lists), b, n,
                                   k.shape[1], h, k.shape[2], d, dtype_of(q), _ptr(kv_len), int(bool(causal)),
                                   lists.shape[3], d ** -0.5 if sm_scale is None else sm_scale, _tok(gq), _tok(gk),
                                   _tok(gv), *_ws(ws), _current(q, stream)), "gs_block_attn_bwd")


# Matrices are [rows][columns], any row stride, columns contiguous.
_pack_matrix = struct.Struct("@Pq").pack


def _mat(t):
    if t is None:
        return None
    (rows, columns), (sr, sc) = t.shape, t.stride()
    if sc != 1 and columns > 1:
        raise GsError("the rows of a matrix must be contiguous")
    return _pack_matrix(t.data_ptr(), sr if rows > 1 else columns)


def gs_layer_norm_fwd(x, w, b, y, stats, eps=1e-5, stream=None):
    """x any row stride, y contiguous; w and b may be None."""
    rows, c = x.shape
    _check(_at(x).gs_layer_norm_fwd(_mat(x), _ptr(w), _ptr(b), _ptr(y), _ptr(stats), rows, c, eps, dtype_of(x),
                                    _current(x, stream)), "gs_layer_norm_fwd")


def layer_norm_bwd_workspace_bytes(rows: int, channels: int) -> int:
    return lib().gs_layer_norm_bwd_workspace_bytes(rows, channels)


def gs_layer_norm_bwd(gy, x, w, stats, gx, gw, gb, ws, stream=None):
    """gy and x any row stride, gx contiguous; w, gw and gb may be None."""
    rows, c = x.shape
    _check(_at(x).gs_layer_norm_bwd(_mat(gy), _mat(x), _ptr(w), _ptr(stats), _ptr(gx), _ptr(gw), _ptr(gb), rows, c,
                                    dtype_of(x), *_ws(ws), _current(x, stream)), "gs_layer_norm_bwd")


def gated_ff_kept_bytes(rows: int, hidden: int, dtype: int) -> int:
    return lib().gs_gated_ff_kept_bytes(rows, hidden, dtype)


def gated_ff_fwd_workspace_bytes(rows: int, channels: int, hidden: int, channels_out: int) -> int:
    return lib().gs_gated_ff_fwd_workspace_bytes(rows, channels, hidden, channels_out)


def gs_gated_ff_fwd(x, w_gate, w_up, w_down, act, h, kept, y, ws=None, stream=None):
    """x, w_gate, w_up, w_down any row stride of 8 elements; kept may be None."""
    rows, c = x.shape
    _check(_at(x).gs_gated_ff_fwd(_mat(x), _mat(w_gate), _mat(w_up), _mat(w_down), rows, c, w_gate.shape[0],
                                  w_down.shape[0], act, dtype_of(x), _ptr(h), _ptr(kept), _ptr(y), *_ws(ws),
                                  _current(x, stream)), "gs_gated_ff_fwd")


def gated_ff_bwd_workspace_bytes(rows: int, channels: int, hidden: int, channels_out: int) -> int:
    return lib().gs_gated_ff_bwd_workspace_bytes(rows, channels, hidden, channels_out)


def gs_gated_ff_bwd(gy, x, w_gate, w_up, w_down, h, kept, act, gx, gw_gate, gw_up, gw_down, ws, stream=None):
    """gx, gw_gate with gw_up, and gw_down may be None; rows apart (no stride of 0)."""
    rows, c = x.shape
    _check(_at(x).gs_gated_ff_bwd(_mat(gy), _mat(x), _mat(w_gate), _mat(w_up), _mat(w_down), _ptr(h), _ptr(kept), rows, c,
                                  w_gate.shape[0], w_down.shape[0], act, dtype_of(x), _ptr(gx), _ptr(gw_gate), _ptr(gw_up),
                                  _ptr(gw_down), *_ws(ws), _current(x, stream)), "gs_gated_ff_bwd")


def gs_quantise_fp4(x, codes, scales, stream=None):
    """codes uint8 [rows][channels / 2], scales uint8 [rows][4 ceil(channels / 128)], contiguous."""
    rows, c = x.shape
    _check(_at(x).gs_quantise_fp4(_mat(x), rows, c, dtype_of(x), _ptr(codes), _ptr(scales), _current(x, stream)),
           "gs_quantise_fp4")


def gs_dequantise_fp4(codes, scales, out, stream=None):
    rows, c = out.shape
    _check(_at(out).gs_dequantise_fp4(_mat(codes), _mat(scales), rows, c, dtype_of(out), _ptr(out), _current(out, stream)),
           "gs_dequantise_fp4")


def linear_fp4_workspace_bytes(rows: int, channels: int, out: int) -> int:
    return lib().gs_linear_fp4_workspace_bytes(rows, channels, out)


def gs_linear_fp4(x, codes, scales, y, ws, stream=None):
    rows, c = x.shape
    _check(_at(x).gs_linear_fp4(_mat(x), _mat(codes), _mat(scales), rows, c, codes.shape[0], dtype_of(x), _ptr(y), *_ws(ws),
                                _current(x, stream)), "gs_linear_fp4")
