"""Thin ctypes binding of libridgefill.so (C ABI in include/ridgefill.h).

Argument marshalling only: every step of the fill, calibration and solve runs in the
HIP library.  torch tensors supply device memory and the current stream.  There is no
fallback: if the library is missing, `lib()` raises.
"""

from __future__ import annotations

import ctypes as C
import os

import numpy as np

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libridgefill.so")

RF_OK, RF_E_INVALID, RF_E_SHAPE, RF_E_WORKSPACE, RF_E_HIP, RF_E_NOT_SPD, RF_E_ROWS, \
    RF_E_UNSUPPORTED = range(8)

EXPORTED = [
    "ridgefill_partition",
    "ridgefill_fill_workspace_bytes",
    "ridgefill_fill_workspace_bytes_ex",
    "ridgefill_fill",
    "ridgefill_fill_streamed",
    "ridgefill_fill_noalloc",
    "ridgefill_value_scale_workspace_bytes",
    "ridgefill_value_scale",
    "ridgefill_quantize_map",
    "ridgefill_fold_bytes",
    "ridgefill_fold_workspace_bytes",
    "ridgefill_fold_workspace_bytes_ex",
    "ridgefill_fold_workspace_bytes_maps",
    "ridgefill_fold_maps",
    "ridgefill_select_workspace_bytes",
    "ridgefill_select_rows",
    "ridgefill_calib_state_bytes",
    "ridgefill_calib_reset",
    "ridgefill_calibrate",
    "ridgefill_calib_state_bytes_ex",
    "ridgefill_calib_reset_ex",
    "ridgefill_calibrate_ex",
    "ridgefill_solve_workspace_bytes",
    "ridgefill_solve",
    "ridgefill_solve_workspace_bytes_ex",
    "ridgefill_solve_ex",
    "ridgefill_rope",
    "ridgefill_append_rows",
    "ridgefill_tree_attention_workspace_bytes",
    "ridgefill_tree_attention",
    "ridgefill_attention_weight_workspace_bytes",
    "ridgefill_attention_weight",
    "ridgefill_evict_workspace_bytes",
    "ridgefill_evict_rows",
    "ridgefill_norm_rope",
    "ridgefill_norm_rope_grad_workspace_bytes",
    "ridgefill_norm_rope_grad",
    "ridgefill_append_cache",
    "ridgefill_read_rows",
    "ridgefill_cache_attention_workspace_bytes",
    "ridgefill_cache_attention",
    "ridgefill_read_status",
    "ridgefill_solve_info",
    "ridgefill_profile_enable",
    "ridgefill_profile_read",
    "ridgefill_profile_reset",
    "ridgefill_status_string",
    "ridgefill_last_error",
]


class RidgeFillError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"ridgefill status {status}: {msg}")
        self.status = status


RF_MAPS_INT8 = 1
RF_MAPS_STREAMED = 2
RF_MAPS_FOLDED = 4


class rf_shape(C.Structure):
    _fields_ = [("d", C.c_int32), ("n_kv_heads", C.c_int32), ("head_dim", C.c_int32),
                ("rms_eps", C.c_float), ("rope_theta", C.c_double), ("d_in", C.c_int32),
                ("reserved", C.c_int32)]


class rf_layer(C.Structure):
    _fields_ = [("A", C.c_void_p), ("b", C.c_void_p), ("norm_w", C.c_void_p),
                ("W_K", C.c_void_p), ("W_V", C.c_void_p), ("k_pages", C.c_void_p),
                ("v_pages", C.c_void_p), ("k_norm_w", C.c_void_p), ("v_scale", C.c_void_p),
                ("A_q", C.c_void_p), ("A_scale", C.c_void_p), ("folded", C.c_void_p)]


class rf_paged_kv(C.Structure):
    _fields_ = [("block_table", C.c_void_p), ("n_logical", C.c_int64),
                ("page_size", C.c_int32), ("num_pages", C.c_int32)]


class rf_paged_batch(C.Structure):
    _fields_ = [("block_tables", C.c_void_p), ("lengths", C.c_void_p), ("table_stride", C.c_int64),
                ("batch", C.c_int32), ("max_len", C.c_int32), ("page_size", C.c_int32),
                ("num_pages", C.c_int32), ("n_kv_heads", C.c_int32), ("head_dim", C.c_int32)]


class rf_rope(C.Structure):
    _fields_ = [("theta", C.c_double), ("rotary_dim", C.c_int32), ("layout", C.c_int32),
                ("scaling", C.c_int32), ("orig_len", C.c_int32), ("factor", C.c_double),
                ("low", C.c_double), ("high", C.c_double), ("mscale", C.c_double)]


class rf_head_norm(C.Structure):
    _fields_ = [("q_w", C.c_void_p), ("k_w", C.c_void_p), ("eps", C.c_float), ("reserved", C.c_int32)]


class rf_cache(C.Structure):
    _fields_ = [("type", C.c_int32), ("reserved", C.c_int32), ("k_pages", C.c_void_p),
                ("v_pages", C.c_void_p), ("k_scales", C.c_void_p), ("v_scales", C.c_void_p)]


class rf_prefix(C.Structure):
    _fields_ = [("block_tables", C.c_void_p), ("lengths", C.c_void_p), ("group_start", C.c_void_p),
                ("table_stride", C.c_int64), ("groups", C.c_int32), ("max_len", C.c_int32)]


RF_ROPE_HALF, RF_ROPE_INTERLEAVED = range(2)
RF_ROPE_PLAIN, RF_ROPE_LINEAR, RF_ROPE_NTK, RF_ROPE_BANDS, RF_ROPE_YARN = range(5)
RF_TYPE_BF16, RF_TYPE_F32 = range(2)
RF_CACHE_BF16, RF_CACHE_FP8, RF_CACHE_INT8 = range(3)

_lib = None


def lib() -> C.CDLL:
    """Load the HIP library (once).  Raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                           "`python -m ridge_map_kv_amd.build` (there is no CPU fallback)")
    L = C.CDLL(LIB_PATH)
    vp, i32, i64, sz = C.c_void_p, C.c_int32, C.c_int64, C.c_size_t
    st = C.c_int
    sig = {
        "ridgefill_partition": (st, [i64, i64, vp, vp, C.POINTER(i64)]),
        "ridgefill_fill_workspace_bytes": (sz, [C.POINTER(rf_shape), i64, i32]),
        "ridgefill_fill_workspace_bytes_ex": (sz, [C.POINTER(rf_shape), i64, i32, i32]),
        "ridgefill_fill": (st, [C.POINTER(rf_shape), vp, i64, i64, i64, vp, i64,
                                C.POINTER(rf_layer), i32, C.POINTER(rf_paged_kv), vp, sz, vp]),
        "ridgefill_fill_streamed": (st, [C.POINTER(rf_shape), vp, i64, i64, i64, vp, i64,
                                         C.POINTER(rf_layer), i32, C.POINTER(rf_paged_kv), vp,
                                         sz, vp, vp]),
        "ridgefill_fill_noalloc": (st, [C.POINTER(rf_shape), vp, i64, i64, i64, vp, i64,
                                        C.POINTER(rf_layer), i32, C.POINTER(rf_paged_kv), vp, vp]),
        "ridgefill_value_scale_workspace_bytes": (sz, [C.POINTER(rf_shape), i64, i32, i32]),
        "ridgefill_value_scale": (st, [C.POINTER(rf_shape), vp, i64, C.POINTER(vp), i64,
                                       C.POINTER(rf_layer), i32, vp, vp, sz, vp]),
        "ridgefill_quantize_map": (st, [vp, i64, i64, vp, vp, vp]),
        "ridgefill_fold_bytes": (sz, [C.POINTER(rf_shape)]),
        "ridgefill_fold_workspace_bytes": (sz, [C.POINTER(rf_shape)]),
        "ridgefill_fold_workspace_bytes_ex": (sz, [C.POINTER(rf_shape), i32]),
        "ridgefill_fold_workspace_bytes_maps": (sz, [C.POINTER(rf_shape), i32, C.c_uint32]),
        "ridgefill_fold_maps": (st, [C.POINTER(rf_shape), C.POINTER(rf_layer), i32,
                                     C.POINTER(vp), vp, sz, vp]),
        "ridgefill_select_workspace_bytes": (sz, [i64]),
        "ridgefill_select_rows": (st, [vp, i64, i64, vp, vp, vp, sz, vp]),
        "ridgefill_calib_state_bytes": (sz, [i32, i32]),
        "ridgefill_calib_reset": (st, [vp, sz, i32, i32, vp]),
        "ridgefill_calibrate": (st, [vp, sz, i32, i32, vp, C.POINTER(vp), i64, vp]),
        "ridgefill_solve_workspace_bytes": (sz, [i32, i32]),
        "ridgefill_solve": (st, [vp, sz, i32, i32, C.c_double, vp, vp, vp, vp, sz, vp]),
        "ridgefill_calib_state_bytes_ex": (sz, [i32, i32, i32]),
        "ridgefill_calib_reset_ex": (st, [vp, sz, i32, i32, i32, vp]),
        "ridgefill_calibrate_ex": (st, [vp, sz, i32, i32, i32, vp, C.POINTER(vp), i64, vp]),
        "ridgefill_solve_workspace_bytes_ex": (sz, [i32, i32, i32]),
        "ridgefill_solve_ex": (st, [vp, sz, i32, i32, i32, C.c_double, vp, vp, vp, vp, sz, vp]),
        "ridgefill_rope": (st, [vp, vp, i32, i64, i32, i32, i64, vp, vp, i64, i32, vp]),
        "ridgefill_append_rows": (st, [vp, vp, vp, i32, i64, vp, i64, vp, i64, vp, i64, i64, vp, vp,
                                       vp, vp, vp, vp, vp]),
        "ridgefill_tree_attention_workspace_bytes": (sz, [vp, i32, i32]),
        "ridgefill_tree_attention": (st, [vp, vp, vp, vp, i32, i64, vp, i64, i32, vp, C.c_float, vp,
                                          i64, vp, vp, sz, vp]),
        "ridgefill_attention_weight_workspace_bytes": (sz, [vp, i32, i32]),
        "ridgefill_attention_weight": (st, [vp, vp, vp, i32, i64, vp, i64, i32, vp, C.c_float, vp,
                                            C.c_float, vp, vp, i64, vp, sz, vp]),
        "ridgefill_evict_workspace_bytes": (sz, [vp, i32]),
        "ridgefill_evict_rows": (st, [vp, C.POINTER(rf_layer), i32, vp, vp, i64, i32, i32, i32, vp,
                                      vp, vp, vp, sz, vp]),
        "ridgefill_norm_rope": (st, [vp, vp, i32, i64, i32, vp, vp, i32, i64, vp, i64, vp, i32, i64,
                                     vp, i64, vp]),
        "ridgefill_norm_rope_grad_workspace_bytes": (sz, [i64, i32, i32, i32]),
        "ridgefill_norm_rope_grad": (st, [vp, vp, i32, i64, i32, vp, vp, i32, i64, vp, i64, vp, i64,
                                          vp, vp, i32, i64, vp, i64, vp, i64, vp, vp, sz, vp]),
        "ridgefill_append_cache": (st, [vp, vp, vp, vp, vp, i32, i64, vp, i64, vp, i64, vp, i64, i64,
                                        vp, vp, vp, vp, vp]),
        "ridgefill_read_rows": (st, [vp, vp, i64, vp, vp, i32, vp, i64, vp, i64, vp, vp]),
        "ridgefill_cache_attention_workspace_bytes": (sz, [vp, vp, i32, i32, i64]),
        "ridgefill_cache_attention": (st, [vp, vp, vp, vp, i32, i64, vp, i64, i32, vp, C.c_float, vp, i64,
                                           vp, vp, sz, vp]),
        "ridgefill_read_status": (st, [vp, vp]),
        "ridgefill_solve_info": (st, [vp, C.POINTER(C.c_double), C.POINTER(i32), vp]),
        "ridgefill_profile_enable": (st, [i32]),
        "ridgefill_profile_read": (st, [i32, C.POINTER(i64), C.POINTER(C.c_double)]),
        "ridgefill_profile_reset": (st, []),
        "ridgefill_status_string": (C.c_char_p, [st]),
        "ridgefill_last_error": (C.c_char_p, []),
    }
    for name, (res, args) in sig.items():
        f = getattr(L, name)
        f.restype = res
        f.argtypes = args
    _lib = L
    return L


def _check(status: int) -> None:
    if status != RF_OK:
        msg = lib().ridgefill_last_error().decode() or lib().ridgefill_status_string(status).decode()
        raise RidgeFillError(status, msg)


def _ptr(t) -> int | None:
    if t is None:
        return None
    return t.data_ptr()


def _stream(stream) -> int | None:
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream


def make_shape(d: int, n_kv_heads: int, head_dim: int, rms_eps: float = 1e-5,
               rope_theta: float = 500000.0, d_in: int = 0) -> rf_shape:
    return rf_shape(d, n_kv_heads, head_dim, rms_eps, rope_theta, d_in, 0)


# ------------------------------------------------------------------------------ partition

def ridgefill_partition(N: int, T: int, exact_mask: np.ndarray | None) -> np.ndarray:
    """Host row partition; returns the filled rows (int32, ascending)."""
    P = max(int(N) - int(T), 0)
    out = np.zeros(max(P, 1), dtype=np.int32)
    n = C.c_int64(0)
    m = None
    if exact_mask is not None:
        exact_mask = np.ascontiguousarray(exact_mask, dtype=np.uint8)
        if exact_mask.size < P:
            raise ValueError("exact_mask shorter than the prefix")
        m = exact_mask.ctypes.data
    _check(lib().ridgefill_partition(int(N), int(T), m, out.ctypes.data, C.byref(n)))
    return out[: n.value].copy()


# ------------------------------------------------------------------------------ int8 maps

def ridgefill_quantize_map(A, A_q, A_scale, stream=None) -> None:
    """fp32 [rows][cols] map -> int8 codes A_q (same shape) and fp32 row scales A_scale."""
    _check(lib().ridgefill_quantize_map(_ptr(A), int(A.shape[0]), int(A.shape[1]), _ptr(A_q),
                                        _ptr(A_scale), _stream(stream)))


# ------------------------------------------------------------------------------ selection

def ridgefill_select_workspace_bytes(P: int) -> int:
    return int(lib().ridgefill_select_workspace_bytes(int(P)))


def ridgefill_select_rows(scores, k: int, filled_idx, ws, exact_mask=None, stream=None) -> None:
    """Top-k rows by score (ties to the lower index) -> exact_mask (optional, uint8 [P])
    and the remaining rows in ascending order -> filled_idx (int32 [P - k])."""
    _check(lib().ridgefill_select_rows(_ptr(scores), int(scores.numel()), int(k), _ptr(exact_mask),
                                       _ptr(filled_idx), _ptr(ws), _nbytes(ws), _stream(stream)))


# ------------------------------------------------------------------------------ fill

def ridgefill_fill_workspace_bytes(shape: rf_shape, n_filled: int, n_layers: int,
                                   map_flags: int = 0) -> int:
    return int(lib().ridgefill_fill_workspace_bytes_ex(C.byref(shape), int(n_filled),
                                                       int(n_layers), int(map_flags)))


def _layers(layers: list[dict]):
    """rf_layer array from dicts of torch tensors: A (bf16 [d][d_in]) or A_q (int8) with
    A_scale (fp32 [d]); b (fp32 [d]); norm_w (bf16 [d]); W_K, W_V (bf16 [kv][d]); k_pages,
    v_pages (bf16 [num_pages][page_size][n_kv][hd]); optional k_norm_w (bf16 [hd]) and
    v_scale (fp32 [n_kv]); or, for a folded layer, folded (uint8 device buffer made by
    ridgefill_fold_maps) with the pages and the optional parts."""
    arr = (rf_layer * max(len(layers), 1))()
    for i, l in enumerate(layers):
        g = l.get
        arr[i] = rf_layer(_ptr(g("A")), _ptr(g("b")), _ptr(g("norm_w")), _ptr(g("W_K")),
                          _ptr(g("W_V")), _ptr(g("k_pages")), _ptr(g("v_pages")),
                          _ptr(g("k_norm_w")), _ptr(g("v_scale")), _ptr(g("A_q")),
                          _ptr(g("A_scale")), _ptr(g("folded")))
    return arr


def ridgefill_fold_bytes(shape: rf_shape) -> int:
    """Bytes of one layer's folded buffer (0: the shape cannot be folded)."""
    return int(lib().ridgefill_fold_bytes(C.byref(shape)))


def ridgefill_fold_workspace_bytes(shape: rf_shape) -> int:
    return int(lib().ridgefill_fold_workspace_bytes(C.byref(shape)))


def ridgefill_fold_workspace_bytes_ex(shape: rf_shape, layers_at_once: int) -> int:
    """Fold workspace for layers_at_once layers folded side by side."""
    return int(lib().ridgefill_fold_workspace_bytes_ex(C.byref(shape), layers_at_once))


def ridgefill_fold_workspace_bytes_maps(shape: rf_shape, layers_at_once: int, map_flags: int) -> int:
    """Fold workspace for layers_at_once layers side by side, for bf16 maps (map_flags 0)
    or int8 maps (RF_MAPS_INT8)."""
    return int(lib().ridgefill_fold_workspace_bytes_maps(C.byref(shape), layers_at_once, map_flags))


def ridgefill_fold_maps(shape: rf_shape, layers: list[dict], folded: list, ws, stream=None) -> None:
    """Folded buffers (uint8 device tensors, one per layer) from the layers' plain fields."""
    arr = _layers(layers)
    ptrs = (C.c_void_p * max(len(folded), 1))(*[_ptr(f) for f in folded])
    _check(lib().ridgefill_fold_maps(C.byref(shape), arr, len(layers), ptrs, _ptr(ws),
                                     _nbytes(ws), _stream(stream)))


def ridgefill_fill(shape: rf_shape, x_S, N: int, T: int, filled_idx, n_filled: int,
                   layers: list[dict], block_table, page_size: int, num_pages: int,
                   ws, x_stride: int | None = None, stream=None, copy_stream=None) -> None:
    """The fill; with copy_stream given, the streamed variant (maps in host tensors)."""
    arr = _layers(layers)
    kv = rf_paged_kv(_ptr(block_table), int(block_table.numel()), int(page_size), int(num_pages))
    stride = int(x_stride if x_stride is not None else x_S.stride(0))
    args = (C.byref(shape), _ptr(x_S), int(N), int(T), stride, _ptr(filled_idx), int(n_filled),
            arr, len(layers), C.byref(kv), _ptr(ws), int(ws.numel() * ws.element_size()),
            _stream(stream))
    if copy_stream is None:
        _check(lib().ridgefill_fill(*args))
    else:
        _check(lib().ridgefill_fill_streamed(*args, _stream(copy_stream)))


def ridgefill_fill_noalloc(shape: rf_shape, x_S, N: int, T: int, filled_idx, n_filled: int,
                           layers: list[dict], block_table, page_size: int, num_pages: int,
                           status, x_stride: int | None = None, stream=None) -> None:
    """The fill with the library's fixed device scratch as its workspace (no allocation);
    the device status goes to `status` (a device int32/uint32 tensor of >= 1 element)."""
    arr = _layers(layers)
    kv = rf_paged_kv(_ptr(block_table), int(block_table.numel()), int(page_size), int(num_pages))
    stride = int(x_stride if x_stride is not None else x_S.stride(0))
    _check(lib().ridgefill_fill_noalloc(C.byref(shape), _ptr(x_S), int(N), int(T), stride,
                                        _ptr(filled_idx), int(n_filled), arr, len(layers),
                                        C.byref(kv), _ptr(status), _stream(stream)))


RIDGEFILL_NOALLOC_SCRATCH_BYTES = 64 << 20


def ridgefill_value_scale_workspace_bytes(shape: rf_shape, c: int, n_layers: int,
                                          map_flags: int = 0) -> int:
    return int(lib().ridgefill_value_scale_workspace_bytes(C.byref(shape), int(c), int(n_layers),
                                                           int(map_flags)))


def ridgefill_value_scale(shape: rf_shape, x_S_tail, x_l_tail: list, layers: list[dict], out,
                          ws, x_stride: int | None = None, stream=None) -> None:
    """Value-rescale factors of every layer into out (fp32 [n_layers][n_kv])."""
    arr = _layers(layers)
    ptrs = (C.c_void_p * max(len(x_l_tail), 1))(*[_ptr(t) for t in x_l_tail])
    stride = int(x_stride if x_stride is not None else x_S_tail.stride(0))
    _check(lib().ridgefill_value_scale(C.byref(shape), _ptr(x_S_tail), stride, ptrs,
                                       int(x_S_tail.shape[0]), arr, len(layers), _ptr(out),
                                       _ptr(ws), int(ws.numel() * ws.element_size()),
                                       _stream(stream)))


# ------------------------------------------------------------------------------ the cache
#
# These calls check what the C side cannot see (types, devices, shapes of the tensors), run on
# the tensors' own device and, unless a stream is given, on that device's current stream.

def _need(name: str, t, dtype, device, ndim: int) -> None:
    if t.dtype is not dtype or t.device != device or t.dim() != ndim:
        raise ValueError(f"{name} must be a {dtype} tensor of {ndim} dimensions on {device}, not "
                         f"{t.dtype} of {t.dim()} on {t.device}")


def _flat(name: str, t, dtype, device, ndim: int, shape: tuple | None = None) -> None:
    """A contiguous tensor, of the given shape where one is given."""
    if (t.dtype is dtype and t.device == device and t.is_contiguous()
            and (t.shape == shape if shape is not None else t.dim() == ndim)):
        return
    _need(name, t, dtype, device, ndim)
    raise ValueError(f"{name} must be contiguous" + (f" {shape}" if shape else "") +
                     f", not {tuple(t.shape)} with strides {t.stride()}")


def _fits(*values: int) -> bool:
    """Whether integers are what the C side will get: ctypes cuts off what is past 32 bits."""
    for v in values:
        if not -0x80000000 <= v <= 0x7fffffff:
            return False
    return True


def _ints(**values: int) -> None:
    for name, v in values.items():
        if not _fits(v):
            raise ValueError(f"{name} = {v} does not fit 32 bits")


def _rows_of(name: str, t, dtype, device, width: int, n: int | None = None) -> int:
    """Elements between the rows of [rows][heads][head_dim]; each row lies in one piece.  A single
    row's stride means nothing and is taken as the row's own size."""
    shape, stride = t.shape, t.stride()
    if (t.dtype is dtype and t.device == device and len(shape) == 3 and shape[2] == width
            and stride[2] == 1 and (stride[1] == width or shape[1] == 1) and shape[1] > 0
            and (n is None or shape[0] == n)):
        return stride[0] if shape[0] > 1 else shape[1] * width
    _need(name, t, dtype, device, 3)
    raise ValueError(f"{name} must be [{'rows' if n is None else n}][heads][{width}] with each "
                     f"row in one piece, not {tuple(shape)} with strides {stride}")


def _go(f, device, stream, *args) -> None:
    """f(*args, stream) with `device` current."""
    import torch
    if device.type != "cuda":
        raise ValueError(f"the tensors must be in GPU memory, not on {device}")
    index = device.index
    if stream is None:      # the handle alone: a stream object takes longer to make than the checks
        handle = torch._C._cuda_getCurrentRawStream(index)
    else:
        handle = stream.cuda_stream
    if index == torch.cuda.current_device():
        status = f(*args, handle)
    else:
        with torch.cuda.device(device):
            status = f(*args, handle)
    if status != RF_OK:
        _check(status)


def make_rope(theta: float = 500000.0, rotary_dim: int = 0, layout: int = RF_ROPE_HALF,
              scaling: int = RF_ROPE_PLAIN, factor: float = 1.0, orig_len: int = 0,
              low: float = 0.0, high: float = 0.0, mscale: float = 0.0) -> rf_rope:
    _ints(rotary_dim=rotary_dim, layout=layout, scaling=scaling, orig_len=orig_len)
    return rf_rope(theta, rotary_dim, layout, scaling, orig_len, factor, low, high, mscale)


def make_batch(block_tables, lengths, page_size: int, num_pages: int, n_kv_heads: int,
               head_dim: int, max_len: int | None = None) -> rf_paged_batch:
    """Descriptor of a batch of sequences in a paged pool: block_tables int32 [batch][pages],
    lengths int32 [batch] (None where only rows are appended).  max_len bounds the lengths
    (default: all the rows that a table holds).  It keeps both tensors alive."""
    import torch
    dev = block_tables.device
    _need("block_tables", block_tables, torch.int32, dev, 2)
    batch, per = block_tables.shape
    if block_tables.stride(1) != 1 and per > 1:
        raise ValueError("the entries of a block table must lie in one piece")
    if lengths is not None:
        _flat("lengths", lengths, torch.int32, dev, 1, (batch,))
    if max_len is None:
        max_len = per * page_size
    _ints(max_len=max_len, page_size=page_size, num_pages=num_pages, n_kv_heads=n_kv_heads,
          head_dim=head_dim)
    kv = rf_paged_batch(block_tables.data_ptr(), _ptr(lengths),
                        block_tables.stride(0) if batch > 1 else per, batch, max_len, page_size,
                        num_pages, n_kv_heads, head_dim)
    if per * page_size < kv.max_len:
        raise ValueError(f"a block table of {per} pages holds fewer than max_len = {kv.max_len} rows")
    kv._keep = (block_tables, lengths)
    kv._pool = (num_pages, page_size, n_kv_heads, head_dim)
    kv._device = dev
    return kv


def make_pools(k_pages: list, v_pages: list):
    """Array of layers that carry only their page pools, for ridgefill_evict_rows; it keeps
    the pools alive."""
    pools = (rf_layer * max(len(k_pages), 1))()
    for i, (k, v) in enumerate(zip(k_pages, v_pages, strict=True)):
        pools[i].k_pages, pools[i].v_pages = k.data_ptr(), v.data_ptr()
    pools._keep = (list(k_pages), list(v_pages))
    return pools


def ridgefill_rope(rope: rf_rope, x, positions, out, transpose: bool = False, stream=None) -> None:
    """x [rows][heads][head_dim] (bf16 or fp32) rotated by positions (int32 [rows]) into out
    (may be x); transpose=True takes the gradient of out to the gradient of x."""
    import torch
    dev, hd = x.device, x.shape[-1]
    kind = RF_TYPE_F32 if x.dtype == torch.float32 else RF_TYPE_BF16
    dtype = torch.float32 if kind else torch.bfloat16
    xs = _rows_of("x", x, dtype, dev, hd)
    n, heads = x.shape[0], x.shape[1]
    os_ = _rows_of("out", out, dtype, dev, hd, n)
    if out.shape[1] != heads:
        raise ValueError(f"out has {out.shape[1]} heads, x {heads}")
    _flat("positions", positions, torch.int32, dev, 1, (n,))
    _go(lib().ridgefill_rope, dev, stream, C.byref(rope), x.data_ptr(), kind, n, heads, hd, xs,
        positions.data_ptr(), out.data_ptr(), os_, 1 if transpose else 0)


def _status_of(status, device) -> None:
    if status.device != device or status.numel() < 1 or status.element_size() != 4:
        raise ValueError("status must be a 4-byte integer tensor on the cache's device")


def _appended(kv: rf_paged_batch, k, v, rows, status, seq, positions, q, q_out) -> tuple:
    """Checks of what an append writes; q, k and v as the C side takes them."""
    import torch
    dev, n, hd = kv._device, k.shape[0], kv.head_dim
    ks = _rows_of("k", k, torch.bfloat16, dev, hd, n)
    vs = _rows_of("v", v, torch.bfloat16, dev, hd, n)
    if k.shape[1] != kv.n_kv_heads or v.shape[1] != kv.n_kv_heads:
        raise ValueError(f"k and v must have {kv.n_kv_heads} heads")
    _flat("rows", rows, torch.int32, dev, 1, (n,))
    if seq is not None:
        _flat("seq", seq, torch.int32, dev, 1, (n,))
    if positions is not None:
        _flat("positions", positions, torch.int32, dev, 1, (n,))
    _status_of(status, dev)
    heads = qs = qos = 0
    if q is not None:
        if q_out is None:
            raise ValueError("q without q_out")
        qs = _rows_of("q", q, torch.bfloat16, dev, hd, n)
        qos = _rows_of("q_out", q_out, torch.bfloat16, dev, hd, n)
        heads = q.shape[1]
        if q_out.shape[1] != heads:
            raise ValueError(f"q_out has {q_out.shape[1]} heads, q {heads}")
    elif q_out is not None:
        raise ValueError("q_out without q")
    return _ptr(q), heads, qs, _ptr(q_out), qos, k.data_ptr(), ks, v.data_ptr(), vs


def ridgefill_append_rows(rope: rf_rope | None, kv: rf_paged_batch, k, v, rows, k_pages, v_pages,
                          status, seq=None, positions=None, q=None, q_out=None, stream=None) -> None:
    """k (rotated) and v, bf16 [n][n_kv][head_dim], into cache rows `rows` (int32 [n]) of
    sequences `seq` (int32 [n]; None: sequence 0; negative: a padding row); q rotated into
    q_out.  positions (int32 [n]) default to the rows.  status: device int32 tensor."""
    import torch
    dev = kv._device
    _flat("k_pages", k_pages, torch.bfloat16, dev, 4, kv._pool)
    _flat("v_pages", v_pages, torch.bfloat16, dev, 4, kv._pool)
    args = _appended(kv, k, v, rows, status, seq, positions, q, q_out)
    _go(lib().ridgefill_append_rows, dev, stream, None if rope is None else C.byref(rope),
        C.byref(kv), *args, k.shape[0], _ptr(seq), rows.data_ptr(), _ptr(positions),
        k_pages.data_ptr(), v_pages.data_ptr(), status.data_ptr())


def ridgefill_tree_attention_workspace_bytes(kv: rf_paged_batch, n_q_heads: int, max_q: int) -> int:
    return int(lib().ridgefill_tree_attention_workspace_bytes(C.byref(kv), n_q_heads, max_q)) if _fits(n_q_heads, max_q) else 0


def _queries(kv: rf_paged_batch, k_pages, q, q_start, max_q, tree_mask, lse, ws) -> int:
    """Checks shared by the attention and the weight accumulation; q's row stride."""
    import torch
    dev = kv._device
    if not _fits(max_q):
        raise ValueError(f"max_q = {max_q} does not fit 32 bits")
    if kv._keep[1] is None:
        raise ValueError("the batch was made without lengths")
    stride = _rows_of("q", q, torch.bfloat16, dev, kv.head_dim)
    if k_pages is not None:
        _flat("k_pages", k_pages, torch.bfloat16, dev, 4, kv._pool)
    _flat("q_start", q_start, torch.int32, dev, 1, (kv.batch + 1,))
    n, heads = q.shape[0], q.shape[1]
    if tree_mask is not None:
        _flat("tree_mask", tree_mask, torch.int64, dev, 1, (n,))
    if lse is not None:
        _flat("lse", lse, torch.float32, dev, 2, (n, heads))
    if ws.device != dev or not ws.is_contiguous():
        raise ValueError("the workspace must be contiguous and on the cache's device")
    return stride


def ridgefill_tree_attention(kv: rf_paged_batch, k_pages, v_pages, q, q_start, max_q: int,
                             scale: float, out, ws, lse=None, tree_mask=None, stream=None) -> None:
    """Attention of q (bf16 [n][heads][head_dim]), the last rows of each sequence, over the
    cache.  q_start int32 [batch + 1]; tree_mask int64 [n] (bit j: sees draft j) or None (a
    chain); out bf16 like q or None; lse fp32 [n][heads] or None."""
    import torch
    qs = _queries(kv, k_pages, q, q_start, max_q, tree_mask, lse, ws)
    os_ = 0
    if out is not None:
        if v_pages is None:
            raise ValueError("out without v_pages")
        _flat("v_pages", v_pages, torch.bfloat16, kv._device, 4, kv._pool)
        os_ = _rows_of("out", out, torch.bfloat16, kv._device, kv.head_dim, q.shape[0])
        if out.shape[1] != q.shape[1]:
            raise ValueError(f"out has {out.shape[1]} heads, q {q.shape[1]}")
    _go(lib().ridgefill_tree_attention, kv._device, stream, C.byref(kv), k_pages.data_ptr(),
        _ptr(v_pages), q.data_ptr(), q.shape[1], qs, q_start.data_ptr(), q.shape[0], max_q,
        _ptr(tree_mask), scale, _ptr(out), os_, _ptr(lse), ws.data_ptr(), _nbytes(ws))


def ridgefill_attention_weight_workspace_bytes(kv: rf_paged_batch, n_q_heads: int, max_q: int) -> int:
    return int(lib().ridgefill_attention_weight_workspace_bytes(C.byref(kv), n_q_heads, max_q)) if _fits(n_q_heads, max_q) else 0


def ridgefill_attention_weight(kv: rf_paged_batch, k_pages, q, q_start, max_q: int, scale: float,
                               lse, acc_out, ws, acc=None, decay: float = 1.0, tree_mask=None,
                               stream=None) -> None:
    """acc_out (fp32 [batch][>= max_len]) = decay * acc + the weight that q's queries, with
    their lse, give to each cached row; acc=None where nothing is accumulated yet."""
    import torch
    qs = _queries(kv, k_pages, q, q_start, max_q, tree_mask, lse, ws)
    dev = kv._device
    if lse is None:
        raise ValueError("the weights need the queries' lse")
    _flat("acc_out", acc_out, torch.float32, dev, 2)
    if acc_out.shape[0] != kv.batch:
        raise ValueError(f"acc_out has {acc_out.shape[0]} rows for {kv.batch} sequences")
    if acc is not None:
        _flat("acc", acc, torch.float32, dev, 2, tuple(acc_out.shape))
    _go(lib().ridgefill_attention_weight, dev, stream, C.byref(kv), k_pages.data_ptr(), q.data_ptr(),
        q.shape[1], qs, q_start.data_ptr(), q.shape[0], max_q, _ptr(tree_mask), scale,
        lse.data_ptr(), decay, _ptr(acc), acc_out.data_ptr(), acc_out.shape[1], ws.data_ptr(),
        _nbytes(ws))


def ridgefill_evict_workspace_bytes(kv: rf_paged_batch, n_keep: int) -> int:
    return int(lib().ridgefill_evict_workspace_bytes(C.byref(kv), n_keep)) if _fits(n_keep) else 0


def ridgefill_evict_rows(kv: rf_paged_batch, layers, acc, positions, n_keep: int, acc_out,
                         positions_out, lengths_out, ws, n_sink: int = 0, n_recent: int = 0,
                         stream=None) -> None:
    """Every sequence of more than n_keep rows cut to them, in the pools of `layers` (from
    make_pools, or dicts with k_pages and v_pages).  acc fp32 and positions int32
    [batch][>= max_len]; the three outputs may be the inputs."""
    import torch
    dev = kv._device
    if kv._keep[1] is None:
        raise ValueError("the batch was made without lengths")
    if not _fits(n_keep, n_sink, n_recent):
        raise ValueError(f"n_keep = {n_keep}, n_sink = {n_sink}, n_recent = {n_recent}: more than 32 bits")
    if isinstance(layers, (list, tuple)):
        layers = make_pools([l["k_pages"] for l in layers], [l["v_pages"] for l in layers])
    for pool in layers._keep[0] + layers._keep[1]:
        _flat("k_pages and v_pages", pool, torch.bfloat16, dev, 4, kv._pool)
    shape = (kv.batch, acc.shape[-1])
    _flat("acc", acc, torch.float32, dev, 2, shape)
    _flat("acc_out", acc_out, torch.float32, dev, 2, shape)
    _flat("positions", positions, torch.int32, dev, 2, shape)
    _flat("positions_out", positions_out, torch.int32, dev, 2, shape)
    _flat("lengths_out", lengths_out, torch.int32, dev, 1, (kv.batch,))
    if ws.device != dev or not ws.is_contiguous():
        raise ValueError("the workspace must be contiguous and on the cache's device")
    _go(lib().ridgefill_evict_rows, dev, stream, C.byref(kv), layers, len(layers._keep[0]),
        acc.data_ptr(), positions.data_ptr(), shape[1], n_keep, n_sink, n_recent,
        acc_out.data_ptr(), positions_out.data_ptr(), lengths_out.data_ptr(), ws.data_ptr(),
        _nbytes(ws))


def make_head_norm(q_w=None, k_w=None, eps: float = 1e-6) -> rf_head_norm:
    """Norms of query and key heads: weights [head_dim] (None: that tensor is not normed), of the
    type of the tensors they are used on.  It keeps them alive."""
    for name, w in (("q_w", q_w), ("k_w", k_w)):
        if w is not None and (w.dim() != 1 or not w.is_contiguous()):
            raise ValueError(f"{name} must be contiguous [head_dim], not {tuple(w.shape)} with strides {w.stride()}")
    norm = rf_head_norm(_ptr(q_w), _ptr(k_w), eps, 0)
    norm._keep = (q_w, k_w)
    return norm


def make_cache(k_pages, v_pages, k_scales=None, v_scales=None) -> rf_cache:
    """One layer's pools [num_pages][page_size][n_kv][head_dim]: bf16, or 8-bit codes
    (float8_e4m3fn or int8) with their blocks' scales, uint8 [num_pages][page_size][n_kv]
    [head_dim / 32].  v_pages may be None for attention that gives only lse.  It keeps them alive."""
    import torch
    kinds = {torch.bfloat16: RF_CACHE_BF16, torch.float8_e4m3fn: RF_CACHE_FP8, torch.int8: RF_CACHE_INT8}
    dtype, dev = k_pages.dtype, k_pages.device
    if dtype not in kinds:
        raise ValueError(f"k_pages must be bfloat16, float8_e4m3fn or int8, not {dtype}")
    _flat("k_pages", k_pages, dtype, dev, 4)
    shape = tuple(k_pages.shape)
    if v_pages is not None:
        _flat("v_pages", v_pages, dtype, dev, 4, shape)
    for name, pages, scales in (("k_scales", k_pages, k_scales), ("v_scales", v_pages, v_scales)):
        if (scales is not None) != (dtype is not torch.bfloat16 and pages is not None):
            raise ValueError(f"{name}: pages of 8 bits have scales, others have none")
        if scales is not None:
            _flat(name, scales, torch.uint8, dev, 4, shape[:3] + (shape[3] // 32,))
    cache = rf_cache(kinds[dtype], 0, k_pages.data_ptr(), _ptr(v_pages), _ptr(k_scales), _ptr(v_scales))
    cache._keep = (k_pages, v_pages, k_scales, v_scales)
    cache._pool, cache._device = shape, dev
    return cache


def _cache_of(kv: rf_paged_batch, cache: rf_cache) -> None:
    if cache._pool != kv._pool or cache._device != kv._device:
        raise ValueError(f"the cache's pools are {cache._pool} on {cache._device}, the batch's {kv._pool} on {kv._device}")


def _normed(norm: rf_head_norm | None, dtype, device, head_dim: int) -> None:
    """The weights of a norm that is used on tensors of this type."""
    for name, w in zip(("q_w", "k_w"), norm._keep if norm is not None else ()):
        if w is not None:
            _flat(name, w, dtype, device, 1, (head_dim,))


def ridgefill_norm_rope(rope: rf_rope | None, norm: rf_head_norm | None, positions, q=None, q_out=None,
                        k=None, k_out=None, stream=None) -> None:
    """q and k [rows][heads][head_dim] (bf16 or fp32; either may be None), normed per head where
    `norm` has a weight and rotated by positions (int32 [rows]), into q_out and k_out (which may
    be q and k)."""
    import torch
    x = q if q is not None else k
    if x is None:
        raise ValueError("neither q nor k")
    dev, n, hd = x.device, x.shape[0], x.shape[-1]
    dtype = torch.float32 if x.dtype is torch.float32 else torch.bfloat16
    _normed(norm, dtype, dev, hd)
    args = []
    for name, t, out in (("q", q, q_out), ("k", k, k_out)):
        if (t is None) != (out is None):
            raise ValueError(f"{name} and {name}_out go together")
        if t is None:
            args += [None, 0, 0, None, 0]
            continue
        stride = _rows_of(name, t, dtype, dev, hd, n)
        out_stride = _rows_of(name + "_out", out, dtype, dev, hd, n)
        if out.shape[1] != t.shape[1]:
            raise ValueError(f"{name}_out has {out.shape[1]} heads, {name} {t.shape[1]}")
        args += [t.data_ptr(), t.shape[1], stride, out.data_ptr(), out_stride]
    if rope is not None:
        _flat("positions", positions, torch.int32, dev, 1, (n,))
    _go(lib().ridgefill_norm_rope, dev, stream, None if rope is None else C.byref(rope),
        None if norm is None else C.byref(norm), RF_TYPE_F32 if dtype is torch.float32 else RF_TYPE_BF16, n, hd,
        None if rope is None else positions.data_ptr(), *args)


def ridgefill_norm_rope_grad_workspace_bytes(n_rows: int, n_q_heads: int, n_k_heads: int, head_dim: int) -> int:
    if not _fits(n_rows, n_q_heads, n_k_heads, head_dim):
        return 0
    return int(lib().ridgefill_norm_rope_grad_workspace_bytes(n_rows, n_q_heads, n_k_heads, head_dim))


def ridgefill_norm_rope_grad(rope: rf_rope | None, norm: rf_head_norm | None, positions, ws, q=None, gq=None,
                             q_grad=None, qw_grad=None, k=None, gk=None, k_grad=None, kw_grad=None,
                             stream=None) -> None:
    """From the gradients gq and gk of the outputs of ridgefill_norm_rope on q and k: q_grad and
    k_grad (which may be gq and gk), and qw_grad and kw_grad (fp32 [head_dim], None: not wanted)
    of the weights.  q or k may be None where it has no weight."""
    import torch
    x = gq if gq is not None else gk
    if x is None:
        raise ValueError("neither gq nor gk")
    dev, n, hd = x.device, x.shape[0], x.shape[-1]
    dtype = torch.float32 if x.dtype is torch.float32 else torch.bfloat16
    _normed(norm, dtype, dev, hd)
    args = []
    weights = norm._keep if norm is not None else (None, None)
    for name, w, t, g, out, dw in (("q", weights[0], q, gq, q_grad, qw_grad), ("k", weights[1], k, gk, k_grad, kw_grad)):
        if (g is None) != (out is None) or (g is None and (t is not None or dw is not None)):
            raise ValueError(f"{name}: g{name} and {name}_grad go together")
        if g is None:
            args += [None, 0, 0, None, 0, None, 0, None]
            continue
        if w is not None and t is None:
            raise ValueError(f"the gradient of normed {name} needs {name}")
        stride = _rows_of(name, t, dtype, dev, hd, n) if t is not None else 0
        g_stride = _rows_of("g" + name, g, dtype, dev, hd, n)
        out_stride = _rows_of(name + "_grad", out, dtype, dev, hd, n)
        if out.shape[1] != g.shape[1] or (t is not None and t.shape[1] != g.shape[1]):
            raise ValueError(f"{name}, g{name} and {name}_grad differ in heads")
        if dw is not None:
            _flat(name + "w_grad", dw, torch.float32, dev, 1, (hd,))
        args += [_ptr(t), g.shape[1], stride, g.data_ptr(), g_stride, out.data_ptr(), out_stride, _ptr(dw)]
    if rope is not None:
        _flat("positions", positions, torch.int32, dev, 1, (n,))
    if ws.device != dev or not ws.is_contiguous():
        raise ValueError("the workspace must be contiguous and on the tensors' device")
    _go(lib().ridgefill_norm_rope_grad, dev, stream, None if rope is None else C.byref(rope),
        None if norm is None else C.byref(norm), RF_TYPE_F32 if dtype is torch.float32 else RF_TYPE_BF16, n, hd,
        None if rope is None else positions.data_ptr(), *args, ws.data_ptr(), _nbytes(ws))


def ridgefill_append_cache(rope: rf_rope | None, norm: rf_head_norm | None, kv: rf_paged_batch, cache: rf_cache, k, v,
                           rows, status, seq=None, positions=None, q=None, q_out=None, stream=None) -> None:
    """ridgefill_append_rows into a cache of any type (from make_cache), with q and k normed per
    head where `norm` has a weight (bf16)."""
    import torch
    dev, n, hd = kv._device, k.shape[0], kv.head_dim
    _cache_of(kv, cache)
    _normed(norm, torch.bfloat16, dev, hd)
    if cache._keep[1] is None:
        raise ValueError("the cache was made without v_pages")
    args = _appended(kv, k, v, rows, status, seq, positions, q, q_out)
    _go(lib().ridgefill_append_cache, dev, stream, None if rope is None else C.byref(rope),
        None if norm is None else C.byref(norm), C.byref(kv), C.byref(cache), *args, n, _ptr(seq),
        rows.data_ptr(), _ptr(positions), status.data_ptr())


def ridgefill_read_rows(kv: rf_paged_batch, cache: rf_cache, rows, status, seq=None, k_out=None, v_out=None,
                        stream=None) -> None:
    """Cache rows `rows` (int32 [n]) of sequences `seq` (int32 [n]; None: sequence 0; negative:
    left out) into k_out and v_out [n][n_kv][head_dim], bf16 or fp32; one of them may be None."""
    import torch
    dev, n, hd = kv._device, rows.shape[0], kv.head_dim
    _cache_of(kv, cache)
    out = k_out if k_out is not None else v_out
    if out is None:
        raise ValueError("neither k_out nor v_out")
    if v_out is not None and cache._keep[1] is None:
        raise ValueError("v_out, and the cache was made without v_pages")
    dtype = torch.float32 if out.dtype is torch.float32 else torch.bfloat16
    strides = []
    for name, t in (("k_out", k_out), ("v_out", v_out)):
        strides.append(0 if t is None else _rows_of(name, t, dtype, dev, hd, n))
        if t is not None and t.shape[1] != kv.n_kv_heads:
            raise ValueError(f"{name} must have {kv.n_kv_heads} heads")
    _flat("rows", rows, torch.int32, dev, 1, (n,))
    if seq is not None:
        _flat("seq", seq, torch.int32, dev, 1, (n,))
    _status_of(status, dev)
    _go(lib().ridgefill_read_rows, dev, stream, C.byref(kv), C.byref(cache), n, _ptr(seq), rows.data_ptr(),
        RF_TYPE_F32 if dtype is torch.float32 else RF_TYPE_BF16, _ptr(k_out), strides[0], _ptr(v_out), strides[1],
        status.data_ptr())


def make_prefix(block_tables, lengths, group_start, max_len: int) -> rf_prefix:
    """Prefixes that groups of sequences share: block_tables int32 [groups][pages], lengths int32
    [groups], group_start int32 [groups + 1] (the groups' sequences, ascending); max_len bounds the
    lengths.  It keeps the tensors alive."""
    import torch
    dev = block_tables.device
    _need("block_tables", block_tables, torch.int32, dev, 2)
    groups, per = block_tables.shape
    if block_tables.stride(1) != 1 and per > 1:
        raise ValueError("the entries of a block table must lie in one piece")
    _flat("lengths", lengths, torch.int32, dev, 1, (groups,))
    _flat("group_start", group_start, torch.int32, dev, 1, (groups + 1,))
    _ints(max_len=max_len, groups=groups)
    prefix = rf_prefix(block_tables.data_ptr(), lengths.data_ptr(), group_start.data_ptr(),
                       block_tables.stride(0) if groups > 1 else per, groups, max_len)
    prefix._keep = (block_tables, lengths, group_start)
    prefix._per, prefix._device = per, dev
    return prefix


def ridgefill_cache_attention_workspace_bytes(kv: rf_paged_batch, n_q_heads: int, max_q: int, n_q: int,
                                              prefix: rf_prefix | None = None) -> int:
    if not _fits(n_q_heads, max_q, n_q):
        return 0
    return int(lib().ridgefill_cache_attention_workspace_bytes(C.byref(kv), None if prefix is None else C.byref(prefix),
                                                               n_q_heads, max_q, n_q))


def ridgefill_cache_attention(kv: rf_paged_batch, cache: rf_cache, q, q_start, max_q: int, scale: float, out, ws,
                              prefix: rf_prefix | None = None, lse=None, tree_mask=None, stream=None) -> None:
    """ridgefill_tree_attention over a cache of any type (from make_cache); with `prefix` (from
    make_prefix) the sequences of a group see their prefix's rows before their own."""
    _cache_of(kv, cache)
    qs = _queries(kv, None, q, q_start, max_q, tree_mask, lse, ws)
    os_ = 0
    if out is not None:
        if cache._keep[1] is None:
            raise ValueError("out, and the cache was made without v_pages")
        os_ = _rows_of("out", out, q.dtype, kv._device, kv.head_dim, q.shape[0])
        if out.shape[1] != q.shape[1]:
            raise ValueError(f"out has {out.shape[1]} heads, q {q.shape[1]}")
    if prefix is not None:
        if prefix._device != kv._device:
            raise ValueError(f"the prefix's tables are on {prefix._device}, the batch's on {kv._device}")
        if prefix._per * kv.page_size < prefix.max_len:
            raise ValueError(f"a prefix's table of {prefix._per} pages holds fewer than max_len = {prefix.max_len} rows")
    _go(lib().ridgefill_cache_attention, kv._device, stream, C.byref(kv), None if prefix is None else C.byref(prefix),
        C.byref(cache), q.data_ptr(), q.shape[1], qs, q_start.data_ptr(), q.shape[0], max_q, _ptr(tree_mask), scale,
        _ptr(out), os_, _ptr(lse), ws.data_ptr(), _nbytes(ws))


# ------------------------------------------------------------------------------ calibration

def ridgefill_calib_state_bytes(d: int, n_layers: int, d_out: int | None = None) -> int:
    """State size for x_S of width d (= d_in) and layer inputs of width d_out (default d)."""
    return int(lib().ridgefill_calib_state_bytes_ex(int(d), int(d_out or d), int(n_layers)))


def _nbytes(t) -> int:
    return int(t.numel() * t.element_size())


def ridgefill_calib_reset(state, d: int, n_layers: int, stream=None,
                          d_out: int | None = None) -> None:
    _check(lib().ridgefill_calib_reset_ex(_ptr(state), _nbytes(state), int(d), int(d_out or d),
                                          int(n_layers), _stream(stream)))


def ridgefill_calibrate(state, d: int, n_layers: int, x_S, x_l: list, n_rows: int | None = None,
                        stream=None, d_out: int | None = None) -> None:
    ptrs = (C.c_void_p * max(len(x_l), 1))(*[_ptr(t) for t in x_l])
    n = int(n_rows if n_rows is not None else x_S.shape[0])
    _check(lib().ridgefill_calibrate_ex(_ptr(state), _nbytes(state), int(d), int(d_out or d),
                                        int(n_layers), _ptr(x_S), ptrs, n, _stream(stream)))


def ridgefill_solve_workspace_bytes(d: int, n_layers: int, d_out: int | None = None) -> int:
    return int(lib().ridgefill_solve_workspace_bytes_ex(int(d), int(d_out or d), int(n_layers)))


def ridgefill_solve(state, d: int, n_layers: int, lam: float, A_out, b_out, A_bf16_out, ws,
                    stream=None, d_out: int | None = None) -> None:
    """A_out fp32 [n_layers][d_out][d], b_out [n_layers][d_out] (d_out defaults to d)."""
    _check(lib().ridgefill_solve_ex(_ptr(state), _nbytes(state), int(d), int(d_out or d),
                                    int(n_layers), float(lam), _ptr(A_out), _ptr(b_out),
                                    _ptr(A_bf16_out), _ptr(ws), _nbytes(ws), _stream(stream)))


def ridgefill_read_status(ws, stream=None) -> int:
    """Device status of the last fill/solve/selection on this workspace (waits for the
    stream): RF_OK, RF_E_ROWS, RF_E_NOT_SPD, RF_E_INVALID (a NaN selection score) or
    RF_E_WORKSPACE (a solve on a calibration state that does not match its sizes)."""
    if ws is None:
        raise ValueError("ws is None")
    s = lib().ridgefill_read_status(_ptr(ws), _stream(stream))
    if s not in (RF_OK, RF_E_ROWS, RF_E_NOT_SPD, RF_E_INVALID, RF_E_WORKSPACE):
        _check(s)
    return int(s)


def ridgefill_solve_info(ws, stream=None) -> tuple[float, int]:
    """(kappa_F, parts) of the last solve on this workspace (waits for the stream)."""
    kap = C.c_double(0.0)
    parts = C.c_int32(0)
    _check(lib().ridgefill_solve_info(_ptr(ws), C.byref(kap), C.byref(parts), _stream(stream)))
    return float(kap.value), int(parts.value)


RF_KERNEL_FILL_MAP, RF_KERNEL_FILL_KV, RF_KERNEL_CALIB_MOMENTS, RF_KERNEL_CALIB_SUMS, \
    RF_KERNEL_SOLVE_MAP, RF_KERNEL_FILL_NORM = range(6)


def ridgefill_profile_enable(enable: bool) -> None:
    _check(lib().ridgefill_profile_enable(1 if enable else 0))


def ridgefill_profile_read(kernel: int) -> tuple[int, float]:
    """(launches, summed milliseconds) of one kernel since the last reset."""
    n = C.c_int64(0)
    ms = C.c_double(0.0)
    _check(lib().ridgefill_profile_read(int(kernel), C.byref(n), C.byref(ms)))
    return int(n.value), float(ms.value)


def ridgefill_profile_reset() -> None:
    _check(lib().ridgefill_profile_reset())


def ridgefill_status_string(s: int) -> str:
    return lib().ridgefill_status_string(int(s)).decode()
