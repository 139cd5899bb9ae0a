"""Submanifold sparse 3x3x3 convolution on MI355X: Python binding.

A thin ctypes layer over libsmconv.so (C ABI in include/smconv.h). It only
marshals arguments: torch tensors supply device memory and the current HIP
stream, every step of the computation runs in the library's HIP kernels.
There is no fallback: if the library is not built, every call raises.

    m = KernelMap()
    m.build(coords, spatial_shape=(1440, 1440, 41))     # int32 [N, 4] on the GPU
    wp = pack_weights(w)                                 # bf16 [27, C_in, C_out]
    y = m.forward(x, wp, relu=True)                      # bf16 [N, C_in] -> [N, C_out]
"""
from __future__ import annotations

import ctypes
import os

__all__ = ["KernelMap", "PackedWeights", "pack_weights", "subm_conv3d", "lib", "library_path",
           "SmconvError", "ROUTES", "EXPORTED_SYMBOLS", "use_torch_allocator", "probe_mfma_bf16",
           "probe_copy", "rms_norm", "rms_norm_backward", "linear", "linear_backward", "gated",
           "gated_backward", "quantize_weight", "ACTIVATIONS", "group_norm", "group_norm_backward",
           "Windows", "window_attention", "window_attention_backward"]

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_HERE, "libsmconv.so")

ROUTES = {"auto": 0, "dense": 1, "sorted": 2}
_ROUTE_NAMES = {v: k for k, v in ROUTES.items()}
SMC_BUILD_ASYNC = 1
SMC_FWD_RELU = 1
SMC_FWD_OUT_F32 = 2
SMC_FWD_MASK_TILES = 4
SMC_FWD_SLAB_IN_MEMORY = 8
SMC_BUILD_NO_PAIRS = 2
SMC_BUILD_NO_SORT = 4
SMC_BUILD_TABLE = 8
ALGOS = ("pairs", "pairs_slab", "mask_tiles")

EXPORTED_SYMBOLS = [
    "smc_map_create", "smc_map_destroy", "smc_map_build", "smc_map_sync", "smc_map_info",
    "smc_map_export", "smc_weight_packed_bytes", "smc_weight_pack", "smc_conv_forward",
    "smc_status_string", "smc_last_error", "smc_version", "smc_timing_enable", "smc_timing_read",
    "smc_map_set_order", "smc_map_calibrate", "smc_map_build_strided",
    "smc_map_export_out_coords", "smc_set_allocator", "smc_probe_mfma_out_bytes",
    "smc_probe_mfma_bf16", "smc_probe_copy", "smc_conv_forward_noalloc",
    "smc_test_force_lookback_timeout", "smc_map_rows", "smc_rms_norm", "smc_rms_norm_backward",
    "smc_rms_norm_backward_workspace", "smc_linear", "smc_gated", "smc_linear_backward",
    "smc_gated_backward", "smc_linear_workspace", "smc_gated_workspace",
    "smc_linear_backward_workspace", "smc_gated_backward_workspace", "smc_weight_quantize",
    "smc_group_norm", "smc_group_norm_backward", "smc_group_norm_workspace",
    "smc_group_norm_backward_workspace", "smc_windows_bytes", "smc_windows_build",
    "smc_window_attention", "smc_window_attention_backward",
    "smc_window_attention_backward_workspace",
]
STAGES = ["map", "neighbours", "mask_sort", "compact", "gemm", "centre"]


class SmconvError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(msg)
        self.status = status


class MapInfo(ctypes.Structure):
    _fields_ = [
        ("n", ctypes.c_int64), ("route", ctypes.c_int32), ("key_bits", ctypes.c_int32),
        ("origin", ctypes.c_int32 * 3), ("extent", ctypes.c_int32 * 3),
        ("batch", ctypes.c_int32), ("tile_m", ctypes.c_int32), ("grid_cells", ctypes.c_int64),
        ("pairs", ctypes.c_int64), ("pairs_padded", ctypes.c_int64), ("n_tiles", ctypes.c_int64),
        ("tap_count", ctypes.c_int64 * 125), ("status", ctypes.c_int32),
        ("n_groups", ctypes.c_int32), ("group_rows", ctypes.c_int64 * 4),
        ("kernel_size", ctypes.c_int32), ("taps", ctypes.c_int32),
        ("n_in", ctypes.c_int64), ("strided", ctypes.c_int32), ("out_extent", ctypes.c_int32 * 3),
    ]


class NormArgs(ctypes.Structure):
    _fields_ = [
        ("n", ctypes.c_int64), ("c", ctypes.c_int32), ("dtype", ctypes.c_int32),
        ("eps", ctypes.c_float), ("x", ctypes.c_void_p), ("ldx", ctypes.c_int64),
        ("residual", ctypes.c_void_p), ("ld_residual", ctypes.c_int64),
        ("weight", ctypes.c_void_p), ("y", ctypes.c_void_p), ("ldy", ctypes.c_int64),
        ("y_scale", ctypes.c_void_p), ("s", ctypes.c_void_p), ("lds", ctypes.c_int64),
    ]


class NormBackwardArgs(ctypes.Structure):
    _fields_ = [
        ("n", ctypes.c_int64), ("c", ctypes.c_int32), ("dtype", ctypes.c_int32),
        ("eps", ctypes.c_float), ("dy", ctypes.c_void_p), ("ld_dy", ctypes.c_int64),
        ("s", ctypes.c_void_p), ("lds", ctypes.c_int64), ("weight", ctypes.c_void_p),
        ("ds", ctypes.c_void_p), ("ld_ds", ctypes.c_int64), ("dx", ctypes.c_void_p),
        ("ld_dx", ctypes.c_int64), ("dweight", ctypes.c_void_p), ("workspace", ctypes.c_void_p),
        ("workspace_bytes", ctypes.c_size_t),
    ]


class ProductArgs(ctypes.Structure):
    _fields_ = [
        ("n", ctypes.c_int64), ("c_in", ctypes.c_int32), ("c_out", ctypes.c_int32),
        ("dtype", ctypes.c_int32), ("x_dtype", ctypes.c_int32), ("activation", ctypes.c_int32),
        ("x", ctypes.c_void_p), ("ldx", ctypes.c_int64), ("x_scale", ctypes.c_void_p),
        ("w", ctypes.c_void_p), ("ldw", ctypes.c_int64), ("w_transposed", ctypes.c_int32),
        ("w_scale", ctypes.c_void_p), ("bias", ctypes.c_void_p), ("residual", ctypes.c_void_p),
        ("ld_residual", ctypes.c_int64), ("y", ctypes.c_void_p), ("ldy", ctypes.c_int64),
        ("dy", ctypes.c_void_p), ("ld_dy", ctypes.c_int64), ("dx", ctypes.c_void_p),
        ("ld_dx", ctypes.c_int64), ("dw", ctypes.c_void_p), ("ld_dw", ctypes.c_int64),
        ("db", ctypes.c_void_p), ("workspace", ctypes.c_void_p),
        ("workspace_bytes", ctypes.c_size_t),
    ]


class GroupNormArgs(ctypes.Structure):
    _fields_ = [
        ("n", ctypes.c_int64), ("c", ctypes.c_int32), ("groups", ctypes.c_int32),
        ("samples", ctypes.c_int32), ("dtype", ctypes.c_int32), ("activation", ctypes.c_int32),
        ("eps", ctypes.c_float), ("offsets", ctypes.c_void_p), ("x", ctypes.c_void_p),
        ("ldx", ctypes.c_int64), ("weight", ctypes.c_void_p), ("bias", ctypes.c_void_p),
        ("y", ctypes.c_void_p), ("ldy", ctypes.c_int64), ("stats", ctypes.c_void_p),
        ("dy", ctypes.c_void_p), ("ld_dy", ctypes.c_int64), ("dx", ctypes.c_void_p),
        ("ld_dx", ctypes.c_int64), ("dweight", ctypes.c_void_p), ("dbias", ctypes.c_void_p),
        ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t),
    ]


class WindowsArgs(ctypes.Structure):
    _fields_ = [
        ("n", ctypes.c_int64), ("windows", ctypes.c_int64), ("offsets", ctypes.c_void_p),
        ("order", ctypes.c_void_p), ("coords", ctypes.c_void_p), ("coord_cols", ctypes.c_int32),
        ("ex", ctypes.c_int32), ("ey", ctypes.c_int32), ("ez", ctypes.c_int32),
        ("plan", ctypes.c_void_p), ("plan_bytes", ctypes.c_size_t), ("tiles32", ctypes.c_int32),
        ("tiles64", ctypes.c_int32), ("tiles128", ctypes.c_int32), ("longest", ctypes.c_int32),
        ("pairs", ctypes.c_int64),
    ]


class AttentionArgs(ctypes.Structure):
    _fields_ = [
        ("windows", ctypes.POINTER(WindowsArgs)), ("heads", ctypes.c_int32),
        ("kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32), ("dtype", ctypes.c_int32),
        ("scale", ctypes.c_float), ("reach", ctypes.c_int32), ("bias", ctypes.c_void_p),
        ("q", ctypes.c_void_p), ("ldq", ctypes.c_int64), ("k", ctypes.c_void_p),
        ("ldk", ctypes.c_int64), ("v", ctypes.c_void_p), ("ldv", ctypes.c_int64),
        ("out", ctypes.c_void_p), ("ld_out", ctypes.c_int64), ("lse", ctypes.c_void_p),
        ("dout", ctypes.c_void_p), ("ld_dout", ctypes.c_int64), ("dq", ctypes.c_void_p),
        ("ld_dq", ctypes.c_int64), ("dk", ctypes.c_void_p), ("ld_dk", ctypes.c_int64),
        ("dv", ctypes.c_void_p), ("ld_dv", ctypes.c_int64), ("dbias", ctypes.c_void_p),
        ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t),
    ]


_lib = None


def library_path() -> str:
    return _LIB_PATH


def lib():
    """Load libsmconv.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(_LIB_PATH):
        raise RuntimeError(f"{_LIB_PATH} is not built; run `python __graft_entry__.py build` "
                           "(hipcc --offload-arch=gfx950) first")
    # torch ships its own HIP runtime under the same soname (libamdhip64.so.7).
    # Importing torch first makes the library bind to that runtime, the one
    # that owns the tensors and streams handed over; loaded first, the library
    # would pull in a second runtime that cannot use them.
    import torch  # noqa: F401
    L = ctypes.CDLL(_LIB_PATH)
    vp, i32, i64, u32 = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_uint
    L.smc_map_create.argtypes = [ctypes.POINTER(vp)]
    L.smc_map_destroy.argtypes = [vp]
    L.smc_map_build.argtypes = [vp, vp, i64, i32, vp, i32, i32, i32, u32, vp]
    L.smc_map_sync.argtypes = [vp]
    L.smc_map_info.argtypes = [vp, ctypes.POINTER(MapInfo)]
    L.smc_map_rows.argtypes = [vp, ctypes.POINTER(i64), ctypes.POINTER(i64)]
    L.smc_map_export.argtypes = [vp, vp, vp, vp, vp, vp, vp]
    L.smc_weight_packed_bytes.argtypes = [i32, i32, i32]
    L.smc_weight_packed_bytes.restype = ctypes.c_size_t
    L.smc_weight_pack.argtypes = [vp, i32, i32, i32, vp, vp]
    L.smc_conv_forward.argtypes = [vp, vp, i32, vp, i32, vp, u32, vp]
    L.smc_conv_forward_noalloc.argtypes = [vp, vp, i32, vp, i32, vp, u32, vp]
    L.smc_test_force_lookback_timeout.argtypes = [vp, i32]
    L.smc_status_string.argtypes = [i32]
    L.smc_status_string.restype = ctypes.c_char_p
    L.smc_last_error.argtypes = []
    L.smc_last_error.restype = ctypes.c_char_p
    L.smc_version.restype = i32
    L.smc_timing_enable.argtypes = [vp, i32]
    L.smc_timing_read.argtypes = [vp, vp, vp, i32]
    L.smc_map_set_order.argtypes = [vp, vp, vp]
    L.smc_map_calibrate.argtypes = [vp, i32, vp, vp]
    L.smc_map_build_strided.argtypes = [vp, vp, i64, i32, vp, i32, i32, i32, i32, u32, vp]
    L.smc_map_export_out_coords.argtypes = [vp, vp]
    L.smc_set_allocator.argtypes = [vp, vp, vp]
    L.smc_probe_mfma_out_bytes.argtypes = [i32]
    L.smc_probe_mfma_out_bytes.restype = ctypes.c_size_t
    L.smc_probe_mfma_bf16.argtypes = [i64, vp, ctypes.c_size_t, ctypes.POINTER(ctypes.c_double), vp]
    L.smc_probe_copy.argtypes = [vp, vp, ctypes.c_size_t, vp]
    for name in ("smc_map_create", "smc_map_destroy", "smc_map_build", "smc_map_sync",
                 "smc_map_info", "smc_map_export", "smc_weight_pack", "smc_conv_forward",
                 "smc_timing_enable", "smc_timing_read", "smc_map_set_order",
                 "smc_map_calibrate", "smc_map_build_strided", "smc_map_export_out_coords",
                 "smc_set_allocator", "smc_probe_mfma_bf16", "smc_probe_copy",
                 "smc_conv_forward_noalloc", "smc_test_force_lookback_timeout", "smc_map_rows"):
        getattr(L, name).restype = i32
    for name, args in (("smc_rms_norm", NormArgs), ("smc_rms_norm_backward", NormBackwardArgs),
                       ("smc_linear", ProductArgs), ("smc_gated", ProductArgs),
                       ("smc_linear_backward", ProductArgs), ("smc_gated_backward", ProductArgs),
                       ("smc_group_norm", GroupNormArgs), ("smc_group_norm_backward", GroupNormArgs),
                       ("smc_windows_build", WindowsArgs), ("smc_window_attention", AttentionArgs),
                       ("smc_window_attention_backward", AttentionArgs)):
        getattr(L, name).argtypes = [ctypes.POINTER(args), vp]
        getattr(L, name).restype = i32
    for name, args in (("smc_linear_workspace", ProductArgs), ("smc_gated_workspace", ProductArgs),
                       ("smc_linear_backward_workspace", ProductArgs),
                       ("smc_gated_backward_workspace", ProductArgs),
                       ("smc_group_norm_workspace", GroupNormArgs),
                       ("smc_group_norm_backward_workspace", GroupNormArgs),
                       ("smc_window_attention_backward_workspace", AttentionArgs)):
        getattr(L, name).argtypes = [ctypes.POINTER(args)]
        getattr(L, name).restype = ctypes.c_size_t
    L.smc_rms_norm_backward_workspace.argtypes = [i64, i32]
    L.smc_rms_norm_backward_workspace.restype = ctypes.c_size_t
    L.smc_windows_bytes.argtypes = [i64, i64]
    L.smc_windows_bytes.restype = ctypes.c_size_t
    L.smc_weight_quantize.argtypes = [vp, i64, i32, i32, i32, vp, i64, vp, vp]
    L.smc_weight_quantize.restype = i32
    _lib = L
    return L


_ALLOC_T = ctypes.CFUNCTYPE(ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p)
_FREE_T = ctypes.CFUNCTYPE(None, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p)
_allocator_refs = []        # every callback pair ever handed over: buffers free through them


def use_torch_allocator(on: bool = True):
    """Take every device buffer that map handles allocate from now on (builds,
    forwards, growth) from torch's caching allocator, on the stream of the call
    that needs it, so that torch's pool holds all of the library's device
    memory; on=False goes back to hipMalloc/hipFree. Buffers keep the
    allocator that made them (smc_set_allocator)."""
    import torch
    L = lib()
    if not on:
        _check(L.smc_set_allocator(None, None, None))
        return

    def _alloc(ctx, nbytes, stream):
        try:
            return torch.cuda.caching_allocator_alloc(int(nbytes), stream=stream or None)
        except Exception:
            return None                # the library reports SMC_ERR_ALLOC

    def _free(ctx, ptr, stream):
        try:
            torch.cuda.caching_allocator_delete(ptr)
        except Exception:
            pass

    fa, ff = _ALLOC_T(_alloc), _FREE_T(_free)
    _allocator_refs.append((fa, ff))
    _check(L.smc_set_allocator(ctypes.cast(fa, ctypes.c_void_p), ctypes.cast(ff, ctypes.c_void_p),
                               None))


def _check(status: int):
    if status != 0:
        L = lib()
        raise SmconvError(status, f"{L.smc_status_string(status).decode()}: "
                                  f"{L.smc_last_error().decode()}")


def _stream(stream):
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _need(t, dtype, name, ndim=None):
    import torch
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA (HIP) torch tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dimensions")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


class PackedWeights:
    """Weights packed for the GEMM; holds the device buffer."""

    def __init__(self, buf, c_in: int, c_out: int, kernel_size: int = 3):
        self.buf, self.c_in, self.c_out, self.kernel_size = buf, c_in, c_out, kernel_size


_KSIZE_OF_TAPS = {27: 3, 125: 5}


def pack_weights(w, out: PackedWeights = None, stream=None) -> PackedWeights:
    """bf16 [K^3, C_in, C_out] CUDA tensor (K = 3 or 5) -> PackedWeights
    (into ``out`` if given)."""
    import torch
    _need(w, torch.bfloat16, "w", 3)
    if int(w.shape[0]) not in _KSIZE_OF_TAPS:
        raise ValueError("w must be [27, C_in, C_out] or [125, C_in, C_out]")
    k = _KSIZE_OF_TAPS[int(w.shape[0])]
    c_in, c_out = int(w.shape[1]), int(w.shape[2])
    L = lib()
    nbytes = L.smc_weight_packed_bytes(k, c_in, c_out)
    if out is not None:
        if (out.c_in, out.c_out, out.kernel_size) != (c_in, c_out, k):
            raise ValueError("out was packed for other channel counts or kernel size")
        buf = out.buf
    else:
        buf = torch.empty(nbytes, dtype=torch.uint8, device=w.device)
    _check(L.smc_weight_pack(ctypes.c_void_p(w.data_ptr()), k, c_in, c_out,
                             ctypes.c_void_p(buf.data_ptr()), _stream(stream)))
    return PackedWeights(buf, c_in, c_out, k)


class KernelMap:
    """A kernel map handle: built from coordinates, reused by every layer."""

    def __init__(self):
        self._h = ctypes.c_void_p()
        _check(lib().smc_map_create(ctypes.byref(self._h)))
        self.n = 0
        self.n_in = 0
        self.kernel_size = 3
        self.strided = False
        self._coords = None

    def close(self):
        """Destroy the handle (waits for its work) and drop the last coordinates."""
        if self._h:
            lib().smc_map_destroy(self._h)
            self._h = ctypes.c_void_p()
        self._coords = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def build(self, coords, spatial_shape=None, batch_size: int = 0, route: str = "auto",
              sync: bool = True, pairs: bool = True, sort: bool = True,
              kernel_size: int = 3, table: bool = False, stream=None) -> "KernelMap":
        """coords: int32 [N, 4] (b, x, y, z) or [N, 3] (x, y, z) CUDA tensor.

        pairs=False skips the per-tap pair lists (algo="pairs" then refuses the
        map); sort=False skips the mask-sorted row order (algo="mask_tiles"
        then refuses it). kernel_size 3 or 5 (a 5x5x5 map has pair lists and
        no mask order). table=True keeps the neighbour table in device memory
        where the build would leave it out (dense route, 3x3x3, pair lists
        without the mask order); export() returns the table either way."""
        import torch
        _need(coords, torch.int32, "coords", 2)
        n, ncols = int(coords.shape[0]), int(coords.shape[1])
        shape = None
        if spatial_shape is not None:
            shape = (ctypes.c_int32 * 3)(*[int(v) for v in spatial_shape])
        flags = ((0 if sync else SMC_BUILD_ASYNC) | (0 if pairs else SMC_BUILD_NO_PAIRS)
                 | (0 if sort else SMC_BUILD_NO_SORT) | (SMC_BUILD_TABLE if table else 0))
        if kernel_size == 5:
            flags |= SMC_BUILD_NO_SORT
        self._coords = coords          # keep alive while the stream reads it
        self.n = self.n_in = n
        self.strided = False
        _check(lib().smc_map_build(self._h, ctypes.c_void_p(coords.data_ptr() if n else 0), n,
                                   ncols, shape, int(batch_size), int(kernel_size), ROUTES[route],
                                   flags, _stream(stream)))
        self.kernel_size = int(kernel_size)
        return self

    def build_strided(self, coords, spatial_shape=None, batch_size: int = 0, route: str = "auto",
                      sync: bool = True, kernel_size: int = 3, stride: int = 2,
                      pairs: bool = True, sort: bool = True, stream=None) -> "KernelMap":
        """Downsampling map (kernel 3, stride 2, padding 1) of int32 [N, 4] / [N, 3]
        CUDA coordinates; outputs are new cells (``out_coords()``), ``n`` of them.
        pairs: per-tap pair lists over the output rows (forward algo "pairs");
        sort: the mask order of the output rows (forward algo "mask_tiles")."""
        import torch
        _need(coords, torch.int32, "coords", 2)
        n, ncols = int(coords.shape[0]), int(coords.shape[1])
        shape = None
        if spatial_shape is not None:
            shape = (ctypes.c_int32 * 3)(*[int(v) for v in spatial_shape])
        self._coords = coords
        self.n, self.n_in, self.strided = 0, n, True
        _check(lib().smc_map_build_strided(
            self._h, ctypes.c_void_p(coords.data_ptr() if n else 0), n, ncols, shape,
            int(batch_size), int(kernel_size), int(stride), ROUTES[route],
            (0 if sync else SMC_BUILD_ASYNC) | (0 if pairs else SMC_BUILD_NO_PAIRS)
            | (0 if sort else SMC_BUILD_NO_SORT), _stream(stream)))
        # the output count: waits for its own event only (the lookup and
        # compaction after it are still running)
        rows = ctypes.c_int64()
        _check(lib().smc_map_rows(self._h, ctypes.byref(rows), None))
        self.n, self.n_in, self.kernel_size, self.strided = rows.value, n, int(kernel_size), True
        return self

    def out_coords(self):
        """Output coordinates of a strided map: numpy int32 [n, 4] (b, x, y, z)."""
        import numpy as np
        out = np.empty((self.n, 4), np.int32)
        _check(lib().smc_map_export_out_coords(
            self._h, ctypes.c_void_p(out.ctypes.data) if out.size else None))
        return out

    def sync(self):
        _check(lib().smc_map_sync(self._h))

    def set_order(self, bit_order=None, group_of=None) -> "KernelMap":
        """Bit order (27 taps, most significant first) and offset groups (group
        of each tap) of the mask sort of later builds; None: plain / one group."""
        arr = {}
        for name, v in (("bit_order", bit_order), ("group_of", group_of)):
            if v is not None:
                v = [int(t) for t in v]
                if len(v) != 27:
                    raise ValueError(f"{name} must have 27 entries")
                arr[name] = (ctypes.c_int32 * 27)(*v)
        _check(lib().smc_map_set_order(self._h, arr.get("bit_order"), arr.get("group_of")))
        return self

    def calibrate(self, n_groups: int = 1):
        """(bit_order, group_of) chosen on this built map (see smc_map_calibrate)."""
        order = (ctypes.c_int32 * 27)()
        groups = (ctypes.c_int32 * 27)()
        _check(lib().smc_map_calibrate(self._h, int(n_groups), order, groups))
        return list(order), list(groups)

    def timing(self, on: bool = True):
        """Record HIP events around each stage of later builds and forwards."""
        _check(lib().smc_timing_enable(self._h, 1 if on else 0))

    def timing_read(self, reset: bool = True) -> dict:
        """{stage: (total_ms, calls)} of the timed work (waits for it)."""
        ms = (ctypes.c_double * len(STAGES))()
        calls = (ctypes.c_int64 * len(STAGES))()
        _check(lib().smc_timing_read(self._h, ms, calls, 1 if reset else 0))
        return {name: (ms[i], calls[i]) for i, name in enumerate(STAGES)}

    def info(self) -> dict:
        inf = MapInfo()
        _check(lib().smc_map_info(self._h, ctypes.byref(inf)))
        return dict(n=inf.n, route=_ROUTE_NAMES.get(inf.route, inf.route), key_bits=inf.key_bits,
                    origin=tuple(inf.origin), extent=tuple(inf.extent), batch=inf.batch,
                    tile_m=inf.tile_m, grid_cells=inf.grid_cells, pairs=inf.pairs,
                    pairs_padded=inf.pairs_padded, n_tiles=inf.n_tiles,
                    tap_count=list(inf.tap_count)[:inf.taps], status=inf.status,
                    n_groups=inf.n_groups, group_rows=list(inf.group_rows)[:inf.n_groups],
                    kernel_size=inf.kernel_size, taps=inf.taps, n_in=inf.n_in,
                    strided=bool(inf.strided), out_extent=tuple(inf.out_extent))

    def export(self, pairs: bool = True, perm: bool = True) -> dict:
        """Copy nbr, mask, tap offsets (and the mask-tile row orders [G, N], the
        pair lists) to numpy (host)."""
        import numpy as np
        info = self.info()
        n, p, taps = info["n"], info["pairs"], info["taps"]
        out = dict(nbr=np.empty((n, taps), np.int32),
                   mask=np.empty(n if taps == 27 else (n, 4), np.uint32),
                   tap_off=np.empty(taps + 1, np.int64))
        if perm:
            out["perm"] = np.empty((max(info["n_groups"], 1), n), np.int32)
            out["group_rows"] = np.asarray(info["group_rows"], np.int64)
        if pairs:
            out["pair_in"] = np.empty(p, np.int32)
            out["pair_out"] = np.empty(p, np.int32)

        def ptr(key):
            a = out.get(key)
            return ctypes.c_void_p(a.ctypes.data) if a is not None and a.size else None
        _check(lib().smc_map_export(self._h, ptr("nbr"), ptr("mask"), ptr("perm"),
                                    ptr("pair_in"), ptr("pair_out"), ptr("tap_off")))
        return out

    def forward(self, x, w: PackedWeights, relu: bool = False, out=None, out_f32: bool = False,
                algo: str = "pairs", stream=None):
        """x: bf16 [N, C_in] CUDA tensor -> bf16 [N, C_out] (float32 with out_f32).

        algo: "pairs" (per-tap pair lists: each row is its centre product plus
        its partial-product slab rows; one kernel with the slab in LDS for
        3x3x3 maps and C_in, C_out <= 64 (C_in a multiple of 8), else two kernels with the
        slab in device memory), "pairs_slab" (always the two-kernel form) or
        "mask_tiles" (output-stationary tiles of mask-sorted rows)."""
        if algo not in ALGOS:
            raise ValueError(f"algo must be one of {ALGOS}")
        import torch
        _need(x, torch.bfloat16, "x", 2)
        if x.shape[0] != self.n_in:
            raise ValueError(f"x has {x.shape[0]} rows, the map has {self.n_in} inputs")
        if x.shape[1] != w.c_in:
            raise ValueError(f"x has {x.shape[1]} channels, weights expect {w.c_in}")
        if w.kernel_size != self.kernel_size:
            raise ValueError(f"weights are {w.kernel_size}^3, the map is {self.kernel_size}^3")
        odt = torch.float32 if out_f32 else torch.bfloat16
        if out is None:
            out = torch.empty((self.n, w.c_out), dtype=odt, device=x.device)
        else:
            _need(out, odt, "out", 2)
            if tuple(out.shape) != (self.n, w.c_out):
                raise ValueError("out has the wrong shape")
        _check(lib().smc_conv_forward(self._h, ctypes.c_void_p(x.data_ptr()), w.c_in,
                                      ctypes.c_void_p(w.buf.data_ptr()), w.c_out,
                                      ctypes.c_void_p(out.data_ptr()),
                                      (SMC_FWD_RELU if relu else 0)
                                      | (SMC_FWD_OUT_F32 if out_f32 else 0)
                                      | (SMC_FWD_MASK_TILES if algo == "mask_tiles" else 0)
                                      | (SMC_FWD_SLAB_IN_MEMORY if algo == "pairs_slab" else 0),
                                      _stream(stream)))
        return out


def subm_conv3d(coords, x, w, spatial_shape=None, relu: bool = False, route: str = "auto"):
    """One layer from raw inputs: builds a map (kernel size from w: 27 or 125
    taps), packs w, runs the layer."""
    wp = pack_weights(w)
    m = KernelMap().build(coords, spatial_shape=spatial_shape, route=route,
                          kernel_size=wp.kernel_size)
    return m.forward(x, wp, relu=relu)


# ---- row operators ------------------------------------------------------------
# Like the convolution they are not connected to autograd: results are detached, also
# where an input requires gradients; the _backward functions give the gradients.

ACTIVATIONS = {None: 0, "none": 0, "relu": 1, "silu": 2, "gelu": 3}


def _dtype_code(t, name):
    import torch
    dtype = t.dtype if isinstance(t, torch.Tensor) else t
    if dtype == torch.bfloat16:
        return 0
    if dtype == torch.float16:
        return 1
    raise TypeError(f"{name} must be bfloat16 or float16, got {dtype}")


def _of(t, name, dtype, device):
    import torch
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA (HIP) torch tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, not on {device}")


def _rows(t, name, dtype, device, shape=None):
    """A 2-D CUDA tensor's (address, row distance in elements): the elements of
    a row must be adjacent, rows may lie any distance apart without overlap."""
    _of(t, name, dtype, device)
    size = t.shape
    if len(size) != 2 or (shape is not None and size != shape):
        raise ValueError(f"{name} must be {list(shape) if shape else '2-dimensional'}, "
                         f"got {list(size)}")
    n, c = size
    ld, step = t.stride()
    if c > 1 and step != 1:
        raise ValueError(f"{name}: the elements of a row must be adjacent")
    if n <= 1:
        ld = c
    elif ld < c:
        raise ValueError(f"{name}: rows overlap (row distance {ld} < {c})")
    return t.data_ptr(), ld


def _vector(t, name, dtype, device, size):
    _of(t, name, dtype, device)
    if t.shape != (size,) or (size > 1 and t.stride(0) != 1):
        raise ValueError(f"{name} must be contiguous [{size}], got {list(t.shape)}")
    return t.data_ptr()


def _elsewhere(x, stream):
    """None where a call runs as it stands, on x's device and its current
    stream; else the context to run it in, so that outputs and scratch memory
    belong to the stream that runs the kernels."""
    import torch
    if not isinstance(x, torch.Tensor) or not x.is_cuda:
        raise TypeError("x must be a CUDA (HIP) torch tensor")
    if x.dim() != 2:
        raise ValueError(f"x must be 2-dimensional, got {list(x.shape)}")
    if stream is not None:
        if stream.device != x.device:
            raise ValueError(f"stream is on {stream.device}, x on {x.device}")
        return torch.cuda.stream(stream)                    # switches the device too
    if torch._C._cuda_getDevice() != x.device.index:
        return torch.cuda.device(x.device.index)
    return None


def _raw_stream(device):
    import torch
    return torch._C._cuda_getCurrentRawStream(device.index)


def rms_norm(x, weight, residual=None, eps: float = 1e-6, e4m3: bool = False, stream=None):
    """s = x + residual (or x); y = s / sqrt(mean(s^2) + eps) * weight, per row.

    x, residual: bf16 or f16 [N, C] CUDA tensors (rows may be strided), weight
    [C]. Returns y; with a residual (y, s), s the new residual stream. e4m3:
    (q, scale) in y's place, q float8_e4m3fn [N, C] and scale float32 [N] with
    y = q * scale[:, None], as linear and gated take them."""
    import torch
    ctx = _elsewhere(x, stream)
    if ctx is not None:
        with ctx:
            return rms_norm(x, weight, residual, eps, e4m3)
    dev, dt = x.device, x.dtype
    code = _dtype_code(x, "x")
    n, c = x.shape
    xp, ldx = _rows(x, "x", dt, dev)
    rp, ldr, s = None, 0, None
    wp = _vector(weight, "weight", dt, dev, c)
    if residual is not None:
        rp, ldr = _rows(residual, "residual", dt, dev, (n, c))
        s = x.new_empty((n, c))
    y = x.new_empty((n, c), dtype=torch.float8_e4m3fn) if e4m3 else x.new_empty((n, c))
    scale = x.new_empty(n, dtype=torch.float32) if e4m3 else None
    _check(lib().smc_rms_norm(NormArgs(
        n, c, code, eps, xp, ldx, rp, ldr, wp, y.data_ptr(), c,
        scale.data_ptr() if e4m3 and n else None, s.data_ptr() if s is not None else None, c),
        _raw_stream(dev)))
    out = ((y, scale) if e4m3 else (y,)) + ((s,) if s is not None else ())
    return out if len(out) > 1 else y


def rms_norm_backward(dy, s, weight, eps: float = 1e-6, ds=None, stream=None):
    """Gradients of rms_norm: (dx, dweight). s: the rows that were normalised
    (rms_norm's s, or x without a residual); ds: the gradient that reaches s by
    other paths, added to dx. dx is the gradient of x and of the residual."""
    import torch
    ctx = _elsewhere(s, stream)
    if ctx is not None:
        with ctx:
            return rms_norm_backward(dy, s, weight, eps, ds)
    dev, dt = s.device, s.dtype
    code = _dtype_code(s, "s")
    n, c = s.shape
    sp, lds = _rows(s, "s", dt, dev)
    dyp, lddy = _rows(dy, "dy", dt, dev, (n, c))
    wp = _vector(weight, "weight", dt, dev, c)
    dsp, ldds = _rows(ds, "ds", dt, dev, (n, c)) if ds is not None else (None, 0)
    L = lib()
    dx = s.new_empty((n, c))
    dweight = s.new_empty(c)
    nbytes = L.smc_rms_norm_backward_workspace(n, c)
    ws = s.new_empty(nbytes, dtype=torch.uint8)
    _check(L.smc_rms_norm_backward(NormBackwardArgs(
        n, c, code, eps, dyp, lddy, sp, lds, wp, dsp, ldds, dx.data_ptr(), c,
        dweight.data_ptr(), ws.data_ptr(), nbytes), _raw_stream(dev)))
    return dx, dweight


def _activation(name):
    if name not in ACTIVATIONS:
        raise ValueError(f"activation must be one of {[a for a in ACTIVATIONS if a]} or None")
    return ACTIVATIONS[name]


def _product_args(halves, x, w, bias, activation, x_scale, w_scale, dtype, backward=False):
    """(args with the shared fields, output dtype, output shape) of a linear or gated layer."""
    import torch
    act = _activation(activation)
    dev = x.device
    e4m3 = x.dtype == torch.float8_e4m3fn
    dt = (torch.bfloat16 if dtype is None else dtype) if e4m3 else x.dtype
    if not e4m3 and (dtype not in (None, dt) or x_scale is not None or w_scale is not None):
        raise ValueError("dtype and scales are for e4m3 rows")
    code = _dtype_code(dt, "dtype" if e4m3 else "x")
    n, c_in = x.shape
    xp, ldx = _rows(x, "x", x.dtype, dev)
    along = e4m3 and (w.dim() != 2 or w.stride(1) == 1)     # else [c_in, c_out] in memory
    wp, ldw = _rows(w.t() if e4m3 and not along else w, "w", x.dtype, dev)
    if w.shape[1 if e4m3 else 0] != c_in:
        raise ValueError(f"w is {list(w.shape)}, x has {c_in} channels "
                         f"(e4m3 weights are [c_out, c_in])")
    wide = w.shape[0 if e4m3 else 1]
    if wide % halves or wide == 0:
        raise ValueError(f"a gated layer's w holds two halves, got {wide} columns")
    xsp = wsp = None
    if e4m3 and not backward:          # the library refuses gradients of e4m3 layers
        xsp = _vector(x_scale, "x_scale", torch.float32, dev, n) if n else None
        wsp = _vector(w_scale, "w_scale", torch.float32, dev, wide)
    bp = _vector(bias, "bias", dt, dev, wide) if bias is not None else None
    return ProductArgs(n, c_in, wide // halves, code, 2 if e4m3 else code, act, xp, ldx, xsp, wp, ldw,
                       along, wsp, bp), dt, (n, wide // halves)


def _product_out(a, x, out, dt, shape):
    if out is None:
        out = x.new_empty(shape, dtype=dt)
        a.y, a.ldy = out.data_ptr(), shape[1]
    else:
        a.y, a.ldy = _rows(out, "out", dt, x.device, shape)
    return out


def _product_forward(halves, a, x):
    import torch
    L = lib()
    need, call = ((L.smc_linear_workspace, L.smc_linear) if halves == 1 else
                  (L.smc_gated_workspace, L.smc_gated))
    # rows that are not whole 16-byte words: room for padded copies of them
    if (a.ldx | a.ldw | a.c_in | a.c_out) & (15 if a.x_dtype == 2 else 7) or ((a.x or 0) | a.w) & 15:
        nbytes = need(a)
        if nbytes:
            ws = x.new_empty(nbytes, dtype=torch.uint8)
            a.workspace, a.workspace_bytes = ws.data_ptr(), nbytes
    _check(call(a, _raw_stream(x.device)))


def linear(x, w, bias=None, residual=None, activation=None, x_scale=None, w_scale=None, dtype=None,
           out=None, stream=None):
    """y = activation(x @ w + bias) + residual in one kernel.

    x: bf16 or f16 [N, C_in] CUDA tensor, w: [C_in, C_out] (rows of both may be
    strided), bias [C_out], residual [N, C_out]; activation None, "relu",
    "silu" or "gelu" (erf). Served in 8 bits: x float8_e4m3fn with x_scale [N]
    (rms_norm's e4m3 output), w float8_e4m3fn [C_out, C_in] with w_scale [C_out]
    (quantize_weight; its transpose's memory order is taken too), y of `dtype`
    (default bf16). out may be the residual, not x."""
    ctx = _elsewhere(x, stream)
    if ctx is not None:
        with ctx:
            return linear(x, w, bias, residual, activation, x_scale, w_scale, dtype, out)
    a, dt, shape = _product_args(1, x, w, bias, activation, x_scale, w_scale, dtype)
    if residual is not None:
        a.residual, a.ld_residual = _rows(residual, "residual", dt, x.device, shape)
    out = _product_out(a, x, out, dt, shape)
    _product_forward(1, a, x)
    return out


def gated(x, w, bias=None, activation="silu", x_scale=None, w_scale=None, dtype=None, out=None,
          stream=None):
    """h = activation(x @ wg + bias_g) * (x @ wu + bias_u) in one kernel, with
    w = [wg | wu] [C_in, 2 C_out] and bias [2 C_out]. Types and the 8-bit form
    as in linear (e4m3 w: [2 C_out, C_in], the gate's rows first)."""
    ctx = _elsewhere(x, stream)
    if ctx is not None:
        with ctx:
            return gated(x, w, bias, activation, x_scale, w_scale, dtype, out)
    a, dt, shape = _product_args(2, x, w, bias, activation, x_scale, w_scale, dtype)
    out = _product_out(a, x, out, dt, shape)
    _product_forward(2, a, x)
    return out


def _product_backward(halves, dy, x, w, bias, activation, stream):
    import torch
    ctx = _elsewhere(x, stream)
    if ctx is not None:
        with ctx:
            return _product_backward(halves, dy, x, w, bias, activation, None)
    a, dt, (n, c_out) = _product_args(halves, x, w, bias, activation, None, None, None, True)
    dev, c_in, wide = x.device, x.shape[1], c_out * halves
    a.dy, a.ld_dy = _rows(dy, "dy", dt, dev, (n, c_out))
    dx = x.new_empty((n, c_in))
    dw = x.new_empty((c_in, wide))
    db = x.new_empty(wide) if bias is not None else None
    a.dx, a.ld_dx, a.dw, a.ld_dw = dx.data_ptr(), c_in, dw.data_ptr(), wide
    a.db = db.data_ptr() if db is not None else None
    L = lib()
    need, call = ((L.smc_linear_backward_workspace, L.smc_linear_backward) if halves == 1 else
                  (L.smc_gated_backward_workspace, L.smc_gated_backward))
    nbytes = need(a)
    ws = x.new_empty(nbytes, dtype=torch.uint8)
    a.workspace, a.workspace_bytes = ws.data_ptr(), nbytes
    _check(call(a, _raw_stream(dev)))
    return dx, dw, db


def linear_backward(dy, x, w, bias=None, activation=None, stream=None):
    """(dx, dw, db) of linear for the gradient dy of its output (db None without
    a bias); the residual's gradient is dy itself. The pre-activations are
    computed again from x, w and bias: nothing of the forward pass is kept."""
    return _product_backward(1, dy, x, w, bias, activation, stream)


def gated_backward(dh, x, w, bias=None, activation="silu", stream=None):
    """(dx, dw, db) of gated for the gradient dh of its output (db None without
    a bias), from x, w and bias alone."""
    return _product_backward(2, dh, x, w, bias, activation, stream)


def quantize_weight(w, stream=None):
    """bf16 or f16 w [C_in, C_out] -> (float8_e4m3fn [C_out, C_in], float32 scale
    [C_out]) for linear and gated on e4m3 rows; scale[j] = max |w[:, j]| / 448."""
    import torch
    ctx = _elsewhere(w, stream)
    if ctx is not None:
        with ctx:
            return quantize_weight(w)
    code = _dtype_code(w, "w")
    c_in, c_out = w.shape
    wp, ldw = _rows(w, "w", w.dtype, w.device)
    q = torch.empty((c_out, c_in), dtype=torch.float8_e4m3fn, device=w.device)
    scale = torch.empty(c_out, dtype=torch.float32, device=w.device)
    _check(lib().smc_weight_quantize(wp, ldw, c_in, c_out, code, q.data_ptr(), c_in,
                                     scale.data_ptr(), _raw_stream(w.device)))
    return q, scale


# ---- operators that mix rows ---------------------------------------------------


def _group_args(x, weight, bias, groups, offsets, eps, activation):
    import torch
    act = _activation(activation)
    dev, dt = x.device, x.dtype
    code = _dtype_code(x, "x")
    n, c = x.shape
    xp, ldx = _rows(x, "x", dt, dev)
    if groups < 1 or c % groups:
        raise ValueError(f"{c} channels in {groups} groups")
    op, samples = None, 1
    if offsets is not None:
        if offsets.dim() != 1 or offsets.shape[0] < 2:
            raise ValueError(f"offsets must be [samples + 1], got {list(offsets.shape)}")
        op, samples = _vector(offsets, "offsets", torch.int32, dev, offsets.shape[0]), offsets.shape[0] - 1
    return GroupNormArgs(n, c, groups, samples, code, act, eps, op, xp, ldx,
                         _vector(weight, "weight", dt, dev, c), _vector(bias, "bias", dt, dev, c))


def group_norm(x, weight, bias, groups: int, offsets=None, eps: float = 1e-5, activation=None,
               stats: bool = False, stream=None):
    """y = activation((x - mean) / sqrt(var + eps) * weight + bias), mean and variance
    over the rows of each sample and the channels of each of `groups` groups.

    x: bf16 or f16 [N, C] CUDA tensor (rows may be strided), weight and bias [C],
    offsets: int32 [samples + 1] CUDA tensor, sample s being the rows offsets[s] ..
    offsets[s + 1] - 1 (None: one sample of all rows; rows of no sample come out as
    zeros); activation as in linear. With stats (y, stats), stats float32 [samples,
    groups, 2] (mean, 1 / sqrt(var + eps)), as group_norm_backward takes it."""
    import torch
    ctx = _elsewhere(x, stream)
    if ctx is not None:
        with ctx:
            return group_norm(x, weight, bias, groups, offsets, eps, activation, stats)
    a = _group_args(x, weight, bias, groups, offsets, eps, activation)
    L = lib()
    y = x.new_empty((a.n, a.c))
    a.y, a.ldy = y.data_ptr(), a.c
    if stats:
        kept = x.new_empty((a.samples, groups, 2), dtype=torch.float32)
        a.stats = kept.data_ptr()
    nbytes = L.smc_group_norm_workspace(a)
    ws = x.new_empty(nbytes, dtype=torch.uint8)
    a.workspace, a.workspace_bytes = ws.data_ptr(), nbytes
    _check(L.smc_group_norm(a, _raw_stream(x.device)))
    return (y, kept) if stats else y


def group_norm_backward(dy, x, weight, bias, groups: int, stats, offsets=None, activation=None,
                        stream=None):
    """Gradients of group_norm for the gradient dy of its output: (dx, dweight,
    dbias). stats: what group_norm returned for the same x, groups and offsets."""
    import torch
    ctx = _elsewhere(x, stream)
    if ctx is not None:
        with ctx:
            return group_norm_backward(dy, x, weight, bias, groups, stats, offsets, activation)
    a = _group_args(x, weight, bias, groups, offsets, 0.0, activation)
    L = lib()
    dev, dt, shape = x.device, x.dtype, (a.n, a.c)
    a.dy, a.ld_dy = _rows(dy, "dy", dt, dev, shape)
    _of(stats, "stats", torch.float32, dev)
    if stats.shape != (a.samples, groups, 2) or not stats.is_contiguous():
        raise ValueError(f"stats must be contiguous {[a.samples, groups, 2]}, got {list(stats.shape)}")
    a.stats = stats.data_ptr()
    dx, dweight, dbias = x.new_empty(shape), x.new_empty(a.c), x.new_empty(a.c)
    a.dx, a.ld_dx, a.dweight, a.dbias = dx.data_ptr(), a.c, dweight.data_ptr(), dbias.data_ptr()
    nbytes = L.smc_group_norm_backward_workspace(a)
    ws = x.new_empty(nbytes, dtype=torch.uint8)
    a.workspace, a.workspace_bytes = ws.data_ptr(), nbytes
    _check(L.smc_group_norm_backward(a, _raw_stream(dev)))
    return dx, dweight, dbias


class Windows:
    """The windows that window_attention works in, made once for all layers on the
    same rows (waits for the device once).

    order: int32 [N] CUDA tensor, every row once, window after window (None: the rows as
    they lie); window w is the places offsets[w] .. offsets[w + 1] - 1 of it (int32
    [windows + 1] CUDA tensor); places of no window may be left at both ends. For a
    relative position bias: coords, the rows' int32 [N, 4] (b, x, y, z) or [N, 3]
    coordinates, and extent, how many cells a window spans along x, y and z at most (each
    rounded up to a multiple of 4, 128 in all). SmconvError where a row is listed twice, an
    offset or row is out of range or a window is larger than that. The tensors are not read
    again; the object has to outlive the calls that it is used in on other streams."""

    def __init__(self, offsets, n: int, order=None, coords=None, extent=None, stream=None):
        import torch
        if not isinstance(offsets, torch.Tensor) or not offsets.is_cuda:
            raise TypeError("offsets must be a CUDA (HIP) torch tensor")
        dev = offsets.device
        if offsets.dim() != 1 or offsets.shape[0] < 1:
            raise ValueError(f"offsets must be [windows + 1], got {list(offsets.shape)}")
        if stream is not None and stream.device != dev:
            raise ValueError(f"stream is on {stream.device}, offsets on {dev}")
        if (coords is None) != (extent is None):
            raise ValueError("coords and extent come together")
        with torch.cuda.stream(stream) if stream is not None else torch.cuda.device(dev):
            a = WindowsArgs(int(n), offsets.shape[0] - 1,
                            _vector(offsets, "offsets", torch.int32, dev, offsets.shape[0]))
            if order is not None:
                a.order = _vector(order, "order", torch.int32, dev, a.n)
            if coords is not None:
                _need(coords, torch.int32, "coords", 2)
                if coords.device != dev or coords.shape[0] != a.n or coords.shape[1] not in (3, 4):
                    raise ValueError(f"coords must be [{a.n}, 3 or 4] on {dev}, got {list(coords.shape)}")
                a.coords, a.coord_cols = coords.data_ptr(), coords.shape[1]
                a.ex, a.ey, a.ez = (int(e) for e in extent)
            a.plan_bytes = lib().smc_windows_bytes(a.n, a.windows)
            self._plan = torch.empty(a.plan_bytes, dtype=torch.uint8, device=dev)
            a.plan = self._plan.data_ptr()
            _check(lib().smc_windows_build(a, _raw_stream(dev)))
        a.offsets = a.order = a.coords = None
        self._args, self.device, self.n = a, dev, a.n
        self.longest = a.longest


def _attention_args(q, k, v, windows, heads, bias, scale):
    dev, dt = q.device, q.dtype
    code = _dtype_code(q, "q")
    n, c = q.shape
    if not isinstance(windows, Windows):
        raise TypeError("windows must be a Windows")
    if windows.device != dev or windows.n != n:
        raise ValueError(f"windows are of {windows.n} rows on {windows.device}, q has {n} on {dev}")
    if heads < 1 or c < 1 or c % heads:
        raise ValueError(f"{c} channels in {heads} heads")
    dim = c // heads
    if k.dim() != 2 or k.shape[1] < dim or k.shape[1] % dim or heads % (k.shape[1] // dim):
        raise ValueError(f"k is {list(k.shape)}, heads are {heads} of {dim}")
    qp, ldq = _rows(q, "q", dt, dev)
    kp, ldk = _rows(k, "k", dt, dev, (n, k.shape[1]))
    vp, ldv = _rows(v, "v", dt, dev, (n, k.shape[1]))
    bp, reach = None, 0
    if bias is not None:
        _of(bias, "bias", dt, dev)
        if bias.dim() != 3 or bias.shape[0] != 3 or bias.shape[1] % 2 == 0 or bias.shape[2] != heads \
                or not bias.is_contiguous():
            raise ValueError(f"bias must be contiguous [3, 2 reach + 1, {heads}], got {list(bias.shape)}")
        if windows._args.ex == 0:
            raise ValueError("a bias needs windows with coords")
        bp, reach = bias.data_ptr(), bias.shape[1] // 2
    return AttentionArgs(ctypes.pointer(windows._args), heads, k.shape[1] // dim, dim, code,
                         dim ** -0.5 if scale is None else scale, reach, bp, qp, ldq, kp, ldk, vp, ldv)


def window_attention(q, k, v, windows: Windows, heads: int, bias=None, scale=None, lse: bool = False,
                     out=None, stream=None):
    """out_i = sum over the rows j of i's window of softmax_j(scale q_i k_j + bias_ij) v_j,
    head by head.

    q: bf16 or f16 [N, heads D] CUDA tensor, k and v [N, kv_heads D] with kv_heads dividing
    heads (rows of all may be strided, such as columns of one projection's output), D up to
    128; scale: D ** -0.5 by default. bias: a learned table [3, 2 reach + 1, heads], bias_ij
    the sum over the axes of bias[axis, reach + clamp(c_i - c_j, -reach, reach)] with c the
    windows' coords. Rows of no window come out as zeros. With lse (out, lse), lse float32
    [heads, N] by place of the window order, as window_attention_backward takes it."""
    import torch
    ctx = _elsewhere(q, stream)
    if ctx is not None:
        with ctx:
            return window_attention(q, k, v, windows, heads, bias, scale, lse, out)
    a = _attention_args(q, k, v, windows, heads, bias, scale)
    n, c = q.shape
    if out is None:
        out = q.new_empty((n, c))
        a.out, a.ld_out = out.data_ptr(), c
    else:
        a.out, a.ld_out = _rows(out, "out", q.dtype, q.device, (n, c))
    if lse:
        kept = q.new_empty((heads, n), dtype=torch.float32)
        a.lse = kept.data_ptr()
    _check(lib().smc_window_attention(a, _raw_stream(q.device)))
    return (out, kept) if lse else out


def window_attention_backward(dout, q, k, v, out, lse, windows: Windows, heads: int, bias=None,
                              scale=None, grads=None, stream=None):
    """Gradients of window_attention for the gradient dout of its output: (dq, dk,
    dv, dbias), dbias None without a bias. out and lse: what window_attention returned for
    the same inputs. grads: (dq, dk, dv) to write to, which may be columns of one buffer
    (the gradient of a projection's output)."""
    import torch
    ctx = _elsewhere(q, stream)
    if ctx is not None:
        with ctx:
            return window_attention_backward(dout, q, k, v, out, lse, windows, heads, bias, scale, grads)
    a = _attention_args(q, k, v, windows, heads, bias, scale)
    dev, dt, n = q.device, q.dtype, q.shape[0]
    a.dout, a.ld_dout = _rows(dout, "dout", dt, dev, q.shape)
    a.out, a.ld_out = _rows(out, "out", dt, dev, q.shape)
    _of(lse, "lse", torch.float32, dev)
    if lse.shape != (heads, n) or not lse.is_contiguous():
        raise ValueError(f"lse must be contiguous {[heads, n]}, got {list(lse.shape)}")
    a.lse = lse.data_ptr()
    dq, dk, dv = grads if grads is not None else (q.new_empty(t.shape) for t in (q, k, v))
    a.dq, a.ld_dq = _rows(dq, "dq", dt, dev, q.shape)
    a.dk, a.ld_dk = _rows(dk, "dk", dt, dev, k.shape)
    a.dv, a.ld_dv = _rows(dv, "dv", dt, dev, v.shape)
    dbias = None
    if bias is not None:
        dbias = torch.empty_like(bias)
        a.dbias = dbias.data_ptr()
    L = lib()
    nbytes = L.smc_window_attention_backward_workspace(a)
    ws = q.new_empty(nbytes, dtype=torch.uint8)
    a.workspace, a.workspace_bytes = ws.data_ptr(), nbytes
    _check(L.smc_window_attention_backward(a, _raw_stream(dev)))
    return dq, dk, dv, dbias


def probe_mfma_bf16(iters: int, stream=None) -> float:
    """Enqueue the MFMA-only probe kernel on the stream; returns the flops it
    executes (the caller times it)."""
    import torch
    L = lib()
    n_cu = torch.cuda.get_device_properties(torch.cuda.current_device()).multi_processor_count
    nbytes = L.smc_probe_mfma_out_bytes(n_cu)
    out = torch.empty(nbytes // 4, dtype=torch.float32, device="cuda")
    flops = ctypes.c_double()
    _check(L.smc_probe_mfma_bf16(int(iters), ctypes.c_void_p(out.data_ptr()), nbytes,
                                 ctypes.byref(flops), _stream(stream)))
    probe_mfma_bf16._keep = out          # alive until the stream has run the kernel
    return flops.value


def probe_copy(dst, src, stream=None):
    """dst[:] = src[:] (CUDA tensors of equal byte size) by the library's copy probe."""
    nbytes = src.numel() * src.element_size()
    if dst.numel() * dst.element_size() != nbytes:
        raise ValueError("dst and src differ in size")
    _check(lib().smc_probe_copy(ctypes.c_void_p(dst.data_ptr()), ctypes.c_void_p(src.data_ptr()),
                                nbytes, _stream(stream)))
