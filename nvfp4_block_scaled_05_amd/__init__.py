"""Python binding of the MI355X NVFP4 quantize library (``libnvfp4.so``).

Thin ctypes marshalling over the C ABI declared in ``include/nvfp4.h``; the
functions keep the C names. Every step of the quantize path runs in the
library's HIP kernels; torch only supplies device memory and the current
stream. If the library is missing or cannot be loaded, every call raises:
there is no fallback.

Tensors passed in are torch CUDA tensors (on ROCm, HIP devices):
  x         bfloat16 or float32, 2-D, contiguous
  data      uint8 [n][k/2]      scales  uint8 (compact [n][k/16] or swizzled, flat)
  amax      float32 [1] or [n]
"""

from __future__ import annotations

import contextlib
import ctypes
import dataclasses
import functools
import os
from typing import Optional

import torch

from . import build as _build

_LIB_PATH = _build.LIB

NVFP4_OK = 0
NVFP4_ERR_NULL = 1
NVFP4_ERR_SHAPE = 2
NVFP4_ERR_ALIGN = 3
NVFP4_ERR_UNSUPPORTED = 4
NVFP4_ERR_HIP = 5

NVFP4_IN_BF16 = 0
NVFP4_IN_FP32 = 1

NVFP4_SCALES_COMPACT = 0
NVFP4_SCALES_GEMM_SWIZZLED = 1

NVFP4_SCALE_E4M3 = 0
NVFP4_SCALE_UE5M3 = 1

NVFP4_AMAX_PATH_AUTO = 0
NVFP4_AMAX_PATH_TWO_PASS = 1
NVFP4_AMAX_PATH_SINGLE_PASS = 2

NVFP4_DEBUG_SR = 1
NVFP4_DEBUG_PAIRWISE = 2

NVFP4_MAX_GROUPS = 256
NVFP4_EXPERT_MLP_MAX_SLOTS = 1024

EXPORTED = ("nvfp4_compute_amax", "nvfp4_quantize", "nvfp4_dequantize", "nvfp4_last_error",
            "nvfp4_workspace_bytes", "nvfp4_swizzle_scales", "nvfp4_swizzled_scales_bytes", "nvfp4_quantize_grouped",
            "nvfp4_debug_rht_colwise", "nvfp4_debug_e2m1_pack", "nvfp4_debug_set_wait_ticks",
            "nvfp4_quantize_noalloc", "nvfp4_debug_set_rht_unit", "nvfp4_debug_set_resident_variant",
            "nvfp4_expert_rows", "nvfp4_expert_sort_workspace_bytes", "nvfp4_expert_sort", "nvfp4_expert_gather",
            "nvfp4_expert_combine", "nvfp4_expert_combine_grad", "nvfp4_fp8_pitch", "nvfp4_fp8_quantize",
            "nvfp4_fp8_matmul", "nvfp4_fp8_matmul_grouped", "nvfp4_fp8_matmul_grouped_k",
            "nvfp4_mxfp4_quantize", "nvfp4_mxfp4_dequantize", "nvfp4_mxfp4_matmul", "nvfp4_mxfp4_matmul_grouped",
            "nvfp4_mxfp4_matmul_grouped_k", "nvfp4_expert_mlp_workspace_bytes", "nvfp4_expert_mlp_mxfp4", "nvfp4_expert_mlp_fp8")


class nvfp4_out_t(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("amax", ctypes.c_void_p)]


class nvfp4_fp8_t(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("scales", ctypes.c_void_p)]


class nvfp4_mxfp4_t(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("scales", ctypes.c_void_p)]


class nvfp4_config_t(ctypes.Structure):
    _fields_ = [
        ("block_2d", ctypes.c_uint32),
        ("scale_layout", ctypes.c_uint32),
        ("scale_fmt", ctypes.c_uint32),
        ("stochastic", ctypes.c_uint32),
        ("sr_seed", ctypes.c_uint32),
        ("row_scaled", ctypes.c_uint32),
        ("rht", ctypes.c_uint32),
        ("rht_sign_mask", ctypes.c_uint32),
        ("rht_bf16", ctypes.c_uint32),
        ("compute_amax", ctypes.c_uint32),
        ("noop", ctypes.c_void_p),
        ("workspace", ctypes.c_void_p),
        ("cast_events", ctypes.c_void_p),
        ("amax_path", ctypes.c_uint32),
    ]


class NVFP4Error(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"nvfp4 status {status}: {message}")
        self.status = status


_lib = None


def library_path() -> str:
    return _LIB_PATH


def load(build_if_missing: bool = True) -> ctypes.CDLL:
    """Load libnvfp4.so (building it first only when it does not exist)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(_LIB_PATH):
        if not build_if_missing:
            raise RuntimeError(f"{_LIB_PATH} is not built")
        _build.build()
    lib = ctypes.CDLL(_LIB_PATH)
    P = ctypes.c_void_p
    I64 = ctypes.c_int64
    U32 = ctypes.c_uint32
    I = ctypes.c_int
    lib.nvfp4_compute_amax.restype = I
    lib.nvfp4_compute_amax.argtypes = [P, I, I64, I64, P, P, ctypes.POINTER(nvfp4_config_t), P]
    lib.nvfp4_quantize.restype = I
    lib.nvfp4_quantize.argtypes = [P, I, I64, I64, ctypes.POINTER(nvfp4_out_t), ctypes.POINTER(nvfp4_out_t),
                                   ctypes.POINTER(nvfp4_config_t), P]
    lib.nvfp4_quantize_noalloc.restype = I
    lib.nvfp4_quantize_noalloc.argtypes = lib.nvfp4_quantize.argtypes
    lib.nvfp4_dequantize.restype = I
    lib.nvfp4_dequantize.argtypes = [ctypes.POINTER(nvfp4_out_t), I64, I64, U32, U32, U32, P, P]
    lib.nvfp4_last_error.restype = ctypes.c_char_p
    lib.nvfp4_last_error.argtypes = []
    lib.nvfp4_workspace_bytes.restype = ctypes.c_uint64
    lib.nvfp4_workspace_bytes.argtypes = []
    lib.nvfp4_quantize_grouped.restype = I
    lib.nvfp4_quantize_grouped.argtypes = [P, I, I64, ctypes.POINTER(ctypes.c_int64), I64,
                                           ctypes.POINTER(nvfp4_out_t), ctypes.POINTER(nvfp4_out_t),
                                           ctypes.POINTER(nvfp4_config_t), P]
    lib.nvfp4_swizzle_scales.restype = I
    lib.nvfp4_swizzle_scales.argtypes = [P, I64, I64, P, P]
    lib.nvfp4_swizzled_scales_bytes.restype = ctypes.c_uint64
    lib.nvfp4_swizzled_scales_bytes.argtypes = [I64, I64]
    lib.nvfp4_debug_rht_colwise.restype = I
    lib.nvfp4_debug_rht_colwise.argtypes = [P, I, I64, I64, U32, P, P]
    lib.nvfp4_debug_e2m1_pack.restype = I
    lib.nvfp4_debug_e2m1_pack.argtypes = [P, P, P, I64, U32, P]
    lib.nvfp4_debug_set_wait_ticks.restype = I
    lib.nvfp4_debug_set_wait_ticks.argtypes = [U32]
    lib.nvfp4_debug_set_rht_unit.restype = I
    lib.nvfp4_debug_set_rht_unit.argtypes = [U32]
    lib.nvfp4_debug_set_resident_variant.restype = I
    lib.nvfp4_debug_set_resident_variant.argtypes = [U32]
    FP8 = ctypes.POINTER(nvfp4_fp8_t)
    lib.nvfp4_expert_rows.restype = ctypes.c_uint64
    lib.nvfp4_expert_rows.argtypes = [I64, I64, I64, I64]
    lib.nvfp4_expert_sort_workspace_bytes.restype = ctypes.c_uint64
    lib.nvfp4_expert_sort_workspace_bytes.argtypes = [I64, I64, I64]
    lib.nvfp4_expert_sort.restype = I
    lib.nvfp4_expert_sort.argtypes = [P, U32, I64, I64, I64, I64, I64, P, P, P, P, P, P]
    lib.nvfp4_expert_gather.restype = I
    lib.nvfp4_expert_gather.argtypes = [P, I, I64, I64, I64, P, P, I64, P, P]
    lib.nvfp4_expert_combine.restype = I
    lib.nvfp4_expert_combine.argtypes = [P, I, I64, I64, I64, P, I64, P, P, P]
    lib.nvfp4_expert_combine_grad.restype = I
    lib.nvfp4_expert_combine_grad.argtypes = [P, P, I, I64, I64, I64, P, P, I64, P, P, P, P]
    lib.nvfp4_fp8_pitch.restype = ctypes.c_uint64
    lib.nvfp4_fp8_pitch.argtypes = [I64]
    lib.nvfp4_fp8_quantize.restype = I
    lib.nvfp4_fp8_quantize.argtypes = [P, I, I64, I64, I64, P, I64, I64, U32, FP8, FP8, P]
    lib.nvfp4_fp8_matmul.restype = I
    lib.nvfp4_fp8_matmul.argtypes = [FP8, FP8, I64, I64, I64, U32, P, I, P]
    lib.nvfp4_fp8_matmul_grouped.restype = I
    lib.nvfp4_fp8_matmul_grouped.argtypes = [FP8, FP8, P, I64, I64, I64, I64, P, I, P]
    lib.nvfp4_fp8_matmul_grouped_k.restype = I
    lib.nvfp4_fp8_matmul_grouped_k.argtypes = [FP8, FP8, P, I64, I64, I64, I64, P, I, P]
    MX = ctypes.POINTER(nvfp4_mxfp4_t)
    lib.nvfp4_mxfp4_quantize.restype = I
    lib.nvfp4_mxfp4_quantize.argtypes = [P, I, I64, I64, I64, P, I64, I64, U32, MX, MX, P]
    lib.nvfp4_mxfp4_dequantize.restype = I
    lib.nvfp4_mxfp4_dequantize.argtypes = [MX, I64, I64, I64, P, I, P]
    lib.nvfp4_mxfp4_matmul.restype = I
    lib.nvfp4_mxfp4_matmul.argtypes = [MX, MX, I64, I64, I64, P, I, P]
    lib.nvfp4_mxfp4_matmul_grouped.restype = I
    lib.nvfp4_mxfp4_matmul_grouped.argtypes = [MX, MX, P, I64, I64, I64, I64, P, I, P]
    lib.nvfp4_mxfp4_matmul_grouped_k.restype = I
    lib.nvfp4_mxfp4_matmul_grouped_k.argtypes = [MX, MX, P, I64, I64, I64, I64, P, I, P]
    lib.nvfp4_expert_mlp_workspace_bytes.restype = ctypes.c_uint64
    lib.nvfp4_expert_mlp_workspace_bytes.argtypes = [I64, I64, I64, I64]
    lib.nvfp4_expert_mlp_mxfp4.restype = I
    lib.nvfp4_expert_mlp_mxfp4.argtypes = [P, I64, I64, P, U32, P, I64, I64, MX, MX, I64, U32, P, P, P]
    lib.nvfp4_expert_mlp_fp8.restype = I
    lib.nvfp4_expert_mlp_fp8.argtypes = [P, I64, I64, P, U32, P, I64, I64, FP8, FP8, I64, U32, P, P, P]
    _lib = lib
    return lib


def _check(status: int) -> None:
    if status != NVFP4_OK:
        raise NVFP4Error(status, nvfp4_last_error())


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _dtype_code(x: torch.Tensor) -> int:
    if x.dtype == torch.bfloat16:
        return NVFP4_IN_BF16
    if x.dtype == torch.float32:
        return NVFP4_IN_FP32
    raise TypeError(f"input must be bfloat16 or float32, got {x.dtype}")


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _under(stream, device):
    """The context of a call that was given a stream of its own: torch's, an
    object with its handle in cuda_stream, or the handle."""
    if not isinstance(stream, torch.cuda.Stream):
        handle = int(getattr(stream, "cuda_stream", stream))
        # ExternalStream takes 0, the default stream's handle, for none given and makes a new stream
        stream = torch.cuda.ExternalStream(handle, device) if handle else torch.cuda.default_stream(device)
    return torch.cuda.stream(stream)


def _current_device() -> int:
    # torch.cuda.current_device() without its check for a first use, which a tensor on a GPU has behind it
    return torch._C._cuda_getDevice()


def _elsewhere(stream, device):
    """The context that a call on tensors of `device` enters before it goes on:
    that of its stream, or of the device where that is not the current one (the
    library launches on the current one). None if neither is needed."""
    if stream is not None:
        if getattr(stream, "device", device) != device:
            raise ValueError(f"the stream is on {stream.device}, the tensors on {device}")
        return _under(stream, device)
    return None if _current_device() == device.index else torch.cuda.device(device)


def _on_its_device(call):
    """`call` with the device of its first argument as the current one."""
    @functools.wraps(call)
    def guarded(*args, **kwargs):
        x = args[0] if args else next(iter(kwargs.values()), None)
        t = x if isinstance(x, torch.Tensor) else getattr(x, "data", None)
        index = t.get_device() if isinstance(t, torch.Tensor) else -1  # -1: not on a GPU, which the call refuses
        if index < 0 or index == _current_device():
            return call(*args, **kwargs)
        with torch.cuda.device(index):
            return call(*args, **kwargs)
    return guarded


def _shape2d(x: torch.Tensor):
    if x.dim() != 2 or not x.is_contiguous() or not x.is_cuda:
        raise ValueError("x must be a contiguous 2-D CUDA tensor")
    return x.shape[0], x.shape[1]


# The C ABI takes plain pointers and cannot see buffer sizes; the binding
# checks every tensor it passes against what the call will touch.
def _need(t: Optional[torch.Tensor], n: int, dtypes, what: str) -> None:
    dtypes = dtypes if isinstance(dtypes, tuple) else (dtypes,)
    if t is None or not t.is_cuda or not t.is_contiguous() or t.dtype not in dtypes or t.numel() < n:
        raise ValueError(f"{what} must be a contiguous CUDA tensor of {'/'.join(str(d) for d in dtypes)} "
                         f"with at least {n} elements")


def _need_orientation(o, n: int, k: int, amax_len: int, what: str) -> None:
    if o is None:
        return
    _need(o.data, n * k // 2, torch.uint8, f"{what} data")
    _need(o.scales, n * k // 16, torch.uint8, f"{what} scales")
    _need(o.amax, amax_len, torch.float32, f"{what} amax")


def make_config(*, block_2d=False, swizzled=False, scale_fmt=NVFP4_SCALE_E4M3, stochastic=False, sr_seed=0,
                row_scaled=False, rht=False, rht_sign_mask=0, compute_amax=True,
                noop: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                rht_bf16=False, amax_path=0) -> nvfp4_config_t:
    """The config struct. It holds references to the noop and workspace
    tensors (a copy made with from_buffer_copy does not: keep them alive
    while such a copy is used)."""
    if noop is not None:
        _need(noop, 1, torch.float32, "noop")
    if workspace is not None and (not workspace.is_cuda or not workspace.is_contiguous()
                                  or workspace.numel() * workspace.element_size() < nvfp4_workspace_bytes()):
        raise ValueError(f"workspace must be contiguous CUDA memory of at least {nvfp4_workspace_bytes()} bytes")
    cfg = nvfp4_config_t(int(block_2d), NVFP4_SCALES_GEMM_SWIZZLED if swizzled else NVFP4_SCALES_COMPACT,
                         int(scale_fmt), int(stochastic), int(sr_seed) & 0xFFFFFFFF, int(row_scaled), int(rht),
                         int(rht_sign_mask) & 0xFFFFFFFF, int(rht_bf16), int(compute_amax),
                         None if noop is None else noop.data_ptr(),
                         None if workspace is None else workspace.data_ptr())
    cfg.amax_path = int(amax_path)
    cfg._tensors = (noop, workspace)
    return cfg


@dataclasses.dataclass
class Orientation:
    """One orientation of an NVFP4 tensor: data [n][k/2], scales, amax."""
    data: torch.Tensor
    scales: torch.Tensor
    amax: torch.Tensor

    def as_c(self) -> nvfp4_out_t:
        return nvfp4_out_t(self.data.data_ptr(), self.scales.data_ptr(), self.amax.data_ptr())


def nvfp4_last_error() -> str:
    return load().nvfp4_last_error().decode()


def nvfp4_workspace_bytes() -> int:
    return int(load().nvfp4_workspace_bytes())


@_on_its_device
def nvfp4_compute_amax(x: torch.Tensor, row_amax: Optional[torch.Tensor], col_amax: Optional[torch.Tensor],
                       cfg: Optional[nvfp4_config_t] = None, stream=None) -> None:
    rows, cols = _shape2d(x)
    if row_amax is not None:
        _need(row_amax, rows if (cfg is not None and cfg.row_scaled) else 1, torch.float32, "row_amax")
    if col_amax is not None:
        _need(col_amax, cols if (cfg is not None and cfg.row_scaled) else 1, torch.float32, "col_amax")
    _check(load().nvfp4_compute_amax(_ptr(x), _dtype_code(x), rows, cols, _ptr(row_amax), _ptr(col_amax),
                                     None if cfg is None else ctypes.byref(cfg), _stream(stream)))


@_on_its_device
def nvfp4_quantize(x: torch.Tensor, row: Optional[Orientation], col: Optional[Orientation],
                   cfg: Optional[nvfp4_config_t] = None, stream=None) -> None:
    rows, cols = _shape2d(x)
    _need_orientation(row, rows, cols, rows if (cfg is not None and cfg.row_scaled) else 1, "row-wise")
    _need_orientation(col, cols, rows, cols if (cfg is not None and cfg.row_scaled) else 1, "column-wise")
    r = row.as_c() if row is not None else None
    c = col.as_c() if col is not None else None
    _check(load().nvfp4_quantize(_ptr(x), _dtype_code(x), rows, cols, None if r is None else ctypes.byref(r),
                                 None if c is None else ctypes.byref(c), None if cfg is None else ctypes.byref(cfg),
                                 _stream(stream)))


@_on_its_device
def nvfp4_quantize_noalloc(x: torch.Tensor, row: Optional[Orientation], col: Optional[Orientation],
                           cfg: Optional[nvfp4_config_t] = None, stream=None) -> None:
    """nvfp4_quantize with the library's own per-device scratch in place of a
    workspace (cfg.workspace must be unset); allocates nothing."""
    rows, cols = _shape2d(x)
    _need_orientation(row, rows, cols, rows if (cfg is not None and cfg.row_scaled) else 1, "row-wise")
    _need_orientation(col, cols, rows, cols if (cfg is not None and cfg.row_scaled) else 1, "column-wise")
    r = row.as_c() if row is not None else None
    c = col.as_c() if col is not None else None
    _check(load().nvfp4_quantize_noalloc(_ptr(x), _dtype_code(x), rows, cols, None if r is None else ctypes.byref(r),
                                         None if c is None else ctypes.byref(c),
                                         None if cfg is None else ctypes.byref(cfg), _stream(stream)))


@_on_its_device
def nvfp4_dequantize(q: Orientation, rows: int, cols: int, scale_layout: int, row_scaled: bool, y: torch.Tensor,
                     stream=None, scale_fmt: int = 0) -> None:
    _need_orientation(q, rows, cols, rows if row_scaled else 1, "quantized tensor")
    _need(y, rows * cols, torch.float32, "y")
    qc = q.as_c()
    _check(load().nvfp4_dequantize(ctypes.byref(qc), rows, cols, scale_layout, scale_fmt, int(row_scaled), _ptr(y),
                                   _stream(stream)))


@_on_its_device
def nvfp4_quantize_grouped(x: torch.Tensor, group_rows, row: Optional[Orientation], col: Optional[Orientation],
                           cfg: Optional[nvfp4_config_t] = None, stream=None) -> None:
    """x [sum(group_rows)][C]; row/col hold the concatenated per-group outputs
    (data and scales flat or shaped, amax [G])."""
    rows, cols = _shape2d(x)
    _need_orientation(row, rows, cols, rows if (cfg is not None and cfg.row_scaled) else len(group_rows), "row-wise")
    _need_orientation(col, cols, rows, len(group_rows), "column-wise")
    g = (ctypes.c_int64 * len(group_rows))(*[int(m) for m in group_rows])
    r = row.as_c() if row is not None else None
    c = col.as_c() if col is not None else None
    _check(load().nvfp4_quantize_grouped(_ptr(x), _dtype_code(x), len(group_rows), g, cols,
                                         None if r is None else ctypes.byref(r), None if c is None else ctypes.byref(c),
                                         None if cfg is None else ctypes.byref(cfg), _stream(stream)))


@_on_its_device
def quantize_grouped(x: torch.Tensor, group_rows, *, rowwise=True, columnwise=True,
                     cfg: Optional[nvfp4_config_t] = None, stream=None, use_workspace: bool = True):
    """Allocate the concatenated per-group outputs and run nvfp4_quantize_grouped.
    Returns (row, col) with flat data and scales and amax [G] ([R] for a
    row-scaled config). A workspace is allocated for the call as in
    quantize()."""
    rows, cols = _shape2d(x)
    G = len(group_rows)
    dev = x.device
    cfg = cfg if cfg is not None else make_config()

    def orient(amax_len):
        return Orientation(torch.empty((rows * cols // 2,), dtype=torch.uint8, device=dev),
                           torch.empty((rows * cols // 16,), dtype=torch.uint8, device=dev),
                           torch.empty((amax_len,), dtype=torch.float32, device=dev))

    row = orient(rows if cfg.row_scaled else G) if rowwise else None
    col = orient(G) if columnwise else None
    ws = None
    if use_workspace and not cfg.workspace and cfg.compute_amax and not cfg.row_scaled:
        ws = _clear_workspace(dev, stream)
        cfg = nvfp4_config_t.from_buffer_copy(cfg)
        cfg.workspace = ws.data_ptr()
    nvfp4_quantize_grouped(x, group_rows, row, col, cfg, stream)
    del ws
    return row, col


def nvfp4_swizzled_scales_bytes(rows: int, scale_cols: int) -> int:
    return int(load().nvfp4_swizzled_scales_bytes(rows, scale_cols))


@_on_its_device
def nvfp4_swizzle_scales(compact: torch.Tensor, rows: int, scale_cols: int, swizzled: torch.Tensor,
                         stream=None) -> None:
    """compact: uint8 with rows * scale_cols bytes; swizzled: uint8 with
    nvfp4_swizzled_scales_bytes(rows, scale_cols) bytes."""
    _need(compact, rows * scale_cols, torch.uint8, "compact")
    _need(swizzled, nvfp4_swizzled_scales_bytes(rows, scale_cols), torch.uint8, "swizzled")
    _check(load().nvfp4_swizzle_scales(_ptr(compact), rows, scale_cols, _ptr(swizzled), _stream(stream)))


@_on_its_device
def nvfp4_debug_rht_colwise(x: torch.Tensor, sign_mask: int, t: torch.Tensor, stream=None) -> None:
    rows, cols = _shape2d(x)
    _need(t, rows * cols, torch.float32, "t")
    _check(load().nvfp4_debug_rht_colwise(_ptr(x), _dtype_code(x), rows, cols, sign_mask & 0xFFFFFFFF, _ptr(t),
                                          _stream(stream)))


@_on_its_device
def nvfp4_debug_e2m1_pack(v: torch.Tensor, r: Optional[torch.Tensor], out: torch.Tensor, flags: int,
                          stream=None) -> None:
    """v: float32 [2n]; r: int32/uint32 [n] or None; out: uint8 [n]."""
    n = out.numel()
    _need(out, n, torch.uint8, "out")
    _need(v, 2 * n, torch.float32, "v")
    if r is not None:
        _need(r, n, (torch.int32, torch.uint32), "r")
    _check(load().nvfp4_debug_e2m1_pack(_ptr(v), _ptr(r), _ptr(out), n, flags, _stream(stream)))


# ---- allocation helpers (device memory only; no arithmetic) -----------------

def empty_orientation(n: int, k: int, device, amax_len: int = 1) -> Orientation:
    """Uninitialized buffers for one orientation with n rows of k elements."""
    return Orientation(torch.empty((n, k // 2), dtype=torch.uint8, device=device),
                       torch.empty((n * (k // 16),), dtype=torch.uint8, device=device),
                       torch.empty((amax_len,), dtype=torch.float32, device=device))


def empty_workspace(device) -> torch.Tensor:
    """A zero-filled quantize workspace, as its first use needs (torch's
    allocator aligns it to 512 bytes). Reuse it for later calls on one stream:
    the library keeps its arrival counters valid from call to call."""
    return torch.zeros((nvfp4_workspace_bytes(),), dtype=torch.uint8, device=device)


def _clear_workspace(device, stream) -> torch.Tensor:
    """An empty_workspace() that is allocated and cleared on `stream`, so that
    the call on it comes after that and its memory is not used again before."""
    with contextlib.nullcontext() if stream is None else _under(stream, device):
        return empty_workspace(device)


_workspaces = {}


def stream_workspace(device, stream=None) -> torch.Tensor:
    """The workspace that quantize() uses for calls on (device, stream): made
    once, zero-filled, then reused, so that a call costs no extra launch.
    Calls on one stream run in order, so they never share it concurrently."""
    dev = torch.device(device)
    if dev.index is None:
        dev = torch.device(dev.type, torch.cuda.current_device())
    if stream is None:
        handle = torch.cuda.current_stream(dev).cuda_stream
    else:
        handle = int(getattr(stream, "cuda_stream", stream))
    key = (dev.index, handle)
    ws = _workspaces.get(key)
    if ws is None:
        ws = _clear_workspace(dev, stream)
        _workspaces[key] = ws
    return ws


def nvfp4_debug_set_wait_ticks(ticks: int) -> None:
    _check(load().nvfp4_debug_set_wait_ticks(int(ticks) & 0xFFFFFFFF))


def nvfp4_debug_set_resident_variant(tiles_per_workgroup: int) -> None:
    _check(load().nvfp4_debug_set_resident_variant(int(tiles_per_workgroup) & 0xFFFFFFFF))


RHT_UNIT_DEFAULT = 0
RHT_UNIT_VALU = 1
RHT_UNIT_MATRIX = 2


def nvfp4_debug_set_rht_unit(unit: int) -> None:
    _check(load().nvfp4_debug_set_rht_unit(int(unit) & 0xFFFFFFFF))


@_on_its_device
def quantize(x: torch.Tensor, *, rowwise=True, columnwise=True, cfg: Optional[nvfp4_config_t] = None,
             stream=None, use_workspace: bool = True):
    """Allocate outputs for x [R][C] and run nvfp4_quantize. Returns (row, col).

    With use_workspace (and no workspace in cfg) the stream's cached
    workspace is passed, so a computed per-tensor amax takes one launch
    (single pass) or two instead of three."""
    rows, cols = _shape2d(x)
    cfg = cfg if cfg is not None else make_config()
    row = empty_orientation(rows, cols, x.device, rows if cfg.row_scaled else 1) if rowwise else None
    col = empty_orientation(cols, rows, x.device, cols if cfg.row_scaled else 1) if columnwise else None
    ws = None
    if use_workspace and not cfg.workspace and cfg.compute_amax and not cfg.row_scaled:
        ws = stream_workspace(x.device, stream)
        cfg = nvfp4_config_t.from_buffer_copy(cfg)
        cfg.workspace = ws.data_ptr()
    nvfp4_quantize(x, row, col, cfg, stream)
    return row, col


# ---- expert layers: tokens by expert, block-scaled FP8, products -------------
#
# Outputs are allocated on the stream that the call runs on, so a caller who
# passes `stream` may let go of them as with any tensor made under it.

FP8_BLOCK = 128


@dataclasses.dataclass
class ExpertPlan:
    """Where expert_sort put each slot (choice j of token t is slot t * topk + j).

    slot_rows [tokens][topk] the slot's sorted row (-1: dropped); row_slots
    [rows] the row's slot (-1: padding); offsets [experts + 1] each expert's
    first row, a multiple of align; counts [experts] its slots. All int32, on
    the device: nothing is read back to the host."""
    slot_rows: torch.Tensor
    row_slots: torch.Tensor
    offsets: torch.Tensor
    counts: torch.Tensor
    align: int

    @property
    def tokens(self) -> int:
        return self.slot_rows.shape[0]

    @property
    def topk(self) -> int:
        return self.slot_rows.shape[1]

    @property
    def experts(self) -> int:
        return self.counts.shape[0]

    @property
    def rows(self) -> int:
        return self.row_slots.shape[0]


@dataclasses.dataclass
class Fp8Tensor:
    """n rows of k values in block-scaled FP8, or a batch of such matrices.

    data float8_e4m3fn [..][n][pitch(k)], zero from k on; scales float32
    [..][ceil(k / 128)][n] (1x128 blocks) or [..][ceil(k / 128)][ceil(n / 128)]
    (block_2d: 128x128 blocks)."""
    data: torch.Tensor
    scales: torch.Tensor
    n: int
    k: int
    block_2d: bool = False

    def as_c(self) -> nvfp4_fp8_t:
        return nvfp4_fp8_t(self.data.data_ptr(), self.scales.data_ptr())


# These checks run on every call, most of which are short: each looks at the
# tensor's attributes in place and builds its message only when it refuses.
def _want(t, dtype, shape, device, what: str) -> None:
    if (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.device == device
            and t.is_contiguous()):
        return
    got = f"{t.dtype} {tuple(t.shape)} on {t.device}" if isinstance(t, torch.Tensor) else type(t).__name__
    raise ValueError(f"{what} must be a contiguous {dtype} tensor of shape {tuple(shape)} on {device}, got {got}")


def _on(x: torch.Tensor, what: str) -> torch.device:
    if not isinstance(x, torch.Tensor) or not x.is_cuda or not x.is_contiguous():
        raise ValueError(f"{what} must be a contiguous CUDA tensor")
    return x.device


def _current(device) -> int:
    # the handle that torch.cuda.current_stream(device).cuda_stream has, without the object around it
    return torch._C._cuda_getCurrentRawStream(device.index)


def _want_plan(plan: ExpertPlan, device) -> None:
    a, b, o, c, i32 = plan.slot_rows, plan.row_slots, plan.offsets, plan.counts, torch.int32
    if not (a.dtype is i32 and b.dtype is i32 and o.dtype is i32 and c.dtype is i32 and a.device == device
            and b.device == device and o.device == device and c.device == device and a.is_contiguous()
            and b.is_contiguous() and o.is_contiguous() and c.is_contiguous()):
        raise ValueError(f"a plan's tensors must be contiguous int32 tensors on {device}")
    if a.dim() != 2 or b.dim() != 1 or c.dim() != 1 or o.dim() != 1 or o.shape[0] != c.shape[0] + 1:
        raise ValueError("a plan has slot_rows [tokens][topk], row_slots [rows], offsets [experts + 1] and counts [experts]")


def expert_sort(ids: torch.Tensor, experts: int, *, align: int = FP8_BLOCK, rows: Optional[int] = None,
                stream=None) -> ExpertPlan:
    """Sort the slots of a router (ids int32 or int64 [tokens][topk]; an id
    outside 0 .. experts - 1 drops its slot) by expert, each expert's rows
    starting at a multiple of align (a power of two up to 128). rows: rows of
    the sorted matrix, by default as many as any ids could need."""
    dev = _on(ids, "ids")
    if ids.dim() != 2 or ids.dtype not in (torch.int32, torch.int64):
        raise ValueError("ids must be int32 or int64 [tokens][topk]")
    lib = load()
    tokens, topk = ids.shape
    if rows is None:
        rows = int(lib.nvfp4_expert_rows(tokens, topk, experts, align))
    if (context := _elsewhere(stream, dev)) is not None:
        with context:
            return expert_sort(ids, experts, align=align, rows=rows)
    # one allocation for all five arrays (each costs more than cutting them apart)
    sizes = (tokens * topk, max(rows, 0), max(experts, 0) + 1, max(experts, 0),
             lib.nvfp4_expert_sort_workspace_bytes(tokens, topk, experts) // 4)
    slot_rows, row_slots, offsets, counts, ws = torch.split_with_sizes(ids.new_empty((sum(sizes),), dtype=torch.int32), sizes)
    slot_rows = slot_rows.view(tokens, topk)
    _check(lib.nvfp4_expert_sort(ids.data_ptr(), ids.element_size(), tokens, topk, experts, align, rows, slot_rows.data_ptr(),
                                 row_slots.data_ptr(), offsets.data_ptr(), counts.data_ptr(), _ptr(ws) if sizes[4] else None, _current(dev)))
    return ExpertPlan(slot_rows, row_slots, offsets, counts, align)


def expert_gather(x: torch.Tensor, plan: ExpertPlan, *, stream=None) -> torch.Tensor:
    """x [tokens][cols] to the sorted rows [rows][cols], zeros in padding."""
    dev = _on(x, "x")
    _want_plan(plan, dev)
    if x.dim() != 2 or x.shape[0] != plan.tokens:
        raise ValueError(f"x must be [{plan.tokens}][cols], got {tuple(x.shape)}")
    code = _dtype_code(x)
    if (context := _elsewhere(stream, dev)) is not None:
        with context:
            return expert_gather(x, plan)
    y = torch.empty((plan.rows, x.shape[1]), dtype=x.dtype, device=dev)
    _check(load().nvfp4_expert_gather(x.data_ptr(), code, plan.tokens, plan.topk, x.shape[1], plan.slot_rows.data_ptr(),
                                      plan.row_slots.data_ptr(), plan.rows, y.data_ptr(), _current(dev)))
    return y


def expert_combine(y: torch.Tensor, plan: ExpertPlan, weights: Optional[torch.Tensor] = None, *, stream=None) -> torch.Tensor:
    """The sorted rows y [rows][cols] back to tokens [tokens][cols], summed
    over each token's slots with weights (float32 [tokens][topk]; None: ones).
    Padding rows and dropped slots are not read."""
    dev = _on(y, "y")
    _want_plan(plan, dev)
    if y.dim() != 2 or y.shape[0] != plan.rows:
        raise ValueError(f"y must be [{plan.rows}][cols], got {tuple(y.shape)}")
    if weights is not None:
        _want(weights, torch.float32, (plan.tokens, plan.topk), dev, "weights")
    code = _dtype_code(y)
    if (context := _elsewhere(stream, dev)) is not None:
        with context:
            return expert_combine(y, plan, weights)
    out = torch.empty((plan.tokens, y.shape[1]), dtype=y.dtype, device=dev)
    _check(load().nvfp4_expert_combine(y.data_ptr(), code, plan.tokens, plan.topk, y.shape[1], plan.slot_rows.data_ptr(), plan.rows,
                                       _ptr(weights), out.data_ptr(), _current(dev)))
    return out


def expert_gather_grad(dy: torch.Tensor, plan: ExpertPlan, *, stream=None) -> torch.Tensor:
    """The gradient of expert_gather's x from that of its sorted rows."""
    return expert_combine(dy, plan, None, stream=stream)


def expert_combine_grad(dout: torch.Tensor, y: torch.Tensor, plan: ExpertPlan, weights: torch.Tensor, *, stream=None):
    """The gradients (dy [rows][cols], dweights float32 [tokens][topk]) of
    expert_combine(y, plan, weights) from dout [tokens][cols]."""
    dev = _on(dout, "dout")
    _want_plan(plan, dev)
    if dout.dim() != 2 or dout.shape[0] != plan.tokens:
        raise ValueError(f"dout must be [{plan.tokens}][cols], got {tuple(dout.shape)}")
    cols = dout.shape[1]
    _want(y, dout.dtype, (plan.rows, cols), dev, "y")
    _want(weights, torch.float32, (plan.tokens, plan.topk), dev, "weights")
    code = _dtype_code(dout)
    if (context := _elsewhere(stream, dev)) is not None:
        with context:
            return expert_combine_grad(dout, y, plan, weights)
    dy = torch.empty((plan.rows, cols), dtype=dout.dtype, device=dev)
    dw = torch.empty((plan.tokens, plan.topk), dtype=torch.float32, device=dev)
    _check(load().nvfp4_expert_combine_grad(dout.data_ptr(), y.data_ptr(), code, plan.tokens, plan.topk, cols, plan.slot_rows.data_ptr(),
                                            plan.row_slots.data_ptr(), plan.rows, _ptr(weights), dy.data_ptr(), dw.data_ptr(), _current(dev)))
    return dy, dw


def nvfp4_fp8_pitch(k: int) -> int:
    return int(load().nvfp4_fp8_pitch(k))


def _blocks(n: int) -> int:
    return (n + FP8_BLOCK - 1) // FP8_BLOCK


def _matrices(x: torch.Tensor, plan: Optional[ExpertPlan]):
    """What a quantize call takes x [R][C] or [B][R][C] for, or x [tokens][C] with a plan: its
    device, leading shape, matrices, their rows and columns, and the plan's row_slots, tokens and topk."""
    dev = _on(x, "x")
    if x.dim() != 2 and (x.dim() != 3 or plan is not None):
        raise ValueError("x must be [R][C] or, without a plan, [B][R][C]")
    lead, batch = tuple(x.shape[:-2]), x.shape[0] if x.dim() == 3 else 1
    rows, cols = x.shape[-2:]
    if plan is None:
        return dev, lead, batch, rows, cols, None, 0, 1
    _want_plan(plan, dev)
    if rows != plan.tokens:
        raise ValueError(f"x must be [{plan.tokens}][cols], got {tuple(x.shape)}")
    return dev, lead, batch, plan.rows, cols, plan.row_slots, plan.tokens, plan.topk


def fp8_quantize(x: torch.Tensor, *, rowwise=True, columnwise=False, block_2d=False, plan: Optional[ExpertPlan] = None,
                 stream=None):
    """Quantize x [R][C], or a batch [B][R][C], to block-scaled FP8 (1x128
    blocks, or 128x128 with block_2d). Returns (row, col): x itself with k = C,
    and its transpose with k = R; None for one not asked for. With a plan, x
    is [tokens][C] and the matrix is expert_gather(x, plan)."""
    dev, lead, batch, rows, cols, slots, tokens, topk = _matrices(x, plan)
    code = _dtype_code(x)
    if (context := _elsewhere(stream, dev)) is not None:
        with context:
            return fp8_quantize(x, rowwise=rowwise, columnwise=columnwise, block_2d=block_2d, plan=plan)

    def empty(n, k):
        return Fp8Tensor(torch.empty((*lead, n, _blocks(k) * FP8_BLOCK), dtype=torch.float8_e4m3fn, device=dev),
                         torch.empty((*lead, _blocks(k), _blocks(n) if block_2d else n), dtype=torch.float32, device=dev),
                         n, k, bool(block_2d))

    row = empty(rows, cols) if rowwise else None
    col = empty(cols, rows) if columnwise else None
    r, c = row.as_c() if row is not None else None, col.as_c() if col is not None else None
    _check(load().nvfp4_fp8_quantize(x.data_ptr(), code, batch, rows, cols, _ptr(slots), tokens, topk, int(block_2d), r, c, _current(dev)))
    return row, col


def _want_fp8(q: Fp8Tensor, lead, n: int, k: int, block_2d: bool, device, what: str) -> None:
    if q.n != n or q.k != k or bool(q.block_2d) != block_2d:
        raise ValueError(f"{what} must have {n} rows of {k} values in {'128x128' if block_2d else '1x128'} blocks, got "
                         f"{q.n} x {q.k}, block_2d={q.block_2d}")
    kb = (k + FP8_BLOCK - 1) // FP8_BLOCK
    _want(q.data, torch.float8_e4m3fn, (*lead, n, kb * FP8_BLOCK), device, what)
    _want(q.scales, torch.float32, (*lead, kb, (n + FP8_BLOCK - 1) // FP8_BLOCK if block_2d else n), device, what)


def _out_code(dtype) -> int:
    if dtype not in (torch.bfloat16, torch.float32):
        raise TypeError(f"the output type must be bfloat16 or float32, got {dtype}")
    return NVFP4_IN_BF16 if dtype == torch.bfloat16 else NVFP4_IN_FP32


def fp8_matmul(a: Fp8Tensor, b: Fp8Tensor, *, out_dtype=torch.bfloat16, stream=None) -> torch.Tensor:
    """a b^T [a.n][b.n]; a in 1x128 blocks, b in 1x128 or 128x128 blocks."""
    dev = _on(a.data, "operand a")
    code = _out_code(out_dtype)
    _want_fp8(a, (), a.n, a.k, False, dev, "operand a")
    _want_fp8(b, (), b.n, a.k, bool(b.block_2d), dev, "operand b")
    if (context := _elsewhere(stream, dev)) is not None:
        with context:
            return fp8_matmul(a, b, out_dtype=out_dtype)
    d = torch.empty((a.n, b.n), dtype=out_dtype, device=dev)
    _check(load().nvfp4_fp8_matmul(a.as_c(), b.as_c(), a.n, b.n, a.k, int(b.block_2d), d.data_ptr(), code, _current(dev)))
    return d


def fp8_matmul_grouped(a: Fp8Tensor, b: Fp8Tensor, plan: ExpertPlan, *, out_dtype=torch.bfloat16, stream=None) -> torch.Tensor:
    """Each expert's rows of a (1x128 blocks, plan.rows rows) times its matrix
    of the batch b ([experts], 128x128 blocks): [plan.rows][b.n], zeros past
    the last expert's rows."""
    dev = _on(a.data, "operand a")
    code = _out_code(out_dtype)
    _want_plan(plan, dev)
    _want_fp8(a, (), plan.rows, a.k, False, dev, "operand a")
    _want_fp8(b, (plan.experts,), b.n, a.k, True, dev, "operand b")
    if (context := _elsewhere(stream, dev)) is not None:
        with context:
            return fp8_matmul_grouped(a, b, plan, out_dtype=out_dtype)
    d = torch.empty((plan.rows, b.n), dtype=out_dtype, device=dev)
    _check(load().nvfp4_fp8_matmul_grouped(a.as_c(), b.as_c(), plan.offsets.data_ptr(), plan.experts, plan.rows, b.n, a.k,
                                           d.data_ptr(), code, _current(dev)))
    return d


def fp8_matmul_grouped_k(a: Fp8Tensor, b: Fp8Tensor, plan: ExpertPlan, *, out_dtype=torch.float32, stream=None) -> torch.Tensor:
    """Per expert, a b^T over its rows, which are k here: [experts][a.n][b.n],
    zeros for an expert without rows. a and b are column-wise orientations of
    sorted rows (k = plan.rows, 1x128 blocks) and the plan's align is 128."""
    dev = _on(a.data, "operand a")
    code = _out_code(out_dtype)
    _want_plan(plan, dev)
    if plan.align != FP8_BLOCK:
        raise ValueError(f"the plan must be aligned to {FP8_BLOCK} rows, got {plan.align}")
    _want_fp8(a, (), a.n, plan.rows, False, dev, "operand a")
    _want_fp8(b, (), b.n, plan.rows, False, dev, "operand b")
    if (context := _elsewhere(stream, dev)) is not None:
        with context:
            return fp8_matmul_grouped_k(a, b, plan, out_dtype=out_dtype)
    d = torch.empty((plan.experts, a.n, b.n), dtype=out_dtype, device=dev)
    _check(load().nvfp4_fp8_matmul_grouped_k(a.as_c(), b.as_c(), plan.offsets.data_ptr(), plan.experts, a.n, b.n, plan.rows,
                                             d.data_ptr(), code, _current(dev)))
    return d


# ---- MXFP4: quantization and back, products -----------------------------------

@dataclasses.dataclass
class Mxfp4Tensor:
    """n rows of k values in MXFP4, or a batch of such matrices.

    data uint8 [..][n][pitch(k) / 2], two E2M1 codes a byte (the even element in
    the low half), zero from k on; scales uint8 [..][ceil(k / 128)][n][4], an E8M0
    byte for each 32 values of a row."""
    data: torch.Tensor
    scales: torch.Tensor
    n: int
    k: int

    def as_c(self) -> nvfp4_mxfp4_t:
        return nvfp4_mxfp4_t(self.data.data_ptr(), self.scales.data_ptr())


def mxfp4_quantize(x: torch.Tensor, *, rowwise=True, columnwise=False, block_2d=False, plan: Optional[ExpertPlan] = None,
                   stream=None):
    """Quantize x [R][C], or a batch [B][R][C], to MXFP4 (a scale for 32 values
    of a row, or with block_2d for 32x32). Returns (row, col): x itself with k =
    C, and its transpose with k = R; None for one not asked for. With a plan, x
    is [tokens][C] and the matrix is expert_gather(x, plan)."""
    dev, lead, batch, rows, cols, slots, tokens, topk = _matrices(x, plan)
    code = _dtype_code(x)
    if (context := _elsewhere(stream, dev)) is not None:
        with context:
            return mxfp4_quantize(x, rowwise=rowwise, columnwise=columnwise, block_2d=block_2d, plan=plan)

    def empty(n, k):
        return Mxfp4Tensor(torch.empty((*lead, n, _blocks(k) * (FP8_BLOCK // 2)), dtype=torch.uint8, device=dev),
                           torch.empty((*lead, _blocks(k), n, 4), dtype=torch.uint8, device=dev), n, k)

    row = empty(rows, cols) if rowwise else None
    col = empty(cols, rows) if columnwise else None
    r, c = row.as_c() if row is not None else None, col.as_c() if col is not None else None
    _check(load().nvfp4_mxfp4_quantize(x.data_ptr(), code, batch, rows, cols, _ptr(slots), tokens, topk, int(block_2d), r, c, _current(dev)))
    return row, col


def _want_mxfp4(q: Mxfp4Tensor, lead, n: int, k: int, device, what: str) -> None:
    if q.n != n or q.k != k:
        raise ValueError(f"{what} must have {n} rows of {k} values, got {q.n} x {q.k}")
    kb = (k + FP8_BLOCK - 1) // FP8_BLOCK
    _want(q.data, torch.uint8, (*lead, n, kb * (FP8_BLOCK // 2)), device, what)
    _want(q.scales, torch.uint8, (*lead, kb, n, 4), device, what)


def mxfp4_dequantize(q: Mxfp4Tensor, *, out_dtype=torch.bfloat16, stream=None) -> torch.Tensor:
    """The values of q, [n][k] or [B][n][k]; bfloat16 and float32 hold them exactly, but for those of
    scales 253 and 254 that are past their largest number: infinities."""
    dev = _on(q.data, "the tensor")
    code = _out_code(out_dtype)
    lead = tuple(q.data.shape[:-2])
    if len(lead) > 1:
        raise ValueError(f"the tensor must be one matrix or a batch of them, got {tuple(q.data.shape)}")
    _want_mxfp4(q, lead, q.n, q.k, dev, "the tensor")
    if (context := _elsewhere(stream, dev)) is not None:
        with context:
            return mxfp4_dequantize(q, out_dtype=out_dtype)
    y = torch.empty((*lead, q.n, q.k), dtype=out_dtype, device=dev)
    _check(load().nvfp4_mxfp4_dequantize(q.as_c(), lead[0] if lead else 1, q.n, q.k, y.data_ptr(), code, _current(dev)))
    return y


def mxfp4_matmul(a: Mxfp4Tensor, b: Mxfp4Tensor, *, out_dtype=torch.bfloat16, stream=None) -> torch.Tensor:
    """a b^T [a.n][b.n]."""
    dev = _on(a.data, "operand a")
    code = _out_code(out_dtype)
    _want_mxfp4(a, (), a.n, a.k, dev, "operand a")
    _want_mxfp4(b, (), b.n, a.k, dev, "operand b")
    if (context := _elsewhere(stream, dev)) is not None:
        with context:
            return mxfp4_matmul(a, b, out_dtype=out_dtype)
    d = torch.empty((a.n, b.n), dtype=out_dtype, device=dev)
    _check(load().nvfp4_mxfp4_matmul(a.as_c(), b.as_c(), a.n, b.n, a.k, d.data_ptr(), code, _current(dev)))
    return d


def mxfp4_matmul_grouped(a: Mxfp4Tensor, b: Mxfp4Tensor, plan: ExpertPlan, *, out_dtype=torch.bfloat16, stream=None) -> torch.Tensor:
    """Each expert's rows of a (plan.rows rows) times its matrix of the batch b
    ([experts]): [plan.rows][b.n], zeros past the last expert's rows."""
    dev = _on(a.data, "operand a")
    code = _out_code(out_dtype)
    _want_plan(plan, dev)
    _want_mxfp4(a, (), plan.rows, a.k, dev, "operand a")
    _want_mxfp4(b, (plan.experts,), b.n, a.k, dev, "operand b")
    if (context := _elsewhere(stream, dev)) is not None:
        with context:
            return mxfp4_matmul_grouped(a, b, plan, out_dtype=out_dtype)
    d = torch.empty((plan.rows, b.n), dtype=out_dtype, device=dev)
    _check(load().nvfp4_mxfp4_matmul_grouped(a.as_c(), b.as_c(), plan.offsets.data_ptr(), plan.experts, plan.rows, b.n, a.k,
                                             d.data_ptr(), code, _current(dev)))
    return d


def mxfp4_matmul_grouped_k(a: Mxfp4Tensor, b: Mxfp4Tensor, plan: ExpertPlan, *, out_dtype=torch.float32, stream=None) -> torch.Tensor:
    """Per expert, a b^T over its rows, which are k here: [experts][a.n][b.n],
    zeros for an expert without rows. a and b are column-wise orientations of
    sorted rows (k = plan.rows) and the plan's align is 128."""
    dev = _on(a.data, "operand a")
    code = _out_code(out_dtype)
    _want_plan(plan, dev)
    if plan.align != FP8_BLOCK:
        raise ValueError(f"the plan must be aligned to {FP8_BLOCK} rows, got {plan.align}")
    _want_mxfp4(a, (), a.n, plan.rows, dev, "operand a")
    _want_mxfp4(b, (), b.n, plan.rows, dev, "operand b")
    if (context := _elsewhere(stream, dev)) is not None:
        with context:
            return mxfp4_matmul_grouped_k(a, b, plan, out_dtype=out_dtype)
    d = torch.empty((plan.experts, a.n, b.n), dtype=out_dtype, device=dev)
    _check(load().nvfp4_mxfp4_matmul_grouped_k(a.as_c(), b.as_c(), plan.offsets.data_ptr(), plan.experts, a.n, b.n, plan.rows,
                                               d.data_ptr(), code, _current(dev)))
    return d


# ---- an expert layer for a few tokens -----------------------------------------

def expert_mlp(x: torch.Tensor, ids: torch.Tensor, weights: torch.Tensor, w1, w2, *, gated=True, stream=None) -> torch.Tensor:
    """An expert layer for a decoding step, in three launches: out[t] = the sum over
    j of weights[t][j] w2[e] act(w1[e] x[t]) with e = ids[t][j], [tokens][cols] bfloat16.

    x bfloat16 [tokens][cols]; ids int32 or int64 [tokens][topk] (an id outside 0
    .. experts - 1 leaves its choice out); weights float32 [tokens][topk]; tokens *
    topk at most 1024. w1 is a batch [experts] with k = cols and n = 2 hidden, act
    = silu of the first half's products times the second half's, or (not gated) n =
    hidden and act = silu; w2 has n = cols and k = hidden. Both are Mxfp4Tensors
    or both Fp8Tensors in 128x128 blocks. Larger batches go through expert_sort
    and the grouped products, which are also the faster form from about 32 slots an
    expert on (16 where rows are of 8192 values)."""
    dev = _on(x, "x")
    if x.dim() != 2 or x.dtype is not torch.bfloat16:
        raise ValueError(f"x must be bfloat16 [tokens][cols], got {x.dtype} {tuple(x.shape)}")
    tokens, cols = x.shape
    if not isinstance(ids, torch.Tensor) or ids.dim() != 2 or ids.dtype not in (torch.int32, torch.int64):
        raise ValueError("ids must be int32 or int64 [tokens][topk]")
    topk = ids.shape[1]
    _want(ids, ids.dtype, (tokens, topk), dev, "ids")
    _want(weights, torch.float32, (tokens, topk), dev, "weights")
    if isinstance(w1, Fp8Tensor) != isinstance(w2, Fp8Tensor):
        raise ValueError("w1 and w2 must have one format")
    hidden, experts = w2.k, w2.data.shape[0]
    n1 = 2 * hidden if gated else hidden
    lib = load()
    if isinstance(w1, Fp8Tensor):
        _want_fp8(w1, (experts,), n1, cols, True, dev, "w1")
        _want_fp8(w2, (experts,), cols, hidden, True, dev, "w2")
        call = lib.nvfp4_expert_mlp_fp8
    else:
        _want_mxfp4(w1, (experts,), n1, cols, dev, "w1")
        _want_mxfp4(w2, (experts,), cols, hidden, dev, "w2")
        call = lib.nvfp4_expert_mlp_mxfp4
    if (context := _elsewhere(stream, dev)) is not None:
        with context:
            return expert_mlp(x, ids, weights, w1, w2, gated=gated)
    out = torch.empty_like(x)
    workspace = torch.empty((lib.nvfp4_expert_mlp_workspace_bytes(tokens, topk, cols, hidden),), dtype=torch.uint8, device=dev)
    _check(call(x.data_ptr(), tokens, cols, ids.data_ptr(), ids.element_size(), weights.data_ptr(), topk, experts, w1.as_c(), w2.as_c(),
                hidden, int(gated), workspace.data_ptr(), out.data_ptr(), _current(dev)))
    return out
