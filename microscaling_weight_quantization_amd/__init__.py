"""Python binding of the gfx950 block-scaled weight-quantization library (libmxq.so).

The ``mxq_*`` functions carry the names of the C entry points in
``include/mxq.h`` and only marshal arguments: tensors become device pointers,
row strides and sizes, and the call is enqueued on torch's current stream.
Every step of the computation runs in the HIP kernels of ``csrc/`` (``mxq.hip``;
``group_quant.hip``, ``product.hip`` and ``experts.hip`` for the FP8 products, their
operands and the experts' rows; ``norm.hip``, ``activate.hip`` and ``route.hip`` for what stands
between the products); there is no fallback of any kind, and a missing library raises.

PyTorch is used for device memory and streams only.  A [rows, K] operand is a
tensor whose last dimension is contiguous; leading dimensions of a contiguous
tensor are flattened into rows.

Sources (page title, section): "[PyTorch] MXFP4 weight QAT on MXFP8 and FP8
block-scaling recipes" -- Description, Test results, Known limitations; and
"MXFP8TensorStorage.export_components()" -- Description.
"""
from __future__ import annotations

import ctypes
import functools
import os
import threading
from typing import NamedTuple, Optional

import torch

from . import build as _build

MXQ_BF16, MXQ_FP32, MXQ_FP16 = 0, 1, 2
MXQ_E4M3, MXQ_E5M2 = 0, 1
MXQ_SCALE_ROW_1X32, MXQ_SCALE_TILE_128X128, MXQ_SCALE_COL_32X1 = 0, 1, 2
MXQ_SILU, MXQ_GELU_TANH, MXQ_RELU2 = 0, 1, 2
MXQ_SOFTMAX, MXQ_SIGMOID = 0, 1
MXQ_OK, MXQ_ERR_NULL, MXQ_ERR_SHAPE, MXQ_ERR_DTYPE, MXQ_ERR_NO_ROWWISE_DATA, MXQ_ERR_ALIAS, MXQ_ERR_HIP = range(7)

ENTRY_POINTS = ("mxq_status_string", "mxq_fake_quantize_mxfp4", "mxq_mxfp4_to_mxfp8_row",
                "mxq_mxfp4_to_fp8_block128", "mxq_export_mxfp8", "mxq_dequantize",
                "mxq_fake_quantize_mxfp4_with_mxfp8_row", "mxq_mxfp4_to_mxfp8_row_guarded",
                "mxq_mxfp4_to_fp8_block128_guarded", "mxq_quantize_mxfp4", "mxq_dequantize_mxfp4",
                "mxq_mxfp4_packed_to_mxfp8_row", "mxq_mxfp4_packed_to_fp8_block128", "mxq_mxfp4_to_mxfp8_col",
                "mxq_mxfp4_to_mxfp8_row_col", "mxq_mxfp4_to_mxfp8_col_guarded", "mxq_mxfp4_to_mxfp8_row_col_guarded",
                "mxq_mxfp4_to_mxfp8_row_grouped", "mxq_fake_quantize_mxfp4_grouped",
                "mxq_mxfp4_to_fp8_block128_grouped", "mxq_dequantize_grouped", "mxq_quantize_mxfp4_grouped",
                "mxq_quantize_fp8_group128", "mxq_quantize_fp8_group128_col", "mxq_quantize_fp8_group128_row_col",
                "mxq_matmul_fp8_block128", "mxq_matmul_fp8_block128_dgrad", "mxq_matmul_fp8_group128_wgrad",
                "mxq_sort_experts", "mxq_sort_experts_workspace", "mxq_dispatch_rows", "mxq_combine_rows",
                "mxq_combine_rows_backward", "mxq_rms_norm", "mxq_rms_norm_fp8_group128",
                "mxq_rms_norm_fp8_group128_row_col_workspace", "mxq_rms_norm_fp8_group128_row_col",
                "mxq_rms_norm_backward_workspace", "mxq_rms_norm_backward", "mxq_activate_fp8_group128",
                "mxq_activate_fp8_group128_row_col", "mxq_activate_fp8_group128_backward", "mxq_route_experts",
                "mxq_route_experts_backward")

_libs = {}
_lock = threading.Lock()


class _RowGroup(ctypes.Structure):
    """mxq_row_group of include/mxq.h."""
    _fields_ = [("x", ctypes.c_void_p), ("ld_x", ctypes.c_int64), ("rows", ctypes.c_int64), ("K", ctypes.c_int64),
                ("data", ctypes.c_void_p), ("scale", ctypes.c_void_p), ("scale_ld", ctypes.c_int64)]


class _ProjGroup(ctypes.Structure):
    """mxq_proj_group of include/mxq.h."""
    _fields_ = [("x", ctypes.c_void_p), ("ld_x", ctypes.c_int64), ("y", ctypes.c_void_p), ("ld_y", ctypes.c_int64),
                ("rows", ctypes.c_int64), ("K", ctypes.c_int64)]


class _Block128Group(ctypes.Structure):
    """mxq_block128_group of include/mxq.h."""
    _fields_ = [("x", ctypes.c_void_p), ("ld_x", ctypes.c_int64), ("rows", ctypes.c_int64), ("K", ctypes.c_int64),
                ("data", ctypes.c_void_p), ("tile_code", ctypes.c_void_p), ("tile_ld", ctypes.c_int64)]


class _DequantGroup(ctypes.Structure):
    """mxq_dequant_group of include/mxq.h."""
    _fields_ = [("data", ctypes.c_void_p), ("scale", ctypes.c_void_p), ("scale_ld", ctypes.c_int64),
                ("rows", ctypes.c_int64), ("K", ctypes.c_int64), ("out", ctypes.c_void_p), ("ld_out", ctypes.c_int64)]


class _Mxfp4Group(ctypes.Structure):
    """mxq_mxfp4_group of include/mxq.h."""
    _fields_ = [("x", ctypes.c_void_p), ("ld_x", ctypes.c_int64), ("rows", ctypes.c_int64), ("K", ctypes.c_int64),
                ("packed", ctypes.c_void_p), ("scale", ctypes.c_void_p), ("scale_ld", ctypes.c_int64)]


class MxqError(RuntimeError):
    def __init__(self, status: int, text: str):
        super().__init__(f"mxq status {status}: {text}")
        self.status = status


def load(name: str = "libmxq.so") -> ctypes.CDLL:
    """Load a built variant of the library (build it first: ``__graft_entry__.build()``)."""
    with _lock:
        if name in _libs:
            return _libs[name]
        path = _build.library_path(name)
        if not os.path.exists(path):
            raise FileNotFoundError(f"{path} is not built; run __graft_entry__.build() "
                                    "(python -m microscaling_weight_quantization_amd.build)")
        L = ctypes.CDLL(path)
        i64, vp, i32, u8p = ctypes.c_int64, ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p
        L.mxq_status_string.argtypes = [i32]
        L.mxq_status_string.restype = ctypes.c_char_p
        L.mxq_fake_quantize_mxfp4.argtypes = [vp, i64, vp, i64, i64, i64, i32, vp]
        L.mxq_mxfp4_to_mxfp8_row.argtypes = [vp, i64, i64, i64, i32, u8p, u8p, i64, vp]
        L.mxq_mxfp4_to_fp8_block128.argtypes = [vp, i64, i64, i64, i32, u8p, u8p, i64, vp]
        L.mxq_export_mxfp8.argtypes = [u8p, u8p, i64, i64, i64, u8p, vp]
        L.mxq_dequantize.argtypes = [u8p, u8p, i64, i64, i64, i32, i32, vp, i64, i32, vp]
        L.mxq_fake_quantize_mxfp4_with_mxfp8_row.argtypes = [vp, i64, vp, i64, i64, i64, i32, u8p, u8p, i64, vp]
        L.mxq_mxfp4_to_mxfp8_row_guarded.argtypes = [vp, i64, i64, i64, i32, u8p, u8p, i64, vp, vp]
        L.mxq_mxfp4_to_fp8_block128_guarded.argtypes = [vp, i64, i64, i64, i32, u8p, u8p, i64, vp, vp]
        L.mxq_quantize_mxfp4.argtypes = [vp, i64, i64, i64, i32, u8p, u8p, i64, vp]
        L.mxq_dequantize_mxfp4.argtypes = [u8p, u8p, i64, i64, i64, vp, i64, i32, vp]
        L.mxq_mxfp4_packed_to_mxfp8_row.argtypes = [u8p, u8p, i64, i64, i64, u8p, u8p, i64, vp]
        L.mxq_mxfp4_packed_to_fp8_block128.argtypes = [u8p, u8p, i64, i64, i64, u8p, u8p, i64, vp]
        L.mxq_mxfp4_to_mxfp8_col.argtypes = [vp, i64, i64, i64, i32, u8p, u8p, i64, vp]
        L.mxq_mxfp4_to_mxfp8_row_col.argtypes = [vp, i64, i64, i64, i32, u8p, u8p, i64, u8p, u8p, i64, vp]
        L.mxq_mxfp4_to_mxfp8_col_guarded.argtypes = [vp, i64, i64, i64, i32, u8p, u8p, i64, vp, vp]
        L.mxq_mxfp4_to_mxfp8_row_col_guarded.argtypes = [vp, i64, i64, i64, i32, u8p, u8p, i64, u8p, u8p, i64, vp, vp]
        L.mxq_mxfp4_to_mxfp8_row_grouped.argtypes = [ctypes.POINTER(_RowGroup), i64, i32, vp]
        L.mxq_fake_quantize_mxfp4_grouped.argtypes = [ctypes.POINTER(_ProjGroup), i64, i32, vp]
        L.mxq_mxfp4_to_fp8_block128_grouped.argtypes = [ctypes.POINTER(_Block128Group), i64, i32, vp]
        L.mxq_dequantize_grouped.argtypes = [ctypes.POINTER(_DequantGroup), i64, i32, i32, i32, vp]
        L.mxq_quantize_mxfp4_grouped.argtypes = [ctypes.POINTER(_Mxfp4Group), i64, i32, vp]
        quant = [vp, i64, i64, i64, i64, i32, vp, i64]                  # x, ld, x_rows, rows, K, dtype, slots, top_k
        L.mxq_quantize_fp8_group128.argtypes = quant + [u8p, i64, u8p, i64, vp]
        L.mxq_quantize_fp8_group128_col.argtypes = quant + [vp, i64, u8p, i64, u8p, i64, vp]
        L.mxq_quantize_fp8_group128_row_col.argtypes = quant + [vp, i64] + [u8p, i64] * 4 + [vp]
        product = [u8p, i64, u8p, i64, u8p, i64, i64, u8p, i64, i64, i64, i64, i64, vp, i64, vp, i64, i32, i32, vp]
        L.mxq_matmul_fp8_block128.argtypes = product
        L.mxq_matmul_fp8_block128_dgrad.argtypes = product
        L.mxq_matmul_fp8_group128_wgrad.argtypes = [u8p, i64] * 4 + [i64, i64, i64, vp, i64, vp, i64, i64, i32, vp]
        L.mxq_sort_experts.argtypes = [vp, i64, i64, i64, i64, vp, vp, vp, vp, i64, vp]
        L.mxq_sort_experts_workspace.argtypes = [i64, i64, i64]
        L.mxq_dispatch_rows.argtypes = [vp, i64, i64, vp, i64, i64, i64, i32, vp, i64, vp]
        L.mxq_combine_rows.argtypes = [vp, i64, i64, vp, vp, i64, i64, i64, i32, vp, i64, vp]
        L.mxq_combine_rows_backward.argtypes = [vp, i64, vp, i64, i64, vp, vp, i64, i64, i64, i32, vp, i64, vp, vp]
        f32 = ctypes.c_float
        norm = [vp, i64, vp, i64, i32, vp, i32, f32, i64, i64, i32, vp, i64, vp, i64]   # ... sum, ld_sum, y, ld_y
        L.mxq_rms_norm.argtypes = norm + [vp]
        L.mxq_rms_norm_fp8_group128.argtypes = norm + [u8p, i64] * 2 + [vp]
        L.mxq_rms_norm_fp8_group128_row_col_workspace.argtypes = [i64]
        L.mxq_rms_norm_fp8_group128_row_col.argtypes = norm + [u8p, i64] * 4 + [vp, i64, vp]
        L.mxq_rms_norm_backward_workspace.argtypes = [i64, i64]
        L.mxq_rms_norm_backward.argtypes = [vp, i64, i32, vp, i64, i32, vp, i32, f32, vp, i64, i64, i64, vp, i64, vp, vp,
                                            i64, vp]
        act = [vp, i64, vp, i64, i64, i64, i32, i32]                    # gate, ld, up, ld, rows, F, dtype, activation
        L.mxq_activate_fp8_group128.argtypes = act + [u8p, i64] * 2 + [vp]
        L.mxq_activate_fp8_group128_row_col.argtypes = act + [vp, i64] + [u8p, i64] * 4 + [vp]
        L.mxq_activate_fp8_group128_backward.argtypes = [vp, i64] + act + [vp, i64] + [u8p, i64] * 4 + [vp]
        L.mxq_route_experts.argtypes = [vp, i64, i64, i64, i32, vp, vp, i32, i32, f32, i64, i64, i64, i64, vp, vp, vp]
        L.mxq_route_experts_backward.argtypes = [vp, vp, i64, vp, i64, i64, i64, i32, i32, i32, f32, vp, i64, vp]
        for n in ENTRY_POINTS[1:]:
            getattr(L, n).restype = i64 if n.endswith("_workspace") else i32
        _libs[name] = L
        return L


_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _device_operands(fn):
    """Every tensor argument of an entry point must be a device tensor, all on one
    device: the library takes raw device pointers, and a host pointer or one
    from another GPU would reach a kernel as an invalid address."""
    tensor = torch.Tensor

    @functools.wraps(fn)
    def wrapper(*args, **kwargs):
        dev = -2                                            # get_device(): -1 for a host tensor
        for t in (*args, *kwargs.values()):
            if isinstance(t, tensor):
                d = t.get_device()
                if d == dev:
                    continue
                if d < 0 or not t.is_cuda:
                    raise ValueError(f"{fn.__name__}: operands must be device tensors, got one on {t.device}")
                if dev == -2:
                    dev = d
                else:
                    raise ValueError(f"{fn.__name__}: operands on cuda:{dev} and cuda:{d}; all must be on one device")
        if dev >= 0 and dev != _current_device():   # a launch goes to the current device
            with torch.cuda.device(dev):
                return fn(*args, **kwargs)
        return fn(*args, **kwargs)
    return wrapper


def _check(L, rc: int):
    if rc != MXQ_OK:
        raise MxqError(rc, L.mxq_status_string(rc).decode())


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return MXQ_BF16
    if t.dtype == torch.float32:
        return MXQ_FP32
    if t.dtype == torch.float16:
        return MXQ_FP16
    raise TypeError(f"unsupported dtype {t.dtype}: bf16 or fp32 expected")


def _matrix(t: torch.Tensor):
    """(pointer, rows, K, row stride in elements) of a tensor with a contiguous last dim."""
    if t.dim() == 0:
        raise ValueError("a matrix needs at least one dimension")
    if t.dim() == 1:
        t = t.view(1, -1)
    if t.dim() > 2:
        if not t.is_contiguous():
            raise ValueError("leading dimensions can only be flattened for a contiguous tensor")
        t = t.view(-1, t.shape[-1])
    rows, K = t.shape
    if K > 1 and t.stride(1) != 1:
        raise ValueError("the last dimension must be contiguous")
    ld = t.stride(0) if rows > 1 else K
    return t.data_ptr(), rows, K, ld


def _operand(t: torch.Tensor, rows: int, cols: int, what: str, contiguous: bool = False, byte: bool = False):
    """(pointer, row stride) of an operand the call reads or writes as a
    [rows, cols] matrix.  Raises ValueError, before anything is launched, when
    the tensor is smaller than that region (the C entry points only see a
    pointer and a stride, so a short buffer would be accessed out of bounds),
    when `contiguous` is set and its rows are not packed (payloads have row
    stride cols), or when `byte` is set and its elements are not bytes."""
    if byte and t.element_size() != 1:
        raise ValueError(f"{what} holds bytes (uint8), got {t.dtype}")
    p, trows, tcols, ld = _matrix(t)
    if rows * cols == 0:
        return p, max(ld, cols)
    if trows < rows or tcols < cols:
        raise ValueError(f"{what} must cover [{rows}, {cols}], got [{trows}, {tcols}]")
    if contiguous and ld != cols:
        raise ValueError(f"{what} must be a contiguous [{rows}, {cols}] tensor (row stride {cols}), got row stride {ld}")
    return p, ld


def _flag(t: torch.Tensor) -> int:
    if t.dtype != torch.int32 or not t.is_cuda or t.numel() < 1:
        raise ValueError("the no-op flag is a device int32 tensor")
    return t.data_ptr()


# torch's current stream as a raw handle.  The internal accessor returns the
# handle directly (a tenth of the time of building a Stream object); the public
# call is the fallback where a torch build lacks it.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(t: torch.Tensor):
    if _raw_stream is not None:
        return ctypes.c_void_p(_raw_stream(t.get_device()))
    return ctypes.c_void_p(torch.cuda.current_stream(t.device).cuda_stream)


# ---- the C entry points, one to one ---------------------------------------------------

def _nb(K: int) -> int:
    return (K + 31) // 32


def _scale_for(x: torch.Tensor, rows: int, cols: int, ld: Optional[int]) -> torch.Tensor:
    """A zeroed code array [rows, ld or cols] on x's device (padding stays 0)."""
    return torch.zeros((rows, ld or cols), dtype=torch.uint8, device=x.device)


def _payload_for(x: torch.Tensor, rows: int, K: int, data: Optional[torch.Tensor], what: str = "payload"):
    if data is None:
        data = torch.empty((rows, K), dtype=torch.uint8, device=x.device)
    pd, _ = _operand(data, rows, K, what, contiguous=True, byte=True)
    return data, pd


@_device_operands
def mxq_fake_quantize_mxfp4(x: torch.Tensor, y: Optional[torch.Tensor] = None, lib: str = "libmxq.so") -> torch.Tensor:
    """MXFP4 projection of x (bf16 / fp32) into y (same dtype; y may be x)."""
    L = load(lib)
    dt = _dtype_code(x)
    if y is None:
        y = torch.empty_like(x, memory_format=torch.contiguous_format)
    if y.dtype != x.dtype or y.shape != x.shape:
        raise ValueError("y must have x's dtype and shape")
    px, rows, K, ldx = _matrix(x)
    py, ldy = _operand(y, rows, K, "y")
    _check(L, L.mxq_fake_quantize_mxfp4(px, ldx, py, ldy, rows, K, dt, _stream(x)))
    return y


@_device_operands
def mxq_mxfp4_to_mxfp8_row(x: torch.Tensor, data: Optional[torch.Tensor] = None, scale: Optional[torch.Tensor] = None,
                           scale_ld: Optional[int] = None, lib: str = "libmxq.so",
                           noop: Optional[torch.Tensor] = None):
    """Direct MXFP8 rowwise lift -> (payload uint8 [rows, K], E8M0 codes uint8 [rows, scale_ld]).
    With `noop` (an int32 device tensor) this is mxq_mxfp4_to_mxfp8_row_guarded."""
    L = load(lib)
    dt = _dtype_code(x)
    px, rows, K, ldx = _matrix(x)
    scale = _scale_for(x, rows, _nb(K), scale_ld) if scale is None else scale
    data, pd = _payload_for(x, rows, K, data)
    ps, ld_s = _operand(scale, rows, _nb(K), "scale", byte=True)
    if noop is None:
        _check(L, L.mxq_mxfp4_to_mxfp8_row(px, ldx, rows, K, dt, pd, ps, ld_s, _stream(x)))
    else:
        _check(L, L.mxq_mxfp4_to_mxfp8_row_guarded(px, ldx, rows, K, dt, pd, ps, ld_s, _flag(noop), _stream(x)))
    return data, scale


@_device_operands
def mxq_mxfp4_to_fp8_block128(x: torch.Tensor, data: Optional[torch.Tensor] = None,
                              tile_code: Optional[torch.Tensor] = None, lib: str = "libmxq.so",
                              noop: Optional[torch.Tensor] = None):
    """Direct 128x128 blockwise FP8 -> (payload uint8 [rows, K], tile codes uint8 [ceil(rows/128), tile_ld]).
    With `noop` (an int32 device tensor) this is mxq_mxfp4_to_fp8_block128_guarded."""
    L = load(lib)
    dt = _dtype_code(x)
    px, rows, K, ldx = _matrix(x)
    ntr, ntc = (rows + 127) // 128, (K + 127) // 128
    tile_code = _scale_for(x, ntr, ntc, None) if tile_code is None else tile_code
    data, pd = _payload_for(x, rows, K, data)
    pt, ldt = _operand(tile_code, ntr, ntc, "tile_code", byte=True)
    if noop is None:
        _check(L, L.mxq_mxfp4_to_fp8_block128(px, ldx, rows, K, dt, pd, pt, ldt, _stream(x)))
    else:
        _check(L, L.mxq_mxfp4_to_fp8_block128_guarded(px, ldx, rows, K, dt, pd, pt, ldt, _flag(noop), _stream(x)))
    return data, tile_code


@_device_operands
def mxq_mxfp4_to_mxfp8_col(x: torch.Tensor, data: Optional[torch.Tensor] = None, scale: Optional[torch.Tensor] = None,
                           scale_ld: Optional[int] = None, lib: str = "libmxq.so",
                           noop: Optional[torch.Tensor] = None):
    """MXFP8 columnwise (32x1 blocks) from the decomposition ->
    (payload uint8 [rows, K], E8M0 codes uint8 [ceil(rows/32), scale_ld]).
    With `noop` (an int32 device tensor) this is mxq_mxfp4_to_mxfp8_col_guarded."""
    L = load(lib)
    dt = _dtype_code(x)
    px, rows, K, ldx = _matrix(x)
    bands = (rows + 31) // 32
    scale = _scale_for(x, bands, K, scale_ld) if scale is None else scale
    data, pd = _payload_for(x, rows, K, data)
    ps, ld_s = _operand(scale, bands, K, "scale", byte=True)
    if noop is None:
        _check(L, L.mxq_mxfp4_to_mxfp8_col(px, ldx, rows, K, dt, pd, ps, ld_s, _stream(x)))
    else:
        _check(L, L.mxq_mxfp4_to_mxfp8_col_guarded(px, ldx, rows, K, dt, pd, ps, ld_s, _flag(noop), _stream(x)))
    return data, scale


@_device_operands
def mxq_mxfp4_to_mxfp8_row_col(x: torch.Tensor, row_data: Optional[torch.Tensor] = None,
                               row_scale: Optional[torch.Tensor] = None, col_data: Optional[torch.Tensor] = None,
                               col_scale: Optional[torch.Tensor] = None, row_scale_ld: Optional[int] = None,
                               col_scale_ld: Optional[int] = None, lib: str = "libmxq.so",
                               noop: Optional[torch.Tensor] = None):
    """Row lift and columnwise conversion from one read of x ->
    (row payload, row codes [rows, row_scale_ld], column payload, column codes [ceil(rows/32), col_scale_ld]).
    With `noop` (an int32 device tensor) this is mxq_mxfp4_to_mxfp8_row_col_guarded."""
    L = load(lib)
    dt = _dtype_code(x)
    px, rows, K, ldx = _matrix(x)
    bands = (rows + 31) // 32
    row_scale = _scale_for(x, rows, _nb(K), row_scale_ld) if row_scale is None else row_scale
    col_scale = _scale_for(x, bands, K, col_scale_ld) if col_scale is None else col_scale
    row_data, prd = _payload_for(x, rows, K, row_data, "row payload")
    col_data, pcd = _payload_for(x, rows, K, col_data, "column payload")
    prs, ld_rs = _operand(row_scale, rows, _nb(K), "row_scale", byte=True)
    pcs, ld_cs = _operand(col_scale, bands, K, "col_scale", byte=True)
    if noop is None:
        _check(L, L.mxq_mxfp4_to_mxfp8_row_col(px, ldx, rows, K, dt, prd, prs, ld_rs, pcd, pcs, ld_cs, _stream(x)))
    else:
        _check(L, L.mxq_mxfp4_to_mxfp8_row_col_guarded(px, ldx, rows, K, dt, prd, prs, ld_rs, pcd, pcs, ld_cs,
                                                       _flag(noop), _stream(x)))
    return row_data, row_scale, col_data, col_scale


@_device_operands
def mxq_fake_quantize_mxfp4_with_mxfp8_row(x: torch.Tensor, y: Optional[torch.Tensor] = None,
                                           data: Optional[torch.Tensor] = None, scale: Optional[torch.Tensor] = None,
                                           scale_ld: Optional[int] = None, lib: str = "libmxq.so"):
    """Projection and row lift from one read of x -> (y, payload, codes)."""
    L = load(lib)
    dt = _dtype_code(x)
    px, rows, K, ldx = _matrix(x)
    if y is None:
        y = torch.empty_like(x, memory_format=torch.contiguous_format)
    if y.dtype != x.dtype or y.shape != x.shape:
        raise ValueError("y must have x's dtype and shape")
    scale = _scale_for(x, rows, _nb(K), scale_ld) if scale is None else scale
    py, ldy = _operand(y, rows, K, "y")
    data, pd = _payload_for(x, rows, K, data)
    ps, ld_s = _operand(scale, rows, _nb(K), "scale", byte=True)
    _check(L, L.mxq_fake_quantize_mxfp4_with_mxfp8_row(px, ldx, py, ldy, rows, K, dt, pd, ps, ld_s, _stream(x)))
    return y, data, scale


@_device_operands
def mxq_export_mxfp8(data: Optional[torch.Tensor], scale_storage: Optional[torch.Tensor], K: int,
                     scale_out: Optional[torch.Tensor] = None, lib: str = "libmxq.so") -> torch.Tensor:
    """Compact [rows, ceil(K/32)] copy of padded E8M0 scale storage (rows, scale_ld)."""
    L = load(lib)
    if data is None or scale_storage is None:
        rc = L.mxq_export_mxfp8(None, None, 0, K, 0, None, None)
        _check(L, rc)
    ps, rows, _, ld_s = _matrix(scale_storage)
    nb = _nb(K)
    if scale_out is None:
        scale_out = torch.empty((rows, nb), dtype=torch.uint8, device=scale_storage.device)
    _operand(scale_storage, rows, nb, "scale_storage", byte=True)
    po, _ = _operand(scale_out, rows, nb, "scale_out", contiguous=True, byte=True)
    _check(L, L.mxq_export_mxfp8(data.data_ptr(), ps, rows, K, ld_s, po, _stream(scale_storage)))
    return scale_out


_SCALE_GRID = {MXQ_SCALE_ROW_1X32: lambda rows, K: (rows, _nb(K)),
               MXQ_SCALE_TILE_128X128: lambda rows, K: ((rows + 127) // 128, (K + 127) // 128),
               MXQ_SCALE_COL_32X1: lambda rows, K: ((rows + 31) // 32, K)}


@_device_operands
def mxq_dequantize(data: torch.Tensor, scale: torch.Tensor, layout: int = MXQ_SCALE_ROW_1X32, fmt: int = MXQ_E4M3,
                   out: Optional[torch.Tensor] = None, out_dtype: torch.dtype = torch.bfloat16,
                   lib: str = "libmxq.so") -> torch.Tensor:
    """Decode FP8 payload bytes with E8M0 codes into bf16 / fp32."""
    L = load(lib)
    _, rows, K, _ = _matrix(data)
    pd, _ = _operand(data, rows, K, "payload", contiguous=True, byte=True)
    if out is None:
        out = torch.empty((rows, K), dtype=out_dtype, device=data.device)
    srows, scols = _SCALE_GRID[layout](rows, K) if layout in _SCALE_GRID else (0, 0)   # the C call rejects others
    ps, lds = _operand(scale, srows, scols, "scale", byte=True)
    po, ldo = _operand(out, rows, K, "out")
    _check(L, L.mxq_dequantize(pd, ps, lds, rows, K, fmt, layout, po, ldo, _dtype_code(out), _stream(data)))
    return out


@_device_operands
def mxq_quantize_mxfp4(x: torch.Tensor, packed: Optional[torch.Tensor] = None, scale: Optional[torch.Tensor] = None,
                       scale_ld: Optional[int] = None, lib: str = "libmxq.so"):
    """Packed MXFP4 (deployment format) -> (nibble pairs uint8 [rows, ceil(K/2)], E8M0 codes)."""
    L = load(lib)
    dt = _dtype_code(x)
    px, rows, K, ldx = _matrix(x)
    pw = (K + 1) // 2
    if packed is None:
        packed = torch.empty((rows, pw), dtype=torch.uint8, device=x.device)
    scale = _scale_for(x, rows, _nb(K), scale_ld) if scale is None else scale
    pp, _ = _operand(packed, rows, pw, "packed", contiguous=True, byte=True)
    ps, ld_s = _operand(scale, rows, _nb(K), "scale", byte=True)
    _check(L, L.mxq_quantize_mxfp4(px, ldx, rows, K, dt, pp, ps, ld_s, _stream(x)))
    return packed, scale


def _packed_args(packed: torch.Tensor, scale: torch.Tensor, K: int):
    _, rows, _, _ = _matrix(packed)
    pp, _ = _operand(packed, rows, (K + 1) // 2, "packed", contiguous=True, byte=True)
    ps, ld_s = _operand(scale, rows, _nb(K), "scale", byte=True)
    return pp, ps, ld_s, rows


@_device_operands
def mxq_dequantize_mxfp4(packed: torch.Tensor, scale: torch.Tensor, K: int, out: Optional[torch.Tensor] = None,
                         out_dtype: torch.dtype = torch.bfloat16, lib: str = "libmxq.so") -> torch.Tensor:
    """Decode packed MXFP4 into bf16 / fp32 [rows, K]."""
    L = load(lib)
    pp, ps, ld_s, rows = _packed_args(packed, scale, K)
    if out is None:
        out = torch.empty((rows, K), dtype=out_dtype, device=packed.device)
    po, ldo = _operand(out, rows, K, "out")
    _check(L, L.mxq_dequantize_mxfp4(pp, ps, ld_s, rows, K, po, ldo, _dtype_code(out), _stream(packed)))
    return out


@_device_operands
def mxq_mxfp4_packed_to_mxfp8_row(packed: torch.Tensor, scale: torch.Tensor, K: int,
                                  data: Optional[torch.Tensor] = None, scale_out: Optional[torch.Tensor] = None,
                                  lib: str = "libmxq.so"):
    """Direct MXFP8 row lift from packed MXFP4 -> (payload uint8 [rows, K], codes)."""
    L = load(lib)
    pp, ps, ld_s, rows = _packed_args(packed, scale, K)
    data, pd = _payload_for(packed, rows, K, data)
    scale_out = _scale_for(packed, rows, _nb(K), None) if scale_out is None else scale_out
    po, ldo = _operand(scale_out, rows, _nb(K), "scale_out", byte=True)
    _check(L, L.mxq_mxfp4_packed_to_mxfp8_row(pp, ps, ld_s, rows, K, pd, po, ldo, _stream(packed)))
    return data, scale_out


@_device_operands
def mxq_mxfp4_packed_to_fp8_block128(packed: torch.Tensor, scale: torch.Tensor, K: int,
                                     data: Optional[torch.Tensor] = None, tile_code: Optional[torch.Tensor] = None,
                                     lib: str = "libmxq.so"):
    """Direct 128x128 blockwise FP8 from packed MXFP4 -> (payload uint8 [rows, K], tile codes)."""
    L = load(lib)
    pp, ps, ld_s, rows = _packed_args(packed, scale, K)
    ntr, ntc = (rows + 127) // 128, (K + 127) // 128
    data, pd = _payload_for(packed, rows, K, data)
    tile_code = _scale_for(packed, ntr, ntc, None) if tile_code is None else tile_code
    pt, ldt = _operand(tile_code, ntr, ntc, "tile_code", byte=True)
    _check(L, L.mxq_mxfp4_packed_to_fp8_block128(pp, ps, ld_s, rows, K, pd, pt, ldt, _stream(packed)))
    return data, tile_code


# ---- grouped calls ------------------------------------------------------------------------

class _Grouped:
    """A grouped entry point prepared once for a fixed list of weights and
    outputs: the descriptor table is built (and every operand checked) here,
    and each call enqueues the whole list on torch's current stream with one
    call into the library, for weights re-converted every training step.  The
    object keeps the tensors alive.

    Subclasses name the C function and its descriptor struct, the list
    arguments (the first is the per-weight input that sets rows and K),
    `_describe`, which fills in missing outputs for weight i, checks its
    operands and returns its descriptor, and `_extra_args`, the call's
    arguments between the table and the stream."""
    _fn: str
    _struct: type
    _lists: tuple

    def __init__(self, lists, lib: str):
        self._L = load(lib)
        lists = [list(l) if l is not None else None for l in lists]
        self.n = n = len(lists[0])
        lists = [[None] * n if l is None else l for l in lists]
        if any(len(l) != n for l in lists):
            raise ValueError(f"{self._fn}: {', '.join(self._lists[1:])} must have one entry per weight")
        self._tensors = lists
        self._first = None
        if n == 0:
            return
        for l in lists:
            for t in l:
                if t is not None and not (isinstance(t, torch.Tensor) and t.is_cuda):
                    raise ValueError(f"{self._fn}: operands must be device tensors on one device")
        dev = lists[0][0].device
        if any(t is not None and t.device != dev for l in lists for t in l):
            raise ValueError(f"{self._fn}: operands must be device tensors on one device")
        self._first = lists[0][0]
        self._table = (self._struct * n)(*[self._describe(i, dev) for i in range(n)])
        self._extra = self._extra_args()

    def _describe(self, i: int, dev):
        raise NotImplementedError

    def _extra_args(self):
        return (self._same_dtype(self._tensors[0], "weights"),)

    def _same_dtype(self, ts, what: str) -> int:
        if any(t.dtype != ts[0].dtype for t in ts):
            raise ValueError(f"all {what} of a group call must have one dtype")
        return _dtype_code(ts[0])

    def __call__(self):
        if self.n:
            _check(self._L, getattr(self._L, self._fn)(self._table, self.n, *self._extra, _stream(self._first)))
        return self._outputs()


class GroupedRowLift(_Grouped):
    """The grouped row lift (mxq_mxfp4_to_mxfp8_row_grouped); `datas` / `scales` are the outputs."""
    _fn, _struct, _lists = "mxq_mxfp4_to_mxfp8_row_grouped", _RowGroup, ("xs", "datas", "scales")

    def __init__(self, xs, datas=None, scales=None, scale_ld: Optional[int] = None, lib: str = "libmxq.so"):
        self._scale_ld = scale_ld
        super().__init__((xs, datas, scales), lib)

    def _describe(self, i, dev):
        xs, datas, scales = self._tensors
        px, rows, K, ldx = _matrix(xs[i])
        if scales[i] is None:
            scales[i] = _scale_for(xs[i], rows, _nb(K), self._scale_ld)
        datas[i], pd = _payload_for(xs[i], rows, K, datas[i])
        ps, ld_s = _operand(scales[i], rows, _nb(K), "scale", byte=True)
        return _RowGroup(px, ldx, rows, K, pd, ps, ld_s)

    def _outputs(self):
        return self._tensors[1], self._tensors[2]

    xs = property(lambda self: self._tensors[0])
    datas = property(lambda self: self._tensors[1])
    scales = property(lambda self: self._tensors[2])


class GroupedProjection(_Grouped):
    """The grouped MXFP4 projection (mxq_fake_quantize_mxfp4_grouped); an
    output may be its weight itself (in place); `ys` are the outputs."""
    _fn, _struct, _lists = "mxq_fake_quantize_mxfp4_grouped", _ProjGroup, ("xs", "ys")

    def __init__(self, xs, ys=None, lib: str = "libmxq.so"):
        super().__init__((xs, ys), lib)

    def _describe(self, i, dev):
        xs, ys = self._tensors
        if ys[i] is None:
            ys[i] = torch.empty_like(xs[i], memory_format=torch.contiguous_format)
        if ys[i].dtype != xs[i].dtype or ys[i].shape != xs[i].shape:
            raise ValueError("each output must have its weight's dtype and shape")
        px, rows, K, ldx = _matrix(xs[i])
        py, ldy = _operand(ys[i], rows, K, "y")
        return _ProjGroup(px, ldx, py, ldy, rows, K)

    def _outputs(self):
        return self._tensors[1]

    xs = property(lambda self: self._tensors[0])
    ys = property(lambda self: self._tensors[1])


class GroupedBlock128(_Grouped):
    """The grouped 128x128 fold (mxq_mxfp4_to_fp8_block128_grouped); `datas` / `tile_codes` are the outputs."""
    _fn, _struct, _lists = "mxq_mxfp4_to_fp8_block128_grouped", _Block128Group, ("xs", "datas", "tile_codes")

    def __init__(self, xs, datas=None, tile_codes=None, lib: str = "libmxq.so"):
        super().__init__((xs, datas, tile_codes), lib)

    def _describe(self, i, dev):
        xs, datas, tcs = self._tensors
        px, rows, K, ldx = _matrix(xs[i])
        ntr, ntc = (rows + 127) // 128, (K + 127) // 128
        if tcs[i] is None:
            tcs[i] = _scale_for(xs[i], ntr, ntc, None)
        datas[i], pd = _payload_for(xs[i], rows, K, datas[i])
        pt, ldt = _operand(tcs[i], ntr, ntc, "tile_code", byte=True)
        return _Block128Group(px, ldx, rows, K, pd, pt, ldt)

    def _outputs(self):
        return self._tensors[1], self._tensors[2]

    xs = property(lambda self: self._tensors[0])
    datas = property(lambda self: self._tensors[1])
    tile_codes = property(lambda self: self._tensors[2])


class GroupedDequantize(_Grouped):
    """The grouped decode (mxq_dequantize_grouped) of payloads with one format,
    scale layout and output dtype; `outs` are the outputs."""
    _fn, _struct, _lists = "mxq_dequantize_grouped", _DequantGroup, ("datas", "scales", "outs")

    def __init__(self, datas, scales, layout: int = MXQ_SCALE_ROW_1X32, fmt: int = MXQ_E4M3, outs=None,
                 out_dtype: torch.dtype = torch.bfloat16, lib: str = "libmxq.so"):
        self._layout, self._fmt, self._out_dtype = layout, fmt, out_dtype
        super().__init__((datas, scales, outs), lib)

    def _extra_args(self):
        return (self._fmt, self._layout, self._same_dtype(self._tensors[2], "outputs"))

    def _describe(self, i, dev):
        datas, scales, outs = self._tensors
        _, rows, K, _ = _matrix(datas[i])
        if outs[i] is None:
            outs[i] = torch.empty(tuple(datas[i].shape), dtype=self._out_dtype, device=dev)
        pd, _ = _operand(datas[i], rows, K, "payload", contiguous=True, byte=True)
        srows, scols = _SCALE_GRID[self._layout](rows, K) if self._layout in _SCALE_GRID else (0, 0)
        ps, lds = _operand(scales[i], srows, scols, "scale", byte=True)
        po, ldo = _operand(outs[i], rows, K, "out")
        return _DequantGroup(pd, ps, lds, rows, K, po, ldo)

    def _outputs(self):
        return self._tensors[2]

    datas = property(lambda self: self._tensors[0])
    outs = property(lambda self: self._tensors[2])


class GroupedQuantizeMxfp4(_Grouped):
    """The grouped packed MXFP4 encode (mxq_quantize_mxfp4_grouped); `packeds` / `scales` are the outputs."""
    _fn, _struct, _lists = "mxq_quantize_mxfp4_grouped", _Mxfp4Group, ("xs", "packeds", "scales")

    def __init__(self, xs, packeds=None, scales=None, scale_ld: Optional[int] = None, lib: str = "libmxq.so"):
        self._scale_ld = scale_ld
        super().__init__((xs, packeds, scales), lib)

    def _describe(self, i, dev):
        xs, packeds, scales = self._tensors
        px, rows, K, ldx = _matrix(xs[i])
        pw = (K + 1) // 2
        if packeds[i] is None:
            packeds[i] = torch.empty((rows, pw), dtype=torch.uint8, device=dev)
        if scales[i] is None:
            scales[i] = _scale_for(xs[i], rows, _nb(K), self._scale_ld)
        pp, _ = _operand(packeds[i], rows, pw, "packed", contiguous=True, byte=True)
        ps, ld_s = _operand(scales[i], rows, _nb(K), "scale", byte=True)
        return _Mxfp4Group(px, ldx, rows, K, pp, ps, ld_s)

    def _outputs(self):
        return self._tensors[1], self._tensors[2]

    xs = property(lambda self: self._tensors[0])
    packeds = property(lambda self: self._tensors[1])
    scales = property(lambda self: self._tensors[2])


@_device_operands
def mxq_mxfp4_to_mxfp8_row_grouped(xs, datas=None, scales=None, scale_ld: Optional[int] = None,
                                   lib: str = "libmxq.so"):
    """Direct MXFP8 rowwise lift of a list of weights of one dtype, in as few
    launches as possible -> (list of payloads, list of E8M0 codes); the same
    bytes as one mxq_mxfp4_to_mxfp8_row per weight.  `datas` / `scales`: lists
    of outputs (None entries, or None for the whole list, are allocated)."""
    return GroupedRowLift(xs, datas, scales, scale_ld, lib)()


@_device_operands
def mxq_fake_quantize_mxfp4_grouped(xs, ys=None, lib: str = "libmxq.so"):
    """MXFP4 projection of a list of weights of one dtype, in as few launches as
    possible -> list of outputs; the same bits as one mxq_fake_quantize_mxfp4 per
    weight (an entry of `ys` may be its weight, in place)."""
    return GroupedProjection(xs, ys, lib)()


@_device_operands
def mxq_mxfp4_to_fp8_block128_grouped(xs, datas=None, tile_codes=None, lib: str = "libmxq.so"):
    """Direct 128x128 blockwise FP8 of a list of weights of one dtype, in as few
    launches as possible -> (list of payloads, list of tile codes)."""
    return GroupedBlock128(xs, datas, tile_codes, lib)()


@_device_operands
def mxq_dequantize_grouped(datas, scales, layout: int = MXQ_SCALE_ROW_1X32, fmt: int = MXQ_E4M3, outs=None,
                           out_dtype: torch.dtype = torch.bfloat16, lib: str = "libmxq.so"):
    """Decode a list of FP8 payloads with their E8M0 codes (one format, scale
    layout and output dtype), in as few launches as possible -> list of outputs."""
    return GroupedDequantize(datas, scales, layout, fmt, outs, out_dtype, lib)()


@_device_operands
def mxq_quantize_mxfp4_grouped(xs, packeds=None, scales=None, scale_ld: Optional[int] = None,
                               lib: str = "libmxq.so"):
    """Packed MXFP4 (deployment format) of a list of weights of one dtype, in as
    few launches as possible -> (list of nibble pairs, list of E8M0 codes)."""
    return GroupedQuantizeMxfp4(xs, packeds, scales, scale_ld, lib)()


# ---- FP8 products and the routing of a layer of experts ------------------------------------

# A call on a single token costs more on the host than on the GPU, so these
# functions take the short way where there is one.

_UINT8, _INT32, _FLOAT32 = torch.uint8, torch.int32, torch.float32
_FLOAT_CODES = {torch.bfloat16: MXQ_BF16, torch.float32: MXQ_FP32}


def _library(name: str) -> ctypes.CDLL:
    return _libs.get(name) or load(name)


def _mat(t: torch.Tensor):
    """_matrix, at once for the usual [rows, K] with contiguous rows."""
    s = t.shape
    if len(s) == 2:
        rows, K = s
        if t.is_contiguous():
            return t.data_ptr(), rows, K, K
        ld, step = t.stride()
        if step == 1 and rows > 1:
            return t.data_ptr(), rows, K, ld
    return _matrix(t)


def _handle(t: torch.Tensor):
    """torch's current stream on t's device as the C calls take it."""
    return _raw_stream(t.get_device()) if _raw_stream is not None else torch.cuda.current_stream(t.device).cuda_stream


def _float_code(t: torch.Tensor) -> int:
    code = _FLOAT_CODES.get(t.dtype)
    return _dtype_code(t) if code is None else code


def _ng(n: int) -> int:
    return (n + 127) // 128


def _vector(t: torch.Tensor, n: int, dtype: torch.dtype, what: str) -> int:
    """Pointer of a contiguous array of n elements of `dtype`."""
    if t.dtype != dtype or t.numel() != n or not t.is_contiguous():
        raise ValueError(f"{what} is a contiguous {dtype} tensor of {n} elements, "
                         f"got {t.dtype} {list(t.shape)}")
    return t.data_ptr()


def _experts_of(offsets: Optional[torch.Tensor]):
    """(pointer, number of experts) of an offsets tensor; (None, 0) for None."""
    if offsets is None:
        return None, 0
    if offsets.dim() != 1 or offsets.shape[0] < 2:
        raise ValueError("offsets is a tensor of n_experts + 1 elements")
    return _vector(offsets, offsets.shape[0], torch.int32, "offsets"), offsets.shape[0] - 1


def _code_rows(rows: int, n_experts: int) -> int:
    """Code rows of groups of 128 rows: begun anew with each expert, or at row 0."""
    return rows // 128 + n_experts if n_experts else _ng(rows)


def _source(x: torch.Tensor, slots: Optional[torch.Tensor], top_k: int):
    """The quantizer's leading arguments, and the rows and columns of its result."""
    px, x_rows, K, ldx = _mat(x)
    if slots is None:
        return (px, ldx, x_rows, x_rows, K, _float_code(x), None, 1), x_rows, K
    rows = slots.numel()
    return (px, ldx, x_rows, rows, K, _float_code(x), _vector(slots, rows, torch.int32, "slots"), top_k), rows, K


def _bytes_for(x: torch.Tensor, t: Optional[torch.Tensor], rows: int, cols: int, what: str):
    """(tensor, pointer, row stride) of a byte output, allocated if missing."""
    if t is None:
        t = x.new_empty((rows, cols), dtype=_UINT8)
        return t, t.data_ptr(), cols
    p, ld = _operand(t, rows, cols, what, byte=True)
    return t, p, ld


@_device_operands
def mxq_quantize_fp8_group128(x: torch.Tensor, slots: Optional[torch.Tensor] = None, top_k: int = 1,
                              data: Optional[torch.Tensor] = None, scale: Optional[torch.Tensor] = None,
                              lib: str = "libmxq.so"):
    """FP8 payload and E8M0 codes of groups of 128 along the rows of x (bf16 / fp32) ->
    (payload uint8 [rows, K], codes uint8 [rows, ceil(K/128)]).  With `slots` (int32, as
    mxq_sort_experts returns them) row r of the result is x's row slots[r] // top_k, zeros for a
    dropped slot."""
    L = _library(lib)
    args, rows, K = _source(x, slots, top_k)
    data, pd, ldd = _bytes_for(x, data, rows, K, "payload")
    scale, ps, lds = _bytes_for(x, scale, rows, _ng(K), "scale")
    _check(L, L.mxq_quantize_fp8_group128(*args, pd, ldd, ps, lds, _handle(x)))
    return data, scale


@_device_operands
def mxq_quantize_fp8_group128_col(x: torch.Tensor, slots: Optional[torch.Tensor] = None, top_k: int = 1,
                                  offsets: Optional[torch.Tensor] = None, data: Optional[torch.Tensor] = None,
                                  scale: Optional[torch.Tensor] = None, lib: str = "libmxq.so"):
    """The same with groups of 128 rows of a column, the operand of a weight gradient ->
    (payload uint8 [rows, K], codes uint8 [groups, K]).  With `offsets` (int32 [n_experts + 1])
    groups begin anew with each expert's rows and there are rows // 128 + n_experts code rows."""
    L = _library(lib)
    args, rows, K = _source(x, slots, top_k)
    po, n = _experts_of(offsets)
    data, pd, ldd = _bytes_for(x, data, rows, K, "payload")
    scale, ps, lds = _bytes_for(x, scale, _code_rows(rows, n), K, "scale")
    _check(L, L.mxq_quantize_fp8_group128_col(*args, po, n, pd, ldd, ps, lds, _handle(x)))
    return data, scale


@_device_operands
def mxq_quantize_fp8_group128_row_col(x: torch.Tensor, slots: Optional[torch.Tensor] = None, top_k: int = 1,
                                      offsets: Optional[torch.Tensor] = None,
                                      row_data: Optional[torch.Tensor] = None, row_scale: Optional[torch.Tensor] = None,
                                      col_data: Optional[torch.Tensor] = None, col_scale: Optional[torch.Tensor] = None,
                                      lib: str = "libmxq.so"):
    """Groups along the rows and along the columns from one read of x ->
    (row payload, row codes, column payload, column codes)."""
    L = _library(lib)
    args, rows, K = _source(x, slots, top_k)
    po, n = _experts_of(offsets)
    row_data, prd, ldrd = _bytes_for(x, row_data, rows, K, "row payload")
    row_scale, prs, ldrs = _bytes_for(x, row_scale, rows, _ng(K), "row_scale")
    col_data, pcd, ldcd = _bytes_for(x, col_data, rows, K, "column payload")
    col_scale, pcs, ldcs = _bytes_for(x, col_scale, _code_rows(rows, n), K, "col_scale")
    _check(L, L.mxq_quantize_fp8_group128_row_col(*args, po, n, prd, ldrd, prs, ldrs, pcd, ldcd, pcs, ldcs, _handle(x)))
    return row_data, row_scale, col_data, col_scale


def _weights(w: torch.Tensor, tile_code: torch.Tensor, n_experts: int):
    """(N, K, the C call's arguments) of [N, K] payloads and their tile codes, n_experts of them if not 0."""
    lead = 3 if n_experts else 2
    ws, ts = w.shape, tile_code.shape
    if (len(ws) == len(ts) == lead and w.is_contiguous() and tile_code.is_contiguous() and w.element_size() == 1
            and tile_code.element_size() == 1 and ts[-2:] == (_ng(ws[-2]), _ng(ws[-1]))
            and (not n_experts or ws[0] == ts[0] == n_experts)):
        N, K, tc = ws[-2], ws[-1], ts[-1]
        return N, K, (w.data_ptr(), K, N * K, tile_code.data_ptr(), tc, ts[-2] * tc)
    if w.dim() != lead or tile_code.dim() != lead or (n_experts and not w.shape[0] == tile_code.shape[0] == n_experts):
        raise ValueError("w and tile_code are [N, K] and [ceil(N/128), ceil(K/128)], with offsets [n_experts, ...] "
                         f"of them; got {list(w.shape)} and {list(tile_code.shape)}")
    if w.element_size() != 1 or tile_code.element_size() != 1:
        raise ValueError(f"w and tile_code hold bytes, got {w.dtype} and {tile_code.dtype}")
    N, K = w.shape[-2:]
    tr, tc = _ng(N), _ng(K)
    if tile_code.shape[-2] < tr or tile_code.shape[-1] < tc:
        raise ValueError(f"tile_code must cover [{tr}, {tc}], got {list(tile_code.shape)}")
    if (K > 1 and w.stride(-1) != 1) or (tc > 1 and tile_code.stride(-1) != 1):
        raise ValueError("the last dimension must be contiguous")
    return N, K, (w.data_ptr(), w.stride(-2) if N > 1 else K, w.stride(0) if n_experts else 0, tile_code.data_ptr(),
                  tile_code.stride(-2) if tr > 1 else tc, tile_code.stride(0) if n_experts else 0)


def _rows_operand(t: torch.Tensor, scale: torch.Tensor, cols: int, what: str):
    """(rows, the C call's arguments) of a payload [rows, cols] with row groups."""
    p, rows, tcols, ld = _mat(t)
    if tcols != cols or t.element_size() != 1:
        raise ValueError(f"{what} holds bytes, [rows, {cols}], got {t.dtype} {list(t.shape)}")
    groups = _ng(cols)
    if scale.shape == (rows, groups) and scale.is_contiguous() and scale.element_size() == 1:
        return rows, (p, ld, scale.data_ptr(), groups)
    ps, lds = _operand(scale, rows, groups, what + "_scale", byte=True)
    return rows, (p, ld, ps, lds)


def _result(like: torch.Tensor, out: Optional[torch.Tensor], shape, out_dtype: torch.dtype):
    """(tensor, pointer, row stride, stride of a leading dimension, dtype) of an output, allocated if missing."""
    if out is None:
        out = torch.empty(shape, dtype=out_dtype, device=like.device)
        return out, out.data_ptr(), shape[-1], shape[-2] * shape[-1], _float_code(out)
    if tuple(out.shape) != tuple(shape):
        raise ValueError(f"the output is {list(shape)}, got {list(out.shape)}")
    if shape[-1] > 1 and out.stride(-1) != 1:
        raise ValueError("the last dimension must be contiguous")
    return out, out.data_ptr(), out.stride(-2) if shape[-2] > 1 else shape[-1], out.stride(0), _float_code(out)


@_device_operands
def mxq_matmul_fp8_block128(x: torch.Tensor, x_scale: torch.Tensor, w: torch.Tensor, tile_code: torch.Tensor,
                            offsets: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                            out_dtype: torch.dtype = torch.bfloat16, fast_accum: bool = False,
                            lib: str = "libmxq.so") -> torch.Tensor:
    """y = x w^T in FP8: x [M, K] with its codes [M, ceil(K/128)] (mxq_quantize_fp8_group128), w [N, K]
    with its tile codes (mxq_mxfp4_to_fp8_block128) -> [M, N] bf16 / fp32.  With `offsets` (int32
    [n_experts + 1]) the rows of x are sorted by expert, w is [n_experts, N, K] and expert e's rows
    meet w[e]; rows of no expert give zeros.  Products are summed in fp32; with `fast_accum` the FP8
    matrix instructions sum them, at about twice the rate and up to 2^-10 of the sum of magnitudes off."""
    L = _library(lib)
    po, n = (None, 0) if offsets is None else _experts_of(offsets)
    N, K, pw = _weights(w, tile_code, n)
    M, px = _rows_operand(x, x_scale, K, "x")
    out, py, ldy, _, dt = _result(x, out, (M, N), out_dtype)
    _check(L, L.mxq_matmul_fp8_block128(*px, *pw, M, N, K, po, n, py, ldy, dt, fast_accum, _handle(x)))
    return out


@_device_operands
def mxq_matmul_fp8_block128_dgrad(dy: torch.Tensor, dy_scale: torch.Tensor, w: torch.Tensor, tile_code: torch.Tensor,
                                  offsets: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                                  out_dtype: torch.dtype = torch.bfloat16, fast_accum: bool = False,
                                  lib: str = "libmxq.so") -> torch.Tensor:
    """dx = dy w in FP8, the input's gradient of mxq_matmul_fp8_block128: dy [M, N] with its codes
    [M, ceil(N/128)], the same w and tile codes -> [M, K]."""
    L = _library(lib)
    po, n = (None, 0) if offsets is None else _experts_of(offsets)
    N, K, pw = _weights(w, tile_code, n)
    M, pg = _rows_operand(dy, dy_scale, N, "dy")
    out, px, ldx, _, dt = _result(dy, out, (M, K), out_dtype)
    _check(L, L.mxq_matmul_fp8_block128_dgrad(*pg, *pw, M, N, K, po, n, px, ldx, dt, fast_accum, _handle(dy)))
    return out


@_device_operands
def mxq_matmul_fp8_group128_wgrad(dy: torch.Tensor, dy_scale: torch.Tensor, x: torch.Tensor, x_scale: torch.Tensor,
                                  offsets: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                                  out_dtype: torch.dtype = torch.float32, lib: str = "libmxq.so") -> torch.Tensor:
    """dw = dy^T x in FP8, the weight's gradient: dy [M, N] and x [M, K] with the codes of column groups
    (mxq_quantize_fp8_group128_col, both with the same `offsets`) -> [N, K], or [n_experts, N, K]."""
    L = _library(lib)
    po, n = _experts_of(offsets)
    pg, M, N, ldg = _mat(dy)
    px, mx, K, ldx = _mat(x)
    if mx != M or dy.element_size() != 1 or x.element_size() != 1:
        raise ValueError(f"dy and x hold bytes and have the same rows, got {dy.dtype} {list(dy.shape)} and "
                         f"{x.dtype} {list(x.shape)}")
    groups = _code_rows(M, n)
    pgs, ldgs = _operand(dy_scale, groups, N, "dy_scale", byte=True)
    pxs, ldxs = _operand(x_scale, groups, K, "x_scale", byte=True)
    out, pw, ldw, stride, dt = _result(dy, out, (n, N, K) if n else (N, K), out_dtype)
    _check(L, L.mxq_matmul_fp8_group128_wgrad(pg, ldg, pgs, ldgs, px, ldx, pxs, ldxs, M, N, K, po, n, pw, ldw, stride,
                                              dt, _handle(dy)))
    return out


@_device_operands
def mxq_sort_experts(ids: torch.Tensor, n_experts: int, lib: str = "libmxq.so"):
    """Slots of ids (int32 [tokens, top_k], the experts of each token) sorted by expert, stably ->
    (offsets [n_experts + 1], slots [tokens * top_k], position [tokens, top_k]), all int32.  Expert e
    owns sorted rows offsets[e] .. offsets[e + 1]; slots[r] is the slot of sorted row r and
    position[t, j] the sorted row of slot t * top_k + j.  Ids outside [0, n_experts) are dropped:
    their slots come last and both directions hold the complement."""
    L = _library(lib)
    if ids.dim() != 2 or ids.dtype != torch.int32:
        raise ValueError(f"ids is int32 [tokens, top_k], got {ids.dtype} {list(ids.shape)}")
    pi, T, k, ldi = _mat(ids)
    need = L.mxq_sort_experts_workspace(T, k, n_experts)
    # one allocation: offsets, slots, position, workspace
    n = T * k
    a = n_experts + 1
    buf = torch.empty(a + 2 * n + need // 4, dtype=_INT32, device=ids.device)
    at = buf.data_ptr()
    _check(L, L.mxq_sort_experts(pi, ldi, T, k, n_experts, at, at + 4 * a, at + 4 * (a + n), at + 4 * (a + 2 * n), need,
                                 _handle(ids)))
    offsets, slots, position = (buf[:a + 2 * n] if need else buf).split_with_sizes((a, n, n))
    return offsets, slots, position.view(T, k)


@_device_operands
def mxq_dispatch_rows(x: torch.Tensor, slots: torch.Tensor, top_k: int, out: Optional[torch.Tensor] = None,
                      lib: str = "libmxq.so") -> torch.Tensor:
    """x's rows (bf16 / fp32 [tokens, H]) in sorted order: row r is x[slots[r] // top_k], zeros for a
    dropped slot -> [slots, H].  Its gradient is mxq_combine_rows without weights."""
    L = _library(lib)
    px, T, H, ldx = _mat(x)
    rows = slots.numel()
    ps = _vector(slots, rows, torch.int32, "slots")
    out, po, ldo, _, dt = _result(x, out, (rows, H), x.dtype)
    if out.dtype != x.dtype:
        raise ValueError("out must have x's dtype")
    _check(L, L.mxq_dispatch_rows(px, ldx, T, ps, rows, top_k, H, dt, po, ldo, _handle(x)))
    return out


def _slots_of(position: torch.Tensor, weights: Optional[torch.Tensor]):
    if position.dim() != 2:
        raise ValueError(f"position is int32 [tokens, top_k], got {list(position.shape)}")
    T, k = position.shape
    return (T, k, _vector(position, T * k, torch.int32, "position"),
            None if weights is None else _vector(weights, T * k, torch.float32, "weights"))


@_device_operands
def mxq_combine_rows(rows: torch.Tensor, position: torch.Tensor, weights: Optional[torch.Tensor] = None,
                     out: Optional[torch.Tensor] = None, lib: str = "libmxq.so") -> torch.Tensor:
    """Sorted rows (bf16 / fp32 [rows, H]) back to their tokens: y[t] = sum over j of weights[t, j] *
    rows[position[t, j]] -> [tokens, H].  `weights` fp32 [tokens, top_k], None: all 1."""
    L = _library(lib)
    pr, R, H, ldr = _mat(rows)
    T, k, pp, pw = _slots_of(position, weights)
    out, py, ldy, _, dt = _result(rows, out, (T, H), rows.dtype)
    if out.dtype != rows.dtype:
        raise ValueError("out must have the rows' dtype")
    _check(L, L.mxq_combine_rows(pr, ldr, R, pp, pw, T, k, H, dt, py, ldy, _handle(rows)))
    return out


@_device_operands
def mxq_combine_rows_backward(dy: torch.Tensor, rows: torch.Tensor, position: torch.Tensor,
                              weights: Optional[torch.Tensor] = None, drows: Optional[torch.Tensor] = None,
                              dweights: Optional[torch.Tensor] = None, lib: str = "libmxq.so"):
    """Gradients of mxq_combine_rows for dy [tokens, H] -> (drows [rows, H], dweights fp32 [tokens, top_k]).
    `position` names a row at most once, as mxq_sort_experts returns it.  Where `rows` has more of them than
    there are slots, the gradient of the others is 0; a `drows` that is given keeps what it holds there."""
    L = _library(lib)
    pg, T0, H, ldg = _mat(dy)
    pr, R, hr, ldr = _mat(rows)
    T, k, pp, pw = _slots_of(position, weights)
    if (T0, hr) != (T, H) or dy.dtype != rows.dtype:
        raise ValueError(f"dy is [tokens, H] of the rows' dtype, got {dy.dtype} {list(dy.shape)} for "
                         f"{T} tokens and rows {rows.dtype} {list(rows.shape)}")
    if drows is None and R > T * k:
        drows = torch.zeros((R, H), dtype=rows.dtype, device=rows.device)
    drows, pd, ldd, _, dt = _result(dy, drows, (R, H), rows.dtype)
    if drows.dtype != rows.dtype:
        raise ValueError("drows must have the rows' dtype")
    if dweights is None:
        dweights = torch.empty((T, k), dtype=torch.float32, device=dy.device)
    pv = _vector(dweights, T * k, torch.float32, "dweights")
    _check(L, L.mxq_combine_rows_backward(pg, ldg, pr, ldr, R, pp, pw, T, k, H, dt, pd, ldd, pv, _handle(dy)))
    return drows, dweights


# ---- between the FP8 products: norm, activation, routing -----------------------------------

def _weight_of(weight: Optional[torch.Tensor], K: int):
    """(pointer, dtype code) of a norm's weight."""
    if weight is None:
        return None, MXQ_FP32
    if weight.shape != (K,) or not weight.is_contiguous():
        raise ValueError(f"weight is a contiguous tensor of {K} elements, got {list(weight.shape)}")
    return weight.data_ptr(), _float_code(weight)


def _same_rows(t: torch.Tensor, rows: int, cols: int, what: str):
    """(pointer, row stride) of an input [rows, cols], no more and no less."""
    p, r, c, ld = _mat(t)
    if (r, c) != (rows, cols):
        raise ValueError(f"{what} is [{rows}, {cols}], got {list(t.shape)}")
    return p, ld


def _float_out(like: torch.Tensor, out: Optional[torch.Tensor], rows: int, cols: int, dtype: torch.dtype, what: str):
    """(tensor, pointer, row stride) of a floating output shaped as `like`, allocated if missing."""
    if out is None:
        out = torch.empty_like(like, dtype=dtype, memory_format=torch.contiguous_format)
        return out, out.data_ptr(), cols
    if out.dtype != dtype:
        raise ValueError(f"{what} must be {dtype}, got {out.dtype}")
    return (out, *_same_rows(out, rows, cols, what))


def _vector_out(like: torch.Tensor, out: Optional[torch.Tensor], shape, dtype: torch.dtype, what: str):
    """(tensor, pointer) of a contiguous output, allocated if missing."""
    if out is None:
        out = like.new_empty(shape, dtype=dtype)
        return out, out.data_ptr()
    n = 1
    for s in shape:
        n *= s
    return out, _vector(out, n, dtype, what)


def _norm_operands(x, weight, eps, residual, residual_out, y, with_y):
    """The norm's leading arguments, rows, K, and its floating outputs (s or None, y or None)."""
    px, rows, K, ldx = _mat(x)
    pw, wdt = _weight_of(weight, K)
    dt = _float_code(x)
    if residual is None:
        if residual_out is not None:
            raise ValueError("residual_out needs a residual")
        pr, ldr, rdt, s, ps, lds = None, 0, dt, None, None, 0
    else:
        rdt = _float_code(residual)
        pr, ldr = _same_rows(residual, rows, K, "residual")
        s, ps, lds = _float_out(x, residual_out, rows, K, residual.dtype, "residual_out")
    py, ldy = None, 0
    if y is not None or with_y:
        y, py, ldy = _float_out(x, y, rows, K, x.dtype, "y")
    return (px, ldx, pr, ldr, rdt, pw, wdt, eps, rows, K, dt, ps, lds, py, ldy), rows, K, s, y


@_device_operands
def mxq_rms_norm(x: torch.Tensor, weight: Optional[torch.Tensor], eps: float = 1e-6,
                 residual: Optional[torch.Tensor] = None, residual_out: Optional[torch.Tensor] = None,
                 y: Optional[torch.Tensor] = None, lib: str = "libmxq.so"):
    """y = s / sqrt(mean(s^2) + eps) * weight over each row of s = x + residual (bf16 / fp32), s rounded
    to the residual's type -> (y of x's type, s).  s goes to `residual_out`, which may be `residual`
    itself; without a residual s is x and None comes back for it.  `weight` [K] bf16 / fp32, None: all 1."""
    L = _library(lib)
    args, _, _, s, y = _norm_operands(x, weight, eps, residual, residual_out, y, True)
    _check(L, L.mxq_rms_norm(*args, _handle(x)))
    return y, s


@_device_operands
def mxq_rms_norm_fp8_group128(x: torch.Tensor, weight: Optional[torch.Tensor], eps: float = 1e-6,
                              residual: Optional[torch.Tensor] = None, residual_out: Optional[torch.Tensor] = None,
                              y: Optional[torch.Tensor] = None, with_y: bool = False,
                              data: Optional[torch.Tensor] = None, scale: Optional[torch.Tensor] = None,
                              lib: str = "libmxq.so"):
    """The norm in FP8, groups of 128 along the rows -> (payload uint8 [rows, K], codes uint8
    [rows, ceil(K/128)], s, y).  s as mxq_rms_norm returns it; y None unless `with_y` or a tensor for it."""
    L = _library(lib)
    args, rows, K, s, y = _norm_operands(x, weight, eps, residual, residual_out, y, with_y)
    data, pd, ldd = _bytes_for(x, data, rows, K, "payload")
    scale, pc, ldc = _bytes_for(x, scale, rows, _ng(K), "scale")
    _check(L, L.mxq_rms_norm_fp8_group128(*args, pd, ldd, pc, ldc, _handle(x)))
    return data, scale, s, y


@_device_operands
def mxq_rms_norm_fp8_group128_row_col(x: torch.Tensor, weight: Optional[torch.Tensor], eps: float = 1e-6,
                                      residual: Optional[torch.Tensor] = None,
                                      residual_out: Optional[torch.Tensor] = None, y: Optional[torch.Tensor] = None,
                                      with_y: bool = False, row_data: Optional[torch.Tensor] = None,
                                      row_scale: Optional[torch.Tensor] = None, col_data: Optional[torch.Tensor] = None,
                                      col_scale: Optional[torch.Tensor] = None, lib: str = "libmxq.so"):
    """The norm in FP8, groups of 128 along the rows and along the columns (the operand of a weight
    gradient) -> (row payload, row codes, column payload, column codes, s, y)."""
    L = _library(lib)
    args, rows, K, s, y = _norm_operands(x, weight, eps, residual, residual_out, y, with_y)
    row_data, prd, ldrd = _bytes_for(x, row_data, rows, K, "row payload")
    row_scale, prs, ldrs = _bytes_for(x, row_scale, rows, _ng(K), "row_scale")
    col_data, pcd, ldcd = _bytes_for(x, col_data, rows, K, "column payload")
    col_scale, pcs, ldcs = _bytes_for(x, col_scale, _ng(rows), K, "col_scale")
    need = L.mxq_rms_norm_fp8_group128_row_col_workspace(rows)
    ws = x.new_empty((need,), dtype=_UINT8)
    _check(L, L.mxq_rms_norm_fp8_group128_row_col(*args, prd, ldrd, prs, ldrs, pcd, ldcd, pcs, ldcs, ws.data_ptr(), need,
                                                  _handle(x)))
    return row_data, row_scale, col_data, col_scale, s, y


@_device_operands
def mxq_rms_norm_backward(dy: torch.Tensor, x: torch.Tensor, weight: Optional[torch.Tensor], eps: float = 1e-6,
                          dresidual: Optional[torch.Tensor] = None, dx: Optional[torch.Tensor] = None,
                          dweight: Optional[torch.Tensor] = None, lib: str = "libmxq.so"):
    """Gradients of the norm for dy -> (dx of x's type, dweight fp32 [K]).  `x` is what was normalized: s where
    there was a residual.  `dresidual` (x's type) is the gradient that reaches s past the norm; dx holds
    both, the gradient of the norm's x and of its residual alike."""
    L = _library(lib)
    px, rows, K, ldx = _mat(x)
    pg, ldg = _same_rows(dy, rows, K, "dy")
    pw, wdt = _weight_of(weight, K)
    pr, ldr = None, 0
    if dresidual is not None:
        if dresidual.dtype != x.dtype:
            raise ValueError(f"dresidual must be {x.dtype}, got {dresidual.dtype}")
        pr, ldr = _same_rows(dresidual, rows, K, "dresidual")
    dx, pd, ldd = _float_out(x, dx, rows, K, x.dtype, "dx")
    dweight, pv = _vector_out(x, dweight, (K,), _FLOAT32, "dweight")
    need = L.mxq_rms_norm_backward_workspace(rows, K)
    ws = x.new_empty((need,), dtype=_UINT8)
    _check(L, L.mxq_rms_norm_backward(pg, ldg, _float_code(dy), px, ldx, _float_code(x), pw, wdt, eps, pr, ldr, rows, K,
                                      pd, ldd, pv, ws.data_ptr(), need, _handle(x)))
    return dx, dweight


_ACTIVATIONS = {"silu": MXQ_SILU, "gelu_tanh": MXQ_GELU_TANH, "relu2": MXQ_RELU2}
_SCORES = {"softmax": MXQ_SOFTMAX, "sigmoid": MXQ_SIGMOID}


def _named(names: dict, name: str, what: str) -> int:
    if name not in names:
        raise ValueError(f"{what} is one of {', '.join(names)}, got {name!r}")
    return names[name]


def _halves(gate: torch.Tensor, up: Optional[torch.Tensor], activation: str):
    """The activation's leading arguments, rows and F."""
    pg, rows, F, ldg = _mat(gate)
    pu, ldu = None, 0
    if up is not None:
        if up.dtype != gate.dtype:
            raise ValueError(f"gate and up must have one dtype, got {gate.dtype} and {up.dtype}")
        pu, ldu = _same_rows(up, rows, F, "up")
        pu = pu or 16                   # a tensor of no rows has no address, and none would stand for no second half
    return (pg, ldg, pu, ldu, rows, F, _float_code(gate), _named(_ACTIVATIONS, activation, "activation")), rows, F


@_device_operands
def mxq_activate_fp8_group128(gate: torch.Tensor, up: Optional[torch.Tensor] = None, activation: str = "silu",
                              data: Optional[torch.Tensor] = None, scale: Optional[torch.Tensor] = None,
                              lib: str = "libmxq.so"):
    """act(gate) * up (bf16 / fp32 [rows, F], `up` None: act(gate)) in FP8, groups of 128 along the rows ->
    (payload uint8 [rows, F], codes uint8 [rows, ceil(F/128)]).  `activation`: "silu", "gelu_tanh" or "relu2"
    (the squared relu).  gate and up may be the halves of one matrix: h[:, :F], h[:, F:]."""
    L = _library(lib)
    args, rows, F = _halves(gate, up, activation)
    data, pd, ldd = _bytes_for(gate, data, rows, F, "payload")
    scale, ps, lds = _bytes_for(gate, scale, rows, _ng(F), "scale")
    _check(L, L.mxq_activate_fp8_group128(*args, pd, ldd, ps, lds, _handle(gate)))
    return data, scale


@_device_operands
def mxq_activate_fp8_group128_row_col(gate: torch.Tensor, up: Optional[torch.Tensor] = None, activation: str = "silu",
                                      offsets: Optional[torch.Tensor] = None,
                                      row_data: Optional[torch.Tensor] = None, row_scale: Optional[torch.Tensor] = None,
                                      col_data: Optional[torch.Tensor] = None, col_scale: Optional[torch.Tensor] = None,
                                      lib: str = "libmxq.so"):
    """The same with groups of 128 along the rows and along the columns, these begun anew with each expert's rows
    where `offsets` is given -> (row payload, row codes, column payload, column codes)."""
    L = _library(lib)
    args, rows, F = _halves(gate, up, activation)
    po, n = (None, 0) if offsets is None else _experts_of(offsets)
    row_data, prd, ldrd = _bytes_for(gate, row_data, rows, F, "row payload")
    row_scale, prs, ldrs = _bytes_for(gate, row_scale, rows, _ng(F), "row_scale")
    col_data, pcd, ldcd = _bytes_for(gate, col_data, rows, F, "column payload")
    col_scale, pcs, ldcs = _bytes_for(gate, col_scale, _code_rows(rows, n), F, "col_scale")
    _check(L, L.mxq_activate_fp8_group128_row_col(*args, po, n, prd, ldrd, prs, ldrs, pcd, ldcd, pcs, ldcs,
                                                  _handle(gate)))
    return row_data, row_scale, col_data, col_scale


@_device_operands
def mxq_activate_fp8_group128_backward(da: torch.Tensor, gate: torch.Tensor, up: Optional[torch.Tensor] = None,
                                       activation: str = "silu", offsets: Optional[torch.Tensor] = None,
                                       row_data: Optional[torch.Tensor] = None,
                                       row_scale: Optional[torch.Tensor] = None,
                                       col_data: Optional[torch.Tensor] = None,
                                       col_scale: Optional[torch.Tensor] = None, lib: str = "libmxq.so"):
    """Gradients of gate and up for da [rows, F], side by side as one [rows, 2 F] ([rows, F] without `up`) in FP8
    with groups of 128 along the rows and along the columns: what the up projection's input and weight
    gradients take -> (row payload, row codes, column payload, column codes)."""
    L = _library(lib)
    args, rows, F = _halves(gate, up, activation)
    if da.dtype != gate.dtype:
        raise ValueError(f"da and gate must have one dtype, got {da.dtype} and {gate.dtype}")
    pa, lda = _same_rows(da, rows, F, "da")
    po, n = (None, 0) if offsets is None else _experts_of(offsets)
    K = F if up is None else 2 * F
    row_data, prd, ldrd = _bytes_for(gate, row_data, rows, K, "row payload")
    row_scale, prs, ldrs = _bytes_for(gate, row_scale, rows, _ng(K), "row_scale")
    col_data, pcd, ldcd = _bytes_for(gate, col_data, rows, K, "column payload")
    col_scale, pcs, ldcs = _bytes_for(gate, col_scale, _code_rows(rows, n), K, "col_scale")
    _check(L, L.mxq_activate_fp8_group128_backward(pa, lda, *args, po, n, prd, ldrd, prs, ldrs, pcd, ldcd, pcs, ldcs,
                                                   _handle(gate)))
    return row_data, row_scale, col_data, col_scale


def _logits_of(logits: torch.Tensor):
    if logits.dim() != 2:
        raise ValueError(f"logits is [tokens, experts], got {list(logits.shape)}")
    return _mat(logits)


@_device_operands
def mxq_route_experts(logits: torch.Tensor, top_k: int, bias: Optional[torch.Tensor] = None, score: str = "softmax",
                      renormalize: bool = True, scale: float = 1.0, n_groups: int = 1, top_groups: int = 1,
                      group_top: int = 1, mask: Optional[torch.Tensor] = None, ids: Optional[torch.Tensor] = None,
                      weights: Optional[torch.Tensor] = None, lib: str = "libmxq.so"):
    """Each token's experts and their weights from a router's logits (bf16 / fp32 [tokens, experts]) ->
    (ids int32 [tokens, top_k], weights fp32 [tokens, top_k]), the operands of mxq_sort_experts and
    mxq_combine_rows.  `score` "softmax" or "sigmoid"; `bias` fp32 [experts] is added to the scores for the choice
    alone; with `n_groups` > 1 only the experts of the `top_groups` best groups take part, a group ranked by
    its largest key (`group_top` 1) or by the sum of its two best (2).  The chosen scores are the weights,
    made to sum to 1 with `renormalize`, times `scale`.  An expert whose logit is -inf is closed;
    a token whose `mask` (bool [tokens]) is False has none.  Slots that no expert is left for hold -1 and 0."""
    L = _library(lib)
    pl, T, E, ldl = _logits_of(logits)
    pb = None if bias is None else _vector(bias, E, _FLOAT32, "bias")
    pm = None
    if mask is not None:
        if mask.dtype not in (torch.bool, _UINT8) or mask.numel() != T or not mask.is_contiguous():
            raise ValueError(f"mask is a contiguous bool tensor of {T} elements, got {mask.dtype} {list(mask.shape)}")
        pm = mask.data_ptr()
    if top_k < 1:
        raise ValueError(f"top_k is at least 1, got {top_k}")
    ids, pi = _vector_out(logits, ids, (T, top_k), _INT32, "ids")
    weights, pw = _vector_out(logits, weights, (T, top_k), _FLOAT32, "weights")
    _check(L, L.mxq_route_experts(pl, ldl, T, E, _float_code(logits), pb, pm, _named(_SCORES, score, "score"), renormalize,
                                  scale, n_groups, top_groups, group_top, top_k, pi, pw, _handle(logits)))
    return ids, weights


@_device_operands
def mxq_route_experts_backward(dweights: torch.Tensor, logits: torch.Tensor, ids: torch.Tensor, score: str = "softmax",
                               renormalize: bool = True, scale: float = 1.0, dlogits: Optional[torch.Tensor] = None,
                               lib: str = "libmxq.so") -> torch.Tensor:
    """Gradient of mxq_route_experts' logits for that of its weights, the choice `ids` held fixed ->
    [tokens, experts] of the logits' type.  `score`, `renormalize` and `scale` as in the forward call."""
    L = _library(lib)
    pl, T, E, ldl = _logits_of(logits)
    if ids.dim() != 2 or ids.shape[0] != T:
        raise ValueError(f"ids is int32 [{T}, top_k], got {list(ids.shape)}")
    top_k = ids.shape[1]
    pi, pg = _vector(ids, T * top_k, _INT32, "ids"), _vector(dweights, T * top_k, _FLOAT32, "dweights")
    dlogits, pd, ldd = _float_out(logits, dlogits, T, E, logits.dtype, "dlogits")
    _check(L, L.mxq_route_experts_backward(pg, pl, ldl, pi, T, E, top_k, _float_code(logits),
                                           _named(_SCORES, score, "score"), renormalize, scale, pd, ldd, _handle(logits)))
    return dlogits


# ---- convenience layer ------------------------------------------------------------------

class MXFP8Components(NamedTuple):
    """FP8 values and unpadded E8M0 scales of an MXFP8 rowwise tensor."""
    data: torch.Tensor        # payload viewed as float8 with the tensor's shape
    scale_inv: torch.Tensor   # uint8 E8M0 codes, shape (*shape[:-1], ceil(K/32))


def export_components(data: Optional[torch.Tensor], scale_storage: Optional[torch.Tensor], shape,
                      fp8_dtype: torch.dtype = torch.float8_e4m3fn, lib: str = "libmxq.so") -> MXFP8Components:
    """Export values and scales in a storage-independent layout.  The values are
    always a view of `data`; the scales are a view when the storage has exactly
    ceil(K/32) columns and a copy (made by the library's kernel) when it is
    padded.  Missing row-scaled data raises ValueError."""
    if data is None or scale_storage is None:
        raise ValueError("tensor has no row-scaled data to export")
    shape = tuple(shape)
    K = shape[-1]
    nb = (K + 31) // 32
    values = data.view(fp8_dtype).view(shape)
    scale2d = scale_storage.view(-1, scale_storage.shape[-1]) if scale_storage.dim() != 2 else scale_storage
    if scale2d.shape[1] == nb:
        scale_inv = scale2d
    else:
        scale_inv = mxq_export_mxfp8(data, scale2d, K, lib=lib)
    return MXFP8Components(values, scale_inv.view(*shape[:-1], nb))


def fake_quantize_mxfp4(t: torch.Tensor, lib: str = "libmxq.so") -> torch.Tensor:
    if t.dtype == torch.float16:
        raise TypeError("fp16 is not supported: the MXFP4 grid exceeds fp16's range")
    return mxq_fake_quantize_mxfp4(t, lib=lib)
