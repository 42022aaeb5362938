"""torch-facing wrappers of the C ABI: allocate outputs with torch (device
memory and the current stream are the only things torch supplies) and call
libnvfp4.so.  Every step of the computation runs in the library's kernels.
"""
import contextlib
import ctypes
import importlib.util
import math
import types
import warnings
from dataclasses import dataclass
from typing import Optional

import torch

from . import _lib as L
from .build import fastcall_path
from ._lib import (NVFP4_ALPHA_PROVIDED, NVFP4_AMAX_PROVIDED, NVFP4_BLOCK2D, NVFP4_COLWISE, NVFP4_FOUR_SIX,  # noqa: F401
                   NVFP4_GEMM_SCALE_LAYOUT, NVFP4_HEADROOM, NVFP4_INVERSE_RHT, NVFP4_MS_EDEN, NVFP4_OUT_BF16,
                   NVFP4_OUT_DTYPE_BF16, NVFP4_OUT_DTYPE_FP32, NVFP4_RHT, NVFP4_RHT_SR, NVFP4_RHT_SR_HW,
                   NVFP4_ROUTE_GROUP_PAIR, NVFP4_ROUTE_RENORM, NVFP4_ROUTE_SIGMOID, NVFP4_ROUTE_SOFTMAX,
                   NVFP4_ROWWISE, NVFP4_RTN, NVFP4_SINGLE_PASS, NVFP4_VECTOR_SCALES)


class NVFP4Error(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: {L.nvfp4_status_string(status)} (status {status})")
        self.status = status


def _check(status: int, what: str):
    if status != L.NVFP4_OK:
        raise NVFP4Error(status, what)


def _p(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _stream():
    return torch.cuda.current_stream().cuda_stream


def _need(t: Optional[torch.Tensor], numel: int, dtype, what: str, device=None):
    """Raise unless t can hold `numel` contiguous elements of `dtype` (on
    `device`): the library writes through raw pointers and cannot check."""
    if t is None:
        raise ValueError(f"{what}: buffer missing")
    if t.dtype != dtype:
        raise TypeError(f"{what}: dtype {t.dtype}, expected {dtype}")
    if device is not None and t.device != device:
        raise ValueError(f"{what}: on {t.device}, expected {device}")
    if not t.is_contiguous():
        raise ValueError(f"{what}: must be contiguous")
    if t.numel() < numel:
        raise ValueError(f"{what}: {t.numel()} elements, {numel} needed")


def _need_matrix(t: torch.Tensor, rows: int, cols: int, dtype, what: str, device=None):
    """A row-major matrix view of at least rows x cols (row stride >= cols)."""
    if t.dtype != dtype:
        raise TypeError(f"{what}: dtype {t.dtype}, expected {dtype}")
    if device is not None and t.device != device:
        raise ValueError(f"{what}: on {t.device}, expected {device}")
    if t.dim() != 2 or t.shape[0] < rows or t.shape[1] < cols or t.stride(1) != 1:
        raise ValueError(f"{what}: shape {tuple(t.shape)} / strides {t.stride()}, need a row-major "
                         f"[>= {rows}, >= {cols}] matrix")


def check_outputs(q: "QTensor", R: int, C: int, flags: int, device=None):
    """Raise unless q's buffers can take the outputs of nvfp4_quantize on an
    [R, C] tensor with these flags."""
    vec = bool(flags & NVFP4_VECTOR_SCALES)
    if flags & NVFP4_ROWWISE:
        _need(q.codes_row, R * (C // 2), torch.uint8, "codes_row", device)
        _need(q.scales_row, math.prod(scale_shape(R, C, flags)), torch.uint8, "scales_row", device)
        _need(q.alpha_row, R if vec else 1, torch.float32, "alpha_row", device)
    if flags & NVFP4_COLWISE:
        _need(q.codes_col, C * (R // 2), torch.uint8, "codes_col", device)
        _need(q.scales_col, math.prod(scale_shape(C, R, flags)), torch.uint8, "scales_col", device)
        _need(q.alpha_col, C if vec else 1, torch.float32, "alpha_col", device)
    if q.amax is not None:
        _need(q.amax, 2, torch.float32, "amax", device)


@dataclass
class QTensor:
    """NVFP4 outputs of one quantize call (device tensors)."""
    codes_row: Optional[torch.Tensor] = None
    scales_row: Optional[torch.Tensor] = None
    alpha_row: Optional[torch.Tensor] = None
    codes_col: Optional[torch.Tensor] = None
    scales_col: Optional[torch.Tensor] = None
    alpha_col: Optional[torch.Tensor] = None
    amax: Optional[torch.Tensor] = None


def scale_shape(rows: int, cols: int, flags: int):
    """Shape of the scale tensor of an operand [rows, cols] (cols = the
    blocked axis)."""
    if flags & NVFP4_GEMM_SCALE_LAYOUT:
        return (rows * (cols // 16),)
    if flags & NVFP4_BLOCK2D:
        return (rows // 16, cols // 16)
    return (rows, cols // 16)


def alloc_outputs(R: int, C: int, flags: int, device) -> QTensor:
    q = QTensor()
    u8 = dict(dtype=torch.uint8, device=device)
    vec = bool(flags & NVFP4_VECTOR_SCALES)   # one tensor scale per row / column
    if flags & NVFP4_ROWWISE:
        q.codes_row = torch.empty((R, C // 2), **u8)
        q.scales_row = torch.empty(scale_shape(R, C, flags), **u8)
        q.alpha_row = torch.empty(max(R, 1) if vec else 1, dtype=torch.float32, device=device)
    if flags & NVFP4_COLWISE:
        q.codes_col = torch.empty((C, R // 2), **u8)
        q.scales_col = torch.empty(scale_shape(C, R, flags), **u8)
        q.alpha_col = torch.empty(max(C, 1) if vec else 1, dtype=torch.float32, device=device)
    q.amax = torch.zeros(2, dtype=torch.float32, device=device)
    return q


def workspace_for(R: int, C: int, flags: int, device) -> Optional[torch.Tensor]:
    n = L.nvfp4_workspace_size(R, C, flags)
    return torch.empty(n, dtype=torch.uint8, device=device) if n else None


def nvfp4_amax(x: torch.Tensor, flags: int = 0, seed: int = 0, out: Optional[torch.Tensor] = None,
               status: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The amax values of Eq. 1 from one read of x with the C ABI's
    nvfp4_amax: [plain, rotated rows, rotated columns] as a float32 CUDA
    tensor of 3 (rotated entries with NVFP4_RHT and the orientation flag)."""
    if x.dtype != torch.bfloat16 or x.dim() != 2 or not x.is_cuda:
        raise TypeError("x must be a 2D bfloat16 CUDA tensor")
    if x.numel() and x.stride(1) != 1:
        raise ValueError("x must have unit column stride")
    R, C = x.shape
    ld = x.stride(0) if x.numel() else C
    if out is not None:
        _need(out, 3, torch.float32, "out", x.device)
    if status is not None:
        _need(status, 1, torch.int32, "status", x.device)
    a = out if out is not None else torch.empty(3, dtype=torch.float32, device=x.device)
    st = L.nvfp4_amax(_p(x), R, C, ld, flags, seed, _p(a), _p(status), _stream())
    _check(st, "nvfp4_amax")
    return a


def nvfp4_quantize(x: torch.Tensor, mode: int, flags: int, seed: int = 0, stream_id: int = 0,
                   alpha: Optional[torch.Tensor] = None, out: Optional[QTensor] = None,
                   workspace: Optional[torch.Tensor] = None,
                   status: Optional[torch.Tensor] = None, amax: Optional[torch.Tensor] = None) -> QTensor:
    """Quantize a 2D bf16 CUDA tensor (unit column stride) with the C ABI's
    nvfp4_quantize; allocates outputs and workspace when not given.  alpha
    (a device float) replaces Eq. 1 (NVFP4_ALPHA_PROVIDED); amax (the three
    device floats nvfp4_amax writes) replaces the amax pass
    (NVFP4_AMAX_PROVIDED)."""
    if x.dtype != torch.bfloat16 or x.dim() != 2 or not x.is_cuda:
        raise TypeError("x must be a 2D bfloat16 CUDA tensor")
    if x.numel() and x.stride(1) != 1:
        raise ValueError("x must have unit column stride")
    R, C = x.shape
    ld = x.stride(0) if x.numel() else C
    if alpha is not None and amax is not None:
        raise ValueError("give alpha or amax, not both")
    if alpha is not None:
        flags |= NVFP4_ALPHA_PROVIDED
    if amax is not None:
        if amax.dtype != torch.float32 or not amax.is_cuda or amax.device != x.device or amax.numel() < 3 \
                or not amax.is_contiguous():
            raise ValueError("amax must be a contiguous float32 tensor on x's device")
        flags |= NVFP4_AMAX_PROVIDED
        alpha = amax
    if out is not None:
        check_outputs(out, R, C, flags, x.device)
    if status is not None:
        _need(status, 1, torch.int32, "status", x.device)
    q = out if out is not None else alloc_outputs(R, C, flags, x.device)
    ws = workspace if workspace is not None else workspace_for(R, C, flags, x.device)
    qt = L.nvfp4_qtensor_t(_p(q.codes_row), _p(q.scales_row), _p(q.alpha_row), _p(q.codes_col),
                           _p(q.scales_col), _p(q.alpha_col), _p(q.amax), _p(status))
    st = L.nvfp4_quantize(_p(x), R, C, ld, mode, flags, seed, stream_id, _p(alpha), qt, _p(ws),
                          0 if ws is None else ws.numel(), _stream())
    _check(st, "nvfp4_quantize")
    return q


def nvfp4_dequantize(codes: torch.Tensor, scales: torch.Tensor, alpha: torch.Tensor, R: int, C: int,
                     flags: int = 0, seed: int = 0, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Decode [R, C/2] codes to fp32 (or bf16 with NVFP4_OUT_BF16)."""
    dtype = torch.bfloat16 if flags & NVFP4_OUT_BF16 else torch.float32
    if out is not None:
        _need(out, R * C, dtype, "out", codes.device)
    y = out if out is not None else torch.empty((R, C), dtype=dtype, device=codes.device)
    st = L.nvfp4_dequantize(_p(codes), _p(scales), _p(alpha), R, C, flags, seed, _p(y), _stream())
    _check(st, "nvfp4_dequantize")
    return y


def nvfp4_gemm(A: torch.Tensor, sA: torch.Tensor, alphaA: torch.Tensor, B: torch.Tensor,
               sB: torch.Tensor, alphaB: torch.Tensor, out_dtype: int = NVFP4_OUT_DTYPE_BF16,
               out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """D[M, N] = alphaA alphaB (A dequantized) (B dequantized)^T; A codes
    [M, K/2], B codes [N, K/2], scales in the GEMM layout."""
    M, K2 = A.shape
    N = B.shape[0]
    K = 2 * K2
    dt = torch.bfloat16 if out_dtype == NVFP4_OUT_DTYPE_BF16 else torch.float32
    if out is not None:
        _need_matrix(out, M, N, dt, "out", A.device)
    D = out if out is not None else torch.empty((M, N), dtype=dt, device=A.device)
    st = L.nvfp4_gemm(_p(A), _p(sA), _p(alphaA), _p(B), _p(sB), _p(alphaB), M, N, K, _p(D), out_dtype,
                      D.stride(0), None, 0, _stream())
    _check(st, "nvfp4_gemm")
    return D


def nvfp4_gemm_vector_scales(A: torch.Tensor, sA: torch.Tensor, alphaA: torch.Tensor, B: torch.Tensor,
                             sB: torch.Tensor, alphaB: torch.Tensor, out_dtype: int = NVFP4_OUT_DTYPE_BF16,
                             out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """nvfp4_gemm for operands quantized with NVFP4_VECTOR_SCALES: alphaA
    holds one tensor scale per row of A ([M]), alphaB one per row of B ([N])."""
    M, K2 = A.shape
    N = B.shape[0]
    K = 2 * K2
    _need(alphaA, M, torch.float32, "alphaA", A.device)
    _need(alphaB, N, torch.float32, "alphaB", A.device)
    dt = torch.bfloat16 if out_dtype == NVFP4_OUT_DTYPE_BF16 else torch.float32
    if out is not None:
        _need_matrix(out, M, N, dt, "out", A.device)
    D = out if out is not None else torch.empty((M, N), dtype=dt, device=A.device)
    st = L.nvfp4_gemm_vector_scales(_p(A), _p(sA), _p(alphaA), _p(B), _p(sB), _p(alphaB), M, N, K, _p(D),
                                    out_dtype, D.stride(0), None, 0, _stream())
    _check(st, "nvfp4_gemm_vector_scales")
    return D


def nvfp4_gemm_quantize(A: torch.Tensor, sA: torch.Tensor, alphaA: torch.Tensor, B: torch.Tensor,
                        sB: torch.Tensor, alphaB: torch.Tensor, mode: int, alpha_out: torch.Tensor,
                        flags: int = NVFP4_GEMM_SCALE_LAYOUT, write_d: bool = True,
                        out: Optional[torch.Tensor] = None):
    """nvfp4_gemm with the bf16 output also quantized rowwise in the epilogue
    (RTN or FOUR_SIX, tensor scale alpha_out).  Returns (D or None, codes
    [M, N/2], scales, amax [1])."""
    M, K2 = A.shape
    N = B.shape[0]
    K = 2 * K2
    dev = A.device
    D = None
    if write_d:
        if out is not None:
            _need_matrix(out, M, N, torch.bfloat16, "out", dev)
        D = out if out is not None else torch.empty((M, N), dtype=torch.bfloat16, device=dev)
    codes = torch.empty((M, N // 2), dtype=torch.uint8, device=dev)
    scales = torch.empty((M, N // 16), dtype=torch.uint8, device=dev)
    amax = torch.empty(1, dtype=torch.float32, device=dev)
    st = L.nvfp4_gemm_quantize(_p(A), _p(sA), _p(alphaA), _p(B), _p(sB), _p(alphaB), M, N, K,
                               _p(D) if D is not None else None, D.stride(0) if D is not None else N,
                               mode, flags, _p(alpha_out), _p(codes), _p(scales), _p(amax), None, 0, _stream())
    _check(st, "nvfp4_gemm_quantize")
    return D, codes, scales, amax


@dataclass
class MXTensor:
    """MXFP4 outputs of one quantize call (device tensors): codes [rows, len/2],
    UE8M0 scale bytes [rows, len/32] per requested orientation."""
    codes_row: Optional[torch.Tensor] = None
    scales_row: Optional[torch.Tensor] = None
    codes_col: Optional[torch.Tensor] = None
    scales_col: Optional[torch.Tensor] = None


def mx_alloc_outputs(R: int, C: int, flags: int, device) -> MXTensor:
    """Output buffers of mxfp4_quantize on an [R, C] tensor: codes [rows,
    len/2] and UE8M0 scales [rows, len/32] (flat in the GEMM layout)."""
    q = MXTensor()
    u8 = dict(dtype=torch.uint8, device=device)
    gemm = bool(flags & NVFP4_GEMM_SCALE_LAYOUT)
    if flags & NVFP4_ROWWISE:
        q.codes_row = torch.empty((R, C // 2), **u8)
        q.scales_row = torch.empty((R * (C // 32),) if gemm else (R, C // 32), **u8)
    if flags & NVFP4_COLWISE:
        q.codes_col = torch.empty((C, R // 2), **u8)
        q.scales_col = torch.empty((C * (R // 32),) if gemm else (C, R // 32), **u8)
    return q


def mx_check_outputs(q: MXTensor, R: int, C: int, flags: int, device=None):
    """Raise unless q's buffers can take the outputs of mxfp4_quantize."""
    if flags & NVFP4_ROWWISE:
        _need(q.codes_row, R * (C // 2), torch.uint8, "codes_row", device)
        _need(q.scales_row, R * (C // 32), torch.uint8, "scales_row", device)
    if flags & NVFP4_COLWISE:
        _need(q.codes_col, C * (R // 2), torch.uint8, "codes_col", device)
        _need(q.scales_col, C * (R // 32), torch.uint8, "scales_col", device)


def mxfp4_quantize(x: torch.Tensor, flags: int, seed: int = 0, status: Optional[torch.Tensor] = None,
                   out: Optional[MXTensor] = None) -> MXTensor:
    """Quantize a 2D bf16 CUDA tensor (unit column stride) to MXFP4 with the C
    ABI's mxfp4_quantize (flags: NVFP4_ROWWISE / NVFP4_COLWISE, NVFP4_RHT)."""
    if x.dtype != torch.bfloat16 or x.dim() != 2 or not x.is_cuda:
        raise TypeError("x must be a 2D bfloat16 CUDA tensor")
    if x.numel() and x.stride(1) != 1:
        raise ValueError("x must have unit column stride")
    R, C = x.shape
    ld = x.stride(0) if x.numel() else C
    if out is not None:
        mx_check_outputs(out, R, C, flags, x.device)
    if status is not None:
        _need(status, 1, torch.int32, "status", x.device)
    q = out if out is not None else mx_alloc_outputs(R, C, flags, x.device)
    st = L.mxfp4_quantize(_p(x), R, C, ld, flags, seed, _p(q.codes_row), _p(q.scales_row), _p(q.codes_col),
                          _p(q.scales_col), _p(status), _stream())
    _check(st, "mxfp4_quantize")
    return q


def mxfp4_dequantize(codes: torch.Tensor, scales: torch.Tensor, R: int, C: int, flags: int = 0, seed: int = 0,
                     out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Decode MXFP4 codes [R, C/2] and scales [R, C/32] to fp32 (or bf16 with
    NVFP4_OUT_BF16)."""
    dtype = torch.bfloat16 if flags & NVFP4_OUT_BF16 else torch.float32
    if out is not None:
        _need(out, R * C, dtype, "out", codes.device)
    y = out if out is not None else torch.empty((R, C), dtype=dtype, device=codes.device)
    st = L.mxfp4_dequantize(_p(codes), _p(scales), R, C, flags, seed, _p(y), _stream())
    _check(st, "mxfp4_dequantize")
    return y


def mxfp4_gemm(A: torch.Tensor, sA: torch.Tensor, B: torch.Tensor, sB: torch.Tensor,
               out_dtype: int = NVFP4_OUT_DTYPE_BF16, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """D[M, N] = (A dequantized) (B dequantized)^T for MXFP4 operands: codes
    [M, K/2] and [N, K/2], UE8M0 scales in the GEMM layout."""
    M, K2 = A.shape
    N = B.shape[0]
    K = 2 * K2
    dt = torch.bfloat16 if out_dtype == NVFP4_OUT_DTYPE_BF16 else torch.float32
    if out is not None:
        _need_matrix(out, M, N, dt, "out", A.device)
    D = out if out is not None else torch.empty((M, N), dtype=dt, device=A.device)
    st = L.mxfp4_gemm(_p(A), _p(sA), _p(B), _p(sB), M, N, K, _p(D), out_dtype, D.stride(0), None, 0, _stream())
    _check(st, "mxfp4_gemm")
    return D


# ---------------------------------------------------------------------------
# Ragged groups (the expert layers of a mixture model): rows sorted by group,
# offsets [E + 1] on the device.
# ---------------------------------------------------------------------------
def _check_groups(offsets: torch.Tensor, device) -> int:
    """Number of groups of an offsets tensor (int32 [E + 1] on `device`)."""
    if offsets.dtype != torch.int32 or offsets.dim() != 1:
        raise TypeError("offsets must be a 1D int32 tensor of E + 1 values")
    if offsets.numel() < 2:
        raise ValueError("offsets: at least two values (one group) are needed")
    _need(offsets, 2, torch.int32, "offsets", device)
    return offsets.numel() - 1


def _check_status(status: Optional[torch.Tensor], device):
    if status is not None:
        _need(status, 1, torch.int32, "status", device)


# The small calls of these operators take a few microseconds on the GPU, so
# their host path avoids what costs as much: the current stream's raw handle
# instead of a stream object (2.2 us), a device guard only where the tensors
# are not on the current device (1.4 us), sizes computed here.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_device = getattr(torch._C, "_cuda_getDevice", None)
_HERE = contextlib.nullcontext()


def _stream_of(device):
    if _raw_stream is None:
        return torch.cuda.current_stream(device).cuda_stream
    return _raw_stream(device.index)


def _guard(device):
    """Context in which `device` is current."""
    if device.type != "cuda":
        raise TypeError(f"the tensors must be CUDA tensors, not on {device}")
    if _current_device is not None and _current_device() == device.index:
        return _HERE
    return torch.cuda.device(device)


def _capacity(T: int, E: int, step: int) -> int:
    """nvfp4_grouped_capacity."""
    return (T + min(T, E) * (step - 1)) // step * step


def grouped_alloc_outputs(T: int, C: int, E: int, flags: int, device) -> QTensor:
    """Output buffers of nvfp4_quantize_grouped: a row operand (codes [T, C/2],
    scales of the 128-row padded groups) and / or a column operand (codes
    [C, Kcap/2] and scales over the 64-row padded groups), one alpha per group,
    amax [2, E]."""
    row, col = bool(flags & NVFP4_ROWWISE), bool(flags & NVFP4_COLWISE)
    q = QTensor()
    f = torch.empty((2 + row + col, E), dtype=torch.float32, device=device)   # maxima first: a workspace too
    q.amax = f[:2]
    if row:
        q.codes_row = torch.empty((T, C // 2), dtype=torch.uint8, device=device)
        q.scales_row = torch.empty(_capacity(T, E, 128) * (C // 16), dtype=torch.uint8, device=device)
        q.alpha_row = f[2]
    if col:
        kcap = _capacity(T, E, 64)
        q.codes_col = torch.empty((C, kcap // 2), dtype=torch.uint8, device=device)
        q.scales_col = torch.empty(C * (kcap // 16), dtype=torch.uint8, device=device)
        q.alpha_col = f[2 + row]
    return q


def grouped_check_outputs(q: QTensor, T: int, C: int, E: int, flags: int, device=None):
    """Raise unless q's buffers can take the outputs of nvfp4_quantize_grouped."""
    if flags & NVFP4_ROWWISE:
        _need(q.codes_row, T * (C // 2), torch.uint8, "codes_row", device)
        _need(q.scales_row, _capacity(T, E, 128) * (C // 16), torch.uint8, "scales_row", device)
        _need(q.alpha_row, E, torch.float32, "alpha_row", device)
    if flags & NVFP4_COLWISE:
        kcap = _capacity(T, E, 64)
        _need(q.codes_col, C * (kcap // 2), torch.uint8, "codes_col", device)
        _need(q.scales_col, C * (kcap // 16), torch.uint8, "scales_col", device)
        _need(q.alpha_col, E, torch.float32, "alpha_col", device)
    if q.amax is not None:
        _need(q.amax, 2 * E, torch.float32, "amax", device)


def nvfp4_quantize_grouped(x: torch.Tensor, offsets: torch.Tensor, mode: int, flags: int, seed: int = 0,
                           stream_id: int = 0, out: Optional[QTensor] = None,
                           workspace: Optional[torch.Tensor] = None,
                           status: Optional[torch.Tensor] = None) -> QTensor:
    """Quantize rows sorted by group (x [T, C] bf16, group e: rows offsets[e]
    .. offsets[e + 1] - 1) with one tensor scale per group: operands of
    nvfp4_gemm_grouped (NVFP4_ROWWISE) and nvfp4_gemm_grouped_wgrad
    (NVFP4_COLWISE).  offsets stays on the device."""
    if x.dtype != torch.bfloat16 or x.dim() != 2 or not x.is_cuda:
        raise TypeError("x must be a 2D bfloat16 CUDA tensor")
    if x.numel() and x.stride(1) != 1:
        raise ValueError("x must have unit column stride")
    T, C = x.shape
    E = _check_groups(offsets, x.device)
    ld = x.stride(0) if T > 1 else C
    _check_status(status, x.device)
    if out is not None:
        grouped_check_outputs(out, T, C, E, flags, x.device)
    if workspace is not None:
        _need(workspace, 8 * E, torch.uint8, "workspace", x.device)
    with _guard(x.device):
        q = out if out is not None else grouped_alloc_outputs(T, C, E, flags, x.device)
        # without a workspace the groups' maxima are gathered where they are returned
        ws = workspace
        if ws is None:
            ws = q.amax if out is None else torch.empty((2, E), dtype=torch.float32, device=x.device)
        qt = L.nvfp4_qtensor_t(_p(q.codes_row), _p(q.scales_row), _p(q.alpha_row), _p(q.codes_col), _p(q.scales_col),
                               _p(q.alpha_col), _p(q.amax), _p(status))
        st = L.nvfp4_quantize_grouped(_p(x), T, C, ld, _p(offsets), E, mode, flags, seed, stream_id, qt, _p(ws),
                                      ws.numel() * ws.element_size(), _stream_of(x.device))
    _check(st, "nvfp4_quantize_grouped")
    return q


def nvfp4_dequantize_grouped(codes: torch.Tensor, scales: torch.Tensor, alpha: torch.Tensor, offsets: torch.Tensor,
                             T: int, C: int, flags: int, seed: int = 0, out: Optional[torch.Tensor] = None,
                             status: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Decode a grouped operand (flags: NVFP4_ROWWISE or NVFP4_COLWISE, as it
    was quantized) to [T, C] fp32, or bf16 with NVFP4_OUT_BF16.  Rows of no
    group are left as they are in `out` (unspecified in a new tensor)."""
    dev = codes.device
    E = _check_groups(offsets, dev)
    col = bool(flags & NVFP4_COLWISE)
    cap = _capacity(T, E, 64 if col else 128)
    _need(codes, C * (cap // 2) if col else T * (C // 2), torch.uint8, "codes", dev)
    _need(scales, cap * (C // 16), torch.uint8, "scales", dev)
    _need(alpha, E, torch.float32, "alpha", dev)
    _check_status(status, dev)
    dtype = torch.bfloat16 if flags & NVFP4_OUT_BF16 else torch.float32
    if out is not None:
        _need(out, T * C, dtype, "out", dev)
    with _guard(dev):
        y = out if out is not None else torch.empty((T, C), dtype=dtype, device=dev)
        st = L.nvfp4_dequantize_grouped(_p(codes), _p(scales), _p(alpha), T, C, _p(offsets), E, flags, seed, _p(y),
                                        _p(status), _stream_of(dev))
    _check(st, "nvfp4_dequantize_grouped")
    return y


def nvfp4_gemm_grouped(A: torch.Tensor, sA: torch.Tensor, alphaA: torch.Tensor, B: torch.Tensor, sB: torch.Tensor,
                       alphaB: torch.Tensor, offsets: torch.Tensor, out_dtype: int = NVFP4_OUT_DTYPE_BF16,
                       out: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None) -> torch.Tensor:
    """D[m] = alphaA[e] alphaB[e] A[m] B[e]^T for the rows m of each group e:
    A codes [T, K/2] and scales as nvfp4_quantize_grouped writes them
    (NVFP4_ROWWISE), B codes [E, N, K/2] with the experts' GEMM-layout scales
    one after the other, one alpha per group.  Rows of no group are left as
    they are in `out` (unspecified in a new tensor)."""
    dev = A.device
    if A.dim() != 2 or B.dim() != 3 or A.shape[1] != B.shape[2]:
        raise ValueError("A must be codes [T, K/2] and B codes [E, N, K/2]")
    E = _check_groups(offsets, dev)
    T, K2 = A.shape
    N, K = B.shape[1], 2 * K2
    if B.shape[0] != E:
        raise ValueError(f"B holds {B.shape[0]} experts, offsets {E}")
    _need(A, T * K2, torch.uint8, "A", dev)
    _need(B, E * N * K2, torch.uint8, "B", dev)
    _need(sA, _capacity(T, E, 128) * (K // 16), torch.uint8, "sA", dev)
    _need(sB, E * N * (K // 16), torch.uint8, "sB", dev)
    _need(alphaA, E, torch.float32, "alphaA", dev)
    _need(alphaB, E, torch.float32, "alphaB", dev)
    _check_status(status, dev)
    dt = torch.bfloat16 if out_dtype == NVFP4_OUT_DTYPE_BF16 else torch.float32
    if out is not None:
        _need_matrix(out, T, N, dt, "out", dev)
    with _guard(dev):
        D = out if out is not None else torch.empty((T, N), dtype=dt, device=dev)
        st = L.nvfp4_gemm_grouped(_p(A), _p(sA), _p(alphaA), _p(B), _p(sB), _p(alphaB), _p(offsets), E, T, N, K, _p(D),
                                  out_dtype, D.stride(0) if T > 1 else N, _p(status), _stream_of(dev))
    _check(st, "nvfp4_gemm_grouped")
    return D


def nvfp4_gemm_grouped_wgrad(A: torch.Tensor, sA: torch.Tensor, alphaA: torch.Tensor, B: torch.Tensor,
                             sB: torch.Tensor, alphaB: torch.Tensor, offsets: torch.Tensor, T: int,
                             out_dtype: int = NVFP4_OUT_DTYPE_FP32, out: Optional[torch.Tensor] = None,
                             status: Optional[torch.Tensor] = None) -> torch.Tensor:
    """D[e] = alphaA[e] alphaB[e] A_e B_e^T over the tokens of each group: A
    codes [M, Kcap/2] (the output gradient) and B codes [N, Kcap/2] (the
    layer's input) as nvfp4_quantize_grouped writes them (NVFP4_COLWISE) for
    the same T rows and offsets.  Groups without rows get zeros."""
    dev = A.device
    if A.dim() != 2 or B.dim() != 2:
        raise ValueError("A and B must be codes [M, Kcap/2] and [N, Kcap/2]")
    E = _check_groups(offsets, dev)
    M, N = A.shape[0], B.shape[0]
    kcap = _capacity(T, E, 64)
    if A.shape[1] != kcap // 2 or B.shape[1] != kcap // 2:
        raise ValueError(f"A and B must have {kcap // 2} bytes per row for T = {T}, E = {E}")
    _need(A, M * (kcap // 2), torch.uint8, "A", dev)
    _need(B, N * (kcap // 2), torch.uint8, "B", dev)
    _need(sA, M * (kcap // 16), torch.uint8, "sA", dev)
    _need(sB, N * (kcap // 16), torch.uint8, "sB", dev)
    _need(alphaA, E, torch.float32, "alphaA", dev)
    _need(alphaB, E, torch.float32, "alphaB", dev)
    _check_status(status, dev)
    dt = torch.bfloat16 if out_dtype == NVFP4_OUT_DTYPE_BF16 else torch.float32
    if out is not None:
        _need(out, E * M * N, dt, "out", dev)
    with _guard(dev):
        D = out if out is not None else torch.empty((E, M, N), dtype=dt, device=dev)
        st = L.nvfp4_gemm_grouped_wgrad(_p(A), _p(sA), _p(alphaA), _p(B), _p(sB), _p(alphaB), _p(offsets), E, T, M, N,
                                        _p(D), out_dtype, _p(status), _stream_of(dev))
    _check(st, "nvfp4_gemm_grouped_wgrad")
    return D


# ---------------------------------------------------------------------------
# Low-rank adapters of many requests beside a shared projection.
# ---------------------------------------------------------------------------
def _rows(t: torch.Tensor, T: int, cols: int, what: str, device):
    """Row stride of a bf16 matrix [T, cols] with unit column stride."""
    if t.dtype != torch.bfloat16:
        raise TypeError(f"{what}: dtype {t.dtype}, expected {torch.bfloat16}")
    if t.device != device:
        raise ValueError(f"{what}: on {t.device}, expected {device}")
    st = t.stride()
    if t.shape != (T, cols) or (T and st[1] != 1):
        raise ValueError(f"{what}: shape {tuple(t.shape)} / strides {st}, need a row-major [{T}, {cols}] matrix")
    return st[0] if T > 1 else cols


def _check_lora(A, B, scaling, ids, T, device):
    """(K, N, r, n) of adapters A [n, r, K], B [n, N, r] and the tokens' ids [T]."""
    sa, sb = A.shape, B.shape
    if len(sa) != 3 or len(sb) != 3 or sa[0] != sb[0] or sa[1] != sb[2]:
        raise ValueError("A must be [n, r, K] and B [n, N, r]")
    n, r, K = sa
    N = sb[1]
    _need(A, n * r * K, torch.bfloat16, "A", device)
    _need(B, n * N * r, torch.bfloat16, "B", device)
    _need(scaling, n, torch.float32, "scaling", device)
    if ids.shape != (T,):
        raise ValueError(f"ids: shape {tuple(ids.shape)}, need [{T}]")
    _need(ids, T, torch.int32, "ids", device)
    return K, N, r, n


def _lora_workspace(workspace, T, K, N, r, n, device):
    need = L.nvfp4_lora_workspace_size(T, K, N, r, n, True)
    if workspace is None:
        return torch.empty(max(need, 16), dtype=torch.uint8, device=device)
    _need(workspace, need, torch.uint8, "workspace", device)
    return workspace


def nvfp4_lora_apply(x: torch.Tensor, A: torch.Tensor, B: torch.Tensor, scaling: torch.Tensor, ids: torch.Tensor,
                     y: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                     h: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None):
    """out[t] = y[t] + scaling[a] B[a] (A[a] x[t]) with a = ids[t] (-1: y[t]
    alone), beside the shared projection y = nvfp4_gemm(x, frozen weight).
    x [T, K], y and out [T, N] bf16 (out may be y); A [n, r, K], B [n, N, r]
    bf16; scaling [n] fp32; ids [T] int32.  Returns (out, h) with h = A[a] x[t]
    (fp32 [T, r]), which nvfp4_lora_backward takes."""
    if x.dtype != torch.bfloat16 or x.dim() != 2 or not x.is_cuda:
        raise TypeError("x must be a 2D bfloat16 CUDA tensor")
    dev, T = x.device, x.shape[0]
    K, N, r, n = _check_lora(A, B, scaling, ids, T, dev)
    ldx = _rows(x, T, K, "x", dev)
    ldy = 0 if y is None else _rows(y, T, N, "y", dev)
    ldo = N if out is None else _rows(out, T, N, "out", dev)
    if h is not None:
        _need(h, T * r, torch.float32, "h", dev)
    _check_status(status, dev)
    with _guard(dev):
        if out is None:
            out = torch.empty((T, N), dtype=torch.bfloat16, device=dev)
        if h is None:
            h = torch.empty((T, r), dtype=torch.float32, device=dev)
        # h serves as the workspace, whose only use is to hold h
        st = L.nvfp4_lora_apply(_p(x), ldx, _p(A), _p(B), _p(scaling), _p(ids), T, K, N, r, n, _p(y), ldy, _p(out), ldo,
                                _p(h), _p(h), 4 * T * r, _p(status), _stream_of(dev))
    _check(st, "nvfp4_lora_apply")
    return out, h


def nvfp4_lora_backward(dy: torch.Tensor, x: torch.Tensor, h: torch.Tensor, A: torch.Tensor, B: torch.Tensor,
                        scaling: torch.Tensor, ids: torch.Tensor, dx: Optional[torch.Tensor] = None,
                        dx_out: Optional[torch.Tensor] = None, out_dtype: int = NVFP4_OUT_DTYPE_BF16,
                        workspace: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None):
    """Gradients of nvfp4_lora_apply: returns (dx, dA, dB) for the output
    gradient dy [T, N].  dx (bf16 [T, K], the shared projection's input
    gradient, optional) is added to the adapters' part; the sum goes to dx_out
    (which may be dx) or a new tensor.  h as the forward call returned it.  dA
    [n, r, K] and dB [n, N, r] are bf16 or fp32 (out_dtype); an adapter
    without tokens gets zeros."""
    if dy.dtype != torch.bfloat16 or dy.dim() != 2 or not dy.is_cuda:
        raise TypeError("dy must be a 2D bfloat16 CUDA tensor")
    dev, T = dy.device, dy.shape[0]
    K, N, r, n = _check_lora(A, B, scaling, ids, T, dev)
    lddy, ldx = _rows(dy, T, N, "dy", dev), _rows(x, T, K, "x", dev)
    _need(h, T * r, torch.float32, "h", dev)
    ld_in = 0 if dx is None else _rows(dx, T, K, "dx", dev)
    lddx = K if dx_out is None else _rows(dx_out, T, K, "dx_out", dev)
    _check_status(status, dev)
    dt = torch.bfloat16 if out_dtype == NVFP4_OUT_DTYPE_BF16 else torch.float32
    with _guard(dev):
        ws = _lora_workspace(workspace, T, K, N, r, n, dev)
        if dx_out is None:
            dx_out = torch.empty((T, K), dtype=torch.bfloat16, device=dev)
        dA = torch.empty((n, r, K), dtype=dt, device=dev)
        dB = torch.empty((n, N, r), dtype=dt, device=dev)
        st = L.nvfp4_lora_backward(_p(dy), lddy, _p(x), ldx, _p(h), _p(A), _p(B), _p(scaling), _p(ids), T, K, N, r, n,
                                   _p(dx), ld_in, _p(dx_out) if T else None, lddx, _p(dA), _p(dB), out_dtype, _p(ws),
                                   ws.numel(), _p(status), _stream_of(dev))
    _check(st, "nvfp4_lora_backward")
    return dx_out, dA, dB


# ---------------------------------------------------------------------------
# Around the experts' products: routing, sorting rows by expert, the way back,
# and products of a few unquantized rows.  Their small calls are as long as
# their host path, so each goes to C++ first (csrc/fastcall.cpp: 4 to 5 us a
# call).  What that declines, and every call where it is not built, goes through
# the checks below it: they say what is wrong, or make the call (9 to 11 us).
# Tensors on another device than the current one take a second call under it.
# ---------------------------------------------------------------------------
_SMALL = ("route", "route_backward", "dispatch", "combine", "combine_backward", "gemv")
_fast = None


def _load_fast():
    """The small calls' C++ host path, with the library's entry points.  Its
    functions return the results, a status, or None where a call is not of the
    plain form: then the checks below say what is wrong, or make the call.
    Where it is not built for this torch and Python they make every call."""
    global _fast
    lib = L.load()
    try:
        spec = importlib.util.spec_from_file_location(f"{__package__}._fastcall", fastcall_path())
        fast = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(fast)
        fast.use(*(ctypes.cast(getattr(lib, "nvfp4_" + n), ctypes.c_void_p).value for n in _SMALL))
    except ImportError as e:
        warnings.warn(f"the small calls take about 5 us longer: their C++ host path is not built for this torch and Python "
                      f"(nvfp4_block_quantization_amax_b200/build.py builds it): {e}", RuntimeWarning, stacklevel=3)
        fast = types.SimpleNamespace(**{n: lambda *args: None for n in _SMALL})
    _fast = fast
    return fast


def _new(rows: int, cols: int, dtype, device) -> torch.Tensor:
    return torch.empty_strided((rows, cols), (cols, 1), dtype=dtype, device=device)


def _within(v: int, most: int, what: str):
    """Raise unless 1 <= v <= most: a size of tensors that are yet to be made."""
    if not 1 <= v <= most:
        raise NVFP4Error(L.NVFP4_ERR_SHAPE, what)


def _elsewhere(device) -> bool:
    """Whether `device`, a GPU, is not the current one."""
    return (_current_device or torch.cuda.current_device)() != device.index


def _pairs(t: torch.Tensor, dtype, what: str, device):
    """Shape (T, k) of a contiguous tensor of one value per token and choice."""
    shape = t.shape
    if len(shape) != 2:
        raise ValueError(f"{what}: shape {tuple(shape)}, need [T, k]")
    if t.dtype is not dtype or t.device != device or not t.is_contiguous():
        _need(t, 0, dtype, what, device)
    return shape


def _like_pairs(t: torch.Tensor, shape, dtype, what: str, device):
    if t.shape != shape:
        raise ValueError(f"{what}: shape {tuple(t.shape)}, need {tuple(shape)}")
    if t.dtype is not dtype or t.device != device or not t.is_contiguous():
        _need(t, 0, dtype, what, device)


def _logits(t: torch.Tensor, what: str):
    """(row stride, dtype flag) of router logits, fp32 or bf16."""
    if t.dim() != 2 or not t.is_cuda:
        raise TypeError(f"{what} must be a 2D CUDA tensor")
    if t.dtype == torch.float32:
        kind = NVFP4_OUT_DTYPE_FP32
    elif t.dtype == torch.bfloat16:
        kind = NVFP4_OUT_DTYPE_BF16
    else:
        raise TypeError(f"{what}: dtype {t.dtype}, expected {torch.float32} or {torch.bfloat16}")
    T, E = t.shape
    stride = t.stride()
    if T and E > 1 and stride[1] != 1:
        raise ValueError(f"{what} must have unit column stride")
    return stride[0] if T > 1 else E, kind


def nvfp4_route(logits: torch.Tensor, k: int, score: int = NVFP4_ROUTE_SOFTMAX, flags: int = 0,
                bias: Optional[torch.Tensor] = None, groups: int = 1, groups_kept: int = 1, scale: float = 1.0,
                ids: Optional[torch.Tensor] = None, weights: Optional[torch.Tensor] = None,
                status: Optional[torch.Tensor] = None):
    """Choose k experts of each token from router logits [T, E] (fp32 or
    bf16): returns (ids [T, k] int32, weights [T, k] fp32), best first.
    score: NVFP4_ROUTE_SOFTMAX or NVFP4_ROUTE_SIGMOID; bias [E] fp32 is added
    for the choice alone; groups / groups_kept restrict it to the best groups
    of experts; flags: NVFP4_ROUTE_RENORM, NVFP4_ROUTE_GROUP_PAIR.  Experts
    with a logit of -inf are never chosen; -1 stands where none is left."""
    done = (_fast or _load_fast()).route(logits, k, score, flags, bias, groups, groups_kept, scale, ids, weights, status)
    if done.__class__ is tuple:
        return done
    if done is not None:
        _check(done, "nvfp4_route")
    ldl, kind = _logits(logits, "logits")
    dev = logits.device
    if _elsewhere(dev):
        with torch.cuda.device(dev):
            return nvfp4_route(logits, k, score, flags, bias, groups, groups_kept, scale, ids, weights, status)
    T, E = logits.shape
    _within(k, 32, "nvfp4_route")
    if bias is not None:
        _need(bias, E, torch.float32, "bias", dev)
    if ids is not None:
        _like_pairs(ids, (T, k), torch.int32, "ids", dev)
    if weights is not None:
        _like_pairs(weights, (T, k), torch.float32, "weights", dev)
    if status is not None:
        _check_status(status, dev)
    if ids is None:
        ids = _new(T, k, torch.int32, dev)
    if weights is None:
        weights = torch.empty_like(ids, dtype=torch.float32)
    st = L.nvfp4_route(
        logits.data_ptr(), ldl, kind, _p(bias), T, E, k, groups, groups_kept, score, flags, scale, ids.data_ptr(),
        weights.data_ptr(), _p(status), _stream_of(dev))
    if st:
        _check(st, "nvfp4_route")
    return ids, weights


def nvfp4_route_backward(dweights: torch.Tensor, ids: torch.Tensor, logits: torch.Tensor, score: int = NVFP4_ROUTE_SOFTMAX,
                         flags: int = 0, scale: float = 1.0, out: Optional[torch.Tensor] = None,
                         status: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Gradient of nvfp4_route's weights with respect to the logits ([T, E],
    the logits' type) for dweights [T, k]; ids, score, flags and scale as in
    the forward call.  out may be the logits."""
    done = (_fast or _load_fast()).route_backward(dweights, ids, logits, score, flags, scale, out, status)
    if done.__class__ is tuple:
        return done[0]
    if done is not None:
        _check(done, "nvfp4_route_backward")
    ldl, kind = _logits(logits, "logits")
    dev = logits.device
    if _elsewhere(dev):
        with torch.cuda.device(dev):
            return nvfp4_route_backward(dweights, ids, logits, score, flags, scale, out, status)
    T, E = logits.shape
    shape = _pairs(ids, torch.int32, "ids", dev)
    if shape[0] != T:
        raise ValueError(f"ids: {shape[0]} tokens, logits {T}")
    _like_pairs(dweights, shape, torch.float32, "dweights", dev)
    ldd = E
    if out is not None:
        if out.dtype != logits.dtype or out.device != dev or out.shape != logits.shape:
            raise ValueError("out must have the logits' type, device and shape")
        ldd = _logits(out, "out")[0]
    if status is not None:
        _check_status(status, dev)
    if out is None:
        out = torch.empty_like(logits) if logits.is_contiguous() else _new(T, E, logits.dtype, dev)
    st = L.nvfp4_route_backward(
        dweights.data_ptr(), ids.data_ptr(), logits.data_ptr(), ldl, kind, T, E, shape[1], score, flags, scale,
        out.data_ptr(), ldd, _p(status), _stream_of(dev))
    if st:
        _check(st, "nvfp4_route_backward")
    return out


def nvfp4_dispatch(x: Optional[torch.Tensor], ids: torch.Tensor, E: int, out: Optional[torch.Tensor] = None,
                   rows: Optional[torch.Tensor] = None, offsets: Optional[torch.Tensor] = None,
                   status: Optional[torch.Tensor] = None):
    """Sort token rows x [T, C] (bf16) by the experts ids [T, k]: returns (xs
    [T k, C], rows [T, k], offsets [E + 1]); xs and offsets are the operands of
    nvfp4_quantize_grouped, rows those of nvfp4_combine.  Rows of xs from
    offsets[E] on are left as they are (unspecified in a new tensor).  Without
    x only rows and offsets are computed (xs is None)."""
    done = (_fast or _load_fast()).dispatch(x, ids, E, out, rows, offsets, status)
    if done.__class__ is tuple:
        return done
    if done is not None:
        _check(done, "nvfp4_dispatch")
    if not ids.is_cuda:
        raise TypeError("ids must be a 2D int32 CUDA tensor")
    dev = ids.device
    if _elsewhere(dev):
        with torch.cuda.device(dev):
            return nvfp4_dispatch(x, ids, E, out, rows, offsets, status)
    T, k = _pairs(ids, torch.int32, "ids", dev)
    _within(E, 1024, "nvfp4_dispatch")
    C = ldx = ldo = 8
    if x is not None:
        if x.dim() != 2:
            raise ValueError("x must be [T, C]")
        C = x.shape[1]
        ldx, ldo = _rows(x, T, C, "x", dev), C
        if out is not None:
            ldo = _rows(out, T * k, C, "out", dev)
    elif out is not None:
        raise ValueError("out without x")
    if rows is not None:
        _like_pairs(rows, (T, k), torch.int32, "rows", dev)
    if offsets is not None:
        _need(offsets, E + 1, torch.int32, "offsets", dev)
    if status is not None:
        _check_status(status, dev)
    if rows is None:
        rows = torch.empty_like(ids)
    if offsets is None:
        offsets = torch.empty_strided((E + 1,), (1,), dtype=torch.int32, device=dev)
    if x is not None and out is None:
        out = _new(T * k, C, torch.bfloat16, dev)
    st = L.nvfp4_dispatch(
        _p(x), ldx, ids.data_ptr(), T, k, E, C, _p(out), ldo, offsets.data_ptr(), rows.data_ptr(), _p(status),
        _stream_of(dev))
    if st:
        _check(st, "nvfp4_dispatch")
    return out, rows, offsets


def _places(rows, weights, device):
    """Shape (T, k) of the pairs: that of rows, or of weights without rows."""
    if rows is not None:
        shape = _pairs(rows, torch.int32, "rows", device)
    elif weights is None:
        raise ValueError("rows or weights are needed")
    else:
        return _pairs(weights, torch.float32, "weights", device)
    if weights is not None:
        _like_pairs(weights, shape, torch.float32, "weights", device)
    return shape


def nvfp4_combine(y: torch.Tensor, rows: Optional[torch.Tensor], weights: Optional[torch.Tensor] = None,
                  residual: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                  status: Optional[torch.Tensor] = None) -> torch.Tensor:
    """out[t] = residual[t] + sum_j weights[t, j] y[rows[t, j]] (bf16 [T, C]):
    the experts' rows y [R, C] back to their tokens.  rows as nvfp4_dispatch
    returned them (-1: nothing), or None: y's rows are those of the pairs in
    order, as nvfp4_gemv returns them; weights [T, k] fp32, or all 1; residual
    optional, may be out.  Without weights it is nvfp4_dispatch's gradient."""
    done = (_fast or _load_fast()).combine(y, rows, weights, residual, out, status)
    if done.__class__ is tuple:
        return done[0]
    if done is not None:
        _check(done, "nvfp4_combine")
    if y.dtype != torch.bfloat16 or y.dim() != 2 or not y.is_cuda:
        raise TypeError("y must be a 2D bfloat16 CUDA tensor")
    dev = y.device
    if _elsewhere(dev):
        with torch.cuda.device(dev):
            return nvfp4_combine(y, rows, weights, residual, out, status)
    R, C = y.shape
    T, k = _places(rows, weights, dev)
    ldy = _rows(y, R, C, "y", dev)
    ldr = 0 if residual is None else _rows(residual, T, C, "residual", dev)
    ldo = C if out is None else _rows(out, T, C, "out", dev)
    if status is not None:
        _check_status(status, dev)
    if out is None:
        if residual is not None and residual.is_contiguous():
            out = torch.empty_like(residual)
        else:
            out = _new(T, C, torch.bfloat16, dev)
    st = L.nvfp4_combine(
        y.data_ptr(), ldy, R, _p(rows), _p(weights), T, k, C, _p(residual), ldr, out.data_ptr(), ldo, _p(status),
        _stream_of(dev))
    if st:
        _check(st, "nvfp4_combine")
    return out


def nvfp4_combine_backward(dout: torch.Tensor, rows: Optional[torch.Tensor], weights: Optional[torch.Tensor],
                           y: torch.Tensor, need_dy: bool = True, need_dweights: bool = True, out: Optional[torch.Tensor] = None,
                           status: Optional[torch.Tensor] = None):
    """Gradients of nvfp4_combine for dout [T, C]: returns (dy [R, C], dweights
    [T, k]), None in the place of one that is not needed.  rows, weights and y
    as in the forward call; no place may occur twice in rows.  Rows of dy that
    do not occur are left as they are in `out` (unspecified in a new tensor)."""
    done = (_fast or _load_fast()).combine_backward(dout, rows, weights, y, need_dy, need_dweights, out, status)
    if done.__class__ is tuple:
        return done
    if done is not None:
        _check(done, "nvfp4_combine_backward")
    if dout.dtype != torch.bfloat16 or dout.dim() != 2 or not dout.is_cuda:
        raise TypeError("dout must be a 2D bfloat16 CUDA tensor")
    dev = dout.device
    if _elsewhere(dev):
        with torch.cuda.device(dev):
            return nvfp4_combine_backward(dout, rows, weights, y, need_dy, need_dweights, out, status)
    T, C = dout.shape
    shape = _places(rows, weights, dev)
    if shape[0] != T:
        raise ValueError(f"rows: {shape[0]} tokens, dout {T}")
    if y.dim() != 2:
        raise ValueError("y must be [R, C]")
    R = y.shape[0]
    lddo, ldy = _rows(dout, T, C, "dout", dev), _rows(y, R, C, "y", dev)
    if out is not None and not need_dy:
        raise ValueError("out without need_dy")
    lddy = C if out is None else _rows(out, R, C, "out", dev)
    if status is not None:
        _check_status(status, dev)
    if need_dy and out is None:
        out = _new(R, C, torch.bfloat16, dev)
    dw = _new(shape[0], shape[1], torch.float32, dev) if need_dweights else None
    st = L.nvfp4_combine_backward(
        dout.data_ptr(), lddo, y.data_ptr(), ldy, R, _p(rows), _p(weights), T, shape[1], C, _p(out), lddy, _p(dw),
        _p(status), _stream_of(dev))
    if st:
        _check(st, "nvfp4_combine_backward")
    return out, dw


def nvfp4_gemv(x: torch.Tensor, W: torch.Tensor, sW: torch.Tensor, alphaW: torch.Tensor, ids: Optional[torch.Tensor] = None,
               out_dtype: int = NVFP4_OUT_DTYPE_BF16, out: Optional[torch.Tensor] = None,
               status: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Products of a few bf16 rows with NVFP4 weights, the rows not quantized
    (at most 1024 results).  Without ids: x [P, K], W codes [N, K/2] -> [P, N].
    With ids [T, k]: W codes [E, N, K/2], and x [T, K] (a token's choices share
    its row) or [T k, K] (a row each) -> [T k, N], zeros for a choice of -1.
    Scales in the GEMM layout, alphaW one float per weight."""
    done = (_fast or _load_fast()).gemv(x, W, sW, alphaW, ids, out_dtype, out, status)
    if done.__class__ is tuple:
        return done[0]
    if done is not None:
        _check(done, "nvfp4_gemv")
    if x.dtype != torch.bfloat16 or x.dim() != 2 or not x.is_cuda:
        raise TypeError("x must be a 2D bfloat16 CUDA tensor")
    dev = x.device
    if _elsewhere(dev):
        with torch.cuda.device(dev):
            return nvfp4_gemv(x, W, sW, alphaW, ids, out_dtype, out, status)
    X, K = x.shape
    if W.dim() != (2 if ids is None else 3) or 2 * W.shape[-1] != K:
        raise ValueError(f"W must be codes [{'' if ids is None else 'E, '}N, {K // 2}], not {tuple(W.shape)}")
    N = W.shape[-2]
    E = 1 if ids is None else W.shape[0]
    P, rep = X, 1
    if ids is not None:
        T, k = _pairs(ids, torch.int32, "ids", dev)
        P = T * k
        if X == T:
            rep = k
        elif X != P:
            raise ValueError(f"x: {X} rows, need {T} or {P}")
    if P:
        _within(P, 1024, "nvfp4_gemv")
    ldx = _rows(x, X, K, "x", dev)
    _need(W, E * N * (K // 2), torch.uint8, "W", dev)
    _need(sW, E * N * (K // 16), torch.uint8, "sW", dev)
    _need(alphaW, E, torch.float32, "alphaW", dev)
    if status is not None:
        _check_status(status, dev)
    dt = torch.bfloat16 if out_dtype == NVFP4_OUT_DTYPE_BF16 else torch.float32
    ldo = N
    if out is None:
        out = _new(P, N, dt, dev)
    else:
        _need_matrix(out, P, N, dt, "out", dev)
        if P > 1:
            ldo = out.stride(0)
    st = L.nvfp4_gemv(
        x.data_ptr(), ldx, _p(ids), P, rep or 1, W.data_ptr(), sW.data_ptr(), alphaW.data_ptr(), E, N, K, out.data_ptr(),
        out_dtype, ldo, _p(status), _stream_of(dev))
    if st:
        _check(st, "nvfp4_gemv")
    return out
