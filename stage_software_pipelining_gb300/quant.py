"""ctypes binding over libgemm.so's quantised-linear operators (include/quant.h).

Argument marshalling only, as in ``gemm.py``: tensors become (pointer, leading
dimension) pairs and a type code; all arithmetic runs in the CUDA kernels of
libgemm.so.  The caller owns every buffer, outputs included; ``empty_rows``
makes one whose rows start on 16-byte boundaries.
"""
from __future__ import annotations

import ctypes
import threading

import torch

from . import gemm as G
from .gemm import GemmError

QUANT_F32 = 0
QUANT_F16 = 1
QUANT_BF16 = 2

GROUPS = (32, 64, 128)          # K per scale of the 4-bit weights
E4M3_MAX = 448.0                # largest e4m3 value

# Every extern "C" symbol include/quant.h declares.
EXPORTS = ("add_rmsnorm", "quantize_fp8", "gemm_fp8", "gemm_fp8_checked", "gemv_w4", "quantize_w4")

_TYPES = {torch.float32: QUANT_F32, torch.float16: QUANT_F16, torch.bfloat16: QUANT_BF16}
_E4M3 = torch.float8_e4m3fn
_lock = threading.Lock()
_lib = None


def load_library():
    """libgemm.so with these operators' signatures.  Raises if it is missing."""
    global _lib
    with _lock:
        if _lib is None:
            lib = G.load_library()
            i64, p, i32, f32 = ctypes.c_int64, ctypes.c_void_p, ctypes.c_int, ctypes.c_float
            lib.add_rmsnorm.argtypes = [i64, i64, p, i64, p, i64, p, f32, i32, p, i64, p, i64, p,
                                        i64, p, p]
            lib.quantize_fp8.argtypes = [i64, i64, p, i64, i32, p, i64, p, p]
            lib.gemm_fp8.argtypes = [i64, i64, i64, p, i64, p, i64, p, i64, p, p, i32, p]
            lib.gemm_fp8_checked.argtypes = lib.gemm_fp8.argtypes
            lib.gemv_w4.argtypes = [i64, i64, i64, p, i64, p, i64, p, i64, p, i64, i32, p, i64,
                                    i32, p]
            lib.quantize_w4.argtypes = [i64, i64, p, i64, i32, i32, p, i64, p, i64, i32, p, i64, p]
            for name in EXPORTS:
                getattr(lib, name).restype = i32
            _lib = lib
        return _lib


def empty_rows(rows: int, cols: int, dtype: torch.dtype, device="cuda") -> torch.Tensor:
    """An uninitialised rows x cols tensor whose rows start on 16-byte
    boundaries, as gemm_fp8 (and the fast case of the row kernels) wants them."""
    unit = 16 // torch.empty((), dtype=dtype).element_size()
    return torch.empty((rows, (cols + unit - 1) // unit * unit), dtype=dtype,
                       device=device)[:, :cols]


def _type(t: torch.Tensor, name: str) -> int:
    try:
        return _TYPES[t.dtype]
    except KeyError:
        raise ValueError(f"{name} has unsupported type {t.dtype}") from None


def _rows(t: torch.Tensor, name: str, dtype, shape, device) -> int:
    """Leading dimension of a row-major matrix argument, after its checks."""
    if t.dtype != dtype:
        raise ValueError(f"{name} must have type {dtype}, not {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}")
    if tuple(t.shape) != shape:
        raise ValueError(f"{name} must be {shape}, not {tuple(t.shape)}")
    st = t.stride()
    if shape[1] > 1 and shape[0] > 0 and st[1] != 1:
        raise ValueError(f"{name} must be row-major (unit column stride)")
    if shape[0] > 1 and st[0] < shape[1]:
        raise ValueError(f"{name}'s rows overlap")
    return st[0]


def _vector(t: torch.Tensor, name: str, dtype, n: int, device) -> None:
    if t.dtype != dtype:
        raise ValueError(f"{name} must have type {dtype}, not {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}")
    if t.dim() != 1 or t.shape[0] != n:
        raise ValueError(f"{name} must have {n} elements, not {tuple(t.shape)}")
    if n > 1 and t.stride(0) != 1:
        raise ValueError(f"{name} must be contiguous")


def _matrix(t: torch.Tensor, name: str):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dim() != 2:
        raise ValueError(f"{name} must be 2-D")
    return t.device


def _call(name: str, device: torch.device, stream, *args) -> None:
    lib = _lib or load_library()
    s = (stream or torch.cuda.current_stream(device)).cuda_stream
    if device.index == torch.cuda.current_device():
        status = getattr(lib, name)(*args, s)
    else:
        with torch.cuda.device(device):
            status = getattr(lib, name)(*args, s)
    if status != G.GEMM_OK:
        raise GemmError(status, name)


def add_rmsnorm(x: torch.Tensor, weight: torch.Tensor, residual: torch.Tensor | None = None, *,
                eps: float = 1e-6, residual_out: torch.Tensor | None = None,
                y: torch.Tensor | None = None, q: torch.Tensor | None = None,
                scale: torch.Tensor | None = None,
                stream: torch.cuda.Stream | None = None) -> None:
    """h = x + residual, y = h / sqrt(mean(h^2) + eps) * weight a row, and its
    8-bit form q = e4m3(y / scale) with scale = max(max|y| / 448, 2^-126).

    x, residual, residual_out, y: rows x cols in fp32, fp16 or bf16 (one
    type); weight: cols of that type; q: rows x cols float8_e4m3fn; scale:
    rows fp32.  Outputs that are None are not computed; residual_out and y may
    be x or residual itself.  Raises ValueError or GemmError.
    """
    device = _matrix(x, "x")
    code = _type(x, "x")
    shape = tuple(x.shape)
    rows, cols = shape
    dt = x.dtype
    ldx = _rows(x, "x", dt, shape, device)
    _vector(weight, "weight", dt, cols, device)
    ldr = ldro = ldy = ldq = 0
    pr = pro = py = pq = ps = None
    if residual is not None:
        ldr, pr = _rows(residual, "residual", dt, shape, device), residual.data_ptr()
    if residual_out is not None:
        ldro = _rows(residual_out, "residual_out", dt, shape, device)
        pro = residual_out.data_ptr()
    if y is not None:
        ldy, py = _rows(y, "y", dt, shape, device), y.data_ptr()
    if (q is None) != (scale is None):
        raise ValueError("q and scale go together")
    if q is not None:
        ldq, pq = _rows(q, "q", _E4M3, shape, device), q.data_ptr()
        _vector(scale, "scale", torch.float32, rows, device)
        ps = scale.data_ptr()
    if residual_out is None and y is None and q is None:
        raise ValueError("add_rmsnorm needs an output: residual_out, y, or q with scale")
    if rows == 0:
        return
    _call("add_rmsnorm", device, stream, rows, cols, x.data_ptr(), ldx, pr, ldr,
          weight.data_ptr(), eps, code, pro, ldro, py, ldy, pq, ldq, ps)


def quantize_fp8(x: torch.Tensor, q: torch.Tensor, scale: torch.Tensor, *,
                 stream: torch.cuda.Stream | None = None) -> torch.Tensor:
    """q = e4m3(x / scale) with scale = max(max|x| / 448, 2^-126) a row: rows
    of activations, or a weight matrix stored N x K (a scale an output
    column).  x: fp32, fp16 or bf16; q: float8_e4m3fn; scale: fp32.  Returns q."""
    device = _matrix(x, "x")
    code = _type(x, "x")
    shape = tuple(x.shape)
    ldx = _rows(x, "x", x.dtype, shape, device)
    ldq = _rows(q, "q", _E4M3, shape, device)
    _vector(scale, "scale", torch.float32, shape[0], device)
    if shape[0]:
        _call("quantize_fp8", device, stream, shape[0], shape[1], x.data_ptr(), ldx, code,
              q.data_ptr(), ldq, scale.data_ptr())
    return q


def gemm_fp8(A: torch.Tensor, B: torch.Tensor, C: torch.Tensor, a_scale: torch.Tensor,
             b_scale: torch.Tensor, *, stream: torch.cuda.Stream | None = None,
             checked: bool = False) -> torch.Tensor:
    """C = diag(a_scale) A B diag(b_scale) in place (libgemm.so gemm_fp8, or
    gemm_fp8_checked, which synchronises and reports a wait that ran out).

    A: M x K float8_e4m3fn, row-major; B: K x N float8_e4m3fn, column-major (a
    transposed view of the N x K weights); C: M x N fp16 or bf16, row-major;
    a_scale, b_scale: M and N fp32.  A, B and C start on 16-byte boundaries
    and so do their rows (B's columns).  Returns C.
    """
    device = _matrix(A, "A")
    _matrix(B, "B")
    _matrix(C, "C")
    M, K = A.shape
    N = B.shape[1]
    if C.dtype != torch.float16 and C.dtype != torch.bfloat16:
        raise ValueError(f"C must be fp16 or bf16, not {C.dtype}")
    lda = _rows(A, "A", _E4M3, (M, K), device)
    ldb = _rows(B.t(), "B (transposed: B is column-major)", _E4M3, (N, K), device)
    ldc = _rows(C, "C", C.dtype, (M, N), device)
    _vector(a_scale, "a_scale", torch.float32, M, device)
    _vector(b_scale, "b_scale", torch.float32, N, device)
    _call("gemm_fp8_checked" if checked else "gemm_fp8", device, stream, M, N, K, A.data_ptr(), lda, B.data_ptr(), ldb, C.data_ptr(),
          ldc, a_scale.data_ptr(), b_scale.data_ptr(), _TYPES[C.dtype])
    return C


def gemv_w4(x: torch.Tensor, W: torch.Tensor, scales: torch.Tensor, C: torch.Tensor,
            zeros: torch.Tensor | None = None, *,
            stream: torch.cuda.Stream | None = None) -> torch.Tensor:
    """C = x @ ((w - zeros) * scales)^T with 4-bit weights w (libgemm.so gemv_w4).

    x: M x K fp16 or bf16; W: N x K/2 uint8, the even k in the low four bits;
    scales: N x K/group of x's type, group 32, 64 or 128; zeros: N x K/group
    uint8 (None: 8 everywhere); C: M x N of x's type.  x and W start on
    16-byte boundaries and so do their rows.  Returns C.
    """
    device = _matrix(x, "x")
    _matrix(W, "W")
    _matrix(scales, "scales")
    M, K = x.shape
    N = W.shape[0]
    dt = x.dtype
    if dt != torch.float16 and dt != torch.bfloat16:
        raise ValueError(f"x must be fp16 or bf16, not {dt}")
    groups = scales.shape[1]
    group = K // groups if groups else 32
    if (groups * group != K or group not in GROUPS):
        raise ValueError(f"K = {K} and {groups} scales a row: the group must be 32, 64 or 128")
    ldx = _rows(x, "x", dt, (M, K), device)
    ldw = _rows(W, "W", torch.uint8, (N, K // 2), device)
    lds = _rows(scales, "scales", dt, (N, groups), device)
    ldz, pz = 0, None
    if zeros is not None:
        ldz, pz = _rows(zeros, "zeros", torch.uint8, (N, groups), device), zeros.data_ptr()
    ldc = _rows(C, "C", dt, (M, N), device)
    _call("gemv_w4", device, stream, M, N, K, x.data_ptr(), ldx, W.data_ptr(), ldw,
          scales.data_ptr(), lds, pz, ldz, group, C.data_ptr(), ldc, _TYPES[dt])
    return C


def quantize_w4(w: torch.Tensor, W: torch.Tensor, scales: torch.Tensor,
                zeros: torch.Tensor | None = None, *,
                stream: torch.cuda.Stream | None = None) -> torch.Tensor:
    """The 4-bit form of a weight matrix w (N x K, fp32, fp16 or bf16) that
    gemv_w4 reads: W (N x K/2 uint8), scales (N x K/group, fp16 or bf16) and,
    if given, zeros (N x K/group uint8; without them the zero point is 8).
    Returns W."""
    device = _matrix(w, "w")
    code = _type(w, "w")
    _matrix(scales, "scales")
    N, K = w.shape
    if scales.dtype != torch.float16 and scales.dtype != torch.bfloat16:
        raise ValueError(f"scales must be fp16 or bf16, not {scales.dtype}")
    groups = scales.shape[1]
    group = K // groups if groups else 32
    if groups * group != K or group not in GROUPS:
        raise ValueError(f"K = {K} and {groups} scales a row: the group must be 32, 64 or 128")
    ld = _rows(w, "w", w.dtype, (N, K), device)
    ldw = _rows(W, "W", torch.uint8, (N, K // 2), device)
    lds = _rows(scales, "scales", scales.dtype, (N, groups), device)
    ldz, pz = 0, None
    if zeros is not None:
        ldz, pz = _rows(zeros, "zeros", torch.uint8, (N, groups), device), zeros.data_ptr()
    _call("quantize_w4", device, stream, N, K, w.data_ptr(), ld, code, group, W.data_ptr(), ldw,
          scales.data_ptr(), lds, _TYPES[scales.dtype], pz, ldz)
    return W
