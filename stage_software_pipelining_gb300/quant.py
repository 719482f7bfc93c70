"""Binding over libgemm.so's quantised-linear operators (include/quant.h).

The operators of a linear layer whose weights or activations are held in few
bits: the residual's addition with the RMS norm and 8-bit rows
(``add_rmsnorm``), the 8-bit matrix product (``gemm_fp8``) and the product of a
few rows with 4-bit weights (``gemv_w4``), with the kernels that make such
weights (``quantize_fp8``, ``quantize_w4``).

Signatures and documentation are here; the checks of the arguments and their
marshalling are in the extension ``_quant.so`` (csrc/binding.cpp), and all
arithmetic runs in the CUDA kernels of libgemm.so.  The caller owns every
buffer, outputs included; ``empty_rows`` makes one whose rows start on 16-byte
boundaries.  A tensor that an operator cannot take raises ValueError, a status
other than GEMM_OK raises GemmError.  There is no CPU fallback.

A call runs on the current stream of its tensors' device, or on ``stream``; with
another stream than the one a tensor was made on, the caller orders the two and
keeps the tensor until the call has run (torch's ``wait_stream`` and
``record_stream``).
"""
from __future__ import annotations

import ctypes
import importlib.util
import os
import threading

import torch

from . import gemm as G
from .gemm import GemmError

HERE = os.path.dirname(os.path.abspath(__file__))
BINDING_PATH = os.path.join(HERE, "_quant.so")

QUANT_F32 = 0
QUANT_F16 = 1
QUANT_BF16 = 2

GROUPS = (32, 64, 128)          # K per scale of the 4-bit weights
E4M3_MAX = 448.0                # largest e4m3 value

# Every extern "C" symbol include/quant.h declares.
EXPORTS = ("add_rmsnorm", "quantize_fp8", "gemm_fp8", "gemm_fp8_checked", "gemm_fp8_plan", "gemv_w4",
           "gemv_w4_checked", "gemv_w4_plan", "quantize_w4")

# The products' kernels, in quant_kernel_t's order.
KERNELS = ("fp8_few", "fp8_pair", "w4_warp", "w4_tc")


class _Plan(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in ("kernel", "tile_rows", "split", "stages", "grid", "smem_bytes")]

_lock = threading.Lock()
_lib = None
_ext = None


def load_library():
    """libgemm.so with these operators' signatures, for calls with raw
    arguments.  Raises if it is missing."""
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
            lib.gemv_w4_checked.argtypes = lib.gemv_w4.argtypes
            lib.gemm_fp8_plan.argtypes = [i64, i64, i64, i32, p]
            lib.gemv_w4_plan.argtypes = [i64, i64, i64, i32, i32, i32, p]
            lib.quantize_w4.argtypes = [i64, i64, p, i64, i32, i32, p, i64, p, i64, i32, p, i64, p]
            for name in EXPORTS:
                getattr(lib, name).restype = i32
            _lib = lib
        return _lib


def load_binding():
    """The extension that marshals tensors into libgemm.so.  Raises if it is missing."""
    global _ext
    with _lock:
        if _ext is None:
            if not os.path.exists(BINDING_PATH):
                raise RuntimeError(
                    f"{BINDING_PATH} is missing: build it first (python -c 'import __graft_entry__ "
                    "as g; g.build()'); there is no CPU fallback")
            spec = importlib.util.spec_from_file_location("_quant", BINDING_PATH)
            ext = importlib.util.module_from_spec(spec)
            spec.loader.exec_module(ext)
            _ext = ext
        return _ext


def empty_rows(rows: int, cols: int, dtype: torch.dtype, device="cuda") -> torch.Tensor:
    """An uninitialised rows x cols tensor whose rows start on 16-byte
    boundaries, as gemm_fp8 (and the fast case of the row kernels) wants them."""
    unit = 16 // torch.empty((), dtype=dtype).element_size()
    return torch.empty((rows, (cols + unit - 1) // unit * unit), dtype=dtype,
                       device=device)[:, :cols]


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
    be x or residual itself.
    """
    st = (_ext or load_binding()).add_rmsnorm(x, weight, residual, eps, residual_out, y, q, scale,
                                              stream)
    if st:
        raise GemmError(st, "add_rmsnorm")


def quantize_fp8(x: torch.Tensor, q: torch.Tensor, scale: torch.Tensor, *,
                 stream: torch.cuda.Stream | None = None) -> torch.Tensor:
    """q = e4m3(x / scale) with scale = max(max|x| / 448, 2^-126) a row: rows
    of activations, or a weight matrix stored N x K (a scale an output
    column).  x: fp32, fp16 or bf16; q: float8_e4m3fn; scale: fp32.  Returns q."""
    st = (_ext or load_binding()).quantize_fp8(x, q, scale, stream)
    if st:
        raise GemmError(st, "quantize_fp8")
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
    st = (_ext or load_binding()).gemm_fp8(A, B, C, a_scale, b_scale, stream, checked)
    if st:
        raise GemmError(st, "gemm_fp8")
    return C


def gemv_w4(x: torch.Tensor, W: torch.Tensor, scales: torch.Tensor, C: torch.Tensor,
            zeros: torch.Tensor | None = None, *, stream: torch.cuda.Stream | None = None,
            checked: bool = False) -> torch.Tensor:
    """C = x @ ((w - zeros) * scales)^T with 4-bit weights w (libgemm.so gemv_w4,
    or gemv_w4_checked, which synchronises and reports a wait that ran out).

    x: M x K fp16 or bf16; W: N x K/2 uint8, the even k in the low four bits;
    scales: N x K/group of x's type, group 32, 64 or 128; zeros: N x K/group
    uint8 (None: 8 everywhere); C: M x N of x's type.  x and W start on
    16-byte boundaries and so do their rows.  Returns C.
    """
    st = (_ext or load_binding()).gemv_w4(x, W, scales, C, zeros, stream, checked)
    if st:
        raise GemmError(st, "gemv_w4")
    return C


def quantize_w4(w: torch.Tensor, W: torch.Tensor, scales: torch.Tensor,
                zeros: torch.Tensor | None = None, *,
                stream: torch.cuda.Stream | None = None) -> torch.Tensor:
    """The 4-bit form of a weight matrix w (N x K, fp32, fp16 or bf16) that
    gemv_w4 reads: W (N x K/2 uint8), scales (N x K/group, fp16 or bf16) and,
    if given, zeros (N x K/group uint8; without them the zero point is 8).
    Returns W."""
    st = (_ext or load_binding()).quantize_w4(w, W, scales, zeros, stream)
    if st:
        raise GemmError(st, "quantize_w4")
    return W


def _plan(name: str, *args) -> dict:
    plan = _Plan()
    st = getattr(load_library(), name)(*args, ctypes.byref(plan))
    if st:
        raise GemmError(st, name)
    out = {n: getattr(plan, n) for n, _ in _Plan._fields_}
    out["kernel"] = KERNELS[plan.kernel]
    return out


_TYPES = {torch.float32: QUANT_F32, torch.float16: QUANT_F16, torch.bfloat16: QUANT_BF16}


def gemm_fp8_plan(M: int, N: int, K: int, dtype: torch.dtype = torch.bfloat16) -> dict:
    """The launch gemm_fp8 would make on the current device for an M x N result
    of `dtype`: its kernel (one of KERNELS), the rows of A a tile, the CTAs that
    share a tile's K, the ring's stages, the CTAs and their dynamic shared memory."""
    return _plan("gemm_fp8_plan", int(M), int(N), int(K), _TYPES.get(dtype, -1))


def gemv_w4_plan(M: int, N: int, K: int, group: int, zeros: bool = False,
                 dtype: torch.dtype = torch.bfloat16) -> dict:
    """The same for gemv_w4 with groups of `group`, with or without zero points."""
    return _plan("gemv_w4_plan", int(M), int(N), int(K), int(group), int(bool(zeros)),
                 _TYPES.get(dtype, -1))
