"""Binding over libgemm.so's training operators (include/linear.h).

A 16-bit linear layer (``linear``: product, bias, activation and residual in one
kernel), its gradients (``act_grad``, ``linear_dx``, ``linear_dw``) and the update
of its weights with all singular values brought near one (``orthogonalize``).

    linear(x, W, y, bias=b, act="gelu", pre=z)      # y = gelu(x W^T + b), z kept
    act_grad(dy, dz, pre=z, act="gelu", dbias=db)   # dz = dy gelu'(z), db = sum of its rows
    linear_dx(dz, W, dx)                            # dx = dz W
    linear_dw(dz, x, dW)                            # dW = dz^T x
    orthogonalize(dW, update, workspace)

Buffers, streams and errors are as in quant.py: the caller owns every buffer, a
tensor that an operator cannot take raises ValueError, a status other than GEMM_OK
raises GemmError, and a call runs on the current stream of its tensors' device,
or on ``stream``.  Matrices start on 16-byte boundaries and so do their rows
(``quant.empty_rows`` makes such); ``act_grad`` takes any.  There is no CPU
fallback.  ``checked`` waits for the stream and reports a pipeline wait that ran
out.
"""
from __future__ import annotations

import ctypes
import threading

import torch

from . import gemm as G
from . import quant as Q
from .gemm import GemmError

# linear_act_t
ACTIVATIONS = {"none": 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4}

# Every extern "C" symbol include/linear.h declares.
EXPORTS = ("linear", "linear_checked", "act_grad", "linear_dx", "linear_dx_checked", "linear_dw",
           "linear_dw_checked", "linear_plan", "orthogonalize", "orthogonalize_checked",
           "orthogonalize_workspace")

# The products' kernels, in linear_kernel_t's order, and linear_op_t.
KERNELS = ("few", "pair")
OPS = {"linear": 0, "dx": 1, "dw": 2}

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
            i64, p, i32, f32, size = (ctypes.c_int64, ctypes.c_void_p, ctypes.c_int, ctypes.c_float,
                                      ctypes.c_size_t)
            lib.linear.argtypes = [i64, i64, i64, p, i64, p, i64, p, p, i64, i32, p, i64, p, i64, i32, p]
            lib.act_grad.argtypes = [i64, i64, p, i64, p, i64, i32, p, i64, p, p, i32, p]
            lib.linear_dx.argtypes = [i64, i64, i64, p, i64, p, i64, p, i64, i32, p, i64, p, i64, i32, p]
            lib.linear_dw.argtypes = [i64, i64, i64, p, i64, p, i64, p, i64, p, i64, i32, i32, p]
            lib.orthogonalize.argtypes = [i64, i64, i64, p, i64, i64, i32, p, i64, i64, i32, i32, p, f32,
                                          f32, p, size, p]
            for name in ("linear", "linear_dx", "linear_dw", "orthogonalize"):
                getattr(lib, name + "_checked").argtypes = getattr(lib, name).argtypes
            lib.linear_plan.argtypes = [i32, i64, i64, i64, i32, p]
            lib.orthogonalize_workspace.argtypes = [i64, i64, i64, p]
            for name in EXPORTS:
                getattr(lib, name).restype = i32
            _lib = lib
        return _lib


def _binding():
    """The extension that marshals tensors into libgemm.so.  Raises if it is missing."""
    global _ext
    _ext = Q.load_binding()
    return _ext


def _act(name: str) -> int:
    try:
        return ACTIVATIONS[name]
    except (KeyError, TypeError):
        raise ValueError(f"act must be one of {', '.join(ACTIVATIONS)}, not {name!r}") from None


def linear(x: torch.Tensor, W: torch.Tensor, y: torch.Tensor, *, bias: torch.Tensor | None = None,
           residual: torch.Tensor | None = None, act: str = "none", pre: torch.Tensor | None = None,
           stream: torch.cuda.Stream | None = None, checked: bool = False) -> torch.Tensor:
    """y = act(z) + residual with z = x W^T + bias, kept in pre if given.

    x: M x K; W: N x K; y, residual, pre: M x N; bias: N; all fp16 or all
    bf16.  act: one of ACTIVATIONS.  residual may be y itself.  Returns y."""
    st = (_ext or _binding()).linear(x, W, y, bias, residual, _act(act), pre, stream, checked)
    if st:
        raise GemmError(st, "linear")
    return y


def act_grad(dy: torch.Tensor, dz: torch.Tensor | None = None, *, pre: torch.Tensor | None = None,
             act: str = "none", dbias: torch.Tensor | None = None,
             addend: torch.Tensor | None = None, stream: torch.cuda.Stream | None = None) -> None:
    """dz = dy act'(pre) and dbias = addend + the sum of dz's (unrounded) rows.

    dy, pre, dz: M x N of one 16-bit type; dbias, addend: N fp32.  dz or dbias may
    be None (not computed); dz may be dy or pre itself, addend dbias itself."""
    st = (_ext or _binding()).act_grad(dy, dz, pre, _act(act), dbias, addend, stream)
    if st:
        raise GemmError(st, "act_grad")


def linear_dx(dz: torch.Tensor, W: torch.Tensor, dx: torch.Tensor, *,
              residual: torch.Tensor | None = None, act: str = "none",
              pre: torch.Tensor | None = None, stream: torch.cuda.Stream | None = None,
              checked: bool = False) -> torch.Tensor:
    """dx = (dz W + residual) act'(pre): the gradient of linear's x, joined with
    one that arrives by another way, and taken through the activation that made x.

    dz: M x N; W: N x K; dx, residual, pre: M x K; all fp16 or all bf16.  pre
    and an act other than "none" go together.  dx may be residual or pre itself.
    Returns dx."""
    st = (_ext or _binding()).linear_dx(dz, W, dx, residual, _act(act), pre, stream, checked)
    if st:
        raise GemmError(st, "linear_dx")
    return dx


def linear_dw(dz: torch.Tensor, x: torch.Tensor, dw: torch.Tensor, *,
              addend: torch.Tensor | None = None, stream: torch.cuda.Stream | None = None,
              checked: bool = False) -> torch.Tensor:
    """dw = dz^T x + addend: the gradient of linear's W.

    dz: M x N; x: M x K; both fp16 or both bf16; dw, addend: N x K, fp32 or dz's
    type.  addend may be dw itself (micro-batches).  Returns dw."""
    st = (_ext or _binding()).linear_dw(dz, x, dw, addend, stream, checked)
    if st:
        raise GemmError(st, "linear_dw")
    return dw


def orthogonalize_workspace(g: torch.Tensor) -> int:
    """Bytes of workspace that orthogonalize needs for g."""
    if g.dim() not in (2, 3):
        raise ValueError("g must be 2-D or 3-D")
    n = ctypes.c_size_t()
    st = load_library().orthogonalize_workspace(g.shape[0] if g.dim() == 3 else 1, g.shape[-2], g.shape[-1],
                                                ctypes.byref(n))
    if st:
        raise GemmError(st, "orthogonalize_workspace")
    return n.value


def orthogonalize(g: torch.Tensor, out: torch.Tensor, workspace: torch.Tensor, *, steps: int = 5,
                  coefficients: tuple = (3.4445, -4.7750, 2.0315), eps: float = 1e-7,
                  scale: float = 1.0, stream: torch.cuda.Stream | None = None,
                  checked: bool = False) -> torch.Tensor:
    """out = scale X, where X = g / (|g| + eps) and then, `steps` times,
    X <- a X + (b A + c A^2) X with A = X X^T and a, b, c = coefficients.

    g: rows x cols, or a batch of such, fp32, fp16 or bf16; out: the same shape,
    fp16 or bf16; workspace: a contiguous tensor of orthogonalize_workspace(g) bytes,
    which calls that may run at the same time do not share.  Returns out."""
    try:
        a, b, c = coefficients
    except (TypeError, ValueError):
        raise ValueError("coefficients must be three numbers") from None
    st = (_ext or _binding()).orthogonalize(g, out, workspace, steps, a, b, c, eps, scale, stream, checked)
    if st:
        raise GemmError(st, "orthogonalize")
    return out


_TYPES = {torch.float32: Q.QUANT_F32, torch.float16: Q.QUANT_F16, torch.bfloat16: Q.QUANT_BF16}


def linear_plan(op: str, M: int, N: int, K: int, out_dtype: torch.dtype = torch.bfloat16) -> dict:
    """The launch that linear (op "linear"), linear_dx ("dx") or linear_dw ("dw")
    would make on the current device for these sizes and this type of output: its
    kernel (one of KERNELS), the rows of the result a tile, the CTAs that share a
    tile's sum, the ring's stages, the CTAs and their dynamic shared memory."""
    plan = Q._Plan()
    st = load_library().linear_plan(OPS.get(op, -1), int(M), int(N), int(K), _TYPES.get(out_dtype, -1),
                                    ctypes.byref(plan))
    if st:
        raise GemmError(st, "linear_plan")
    out = {n: getattr(plan, n) for n, _ in Q._Plan._fields_}
    out["kernel"] = KERNELS[plan.kernel]
    return out
