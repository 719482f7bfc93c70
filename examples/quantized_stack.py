"""A stack of pre-norm residual linear layers with quantised weights:

    h <- h + W_l norm_l(h),   l = 0 .. L-1,   then a last norm.

A prompt runs through 8-bit products (add_rmsnorm hands gemm_fp8 its e4m3 rows
and their scales, and adds the previous layer's output to the residual stream
on the way), a single token through 4-bit ones (add_rmsnorm's 16-bit row to
gemv_w4) inside one CUDA graph.  Both keep every buffer they need and allocate
nothing once built.

    python examples/quantized_stack.py [--dim 4096] [--layers 8] [--prompt 2048] [--steps 64]

prints the time of a prompt and of a decoding step, and how far both are from
the same stack in fp32 with the unquantised weights.
"""
from __future__ import annotations

import argparse
import os
import sys
import time

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

from stage_software_pipelining_gb300 import quant as Q  # noqa: E402

DTYPE = torch.bfloat16
EPS = 1e-6


class QuantizedStack:
    """weights: L matrices D x D (fp32, on the GPU); norms: L + 1 vectors of D."""

    def __init__(self, weights, norms, group: int = 128):
        dim = weights[0].shape[0]
        self.dim = dim
        self.norms = [n.to(DTYPE) for n in norms]
        self.w8, self.w4 = [], []
        for w in weights:
            q, s = Q.empty_rows(dim, dim, torch.float8_e4m3fn), torch.empty(dim, device="cuda")
            Q.quantize_fp8(w, q, s)
            self.w8.append((q.t(), s))
            packed = torch.empty(dim, dim // 2, dtype=torch.uint8, device="cuda")
            scales = torch.empty(dim, dim // group, dtype=DTYPE, device="cuda")
            zeros = torch.empty(dim, dim // group, dtype=torch.uint8, device="cuda")
            Q.quantize_w4(w, packed, scales, zeros)
            self.w4.append((packed, scales, zeros))

    def prompt_buffers(self, tokens: int) -> dict:
        d = self.dim
        return {"h": torch.empty(tokens, d, dtype=DTYPE, device="cuda"),
                "out": Q.empty_rows(tokens, d, DTYPE),
                "q": Q.empty_rows(tokens, d, torch.float8_e4m3fn),
                "scale": torch.empty(tokens, device="cuda"),
                "last": torch.empty(tokens, d, dtype=DTYPE, device="cuda")}

    def prompt(self, x: torch.Tensor, b: dict) -> torch.Tensor:
        """The normalised stack output of x (tokens x D bf16), in b["last"]."""
        y, residual = x, None
        for norm, (w, s) in zip(self.norms, self.w8):
            Q.add_rmsnorm(y, norm, residual, eps=EPS, residual_out=b["h"], q=b["q"], scale=b["scale"])
            Q.gemm_fp8(b["q"], w, b["out"], b["scale"], s)
            y, residual = b["out"], b["h"]
        Q.add_rmsnorm(y, self.norms[-1], residual, eps=EPS, y=b["last"])
        return b["last"]

    def step_buffers(self) -> dict:
        row = lambda: torch.empty(1, self.dim, dtype=DTYPE, device="cuda")  # noqa: E731
        return {"x": row(), "h": row(), "out": row(), "normed": row(), "last": row()}

    def step(self, b: dict) -> torch.Tensor:
        """The same for one token, from b["x"] into b["last"]."""
        y, residual = b["x"], None
        for norm, (w, s, z) in zip(self.norms, self.w4):
            Q.add_rmsnorm(y, norm, residual, eps=EPS, residual_out=b["h"], y=b["normed"])
            Q.gemv_w4(b["normed"], w, s, b["out"], zeros=z)
            y, residual = b["out"], b["h"]
        Q.add_rmsnorm(y, self.norms[-1], residual, eps=EPS, y=b["last"])
        return b["last"]

    def capture_step(self, b: dict) -> torch.cuda.CUDAGraph:
        """step() as a CUDA graph over b's buffers."""
        stream = torch.cuda.Stream()
        stream.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.stream(stream):
            self.step(b)                      # the kernels' one-time settings, outside the capture
            with torch.cuda.graph(graph, stream=stream):
                self.step(b)
        torch.cuda.current_stream().wait_stream(stream)
        return graph


def reference(x: torch.Tensor, weights, norms) -> torch.Tensor:
    """The stack in fp32 with the weights as they were before quantisation."""
    h = x.float()
    norm = lambda v, w: v * torch.rsqrt((v * v).mean(-1, keepdim=True) + EPS) * w  # noqa: E731
    for w, n in zip(weights, norms):
        h = h + norm(h, n) @ w.t()
    return norm(h, norms[-1])


def make(dim: int, layers: int, seed: int = 0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    weights = [torch.randn(dim, dim, generator=g, device="cuda") * dim ** -0.5 for _ in range(layers)]
    norms = [1.0 + 0.1 * torch.randn(dim, generator=g, device="cuda") for _ in range(layers + 1)]
    return weights, norms


def timed(fn, n: int) -> float:
    for _ in range(3):
        fn()
    torch.cuda.synchronize()
    t = time.perf_counter()
    for _ in range(n):
        fn()
    torch.cuda.synchronize()
    return (time.perf_counter() - t) / n


def main(argv=None) -> dict:
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--dim", type=int, default=4096)
    ap.add_argument("--layers", type=int, default=8)
    ap.add_argument("--prompt", type=int, default=2048)
    ap.add_argument("--steps", type=int, default=64)
    a = ap.parse_args(argv)
    weights, norms = make(a.dim, a.layers)
    stack = QuantizedStack(weights, norms)
    x = torch.randn(a.prompt, a.dim, device="cuda").to(DTYPE)
    pb, sb = stack.prompt_buffers(a.prompt), stack.step_buffers()
    ref = reference(x, weights, norms)
    sb["x"].copy_(x[-1:])
    graph = stack.capture_step(sb)
    graph.replay()
    off = lambda out, r: float((out.float() - r).norm() / r.norm())  # noqa: E731
    result = {"prompt_error": off(stack.prompt(x, pb), ref), "step_error": off(sb["last"], ref[-1:]),
              "prompt_ms": timed(lambda: stack.prompt(x, pb), 10) * 1e3,
              "step_us": timed(graph.replay, a.steps) * 1e6}
    print(f"{a.layers} layers of {a.dim}: prompt of {a.prompt} tokens {result['prompt_ms']:.3f} ms "
          f"(8-bit, {result['prompt_error']:.3f} from fp32), step {result['step_us']:.1f} us "
          f"(4-bit, {result['step_error']:.3f} from fp32)")
    return result


if __name__ == "__main__":
    main()
