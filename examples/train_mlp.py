"""Training a stack of 16-bit linear layers with the framework's operators:

    h <- h + W2_l act(W1_l h + b1_l) + b2_l,    l = 0 .. L-1,

against a target in mean squares.  Every product, activation, residual and gradient
is one of linear, act_grad, linear_dx and linear_dw; the weights (fp32, with a bf16
copy that the products read) follow their momentum, orthogonalised by orthogonalize,
and the biases plain gradient descent.  A step allocates nothing and runs as one CUDA
graph.

    python examples/train_mlp.py [--dim 1024] [--hidden 4096] [--layers 4] [--tokens 4096] [--steps 20]

prints the loss and the time of a step.
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

from stage_software_pipelining_gb300 import linear as L  # noqa: E402

DTYPE = torch.bfloat16


class Mlp:
    """The stack's parameters, their gradients and every buffer of a step."""

    def __init__(self, dim: int, hidden: int, layers: int, tokens: int, act: str = "gelu", seed: int = 0):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def empty(*shape, dtype=DTYPE):
            return torch.empty(shape, dtype=dtype, device="cuda")

        self.act, self.tokens = act, tokens
        self.layers = []
        for _ in range(layers):
            layer = {}
            for name, (n, k) in (("1", (hidden, dim)), ("2", (dim, hidden))):
                w = torch.randn((n, k), generator=g, device="cuda") * k ** -0.5
                layer["W" + name], layer["w" + name] = w, w.to(DTYPE)      # fp32, and what products read
                layer["b" + name] = torch.zeros(n, device="cuda")
                layer["c" + name] = layer["b" + name].to(DTYPE)
                layer["dW" + name], layer["db" + name] = torch.zeros_like(w), torch.zeros(n, device="cuda")
                layer["momentum" + name] = torch.zeros_like(w)
                layer["update" + name] = empty(n, k)
                layer["room" + name] = torch.empty(L.orthogonalize_workspace(w), dtype=torch.uint8, device="cuda")
            layer["h"] = empty(tokens, dim)           # the layer's input
            layer["z"], layer["a"] = empty(tokens, hidden), empty(tokens, hidden)
            self.layers.append(layer)
        self.out, self.dh = empty(tokens, dim), empty(tokens, dim)
        self.dz = empty(tokens, hidden)
        self.loss = torch.zeros((), device="cuda")

    def forward(self) -> torch.Tensor:
        """The stack's output from the first layer's input h."""
        for i, p in enumerate(self.layers):
            L.linear(p["h"], p["w1"], p["a"], bias=p["c1"], act=self.act, pre=p["z"])
            to = self.layers[i + 1]["h"] if i + 1 < len(self.layers) else self.out
            L.linear(p["a"], p["w2"], to, bias=p["c2"], residual=p["h"])
        return self.out

    def backward(self) -> None:
        """The gradients of every parameter from dh, that of the output; dh becomes the input's."""
        for p in reversed(self.layers):
            L.act_grad(self.dh, dbias=p["db2"])
            L.linear_dw(self.dh, p["a"], p["dW2"])
            # through W2 and, in the same pass, the activation that made a
            L.linear_dx(self.dh, p["w2"], self.dz, act=self.act, pre=p["z"])
            L.act_grad(self.dz, dbias=p["db1"])
            L.linear_dw(self.dz, p["h"], p["dW1"])
            # joined with the residual's gradient, in place
            L.linear_dx(self.dz, p["w1"], self.dh, residual=self.dh)

    def gradients(self, target: torch.Tensor) -> None:
        """Loss and gradients of mean((out - target)^2)."""
        d = self.forward().float() - target.float()
        self.loss.copy_((d * d).mean())
        self.dh.copy_(d * (2.0 / d.numel()))
        self.backward()

    def update(self, rate: float, beta: float = 0.9) -> None:
        for p in self.layers:
            for name in ("1", "2"):
                w, m, u = p["W" + name], p["momentum" + name], p["update" + name]
                m.mul_(beta).add_(p["dW" + name])
                L.orthogonalize(m, u, p["room" + name], scale=max(1.0, w.shape[0] / w.shape[1]) ** 0.5)
                w.sub_(u, alpha=rate)
                p["w" + name].copy_(w)
                p["b" + name].sub_(p["db" + name], alpha=rate)
                p["c" + name].copy_(p["b" + name])

    def capture_step(self, target: torch.Tensor, rate: float) -> torch.cuda.CUDAGraph:
        """A whole step as a CUDA graph over this object's buffers."""
        stream = torch.cuda.Stream()
        stream.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.stream(stream):
            self.gradients(target)            # the kernels' one-time settings, outside the capture
            with torch.cuda.graph(graph, stream=stream):
                self.gradients(target)
                self.update(rate)
        torch.cuda.current_stream().wait_stream(stream)
        return graph


def main(argv=None) -> dict:
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--dim", type=int, default=1024)
    ap.add_argument("--hidden", type=int, default=4096)
    ap.add_argument("--layers", type=int, default=4)
    ap.add_argument("--tokens", type=int, default=4096)
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--rate", type=float, default=0.01)
    a = ap.parse_args(argv)
    for name in ("dim", "hidden", "layers", "tokens", "steps"):
        if getattr(a, name) < 1:
            ap.error(f"--{name} must be at least 1")
    net = Mlp(a.dim, a.hidden, a.layers, a.tokens)
    x = torch.randn(a.tokens, a.dim, device="cuda").to(DTYPE)
    target = torch.roll(x, 1, dims=1)
    net.layers[0]["h"].copy_(x)
    graph = net.capture_step(target, a.rate)
    losses = []
    torch.cuda.synchronize()
    began = time.perf_counter()
    for _ in range(a.steps):
        graph.replay()
        losses.append(net.loss.clone())
    torch.cuda.synchronize()
    ms = (time.perf_counter() - began) / a.steps * 1e3
    result = {"first": float(losses[0]), "last": float(losses[-1]), "ms": ms}
    print(f"{a.layers} layers of {a.dim} x {a.hidden}, {a.tokens} tokens: loss {result['first']:.4f} -> "
          f"{result['last']:.4f} in {a.steps} steps of {ms:.3f} ms")
    return result


if __name__ == "__main__":
    main()
