"""examples/train_mlp.py: the training operators run together as they are used."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def example(gpu):
    spec = importlib.util.spec_from_file_location("train_mlp", os.path.join(ROOT, "examples", "train_mlp.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def net_of(m, layers=2, tokens=96, act="gelu"):
    net = m.Mlp(136, 264, layers, tokens, act=act, seed=3)
    g = torch.Generator(device="cuda").manual_seed(4)
    for p in net.layers:
        for name in ("1", "2"):
            b = torch.randn(p["b" + name].shape, generator=g, device="cuda") * 0.3
            p["b" + name].copy_(b)
            p["c" + name].copy_(b)
    net.layers[0]["h"].copy_(torch.randn(tokens, 136, generator=g, device="cuda"))
    return net, torch.randn(tokens, 136, generator=g, device="cuda").to(BF16)


def stack(params, x, act):
    """The stack in 64 bits, from the 16-bit parameters."""
    f = {"gelu": torch.nn.functional.gelu, "silu": torch.nn.functional.silu, "relu": torch.relu}[act]
    h = x.double()
    for w1, c1, w2, c2 in params:
        h = h + f(h @ w1.t() + c1) @ w2.t() + c2
    return h


@pytest.mark.parametrize("act", ["gelu", "silu", "relu"])
def test_gradients(example, act):
    """Against torch's own differentiation in 64 bits.  Each layer's h, z, a, dz and dh
    is rounded to bf16 (2^-9 on average at most, 2^-8 of an element): ten roundings on
    the way to the first layer's gradients, of independent sign, and the sums over
    elements average them: 10^0.5 2^-8 = 0.0124 in norm, doubled for the residual
    stream's amplification.  relu's derivative jumps where z rounds across 0, for a
    share 2^-8 of the elements at most, which adds 2^-4 in norm."""
    net, target = net_of(example, act=act)
    net.gradients(target)
    params = [[p[k].double().requires_grad_() for k in ("w1", "c1", "w2", "c2")] for p in net.layers]
    x = net.layers[0]["h"].double().requires_grad_()
    loss = ((stack(params, x, act) - target.double()) ** 2).mean()
    loss.backward()
    limit = 0.025 + (2.0 ** -4 if act == "relu" else 0.0)
    loss = loss.detach()
    assert abs(float(net.loss) - float(loss)) < limit * float(loss)
    assert (net.dh.double() - x.grad).norm() < limit * x.grad.norm()
    for p, ref in zip(net.layers, params):
        for k, r in zip(("dW1", "db1", "dW2", "db2"), ref):
            assert (p[k].double() - r.grad).norm() < limit * r.grad.norm(), k


def test_gradients_are_differences(example):
    """A step along the gradient changes the 64-bit loss by what the gradient says: with
    the bound above, and h^2 of the second order for a step that changes it by 1e-4."""
    net, target = net_of(example)
    net.gradients(target)
    params = [[p[k].double() for k in ("w1", "c1", "w2", "c2")] for p in net.layers]
    grads = [[p[k].double() for k in ("dW1", "db1", "dW2", "db2")] for p in net.layers]
    x = net.layers[0]["h"].double()
    square = sum((g * g).sum() for layer in grads for g in layer)
    at = lambda e: ((stack([[v + e * g for v, g in zip(a, b)] for a, b in zip(params, grads)], x, "gelu")  # noqa: E731
                     - target.double()) ** 2).mean()
    e = 1e-4 * float(at(0.0)) / float(square)
    assert abs(float(at(e) - at(-e)) / (2 * e) - float(square)) < 0.03 * float(square)


def test_a_captured_step_is_the_eager_one(example):
    a, target = net_of(example)
    b, _ = net_of(example)
    graph = a.capture_step(target, 0.01)
    for _ in range(2):
        graph.replay()
        b.gradients(target)
        b.update(0.01)
    torch.cuda.synchronize()
    for p, r in zip(a.layers, b.layers):
        for k in ("W1", "W2", "b1", "b2", "dW1", "db2", "update1"):
            assert torch.equal(p[k], r[k]), k
    assert torch.equal(a.loss, b.loss)


def test_runs_as_a_program(example, capsys):
    r = example.main(["--dim", "128", "--hidden", "256", "--layers", "2", "--tokens", "200", "--steps", "2"])
    assert r["first"] > 0 and r["last"] > 0 and "2 layers of 128" in capsys.readouterr().out
