"""examples/quantized_stack.py: the operators run together as they are used."""
import importlib.util
import os

import pytest
import torch

import quant_reference as R

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def stack_module(gpu):
    spec = importlib.util.spec_from_file_location(
        "quantized_stack", os.path.join(ROOT, "examples", "quantized_stack.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_stack_matches_its_quantised_weights(stack_module):
    """One layer against 64 bits with the quantised weights themselves: what is
    left is the roundings of the 16-bit tensors (2^-8 of a value each: the
    residual's, the product's, the last norm's, and for the 8-bit path the e4m3
    row's 2^-4 an element, 0.03 in the norm of a product of hundreds)."""
    m = stack_module
    weights, norms = m.make(512, 1, seed=3)
    s = m.QuantizedStack(weights, norms)
    x = torch.randn(33, 512, device="cuda").to(m.DTYPE)
    n0, n1 = (R.f64(n) for n in s.norms)

    def run(w):
        h = R.f64(x)
        y = h / (((h * h).mean(1, keepdims=True) + m.EPS) ** 0.5) * n0
        h = h + y @ w.T
        return h / (((h * h).mean(1, keepdims=True) + m.EPS) ** 0.5) * n1

    def off(a, b):
        return float(((a - b) ** 2).sum() ** 0.5 / (b ** 2).sum() ** 0.5)

    w8, s8 = s.w8[0]
    out = R.f64(s.prompt(x, s.prompt_buffers(33)))
    assert off(out, run(R.f64(w8).T * R.f64(s8)[:, None])) < 0.05
    b = s.step_buffers()
    b["x"].copy_(x[5:6])
    graph = s.capture_step(b)
    b["last"].zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert off(R.f64(b["last"]), run(R.w4_weights(*s.w4[0], 128))[5:6]) < 4 * 2.0 ** -8


def test_stack_runs_as_a_program(stack_module, capsys):
    r = stack_module.main(["--dim", "512", "--layers", "3", "--prompt", "70", "--steps", "3"])
    # 4-bit weights are off by a step's twelfth root, a fifteenth of a group's
    # range of 5.5 standard deviations: 0.11 of a weight; 8-bit ones by 0.03.
    assert r["prompt_error"] < 0.08 and r["step_error"] < 0.3
    assert "3 layers of 512" in capsys.readouterr().out
