"""include/linear.h without a GPU: the symbols are there, the host-side argument
checks answer before any CUDA call, and the 64-bit forms the GPU tests use are
themselves right.  No test here launches a kernel."""
import ctypes
import os
import re
import subprocess

import numpy as np
import pytest
import torch

import linear_reference as R
from stage_software_pipelining_gb300 import build as gemm_build
from stage_software_pipelining_gb300 import gemm as G
from stage_software_pipelining_gb300 import linear as L
from stage_software_pipelining_gb300 import quant as Q

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = 0x7F0000000000      # never dereferenced: every call below is refused first
BIG = 2 ** 31
ARG, ALIGN, UNSUPPORTED, OK = G.GEMM_ERR_ARG, G.GEMM_ERR_ALIGN, G.GEMM_ERR_UNSUPPORTED, G.GEMM_OK


@pytest.fixture(scope="module")
def lib():
    gemm_build.build()
    return L.load_library()


def test_header_declares_the_binding_exports(lib):
    text = open(os.path.join(ROOT, "include", "linear.h"), encoding="utf-8").read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    names = re.findall(r"^\s*int\s+(\w+)\s*\(", text, flags=re.M)
    assert sorted(names) == sorted(L.EXPORTS)
    for n in names:
        assert hasattr(lib, n)


def test_header_compiles_as_c(tmp_path):
    src = tmp_path / "t.c"
    src.write_text('#include "linear.h"\nint main(void) { return LINEAR_ACT_NONE; }\n')
    subprocess.run(["gcc", "-std=c11", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"), "-c", str(src),
                    "-o", str(tmp_path / "t.o")], check=True, capture_output=True)


def test_activation_numbers_are_the_headers():
    text = open(os.path.join(ROOT, "include", "linear.h"), encoding="utf-8").read()
    for name, number in L.ACTIVATIONS.items():
        assert re.search(rf"LINEAR_ACT_{name.upper()} = {number}\b", text)


def fwd(lib, M=8, N=16, K=32, x=P, ldx=32, W=P, ldw=32, b=None, r=None, ldr=16, act=0, pre=None, ldp=16, y=P, ldy=16,
        dt=Q.QUANT_BF16, f="linear"):
    return getattr(lib, f)(M, N, K, x, ldx, W, ldw, b, r, ldr, act, pre, ldp, y, ldy, dt, None)


@pytest.mark.parametrize("f", ["linear", "linear_checked"])
def test_linear_arguments(lib, f):
    def call(**k):
        return fwd(lib, f=f, **k)
    for bad in (dict(M=-1), dict(N=-1), dict(K=-1), dict(dt=3), dict(dt=-1), dict(act=5), dict(act=-1), dict(x=None),
                dict(W=None), dict(y=None), dict(ldx=31), dict(ldw=16), dict(ldy=15), dict(r=P, ldr=8),
                dict(pre=P, ldp=8)):
        assert call(**bad) == ARG, bad
    for bad in (dict(dt=Q.QUANT_F32), dict(M=BIG), dict(N=BIG, ldy=BIG), dict(K=BIG, ldx=BIG, ldw=BIG)):
        assert call(**bad) == UNSUPPORTED, bad
    for bad in (dict(x=P + 8), dict(W=P + 2), dict(y=P + 4), dict(r=P + 8), dict(pre=P + 2), dict(b=P + 1),
                dict(ldx=36), dict(ldw=33), dict(ldy=20), dict(r=P, ldr=20), dict(pre=P, ldp=17)):
        assert call(**bad) == ALIGN, bad
    if f == "linear":
        assert call(M=0) == call(N=0, y=None) == OK


def grad(lib, M=8, N=16, dy=P, lddy=16, pre=P, ldp=16, act=2, dz=P, lddz=16, db=P, c=None, dt=Q.QUANT_F16):
    return lib.act_grad(M, N, dy, lddy, pre, ldp, act, dz, lddz, db, c, dt, None)


def test_act_grad_arguments(lib):
    for bad in (dict(M=-1), dict(N=-1), dict(dt=3), dict(act=5), dict(act=-1), dict(dy=None), dict(pre=None),
                dict(dz=None, db=None), dict(lddy=15), dict(ldp=15), dict(lddz=15)):
        assert grad(lib, **bad) == ARG, bad
    assert grad(lib, dt=Q.QUANT_F32) == grad(lib, M=BIG) == grad(lib, N=BIG, lddy=BIG, ldp=BIG, lddz=BIG) == UNSUPPORTED
    for bad in (dict(dy=P + 1), dict(pre=P + 1), dict(dz=P + 1), dict(db=P + 2), dict(c=P + 2)):
        assert grad(lib, **bad) == ALIGN, bad
    assert grad(lib, N=0) == grad(lib, M=0, db=None) == OK


def dx(lib, M=8, N=16, K=32, dz=P, lddz=16, W=P, ldw=32, r=None, ldr=32, act=0, pre=None, ldp=32, out=P, ldo=32,
       dt=Q.QUANT_BF16, f="linear_dx"):
    return getattr(lib, f)(M, N, K, dz, lddz, W, ldw, r, ldr, act, pre, ldp, out, ldo, dt, None)


@pytest.mark.parametrize("f", ["linear_dx", "linear_dx_checked"])
def test_linear_dx_arguments(lib, f):
    for bad in (dict(M=-1), dict(N=-1), dict(K=-1), dict(dt=9), dict(act=7), dict(dz=None), dict(W=None), dict(out=None),
                dict(lddz=15), dict(ldw=31), dict(ldo=31), dict(r=P, ldr=31), dict(act=2), dict(pre=P),
                dict(act=2, pre=P, ldp=31)):
        assert dx(lib, f=f, **bad) == ARG, bad
    for bad in (dict(dt=Q.QUANT_F32), dict(M=BIG), dict(N=BIG, lddz=BIG), dict(K=BIG, ldw=BIG, ldo=BIG)):
        assert dx(lib, f=f, **bad) == UNSUPPORTED, bad
    for bad in (dict(dz=P + 2), dict(W=P + 8), dict(out=P + 2), dict(lddz=20), dict(ldw=36), dict(ldo=36),
                dict(r=P + 2), dict(act=4, pre=P + 2)):
        assert dx(lib, f=f, **bad) == ALIGN, bad
    if f == "linear_dx":
        assert dx(lib, M=0) == dx(lib, K=0, out=None) == OK


def dw(lib, M=8, N=16, K=32, dz=P, lddz=16, x=P, ldx=32, c=None, ldc=32, out=P, ldo=32, dt=Q.QUANT_BF16,
       to=Q.QUANT_F32, f="linear_dw"):
    return getattr(lib, f)(M, N, K, dz, lddz, x, ldx, c, ldc, out, ldo, dt, to, None)


@pytest.mark.parametrize("f", ["linear_dw", "linear_dw_checked"])
def test_linear_dw_arguments(lib, f):
    for bad in (dict(M=-1), dict(N=-1), dict(K=-1), dict(dt=9), dict(to=-1), dict(dz=None), dict(x=None),
                dict(out=None), dict(lddz=15), dict(ldx=31), dict(ldo=31), dict(c=P, ldc=31)):
        assert dw(lib, f=f, **bad) == ARG, bad
    for bad in (dict(dt=Q.QUANT_F32), dict(to=Q.QUANT_F16), dict(M=BIG), dict(N=BIG, lddz=BIG),
                dict(K=BIG, ldx=BIG, ldo=BIG)):
        assert dw(lib, f=f, **bad) == UNSUPPORTED, bad
    for bad in (dict(dz=P + 2), dict(x=P + 8), dict(out=P + 4), dict(lddz=20), dict(ldx=36), dict(ldo=33),
                dict(c=P + 4), dict(ldo=36, to=Q.QUANT_BF16)):
        assert dw(lib, f=f, **bad) == ALIGN, bad
    if f == "linear_dw":
        assert dw(lib, N=0) == dw(lib, K=0, out=None) == OK


def ortho(lib, B=2, rows=16, cols=32, g=P, ldg=32, sg=512, dt=Q.QUANT_F32, o=P, ldo=32, so=512, to=Q.QUANT_BF16,
          steps=5, coef=True, eps=1e-7, ws=P, n=1 << 30, f="orthogonalize"):
    c = (ctypes.c_float * 3)(1, 2, 3) if coef else None
    return getattr(lib, f)(B, rows, cols, g, ldg, sg, dt, o, ldo, so, to, steps, c, eps, 1.0, ws, n, None)


@pytest.mark.parametrize("f", ["orthogonalize", "orthogonalize_checked"])
def test_orthogonalize_arguments(lib, f):
    for bad in (dict(B=-1), dict(rows=-1), dict(cols=-1), dict(dt=3), dict(to=-1), dict(steps=-1), dict(steps=101),
                dict(coef=False), dict(eps=-1.0), dict(eps=float("nan")), dict(g=None), dict(o=None), dict(ws=None),
                dict(ldg=31), dict(ldo=24), dict(sg=500), dict(so=508)):
        assert ortho(lib, f=f, **bad) == ARG, bad
    for bad in (dict(to=Q.QUANT_F32), dict(rows=32769, sg=1 << 40, so=1 << 40),
                dict(cols=32769, ldg=40000, ldo=40000, sg=1 << 40, so=1 << 40), dict(B=65536)):
        assert ortho(lib, f=f, **bad) == UNSUPPORTED, bad
    for bad in (dict(g=P + 4), dict(o=P + 2), dict(ws=P + 16), dict(ldg=33, sg=1024), dict(ldo=36, so=1024),
                dict(sg=514), dict(so=516)):
        assert ortho(lib, f=f, **bad) == ALIGN, bad
    assert ortho(lib, f=f, n=100) == G.GEMM_ERR_SCRATCH
    if f == "orthogonalize":
        assert ortho(lib, B=0) == ortho(lib, rows=0) == ortho(lib, cols=0, g=None) == OK


def test_orthogonalize_workspace(lib):
    n = ctypes.c_size_t(7)
    assert lib.orthogonalize_workspace(1, 4, 4, None) == lib.orthogonalize_workspace(-1, 4, 4, ctypes.byref(n)) == ARG
    assert lib.orthogonalize_workspace(1, 4, 32769, ctypes.byref(n)) == UNSUPPORTED
    assert lib.orthogonalize_workspace(0, 4, 4, ctypes.byref(n)) == OK and n.value == 0
    for B, r, c in ((1, 1, 1), (3, 100, 999), (2, 999, 100), (1, 4096, 8192)):
        g = torch.empty(B, r, c, device="meta")
        small = min(r, c)
        # two X and two squares in 16 bits, rows padded by 63 elements at most, the norm's
        # parts, and each on a boundary of 256
        least = B * (4 * r * c + 4 * small * small)
        assert least <= L.orthogonalize_workspace(g) <= B * (4 * r * (c + 63) + 4 * small * (small + 63) + 8196) + 2048
        assert L.orthogonalize_workspace(g[0]) <= L.orthogonalize_workspace(g)
    with pytest.raises(ValueError):
        L.orthogonalize_workspace(torch.empty(4))


def test_plan_arguments(lib):
    assert lib.linear_plan(3, 1, 1, 1, Q.QUANT_F16, P) == lib.linear_plan(0, 0, 1, 1, Q.QUANT_F16, P) == ARG
    assert lib.linear_plan(0, 1, 1, 1, 5, P) == lib.linear_plan(0, 1, 1, 1, Q.QUANT_F16, None) == ARG
    assert lib.linear_plan(1, 1, 1, 1, Q.QUANT_F32, P) == lib.linear_plan(0, BIG, 1, 1, Q.QUANT_F16, P) == UNSUPPORTED
    with pytest.raises(G.GemmError):
        L.linear_plan("dy", 1, 1, 1)


def test_python_refusals():
    t = torch.zeros(4, 8)
    for call in (lambda: L.linear(t, t, t), lambda: L.linear(t, t, t, act="tanh"), lambda: L.linear(t, t, t, act=None),
                 lambda: L.act_grad(t, t), lambda: L.linear_dx(t, t, t), lambda: L.linear_dw(t, t, t),
                 lambda: L.orthogonalize(t, t, t), lambda: L.orthogonalize(t, t, t, coefficients=(1, 2)),
                 lambda: L.linear("x", t, t)):
        with pytest.raises(ValueError):
            call()


# ---------------------------------------------------------------- the 64-bit forms
@pytest.mark.parametrize("name", list(L.ACTIVATIONS))
def test_derivatives_are_differences(name):
    z = np.linspace(-9, 9, 1001) + 1e-3      # not at relu's corner
    h = 1e-5
    diff = (R.act(z + h, name) - R.act(z - h, name)) / (2 * h)
    assert np.abs(diff - R.derivative(z, name)).max() < 1e-8


@pytest.mark.parametrize("name", list(L.ACTIVATIONS))
def test_activations_are_torchs(name):
    z = torch.linspace(-12, 12, 501, dtype=torch.float64)
    t = {"none": lambda v: v, "relu": torch.relu, "gelu": torch.nn.functional.gelu,
         "gelu_tanh": lambda v: torch.nn.functional.gelu(v, approximate="tanh"),
         "silu": torch.nn.functional.silu}[name](z)
    assert np.abs(R.act(z.numpy(), name) - t.numpy()).max() < 1e-14
    ends = R.act(np.array([-np.inf, np.inf, np.nan]), name)
    assert (ends[0] == 0 or name == "none") and ends[1] == np.inf and np.isnan(ends[2])
    if name not in ("none", "relu"):
        d = R.derivative(np.array([-np.inf, np.inf, np.nan]), name)
        assert abs(d[0]) < R.LEAST and d[1] == 1 and np.isnan(d[2])      # 200 exp(-200) for silu


def test_steps_act_on_singular_values():
    g = np.random.default_rng(0).standard_normal((12, 30))
    abc = (3.4445, -4.7750, 2.0315)
    for m in (g, g.T):
        _, x = R.orthogonalized(m, 5, abc, 0.0, 1.0)
        p = np.linalg.svd(m, compute_uv=False) / np.linalg.norm(m)
        for _ in range(5):
            p = abc[0] * p + abc[1] * p ** 3 + abc[2] * p ** 5
        assert np.allclose(np.sort(np.linalg.svd(x, compute_uv=False)), np.sort(p), atol=1e-12)


def test_ortho_bound_holds_for_rounded_steps():
    """The bound against the same steps with fp16 roundings put in, in 64 bits."""
    def h(v, s):
        return (v * s).astype(np.float16).astype(np.float64) / s
    abc = (3.4445, -4.7750, 2.0315)
    for shape in ((24, 100), (60, 61)):
        g = np.random.default_rng(1).standard_normal(shape)
        xs, ref = R.orthogonalized(g, 5, abc, 0.0, 1.0)
        n, m = shape
        sa, sx = 2.0 ** int(np.log2(n)), 2.0 ** int(np.log2(np.sqrt(m)))
        x = h(xs[0], 64.0)
        for _ in range(5):
            A = h(x @ x.T, sa)
            B = h(abc[1] * A + abc[2] * A @ A, sa)
            x = h(abc[0] * x + B @ x, sx)
        off = np.linalg.norm(x - ref)
        assert 0 < off <= R.ortho_bound(xs, abc, 2.0 ** -11)
