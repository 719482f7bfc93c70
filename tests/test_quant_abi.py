"""include/quant.h without a GPU: the symbols are there, the host-side argument
checks answer before any CUDA call, and the 64-bit forms the GPU tests use are
themselves right.  No test here launches a kernel."""
import os
import re
import subprocess

import numpy as np
import pytest
import torch

import quant_reference as R
from stage_software_pipelining_gb300 import build as gemm_build
from stage_software_pipelining_gb300 import gemm as G
from stage_software_pipelining_gb300 import quant as Q

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = 0x7F0000000000      # never dereferenced: every call below is refused first


@pytest.fixture(scope="module")
def lib():
    gemm_build.build()
    return Q.load_library()


def test_header_declares_the_binding_exports(lib):
    text = open(os.path.join(ROOT, "include", "quant.h"), encoding="utf-8").read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    names = re.findall(r"^\s*int\s+(\w+)\s*\(", text, flags=re.M)
    assert sorted(names) == sorted(Q.EXPORTS)
    for n in names:
        assert hasattr(lib, n)


def test_header_compiles_as_c(tmp_path):
    src = tmp_path / "t.c"
    src.write_text('#include "quant.h"\nint main(void) { return QUANT_F32; }\n')
    subprocess.run(["gcc", "-std=c11", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"), "-c", str(src),
                    "-o", str(tmp_path / "t.o")], check=True, capture_output=True)


def norm(lib, rows=4, cols=64, x=P, ldx=64, r=None, ldr=0, w=P, eps=1e-6, dt=Q.QUANT_BF16, ro=None, ldro=0, y=P,
         ldy=64, q=None, ldq=0, s=None):
    return lib.add_rmsnorm(rows, cols, x, ldx, r, ldr, w, eps, dt, ro, ldro, y, ldy, q, ldq, s, None)


def test_norm_arguments(lib):
    assert norm(lib, rows=-1) == norm(lib, cols=-1) == norm(lib, dt=3) == norm(lib, dt=-1) == G.GEMM_ERR_ARG
    assert norm(lib, x=None) == norm(lib, w=None) == norm(lib, y=None) == G.GEMM_ERR_ARG
    assert norm(lib, q=P, ldq=64) == norm(lib, s=P) == G.GEMM_ERR_ARG          # q and scale go together
    assert norm(lib, eps=-1.0) == norm(lib, eps=float("nan")) == G.GEMM_ERR_ARG
    assert norm(lib, ldx=63) == norm(lib, ldy=63) == norm(lib, r=P, ldr=63) == G.GEMM_ERR_ARG
    assert norm(lib, ro=P, ldro=1) == norm(lib, q=P, ldq=8, s=P) == G.GEMM_ERR_ARG
    assert norm(lib, x=P + 1) == norm(lib, y=P + 1) == norm(lib, q=P, ldq=64, s=P + 2) == G.GEMM_ERR_ALIGN
    assert norm(lib, cols=2 ** 31, ldx=2 ** 31, ldy=2 ** 31) == G.GEMM_ERR_UNSUPPORTED
    assert norm(lib, rows=0) == G.GEMM_OK
    qf = lib.quantize_fp8
    assert qf(4, 64, P, 64, Q.QUANT_F32, None, 64, P, None) == G.GEMM_ERR_ARG
    assert qf(4, 64, P, 64, Q.QUANT_F32, P, 64, None, None) == G.GEMM_ERR_ARG
    assert qf(4, 64, P, 63, Q.QUANT_F32, P, 64, P, None) == G.GEMM_ERR_ARG
    assert qf(0, 64, None, 64, Q.QUANT_F32, None, 64, None, None) == G.GEMM_OK


def fp8(lib, M=8, N=16, K=32, A=P, lda=32, B=P, ldb=32, C=P, ldc=16, sa=P, sb=P, dt=Q.QUANT_BF16):
    return lib.gemm_fp8(M, N, K, A, lda, B, ldb, C, ldc, sa, sb, dt, None)


def test_gemm_fp8_arguments(lib):
    assert fp8(lib, M=-1) == fp8(lib, N=-1) == fp8(lib, K=-1) == fp8(lib, dt=5) == G.GEMM_ERR_ARG
    assert fp8(lib, A=None) == fp8(lib, B=None) == fp8(lib, C=None) == G.GEMM_ERR_ARG
    assert fp8(lib, sa=None) == fp8(lib, sb=None) == G.GEMM_ERR_ARG
    assert fp8(lib, lda=31) == fp8(lib, ldb=16) == fp8(lib, ldc=15) == G.GEMM_ERR_ARG
    assert fp8(lib, dt=Q.QUANT_F32) == G.GEMM_ERR_UNSUPPORTED
    assert fp8(lib, A=P + 8) == fp8(lib, B=P + 1) == fp8(lib, C=P + 2) == G.GEMM_ERR_ALIGN
    assert fp8(lib, lda=40) == fp8(lib, ldb=33) == fp8(lib, ldc=20) == fp8(lib, sa=P + 2) == G.GEMM_ERR_ALIGN
    assert fp8(lib, M=2 ** 31) == G.GEMM_ERR_UNSUPPORTED
    assert fp8(lib, M=0) == fp8(lib, N=0, C=None) == G.GEMM_OK


def w4(lib, M=2, N=16, K=128, x=P, ldx=128, W=P, ldw=64, s=P, lds=4, z=None, ldz=4, g=32, C=P, ldc=16,
       dt=Q.QUANT_F16):
    return lib.gemv_w4(M, N, K, x, ldx, W, ldw, s, lds, z, ldz, g, C, ldc, dt, None)


def test_gemv_w4_arguments(lib):
    assert w4(lib, M=-1) == w4(lib, N=-1) == w4(lib, K=-32) == w4(lib, dt=7) == G.GEMM_ERR_ARG
    assert w4(lib, g=16) == w4(lib, g=256) == w4(lib, K=96, g=64) == G.GEMM_ERR_ARG
    assert w4(lib, x=None) == w4(lib, W=None) == w4(lib, s=None) == w4(lib, C=None) == G.GEMM_ERR_ARG
    assert w4(lib, ldx=64) == w4(lib, ldw=63) == w4(lib, lds=3) == w4(lib, ldc=8) == G.GEMM_ERR_ARG
    assert w4(lib, z=P, ldz=3) == G.GEMM_ERR_ARG
    assert w4(lib, dt=Q.QUANT_F32) == G.GEMM_ERR_UNSUPPORTED
    assert w4(lib, x=P + 2) == w4(lib, W=P + 4) == w4(lib, ldw=72) == w4(lib, ldx=132) == G.GEMM_ERR_ALIGN
    assert w4(lib, C=P + 1) == w4(lib, s=P + 1) == G.GEMM_ERR_ALIGN
    assert w4(lib, K=2 ** 31, ldx=2 ** 31, ldw=2 ** 30, lds=2 ** 26) == G.GEMM_ERR_UNSUPPORTED
    assert w4(lib, M=0) == w4(lib, N=0) == G.GEMM_OK
    qw = lib.quantize_w4
    assert qw(4, 64, P, 64, Q.QUANT_F32, 48, P, 32, P, 2, Q.QUANT_F16, None, 0, None) == G.GEMM_ERR_ARG
    assert qw(4, 64, P, 64, Q.QUANT_F32, 32, P, 31, P, 2, Q.QUANT_F16, None, 0, None) == G.GEMM_ERR_ARG
    assert qw(4, 64, P, 64, Q.QUANT_F32, 32, P, 32, P, 2, Q.QUANT_F32, None, 0, None) == G.GEMM_ERR_UNSUPPORTED
    assert qw(4, 64, P, 64, Q.QUANT_F32, 32, P, 32, P, 2, Q.QUANT_F16, P, 1, None) == G.GEMM_ERR_ARG


def test_binding_refuses_host_tensors():
    x = torch.zeros(2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        Q.add_rmsnorm(x, x[0], y=x)
    with pytest.raises(ValueError, match="CUDA"):
        Q.gemv_w4(x, torch.zeros(4, 32, dtype=torch.uint8), x[:, :2], x[:, :4])


def test_empty_rows_are_aligned():
    for cols in (1, 15, 16, 17, 100):
        for dt, es in ((torch.float8_e4m3fn, 1), (torch.bfloat16, 2), (torch.float32, 4)):
            t = Q.empty_rows(3, cols, dt, device="cpu")
            assert t.shape == (3, cols) and t.stride(0) * es % 16 == 0 and t.stride(1) == 1


def test_reference_e4m3_matches_the_format():
    """Every finite e4m3 value rounds to itself, and midpoints go to even."""
    v = torch.arange(0, 127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(R.e4m3(v), v)
    mid = (v[1:] + v[:-1]) / 2
    even = np.where(np.arange(126) % 2 == 0, v[:-1], v[1:])
    assert np.array_equal(R.e4m3(mid), even)
    assert np.array_equal(R.e4m3(-mid), -even)


def test_reference_w4_by_hand():
    W = torch.tensor([[0x10, 0xF8] + [0x88] * 14], dtype=torch.uint8)
    s = torch.tensor([[0.5]])
    w = R.w4_weights(W, s, None, 32)
    assert w[0, :4].tolist() == [-4.0, -3.5, 0.0, 3.5] and not w[0, 4:].any()
    x = torch.zeros(1, 32)
    x[0, :4] = torch.tensor([1.0, 2.0, 3.0, 4.0])
    ref, absb = R.gemv_w4(x, W, s, torch.tensor([[0]], dtype=torch.uint8), 32)
    assert ref[0, 0] == 0 * 1 + 0.5 * 2 + 4 * 3 + 7.5 * 4 and absb[0, 0] == ref[0, 0]


def test_reference_catches_planted_mistakes():
    """The checks fail for a scale, a rounding and a nibble order that are wrong."""
    x = torch.randn(3, 64, generator=torch.Generator().manual_seed(1))
    h, y = R.norm(x, torch.ones(64), None, 1e-6)
    s = R.row_scale(y)
    q = torch.from_numpy(R.e4m3(y / s[:, None]))
    R.check_q(q, torch.from_numpy(s), y, "right")
    with pytest.raises(AssertionError):
        R.check_q(q, torch.from_numpy(s * 1.001), y, "scale")
    down = torch.from_numpy(R.e4m3(y / s[:, None] * 0.97))
    with pytest.raises(AssertionError):
        R.check_q(down, torch.from_numpy(s), y, "rounding")
    W = torch.randint(0, 256, (8, 32), generator=torch.Generator().manual_seed(2), dtype=torch.uint8)
    sc = torch.ones(8, 2)
    ref, absb = R.gemv_w4(x, W, sc, None, 32)
    swapped = (W >> 4) | ((W & 15) << 4)
    wrong, _ = R.gemv_w4(x, swapped, sc, None, 32)
    R.check_rounded(torch.from_numpy(ref).float(), ref, 1e-6, R.W4_REL * absb, "right")
    with pytest.raises(AssertionError):
        R.check_rounded(torch.from_numpy(wrong).float(), ref, 1e-6, R.W4_REL * absb, "nibbles")
