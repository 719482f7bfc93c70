"""The plan queries of include/quant.h: arguments without a GPU, answers on one.
No test here launches a kernel."""
import ctypes
import os
import re

import pytest
import torch

from stage_software_pipelining_gb300 import build as gemm_build
from stage_software_pipelining_gb300 import gemm as G
from stage_software_pipelining_gb300 import quant as Q

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def lib():
    gemm_build.build()
    return Q.load_library()


def test_header_and_binding_agree():
    text = open(os.path.join(ROOT, "include", "quant.h"), encoding="utf-8").read()
    names = re.findall(r"QUANT_KERNEL_(\w+) = (\d+)", text)
    assert [n.lower() for n, _ in names] == list(Q.KERNELS)
    assert [int(i) for _, i in names] == list(range(len(Q.KERNELS)))
    body = re.sub(r"/\*.*?\*/", "", text, flags=re.S).split("quant_kernel_t;")[1].split("quant_plan_t;")[0]
    assert re.findall(r"int (\w+);", body) == [n for n, _ in Q._Plan._fields_]


def test_plan_arguments(lib):
    p = Q._Plan()
    out = ctypes.byref(p)
    f, w = lib.gemm_fp8_plan, lib.gemv_w4_plan
    for bad in ((0, 8, 8, 2), (8, 0, 8, 2), (8, 8, 0, 2), (-1, 8, 8, 2), (8, 8, 8, 3), (8, 8, 8, -1)):
        assert f(*bad, out) == G.GEMM_ERR_ARG
    assert f(8, 8, 8, Q.QUANT_BF16, None) == G.GEMM_ERR_ARG
    assert f(8, 8, 8, Q.QUANT_F32, out) == f(2 ** 31, 8, 8, Q.QUANT_F16, out) == G.GEMM_ERR_UNSUPPORTED
    for bad in ((0, 8, 64, 32, 0, 2), (8, 8, 64, 48, 0, 2), (8, 8, 64, 128, 0, 2), (8, 8, 64, 32, 2, 2),
                (8, 8, 64, 32, 0, 9)):
        assert w(*bad, out) == G.GEMM_ERR_ARG
    assert w(8, 8, 64, 32, 0, Q.QUANT_F16, None) == G.GEMM_ERR_ARG
    assert w(8, 8, 64, 32, 0, Q.QUANT_F32, out) == G.GEMM_ERR_UNSUPPORTED
    assert w(8, 8, 2 ** 27, 32, 0, Q.QUANT_F16, out) == G.GEMM_ERR_UNSUPPORTED
    with pytest.raises(G.GemmError):
        Q.gemm_fp8_plan(8, 8, 8, torch.float64)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_plans_on_the_gpu(gpu, lib, dtype):
    one = Q.gemm_fp8_plan(1, 4096, 4096, dtype)
    assert one["kernel"] == "fp8_few" and one["tile_rows"] == 16 and one["split"] > 1
    assert one["grid"] == 32 * one["split"] and 2 <= one["stages"] <= 12
    many = Q.gemm_fp8_plan(8191, 28672, 4096, dtype)
    assert many["kernel"] == "fp8_pair" and many["tile_rows"] == 256 and many["split"] == 1
    assert many["stages"] == 6 and many["grid"] % 2 == 0
    assert many["grid"] <= torch.cuda.get_device_properties(0).multi_processor_count
    for M, kernel, rows in ((1, "w4_warp", 8), (8, "w4_warp", 8), (9, "w4_warp", 16), (20, "w4_tc", 32)):
        p = Q.gemv_w4_plan(M, 8192, 8192, 64, True, dtype)
        assert p["kernel"] == kernel and p["tile_rows"] == rows and p["grid"] % p["split"] == 0


# Shared memory of an SM and, of that, the system's part of each CTA.
SM_SMEM, CTA_SMEM = 228 * 1024, 1024


def few_row_plans():
    """Every few-row tile of gemm_fp8 and its cuts, and gemv_w4's tcgen05 kernel."""
    for M in (1, 5, 16, 20, 32, 40, 64, 100, 200, 256, 300, 600, 700):
        for N, K in ((64, 128), (520, 768), (600, 2048), (4096, 4096), (28672, 4096), (8192, 300), (40000, 256)):
            yield f"gemm_fp8 {M} x {N} x {K}", Q.gemm_fp8_plan(M, N, K)
    for M, N, K, group in ((17, 13001, 128, 32), (32, 8192, 28672, 128), (24, 8192, 8192, 64)):
        for zeros in (False, True):
            yield f"gemv_w4 {M} x {N} x {K}", Q.gemv_w4_plan(M, N, K, group, zeros)


@pytest.mark.gpu
def test_no_tensor_memory_neighbour_of_the_gemm(gpu, lib):
    """A CTA of the GEMM may take all of an SM's tensor memory: no CTA of a
    kernel with tensor memory fits beside it, on whichever stream it runs."""
    least = min(G.plan(1024, 1024, 1024, G.GEMM_BF16_F32, stages, tile=tile)["smem_bytes"]
                for tile in G.TILE_MAX_STAGES for stages in (1, 2))
    for name, p in few_row_plans():
        if p["kernel"] != "w4_warp":  # no tensor memory
            assert least + p["smem_bytes"] + 2 * CTA_SMEM > SM_SMEM, f"{name}: {p}"


@pytest.mark.gpu
def test_two_small_ctas_still_share_an_sm(gpu, lib):
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    for name, p in few_row_plans():
        if p["grid"] > 2 * sms or p["tile_rows"] > 64 or p["kernel"] == "fp8_pair":
            continue
        if p["kernel"] == "w4_tc" or (p["grid"] > sms and p["kernel"] == "fp8_few" and p["stages"] < 6):
            assert 2 * (p["smem_bytes"] + CTA_SMEM) <= SM_SMEM, f"{name}: {p}"
