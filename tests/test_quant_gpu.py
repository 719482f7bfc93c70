"""The quantised operators on the GPU against their 64-bit forms (quant_reference.py)."""
import numpy as np
import pytest
import torch

import quant_reference as R
from gpu_helpers import GuardedC
from stage_software_pipelining_gb300 import build as gemm_build
from stage_software_pipelining_gb300 import gemm as G
from stage_software_pipelining_gb300 import quant as Q

pytestmark = pytest.mark.gpu
F32, F16, BF16, E4M3 = torch.float32, torch.float16, torch.bfloat16, torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def lib(gpu):
    gemm_build.build()
    return Q.load_library()


def rand(seed, *shape):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed))


def wide(t, extra=8, offset=0):
    """A device copy of t in a buffer of longer rows, NaN outside it, that
    starts `offset` elements past an aligned address."""
    rows, cols = t.shape
    buf = torch.full((rows * (cols + extra) + offset,), float("nan"), device="cuda").to(t.dtype)
    v = buf[offset:].view(rows, cols + extra)[:, :cols]
    v.copy_(t)
    return v


# ---------------------------------------------------------------- add_rmsnorm
NORM_SHAPES = [(1, 1), (3, 2), (1, 4096), (5, 31), (4, 128), (300, 64), (7, 1999), (37, 8192), (9, 1000),
               (2, 16384), (3, 16385), (1, 40000), (640, 2048)]


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("rows,cols", NORM_SHAPES)
def test_norm_all_outputs(rows, cols, dtype):
    x, r = rand(1, rows, cols).to(dtype), (3 * rand(2, rows, cols)).to(dtype)
    w = (1 + 0.2 * rand(3, cols)).to(dtype)
    out = [GuardedC(rows, cols, dtype) for _ in range(2)]
    q = Q.empty_rows(rows, cols, E4M3)
    scale = torch.empty(rows, device="cuda")
    Q.add_rmsnorm(x.cuda(), w.cuda(), r.cuda(), eps=1e-5, residual_out=out[0].view, y=out[1].view,
                  q=q, scale=scale)
    h, y = R.norm(x, w, r, 1e-5)
    for o in out:
        o.check()
    R.check_rounded(out[0].view, h, 2.0 ** -24, 0.0, "residual_out")
    R.check_rounded(out[1].view, y, R.NORM_REL, 0.0, "y")
    R.check_q(q, scale, y, "q")


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("cols", [96, 1999, 4096, 20000])
@pytest.mark.parametrize("outs", ["r", "y", "q", "ry", "rq", "yq"])
@pytest.mark.parametrize("with_residual", [False, True])
def test_norm_any_set_of_outputs(cols, outs, with_residual, dtype):
    rows = 5
    x = rand(4, rows, cols).to(dtype)
    r = rand(5, rows, cols).to(dtype) if with_residual else None
    w = rand(6, cols).to(dtype)
    ro = torch.empty(rows, cols, dtype=dtype, device="cuda") if "r" in outs else None
    yo = torch.empty(rows, cols, dtype=dtype, device="cuda") if "y" in outs else None
    q = torch.empty(rows, cols, dtype=E4M3, device="cuda") if "q" in outs else None
    scale = torch.empty(rows, device="cuda") if "q" in outs else None
    Q.add_rmsnorm(x.cuda(), w.cuda(), r.cuda() if with_residual else None, residual_out=ro, y=yo, q=q,
                  scale=scale)
    h, y = R.norm(x, w, r, 1e-6)
    if ro is not None:
        R.check_rounded(ro, h, 2.0 ** -24, 0.0, "residual_out")
    if yo is not None:
        R.check_rounded(yo, y, R.NORM_REL, 0.0, "y")
    if q is not None:
        R.check_q(q, scale, y, "q")


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("cols,extra,offset", [(512, 8, 0), (512, 3, 0), (512, 8, 1), (1000, 24, 5), (17, 1, 1),
                                               (16400, 9, 3)])
def test_norm_strides_and_offsets(cols, extra, offset, dtype):
    rows = 6
    x, r, w = rand(7, rows, cols).to(dtype), rand(8, rows, cols).to(dtype), rand(9, cols).to(dtype)
    dx, dr, dw = wide(x, extra, offset), wide(r, extra + 1, 0), wide(w[None], 0, offset)[0]
    y = wide(torch.zeros(rows, cols, dtype=dtype), extra, offset)
    qb = torch.zeros(rows, cols + extra + offset, dtype=torch.uint8, device="cuda")
    q = qb.view(E4M3)[:, offset:offset + cols]
    scale = torch.empty(rows, device="cuda")
    Q.add_rmsnorm(dx, dw, dr, residual_out=dr, y=y, q=q, scale=scale)      # dr in place
    h, ref = R.norm(x, w, r, 1e-6)
    R.check_rounded(dr, h, 2.0 ** -24, 0.0, "residual_out in place")
    R.check_rounded(y, ref, R.NORM_REL, 0.0, "y")
    R.check_q(q, scale, ref, "q")
    outside = torch.ones_like(qb, dtype=torch.bool)
    outside[:, offset:offset + cols] = False
    assert not qb[outside].any(), "a write landed outside q"


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("rows,cols", [(2000, 1277), (2000, 1503), (1900, 2999), (400, 3501), (1900, 6001)])
def test_norm_many_rows_of_odd_width(rows, cols, dtype):
    test_norm_all_outputs(rows, cols, dtype)


@pytest.mark.parametrize("cols", [256, 4096, 33000])
def test_norm_in_place_on_x(cols):
    x, w = rand(10, 4, cols).to(BF16), rand(11, cols).to(BF16)
    d = x.cuda()
    Q.add_rmsnorm(d, w.cuda(), y=d)
    R.check_rounded(d, R.norm(x, w, None, 1e-6)[1], R.NORM_REL, 0.0, "y over x")


@pytest.mark.parametrize("cols", [40, 4096, 20000])
def test_norm_special_rows(cols):
    """Zero rows, NaN, infinity and values whose squares leave fp32's range."""
    x = rand(12, 6, cols)
    x[1] = 0
    x[2, cols // 2] = float("nan")
    x[3, cols - 1] = float("inf")
    x[4] = 1e-30
    w = torch.ones(cols)
    y = torch.empty(6, cols, device="cuda")
    q, scale = torch.empty(6, cols, dtype=E4M3, device="cuda"), torch.empty(6, device="cuda")
    Q.add_rmsnorm(x.cuda(), w.cuda(), y=y, q=q, scale=scale)
    y, qf, scale = y.cpu(), q.float().cpu(), scale.cpu()
    ok = [0, 4, 5]
    ref = R.norm(x, w, None, 1e-6)[1]
    R.check_rounded(y[ok], ref[ok], R.NORM_REL, 0.0, "y")
    R.check_q(qf[ok], scale[ok], ref[ok], "q")
    assert not y[1].any() and not qf[1].any() and scale[1].item() == R.SCALE_MIN
    for i in (2, 3):
        assert torch.isnan(scale[i]) and torch.isnan(qf[i]).all()
    assert torch.isnan(y[2]).all()
    # a NaN weight reaches every row's scale, not only its own column
    w[0] = float("nan")
    Q.add_rmsnorm(x.cuda(), w.cuda(), q=q, scale=(s := torch.empty(6, device="cuda")))
    assert torch.isnan(s).all() and torch.isnan(q.float()).all()


def test_norm_tiny_rows_have_finite_scales():
    x = torch.full((2, 64), 1e-42)
    q, scale = torch.empty(2, 64, dtype=E4M3, device="cuda"), torch.empty(2, device="cuda")
    Q.quantize_fp8(x.cuda(), q, scale)
    assert (scale.cpu() == R.SCALE_MIN).all()
    assert (q.float().cpu() * scale.cpu()[:, None] <= 1e-42 * 1.1).all()


@pytest.mark.parametrize("rows,cols", [(0, 64), (3, 0)])
def test_norm_empty(rows, cols):
    x = torch.empty(rows, cols, device="cuda")
    scale = torch.full((rows,), 5.0, device="cuda")
    Q.add_rmsnorm(x, torch.empty(cols, device="cuda"), y=torch.empty_like(x),
                  q=torch.empty(rows, cols, dtype=E4M3, device="cuda"), scale=scale)
    assert (scale.cpu() == R.SCALE_MIN).all()


def test_norm_offsets_past_32_bits():
    """Rows more than 2^31 elements apart."""
    rows, ld, cols = 2051, 1 << 20, 256
    x = rand(13, rows, cols).to(BF16)
    big = torch.empty(rows * ld, dtype=BF16, device="cuda").view(rows, ld)[:, :cols]
    big.copy_(x)
    w = torch.ones(cols, dtype=BF16)
    Q.add_rmsnorm(big, w.cuda(), y=big)
    R.check_rounded(big, R.norm(x, w, None, 1e-6)[1], R.NORM_REL, 0.0, "y")


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("rows,cols", [(1, 1), (5, 100), (64, 4096), (2, 33000)])
def test_quantize_fp8(rows, cols, dtype):
    x = (0.02 * rand(14, rows, cols)).to(dtype)
    q, scale = torch.empty(rows, cols, dtype=E4M3, device="cuda"), torch.empty(rows, device="cuda")
    assert Q.quantize_fp8(x.cuda(), q, scale) is q
    R.check_q(q, scale, R.f64(x), "q", rel=1e-6)


def test_norm_on_another_stream():
    x, w = rand(15, 64, 4096).to(BF16).cuda(), torch.ones(4096, dtype=BF16, device="cuda")
    a, b = torch.empty_like(x), torch.empty_like(x)
    Q.add_rmsnorm(x, w, y=a)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    Q.add_rmsnorm(x, w, y=b, stream=s)
    with torch.cuda.stream(s):
        b2 = b.clone()
    s.synchronize()
    torch.cuda.synchronize()
    assert torch.equal(a, b2)


# ---------------------------------------------------------------- gemm_fp8
def fp8_rows(v):
    """Quantised rows on the device, NaN beyond them, and their scales."""
    s = (v.abs().amax(dim=1) / 448).clamp_min(R.SCALE_MIN)
    q = (v / s[:, None]).clamp(-448, 448).to(E4M3)
    rows, cols = q.shape
    ld = (cols + 15) // 16 * 16 + 16
    buf = torch.full((rows, ld), 0x7F, dtype=torch.uint8, device="cuda").view(E4M3)
    buf[:, :cols].copy_(q)
    return buf[:, :cols], s.cuda()


def fp8_case(M, N, K, dtype, seed=20):
    A, sa = fp8_rows(rand(seed, M, K))
    W, sb = fp8_rows(0.05 * rand(seed + 1, N, K))
    C = GuardedC(M, N, dtype)
    assert Q.gemm_fp8(A, W.t(), C.view, sa, sb) is C.view
    C.check()
    ref, absb = R.gemm_fp8(A, W.t(), sa, sb)
    R.check_rounded(C.view, ref, 2.0 ** -22, R.SUM_REL * absb, f"{M}x{N}x{K}")
    return C.view


FP8_SHAPES = [(600, 300, 2048), (2000, 400, 1024), (400, 2000, 1500), (1, 40000, 256), (40, 40000, 300),
              (90, 20000, 130), (300, 700, 8), (2000, 900, 512), (1300, 2600, 300), (1, 1, 1), (1, 64, 128),
              (1, 4096, 512), (2, 130, 33), (8, 256, 1000), (15, 17, 129), (16, 384, 2048), (17, 100, 256),
              (33, 1000, 640), (48, 2048, 512), (64, 129, 127), (65, 512, 384), (100, 260, 512),
              (128, 128, 128), (129, 129, 129), (200, 520, 192), (255, 777, 1040), (256, 256, 2048),
              (300, 4096, 256), (513, 1025, 257), (1000, 1504, 1000), (2048, 512, 64), (1, 3, 2000)]


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("M,N,K", FP8_SHAPES)
def test_gemm_fp8(M, N, K, dtype):
    fp8_case(M, N, K, dtype)


@pytest.mark.parametrize("M", [1, 16, 64, 128, 200, 640])
def test_gemm_fp8_is_repeatable(M):
    a = fp8_case(M, 1100, 1024, BF16, seed=30).clone()
    assert torch.equal(a, fp8_case(M, 1100, 1024, BF16, seed=30))


@pytest.mark.parametrize("M,N,K", [(1, 256, 256), (20, 300, 200), (300, 300, 300)])
def test_gemm_fp8_nan_stays_in_its_row_and_column(M, N, K):
    A, sa = fp8_rows(rand(40, M, K))
    W, sb = fp8_rows(rand(41, N, K))
    A[M - 1, K - 1] = float("nan")
    W[N // 2, 0] = float("nan")
    C = torch.zeros(M, (N + 7) // 8 * 8, dtype=F16, device="cuda")[:, :N]
    Q.gemm_fp8(A, W.t(), C, sa, sb)
    nan = torch.isnan(C).cpu()
    expect = torch.zeros_like(nan)
    expect[M - 1] = True
    expect[:, N // 2] = True
    assert torch.equal(nan, expect)


@pytest.mark.parametrize("M", [3, 300])
def test_gemm_fp8_overflow_and_scales(M):
    """fp16 results past its range are infinities; scales may be zero or negative."""
    K, N = 256, 160
    A = torch.ones(M, K, device="cuda").to(E4M3)
    W = torch.ones(N, K, device="cuda").to(E4M3)
    sa = torch.linspace(0, 400, M, device="cuda")
    sb = torch.where(torch.arange(N, device="cuda") % 2 == 0, 1.0, -1.0)
    C = torch.empty(M, N, dtype=F16, device="cuda")
    Q.gemm_fp8(A, W.t(), C, sa, sb)
    expect = (K * sa[:, None] * sb[None, :]).to(F16)
    assert torch.equal(C, expect) and torch.isinf(C).any() and not C[0].any()


@pytest.mark.parametrize("M,N,K", [(5, 600, 2048), (600, 600, 2048), (200, 300, 1500)])
def test_gemm_fp8_stuck_pipeline_is_reported(M, N, K):
    """A stage whose copy never comes ends in GEMM_ERR_TIMEOUT, and the next call is right."""
    A, sa = fp8_rows(rand(42, M, K))
    W, sb = fp8_rows(rand(43, N, K))
    C = torch.empty(M, (N + 7) // 8 * 8, dtype=BF16, device="cuda")[:, :N]
    try:
        G.debug_set(wait_limit_ns=50_000_000, withhold_arrive=0)
        with pytest.raises(G.GemmError, match="TIMEOUT"):
            Q.gemm_fp8(A, W.t(), C, sa, sb, checked=True)
    finally:
        G.debug_set()
    Q.gemm_fp8(A, W.t(), C, sa, sb, checked=True)
    ref, absb = R.gemm_fp8(A, W.t(), sa, sb)
    R.check_rounded(C, ref, 2.0 ** -22, R.SUM_REL * absb, "after a timeout")


def test_gemm_fp8_empty():
    e = torch.empty(0, device="cuda")
    A, W = torch.empty(4, 0, dtype=E4M3, device="cuda"), torch.empty(8, 0, dtype=E4M3, device="cuda")
    C = torch.full((4, 8), 3.0, dtype=BF16, device="cuda")
    Q.gemm_fp8(A, W.t(), C, torch.ones(4, device="cuda"), torch.ones(8, device="cuda"))
    assert not C.any()
    Q.gemm_fp8(torch.empty(0, 16, dtype=E4M3, device="cuda"), torch.empty(8, 16, dtype=E4M3, device="cuda").t(),
               torch.empty(0, 8, dtype=BF16, device="cuda"), e, torch.ones(8, device="cuda"))


# ---------------------------------------------------------------- gemv_w4
def w4_case(M, N, K, group, zeros, dtype, seed=50, extra=16):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(M, K, generator=g).to(dtype)
    W = torch.randint(0, 256, (N, K // 2), generator=g, dtype=torch.uint8)
    s = (torch.rand(N, K // group, generator=g) * 0.02 - 0.005).to(dtype)
    z = torch.randint(0, 16, (N, K // group), generator=g, dtype=torch.uint8) if zeros else None
    dx = wide(x, extra)
    dW = torch.full((N, K // 2 + extra), 0xFF, dtype=torch.uint8, device="cuda")[:, :K // 2]
    dW.copy_(W)
    ds = wide(s, 3)
    dz = None
    if zeros:
        dz = torch.full((N, K // group + 5), 99, dtype=torch.uint8, device="cuda")[:, :K // group]
        dz.copy_(z)
    C = GuardedC(M, N, dtype)
    assert Q.gemv_w4(dx, dW, ds, C.view, zeros=dz) is C.view
    C.check()
    ref, absb = R.gemv_w4(x, W, s, z, group)
    R.check_rounded(C.view, ref, 2.0 ** -22, R.W4_REL * absb, f"{M}x{N}x{K} group {group}")
    return C.view


W4_SHAPES = [(1, 1, 128), (1, 16, 128), (1, 17, 256), (1, 1000, 4096), (2, 33, 384), (5, 100, 8192), (7, 64, 640),
             (8, 257, 1024), (9, 128, 2048), (16, 130, 512), (17, 48, 1152), (31, 99, 128), (32, 272, 4096),
             (33, 80, 256), (70, 31, 512)]


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("group,zeros", [(32, False), (32, True), (64, True), (128, False), (128, True)])
@pytest.mark.parametrize("M,N,K", W4_SHAPES)
def test_gemv_w4(M, N, K, group, zeros, dtype):
    w4_case(M, N, K, group, zeros, dtype)


# More than 16 rows with more weights than the few-row kernel's tiles are taken for.
@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("group,zeros", [(32, False), (32, True), (64, True), (128, False), (128, True)])
@pytest.mark.parametrize("M,N,K", [(17, 13001, 128), (31, 12999, 384), (32, 13008, 1152), (33, 8900, 640),
                                   (70, 5100, 512), (20, 1030, 24576), (64, 1100, 9216), (24, 300, 81920)])
def test_gemv_w4_many_weights(M, N, K, group, zeros, dtype):
    w4_case(M, N, K, group, zeros, dtype)


@pytest.mark.parametrize("M,N,K,group", [(17, 13001, 32, 32), (24, 13001, 2080, 32), (32, 13001, 192, 64)])
def test_gemv_w4_many_weights_k_that_is_not_a_multiple_of_128(M, N, K, group):
    w4_case(M, N, K, group, True, BF16)


@pytest.mark.parametrize("M", [20, 40])
def test_gemv_w4_many_weights_is_repeatable(M):
    a = w4_case(M, 8200, 4096, 64, True, F16).clone()
    assert torch.equal(a, w4_case(M, 8200, 4096, 64, True, F16))


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("group,zeros", [(32, True), (64, False), (128, True)])
def test_gemv_w4_many_weights_infinite_and_large_x(group, zeros, dtype):
    test_gemv_w4_infinite_and_large_x(20, group, zeros, dtype, N=13001)


def test_gemv_w4_many_weights_stuck_pipeline_is_reported():
    M, N, K = 20, 13001, 2048
    g = torch.Generator().manual_seed(64)
    x = torch.randn(M, K, generator=g).to(BF16).cuda()
    W = torch.randint(0, 256, (N, K // 2), generator=g, dtype=torch.uint8).cuda()
    s = (torch.rand(N, K // 64, generator=g) * 0.01).to(BF16).cuda()
    C = torch.empty(M, N, dtype=BF16, device="cuda")
    try:
        G.debug_set(wait_limit_ns=50_000_000, withhold_arrive=0)
        with pytest.raises(G.GemmError, match="TIMEOUT"):
            Q.gemv_w4(x, W, s, C, checked=True)
    finally:
        G.debug_set()
    Q.gemv_w4(x, W, s, C, checked=True)
    ref, absb = R.gemv_w4(x, W, s, None, 64)
    R.check_rounded(C, ref, 2.0 ** -22, R.W4_REL * absb, "after a timeout")


@pytest.mark.parametrize("M,N,K,group", [(1, 40, 32, 32), (3, 40, 96, 32), (1, 50, 192, 64), (12, 20, 2080, 32),
                                         (32, 64, 1056, 32)])
def test_gemv_w4_k_that_is_not_a_multiple_of_128(M, N, K, group):
    w4_case(M, N, K, group, True, BF16)


@pytest.mark.parametrize("M", [1, 4, 16, 32])
def test_gemv_w4_is_repeatable(M):
    a = w4_case(M, 600, 4096, 64, True, F16).clone()
    assert torch.equal(a, w4_case(M, 600, 4096, 64, True, F16))


@pytest.mark.parametrize("M", [1, 6, 20])
def test_gemv_w4_special_values_stay_in_their_row(M):
    K, N = 256, 48
    g = torch.Generator().manual_seed(60)
    x = torch.randn(M, K, generator=g).to(F16).cuda()
    W = torch.randint(0, 256, (N, K // 2), generator=g, dtype=torch.uint8).cuda()
    s = torch.ones(N, K // 128, dtype=F16, device="cuda")
    C = torch.empty(M, N, dtype=F16, device="cuda")
    x[M // 2, 3] = float("nan")
    s[7, 1] = float("nan")
    Q.gemv_w4(x, W, s, C)
    nan = torch.isnan(C).cpu()
    expect = torch.zeros_like(nan)
    expect[M // 2] = True
    expect[:, 7] = True
    assert torch.equal(nan, expect)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("group,zeros", [(32, False), (32, True), (64, True), (128, False), (128, True)])
@pytest.mark.parametrize("M", [1, 2, 6, 12, 20])
def test_gemv_w4_infinite_and_large_x(M, group, zeros, dtype, N=150):
    """An infinity takes the sign of its weight less the zero point (NaN where
    they are equal); the largest finite values do not overflow on the way."""
    K = 1600 // group * group
    g = torch.Generator().manual_seed(62)
    x = torch.randn(M, K, generator=g).to(dtype)
    W = torch.randint(0, 256, (N, K // 2), generator=g, dtype=torch.uint8)
    z = torch.full((N, K // group), 7 if zeros else 8, dtype=torch.uint8)
    W[:, 20] = 0x10 * (z[:, 0] + 1) + torch.randint(0, 3, (N,), generator=g, dtype=torch.uint8) + z[:, 0] - 1
    s = torch.full((N, K // group), 2.0 ** -12, dtype=dtype)
    C = torch.empty(M, N, dtype=dtype, device="cuda")
    dev = (W.cuda(), s.cuda(), C)
    huge = float(torch.finfo(dtype).max)
    x[M - 1, 40] = huge  # weights z - 1, z, z + 1
    Q.gemv_w4(x.cuda(), *dev, zeros=z.cuda() if zeros else None)
    ref, absb = R.gemv_w4(x, W, s, z, group)
    R.check_rounded(C, ref, 2.0 ** -22, R.W4_REL * absb, "the largest finite value")
    x[M - 1, 40] = float("inf")
    Q.gemv_w4(x.cuda(), *dev, zeros=z.cuda() if zeros else None)
    d = (W[:, 20] & 15).double() - z[:, 0].double()
    assert torch.equal(C[M - 1].isnan().cpu(), d == 0)
    assert torch.equal(C[M - 1].isinf().cpu(), d != 0)
    assert torch.equal(C[M - 1].cpu()[d != 0].sign().double(), d[d != 0].sign())
    assert C[:M - 1].isfinite().all()


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("groups", [1, 7, 8, 13, 26, 40])
def test_gemv_w4_rows_of_groups_on_their_boundaries(groups, group, dtype):
    """One row of x; scales and zero points in rows of a multiple of eight."""
    N, K, pitch = 77, groups * group, (groups + 7) // 8 * 8
    g = torch.Generator().manual_seed(63)
    x = torch.randn(1, K, generator=g).to(dtype)
    W = torch.randint(0, 256, (N, K // 2), generator=g, dtype=torch.uint8)
    s = (torch.rand(N, groups, generator=g) * 0.02 - 0.005).to(dtype)
    z = torch.randint(0, 16, (N, groups), generator=g, dtype=torch.uint8)
    ds = wide(s, pitch - groups)
    dz = torch.full((N, pitch), 99, dtype=torch.uint8, device="cuda")[:, :groups]
    dz.copy_(z)
    for dz, hz in ((None, None), (dz, z)):
        C = GuardedC(1, N, dtype)
        Q.gemv_w4(x.cuda(), W.cuda(), ds, C.view, zeros=dz)
        C.check()
        ref, absb = R.gemv_w4(x, W, s, hz, group)
        R.check_rounded(C.view, ref, 2.0 ** -22, R.W4_REL * absb, f"{groups} groups of {group}")


def test_gemv_w4_fp16_range():
    """Group sums past fp16's range are not lost before a small scale brings them back."""
    K, N = 1024, 16
    x = torch.full((1, K), 60000.0, dtype=F16, device="cuda")
    W = torch.full((N, K // 2), 0xFF, dtype=torch.uint8, device="cuda")
    s = torch.full((N, K // 128), 2.0 ** -20, dtype=F16, device="cuda")
    C = torch.empty(1, N, dtype=F16, device="cuda")
    Q.gemv_w4(x, W, s, C)
    exact = float(x[0, 0]) * 7 * K * 2.0 ** -20
    assert torch.allclose(C.double(), torch.full_like(C, exact).double(), rtol=2.0 ** -11)


@pytest.mark.parametrize("M", [1, 3, 7, 12, 20])
def test_gemv_w4_stuck_pipeline_is_reported(M):
    K, N = 2048, 200
    g = torch.Generator().manual_seed(61)
    x = torch.randn(M, K, generator=g).to(BF16).cuda()
    W = torch.randint(0, 256, (N, K // 2), generator=g, dtype=torch.uint8).cuda()
    s = (torch.rand(N, K // 64, generator=g) * 0.01).to(BF16).cuda()
    C = torch.empty(M, N, dtype=BF16, device="cuda")
    try:
        G.debug_set(wait_limit_ns=50_000_000, withhold_arrive=0)
        with pytest.raises(G.GemmError, match="TIMEOUT"):
            Q.gemv_w4(x, W, s, C, checked=True)
    finally:
        G.debug_set()
    Q.gemv_w4(x, W, s, C, checked=True)
    ref, absb = R.gemv_w4(x, W, s, None, 64)
    R.check_rounded(C, ref, 2.0 ** -22, R.W4_REL * absb, "after a timeout")


def test_gemv_w4_empty():
    C = torch.full((2, 8), 3.0, dtype=BF16, device="cuda")
    Q.gemv_w4(torch.empty(2, 0, dtype=BF16, device="cuda"), torch.empty(8, 0, dtype=torch.uint8, device="cuda"),
              torch.empty(8, 0, dtype=BF16, device="cuda"), C)
    assert not C.any()


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("zeros", [False, True])
def test_quantize_w4_is_near_its_weights(group, zeros, dtype):
    N, K = 37, 640
    w = (0.03 * rand(70, N, K) + (0.02 if zeros else 0.0)).to(dtype)
    w[5] = 0
    W = torch.empty(N, K // 2, dtype=torch.uint8, device="cuda")
    s = torch.empty(N, K // group, dtype=BF16, device="cuda")
    z = torch.empty(N, K // group, dtype=torch.uint8, device="cuda") if zeros else None
    assert Q.quantize_w4(w.cuda(), W, s, z) is W
    back = R.w4_weights(W, s, z, group)
    step = R.f64(s).repeat(group, axis=1)
    # Half a step; where the scale was rounded down to bf16 (2^-8) the ends of
    # the range move by 15 * 2^-8 of a step at most, and the zero point's own
    # rounding shifts the range by half a step.
    limit = step * (0.5 + 15 * 2.0 ** -8 + (0.5 if zeros else 0.0)) + 1e-7
    assert (np.abs(back - R.f64(w)) <= limit).all()
    assert not back[5].any()


# ---------------------------------------------------------------- together
@pytest.mark.parametrize("T", [1, 40, 300])
def test_norm_then_products(T):
    """The norm's 8-bit rows through gemm_fp8 and its 16-bit rows through gemv_w4."""
    D, N = 512, 384
    x, r, w = rand(80, T, D).to(BF16), rand(81, T, D).to(BF16), (1 + 0.1 * rand(82, D)).to(BF16)
    y, q = torch.empty(T, D, dtype=BF16, device="cuda"), torch.empty(T, D, dtype=E4M3, device="cuda")
    scale = torch.empty(T, device="cuda")
    Q.add_rmsnorm(x.cuda(), w.cuda(), r.cuda(), y=y, q=q, scale=scale)
    weights = 0.05 * rand(83, N, D)
    Wq, ws = torch.empty(N, D, dtype=E4M3, device="cuda"), torch.empty(N, device="cuda")
    Q.quantize_fp8(weights.cuda(), Wq, ws)
    C8 = torch.empty(T, N, dtype=BF16, device="cuda")
    Q.gemm_fp8(q, Wq.t(), C8, scale, ws)
    ref, absb = R.gemm_fp8(q, Wq.t(), scale, ws)
    R.check_rounded(C8, ref, 2.0 ** -22, R.SUM_REL * absb, "8-bit product")
    W4 = torch.empty(N, D // 2, dtype=torch.uint8, device="cuda")
    s4 = torch.empty(N, D // 64, dtype=BF16, device="cuda")
    Q.quantize_w4(weights.cuda(), W4, s4)
    C4 = torch.empty(T, N, dtype=BF16, device="cuda")
    Q.gemv_w4(y, W4, s4, C4)
    ref, absb = R.gemv_w4(y, W4, s4, None, 64)
    R.check_rounded(C4, ref, 2.0 ** -22, R.W4_REL * absb, "4-bit product")


# ---------------------------------------------------------------- refusals
def test_refusals():
    x = torch.zeros(4, 64, dtype=BF16, device="cuda")
    w = torch.ones(64, dtype=BF16, device="cuda")
    q, s = torch.zeros(4, 64, dtype=E4M3, device="cuda"), torch.zeros(4, device="cuda")
    bad = [lambda: Q.add_rmsnorm(x, w),                                        # no output
           lambda: Q.add_rmsnorm(x, w, q=q),                                   # q without scale
           lambda: Q.add_rmsnorm(x, w[:63], y=x),                              # width
           lambda: Q.add_rmsnorm(x, w.float(), y=x),                           # type
           lambda: Q.add_rmsnorm(x, w, x[:3], y=x),                            # shape
           lambda: Q.add_rmsnorm(x.t(), w[:4], y=x.t()),                       # column-major
           lambda: Q.add_rmsnorm(x[:1].expand(4, 64), w, y=x),                 # overlapping rows
           lambda: Q.add_rmsnorm(x.cpu(), w, y=x),                             # host tensor
           lambda: Q.add_rmsnorm(x, w, y=x.float()),
           lambda: Q.quantize_fp8(x, q[:, :32], s),
           lambda: Q.quantize_fp8(x, q, s[:3]),
           lambda: Q.gemm_fp8(q, q.t(), torch.zeros(4, 4, device="cuda"), s, s),          # fp32 C
           lambda: Q.gemm_fp8(q, q, x[:, :4], s, s),                           # B row-major
           lambda: Q.gemm_fp8(q, q[:, :32].t(), x[:, :4], s, s),               # K
           lambda: Q.gemm_fp8(x, q.t(), x[:, :4], s, s),                       # A not e4m3
           lambda: Q.gemm_fp8(q, q.t(), x[:, :8], s, s),                       # C's shape
           lambda: Q.gemv_w4(x, q.view(torch.uint8)[:, :32], x[:, :3], x[:, :4]),          # group
           lambda: Q.gemv_w4(x, q.view(torch.uint8)[:, :31], x[:, :1], x[:, :4]),          # W's width
           lambda: Q.gemv_w4(x.float(), q.view(torch.uint8)[:, :32], x[:, :1], x[:, :4]),  # fp32 x
           lambda: Q.gemv_w4(x, q.view(torch.uint8)[:, :32], x[:, :1].to(F16), x[:, :4])]  # scales' type
    for i, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
            pytest.fail(f"case {i} was accepted")
    with pytest.raises(G.GemmError, match="ALIGN"):
        Q.gemm_fp8(torch.zeros(4, 72, dtype=E4M3, device="cuda")[:, :64], q.t(), torch.zeros(4, 8, dtype=BF16,
                   device="cuda")[:, :4], s, s)
    with pytest.raises(G.GemmError, match="ALIGN"):
        Q.gemv_w4(torch.zeros(4, 65, dtype=BF16, device="cuda")[:, 1:], q.view(torch.uint8)[:, :32], x[:, :1],
                  torch.zeros(4, 4, dtype=BF16, device="cuda"))
