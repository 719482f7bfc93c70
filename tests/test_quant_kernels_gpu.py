"""The products on kernel instances that their sizes choose, with the choice
asserted (so that a change of the choice cannot move a test elsewhere unseen).

Bounds as derived in quant_reference.py.  gemm_fp8 with more K than there: a
tensor-core step of 32 products is off by 2^-22 of the magnitudes at most, so
K / 32 steps by K / 32 * 2^-22 (a cut K's partials, eight at most, are part of
the steps that are saved)."""
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


def fp8_rows(v):
    """Quantised rows on the device, NaN beyond them, and their scales."""
    s = (v.abs().amax(dim=1) / 448).clamp_min(R.SCALE_MIN)
    q = (v / s[:, None]).clamp(-448, 448).to(E4M3)
    rows, cols = q.shape
    buf = torch.full((rows, (cols + 15) // 16 * 16 + 16), 0x7F, dtype=torch.uint8, device="cuda").view(E4M3)
    buf[:, :cols].copy_(q)
    return buf[:, :cols], s.cuda()


def fp8_bound(K, absb):
    return max(R.SUM_REL, K / 32 * 2.0 ** -22) * absb


def fp8_case(M, N, K, dtype, seed=1, scale_offset=0):
    A, sa = fp8_rows(rand(seed, M, K))
    W, sb = fp8_rows(0.05 * rand(seed + 1, N, K))
    if scale_offset:
        sb = torch.cat((torch.full((scale_offset,), float("nan"), device="cuda"), sb))[scale_offset:]
        assert sb.data_ptr() % 16 == 4 * scale_offset
    C = GuardedC(M, N, dtype)
    Q.gemm_fp8(A, W.t(), C.view, sa, sb)
    C.check()
    ref, absb = R.gemm_fp8(A, W.t(), sa, sb)
    R.check_rounded(C.view, ref, 2.0 ** -22, fp8_bound(K, absb), f"{M}x{N}x{K}")
    return C.view


# On the pair kernel: (M, N, K, stages).  More tiles than pairs, two groups of tile
# rows (of which the second walks backwards); tiles fewer than pairs; K on both
# sides of 2048; columns that are not whole 16-byte units.
PAIR = [(4500, 2600, 2100, 6), (4500, 2603, 2100, 6), (4500, 1100, 300, 5), (4500, 1103, 300, 5),
        (1300, 2600, 2048, 5), (1300, 2600, 2049, 6), (1300, 2603, 2100, 6), (1300, 2603, 300, 5),
        (2304, 2310, 2304, 6)]
# On the few-row kernel: (M, N, K, tile_rows, split): the widest tiles, whole and
# with K cut (partials over the ring), and narrower ones with one CTA an SM.
FEW = [(256, 4096, 14336, 256, 4), (250, 5003, 4096, 256, 3), (2100, 4101, 500, 256, 1),
       (200, 4096, 4096, 128, 2), (100, 3000, 8192, 128, 5), (90, 19000, 1000, 128, 1),
       (60, 3001, 8192, 64, 5), (70, 1500, 8192, 32, 4)]


def assert_pair(M, N, K, stages, dtype):
    p = Q.gemm_fp8_plan(M, N, K, dtype)
    assert p["kernel"] == "fp8_pair" and p["stages"] == stages, p
    return p


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("M,N,K,stages", PAIR)
def test_gemm_fp8_pair(M, N, K, stages, dtype):
    p = assert_pair(M, N, K, stages, dtype)
    tiles = -(-M // 256) * -(-N // 256)
    assert (tiles > p["grid"] // 2) == (M == 4500 or M == 2304)
    fp8_case(M, N, K, dtype)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("M,N,K,rows,split", FEW)
def test_gemm_fp8_few(M, N, K, rows, split, dtype):
    p = Q.gemm_fp8_plan(M, N, K, dtype)
    assert p["kernel"] == "fp8_few" and p["tile_rows"] == rows, p
    assert (p["split"] > 1) == (split > 1), p
    fp8_case(M, N, K, dtype)


@pytest.mark.parametrize("M,N,K", [(1300, 2600, 300), (1300, 2603, 2100), (40, 1000, 640), (200, 4096, 4096)])
@pytest.mark.parametrize("offset", [1, 2, 3])
def test_gemm_fp8_column_scales_on_any_address(M, N, K, offset):
    fp8_case(M, N, K, BF16, scale_offset=offset)


@pytest.mark.parametrize("M,N,K,stages", [(1300, 2600, 1024, 5), (4500, 2600, 2100, 6)])
def test_gemm_fp8_pair_is_repeatable(M, N, K, stages):
    assert_pair(M, N, K, stages, BF16)
    a = fp8_case(M, N, K, BF16, seed=5).clone()
    assert torch.equal(a, fp8_case(M, N, K, BF16, seed=5))


@pytest.mark.parametrize("M,N,K,stages", [(1300, 2603, 300, 5), (4500, 2600, 2100, 6)])
def test_gemm_fp8_pair_nan_stays_in_its_row_and_column(M, N, K, stages):
    assert_pair(M, N, K, stages, F16)
    A, sa = fp8_rows(rand(7, M, K))
    W, sb = fp8_rows(rand(8, N, K))
    A[M - 1, K - 1] = float("nan")
    W[N // 2, 0] = float("nan")
    C = torch.zeros(M, (N + 7) // 8 * 8, dtype=F16, device="cuda")[:, :N]
    Q.gemm_fp8(A, W.t(), C, sa, sb)
    nan = torch.isnan(C).cpu()
    expect = torch.zeros_like(nan)
    expect[M - 1] = True
    expect[:, N // 2] = True
    assert torch.equal(nan, expect)


@pytest.mark.parametrize("M,N,K,stages", [(1300, 2600, 256, 5), (2304, 2312, 2304, 6)])
def test_gemm_fp8_pair_overflow_and_scales(M, N, K, stages):
    """fp16 results past its range are infinities; scales may be zero or negative."""
    assert_pair(M, N, K, stages, F16)
    A, W = torch.ones(M, K, device="cuda").to(E4M3), torch.ones(N, K, device="cuda").to(E4M3)
    sa = torch.linspace(0, 400, M, device="cuda")
    sb = torch.where(torch.arange(N, device="cuda") % 2 == 0, 1.0, -1.0)
    C = torch.empty(M, N, dtype=F16, device="cuda")
    Q.gemm_fp8(A, W.t(), C, sa, sb)
    expect = (K * sa[:, None] * sb[None, :]).to(F16)
    assert torch.equal(C, expect) and torch.isinf(C).any() and not C[0].any()


@pytest.mark.parametrize("M,N,K,stages", [(1300, 2600, 1024, 5), (4500, 2600, 2100, 6)])
def test_gemm_fp8_pair_stuck_pipeline_is_reported(M, N, K, stages):
    """A stage whose copy never comes ends in GEMM_ERR_TIMEOUT, and the next call is right."""
    assert_pair(M, N, K, stages, BF16)
    A, sa = fp8_rows(rand(9, M, K))
    W, sb = fp8_rows(rand(10, N, K))
    C = torch.empty(M, N, dtype=BF16, device="cuda")
    try:
        G.debug_set(wait_limit_ns=50_000_000, withhold_arrive=0)
        with pytest.raises(G.GemmError, match="TIMEOUT"):
            Q.gemm_fp8(A, W.t(), C, sa, sb, checked=True)
    finally:
        G.debug_set()
    Q.gemm_fp8(A, W.t(), C, sa, sb, checked=True)
    ref, absb = R.gemm_fp8(A, W.t(), sa, sb)
    R.check_rounded(C, ref, 2.0 ** -22, fp8_bound(K, absb), "after a timeout")


# The tcgen05 kernel of gemv_w4 with scales and zero points as a checkpoint holds
# them: rows of a multiple of eight, on their boundaries, read in vectors.  Group
# counts that end inside a run of eight, and cuts of K that begin inside one.
W4_TC = [(20, 13001, 1024, 32), (20, 13001, 1024, 64), (20, 13001, 2048, 128), (20, 13001, 1152, 128),
         (33, 9000, 2304, 128), (32, 4100, 8192, 64), (20, 9000, 4128, 32)]


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("M,N,K,group", W4_TC)
def test_gemv_w4_tc_rows_of_groups_on_their_boundaries(M, N, K, group, zeros, dtype):
    assert Q.gemv_w4_plan(M, N, K, group, zeros, dtype)["kernel"] == "w4_tc"
    g = torch.Generator().manual_seed(11)
    groups, pitch = K // group, (K // group + 7) // 8 * 8
    x = torch.randn(M, K, generator=g).to(dtype)
    W = torch.randint(0, 256, (N, K // 2), generator=g, dtype=torch.uint8)
    s = (torch.rand(N, groups, generator=g) * 0.02 - 0.005).to(dtype)
    z = torch.randint(0, 16, (N, groups), generator=g, dtype=torch.uint8) if zeros else None
    ds = torch.full((N, pitch), float("nan"), dtype=dtype, device="cuda")[:, :groups]
    ds.copy_(s)
    dz = None
    if zeros:
        dz = torch.full((N, pitch), 99, dtype=torch.uint8, device="cuda")[:, :groups]
        dz.copy_(z)
        assert dz.data_ptr() % 8 == 0
    assert ds.data_ptr() % 16 == 0
    C = GuardedC(M, N, dtype)
    Q.gemv_w4(x.cuda(), W.cuda(), ds, C.view, zeros=dz)
    C.check()
    ref, absb = R.gemv_w4(x, W, s, z, group)
    R.check_rounded(C.view, ref, 2.0 ** -22, R.W4_REL * absb, f"{M}x{N}x{K} group {group}")


# Longer rows than a block's shared memory holds: the mean's terms are added 1024
# threads at a time, n / 1024 in a row by one, fewer than NORM_REL's derivation allows.
@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("rows,cols,extra,offset", [(3, 45001, 0, 0), (2, 100003, 5, 1), (200, 46000, 8, 0)])
def test_norm_of_very_long_rows(rows, cols, extra, offset, dtype):
    def wide(t):
        buf = torch.full((t.shape[0] * (cols + extra) + offset,), float("nan"), device="cuda").to(t.dtype)
        v = buf[offset:].view(t.shape[0], cols + extra)[:, :cols]
        v.copy_(t)
        return v
    x, r, w = rand(12, rows, cols).to(dtype), (3 * rand(13, rows, cols)).to(dtype), (1 + 0.2 * rand(14, cols)).to(dtype)
    ro, y = GuardedC(rows, cols, dtype), GuardedC(rows, cols, dtype)
    q, scale = Q.empty_rows(rows, cols, E4M3), torch.empty(rows, device="cuda")
    dx, dr = wide(x), wide(r)
    Q.add_rmsnorm(dx, w.cuda(), dr, eps=1e-5, residual_out=ro.view, y=y.view, q=q, scale=scale)
    h, ref = R.norm(x, w, r, 1e-5)
    ro.check()
    y.check()
    R.check_rounded(ro.view, h, 2.0 ** -24, 0.0, "residual_out")
    R.check_rounded(y.view, ref, R.NORM_REL, 0.0, "y")
    R.check_q(q, scale, ref, "q")
    Q.add_rmsnorm(dx, w.cuda(), dr, eps=1e-5, residual_out=dr, y=dx)        # both in place
    R.check_rounded(dr, h, 2.0 ** -24, 0.0, "residual_out in place")
    R.check_rounded(dx, ref, R.NORM_REL, 0.0, "y in place")
    Q.quantize_fp8(y.view, q, scale)
    R.check_q(q, scale, R.f64(y.view), "q of y", rel=1e-6)
