"""The training operators at their limits: the derivatives' tails, the longest sums,
and waits that run out."""
import math
import time

import numpy as np
import pytest
import torch

import linear_reference as R
from stage_software_pipelining_gb300 import build as gemm_build
from stage_software_pipelining_gb300 import gemm as G
from stage_software_pipelining_gb300 import linear as L
from stage_software_pipelining_gb300 import quant as Q

pytestmark = pytest.mark.gpu
F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def lib(gpu):
    gemm_build.build()
    return L.load_library()


# ---------------------------------------------------------------- gelu' below zero
# gelu'(z) = Phi(z) + z phi(z) of its own size, -9 <= z <= -4.  phi's exponent z^2 / 2 log2(e)
# is below 58.5 and rounded twice (its factor and itself): 58.5 ln 2 2 2^-24 = 4.9e-6 of phi
# and of the tail alike.  exp2 itself, z times 1 / sqrt(2 pi) and the sum: 2^-22 + 3 2^-24 =
# 4.2e-7.  The tail is at most 0.06 of the other term; its fit (9e-7), reciprocal and
# polynomial (16 2^-24) add 0.06 * 1.9e-6 = 1.2e-7.  |Phi| + |z phi| is at most 1.13 |gelu'|:
# 1.13 * 5.5e-6 = 6.2e-6 < 2^-17.
TAIL_REL = 2.0 ** -17


def tail(dtype):
    """Every value of dtype from -9 to -4, and gelu' there in 64 bits."""
    first, last = (torch.tensor(v, dtype=dtype).view(torch.int16).item() for v in (-4.0, -9.0))
    z = torch.arange(first, last + 1, dtype=torch.int16).view(dtype)
    assert z[0] == -4 and z[-1] == -9
    v = z.double()
    return z, 0.5 * torch.special.erfc(v * -math.sqrt(0.5)) + v * torch.exp(-0.5 * v * v) / math.sqrt(2 * math.pi)


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_gelu_derivative_keeps_its_tail(dtype):
    z, ref = tail(dtype)
    one = torch.ones(1, z.numel(), dtype=dtype, device="cuda")
    db = torch.empty(z.numel(), device="cuda")
    L.act_grad(one, pre=z[None].cuda(), act="gelu", dbias=db)
    off = ((db.cpu().double() - ref) / ref).abs()
    assert off.max() <= TAIL_REL, (float(off.max()), float(z[off.argmax()]))


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("M", [1, 600])
def test_gelu_derivative_keeps_its_tail_in_16_bits(M, dtype):
    """Times 2^10, by act_grad and by linear_dx on either kernel."""
    z, ref = tail(dtype)
    n = z.numel()
    up, pre = Q.empty_rows(M, n, dtype), Q.empty_rows(M, n, dtype)
    up.fill_(1024.0)
    pre.copy_(z.expand(M, n))
    ref = np.broadcast_to(1024.0 * ref.numpy(), (M, n))
    dz, dx = Q.empty_rows(M, n, dtype), Q.empty_rows(M, n, dtype)
    L.act_grad(up, dz, pre=pre, act="gelu")
    R.check_rounded(dz, ref, TAIL_REL, 0.0, "act_grad")
    W = Q.empty_rows(64, n, dtype)
    W.zero_()
    L.linear_dx(torch.zeros(M, 64, dtype=dtype, device="cuda"), W, dx, residual=up, act="gelu", pre=pre, checked=True)
    R.check_rounded(dx, ref, TAIL_REL, 0.0, "linear_dx")


# ---------------------------------------------------------------- the longest fp32 weight gradients
def zeros_and_ones(seed, rows, cols, dtype):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(0, 2, (rows, cols), generator=g, device="cuda", dtype=torch.int8).to(dtype)


@pytest.mark.parametrize("M,N,K,dtype", [(262145, 128, 128, F16), (300001, 40, 264, BF16), (1048577, 24, 8, F16),
                                         (12000001, 24, 40, BF16), (16000000, 8, 16, F16)])
def test_linear_dw_of_many_rows(M, N, K, dtype):
    """Sums of zeros and ones below 2^24 are exact in fp32, whatever their order."""
    dz, x = zeros_and_ones(1, M, N, dtype), zeros_and_ones(2, M, K, dtype)
    dw = torch.full((N, K), 3.0, device="cuda")
    L.linear_dw(dz, x, dw, addend=dw, checked=True)
    ref = torch.full((N, K), 3.0, dtype=torch.float64, device="cuda")
    for at in range(0, M, 1 << 20):
        ref += dz[at:at + (1 << 20)].double().t() @ x[at:at + (1 << 20)].double()
    assert torch.equal(dw.double(), ref)


@pytest.mark.parametrize("M,N,K,kernel,rows", [(17000, 40, 24, "few", 64), (40000, 300, 72, "few", None),
                                               (9000, 1400, 300, "few", None), (600, 40, 40, "few", 64), (32768, 1024, 1024, "few", 256),
                                               (262144, 128, 128, "few", 64), (300000, 128, 128, "few", 64),
                                               (8192, 2304, 2048, "pair", 256), (5000, 2304, 2048, "pair", 256)])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_linear_dw_sums_512_rows_in_an_accumulator(M, N, K, kernel, rows, dtype):
    """Of equal signs.  An accumulator of 512 rows takes 32 steps of 16 products, each of which
    may drop 2^-22 of the sum so far (linear_reference.py; sixteen products and the sum, cut off
    two bits below fp32's last: 17 2^-26): in an evenly growing sum (1 + ... + 32) / 32 2^-22 =
    4e-6 of the whole.  Accumulations join rounded to nearest, 2^-24 of the sum so far each,
    M/512 of them and of 8 CTAs: (M / 1024 + 8) 2^-24 of the whole at most.  Two accumulations of
    1024 rows, of 6144 or more on the pair kernel, drop (1 + ... + 64) / 64 2^-22 = 7.8e-6 of
    their share of M."""
    plan = L.linear_plan("dw", M, N, K, F32)
    assert plan["kernel"] == kernel and plan["tile_rows"] == (rows or plan["tile_rows"])
    g = torch.Generator(device="cuda").manual_seed(9)

    def positive(cols):
        t = Q.empty_rows(M, cols, dtype)
        t.copy_(1.0 + torch.rand(M, cols, generator=g, device="cuda"))
        return t
    dz, x, dw = positive(N), positive(K), Q.empty_rows(N, K, F32)
    L.linear_dw(dz, x, dw, checked=True)
    ref = torch.zeros(N, K, dtype=torch.float64, device="cuda")
    for at in range(0, M, 1 << 16):
        ref += dz[at:at + (1 << 16)].double().t() @ x[at:at + (1 << 16)].double()
    off = (dw.double() - ref) / ref
    longer = 2048 / M if kernel == "pair" and M >= 6144 else 0.0
    assert off.abs().max() <= 4e-6 * (1 - longer) + 7.8e-6 * longer + (M / 1024 + 8) * 2.0 ** -24


# M, N, K, tile rows, CTAs of a cut: more than 512 rows a CTA, uncut, cut and cut unevenly
LONG = [(633, 1836, 33, 64, 1), (1639, 2600, 37, 64, 3), (4660, 35, 36, 64, 8), (674, 4946, 152, 128, 1),
        (1845, 68, 5159, 128, 3), (4614, 67, 1162, 128, 8), (658, 4009, 1040, 256, 1), (2191, 195, 5131, 256, 3),
        (8067, 134, 1565, 256, 8)]


def rand(seed, rows, cols, dtype):
    t = Q.empty_rows(rows, cols, dtype)
    t.copy_(torch.randn(rows, cols, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda"))
    return t


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("M,N,K,rows,cut", LONG)
def test_long_fp32_sums_on_every_instance(M, N, K, rows, cut, dtype):
    plan = L.linear_plan("dw", M, N, K, F32)
    assert (plan["kernel"], plan["tile_rows"], plan["split"]) == ("few", rows, cut) and -(-M // 64) > 8 * cut
    dz, x, c = rand(1, M, N, dtype), rand(2, M, K, dtype), rand(3, N, K, F32)
    s = dz.double().t() @ x.double()
    err = R.sum_rel(M, 512) * (dz.double().abs().t() @ x.double().abs())
    wide = torch.full((N, (K + 3) // 4 * 4 + 8), 7.0, device="cuda")
    dw = wide[:, :K]
    L.linear_dw(dz, x, dw, checked=True)
    assert ((dw.double() - s).abs() <= err + 2.0 ** -23 * s.abs()).all() and (wide[:, K:] == 7.0).all()
    sums = dw.clone()
    L.linear_dw(dz, x, dw)
    assert torch.equal(dw, sums)
    dw.copy_(c)
    L.linear_dw(dz, x, dw, addend=dw, checked=True)      # accumulated in place
    assert torch.equal(dw, c + sums) and (wide[:, K:] == 7.0).all()


def test_long_fp32_sums_in_two_graphs_at_once():
    sets = []
    for i, (M, N, K) in enumerate([(40000, 72, 304), (32768, 1024, 1024)]):
        dz, x, dw = rand(10 + i, M, N, F16), rand(20 + i, M, K, F16), Q.empty_rows(N, K, F32)
        L.linear_dw(dz, x, dw)
        torch.cuda.synchronize()
        expect, graph = dw.clone(), torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            for _ in range(4):
                L.linear_dw(dz, x, dw)
        dw.zero_()
        sets.append((graph, torch.cuda.Stream(), dw, expect, (dz, x)))
    torch.cuda.synchronize()
    for _ in range(3):
        for graph, stream, *_ in sets:
            with torch.cuda.stream(stream):
                graph.replay()
    torch.cuda.synchronize()
    for _, _, dw, expect, _ in sets:
        assert torch.equal(dw, expect)


@pytest.mark.parametrize("M", [11863232, 11863233, 100000000, 2 ** 31 - 4097])
@pytest.mark.parametrize("out", [F32, BF16])
def test_any_number_of_rows_has_a_plan(M, out):
    """The header's limit is the only one: sizes up to 2^31 - 4097."""
    assert L.linear_plan("dw", M, 64, 64, out)["grid"] > 0
    with pytest.raises(G.GemmError) as e:
        L.linear_plan("dw", 2 ** 31 - 4096, 64, 64, out)
    assert e.value.status == G.GEMM_ERR_UNSUPPORTED


# ---------------------------------------------------------------- waits that run out
def late(rows, cols, step, limit_ms=50, steps=5, batch=()):
    """orthogonalize with the copy or commit number `step` of its first CTA left out:
    the status, and how long the call took."""
    g = torch.randn(*batch, rows, cols, generator=torch.Generator().manual_seed(6)).cuda()
    out = torch.empty(*batch, rows, cols, dtype=BF16, device="cuda")
    ws = torch.empty(L.orthogonalize_workspace(g), dtype=torch.uint8, device="cuda")
    L.orthogonalize(g, out, ws, steps=steps, checked=True)      # the kernels' one-time settings
    right = out.clone()
    try:
        G.debug_set(wait_limit_ns=limit_ms * 1000000, withhold_arrive=step)
        began = time.perf_counter()
        with pytest.raises(G.GemmError) as e:
            L.orthogonalize(g, out, ws, steps=steps, checked=True)
        took = time.perf_counter() - began
    finally:
        G.debug_set()
    L.orthogonalize(g, out, ws, steps=steps, checked=True)
    assert torch.equal(out, right)      # the next call is as the one before
    return e.value.status, took


@pytest.mark.parametrize("rows,cols,batch", [(304, 400, ()), (400, 304, (2,))])
@pytest.mark.parametrize("step", [0, 3])
def test_products_of_orthogonalize_say_that_they_ran_out(rows, cols, batch, step):
    """Withheld: a stage of every product."""
    assert late(rows, cols, step, batch=batch)[0] == G.GEMM_ERR_TIMEOUT


@pytest.mark.parametrize("M,N,K,rows", [(262144, 128, 128, 64), (8053, 296, 3016, 128), (32768, 1024, 1024, 256)])
@pytest.mark.parametrize("step", [0, 7, 8, 20])
def test_long_fp32_sums_say_that_they_ran_out(M, N, K, rows, step):
    """A stage withheld in the first, at an end, and in a later accumulation."""
    assert L.linear_plan("dw", M, N, K, F32)["tile_rows"] == rows
    dz, x = zeros_and_ones(1, M, N, F16), zeros_and_ones(2, M, K, F16)
    dw = torch.empty(N, K, device="cuda")
    try:
        G.debug_set(wait_limit_ns=50_000_000, withhold_arrive=step)
        began = time.perf_counter()
        with pytest.raises(G.GemmError) as e:
            L.linear_dw(dz, x, dw, checked=True)
        assert e.value.status == G.GEMM_ERR_TIMEOUT and time.perf_counter() - began < 0.5
    finally:
        G.debug_set()
    L.linear_dw(dz, x, dw, checked=True)
    assert torch.equal(dw, dz.float().t() @ x.float())      # whole numbers below 2^24


@pytest.mark.parametrize("rows,cols,batch", [(104, 304, ()), (304, 64, (3,)), (120, 2048, ()), (2560, 128, ()),
                                             (128, 1024, (2,))])
@pytest.mark.parametrize("step", [0, 1, 2, 7, 149])
def test_orthogonalize_in_one_launch_says_that_it_ran_out(rows, cols, batch, step):
    """Withheld: the end of one product of 150, in one CTA and in clusters.  The call ends
    within some limits, not one for each of the waits that are left."""
    status, took = late(rows, cols, step, steps=50, batch=batch)
    assert status == G.GEMM_ERR_TIMEOUT and took < 0.5
