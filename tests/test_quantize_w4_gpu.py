"""quantize_w4 against its formula, equal in every value: the scale's one fp32
division and rounding, the quotients' fp32 divisions and nearest-even roundings
are all defined."""
import numpy as np
import pytest
import torch

from stage_software_pipelining_gb300 import build as gemm_build
from stage_software_pipelining_gb300 import quant as Q

pytestmark = pytest.mark.gpu
F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def lib(gpu):
    gemm_build.build()
    return Q.load_library()


def formula(w, group, zeros, stype):
    """(values N x K, scales, zero points or None) of fp32 weights."""
    g = w.float().numpy().reshape(w.shape[0], -1, group)
    lo, hi = np.minimum(g.min(axis=2), 0), np.maximum(g.max(axis=2), 0)
    f = np.float32
    with np.errstate(over="ignore"):
        range_ = hi - lo
        scale = np.where(np.isfinite(range_), range_ / f(15), hi / f(15) - lo / f(15)) if zeros \
            else np.maximum(hi, -lo) / f(7)
    scale = torch.from_numpy(np.minimum(scale, f(torch.finfo(stype).max))).to(stype)
    s = scale.float().numpy()
    with np.errstate(divide="ignore", invalid="ignore"):
        steps = np.where(s[:, :, None] > 0, np.rint(g / s[:, :, None]), f(0))
        z = np.minimum(np.where(s > 0, np.rint(-lo / s), f(0)), 15) if zeros else np.full_like(s, 8)
    q = np.clip(steps + z[:, :, None], 0, 15)
    return q.reshape(w.shape).astype(np.uint8), scale, z.astype(np.uint8) if zeros else None


def check(w, group, zeros, stype):
    N, K = w.shape
    W = torch.empty(N, K // 2, dtype=torch.uint8, device="cuda")
    s = torch.empty(N, K // group, dtype=stype, device="cuda")
    z = torch.empty(N, K // group, dtype=torch.uint8, device="cuda") if zeros else None
    Q.quantize_w4(w.cuda(), W, s, z)
    q, scale, zp = formula(w, group, zeros, stype)
    assert torch.equal(s.cpu(), scale)
    if zeros:
        assert np.array_equal(z.cpu().numpy(), zp)
    b = W.cpu().numpy()
    assert np.array_equal(np.stack((b & 15, b >> 4), axis=2).reshape(N, K), q)
    return q, scale


@pytest.mark.parametrize("stype", [F16, BF16])
@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("zeros", [False, True])
def test_random_weights(zeros, group, dtype, stype):
    g = torch.Generator().manual_seed(1)
    w = (torch.randn(37, 640, generator=g) * 0.03 + (0.02 if zeros else 0.0)).to(dtype)
    w[5] = 0
    w[6] = w[6].abs()
    w[7] = -w[7].abs()
    check(w, group, zeros, stype)


@pytest.mark.parametrize("stype", [F16, BF16])
@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("zeros", [False, True])
def test_weights_half_way_between_two_values(zeros, dtype, stype):
    """Groups whose scale is an odd number s / 64 and whose weights are odd
    multiples of half of it (of which bf16 weights hold those up to 255 / 128)."""
    group, odd = 32, torch.arange(1, 256, 2).float()
    top = 15 if zeros else 7
    k = torch.arange(group) % (top - 1 if zeros else 2 * top - 1) - (0 if zeros else top - 1)
    w = odd[:, None] * (k + 0.5) / 64
    w[:, 0] = odd * top / 64
    if zeros:
        w[:, 1] = 0
    held = (w.to(dtype).float() == w).all(dim=1)
    w = w[held].to(dtype)
    assert len(w) >= 5
    _, scale = check(w, group, zeros, stype)
    assert torch.equal(scale.float()[:, 0], (odd / 64)[held])


@pytest.mark.parametrize("stype", [F16, BF16])
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("size", [3e38, 1e6, 4.6e5, 1e-6, 1e-30, 1e-38, 2.0 ** -140])
def test_weights_at_the_ends_of_the_range(size, zeros, stype):
    """Scales stay finite: weights past the largest one's reach are limited."""
    w = (torch.rand(9, 256, generator=torch.Generator().manual_seed(2)) * 2 - 1) * size
    q, scale = check(w, 64, zeros, stype)
    assert torch.isfinite(scale).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("offset", [0, 1, 4])
@pytest.mark.parametrize("pitch", [0, 1, 8])
def test_rows_on_any_address(pitch, offset, dtype):
    """Rows of weights and of packed values that do not start on 16- and 4-byte
    boundaries, and nothing written beside them."""
    N, K, group = 7, 192, 64
    w = torch.randn(N, K, generator=torch.Generator().manual_seed(3)).to(dtype)
    buf = torch.full((N * (K + pitch) + offset,), float("nan"), dtype=dtype, device="cuda")
    dw = buf[offset:].view(N, K + pitch)[:, :K]
    dw.copy_(w)
    packed = torch.full((N * (K // 2 + pitch) + offset + 3,), 0xA5, dtype=torch.uint8, device="cuda")
    W = packed[offset:offset + N * (K // 2 + pitch)].view(N, K // 2 + pitch)[:, :K // 2]
    s = torch.empty(N, K // group, dtype=BF16, device="cuda")
    Q.quantize_w4(dw, W, s)
    q, scale, _ = formula(w, group, False, BF16)
    b = W.cpu().numpy()
    assert np.array_equal(np.stack((b & 15, b >> 4), axis=2).reshape(N, K), q) and torch.equal(s.cpu(), scale)
    outside = torch.ones_like(packed, dtype=torch.bool)
    outside[offset:offset + N * (K // 2 + pitch)].view(N, K // 2 + pitch)[:, :K // 2] = False
    assert (packed[outside] == 0xA5).all()
