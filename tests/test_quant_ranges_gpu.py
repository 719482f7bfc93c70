"""The row-wise operators at the ends of their types' ranges, on each of their
kernels: a warp a row (256 columns), a block a row (4096), rows by way of shared
memory (20000 columns, or many rows of odd width) and longer rows (46000)."""
import numpy as np
import pytest
import torch

import quant_reference as R
from stage_software_pipelining_gb300 import build as gemm_build
from stage_software_pipelining_gb300 import quant as Q

pytestmark = pytest.mark.gpu
F32, F16, BF16, E4M3 = torch.float32, torch.float16, torch.bfloat16, torch.float8_e4m3fn
COLS = [40, 256, 4096, 20000, 46000]


@pytest.fixture(scope="module", autouse=True)
def lib(gpu):
    gemm_build.build()
    return Q.load_library()


def rand(seed, *shape):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed))


def outputs(rows, cols):
    return torch.empty(rows, cols, dtype=E4M3, device="cuda"), torch.empty(rows, device="cuda")


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("cols", COLS)
@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan")])
def test_quantize_fp8_values_that_are_not_finite(value, cols, dtype):
    """They make their own row's scale and values NaN and leave the others alone."""
    x = rand(1, 4, cols).to(dtype)
    x[1, cols // 3] = value
    x[2, cols - 1] = value
    q, scale = outputs(4, cols)
    Q.quantize_fp8(x.cuda(), q, scale)
    for i in (1, 2):
        assert torch.isnan(scale[i]) and torch.isnan(q[i].float()).all()
    ok = [0, 3]
    R.check_q(q.float().cpu()[ok], scale.cpu()[ok], R.f64(x[ok]), "q", rel=1e-6)


@pytest.mark.parametrize("cols", COLS)
def test_norm_of_an_infinite_weight(cols):
    """y is what the formula gives; a row of it that holds an infinity has no scale."""
    x, w = rand(2, 3, cols), 1 + 0.1 * rand(3, cols)
    w[cols // 2] = float("inf")
    y = torch.empty(3, cols, device="cuda")
    q, scale = outputs(3, cols)
    Q.add_rmsnorm(x.cuda(), w.cuda(), y=y, q=q, scale=scale)
    assert torch.isnan(scale).all() and torch.isnan(q.float()).all()
    keep = torch.arange(cols) != cols // 2
    R.check_rounded(y[:, keep], R.norm(x, torch.where(keep, w, torch.ones(())), None, 1e-6)[1][:, keep.numpy()],
                    R.NORM_REL, 0.0, "y")
    assert torch.isinf(y[:, cols // 2]).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rows,cols", [(2000, 1503), (2000, 2999)])
def test_quantize_fp8_infinities_in_many_rows_of_odd_width(rows, cols, dtype):
    x = rand(4, rows, cols).to(dtype)
    x[7::50, cols - 2] = float("inf")
    q, scale = outputs(rows, cols)
    Q.quantize_fp8(x.cuda(), q, scale)
    bad = torch.isinf(x).any(dim=1)
    assert torch.equal(torch.isnan(scale).cpu(), bad)
    assert torch.equal(torch.isnan(q.float()).any(dim=1).cpu(), bad)
    assert torch.isnan(q.float()).all(dim=1).cpu()[bad].all()
    R.check_q(q.float().cpu()[~bad], scale.cpu()[~bad], R.f64(x[~bad]), "q", rel=1e-6)
    assert np.isfinite(R.f64(scale)[~bad.numpy()]).all()
