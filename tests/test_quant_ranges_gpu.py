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


def check_norm(x, r, w, eps, what, rows=None):
    """All outputs of a call, of all or some of its rows, against the 64-bit form."""
    n, cols = x.shape
    ro, y = (torch.empty(n, cols, dtype=x.dtype, device="cuda") for _ in range(2))
    q, scale = outputs(n, cols)
    Q.add_rmsnorm(x.cuda(), w.cuda(), r.cuda() if r is not None else None, eps=eps, residual_out=ro, y=y, q=q,
                  scale=scale)
    eps = float(np.float32(eps))
    rows = list(range(n)) if rows is None else rows
    h, ref = R.norm(x[rows], w, r[rows] if r is not None else None, eps)
    R.check_rounded(ro[rows], h, 2.0 ** -24, 0.0, f"{what}: residual_out")
    R.check_rounded(y[rows], ref, R.NORM_REL, 0.0, f"{what}: y")
    R.check_q(q[rows].float(), scale[rows], ref, f"{what}: q")
    alone = torch.empty_like(y)  # without the 8-bit outputs
    Q.add_rmsnorm(x.cuda(), w.cuda(), r.cuda() if r is not None else None, eps=eps, y=alone)
    R.check_rounded(alone[rows], ref, R.NORM_REL, 0.0, f"{what}: y alone")
    return ro, y, q, scale


# The squares of 3e17 sum to infinity only in long rows; 2^-70 and less lose bits or vanish.
SIZES = [3e17, 2e19, 1e30, 4e37, 2.0 ** -50, 2.0 ** -65, 2.0 ** -73, 1e-25, 1e-38, 2.0 ** -130]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("cols", COLS)
@pytest.mark.parametrize("with_residual", [False, True])
@pytest.mark.parametrize("eps", [0.0, 1e-36, 1e-6])
def test_norm_rows_whose_squares_leave_the_range(eps, with_residual, cols, dtype):
    """Large and small rows side by side with ordinary ones."""
    size = torch.tensor([1.0] + SIZES + [0.5])[:, None]
    # 7-bit values, which fp32 holds down to 2^-142 and bf16 down to 2^-126
    x = (torch.randint(64, 128, (len(size), cols), generator=torch.Generator().manual_seed(5)) / 64.0 * size).to(dtype)
    x[:, ::3] *= -1
    r = (x.float() * 0.25).flip(1).to(dtype) if with_residual else None
    w = (1 + 0.1 * rand(6, cols)).to(dtype)
    check_norm(x, r, w, eps, f"{cols} columns")


@pytest.mark.parametrize("cols", COLS)
def test_norm_products_with_the_weight_that_leave_the_range(cols):
    """h w overflows or vanishes where y = h w / rms is an ordinary number."""
    x = rand(7, 3, cols) * torch.tensor([1e15, 1.0, 3e-9])[:, None]
    check_norm(x, None, 1e25 * (1 + rand(8, cols).abs()), 0.0, "large weights")
    check_norm(x, None, 1e-33 * (1 + rand(9, cols).abs()), 0.0, "small weights")


@pytest.mark.parametrize("cols", COLS)
def test_norm_rows_of_zeros(cols):
    x = rand(10, 3, cols)
    x[1] = 0
    w = torch.ones(cols)
    for eps in (1e-36, 1e-6):
        _, y, q, scale = check_norm(x, None, w, eps, f"eps {eps}")
        assert not y[1].any() and not q[1].float().any() and scale[1].item() == R.SCALE_MIN
    _, y, q, scale = check_norm(x, None, w, 0.0, "eps 0", rows=[0, 2])
    assert torch.isnan(y[1]).all() and torch.isnan(q[1].float()).all() and torch.isnan(scale[1])


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rows,cols", [(2000, 1503), (2000, 2999)])
def test_norm_ranges_in_many_rows_of_odd_width(rows, cols, dtype):
    size = torch.tensor(SIZES)[torch.arange(rows) % len(SIZES)][:, None]
    x = (torch.randint(64, 128, (rows, cols), generator=torch.Generator().manual_seed(11)) / 64.0 * size).to(dtype)
    check_norm(x, None, (1 + 0.1 * rand(12, cols)).to(dtype), 0.0, "many rows")


@pytest.mark.parametrize("cols", COLS)
def test_norm_ranges_in_place(cols):
    """residual_out over the residual and y over x, also where h is read twice."""
    x = rand(13, 2, cols) * torch.tensor([1e25, 1e-25])[:, None]
    r = rand(14, 2, cols) * torch.tensor([1e25, 1e-25])[:, None]
    w = 1 + 0.1 * rand(15, cols)
    dx, dr = x.cuda(), r.cuda()
    Q.add_rmsnorm(dx, w.cuda(), dr, eps=0.0, residual_out=dr, y=dx)
    h, y = R.norm(x, w, r, 0.0)
    # h is one rounded addition, whose error a cancellation leaves whole: off by 2^-24 of |x| + |r| at most
    R.check_rounded(dr, h, 2.0 ** -24, 0.0, "residual_out")
    R.check_rounded(dx, y, R.NORM_REL, 0.0, "y")


def test_quantize_fp8_of_large_and_small_values_is_as_it_was():
    x = rand(16, 3, 4096) * torch.tensor([1e37, 1.0, 1e-30])[:, None]
    q, scale = outputs(3, 4096)
    Q.quantize_fp8(x.cuda(), q, scale)
    R.check_q(q.float(), scale, R.f64(x), "q", rel=1e-6)


@pytest.mark.parametrize("eps", [0.0, 1e-36, 1e-6])
@pytest.mark.parametrize("dtype", [F32, F16, BF16])
def test_norm_rows_without_elements_have_the_least_scale(dtype, eps):
    x = torch.empty(5, 0, dtype=dtype, device="cuda")
    q, scale = outputs(5, 0)
    scale.fill_(7.0)
    Q.add_rmsnorm(x, torch.empty(0, dtype=dtype, device="cuda"), eps=eps, q=q, scale=scale)
    assert (scale.cpu() == R.SCALE_MIN).all()


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("cols", COLS)
def test_norm_keeps_the_sign_of_zeros(cols, dtype):
    """Without a residual h is x: a -0 stays one in every output."""
    x = rand(17, 2, cols).to(dtype)
    x[:, ::2] = -0.0
    ro, y = (torch.empty(2, cols, dtype=dtype, device="cuda") for _ in range(2))
    q, scale = outputs(2, cols)
    Q.add_rmsnorm(x.cuda(), torch.ones(cols, dtype=dtype, device="cuda"), residual_out=ro, y=y, q=q, scale=scale)
    Q.quantize_fp8(x.cuda(), (q2 := torch.empty_like(q)), scale)
    assert torch.equal(ro.cpu(), x)
    for out in (ro, y, q.float(), q2.float()):
        assert torch.equal(torch.signbit(out).cpu(), torch.signbit(x))


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("cols", [510, 4096, 20000, 46000])
def test_quantize_fp8_half_way_between_two_values(cols, dtype):
    """Rows of small multiples of 1/64 whose largest is an integer: many of
    their quotients by the scale lie half-way between two e4m3 values and go to
    the even one.  The scale is the nearest fp32 value to max / 448, the
    quotient the nearest one to x / scale."""
    top = torch.arange(7, 128)
    x = torch.randint(0, 256, (len(top), cols), generator=torch.Generator().manual_seed(18)).float()
    x = torch.minimum(x / 64 * 2.0 ** torch.randint(0, 6, x.shape, generator=torch.Generator().manual_seed(19)),
                      top[:, None])
    x[:, 1::2] *= -1
    x[:, 0] = top
    x = x.to(dtype)
    q, scale = outputs(len(top), cols)
    Q.quantize_fp8(x.cuda(), q, scale)
    s = top.numpy().astype(np.float32) / np.float32(448)
    assert np.array_equal(scale.cpu().numpy(), s)
    quotient = x.float().numpy() / s[:, None]
    assert quotient.dtype == np.float32 and np.isin(np.abs(quotient), ties()).sum() > 100
    assert np.array_equal(R.f64(q.float()), R.e4m3(quotient.astype(np.float64)))


def ties():
    v = torch.arange(0, 127, dtype=torch.uint8).view(E4M3).double().numpy()
    return (v[1:] + v[:-1]) / 2


@pytest.mark.parametrize("cols", COLS)
def test_norm_quantises_the_values_that_it_writes(cols):
    """q is e4m3 of the fp32 quotient of y and scale, as both are written."""
    x, r, w = rand(20, 5, cols), rand(21, 5, cols), 1 + 0.2 * rand(22, cols)
    y = torch.empty(5, cols, device="cuda")
    q, scale = outputs(5, cols)
    Q.add_rmsnorm(x.cuda(), w.cuda(), r.cuda(), y=y, q=q, scale=scale)
    quotient = y.cpu().numpy() / scale.cpu().numpy()[:, None]
    assert quotient.dtype == np.float32
    assert np.array_equal(R.f64(q.float()), R.e4m3(quotient.astype(np.float64)))
