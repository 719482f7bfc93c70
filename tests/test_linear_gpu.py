"""The training operators on the GPU against their 64-bit forms (linear_reference.py)."""
import pytest
import torch

import linear_reference as R
from gpu_helpers import GuardedC
from stage_software_pipelining_gb300 import build as gemm_build
from stage_software_pipelining_gb300 import gemm as G
from stage_software_pipelining_gb300 import linear as L
from stage_software_pipelining_gb300 import quant as Q

pytestmark = pytest.mark.gpu
F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
ACTS = list(L.ACTIVATIONS)
NAN = float("nan")


@pytest.fixture(scope="module", autouse=True)
def lib(gpu):
    gemm_build.build()
    return L.load_library()


def rand(seed, *shape, std=1.0):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)) * std


def rows(t, extra=8):
    """A device copy of t whose rows start on 16-byte boundaries, NaN outside it."""
    r, c = t.shape
    unit = 16 // t.element_size()
    buf = torch.full((r, (c + unit - 1) // unit * unit + extra), NAN, device="cuda").to(t.dtype)
    buf[:, :c] = t
    return buf[:, :c]


# Few rows by every tile width and cut, MN-major chunks, the pair kernel; odd sizes;
# one element.
SHAPES = [(1, 1, 1), (1, 8, 8), (1, 4096, 512), (3, 7, 5), (16, 128, 64), (17, 129, 65), (5, 1000, 4097),
          (33, 520, 130), (64, 256, 2048), (100, 300, 50), (129, 384, 257), (200, 1000, 1000), (257, 255, 513),
          (700, 1111, 333), (1100, 2049, 200)]


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_linear_all_parts(M, N, K, dtype):
    x, W = rand(1, M, K).to(dtype), rand(2, N, K, std=K ** -0.5).to(dtype)
    b, r = rand(3, N).to(dtype), rand(4, M, N).to(dtype)
    y, z = GuardedC(M, N, dtype), GuardedC(M, N, dtype)
    L.linear(rows(x), rows(W), y.view, bias=b.cuda(), residual=rows(r), act="gelu", pre=z.view, checked=True)
    y.check()
    z.check()
    R.check_linear(y.view, z.view, x, W, b, r, "gelu")


@pytest.mark.parametrize("name", ACTS)
@pytest.mark.parametrize("bias,residual,pre", [(0, 0, 0), (1, 0, 0), (0, 1, 0), (0, 0, 1), (1, 0, 1)])
@pytest.mark.parametrize("M,N,K", [(2, 300, 96), (80, 136, 70), (600, 1027, 130), (2000, 2304, 64)])
def test_linear_any_set_of_parts(M, N, K, name, bias, residual, pre):
    dtype = BF16 if (M + bias) % 4 else F16
    x, W = rand(5, M, K).to(dtype), rand(6, N, K, std=2 * K ** -0.5).to(dtype)
    b, r = rand(7, N).to(dtype) if bias else None, rand(8, M, N).to(dtype) if residual else None
    y, z = GuardedC(M, N, dtype), GuardedC(M, N, dtype)
    L.linear(rows(x), rows(W), y.view, bias=b.cuda() if bias else None, residual=rows(r) if residual else None,
             act=name, pre=z.view if pre else None, checked=True)
    y.check()
    R.check_linear(y.view, z.view if pre else None, x, W, b, r, name)
    if not pre:
        assert (z.view.float() == torch.tensor(12345.0).to(dtype).float().item()).all()


@pytest.mark.parametrize("M,N,K", [(3, 64, 64), (700, 1100, 200), (1300, 2048, 200)])
def test_linear_residual_in_place(M, N, K):
    x, W, r = rand(1, M, K).to(BF16), rand(2, N, K, std=0.1).to(BF16), rand(3, M, N).to(BF16)
    h = GuardedC(M, N, BF16, init=r)
    L.linear(rows(x), rows(W), h.view, residual=h.view, checked=True)
    h.check()
    R.check_linear(h.view, None, x, W, None, r)


@pytest.mark.parametrize("offset", [0, 1, 3, 8])
@pytest.mark.parametrize("M", [4, 900])
def test_bias_on_any_address(M, offset):
    N, K = 1000, 64
    x, W, b = rand(1, M, K).to(F16), rand(2, N, K).to(F16), rand(3, N).to(F16)
    buf = torch.full((N + offset,), NAN, device="cuda", dtype=F16)
    buf[offset:] = b
    y = GuardedC(M, N, F16)
    L.linear(rows(x), rows(W), y.view, bias=buf[offset:], checked=True)
    y.check()
    R.check_linear(y.view, None, x, W, b)


def test_both_kernels_are_reached():
    plans = [L.linear_plan("linear", *s) for s in SHAPES] + [L.linear_plan("dx", *s) for s in SHAPES] + \
            [L.linear_plan("dw", *s, F32) for s in SHAPES + DW_SHAPES]
    assert {p["kernel"] for p in plans} == {"few", "pair"}
    assert {1, 2, 4} <= {p["split"] for p in plans}


# ---------------------------------------------------------------- act_grad
@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("name", ACTS)
@pytest.mark.parametrize("M,N,extra,offset", [(1, 1, 0, 0), (1, 64, 0, 0), (61, 1000, 0, 0), (128, 70, 2, 0),
                                              (300, 129, 7, 0), (1000, 96, 8, 1), (4099, 200, 0, 0), (33, 517, 3, 5),
                                              (20000, 40, 0, 0), (9001, 210, 6, 0), (9001, 130, 1, 3)])
def test_act_grad(M, N, extra, offset, name, dtype):
    dy, z = rand(1, M, N).to(dtype), rand(2, M, N, std=2.0).to(dtype)

    def wide(t):
        buf = torch.full((M * (N + extra) + offset,), NAN, device="cuda").to(dtype)
        v = buf[offset:].view(M, N + extra)[:, :N]
        v.copy_(t)
        return v

    dz, db = wide(torch.zeros(M, N, dtype=dtype)), torch.full((N + 2,), 77.0, device="cuda")
    c = rand(3, N)
    L.act_grad(wide(dy), dz, pre=wide(z) if name != "none" else None, act=name, dbias=db[1:N + 1], addend=c.cuda())
    R.check_act_grad(dz, db[1:N + 1], dy, z, name, c)
    assert db[0] == 77 and db[-1] == 77
    # one output alone, and no addend
    other = torch.empty(N, device="cuda")
    L.act_grad(wide(dy), pre=wide(z), act=name, dbias=other)
    R.check_act_grad(None, other, dy, z, name)
    alone = wide(torch.zeros(M, N, dtype=dtype))
    L.act_grad(wide(dy), alone, pre=wide(z), act=name)
    assert torch.equal(alone, dz)


def test_act_grad_in_place_and_accumulated():
    M, N = 700, 264
    dy, z = rand(1, M, N).to(BF16), rand(2, M, N).to(BF16)
    d, p, db = dy.cuda(), z.cuda(), torch.ones(N, device="cuda")
    L.act_grad(d, d, pre=p, act="silu", dbias=db, addend=db)
    R.check_act_grad(d, db, dy, z, "silu", torch.ones(N))
    d = dy.cuda()
    L.act_grad(d, p, pre=p, act="silu")
    R.check_act_grad(p, None, dy, z, "silu")


def test_act_grad_without_rows():
    db, c = torch.full((5,), 3.0, device="cuda"), torch.arange(5.0, device="cuda")
    L.act_grad(torch.empty(0, 5, device="cuda", dtype=F16), dbias=db, addend=c)
    assert torch.equal(db, c)
    L.act_grad(torch.empty(0, 5, device="cuda", dtype=F16), dbias=db)
    assert torch.equal(db, torch.zeros_like(c))


# ---------------------------------------------------------------- linear_dx
@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_linear_dx_all_parts(M, N, K, dtype):
    dz, W = rand(1, M, N).to(dtype), rand(2, N, K, std=N ** -0.5).to(dtype)
    r, z = rand(3, M, K).to(dtype), rand(4, M, K, std=1.5).to(dtype)
    dx = GuardedC(M, K, dtype)
    L.linear_dx(rows(dz), rows(W), dx.view, residual=rows(r), act="gelu_tanh", pre=rows(z), checked=True)
    dx.check()
    R.check_dx(dx.view, dz, W, r, z, "gelu_tanh")


@pytest.mark.parametrize("name", ACTS)
@pytest.mark.parametrize("residual", [0, 1])
@pytest.mark.parametrize("M,N,K", [(2, 96, 300), (80, 70, 136), (600, 130, 1027), (2000, 64, 2304)])
def test_linear_dx_any_set_of_parts(M, N, K, name, residual):
    dtype = F16 if residual else BF16
    dz, W = rand(1, M, N).to(dtype), rand(2, N, K, std=N ** -0.5).to(dtype)
    r = rand(3, M, K).to(dtype) if residual else None
    z = rand(4, M, K, std=1.5).to(dtype) if name != "none" else None
    dx = GuardedC(M, K, dtype)
    L.linear_dx(rows(dz), rows(W), dx.view, residual=rows(r) if residual else None, act=name,
                pre=rows(z) if z is not None else None, checked=True)
    dx.check()
    R.check_dx(dx.view, dz, W, r, z, name)


@pytest.mark.parametrize("M,N,K", [(3, 64, 72), (700, 200, 1100), (1300, 200, 2048)])
@pytest.mark.parametrize("over", ["residual", "pre"])
def test_linear_dx_in_place(M, N, K, over):
    dz, W = rand(1, M, N).to(F16), rand(2, N, K, std=0.1).to(F16)
    r, z = rand(3, M, K).to(F16), rand(4, M, K).to(F16)
    d = {"residual": rows(r), "pre": rows(z)}
    L.linear_dx(rows(dz), rows(W), d[over], act="gelu", checked=True, **d)
    R.check_dx(d[over], dz, W, r, z, "gelu")


# ---------------------------------------------------------------- linear_dw
DW_SHAPES = [(9000, 100, 200), (17000, 300, 64), (70000, 40, 24), (5000, 1500, 2100), (8300, 2304, 2048)]


@pytest.mark.parametrize("dtype,out", [(F16, F32), (BF16, F32), (F16, F16), (BF16, BF16)])
@pytest.mark.parametrize("M,N,K", SHAPES + DW_SHAPES[:4])
def test_linear_dw(M, N, K, dtype, out):
    dz, x = rand(1, M, N).to(dtype), rand(2, M, K).to(dtype)
    c = rand(3, N, K, std=M ** 0.5).to(out)
    dw = GuardedC(N, K, out)
    L.linear_dw(rows(dz), rows(x), dw.view, addend=rows(c), checked=True)
    dw.check()
    R.check_dw(dw.view, dz, x, c)
    again = GuardedC(N, K, out)
    L.linear_dw(rows(dz), rows(x), again.view, checked=True)
    again.check()
    R.check_dw(again.view, dz, x)


@pytest.mark.parametrize("M,N,K", DW_SHAPES[2:])
def test_linear_dw_long_sums_keep_their_precision(M, N, K):
    """In fp32 no accumulator sums more than 4096 rows.  Of equal signs, a sum of
    4096 truncates at most 256 steps, 2^-23 each for a sum that grows evenly (half
    the last value on average, 2^-24 of a step's own): 256 * 2^-23 / 2 = 1.5e-5."""
    dz, x = rand(1, M, N).abs().to(BF16), rand(2, M, K).abs().to(BF16)
    dw = torch.empty(N, K, device="cuda")
    L.linear_dw(rows(dz), rows(x), dw, checked=True)
    ref = dz.cuda().double().t() @ x.cuda().double()
    assert ((dw.double() - ref).abs() / ref).max() < 1.6e-5


@pytest.mark.parametrize("M,N,K", [(50, 40, 72), (5000, 1500, 2104)])
def test_linear_dw_accumulates_in_place(M, N, K):
    dz, x, c = rand(1, M, N).to(BF16), rand(2, M, K).to(BF16), rand(3, N, K)
    dw = GuardedC(N, K, F32, init=c)
    L.linear_dw(rows(dz), rows(x), dw.view, addend=dw.view, checked=True)
    dw.check()
    R.check_dw(dw.view, dz, x, c)


# ---------------------------------------------------------------- sums of nothing
def test_sums_of_nothing():
    e = torch.empty(0, 16, device="cuda", dtype=F16)
    c = rand(1, 16, 8).cuda()
    out = torch.full((16, 8), NAN, device="cuda")
    L.linear_dw(e, torch.empty(0, 8, device="cuda", dtype=F16), out, addend=c)
    assert torch.equal(out, c)
    L.linear_dw(e, torch.empty(0, 8, device="cuda", dtype=F16), out)
    assert torch.equal(out, torch.zeros_like(out))
    b, r = rand(2, 24).to(F16).cuda(), rand(3, 300, 24).to(F16).cuda()
    y, z = torch.empty_like(r), torch.empty_like(r)
    x0, w0 = torch.empty(300, 0, device="cuda", dtype=F16), torch.empty(24, 0, device="cuda", dtype=F16)
    L.linear(x0, w0, y, bias=b, residual=r, act="relu", pre=z)
    assert torch.equal(z, b.expand_as(z)) and torch.equal(y, (b.float().clamp_min(0) + r.float()).to(F16))
    d = torch.empty(300, 24, device="cuda", dtype=F16)
    L.linear_dx(x0, torch.empty(0, 24, device="cuda", dtype=F16), d, residual=r, act="relu", pre=z)
    assert torch.equal(d, torch.where(z <= 0, torch.zeros_like(r), r))
    for f, args in ((L.linear, (torch.empty(0, 8, device="cuda", dtype=F16), w0.new_empty(3, 8), w0.new_empty(0, 3))),
                    (L.linear, (w0.new_empty(5, 8), w0.new_empty(0, 8), w0.new_empty(5, 0)))):
        f(*args)
    torch.cuda.synchronize()


# ---------------------------------------------------------------- special values
@pytest.mark.parametrize("name", ACTS[1:])
@pytest.mark.parametrize("M", [1, 600])
def test_special_values(M, name):
    """Infinities and NaN through an activation and its derivative."""
    N, K = 520, 64
    W = torch.zeros(N, K, dtype=F16)
    b = torch.zeros(N, dtype=F16)
    ends = [float("inf"), float("-inf"), NAN, 65504.0, -65504.0, 0.0, -0.0, 30.0, -30.0]
    b[:len(ends)] = torch.tensor(ends)
    b[32:50:2] = torch.tensor(ends)         # alone beside an ordinary value
    b[65:83:2] = torch.tensor(ends)
    b[100:200] = torch.linspace(-12, 12, 100)
    y, z = torch.empty(M, N, device="cuda", dtype=F16), torch.empty(M, N, device="cuda", dtype=F16)
    L.linear(rows(torch.zeros(M, K, dtype=F16)), rows(W), y, bias=b.cuda(), act=name, pre=z, checked=True)
    ref = torch.from_numpy(R.act(b.double().numpy(), name)).to(F16)
    assert torch.allclose(y.cpu(), ref.expand(M, N), rtol=2.0 ** -10, atol=2.0 ** -24, equal_nan=True)
    assert torch.equal(torch.nan_to_num(z.cpu(), nan=7.0), torch.nan_to_num(b, nan=7.0).expand(M, N))
    d = torch.empty(M, N, device="cuda", dtype=F16)
    L.act_grad(torch.ones(M, N, device="cuda", dtype=F16), d, pre=z, act=name)
    slope = torch.from_numpy(R.derivative(b.double().numpy(), name)).to(F16)
    if name == "relu":
        slope[b.isnan()] = 1.0
    assert torch.allclose(d.cpu(), slope.expand(M, N), rtol=2.0 ** -10, atol=1.1e-5, equal_nan=True)
    e = torch.empty(M, N, device="cuda", dtype=F16)
    L.linear_dx(rows(torch.zeros(M, K, dtype=F16)), rows(torch.zeros(K, N, dtype=F16)), e, pre=z, act=name,
                residual=torch.ones(M, N, device="cuda", dtype=F16), checked=True)
    assert torch.equal(torch.nan_to_num(e, nan=7.0), torch.nan_to_num(d, nan=7.0))


@pytest.mark.parametrize("M,N", [(5, 200), (600, 1024)])
def test_a_nan_stays_in_its_row_and_column(M, N):
    K = 100
    x, W = rand(1, M, K).to(BF16), rand(2, N, K).to(BF16)
    x[M // 2, 3] = NAN
    W[N // 3, 7] = float("inf")
    y = torch.empty(M, N, device="cuda", dtype=BF16)
    L.linear(rows(x), rows(W), y, checked=True)
    bad = ~torch.isfinite(y.cpu())
    expect = torch.zeros(M, N, dtype=torch.bool)
    expect[M // 2] = True
    expect[:, N // 3] = True
    assert torch.equal(bad, expect)


# ---------------------------------------------------------------- orthogonalize
ABC = (3.4445, -4.7750, 2.0315)


def batch(t, extra=8):
    """A device copy of a batch of matrices, rows and matrices apart, NaN between."""
    n, r, c = t.shape
    unit = 16 // t.element_size()
    buf = torch.full((n, r + 1, (c + unit - 1) // unit * unit + extra), NAN, device="cuda").to(t.dtype)
    buf[:, :r, :c] = t
    return buf[:, :r, :c]


def workspace(g):
    n = L.orthogonalize_workspace(g)
    return torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")     # NaN wherever it is read before it is written


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("out", [F16, BF16])
@pytest.mark.parametrize("B,rows_,cols", [(1, 1, 1), (1, 1, 50), (2, 40, 3), (3, 24, 100), (2, 130, 60), (1, 257, 300),
                                          (2, 300, 1000), (1, 1000, 301), (1, 520, 2100), (5, 128, 513), (2, 100, 2560),
                                          (1, 3000, 128), (40, 64, 700), (1, 17, 2049), (1, 128, 2561), (200, 9, 65)])
def test_orthogonalize(B, rows_, cols, dtype, out):
    g = rand(1, B, rows_, cols, std=1e-3).to(dtype)
    o = batch(torch.zeros(B, rows_, cols, dtype=out))
    d = batch(g)
    L.orthogonalize(d, o, workspace(d), scale=0.75, checked=True)
    for k in range(B):
        R.check_ortho(o[k], g[k], 5, ABC, 1e-7, 0.75)
    assert torch.isnan(o.as_strided((B, rows_ + 1, o.stride(1)), o.stride())[:, rows_]).all()


@pytest.mark.parametrize("steps", [0, 1, 2, 3])
@pytest.mark.parametrize("coefficients", [ABC, (1.5, -0.5, 0.0), (2.0, -1.5, 0.5)])
@pytest.mark.parametrize("rows_,cols", [(64, 200), (200, 64), (129, 129)])
def test_orthogonalize_steps(rows_, cols, steps, coefficients):
    g = rand(2, rows_, cols).to(BF16)
    o = torch.empty(rows_, (cols + 7) // 8 * 8, device="cuda", dtype=F16)[:, :cols]
    d = rows(g)
    L.orthogonalize(d, o, workspace(d), steps=steps, coefficients=coefficients, eps=0.0, checked=True)
    R.check_ortho(o, g, steps, coefficients, 0.0, 1.0)


@pytest.mark.parametrize("rows_,cols", [(1500, 1700), (2304, 2100), (2500, 2304)])
def test_orthogonalize_symmetric_tiles(rows_, cols):
    """Sizes whose squares are computed on the pair kernel, on one side of the diagonal."""
    g = rand(3, rows_, cols).to(BF16)
    d = batch(g.expand(3, rows_, cols))
    o = batch(torch.zeros(3, rows_, cols, dtype=BF16))
    L.orthogonalize(d, o, workspace(d), steps=2, checked=True)
    assert torch.equal(o[0], o[1]) and torch.equal(o[0], o[2])
    x = g.cuda().double()
    x = x / (x.norm() + 1e-7)
    for _ in range(2):
        m = x @ x.t()
        x = ABC[0] * x + (ABC[1] * m + ABC[2] * m @ m) @ x
    # Two steps: each rounding of A, B and X (2^-11 an element) comes through with
    # at most 3.45 times its size (the slope at zero) and 4.775 + 2 * 2.04 times for A's.
    bound = (2 * 2.0 ** -11 * (1 + 1 + 9) * 3.45 + 2.0 ** -8) * x.norm()
    assert (o[0].double() - x).norm() <= bound
    assert torch.equal(o.isnan().any(), torch.tensor(False, device="cuda"))


@pytest.mark.parametrize("dtype,size", [(F32, 1e-42), (F32, 1e-30), (F32, 1e-18), (F32, 1e18), (F32, 3e37), (BF16, 1e-30),
                                        (BF16, 1e30), (F16, 6e-8), (F16, 6e4)])
def test_orthogonalize_any_magnitude(dtype, size):
    g = (torch.randint(0, 2, (40, 120), generator=torch.Generator().manual_seed(5)) * 2 - 1) * torch.tensor(size)
    g = g.to(dtype)
    d = rows(g)
    o = torch.empty(40, 120, device="cuda", dtype=F16)
    L.orthogonalize(d, o, workspace(d), eps=0.0, checked=True)
    R.check_ortho(o, (g.double() / g.double().abs().max()).float(), 5, ABC, 0.0, 1.0)


def test_orthogonalize_special_matrices():
    g = torch.zeros(4, 33, 70)
    g[1, 3, 4] = 2.5            # a single element: a single singular value
    g[2, 5, 6] = NAN
    g[3, 32, 69] = float("inf")
    d = batch(g)
    o = torch.empty(4, 33, 72, device="cuda", dtype=BF16)[:, :, :70]
    L.orthogonalize(d, o, workspace(d), checked=True)
    assert torch.equal(o[0].float(), torch.zeros(33, 70, device="cuda"))
    R.check_ortho(o[1], g[1], 5, ABC, 1e-7, 1.0)
    assert o[2].isnan().all() and o[3].isnan().all()
    L.orthogonalize(d, o, workspace(d), eps=0.0, steps=0, checked=True)
    assert o[0].isnan().all() and o[2].isnan().all() and o[3].isnan().all()
    assert o[1, 3, 4] == 1 and o[1].float().abs().sum() == 1


# ---------------------------------------------------------------- calls
def run_all(t, stream=None):
    """Every operator on the tensors of t, on `stream`."""
    L.linear(t["x"], t["W"], t["y"], bias=t["b"], act="silu", pre=t["z"], stream=stream)
    L.act_grad(t["y"], t["dz"], pre=t["z"], act="silu", dbias=t["db"], stream=stream)
    L.linear_dx(t["dz"], t["W"], t["dx"], residual=t["x"], stream=stream)
    L.linear_dw(t["dz"], t["x"], t["dw"], stream=stream)
    L.orthogonalize(t["dw"], t["o"], t["ws"], stream=stream)


def tensors(seed, M=300, N=264, K=520):
    t = {"x": rand(seed, M, K).to(BF16).cuda(), "W": rand(seed + 1, N, K, std=K ** -0.5).to(BF16).cuda(),
         "b": rand(seed + 2, N).to(BF16).cuda()}
    for k, s, d in (("y", (M, N), BF16), ("z", (M, N), BF16), ("dz", (M, N), BF16), ("dx", (M, K), BF16),
                    ("dw", (N, K), F32), ("o", (N, K), BF16), ("db", (N,), F32)):
        t[k] = torch.zeros(s, device="cuda", dtype=d)
    t["ws"] = workspace(t["dw"])
    return t


OUTS = ("y", "z", "dz", "dx", "dw", "o", "db")


def test_same_bits_every_call_on_any_stream_and_in_a_graph():
    a, b = tensors(1), tensors(1)
    run_all(a)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    run_all(b, side)
    torch.cuda.current_stream().wait_stream(side)
    for k in OUTS:
        assert torch.equal(a[k], b[k]), k
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run_all(b)
    fresh = tensors(50)
    for k in ("x", "W", "b"):
        b[k].copy_(fresh[k])
    graph.replay()
    run_all(fresh)
    torch.cuda.synchronize()
    for k in OUTS:
        assert torch.equal(fresh[k], b[k]), k


def test_two_streams_at_once():
    sets = [tensors(10 * i, 200 + 57 * i) for i in range(4)]
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    for _ in range(5):
        for t, s in zip(sets, streams):
            run_all(t, s)
    torch.cuda.synchronize()
    for i, t in enumerate(sets):
        alone = tensors(10 * i, 200 + 57 * i)
        run_all(alone)
        torch.cuda.synchronize()
        for k in OUTS:
            assert torch.equal(alone[k], t[k]), (i, k)


@pytest.mark.parametrize("M", [4, 800])
def test_a_withheld_stage_times_out(M):
    """A stage that never arrives ends every role within the limit, and the next call is sound."""
    x, W = rand(1, M, 256).to(BF16), rand(2, 512, 256).to(BF16)
    dx_, dW = rows(x), rows(W)
    y = torch.empty(M, 512, device="cuda", dtype=BF16)
    G.debug_set(wait_limit_ns=50_000_000, withhold_arrive=0)
    try:
        with pytest.raises(G.GemmError) as e:
            L.linear(dx_, dW, y, checked=True)
        assert e.value.status == G.GEMM_ERR_TIMEOUT
    finally:
        G.debug_set()
    L.linear(dx_, dW, y, checked=True)
    R.check_linear(y, None, x, W)


def test_binding_refusals():
    x, W, y = (torch.zeros(s, device="cuda", dtype=F16) for s in ((4, 16), (8, 16), (4, 8)))
    b = torch.zeros(8, device="cuda", dtype=F16)
    f = torch.zeros(8, device="cuda")
    for call in (lambda: L.linear(x, W.t(), y), lambda: L.linear(x, W, y.t()), lambda: L.linear(x, W, y, bias=f),
                 lambda: L.linear(x.to(BF16), W, y), lambda: L.linear(x, W, y, bias=b[:7]),
                 lambda: L.linear(x, W, y, residual=x), lambda: L.linear(x, W, y.cpu()),
                 lambda: L.linear(x, W, y, stream=3), lambda: L.linear(x.float(), W.float(), y.float()),
                 lambda: L.act_grad(y), lambda: L.act_grad(y, y, act="silu"), lambda: L.act_grad(y, y, addend=f),
                 lambda: L.act_grad(y, dbias=b), lambda: L.linear_dx(y, W, x, act="gelu"),
                 lambda: L.linear_dx(y, W, x, pre=x), lambda: L.linear_dw(y, x, W.to(BF16)),
                 lambda: L.linear_dw(y, x, W.double()), lambda: L.linear_dw(y, x[:3], W),
                 lambda: L.orthogonalize(x, y, f), lambda: L.orthogonalize(x, x.float(), f),
                 lambda: L.orthogonalize(x.t(), x.t().clone(), f), lambda: L.orthogonalize(x, x.clone(), f.cpu()),
                 lambda: L.orthogonalize(x, x.clone(), f, steps=101), lambda: L.orthogonalize(x, x.clone(), f, steps=-1),
                 lambda: L.orthogonalize(x, x.clone(), f, steps=1.5), lambda: L.orthogonalize(x, x.clone(), f, eps="a"),
                 lambda: L.orthogonalize(x[None].expand(3, 4, 16), x[None].repeat(3, 1, 1), f)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(G.GemmError):
        L.orthogonalize(x, x.clone(), f)        # the workspace is too small
    with pytest.raises(G.GemmError):
        L.linear(x[:, 1:9], W[:, :8], y)        # rows that do not start on a boundary
    with pytest.raises(G.GemmError):
        L.orthogonalize(x, x.clone(), torch.empty(1 << 20, dtype=torch.uint8, device="cuda"), eps=-1.0)
