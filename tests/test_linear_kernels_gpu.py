"""The products of the training operators on every instance of their kernels, the plan
asserted, and at the ends of their ranges."""
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


def rand(seed, rows, cols, dtype, std=1.0):
    t = Q.empty_rows(rows, cols, dtype)
    g = torch.Generator(device="cuda").manual_seed(seed)
    t.copy_(torch.randn(rows, cols, generator=g, device="cuda") * std)
    return t


def check(out, ref, bound, what):
    """All in 64 bits on the GPU (quant_reference.check_rounded's rule)."""
    off = (out.double() - ref).abs()
    limit = R.UNIT[out.dtype] * ref.abs() + bound + R.TINY[out.dtype]
    bad = ~(off <= limit)
    assert not bad.any(), f"{what}: {int(bad.sum())} out of bound, first at {tuple(bad.nonzero()[0].tolist())}"


def run(op, M, N, K, dtype, out=None, parts=True):
    """One product with every part of its epilogue, against 64 bits."""
    if op == "linear":
        x, W = rand(1, M, K, dtype), rand(2, N, K, dtype, K ** -0.5)
        b, r = rand(3, 1, N, dtype)[0].contiguous(), rand(4, M, N, dtype)
        y, z = Q.empty_rows(M, N, dtype), Q.empty_rows(M, N, dtype)
        L.linear(x, W, y, bias=b if parts else None, residual=r if parts else None, act="relu" if parts else "none",
                 pre=z if parts else None, checked=True)
        s, mag = x.double() @ W.double().t(), x.double().abs() @ W.double().t().abs()
        err = R.sum_rel(K) * mag
        if parts:
            s = s + b.double()
            err = err + 2.0 ** -23 * s.abs()
            check(z, s, err, "pre")
            s = s.clamp_min(0) + r.double()
            err = err + 2.0 ** -23 * (s.abs() + r.double().abs())
        check(y, s, err, "y")
    elif op == "dx":
        dz, W = rand(1, M, N, dtype), rand(2, N, K, dtype, N ** -0.5)
        r, z = rand(3, M, K, dtype), rand(4, M, K, dtype)
        dx = Q.empty_rows(M, K, dtype)
        L.linear_dx(dz, W, dx, residual=r if parts else None, act="relu" if parts else "none", pre=z if parts else None,
                    checked=True)
        s, mag = dz.double() @ W.double(), dz.double().abs() @ W.double().abs()
        err = R.sum_rel(N) * mag
        if parts:
            s = (s + r.double()) * (z > 0)
            err = err + 2.0 ** -23 * s.abs()
        check(dx, s, err, "dx")
    else:
        dz, x = rand(1, M, N, dtype), rand(2, M, K, dtype)
        dw, c = Q.empty_rows(N, K, out), rand(3, N, K, out, M ** 0.5)
        L.linear_dw(dz, x, dw, addend=c if parts else None, checked=True)
        s, mag = dz.double().t() @ x.double(), dz.double().t().abs() @ x.double().abs()
        err = R.sum_rel(M, 4096 if out == F32 else None) * mag
        if parts:
            s = s + c.double()
            err = err + 2.0 ** -23 * (s.abs() + c.double().abs())
        check(dw, s, err, "dw")


# op, M, N, K, kernel, tile rows, CTAs of a cut (0: uncut, 2: cut), CTAs of the launch (None: any)
CASES = [
    ("linear", 1, 40, 40, "few", 16, 0, None), ("linear", 1, 40, 200, "few", 16, 2, None),
    ("linear", 3000, 40, 40, "few", 32, 0, None), ("linear", 20, 3000, 500, "few", 32, 2, None),
    ("linear", 5000, 40, 200, "few", 64, 0, None), ("linear", 40, 3000, 1500, "few", 64, 2, None),
    ("linear", 100, 3000, 3000, "few", 128, 2, None), ("linear", 130, 5000, 3000, "few", 256, 2, None),
    ("linear", 1000, 2700, 64, "pair", 256, 0, 120),      # tiles of 192 columns
    ("linear", 300, 8512, 1030, "pair", 256, 0, 152),     # of 224
    ("linear", 2000, 2041, 2000, "pair", 256, 0, 128),    # of 256
    ("dx", 1, 40, 40, "few", 16, 0, None), ("dx", 1, 200, 40, "few", 16, 2, None),
    ("dx", 3000, 40, 40, "few", 32, 0, None), ("dx", 20, 500, 3000, "few", 32, 2, None),
    ("dx", 5000, 200, 40, "few", 64, 0, None), ("dx", 40, 1500, 3000, "few", 64, 2, None),
    ("dx", 100, 3000, 3000, "few", 128, 2, None), ("dx", 130, 3000, 5000, "few", 256, 2, None),
    ("dx", 1000, 64, 2700, "pair", 256, 0, 120), ("dx", 2000, 2000, 2041, "pair", 256, 0, 128),
    ("dw", 1, 40, 40, "few", 64, 0, None), ("dw", 500, 40, 40, "few", 64, 2, None),
    ("dw", 3000, 100, 3000, "few", 128, 2, None), ("dw", 3000, 130, 5000, "few", 256, 2, None),
    ("dw", 64, 1000, 2700, "pair", 256, 0, 120), ("dw", 2000, 2000, 2041, "pair", 256, 0, 128),
    ("dw", 20000, 130, 5000, "few", 256, 2, None),        # several accumulators a CTA
]


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("op,M,N,K,kernel,rows,cut,grid", CASES)
def test_every_instance(op, M, N, K, kernel, rows, cut, grid, dtype):
    for out in ((F32, dtype) if op == "dw" else (dtype,)):
        plan = L.linear_plan(op, M, N, K, out)
        assert (plan["kernel"], plan["tile_rows"]) == (kernel, rows)
        assert plan["split"] == 1 if cut == 0 else plan["split"] >= cut
        assert grid is None or plan["grid"] == grid
        run(op, M, N, K, dtype, out)
        run(op, M, N, K, dtype, out, parts=False)


@pytest.mark.parametrize("M,N,K", [(300, 257, 100), (520, 513, 64), (700, 1025, 77), (257, 4100, 200), (400, 2305, 33),
                                   (1000, 2689, 64), (1300, 2041, 500)])
def test_every_remainder_of_a_row(M, N, K):
    """Rows that end inside 16 bytes, by 1 to 7 columns: none is missed, none written past it."""
    for extra in range(8):
        n = N + extra
        for dtype, out in ((F16, F16), (BF16, F32)):
            dz, x = rand(1, K, M, dtype), rand(2, K, n, dtype)
            dw = torch.full((M, (n + 7) // 8 * 8 + 8), 7.0, device="cuda", dtype=out)
            L.linear_dw(dz, x, dw[:, :n], checked=True)
            s, mag = dz.double().t() @ x.double(), dz.double().t().abs() @ x.double().abs()
            check(dw[:, :n], s, R.sum_rel(K) * mag, f"{n} columns")
            assert (dw[:, n:] == 7.0).all()


def test_offsets_past_32_bits():
    """A matrix whose last rows lie 2^32 elements and more behind its first."""
    rows, ld = 530, (1 << 23) + 64
    big = torch.empty(rows * ld, dtype=BF16, device="cuda")
    x = big.as_strided((rows, 200), (ld, 1))
    assert (rows - 1) * ld > 1 << 32
    x.copy_(rand(1, rows, 200, BF16))
    W = rand(2, 300, 200, BF16, 0.1)
    y = rand(3, rows, 300, BF16)
    far = big.as_strided((rows, 300), (ld, 1), 1 << 20)
    far.copy_(y)
    s, mag = x.double() @ W.double().t(), x.double().abs() @ W.double().t().abs()
    L.linear(x, W, far, residual=far, checked=True)
    err = R.sum_rel(200) * mag + 2.0 ** -23 * (s.abs() + y.double().abs())
    check(far, s + y.double(), err, "y")
    few = big.as_strided((5, 300), (ld * 131, 1), 1 << 21)
    L.linear(x[::131][:5], W, few, checked=True)
    check(few, s[::131][:5], R.sum_rel(200) * mag[::131][:5], "few rows")
    d = big.as_strided((rows, 300), (ld, 1), 1 << 22)
    db = torch.empty(300, device="cuda")
    L.act_grad(far, d, pre=y, act="relu", dbias=db)
    assert torch.equal(d, torch.where(y > 0, far, torch.zeros_like(far)))
    g = far.double() * (y > 0)
    assert ((db.double() - g.sum(0)).abs() <= (rows / 16 + 48) * 2.0 ** -24 * g.abs().sum(0)).all()


@pytest.mark.parametrize("M,N,K", [(3, 520, 256), (600, 520, 256)])
def test_two_graphs_at_once(M, N, K):
    """Two captured calls replayed on two streams together: nothing of one is the other's."""
    sets = []
    for i in range(2):
        x, W = rand(10 + i, M, K, BF16), rand(20 + i, N, K, BF16, 0.1)
        y = Q.empty_rows(M, N, BF16)
        g, ws = rand(30 + i, 200, 700, F32), None
        ws = torch.empty(L.orthogonalize_workspace(g), dtype=torch.uint8, device="cuda")
        o = torch.empty(200, 704, device="cuda", dtype=BF16)[:, :700]
        L.linear(x, W, y)
        L.orthogonalize(g, o, ws)
        torch.cuda.synchronize()
        expect = y.clone(), o.clone()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            for _ in range(5):
                L.linear(x, W, y)
                L.orthogonalize(g, o, ws)
        y.zero_()
        o.zero_()
        sets.append((graph, torch.cuda.Stream(), y, o, expect, (x, W, g, ws)))
    torch.cuda.synchronize()
    for _ in range(3):
        for graph, stream, *_ in sets:
            with torch.cuda.stream(stream):
                graph.replay()
    torch.cuda.synchronize()
    for _, _, y, o, (ey, eo), _ in sets:
        assert torch.equal(y, ey) and torch.equal(o, eo)


def test_captured_before_any_call():
    """The first call of a process may be a captured one."""
    import subprocess
    import sys
    code = ("import torch\n"
            "from stage_software_pipelining_gb300 import linear as L\n"
            "x = torch.ones(300, 64, device='cuda', dtype=torch.bfloat16)\n"
            "y = torch.zeros(300, 304, device='cuda', dtype=torch.bfloat16)[:, :300]\n"
            "dw = torch.zeros(64, 64, device='cuda')\n"
            "o = torch.zeros(64, 64, device='cuda', dtype=torch.bfloat16)\n"
            "ws = torch.empty(L.orthogonalize_workspace(dw), dtype=torch.uint8, device='cuda')\n"
            "db = torch.zeros(64, device='cuda')\n"
            "torch.cuda.synchronize()\n"
            "g = torch.cuda.CUDAGraph()\n"
            "with torch.cuda.graph(g):\n"
            "    L.linear(x, x, y)\n"
            "    L.linear_dw(x, x, dw)\n"
            "    L.act_grad(x, dbias=db)\n"
            "    L.orthogonalize(dw, o, ws)\n"
            "g.replay()\n"
            "torch.cuda.synchronize()\n"
            "assert (y == 64).all() and (dw == 300).all() and (db == 300).all() and o.float().abs().max() > 0\n")
    subprocess.run([sys.executable, "-c", code], check=True, timeout=300)


@pytest.mark.parametrize("n", [1, 7, 64, 65, 127, 128])
@pytest.mark.parametrize("m", [128, 320, 321, 641, 2560])
@pytest.mark.parametrize("tall", [False, True])
def test_orthogonalize_in_one_launch(n, m, tall):
    """Matrices that one launch takes: every number of CTAs that share one, both ways round."""
    g = rand(5, n, m, BF16)
    g = g.t().contiguous() if tall else g
    d = Q.empty_rows(*g.shape, BF16)
    d.copy_(g)
    out = Q.empty_rows(*g.shape, F16)
    ws = torch.full((L.orthogonalize_workspace(d),), 0xFF, dtype=torch.uint8, device="cuda")
    abc = (2.0, -1.5, 0.5)
    L.orthogonalize(d, out, ws, steps=3, coefficients=abc, checked=True)
    R.check_ortho(out, d, 3, abc, 1e-7, 1.0)
    again = Q.empty_rows(*g.shape, F16)
    L.orthogonalize(d, again, ws, steps=3, coefficients=abc)
    assert torch.equal(out, again)


@pytest.mark.parametrize("rows,cols", [(100, 300), (300, 400)])
def test_orthogonalize_times_out_soundly(rows, cols):
    """With no time to wait at all, a call ends and says so or is right; the next is right."""
    g = rand(6, rows, cols, F32)
    out = Q.empty_rows(rows, cols, BF16)
    ws = torch.empty(L.orthogonalize_workspace(g), dtype=torch.uint8, device="cuda")
    try:
        G.debug_set(wait_limit_ns=50_000_000, withhold_arrive=0)
        try:
            L.orthogonalize(g, out, ws, checked=True)
        except G.GemmError as e:
            assert e.status == G.GEMM_ERR_TIMEOUT
    finally:
        G.debug_set()
    L.orthogonalize(g, out, ws, checked=True)
    R.check_ortho(out, g, 5, (3.4445, -4.7750, 2.0315), 1e-7, 1.0)


def test_singular_values_come_near_one():
    g = rand(7, 256, 1000, F32)
    out = Q.empty_rows(256, 1000, BF16)
    ws = torch.empty(L.orthogonalize_workspace(g), dtype=torch.uint8, device="cuda")
    L.orthogonalize(g, out, ws)
    s = np.linalg.svd(R.f64(out), compute_uv=False)
    assert 0.65 < s.min() and s.max() < 1.25
