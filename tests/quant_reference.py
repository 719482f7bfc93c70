"""64-bit forms of the quantised operators and the bounds their results are held to.

Unit roundoffs (half a unit in the last place over the value): bf16 2^-8, fp16
2^-11, fp32 2^-24, e4m3 2^-4 (2^-10 absolute below 2^-6, fp16 2^-25 below
2^-14).

* add_rmsnorm: h is one fp32 addition (2^-24).  The mean of squares is a sum
  of positive fp32 terms, at most 100 of which one thread adds in a row (a row
  of 1024 by a warp, 45000 by 512 threads, 100000 by 1024), and then at most 40
  partial sums, so its relative error is below 142 * 2^-24 = 9e-6, of which the
  square root halves; the other factors of y add five roundings, 3e-7.
  NORM_REL = 2.5e-5.  The output's own rounding comes on top.  q is compared
  with the roundings of the exact quotient moved down and up by 2 NORM_REL
  (y's error and the scale's), between which a monotone rounding must fall.
* gemm_fp8: e4m3 products are exact in fp32.  A tensor-core step adds 32 of
  them to the running sum and may truncate: at most 2^-22 of the sum of
  magnitudes a step, K/32 <= 64 steps for K <= 2048: SUM_REL = 2e-5 of
  (|A||B|)_ij, the scales' two roundings and the output's one on top.
* gemv_w4: a group's sum is at most 8 steps of 16 products, each off by 2^-22
  of its magnitudes: 8 * 2^-22 < 2e-6.  The groups' sums are scaled and added in
  fp32, one 2^-24 each, at most K/group of them in a row by one thread (fewer
  where K is cut over warps and CTAs), and the cut's 32 partials at most:
  (K/32 + 32) 2^-24 < 2e-5 for K <= 8192; 24576 uncut 5e-5; 81920, which is cut
  in eight, 2.5e-5.  W4_REL = 1e-4 of (|x||w|)_ij holds all of them.
"""
import numpy as np
import torch

UNIT = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
TINY = {torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -149}
NORM_REL = 2.5e-5
SUM_REL = 2e-5
W4_REL = 1e-4
SCALE_MIN = 2.0 ** -126


def f64(t):
    return t.detach().cpu().double().numpy()


def norm(x, weight, residual, eps):
    h = f64(x) + (f64(residual) if residual is not None else 0.0)
    y = h / np.sqrt((h * h).mean(axis=1, keepdims=True) + eps) * f64(weight)
    return h, y


def row_scale(y):
    return np.maximum(np.abs(y).max(axis=1) / 448.0, SCALE_MIN)


def e4m3(v):
    """Nearest-even e4m3 of finite values in [-448 (1 + 2^-4), 448 (1 + 2^-4))."""
    a = np.abs(v)
    e = np.floor(np.log2(np.maximum(a, 2.0 ** -6)))
    step = 2.0 ** (np.maximum(e, -6) - 3)
    return np.copysign(np.minimum(np.rint(a / step) * step, 448.0), v)


def check_rounded(out, ref, rel, abs_, what):
    """|out - ref| <= (unit roundoff of out's type + rel) |ref| + abs_ + the type's tiny."""
    got = f64(out)
    bound = (UNIT[out.dtype] * (1 + 2 * rel) + rel) * np.abs(ref) + abs_ + TINY[out.dtype]
    bad = ~(np.abs(got - ref) <= bound)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.size} out of bound, first at "
                           f"{tuple(np.argwhere(bad)[0])}: {got[bad][0]!r} for {ref[bad][0]!r}")


def check_q(q, scale, y, what, rel=NORM_REL):
    s = row_scale(y)
    got_s, got = f64(scale), f64(q)
    assert np.all(np.abs(got_s - s) <= 2 * rel * s), f"{what}: scale"
    v = np.abs(y / s[:, None])
    lo, hi = e4m3(v * (1 - 2 * rel)), e4m3(np.minimum(v * (1 + 2 * rel), 448.0))
    bad = ~((lo <= np.abs(got)) & (np.abs(got) <= hi))
    assert not bad.any(), f"{what}: q at {tuple(np.argwhere(bad)[0])}: {got[bad][0]} for {v[bad][0]}"
    wrong_sign = (np.sign(got) != np.sign(y)) & (got != 0)
    assert not wrong_sign.any(), f"{what}: sign of q"


def gemm_fp8(A, B, a_scale, b_scale):
    a, b = f64(A), f64(B)
    sa, sb = f64(a_scale)[:, None], f64(b_scale)[None, :]
    return a @ b * sa * sb, np.abs(a) @ np.abs(b) * np.abs(sa) * np.abs(sb)


def w4_weights(W, scales, zeros, group):
    b = W.detach().cpu().numpy()
    q = np.stack((b & 15, b >> 4), axis=2).reshape(b.shape[0], -1).astype(np.float64)
    z = zeros.detach().cpu().numpy().astype(np.float64).repeat(group, axis=1) if zeros is not None else 8.0
    return (q - z) * f64(scales).repeat(group, axis=1)


def gemv_w4(x, W, scales, zeros, group):
    w = w4_weights(W, scales, zeros, group)
    return f64(x) @ w.T, np.abs(f64(x)) @ np.abs(w).T
