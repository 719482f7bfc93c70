"""64-bit forms of the training operators and the bounds their results are held to.

Unit roundoffs as in quant_reference.py (bf16 2^-8, fp16 2^-11, fp32 2^-24).

* A product's sum: products of 16-bit values are exact in fp32; a tensor-core
  step adds 16 of them to the running sum and may truncate, at most 2^-22 of the
  sum of magnitudes a step, K/16 steps; at most 7 partial sums of a cut K and the
  accumulators of a long one join in fp32, 2^-24 each.  sum_rel(K) of (|A||B|)_ij.
  An fp32 dw sums 4096 rows at most in one accumulator, so its steps stop at 256.
* Activations: exp, the reciprocal and the normal tail are good to 2^-20 of their value
  where the argument is moderate; an argument v of exp is itself rounded, which
  adds |v| 2^-24, below 2^-17 where the result is not tiny.  ACT_REL = 2^-16 of
  |act(z)|.  |act'| is below 1.13, so an error of z comes through at most 1.13
  times.
* Derivatives are sums of terms of at most about one (p, f p (1-p), f phi), each
  good to 2^-19: DERIVATIVE = 1e-5, absolute.  Their second derivatives are not
  needed: z comes rounded, and is taken as given.
* dbias: a thread adds at most M/16 + 1 rows (sixteen row lanes, of the kernel for
  unaligned rows), then two lanes' steps, 32 warps and 8 CTAs follow:
  (M/16 + 48) 2^-24 of the sum of magnitudes, and DERIVATIVE of that of |dy|.
"""
import math

import numpy as np
import torch

from quant_reference import TINY, UNIT, check_rounded, f64  # noqa: F401

ACT_REL = 2.0 ** -16
DERIVATIVE = 1e-5
LEAST = 1e-16           # arguments end where the function is within 43 exp(-43) = 9e-18 of its limit
GELU_C = math.sqrt(2 / math.pi)


def sum_rel(K, chunk=None):
    steps = -(-min(K, chunk or K) // 16)
    return steps * 2.0 ** -22 + (8 + (K // chunk if chunk else 0)) * 2.0 ** -24


def _phi(z):
    return 0.5 * torch.special.erfc(-torch.as_tensor(z) * math.sqrt(0.5)).numpy()


def act(z, name):
    z = np.asarray(z, dtype=np.float64)
    with np.errstate(over="ignore", invalid="ignore"):
        if name == "none":
            return z
        if name == "relu":
            return np.where(z < 0, 0.0, z)
        if name == "gelu":
            y = z * _phi(z)
        elif name == "gelu_tanh":
            y = z / (1 + np.exp(-2 * GELU_C * (z + 0.044715 * z ** 3)))
        else:
            y = z / (1 + np.exp(-z))
    return np.where(np.isneginf(z), 0.0, y)


def derivative(z, name):
    z = np.asarray(z, dtype=np.float64)
    if name == "none":
        return np.ones_like(z)
    if name == "relu":
        return np.where(z <= 0, 0.0, 1.0)
    f = np.clip(z, -200, 200)
    with np.errstate(over="ignore"):
        if name == "gelu":
            d = _phi(f) + f * np.exp(-f * f / 2) / math.sqrt(2 * math.pi)
        elif name == "gelu_tanh":
            p = 1 / (1 + np.exp(-2 * GELU_C * (f + 0.044715 * f ** 3)))
            d = p + f * p * (1 - p) * 2 * GELU_C * (1 + 3 * 0.044715 * f * f)
        else:
            p = 1 / (1 + np.exp(-f))
            d = p + f * p * (1 - p)
    return np.where(np.isnan(z), np.nan, d)


def product(a, b):
    return a @ b, np.abs(a) @ np.abs(b)


def check_linear(y, pre, x, W, bias=None, residual=None, name="none", what="linear"):
    z, mag = product(f64(x), f64(W).T)
    if bias is not None:
        z = z + f64(bias)
    err = sum_rel(x.shape[1]) * mag + 2.0 ** -24 * np.abs(z)
    if pre is not None:
        check_rounded(pre, z, 0.0, err, what + ": pre")
    a = act(z, name)
    r = f64(residual) if residual is not None else 0.0
    rel = 0.0 if name in ("none", "relu") else ACT_REL
    check_rounded(y, a + r, 0.0, 1.13 * err + rel * np.abs(a) + 2.0 ** -23 * (np.abs(a) + np.abs(r)) + LEAST, what)


def check_act_grad(dz, dbias, dy, pre, name, addend=None, what="act_grad"):
    g = f64(dy)
    d = derivative(f64(pre), name) if name != "none" else np.ones_like(g)
    off = 0.0 if name in ("none", "relu") else DERIVATIVE
    if dz is not None:
        check_rounded(dz, g * d, 2.0 ** -23, off * np.abs(g), what + ": dz")
    if dbias is not None:
        c = f64(addend) if addend is not None else 0.0
        ref = (g * d).sum(0) + c
        mag = np.abs(g * d).sum(0)
        bound = ((dy.shape[0] / 16 + 48) * 2.0 ** -24 * mag + off * np.abs(g).sum(0)
                 + 2.0 ** -23 * (np.abs(ref) + np.abs(c)) + TINY[torch.float32])
        bad = ~(np.abs(f64(dbias) - ref) <= bound)
        assert not bad.any(), f"{what}: dbias at {np.argwhere(bad)[0]}: {f64(dbias)[bad][0]} for {ref[bad][0]}"


def check_dx(dx, dz, W, residual=None, pre=None, name="none", what="linear_dx"):
    s, mag = product(f64(dz), f64(W))
    err = sum_rel(dz.shape[1]) * mag
    r = f64(residual) if residual is not None else 0.0
    t = s + r
    d = derivative(f64(pre), name) if name != "none" else 1.0
    off = 0.0 if name in ("none", "relu") else DERIVATIVE
    check_rounded(dx, t * d, 2.0 ** -22, np.abs(d) * (err + 2.0 ** -24 * np.abs(t)) + off * (np.abs(t) + err), what)


def check_dw(dw, dz, x, addend=None, what="linear_dw"):
    s, mag = product(f64(dz).T, f64(x))
    c = f64(addend) if addend is not None else 0.0
    err = sum_rel(dz.shape[0], 4096 if dw.dtype == torch.float32 else None) * mag
    check_rounded(dw, s + c, 0.0, err + 2.0 ** -23 * (np.abs(s) + np.abs(c)), what)


# ---------------------------------------------------------------- orthogonalize
def orthogonalized(g, steps, coefficients, eps, scale):
    """All X of the steps in 64 bits, of one matrix."""
    x = np.asarray(g, dtype=np.float64)
    a, b, c = coefficients
    xs = [x / (np.linalg.norm(x) + eps)]
    for _ in range(steps):
        x = xs[-1]
        m = x @ x.T if x.shape[0] <= x.shape[1] else x.T @ x
        p = b * m + c * m @ m
        xs.append(a * x + (p @ x if x.shape[0] <= x.shape[1] else x @ p))
    return xs, scale * xs[-1]


def ortho_bound(xs, coefficients, u0):
    """A bound of the 2-norm of the computed last X's error (over all elements).

    Each step rounds A, B = b A + c A^2 and the new X to fp16: u = 2^-11 of an
    element, or (below fp16's normal range, 2^-14 at the tensors' scales) 2^-25
    of the scale's unit.  The first X is off by u0 (0 where it is exact).  To first
    order, in Frobenius norms, with s the largest singular value of X:
        dA <= u |A| + sum error;  dB <= u |B| + (|b| + 2 |c| s^2) dA;
        dX' <= s dB + u |X'| + sum errors,
    and an error before a step leaves it at most L times as large, L the largest
    of |f(p) -+ f(q)| / |p -+ q| over X's singular values p, q (and f(p)/p), where
    f(p) = a p + b p^3 + c p^5: the derivative of a function of the singular
    values is bounded by its divided differences.  Terms of second order: 1.5.
    """
    a, b, c = coefficients
    u = 2.0 ** -11
    n, m = sorted(xs[0].shape)
    sa = 2.0 ** min(14, math.floor(math.log2(n)))
    sx = 2.0 ** math.floor(math.log2(math.sqrt(m)))
    fro = np.linalg.norm
    err = u0 * fro(xs[0])
    for k, x in enumerate(xs[:-1]):
        w = x if x.shape[0] <= x.shape[1] else x.T
        p = np.linalg.svd(w, compute_uv=False)
        s = p.max()
        A = w @ w.T
        B = b * A + c * A @ A
        dA = u * fro(A) + sum_rel(m) * fro(np.abs(w) @ np.abs(w).T) + 2.0 ** -25 / sa * n
        dB = (u * fro(B) + (abs(b) + 2 * abs(c) * s * s) * dA + abs(c) * sum_rel(n) * fro(np.abs(A) @ np.abs(A))
              + 2.0 ** -25 / sa * n)
        step = s * dB + u * fro(xs[k + 1]) + sum_rel(n) * fro(np.abs(B) @ np.abs(w)) + 2.0 ** -25 / sx * math.sqrt(n * m)
        f = a * p + b * p ** 3 + c * p ** 5
        with np.errstate(divide="ignore", invalid="ignore"):
            d = np.abs(f[:, None] - f[None, :]) / np.abs(p[:, None] - p[None, :])
        d[~np.isfinite(d)] = 0.0
        slope = np.abs(a + 3 * b * p ** 2 + 5 * c * p ** 4)
        L = max(d.max(), slope.max(), (np.abs(f[:, None] + f[None, :]) / (p[:, None] + p[None, :])).max(),
                np.abs(f / p).max())
        err = L * err + step
    return 1.5 * err


def check_ortho(out, g, steps, coefficients, eps, scale, what="orthogonalize"):
    u0 = 2.0 ** -11 if g.dtype == torch.float32 else 0.0
    xs, ref = orthogonalized(f64(g), steps, coefficients, eps, scale)
    bound = abs(scale) * ortho_bound(xs, coefficients, u0) + UNIT[out.dtype] * np.linalg.norm(ref)
    off = np.linalg.norm(f64(out) - ref)
    assert off <= bound, f"{what}: {off:.3e} off, bound {bound:.3e}, of {np.linalg.norm(ref):.3e}"
    return off / max(np.linalg.norm(ref), 1e-300)
