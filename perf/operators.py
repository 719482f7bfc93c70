"""Cases, plain forms and 64-bit forms of the quantised-linear operators.

The operators are those of a linear layer whose weights are held in few bits:

* ``norm``: the residual's addition, the root-mean-square norm and, for the
  8-bit product that follows, e4m3 values with one scale a row;
* ``fp8``: the matrix product of e4m3 activations (a scale a row) and e4m3
  weights (a scale an output column), with a 16-bit result;
* ``w4``: the product of a few rows of 16-bit activations with 4-bit weights
  that carry a scale (and a zero point, where they have one) a group of K.

``run`` computes a case in elementary torch operations in 32 bits, or, with
``own`` set, through stage_software_pipelining_gb300.quant.
"""
import math

import torch

own = False

E4M3_MAX = 448.0
SCALE_MIN = 2.0 ** -126          # a scale never underflows, so that 1/scale is finite
EPS = 1e-6
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def listed():
    return [
        # one token of a decoding step: the 16-bit row that a 4-bit product reads
        {"name": "norm_1x4096_bf16", "op": "norm", "rows": 1, "cols": 4096, "type": "bf16", "outs": "y"},
        # a decoding batch in front of an 8-bit product
        {"name": "norm_37x8192_f16", "op": "norm", "rows": 37, "cols": 8192, "type": "f16", "outs": "q"},
        # odd rows of an odd width, in 32 bits, all outputs
        {"name": "norm_1021x1999_f32", "op": "norm", "rows": 1021, "cols": 1999, "type": "f32", "outs": "yq"},
        # a long prompt in front of an 8-bit product
        {"name": "norm_8191x8192_bf16", "op": "norm", "rows": 8191, "cols": 8192, "type": "bf16", "outs": "q"},
        # one token through an 8-bit layer: the weights are read once
        {"name": "fp8_1x4096x4096_bf16", "op": "fp8", "M": 1, "N": 4096, "K": 4096, "type": "bf16"},
        # a decoding batch through a wide 8-bit layer
        {"name": "fp8_48x28672x4096_f16", "op": "fp8", "M": 48, "N": 28672, "K": 4096, "type": "f16"},
        # a short prompt through a square layer
        {"name": "fp8_2048x2048x2048_f16", "op": "fp8", "M": 2048, "N": 2048, "K": 2048, "type": "f16"},
        # a long prompt through a wide layer, its rows not a multiple of a tile
        {"name": "fp8_8191x28672x4096_bf16", "op": "fp8", "M": 8191, "N": 28672, "K": 4096, "type": "bf16"},
        # one token through a square 4-bit layer
        {"name": "w4_1x4096x4096_g128_bf16", "op": "w4", "M": 1, "N": 4096, "K": 4096, "group": 128,
         "zeros": False, "type": "bf16"},
        # one token through a wide 4-bit layer with zero points
        {"name": "w4_1x28672x8192_g64_f16", "op": "w4", "M": 1, "N": 28672, "K": 8192, "group": 64,
         "zeros": True, "type": "f16"},
        # a few sequences, an odd number of outputs, the smallest groups
        {"name": "w4_5x4099x8192_g32_bf16", "op": "w4", "M": 5, "N": 4099, "K": 8192, "group": 32,
         "zeros": True, "type": "bf16"},
        # the largest batch of the single-token form, long K
        {"name": "w4_32x8192x28672_g128_f16", "op": "w4", "M": 32, "N": 8192, "K": 28672, "group": 128,
         "zeros": False, "type": "f16"},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("norm", "fp8", "w4"))
    if op == "norm":
        case = {"op": op, "rows": _log(rng, 1, 8192), "cols": _log(rng, 32, 16384),
                "type": rng.choice(("bf16", "f16", "f32")), "outs": rng.choice(("y", "q", "yq"))}
        if rng.random() < 0.5:      # half of the widths are whole vectors, as a model's are
            case["cols"] = (case["cols"] + 31) // 32 * 32
        if case["type"] == "f32":
            case["rows"] = min(case["rows"], 4096)
        return case
    if op == "fp8":
        case = {"op": op, "M": _log(rng, 1, 8192), "N": _log(rng, 64, 28672), "K": _log(rng, 32, 8192),
                "type": rng.choice(("bf16", "f16"))}
        while case["M"] * case["N"] * case["K"] > 8191 * 28672 * 4096:
            case["M"] = (case["M"] + 1) // 2
        if rng.random() < 0.5:
            case["N"] = (case["N"] + 63) // 64 * 64
            case["K"] = (case["K"] + 127) // 128 * 128
        return case
    group = rng.choice((32, 64, 128))
    return {"op": op, "M": _log(rng, 1, 32), "N": _log(rng, 64, 28672),
            "K": group * _log(rng, 1, 8192 // group), "group": group,
            "zeros": rng.random() < 0.5, "type": rng.choice(("bf16", "f16"))}


def _padded(rows, cols, dtype):
    """rows x cols whose rows start on 16-byte boundaries, as the library asks."""
    unit = 16 // torch.empty((), dtype=dtype).element_size()
    return torch.empty((rows, (cols + unit - 1) // unit * unit), dtype=dtype, device="cuda")[:, :cols]


def _quantised_rows(v):
    """e4m3 values (rows on 16-byte boundaries) and one scale a row of an fp32 matrix."""
    scale = (v.abs().amax(dim=1) / E4M3_MAX).clamp_min(SCALE_MIN)
    q = _padded(v.shape[0], v.shape[1], torch.float8_e4m3fn)
    q.copy_((v / scale[:, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn))
    return q, scale


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    dt = TYPES[case["type"]]

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)

    state = dict(case)
    if case["op"] == "norm":
        T, D = case["rows"], case["cols"]
        # a layer's output, and a residual stream that some channels dominate
        loud = torch.where(torch.rand(D, generator=g, device="cuda") < 0.01, 20.0, 1.0)
        state["x"] = normal(T, D).mul_(0.5).to(dt)
        state["residual"] = normal(T, D).mul_(loud).to(dt)
        state["weight"] = normal(D).mul_(0.2).add_(1.0).to(dt)
        state["residual_out"] = torch.empty(T, D, device="cuda", dtype=dt)
        state["y"] = torch.empty(T, D, device="cuda", dtype=dt) if "y" in case["outs"] else None
        state["q"] = _padded(T, D, torch.float8_e4m3fn) if "q" in case["outs"] else None
        state["scale"] = torch.empty(T, device="cuda") if "q" in case["outs"] else None
    elif case["op"] == "fp8":
        M, N, K = case["M"], case["N"], case["K"]
        state["A"], state["a_scale"] = _quantised_rows(normal(M, K))
        state["W"], state["w_scale"] = _quantised_rows(normal(N, K).mul_(0.02))
        state["C"] = _padded(M, N, dt)
    else:
        M, N, K, G = case["M"], case["N"], case["K"], case["group"]
        state["x"] = normal(M, K).to(dt)
        state["W"] = torch.randint(0, 256, (N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
        state["scales"] = torch.rand(N, K // G, generator=g, device="cuda").mul_(0.004).add_(0.002).to(dt)
        state["zeros"] = torch.randint(5, 11, (N, K // G), generator=g, device="cuda",
                                       dtype=torch.uint8) if case["zeros"] else None
        state["C"] = torch.empty(M, N, device="cuda", dtype=dt)
    return state


def _run_own(s):
    from stage_software_pipelining_gb300 import quant as Q
    if s["op"] == "norm":
        Q.add_rmsnorm(s["x"], s["weight"], s["residual"], eps=EPS, residual_out=s["residual_out"],
                      y=s["y"], q=s["q"], scale=s["scale"])
        return {k: s[k] for k in ("residual_out", "y", "q", "scale") if s[k] is not None}
    if s["op"] == "fp8":
        return Q.gemm_fp8(s["A"], s["W"].t(), s["C"], s["a_scale"], s["w_scale"])
    return Q.gemv_w4(s["x"], s["W"], s["scales"], s["C"], zeros=s["zeros"])


def run(s):
    if own:
        return _run_own(s)
    dt = TYPES[s["type"]]
    if s["op"] == "norm":
        h = s["x"].float() + s["residual"].float()
        y = h * torch.rsqrt((h * h).mean(dim=1, keepdim=True) + EPS) * s["weight"].float()
        out = {"residual_out": h.to(dt)}
        if "y" in s["outs"]:
            out["y"] = y.to(dt)
        if "q" in s["outs"]:
            scale = (y.abs().amax(dim=1) / E4M3_MAX).clamp_min(SCALE_MIN)
            out["scale"] = scale
            out["q"] = (y / scale[:, None]).to(torch.float8_e4m3fn)
        return out
    if s["op"] == "fp8":
        c = s["A"].float() @ s["W"].float().t()
        return (c * s["a_scale"][:, None] * s["w_scale"][None, :]).to(dt)
    N, G = s["W"].shape[0], s["group"]
    w = torch.stack((s["W"] & 15, s["W"] >> 4), dim=2).reshape(N, -1, G).float()
    w = w - (s["zeros"].float()[:, :, None] if s["zeros"] is not None else 8.0)
    w = (w * s["scales"].float()[:, :, None]).reshape(N, -1)
    return (s["x"].float() @ w.t()).to(dt)


def work(case):
    size = {"bf16": 2, "f16": 2, "f32": 4}[case["type"]]
    if case["op"] == "norm":
        T, D = case["rows"], case["cols"]
        b = 3 * T * D * size + D * size
        b += T * D * size if "y" in case["outs"] else 0
        b += T * D + 4 * T if "q" in case["outs"] else 0
        return {"bytes": b, "flops": 8 * T * D}
    M, N, K = case["M"], case["N"], case["K"]
    if case["op"] == "fp8":
        return {"bytes": M * K + N * K + 4 * (M + N) + M * N * size, "flops": 2 * M * N * K}
    groups = N * (K // case["group"])
    return {"bytes": N * K // 2 + groups * (size + (1 if case["zeros"] else 0)) + M * K * size + M * N * size,
            "flops": 2 * M * N * K}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        h = s["x"].double().add_(s["residual"].double())
        norm = torch.linalg.vector_norm(h, dim=1, keepdim=True)
        y = (h / torch.sqrt(norm ** 2 / case["cols"] + EPS)) * s["weight"].double()
        out = {"residual_out": h}
        if "y" in case["outs"]:
            out["y"] = y
        if "q" in case["outs"]:
            out["scale"] = torch.maximum(y.max(dim=1).values, -y.min(dim=1).values).div(E4M3_MAX)
            out["q"] = y / out["scale"].unsqueeze(1)
        return out
    if case["op"] == "fp8":
        a = s["A"].double().mul_(s["a_scale"].double().unsqueeze(1))
        w = s["W"].double().mul_(s["w_scale"].double().unsqueeze(1))
        return torch.mm(a, w.t())
    low, high = (s["W"] % 16).double(), (s["W"] // 16).double()
    spread = case["group"] // 2
    zero = s["zeros"].double().repeat_interleave(spread, dim=1) if case["zeros"] else 8.0
    scale = s["scales"].double().repeat_interleave(spread, dim=1)
    x = s["x"].double()
    return torch.mm(x[:, 0::2], ((low - zero) * scale).t()) + torch.mm(x[:, 1::2], ((high - zero) * scale).t())
