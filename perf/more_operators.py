"""Cases, plain forms and 64-bit forms of the operators that train a 16-bit linear layer.

* ``linear``: y = act(x W^T + bias) + residual, with z = x W^T + bias kept for
  the backward pass where it is asked for; one token to a long batch;
* ``act``: dz = dy act'(z) and the bias gradient, the sum of dz's columns;
* ``dx``: (dz W + residual) act'(z), the gradient handed to the layer below;
* ``dw``: dz^T x + addend, the weight gradient, added to what earlier
  micro-batches left;
* ``ortho``: that gradient's update with all singular values brought near one
  by Newton-Schulz steps, X <- a X + (b X X^T + c (X X^T)^2) X.

``run`` computes a case in elementary torch operations in 32 bits, or, with
``own`` set, through stage_software_pipelining_gb300.linear.
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")
EPS = 1e-7
STEPS = 5
COEFFICIENTS = (3.4445, -4.7750, 2.0315)
GELU_C = math.sqrt(2.0 / math.pi)


def listed():
    return [
        # one token's projection back into the residual stream
        {"name": "linear_1x4096x4096_bf16", "op": "linear", "M": 1, "N": 4096, "K": 4096, "type": "bf16",
         "act": "none", "bias": False, "residual": True, "pre": False},
        # a decoding batch through a wide layer with its activation
        {"name": "linear_48x28672x4096_f16", "op": "linear", "M": 48, "N": 28672, "K": 4096, "type": "f16",
         "act": "gelu_tanh", "bias": True, "residual": False, "pre": False},
        # a short training batch, z kept for the backward pass
        {"name": "linear_2048x2048x2048_f16", "op": "linear", "M": 2048, "N": 2048, "K": 2048, "type": "f16",
         "act": "gelu", "bias": True, "residual": False, "pre": True},
        # a long training batch through a wide layer, its rows not a multiple of a tile
        {"name": "linear_8191x28672x4096_bf16", "op": "linear", "M": 8191, "N": 28672, "K": 4096, "type": "bf16",
         "act": "silu", "bias": True, "residual": False, "pre": True},
        # the smallest backward call: a few rows of an odd width
        {"name": "act_61x1000_f16", "op": "act", "M": 61, "N": 1000, "type": "f16", "act": "gelu", "dbias": True},
        # a long batch's gradient back through its activation
        {"name": "act_8192x8192_bf16", "op": "act", "M": 8192, "N": 8192, "type": "bf16", "act": "gelu_tanh",
         "dbias": True},
        # a short batch's gradient through a layer and the activation below it
        {"name": "dx_2048x2048x2048_f16", "op": "dx", "M": 2048, "N": 2048, "K": 2048, "type": "f16",
         "act": "gelu", "residual": False},
        # a long batch's gradient through a layer, joined with the residual stream's
        {"name": "dx_8191x8192x4096_bf16", "op": "dx", "M": 8191, "N": 8192, "K": 4096, "type": "bf16",
         "act": "none", "residual": True},
        # many tokens into a small weight: few tiles, a long sum
        {"name": "dw_32768x1024x1024_f16", "op": "dw", "M": 32768, "N": 1024, "K": 1024, "type": "f16",
         "out": "f32", "addend": False},
        # a long batch's weight gradient, added to the earlier micro-batches'
        {"name": "dw_8192x8192x4096_bf16", "op": "dw", "M": 8192, "N": 8192, "K": 4096, "type": "bf16",
         "out": "f32", "addend": True},
        # the update of a few small tall weights at once, where launches count
        {"name": "ortho_6x2048x512_bf16", "op": "ortho", "B": 6, "R": 2048, "C": 512, "type": "bf16", "out": "bf16"},
        # the update of one large weight
        {"name": "ortho_1x4096x8192_f32", "op": "ortho", "B": 1, "R": 4096, "C": 8192, "type": "f32", "out": "bf16"},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("linear", "act", "dx", "dw", "ortho"))
    case = {"op": op, "type": rng.choice(("bf16", "f16"))}
    if op == "ortho":
        case |= {"type": rng.choice(("bf16", "f16", "f32")), "B": _log(rng, 1, 8), "R": _log(rng, 16, 8192),
                 "C": _log(rng, 16, 8192), "out": rng.choice(("bf16", "f16"))}
        while case["B"] * case["R"] * case["C"] * min(case["R"], case["C"]) > 4096 * 4096 * 8192:
            if case["B"] > 1:
                case["B"] -= 1
            else:
                case["C"] = (case["C"] + 1) // 2
        return case
    case["M"] = _log(rng, 1, 32768 if op in ("act", "dw") else 8192)
    case["N"] = _log(rng, 64, 28672 if op in ("linear", "act") else 8192)
    if op == "act":
        while case["M"] * case["N"] > 8192 * 28672:
            case["M"] = (case["M"] + 1) // 2
        return case | {"act": rng.choice(ACTS[1:]), "dbias": rng.random() < 0.7}
    case["K"] = _log(rng, 32, 8192)
    while case["M"] * case["N"] * case["K"] > 8191 * 28672 * 4096:
        case["M"] = (case["M"] + 1) // 2
    if rng.random() < 0.5:      # half of the widths are whole vectors, as a model's are
        case["N"] = (case["N"] + 63) // 64 * 64
        case["K"] = (case["K"] + 63) // 64 * 64
    if op == "linear":
        return case | {"act": rng.choice(ACTS), "bias": rng.random() < 0.5, "residual": rng.random() < 0.3,
                       "pre": rng.random() < 0.5}
    if op == "dx":
        return case | {"act": rng.choice(ACTS), "residual": rng.random() < 0.5}
    return case | {"out": rng.choice(("f32", case["type"])), "addend": rng.random() < 0.5}


def _padded(rows, cols, dtype):
    """rows x cols whose rows start on 16-byte boundaries, as the library asks."""
    unit = 16 // torch.empty((), dtype=dtype).element_size()
    return torch.empty((rows, (cols + unit - 1) // unit * unit), dtype=dtype, device="cuda")[:, :cols]


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    dt = TYPES[case["type"]]

    def normal(rows, cols, std, dtype=dt):
        t = _padded(rows, cols, dtype)
        t.copy_(torch.randn((rows, cols), generator=g, device="cuda").mul_(std))
        return t

    s = dict(case)
    if case["op"] == "ortho":
        B, R, C = case["B"], case["R"], case["C"]
        # a gradient: a fast decaying part over many small directions
        unit = 16 // torch.empty((), dtype=dt).element_size()
        grad = torch.empty((B, R, (C + unit - 1) // unit * unit), dtype=dt, device="cuda")[:, :, :C]
        r = min(R, C, 64)
        loud = torch.randn((B, R, r), generator=g, device="cuda") * 0.9 ** torch.arange(r, device="cuda")
        low = loud @ torch.randn((B, r, C), generator=g, device="cuda")
        grad.copy_((torch.randn((B, R, C), generator=g, device="cuda") + 0.5 * low).mul_(1e-3))
        s["g"] = grad
        s["scale"] = math.sqrt(max(1.0, R / C))
        to = TYPES[case["out"]]
        s["o"] = torch.empty((B, R, (C + 7) // 8 * 8), dtype=to, device="cuda")[:, :, :C]
        # the room that a program keeps for its updates: as many bytes as eight 16-bit
        # copies of the weights and four of their smaller squares, and a page
        small = min(R, C)
        s["workspace"] = torch.empty(B * (8 * (R + 8) * (C + 8) + 8 * (small + 8) ** 2) + 65536, dtype=torch.uint8,
                                     device="cuda")
        return s
    M, N = case["M"], case["N"]
    if case["op"] == "act":
        s["dy"] = normal(M, N, 1e-2)
        s["z"] = normal(M, N, 1.5)
        s["dz"] = _padded(M, N, dt)
        s["db"] = torch.empty(N, device="cuda") if case["dbias"] else None
        return s
    K = case["K"]
    if case["op"] == "linear":
        s["x"] = normal(M, K, 1.0)
        s["W"] = normal(N, K, 1.5 * K ** -0.5)
        s["b"] = normal(1, N, 0.5)[0] if case["bias"] else None
        s["r"] = normal(M, N, 2.0) if case["residual"] else None
        s["z"] = _padded(M, N, dt) if case["pre"] else None
        s["y"] = _padded(M, N, dt)
    elif case["op"] == "dx":
        s["dz"] = normal(M, N, 1e-2)
        s["W"] = normal(N, K, N ** -0.5)
        s["r"] = normal(M, K, 1e-2) if case["residual"] else None
        s["z"] = normal(M, K, 1.5) if case["act"] != "none" else None
        s["dx"] = _padded(M, K, dt)
    else:
        to = TYPES[case["out"]]
        s["dz"] = normal(M, N, 1e-2)
        s["x"] = normal(M, K, 1.0)
        s["c"] = normal(N, K, 1e-2 * M ** 0.5, to) if case["addend"] else None
        s["dw"] = _padded(N, K, to)
    return s


def _run_own(s):
    from stage_software_pipelining_gb300 import linear as L
    if s["op"] == "linear":
        L.linear(s["x"], s["W"], s["y"], bias=s["b"], residual=s["r"], act=s["act"], pre=s["z"])
        return {"y": s["y"], "z": s["z"]} if s["pre"] else {"y": s["y"]}
    if s["op"] == "act":
        L.act_grad(s["dy"], s["dz"], pre=s["z"], act=s["act"], dbias=s["db"])
        return {"dz": s["dz"], "db": s["db"]} if s["dbias"] else {"dz": s["dz"]}
    if s["op"] == "dx":
        return L.linear_dx(s["dz"], s["W"], s["dx"], residual=s["r"], act=s["act"], pre=s["z"])
    if s["op"] == "dw":
        return L.linear_dw(s["dz"], s["x"], s["dw"], addend=s["c"])
    return L.orthogonalize(s["g"], s["o"], s["workspace"], steps=STEPS, coefficients=COEFFICIENTS, eps=EPS,
                           scale=s["scale"])


def _act(z, act):
    if act == "relu":
        return z * (z > 0)
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(GELU_C * (z + 0.044715 * z * z * z)))
    if act == "silu":
        return z / (1 + torch.exp(-z))
    return z


def _act_grad(z, act):
    if act == "relu":
        return (z > 0).float()
    if act == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    if act == "gelu_tanh":
        t = torch.tanh(GELU_C * (z + 0.044715 * z * z * z))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * GELU_C * (1 + 3 * 0.044715 * z * z)
    p = 1 / (1 + torch.exp(-z))
    return p * (1 + z * (1 - p))


def run(s):
    if own:
        return _run_own(s)
    dt = TYPES[s["type"]]
    if s["op"] == "linear":
        z = s["x"].float() @ s["W"].float().t()
        if s["b"] is not None:
            z = z + s["b"].float()
        y = _act(z, s["act"])
        if s["r"] is not None:
            y = y + s["r"].float()
        return {"y": y.to(dt), "z": z.to(dt)} if s["pre"] else {"y": y.to(dt)}
    if s["op"] == "act":
        dz = s["dy"].float() * _act_grad(s["z"].float(), s["act"])
        # in 64 bits: sums of tens of thousands of values that cancel
        return {"dz": dz.to(dt), "db": dz.double().sum(0).float()} if s["dbias"] else {"dz": dz.to(dt)}
    if s["op"] == "dx":
        dx = s["dz"].float() @ s["W"].float()
        if s["r"] is not None:
            dx = dx + s["r"].float()
        if s["act"] != "none":
            dx = dx * _act_grad(s["z"].float(), s["act"])
        return dx.to(dt)
    if s["op"] == "dw":
        dw = s["dz"].float().t() @ s["x"].float()
        if s["c"] is not None:
            dw = dw + s["c"].float()
        return dw.to(TYPES[s["out"]])
    x = s["g"].float()
    tall = s["R"] > s["C"]
    if tall:
        x = x.transpose(1, 2)
    x = x / (torch.sqrt((x.double() * x.double()).sum((1, 2), keepdim=True)).float() + EPS)
    a, b, c = COEFFICIENTS
    for _ in range(STEPS):
        m = x @ x.transpose(1, 2)
        x = a * x + (b * m + c * (m @ m)) @ x
    x = x * s["scale"]
    return (x.transpose(1, 2) if tall else x).to(TYPES[s["out"]])


def work(case):
    size = {"bf16": 2, "f16": 2, "f32": 4}
    e = size[case["type"]]
    if case["op"] == "ortho":
        B, n, m = case["B"], min(case["R"], case["C"]), max(case["R"], case["C"])
        # X X^T and its square are symmetric: half of each is all there is to compute
        return {"bytes": B * n * m * (e + size[case["out"]]), "flops": STEPS * B * (3 * n * n * m + n * n * n)}
    M, N = case["M"], case["N"]
    if case["op"] == "act":
        return {"bytes": 3 * M * N * e + (4 * N if case["dbias"] else 0), "flops": 20 * M * N}
    K = case["K"]
    if case["op"] == "linear":
        b = e * (M * K + N * K + M * N * (1 + case["residual"] + case["pre"]) + N * case["bias"])
    elif case["op"] == "dx":
        b = e * (M * N + N * K + M * K * (1 + case["residual"] + (case["act"] != "none")))
    else:
        b = e * (M * N + M * K) + size[case["out"]] * N * K * (1 + case["addend"])
    return {"bytes": b, "flops": 2 * M * N * K}


def _phi(z):
    """The normal distribution's share below z."""
    return torch.special.erfc(z.mul(-math.sqrt(0.5))).mul_(0.5)


def _exact_act(z, act):
    return {"none": lambda: z, "relu": lambda: z.clamp_min(0), "gelu": lambda: z * _phi(z),
            "gelu_tanh": lambda: z * torch.sigmoid(2 * GELU_C * (z + 0.044715 * z ** 3)),
            "silu": lambda: z * torch.sigmoid(z)}[act]()


def _exact_slope(z, act):
    if act == "relu":
        return torch.where(z > 0, 1.0, 0.0).double()
    if act == "gelu":
        return _phi(z) + z * torch.exp(-z ** 2 / 2) * (2 * math.pi) ** -0.5
    if act == "gelu_tanh":
        p = torch.sigmoid(2 * GELU_C * (z + 0.044715 * z ** 3))
        return p + z * p * (1 - p) * 2 * GELU_C * (1 + 0.134145 * z ** 2)
    if act == "silu":
        p = torch.sigmoid(z)
        return p + z * p * (1 - p)
    return torch.ones_like(z)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "linear":
        z = torch.mm(s["x"].double(), s["W"].double().t())
        if case["bias"]:
            z += s["b"].double()
        y = _exact_act(z, case["act"])
        if case["residual"]:
            y = y + s["r"].double()
        return {"y": y, "z": z} if case["pre"] else {"y": y}
    if case["op"] == "act":
        dz = _exact_slope(s["z"].double(), case["act"]).mul_(s["dy"].double())
        if not case["dbias"]:
            return {"dz": dz}
        return {"dz": dz, "db": torch.mv(dz.t(), torch.ones(case["M"], dtype=torch.float64, device="cuda"))}
    if case["op"] == "dx":
        dx = torch.mm(s["dz"].double(), s["W"].double())
        if case["residual"]:
            dx += s["r"].double()
        return dx * _exact_slope(s["z"].double(), case["act"]) if case["act"] != "none" else dx
    if case["op"] == "dw":
        dw = torch.mm(s["dz"].double().t(), s["x"].double())
        return dw + s["c"].double() if case["addend"] else dw
    # The steps act on singular values alone: on the smaller Gram matrix G they are
    # X P with P <- P (a + b (P G P) + c (P G P)^2), polynomials of G that commute.
    x = s["g"].double()
    wide = case["R"] <= case["C"]
    norm = torch.linalg.vector_norm(x, dim=(1, 2), keepdim=True) + EPS
    x.div_(norm)
    gram = torch.bmm(x, x.mT) if wide else torch.bmm(x.mT, x)
    eye = torch.eye(gram.shape[1], dtype=torch.float64, device="cuda").expand_as(gram)
    a, b, c = COEFFICIENTS
    p, lam = eye, gram
    for k in range(STEPS):
        q = torch.baddbmm(b * lam + a * eye, lam, lam, beta=1.0, alpha=c)
        p = torch.bmm(p, q)
        if k + 1 < STEPS:
            lam = torch.bmm(torch.bmm(q, lam), q)
    return s["scale"] * (torch.bmm(p, x) if wide else torch.bmm(x, p))
