"""The operators of a pre-norm MLP block, as cases to time: layer norm, the matrix product with
bias, activation and residual in its epilogue, and the same product grouped by expert over ragged
row counts; each forward, and backward with the gradients of everything that has one.

`run` computes them in a plain form (elementary torch operations in 32 bits, rounded once) or, with
`own` set, through the package's entry points.
"""
import math

import numpy as np
import torch

own = False

EPS = 1e-5
BF16, F32 = torch.bfloat16, torch.float32


# ----------------------------------------------------------------------------------- cases --
def listed():
    return [
        # The norm in front of the block for one token of a decoding sequence: latency only.
        {"name": "norm_token", "op": "norm", "rows": 1, "cols": 4096, "dtype": "bf16"},
        # The norm over a prefill batch, the largest forward call.
        {"name": "norm_prefill", "op": "norm", "rows": 2048, "cols": 8192, "dtype": "bf16"},
        # Training: the gradient of the norm, joined with the gradient of the skip connection.
        {"name": "norm_grad", "op": "norm_grad", "rows": 4096, "cols": 8192, "dtype": "bf16", "skip": True},
        # A small model trained in 32 bits with a width that no vector divides.
        {"name": "norm_grad_odd_f32", "op": "norm_grad", "rows": 333, "cols": 1357, "dtype": "f32", "skip": False},
        # Up-projection of one token: the weights are read once, nothing else counts.
        {"name": "linear_token", "op": "linear", "rows": 1, "K": 4096, "N": 14336, "act": "gelu", "layout": "kn",
         "residual": False, "save": False},
        # A decoding batch of 128 sequences through a square projection, weights stored N x K.
        {"name": "linear_batch", "op": "linear", "rows": 128, "K": 4096, "N": 4096, "act": "none", "layout": "nk",
         "residual": True, "save": False},
        # Down-projection of a short prompt of odd length, with the block's residual.
        {"name": "linear_prompt", "op": "linear", "rows": 301, "K": 14336, "N": 4096, "act": "none", "layout": "kn",
         "residual": True, "save": False},
        # The forward pass of a training step: the pre-activation is kept for the backward pass.
        {"name": "linear_train", "op": "linear", "rows": 2048, "K": 8192, "N": 8192, "act": "gelu", "layout": "kn",
         "residual": False, "save": True},
        # Its backward pass: gradients of the input, the weights and the bias.
        {"name": "linear_grad", "op": "linear_grad", "rows": 2048, "K": 8192, "N": 8192, "act": "gelu",
         "layout": "kn"},
        # Eight sequences decode one token each, two experts of eight per token: a few rows an expert.
        {"name": "experts_tokens", "op": "experts", "rows": 16, "experts": 8, "K": 4096, "N": 14336, "act": "silu",
         "layout": "kn", "route": 9},
        # A prefill of 2048 tokens, two experts each: large products of ragged height.
        {"name": "experts_prefill", "op": "experts", "rows": 4096, "experts": 8, "K": 4096, "N": 14336,
         "act": "gelu", "layout": "kn", "route": 8},
        # Training with many smaller experts, some of which get no row: all gradients.
        {"name": "experts_grad", "op": "experts_grad", "rows": 4000, "experts": 32, "K": 2048, "N": 4096,
         "act": "gelu", "layout": "kn", "route": 3},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _log_int8(rng, lo, hi):
    return 8 * max(1, _log_int(rng, lo, hi) // 8)


def draw(rng):
    op = rng.choice(["norm", "norm_grad", "linear", "linear", "linear_grad", "experts", "experts", "experts_grad"])
    if op in ("norm", "norm_grad"):
        case = {"op": op, "rows": _log_int(rng, 1, 8192), "cols": _log_int(rng, 64, 16384),
                "dtype": rng.choice(["bf16", "bf16", "f32"])}
        while case["rows"] * case["cols"] > 4096 * 8192:
            case["rows"] = case["rows"] // 2
        if op == "norm_grad":
            case["skip"] = rng.random() < 0.5
        return case
    act = rng.choice(["none", "gelu", "silu", "relu"])
    layout = rng.choice(["kn", "kn", "nk"])
    if op.startswith("linear"):
        case = {"op": op, "rows": _log_int(rng, 1 if op == "linear" else 16, 4096), "K": _log_int8(rng, 256, 14336),
                "N": _log_int8(rng, 256, 14336), "act": act, "layout": layout}
        if op == "linear":
            case["residual"] = rng.random() < 0.5
            case["save"] = rng.random() < 0.3
    else:
        case = {"op": op, "rows": _log_int(rng, 8, 4096), "experts": _log_int(rng, 4, 64), "K": _log_int8(rng, 256, 8192),
                "N": _log_int8(rng, 256, 8192), "act": act, "layout": layout, "route": rng.randrange(1, 1000)}
        while case["experts"] * case["K"] * case["N"] > 32 * 2048 * 4096:
            case["experts"] = max(case["experts"] // 2, 4)
            case["K"] = max(case["K"] // 16 * 8, 256)
    while case["rows"] * case["K"] * case["N"] > 2048 * 8192 * 8192:
        case["rows"] = case["rows"] // 2
    return case


def _sizes(case):
    """Rows of each expert: uneven popularity, some experts without a row; the same for every seed."""
    r = np.random.RandomState(case["route"])
    p = r.gamma(3.0, size=case["experts"])
    p[r.rand(case["experts"]) < 0.1] = 0.0
    if p.sum() == 0.0:
        p[0] = 1.0
    return [int(v) for v in r.multinomial(case["rows"], p / p.sum())]


# ---------------------------------------------------------------------------------- inputs --
def _normal(gen, shape, std, dtype):
    return (torch.randn(shape, generator=gen, device="cuda", dtype=F32) * std).to(dtype)


def _inputs(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed * 1000003 + 17)
    s = {}
    if case["op"] in ("norm", "norm_grad"):
        dt = BF16 if case["dtype"] == "bf16" else F32
        R, C = case["rows"], case["cols"]
        # a residual stream: spread over rows, an offset, and a few channels far larger than the rest
        x = torch.randn((R, C), generator=gen, device="cuda", dtype=F32) * 1.5 + 0.25
        x[:, torch.randint(0, C, (max(C // 512, 1),), generator=gen, device="cuda")] *= 20.0
        s["x"] = x.to(dt)
        s["gamma"] = (1.0 + torch.randn(C, generator=gen, device="cuda", dtype=F32) * 0.1).to(dt)
        s["beta"] = _normal(gen, C, 0.1, dt)
        if case["op"] == "norm_grad":
            d = s["x"].float()
            s["mean"] = d.mean(dim=1)
            s["rstd"] = torch.rsqrt((d - s["mean"][:, None]).square().mean(dim=1) + EPS)
            s["dy"] = _normal(gen, (R, C), 1.0 / 16, dt)
            s["skip"] = _normal(gen, (R, C), 1.0 / 16, dt) if case["skip"] else None
        return s
    R, K, N = case["rows"], case["K"], case["N"]
    lead = (case["experts"],) if "experts" in case else ()
    s["X"] = _normal(gen, (R, K), 1.0, BF16)
    s["W"] = _normal(gen, lead + ((K, N) if case["layout"] == "kn" else (N, K)), K ** -0.5, BF16)
    if lead:
        s["sizes"] = _sizes(case)
        s["offsets"] = torch.tensor(np.concatenate([[0], np.cumsum(s["sizes"])]), dtype=torch.int32, device="cuda")
    if case["op"].endswith("_grad"):
        # X ~ N(0, 1) and W ~ N(0, 1/K) make a pre-activation ~ N(0, 1)
        s["Z"] = _normal(gen, (R, N), 1.0, BF16) if case["act"] != "none" else None
        s["dY"] = _normal(gen, (R, N), 1.0 / 16, BF16)
    else:
        s["bias"] = _normal(gen, lead + (N,), 0.1, BF16)
        s["residual"] = _normal(gen, (R, N), 1.0, BF16) if case.get("residual") else None
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    if not own:
        return s
    import mlp_latency_gb300 as mc

    op = case["op"]
    if op in ("norm", "norm_grad"):
        s["out"] = torch.empty_like(s["x"])
        if op == "norm":
            s["mean"] = torch.empty(case["rows"], dtype=F32, device="cuda")
            s["rstd"] = torch.empty(case["rows"], dtype=F32, device="cuda")
        else:
            s["dgamma"], s["dbeta"] = torch.empty_like(s["gamma"]), torch.empty_like(s["gamma"])
            s["ws"] = torch.empty(max(mc.layer_norm_workspace_size(case["rows"], case["cols"]), 256),
                                  dtype=torch.uint8, device="cuda")
        return s
    s["linear"] = mc.Linear(case["K"], case["N"], activation=case["act"], experts=case.get("experts", 0),
                            weight_layout=case["layout"])
    s["ws"] = torch.empty(max(s["linear"].workspace_size(case["rows"]), 256), dtype=torch.uint8, device="cuda")
    if op.endswith("_grad"):
        s["dX"], s["dW"] = torch.empty_like(s["X"]), torch.empty_like(s["W"])
        s["dbias"] = torch.empty(s["W"].shape[:-2] + (case["N"],), dtype=BF16, device="cuda")
    else:
        s["Y"] = torch.empty((case["rows"], case["N"]), dtype=BF16, device="cuda")
        s["Z"] = torch.empty_like(s["Y"]) if case.get("save") else None
    return s


# ------------------------------------------------------------------------------ plain forms --
def _act(act, z):
    if act == "none":
        return z
    if act == "relu":
        return torch.clamp_min(z, 0.0)
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    u = math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)
    return 0.5 * z * (1.0 + torch.tanh(u))


def _act_grad(act, z):
    if act == "relu":
        return (z > 0.0).to(z.dtype)
    if act == "silu":
        sg = 1.0 / (1.0 + torch.exp(-z))
        return sg * (1.0 + z * (1.0 - sg))
    c = math.sqrt(2.0 / math.pi)
    t = torch.tanh(c * (z + 0.044715 * z * z * z))
    return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * c * (1.0 + 3.0 * 0.044715 * z * z)


def _plain_norm(s):
    x = s["x"].float()
    mean = x.mean(dim=1)
    d = x - mean[:, None]
    rstd = 1.0 / torch.sqrt((d * d).mean(dim=1) + EPS)
    y = d * rstd[:, None] * s["gamma"].float() + s["beta"].float()
    return {"y": y.to(s["x"].dtype), "mean": mean, "rstd": rstd}


def _plain_norm_grad(s):
    dt = s["x"].dtype
    dy = s["dy"].float()
    xh = (s["x"].float() - s["mean"][:, None]) * s["rstd"][:, None]
    g = dy * s["gamma"].float()
    dx = (g - g.mean(dim=1, keepdim=True) - xh * (g * xh).mean(dim=1, keepdim=True)) * s["rstd"][:, None]
    if s["skip"] is not None:
        dx = dx + s["skip"].float()
    return {"dx": dx.to(dt), "dgamma": (dy * xh).sum(dim=0).to(dt), "dbeta": dy.sum(dim=0).to(dt)}


def _groups(s):
    """(row slice, expert) of every expert; the dense product is one group."""
    if "sizes" not in s:
        return [(slice(0, s["case"]["rows"]), None)]
    out, r0 = [], 0
    for e, n in enumerate(s["sizes"]):
        out.append((slice(r0, r0 + n), e))
        r0 += n
    return out


def _plain_linear(s):
    case = s["case"]
    Y = torch.empty((case["rows"], case["N"]), dtype=BF16, device="cuda")
    Z = torch.empty_like(Y) if case.get("save") else None
    for rows, e in _groups(s):
        W, b = (s["W"], s["bias"]) if e is None else (s["W"][e], s["bias"][e])
        z = s["X"][rows].float() @ (W.float() if case["layout"] == "kn" else W.float().t()) + b.float()
        y = _act(case["act"], z)
        if s["residual"] is not None:
            y = y + s["residual"][rows].float()
        Y[rows] = y.to(BF16)
        if Z is not None:
            Z[rows] = z.to(BF16)
    return {"Y": Y} if Z is None else {"Y": Y, "Z": Z}


def _plain_linear_grad(s):
    case = s["case"]
    dX, dW = torch.empty_like(s["X"]), torch.empty_like(s["W"])
    dbias = torch.empty(s["W"].shape[:-2] + (case["N"],), dtype=BF16, device="cuda")
    for rows, e in _groups(s):
        W, gW, gb = (s["W"], dW, dbias) if e is None else (s["W"][e], dW[e], dbias[e])
        dz = s["dY"][rows].float()
        if case["act"] != "none":
            dz = dz * _act_grad(case["act"], s["Z"][rows].float())
        x = s["X"][rows].float()
        if case["layout"] == "kn":
            dX[rows] = (dz @ W.float().t()).to(BF16)
            gW.copy_((x.t() @ dz).to(BF16))
        else:
            dX[rows] = (dz @ W.float()).to(BF16)
            gW.copy_((dz.t() @ x).to(BF16))
        gb.copy_(dz.sum(dim=0).to(BF16))
    return {"dX": dX, "dW": dW, "dbias": dbias}


# ------------------------------------------------------------------------------------- run --
def run(s):
    op = s["case"]["op"]
    if not own:
        if op == "norm":
            return _plain_norm(s)
        if op == "norm_grad":
            return _plain_norm_grad(s)
        return _plain_linear_grad(s) if op.endswith("_grad") else _plain_linear(s)
    import mlp_latency_gb300 as mc

    if op == "norm":
        mc.layer_norm_forward(s["x"], s["gamma"], s["beta"], s["out"], mean=s["mean"], rstd=s["rstd"], eps=EPS)
        return {"y": s["out"], "mean": s["mean"], "rstd": s["rstd"]}
    if op == "norm_grad":
        mc.layer_norm_backward(s["dy"], s["x"], s["gamma"], s["mean"], s["rstd"], s["out"], dgamma=s["dgamma"],
                               dbeta=s["dbeta"], dx_add=s["skip"], workspace=s["ws"])
        return {"dx": s["out"], "dgamma": s["dgamma"], "dbeta": s["dbeta"]}
    if op.endswith("_grad"):
        s["linear"].backward(s["dY"], s["X"], s["W"], Z=s["Z"], dX=s["dX"], dW=s["dW"], dbias=s["dbias"],
                             offsets=s.get("offsets"), workspace=s["ws"])
        return {"dX": s["dX"], "dW": s["dW"], "dbias": s["dbias"]}
    s["linear"].forward(s["X"], s["W"], s["Y"], bias=s["bias"], residual=s["residual"], Z=s["Z"],
                        offsets=s.get("offsets"), workspace=s["ws"])
    return {"Y": s["Y"]} if s["Z"] is None else {"Y": s["Y"], "Z": s["Z"]}


# ------------------------------------------------------------------------------------ work --
def work(case):
    if case["op"] in ("norm", "norm_grad"):
        R, C, b = case["rows"], case["cols"], 2 if case["dtype"] == "bf16" else 4
        if case["op"] == "norm":
            return {"bytes": 2 * R * C * b + 2 * C * b + 8 * R, "flops": 8 * R * C}
        return {"bytes": (3 + bool(case["skip"])) * R * C * b + 3 * C * b + 8 * R, "flops": 14 * R * C}
    R, K, N = case["rows"], case["K"], case["N"]
    E = case.get("experts", 1)
    used = sum(n > 0 for n in _sizes(case)) if "experts" in case else 1   # experts whose weights are read
    if case["op"].endswith("_grad"):
        acts = R * N * (1 if case["act"] == "none" else 2)
        return {"bytes": 2 * (2 * R * K + acts + used * K * N + E * K * N + E * N), "flops": 4 * R * K * N}
    outs = R * N * (1 + bool(case.get("save")) + bool(case.get("residual")))
    return {"bytes": 2 * (R * K + used * (K * N + N) + outs), "flops": 2 * R * K * N}


# ----------------------------------------------------------------------------------- exact --
def exact(case, seed):
    """The outputs from the definitions, in 64 bits: centred moments, tanh(u) = 2 sigmoid(2u) - 1,
    products by torch's 64-bit matmul."""
    if case["op"].startswith(("linear", "experts")) and case["rows"] * case["K"] * case["N"] > 3e11:
        return None
    s = _inputs(case, seed)
    D = torch.float64
    if case["op"] in ("norm", "norm_grad"):
        x, gamma = s["x"].to(D), s["gamma"].to(D)
        if case["op"] == "norm":
            var, mean = torch.var_mean(x, dim=1, correction=0)
            rstd = (var + EPS) ** -0.5
            return {"y": torch.addcmul(s["beta"].to(D), (x - mean[:, None]) * rstd[:, None], gamma), "mean": mean,
                    "rstd": rstd}
        C = case["cols"]
        mean, rstd, dy = s["mean"].to(D)[:, None], s["rstd"].to(D)[:, None], s["dy"].to(D)
        xh = rstd * (x - mean)
        # J^T g with J = rstd (I - 1 1^T / C - xh xh^T / C)
        g = dy * gamma
        dx = rstd * (g - g.sum(1, keepdim=True) / C - xh * ((xh * g).sum(1, keepdim=True) / C))
        if s["skip"] is not None:
            dx = dx + s["skip"].to(D)
        return {"dx": dx, "dgamma": torch.einsum("rc,rc->c", dy, xh), "dbeta": torch.einsum("rc->c", dy)}
    K, N, R = case["K"], case["N"], case["rows"]
    E = case.get("experts", 1)
    W = s["W"].view(E, *s["W"].shape[-2:])
    if case["layout"] == "nk":
        W = W.transpose(1, 2)
    bounds = np.concatenate([[0], np.cumsum(s["sizes"] if "sizes" in s else [R])])
    c = math.sqrt(2.0 / math.pi)
    if not case["op"].endswith("_grad"):
        Z = torch.empty((R, N), dtype=D, device="cuda")
        for e in range(E):
            lo, hi = int(bounds[e]), int(bounds[e + 1])
            if hi > lo:
                torch.matmul(s["X"][lo:hi].to(D), W[e].to(D), out=Z[lo:hi])
                Z[lo:hi] += s["bias"].view(E, N)[e].to(D)
        if case["act"] == "gelu":
            Y = Z * torch.sigmoid(2.0 * c * Z * (1.0 + 0.044715 * Z ** 2))
        elif case["act"] == "silu":
            Y = Z * torch.sigmoid(Z)
        elif case["act"] == "relu":
            Y = torch.where(Z > 0, Z, torch.zeros_like(Z))
        else:
            Y = Z.clone()
        if s["residual"] is not None:
            Y += s["residual"].to(D)
        return {"Y": Y, "Z": Z} if case.get("save") else {"Y": Y}
    dZ = s["dY"].to(D)
    if case["act"] == "relu":
        dZ = torch.where(s["Z"] > 0, dZ, torch.zeros_like(dZ))
    elif case["act"] == "silu":
        z = s["Z"].to(D)
        p = torch.sigmoid(z)
        dZ = dZ * (p + z * p * torch.sigmoid(-z))
    elif case["act"] == "gelu":
        z = s["Z"].to(D)
        p = torch.sigmoid(2.0 * c * z * (1.0 + 0.044715 * z ** 2))
        dZ = dZ * (p + z * p * (1.0 - p) * 2.0 * c * (1.0 + 3.0 * 0.044715 * z ** 2))
    dX = torch.zeros((R, K), dtype=D, device="cuda")
    dW = torch.zeros((E, K, N), dtype=D, device="cuda")
    db = torch.zeros((E, N), dtype=D, device="cuda")
    for e in range(E):
        lo, hi = int(bounds[e]), int(bounds[e + 1])
        if hi > lo:
            dX[lo:hi] = dZ[lo:hi] @ W[e].to(D).t()
            dW[e] = s["X"][lo:hi].to(D).t() @ dZ[lo:hi]
            db[e] = dZ[lo:hi].sum(0)
    if case["layout"] == "nk":
        dW = dW.transpose(1, 2)
    return {"dX": dX, "dW": dW.reshape(s["W"].shape), "dbias": db.view(s["W"].shape[:-2] + (N,))}
