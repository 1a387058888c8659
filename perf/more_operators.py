"""What stands around the experts' products of an MLP block, and at the end of a training step, as cases to time:
routing (top choices, gates, per-expert counts and rows, balance loss) and its gradient, the exchange of rows between
tokens and experts in its four directions, and the global gradient norm with clipping.

`run` computes them in a plain form (elementary torch operations in 32 bits, rounded once) or, with `own` set, through
the package's entry points.
"""
import math

import numpy as np
import torch

own = False

EPS = 1e-6
BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64
TYPES = {"bf16": BF16, "f32": F32}


# ----------------------------------------------------------------------------------- cases --
def listed():
    return [
        # One decoding sequence chooses its experts: latency only.
        {"name": "route_token", "op": "route", "tokens": 1, "experts": 8, "top": 2, "dtype": "f32", "normalize": True, "pad": 0},
        # The router of a prefill, the last prompt padded; 32-bit logits.
        {"name": "route_prefill", "op": "route", "tokens": 2048, "experts": 8, "top": 2, "dtype": "f32", "normalize": False, "pad": 45},
        # Training with many small experts, logits as a bf16 product left them (with ties).
        {"name": "route_many", "op": "route", "tokens": 8192, "experts": 256, "top": 8, "dtype": "bf16", "normalize": True, "pad": 0},
        # The gradient of the gates and of the balance loss, 32 experts.
        {"name": "route_grad", "op": "route_grad", "tokens": 16000, "experts": 32, "top": 4, "dtype": "f32", "normalize": False, "pad": 77},
        # The end of a block for eight decoding sequences: two rows each, gates and the skip connection.
        {"name": "combine_tokens", "op": "combine", "tokens": 8, "experts": 8, "top": 2, "cols": 4096, "dtype": "bf16", "add": True,
         "pad": 0},
        # The experts' rows of a prefill, put in order.
        {"name": "dispatch_prefill", "op": "dispatch", "tokens": 2048, "experts": 8, "top": 2, "cols": 4096, "dtype": "bf16", "pad": 45},
        # The end of the block in a training step: gates and the skip connection.
        {"name": "combine_train", "op": "combine", "tokens": 4096, "experts": 32, "top": 4, "cols": 2048, "dtype": "bf16", "add": True,
         "pad": 0},
        # Its gradient, for the rows and the gates.
        {"name": "combine_grad", "op": "combine_grad", "tokens": 4096, "experts": 8, "top": 2, "cols": 8192, "dtype": "bf16", "pad": 0},
        # A small model trained in 32 bits, odd sizes: the gradient of the rows' order, joined with the router's part.
        {"name": "dispatch_grad_odd_f32", "op": "dispatch_grad", "tokens": 333, "experts": 5, "top": 3, "cols": 1357, "dtype": "f32",
         "add": True, "pad": 10},
        # The gradients of a large dense block, clipped on their way to the update.
        {"name": "clip_block", "op": "clip", "blocks": 1, "width": 8192, "hidden": 8192, "experts": 0, "dtype": "bf16", "limit": 0.3},
        # A small model in 32 bits: many tensors, odd sizes.
        {"name": "clip_odd_f32", "op": "clip", "blocks": 6, "width": 333, "hidden": 1357, "experts": 0, "dtype": "f32", "limit": 0.3},
        # Experts' gradients in place, with a norm below the limit: read, and left as they are.
        {"name": "clip_experts_below", "op": "clip", "blocks": 1, "width": 1024, "hidden": 2048, "experts": 8, "dtype": "mixed",
         "limit": 4.0},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "route", "route_grad", "dispatch", "dispatch_grad", "combine", "combine_grad", "clip", "clip"])
    if op == "clip":
        case = {"op": op, "blocks": _log_int(rng, 1, 24), "width": _log_int(rng, 64, 4096), "hidden": _log_int(rng, 64, 8192),
                "experts": rng.choice([0, 0, rng.randrange(2, 17)]), "dtype": rng.choice(["bf16", "f32", "mixed"]),
                "limit": rng.choice([0.3, 0.3, 4.0])}
        while case["blocks"] * max(case["experts"], 1) * case["width"] * case["hidden"] > 4096 * 8192:
            if case["blocks"] > 1:
                case["blocks"] //= 2
            else:
                case["hidden"] = max(case["hidden"] // 2, 64)
                case["experts"] //= 2 if case["experts"] > 3 else 1
        return case
    case = {"op": op, "tokens": _log_int(rng, 1, 16384), "experts": _log_int(rng, 4, 256), "dtype": rng.choice(["bf16", "f32"])}
    case["top"] = min(rng.choice([1, 2, 2, 3, 4, 6, 8]), case["experts"])
    case["pad"] = rng.choice([0, int(case["tokens"] * rng.uniform(0.0, 0.3))])
    if op.startswith("route"):
        case["normalize"] = rng.random() < 0.5
        while case["tokens"] * case["experts"] > 8192 * 256:
            case["tokens"] //= 2
            case["pad"] //= 2
        return case
    case["cols"] = _log_int(rng, 64, 8192)
    if rng.random() < 0.6:
        case["cols"] = case["cols"] // 8 * 8
    if op in ("combine", "dispatch_grad"):
        case["add"] = rng.random() < 0.5
    while case["tokens"] * case["top"] * case["cols"] * (1 + (case["dtype"] == "f32")) > 4096 * 2 * 8192:
        case["tokens"] //= 2
        case["pad"] //= 2
    return case


def _shapes(case):
    """The gradients of `blocks` blocks, in the order of their parameters, with their types."""
    w, h, e = case["width"], case["hidden"], case["experts"]
    lead = (e,) if e else ()
    big = BF16 if case["dtype"] == "bf16" else F32
    small = F32 if case["dtype"] == "f32" else BF16
    one = [((w,), small), ((w,), small), (lead + (w, h), big), (lead + (h,), small), (lead + (h, w), big), (lead + (w,), small)]
    return (one + ([((w, e), small)] if e else [])) * case["blocks"]


def _max_norm(case):
    """Near `limit` times the norm of the gradients that _inputs makes: never near the norm itself."""
    return case["limit"] * 0.02 * math.sqrt(sum(math.prod(s) for s, _ in _shapes(case)))


# ---------------------------------------------------------------------------------- inputs --
def _normal(gen, shape, std, dtype):
    return (torch.randn(shape, generator=gen, device="cuda", dtype=F32) * std).to(dtype)


def _route_inputs(case, gen):
    """Logits with experts of uneven popularity, and which tokens are no padding."""
    T, E = case["tokens"], case["experts"]
    logits = torch.randn((T, E), generator=gen, device="cuda", dtype=F32) + 0.7 * torch.randn(E, generator=gen, device="cuda", dtype=F32)
    mask = torch.arange(T, device="cuda") < T - case["pad"] if case["pad"] else None
    return logits, mask


def _order(chosen, experts):
    """slots and offsets of chosen [T, k] (-1: none): a stable sort by expert, counted in 64 bits."""
    flat = chosen.reshape(-1).long()
    place = torch.argsort(torch.where(flat < 0, experts, flat), stable=True)
    slots = torch.empty_like(flat)
    slots[place] = torch.arange(flat.numel(), device=flat.device)
    slots = torch.where(flat < 0, -1, slots).reshape(chosen.shape).to(torch.int32)
    ends = torch.bincount(flat[flat >= 0], minlength=experts).cumsum(0)
    return slots, torch.cat([ends.new_zeros(1), ends]).to(torch.int32)


def _inputs(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed * 1000003 + 29)
    s = {}
    if case["op"] == "clip":
        s["grads"] = [_normal(gen, shape, 0.02, dt) for shape, dt in _shapes(case)]
        return s
    logits, mask = _route_inputs(case, gen)
    if case["op"] == "route":
        s["logits"], s["mask"] = logits.to(TYPES[case["dtype"]]), mask
        return s
    # what the forward pass left: each token's choices and their rows
    T, E, k = case["tokens"], case["experts"], case["top"]
    value, chosen = torch.sort(logits, dim=1, descending=True, stable=True)
    gates = torch.softmax(value, dim=1)[:, :k].contiguous()
    chosen = chosen[:, :k].to(torch.int32).contiguous()
    if mask is not None:
        chosen[~mask] = -1
        gates[~mask] = 0.0
    slots, offsets = _order(chosen, E)
    dt = TYPES[case["dtype"]]
    if case["op"] == "route_grad":
        s["logits"], s["chosen"], s["offsets"] = logits.to(dt), chosen, offsets
        s["dgates"] = _normal(gen, (T, k), 1.0 / 16, F32)
        s["dloss"] = torch.full((1,), 0.01, dtype=F32, device="cuda")
        return s
    s["slots"] = slots
    D = case["cols"]
    if case["op"] == "dispatch":
        s["x"] = _normal(gen, (T, D), 1.0, dt)
    elif case["op"] == "dispatch_grad":
        s["dy"] = _normal(gen, (T * k, D), 1.0 / 16, dt)
    else:
        s["gates"] = gates
        s["z"] = _normal(gen, (T * k, D), 1.0, dt)
        if case["op"] == "combine_grad":
            s["dy"] = _normal(gen, (T, D), 1.0 / 16, dt)
    if "add" in case:
        s["add"] = _normal(gen, (T, D), 1.0, dt) if case["add"] else None
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    op = case["op"]
    if op == "clip":
        s["max_norm"] = _max_norm(case)
        if case["limit"] < 1.0:
            s["out"] = [torch.empty_like(g) for g in s["grads"]]
    if op in ("dispatch", "combine_grad"):   # rows of no token stay as they are
        s["rows_out"] = torch.zeros((case["tokens"] * case["top"], case["cols"]), dtype=TYPES[case["dtype"]], device="cuda")
    if not own:
        return s
    import mlp_latency_gb300 as mc

    new = lambda *shape, dtype=F32: torch.empty(shape, dtype=dtype, device="cuda")
    if op == "clip":
        s["norm"] = new(1)
        s["ws"] = new(mc.clip_workspace_size(len(s["grads"])), dtype=torch.uint8)
        return s
    T, E, k = case["tokens"], case["experts"], case["top"]
    if op == "route":
        s["gates"], s["chosen"], s["slots"] = new(T, k), new(T, k, dtype=torch.int32), new(T, k, dtype=torch.int32)
        s["counts"], s["offsets"], s["loss"] = new(E, dtype=torch.int32), new(E + 1, dtype=torch.int32), new(1)
        s["ws"] = new(mc.route_workspace_size(T, E), dtype=torch.uint8)
    elif op == "route_grad":
        s["dlogits"] = torch.empty_like(s["logits"])
    elif op == "combine_grad":
        s["dgates"] = torch.empty_like(s["gates"])
    elif op != "dispatch":
        s["tokens_out"] = new(T, case["cols"], dtype=TYPES[case["dtype"]])
    return s


# ------------------------------------------------------------------------------ plain forms --
def _plain_route(s):
    case = s["case"]
    T, E, k = case["tokens"], case["experts"], case["top"]
    logits = s["logits"].float()
    p = torch.exp(logits - logits.max(dim=1, keepdim=True).values)
    p = p / p.sum(dim=1, keepdim=True)
    if s["mask"] is not None:
        p = torch.where(s["mask"][:, None], p, torch.zeros_like(p))
    column = torch.arange(E, device="cuda")
    left, chosen = logits.clone(), []
    for _ in range(k):   # the largest that is left, the first of equals
        e = torch.where(left == left.max(dim=1, keepdim=True).values, column, E).min(dim=1).values
        left[torch.arange(T, device="cuda"), e] = -math.inf
        chosen.append(e)
    chosen = torch.stack(chosen, dim=1)
    gates = torch.gather(p, 1, chosen)
    if case["normalize"]:
        c = torch.gather(logits, 1, chosen)
        gates = torch.exp(c - c[:, :1])
        gates = gates / gates.sum(dim=1, keepdim=True)
    if s["mask"] is not None:
        gates = torch.where(s["mask"][:, None], gates, torch.zeros_like(gates))
        chosen = torch.where(s["mask"][:, None], chosen, -1)
    hit = (column[:, None] == chosen.reshape(1, -1)).to(torch.int32)   # an expert's choices along a row
    counts = hit.sum(dim=1)
    ends = counts.cumsum(0)
    offsets = torch.cat([ends.new_zeros(1), ends])
    rank = torch.gather(hit.cumsum(1, dtype=torch.int32), 0, chosen.reshape(1, -1).clamp_min(0))[0] - 1
    slots = torch.where(chosen >= 0, offsets[chosen.clamp_min(0)] + rank.view(T, k), -1)
    M = counts.sum().clamp_min(1).to(F64)
    loss = E * k * (counts * p.sum(dim=0, dtype=F64)).sum() / (M * M)
    i32 = torch.int32
    return {"gates": gates, "experts": chosen.to(i32), "slots": slots.to(i32), "counts": counts.to(i32), "offsets": offsets.to(i32),
            "loss": loss.to(F32).view(1)}


def _plain_route_grad(s):
    case = s["case"]
    E, k = case["experts"], case["top"]
    logits = s["logits"].float()
    p = torch.exp(logits - logits.max(dim=1, keepdim=True).values)
    p = p / p.sum(dim=1, keepdim=True)
    routed = s["chosen"] >= 0
    column = s["chosen"].clamp_min(0).long()
    dgates = torch.where(routed, s["dgates"], torch.zeros_like(s["dgates"]))
    counts = (s["offsets"][1:] - s["offsets"][:-1]).float()
    M = counts.sum().clamp_min(1.0)
    g = (s["dloss"] * E * k * counts / (M * M)).expand_as(p)
    if not case["normalize"]:
        g = g + torch.zeros_like(p).scatter_add_(1, column, dgates)
    d = p * (g - (g * p).sum(dim=1, keepdim=True))
    if case["normalize"]:
        c = torch.gather(logits, 1, column)
        gates = torch.where(routed, torch.exp(c - c.max(dim=1, keepdim=True).values), torch.zeros_like(c))
        gates = gates / gates.sum(dim=1, keepdim=True).clamp_min(1e-30)
        d = d + torch.zeros_like(p).scatter_add_(1, column, gates * (dgates - (gates * dgates).sum(dim=1, keepdim=True)))
    return {"dlogits": torch.where(routed[:, :1], d, torch.zeros_like(d)).to(s["logits"].dtype)}


def _plain_gather(rows, slots, gates, add):
    """sum_j gates[t, j] rows[slots[t, j]] + add[t]"""
    out = torch.zeros((slots.shape[0], rows.shape[1]), dtype=F32, device="cuda") if add is None else add.float()
    for j in range(slots.shape[1]):
        at = slots[:, j]
        v = rows[at.clamp_min(0)].float()
        if gates is not None:
            v = v * gates[:, j:j + 1]
        out = out + torch.where(at[:, None] >= 0, v, torch.zeros_like(v))
    return out.to(rows.dtype)


def _plain_scatter(out, tokens, slots, gates):
    """out[slots[t, j]] = gates[t, j] tokens[t]"""
    for j in range(slots.shape[1]):
        t = torch.nonzero(slots[:, j] >= 0)[:, 0]
        v = tokens[t]
        if gates is not None:
            v = (v.float() * gates[t, j:j + 1]).to(out.dtype)
        out[slots[t, j].long()] = v
    return out


def _plain_exchange(s):
    op, slots = s["case"]["op"], s["slots"]
    if op == "dispatch":
        return {"y": _plain_scatter(s["rows_out"], s["x"], slots, None)}
    if op == "dispatch_grad":
        return {"dx": _plain_gather(s["dy"], slots, None, s["add"])}
    if op == "combine":
        return {"y": _plain_gather(s["z"], slots, s["gates"], s["add"])}
    dgates = torch.stack([torch.where(slots[:, j] >= 0, (s["dy"].float() * s["z"][slots[:, j].clamp_min(0)].float()).sum(dim=1), 0.0)
                          for j in range(slots.shape[1])], dim=1)
    return {"dz": _plain_scatter(s["rows_out"], s["dy"], slots, s["gates"]), "dgates": dgates}


def _plain_clip(s):
    total = sum(g.float().square().sum(dtype=F64) for g in s["grads"])
    norm = torch.sqrt(total).to(F32)
    c = torch.clamp_max(s["max_norm"] / (norm + EPS), 1.0)
    out = s.get("out", s["grads"])
    for g, o in zip(s["grads"], out):
        o.copy_(g.float() * c)
    return {"norm": norm.view(1), "grads": out}


# ------------------------------------------------------------------------------------- run --
def run(s):
    op = s["case"]["op"]
    if not own:
        if op == "clip":
            return _plain_clip(s)
        return _plain_route(s) if op == "route" else _plain_route_grad(s) if op == "route_grad" else _plain_exchange(s)
    import mlp_latency_gb300 as mc

    if op == "route":
        mc.route_forward(s["logits"], s["gates"], s["chosen"], s["offsets"], slots=s["slots"], counts=s["counts"], loss=s["loss"],
                         mask=s["mask"], normalize=s["case"]["normalize"], workspace=s["ws"])
        return {"gates": s["gates"], "experts": s["chosen"], "slots": s["slots"], "counts": s["counts"], "offsets": s["offsets"],
                "loss": s["loss"]}
    if op == "route_grad":
        mc.route_backward(s["logits"], s["chosen"], s["offsets"], s["dlogits"], dgates=s["dgates"], dloss=s["dloss"],
                          normalize=s["case"]["normalize"])
        return {"dlogits": s["dlogits"]}
    if op == "dispatch":
        mc.dispatch_forward(s["x"], s["slots"], s["rows_out"])
        return {"y": s["rows_out"]}
    if op == "dispatch_grad":
        mc.dispatch_backward(s["dy"], s["slots"], s["tokens_out"], dx_add=s["add"])
        return {"dx": s["tokens_out"]}
    if op == "combine":
        mc.combine_forward(s["z"], s["gates"], s["slots"], s["tokens_out"], residual=s["add"])
        return {"y": s["tokens_out"]}
    if op == "combine_grad":
        mc.combine_backward(s["dy"], s["z"], s["gates"], s["slots"], dz=s["rows_out"], dgates=s["dgates"])
        return {"dz": s["rows_out"], "dgates": s["dgates"]}
    mc.clip_gradients(s["grads"], s["max_norm"], s["norm"], out=s.get("out"), eps=EPS, workspace=s["ws"])
    return {"norm": s["norm"], "grads": s.get("out", s["grads"])}


# ------------------------------------------------------------------------------------ work --
def work(case):
    op = case["op"]
    if op == "clip":
        shapes = _shapes(case)
        n = sum(math.prod(shape) for shape, _ in shapes)
        b = sum(math.prod(shape) * (2 if dt == BF16 else 4) for shape, dt in shapes)
        clipped = case["limit"] < 1.0
        return {"bytes": b * (1 + clipped), "flops": n * (2 + clipped)}
    T, E, k, b = case["tokens"], case["experts"], case["top"], 2 if case["dtype"] == "bf16" else 4
    if op == "route":
        return {"bytes": T * E * b + T * bool(case["pad"]) + 12 * T * k + 8 * E + 8, "flops": (5 + k) * T * E}
    if op == "route_grad":
        return {"bytes": 2 * T * E * b + 8 * T * k + 4 * E + 8, "flops": 9 * T * E}
    D, pairs = case["cols"], (T - case["pad"]) * k
    tokens = T - case["pad"]   # a token of no expert need not be read on its way to one
    if op == "dispatch":
        return {"bytes": (tokens + pairs) * D * b + 4 * T * k, "flops": 0}
    if op == "combine_grad":
        return {"bytes": (tokens + 2 * pairs) * D * b + 12 * T * k, "flops": 3 * pairs * D}
    gates = 4 * T * k if op == "combine" else 0
    return {"bytes": (pairs + T * (1 + case["add"])) * D * b + 4 * T * k + gates, "flops": 2 * pairs * D}


# ----------------------------------------------------------------------------------- exact --
def exact(case, seed):
    """The outputs from the definitions, in 64 bits: softmax by log-sum-exp, choices by a stable sort, rows by a stable
    sort, the exchange as a product with the choices' matrix taken row by row, gradients by the Jacobians."""
    s = _inputs(case, seed)
    op = case["op"]
    if op == "clip":
        squares = [torch.linalg.vector_norm(g.reshape(-1), dtype=F64) for g in s["grads"]]
        norm = torch.linalg.vector_norm(torch.stack(squares))
        c = min(1.0, _max_norm(case) / (float(norm) + EPS))
        return {"norm": norm.view(1), "grads": [g.to(F64) * c for g in s["grads"]]}
    T, E, k = case["tokens"], case["experts"], case["top"]
    if op == "route":
        logits = s["logits"].to(F64)
        p = torch.exp(logits - torch.logsumexp(logits, dim=1, keepdim=True))
        place = np.argsort(-logits.cpu().numpy(), axis=1, kind="stable")[:, :k]
        chosen = torch.from_numpy(np.ascontiguousarray(place)).cuda()
        gates = p.gather(1, chosen)
        if case["normalize"]:
            gates = gates / gates.sum(1, keepdim=True)
        if s["mask"] is not None:
            p[~s["mask"]] = 0.0
            gates[~s["mask"]] = 0.0
            chosen[~s["mask"]] = -1
        slots, offsets = _order(chosen, E)
        counts = offsets.diff()
        fraction = counts.to(F64) / max(int(offsets[-1]), 1)
        loss = E * (fraction * p.sum(0) * k / max(int(offsets[-1]), 1)).sum()
        return {"gates": gates, "experts": chosen.to(torch.int32), "slots": slots, "counts": counts, "offsets": offsets,
                "loss": loss.view(1)}
    if op == "route_grad":
        p = torch.softmax(s["logits"].to(F64), dim=1)
        counts = s["offsets"].diff().to(F64)
        pull = float(s["dloss"]) * E * k / max(float(counts.sum()), 1.0) ** 2 * counts
        d = p * pull - p * (p @ pull)[:, None]
        row, column = torch.nonzero(s["chosen"] >= 0, as_tuple=True)
        e = s["chosen"][row, column].long()
        chosen = torch.zeros((T, E), dtype=F64, device="cuda")
        chosen[row, e] = 1.0
        dg = torch.zeros((T, E), dtype=F64, device="cuda")
        dg[row, e] = s["dgates"].to(F64)[row, column]
        gate = p * chosen
        if case["normalize"]:
            gate = gate / gate.sum(1, keepdim=True).clamp_min(1e-300)
            d = d + gate * dg - gate * (gate * dg).sum(1, keepdim=True)
        else:
            d = d + gate * dg - p * (gate * dg).sum(1, keepdim=True)
        return {"dlogits": d * chosen.amax(1, keepdim=True)}
    D = case["cols"]
    token, choice = torch.nonzero(s["slots"] >= 0, as_tuple=True)
    row = s["slots"][token, choice].long()
    if op == "dispatch":
        y = torch.zeros((T * k, D), dtype=F64, device="cuda")
        y[row] = s["x"].to(F64)[token]
        return {"y": y}
    if op == "combine_grad":
        dz = torch.zeros((T * k, D), dtype=F64, device="cuda")
        dz[row] = s["dy"].to(F64)[token] * s["gates"].to(F64)[token, choice][:, None]
        dgates = torch.zeros((T, k), dtype=F64, device="cuda")
        for at in torch.split(torch.arange(row.numel(), device="cuda"), 4096):
            dgates[token[at], choice[at]] = torch.einsum("nd,nd->n", s["dy"].to(F64)[token[at]], s["z"][row[at]].to(F64))
        return {"dz": dz, "dgates": dgates}
    out = torch.zeros((T, D), dtype=F64, device="cuda") if s["add"] is None else s["add"].to(F64)
    rows = (s["dy"] if op == "dispatch_grad" else s["z"])[row].to(F64)
    if op == "combine":
        rows = rows * s["gates"].to(F64)[token, choice][:, None]
    return {"dx" if op == "dispatch_grad" else "y": out.index_add_(0, token, rows)}
