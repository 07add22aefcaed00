"""The measured cases of training the experts in 16 bits: rows to the experts and back, the grouped
products and their gradients, and the router weights' gradient.

Five kinds of case, each one pass of an operator as a program calls it:

  dispatch  each token's row copied to its K expert rows, and the gradient of that, the sum of a
            token's K rows
  combine   the weighted sum of each token's K expert rows onto a residual, and its gradient: the
            rows' and the weights'
  mm        the grouped product of 16-bit rows and weights, out = act(a W^T + bias) + residual, with
            the SwiGLU of gate and up (and their values before it, kept for the gradient) or none
  grad      that product's gradients: its input's (through the SwiGLU that made the input, where
            there is one), its weights' and its bias's
  route     the gradient of the router's logits from that of the K routing weights

``own = False`` computes them from elementary torch operations in 32 bits, ``own = True`` with the
library's kernels.  Rows are grouped by expert: rows offsets[e] .. offsets[e+1]-1 are expert e's,
src[r] = t * K + k names row r's route and slot is its inverse.  A padded token's routes go to no
expert: its slots are -1, and the rows from offsets[E] on stay as they were (here 0).
"""
import math

import torch

own = False

DTYPES = {"float32": torch.float32, "bfloat16": torch.bfloat16, "float16": torch.float16}


def listed():
    return [
        # a small batch of decode steps, and a chunk at the layer's sizes with padded tokens
        {"name": "dispatch_17", "kind": "dispatch", "T": 17, "H": 2048, "E": 512, "K": 10,
         "skew": 0.0, "pad": 0.0, "dtype": "bfloat16"},
        {"name": "dispatch_8k", "kind": "dispatch", "T": 8192, "H": 2048, "E": 512, "K": 10,
         "skew": 0.6, "pad": 0.1, "dtype": "bfloat16"},
        # an odd batch of odd rows, and a training chunk with fp32 token gradients
        {"name": "combine_61_odd", "kind": "combine", "T": 61, "H": 1001, "E": 64, "K": 3,
         "skew": 0.0, "pad": 0.2, "dtype": "float16", "out": "float16", "residual": True},
        {"name": "combine_8k", "kind": "combine", "T": 8192, "H": 2048, "E": 512, "K": 10,
         "skew": 0.0, "pad": 0.0, "dtype": "bfloat16", "out": "float32", "residual": False},
        # gate/up of one decoded token; of a training chunk, which keeps gate and up for the gradient
        {"name": "mm_one_token", "kind": "mm", "T": 1, "N": 512, "Kin": 2048, "E": 512, "K": 10,
         "skew": 0.0, "pad": 0.0, "gather": True, "swiglu": True, "bias": False, "residual": False,
         "keep": False, "dtype": "bfloat16", "out": "bfloat16"},
        {"name": "mm_gate_up_8k", "kind": "mm", "T": 8192, "N": 512, "Kin": 2048, "E": 512, "K": 10,
         "skew": 0.0, "pad": 0.0, "gather": True, "swiglu": True, "bias": False, "residual": False,
         "keep": True, "dtype": "bfloat16", "out": "bfloat16"},
        # one matrix that every token takes (a shared expert), onto what the others gave
        {"name": "mm_dense", "kind": "mm", "T": 8191, "N": 4096, "Kin": 4096, "E": 1, "K": 1,
         "skew": 0.0, "pad": 0.0, "gather": False, "swiglu": False, "bias": True, "residual": True,
         "keep": False, "dtype": "bfloat16", "out": "bfloat16"},
        # gradients: of a small layer on a short chunk, where launches count; of the down product at
        # the layer's sizes, through the SwiGLU before it; of the matrix that every token takes
        {"name": "grad_300_small", "kind": "grad", "T": 300, "N": 640, "Kin": 264, "E": 16, "K": 4,
         "skew": 0.8, "pad": 0.1, "gather": True, "swiglu": False, "bias": True,
         "dtype": "float16", "out": "float32"},
        {"name": "grad_down_8k", "kind": "grad", "T": 8192, "N": 2048, "Kin": 512, "E": 512, "K": 10,
         "skew": 0.0, "pad": 0.0, "gather": False, "swiglu": True, "bias": False,
         "dtype": "bfloat16", "out": "bfloat16"},
        {"name": "grad_dense", "kind": "grad", "T": 8191, "N": 4096, "Kin": 4096, "E": 1, "K": 1,
         "skew": 0.0, "pad": 0.0, "gather": False, "swiglu": False, "bias": True,
         "dtype": "bfloat16", "out": "float32"},
        # router training: a short batch, and a chunk with padded tokens
        {"name": "route_61", "kind": "route", "T": 61, "E": 512, "K": 10, "pad": 0.0,
         "dtype": "float32"},
        {"name": "route_30118", "kind": "route", "T": 30118, "E": 512, "K": 10, "pad": 0.2,
         "dtype": "bfloat16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["dispatch", "combine", "mm", "mm", "mm", "grad", "grad", "route"])
    T = _log(rng, 1, 8192)
    E = _log(rng, 1, 512)
    K = rng.randint(1, min(E, 10))
    skew = round(rng.choice([0.0, rng.uniform(0.1, 0.8)]), 2)
    pad = round(rng.uniform(0.05, 0.4), 2) if T >= 32 and rng.random() < 0.4 else 0.0
    case = {"kind": kind, "T": T, "E": E, "K": K, "pad": pad}
    if kind == "route":
        return {**case, "T": _log(rng, 1, 30000), "dtype": rng.choice(list(DTYPES))}
    case["skew"] = skew
    if kind in ("dispatch", "combine"):
        H = _log(rng, 16, 4096)
        if rng.random() < 0.6:
            H = max(8, H // 8 * 8)
        case["T"] = max(1, min(T, 8192 * 2048 * 10 // (H * K)))
        case |= {"H": H, "dtype": rng.choice(list(DTYPES))}
        if kind == "combine":
            case |= {"out": rng.choice([case["dtype"], "float32"]), "residual": rng.random() < 0.5}
        return case
    N, Kin = 8 * _log(rng, 4, 512), 8 * _log(rng, 4, 512)
    swiglu = rng.random() < 0.5
    while E * N * Kin > 512 * 2048 * 256:
        if E > 2:
            E = max(2, E // 2)
        else:
            N, Kin = max(32, N // 16 * 8), max(32, Kin // 16 * 8)
    K = min(K, E)
    case |= {"N": N, "Kin": Kin, "E": E, "K": K, "gather": rng.random() < 0.5, "swiglu": swiglu,
             "T": max(1, min(T, 8192 * 10 * 2048 * 256 // (N * Kin * K))), "bias": rng.random() < 0.5,
             "dtype": rng.choice(["bfloat16", "float16"])}
    case["out"] = rng.choice([case["dtype"], "float32"])
    if case["T"] < 32:
        case["pad"] = 0.0
    if kind == "mm":
        if swiglu:
            case["out"] = case["dtype"]
        case |= {"residual": not swiglu and rng.random() < 0.5, "keep": swiglu and rng.random() < 0.5}
    return case


# ---- inputs ---------------------------------------------------------------------------------
def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def _routing(case, g):
    """The top-K experts of logits with a popularity bias of slope `skew`, their softmax, and the
    routes of padded tokens, which go to expert E (no expert)."""
    T, E, K = case["T"], case["E"], case["K"]
    logits = _randn(g, T, E)
    rank = torch.randperm(E, generator=g, device="cuda")
    logits -= case.get("skew", 0.0) * torch.log(rank + 1.0)
    w, idx = torch.topk(logits, K, dim=1)
    padded = torch.rand(T, generator=g, device="cuda") < case["pad"]
    idx[padded] = E
    return idx, torch.softmax(w, 1)


def _maps(idx, E):
    """counts [E]; offsets [E + 1]; src (row -> t * K + k, -1 behind the last) and its inverse."""
    flat = idx.reshape(-1)
    order = torch.sort(flat, stable=True).indices
    slot = torch.empty_like(order)
    slot[order] = torch.arange(len(flat), device="cuda")
    counts = torch.bincount(flat, minlength=E + 1)[:E]
    offsets = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    offsets[1:] = torch.cumsum(counts, 0)
    slot = torch.where(flat < E, slot, -1)
    src = torch.where(flat[order] < E, order, -1)
    return counts, offsets, src.to(torch.int32), slot.view(idx.shape).to(torch.int32)


def _acts(g, T, H, dtype):
    """Activations: normal, a few channels ten times as large, one token all zero."""
    x = _randn(g, T, H)
    x[:, torch.randperm(H, generator=g, device="cuda")[:max(1, H // 256)]] *= 10.0
    if T > 3:
        x[T // 2] = 0.0
    return x.to(dtype)


def _weights(g, E, N, Kin, dtype):
    """Normal weights of deviation 1/sqrt(Kin), some experts at a time."""
    w = torch.empty(E, N, Kin, dtype=dtype, device="cuda")
    step = max(1, (1 << 28) // (N * Kin))
    for e in range(0, E, step):
        w[e:e + step] = _randn(g, min(step, E - e), N, Kin) / math.sqrt(Kin)
    return w


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = dict(case)
    kind, T, E, K = case["kind"], case["T"], case["E"], case["K"]
    dt = DTYPES[case["dtype"]]
    idx, w = _routing(case, g)
    R = T * K
    if kind == "route":
        s["idx"], s["w"] = idx.to(torch.int32), w
        s["grad_w"] = _randn(g, T, K)
        s["grad"] = torch.empty(T, E, dtype=dt, device="cuda")
        return s
    counts, s["offsets"], s["src"], s["slot"] = _maps(idx, E)
    if kind == "dispatch":
        s["x"] = _acts(g, T, case["H"], dt)
        s["grad_rows"] = _randn(g, R, case["H"]).to(dt)
        s["rows"] = torch.zeros_like(s["grad_rows"])
        s["grad_x"] = torch.empty_like(s["x"])
        return s
    if kind == "combine":
        H, out = case["H"], DTYPES[case["out"]]
        s["rows"], s["w"] = _randn(g, R, H).to(dt), w
        s["residual"] = _randn(g, T, H).to(out) if case["residual"] else None
        s["grad_out"] = _randn(g, T, H).to(out)
        s["out"] = torch.empty(T, H, dtype=out, device="cuda")
        s["grad_rows"] = torch.zeros_like(s["rows"])
        s["grad_w"] = torch.empty(T, K, device="cuda")
        return s
    # for the plain form: the experts that have rows, and each row's place among rows padded to the
    # longest expert's
    s["order"] = torch.nonzero(counts).reshape(-1)
    s["cap"], s["live"] = int(counts.max()), int(counts.sum())
    ordinal = (torch.cumsum(counts > 0, 0) - 1).repeat_interleave(counts)
    first = s["offsets"][:-1].long().repeat_interleave(counts)
    s["place"] = ordinal * s["cap"] + torch.arange(s["live"], device="cuda") - first
    N, Kin, out = case["N"], case["Kin"], DTYPES[case["out"]]
    rows = 2 * N if kind == "mm" and case["swiglu"] else N
    s["weight"] = _weights(g, E, rows, Kin, dt)
    s["a"] = _acts(g, T if case["gather"] else R, Kin, dt)
    if kind == "mm":
        s["bias"] = _randn(g, E, rows).to(dt) if case["bias"] else None
        s["residual"] = _randn(g, R, N).to(out) if case["residual"] else None
        s["z"] = torch.zeros(R, rows, dtype=dt, device="cuda") if case["keep"] else None
        s["out"] = torch.zeros(R, N, dtype=out, device="cuda")
        return s
    s["grad"] = _randn(g, R, N).to(dt)
    s["z"] = _randn(g, R, 2 * Kin).to(dt) if case["swiglu"] else None
    s["grad_a"] = torch.zeros(R, Kin * (2 if case["swiglu"] else 1), dtype=dt, device="cuda")
    s["grad_weight"] = torch.empty(E, N, Kin, dtype=out, device="cuda")
    s["grad_bias"] = torch.empty(E, N, dtype=out, device="cuda") if case["bias"] else None
    return s


# ---- the plain form -------------------------------------------------------------------------
def _padded(rows, s):
    """[experts with rows, longest, columns] of the first live rows, in 32 bits."""
    pad = torch.zeros(len(s["order"]) * s["cap"], rows.shape[1], device=rows.device)
    pad[s["place"]] = rows[:s["live"]].float()
    return pad.view(len(s["order"]), s["cap"], -1)


def _whole(y, s, dtype):
    """The live rows of a padded product, rows of 0 behind them."""
    out = torch.zeros(s["T"] * s["K"], y.shape[-1], dtype=dtype, device=y.device)
    out[:s["live"]] = y.flatten(0, 1)[s["place"]].to(dtype)
    return out


def _inputs(s):
    """The rows that the product reads: one to each live row."""
    return s["a"][s["src"][:s["live"]].long() // s["K"]] if s["gather"] else s["a"]


def _expert_rows(s):
    """The expert of each live row."""
    counts = (s["offsets"][1:] - s["offsets"][:-1]).long()
    return torch.repeat_interleave(torch.arange(s["E"], device=counts.device), counts)


def _picked(rows, slot):
    """Each token's K rows in 32 bits, 0 for a route that has none."""
    there = (slot >= 0).unsqueeze(-1)
    return torch.where(there, rows[slot.long().clamp(min=0)].float(), 0.0)


def _plain(s):
    kind, T, K = s["kind"], s["T"], s["K"]
    if kind == "dispatch":
        rows = s["x"][s["src"].long().clamp(min=0) // K]
        rows = torch.where((s["src"] >= 0).unsqueeze(-1), rows, torch.zeros_like(rows))
        return {"rows": rows, "grad_x": _picked(s["grad_rows"], s["slot"]).sum(1).to(rows.dtype)}
    if kind == "combine":
        picked, grad = _picked(s["rows"], s["slot"]), s["grad_out"].float()
        out = (picked * s["w"].unsqueeze(-1)).sum(1)
        if s["residual"] is not None:
            out = out + s["residual"].float()
        there = s["slot"].reshape(-1) >= 0
        grad_rows = torch.zeros_like(s["rows"])
        each = (s["w"].unsqueeze(-1) * grad.unsqueeze(1)).flatten(0, 1).to(grad_rows.dtype)
        grad_rows[s["slot"].reshape(-1)[there].long()] = each[there]
        return {"out": out.to(s["out"].dtype), "grad_rows": grad_rows,
                "grad_w": (picked * grad.unsqueeze(1)).sum(-1)}
    if kind == "route":
        there = s["idx"] < s["E"]
        w, gw = s["w"], torch.where(there, s["grad_w"], 0.0)
        each = w * (gw - (w * gw).sum(1, keepdim=True))
        grad = torch.zeros(T, s["E"] + 1, device=w.device)
        return grad.scatter_(1, s["idx"].long(), each)[:, :-1].to(s["grad"].dtype)
    if not s["live"]:
        shapes = ("out", "z") if kind == "mm" else ("grad_a", "grad_weight", "grad_bias")
        return {k: torch.zeros_like(s[k]) for k in shapes if s[k] is not None}
    weight = s["weight"][s["order"]].float()
    if kind == "mm":
        y = torch.bmm(_padded(_inputs(s), s), weight.transpose(1, 2))
        if s["bias"] is not None:
            y = y + s["bias"][s["order"]].float().unsqueeze(1)
        z = y
        if s["swiglu"]:
            gate, up = z.chunk(2, -1)
            y = gate / (1 + torch.exp(-gate)) * up
        if s["residual"] is not None:
            y = y + _padded(s["residual"], s)
        out = {"out": _whole(y, s, s["out"].dtype)}
        return out | {"z": _whole(z, s, s["z"].dtype)} if s["z"] is not None else out
    grad = _padded(s["grad"], s)
    grad_a = torch.bmm(grad, weight)
    if s["swiglu"]:
        gate, up = _padded(s["z"], s).chunk(2, -1)
        sig = 1 / (1 + torch.exp(-gate))
        grad_a = torch.cat([grad_a * up * sig * (1 + gate * (1 - sig)), grad_a * gate * sig], -1)
    grad_weight = torch.zeros_like(s["grad_weight"])
    grad_weight[s["order"]] = torch.bmm(grad.transpose(1, 2).contiguous(),
                                        _padded(_inputs(s), s)).to(grad_weight.dtype)
    out = {"grad_a": _whole(grad_a, s, s["grad_a"].dtype), "grad_weight": grad_weight}
    if s["bias"]:
        out["grad_bias"] = torch.zeros_like(s["grad_bias"])
        out["grad_bias"][s["order"]] = grad.sum(1).to(out["grad_bias"].dtype)
    return out


# ---- the library's calls --------------------------------------------------------------------
def _own(s):
    from quantized_expert_grouped_amd import abi
    kind = s["kind"]
    if kind == "dispatch":
        abi.dispatch_rows(s["x"], s["src"], s["rows"], K=s["K"])
        abi.combine_rows(s["grad_rows"], s["slot"], None, s["grad_x"])
        return {k: s[k] for k in ("rows", "grad_x")}
    if kind == "combine":
        abi.combine_rows(s["rows"], s["slot"], s["w"], s["out"], residual=s["residual"])
        abi.combine_rows_backward(s["grad_out"], s["slot"], s["w"], s["grad_rows"], rows=s["rows"],
                                  grad_w=s["grad_w"])
        return {k: s[k] for k in ("out", "grad_rows", "grad_w")}
    if kind == "route":
        abi.route_topk_backward(s["idx"], s["w"], s["grad_w"], s["grad"])
        return s["grad"]
    src = s["src"] if s["gather"] else None
    if kind == "mm":
        abi.mm_grouped(s["weight"], s["offsets"], s["a"], s["out"], src=src, K=s["K"],
                       bias=s["bias"], swiglu=s["swiglu"], residual=s["residual"], z=s["z"])
        return {k: s[k] for k in ("out", "z") if s[k] is not None}
    if "ws" not in s:
        s["ws"] = torch.empty(abi.mm_grouped_wgrad_workspace_size(s["T"] * s["K"], s["N"], s["Kin"],
                                                                  s["E"]),
                              dtype=torch.uint8, device="cuda")
    abi.mm_grouped_dgrad(s["weight"], s["offsets"], s["grad"], s["grad_a"], z=s["z"])
    abi.mm_grouped_wgrad(s["grad"], s["offsets"], s["a"], s["grad_weight"], s["ws"], src=src,
                         K=s["K"], grad_bias=s["grad_bias"])
    return {k: s[k] for k in ("grad_a", "grad_weight", "grad_bias") if s[k] is not None}


def run(state):
    return _own(state) if own else _plain(state)


# ---- what a pass cannot do without ----------------------------------------------------------
def _active(case, routes):
    """The experts that the routes are expected to reach (exact where each takes many)."""
    E, K = case["E"], case["K"]
    p = torch.arange(1, E + 1, dtype=torch.float64).pow(-case["skew"])
    p = torch.clamp(K * p / p.sum(), max=1.0)
    return float((1 - (1 - p).pow(routes / K)).sum())


def work(case):
    kind, T, E, K = case["kind"], case["T"], case["E"], case["K"]
    size = 4 if case["dtype"] == "float32" else 2
    live = T * K * (1 - case["pad"])
    if kind == "route":
        return {"bytes": T * E * size + T * K * 12, "flops": T * K * 4}
    if kind == "dispatch":
        H = case["H"]
        return {"bytes": 2 * (T + live) * H * size + 2 * T * K * 4, "flops": live * H}
    out = 4 if case["out"] == "float32" else 2
    if kind == "combine":
        H = case["H"]
        tokens = (2 + case["residual"]) * T * H * out
        return {"bytes": tokens + 2 * live * H * size + T * K * 12, "flops": 5 * live * H}
    N, Kin = case["N"], case["Kin"]
    rows_in = T * (1 - case["pad"]) if case["gather"] else live
    active = _active(case, live)
    if kind == "mm":
        mats = 2 if case["swiglu"] else 1
        return {"bytes": active * mats * N * (Kin + case["bias"]) * 2 + rows_in * Kin * 2
                + live * N * out * (1 + case["residual"]) + live * 2 * N * 2 * case["keep"],
                "flops": 2 * live * mats * N * Kin}
    through = 4 if case["swiglu"] else 1  # gate and up read, their gradients written
    return {"bytes": active * N * Kin * 2 + live * N * 2 + live * Kin * 2 * through
            + rows_in * Kin * 2 + E * N * (Kin + case["bias"]) * out,
            "flops": 4 * live * N * Kin}


# ---- the definition in 64 bits --------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    kind, T, E, K = case["kind"], case["T"], case["E"], case["K"]
    f64 = torch.float64

    def zeros(*shape):
        return torch.zeros(shape, dtype=f64, device="cuda")

    if kind == "route":
        grad = zeros(T, E)
        gw = s["grad_w"].double() * (s["idx"] < E)
        w = s["w"].double()
        mean = (w * gw).sum(1)
        tokens = torch.arange(T, device="cuda")
        for k in range(K):
            at = s["idx"][:, k].long()
            ok = at < E
            grad[tokens[ok], at[ok]] = (w[:, k] * (gw[:, k] - mean))[ok]
        return grad
    live = int(s["offsets"][-1])
    route = s["src"][:live].long()  # of each live row
    token = route // K
    if kind == "dispatch":
        rows, grad_x = zeros(T * K, case["H"]), zeros(T, case["H"])
        rows[:live] = s["x"].double()[token]
        grad_x.index_add_(0, token, s["grad_rows"][:live].double())
        return {"rows": rows, "grad_x": grad_x}
    if kind == "combine":
        rows, grad = s["rows"][:live].double(), s["grad_out"].double()
        w = s["w"].double().reshape(-1)[route].unsqueeze(1)
        out = zeros(T, case["H"]) if s["residual"] is None else s["residual"].double()
        out.index_add_(0, token, rows * w)
        grad_rows, grad_w = zeros(T * K, case["H"]), zeros(T * K)
        grad_rows[:live] = w * grad[token]
        grad_w[route] = (rows * grad[token]).sum(1)
        return {"out": out, "grad_rows": grad_rows, "grad_w": grad_w.view(T, K)}
    at = s["offsets"].tolist()
    N, Kin = case["N"], case["Kin"]
    a = s["a"][token] if case["gather"] else s["a"]
    if kind == "mm":
        z = zeros(T * K, s["weight"].shape[1])
        for e in range(E):
            r = slice(at[e], at[e + 1])
            if at[e + 1] > at[e]:
                z[r] = a[r].double() @ s["weight"][e].double().t().contiguous()
                if s["bias"] is not None:
                    z[r] += s["bias"][e].double()
        out = z[:, :N] * torch.sigmoid(z[:, :N]) * z[:, N:] if case["swiglu"] else z.clone()
        if s["residual"] is not None:
            out[:live] += s["residual"][:live].double()
        return {"out": out} | ({"z": z} if s["z"] is not None else {})
    grad_a, grad_weight = zeros(T * K, Kin), zeros(E, N, Kin)
    grad_bias = zeros(E, N)
    for e in range(E):
        r = slice(at[e], at[e + 1])
        if at[e + 1] > at[e]:
            grad = s["grad"][r].double()
            grad_a[r] = grad @ s["weight"][e].double()
            grad_weight[e] = grad.t().contiguous() @ a[r].double()
            grad_bias[e] = grad.sum(0)
    if case["swiglu"]:
        gate, up = s["z"].double().chunk(2, 1)
        sig = torch.sigmoid(gate)
        grad_a = torch.cat([grad_a * up * sig * (1 + gate - gate * sig), grad_a * gate * sig], 1)
    out = {"grad_a": grad_a, "grad_weight": grad_weight}
    return out | {"grad_bias": grad_bias} if case["bias"] else out
