"""Cases of the operators around the expert-parallel path: the router and its
gradient, the products grouped by expert (forward, input and weight gradients,
with the gated activation between them), and the products of a few rows per
expert with 4-bit weights.

Rows are grouped by expert as a receive buffer holds them: expert e has c_e
rows at off_e, its block padded to the alignment A, padding rows zero.
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def listed():
    return [
        # one decode step's routing: 8 groups of 32 experts, 4 groups kept, a selection bias per expert
        {"name": "router decode", "op": "router", "T": 128, "E": 256, "K": 8, "groups": 8, "kept": 4,
         "score": "sigmoid", "normalize": True, "bias": True, "dtype": "fp32"},
        # the routing of a training batch of 16,384 tokens
        {"name": "router batch", "op": "router", "T": 16384, "E": 256, "K": 8, "groups": 8, "kept": 4,
         "score": "sigmoid", "normalize": True, "bias": True, "dtype": "fp32"},
        # its gradient: only the chosen experts' logits have one
        {"name": "router bwd sigmoid", "op": "router_bwd", "T": 16384, "E": 256, "K": 8, "groups": 8, "kept": 4,
         "score": "sigmoid", "normalize": True, "bias": True, "dtype": "fp32"},
        # a softmax over all experts, not renormalised: every logit has a gradient; logits as a bf16 gate gives them
        {"name": "router bwd softmax", "op": "router_bwd", "T": 8192, "E": 128, "K": 8, "groups": 1, "kept": 1,
         "score": "softmax", "normalize": False, "bias": False, "dtype": "bf16"},
        # gate and up products of a decode batch: a few rows per expert, bound by the weights' bytes
        {"name": "up decode", "op": "up", "T": 128, "H": 7168, "F": 2048, "E": 64, "K": 2, "A": 1,
         "dtype": "bf16", "skew": 0.5, "masked": 0.1},
        # the same of a training batch of which one rank holds 32 experts
        {"name": "up batch", "op": "up", "T": 8192, "H": 7168, "F": 2048, "E": 32, "K": 2, "A": 128,
         "dtype": "bf16", "skew": 0.3, "masked": 0.0},
        # down product in 32 bits, as a numerical reference run uses it
        {"name": "down fp32", "op": "down", "T": 1000, "H": 1024, "F": 1024, "E": 8, "K": 2, "A": 16,
         "dtype": "fp32", "skew": 0.3, "masked": 0.0},
        # backward of the down product and the activation: few large experts, fp16
        {"name": "down bwd fp16", "op": "down_bwd", "T": 4096, "H": 4096, "F": 2048, "E": 8, "K": 2, "A": 128,
         "dtype": "fp16", "wtype": "fp16", "skew": 0.3, "masked": 0.0},
        # backward of the gate and up products: many small experts, weight gradients kept in 32 bits
        {"name": "up bwd", "op": "up_bwd", "T": 8192, "H": 2048, "F": 1024, "E": 128, "K": 8, "A": 128,
         "dtype": "bf16", "wtype": "fp32", "skew": 0.3, "masked": 0.0},
        # one token's gate and up products with 4-bit weights
        {"name": "w4 up one token", "op": "w4_up", "T": 1, "H": 7168, "F": 2048, "E": 64, "K": 8, "A": 1,
         "dtype": "bf16", "group": 128, "skew": 0.0, "masked": 0.0},
        # a decode batch's down products with 4-bit weights
        {"name": "w4 down decode", "op": "w4_down", "T": 128, "H": 7168, "F": 2048, "E": 64, "K": 8, "A": 1,
         "dtype": "bf16", "group": 128, "skew": 0.3, "masked": 0.5},
        # a few tokens on a smaller layer, fp16, fine groups
        {"name": "w4 up few fp16", "op": "w4_up", "T": 5, "H": 2048, "F": 1024, "E": 128, "K": 8, "A": 1,
         "dtype": "fp16", "group": 32, "skew": 0.3, "masked": 0.0},
    ]


def _size(rng, lo, hi):
    """An odd number or a power of two between lo and hi, spread over the logarithm."""
    n = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return int(n) | 1 if rng.random() < 0.7 else 2 ** int(round(math.log2(n)))


def draw(rng):
    op = rng.choice(["router", "router_bwd", "up", "down", "up_bwd", "down_bwd", "w4_up", "w4_down"])
    if op in ("router", "router_bwd"):
        groups = rng.choice([1, 1, 2, 4, 8])
        E = groups * _size(rng, 2, 512 // groups)
        score = rng.choice(["softmax", "sigmoid"])
        kept = rng.randint(1, groups)
        return {"op": op, "T": _size(rng, 1, 16384), "E": E, "K": rng.randint(1, min(8, kept * (E // groups))),
                "groups": groups, "kept": kept, "score": score, "normalize": rng.random() < 0.5,
                "bias": score == "sigmoid" and rng.random() < 0.5, "dtype": rng.choice(["fp32", "bf16", "fp16"])}
    E = _size(rng, 1, 64)
    case = {"op": op, "E": E, "K": rng.randint(1, min(8, E)), "A": rng.choice([1, 1, 8, 50, 128]),
            "skew": rng.choice([0.0, 0.3, 0.6]), "masked": rng.choice([0.0, 0.2])}
    if op.startswith("w4"):
        case = {**case, "T": _size(rng, 1, 256), "H": 128 * _size(rng, 4, 56), "F": 128 * _size(rng, 2, 20),
                "dtype": rng.choice(["bf16", "fp16"]), "group": rng.choice([32, 64, 128])}
    else:
        dtype = rng.choice(["bf16", "bf16", "bf16", "fp16", "fp16", "fp32"])
        case = {**case, "T": _size(rng, 1, 8192 if dtype != "fp32" else 1024), "H": 8 * _size(rng, 16, 896),
                "F": 8 * _size(rng, 16, 256), "dtype": dtype}
        if op.endswith("bwd"):
            case["wtype"] = rng.choice([dtype, "fp32"])
    while work(case)["flops"] > (5e10 if case["dtype"] == "fp32" else 1e12):
        case["T"] = case["T"] // 2 | 1
    while work(case)["bytes"] > 2e9:
        case["E"] = case["E"] // 2
        case["K"] = min(case["K"], case["E"])
    return case


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _randn(g, *shape, dtype=torch.float32, scale=1.0):
    return (torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32) * scale).to(dtype)


def _weights(g, E, N, K, dtype):
    w = torch.empty(E, N, K, dtype=dtype, device="cuda")
    for e in range(E):
        w[e] = _randn(g, N, K, dtype=dtype, scale=K ** -0.5)
    return w


def _route(g, c):
    """topk_idx of a router whose experts differ in popularity; a share of the routes masked."""
    z = _randn(g, c["T"], c["E"]) + c["skew"] * _randn(g, c["E"])
    idx = torch.topk(z, c["K"], dim=1).indices
    return idx.masked_fill(torch.rand(idx.shape, generator=g, device="cuda") < c["masked"], -1).contiguous()


def _plan(idx, E, A):
    """Offsets and counts of the receive blocks, and the rows of each used expert side by side
    ([used experts, longest] row numbers, R where an expert has fewer)."""
    T, K = idx.shape
    R = T * K + min(E, T * K) * (A - 1)
    counts = torch.bincount(idx.reshape(-1) + 1, minlength=E + 1)[1:]
    padded = (counts + A - 1) // A * A
    offsets = torch.cat([torch.zeros(1, dtype=torch.int64, device="cuda"), torch.cumsum(padded, 0)])
    used = torch.nonzero(counts)[:, 0]
    j = torch.arange(max(1, int(counts.max())), device="cuda")
    rows = torch.where(j[None, :] < counts[used, None], offsets[used, None] + j[None, :], R)
    return {"R": R, "counts": counts, "offsets": offsets, "used": used, "rows": rows}


def _live(p):
    r = torch.zeros(p["R"] + 1, 1, dtype=torch.bool, device="cuda")
    r[p["rows"].reshape(-1)] = True
    return r[:-1]


def _recv(g, p, width, dtype):
    x = _randn(g, p["R"], width, dtype=dtype)
    return x.masked_fill(~_live(p), 0)


def prepare(case, seed):
    g = _gen(seed)
    c = dict(case)
    dt = TYPES[c["dtype"]]
    s = {"case": c}
    if c["op"] in ("router", "router_bwd"):
        T, E, K = c["T"], c["E"], c["K"]
        s["logits"] = _randn(g, T, E, dtype=dt, scale=1.5)
        s["bias"] = _randn(g, E, scale=0.1) if c["bias"] else None
        if c["op"] == "router":
            s["topk_idx"] = torch.empty(T, K, dtype=torch.int64, device="cuda")
            s["topk_weights"] = torch.empty(T, K, dtype=torch.float32, device="cuda")
        else:
            s["topk_idx"], s["topk_weights"] = _router_plain(s["logits"], s["bias"], c)
            s["grad"] = _randn(g, T, K)
            s["grad_logits"] = torch.empty(T, E, dtype=dt, device="cuda")
        return s
    E, H, F, A = c["E"], c["H"], c["F"], c["A"]
    idx = _route(g, c)
    p = _plan(idx, E, A)
    R = p["R"]
    s.update(p)
    if c["op"] == "up":
        s["x"], s["w"] = _recv(g, p, H, dt), _weights(g, E, 2 * F, H, dt)
        s["pre"], s["act"] = (torch.zeros(R, n, dtype=dt, device="cuda") for n in (2 * F, F))
    elif c["op"] == "down":
        s["x"], s["w"] = _recv(g, p, F, dt), _weights(g, E, H, F, dt)
        s["y"] = torch.zeros(R, H, dtype=dt, device="cuda")
    elif c["op"] == "down_bwd":
        s["dy"], s["pre"], s["w"] = _recv(g, p, H, dt), _recv(g, p, 2 * F, dt), _weights(g, E, H, F, dt)
        gate, up = s["pre"].float().chunk(2, dim=1)
        s["act"] = (gate / (1 + torch.exp(-gate)) * up).to(dt)
        s["dpre"] = torch.zeros(R, 2 * F, dtype=dt, device="cuda")
        s["dw"] = torch.zeros(E, H, F, dtype=TYPES[c["wtype"]], device="cuda")
    elif c["op"] == "up_bwd":
        s["dpre"], s["x"], s["w"] = _recv(g, p, 2 * F, dt), _recv(g, p, H, dt), _weights(g, E, 2 * F, H, dt)
        s["dx"] = torch.zeros(R, H, dtype=dt, device="cuda")
        s["dw"] = torch.zeros(E, 2 * F, H, dtype=TYPES[c["wtype"]], device="cuda")
    else:
        n, k = (2 * F, H) if c["op"] == "w4_up" else (H, F)
        s["x"] = _recv(g, p, k, dt)
        s["wq"] = torch.randint(0, 256, (E, n, k // 2), generator=g, device="cuda", dtype=torch.uint8)
        s["scales"] = ((0.5 + torch.rand(E, n, k // c["group"], generator=g, device="cuda")) * (0.2 * k ** -0.5)).to(dt)
        s["y"] = torch.zeros(R, F if c["op"] == "w4_up" else n, dtype=dt, device="cuda")
    if own:  # the routing map of the step, as dispatch has used it by then
        import combine_ep_prepare_gb300 as ep
        lid, size = ep.ep_register_layer(E, c["K"], H, c["T"], A, dtype=dt)
        s["handle"] = ep.alloc_handle(lid, size)
        s["token_counts"] = torch.empty(E, dtype=torch.int32, device="cuda")
        ep.ep_prepare(s["handle"], idx, s["token_counts"], A)
    return s


def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_own(s):
    import combine_ep_prepare_gb300 as ep
    c, op = s["case"], s["case"]["op"]
    if op == "router":
        ep.ep_router(s["logits"], s["topk_idx"], s["topk_weights"], bias=s["bias"], score=c["score"],
                     normalize=c["normalize"], num_groups=c["groups"], topk_groups=c["kept"])
        return {"topk_idx": s["topk_idx"], "topk_weights": s["topk_weights"]}
    if op == "router_bwd":
        ep.ep_router_bwd(s["logits"], s["topk_idx"], s["grad"], s["grad_logits"], score=c["score"],
                         normalize=c["normalize"])
        return {"grad_logits": s["grad_logits"]}
    h = s["handle"]
    if op == "up":
        ep.ep_expert_gemm_swiglu(h, s["x"], s["w"], s["act"], pre=s["pre"])
        return {"pre": s["pre"], "act": s["act"]}
    if op == "down":
        ep.ep_expert_gemm(h, s["x"], s["w"], s["y"])
        return {"y": s["y"]}
    if op == "down_bwd":
        ep.ep_expert_dgrad_swiglu(h, s["dy"], s["w"], s["pre"], s["dpre"])
        ep.ep_expert_wgrad(h, s["dy"], s["act"], s["dw"])
        return {"dpre": s["dpre"], "dw": s["dw"]}
    if op == "up_bwd":
        ep.ep_expert_dgrad(h, s["dpre"], s["w"], s["dx"])
        ep.ep_expert_wgrad(h, s["dpre"], s["x"], s["dw"])
        return {"dx": s["dx"], "dw": s["dw"]}
    if op == "w4_up":
        ep.ep_expert_gemv_w4_swiglu(h, s["x"], s["wq"], s["scales"], s["y"])
    else:
        ep.ep_expert_gemv_w4(h, s["x"], s["wq"], s["scales"], s["y"])
    return {"y": s["y"]}


# ---- plain forms: elementary operations in 32 bits, one rounding at the end

def _router_plain(logits, bias, c):
    z = logits.float()
    T, E = z.shape
    if c["score"] == "sigmoid":
        score = 1 / (1 + torch.exp(-z))
        v = score if bias is None else score + bias
    else:
        v = z
    v = v.masked_fill(z == -math.inf, -math.inf)
    if c["groups"] > 1:
        per = E // c["groups"]
        best = torch.sort(v.view(T, c["groups"], per), dim=2, descending=True).values
        value = best[:, :, 0] + best[:, :, 1] if per > 1 else best[:, :, 0]
        order = torch.sort(value, dim=1, descending=True, stable=True).indices
        keep = torch.zeros(T, c["groups"], dtype=torch.bool, device=z.device)
        keep.scatter_(1, order[:, :c["kept"]], True)
        v = v.masked_fill(~keep.repeat_interleave(per, dim=1), -math.inf)
    top = torch.sort(v, dim=1, descending=True, stable=True)
    idx = top.indices[:, :c["K"]].contiguous()
    if c["score"] == "sigmoid":
        w = torch.gather(score, 1, idx)
        w = w / w.sum(1, keepdim=True) if c["normalize"] else w
    else:
        e = torch.exp(z - z.max(1, keepdim=True).values)
        w = torch.gather(e, 1, idx)
        w = w / (w.sum(1, keepdim=True) if c["normalize"] else e.sum(1, keepdim=True))
    return idx, w.contiguous()


def _router_bwd_plain(logits, idx, grad, c):
    z = logits.float()
    d = torch.zeros_like(z)
    if c["score"] == "sigmoid":
        score = 1 / (1 + torch.exp(-torch.gather(z, 1, idx)))
        g = grad
        if c["normalize"]:
            total = score.sum(1, keepdim=True)
            g = (grad - (grad * score).sum(1, keepdim=True) / total) / total
        return d.scatter(1, idx, g * score * (1 - score)).to(logits.dtype)
    e = torch.exp(z - z.max(1, keepdim=True).values)
    if c["normalize"]:
        w = torch.gather(e, 1, idx)
        w = w / w.sum(1, keepdim=True)
        return d.scatter(1, idx, w * (grad - (grad * w).sum(1, keepdim=True))).to(logits.dtype)
    p = e / e.sum(1, keepdim=True)
    inner = (torch.gather(p, 1, idx) * grad).sum(1, keepdim=True)
    return (p * (d.scatter(1, idx, grad) - inner)).to(logits.dtype)


def _blocks(t, s):
    """The rows of each used expert, [used experts, longest, width], zeros where it has fewer."""
    t = torch.cat([t, torch.zeros(1, t.shape[1], dtype=t.dtype, device=t.device)])
    return t[s["rows"]].float()


def _rows(b, s, dtype):
    out = torch.zeros(s["R"] + 1, b.shape[2], dtype=dtype, device=b.device)
    out[s["rows"].reshape(-1)] = b.reshape(-1, b.shape[2]).to(dtype)
    return out[:-1]


def _swiglu(pre):
    gate, up = pre.chunk(2, dim=2)
    return gate / (1 + torch.exp(-gate)) * up


def _wgrad(dy, x, s, dtype):
    dw = torch.zeros(s["case"]["E"], dy.shape[2], x.shape[2], dtype=dtype, device=dy.device)
    dw[s["used"]] = torch.bmm(dy.transpose(1, 2), x).to(dtype)
    return dw


def _run_plain(s):
    c, op = s["case"], s["case"]["op"]
    if op == "router":
        idx, w = _router_plain(s["logits"], s["bias"], c)
        return {"topk_idx": idx, "topk_weights": w}
    if op == "router_bwd":
        return {"grad_logits": _router_bwd_plain(s["logits"], s["topk_idx"], s["grad"], c)}
    dt = TYPES[c["dtype"]]
    if op in ("w4_up", "w4_down"):
        q = s["wq"][s["used"]]
        q = torch.stack([q & 15, q >> 4], dim=3).flatten(2).float() - 8
        w = (q.unflatten(2, (-1, c["group"])) * s["scales"][s["used"]].float()[..., None]).flatten(2)
        y = torch.bmm(_blocks(s["x"], s), w.transpose(1, 2))
        return {"y": _rows(_swiglu(y) if op == "w4_up" else y, s, dt)}
    w = s["w"][s["used"]].float()
    if op == "up":
        pre = torch.bmm(_blocks(s["x"], s), w.transpose(1, 2))
        return {"pre": _rows(pre, s, dt), "act": _rows(_swiglu(pre), s, dt)}
    if op == "down":
        return {"y": _rows(torch.bmm(_blocks(s["x"], s), w.transpose(1, 2)), s, dt)}
    wt = TYPES[c["wtype"]]
    if op == "up_bwd":
        d = _blocks(s["dpre"], s)
        return {"dx": _rows(torch.bmm(d, w), s, dt), "dw": _wgrad(d, _blocks(s["x"], s), s, wt)}
    dy = _blocks(s["dy"], s)
    da = torch.bmm(dy, w)
    gate, up = _blocks(s["pre"], s).chunk(2, dim=2)
    sig = 1 / (1 + torch.exp(-gate))
    dpre = torch.cat([da * up * sig * (1 + gate * (1 - sig)), da * gate * sig], dim=2)
    return {"dpre": _rows(dpre, s, dt), "dw": _wgrad(dy, _blocks(s["act"], s), s, wt)}


# ---- what a pass cannot do without

def work(case):
    c = case
    el = {"bf16": 2, "fp16": 2, "fp32": 4}
    b = el[c["dtype"]]
    if c["op"] == "router":
        T, E, K = c["T"], c["E"], c["K"]
        return {"bytes": T * E * b + T * K * 12, "flops": T * E * 4}
    if c["op"] == "router_bwd":
        T, E, K = c["T"], c["E"], c["K"]
        dense = c["score"] == "softmax" and not c["normalize"]
        return {"bytes": (T * E if dense else T * K) * b + T * K * 12 + T * E * b, "flops": T * (E if dense else K) * 6}
    E, H, F = c["E"], c["H"], c["F"]
    rows = int(round(c["T"] * c["K"] * (1 - c["masked"])))
    used = E * (1 - (1 - 1 / E) ** rows) if E > 1 else min(rows, 1)  # experts with a row, routes spread evenly
    if c["T"] == 1:
        used = min(E, rows)
    if c["op"] == "up":
        return {"bytes": b * (rows * (H + 3 * F) + used * 2 * F * H), "flops": 2 * rows * 2 * F * H}
    if c["op"] == "down":
        return {"bytes": b * (rows * (H + F) + used * F * H), "flops": 2 * rows * F * H}
    if c["op"] == "down_bwd":
        return {"bytes": b * (rows * (H + 5 * F) + used * F * H) + el[c["wtype"]] * E * F * H, "flops": 4 * rows * F * H}
    if c["op"] == "up_bwd":
        return {"bytes": b * (rows * (2 * F + 2 * H) + used * 2 * F * H) + el[c["wtype"]] * E * 2 * F * H,
                "flops": 4 * rows * 2 * F * H}
    n, k, out = (2 * F, H, F) if c["op"] == "w4_up" else (H, F, H)
    return {"bytes": used * n * (k / 2 + b * k / c["group"]) + b * rows * (k + out), "flops": 2 * rows * n * k}


# ---- the same in 64 bits, expert by expert and from the formulas

def _exact_router(s):
    c = s["case"]
    z = s["logits"].double().cpu()
    T, E = z.shape
    sg = torch.sigmoid(z)
    v = z
    if c["score"] == "sigmoid":
        v = sg + s["bias"].double().cpu() if c["bias"] else sg
    if c["groups"] > 1:
        per = E // c["groups"]
        grouped = v.reshape(T, c["groups"], per)
        first = torch.topk(grouped, min(2, per), dim=2).values.sum(2)
        dropped = torch.argsort(-first, dim=1, stable=True)[:, c["kept"]:]
        v = grouped.scatter(1, dropped[:, :, None].expand(-1, -1, per), -math.inf).reshape(T, E)
    idx = torch.topk(v, c["K"], dim=1).indices
    if c["score"] == "sigmoid":
        w = sg.gather(1, idx)
        return w / w.sum(1, keepdim=True) if c["normalize"] else w
    if c["normalize"]:
        return torch.softmax(z.gather(1, idx), dim=1)
    return torch.softmax(z, dim=1).gather(1, idx)


def exact(case, seed):
    s = prepare(case, seed)
    c, op = s["case"], case["op"]
    if op == "router":
        return {"topk_idx": None, "topk_weights": _exact_router(s)}
    if op == "router_bwd":
        z, grad, idx = s["logits"].double().cpu().requires_grad_(), s["grad"].double().cpu(), s["topk_idx"].cpu()
        if c["score"] == "sigmoid":
            w = torch.sigmoid(z).gather(1, idx)
            w = w / w.sum(1, keepdim=True) if c["normalize"] else w
        else:
            w = torch.softmax(z.gather(1, idx), 1) if c["normalize"] else torch.softmax(z, 1).gather(1, idx)
        return {"grad_logits": torch.autograd.grad((w * grad).sum(), z)[0]}
    E, H, F, R = c["E"], c["H"], c["F"], s["R"]
    start, count = s["offsets"].tolist(), s["counts"].tolist()
    new = lambda *shape: torch.zeros(*shape, dtype=torch.float64, device="cuda")  # noqa: E731
    spans = [(e, slice(start[e], start[e] + count[e])) for e in range(E) if count[e]]
    if op in ("up", "w4_up"):
        pre, act = new(R, 2 * F), new(R, F)
    for_y = new(R, H) if op in ("down", "w4_down") else None
    dpre = new(R, 2 * F) if op == "down_bwd" else None
    dx = new(R, H) if op == "up_bwd" else None
    dw = new(*s["dw"].shape) if op.endswith("bwd") else None
    for e, r in spans:
        if op.startswith("w4"):
            q = s["wq"][e].to(torch.int64)
            w = torch.empty(q.shape[0], 2 * q.shape[1], dtype=torch.float64, device="cuda")
            w[:, 0::2], w[:, 1::2] = (q % 16 - 8).double(), (q // 16 - 8).double()
            w *= s["scales"][e].double().repeat_interleave(c["group"], dim=1)
        else:
            w = s["w"][e].double()
        if op in ("up", "w4_up"):
            pre[r] = s["x"][r].double() @ w.t()
            act[r] = torch.nn.functional.silu(pre[r, :F]) * pre[r, F:]
        elif op in ("down", "w4_down"):
            for_y[r] = s["x"][r].double() @ w.t()
        elif op == "up_bwd":
            d = s["dpre"][r].double()
            dx[r], dw[e] = d @ w, d.t() @ s["x"][r].double()
        else:
            dy = s["dy"][r].double()
            p = s["pre"][r].double().requires_grad_()
            a = torch.nn.functional.silu(p[:, :F]) * p[:, F:]
            dpre[r] = torch.autograd.grad(a, p, dy @ w)[0]
            dw[e] = dy.t() @ s["act"][r].double()
    if op == "up":
        return {"pre": pre, "act": act}
    if op == "w4_up":
        return {"y": act}
    if op in ("down", "w4_down"):
        return {"y": for_y}
    return {"dx": dx, "dw": dw} if op == "up_bwd" else {"dpre": dpre, "dw": dw}
