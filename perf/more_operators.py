"""Cases of the 8-bit expert path and of a few tokens' whole layer: the
root-mean-square norm with the residual's addition and an 8-bit output, its
gradient, the quantisation and dispatch of 8-bit rows, the products grouped by
expert in 8-bit floating point with a scale for each block of 128 (forward and
input gradient, gated and not), and a whole MoE layer for a few tokens.

8-bit values are e4m3.  A row has one float32 scale for each 128 of its
features, a weight matrix one for each 128 x 128 block; rows of scales are
padded to a multiple of four.  Quantising a block with largest magnitude m (at
least 2^-100): scale m / 448, values x * (448 / m) rounded to e4m3, the quotient
and the product rounded to float32 before (they decide where a value lies on the
border between two others, which a 16-bit x often does).

Rows are grouped by expert as a receive buffer holds them: expert e has c_e
rows at off_e, its block padded to the alignment A, padding rows zero.
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
F8 = torch.float8_e4m3fn
EPS = 1e-6


def listed():
    return [
        # the norm in front of an expert layer, one decode step: sum, 16-bit rows for the router, 8-bit rows to dispatch
        {"name": "norm decode", "op": "norm", "T": 128, "H": 7168, "dtype": "bf16", "residual": True, "y": True},
        # the same of a training batch of 16,384 tokens
        {"name": "norm batch", "op": "norm", "T": 16384, "H": 7168, "dtype": "bf16", "residual": True, "y": True},
        # its gradient, with the gradient that comes down the residual stream
        {"name": "norm bwd batch", "op": "norm_bwd", "T": 8192, "H": 7168, "dtype": "bf16", "through": True},
        # a small batch's, fp16, rows of an odd number of blocks, nothing down the residual stream
        {"name": "norm bwd fp16", "op": "norm_bwd", "T": 1001, "H": 2176, "dtype": "fp16", "through": False},
        # tokens to 8 bits and to their experts: a decode step with masked routes
        {"name": "dispatch decode", "op": "dispatch", "T": 128, "H": 7168, "E": 256, "K": 8, "A": 1, "dtype": "bf16",
         "skew": 0.0, "masked": 0.5},
        # a training batch
        {"name": "dispatch batch", "op": "dispatch", "T": 8192, "H": 7168, "E": 256, "K": 8, "A": 128, "dtype": "bf16",
         "skew": 0.3, "masked": 0.0},
        # gate and up products of a decode batch, result in 8 bits: a few rows per expert, bound by the weights' bytes
        {"name": "up decode", "op": "up", "T": 128, "H": 7168, "F": 2048, "E": 64, "K": 2, "A": 1, "dtype": "bf16",
         "skew": 0.5, "masked": 0.1},
        # the same of a training batch of which one rank holds 32 experts
        {"name": "up batch", "op": "up", "T": 8192, "H": 7168, "F": 2048, "E": 32, "K": 2, "A": 128, "dtype": "bf16",
         "skew": 0.3, "masked": 0.0},
        # down products of few large experts, fp16 results
        {"name": "down fp16", "op": "down", "T": 4096, "H": 4096, "F": 2048, "E": 8, "K": 2, "A": 128, "dtype": "fp16",
         "skew": 0.3, "masked": 0.0},
        # backward of the down product and the activation, many experts: the gradient rows to 8 bits, then the product
        {"name": "down bwd", "op": "down_bwd", "T": 8192, "H": 2048, "F": 1024, "E": 128, "K": 8, "A": 128, "dtype": "bf16",
         "skew": 0.3, "masked": 0.0},
        # one token through a whole layer, 16-bit weights: latency counts
        {"name": "few one token", "op": "few", "T": 1, "H": 2048, "F": 1024, "E": 128, "K": 8, "groups": 1, "kept": 1,
         "score": "softmax", "normalize": True, "bias": False, "dtype": "bf16", "weights": "16"},
        # sixteen tokens through a large layer, 8-bit weights, grouped sigmoid routing
        {"name": "few 16 f8", "op": "few", "T": 16, "H": 7168, "F": 2048, "E": 64, "K": 8, "groups": 8, "kept": 4,
         "score": "sigmoid", "normalize": True, "bias": True, "dtype": "bf16", "weights": "f8"},
    ]


def _size(rng, lo, hi):
    """An odd number or a power of two between lo and hi, spread over the logarithm."""
    n = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return int(n) | 1 if rng.random() < 0.7 else 2 ** int(round(math.log2(n)))


def draw(rng):
    op = rng.choice(["norm", "norm_bwd", "dispatch", "up", "down", "up_bwd", "down_bwd", "few", "few"])
    if op in ("norm", "norm_bwd"):
        case = {"op": op, "T": _size(rng, 1, 16384), "H": 16 * _size(rng, 4, 512), "dtype": rng.choice(["bf16", "bf16", "fp16", "fp32"])}
        return {**case, "residual": rng.random() < 0.7, "y": rng.random() < 0.5} if op == "norm" else {**case, "through": rng.random() < 0.7}
    if op == "few":
        groups = rng.choice([1, 1, 2, 4])
        E = groups * _size(rng, 2, 128 // groups)
        score, kept = rng.choice(["softmax", "sigmoid"]), rng.randint(1, groups)
        case = {"op": op, "T": _size(rng, 1, 32), "E": E, "K": rng.randint(1, min(8, kept * (E // groups))), "groups": groups,
                "kept": kept, "score": score, "normalize": rng.random() < 0.5, "bias": score == "sigmoid" and rng.random() < 0.5,
                "dtype": rng.choice(["bf16", "fp16"]), "weights": rng.choice(["16", "f8"])}
        if case["weights"] == "f8":
            case.update(H=16 * _size(rng, 16, 448), F=128 * _size(rng, 1, 16))
        else:
            case.update(H=8 * _size(rng, 16, 896), F=8 * _size(rng, 16, 256))
        while work(case)["bytes"] > 2.5e9:
            case["T"] = case["T"] // 2 | 1
        return case
    E = _size(rng, 1, 64)
    case = {"op": op, "E": E, "K": rng.randint(1, min(8, E)), "A": rng.choice([1, 1, 8, 50, 128]),
            "skew": rng.choice([0.0, 0.3, 0.6]), "masked": rng.choice([0.0, 0.2]), "dtype": rng.choice(["bf16", "bf16", "fp16"]),
            "T": _size(rng, 1, 8192), "H": 16 * _size(rng, 8, 448)}
    if op != "dispatch":
        case["F"] = 16 * _size(rng, 8, 128) if op == "down" else 128 * _size(rng, 1, 16)
    while work(case)["flops"] > 9e11 or work(case)["bytes"] > 1.2e9:
        case["T"] = case["T"] // 2 | 1
        if case["T"] < 64:
            case["E"] = max(1, case["E"] // 2)
            case["K"] = min(case["K"], case["E"])
    return case


# ---- inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _randn(g, *shape, dtype=torch.float32, scale=1.0):
    return (torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32) * scale).to(dtype)


def _route(g, c):
    """topk_idx of a router whose experts differ in popularity; a share of the routes masked."""
    z = _randn(g, c["T"], c["E"]) + c["skew"] * _randn(g, c["E"])
    idx = torch.topk(z, c["K"], dim=1).indices
    return idx.masked_fill(torch.rand(idx.shape, generator=g, device="cuda") < c["masked"], -1).contiguous()


def _plan(idx, E, A):
    """Offsets and counts of the receive blocks, the row of each route, and the rows of each used expert side by side
    ([used experts, longest] row numbers, R where an expert has fewer)."""
    T, K = idx.shape
    R = T * K + min(E, T * K) * (A - 1)
    flat = idx.reshape(-1)
    counts = torch.bincount(flat + 1, minlength=E + 1)[1:]
    padded = (counts + A - 1) // A * A
    offsets = torch.cat([torch.zeros(1, dtype=torch.int64, device="cuda"), torch.cumsum(padded, 0)])
    starts = torch.cat([torch.zeros(1, dtype=torch.int64, device="cuda"), torch.cumsum(counts, 0)])
    order = torch.sort(torch.where(flat < 0, E, flat), stable=True).indices[:int(counts.sum())]
    e = flat[order]
    place = torch.full((T * K,), R, dtype=torch.int64, device="cuda")
    place[order] = offsets[e] + torch.arange(order.numel(), device="cuda") - starts[e]
    used = torch.nonzero(counts)[:, 0]
    j = torch.arange(max(1, int(counts.max())), device="cuda")
    rows = torch.where(j[None, :] < counts[used, None], offsets[used, None] + j[None, :], R)
    live = torch.zeros(R + 1, 1, dtype=torch.bool, device="cuda")
    live[rows.reshape(-1)] = True
    return {"R": R, "counts": counts, "offsets": offsets, "used": used, "rows": rows, "place": place, "live": live[:-1]}


def _columns(n):
    """Scales of a row of n features: one for each 128, padded to a multiple of four."""
    return ((n + 127) // 128 + 3) // 4 * 4


def _blocks_of(n):
    return (n + 127) // 128


def _quantize(x):
    """Rows [T, n] in 32 bits to e4m3 and one scale for each 128 features."""
    T, n = x.shape
    b = torch.nn.functional.pad(x, (0, _blocks_of(n) * 128 - n)).view(T, -1, 128)
    m = b.abs().amax(2).clamp_min(2.0 ** -100)
    q = (b * (torch.full_like(m, 448) / m)[:, :, None]).clamp(-448, 448).to(F8).view(T, -1)[:, :n].contiguous()
    return q, torch.nn.functional.pad(m / 448, (0, _columns(n) - _blocks_of(n)))


def _weights8(g, E, N, K):
    """Weights in 8 bits with one scale for each 128 x 128 block, as a trained model's file holds them."""
    w = torch.empty(E, N, K, dtype=F8, device="cuda")
    for e in range(E):
        w[e] = (torch.randn(N, K, generator=g, device="cuda") * 100).clamp(-448, 448).to(F8)
    s = (0.5 + torch.rand(E, _blocks_of(N), _blocks_of(K), generator=g, device="cuda")) * (0.01 * K ** -0.5)
    return w, s


def _weights16(g, E, N, K, dtype):
    w = torch.empty(E, N, K, dtype=dtype, device="cuda")
    for e in range(E):
        w[e] = _randn(g, N, K, dtype=dtype, scale=K ** -0.5)
    return w


def _recv8(g, p, width):
    q, s = _quantize(_randn(g, p["R"], width))
    return torch.where(p["live"], q.float(), 0).to(F8), s * p["live"]


def prepare(case, seed):
    g = _gen(seed)
    c = dict(case)
    dt = TYPES[c["dtype"]]
    s = {"case": c}
    new = lambda *shape, dtype=dt: torch.zeros(*shape, dtype=dtype, device="cuda")  # noqa: E731
    T, H, op = c["T"], c["H"], c["op"]
    if op in ("norm", "norm_bwd"):
        s["x"] = _randn(g, T, H, dtype=dt, scale=1.5)
        s["w"] = (1 + 0.2 * _randn(g, H)).to(dt)
        if op == "norm":
            s["residual"] = _randn(g, T, H, dtype=dt, scale=2.0) if c["residual"] else None
            s["sum"] = new(T, H) if c["residual"] else None
            s["y"] = new(T, H) if c["y"] else None
            s["q"], s["scales"] = new(T, H, dtype=F8), new(T, _columns(H), dtype=torch.float32)
        else:
            s["dy"] = _randn(g, T, H, dtype=dt)
            s["dsum"] = _randn(g, T, H, dtype=dt) if c["through"] else None
            s["dx"], s["dw"] = new(T, H), new(H, dtype=torch.float32)
            if own:
                import combine_ep_prepare_gb300 as ep
                s["work"] = ep.rmsnorm_bwd_workspace(T, H)
        return s
    E, K = c["E"], c["K"]
    if op == "few":
        F = c["F"]
        s["x"], s["gate"] = _randn(g, T, H, dtype=dt), _randn(g, E, H, dtype=dt, scale=1.5 * H ** -0.5)
        s["bias"] = _randn(g, E, scale=0.1) if c["bias"] else None
        if c["weights"] == "f8":
            (s["w13"], s["s13"]), (s["w2"], s["s2"]) = _weights8(g, E, 2 * F, H), _weights8(g, E, H, F)
        else:
            s["w13"], s["w2"], s["s13"], s["s2"] = _weights16(g, E, 2 * F, H, dt), _weights16(g, E, H, F, dt), None, None
        s["idx"], s["weights"], s["y"] = new(T, K, dtype=torch.int64), new(T, K, dtype=torch.float32), new(T, H)
        if own:
            import combine_ep_prepare_gb300 as ep
            s["work"] = ep.moe_few_workspace(E, K, H, F, T)
        return s
    idx, A = _route(g, c), c["A"]
    p = _plan(idx, E, A)
    s.update(p)
    R = p["R"]
    if op == "dispatch":
        s["idx"], s["x"], s["weights"] = idx, _randn(g, T, H, dtype=dt), torch.rand(T, K, generator=g, device="cuda")
        s["q"], s["scales"] = new(T, H, dtype=F8), new(T, _columns(H), dtype=torch.float32)
        s["recv"], s["recv_scales"], s["recv_weights"] = new(R, H, dtype=F8), new(R, _columns(H), dtype=torch.float32), new(R, dtype=torch.float32)
    elif op == "up":
        F = c["F"]
        s["x"], s["xs"] = _recv8(g, p, H)
        s["w"], s["ws"] = _weights8(g, E, 2 * F, H)
        s["act"], s["act_scales"] = new(R, F, dtype=F8), new(R, _columns(F), dtype=torch.float32)
    elif op == "down":
        F = c["F"]
        s["x"], s["xs"] = _recv8(g, p, F)
        s["w"], s["ws"] = _weights8(g, E, H, F)
        s["y"] = new(R, H)
    else:
        F = c["F"]
        N, Kw = (2 * F, H) if op == "up_bwd" else (H, F)
        s["dy"] = _randn(g, R, N, dtype=dt).masked_fill(~p["live"], 0)
        s["w"], s["ws"] = _weights8(g, E, N, Kw)
        s["pre"] = _randn(g, R, 2 * F, dtype=dt).masked_fill(~p["live"], 0) if op == "down_bwd" else None
        s["q"], s["scales"] = new(R, N, dtype=F8), new(R, _columns(N), dtype=torch.float32)
        s["dx"] = new(R, 2 * F if op == "down_bwd" else H)
    if own:  # the routing map of the step
        import combine_ep_prepare_gb300 as ep
        lid, size = ep.ep_register_layer(E, K, H, T, A, dtype=dt)
        s["handle"] = ep.alloc_handle(lid, size)
        s["token_counts"] = torch.empty(E, dtype=torch.int32, device="cuda")
        ep.ep_prepare(s["handle"], idx, s["token_counts"], A)
    return s


def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_own(s):
    import combine_ep_prepare_gb300 as ep
    c, op = s["case"], s["case"]["op"]
    if op == "norm":
        ep.ep_rmsnorm(s["x"], s["w"], residual=s["residual"], sum=s["sum"], y=s["y"], q=s["q"], scales=s["scales"], eps=EPS)
        return {k: s[k] for k in ("sum", "y", "q", "scales") if s[k] is not None}
    if op == "norm_bwd":
        ep.ep_rmsnorm_bwd(s["dy"], s["x"], s["w"], s["dx"], s["dw"], s["work"], grad_sum=s["dsum"], eps=EPS)
        return {"dx": s["dx"], "dw": s["dw"]}
    if op == "few":
        ep.ep_moe_few(s["x"], s["gate"], s["w13"], s["w2"], s["y"], s["idx"], s["weights"], s["work"], s13=s["s13"], s2=s["s2"],
                      bias=s["bias"], score=c["score"], normalize=c["normalize"], num_groups=c["groups"], topk_groups=c["kept"])
        return {"y": s["y"], "topk_idx": s["idx"], "topk_weights": s["weights"]}
    h = s["handle"]
    if op == "dispatch":
        ep.ep_quantize_rows(s["x"], s["q"], s["scales"])
        ep.ep_dispatch_f8(h, s["idx"], s["q"], s["scales"], s["weights"], s["recv"], s["recv_scales"], s["recv_weights"])
        return {k: s[k] for k in ("recv", "recv_scales", "recv_weights")}
    if op == "up":
        ep.ep_expert_gemm_f8_swiglu(h, s["x"], s["xs"], s["w"], s["ws"], act_q=s["act"], act_scales=s["act_scales"])
        return {"act": s["act"], "act_scales": s["act_scales"]}
    if op == "down":
        ep.ep_expert_gemm_f8(h, s["x"], s["xs"], s["w"], s["ws"], s["y"])
        return {"y": s["y"]}
    ep.ep_expert_quantize(h, s["dy"], s["q"], s["scales"])
    if op == "up_bwd":
        ep.ep_expert_dgrad_f8(h, s["q"], s["scales"], s["w"], s["ws"], s["dx"])
    else:
        ep.ep_expert_dgrad_f8_swiglu(h, s["q"], s["scales"], s["w"], s["ws"], s["pre"], s["dx"])
    return {"dx": s["dx"], "q": s["q"], "scales": s["scales"]}


# ---- plain forms: elementary operations in 32 bits, one rounding at the end

def _values(q, scales):
    """What 8-bit rows stand for, in 32 bits."""
    n = q.shape[-1]
    return q.float() * scales.repeat_interleave(128, dim=-1)[..., :n]


def _weight_values(w, scales):
    N, K = w.shape[-2:]
    return w.float() * scales.repeat_interleave(128, dim=-2)[..., :N, :].repeat_interleave(128, dim=-1)[..., :K]


def _blocks(t, s):
    """The rows of each used expert, [used experts, longest, width], zeros where it has fewer."""
    t = torch.cat([t, torch.zeros(1, t.shape[1], dtype=t.dtype, device=t.device)])
    return t[s["rows"]]


def _rows(b, s):
    out = torch.zeros(s["R"] + 1, b.shape[2], device=b.device)
    out[s["rows"].reshape(-1)] = b.reshape(-1, b.shape[2])
    return out[:-1]


def _sigmoid(z):
    return 1 / (1 + torch.exp(-z))


def _router_plain(z, bias, c):
    T, E = z.shape
    score = _sigmoid(z)
    v = z if c["score"] == "softmax" else score if bias is None else score + bias
    if c["groups"] > 1:
        per = E // c["groups"]
        best = torch.sort(v.view(T, c["groups"], per), dim=2, descending=True).values
        value = best[:, :, 0] + best[:, :, min(1, per - 1)]
        order = torch.sort(value, dim=1, descending=True, stable=True).indices
        keep = torch.zeros(T, c["groups"], dtype=torch.bool, device=z.device).scatter_(1, order[:, :c["kept"]], True)
        v = v.masked_fill(~keep.repeat_interleave(per, dim=1), -math.inf)
    idx = torch.sort(v, dim=1, descending=True, stable=True).indices[:, :c["K"]].contiguous()
    if c["score"] == "sigmoid":
        w = torch.gather(score, 1, idx)
        return idx, w / w.sum(1, keepdim=True) if c["normalize"] else w
    e = torch.exp(z - z.max(1, keepdim=True).values)
    w = torch.gather(e, 1, idx)
    return idx, w / (w.sum(1, keepdim=True) if c["normalize"] else e.sum(1, keepdim=True))


def _few_plain(s):
    c, f8 = s["case"], s["case"]["weights"] == "f8"
    x = s["x"].float()
    # logits in 64 bits: the choice turns on values next to a border
    idx, p = _router_plain((s["x"].double() @ s["gate"].double().t()).float(), s["bias"], c)
    used = torch.unique(idx)
    w13, w2 = s["w13"][used], s["w2"][used]
    w13, w2 = (_weight_values(w13, s["s13"][used]), _weight_values(w2, s["s2"][used])) if f8 else (w13.float(), w2.float())
    x = _values(*_quantize(x)) if f8 else x
    gate, up = (x @ w13.transpose(1, 2)).chunk(2, dim=2)  # [used experts, tokens, F]
    a = gate * _sigmoid(gate) * up
    a = _values(*_quantize(a.flatten(0, 1))).view(a.shape) if f8 else a
    share = (p[None, :, :] * (idx[None, :, :] == used[:, None, None])).sum(2)  # [used experts, tokens]
    y = (torch.bmm(a, w2.transpose(1, 2)) * share[:, :, None]).sum(0)
    return {"y": y.to(s["x"].dtype), "topk_idx": idx, "topk_weights": p.contiguous()}


def _run_plain(s):
    c, op = s["case"], s["case"]["op"]
    dt = TYPES[c["dtype"]]
    if op == "norm":
        h = s["x"].float()
        out = {}
        if s["residual"] is not None:
            out["sum"] = (h + s["residual"].float()).to(dt)
            h = out["sum"].float()
        y = h / torch.sqrt((h * h).mean(1, keepdim=True) + EPS) * s["w"].float()
        if s["y"] is not None:
            out["y"] = y.to(dt)
        out["q"], out["scales"] = _quantize(y)
        return out
    if op == "norm_bwd":
        h, dy, w = s["x"].float(), s["dy"].float(), s["w"].float()
        r = 1 / torch.sqrt((h * h).mean(1, keepdim=True) + EPS)
        dx = r * (dy * w - h * r * r * (dy * w * h).mean(1, keepdim=True))
        dx = dx if s["dsum"] is None else dx + s["dsum"].float()
        return {"dx": dx.to(dt), "dw": (dy * h * r).double().sum(0).float()}
    if op == "few":
        return _few_plain(s)
    if op == "dispatch":
        q, scales = _quantize(s["x"].float())
        token = torch.arange(c["T"] * c["K"], device=q.device) // c["K"]
        recv, recv_scales = torch.zeros(s["R"] + 1, c["H"], device=q.device), torch.zeros(s["R"] + 1, scales.shape[1], device=q.device)
        weights = torch.zeros(s["R"] + 1, device=q.device)
        recv[s["place"]], recv_scales[s["place"]], weights[s["place"]] = q.float()[token], scales[token], s["weights"].reshape(-1)
        return {"recv": recv[:-1].to(F8), "recv_scales": recv_scales[:-1], "recv_weights": weights[:-1]}
    w = _weight_values(s["w"][s["used"]], s["ws"][s["used"]])
    if op in ("up", "down"):
        y = torch.bmm(_blocks(_values(s["x"], s["xs"]), s), w.transpose(1, 2))
        if op == "down":
            return {"y": _rows(y, s).to(dt)}
        gate, up = y.chunk(2, dim=2)
        q, scales = _quantize(_rows(gate * _sigmoid(gate) * up, s))
        return {"act": q, "act_scales": scales * s["live"]}
    q, scales = _quantize(s["dy"].float())
    scales = scales * s["live"]
    dx = torch.bmm(_blocks(_values(q, scales), s), w)
    if op == "down_bwd":
        gate, up = _blocks(s["pre"].float(), s).chunk(2, dim=2)
        sg = _sigmoid(gate)
        dx = torch.cat([dx * up * sg * (1 + gate * (1 - sg)), dx * gate * sg], dim=2)
    return {"dx": _rows(dx, s).to(dt), "q": q, "scales": scales}


# ---- what a pass cannot do without

def work(case):
    c = case
    b, T, H, op = {"bf16": 2, "fp16": 2, "fp32": 4}[c["dtype"]], c["T"], c["H"], c["op"]
    scaled = lambda n: n + 4 * _blocks_of(n)  # noqa: E731  bytes of an 8-bit row with its scales
    if op == "norm":
        return {"bytes": T * (H * b * (1 + 2 * c["residual"] + c["y"]) + scaled(H)) + H * b, "flops": T * H * 8}
    if op == "norm_bwd":
        return {"bytes": T * H * b * (3 + c["through"]) + H * (b + 4), "flops": T * H * 10}
    E, K = c["E"], c["K"]
    if op == "few":
        F, rows, f8 = c["F"], T * K, c["weights"] == "f8"
        used = E * (1 - (1 - K / E) ** T)  # experts that some token chooses, choices spread evenly
        matrix = H * F * (1 + 4 / 16384) if f8 else H * F * b
        return {"bytes": used * 3 * matrix + E * H * b + T * (2 * H * b + 12 * K), "flops": 2 * rows * 3 * H * F + 2 * T * E * H}
    rows = int(round(T * K * (1 - c["masked"])))
    if op == "dispatch":
        return {"bytes": T * H * b + rows * (scaled(H) + 8), "flops": T * H * 3}
    F = c["F"]
    used = E * (1 - (1 - 1 / E) ** rows) if E > 1 else min(rows, 1)  # experts with a row, routes spread evenly
    if T == 1:
        used = min(E, rows)
    N, Kw = (2 * F, H) if op in ("up", "up_bwd") else (H, F)
    weights = used * (N * Kw + 4 * _blocks_of(N) * _blocks_of(Kw))
    if op == "up":
        return {"bytes": weights + rows * (scaled(H) + scaled(F)), "flops": 2 * rows * N * Kw}
    if op == "down":
        return {"bytes": weights + rows * (scaled(F) + H * b), "flops": 2 * rows * N * Kw}
    into = N * b + scaled(N) + (4 * F * b if op == "down_bwd" else H * b)
    return {"bytes": weights + rows * into, "flops": 2 * rows * N * Kw}


# ---- the same in 64 bits, from the formulas, expert by expert

def _exact_quantize(x):
    """(unrounded values, scales, what the rounded values stand for) of rows in 64 bits."""
    T, n = x.shape
    values, scales, stands = torch.empty_like(x), torch.zeros(T, _columns(n), dtype=torch.float64, device=x.device), torch.empty_like(x)
    for i, at in enumerate(range(0, n, 128)):
        b = x[:, at:at + 128]
        m = torch.maximum(b.abs().max(dim=1, keepdim=True).values, torch.tensor(2.0 ** -100, dtype=torch.float64, device=x.device))
        values[:, at:at + 128], scales[:, i:i + 1] = b / m * 448, m / 448
        stands[:, at:at + 128] = (b.float() * (torch.full_like(m, 448) / m).float()).to(F8).double() * m / 448  # a border's side as defined
    return values, scales, stands


def _exact_values(q, scales):
    n = q.shape[-1]
    return q.double() * scales.double()[..., torch.arange(n, device=q.device) // 128]


def _exact_weight(w, s):
    i, j = (torch.arange(n, device=w.device) // 128 for n in w.shape)
    return w.double() * s.double()[i][:, j]


def _exact_few(s):
    c, f8 = s["case"], s["case"]["weights"] == "f8"
    x, T = s["x"].double(), s["case"]["T"]
    z = x @ s["gate"].double().t()
    v = z
    if c["score"] == "sigmoid":
        v = torch.sigmoid(z) + (s["bias"].double() if c["bias"] else 0)
    if c["groups"] > 1:
        per = c["E"] // c["groups"]
        grouped = v.reshape(T, c["groups"], per)
        first = torch.topk(grouped, min(2, per), dim=2).values.sum(2)
        dropped = torch.argsort(-first, dim=1, stable=True)[:, c["kept"]:]
        v = grouped.scatter(1, dropped[:, :, None].expand(-1, -1, per), -math.inf).reshape(T, c["E"])
    idx = torch.topk(v, c["K"], dim=1).indices
    if c["score"] == "sigmoid":
        p = torch.sigmoid(z).gather(1, idx)
        p = p / p.sum(1, keepdim=True) if c["normalize"] else p
    else:
        p = torch.softmax(z.gather(1, idx), 1) if c["normalize"] else torch.softmax(z, 1).gather(1, idx)
    x = _exact_quantize(x)[2] if f8 else x
    y = torch.zeros_like(s["y"], dtype=torch.float64)
    for e in torch.unique(idx).tolist():
        t, k = torch.nonzero(idx == e, as_tuple=True)
        w13 = _exact_weight(s["w13"][e], s["s13"][e]) if f8 else s["w13"][e].double()
        w2 = _exact_weight(s["w2"][e], s["s2"][e]) if f8 else s["w2"][e].double()
        gate, up = (x[t] @ w13.t()).chunk(2, dim=1)
        a = torch.nn.functional.silu(gate) * up
        a = _exact_quantize(a)[2] if f8 else a
        y.index_add_(0, t, (a @ w2.t()) * p[t, k][:, None])
    return {"y": y, "topk_idx": None, "topk_weights": p}


def exact(case, seed):
    s = prepare(case, seed)
    c, op = s["case"], case["op"]
    if op == "norm":
        out = {}
        h = s["x"].double()
        if c["residual"]:
            h = h + s["residual"].double()
            out["sum"] = h
            h = h.to(s["x"].dtype).double()
        y = h * torch.rsqrt(h.square().mean(1, keepdim=True) + EPS) * s["w"].double()
        if c["y"]:
            out["y"] = y
        out["q"], out["scales"], _ = _exact_quantize(y)
        return out
    if op == "norm_bwd":
        h, w = s["x"].double().requires_grad_(), s["w"].double().requires_grad_()
        y = h * torch.rsqrt(h.square().mean(1, keepdim=True) + EPS) * w
        dx, dw = torch.autograd.grad(y, (h, w), s["dy"].double())
        return {"dx": dx + s["dsum"].double() if c["through"] else dx, "dw": dw}
    if op == "few":
        return _exact_few(s)
    if op == "dispatch":
        values, scales, _ = _exact_quantize(s["x"].double())
        f64 = dict(dtype=torch.float64, device="cuda")
        recv, recv_scales, weights = (torch.zeros(s["R"], n, **f64) for n in (c["H"], scales.shape[1], 1))
        flat = torch.nonzero(s["place"] < s["R"])[:, 0]
        to = s["place"][flat]
        recv[to], recv_scales[to] = values[flat // c["K"]], scales[flat // c["K"]]
        weights[to, 0] = s["weights"].double().reshape(-1)[flat]
        return {"recv": recv, "recv_scales": recv_scales, "recv_weights": weights[:, 0]}
    start, count = s["offsets"].tolist(), s["counts"].tolist()
    spans = [(e, slice(start[e], start[e] + count[e])) for e in range(c["E"]) if count[e]]
    new = lambda n: torch.zeros(s["R"], n, dtype=torch.float64, device="cuda")  # noqa: E731
    if op in ("up", "down"):
        out = new(c["F"] if op == "up" else c["H"])
        for e, r in spans:
            y = _exact_values(s["x"][r], s["xs"][r]) @ _exact_weight(s["w"][e], s["ws"][e]).t()
            out[r] = torch.nn.functional.silu(y[:, :c["F"]]) * y[:, c["F"]:] if op == "up" else y
        if op == "down":
            return {"y": out}
        values, scales, _ = _exact_quantize(out)
        return {"act": values, "act_scales": scales * s["live"]}
    values, scales, stands = _exact_quantize(s["dy"].double())
    dx = new(s["dx"].shape[1])
    for e, r in spans:
        d = stands[r] @ _exact_weight(s["w"][e], s["ws"][e])
        if op == "down_bwd":
            p = s["pre"][r].double().requires_grad_()
            a = torch.nn.functional.silu(p[:, :c["F"]]) * p[:, c["F"]:]
            d = torch.autograd.grad(a, p, d)[0]
        dx[r] = d
    return {"dx": dx, "q": values, "scales": scales * s["live"]}
