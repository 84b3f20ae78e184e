"""The operators of a layer of experts around the Muon step, as cases to be timed and compared: the router's choice of
experts with its gradient, the order of the tokens by expert with the weighted sum of what the experts return, the
product with bias, activation and residual (of one matrix or of one a group of rows) with its gradients, and dropout.

`own` chooses the side: False computes each operator from elementary torch operations in 32 bits (64 where a choice
falls next to a border), True calls this package.  `exact` gives the definition in 64 bits, written apart from the
plain form.
"""

import math

import torch

own = False

DEV = "cuda:0"
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
IT = {"int32": torch.int32, "int64": torch.int64}
BYTES = {"bf16": 2, "fp32": 4, "int32": 4, "int64": 8}
NORM_EPS = 1e-20  # added to the sum of the chosen scores that weights are divided by
ACTS = ("none", "relu", "silu", "gelu", "gelu_tanh")


# ------------------------------------------------------------------ cases


def listed():
    return [
        # one short micro-batch through a small model's residual branch: latency counts
        {"name": "dropout 33 x 1024", "op": "dropout", "rows": 33, "cols": 1024, "dtype": "fp32", "p": 0.1,
         "residual": True},
        # a training batch of a wide model, added to the residual stream
        {"name": "dropout 16384 x 8192", "op": "dropout", "rows": 16384, "cols": 8192, "dtype": "bf16", "p": 0.1,
         "residual": True},
        # a few tokens of a small mixture: softmax, the two best of eight, odd count
        {"name": "route 61 x 8", "op": "route", "tokens": 61, "experts": 8, "k": 2, "dtype": "bf16", "ids": "int64",
         "scoring": "softmax", "bias": False, "groups": 1, "keep": 1, "top": 1, "renorm": True, "scale": 1.0,
         "pad": 0.0, "first": True},
        # a global batch of a fine-grained mixture: sigmoid scores, a balancing bias, half of eight groups, eight
        # choices; padded tokens route nowhere
        {"name": "route 131072 x 256", "op": "route", "tokens": 131072, "experts": 256, "k": 8, "dtype": "fp32",
         "ids": "int32", "scoring": "sigmoid", "bias": True, "groups": 8, "keep": 4, "top": 2, "renorm": True,
         "scale": 2.5, "pad": 0.1, "first": True},
        # the tokens of a small mixture sorted by expert, and the experts' rows summed, forwards and backwards
        {"name": "order and combine 509 x 2", "op": "combine", "tokens": 509, "experts": 8, "k": 2, "dim": 1024,
         "dtype": "fp32", "ids": "int64", "pad": 0.0, "residual": True},
        # the same of a fine-grained mixture
        {"name": "order and combine 16384 x 8", "op": "combine", "tokens": 16384, "experts": 256, "k": 8,
         "dim": 4096, "dtype": "bf16", "ids": "int32", "pad": 0.05, "residual": True},
        # one token through a wide layer: the weights' way through memory
        {"name": "linear 1 token", "op": "linear", "rows": 1, "in": 4096, "out": 11008, "groups": 1, "dtype": "bf16",
         "layout": "in_out", "act": "silu", "bias": True, "residual": False, "pre": False, "pad": 0.0},
        # a training batch through the first matrix of a block; what the gradient needs is kept
        {"name": "linear 8192 tokens", "op": "linear", "rows": 8192, "in": 4096, "out": 11008, "groups": 1,
         "dtype": "bf16", "layout": "in_out", "act": "gelu_tanh", "bias": True, "residual": False, "pre": True,
         "pad": 0.0},
        # 32 experts of a mixture on their sorted tokens: very uneven groups, empty ones among them
        {"name": "linear 32 experts", "op": "linear", "rows": 32768, "in": 1024, "out": 4096, "groups": 32,
         "dtype": "bf16", "layout": "out_in", "act": "silu", "bias": True, "residual": False, "pre": True,
         "pad": 0.05},
        # both gradients of the second matrix of a block, through the activation before it; odd count
        {"name": "linear gradients 4091 tokens", "op": "linear_grad", "rows": 4091, "in": 11008, "out": 4096,
         "groups": 1, "dtype": "bf16", "layout": "in_out", "act": "gelu_tanh", "bias": True, "residual": False,
         "first": True, "pad": 0.0},
        # both gradients of the experts' second matrices
        {"name": "linear gradients 32 experts", "op": "linear_grad", "rows": 32768, "in": 4096, "out": 1024,
         "groups": 32, "dtype": "bf16", "layout": "out_in", "act": "silu", "bias": True, "residual": False,
         "first": True, "pad": 0.05},
        # a small model in 32 bits, odd sizes, with the skip connection's gradient
        {"name": "linear gradients 1021 x 1000 fp32", "op": "linear_grad", "rows": 1021, "in": 1000, "out": 257,
         "groups": 1, "dtype": "fp32", "layout": "in_out", "act": "gelu", "bias": True, "residual": True,
         "first": True, "pad": 0.0},
    ]


def _log(rng, lo, hi):
    """A whole number in [lo, hi], spread over the logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["dropout", "route", "combine", "linear", "linear_grad"])
    dtype, ids = rng.choice(["bf16", "fp32"]), rng.choice(["int32", "int64"])
    if op == "dropout":
        cols = _log(rng, 64, 16384)
        return {"op": op, "rows": _log(rng, 1, max(1, (1 << 27) // (cols * BYTES[dtype] // 2))), "cols": cols,
                "dtype": dtype, "p": round(rng.uniform(0.0, 0.6), 3), "residual": rng.random() < 0.5}
    if op == "route":
        softmax = rng.random() < 0.5
        groups = rng.choice([1, 1, 4, 8])
        per = rng.randint(2, 32 if groups > 1 else 256)
        experts = groups * per
        keep = rng.randint((groups + 1) // 2, groups)
        k = rng.randint(1, min(8, keep * per))
        return {"op": op, "tokens": _log(rng, 1, (1 << 25) // max(experts, 64) // 4), "experts": experts, "k": k,
                "dtype": dtype, "ids": ids,
                "scoring": "softmax" if softmax else "sigmoid", "bias": rng.random() < 0.5, "groups": groups,
                "keep": keep, "top": rng.choice([1, 2]), "renorm": k > 1 and rng.random() < 0.7,  # one choice's share is 1
                "scale": rng.choice([1.0, 2.5]), "pad": rng.choice([0.0, 0.1]), "first": rng.random() < 0.7}
    if op == "combine":
        k, dim = rng.randint(1, 8), _log(rng, 64, 8192)
        return {"op": op, "tokens": _log(rng, 1, max(1, (1 << 28) // (k * dim * BYTES[dtype]))),
                "experts": _log(rng, max(2, k), 256), "k": k, "dim": dim, "dtype": dtype, "ids": ids,
                "pad": rng.choice([0.0, 0.1]), "residual": rng.random() < 0.5}
    groups = rng.choice([1, 1, 8, 32])
    d_in, d_out = rng.choice([_log(rng, 64, 8192), 512, 1024, 4096, 11008]), rng.choice([_log(rng, 64, 8192), 512, 1024, 4096])
    if rng.random() < 0.6:
        d_in, d_out = max(64, d_in // 8 * 8), max(64, d_out // 8 * 8)
    cap = (1 << 38) // (16 if dtype == "fp32" else 1) // (d_in * d_out * (2 if op == "linear_grad" else 1))
    case = {"op": op, "rows": _log(rng, 1, max(1, min(32768, cap))), "in": d_in, "out": d_out, "groups": groups,
            "dtype": dtype, "layout": rng.choice(["in_out", "out_in"]), "act": rng.choice(ACTS),
            "bias": rng.random() < 0.7, "residual": rng.random() < 0.5}
    if op == "linear":
        case["pre"] = case["act"] != "none" and rng.random() < 0.5
    else:
        case["first"] = rng.random() < 0.7
    case["pad"] = rng.choice([0.0, 0.1]) if groups > 1 else 0.0
    return case


def work(case):
    op, e = case["op"], BYTES[case["dtype"]]
    if op == "dropout":
        n = case["rows"] * case["cols"]
        return {"bytes": n * e * (3 if case["residual"] else 2), "flops": 2.0 * n}
    if op == "route":
        t, x, k, i = case["tokens"], case["experts"], case["k"], BYTES[case["ids"]]
        live = t * (1.0 - case["pad"])
        # forwards the logits; backwards a softmax needs the whole row, a sigmoid the chosen ones
        back = live * (x if case["scoring"] == "softmax" else k) * e + t * x * e * (1 if case["first"] else 2)
        return {"bytes": live * x * e + back + t * k * (2 * i + 8) + 2 * t, "flops": 12.0 * live * x}
    if op == "combine":
        t, k, d, i = case["tokens"], case["k"], case["dim"], BYTES[case["ids"]]
        slots = t * k * (1.0 - case["pad"])
        rows = t * (3 if case["residual"] else 2) * d * e  # the residual, the sum, the sum's gradient
        return {"bytes": 3 * slots * d * e + rows + t * k * (i + 16), "flops": 5.0 * slots * d}
    n, a, b = case["rows"] * (1.0 - case["pad"]), case["in"], case["out"]
    w = case["groups"] * a * b
    if op == "linear":
        return {"bytes": (n * a + n * b * (1 + case["pre"] + case["residual"]) + w) * e, "flops": 2.0 * n * a * b}
    by = (n * b + n * a * (2 + case["residual"] + (case["act"] != "none")) + w) * e
    return {"bytes": by + w * (4 if case["first"] else 8), "flops": 4.0 * n * a * b}


# ----------------------------------------------------------------- inputs


def _normal(shape, dtype, g, std=1.0):
    return torch.empty(shape, dtype=DT[dtype], device=DEV).normal_(0.0, std, generator=g)


def _groups(case, g):
    """First rows of the groups, uneven and some empty, with what lies behind the last; and the same on the host."""
    n, live = case["groups"], int(case["rows"] * (1.0 - case["pad"]))
    if n == 1:
        return None, [0, case["rows"]]
    share = torch.randn(n, dtype=torch.float64, device=DEV, generator=g).exp()
    share[torch.randint(0, n, (max(1, n // 16),), device=DEV, generator=g)] = 0.0
    ends = (share.cumsum(0) / share.sum() * live).round().int()
    offsets = torch.cat([torch.zeros(1, dtype=torch.int32, device=DEV), ends])
    return offsets, offsets.tolist()


def _matrix(case, g):
    """The weights, indexed [group, in, out] whichever of the two is adjacent in memory."""
    n, a, b = case["groups"], case["in"], case["out"]
    if case["layout"] == "in_out":
        w = _normal((n, a, b), case["dtype"], g, 1.0 / math.sqrt(a))
    else:
        w = _normal((n, b, a), case["dtype"], g, 1.0 / math.sqrt(a)).transpose(1, 2)
    return w[0] if n == 1 else w


def prepare(case, seed):
    g = torch.Generator(DEV).manual_seed(seed)
    s, op, dt = {"case": case}, case["op"], case["dtype"]
    if op == "dropout":
        s["x"] = _normal((case["rows"], case["cols"]), dt, g)
        s["residual"] = _normal((case["rows"], case["cols"]), dt, g) if case["residual"] else None
        s["out"] = torch.empty_like(s["x"])
        # the training step is a number on the device, which a captured graph's replays raise
        s["step"] = torch.randint(0, 1 << 20, (1,), dtype=torch.int64, device=DEV, generator=g)
        s["seed"], s["site"] = 0x9E3779B97F4A7C15 ^ seed, 5
    elif op == "route":
        t, x = case["tokens"], case["experts"]
        s["logits"] = _normal((t, x), dt, g)
        s["logits"] += (0.5 * torch.randn(x, device=DEV, generator=g)).to(DT[dt])  # some experts are favoured
        s["bias"] = 0.1 * torch.randn(x, device=DEV, generator=g) if case["bias"] else None
        s["valid"] = torch.rand(t, device=DEV, generator=g) >= case["pad"] if case["pad"] else None
        s["choices"] = torch.empty(t, case["k"], dtype=IT[case["ids"]], device=DEV)
        s["weights"] = torch.empty(t, case["k"], device=DEV)
        s["dweights"] = torch.randn(t, case["k"], device=DEV, generator=g)
        s["dlogits"] = _normal((t, x), dt, g, 0.01)  # holds the balance loss's gradient where it is added to
    elif op == "combine":
        t, k, x, d = case["tokens"], case["k"], case["experts"], case["dim"]
        score = torch.randn(t, x, device=DEV, generator=g) + 0.5 * torch.randn(x, device=DEV, generator=g)
        c = score.topk(k, 1).indices
        c[torch.rand(t, k, device=DEV, generator=g) < case["pad"]] = -1
        s["choices"] = c.to(IT[case["ids"]])
        s["tokens"] = torch.empty(t * k, dtype=torch.int32, device=DEV)
        s["place"] = torch.empty(t, k, dtype=torch.int32, device=DEV)
        s["offsets"] = torch.empty(x + 1, dtype=torch.int32, device=DEV)
        s["y"] = _normal((t * k, d), dt, g)
        s["weights"] = torch.rand(t, k, device=DEV, generator=g)
        s["residual"] = _normal((t, d), dt, g) if case["residual"] else None
        s["dout"] = _normal((t, d), dt, g)
        s["out"] = torch.empty(t, d, dtype=DT[dt], device=DEV)
        s["dy"] = torch.zeros_like(s["y"])
        s["dweights"] = torch.empty(t, k, device=DEV)
    else:
        n, a, b = case["rows"], case["in"], case["out"]
        s["offsets"], s["bounds"] = _groups(case, g)
        s["w"] = _matrix(case, g)
        s["x"] = _normal((n, a), dt, g)
        if op == "linear":
            s["bias"] = _normal((case["groups"], b) if case["groups"] > 1 else (b,), dt, g, 0.1) if case["bias"] else None
            s["residual"] = _normal((n, b), dt, g) if case["residual"] else None
            s["out"] = torch.zeros(n, b, dtype=DT[dt], device=DEV)
            s["pre"] = torch.zeros_like(s["out"]) if case["pre"] else None
        else:
            s["dy"] = _normal((n, b), dt, g, 0.02)
            s["pre"] = _normal((n, a), dt, g) if case["act"] != "none" else None
            s["residual"] = _normal((n, a), dt, g, 0.02) if case["residual"] else None
            s["dx"] = torch.zeros(n, a, dtype=DT[dt], device=DEV)
            s["dw"] = torch.randn(s["w"].shape, device=DEV, generator=g)
            s["dbias"] = torch.randn((case["groups"], b) if case["groups"] > 1 else (b,), device=DEV,
                                     generator=g) if case["bias"] else None
    return s


# -------------------------------------------------------------- one pass


def run(state):
    return (_run_own if own else _run_plain)(state["case"]["op"], state)


def _workspace(M, op, s):
    """The workspace that a user's program keeps beside its calls of one size; made at the first of them."""
    if "ws" not in s:
        c = s["case"]
        if op == "combine":
            need = M.expert_order_workspace_bytes(c["tokens"], c["k"], c["experts"])
        elif op == "linear":
            need = M.linear_workspace_bytes(c["rows"], c["in"], c["out"], c["groups"])
        else:
            need = max(M.linear_workspace_bytes(c["rows"], c["out"], c["in"], c["groups"]),
                       M.linear_weight_grad_workspace_bytes(c["rows"], c["in"], c["out"], c["groups"]))
        s["ws"] = torch.empty(need, dtype=torch.uint8, device=DEV)
    return s["ws"]


def _run_own(op, s):
    import muon_newton_schulz_step_amd as M
    c = s["case"]
    if op == "dropout":
        M.dropout(s["x"], s["out"], c["p"], s["seed"], site=s["site"], step=s["step"], residual=s["residual"])
        return {"out": s["out"]}
    if op == "route":
        how = dict(scoring=c["scoring"], renormalize=c["renorm"], scale=c["scale"], valid=s["valid"])
        M.route_experts(s["logits"], s["choices"], s["weights"], bias=s["bias"], groups=c["groups"],
                        keep_groups=c["keep"], group_top=c["top"], **how)
        M.route_backward(s["logits"], s["choices"], s["dweights"], s["dlogits"], c["first"], **how)
        return {"choices": s["choices"], "weights": s["weights"], "dlogits": s["dlogits"]}
    if op == "combine":
        M.expert_order(s["choices"], s["tokens"], s["offsets"], s["place"], _workspace(M, op, s))
        M.expert_combine(s["y"], s["place"], s["out"], weights=s["weights"], residual=s["residual"])
        M.expert_combine_backward(s["dout"], s["place"], s["dy"], weights=s["weights"], y=s["y"],
                                  dweights=s["dweights"])
        return {"tokens": s["tokens"], "offsets": s["offsets"], "place": s["place"], "out": s["out"], "dy": s["dy"],
                "dweights": s["dweights"]}
    ws = _workspace(M, op, s)
    if op == "linear":
        M.linear_forward(s["x"], s["w"], s["out"], ws, bias=s["bias"], activation=c["act"], pre=s["pre"],
                         residual=s["residual"], offsets=s["offsets"])
        return {"out": s["out"], "pre": s["pre"]} if c["pre"] else {"out": s["out"]}
    M.linear_input_grad(s["dy"], s["w"], s["dx"], ws, pre=s["pre"], activation=c["act"], residual=s["residual"],
                        offsets=s["offsets"])
    M.linear_weight_grad(s["x"], s["dy"], s["dw"], c["first"], ws, dbias=s["dbias"], offsets=s["offsets"])
    out = {"dx": s["dx"], "dw": s["dw"]}
    return {**out, "dbias": s["dbias"]} if c["bias"] else out


def _philox(counter, key):
    """Philox4x32-10 (Salmon et al., 2011): four words of 32 bits from four of a counter and two of a key."""
    c0, c1, c2, c3 = counter
    k0, k1 = key
    low = 0xFFFFFFFF
    for _ in range(10):
        p, q = c0 * 0xD2511F53, c2 * 0xCD9E8D57  # 64-bit products, modulo 2^64
        c0, c1, c2, c3 = (q >> 32 & low) ^ c1 ^ k0, q & low, (p >> 32 & low) ^ c3 ^ k1, p & low
        k0, k1 = k0 + 0x9E3779B9 & low, k1 + 0xBB67AE85 & low
    return c0, c1, c2, c3


def _act(name, v):
    if name == "relu":
        return torch.where(v < 0.0, 0.0, v)
    if name == "silu":
        return v / (1.0 + (-v).exp())
    if name == "gelu":
        return 0.5 * v * (1.0 + torch.erf(v * math.sqrt(0.5)))
    if name == "gelu_tanh":
        return 0.5 * v * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (v + 0.044715 * v * v * v)))
    return v


def _act_slope(name, v):
    if name == "relu":
        return (v > 0.0).to(v.dtype)
    if name == "silu":
        q = 1.0 / (1.0 + (-v).exp())
        return q * (1.0 + v * (1.0 - q))
    if name == "gelu":
        return 0.5 * (1.0 + torch.erf(v * math.sqrt(0.5))) + v * (-0.5 * v * v).exp() * (1.0 / math.sqrt(2.0 * math.pi))
    if name == "gelu_tanh":
        c = math.sqrt(2.0 / math.pi)
        t = torch.tanh(c * (v + 0.044715 * v * v * v))
        return 0.5 * (1.0 + t) + 0.5 * v * (1.0 - t * t) * c * (1.0 + 0.134145 * v * v)
    return torch.ones_like(v)


def _run_plain(op, s):
    c = s["case"]
    if op == "dropout":
        rows, cols = c["rows"], c["cols"]
        quads = torch.arange((cols + 3) // 4, device=DEV).expand(rows, -1)
        row = torch.arange(rows, device=DEV)[:, None].expand(quads.shape)
        site = torch.full_like(quads, s["site"])
        words = _philox((quads, row, site, (s["step"] & 0xFFFFFFFF).expand(quads.shape)),
                        (s["seed"] & 0xFFFFFFFF, s["seed"] >> 32))
        keep = torch.stack(words, 2).reshape(rows, -1)[:, :cols] >= round(c["p"] * 2.0 ** 32)
        out = torch.where(keep, s["x"].float() * (1.0 / (1.0 - c["p"])), 0.0)
        if s["residual"] is not None:
            out = out + s["residual"].float()
        s["out"].copy_(out)
        return {"out": s["out"]}
    if op == "route":
        x = s["logits"].double()  # experts of nearly equal scores: 32 bits would pick others
        t, n = x.shape
        k = c["k"]
        if c["scoring"] == "softmax":
            e = (x - x.max(1, keepdim=True).values).exp()
            score = e / e.sum(1, keepdim=True)
        else:
            score = 1.0 / (1.0 + (-x).exp())
        rank = score if s["bias"] is None else score + s["bias"].double()
        if c["groups"] > 1:
            per = rank.view(t, c["groups"], -1)
            best = per.sort(dim=2, descending=True, stable=True).values[:, :, :c["top"]].sum(2)
            kept = best.sort(dim=1, descending=True, stable=True).indices[:, :c["keep"]]
            open_ = torch.zeros(t, c["groups"], dtype=torch.bool, device=DEV).scatter_(1, kept, True)
            rank = torch.where(open_[:, :, None], per, -math.inf).view(t, n)
        chosen = rank.sort(dim=1, descending=True, stable=True).indices[:, :k]
        ok = torch.ones(t, 1, dtype=torch.bool, device=DEV) if s["valid"] is None else s["valid"][:, None]
        score = score.float()
        picked = score.gather(1, chosen)
        total = picked.sum(1, keepdim=True) + NORM_EPS if c["renorm"] else 1.0
        s["weights"].copy_(torch.where(ok, c["scale"] * picked / total, 0.0))
        s["choices"].copy_(torch.where(ok, chosen, -1))
        dw = s["dweights"]
        ds = c["scale"] * (dw - (dw * picked).sum(1, keepdim=True) / total if c["renorm"] else dw) / total
        if c["scoring"] == "softmax":
            d = -score * (ds * picked).sum(1, keepdim=True)
            d.scatter_add_(1, chosen, ds * picked)
        else:
            d = torch.zeros_like(score).scatter_(1, chosen, ds * picked * (1.0 - picked))
        d = torch.where(ok, d, 0.0)
        s["dlogits"].copy_(d if c["first"] else d + s["dlogits"].float())
        return {"choices": s["choices"], "weights": s["weights"], "dlogits": s["dlogits"]}
    if op == "combine":
        t, k = c["tokens"], c["k"]
        flat = s["choices"].reshape(-1).long()
        flat = torch.where((flat >= 0) & (flat < c["experts"]), flat, c["experts"])
        by = flat.sort(stable=True).indices
        ends = torch.zeros(c["experts"] + 1, dtype=torch.int64, device=DEV).index_add_(0, flat, torch.ones_like(flat))
        s["offsets"].copy_(torch.cat([ends.new_zeros(1), ends[:-1].cumsum(0)]))
        at = torch.arange(t * k, device=DEV)
        live = at < s["offsets"][-1]
        s["tokens"].copy_(torch.where(live, by // k, -1))
        s["place"].view(-1)[by] = torch.where(live, at, -1).int()
        place = s["place"].long()
        has = (place >= 0)[:, :, None]
        rows = torch.where(has, s["y"][place.clamp(min=0)].float(), 0.0)
        out = (rows * s["weights"][:, :, None]).sum(1)
        s["out"].copy_(out if s["residual"] is None else out + s["residual"].float())
        s["dweights"].copy_((rows * s["dout"].float()[:, None, :]).sum(2))
        source, slot = s["tokens"].long().clamp(min=0), place.reshape(-1)
        wslot = torch.zeros(t * k + 1, device=DEV)
        wslot[torch.where(slot < 0, t * k, slot)] = s["weights"].reshape(-1)
        grad = (s["dout"].float()[source] * wslot[:-1, None]).to(s["dy"].dtype)
        s["dy"].copy_(torch.where(live[:, None], grad, s["dy"]))
        return {"tokens": s["tokens"], "offsets": s["offsets"], "place": s["place"], "out": s["out"], "dy": s["dy"],
                "dweights": s["dweights"]}
    ws = [s["w"]] if c["groups"] == 1 else list(s["w"])
    act = c["act"]
    if op == "linear":
        bias = [None] * len(ws) if s["bias"] is None else [s["bias"]] if c["groups"] == 1 else list(s["bias"])
        for w, b, lo, hi in zip(ws, bias, s["bounds"], s["bounds"][1:]):
            v = s["x"][lo:hi].float() @ w.float()
            if b is not None:
                v = v + b.float()
            if c["pre"]:
                s["pre"][lo:hi].copy_(v)
            v = _act(act, v)
            if s["residual"] is not None:
                v = v + s["residual"][lo:hi].float()
            s["out"][lo:hi].copy_(v)
        return {"out": s["out"], "pre": s["pre"]} if c["pre"] else {"out": s["out"]}
    dws = [s["dw"]] if c["groups"] == 1 else list(s["dw"])
    dbs = [None] * len(ws) if s["dbias"] is None else [s["dbias"]] if c["groups"] == 1 else list(s["dbias"])
    for w, dw, db, lo, hi in zip(ws, dws, dbs, s["bounds"], s["bounds"][1:]):
        dy = s["dy"][lo:hi].float()
        v = dy @ w.float().t()
        if act != "none":
            v = v * _act_slope(act, s["pre"][lo:hi].float())
        if s["residual"] is not None:
            v = v + s["residual"][lo:hi].float()
        s["dx"][lo:hi].copy_(v)
        part = s["x"][lo:hi].float().t() @ dy
        dw.copy_(part if c["first"] else dw + part)
        if db is not None:
            part = dy.double().sum(0).float()
            db.copy_(part if c["first"] else db + part)
    out = {"dx": s["dx"], "dw": s["dw"]}
    return {**out, "dbias": s["dbias"]} if c["bias"] else out


# ------------------------------------------------------------ definition


def _bits(rows, cols, seed, site, step):
    """The 32 random bits of each element, with 32-bit products put together from halves."""
    def mul(a, m):  # (high, low) words of a * m
        part = a * (m & 0xFFFF)
        rest = a * (m >> 16) + (part >> 16)
        return rest >> 16, (rest & 0xFFFF) << 16 | part & 0xFFFF
    quads = (cols + 3) // 4
    ctr = [torch.arange(quads, device=DEV).repeat(rows, 1), torch.arange(rows, device=DEV)[:, None].repeat(1, quads),
           torch.full((rows, quads), site, device=DEV), torch.full((rows, quads), step, device=DEV)]
    key = [seed % 2 ** 32, seed // 2 ** 32]
    for _ in range(10):
        h0, l0 = mul(ctr[0], 0xD2511F53)
        h1, l1 = mul(ctr[2], 0xCD9E8D57)
        ctr = [h1 ^ ctr[1] ^ key[0], l1, h0 ^ ctr[3] ^ key[1], l0]
        key = [(key[0] + 0x9E3779B9) % 2 ** 32, (key[1] + 0xBB67AE85) % 2 ** 32]
    return torch.stack(ctr, 2).reshape(rows, 4 * quads)[:, :cols]


def _exact_route(case, s):
    x, n, k = s["logits"].double(), case["experts"], case["k"]
    score = torch.softmax(x, 1) if case["scoring"] == "softmax" else torch.sigmoid(x)
    rank = score + (0.0 if s["bias"] is None else s["bias"].double())
    rows = torch.arange(x.shape[0], device=DEV)
    if case["groups"] > 1:
        size = n // case["groups"]
        value = rank.view(-1, case["groups"], size).topk(case["top"], 2).values.sum(2)
        closed = torch.ones(value.shape, dtype=torch.bool, device=DEV)
        for _ in range(case["keep"]):  # argmax takes any of equals; no two are equal in 64 bits but by their inputs
            top = (value == value.max(1, keepdim=True).values).int().argmax(1)
            value[rows, top] = -math.inf
            closed[rows, top] = False
        rank = rank.masked_fill(closed.repeat_interleave(size, 1), -math.inf)
    chosen = []
    for _ in range(k):
        top = (rank == rank.max(1, keepdim=True).values).int().argmax(1)
        rank = rank.index_put((rows, top), torch.tensor(-math.inf, dtype=torch.float64, device=DEV))
        chosen.append(top)
    chosen = torch.stack(chosen, 1)
    with torch.enable_grad():
        z = x.clone().requires_grad_()
        q = torch.softmax(z, 1) if case["scoring"] == "softmax" else torch.sigmoid(z)
        w = q.gather(1, chosen)
        w = case["scale"] * (w / (w.sum(1, keepdim=True) + NORM_EPS) if case["renorm"] else w)
        d, = torch.autograd.grad((w * s["dweights"].double()).sum(), z)
    w = w.detach()
    if s["valid"] is not None:
        chosen[~s["valid"]] = -1
        w[~s["valid"]] = 0.0
        d[~s["valid"]] = 0.0
    return {"choices": chosen.to(s["choices"].dtype), "weights": w,
            "dlogits": d if case["first"] else d + s["dlogits"].double()}


def _exact_combine(case, s):
    t, k = case["tokens"], case["k"]
    c = s["choices"].cpu().reshape(-1).tolist()
    lists = [[] for _ in range(case["experts"])]
    for i, e in enumerate(c):
        if 0 <= e < case["experts"]:
            lists[e].append(i)
    offsets, order = [0], []
    for part in lists:
        order += part
        offsets.append(len(order))
    slots, n = torch.tensor(order, dtype=torch.int64, device=DEV), len(order)
    tokens = torch.full((t * k,), -1, dtype=torch.int32, device=DEV)
    tokens[:n] = (slots // k).int()
    place = torch.full((t * k,), -1, dtype=torch.int32, device=DEV)
    place[slots] = torch.arange(n, dtype=torch.int32, device=DEV)
    out = torch.zeros(t, case["dim"], dtype=torch.float64, device=DEV) if s["residual"] is None else s["residual"].double()
    w, dy, dw = s["weights"].reshape(-1).double(), s["dy"].double(), torch.zeros(t * k, dtype=torch.float64, device=DEV)
    for lo in range(0, n, 16384):
        a = slots[lo:lo + 16384]
        rows, grads = s["y"][lo:lo + a.numel()].double(), s["dout"][a // k].double()
        out.index_add_(0, a // k, rows * w[a, None])
        dw[a] = (rows * grads).sum(1)
        dy[lo:lo + a.numel()] = grads * w[a, None]
    return {"tokens": tokens, "offsets": torch.tensor(offsets, dtype=torch.int32, device=DEV), "place": place.view(t, k),
            "out": out, "dy": dy, "dweights": dw.view(t, k)}


def exact(case, seed):
    """The outputs of run() from the operators' definitions, in 64 bits."""
    s, op = prepare(case, seed), case["op"]
    if op == "dropout":
        r = _bits(case["rows"], case["cols"], s["seed"], s["site"], int(s["step"]))
        out = s["x"].double() / (1.0 - case["p"])
        out[r < round(case["p"] * 2 ** 32)] = 0.0
        return {"out": out if s["residual"] is None else out + s["residual"].double()}
    if op == "route":
        return _exact_route(case, s)
    if op == "combine":
        return _exact_combine(case, s)
    F, pi = torch.nn.functional, s["bounds"]
    name = {"none": lambda v: v, "relu": F.relu, "silu": F.silu, "gelu": F.gelu,
            "gelu_tanh": lambda v: F.gelu(v, approximate="tanh")}[case["act"]]
    w = s["w"].reshape(case["groups"], case["in"], case["out"])
    if op == "linear":
        out, pre = s["out"].double(), s["out"].double()
        for i in range(case["groups"]):
            v = torch.mm(s["x"][pi[i]:pi[i + 1]].double(), w[i].double())
            if s["bias"] is not None:
                v += s["bias"].view(case["groups"], -1)[i].double()
            pre[pi[i]:pi[i + 1]] = v
            v = name(v)
            out[pi[i]:pi[i + 1]] = v if s["residual"] is None else v + s["residual"][pi[i]:pi[i + 1]].double()
        return {"out": out, "pre": pre} if case["pre"] else {"out": out}
    dx = s["dx"].double()
    dw = torch.zeros(w.shape, dtype=torch.float64, device=DEV)
    db = torch.zeros(case["groups"], case["out"], dtype=torch.float64, device=DEV)
    for i in range(case["groups"]):
        dy = s["dy"][pi[i]:pi[i + 1]].double()
        v = torch.mm(w[i].double(), dy.t()).t()
        if case["act"] != "none":
            with torch.enable_grad():
                z = s["pre"][pi[i]:pi[i + 1]].double().requires_grad_()
                v, = torch.autograd.grad(name(z), z, v.contiguous())
        dx[pi[i]:pi[i + 1]] = v if s["residual"] is None else v + s["residual"][pi[i]:pi[i + 1]].double()
        dw[i] = torch.mm(dy.t(), s["x"][pi[i]:pi[i + 1]].double()).t()
        db[i] = dy.sum(0)
    dw = dw.view(s["dw"].shape)
    out = {"dx": dx, "dw": dw if case["first"] else dw + s["dw"].double()}
    if case["bias"]:
        db = db.view(s["dbias"].shape)
        out["dbias"] = db if case["first"] else db + s["dbias"].double()
    return out
