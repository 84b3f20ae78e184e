"""The training-step operators around the Muon step, as cases to be timed and compared: embedding lookup and its
gradient, token log-probabilities, the clipped policy loss, the preference loss and the router's balance loss.

`own` chooses the side: False computes each operator from elementary torch operations in 32 bits (64 for long sums),
True calls this package.  `exact` gives the definition in 64 bits, written apart from the plain form.
"""

import math
import random

import torch

own = False

DEV = "cuda:0"
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
IT = {"int32": torch.int32, "int64": torch.int64}
BYTES = {"bf16": 2, "fp32": 4, "int32": 4, "int64": 8}
CLIP_LOW, CLIP_HIGH, KL_COEF = 0.2, 0.28, 0.05
BETA, SMOOTHING = 0.1, 0.05
BALANCE, ZCOEF = 0.01, 0.001
ZIPF = 2.7  # word frequency: rank r is met in proportion to 1 / (r + ZIPF)


# ------------------------------------------------------------------ cases


def listed():
    return [
        # a few tokens at a time, as a sampling loop between updates feeds them: latency counts
        {"name": "lookup, 7 tokens", "op": "embed", "tokens": 7, "vocab": 32000, "dim": 4096, "dtype": "bf16",
         "ids": "int64", "pad": 0.0},
        # a training batch of a wide model with a large vocabulary, right-padded sequences
        {"name": "lookup, 32768 tokens", "op": "embed", "tokens": 32768, "vocab": 131072, "dim": 8192, "dtype": "bf16",
         "ids": "int32", "pad": 0.1},
        # a short micro-batch added to an accumulator that already holds others; odd count, odd vocabulary
        {"name": "embedding gradient, 1021 tokens", "op": "embed_grad", "tokens": 1021, "vocab": 50257, "dim": 1024,
         "dtype": "fp32", "ids": "int64", "pad": 0.0, "first": False},
        # the first micro-batch of a step: the whole dense gradient is written
        {"name": "embedding gradient, 16384 tokens", "op": "embed_grad", "tokens": 16384, "vocab": 32000, "dim": 4096,
         "dtype": "bf16", "ids": "int64", "pad": 0.1, "first": True},
        # scoring the next token of a small batch over a large vocabulary
        {"name": "log-probability, 32 rows", "op": "logprob", "rows": 32, "vocab": 131072, "dtype": "bf16",
         "ids": "int64", "pad": 0.0, "dead": 0},
        # scoring a batch with fp32 logits, odd row length (rows start off 16-byte lines), some rows without a target
        {"name": "log-probability, 4093 rows", "op": "logprob", "rows": 4093, "vocab": 50257, "dtype": "fp32",
         "ids": "int64", "pad": 0.2, "dead": 0},
        # one short answer
        {"name": "policy loss, 61 rows", "op": "policy", "rows": 61, "vocab": 32000, "dtype": "bf16", "ids": "int64",
         "pad": 0.25, "dead": 0},
        # a micro-batch of answers over a large vocabulary, prompts weighted with zero
        {"name": "policy loss, 8192 rows", "op": "policy", "rows": 8192, "vocab": 131072, "dtype": "bf16",
         "ids": "int64", "pad": 0.25, "dead": 0},
        # two pairs of answers, fp32 logits whose last columns pad the vocabulary with -inf
        {"name": "preference loss, 2 pairs", "op": "preference", "pairs": 2, "length": 150, "vocab": 32064,
         "dtype": "fp32", "ids": "int64", "pad": 0.3, "dead": 64},
        # sixteen ragged pairs
        {"name": "preference loss, 16 pairs", "op": "preference", "pairs": 16, "length": 384, "vocab": 50257,
         "dtype": "bf16", "ids": "int64", "pad": 0.3, "dead": 0},
        # a small router
        {"name": "balance loss, 509 tokens", "op": "balance", "tokens": 509, "experts": 8, "k": 2, "dtype": "fp32",
         "ids": "int64", "pad": 0.1},
        # a large batch over many experts
        {"name": "balance loss, 131072 tokens", "op": "balance", "tokens": 131072, "experts": 256, "k": 8,
         "dtype": "fp32", "ids": "int64", "pad": 0.1},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    most = max(work(c)["bytes"] for c in listed())
    while True:
        op = rng.choice(["embed", "embed_grad", "logprob", "policy", "preference", "balance"])
        c = {"op": op, "dtype": rng.choice(["bf16", "bf16", "fp32"]), "ids": rng.choice(["int64", "int64", "int32"]),
             "pad": rng.choice([0.0, 0.1, 0.3])}
        if op in ("embed", "embed_grad"):
            c["tokens"] = _log_int(rng, 1, 32768)
            c["vocab"] = _log_int(rng, 1000, 131072)
            c["dim"] = rng.choice([_log_int(rng, 64, 8192), 64 * rng.randint(1, 128), 1024, 4096, 8192])
            if op == "embed_grad":
                c["first"] = rng.random() < 0.5
        elif op == "balance":
            c["tokens"] = _log_int(rng, 1, 131072)
            c["experts"] = rng.choice([8, 16, 64, 128, 256, rng.randint(3, 256)])
            c["k"] = rng.randint(1, min(8, c["experts"]))
        else:
            c["vocab"] = rng.choice([_log_int(rng, 1000, 131072), 64 * rng.randint(100, 2048), 32000, 50257])
            c["dead"] = rng.choice([0, 0, 17])
            if op == "preference":
                c["pairs"] = _log_int(rng, 1, 24)
                c["length"] = _log_int(rng, 4, 512)
            else:
                c["rows"] = _log_int(rng, 1, 8192)
        if work(c)["bytes"] <= 0.9 * most:
            return c


def _lengths(case):
    """Sequence lengths and prompt lengths of a preference case: ragged, and a matter of the case, not of the seed."""
    r = random.Random("%(pairs)d/%(length)d" % case)
    ls = [max(2, int(case["length"] * r.uniform(0.5, 1.5))) for _ in range(2 * case["pairs"])]
    return ls, [int(x * case["pad"]) for x in ls]


def _distinct(case):
    """Expected number of table rows that a case's tokens meet."""
    p = 1.0 / (torch.arange(case["vocab"], dtype=torch.float64) + ZIPF)
    n = case["tokens"] * (1.0 - case["pad"])
    return float((1.0 - (1.0 - p / p.sum()) ** n).sum())


def work(case):
    op, e, i = case["op"], BYTES[case["dtype"]], BYTES[case["ids"]]
    if op in ("embed", "embed_grad"):
        n, d = case["tokens"], case["dim"]
        live = n * (1.0 - case["pad"])
        if op == "embed":
            return {"bytes": n * i + _distinct(case) * d * e + n * d * e, "flops": live * d}
        out = case["vocab"] * d * 4 if case["first"] else 2 * _distinct(case) * d * 4
        return {"bytes": n * i + live * d * e + out, "flops": 2 * live * d}
    if op == "balance":
        t, x = case["tokens"], case["experts"]
        return {"bytes": t * case["k"] * i + t + t * x * e * (2.0 - case["pad"]) + x * 4, "flops": 12.0 * t * x}
    v = case["vocab"]
    if op == "preference":
        ls, ps = _lengths(case)
        n, live = sum(ls), sum(ls) - sum(ps)
    else:
        n, live = case["rows"], case["rows"] * (1.0 - case["pad"])
    if op == "logprob":
        return {"bytes": live * v * e + n * (i + 8), "flops": 5.0 * live * v}
    return {"bytes": live * v * e + n * v * e + n * (i + 16), "flops": 9.0 * live * v}


# ----------------------------------------------------------------- inputs


def _token_ids(case, n, g):
    p = 1.0 / (torch.arange(case["vocab"], dtype=torch.float64, device=DEV) + ZIPF)
    c = (p / p.sum()).cumsum(0)
    u = torch.rand(n, dtype=torch.float64, device=DEV, generator=g)
    ids = torch.searchsorted(c, u).clamp(max=case["vocab"] - 1)
    # padding: ids outside the table, which have no row and no gradient
    ids[torch.rand(n, device=DEV, generator=g) < case["pad"]] = -1
    return ids.to(IT[case["ids"]])


def _logits_and_targets(case, n, g):
    """Logits whose targets are likelier than the rest, and the targets' log-probabilities."""
    v, live = case["vocab"], case["vocab"] - case["dead"]
    x = torch.empty(n, v, dtype=DT[case["dtype"]], device=DEV).normal_(0.0, 2.0, generator=g)
    t = torch.randint(0, live, (n,), device=DEV, generator=g)
    up = torch.rand(n, 1, device=DEV, generator=g) * 10.0
    x.scatter_(1, t[:, None], (x.gather(1, t[:, None]).float() + up).to(x.dtype))
    if case["dead"]:
        x[:, live:] = -math.inf
    logp = torch.cat([torch.log_softmax(a.float(), 1).gather(1, b[:, None])[:, 0]
                      for a, b in zip(x.split(1024), t.split(1024))])
    return x, t, logp


def prepare(case, seed):
    g = torch.Generator(DEV).manual_seed(seed)
    s = {"case": case}
    op = case["op"]
    if op == "embed":
        s["ids"] = _token_ids(case, case["tokens"], g)
        s["table"] = torch.empty(case["vocab"], case["dim"], dtype=DT[case["dtype"]], device=DEV).normal_(0.0, 0.02, generator=g)
        s["out"] = torch.empty(case["tokens"], case["dim"], dtype=DT[case["dtype"]], device=DEV)
        s["scale"] = math.sqrt(case["dim"])
    elif op == "embed_grad":
        s["ids"] = _token_ids(case, case["tokens"], g)
        s["dout"] = torch.empty(case["tokens"], case["dim"], dtype=DT[case["dtype"]], device=DEV).normal_(0.0, 0.02, generator=g)
        s["acc"] = torch.empty(case["vocab"], case["dim"], dtype=torch.float32, device=DEV).normal_(0.0, 0.02, generator=g)
        s["scale"] = math.sqrt(case["dim"])
    elif op == "balance":
        n, e = case["tokens"], case["experts"]
        x = torch.empty(n, e, dtype=DT[case["dtype"]], device=DEV).normal_(0.0, 1.0, generator=g)
        x += (0.5 * torch.randn(e, device=DEV, generator=g)).to(x.dtype)  # some experts are favoured
        s["logits"] = x
        s["experts"] = x.float().topk(case["k"], 1).indices.to(IT[case["ids"]]).contiguous()
        s["valid"] = torch.rand(n, device=DEV, generator=g) >= case["pad"]
        s["counts"] = torch.empty(e, dtype=torch.int32, device=DEV)
        s["stats"] = torch.empty(3, dtype=torch.float32, device=DEV)
        s["dlogits"] = torch.empty_like(x)
    else:
        if op == "preference":
            ls, ps = _lengths(case)
            n = sum(ls)
        else:
            n = case["rows"]
        x, t, logp = _logits_and_targets(case, n, g)
        s["logits"], s["logp"] = x, torch.empty(n, dtype=torch.float32, device=DEV)
        if op == "preference":
            off = [0]
            for length in ls:
                off.append(off[-1] + length)
            at = torch.arange(n, device=DEV)
            s["offsets"] = torch.tensor(off, dtype=IT[case["ids"]], device=DEV)
            seq = torch.searchsorted(torch.tensor(off[1:], device=DEV), at, right=True)
            prompt = at - torch.tensor(off, device=DEV)[seq] < torch.tensor(ps, device=DEV)[seq]
            t[prompt] = -100  # prompt tokens are no targets
            total = torch.zeros(len(ls), dtype=torch.float64, device=DEV).index_add_(0, seq, torch.where(prompt, 0.0, logp.double()))
            # log ratios of order one per token add up like a random walk
            walk = torch.tensor(ls, dtype=torch.float64, device=DEV).sqrt()
            s["ref_logp"] = (total + walk * torch.randn(len(ls), device=DEV, generator=g, dtype=torch.float64)).float()
            s["loss"] = torch.empty(1, dtype=torch.float32, device=DEV)
            s["rewards"] = torch.empty(len(ls), dtype=torch.float32, device=DEV)
        else:
            keep = torch.rand(n, device=DEV, generator=g) >= case["pad"]
            if op == "logprob":
                t[~keep] = -100
                s["lse"] = torch.empty(n, dtype=torch.float32, device=DEV)
            else:
                lr = 0.15 * torch.randn(n, device=DEV, generator=g)
                # no ratio within rounding of the clip's ends, where the derivative jumps
                for edge in (math.log(1.0 - CLIP_LOW), math.log(1.0 + CLIP_HIGH)):
                    lr = torch.where((lr - edge).abs() < 1e-3, lr + 4e-3, lr)
                s["old_logp"] = logp - lr
                s["ref_logp"] = logp + 0.3 * torch.randn(n, device=DEV, generator=g)
                s["advantages"] = torch.randn(n, device=DEV, generator=g)
                s["weights"] = keep.float() / max(1, n)
                s["stats"] = torch.empty(4, dtype=torch.float32, device=DEV)
        s["targets"] = t.to(IT[case["ids"]])
        if op != "logprob":
            s["dlogits"] = torch.empty_like(x)
    return s


# -------------------------------------------------------------- one pass


def run(state):
    return (_run_own if own else _run_plain)(state["case"]["op"], state)


def _workspace(M, op, s):
    """The workspace that a user's program keeps beside its calls of one size; made at the first of them."""
    if "ws" not in s:
        c = s["case"]
        if op == "embed_grad":
            need = M.embed_backward_workspace_bytes(c["tokens"], c["vocab"], c["dim"])
        elif op == "policy":
            need = M.policy_loss_workspace_bytes(c["rows"])
        elif op == "preference":
            need = M.preference_loss_workspace_bytes(s["logits"].shape[0], c["pairs"])
        else:
            need = M.balance_loss_workspace_bytes(c["tokens"], c["experts"])
        s["ws"] = torch.empty(need, dtype=torch.uint8, device=DEV)
    return s["ws"]


def _run_own(op, s):
    import muon_newton_schulz_step_amd as M
    if op == "embed":
        M.embed_forward(s["table"], s["ids"], s["out"], scale=s["scale"])
        return {"out": s["out"]}
    if op == "embed_grad":
        M.embed_backward(s["ids"], s["dout"], s["acc"], s["case"]["first"], _workspace(M, op, s), scale=s["scale"])
        return {"acc": s["acc"]}
    if op == "logprob":
        M.token_logprob(s["logits"], s["targets"], s["logp"], s["lse"])
        return {"logp": s["logp"], "lse": s["lse"]}
    if op == "policy":
        M.policy_loss(s["logits"], s["targets"], s["advantages"], s["weights"], s["stats"], s["logp"], s["dlogits"],
                      _workspace(M, op, s), old_logp=s["old_logp"], ref_logp=s["ref_logp"], clip_low=CLIP_LOW, clip_high=CLIP_HIGH,
                      kl_coef=KL_COEF)
        return {"stats": s["stats"], "logp": s["logp"], "dlogits": s["dlogits"]}
    if op == "preference":
        M.preference_loss(s["logits"], s["targets"], s["offsets"], s["ref_logp"], s["loss"], s["rewards"],
                          s["dlogits"], _workspace(M, op, s), beta=BETA, label_smoothing=SMOOTHING)
        return {"loss": s["loss"], "rewards": s["rewards"], "dlogits": s["dlogits"]}
    M.balance_loss(s["logits"], s["experts"], s["counts"], s["stats"], s["dlogits"], _workspace(M, op, s),
                   valid=s["valid"], coef=BALANCE, z_coef=ZCOEF)
    return {"counts": s["counts"], "stats": s["stats"], "dlogits": s["dlogits"]}


def _row_logprob(x, targets):
    """Each row's exponentials shifted by its maximum, their sum, and its target's log-probability (from the sum on
    in 64 bits: a sequence adds up many of them, next to a reference of the same size)."""
    z = x.float()
    top = z.max(1, keepdim=True).values
    e = (z - top).exp()
    total = e.sum(1, keepdim=True)
    has = (targets >= 0) & (targets < z.shape[1])
    at = torch.where(has, targets, 0).long()[:, None]
    log_total = total.double().log()
    lse = top.double() + log_total
    logp = torch.where(has, ((z.gather(1, at) - top).double() - log_total)[:, 0], 0.0)
    return e, total, has, at, torch.where(has, lse[:, 0], 0.0), logp


def _logit_grad(e, total, at, dlogp, dtype):
    """d logits of sum(dlogp * logp): dlogp (onehot - softmax)."""
    d = (e / total) * -dlogp[:, None]
    d.scatter_add_(1, at, dlogp[:, None])
    return torch.where(dlogp[:, None] == 0.0, 0.0, d).to(dtype)


def _run_plain(op, s):
    if op == "embed":
        ids, table = s["ids"], s["table"]
        has = (ids >= 0) & (ids < table.shape[0])
        rows = table[torch.where(has, ids, 0).long()].float() * s["scale"]
        s["out"].copy_(torch.where(has[:, None], rows, 0.0))
        return {"out": s["out"]}
    if op == "embed_grad":
        ids, acc = s["ids"], s["acc"]
        has = (ids >= 0) & (ids < acc.shape[0])
        g = torch.where(has[:, None], s["dout"].float() * s["scale"], 0.0)
        if s["case"]["first"]:
            acc.zero_()
        acc.index_add_(0, torch.where(has, ids, 0).long(), g)
        return {"acc": acc}
    if op == "logprob":
        _, _, _, _, lse, logp = _row_logprob(s["logits"], s["targets"])
        return {"logp": logp.float(), "lse": lse.float()}
    if op == "policy":
        e, total, has, at, _, logp = _row_logprob(s["logits"], s["targets"])
        logp = logp.float()
        a = s["advantages"]
        w = torch.where(has, s["weights"], 0.0)
        ratio = (logp - s["old_logp"]).exp()
        clipped = ratio.clamp(1.0 - CLIP_LOW, 1.0 + CLIP_HIGH)
        active = ratio * a <= clipped * a
        d = s["ref_logp"] - logp
        kl = torch.expm1(d) - d
        pg = -torch.minimum(ratio * a, clipped * a)
        dlogp = w * (torch.where(active, -a * ratio, 0.0) - KL_COEF * torch.expm1(d))
        terms = torch.stack([w * (pg + KL_COEF * kl), w * pg, w * kl, torch.where(active, 0.0, w)])
        return {"stats": terms.double().sum(1).float(), "logp": torch.where(w != 0.0, logp, 0.0),
                "dlogits": _logit_grad(e, total, at, dlogp, s["logits"].dtype)}
    if op == "preference":
        e, total, has, at, _, logp = _row_logprob(s["logits"], s["targets"])
        n, pairs = logp.shape[0], s["ref_logp"].shape[0] // 2
        seq = torch.searchsorted(s["offsets"][1:].long(), torch.arange(n, device=logp.device), right=True)
        sums = torch.zeros(2 * pairs, dtype=torch.float64, device=logp.device).index_add_(0, seq, logp)
        gain = sums - s["ref_logp"].double()
        m = BETA * (gain[:pairs] - gain[pairs:])
        up, down = 1.0 / (1.0 + (-m).exp()), 1.0 / (1.0 + m.exp())
        loss = (-(1.0 - SMOOTHING) * up.log() - SMOOTHING * down.log()).mean()
        c = BETA / pairs * (SMOOTHING * up - (1.0 - SMOOTHING) * down)
        dlogp = torch.where(has, torch.cat([c, -c]).float()[seq], 0.0)
        return {"loss": loss.float().reshape(1), "rewards": (BETA * gain).float(),
                "dlogits": _logit_grad(e, total, at, dlogp, s["logits"].dtype)}
    z, ids, valid = s["logits"].float(), s["experts"], s["valid"]
    n_e, k = z.shape[1], ids.shape[1]
    top = z.max(1, keepdim=True).values
    e = (z - top).exp()
    total = e.sum(1, keepdim=True)
    p = torch.where(valid[:, None], e / total, 0.0)
    lse = torch.where(valid, (top + total.log())[:, 0], 0.0)
    counts = torch.zeros(n_e, dtype=torch.int32, device=z.device)
    counts.index_add_(0, ids.reshape(-1).long(), valid.int()[:, None].expand(-1, k).reshape(-1))
    t = valid.sum().clamp(min=1).float()
    f = counts.float() / (t * k)
    balance = n_e * (f.double() * p.double().sum(0)).sum() / t
    zloss = lse.double().square().sum() / t
    mean_f = (p * f).sum(1, keepdim=True)
    d = p * (BALANCE * n_e / t * (f - mean_f) + 2.0 * ZCOEF / t * lse[:, None])
    stats = torch.stack([BALANCE * balance + ZCOEF * zloss, balance, zloss]).float()
    return {"counts": counts, "stats": stats, "dlogits": d.to(s["logits"].dtype)}


# ------------------------------------------------------------ definition


def exact(case, seed):
    """The outputs of run() from the operators' definitions, in 64 bits."""
    s = prepare(case, seed)
    op = case["op"]
    if op == "embed":
        out = torch.zeros(s["out"].shape, dtype=torch.float64, device=DEV)
        live = (s["ids"] >= 0).nonzero()[:, 0]
        out[live] = s["table"].double()[s["ids"][live].long()] * s["scale"]
        return {"out": out}
    if op == "embed_grad":
        live = (s["ids"] >= 0).nonzero()[:, 0]
        acc = torch.zeros(s["acc"].shape, dtype=torch.float64, device=DEV)
        acc.index_add_(0, s["ids"][live].long(), s["dout"][live].double())
        acc *= s["scale"]
        return {"acc": acc if case["first"] else acc + s["acc"].double()}
    x, n = s["logits"], s["logits"].shape[0]
    if op == "balance":
        x, keep = x.double()[s["valid"]], s["valid"]
        lse = torch.logsumexp(x, 1)
        p = (x - lse[:, None]).exp()
        t, k = max(1, x.shape[0]), case["k"]
        counts = torch.bincount(s["experts"][keep].reshape(-1).long(), minlength=case["experts"])
        f = counts.double() / (t * k)
        bal, zl = case["experts"] * (f * p.sum(0) / t).sum(), (lse * lse).sum() / t
        d = torch.zeros(s["logits"].shape, dtype=torch.float64, device=DEV)
        # the gradient of sum_e f_e P_e through the softmax's Jacobian, diag(p) - p p'
        d[keep] = BALANCE * case["experts"] / t * (p * f - p * (p @ f)[:, None]) + ZCOEF / t * 2.0 * lse[:, None] * p
        return {"counts": counts.int(), "stats": torch.stack([BALANCE * bal + ZCOEF * zl, bal, zl]), "dlogits": d}
    live = s["targets"] >= 0
    if op == "policy":
        live = live & (s["weights"] != 0.0)
    lse = torch.zeros(n, dtype=torch.float64, device=DEV)
    logp = torch.zeros(n, dtype=torch.float64, device=DEV)
    for a in range(0, n, 512):
        z = x[a:a + 512].double()
        q = torch.log_softmax(z, 1)
        at = s["targets"][a:a + 512].long().clamp(min=0)[:, None]
        lse[a:a + 512] = torch.logsumexp(z, 1)
        logp[a:a + 512] = q.gather(1, at)[:, 0]
    zero = torch.zeros(n, dtype=torch.float64, device=DEV)
    if op == "logprob":
        return {"logp": torch.where(live, logp, zero), "lse": torch.where(live, lse, zero)}
    if op == "policy":
        w, adv = s["weights"].double() * live, s["advantages"].double()
        r = (logp - s["old_logp"].double()).exp()
        lo, hi = 1.0 - CLIP_LOW, 1.0 + CLIP_HIGH
        # the clipped branch holds where the ratio has left the interval on the side that the advantage favours
        flat = ((adv > 0) & (r > hi)) | ((adv < 0) & (r < lo))
        pg = -adv * torch.where(flat, r.clamp(lo, hi), r)
        d = s["ref_logp"].double() - logp
        kl = d.exp() - 1.0 - d
        dlogp = w * (torch.where(flat, zero, -adv * r) + KL_COEF * (1.0 - d.exp()))
        first = {"stats": torch.stack([(w * (pg + KL_COEF * kl)).sum(), (w * pg).sum(), (w * kl).sum(), (w * flat).sum()]),
                 "logp": torch.where(live, logp, zero)}
    else:
        off, pairs = s["offsets"].tolist(), case["pairs"]
        total = torch.stack([torch.where(live, logp, zero)[a:b].sum() for a, b in zip(off, off[1:])])
        gain = total - s["ref_logp"].double()
        m = BETA * (gain[:pairs] - gain[pairs:])
        soft = torch.nn.functional.softplus
        loss = ((1.0 - SMOOTHING) * soft(-m) + SMOOTHING * soft(m)).mean()
        c = BETA * (torch.sigmoid(m) - (1.0 - SMOOTHING)) / pairs
        each = torch.cat([c, -c])
        dlogp = torch.cat([each[i].expand(b - a) for i, (a, b) in enumerate(zip(off, off[1:]))]) * live
        first = {"loss": loss.reshape(1), "rewards": BETA * gain}
    d = torch.empty(x.shape, dtype=torch.float64, device=DEV)
    for a in range(0, n, 512):
        q = -(x[a:a + 512].double() - lse[a:a + 512, None]).exp()
        at = s["targets"][a:a + 512].long().clamp(min=0)[:, None]
        q.scatter_add_(1, at, torch.ones_like(at, dtype=torch.float64))
        d[a:a + 512] = q * dlogp[a:a + 512, None]
    return {**first, "dlogits": d}
