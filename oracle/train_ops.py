"""Plain fp64 definitions of the operators around the Muon step (embedding
lookup and gradient, token log-probability, policy, preference and balance
losses with their gradients).  Test infrastructure only, like the rest of the
oracle: it shares no code with the library and imports nothing from it.

Arrays are numpy, logits fp64; a target or id outside its range is none.
"""

from __future__ import annotations

import numpy as np


def embed_forward(table, ids, scale):
    table = np.asarray(table, dtype=np.float64)
    out = np.zeros((len(ids), table.shape[1]))
    for t, i in enumerate(ids):
        if 0 <= i < table.shape[0]:
            out[t] = table[i] * scale
    return out


def embed_backward(ids, dout, vocab, scale, acc=None):
    dout = np.asarray(dout, dtype=np.float64)
    g = np.zeros((vocab, dout.shape[1])) if acc is None else np.array(acc, dtype=np.float64)
    for t, i in enumerate(ids):
        if 0 <= i < vocab:
            g[i] += scale * dout[t]
    return g


def log_softmax(x):
    """(log p, lse) of each row; a row of -inf gives lse -inf and NaN."""
    x = np.asarray(x, dtype=np.float64)
    with np.errstate(all="ignore"):
        top = x.max(axis=1, keepdims=True)
        shift = np.where(np.isfinite(top), top, 0.0)
        lse = shift + np.log(np.exp(x - shift).sum(axis=1, keepdims=True))
        return x - lse, lse[:, 0]


def token_logprob(x, targets):
    v = np.asarray(x).shape[1]
    lp, lse = log_softmax(x)
    has = (targets >= 0) & (targets < v)
    at = np.where(has, targets, 0).astype(np.int64)
    return np.where(has, lp[np.arange(len(at)), at], 0.0), np.where(has, lse, 0.0)


def times(c, v):
    """c v, where a factor of 0 leaves nothing of an infinite value."""
    with np.errstate(invalid="ignore"):
        return np.where((np.asarray(c) == 0.0) & np.isinf(v), 0.0, np.multiply(c, v))


def logit_grad(x, targets, dlogp):
    """sum_r dlogp[r] logp[r] by the logits; rows whose dlogp is 0 get 0."""
    x = np.asarray(x, dtype=np.float64)
    lp, _ = log_softmax(x)
    with np.errstate(all="ignore"):
        d = -np.exp(lp)
    for r, t in enumerate(targets):
        if 0 <= t < x.shape[1]:
            d[r, t] += 1.0
    with np.errstate(all="ignore"):
        return np.where(dlogp[:, None] == 0.0, 0.0, d * dlogp[:, None])


def policy_loss(x, targets, advantages, weights, old_logp=None, ref_logp=None, clip_low=0.2, clip_high=0.2,
                kl_coef=0.0):
    """(stats, logp, dlogits, dlogp)."""
    x = np.asarray(x, dtype=np.float64)
    n, v = x.shape
    logp, _ = token_logprob(x, targets)
    stats, dlogp, out = np.zeros(4), np.zeros(n), np.zeros(n)
    for r in range(n):
        w, a = float(weights[r]), float(advantages[r])
        if not 0 <= targets[r] < v or w == 0.0:
            continue
        out[r] = logp[r]
        ratio = (logp[r] if np.isnan(logp[r]) else 1.0) if old_logp is None else np.exp(logp[r] - float(old_logp[r]))
        clipped = min(max(ratio, 1.0 - clip_low), 1.0 + clip_high)
        plain = float(times(a, ratio))
        flat = plain > clipped * a
        pg = -(clipped * a if flat else plain)
        kl = dkl = 0.0
        if ref_logp is not None:
            d = float(ref_logp[r]) - logp[r]
            kl, dkl = np.expm1(d) - (d if d < np.inf else 0.0), -np.expm1(d)
        stats += np.array([w * (pg + times(kl_coef, kl)), w * pg, w * kl, w if flat else 0.0])
        dlogp[r] = w * ((0.0 if flat else -plain) + times(kl_coef, dkl))
    return stats, out, logit_grad(x, targets, dlogp), dlogp


def preference_loss(x, targets, offsets, ref_logp, beta=0.1, label_smoothing=0.0):
    """(loss, rewards, dlogits, dlogp)."""
    x = np.asarray(x, dtype=np.float64)
    n, v = x.shape
    logp, _ = token_logprob(x, targets)
    seqs = len(ref_logp)
    pairs = seqs // 2
    gain = np.array([logp[offsets[s]:offsets[s + 1]].sum() - float(ref_logp[s]) for s in range(seqs)])
    rewards = times(beta, gain)
    m = rewards[:pairs] - rewards[pairs:] if beta == 0.0 else beta * (gain[:pairs] - gain[pairs:])
    loss = (times(1.0 - label_smoothing, np.logaddexp(0.0, -m)) + times(label_smoothing, np.logaddexp(0.0, m))).mean()
    up, down = np.exp(-np.logaddexp(0.0, -m)), np.exp(-np.logaddexp(0.0, m))  # neither as 1 minus the other
    c = beta / pairs * (label_smoothing * up - (1.0 - label_smoothing) * down)
    dlogp = np.zeros(n)
    for s in range(seqs):
        dlogp[offsets[s]:offsets[s + 1]] = c[s] if s < pairs else -c[s - pairs]
    dlogp = np.where((targets >= 0) & (targets < v), dlogp, 0.0)
    return loss, rewards, logit_grad(x, targets, dlogp), dlogp


def balance_loss(x, choices, valid=None, coef=0.01, z_coef=0.0):
    """(counts, stats, dlogits)."""
    x = np.asarray(x, dtype=np.float64)
    n, e = x.shape
    k = choices.shape[1]
    valid = np.ones(n, dtype=bool) if valid is None else np.asarray(valid, dtype=bool)
    counts = np.zeros(e, dtype=np.int64)
    for c in choices[valid].reshape(-1):
        if 0 <= c < e:
            counts[c] += 1
    t = max(1, int(valid.sum()))
    f = counts / (t * k)
    lp, lse = log_softmax(x) if n else (x, np.zeros(0))
    p = np.where(valid[:, None], np.exp(lp), 0.0)
    lse = np.where(valid, lse, 0.0)
    bal = e * float((f * p.sum(axis=0)).sum()) / t
    z = float((lse * lse).sum()) / t
    d = p * (coef * e / t * (f - (p @ f)[:, None]) + 2.0 * z_coef / t * lse[:, None])
    return counts, np.array([coef * bal + z_coef * z, bal, z]), d
