"""Plain fp64 definitions of the operators of a trained layer (dropout, routing to experts, the order of the tokens
by expert, the experts' weighted sum, the product with bias, activation and residual, and their gradients).  Test
infrastructure only, like the rest of the oracle: it shares no code with the library and imports nothing from it.
"""

from __future__ import annotations

import math

import numpy as np

NORM_EPS = 1e-20


# ---------------------------------------------------------------- dropout


def philox(counter, key):
    """One block of Philox4x32-10: four words from four counter words and two key words (Python integers)."""
    c, k = list(counter), list(key)
    for _ in range(10):
        p, q = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57
        c = [(q >> 32) ^ c[1] ^ k[0], q & 0xFFFFFFFF, (p >> 32) ^ c[3] ^ k[1], p & 0xFFFFFFFF]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return c


def dropout_keep(rows, cols, p, seed, site, step, row0=0, col0=0):
    """Which elements of rows [row0, row0 + rows), columns [col0, col0 + cols) stay."""
    limit = round(p * 2 ** 32)
    keep = np.zeros((rows, cols), dtype=bool)
    for r in range(rows):
        for c in range(col0 - col0 % 4, col0 + cols, 4):
            word = philox((c // 4, row0 + r, site, step & 0xFFFFFFFF), (seed & 0xFFFFFFFF, seed >> 32))
            for j in range(4):
                if col0 <= c + j < col0 + cols:
                    keep[r, c + j - col0] = word[j] >= limit
    return keep


def dropout(x, keep, p, residual=None):
    out = np.where(keep, np.asarray(x, dtype=np.float64) / (1.0 - p), 0.0)
    return out if residual is None else out + np.asarray(residual, dtype=np.float64)


# ---------------------------------------------------------------- routing


def scores(x, scoring):
    x = np.asarray(x, dtype=np.float64)
    with np.errstate(all="ignore"):
        if scoring == "sigmoid":
            return 1.0 / (1.0 + np.exp(-x))
        top = x.max(axis=1, keepdims=True)
        e = np.exp(x - np.where(np.isneginf(top), 0.0, top))
        total = e.sum(axis=1, keepdims=True)
        return np.where(total == 0.0, 0.0, e / np.where(total == 0.0, 1.0, total))


def _better(a, b):
    """Whether rank a beats rank b; NaN is below every number."""
    if math.isnan(a):
        return False
    return math.isnan(b) or a > b


def route(x, k, scoring="softmax", bias=None, valid=None, groups=1, keep_groups=1, group_top=1, renormalize=True,
          scale=1.0):
    """(choices, weights)."""
    x = np.asarray(x, dtype=np.float64)
    t, n = x.shape
    s = scores(x, scoring)
    choices, weights = np.full((t, k), -1, dtype=np.int64), np.zeros((t, k))
    for r in range(t):
        if valid is not None and not valid[r]:
            continue
        plain = bias is None and (groups == 1 or group_top == 1)
        rank = x[r] if plain else s[r] + (0.0 if bias is None else np.asarray(bias, dtype=np.float64))
        live = [e for e in range(n) if x[r, e] != -np.inf and (bias is None or bias[e] != -np.inf)]

        def pick(among, count):
            left, out = list(among), []
            while left and len(out) < count:
                best = left[0]
                for e in left[1:]:
                    if _better(rank[e], rank[best]):
                        best = e
                out.append(best)
                left.remove(best)
            return out
        if groups > 1:
            size = n // groups
            value = {}
            for g in range(groups):
                two = pick([e for e in live if e // size == g], group_top)
                if two:
                    v = [rank[e] for e in two]
                    value[g] = sum(-1e39 if math.isnan(q) else q for q in v)
            order = sorted(value, key=lambda g: (-value[g], g))[:keep_groups]
            live = [e for e in live if e // size in order]
        got = pick(live, k)
        choices[r, :len(got)] = got
        w = s[r, got]
        weights[r, :len(got)] = scale * (w / (w.sum() + NORM_EPS) if renormalize else w)
    return choices, weights


def route_backward(x, choices, dweights, scoring="softmax", valid=None, renormalize=True, scale=1.0):
    """The gradient by the logits, through the Jacobians written out."""
    x = np.asarray(x, dtype=np.float64)
    t, n = x.shape
    s = scores(x, scoring)
    d = np.zeros((t, n))
    for r in range(t):
        if valid is not None and not valid[r]:
            continue
        got = [(j, e) for j, e in enumerate(choices[r]) if 0 <= e < n]
        if not got:
            continue
        idx = [e for _, e in got]
        dw = np.array([float(dweights[r, j]) for j, _ in got])
        w = s[r, idx]
        total = w.sum() + NORM_EPS
        ds = scale * ((dw - (dw * w).sum() / total) / total if renormalize else dw)
        for e, g, v in zip(idx, ds, w):
            if scoring == "sigmoid":
                d[r, e] += g * v * (1.0 - v)
            else:
                d[r, e] += g * v
                d[r] -= g * v * s[r]
    return d


# ------------------------------------------------- order and weighted sum


def expert_order(choices, experts):
    """(tokens, offsets, place)."""
    t, k = choices.shape
    tokens, place = np.full(t * k, -1, dtype=np.int64), np.full((t, k), -1, dtype=np.int64)
    offsets, at = [0], 0
    for e in range(experts):
        for r, j in np.argwhere(choices == e):
            tokens[at], place[r, j] = r, at
            at += 1
        offsets.append(at)
    return tokens, np.array(offsets), place


def expert_combine(y, place, weights=None, residual=None):
    y = np.asarray(y, dtype=np.float64)
    t, k = place.shape
    out = np.zeros((t, y.shape[1])) if residual is None else np.array(residual, dtype=np.float64)
    for r in range(t):
        for j in range(k):
            if 0 <= place[r, j] < y.shape[0]:
                out[r] += (1.0 if weights is None else float(weights[r, j])) * y[place[r, j]]
    return out


def expert_combine_backward(dout, y, place, dy, weights=None):
    """(dy, dweights); dy: what the rows of no place keep."""
    y, dout, dy = (np.array(a, dtype=np.float64) for a in (y, dout, dy))
    dw = np.zeros(place.shape)
    for r in range(place.shape[0]):
        for j in range(place.shape[1]):
            p = place[r, j]
            if 0 <= p < y.shape[0]:
                dw[r, j] = (dout[r] * y[p]).sum()
                dy[p] = (1.0 if weights is None else float(weights[r, j])) * dout[r]
    return dy, dw


# ---------------------------------------------------------------- product


def activation(name, v):
    """(value, slope)."""
    v = np.asarray(v, dtype=np.float64)
    if name == "relu":
        return np.where(v > 0.0, v, np.where(np.isnan(v), v, 0.0)), (v > 0.0).astype(np.float64)
    if name == "silu":
        with np.errstate(over="ignore"):
            q = 1.0 / (1.0 + np.exp(-v))
        return v * q, q * (1.0 + v * (1.0 - q))
    if name == "gelu":
        half = 0.5 * np.vectorize(math.erfc, otypes=[np.float64])(-v * math.sqrt(0.5))
        return v * half, half + v * np.exp(-0.5 * v * v) / math.sqrt(2.0 * math.pi)
    if name == "gelu_tanh":
        c = math.sqrt(2.0 / math.pi)
        with np.errstate(over="ignore"):
            q = 1.0 / (1.0 + np.exp(-2.0 * c * (v + 0.044715 * v ** 3)))  # (1 + tanh) / 2
        return v * q, q + v * q * (1.0 - q) * 2.0 * c * (1.0 + 0.134145 * v * v)
    assert name == "none"
    return v, np.ones_like(v)


def linear_forward(x, w, bias=None, act="none", residual=None, offsets=None, out=None, pre=None):
    """(out, pre) of one matrix (w: in x out), or of a matrix a group of rows (w: groups x in x out); rows of no group
    keep what out and pre hold."""
    x = np.asarray(x, dtype=np.float64)
    w = np.asarray(w, dtype=np.float64)
    if offsets is None:
        w, offsets = w[None], [0, x.shape[0]]
    shape = (x.shape[0], w.shape[2])
    out = np.zeros(shape) if out is None else np.array(out, dtype=np.float64)
    pre = np.zeros(shape) if pre is None else np.array(pre, dtype=np.float64)
    for g in range(w.shape[0]):
        r = slice(offsets[g], offsets[g + 1])
        v = x[r] @ w[g]
        if bias is not None:
            v = v + np.asarray(bias, dtype=np.float64).reshape(w.shape[0], -1)[g]
        pre[r] = v
        v = activation(act, v)[0]
        out[r] = v if residual is None else v + np.asarray(residual, dtype=np.float64)[r]
    return out, pre


def linear_input_grad(dy, w, act="none", pre=None, residual=None, offsets=None, dx=None):
    w = np.asarray(w, dtype=np.float64)
    v, _ = linear_forward(dy, np.swapaxes(w, -1, -2), offsets=offsets)
    if act != "none":
        v = v * activation(act, pre)[1]
    if residual is not None:
        v = v + np.asarray(residual, dtype=np.float64)
    if offsets is None:
        return v
    out = np.zeros(v.shape) if dx is None else np.array(dx, dtype=np.float64)
    out[offsets[0]:offsets[-1]] = v[offsets[0]:offsets[-1]]
    return out


def linear_weight_grad(x, dy, offsets=None):
    """(dw, dbias), with a leading axis of groups if there are offsets."""
    x, dy = np.asarray(x, dtype=np.float64), np.asarray(dy, dtype=np.float64)
    if offsets is None:
        return x.T @ dy, dy.sum(axis=0)
    parts = [slice(a, b) for a, b in zip(offsets, offsets[1:])]
    return np.stack([x[p].T @ dy[p] for p in parts]), np.stack([dy[p].sum(axis=0) for p in parts])
