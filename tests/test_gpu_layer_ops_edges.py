"""The operators of a trained layer where digits, experts or limits are easily lost: routers that are sure of an
expert, NaN beside masks, more tokens than a grid has lanes for, long sums of columns, activations far out.

e = 2^-24 (half a step of fp32), h = half a step of the output's type.  Tolerances stand at each test.
"""

from __future__ import annotations

import numpy as np
import pytest

import muon_newton_schulz_step_amd as M
import oracle.layer_ops as L
from test_gpu_train_ops import DEV, E, HALF, TINY, dt, f64, poisoned, torch, vec, within  # noqa: F401

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------- routing


def sure_logits(rng, t, n):
    """Rows whose scores reach from almost 0 to almost 1."""
    x = rng.standard_normal((t, n)).astype(np.float32)
    far = np.linspace(0.0, 40.0, t).astype(np.float32)
    x[:, n // 3] += far
    x[::3, n // 2] += far[::3]
    x[1::4] -= far[1::4, None]
    return x


def gradient(x, choices, dw, scoring, renormalize, scale):
    """(the gradient, the size of what it is a sum of) in fp64, with the differences taken before the sums: of dw_e and
    dw_j instead of dw_e and the mean, of the scores left over instead of 1 and the chosen ones."""
    t, n = x.shape
    x = x.astype(np.float64)
    d, size = np.zeros((t, n)), np.zeros((t, n))
    for r in range(t):
        idx = choices[r]
        g = dw[r].astype(np.float64)
        if scoring == "sigmoid":
            s, comp = 1.0 / (1.0 + np.exp(-x[r, idx])), 1.0 / (1.0 + np.exp(x[r, idx]))
        else:
            e = np.exp(x[r] - x[r].max())
            p = e / e.sum()
            s, left = p[idx], np.delete(e, idx).sum() / e.sum()
        total = s.sum() + L.NORM_EPS
        if renormalize:
            pair = g[:, None] - g[None, :]                       # dw_j - dw_i
            ds = scale / total ** 2 * (pair @ s + L.NORM_EPS * g)
            dsize = scale / total ** 2 * (np.abs(pair) @ s + L.NORM_EPS * np.abs(g))
            diff = scale / total * pair                          # ds_j - ds_i
        else:
            ds, dsize, diff = scale * g, scale * np.abs(g), scale * (g[:, None] - g[None, :])
        if scoring == "sigmoid":
            d[r, idx], size[r, idx] = s * comp * ds, s * comp * dsize
            continue
        inner = (s * ds).sum()
        if renormalize:
            inner = (scale * g * s).sum() * L.NORM_EPS / total ** 2
            d[r] = -p * inner
            d[r, idx] = s * (ds - inner)
            size[r] = p * abs(inner)
            size[r, idx] += s * dsize
        else:
            d[r] = -p * inner
            size[r] = p * (s * np.abs(ds)).sum()
            d[r, idx] = s * (left * ds + diff @ s)
            size[r, idx] = s * (left * np.abs(ds) + np.abs(diff) @ s)
    return d, size


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("n,k", [(8, 1), (8, 2), (40, 6), (256, 8), (700, 20), (30, 30), (200, 32)])
def test_gradient_of_a_sure_router(torch, n, k, scoring, renorm):
    # A score near 1 leaves 1 - s, and a mean of dw that is all but one dw, with few digits: what is left over has to
    # be had from what it is made of.
    # Tolerance: scores carry (|d| + 60) e of themselves (sigmoid: (|x| + 8) e, its complement as much), of which an
    # element has four, and 12 e of operations; 2^-50 of dw s / total for sums in 64 bits.
    rng = np.random.default_rng(n + k)
    t, scale = 41, 2.5
    x = sure_logits(rng, t, n)
    choices = np.stack([rng.permutation(n)[:k] for _ in range(t)])
    choices[:, 0] = n // 3
    for r in range(t):
        others = [e for e in choices[r, 1:] if e != n // 3]
        more = [e for e in range(n) if e != n // 3 and e not in others]
        choices[r, 1:] = (others + more)[:k - 1]
    dw = rng.standard_normal((t, k)).astype(np.float32)
    want, size = gradient(x, choices, dw, scoring, renorm, scale)
    out = torch.full((t, n), 9.0, device=DEV)
    M.route_backward(vec(torch, x), vec(torch, choices, "int32"), vec(torch, dw), out, True, scoring=scoring,
                     renormalize=renorm, scale=scale)
    x = x.astype(np.float64)
    rel = (np.abs(x).max(axis=1) + 8) if scoring == "sigmoid" else (x.max(axis=1) - x.min(axis=1) + 60)
    s = L.scores(x, scoring)
    total = (np.take_along_axis(s, choices, 1).sum(axis=1, keepdims=True) if renorm else 1.0)
    sums = 2.0 ** -50 * scale * np.abs(dw).max(axis=1, keepdims=True) * s / total
    within(f64(out), want, size * (4 * rel[:, None] + 12) * E + np.abs(want) * E + sums + TINY, "gradient by the logits")


def test_gradient_of_repeated_choices(torch):
    # the same expert several times, chosen first and last, beside others
    rng = np.random.default_rng(5)
    for scoring in ("softmax", "sigmoid"):
        for n, k in ((8, 8), (64, 12), (300, 32)):
            x = rng.standard_normal((50, n)).astype(np.float32)
            choices = rng.integers(-1, min(n, k // 2) + 1, (50, k))  # some outside where n is small
            dw = rng.standard_normal((50, k)).astype(np.float32)
            out = torch.empty(50, n, device=DEV)
            for renorm in (True, False):
                M.route_backward(vec(torch, x), vec(torch, choices, "int64"), vec(torch, dw), out, True, scoring=scoring,
                                 renormalize=renorm)
                want = L.route_backward(x, choices, dw, scoring, renormalize=renorm)
                # k products of scores below 1, each within (8 + 60 + 12) 4 e, weights' sums at least 1 / n of a score
                within(f64(out), want, np.abs(dw).sum(axis=1, keepdims=True) * 400 * E * (n if renorm else 1), scoring)


@pytest.mark.parametrize("n,k", [(6, 6), (8, 2), (32, 8), (64, 6), (256, 8), (300, 32), (1000, 8)])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_route_of_nan_beside_masks(torch, n, k, scoring, dtype):
    # A NaN ranks below every number, the lowest one too; an expert masked by its bias stays out whatever its logit is.
    rng = np.random.default_rng(n)
    x = rng.standard_normal((12, n))
    low = -3.4028235e38 if dtype == "fp32" else -3.3895314e38
    x[0, :-1] = low                          # a mask of the type's lowest value
    x[0, 0] = np.nan
    x[1, 1::2] = low
    x[1, ::3] = np.nan
    x[2] = np.nan
    x[3, 0] = np.nan
    x[4, n // 2:] = np.nan
    x[5, 1:] = -np.inf
    x[5, 0] = np.nan
    x[6, :] = low
    x[6, n - 1] = np.nan
    x[7, 0] = np.inf
    x = x.astype(np.float32)
    xd = torch.from_numpy(x).to(DEV).to(dt(torch, dtype))
    x = f64(xd)
    lowest, masked = np.zeros(n, dtype=np.float32), np.zeros(n, dtype=np.float32)
    lowest[::2] = -3.4028235e38
    masked[0], masked[n // 2] = -np.inf, -np.inf
    for bias in (None, masked, lowest):
        for groups in (1, 2):
            choices, weights = torch.full((12, k), 99, dtype=torch.int32, device=DEV), torch.empty(12, k, device=DEV)
            how = dict(scoring=scoring, groups=groups, keep_groups=1, group_top=2)
            if groups > 1 and k > n // 2:
                continue
            M.route_experts(xd, choices, weights, bias=None if bias is None else vec(torch, bias), **how)
            with np.errstate(invalid="ignore"):
                want, w = L.route(x, k, bias=bias, **how)
            assert np.array_equal(choices.cpu().numpy(), want), (bias is None, groups)
            # a row's weights are NaN where a score among them is
            assert np.array_equal(np.isnan(f64(weights)), np.isnan(w)), (bias is None, groups)


@pytest.mark.parametrize("tokens,n", [((1 << 30) + 70, 2), ((1 << 28) + 40, 33)])
def test_route_of_more_tokens_than_a_grid_has_lanes_for(torch, tokens, n):
    # 4 and 16 lanes a token: more than 2^32 in all.  Against calls on the tokens of both sides of the seams.
    torch.cuda.empty_cache()
    x = torch.empty(tokens, n, dtype=torch.bfloat16, device=DEV).normal_(generator=torch.Generator(DEV).manual_seed(1))
    valid = torch.ones(tokens, dtype=torch.bool, device=DEV)
    valid[5::1000] = False
    c, w = torch.full((tokens, 1), 99, dtype=torch.int32, device=DEV), torch.full((tokens, 1), 9.0, device=DEV)
    M.route_experts(x, c, w, valid=valid, renormalize=False)
    assert int(c.min()) == -1 and int(c.max()) == n - 1 and float(w.max()) <= 1.0
    d = torch.full_like(x, 9.0)
    M.route_backward(x, c, w, d, True, valid=valid, renormalize=False)
    assert float(d.max()) < 1.0
    lanes = 4 if n == 2 else 16
    seam = (1 << 32) // lanes
    for at in (0, seam // 2, seam - 4096, tokens - 4096):
        part = slice(at, min(tokens, at + 8192))
        c2, w2, d2 = torch.empty_like(c[part]), torch.empty_like(w[part]), torch.empty_like(d[part])
        M.route_experts(x[part], c2, w2, valid=valid[part], renormalize=False)
        M.route_backward(x[part], c2, w2, d2, True, valid=valid[part], renormalize=False)
        assert torch.equal(c[part], c2) and torch.equal(w[part], w2) and torch.equal(d[part], d2), at
    del x, c, w, d, valid
    torch.cuda.empty_cache()


def test_route_of_a_row_of_any_stride(torch):
    x = torch.randn(40, device=DEV)
    far = torch.as_strided(x, (1, 40), (1 << 54, 1))
    c, w, d = torch.empty(1, 3, dtype=torch.int32, device=DEV), torch.empty(1, 3, device=DEV), torch.empty(1, 40, device=DEV)
    M.route_experts(far, c, w)
    M.route_backward(far, c, w, d, True)
    c2, w2, d2 = torch.empty_like(c), torch.empty_like(w), torch.empty_like(d)
    M.route_experts(x[None], c2, w2)
    M.route_backward(x[None], c2, w2, d2, True)
    assert torch.equal(c, c2) and torch.equal(w, w2) and torch.equal(d, d2)


# ---------------------------------------------------------------- product


@pytest.mark.parametrize("rows,cols,groups,dtype", [(1 << 17, 128, 1024, "fp32"), (1 << 17, 128, 1024, "bf16"), (40000, 4096, 32, "bf16"),
                                                    (100003, 130, 1, "fp32"), (5000, 1000, 3, "fp32")])
def test_bias_gradient_of_long_groups(torch, rows, cols, groups, dtype):
    # One value throughout: every addition in 32 bits would round the same way.  Sums in 64 bits leave each part's
    # rounding, that of the parts' sum, and of what was held: 4 e of the sum of magnitudes.
    value = 0.1
    dy = torch.full((rows, cols), value, dtype=dt(torch, dtype), device=DEV)
    x = torch.ones(rows, 4, dtype=dy.dtype, device=DEV)
    value = float(dy[0, 0].double())
    offsets = torch.zeros(groups + 1, dtype=torch.int32, device=DEV)
    offsets[groups // 2 + 1:] = rows                   # one group has every row
    for first in (True, False):
        dw, db = torch.full((groups, 4, cols), 3.0, device=DEV), torch.full((groups, cols), 3.0, device=DEV)
        M.linear_weight_grad(x, dy, dw, first, poisoned(torch, M.linear_weight_grad_workspace_bytes(rows, 4, cols, groups)),
                             dbias=db, offsets=offsets)
        want = np.full((groups, cols), 0.0 if first else 3.0)
        want[groups // 2] += rows * value
        within(f64(db), want, 4 * E * np.abs(want), "dbias")


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_activations_far_out(torch, act, dtype):
    # Relative to the value itself, down to where results leave the normal numbers.
    #   silu       exp in two parts 4 e, 1 + exp, the quotient, the product: 10 e (bf16: a quotient of 2^-22: 16 e)
    #   gelu_tanh  its exponent u = 1.6 v + 0.07 v^3 is rounded: 4 |u| e more
    #   gelu       fp32: erfc's argument is rounded: (v^2 + 1) 2 e more, erfc itself 16 e;
    #              bf16: the polynomial's 8e-5, the exponent v^2 / 2 in fp32: 4 v^2 e more
    v = np.concatenate([np.linspace(-13.0, 13.0, 5001), np.linspace(-85.0, 85.0, 3001)])
    if act != "silu":
        v = v[np.abs(v) < (13.0 if act == "gelu" else 9.5)]
    x = torch.from_numpy(v).to(dt(torch, dtype)).to(DEV)[:, None].contiguous()
    out = torch.empty_like(x)
    M.linear_forward(x, torch.ones(1, 1, dtype=x.dtype, device=DEV), out, poisoned(torch, M.linear_workspace_bytes(len(v), 1, 1, 1)),
                     activation=act)
    v = f64(x)
    want, _ = L.activation(act, v)
    rel = {"silu": 16.0 + 0 * v, "gelu_tanh": 16.0 + 4 * np.abs(1.6 * v + 0.0714 * v ** 3),
           "gelu": 24.0 + 4 * v * v + (8e-5 / E if dtype == "bf16" else 0.0)}[act] * E
    within(f64(out), want, np.abs(want) * (rel + HALF[dtype]), act)


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
def test_slopes_of_large_numbers(torch, act):
    # The slope's second part is v (1 - q) q with q near 1: 1 - q from exp(-v) instead of q.
    #   silu      a product and three sums near 1: 8 e of the sum of the parts' magnitudes (at most 1.3)
    #   gelu_tanh the same, with its exponent u rounded: 4 |u| e of the second part
    v = np.linspace(0.5, 30.0, 3001)
    x = torch.from_numpy(v).float().to(DEV)[:, None].contiguous()
    d = torch.empty_like(x)
    M.activation_grad(torch.ones_like(x), x, d, act)
    v = f64(x)
    if act == "silu":
        e = np.exp(-v)
        q, second, u = 1 / (1 + e), v * e / (1 + e) ** 2, 0.0
    else:
        c = np.sqrt(2 / np.pi)
        u = 2 * c * (v + 0.044715 * v ** 3)
        e = np.exp(-u)
        q, second = 1 / (1 + e), v * 2 * c * (1 + 0.134145 * v * v) * e / (1 + e) ** 2
    within(f64(d), q + second, (q + second) * 8 * E + second * (4 * u + 16) * E, act + "'")
