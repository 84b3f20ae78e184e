"""Dropout, routing, order and weighted sum on the GPU, against their fp64 definitions (oracle/layer_ops.py) on the
same bits.

Tolerances, from the arithmetic (e = 2^-24, half a step of fp32; h = half a step of the output's type):
  dropout      the scale's rounding, one product, one sum, one rounding: (4 e + h) (|x| scale + |residual|)
  scores       sigmoid of x: (|x| + 8) e of itself; softmax: (|d| + 60) e with d the distance to the row's maximum,
               the sum's error among it (at most 22 additions a path, sum p |d| <= 7)
  weights      the scores' error twice (own and in the sum), k additions, two operations: |w| (2 t + (k + 4) e)
  gradient     of each of the at most k + 1 products that meet in an element, 4 t + (k + 10) e of the sum of their
               magnitudes, and h of the result
  sums         out: (k + 2) e of the sum of magnitudes + h; dweights: (dim / 64 + 10) e of the sum of magnitudes
Whole numbers are equal.
"""

from __future__ import annotations

import numpy as np
import pytest

import muon_newton_schulz_step_amd as M
import oracle.layer_ops as L
from test_gpu_train_ops import DEV, E, HALF, TINY, around_untouched, dt, f64, poisoned, strided, torch, vec, within  # noqa: F401

pytestmark = pytest.mark.gpu
SEED = 0xFEDCBA9876543210


# ---------------------------------------------------------------- dropout


@pytest.mark.parametrize("rows,cols,p", [(1, 1, 0.5), (1, 4, 0.1), (3, 7, 0.9), (2, 1023, 0.3), (33, 130, 0.25), (300, 3, 0.5),
                                         (1, 5000, 0.1), (70, 64, 0.0), (2, 9, 1.0 - 2.0 ** -30), (0, 5, 0.1), (9, 8, 2.0 ** -32)])
@pytest.mark.parametrize("dtype,res,ld,shift", [("bf16", True, 0, 0), ("fp32", False, 3, 1), ("bf16", False, 5, 3), ("fp32", True, 0, 0)])
def test_dropout(torch, rows, cols, p, dtype, res, ld, shift):
    rng = np.random.default_rng(rows * 7 + cols)
    x, _ = strided(torch, rng.standard_normal((rows, cols)), dtype, cols + ld, shift)
    r, _ = strided(torch, rng.standard_normal((rows, cols)), dtype, cols + 2 * ld, 2 * shift)
    out, buf = strided(torch, np.zeros((rows, cols)), dtype, cols + ld, shift)
    M.dropout(x, out, p, SEED, site=3, step=41, residual=r if res else None)
    keep = L.dropout_keep(rows, cols, p, SEED, 3, 41)
    want = L.dropout(f64(x), keep, p, f64(r) if res else None)
    size = np.abs(f64(x)) / (1.0 - p) + (np.abs(f64(r)) if res else 0.0)
    within(f64(out), want, size * (4 * E + HALF[dtype]), "dropout")
    assert around_untouched(torch, out, buf)


@pytest.mark.parametrize("dtype,rows,cols,ld", [("bf16", 5000, 1000, 1003), ("fp32", 4, 1 << 20, 1 << 20), ("bf16", 2100000, 1, 2)])
def test_dropout_of_many_elements(torch, dtype, rows, cols, ld):
    x = torch.ones(rows, ld, dtype=dt(torch, dtype), device=DEV)[:, :cols]
    out = torch.full((rows, ld), 7.0, dtype=x.dtype, device=DEV)
    M.dropout(x, out[:, :cols], 0.5, SEED, site=1 << 31, step=(1 << 32) - 1)
    o = out[:, :cols]
    assert bool(((o == 0) | (o == 2)).all()) and bool((out[:, cols:] == 7).all())
    # five standard deviations of a binomial count
    assert abs(int((o == 2).sum()) - rows * cols / 2) < 2.5 * np.sqrt(rows * cols)
    for r0, c0 in ((0, 0), (rows - 3, max(0, cols - 70)), (rows // 2, cols // 2 // 4 * 4)):
        part = o[r0:r0 + 3, c0:c0 + 70]
        keep = L.dropout_keep(part.shape[0], part.shape[1], 0.5, SEED, 1 << 31, (1 << 32) - 1, r0, c0)
        assert np.array_equal(f64(part) == 2, keep)


def test_dropout_in_place_and_its_gradient(torch):
    rng = np.random.default_rng(0)
    x, g = (vec(torch, rng.standard_normal((37, 130)).astype(np.float32)) for _ in range(2))
    out, dx = torch.empty_like(x), torch.empty_like(x)
    M.dropout(x, out, 0.3, 5, site=2, step=9)
    M.dropout(g, dx, 0.3, 5, site=2, step=9)
    # <out, g> = <x, dx>: the mask is the same, and so is the factor
    assert float((out.double() * g.double()).sum()) == pytest.approx(float((x.double() * dx.double()).sum()), rel=1e-6)
    y = x.clone()
    M.dropout(y, y, 0.3, 5, site=2, step=9)
    assert torch.equal(y, out)
    r = g.clone()
    M.dropout(x, r, 0.3, 5, site=2, step=9, residual=r)
    M.dropout(x, y, 0.3, 5, site=2, step=9, residual=g)
    assert torch.equal(r, y)


def test_dropout_leaves_nothing_of_what_it_drops(torch):
    x = torch.full((16, 64), float("inf"), device=DEV)
    x[::2] = float("nan")
    out = torch.empty_like(x)
    M.dropout(x, out, 0.5, SEED)
    keep = torch.from_numpy(L.dropout_keep(16, 64, 0.5, SEED, 0, 0)).to(DEV)
    assert bool((out[~keep] == 0).all()) and bool(torch.isnan(out[::2][keep[::2]]).all()) and bool(torch.isinf(out[1::2][keep[1::2]]).all())


def test_dropout_step_on_the_device_and_in_a_graph(torch):
    x = torch.randn(64, 256, device=DEV)
    out, step = torch.zeros_like(x), torch.zeros(1, dtype=torch.int64, device=DEV)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        M.dropout(x, out, 0.4, SEED, site=1, step=step)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        M.dropout(x, out, 0.4, SEED, site=1, step=step)
    for k in (0, 1, (1 << 32) + 5, 7):  # the low 32 bits count
        step.fill_(k)
        graph.replay()
        torch.cuda.synchronize()
        want = torch.empty_like(x)
        M.dropout(x, want, 0.4, SEED, site=1, step=k & 0xFFFFFFFF)
        assert torch.equal(out, want)


# ---------------------------------------------------------------- routing


def score_error(x, scoring):
    if scoring == "sigmoid":
        return (np.abs(x) + 8) * E
    with np.errstate(invalid="ignore"):
        return (x.max(axis=1, keepdims=True) - x + 60) * E


def check_route(torch, x, k, dtype, idt, bias=None, valid=None, ld=0, shift=0, first=True, seed=0, **how):
    rng = np.random.default_rng(seed)
    t, n = x.shape
    xd, _ = strided(torch, x, dtype, n + ld, shift)
    x = f64(xd)
    b = None if bias is None else vec(torch, bias)
    v = None if valid is None else torch.from_numpy(valid).to(DEV)
    choices = torch.full((t, k), 99, dtype=dt(torch, idt), device=DEV)
    weights = torch.full((t, k), 9.0, device=DEV)
    M.route_experts(xd, choices, weights, bias=b, valid=v, **how)
    want, w = L.route(x, k, bias=None if bias is None else f64(b), valid=valid, **how)
    assert np.array_equal(choices.cpu().numpy(), want)
    same = {q: how[q] for q in ("scoring", "renormalize", "scale") if q in how}
    scoring, scale = how.get("scoring", "softmax"), how.get("scale", 1.0)
    at = np.maximum(want, 0)
    err = np.take_along_axis(score_error(x, scoring), at, 1)
    err = np.where(want >= 0, err, 0.0)
    bound = np.broadcast_to(err.max(axis=1, keepdims=True), err.shape)
    within(f64(weights), w, np.abs(w) * (2 * bound + (k + 4) * E), "weights")
    # the gradient, with choices that no choice of experts gives
    ch = want.copy()
    if k > 1 and t > 2:
        ch[t // 2, 0] = n
        ch[t // 3, 1] = ch[t // 3, 0]
    dw = rng.standard_normal((t, k)).astype(np.float32)
    held = rng.standard_normal((t, n))
    d, buf = strided(torch, held, dtype, n + ld, shift)
    held = f64(d)
    M.route_backward(xd, vec(torch, ch, idt), vec(torch, dw), d, first, valid=v, **same)
    g = L.route_backward(x, ch, dw, valid=valid, **same)
    s = L.scores(x, scoring)
    dead = np.zeros(t, dtype=bool) if valid is None else ~valid
    s[dead] = 0.0
    live = (ch >= 0) & (ch < n)
    at = np.where(live, ch, 0)
    ws = np.where(live, np.take_along_axis(s, at, 1), 0.0)
    total = ws.sum(axis=1, keepdims=True) + L.NORM_EPS if how.get("renormalize", True) else np.ones((t, 1))
    mean = (np.abs(dw) * ws).sum(axis=1, keepdims=True) / total if how.get("renormalize", True) else 0.0
    parts = scale / total * (np.abs(dw) + mean) * ws
    size = np.zeros((t, n))
    for j in range(k):
        np.add.at(size, (np.arange(t), at[:, j]), np.where(live[:, j], parts[:, j], 0.0))
    if scoring == "softmax":
        size = size + s * parts.sum(axis=1, keepdims=True)
    rel = 4 * np.nanmax(np.where(np.isfinite(score_error(x, scoring)), score_error(x, scoring), 0.0), axis=1, keepdims=True)
    # a score below 2^-126 is 0 in fp32: d x = s (ds - inner) loses at most 2^-126 (|ds| + |inner|) with it, where
    # |ds| <= scale / total (|dw| + mean) and |inner| <= the sum of the parts
    lost = TINY * ((scale / total * (np.abs(dw) + mean)).max(axis=1, keepdims=True) + parts.sum(axis=1, keepdims=True))
    tol = size * (rel + (k + 10) * E) + np.abs(g) * HALF[dtype] + lost
    if not first:
        tol = tol + (np.abs(g) + np.abs(held)) * (HALF[dtype] + E)
        g = g + held
    within(f64(d), g, tol, "gradient by the logits")
    assert around_untouched(torch, d, buf)


SHAPES = [(1, 1, 1), (61, 8, 2), (5, 3, 3), (200, 16, 4), (33, 17, 1), (40, 32, 8), (50, 60, 6), (40, 64, 2), (64, 100, 8), (30, 128, 5),
          (100, 256, 8), (20, 200, 32), (9, 512, 9), (7, 300, 4), (5, 1024, 8), (3, 1000, 32), (0, 8, 2)]


@pytest.mark.parametrize("t,n,k", SHAPES)
@pytest.mark.parametrize("dtype,idt,ld,shift", [("bf16", "int64", 0, 0), ("fp32", "int32", 3, 1)])
@pytest.mark.parametrize("scoring,biased,renorm", [("softmax", False, True), ("sigmoid", True, True), ("softmax", True, False),
                                                  ("sigmoid", False, False)])
def test_route(torch, t, n, k, dtype, idt, ld, shift, scoring, biased, renorm):
    rng = np.random.default_rng(t + n + k)
    x = rng.standard_normal((t, n)) * 1.5
    valid = None
    if t > 20:
        valid = rng.random(t) < 0.8
        x[np.argwhere(~valid)[0]] = np.nan  # not read
    bias = (0.2 * rng.standard_normal(n)).astype(np.float32) if biased else None
    with np.errstate(invalid="ignore"):
        check_route(torch, x, k, dtype, idt, bias, valid, ld, shift, first=renorm, scoring=scoring, renormalize=renorm,
                    scale=2.5)


@pytest.mark.parametrize("n,groups,keep,top,k", [(64, 8, 4, 2, 6), (256, 8, 4, 2, 8), (12, 3, 1, 1, 4), (32, 32, 5, 1, 5), (30, 5, 2, 2, 8),
                                                (1024, 32, 3, 2, 8), (160, 8, 3, 1, 6), (96, 2, 2, 2, 7), (4, 2, 1, 2, 2), (21, 7, 6, 2, 9)])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("scoring,biased", [("softmax", False), ("sigmoid", True), ("sigmoid", False), ("softmax", True)])
def test_route_within_groups(torch, n, groups, keep, top, k, dtype, scoring, biased):
    rng = np.random.default_rng(n + groups)
    x = rng.standard_normal((45, n))
    x[3, :n // groups] = -np.inf           # a group without an expert
    x[4] = -np.inf                         # none at all
    x[5, 1:] = -np.inf                     # one
    x[6] = 0.25                            # all equal: by index
    bias = (0.1 * rng.standard_normal(n)).astype(np.float32) if biased else None
    check_route(torch, x, k, dtype, "int32", bias, scoring=scoring, groups=groups, keep_groups=keep, group_top=top,
                scale=1.5)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_route_of_nearly_equal_ranks(torch, dtype):
    # ranks that differ by a few 2^-26: fp32 sums of score and bias tie or swap, the definition tells them apart
    rng = np.random.default_rng(11)
    n, t = 256, 64
    base = np.round(rng.standard_normal((t, n)) * 4) / 4
    x = base + (rng.integers(-3, 4, (t, n)) * 2.0 ** -22 if dtype == "fp32" else 0.0)
    levels = 1.0 / (1.0 + np.exp(-base[0]))
    bias = (0.9 - levels + rng.integers(-2, 3, n) * 2.0 ** -24).astype(np.float32)
    for scoring in ("sigmoid", "softmax"):
        check_route(torch, x, 8, dtype, "int32", bias, scoring=scoring)
        check_route(torch, x, 8, dtype, "int32", bias, scoring=scoring, groups=8, keep_groups=3, group_top=2)
    check_route(torch, x, 8, dtype, "int64", np.zeros(n, dtype=np.float32), scoring="sigmoid")


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("n,groups,keep,top", [(256, 1, 1, 1), (64, 8, 4, 1), (256, 8, 4, 2), (1024, 1, 1, 1), (100, 1, 1, 1)])
def test_route_of_many_equal_ranks(torch, dtype, n, groups, keep, top):
    # logits of a few values, zeros of both signs among them: most choices are decided by the index
    rng = np.random.default_rng(n)
    x = rng.integers(-2, 3, (200, n)) * 0.25
    x[:, ::3] *= -1.0
    x[:50] = np.where(x[:50] < 0.5, x[:50], np.where(rng.random((50, n)) < 0.01, 0.5, -0.0))
    x[50:60] = np.where(rng.random((10, n)) < 0.5, 0.0, -0.0)
    x[60:70] = 1.0 + rng.integers(0, 3, (10, n)) * 2.0 ** (-23 if dtype == "fp32" else -7)
    for bias in (None, np.zeros(n, dtype=np.float32), (rng.integers(-1, 2, n) * 0.125).astype(np.float32)):
        check_route(torch, x, 8, dtype, "int32", bias, scoring="sigmoid", groups=groups, keep_groups=keep, group_top=top)
        check_route(torch, x, 3, dtype, "int32", bias, scoring="softmax", groups=groups, keep_groups=keep, group_top=top)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_route_of_many_tokens(torch, dtype):
    # against the definition in torch, in 64 bits: with so many tokens some have ranks that fp32 does not tell apart
    g = torch.Generator(DEV).manual_seed(3)
    t, n, k = 20000, 256, 8
    x = torch.randn(t, n, device=DEV, generator=g).to(dt(torch, dtype))
    bias = 0.1 * torch.randn(n, device=DEV, generator=g)
    for scoring in ("sigmoid", "softmax"):
        s = torch.sigmoid(x.double()) if scoring == "sigmoid" else torch.softmax(x.double(), 1)
        for b, groups in ((None, 1), (bias, 1), (bias, 8), (None, 8)):
            rank = s if b is not None or groups > 1 else x.double()
            rank = rank if b is None else rank + b.double()
            if groups > 1:
                value = rank.view(t, groups, -1).topk(2, 2).values.sum(2)
                keep = value.sort(dim=1, descending=True, stable=True).indices[:, :4]
                open_ = torch.zeros(t, groups, dtype=torch.bool, device=DEV).scatter_(1, keep, True)
                rank = torch.where(open_[:, :, None], rank.view(t, groups, -1), -torch.inf).view(t, n)
            want = rank.sort(dim=1, descending=True, stable=True).indices[:, :k]
            c, w = torch.empty(t, k, dtype=torch.int64, device=DEV), torch.empty(t, k, device=DEV)
            M.route_experts(x, c, w, scoring=scoring, bias=b, groups=groups, keep_groups=4 if groups > 1 else 1,
                            group_top=2 if groups > 1 else 1)
            assert torch.equal(c, want), (scoring, b is None, groups)
            sw = s.gather(1, want)
            assert float((w.double() - sw / sw.sum(1, keepdim=True)).abs().max()) < 2e-6


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_route_of_masks_and_extremes(torch, scoring):
    rng = np.random.default_rng(2)
    x = rng.standard_normal((12, 40))
    x[0, 5:] = -np.inf
    x[1] = -np.inf
    x[2] = np.float32(-3.4028235e38)       # a mask of the type's lowest value: all equal
    x[3, ::2] = np.float32(-3.4028235e38)
    x[4] = 90.0 * rng.standard_normal(40)
    x[5] = -200.0                          # sigmoids that underflow
    x[6, 7] = 3.0e38
    check_route(torch, x, 6, "fp32", "int32", scoring=scoring)
    bias = np.zeros(40, dtype=np.float32)
    bias[3], bias[9] = -np.inf, np.inf     # never, and always first
    check_route(torch, x[7:], 6, "fp32", "int32", bias, scoring=scoring)
    bias[9] = 0.0
    check_route(torch, x[:6], 6, "fp32", "int32", bias, scoring=scoring, renormalize=False)


@pytest.mark.parametrize("biased,groups,top", [(False, 1, 1), (True, 1, 1), (True, 4, 2), (False, 4, 2), (False, 4, 1)])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_route_of_nan(torch, biased, groups, top, scoring):
    # a NaN ranks below every number; where it reaches the chosen scores, so do the weights and the gradient
    x = torch.randn(6, 32, device=DEV)
    x[1, 3] = float("nan")
    x[2] = float("nan")
    x[3, :28] = float("nan")
    bias = torch.zeros(32, device=DEV) if biased else None
    c, w = torch.empty(6, 5, dtype=torch.int32, device=DEV), torch.empty(6, 5, device=DEV)
    M.route_experts(x, c, w, scoring=scoring, bias=bias, groups=groups, keep_groups=2 if groups > 1 else 1, group_top=top)
    c = c.cpu().numpy()
    assert all(len(set(r)) == 5 and r.min() >= 0 and r.max() < 32 for r in c)
    assert 3 not in c[1] or scoring == "softmax"
    bad = torch.isnan(w).all(1).tolist()
    assert bad[2] and not bad[0] and not bad[4] and bad[3] and bad[1] == (scoring == "softmax")
    d = torch.empty_like(x)
    M.route_backward(x, vec(torch, c, "int32"), torch.ones_like(w), d, True, scoring=scoring, renormalize=False)
    assert bool(torch.isnan(d[2]).any()) and not bool(torch.isnan(d[0]).any())


def test_route_gradient_against_differences(torch):
    x = torch.randn(40, 24, dtype=torch.float64, generator=torch.Generator().manual_seed(3))
    u = torch.randn(40, 24, dtype=torch.float64, generator=torch.Generator().manual_seed(4))
    dw = torch.randn(40, 3, generator=torch.Generator().manual_seed(5))
    for scoring in ("softmax", "sigmoid"):
        for renorm in (True, False):
            c, w = torch.empty(40, 3, dtype=torch.int64, device=DEV), torch.empty(40, 3, device=DEV)
            xd = x.float().to(DEV)
            M.route_experts(xd, c, w, scoring=scoring, renormalize=renorm)
            d = torch.empty_like(xd)
            M.route_backward(xd, c, dw.to(DEV), d, True, scoring=scoring, renormalize=renorm)

            def value(z):  # the choice held
                s = torch.softmax(z, 1) if scoring == "softmax" else torch.sigmoid(z)
                s = s.gather(1, c.cpu())
                return float(((s / s.sum(1, keepdim=True) if renorm else s) * dw.double()).sum())
            diff = (value(x + 1e-5 * u) - value(x - 1e-5 * u)) / 2e-5
            assert float((d.cpu().double() * u).sum()) == pytest.approx(diff, rel=1e-4, abs=1e-4)


# ------------------------------------------------- order and weighted sum


def make_choices(rng, t, k, experts, kind):
    c = np.stack([rng.permutation(max(experts, k))[:k] for _ in range(t)]) if t else np.zeros((0, k), dtype=np.int64)
    c = c.reshape(t, k)
    if kind == "one":
        c[:] = experts - 1
    elif kind == "none":
        c[:] = -1
    elif kind == "skewed":
        c = np.minimum((rng.pareto(0.8, (t, k)) * 2).astype(np.int64), experts - 1)
        c[rng.random((t, k)) < 0.1] = -1
    if t > 3 and kind != "one":
        c[t // 2, 0], c[t // 3, k - 1] = experts, -2 ** 31
    return c


@pytest.mark.parametrize("t,k,experts,kind", [(0, 2, 4, "any"), (1, 1, 1, "any"), (1, 8, 1024, "any"), (509, 2, 8, "any"), (777, 3, 600, "skewed"),
                                              (2048, 8, 64, "skewed"), (2049, 8, 64, "skewed"), (20000, 1, 5, "one"), (9001, 2, 256, "none"),
                                              (16411, 6, 160, "skewed"), (40000, 8, 1024, "any"), (5461, 3, 512, "any"), (2731, 6, 513, "any")])
@pytest.mark.parametrize("idt", ["int32", "int64"])
def test_order(torch, t, k, experts, kind, idt):
    c = make_choices(np.random.default_rng(t + k), t, k, experts, kind)
    flat = c.reshape(-1)
    key = np.where((flat >= 0) & (flat < experts), flat, experts)
    by = np.argsort(key, kind="stable")
    n = int((key < experts).sum())
    tokens = torch.full((t * k + 8,), 7, dtype=torch.int32, device=DEV)
    offsets = torch.full((experts + 9,), 7, dtype=torch.int32, device=DEV)
    place = torch.full((t * k + 8,), 7, dtype=torch.int32, device=DEV)
    M.expert_order(vec(torch, c, idt), tokens[:t * k], offsets[:experts + 1], place[:t * k].view(t, k),
                   poisoned(torch, M.expert_order_workspace_bytes(t, k, experts)))
    want_place = np.full(t * k, -1)
    want_place[by[:n]] = np.arange(n)
    want_tokens = np.full(t * k, -1)
    want_tokens[:n] = by[:n] // k
    assert np.array_equal(offsets[:experts + 1].cpu().numpy(), np.searchsorted(key[by], np.arange(experts + 1)))
    assert np.array_equal(tokens[:t * k].cpu().numpy(), want_tokens)
    assert np.array_equal(place[:t * k].cpu().numpy(), want_place)
    assert bool((tokens[t * k:] == 7).all()) and bool((offsets[experts + 1:] == 7).all()) and bool((place[t * k:] == 7).all())


@pytest.mark.parametrize("t,k,experts,dim", [(0, 2, 3, 8), (1, 1, 1, 1), (1, 8, 16, 4096), (7, 2, 4, 5), (61, 3, 5, 1001), (40, 9, 20, 130), (300, 2, 8, 64),
                                             (20, 17, 40, 513)])
@pytest.mark.parametrize("dtype,ld,shift,weighted,res", [("bf16", 0, 0, True, True), ("fp32", 3, 1, True, False), ("bf16", 5, 3, False, True),
                                                         ("fp32", 0, 0, False, False)])
def test_combine(torch, t, k, experts, dim, dtype, ld, shift, weighted, res):
    rng = np.random.default_rng(t + dim)
    _, _, place = L.expert_order(make_choices(rng, t, k, experts, "any"), experts)
    rows = t * k + 3
    if t > 3:
        place[1, 0] = rows  # behind the rows: adds nothing
    y, _ = strided(torch, rng.standard_normal((rows, dim)), dtype, dim + ld, shift)
    r, _ = strided(torch, rng.standard_normal((t, dim)), dtype, dim + 2 * ld, shift)
    y[t * k:] = float("nan")  # of no place: not read
    w = rng.standard_normal((t, k)).astype(np.float32)
    out, obuf = strided(torch, np.zeros((t, dim)), dtype, dim + ld, shift)
    p, wd = vec(torch, place, "int32"), vec(torch, w) if weighted else None
    M.expert_combine(y, p, out, weights=wd, residual=r if res else None)
    wh, rh = (w if weighted else None), (f64(r) if res else None)
    want = L.expert_combine(f64(y), place, wh, rh)
    size = L.expert_combine(np.abs(f64(y)), place, np.abs(w) if weighted else None, None if rh is None else np.abs(rh))
    within(f64(out), want, size * (k + 2) * E + np.abs(want) * HALF[dtype], "weighted sum")
    assert around_untouched(torch, out, obuf)
    # backwards
    g, _ = strided(torch, rng.standard_normal((t, dim)), dtype, dim + ld, shift)
    dy, dbuf = strided(torch, rng.standard_normal((rows, dim)), dtype, dim + ld, shift)
    held = f64(dy)
    dw = torch.full((t, k), 9.0, device=DEV)
    M.expert_combine_backward(g, p, dy, weights=wd, y=y, dweights=dw)
    want, wantw = L.expert_combine_backward(f64(g), np.nan_to_num(f64(y)), place, held, wh)
    within(f64(dy), want, np.abs(want) * (HALF[dtype] + E), "gradient of the rows")
    _, sizew = L.expert_combine_backward(np.abs(f64(g)), np.abs(np.nan_to_num(f64(y))), place, held, wh)
    within(f64(dw), wantw, sizew * (dim / 64 + 10) * E, "gradient of the weights")
    assert around_untouched(torch, dy, dbuf)
    # either alone, and over y itself
    dy2, dw2 = torch.empty_like(dy.contiguous()), torch.empty_like(dw)
    dy2.copy_(torch.from_numpy(held))
    M.expert_combine_backward(g, p, dy2, weights=wd)
    M.expert_combine_backward(g, p, weights=wd, y=y, dweights=dw2)
    assert torch.equal(dy2, dy) and torch.equal(dw2, dw)
    last = y.clone().contiguous()
    M.expert_combine_backward(g, p, last, weights=wd, y=last, dweights=dw2)
    at = torch.from_numpy(place[(place >= 0) & (place < rows)].reshape(-1)).to(DEV)
    assert torch.equal(last[at], dy[at]) and torch.equal(dw2, dw)
    if res:
        M.expert_combine(y, p, r, weights=wd, residual=r)
        assert torch.equal(r, out)


def test_gather_and_its_gradient(torch):
    # rows gathered by the slots' tokens; the gradient of that is the weighted sum without weights
    rng = np.random.default_rng(9)
    t, k, experts, dim = 100, 4, 12, 64
    c = make_choices(rng, t, k, experts, "skewed")
    tokens, place = torch.empty(t * k, dtype=torch.int32, device=DEV), torch.empty(t, k, dtype=torch.int32, device=DEV)
    offsets = torch.empty(experts + 1, dtype=torch.int32, device=DEV)
    M.expert_order(vec(torch, c, "int32"), tokens, offsets, place, poisoned(torch, M.expert_order_workspace_bytes(t, k, experts)))
    x, g = torch.randn(t, dim, device=DEV), torch.randn(t * k, dim, device=DEV)
    rows, dx = torch.empty(t * k, dim, device=DEV), torch.empty(t, dim, device=DEV)
    M.embed_forward(x, tokens, rows)
    assert bool((rows[int(offsets[-1]):] == 0).all())
    M.expert_combine(g, place, dx)
    assert float((rows.double() * g.double()).sum()) == pytest.approx(float((x.double() * dx.double()).sum()), rel=1e-5)
