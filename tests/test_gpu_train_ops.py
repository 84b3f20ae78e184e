"""The operators around the step on the GPU, against their fp64 definitions
(oracle/train_ops.py) on the same bits.

Tolerances, from the arithmetic (e = 2^-24, half a step of fp32; h = half a
step of the output's type, 2^-8 for bf16, e for fp32):
  lookup       one fp32 product, one rounding: h (1 + 2 e) + e
  its gradient (n + 4) e (scale sum|g| + |acc|) for n tokens of a row
  row sums     an exponential of a shifted logit d carries (2|d| + 4) e (the
               difference, the change of base, the hardware's exp2), the sum
               at most one e per addition of a thread, plus the tree:
               t = (2 sum p|d| + V / 64 + 64) e, relative to the sum
  lse, logp    t + 2 e (1 + |value|)
  gradient     |p dlogp| ((2|d| + 8) e + t) + p |ddlogp| t + h |value|, where
               ddlogp bounds how dlogp moves with its row's logp
  sums         the rows' own errors, and 2 e of the sum of magnitudes
Values below the smallest normal number may be flushed to 0 (1.2e-38).
"""

from __future__ import annotations

import numpy as np
import pytest

import muon_newton_schulz_step_amd as M
import oracle.train_ops as T

pytestmark = pytest.mark.gpu

E = 2.0 ** -24
HALF = {"bf16": 2.0 ** -8, "fp32": E}
TINY = 1.2e-38
DEV = "cuda:0"


@pytest.fixture(scope="module")
def torch():
    t = pytest.importorskip("torch")
    if not t.cuda.is_available():
        pytest.skip("no GPU")
    M.load()
    return t


def dt(torch, name):
    return {"bf16": torch.bfloat16, "fp32": torch.float32, "int32": torch.int32, "int64": torch.int64}[name]


def strided(torch, a, dtype, ld=None, shift=0, fill=7.0):
    """The matrix on the device with row stride ld, `shift` elements off its
    allocation's start; the allocation around it holds `fill`."""
    rows, cols = a.shape
    ld = ld or cols
    buf = torch.full((shift + max(rows, 1) * ld + 8,), fill, dtype=dt(torch, dtype), device=DEV)
    v = buf[shift:shift + rows * ld].view(rows, ld)[:, :cols]
    v.copy_(torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(DEV))
    return v, buf


def around_untouched(torch, view, buf, fill=7.0):
    mask = torch.ones_like(buf, dtype=torch.bool)
    off = view.storage_offset()
    rows, cols = view.shape
    for r in range(rows):
        mask[off + r * view.stride(0):off + r * view.stride(0) + cols] = False
    return bool((buf[mask].float() == fill).all())


def f64(t):
    return t.detach().double().cpu().numpy()


def vec(torch, a, dtype="fp32"):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV).to(dt(torch, dtype)).contiguous()


def poisoned(torch, nbytes):
    return torch.full((nbytes,), 0xFF, dtype=torch.uint8, device=DEV)


def within(got, want, tol, label):
    got, want, tol = np.asarray(got, np.float64), np.asarray(want, np.float64), np.broadcast_to(tol, np.shape(want))
    same = (got == want) | (np.isnan(got) & np.isnan(want))
    with np.errstate(invalid="ignore"):
        bad = ~(same | (np.abs(got - want) <= tol + TINY))
    if bad.any():
        i = tuple(np.argwhere(bad)[0])
        raise AssertionError(f"{label}: {int(bad.sum())} of {bad.size} off, first at {i}: {got[i]!r}, "
                             f"expected {want[i]!r} within {tol[i]:.3e}")


# -------------------------------------------------------------- embedding


def make_ids(rng, n, vocab, kind):
    if kind == "zipf":
        ids = np.minimum((rng.pareto(0.7, n) * 2).astype(np.int64), vocab - 1)
    elif kind == "one":
        ids = np.full(n, vocab // 2)
    elif kind == "pad":
        ids = np.full(n, -1)
    else:
        ids = rng.integers(0, vocab, n)
    if n > 3 and kind != "one":
        ids[rng.random(n) < 0.15] = -1
        ids[n // 2] = vocab          # just past the table
        ids[n // 3] = -2 ** 31       # the lowest int32
    return ids


@pytest.mark.parametrize("n,vocab,dim,kind", [
    (0, 5, 8, "any"), (1, 1, 1, "any"), (1, 1, 1, "pad"), (7, 1000, 4096, "any"), (5, 3, 7, "any"), (300, 17, 130, "any"),
    (1021, 257, 1001, "zipf"), (64, 100000, 64, "any"), (33, 40, 9, "pad")])
@pytest.mark.parametrize("dtype,idt,ld,shift", [("bf16", "int64", 0, 0), ("fp32", "int32", 3, 1), ("bf16", "int32", 5, 3)])
def test_lookup(torch, n, vocab, dim, kind, dtype, idt, ld, shift):
    rng = np.random.default_rng(n + vocab)
    tab, tbuf = strided(torch, rng.standard_normal((vocab, dim)), dtype, dim + ld, shift)
    ids = make_ids(rng, n, vocab, kind)
    out, obuf = strided(torch, np.zeros((n, dim)), dtype, dim + (ld + 1 if ld else 0), shift)
    scale = float(np.float32(np.sqrt(dim)))
    M.embed_forward(tab, vec(torch, ids, idt), out, scale=scale)
    want = T.embed_forward(f64(tab), ids, scale)
    within(f64(out), want, np.abs(want) * (HALF[dtype] * (1 + 2 * E) + E), "lookup")
    assert around_untouched(torch, out, obuf)


@pytest.mark.parametrize("dtype,dim,ld", [("bf16", 4096, 4096), ("bf16", 4099, 4101), ("fp32", 2050, 2051)])
def test_lookup_of_many_tokens(torch, dtype, dim, ld):
    # outputs of 64 MB and more take another way to memory
    n, vocab = 9000, 700
    g = torch.Generator(DEV).manual_seed(1)
    tab = torch.empty(vocab, ld, dtype=dt(torch, dtype), device=DEV).normal_(generator=g)[:, :dim]
    ids = torch.randint(-30, vocab + 30, (n,), generator=g, device=DEV)
    buf = torch.full((n, ld), 7.0, dtype=tab.dtype, device=DEV)
    M.embed_forward(tab, ids, buf[:, :dim], scale=2.0)  # twice a value: exact
    has = (ids >= 0) & (ids < vocab)
    assert torch.equal(buf[:, :dim], torch.where(has[:, None], tab[ids.clamp(0, vocab - 1)] * 2.0, 0.0).to(tab.dtype))
    assert bool((buf[:, dim:] == 7.0).all())


def check_embed_grad(torch, n, vocab, dim, kind, dtype, idt, first, ld=0, shift=0, scale=1.75, seed=0):
    rng = np.random.default_rng(1000 + n + vocab + seed)
    ids = make_ids(rng, n, vocab, kind)
    dout, _ = strided(torch, rng.standard_normal((n, dim)), dtype, dim + ld, shift)
    acc, abuf = strided(torch, rng.standard_normal((vocab, dim)), "fp32", dim + ld, shift)
    before = f64(acc)
    need = M.embed_backward_workspace_bytes(n, vocab, dim)
    iv, ws = vec(torch, ids, idt), poisoned(torch, need)
    keep = acc.clone()
    M.embed_backward(iv, dout, acc, first, ws, scale=scale)
    d64 = f64(dout)
    want = T.embed_backward(ids, d64, vocab, scale, None if first else before)
    mag = T.embed_backward(ids, np.abs(d64), vocab, abs(scale), None if first else np.abs(before))
    live = ids[(ids >= 0) & (ids < vocab)]
    counts = np.bincount(live, minlength=vocab)[:, None]
    within(f64(acc), want, (counts + 4) * E * mag, "embedding gradient")
    assert around_untouched(torch, acc, abuf)
    if not first:  # rows without a token keep their bits
        rest = torch.from_numpy(np.flatnonzero(counts[:, 0] == 0)).to(DEV)
        assert torch.equal(acc[rest], keep[rest])
    again, _ = strided(torch, before, "fp32", dim + ld, shift)
    again.copy_(keep)
    M.embed_backward(iv, dout, again, first, ws, scale=scale)
    assert torch.equal(again, acc), "a second run gives other bits"


@pytest.mark.parametrize("first", [True, False])
@pytest.mark.parametrize("n,vocab,dim,kind", [
    (0, 5, 8, "any"), (1, 1, 1, "any"), (1, 1, 1, "pad"), (2, 300, 513, "any"), (50, 40, 9, "pad"), (65, 3, 7, "one"),
    (300, 17, 130, "any"), (1021, 5000, 1000, "zipf"), (1024, 70000, 72, "any"), (1025, 300000, 40, "any"),
    (2500, 1, 256, "any"), (4097, 9, 260, "one"), (5000, 700, 1024, "zipf")])
def test_embedding_gradient(torch, n, vocab, dim, kind, first):
    check_embed_grad(torch, n, vocab, dim, kind, "bf16", "int64", first)


@pytest.mark.parametrize("first", [True, False])
@pytest.mark.parametrize("n,vocab,dim,kind,dtype,idt,ld,shift", [
    (700, 90, 515, "zipf", "fp32", "int32", 3, 1), (700, 90, 515, "zipf", "bf16", "int32", 2, 3),
    (3000, 20, 8, "any", "fp32", "int64", 0, 0), (20000, 600, 64, "zipf", "bf16", "int32", 0, 0),
    (20000, 600, 65, "one", "fp32", "int32", 1, 2)])
def test_embedding_gradient_layouts(torch, n, vocab, dim, kind, dtype, idt, ld, shift, first):
    check_embed_grad(torch, n, vocab, dim, kind, dtype, idt, first, ld, shift)


@pytest.mark.parametrize("first", [True, False])
@pytest.mark.parametrize("n,vocab,dim", [(3000, 600000, 9), (1024, 600000, 8), (1025, 600000, 8), (40000, 300, 24),
                                         (9000, 10240, 24)])  # the last: 40 rows of many chunks in one bucket
def test_embedding_gradient_of_one_bucket(torch, n, vocab, dim, first):
    # rows a multiple of 256 apart meet in one bucket of the sort: more than it sorts by counting, and keys of more
    # bits than one radix pass takes
    rng = np.random.default_rng(n)
    ids = rng.integers(0, (vocab + 255) // 256, n) * 256
    dout = torch.from_numpy(rng.integers(-8, 9, (n, dim)).astype(np.float32)).to(DEV)
    acc = torch.from_numpy(rng.integers(-8, 9, (vocab, dim)).astype(np.float32)).to(DEV)
    want = torch.zeros_like(acc) if first else acc.clone()
    iv = vec(torch, ids, "int64")
    want.index_add_(0, iv, dout)  # small whole numbers: exact in any order
    M.embed_backward(iv, dout, acc, first, poisoned(torch, M.embed_backward_workspace_bytes(n, vocab, dim)))
    assert torch.equal(acc, want)


@pytest.mark.parametrize("n,vocab", [(5, 9_000_000), (2000, 34_000_000)])
def test_embedding_gradient_of_a_long_table(torch, n, vocab):
    # more rows than one presence map of the zeros' workgroups covers
    rng = np.random.default_rng(n)
    ids = rng.integers(0, vocab, n)
    ids[0], ids[1] = vocab - 1, 0
    dout = torch.from_numpy(rng.integers(-8, 9, (n, 1)).astype(np.float32)).to(DEV)
    acc = torch.full((vocab, 1), 5.0, device=DEV)
    iv = vec(torch, ids, "int32")
    M.embed_backward(iv, dout, acc, True, poisoned(torch, M.embed_backward_workspace_bytes(n, vocab, 1)))
    want = torch.zeros_like(acc)
    want.index_add_(0, iv.long(), dout)
    assert torch.equal(acc, want)


def test_embedding_gradient_against_differences(torch):
    # the lookup is linear: <g, lookup(table + u) - lookup(table)> = <gradient, u>, in exact arithmetic; here
    # small whole numbers make every product and sum exact, so the two sides are equal bit for bit
    rng = np.random.default_rng(11)
    n, vocab, dim = 900, 50, 96
    ids = vec(torch, make_ids(rng, n, vocab, "zipf"), "int64")
    tab = vec(torch, rng.integers(-4, 5, (vocab, dim)).astype(np.float32))
    u = vec(torch, rng.integers(-4, 5, (vocab, dim)).astype(np.float32))
    g = vec(torch, rng.integers(-4, 5, (n, dim)).astype(np.float32))
    a, b, acc = torch.empty_like(g), torch.empty_like(g), torch.empty_like(tab)
    M.embed_forward(tab + u, ids, a, scale=2.0)
    M.embed_forward(tab, ids, b, scale=2.0)
    M.embed_backward(ids, g, acc, True, poisoned(torch, M.embed_backward_workspace_bytes(n, vocab, dim)), scale=2.0)
    assert float(((a - b).double() * g.double()).sum()) == float((acc.double() * u.double()).sum())


# ------------------------------------------------------- losses over logits


def make_logits(torch, rng, n, v, dtype, ld=0, shift=0, dead=0):
    x = rng.standard_normal((n, v)) * 2.0
    if dead and v > dead:
        x[:, v - dead:] = -np.inf
    live = v - dead if v > dead else v
    t = rng.integers(0, live, n) if n else np.zeros(0, np.int64)
    for r in range(n):
        x[r, t[r]] += rng.random() * 8.0
    lo, buf = strided(torch, x, dtype, v + ld, shift)
    return lo, buf, t


def row_tol(x, targets):
    """t (relative error of a row's sum) and |d| of each logit."""
    lp, lse = T.log_softmax(x)
    with np.errstate(all="ignore"):
        p = np.exp(lp)
        d = np.abs(x - x.max(axis=1, keepdims=True))
        pd = np.where(p > 0, p * np.where(np.isfinite(d), d, 0.0), 0.0)
    return p, np.where(np.isfinite(d), d, 0.0), (2 * np.nansum(pd, axis=1) + x.shape[1] / 64 + 64) * E


def grad_tol(x, targets, dlogp, ddlogp, want, dtype):
    p, d, t = row_tol(x, targets)
    a = np.abs(dlogp)[:, None]
    has = (targets >= 0) & (targets < x.shape[1])
    rows = np.arange(len(targets))[has]
    tol = p * a * ((2 * d + 8) * E + t[:, None]) + p * (ddlogp * t)[:, None]
    one = np.zeros_like(x)
    one[rows, targets[has]] = 1.0 - p[rows, targets[has]]
    # the target's own element: dlogp (1 - p), whose error is that of log p times p, and of dlogp
    tol += one * ((ddlogp * t)[:, None] + 4 * E * a)
    return tol + HALF[dtype] * np.abs(want) * 1.01


SHAPES = [(0, 5, 0), (1, 1, 0), (3, 2, 0), (2, 7, 0), (5, 8, 0), (4, 9, 0), (61, 511, 17), (7, 4099, 0), (2, 4096, 0), (3, 8193, 17),
          (5, 32064, 64), (3, 50257, 0), (2, 131072, 0)]
LAYOUTS = [("bf16", "int64", 0, 0), ("fp32", "int32", 0, 0), ("bf16", "int32", 3, 5), ("fp32", "int64", 1, 3)]


@pytest.mark.parametrize("n,v,dead", SHAPES)
@pytest.mark.parametrize("dtype,idt,ld,shift", LAYOUTS)
def test_token_logprob(torch, n, v, dead, dtype, idt, ld, shift):
    rng = np.random.default_rng(n + v)
    x, _, t = make_logits(torch, rng, n, v, dtype, ld, shift, dead)
    if n > 2:
        t[1], t[2] = -100, v
        x[1] = float("nan")  # a row without a target is not read
    logp = torch.full((n,), 3.0, device=DEV)
    lse = torch.full((n,), 3.0, device=DEV)
    M.token_logprob(x, vec(torch, t, idt), logp, lse)
    with np.errstate(invalid="ignore"):
        wp, wl = T.token_logprob(f64(x), t)
        _, _, tol = row_tol(f64(x), t) if n else (0, 0, np.zeros(0))
    within(f64(logp), wp, tol + 2 * E * (1 + np.abs(wp) + np.abs(wl)), "logp")
    within(f64(lse), wl, tol + 2 * E * (1 + np.abs(wl)), "lse")
    only = torch.full((n,), 3.0, device=DEV)
    M.token_logprob(x, vec(torch, t, idt), only)
    assert torch.equal(only, logp)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_logprob_extremes(torch, dtype):
    low = float(torch.finfo(dt(torch, dtype)).min)
    v = 1030
    x = torch.zeros((7, v), dtype=dt(torch, dtype), device=DEV)
    x[0] = float("-inf")               # nothing but -inf
    x[1] = low                         # masked everywhere with the type's lowest value
    x[2] = float("-inf")
    x[2, 5] = 1.0                      # one logit left, the target
    x[3] = low
    x[3, v - 1] = -low                 # both ends of the range in one row
    x[4, 0] = float("-inf")            # the target itself masked
    x[5, 3] = float("nan")
    x[6, 3] = float("inf")
    t = torch.tensor([0, 3, 5, v - 1, 0, 1, 1], device=DEV)
    logp, lse = torch.empty(7, device=DEV), torch.empty(7, device=DEV)
    M.token_logprob(x, t, logp, lse)
    logp, lse = logp.cpu().numpy(), lse.cpu().numpy()
    assert np.isnan(logp[0]) and lse[0] == -np.inf
    assert logp[1] == pytest.approx(-np.log(v), rel=4 * E) or logp[1] == pytest.approx(-np.log(v), abs=200 * E)
    assert logp[2] == 0.0 and lse[2] == 1.0
    assert logp[3] == 0.0 and lse[3] == np.float32(-low)
    assert logp[4] == -np.inf and lse[4] == pytest.approx(np.log(v - 1), abs=200 * E)
    assert np.isnan(logp[5]) and np.isnan(lse[5]) and np.isnan(logp[6])


def policy_inputs(torch, rng, n, v, dtype, idt, ld=0, shift=0, dead=0):
    x, buf, t = make_logits(torch, rng, n, v, dtype, ld, shift, dead)
    logp, _ = T.token_logprob(f64(x), t)
    lr = 0.15 * rng.standard_normal(n)
    for edge in (np.log(0.8), np.log(1.28)):  # away from where the derivative jumps
        lr = np.where(np.abs(lr - edge) < 1e-3, lr + 4e-3, lr)
    w = rng.random(n).astype(np.float32) / max(1, n)
    old, ref = (logp - lr).astype(np.float32), (logp + 0.3 * rng.standard_normal(n)).astype(np.float32)
    adv = rng.standard_normal(n).astype(np.float32)
    if n > 4:
        t[1], t[2], w[3] = -100, v, 0.0
        x[1], x[3] = float("nan"), float("inf")  # rows that do not count are not read
        old[1] = adv[3] = np.nan
    return x, buf, t, adv, w, old, ref


def check_policy(torch, x, t, adv, w, old, ref, dtype, idt, in_place=False, dl=None, kl=0.05):
    n, v = x.shape
    kw = dict(clip_low=0.2, clip_high=0.28, kl_coef=kl)
    x64 = f64(x)
    stats, logp = torch.full((4,), 9.0, device=DEV), torch.full((n,), 9.0, device=DEV)
    if dl is None:
        dl = x if in_place else torch.full((n, v), 9.0, dtype=x.dtype, device=DEV)
    ws = poisoned(torch, M.policy_loss_workspace_bytes(n))
    opt = dict(old_logp=None if old is None else vec(torch, old), ref_logp=None if ref is None else vec(torch, ref))
    M.policy_loss(x, vec(torch, t, idt), vec(torch, adv), vec(torch, w), stats, logp, dl, ws, **opt, **kw)
    with np.errstate(invalid="ignore"):
        ws_, wl, wd, dlogp = T.policy_loss(x64, t, adv, w, old, ref, **kw)
    if n == 0:
        assert not stats.any()
        return stats, logp, dl
    count = (t >= 0) & (t < v) & (w != 0)
    xc = np.where(count[:, None], x64, 0.0)
    _, _, tol = row_tol(xc, t)
    within(f64(logp), wl, np.where(count, tol + 2 * E * (1 + np.abs(wl)) * 12, 0.0), "logp")
    a, wt = np.where(count, np.abs(adv), 0.0), np.where(count, w, 0.0)
    with np.errstate(all="ignore"):
        r = np.ones(n) if old is None else np.where(count, np.exp(np.where(count, wl - old, 0.0)), 0.0)
        ed = np.zeros(n) if ref is None else np.exp(np.where(count, ref - wl, 0.0))
    ddlogp = wt * (a * r + abs(kl) * ed)
    within(f64(dl), wd, grad_tol(xc, np.where(count, t, -1), dlogp, ddlogp, wd, dtype), "dlogits")
    slack = (wt * ((a * r + abs(kl) * (1 + ed)) * (tol + 4 * E))).sum()
    mag = (wt * (a * np.maximum(r, 1.28) + abs(kl) * (1 + ed))).sum()
    within(f64(stats)[:2], ws_[:2], slack + 2 * E * mag, "loss")
    within(f64(stats)[2:], ws_[2:], (wt * (1 + ed) * (tol + 4 * E)).sum() + 2 * E * wt.sum(), "kl, clipped")
    return stats, logp, dl


@pytest.mark.parametrize("n,v,dead", SHAPES)
@pytest.mark.parametrize("dtype,idt,ld,shift", LAYOUTS)
def test_policy_loss(torch, n, v, dead, dtype, idt, ld, shift):
    rng = np.random.default_rng(n + v + 1)
    x, _, t, adv, w, old, ref = policy_inputs(torch, rng, n, v, dtype, idt, ld, shift, dead)
    dl, dbuf = strided(torch, np.zeros((n, v)), dtype, v + (ld + 2 if ld else 0), shift)
    stats, logp, d = check_policy(torch, x, t, adv, w, old, ref, dtype, idt, dl=dl)
    assert around_untouched(torch, d, dbuf)
    s2, l2, d2 = check_policy(torch, x, t, adv, w, old, ref, dtype, idt)
    assert torch.equal(stats, s2) and torch.equal(logp, l2) and torch.equal(d, d2), "other bits in another layout"
    s3, l3, d3 = check_policy(torch, x, t, adv, w, old, ref, dtype, idt, in_place=True)
    assert torch.equal(stats, s3) and torch.equal(logp, l3) and torch.equal(d, d3), "other bits in place"


@pytest.mark.parametrize("n,v", [(300, 1000), (1500, 257), (2600, 64), (700, 20001)])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_policy_loss_many_rows(torch, n, v, dtype):
    rng = np.random.default_rng(n)
    x, _, t, adv, w, old, ref = policy_inputs(torch, rng, n, v, dtype, "int64")
    check_policy(torch, x, t, adv, w, old, ref, dtype, "int64")


@pytest.mark.parametrize("n,v", [(1, 65537), (9, 70001), (128, 65600), (129, 65600)])
@pytest.mark.parametrize("dtype,ld,shift", [("bf16", 0, 0), ("fp32", 3, 1)])
def test_policy_loss_few_long_rows(torch, n, v, dtype, ld, shift):
    rng = np.random.default_rng(n)
    x, _, t, adv, w, old, ref = policy_inputs(torch, rng, n, v, dtype, "int64", ld, shift)
    t[0] = v - 1 if n < 9 else 0
    old[0] = ref[0] = float(T.token_logprob(f64(x[:1]), t[:1])[0][0]) + 0.01
    dl, dbuf = strided(torch, np.zeros((n, v)), dtype, v + ld, shift)
    stats, logp, d = check_policy(torch, x, t, adv, w, old, ref, dtype, "int64", dl=dl)
    assert around_untouched(torch, d, dbuf)
    again = check_policy(torch, x, t, adv, w, old, ref, dtype, "int64")
    assert all(torch.equal(a, b) for a, b in zip(again, (stats, logp, d))), "a second run gives other bits"
    place = check_policy(torch, x, t, adv, w, old, ref, dtype, "int64", in_place=True)
    assert all(torch.equal(a, b) for a, b in zip(place, (stats, logp, d))), "other bits in place"


@pytest.mark.parametrize("have_old,have_ref,kl", [(False, True, 0.05), (True, False, 0.05), (False, False, 0.0),
                                                  (True, True, 0.0)])
def test_policy_loss_options(torch, have_old, have_ref, kl):
    rng = np.random.default_rng(5)
    x, _, t, adv, w, old, ref = policy_inputs(torch, rng, 40, 333, "fp32", "int32")
    check_policy(torch, x, t, adv, w, old if have_old else None, ref if have_ref else None, "fp32", "int32", kl=kl)


def test_policy_gradient_against_differences(torch):
    # the kernel's gradient along a direction against the fp64 loss's central difference on the same logits:
    # third-order truncation is below 1e-8 of the terms at h = 1e-4; the gradient's own tolerance is relative
    rng = np.random.default_rng(6)
    n, v = 24, 501
    x, _, t, adv, w, old, ref = policy_inputs(torch, rng, n, v, "fp32", "int64")
    x[1], x[3] = 0.0, 0.0
    old[1] = adv[3] = 0.0
    _, _, d = check_policy(torch, x, t, adv, w, old, ref, "fp32", "int64")
    x64, kw = f64(x), dict(clip_low=0.2, clip_high=0.28, kl_coef=0.05)
    for seed in range(3):
        u = np.random.default_rng(seed).standard_normal((n, v))
        u *= 0.05
        h = 1e-3
        diff = (T.policy_loss(x64 + h * u, t, adv, w, old, ref, **kw)[0][0]
                - T.policy_loss(x64 - h * u, t, adv, w, old, ref, **kw)[0][0]) / (2 * h)
        got = float((f64(d) * u).sum())
        assert got == pytest.approx(diff, abs=float((np.abs(f64(d)) * np.abs(u)).sum()) * 1e-5 + 1e-9)


def pref_inputs(torch, rng, lens, lead, tail, v, dtype, ld=0, shift=0, dead=0):
    off = np.cumsum([lead] + list(lens))
    n = int(off[-1]) + tail
    x, buf, t = make_logits(torch, rng, n, v, dtype, ld, shift, dead)
    t[rng.random(n) < 0.3] = -100
    logp, _ = T.token_logprob(f64(x), t)
    ref = np.array([logp[off[s]:off[s + 1]].sum() + rng.standard_normal() * np.sqrt(max(1, lens[s]))
                    for s in range(len(lens))], dtype=np.float32)
    return x, buf, t, off, ref


def check_pref(torch, x, t, off, ref, dtype, idt, beta=0.1, smooth=0.05, in_place=False, dl=None):
    n, v = x.shape
    seqs, x64 = len(ref), f64(x)
    loss, rew = torch.full((1,), 9.0, device=DEV), torch.full((seqs,), 9.0, device=DEV)
    if dl is None:
        dl = x if in_place else torch.full((n, v), 9.0, dtype=x.dtype, device=DEV)
    ws = poisoned(torch, M.preference_loss_workspace_bytes(n, seqs // 2))
    M.preference_loss(x, vec(torch, t, idt), vec(torch, off, idt), vec(torch, ref), loss, rew, dl, ws, beta=beta,
                      label_smoothing=smooth)
    with np.errstate(invalid="ignore"):
        wl, wr, wd, dlogp = T.preference_loss(x64, t, off, ref, beta, smooth)
        logp, _ = T.token_logprob(x64, t)
    live = (t >= 0) & (t < v)
    tol = np.where(live, row_tol(x64, t)[2], 0.0) if n else np.zeros(0)
    seq_tol = np.array([tol[off[s]:off[s + 1]].sum() for s in range(seqs)])
    gain_tol = beta * seq_tol + 4 * E * np.abs(wr)
    within(f64(rew), wr, gain_tol, "rewards")
    pair_tol = gain_tol[:seqs // 2] + gain_tol[seqs // 2:]
    within(f64(loss), [wl], pair_tol.mean() + 4 * E * (1 + abs(wl)), "loss")
    if n:
        # the coefficient is beta / pairs sigmoid(m) + const, of slope at most beta / (4 pairs)
        dd = np.zeros(n)
        for s in range(seqs):
            dd[off[s]:off[s + 1]] = beta / (seqs // 2) / 4 * pair_tol[s % (seqs // 2)]
        xc = np.where(live[:, None], x64, 0.0)
        p, _, t_ = row_tol(xc, t)
        gt = grad_tol(xc, np.where(live, t, -1), dlogp, np.zeros(n), wd, dtype)
        gt += np.where(live, dd + np.abs(dlogp) * t_, 0.0)[:, None] * (p + (np.arange(v) == t[:, None]))
        within(f64(dl), wd, np.where(live[:, None], gt, 0.0), "dlogits")
    return loss, rew, dl


@pytest.mark.parametrize("lens,lead,tail,v,dead", [
    ([1, 1], 0, 0, 1, 0), ([0, 0], 0, 0, 5, 0), ([2, 0], 0, 3, 9, 0), ([3, 5, 1, 7], 1, 2, 513, 17), ([40, 90], 0, 0, 4099, 0),
    ([150, 100, 120, 180], 0, 0, 700, 0), ([300] * 2, 5, 0, 64, 0), ([3] * 24, 0, 1, 8200, 0), ([2, 1], 0, 0, 50257, 0),
    ([1, 2, 2, 1], 0, 0, 131072, 0)])
@pytest.mark.parametrize("dtype,idt,ld,shift", LAYOUTS)
def test_preference_loss(torch, lens, lead, tail, v, dead, dtype, idt, ld, shift):
    rng = np.random.default_rng(sum(lens) + v)
    x, _, t, off, ref = pref_inputs(torch, rng, lens, lead, tail, v, dtype, ld, shift, dead)
    dl, dbuf = strided(torch, np.zeros(tuple(x.shape)), dtype, v + (ld + 2 if ld else 0), shift)
    loss, rew, d = check_pref(torch, x, t, off, ref, dtype, idt, dl=dl)
    assert around_untouched(torch, d, dbuf)
    l2, r2, d2 = check_pref(torch, x, t, off, ref, dtype, idt, in_place=True)
    assert torch.equal(loss, l2) and torch.equal(rew, r2) and torch.equal(d, d2), "other bits in place"


def test_preference_loss_far_apart(torch):
    # margins at which exp would overflow or vanish in the naive form
    v = 50
    x = torch.zeros((4, v), device=DEV)
    t, off = np.array([0, 1, 2, 3]), np.array([0, 1, 2, 3, 4])
    for smooth in (0.0, 0.1):
        check_pref(torch, x, t, off, np.array([1e5, -1e5, -1e5, 1e5], dtype=np.float32), "fp32", "int64", 0.5, smooth)


def test_preference_loss_bad_offsets_touch_no_row_outside(torch):
    # decreasing and out-of-range offsets: results unspecified but the buffers around stay as they are
    rng = np.random.default_rng(9)
    x, _, t = make_logits(torch, rng, 6, 40, "fp32")
    dl, dbuf = strided(torch, np.zeros((6, 40)), "fp32", 40, 4)
    for off in ([0, 100, 3, -7, 6], [2 ** 40, -2 ** 40, 2, 4, 2 ** 62], [5, 4, 3, 2, 1]):
        loss, rew = torch.empty(1, device=DEV), torch.empty(4, device=DEV)
        M.preference_loss(x, vec(torch, t, "int64"), vec(torch, np.array(off), "int64"), torch.zeros(4, device=DEV),
                          loss, rew, dl, poisoned(torch, M.preference_loss_workspace_bytes(6, 2)))
        torch.cuda.synchronize()
        assert around_untouched(torch, dl, dbuf)


def big_pref(torch, lens, lead, tail, v, dtype, ld, seed):
    """A preference case too large for the host: logits, targets (some of them none), offsets, references."""
    g = torch.Generator(DEV).manual_seed(seed)
    off = np.cumsum([lead] + list(lens))
    n = int(off[-1]) + tail
    buf = torch.empty(n * ld, dtype=dt(torch, dtype), device=DEV).normal_(0.0, 2.0, generator=g)
    x = buf.view(n, ld)[:, :v]
    t = torch.randint(0, v, (n,), generator=g, device=DEV)
    t[torch.rand(n, generator=g, device=DEV) < 0.3] = -1
    ref = []
    for s in range(len(lens)):
        lp, _, _, _ = big_rows(torch, x[int(off[s]):int(off[s + 1])], t[int(off[s]):int(off[s + 1])])
        ref.append(float(lp.sum()) + float(torch.randn(1, generator=g, device=DEV)) * np.sqrt(max(1, lens[s])))
    return x, t, torch.tensor(off, device=DEV), torch.tensor(ref, device=DEV, dtype=torch.float32)


def big_rows(torch, x, t):
    """logp, p, |d| and the row sums' relative tolerance of rows, in fp64 (0 where a row has no target)."""
    z = x.double()
    lp = torch.log_softmax(z, 1)
    live = (t >= 0) & (t < x.shape[1])
    logp = torch.where(live, lp.gather(1, t.clamp(0, x.shape[1] - 1)[:, None])[:, 0], 0.0)
    p, d = lp.exp(), (z - z.max(1, keepdim=True).values).abs()
    tol = torch.where(live, (2 * (p * d).sum(1) + x.shape[1] / 64 + 64) * E, 0.0)
    return logp, p, d, tol


@pytest.mark.parametrize("lens,lead,tail,v,dtype,ld", [
    # more than 256 MB: ragged pairs, an empty sequence and an empty pair, rows before and after them
    ([300, 0, 0, 511, 40, 500, 333, 0, 420, 1], 3, 650, 50257, "bf16", 50257),
    ([150, 700, 260, 10, 600, 520], 0, 0, 32001, "fp32", 32003)])
def test_preference_loss_in_one_walk(torch, lens, lead, tail, v, dtype, ld):
    x, t, off, ref = big_pref(torch, lens, lead, tail, v, dtype, ld, 5)
    n, seqs, beta, smooth = x.shape[0], len(lens), 0.1, 0.05
    pairs = seqs // 2
    assert x.numel() * x.element_size() > 256 << 20
    o = off.tolist()

    def call(x, dl):
        loss, rew = torch.full((1,), 9.0, device=DEV), torch.full((seqs,), 9.0, device=DEV)
        M.preference_loss(x, t, off, ref, loss, rew, dl, poisoned(torch, M.preference_loss_workspace_bytes(n, pairs)),
                          beta=beta, label_smoothing=smooth)
        return loss, rew, dl
    loss, rew, dl = call(x, torch.full((n, v), 9.0, dtype=x.dtype, device=DEV))
    sums, seq_tol = np.zeros(seqs), np.zeros(seqs)
    for s in range(seqs):
        lp, _, _, tol = big_rows(torch, x[o[s]:o[s + 1]], t[o[s]:o[s + 1]])
        sums[s], seq_tol[s] = float(lp.sum()), float(tol.sum())
    gain = sums - f64(ref)
    m = beta * (gain[:pairs] - gain[pairs:])
    want = ((1 - smooth) * np.logaddexp(0, -m) + smooth * np.logaddexp(0, m)).mean()
    gain_tol = beta * seq_tol + 4 * E * np.abs(beta * gain)
    pair_tol = gain_tol[:pairs] + gain_tol[pairs:]
    within(f64(rew), beta * gain, gain_tol, "rewards")
    within(f64(loss), [want], pair_tol.mean() + 4 * E * (1 + abs(want)), "loss")
    c = beta / pairs * (1 / (1 + np.exp(-m)) - (1 - smooth))
    assert not dl[:o[0]].any() and not dl[o[-1]:].any()
    for s in range(seqs):
        for r0 in range(o[s], o[s + 1], 128):
            r = slice(r0, min(r0 + 128, o[s + 1]))
            _, p, d, tol = big_rows(torch, x[r], t[r])
            live = ((t[r] >= 0) & (t[r] < v)).double()[:, None]
            a = live * (c[s] if s < pairs else -c[s - pairs])
            one = torch.zeros_like(p).scatter_(1, t[r].clamp(0, v - 1)[:, None], 1.0)
            wd = a * (one - p)
            a = a.abs()
            dd = live * beta / pairs / 4 * pair_tol[s % pairs]
            lim = p * a * ((2 * d + 8) * E + tol[:, None]) + one * (1 - p) * 4 * E * a + 1.01 * HALF[dtype] * wd.abs()
            lim = lim + (dd + a * tol[:, None]) * (p + one) + TINY
            assert bool(((dl[r].double() - wd).abs() <= lim).all()), f"dlogits of sequence {s}, rows {r}"
    again = call(x, torch.full((n, v), 9.0, dtype=x.dtype, device=DEV))
    assert all(torch.equal(p, q) for p, q in zip(again, (loss, rew, dl))), "a second run gives other bits"
    place = call(x, x)
    assert all(torch.equal(p, q) for p, q in zip(place, (loss, rew, dl))), "other bits in place"


def test_preference_loss_walk_in_a_graph(torch):
    n, v, lens = 2700, 50257, [300, 410, 500, 140, 350, 450, 250, 300]
    x, t, off, ref = big_pref(torch, lens, 0, 0, v, "bf16", v, 1)
    assert x.shape[0] == n
    ws = poisoned(torch, M.preference_loss_workspace_bytes(n, 4))

    def outs():
        return torch.empty(1, device=DEV), torch.empty(8, device=DEV), torch.empty_like(x)
    one, two = outs(), outs()

    def call(o):
        M.preference_loss(x, t, off, ref, o[0], o[1], o[2], ws)
    call(two)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(one)
    for k in range(1, 4):
        x.mul_(0.9)
        ref.add_(0.5 * k)
        ws.fill_(0x5A + k)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        call(two)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(one, two)), f"replay {k}"
    graph.reset()


def test_more_rows_than_one_launch_takes(torch):
    n, v = (1 << 21) + 5, 3
    g = torch.Generator(DEV).manual_seed(2)
    x = torch.randn(n, v, generator=g, device=DEV)
    t = torch.randint(0, v, (n,), generator=g, device=DEV, dtype=torch.int32)
    t[::7] = -1
    live = t >= 0
    z = torch.log_softmax(x.double(), 1)
    lp = torch.where(live, z.gather(1, t.clamp(min=0).long()[:, None])[:, 0], 0.0)
    logp = torch.empty(n, device=DEV)
    M.token_logprob(x, t, logp)
    # three terms a row: the sum's relative error is below (2 |d| + 68) e with |d| < 16
    tol = 100 * E * (1 + lp.abs())
    assert bool(((logp.double() - lp).abs() <= tol).all())
    w = torch.full((n,), 1.0 / n, device=DEV)
    adv = torch.randn(n, generator=g, device=DEV)
    stats, lp2, d = torch.empty(4, device=DEV), torch.empty(n, device=DEV), torch.empty_like(x)
    M.policy_loss(x, t, adv, w, stats, lp2, d, poisoned(torch, M.policy_loss_workspace_bytes(n)))
    assert torch.equal(lp2, logp)
    # ratio 1 in every row: the loss is -sum w a over the live rows
    aw = torch.where(live, adv.double() * w.double(), 0.0)
    assert float(stats[0]) == pytest.approx(-float(aw.sum()), abs=2 * E * float(aw.abs().sum()))
    one = torch.zeros_like(z).scatter_(1, t.clamp(min=0).long()[:, None], 1.0)
    want = -aw[:, None] * (one - z.exp())
    assert bool(((d.double() - want).abs() <= 200 * E * aw.abs()[:, None] + TINY).all())
    off = torch.tensor([2, n // 3, n // 2, n - 70, n - 1], device=DEV)
    sums = [float(lp[a:b].sum()) for a, b in zip(off.tolist(), off.tolist()[1:])]
    ref = torch.tensor([round(s) for s in sums], device=DEV, dtype=torch.float32)
    loss, rew = torch.empty(1, device=DEV), torch.empty(4, device=DEV)
    M.preference_loss(x, t, off, ref, loss, rew, d, poisoned(torch, M.preference_loss_workspace_bytes(n, 2)), beta=1e-3)
    gain = np.array(sums) - f64(ref)
    err = np.array([float(tol[a:b].sum()) for a, b in zip(off.tolist(), off.tolist()[1:])])
    within(f64(rew), 1e-3 * gain, 1e-3 * err + 4 * E * 1e-3 * np.abs(gain), "rewards")
    assert not d[:2].any() and not d[n - 1:].any()


# ------------------------------------------------------------ balance loss


def check_balance(torch, n, e, k, dtype, idt, ld=0, shift=0, pad=0.2, in_place=False, seed=0, valid=True, scale=1.0):
    rng = np.random.default_rng(n + e + k + seed)
    x, _ = strided(torch, rng.standard_normal((n, e)) * scale + 0.5 * rng.standard_normal(e), dtype, e + ld, shift)
    ch = rng.integers(0, e, (n, k))
    va = rng.random(n) >= pad
    if n > 2:
        ch[1, 0], ch[2, k - 1], va[2] = -1, e, True
        if valid:
            va[0] = False
            x[0] = float("nan")  # tokens that do not count are not read
    x64 = f64(x)
    d, dbuf = (x, None) if in_place else strided(torch, np.zeros((n, e)), dtype, e + (ld + 1 if ld else 0), shift)
    counts = torch.full((e,), -5, dtype=torch.int32, device=DEV)
    stats = torch.full((3,), 9.0, device=DEV)
    ws = poisoned(torch, M.balance_loss_workspace_bytes(n, e))
    M.balance_loss(x, vec(torch, ch, idt), counts, stats, d, ws,
                   valid=torch.from_numpy(va).to(DEV) if valid else None, coef=0.3, z_coef=0.02)
    with np.errstate(invalid="ignore"):
        wc, wst, wd = T.balance_loss(x64, ch, va if valid else None, 0.3, 0.02)
    assert counts.cpu().numpy().tolist() == wc.tolist()
    live = va if valid else np.ones(n, bool)
    tt = max(1, int(live.sum()))
    f = wc / (tt * k)
    xc = np.where(live[:, None], x64, 0.0)
    if n:
        p, dd, tol = row_tol(xc, np.zeros(n, int))
        lse = np.abs(T.log_softmax(xc)[1])
        mf = p @ f
        # each product of p carries (2|d| + 8) e + t, and f, the mean of f and lse their own rounding
        rel = (2 * dd + 8) * E + tol[:, None]
        body = 0.3 * e / tt * (f + mf[:, None]) + 0.04 / tt * lse[:, None]
        within(f64(d), wd, np.where(live[:, None], p * body * (2 * rel + 8 * E) + p * 0.04 / tt * tol[:, None]
                                    + 1.01 * HALF[dtype] * np.abs(wd), 0.0), "dlogits")
        bt = e * (mf * (tol + 8 * E))[live].sum() / tt
        zt = (2 * lse * (tol + 4 * E * (1 + lse)))[live].sum() / tt
        within(f64(stats), wst, np.array([0.3 * bt + 0.02 * zt, bt, zt]) + 4 * E * np.abs(wst), "stats")
        if dbuf is not None:
            assert around_untouched(torch, d, dbuf)
    else:
        assert not stats.any()
    return counts, stats, d


@pytest.mark.parametrize("n,e,k", [(0, 4, 1), (1, 1, 1), (1, 3, 2), (5, 2, 1), (509, 8, 2), (63, 7, 3), (300, 64, 4), (257, 65, 1),
                                   (100, 255, 8), (1030, 256, 8), (50, 257, 2), (40, 1000, 5), (33, 1024, 8),
                                   (5000, 16, 2), (9001, 60, 6), (20000, 5, 1)])
@pytest.mark.parametrize("dtype,idt,ld,shift", LAYOUTS)
def test_balance_loss(torch, n, e, k, dtype, idt, ld, shift):
    a = check_balance(torch, n, e, k, dtype, idt, ld, shift)
    b = check_balance(torch, n, e, k, dtype, idt, ld, shift, in_place=True)
    assert all(torch.equal(p, q) for p, q in zip(a, b)), "other bits in place"


def test_balance_loss_masks(torch):
    check_balance(torch, 700, 40, 2, "fp32", "int64", valid=False)
    counts, stats, d = check_balance(torch, 2, 40, 2, "fp32", "int64", pad=2.0)  # no valid token
    assert not counts.any() and not stats.any() and not d.any()
    # experts masked with -inf and with the lowest value
    x = torch.zeros((3, 10), device=DEV)
    x[:, 7:], x[1, 2] = float("-inf"), torch.finfo(torch.float32).min
    ch = torch.zeros((3, 1), dtype=torch.int64, device=DEV)
    counts, stats = torch.empty(10, dtype=torch.int32, device=DEV), torch.empty(3, device=DEV)
    d, ws = torch.empty_like(x), poisoned(torch, M.balance_loss_workspace_bytes(3, 10))
    M.balance_loss(x, ch, counts, stats, d, ws, coef=1.0, z_coef=0.1)
    _, wst, wd = T.balance_loss(f64(x), ch.cpu().numpy(), None, 1.0, 0.1)
    within(f64(stats), wst, 100 * E * np.abs(wst), "stats")
    within(f64(d), wd, 200 * E, "dlogits")


def test_balance_gradient_against_differences(torch):
    _, _, _ = check_balance(torch, 60, 12, 2, "fp32", "int64")
    rng = np.random.default_rng(2)
    x = vec(torch, rng.standard_normal((60, 12)).astype(np.float32))
    ch = rng.integers(0, 12, (60, 2))
    counts, stats = torch.empty(12, dtype=torch.int32, device=DEV), torch.empty(3, device=DEV)
    d, ws = torch.empty_like(x), poisoned(torch, M.balance_loss_workspace_bytes(60, 12))
    M.balance_loss(x, vec(torch, ch, "int64"), counts, stats, d, ws, coef=0.3, z_coef=0.02)
    u, h = rng.standard_normal((60, 12)), 1e-4
    diff = (T.balance_loss(f64(x) + h * u, ch, None, 0.3, 0.02)[1][0]
            - T.balance_loss(f64(x) - h * u, ch, None, 0.3, 0.02)[1][0]) / (2 * h)
    assert float((f64(d) * u).sum()) == pytest.approx(diff, abs=float((np.abs(f64(d)) * np.abs(u)).sum()) * 1e-5)


# --------------------------------------------- streams, graphs, large offsets


def _all_operators(torch, seed):
    """Inputs of one call of every operator, and a function that makes the calls."""
    rng = np.random.default_rng(seed)
    n, vocab, dim, e = 700, 900, 264, 16
    ids = vec(torch, make_ids(rng, n, vocab, "zipf"), "int64")
    tab = vec(torch, rng.standard_normal((vocab, dim)).astype(np.float32), "bf16")
    x, _, t, adv, w, old, ref = policy_inputs(torch, rng, n, vocab, "bf16", "int64")
    x[1], x[3] = 0.0, 0.0
    old[1] = adv[3] = 0.0
    inp = [ids, tab, x.contiguous(), vec(torch, t, "int64"), vec(torch, adv), vec(torch, w), vec(torch, old),
           vec(torch, ref), vec(torch, rng.standard_normal((n, e)).astype(np.float32)),
           vec(torch, rng.integers(0, e, (n, 2)), "int32")]
    off = vec(torch, np.array([0, 100, 300, 450, 700]), "int64")
    sref = vec(torch, np.array([-500.0, -900.0, -700.0, -1100.0], dtype=np.float32))

    def empty(*s, dtype=torch.float32):
        return torch.empty(*s, dtype=dtype, device=DEV)
    out = [empty(n, dim, dtype=torch.bfloat16), empty(vocab, dim), empty(n), empty(n), empty(4), empty(n),
           torch.empty_like(inp[2]), empty(1), empty(4), torch.empty_like(inp[2]), empty(e, dtype=torch.int32), empty(3),
           empty(n, e)]
    ws = [poisoned(torch, b) for b in (M.embed_backward_workspace_bytes(n, vocab, dim), M.policy_loss_workspace_bytes(n),
                                       M.preference_loss_workspace_bytes(n, 2), M.balance_loss_workspace_bytes(n, e))]

    def calls(inp=inp, out=out, ws=ws, stream=None):
        M.embed_forward(inp[1], inp[0], out[0], scale=2.0, stream=stream)
        M.embed_backward(inp[0], out[0], out[1], True, ws[0], scale=2.0, stream=stream)
        M.token_logprob(inp[2], inp[3], out[2], out[3], stream=stream)
        M.policy_loss(inp[2], inp[3], inp[4], inp[5], out[4], out[5], out[6], ws[1], old_logp=inp[6], ref_logp=inp[7],
                      kl_coef=0.1, stream=stream)
        M.preference_loss(inp[2], inp[3], off, sref, out[7], out[8], out[9], ws[2], stream=stream)
        M.balance_loss(inp[8], inp[9], out[10], out[11], out[12], ws[3], z_coef=0.001, stream=stream)
    return inp, out, ws, calls


def test_operators_on_another_stream_and_in_a_graph(torch):
    inp, out, ws, calls = _all_operators(torch, 0)
    calls()
    torch.cuda.synchronize()
    eager = [o.clone() for o in out]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out2 = [torch.empty_like(o) for o in out]
    torch.cuda.synchronize()
    calls(out=out2, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out2, eager))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls(out=out2)
    for k in range(1, 4):
        new = _all_operators(torch, k)[0]
        for a, b in zip(inp, new):
            a.copy_(b)
        for w in ws:
            w.fill_(0xA5 + k)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        calls()  # eager, on the same inputs and other outputs
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out2, out)), f"replay {k}"
    graph.reset()


def test_offsets_beyond_32_bits(torch):
    # matrices whose far rows lie more than 2^31 elements in: a stride, not the row count, makes them far
    rng = np.random.default_rng(3)
    ld, rows, v = (1 << 30) + 8, 4, 37
    big = torch.empty(((rows - 1) * ld + v + 3,), dtype=torch.bfloat16, device=DEV)
    x = torch.as_strided(big, (rows, v), (ld, 1), 3)
    vals = rng.standard_normal((rows, v))
    x.copy_(torch.from_numpy(vals).to(DEV))
    t = rng.integers(0, v, rows)
    logp = torch.empty(rows, device=DEV)
    M.token_logprob(x, vec(torch, t, "int64"), logp)
    want, _ = T.token_logprob(f64(x), t)
    within(f64(logp), want, 200 * E * (1 + np.abs(want)), "logp")
    d = torch.empty((rows, v), dtype=torch.bfloat16, device=DEV)
    stats, lp = torch.empty(4, device=DEV), torch.empty(rows, device=DEV)
    adv, w = torch.ones(rows, device=DEV), torch.ones(rows, device=DEV)
    ws = poisoned(torch, M.policy_loss_workspace_bytes(rows))
    M.policy_loss(x, vec(torch, t, "int64"), adv, w, stats, lp, d, ws)
    near = x.contiguous()
    d2 = torch.empty_like(d)
    M.policy_loss(near, vec(torch, t, "int64"), adv, w, stats, lp, d2, ws)
    assert torch.equal(d, d2)
    M.policy_loss(x, vec(torch, t, "int64"), adv, w, stats, lp, x, ws)  # far writes
    assert torch.equal(x.contiguous(), d2)
    # far rows of the table and of its output
    ids = vec(torch, np.array([3, 0, 3, 1]), "int64")
    out = torch.empty((4, v), dtype=torch.bfloat16, device=DEV)
    M.embed_forward(x, ids, out)
    assert torch.equal(out, d2[ids])
    M.embed_forward(out.clone(), vec(torch, np.array([3, 2, 1, 0]), "int64"), x)
    assert torch.equal(x.contiguous(), out.flip(0))
    # the far rows of dout, and of an fp32 accumulator of as many bytes
    acc = torch.zeros((5, v), device=DEV)
    need = M.embed_backward_workspace_bytes(4, 5, v)
    M.embed_backward(ids, x, acc, True, poisoned(torch, need))
    acc2 = torch.zeros((5, v), device=DEV)
    M.embed_backward(ids, x.contiguous(), acc2, True, poisoned(torch, need))
    assert torch.equal(acc, acc2)
