"""The product with a weight matrix, or with one a group of rows, and its gradients on the GPU, against the fp64
definitions (oracle/layer_ops.py) on the same bits.

Small whole numbers have exact sums in fp32, so with them every element of every size, layout and grouping has to be
the definition's, rounded to the output's type.  With others (e = 2^-24, h = half a step of the output's type):
  sums        (K + 4) e of the sum of magnitudes
  activation  of v off by d: |slope| <= 1.2 times d; and its own arithmetic: exponentials carry (|arg| + 4) e, the
              bf16 forms a quotient of 2^-22 of itself, or 2^-23 (1.5e-7 / 2 and a rounding) of v for gelu's cdf;
              over |v| <= 12: (|v| + 1) 40 e in all
  result      h of itself
"""

from __future__ import annotations

import numpy as np
import pytest

import muon_newton_schulz_step_amd as M
import oracle.layer_ops as L
from test_gpu_train_ops import DEV, E, HALF, around_untouched, dt, f64, poisoned, strided, torch, vec, within  # noqa: F401

pytestmark = pytest.mark.gpu
ACTS = ("none", "relu", "silu", "gelu", "gelu_tanh")


def rounded(torch, a, dtype):
    return torch.from_numpy(np.ascontiguousarray(a)).to(dt(torch, dtype)).double().numpy()


def matrices(torch, w, dtype, layout, ld=0, shift=0, gap=0):
    """Weights (groups x in x out) on the device in either layout, with row stride + ld and `gap` between groups."""
    g, a, b = w.shape
    r, c = (a, b) if layout == "in_out" else (b, a)
    stride = r * (c + ld) + gap
    buf = torch.full((shift + g * stride + 8,), 7.0, dtype=dt(torch, dtype), device=DEV)
    v = torch.as_strided(buf, (g, r, c), (stride, c + ld, 1), shift)
    v = v if layout == "in_out" else v.transpose(1, 2)
    v.copy_(torch.from_numpy(np.ascontiguousarray(w)).to(DEV))
    return v, buf


def split_rows(rng, rows, groups, kind):
    """Offsets: uneven, with empty groups, rows before the first and behind the last."""
    if kind == "empty":
        return np.full(groups + 1, rows // 2)
    cuts = np.sort(rng.integers(0, rows + 1, groups + 1))
    if kind == "full":
        cuts[0], cuts[-1] = 0, rows
    return cuts


def check_linear(torch, rows, a, b, dtype, layout, groups=None, kind="any", bias=True, act="none", pre=False, res=True, ld=0, shift=0,
                 first=True, seed=0, whole=True, idt="int32"):
    rng = np.random.default_rng(seed + rows + a + b)

    def draw(*shape):
        return rng.integers(-3, 4, shape).astype(np.float64) if whole else rng.standard_normal(shape)
    n = groups or 1
    off = split_rows(rng, rows, n, kind) if groups else None
    offd = vec(torch, off, idt) if groups else None
    x, _ = strided(torch, draw(rows, a), dtype, a + ld, shift)
    w, _ = matrices(torch, draw(n, a, b) * (1.0 if whole else a ** -0.5), dtype, layout, ld, shift, 3 * ld)
    bv = vec(torch, draw(n, b), dtype) if bias else None
    r, _ = strided(torch, draw(rows, b), dtype, b + ld, 2 * shift)
    out, obuf = strided(torch, np.full((rows, b), 5.0), dtype, b + ld, shift)
    p, pbuf = strided(torch, np.full((rows, b), 5.0), dtype, b + 2 * ld, shift)
    wd = w if groups else w[0]
    # poisoned workspaces: nothing of them may be read before it is written
    M.linear_forward(x, wd, out, poisoned(torch, M.linear_workspace_bytes(rows, a, b, n)),
                     bias=None if bv is None else bv if groups else bv.view(-1), activation=act, pre=p if pre else None,
                     residual=r if res else None, offsets=offd)
    wh = f64(w) if groups else f64(w)[0]
    bh, rh = (None if bv is None else f64(bv)), (f64(r) if res else None)
    held = np.full((rows, b), 5.0)
    want, wpre = L.linear_forward(f64(x), wh, bh, act, rh, off, held, held)
    sums = np.abs(f64(x))
    sums = L.linear_forward(sums, np.abs(wh), None if bh is None else np.abs(bh), offsets=off)[0] * (a + 4) * E * (0.0 if whole else 1.0)
    tol = 1.2 * sums + (0.0 if act == "none" else (np.abs(wpre) + 1) * 40 * E) + (0.0 if whole else np.abs(want) * 2 * E)
    if whole and act in ("none", "relu"):
        assert np.array_equal(f64(out), rounded(torch, want, dtype)), "out"
    else:
        within(f64(out), want, tol + np.abs(want) * HALF[dtype], "out")
    if pre and whole:
        assert np.array_equal(f64(p), rounded(torch, wpre, dtype)), "pre"
    elif pre:
        within(f64(p), wpre, sums + np.abs(wpre) * HALF[dtype], "pre")
    else:
        assert bool((p == 5).all())
    assert around_untouched(torch, out, obuf) and around_untouched(torch, p, pbuf)
    if res:
        again = r.contiguous().clone()
        M.linear_forward(x, wd, again, poisoned(torch, M.linear_workspace_bytes(rows, a, b, n)),
                         bias=None if bv is None else bv if groups else bv.view(-1), activation=act, residual=again, offsets=offd)
        inside = slice(off[0], max(off[0], off[-1])) if groups else slice(None)
        assert torch.equal(again[inside], out[inside])
    # gradient by the input
    dy, _ = strided(torch, draw(rows, b), dtype, b + ld, shift)
    z, _ = strided(torch, draw(rows, a), dtype, a + ld, shift)
    q, _ = strided(torch, draw(rows, a), dtype, a + ld, shift)
    dx, dbuf = strided(torch, np.full((rows, a), 5.0), dtype, a + 2 * ld, shift)
    M.linear_input_grad(dy, wd, dx, poisoned(torch, M.linear_workspace_bytes(rows, b, a, n)), pre=z, activation=act,
                        residual=q if res else None, offsets=offd)
    want = L.linear_input_grad(f64(dy), wh, act, f64(z), f64(q) if res else None, off, np.full((rows, a), 5.0))
    if whole and act in ("none", "relu"):
        assert np.array_equal(f64(dx), rounded(torch, want, dtype)), "dx"
    else:
        v = L.linear_input_grad(f64(dy), wh, offsets=off)
        sums = L.linear_input_grad(np.abs(f64(dy)), np.abs(wh), offsets=off) * (b + 4) * E * (0.0 if whole else 1.0)
        tol = 1.2 * sums + np.abs(v) * ((np.abs(f64(z)) + 1) * 40 + 4) * E + np.abs(want) * (HALF[dtype] + 2 * E)
        within(f64(dx), want, tol, "dx")
    assert around_untouched(torch, dx, dbuf)
    # gradients by the weights and the bias
    dw, wbuf = matrices(torch, draw(n, a, b), "fp32", layout, ld, shift, 3 * ld)
    db = vec(torch, draw(n, b)) if bias else None
    heldw, heldb = f64(dw), (f64(db) if bias else None)
    M.linear_weight_grad(x, dy, dw if groups else dw[0], first, poisoned(torch, M.linear_weight_grad_workspace_bytes(rows, a, b, n)),
                         dbias=None if db is None else db if groups else db.view(-1), offsets=offd)
    wantw, wantb = L.linear_weight_grad(f64(x), f64(dy), off)
    wantw, wantb = wantw.reshape(n, a, b), wantb.reshape(n, b)
    sizew, sizeb = L.linear_weight_grad(np.abs(f64(x)), np.abs(f64(dy)), off)
    if not first:
        wantw, wantb = wantw + heldw, wantb + (heldb if bias else 0.0)
    loose = 0.0 if whole else 1.0
    within(f64(dw), wantw, loose * ((rows + 4) * E * sizew.reshape(n, a, b) + 2 * E * np.abs(wantw)), "dw")
    if bias:
        within(f64(db), wantb, loose * ((rows + 4) * E * sizeb.reshape(n, b) + 2 * E * np.abs(wantb)), "dbias")
    mask = torch.ones_like(wbuf, dtype=torch.bool)
    r_, c_ = (a, b) if layout == "in_out" else (b, a)
    torch.as_strided(mask, (n, r_, c_), (r_ * (c_ + ld) + 3 * ld, c_ + ld, 1), shift).fill_(False)
    assert bool((wbuf[mask] == 7).all())


SIZES = [(1, 1, 1), (0, 5, 3), (1, 64, 128), (7, 130, 17), (128, 128, 128), (129, 64, 136), (300, 72, 264), (33, 1000, 257), (64, 512, 8),
         (3, 4104, 40), (260, 200, 8), (700, 24, 136), (17, 8, 1032)]


@pytest.mark.parametrize("rows,a,b", SIZES)
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("layout", ["in_out", "out_in"])
@pytest.mark.parametrize("ld,shift", [(0, 0), (8, 8), (3, 1)])
def test_linear_of_whole_numbers(torch, rows, a, b, dtype, layout, ld, shift):
    check_linear(torch, rows, a, b, dtype, layout, ld=ld, shift=shift, act="relu" if ld == 8 else "none", pre=ld != 3, res=ld != 8,
                 first=ld == 0)


@pytest.mark.parametrize("rows,a,b,groups,kind", [(1, 8, 8, 1, "full"), (50, 16, 24, 7, "any"), (513, 64, 72, 4, "full"), (700, 136, 40, 70, "any"),
                                                  (300, 128, 128, 3, "empty"), (1000, 40, 264, 9, "any"), (65, 7, 5, 130, "any"), (0, 8, 8, 3, "any"),
                                                  (90, 1032, 16, 5, "full")])
@pytest.mark.parametrize("dtype,idt", [("bf16", "int32"), ("fp32", "int64")])
@pytest.mark.parametrize("layout", ["in_out", "out_in"])
@pytest.mark.parametrize("ld,shift", [(0, 0), (3, 1)])
def test_linear_of_groups(torch, rows, a, b, groups, kind, dtype, idt, layout, ld, shift):
    check_linear(torch, rows, a, b, dtype, layout, groups, kind, ld=ld, shift=shift, act="relu" if ld else "none", pre=True, first=ld == 0,
                 idt=idt)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("rows,a,b,groups", [(130, 96, 136, None), (200, 80, 33, 3)])
def test_linear_activations(torch, act, dtype, rows, a, b, groups):
    check_linear(torch, rows, a, b, dtype, "in_out", groups, act=act, pre=True, whole=False)


@pytest.mark.parametrize("rows,a,b,layout", [(1, 2048, 512, "in_out"), (5, 4096, 1000, "out_in"), (40, 1536, 130, "in_out"), (2000, 24, 40, "out_in")])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_linear_in_parts(torch, rows, a, b, layout, dtype):
    # few tiles, long sums: cut along K, the parts' sums joined
    check_linear(torch, rows, a, b, dtype, layout, act="silu", pre=True, whole=False)
    check_linear(torch, rows, a, b, dtype, layout, act="relu", pre=True, first=False)
    check_linear(torch, rows, a, b, dtype, layout, groups=3, act="relu", pre=True, first=False)


@pytest.mark.parametrize("act", ACTS[1:])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_activations_over_their_range(torch, act, dtype):
    # forwards by a product with 1, backwards by the elementwise call; e of the argument moves an exponential by |arg| e
    v = np.concatenate([np.linspace(-12, 12, 4001), np.geomspace(1e-6, 60, 500), -np.geomspace(1e-6, 60, 500), [0.0]])
    x = torch.from_numpy(v).to(dt(torch, dtype)).to(DEV)[:, None].contiguous()
    out, pre = torch.empty_like(x), torch.empty_like(x)
    M.linear_forward(x, torch.ones(1, 1, dtype=x.dtype, device=DEV), out, poisoned(torch, M.linear_workspace_bytes(len(v), 1, 1, 1)),
                     activation=act, pre=pre)
    assert torch.equal(pre, x)
    val, slope = L.activation(act, f64(x))
    size = np.minimum(np.abs(f64(x)), 12)
    within(f64(out), val, (size + 1) * 40 * E + np.abs(val) * HALF[dtype], act)
    dx = torch.empty_like(x)
    M.activation_grad(torch.full_like(x, 2.0), x, dx, act)
    within(f64(dx), 2 * slope, (size + 1) * 80 * E + 2 * np.abs(slope) * HALF[dtype], act + "'")
    y = x.clone()
    M.activation_grad(torch.full_like(x, 2.0), y, y, act)
    assert torch.equal(y, dx)


def test_linear_of_rows_that_are_not_there(torch):
    # NaN between the rows, behind the groups and in the rows of no group reaches nothing
    for dtype, a, b in (("bf16", 136, 72), ("fp32", 20, 36), ("bf16", 21, 35)):
        x = torch.full((300, a + 8), float("nan"), dtype=dt(torch, dtype), device=DEV)
        dy = torch.full((300, b + 8), float("nan"), dtype=x.dtype, device=DEV)
        x[10:290, :a], dy[10:290, :b] = 1.0, 1.0
        w = torch.full((3, a, b + 8), float("nan"), dtype=x.dtype, device=DEV)[:, :, :b]
        w.fill_(1.0)
        off = torch.tensor([10, 10, 137, 290], dtype=torch.int32, device=DEV)
        out = torch.full((300, b), 7.0, dtype=x.dtype, device=DEV)
        M.linear_forward(x[:, :a], w, out, poisoned(torch, M.linear_workspace_bytes(300, a, b, 3)), offsets=off)
        assert bool((out[10:290] == a).all()) and bool((out[:10] == 7).all()) and bool((out[290:] == 7).all())
        dx = torch.full((300, a), 7.0, dtype=x.dtype, device=DEV)
        M.linear_input_grad(dy[:, :b], w, dx, poisoned(torch, M.linear_workspace_bytes(300, b, a, 3)), offsets=off)
        assert bool((dx[10:290] == b).all()) and bool((dx[:10] == 7).all()) and bool((dx[290:] == 7).all())
        dw, db = torch.full((3, a, b), 7.0, device=DEV), torch.full((3, b), 7.0, device=DEV)
        M.linear_weight_grad(x[:, :a], dy[:, :b], dw, True, poisoned(torch, M.linear_weight_grad_workspace_bytes(300, a, b, 3)), dbias=db,
                             offsets=off)
        for g, n in enumerate((0, 127, 153)):
            assert bool((dw[g] == n).all()) and bool((db[g] == n).all())


def test_linear_offsets_are_cut_off(torch):
    x, w = torch.ones(50, 16, device=DEV), torch.ones(3, 16, 24, device=DEV)
    off = torch.tensor([-7, 20, 1 << 40, 1 << 41], dtype=torch.int64, device=DEV)
    out, dw = torch.full((50, 24), 7.0, device=DEV), torch.empty(3, 16, 24, device=DEV)
    M.linear_forward(x, w, out, poisoned(torch, M.linear_workspace_bytes(50, 16, 24, 3)), offsets=off)
    assert bool((out == 16).all())
    M.linear_weight_grad(x, torch.ones(50, 24, device=DEV), dw, True, poisoned(torch, M.linear_weight_grad_workspace_bytes(50, 16, 24, 3)),
                         offsets=off)
    assert [float(d.mean()) for d in dw] == [20.0, 30.0, 0.0]


def test_linear_gradients_against_differences(torch):
    rng = np.random.default_rng(1)
    rows, a, m, b = 40, 24, 56, 16
    x, w1, w2, b1, up = (rng.standard_normal(s) for s in ((rows, a), (a, m), (m, b), (m,), (rows, b)))

    def loss(dx=0.0, dw1=0.0, db1=0.0, dw2=0.0):
        z = L.activation("gelu", (x + dx) @ (w1 + dw1) / 4 + b1 + db1)[0]
        return float((up * (z @ (w2 + dw2) / 4)).sum())
    d = [vec(torch, t.astype(np.float32)) for t in (x, w1 / 4, w2 / 4, b1, up)]
    pre, z, dpre, dx = (torch.empty(rows, c, device=DEV) for c in (m, m, m, a))
    out = torch.empty(rows, b, device=DEV)

    def ws(f, *s):
        return poisoned(torch, f(*s))
    M.linear_forward(d[0], d[1], z, ws(M.linear_workspace_bytes, rows, a, m, 1), bias=d[3], activation="gelu", pre=pre)
    M.linear_forward(z, d[2], out, ws(M.linear_workspace_bytes, rows, m, b, 1))
    M.linear_input_grad(d[4], d[2], dpre, ws(M.linear_workspace_bytes, rows, b, m, 1), pre=pre, activation="gelu")
    M.linear_input_grad(dpre, d[1], dx, ws(M.linear_workspace_bytes, rows, m, a, 1))
    dw1, dw2, db1 = torch.empty(a, m, device=DEV), torch.empty(m, b, device=DEV), torch.empty(m, device=DEV)
    M.linear_weight_grad(d[0], dpre, dw1, True, ws(M.linear_weight_grad_workspace_bytes, rows, a, m, 1), dbias=db1)
    M.linear_weight_grad(z, d[4], dw2, True, ws(M.linear_weight_grad_workspace_bytes, rows, m, b, 1))
    assert float((out.double() * d[4].double()).sum()) == pytest.approx(loss(), rel=1e-4, abs=1e-3)
    for name, g, scale in (("dx", dx, 1.0), ("dw1", dw1, 0.25), ("db1", db1, 1.0), ("dw2", dw2, 0.25)):
        u = rng.standard_normal(tuple(g.shape))
        diff = (loss(**{name: 1e-5 * u}) - loss(**{name: -1e-5 * u})) / 2e-5
        assert scale * float((f64(g) * u).sum()) == pytest.approx(diff, rel=1e-4, abs=1e-3)


@pytest.mark.parametrize("layout", ["in_out", "out_in"])
@pytest.mark.parametrize("rows,a,b,groups,ld", [
    (3501, 8, 3600, None, 0), (3499, 64, 3592, None, 8), (3585, 136, 3600, None, 0), (3501, 200, 3584, None, 0),   # forwards
    (3500, 3600, 8, None, 8), (3501, 3592, 72, None, 0), (3500, 3584, 192, None, 0),                              # by the input
    (1, 3600, 3504, None, 0), (65, 3592, 3600, None, 8), (129, 3584, 3584, None, 0), (190, 3600, 3600, None, 0),    # by the weights
    (5003, 72, 2568, 5, 0), (5003, 2568, 72, 5, 8), (700, 1032, 1024, 12, 8)])
def test_linear_of_large_tiles(torch, rows, a, b, groups, ld, layout):
    check_linear(torch, rows, a, b, "bf16", layout, groups, ld=ld, shift=ld, act="relu" if ld else "none", pre=True, first=ld == 0)


@pytest.mark.parametrize("layout", ["in_out", "out_in"])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("rows,a,b,groups,ld", [(2050, 40, 2064, None, 0), (2050, 137, 2063, None, 1), (2049, 2064, 72, None, 8), (2051, 2062, 33, None, 0),
                                                (130, 2064, 2048, None, 0), (33, 2065, 2050, None, 1), (900, 504, 520, 20, 8), (900, 501, 515, 20, 0),
                                                (2100, 72, 2064, 7, 0), (2100, 2065, 40, 7, 3)])
def test_linear_of_middle_tiles(torch, rows, a, b, groups, ld, dtype, layout):
    check_linear(torch, rows, a, b, dtype, layout, groups, ld=ld, shift=ld, act="relu" if ld else "none", pre=True, first=ld == 0)


@pytest.mark.parametrize("act", ["gelu", "silu"])
def test_linear_of_large_tiles_with_activations(torch, act):
    check_linear(torch, 3501, 200, 3600, "bf16", "in_out", act=act, pre=True, whole=False)
    check_linear(torch, 3501, 3600, 136, "bf16", "out_in", act=act, pre=True, whole=False)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("rows,a,b", [(1, 1, 1), (1, 3, 1), (3, 1, 1), (1, 1, 3), (2, 2, 2), (1, 33, 67), (5, 65, 1), (130, 7, 3), (131, 197, 129), (2051, 130, 2062)])
@pytest.mark.parametrize("layout", ["in_out", "out_in"])
def test_linear_of_unaligned_rows_between_others(torch, dtype, rows, a, b, layout):
    # NaN before, between and behind the rows of every operand, at every remainder of 16 bytes, reaches nothing
    rng = np.random.default_rng(rows + a)

    def inside(values, shift):
        r, c = values.shape
        buf = torch.full((shift + (r + 1) * (c + 3) + 16,), float("nan"), dtype=dt(torch, dtype), device=DEV)
        v = torch.as_strided(buf, (r, c), (c + 3, 1), shift)
        v.copy_(torch.from_numpy(values).to(DEV))
        return v
    x, w, dy = (rng.integers(-2, 3, s).astype(np.float64) for s in ((rows, a), (a, b), (rows, b)))
    for shift in (1, 2, 3):
        xd, dyd = inside(x, shift), inside(dy, shift)
        wd = inside(w, shift) if layout == "in_out" else inside(np.ascontiguousarray(w.T), shift).t()
        out, dx, dw = (torch.empty(s, dtype=xd.dtype, device=DEV) for s in ((rows, b), (rows, a), (a, b)))
        dw = dw.float()
        ws = poisoned(torch, max(M.linear_workspace_bytes(rows, a, b, 1), M.linear_workspace_bytes(rows, b, a, 1),
                                 M.linear_weight_grad_workspace_bytes(rows, a, b, 1)))
        M.linear_forward(xd, wd, out, ws)
        M.linear_input_grad(dyd, wd, dx, ws)
        M.linear_weight_grad(xd, dyd, dw, True, ws)
        assert np.array_equal(f64(out), rounded(torch, x @ w, dtype))
        assert np.array_equal(f64(dx), rounded(torch, dy @ w.T, dtype))
        assert np.array_equal(f64(dw), x.T @ dy)


@pytest.mark.parametrize("act", ACTS[1:])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_activations_of_huge_numbers(torch, act, dtype):
    # far out every activation is v or 0 and its slope 1 or 0, also where v^2 is no longer a number of the type
    v = np.array([100.0, 1e4, 3e9, 2e19, 1e30, 3e38])
    for sign in (1, -1):
        x = torch.from_numpy(sign * v).to(dt(torch, dtype)).to(DEV)[:, None].contiguous()
        out, dx, one = torch.empty_like(x), torch.empty_like(x), torch.ones(1, 1, dtype=x.dtype, device=DEV)
        ws = poisoned(torch, M.linear_workspace_bytes(len(v), 1, 1, 1))
        M.linear_forward(x, one, out, ws, activation=act)
        M.activation_grad(torch.ones_like(x), x, dx, act)
        assert torch.equal(out, x if sign > 0 else torch.zeros_like(x))
        assert torch.equal(dx, torch.full_like(x, max(sign, 0)))
        M.linear_input_grad(torch.ones_like(x), one, dx, ws, pre=x, activation=act)
        assert torch.equal(dx, torch.full_like(x, max(sign, 0)))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("layout", ["in_out", "out_in"])
@pytest.mark.parametrize("rows", [1, 2, 3, 4, 5, 8, 9])
@pytest.mark.parametrize("a,b,groups", [(8, 8, None), (2056, 72, None), (1032, 4112, None), (136, 264, 5), (3080, 40, 70)])
def test_linear_of_few_rows(torch, rows, dtype, layout, a, b, groups):
    check_linear(torch, rows, a, b, dtype, layout, groups, kind="full" if rows % 2 else "any", pre=True, ld=8, shift=8, first=rows % 2 == 0)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("layout", ["in_out", "out_in"])
def test_linear_of_few_rows_with_activations(torch, act, dtype, layout):
    check_linear(torch, 3, 2048, 136, dtype, layout, act=act, pre=True, whole=False)
    check_linear(torch, 8, 96, 2064, dtype, layout, groups=4, act=act, pre=True, whole=False)


def test_linear_of_few_rows_beside_nan(torch):
    # a row, an expert and what lies between the rows hold NaN: other rows do not see them
    for layout in ("in_out", "out_in"):
        w, _ = matrices(torch, np.ones((3, 1096, 72)), "bf16", layout, 8, 8, 16)
        w[1].fill_(float("nan"))
        x = torch.full((6, 1104), float("nan"), dtype=torch.bfloat16, device=DEV)
        x[1:4, :1096] = 1.0
        x[5, :1096] = 1.0
        off = torch.tensor([1, 4, 4, 6], dtype=torch.int32, device=DEV)
        out = torch.full((6, 72), 7.0, dtype=torch.bfloat16, device=DEV)
        M.linear_forward(x[:, :1096], w, out, poisoned(torch, M.linear_workspace_bytes(6, 1096, 72, 3)), offsets=off)
        assert bool((out[0] == 7).all()) and bool((out[[1, 2, 3, 5]] == 1096).all()) and bool(out[4].isnan().all())
