"""The operators of a trained layer without a GPU: the fp64 definitions against differences, published vectors and
themselves on small hand cases, and every refusal of the C entry points and of the tensor checks (nothing reaches a
device)."""

from __future__ import annotations

import ctypes as C

import numpy as np
import pytest

import muon_newton_schulz_step_amd as M
import oracle.layer_ops as L
from muon_newton_schulz_step_amd import _lib
from test_train_ops_host import BASE, BIG, WS, _directional, _expect

# ------------------------------------------------- the definitions themselves


def test_philox_against_its_published_vectors():
    # the known answers that come with the generator (Salmon et al., 2011): counter, key, block
    assert L.philox((0, 0, 0, 0), (0, 0)) == [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]
    assert L.philox((0xFFFFFFFF,) * 4, (0xFFFFFFFF,) * 2) == [0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD]
    assert L.philox((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0)) == [
        0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1]


def test_dropout_definition():
    keep = L.dropout_keep(40, 50, 0.3, 7, 1, 2)
    assert abs(keep.mean() - 0.7) < 5 * np.sqrt(0.21 / 2000)
    assert np.array_equal(keep[3:9, 5:21], L.dropout_keep(6, 16, 0.3, 7, 1, 2, 3, 5))
    for other in ((8, 1, 2), (7, 2, 2), (7, 1, 3)):
        assert not np.array_equal(keep, L.dropout_keep(40, 50, 0.3, *other))
    assert L.dropout_keep(3, 9, 0.0, 1, 0, 0).all()
    x = np.ones((2, 3))
    assert L.dropout(x, x > 0, 0.5, x) == pytest.approx(3.0 * x)


def test_route_definition_by_hand():
    x = np.array([[0.0, 2.0, 1.0, -1.0]])
    c, w = L.route(x, 2, "softmax", scale=3.0)
    e = np.exp([2.0, 1.0])
    assert list(c[0]) == [1, 2] and w[0] == pytest.approx(3.0 * e / e.sum())
    # a bias moves the choice, not the weights
    s = 1.0 / (1.0 + np.exp(-x[0]))
    c, w = L.route(x, 2, "sigmoid", bias=np.array([5.0, 0.0, 0.0, 4.0]), renormalize=False)
    assert list(c[0]) == [0, 3] and w[0] == pytest.approx(s[[0, 3]])
    # of two groups the one with the larger sum of two
    x = np.array([[3.0, -9.0, 2.0, 2.0]])
    assert list(L.route(x, 1, groups=2, group_top=1)[0][0]) == [0]
    assert list(L.route(x, 1, "sigmoid", bias=x[0], groups=2, group_top=2)[0][0]) == [2]
    # masked and equal experts, tokens that are not valid
    c, w = L.route(np.array([[-np.inf, 1.0, -np.inf], [1.0, 1.0, 1.0], [0.0, 0.0, 0.0]]), 2, valid=[True, True, False])
    assert c.tolist() == [[1, -1], [0, 1], [-1, -1]] and w.tolist() == [[1.0, 0.0], [0.5, 0.5], [0.0, 0.0]]


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_route_gradient_definition_against_differences(scoring, renorm):
    rng = np.random.default_rng(1)
    x, dw = rng.standard_normal((9, 7)), rng.standard_normal((9, 3))
    c, _ = L.route(x, 3, scoring)
    c[2, 1], c[4, 2] = -1, 7
    valid = np.arange(9) != 5

    def value(z):
        s = L.scores(z, scoring)
        total = 0.0
        for r in np.flatnonzero(valid):
            live = [(j, e) for j, e in enumerate(c[r]) if 0 <= e < 7]
            w = s[r, [e for _, e in live]]
            total += ((w / w.sum() if renorm else w) * 1.5 * dw[r, [j for j, _ in live]]).sum()
        return total
    u, d = _directional(value, x, 2)
    g = L.route_backward(x, c, dw, scoring, valid, renorm, 1.5)
    assert (g * u).sum() == pytest.approx(d, rel=1e-6, abs=1e-8) and not g[5].any()


def test_order_and_combine_definitions():
    c = np.array([[2, 0], [0, -1], [2, 5], [0, 2]])
    tokens, offsets, place = L.expert_order(c, 3)
    assert offsets.tolist() == [0, 3, 3, 6]
    assert tokens.tolist() == [0, 1, 3, 0, 2, 3, -1, -1]
    assert place.tolist() == [[3, 0], [1, -1], [4, -1], [2, 5]]
    rng = np.random.default_rng(3)
    y, w, res, g = rng.standard_normal((8, 5)), rng.standard_normal((4, 2)), rng.standard_normal((4, 5)), rng.standard_normal((4, 5))
    assert L.expert_combine(y, place, w, res)[1] == pytest.approx(res[1] + w[1, 0] * y[1])
    dy, dw = L.expert_combine_backward(g, y, place, np.zeros((8, 5)), w)
    u, d = _directional(lambda v: (g * L.expert_combine(v, place, w)).sum(), y, 4)
    assert (dy * u).sum() == pytest.approx(d, rel=1e-8)
    u, d = _directional(lambda v: (g * L.expert_combine(y, place, v)).sum(), w, 5)
    assert (dw * u).sum() == pytest.approx(d, rel=1e-8)


@pytest.mark.parametrize("act", ["relu", "silu", "gelu", "gelu_tanh"])
def test_linear_definitions_against_differences(act):
    v = np.linspace(-6, 6, 241) + 0.013
    val, slope = L.activation(act, v)
    diff = (L.activation(act, v + 1e-6)[0] - L.activation(act, v - 1e-6)[0]) / 2e-6
    assert slope == pytest.approx(diff, rel=1e-6, abs=1e-8)
    assert L.activation(act, np.array([30.0]))[0] == pytest.approx(30.0) and abs(L.activation(act, np.array([-40.0]))[0]) < 1e-10
    rng = np.random.default_rng(7)
    x, w, b, g = rng.standard_normal((10, 4)), rng.standard_normal((3, 4, 6)), rng.standard_normal((3, 6)), rng.standard_normal((10, 6))
    off = np.array([1, 4, 4, 9])
    z = rng.standard_normal((10, 4))

    def loss(xx=None, ww=w, bb=b):
        out, _ = L.linear_forward(L.activation(act, z)[0] if xx is None else xx, ww, bb, offsets=off)
        return float((g * out)[1:9].sum())
    u, d = _directional(lambda t: loss(L.activation(act, t)[0]), z, 8)
    dz = L.linear_input_grad(g, w, act, z, offsets=off, dx=np.zeros((10, 4)))
    assert (dz * u).sum() == pytest.approx(d, rel=1e-6) and not dz[0].any() and not dz[9].any()
    dw, db = L.linear_weight_grad(L.activation(act, z)[0], g, off)
    u, d = _directional(lambda t: loss(ww=t), w, 9)
    assert (dw * u).sum() == pytest.approx(d, rel=1e-7) and not dw[1].any()
    u, d = _directional(lambda t: loss(bb=t), b, 10)
    assert (db * u).sum() == pytest.approx(d, rel=1e-7)


# --------------------------------------------------- refusals of the C entries


def test_dropout_refusals():
    def call(status, **kw):
        a = dict(x=BASE, rows=4, cols=8, ld=8, dt=0, p=0.1, seed=1, site=0, step=0, dev=None, res=BASE + BIG, rld=8, out=BASE + 2 * BIG,
                 old=8, s=None)
        a.update(kw)
        _expect("muon_dropout", status, *a.values())
    for bad in (dict(x=None), dict(out=None), dict(rows=-1), dict(cols=0), dict(ld=7), dict(rld=7), dict(old=7), dict(dt=2), dict(p=-0.1),
                dict(p=1.0), dict(p=1.0 - 2.0 ** -40), dict(p=float("nan")), dict(p=float("inf"))):
        call("MUON_ERR_INVALID_ARG", **bad)
    for bad in (dict(rows=1 << 31), dict(ld=1 << 60), dict(old=1 << 60), dict(rld=1 << 60),
                dict(cols=1 << 31, ld=1 << 31, rld=1 << 31, old=1 << 31), dict(rows=1 << 30, cols=1 << 20, ld=1 << 20, rld=1 << 20, old=1 << 20)):
        call("MUON_ERR_UNSUPPORTED", **bad)
    for bad in (dict(out=BASE + 4), dict(out=BASE, old=9), dict(out=BASE + BIG + 32), dict(dev=BASE + 2 * BIG + 8)):
        call("MUON_ERR_ALIAS", **bad)


def _route_opt(**kw):
    a = dict(scoring=0, renormalize=1, groups=2, keep_groups=1, group_top=1, reserved=0, scale=1.0)
    a.update(kw)
    return C.byref(_lib.muon_route_options(*a.values()))


def test_route_refusals():
    def call(status, opt=None, null=False, **kw):
        a = dict(x=BASE, n=4, e=8, ld=8, dt=0, bias=BASE + BIG, valid=BASE + 2 * BIG, opt=None if null else _route_opt(**(opt or {})),
                 ch=BASE + 3 * BIG, ct=0, k=2, w=BASE + 4 * BIG, s=None)
        a.update(kw)
        _expect("muon_route", status, *a.values())
    for bad in (dict(x=None), dict(ch=None), dict(w=None), dict(null=True), dict(n=-1), dict(e=0), dict(k=0), dict(k=9), dict(ld=7), dict(dt=5),
                dict(ct=9), dict(opt=dict(scoring=2)), dict(opt=dict(scale=float("nan"))), dict(opt=dict(groups=0)), dict(opt=dict(groups=3)),
                dict(opt=dict(keep_groups=0)), dict(opt=dict(keep_groups=3)), dict(opt=dict(group_top=0)), dict(opt=dict(group_top=3))):
        call("MUON_ERR_INVALID_ARG", **bad)
    for bad in (dict(e=1026, ld=1026), dict(e=40, ld=40, k=33), dict(n=1 << 30), dict(ld=1 << 60), dict(e=64, ld=64, opt=dict(groups=64)),
                dict(n=1 << 27, e=512, ld=512)):
        call("MUON_ERR_UNSUPPORTED", **bad)
    for bad in (dict(ch=BASE + 4), dict(w=BASE + 3 * BIG + 28), dict(w=BASE + BIG + 28), dict(ch=BASE + 2 * BIG)):
        call("MUON_ERR_ALIAS", **bad)


def test_route_backward_refusals():
    def call(status, opt=None, null=False, **kw):
        a = dict(x=BASE, n=4, e=8, ld=8, dt=0, valid=None, opt=None if null else _route_opt(**(opt or {})), ch=BASE + 3 * BIG, ct=0, k=2,
                 dw=BASE + 4 * BIG, d=BASE + 5 * BIG, dld=8, first=1, s=None)
        a.update(kw)
        _expect("muon_route_backward", status, *a.values())
    for bad in (dict(x=None), dict(ch=None), dict(dw=None), dict(d=None), dict(null=True), dict(n=-1), dict(e=0), dict(k=0), dict(ld=7),
                dict(dld=7), dict(dt=5), dict(ct=9), dict(opt=dict(scoring=-1)), dict(opt=dict(scale=float("inf")))):
        call("MUON_ERR_INVALID_ARG", **bad)
    for bad in (dict(e=1025, ld=1025, dld=1025), dict(k=33), dict(dld=1 << 60)):
        call("MUON_ERR_UNSUPPORTED", **bad)
    for bad in (dict(d=BASE), dict(d=BASE + 4 * BIG + 28), dict(valid=BASE + 5 * BIG)):
        call("MUON_ERR_ALIAS", **bad)


def test_expert_order_refusals():
    need = M.expert_order_workspace_bytes(4, 2, 8)

    def call(status, **kw):
        a = dict(ch=BASE, ct=1, n=4, k=2, e=8, tok=BASE + BIG, off=BASE + 2 * BIG, pl=BASE + 3 * BIG, ws=WS, wb=need, s=None)
        a.update(kw)
        _expect("muon_expert_order", status, *a.values())
    for bad in (dict(ch=None), dict(tok=None), dict(off=None), dict(pl=None), dict(n=-1), dict(k=0), dict(e=0), dict(ct=7)):
        call("MUON_ERR_INVALID_ARG", **bad)
    for bad in (dict(e=1025), dict(n=1 << 30), dict(n=1 << 31)):
        call("MUON_ERR_UNSUPPORTED", **bad)
    for bad in (dict(ws=None), dict(ws=WS + 64), dict(wb=need - 1)):
        call("MUON_ERR_WORKSPACE", **bad)
    for bad in (dict(tok=BASE + 8), dict(off=BASE + BIG + 28), dict(pl=BASE + 2 * BIG + 32), dict(ws=BASE)):
        call("MUON_ERR_ALIAS", **bad)


def test_expert_combine_refusals():
    def call(status, **kw):
        a = dict(y=BASE, rows=8, dim=16, yld=16, dt=0, pl=BASE + BIG, n=4, k=2, w=BASE + 2 * BIG, res=BASE + 3 * BIG, rld=16, out=BASE + 4 * BIG,
                 old=16, s=None)
        a.update(kw)
        _expect("muon_expert_combine", status, *a.values())
    for bad in (dict(y=None), dict(pl=None), dict(out=None), dict(rows=-1), dict(dim=0), dict(n=-1), dict(k=0), dict(yld=15), dict(rld=15),
                dict(old=15), dict(dt=3)):
        call("MUON_ERR_INVALID_ARG", **bad)
    for bad in (dict(rows=1 << 31), dict(n=1 << 30), dict(yld=1 << 60), dict(n=1 << 27, k=1), dict(n=1 << 25, k=1, dim=1 << 12, yld=1 << 12,
                rld=1 << 12, old=1 << 12)):
        call("MUON_ERR_UNSUPPORTED", **bad)
    for bad in (dict(out=BASE + 64), dict(out=BASE + 3 * BIG, old=17), dict(out=BASE + 2 * BIG + 16), dict(out=BASE + BIG)):
        call("MUON_ERR_ALIAS", **bad)


def test_expert_combine_backward_refusals():
    def call(status, **kw):
        a = dict(g=BASE, n=4, dim=16, gld=16, dt=0, pl=BASE + BIG, k=2, w=None, y=BASE + 2 * BIG, yld=16, rows=8, dy=BASE + 3 * BIG, dyld=16,
                 dw=BASE + 4 * BIG, s=None)
        a.update(kw)
        _expect("muon_expert_combine_backward", status, *a.values())
    for bad in (dict(g=None), dict(pl=None), dict(y=None), dict(dy=None, dw=None), dict(gld=15), dict(yld=15), dict(dyld=15), dict(k=0),
                dict(dim=0), dict(n=-1), dict(dt=-1)):
        call("MUON_ERR_INVALID_ARG", **bad)
    for bad in (dict(gld=1 << 60), dict(dyld=1 << 60), dict(yld=1 << 60)):
        call("MUON_ERR_UNSUPPORTED", **bad)
    for bad in (dict(dy=BASE), dict(dy=BASE + 2 * BIG + 64), dict(dw=BASE + 3 * BIG + 8), dict(dw=BASE + BIG)):
        call("MUON_ERR_ALIAS", **bad)


def _w(**kw):
    a = dict(w=BASE + BIG, in_=16, out=24, ld=24, stride=16 * 24, layout=0, groups=3, offsets=BASE + 2 * BIG, offset_type=0, dtype=0)
    a.update(kw)
    return C.byref(_lib.muon_weights(**a))


BAD_WEIGHTS = (dict(w=None), dict(in_=0), dict(out=0), dict(ld=23), dict(stride=16 * 24 - 1), dict(layout=2), dict(groups=0),
               dict(offsets=None), dict(offset_type=4), dict(dtype=9), dict(layout=1, ld=15))
BIG_WEIGHTS = (dict(in_=1 << 31), dict(groups=1025), dict(ld=1 << 60), dict(stride=1 << 60), dict(in_=1 << 20, out=1 << 20, ld=1 << 20, stride=1 << 40))


def test_linear_forward_refusals():
    need = M.linear_workspace_bytes(10, 16, 24, 3)

    def call(status, w=None, null=False, **kw):
        a = dict(x=BASE, rows=10, xld=16, w=None if null else _w(**(w or {})), bias=BASE + 3 * BIG, act=1, pre=BASE + 4 * BIG, pld=24,
                 res=BASE + 5 * BIG, rld=24, out=BASE + 6 * BIG, old=24, ws=2 * WS, wb=need, s=None)
        a.update(kw)
        _expect("muon_linear_forward", status, *a.values())
    for bad in (dict(x=None), dict(out=None), dict(rows=-1), dict(xld=15), dict(pld=23), dict(rld=23), dict(old=23), dict(act=5), dict(act=-1),
                dict(null=True)) + tuple(dict(w=b) for b in BAD_WEIGHTS):
        call("MUON_ERR_INVALID_ARG", **bad)
    for bad in (dict(rows=1 << 31), dict(xld=1 << 60), dict(old=1 << 60), dict(pld=1 << 60), dict(rld=1 << 60)) + tuple(dict(w=b) for b in BIG_WEIGHTS):
        call("MUON_ERR_UNSUPPORTED", **bad)
    for bad in (dict(ws=None), dict(ws=WS + 128), dict(wb=need - 1)):
        call("MUON_ERR_WORKSPACE", **bad)
    for bad in (dict(out=BASE + 64), dict(out=BASE + BIG + 3 * 16 * 24 * 4 - 4), dict(pre=BASE + 6 * BIG), dict(pre=BASE + 5 * BIG),
                dict(out=BASE + 5 * BIG, old=25), dict(out=BASE + 3 * BIG), dict(out=BASE + 2 * BIG + 12), dict(ws=BASE)):
        call("MUON_ERR_ALIAS", **bad)


def test_linear_input_grad_refusals():
    need = M.linear_workspace_bytes(10, 24, 16, 3)

    def call(status, w=None, null=False, **kw):
        a = dict(dy=BASE, rows=10, yld=24, w=None if null else _w(**(w or {})), act=2, pre=BASE + 4 * BIG, pld=16, res=BASE + 5 * BIG, rld=16,
                 dx=BASE + 6 * BIG, xld=16, ws=2 * WS, wb=need, s=None)
        a.update(kw)
        _expect("muon_linear_input_grad", status, *a.values())
    for bad in (dict(dy=None), dict(dx=None), dict(pre=None), dict(rows=-1), dict(yld=23), dict(pld=15), dict(rld=15), dict(xld=15), dict(act=5),
                dict(null=True)) + tuple(dict(w=b) for b in BAD_WEIGHTS):
        call("MUON_ERR_INVALID_ARG", **bad)
    for bad in (dict(rows=1 << 31), dict(yld=1 << 60), dict(xld=1 << 60)) + tuple(dict(w=b) for b in BIG_WEIGHTS):
        call("MUON_ERR_UNSUPPORTED", **bad)
    for bad in (dict(ws=None), dict(ws=WS + 128), dict(wb=need - 1)):
        call("MUON_ERR_WORKSPACE", **bad)
    for bad in (dict(dx=BASE), dict(dx=BASE + BIG), dict(dx=BASE + 4 * BIG), dict(dx=BASE + 5 * BIG + 16), dict(dx=BASE + 2 * BIG)):
        call("MUON_ERR_ALIAS", **bad)


def test_linear_weight_grad_refusals():
    need = M.linear_weight_grad_workspace_bytes(10, 16, 24, 3)

    def call(status, **kw):
        a = dict(x=BASE, rows=10, i=16, xld=16, dy=BASE + BIG, o=24, yld=24, dt=1, off=BASE + 2 * BIG, ot=0, g=3, dw=BASE + 3 * BIG, ld=24,
                 st=16 * 24, lay=0, db=BASE + 4 * BIG, first=1, ws=2 * WS, wb=need, s=None)
        a.update(kw)
        _expect("muon_linear_weight_grad", status, *a.values())
    for bad in (dict(x=None), dict(dy=None), dict(dw=None), dict(off=None), dict(rows=-1), dict(i=0), dict(o=0), dict(xld=15), dict(yld=23),
                dict(ld=23), dict(st=16 * 24 - 1), dict(lay=3), dict(lay=1, ld=15), dict(g=0), dict(dt=2), dict(ot=2)):
        call("MUON_ERR_INVALID_ARG", **bad)
    for bad in (dict(rows=1 << 31), dict(g=1025), dict(ld=1 << 60), dict(xld=1 << 60), dict(st=1 << 60)):
        call("MUON_ERR_UNSUPPORTED", **bad)
    for bad in (dict(ws=None), dict(ws=WS + 128), dict(wb=need - 1)):
        call("MUON_ERR_WORKSPACE", **bad)
    for bad in (dict(dw=BASE), dict(dw=BASE + BIG + 64), dict(db=BASE + 3 * BIG + 4 * (3 * 16 * 24) - 4), dict(db=BASE + 2 * BIG),
                dict(ws=BASE)):
        call("MUON_ERR_ALIAS", **bad)


def test_activation_grad_refusals():
    def call(status, **kw):
        a = dict(dy=BASE, rows=4, cols=8, yld=8, dt=0, act=3, pre=BASE + BIG, pld=8, out=BASE + 2 * BIG, old=8, s=None)
        a.update(kw)
        _expect("muon_activation_grad", status, *a.values())
    for bad in (dict(dy=None), dict(pre=None), dict(out=None), dict(rows=-1), dict(cols=0), dict(yld=7), dict(pld=7), dict(old=7), dict(dt=4),
                dict(act=9)):
        call("MUON_ERR_INVALID_ARG", **bad)
    for bad in (dict(rows=1 << 31), dict(old=1 << 60), dict(rows=1 << 30, cols=1 << 10, yld=1 << 10, pld=1 << 10, old=1 << 10)):
        call("MUON_ERR_UNSUPPORTED", **bad)
    for bad in (dict(out=BASE + 16), dict(out=BASE + BIG, old=9)):
        call("MUON_ERR_ALIAS", **bad)


def test_layer_workspace_sizes_are_checked():
    for name, good, bad in (("expert_order", (100, 2, 8), [(-1, 2, 8), (100, 0, 8), (100, 2, 0), (100, 2, 1025)]),
                            ("linear", (100, 8, 8, 1), [(-1, 8, 8, 1), (100, 0, 8, 1), (100, 8, 0, 1), (100, 8, 8, 0), (100, 8, 8, 1025)]),
                            ("linear_weight_grad", (100, 8, 8, 1), [(-1, 8, 8, 1), (100, 0, 8, 1), (100, 8, 0, 1), (100, 8, 8, 0)])):
        f = getattr(M, name + "_workspace_bytes")
        assert f(*good) > 0 and f(0, *good[1:]) > 0
        for b in bad:
            with pytest.raises(M.MuonError):
                f(*b)


# ------------------------------------------------------ tensor checks in Python


def test_layer_tensor_checks():
    torch = pytest.importorskip("torch")
    x, v = torch.zeros(4, 8), torch.zeros(8)
    ch, w2 = torch.zeros(4, 2, dtype=torch.int64), torch.zeros(4, 2)
    ws = torch.zeros(1 << 16, dtype=torch.uint8)
    w, w3, off = torch.zeros(8, 6), torch.zeros(3, 8, 6), torch.zeros(4, dtype=torch.int32)
    out = torch.zeros(4, 6)

    def refuse(match, f, *a, **k):
        with pytest.raises(ValueError, match=match):
            f(*a, **k)
    refuse("x: a host tensor", M.dropout, x, x.clone(), 0.1, 1)
    refuse("x: dtype", M.dropout, x.double(), x.clone(), 0.1, 1)
    refuse("logits: a host", M.route_experts, x, ch, w2)
    refuse("logits: .*not adjacent", M.route_experts, torch.zeros(8, 4).t(), ch, w2)
    refuse("logits: a host", M.route_backward, x, ch, w2, x.clone(), True)
    refuse("choices: shape", M.expert_order, v, v, off, v, ws)
    refuse("choices: dtype", M.expert_order, w2, v, off, v, ws)
    refuse("y: a host", M.expert_combine, x, ch.int(), x.clone())
    refuse("neither dy nor dweights", M.expert_combine_backward, x, ch.int())
    refuse("dout: a host", M.expert_combine_backward, x, ch.int(), dy=x.clone())
    refuse("w: 3 dimensions, expected 2", M.linear_forward, x, w3, out, ws)
    refuse("w: 2 dimensions, expected 3", M.linear_forward, x, w, out, ws, offsets=off)
    refuse("w: no groups", M.linear_forward, x, w3[:0], out, ws, offsets=off)
    refuse("w: a host", M.linear_forward, x, w, out, ws)
    refuse("w: a host", M.linear_input_grad, out, w.t().contiguous().t(), x, ws)
    refuse("w: .*not adjacent", M.linear_forward, x, torch.zeros(16, 12)[::2, ::2], out, ws)
    refuse("dw: dtype", M.linear_weight_grad, x, out, w.bfloat16(), True, ws)
    refuse("dw: a host", M.linear_weight_grad, x, out, w, True, ws)
    refuse("dy: a host", M.activation_grad, x, x.clone(), x.clone(), "relu")
