"""The operators around the step without a GPU: the fp64 definitions against
differences and against themselves on small hand cases, and every refusal of
the C entry points and of the tensor checks (nothing reaches a device)."""

from __future__ import annotations

import ctypes as C

import numpy as np
import pytest

import muon_newton_schulz_step_amd as M
import oracle.train_ops as T
from muon_newton_schulz_step_amd import _lib

BASE = 1 << 40
WS = BASE + (1 << 36)
BIG = 1 << 34


# ------------------------------------------------- the definitions themselves


def _directional(loss, x, seed, h=1e-5):
    u = np.random.default_rng(seed).standard_normal(x.shape)
    return u, (loss(x + h * u) - loss(x - h * u)) / (2 * h)


@pytest.mark.parametrize("old,ref", [(True, True), (False, True), (True, False), (False, False)])
def test_policy_definition_against_differences(old, ref):
    rng = np.random.default_rng(1)
    x, t = rng.standard_normal((9, 13)) * 2, rng.integers(0, 13, 9)
    t[3], w = -100, rng.random(9)
    w[5] = 0.0
    logp, _ = T.token_logprob(x, t)
    adv, lr = rng.standard_normal(9), rng.standard_normal(9) * 0.4
    kw = dict(clip_low=0.2, clip_high=0.3, kl_coef=0.1, ref_logp=logp + 0.3 * rng.standard_normal(9) if ref else None)
    full = dict(kw, old_logp=logp - lr if old else None)
    # without old_logp the loss's ratio is 1 by value; its gradient is that of exp(logp - stop(logp))
    frozen = dict(kw, old_logp=full["old_logp"] if old else logp)
    u, d = _directional(lambda y: T.policy_loss(y, t, adv, w, **frozen)[0][0], x, 2)
    assert (T.policy_loss(x, t, adv, w, **full)[2] * u).sum() == pytest.approx(d, rel=1e-7, abs=1e-9)


def test_policy_definition_by_hand():
    # two tokens of probability 1/2: ratio 2 against old logp log(1/4), clipped at 1.2 for a > 0 only
    x, t = np.zeros((2, 2)), np.array([0, 1])
    old = np.log([0.25, 0.25])
    stats, logp, d, dl = T.policy_loss(x, t, np.array([1.0, -1.0]), np.ones(2), old_logp=old)
    assert logp == pytest.approx(np.log([0.5, 0.5]))
    assert stats == pytest.approx([-1.2 + 2.0, -1.2 + 2.0, 0.0, 1.0])
    assert dl == pytest.approx([0.0, 2.0]) and d == pytest.approx(np.array([[0, 0], [-1.0, 1.0]]))


def test_policy_definition_of_an_infinite_kl():
    x = np.zeros((1, 4))
    x[0, 1] = -np.inf
    lp = np.full(1, -np.log(4))
    with np.errstate(over="ignore"):
        stats, _, _, _ = T.policy_loss(x, np.array([1]), np.ones(1), np.ones(1), lp, lp, kl_coef=0.1)
    assert stats[0] == np.inf and stats[2] == np.inf and stats[1] == 0.0


def test_policy_definition_with_a_reference_but_no_kl():
    x = np.zeros((2, 4))
    x[1, 1] = -np.inf
    lp = np.full(2, -np.log(4))
    stats, logp, d, dl = T.policy_loss(x, np.array([0, 1]), np.ones(2), np.ones(2), lp, lp, kl_coef=0.0)
    assert stats[:2] == pytest.approx([-1.0, -1.0]) and dl == pytest.approx([-1.0, 0.0]) and not d[1].any()


def test_policy_definition_without_advantage_at_an_infinite_ratio():
    with np.errstate(over="ignore"):
        stats, _, d, _ = T.policy_loss(np.zeros((2, 4)), np.array([0, 1]), np.zeros(2), np.ones(2), np.array([-np.inf, -2000.0]))
    assert not stats.any() and not d.any()


def test_policy_definition_of_nan_without_old_logp():
    x = np.zeros((2, 4))
    x[1, 2] = np.nan
    stats, logp, _, _ = T.policy_loss(x, np.array([0, 1]), np.ones(2), np.ones(2))
    assert np.isnan(logp[1]) and np.isnan(stats[0]) and np.isnan(stats[1]) and not np.isnan(logp[0])


def test_preference_definition_against_differences_and_by_hand():
    rng = np.random.default_rng(3)
    x, t = rng.standard_normal((12, 7)), rng.integers(0, 7, 12)
    t[[0, 6]] = -100
    off = np.array([1, 4, 4, 9, 11])  # an empty sequence, rows of none
    ref = rng.standard_normal(4)
    for s in (0.0, 0.1):
        u, d = _directional(lambda y: T.preference_loss(y, t, off, ref, 0.5, s)[0], x, 4)
        loss, rew, g, _ = T.preference_loss(x, t, off, ref, 0.5, s)
        assert (g * u).sum() == pytest.approx(d, rel=1e-7, abs=1e-9)
        assert not g[0].any() and not g[11].any() and not g[6].any()
    # equal gains: log 2, and half of beta on each side
    loss, rew, g, dl = T.preference_loss(np.zeros((2, 2)), np.array([0, 1]), np.array([0, 1, 2]), np.zeros(2), 0.3)
    assert loss == pytest.approx(np.log(2)) and dl == pytest.approx([-0.15, 0.15])


@pytest.mark.parametrize("margin", [1.0, 20.0, 40.0, 80.0])
def test_preference_definition_at_large_margins(margin):
    # d log(1 + exp(-m)) / d m = -exp(-m) / (1 + exp(-m)) to full accuracy, however small
    _, _, _, dl = T.preference_loss(np.zeros((2, 4)), np.array([0, 1]), np.array([0, 1, 2]), np.array([-margin, 0.0]), 1.0)
    want = np.exp(-margin) / (1.0 + np.exp(-margin))
    assert dl == pytest.approx([-want, want], rel=1e-13)


@pytest.mark.parametrize("smooth", [0.0, 1.0])
def test_preference_definition_at_an_infinite_margin(smooth):
    # the sequence that should lose has probability 0: loss and gradient 0, whatever the other label would cost
    x = np.zeros((2, 4))
    x[int(smooth == 0.0), 1] = -np.inf
    loss, rew, d, _ = T.preference_loss(x, np.array([1, 1]), np.array([0, 1, 2]), np.zeros(2), 0.5, smooth)
    assert loss == 0.0 and not d.any() and rew[int(smooth == 0.0)] == -np.inf


def test_preference_definition_of_beta_zero():
    x = np.zeros((2, 4))
    x[1, 1] = -np.inf
    loss, rew, d, _ = T.preference_loss(x, np.array([1, 1]), np.array([0, 1, 2]), np.zeros(2), 0.0, 0.1)
    assert loss == pytest.approx(np.log(2)) and not rew.any() and not d.any()


def test_balance_definition_against_differences_and_by_hand():
    rng = np.random.default_rng(5)
    x, ch = rng.standard_normal((11, 5)), rng.integers(0, 5, (11, 2))
    ch[4, 1] = -1
    valid = rng.random(11) < 0.8
    u, d = _directional(lambda y: T.balance_loss(y, ch, valid, 0.7, 0.2)[1][0], x, 6)
    counts, stats, g = T.balance_loss(x, ch, valid, 0.7, 0.2)
    assert (g * u).sum() == pytest.approx(d, rel=1e-7, abs=1e-9)
    # uniform probabilities and even counts: balance 1, z log(E)^2, no gradient from the balance term
    counts, stats, g = T.balance_loss(np.zeros((4, 4)), np.arange(4)[:, None], None, 1.0, 0.0)
    assert list(counts) == [1, 1, 1, 1] and stats == pytest.approx([1.0, 1.0, np.log(4) ** 2]) and not g.any()


def test_embedding_definition_is_its_own_transpose():
    rng = np.random.default_rng(7)
    tab, ids, g = rng.standard_normal((6, 3)), np.array([0, 5, 5, -1, 6, 2]), rng.standard_normal((6, 3))
    out = T.embed_forward(tab, ids, 1.5)
    assert (out * g).sum() == pytest.approx((tab * T.embed_backward(ids, g, 6, 1.5)).sum())
    assert not out[3].any() and not out[4].any()


# --------------------------------------------------- refusals of the C entries


def _expect(name, status, *args, text=""):
    st = getattr(_lib.load(), name)(*args)
    assert _lib.STATUS[st] == status, (name, _lib.STATUS[st], M.muon_last_error())
    assert M.muon_last_error().startswith(name)
    assert text in M.muon_last_error()


def _x(**kw):
    a = dict(logits=BASE, targets=BASE + BIG, rows=4, vocab=100, ld=100, dtype=0, target_type=1)
    a.update(kw)
    return _lib.muon_logits(**a)


def test_embed_forward_refusals():
    def call(status, **kw):
        a = dict(table=BASE, vocab=10, dim=8, tld=8, dt=0, ids=BASE + BIG, it=0, n=5, scale=1.0, out=BASE + 2 * BIG,
                 old=8, s=None)
        a.update(kw)
        _expect("muon_embed_forward", status, *a.values())
    for bad in (dict(table=None), dict(ids=None), dict(out=None), dict(vocab=0), dict(dim=0), dict(n=-1), dict(tld=7),
                dict(old=7), dict(dt=2), dict(it=2), dict(dt=-1), dict(scale=float("nan")), dict(scale=float("inf"))):
        call("MUON_ERR_INVALID_ARG", **bad)
    for bad in (dict(n=1 << 31), dict(vocab=1 << 31), dict(dim=1 << 31, tld=1 << 31, old=1 << 31), dict(tld=1 << 60),
                dict(old=1 << 60)):
        call("MUON_ERR_UNSUPPORTED", **bad)
    for bad in (dict(out=BASE + 4), dict(out=BASE + 10 * 8 * 4 - 4), dict(out=BASE + BIG + 16)):
        call("MUON_ERR_ALIAS", **bad)


def test_embed_backward_refusals():
    need = M.embed_backward_workspace_bytes(5, 10, 8)

    def call(status, **kw):
        a = dict(ids=BASE + BIG, it=0, n=5, dout=BASE, dt=1, dld=8, scale=1.0, acc=BASE + 2 * BIG, vocab=10, dim=8,
                 ald=8, first=1, ws=WS, wb=need, s=None)
        a.update(kw)
        _expect("muon_embed_backward", status, *a.values())
    for bad in (dict(ids=None), dict(dout=None), dict(acc=None), dict(vocab=0), dict(dim=0), dict(n=-1), dict(dld=7),
                dict(ald=7), dict(dt=9), dict(it=-1), dict(scale=float("nan"))):
        call("MUON_ERR_INVALID_ARG", **bad)
    for bad in (dict(ws=None), dict(ws=WS + 128), dict(wb=need - 1)):
        call("MUON_ERR_WORKSPACE", **bad)
    for bad in (dict(acc=BASE), dict(acc=BASE + BIG), dict(ws=BASE + 2 * BIG), dict(dout=WS)):
        call("MUON_ERR_ALIAS", **bad)
    call("MUON_ERR_UNSUPPORTED", n=1 << 31)


def test_token_logprob_refusals():
    f = "muon_token_logprob"
    out = BASE + 2 * BIG
    _expect(f, "MUON_ERR_INVALID_ARG", None, out, None, None)
    for bad in (dict(logits=None), dict(targets=None), dict(rows=-1), dict(vocab=0), dict(ld=99), dict(dtype=3),
                dict(target_type=5)):
        _expect(f, "MUON_ERR_INVALID_ARG", C.byref(_x(**bad)), out, None, None)
    _expect(f, "MUON_ERR_INVALID_ARG", C.byref(_x()), None, None, None)
    _expect(f, "MUON_ERR_UNSUPPORTED", C.byref(_x(rows=1 << 31)), out, None, None)
    _expect(f, "MUON_ERR_UNSUPPORTED", C.byref(_x(ld=1 << 60)), out, None, None)
    _expect(f, "MUON_ERR_ALIAS", C.byref(_x()), BASE + 4, None, None)
    _expect(f, "MUON_ERR_ALIAS", C.byref(_x()), out, out + 12, None)
    _expect(f, "MUON_ERR_ALIAS", C.byref(_x()), BASE + BIG + 28, None, None)


def test_policy_loss_refusals():
    need = M.policy_loss_workspace_bytes(4)

    def call(status, x=None, opt=(0.2, 0.2, 0.0), **kw):
        a = dict(x=C.byref(_x(**(x or {}))), adv=BASE + 2 * BIG, w=BASE + 3 * BIG, old=None, ref=None,
                 opt=C.byref(_lib.muon_policy_options(*opt)) if opt else None, stats=BASE + 4 * BIG,
                 logp=BASE + 5 * BIG, d=BASE + 6 * BIG, dld=100, ws=WS * 2, wb=need, s=None)
        a.update(kw)
        _expect("muon_policy_loss", status, *a.values())
    for bad in (dict(adv=None), dict(w=None), dict(opt=None), dict(stats=None), dict(logp=None), dict(d=None),
                dict(dld=99), dict(opt=(-0.1, 0.2, 0.0)), dict(opt=(0.2, float("nan"), 0.0)),
                dict(opt=(0.2, 0.2, float("inf"))), dict(x=dict(vocab=0)), dict(x=dict(dtype=7))):
        call("MUON_ERR_INVALID_ARG", **bad)
    for bad in (dict(ws=None), dict(ws=WS * 2 + 8), dict(wb=need - 1)):
        call("MUON_ERR_WORKSPACE", **bad)
    # shifted or differently strided over the logits; outputs on inputs and on each other
    for bad in (dict(d=BASE + 4), dict(d=BASE, dld=101), dict(stats=BASE + 2 * BIG), dict(logp=BASE + 4 * BIG + 8),
                dict(ws=BASE), dict(old=BASE + 5 * BIG), dict(ref=BASE + 6 * BIG + 4)):
        call("MUON_ERR_ALIAS", **bad)
    call("MUON_ERR_UNSUPPORTED", dld=1 << 60)


def test_preference_loss_refusals():
    need = M.preference_loss_workspace_bytes(4, 2)

    def call(status, x=None, opt=(0.1, 0.0), **kw):
        a = dict(x=C.byref(_x(**(x or {}))), off=BASE + 2 * BIG, ot=1, pairs=2, ref=BASE + 3 * BIG,
                 opt=C.byref(_lib.muon_preference_options(*opt)) if opt else None, loss=BASE + 4 * BIG,
                 rew=BASE + 5 * BIG, d=BASE + 6 * BIG, dld=100, ws=WS * 2, wb=need, s=None)
        a.update(kw)
        _expect("muon_preference_loss", status, *a.values())
    for bad in (dict(off=None), dict(ref=None), dict(loss=None), dict(rew=None), dict(d=None), dict(pairs=0),
                dict(ot=3), dict(opt=None), dict(opt=(float("inf"), 0.0)), dict(opt=(0.1, -0.1)), dict(opt=(0.1, 1.1)),
                dict(opt=(0.1, float("nan"))), dict(dld=99), dict(x=dict(logits=None))):
        call("MUON_ERR_INVALID_ARG", **bad)
    call("MUON_ERR_WORKSPACE", wb=need - 1)
    for bad in (dict(rew=BASE + 3 * BIG + 12), dict(loss=BASE + 2 * BIG + 32), dict(d=BASE + 8)):
        call("MUON_ERR_ALIAS", **bad)
    call("MUON_ERR_UNSUPPORTED", pairs=1 << 30)


def test_balance_loss_refusals():
    need = M.balance_loss_workspace_bytes(4, 8)

    def call(status, opt=(0.1, 0.0), **kw):
        a = dict(x=BASE, n=4, e=8, ld=8, dt=0, ch=BASE + BIG, ct=0, k=2, valid=None,
                 opt=C.byref(_lib.muon_balance_options(*opt)) if opt else None, counts=BASE + 2 * BIG,
                 stats=BASE + 3 * BIG, d=BASE + 4 * BIG, dld=8, ws=WS, wb=need, s=None)
        a.update(kw)
        _expect("muon_balance_loss", status, *a.values())
    for bad in (dict(x=None), dict(ch=None), dict(counts=None), dict(stats=None), dict(d=None), dict(n=-1), dict(e=0),
                dict(k=0), dict(ld=7), dict(dld=7), dict(dt=4), dict(ct=4), dict(opt=None), dict(opt=(float("nan"), 0.0)),
                dict(opt=(0.0, float("inf")))):
        call("MUON_ERR_INVALID_ARG", **bad)
    for bad in (dict(e=1025, ld=1025, dld=1025), dict(n=1 << 31), dict(n=1 << 30, k=2), dict(ld=1 << 60)):
        call("MUON_ERR_UNSUPPORTED", **bad)
    for bad in (dict(ws=None), dict(ws=WS + 1), dict(wb=need - 1)):
        call("MUON_ERR_WORKSPACE", **bad)
    for bad in (dict(d=BASE + 32), dict(d=BASE, dld=9), dict(counts=BASE + BIG + 4), dict(valid=BASE + 3 * BIG + 8)):
        call("MUON_ERR_ALIAS", **bad)


def test_workspace_sizes_are_checked_and_grow():
    for name, good, bad in (("embed_backward", (100, 50, 8), [(-1, 50, 8), (100, 0, 8), (100, 50, 0)]),
                            ("policy_loss", (100,), [(-1,)]), ("preference_loss", (100, 3), [(-1, 3), (100, 0)]),
                            ("balance_loss", (100, 8), [(-1, 8), (100, 0), (100, 1025)])):
        f = getattr(M, name + "_workspace_bytes")
        assert f(*good) > 0 and f(*[2 * g for g in good]) >= f(*good)
        for b in bad:
            with pytest.raises(M.MuonError):
                f(*b)
    # one element of each still has a workspace that can be handed over
    assert min(M.embed_backward_workspace_bytes(0, 1, 1), M.policy_loss_workspace_bytes(0),
               M.preference_loss_workspace_bytes(0, 1), M.balance_loss_workspace_bytes(0, 1)) > 0


# ------------------------------------------------------ tensor checks in Python


def test_tensor_checks():
    torch = pytest.importorskip("torch")
    tab, ids, out = torch.zeros(10, 8), torch.zeros(5, dtype=torch.int64), torch.zeros(5, 8)
    ws = torch.zeros(1 << 16, dtype=torch.uint8)
    x, t = torch.zeros(4, 6), torch.zeros(4, dtype=torch.int64)
    v4 = torch.zeros(4)

    def refuse(match, f, *a, **k):
        with pytest.raises(ValueError, match=match):
            f(*a, **k)
    refuse("table: dtype", M.embed_forward, tab.double(), ids, out)
    refuse("table: 1 dim", M.embed_forward, tab[0], ids, out)
    refuse("table: .*not adjacent", M.embed_forward, torch.zeros(8, 10).t(), ids, out)
    refuse("table: a host tensor", M.embed_forward, tab, ids, out)
    refuse("ids: a host tensor", M.embed_backward, ids, out, tab, True, ws)
    refuse("ids: dtype", M.embed_backward, ids.short(), out, tab, True, ws)
    refuse("logits: dtype", M.token_logprob, x.half(), t, v4)
    refuse("logits: row stride", M.token_logprob, torch.zeros(1, 6).expand(4, 6), t, v4)
    refuse("logits: a host", M.policy_loss, x, t, v4, v4, v4, v4, x.clone(), ws)
    refuse("logits: a host", M.preference_loss, x, t, torch.zeros(3, dtype=torch.int64), torch.zeros(2), torch.zeros(1),
           torch.zeros(2), x.clone(), ws)
    refuse("logits: a host", M.balance_loss, x, torch.zeros(4, 2, dtype=torch.int64),
           torch.zeros(6, dtype=torch.int32), torch.zeros(3), x.clone(), ws)


def test_a_matrix_counts_with_what_lies_between_its_rows():
    # two column ranges of one allocation: the second is refused as an output, its rows lie between the first's
    _expect("muon_embed_forward", "MUON_ERR_ALIAS", BASE, 10, 8, 16, 0, BASE + BIG, 0, 5, 1.0, BASE + 8 * 4, 16, None,
            text="out and table")
    _expect("muon_balance_loss", "MUON_ERR_ALIAS", BASE, 4, 8, 16, 0, BASE + BIG, 0, 2, None,
            C.byref(_lib.muon_balance_options(0.1, 0.0)), BASE + 2 * BIG, BASE + 3 * BIG, BASE + 32, 16, WS,
            M.balance_loss_workspace_bytes(4, 8), None, text="dlogits and logits")
