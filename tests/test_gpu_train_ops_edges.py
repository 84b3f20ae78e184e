"""The losses at the ends of their range, on the GPU: terms whose factor is 0 beside infinities, margins of any size,
rows that hold NaN, waits that are given up.  Expected values are written out from the formulas in fp64; tolerances as in
test_gpu_train_ops.py (e = 2^-24, half a step of fp32; h = half a step of the output's type)."""

from __future__ import annotations

import ctypes as C

import numpy as np
import pytest

import muon_newton_schulz_step_amd as M
from test_gpu_train_ops import DEV, E, HALF, TINY, big_pref, dt, f64, poisoned, torch, vec, within  # noqa: F401

pytestmark = pytest.mark.gpu

INF = float("inf")


def preference(torch, x, t, ref, beta, smooth, off=None):
    """(loss, rewards, dlogits) of a call."""
    seqs = len(ref)
    off = np.arange(seqs + 1) if off is None else off
    loss, rew = torch.full((1,), 9.0, device=DEV), torch.full((seqs,), 9.0, device=DEV)
    d = torch.full_like(x, 9.0)
    M.preference_loss(x, vec(torch, np.asarray(t), "int64"), vec(torch, np.asarray(off), "int64"),
                      vec(torch, np.asarray(ref, dtype=np.float32)), loss, rew, d,
                      poisoned(torch, M.preference_loss_workspace_bytes(x.shape[0], seqs // 2)), beta=beta,
                      label_smoothing=smooth)
    return f64(loss)[0], f64(rew), f64(d)


def policy(torch, x, t, adv, old, ref, kl):
    """(stats, logp, dlogits) of a call with weights 1 and clips 0.2 and 0.28."""
    n = x.shape[0]
    stats, logp, d = torch.full((4,), 9.0, device=DEV), torch.full((n,), 9.0, device=DEV), torch.full_like(x, 9.0)
    opt = dict(old_logp=None if old is None else vec(torch, np.asarray(old, dtype=np.float32)),
               ref_logp=None if ref is None else vec(torch, np.asarray(ref, dtype=np.float32)))
    M.policy_loss(x, vec(torch, np.asarray(t), "int64"), vec(torch, np.asarray(adv, dtype=np.float32)),
                  torch.ones(n, device=DEV), stats, logp, d, poisoned(torch, M.policy_loss_workspace_bytes(n)),
                  clip_low=0.2, clip_high=0.28, kl_coef=kl, **opt)
    return f64(stats), f64(logp), f64(d)


def masked_pair(torch, dtype, side):
    """Two pairs of one-row sequences over 8 equal logits; the target of pair 0's sequence on `side` (0: chosen) is
    masked.  Rows: chosen 0, chosen 1, rejected 0, rejected 1."""
    x = torch.zeros((4, 8), dtype=dt(torch, dtype), device=DEV)
    x[2 * side, 2 * side] = -INF
    return x, [0, 1, 2, 3]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("smooth", [0.0, 1.0])
def test_preference_masked_target_without_the_other_label(torch, dtype, smooth):
    # the masked sequence has log-probability -inf, so the margin is infinite on the side whose weight is 1: that
    # pair's loss and gradient are 0, and the other label's infinite term has weight 0
    side = 1 if smooth == 0.0 else 0
    x, t = masked_pair(torch, dtype, side)
    loss, rew, d = preference(torch, x, t, [0.0] * 4, 0.5, smooth)
    within(loss, np.log(2) / 2, 100 * E, "loss")
    want = np.full(4, -0.5 * np.log(8))
    want[2 * side] = -INF
    within(rew, want, 100 * E * 0.5, "rewards")
    assert not d[0].any() and not d[2].any()
    c = 0.5 / 2 * (0.5 - (1.0 - smooth))
    for r, a in ((1, c), (3, -c)):
        g = -a / 8 * np.ones(8)
        g[r] += a
        within(d[r], g, 100 * E * abs(c) + HALF[dtype] * np.abs(g) * 1.01, "dlogits")


@pytest.mark.parametrize("side", [0, 1])
def test_preference_of_beta_zero(torch, side):
    # beta 0: margins and rewards are 0, also of a sequence of log-probability -inf
    x, t = masked_pair(torch, "fp32", side)
    loss, rew, d = preference(torch, x, t, [0.0] * 4, 0.0, 0.1)
    within(loss, np.log(2), 2 * E, "loss")
    assert not rew.any() and not d.any()
    # but NaN is not a factor's business
    x[1, 5] = float("nan")
    loss, rew, d = preference(torch, x, t, [0.0] * 4, 0.0, 0.1)
    assert np.isnan(loss) and np.isnan(rew[1]) and not rew[[0, 2, 3]].any()


def test_policy_kl_of_a_target_of_probability_zero(torch):
    # exp(d) - 1 - d at d = +inf is +inf, not inf - inf; at d = -inf likewise
    x = torch.zeros((2, 8), device=DEV)
    x[1, 4] = -INF
    lp = -np.log(8)
    for ref in ([lp, lp], [-INF, lp]):
        stats, _, _ = policy(torch, x, [0, 4], [1.0, 1.0], [lp, lp], ref, 0.1)
        assert stats[0] == INF and stats[2] == INF
        within(stats[1], -1.0, 100 * E, "policy part")


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("n,v", [(3, 8), (3, 5000), (3, 70000)])  # a wave a row, a workgroup a row, pieces (bf16)
@pytest.mark.parametrize("has_old", [True, False])
def test_policy_masked_target_with_a_reference_but_no_kl(torch, dtype, n, v, has_old):
    # kl_coef 0 with a reference to look at: the KL of a target of probability 0 is infinite and its factor 0
    x = torch.zeros((n, v), dtype=dt(torch, dtype), device=DEV)
    x[1, 4] = -INF
    lp = -np.log(v)
    adv = np.array([1.0, 2.0, -0.5])
    stats, logp, d = policy(torch, x, [0, 4, 2], adv, [lp] * n if has_old else None, [lp] * n, 0.0)
    ratio = np.array([1.0, 0.0 if has_old else 1.0, 1.0])
    tol = (v / 64 + 64) * E
    within(logp, [lp, -INF, lp], tol + 2 * E * (1 - lp) * 12, "logp")
    within(stats[:2], np.full(2, -(ratio * adv).sum()), 3.5 * (tol + 20 * E), "loss")
    for r, t in ((0, 0), (1, 4), (2, 2)):
        dl = -adv[r] * ratio[r]
        p = np.full(v, 1.0 / v)
        if r == 1:
            p = np.full(v, 1.0 / (v - 1))
            p[4] = 0.0
        g = -dl * p
        g[t] += dl
        within(d[r], g, np.abs(dl) * (p + (np.arange(v) == t)) * (2 * tol + 30 * E) + 1.01 * HALF[dtype] * np.abs(g), "dlogits")


@pytest.mark.parametrize("n,v", [(3, 8), (3, 5000), (3, 70000)])
def test_policy_without_advantage_at_an_infinite_ratio(torch, n, v):
    # a target that the old policy gave probability 0 (or far less than now): the ratio is infinite, and with
    # advantage 0 both branches are 0
    x = torch.zeros((n, v), dtype=torch.bfloat16, device=DEV)
    lp = -np.log(v)
    stats, _, d = policy(torch, x, [0, 1, 2], [0.0, 0.0, 1.0], [-INF, -2000.0, lp], None, 0.0)
    within(stats[:2], [-1.0, -1.0], (v / 64 + 90) * E, "loss")
    assert stats[2] == 0.0 and stats[3] == 0.0
    assert not d[:2].any() and d[2].any()


@pytest.mark.parametrize("v", [8, 5000, 70000])
def test_policy_nan_without_old_logp_reaches_the_loss(torch, v):
    # the ratio is 1 by value, but of a row without a log-probability there is none
    for bad, row in (("nan", 0), ("all masked", 1)):
        x = torch.zeros((2, v), dtype=torch.bfloat16, device=DEV)
        if row == 0:
            x[0, 5] = float("nan")
        else:
            x[1] = -INF
        stats, logp, d = policy(torch, x, [0, 1], [1.0, 1.0], None, None, 0.0)
        assert np.isnan(logp[row]) and np.isnan(stats[0]) and np.isnan(stats[1]), bad
        assert np.isnan(d[row]).any() and not np.isnan(d[1 - row]).any()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("smooth", [0.0, 1.0])
@pytest.mark.parametrize("margin", [3.0, 20.0, 30.0, 36.0, 40.0, 80.0])
def test_preference_gradient_at_large_margins(torch, dtype, smooth, margin):
    # sigmoid's far side is exp(-|m|) there, a normal number of either type: the coefficient keeps its relative
    # accuracy on the side that is already right, and is near -+1 on the other.  The margin comes from the reference
    # alone: the logits are equal, so gains are -log 8 - ref, whose own error (64 e of log 8, and the reference's
    # rounding) moves the coefficient by as much again.
    beta, v = 0.5, 8
    x = torch.zeros((4, v), dtype=dt(torch, dtype), device=DEV)
    ref = np.array([-margin / beta, margin / beta, 0.0, 0.0], dtype=np.float32)  # pair 0: +margin, pair 1: -margin
    loss, _, d = preference(torch, x, [0, 1, 2, 3], ref, beta, smooth)
    m = np.array([margin, -margin])
    q = np.exp(-margin) / (1.0 + np.exp(-margin))
    far = {1.0: q, -1.0: 1.0 / (1.0 + np.exp(-margin))}  # sigmoid(-m) by the margin's sign
    c = np.array([beta / 2 * (smooth * far[-s] - (1.0 - smooth) * far[s]) for s in np.sign(m)])
    rel = 2 * beta * 200 * E + 40 * E
    for r, a in ((0, c[0]), (1, c[1]), (2, -c[0]), (3, -c[1])):
        g = -a / v * np.ones(v)
        g[r] += a
        within(d[r], g, np.abs(g) * (rel + 1.01 * HALF[dtype]), f"dlogits of row {r}")
    want = np.mean([(1 - smooth) * np.logaddexp(0, -a) + smooth * np.logaddexp(0, a) for a in m])
    within(loss, want, 100 * E * (1 + want), "loss")


def test_preference_walk_gives_up_a_wait_that_does_not_end(torch):
    # with no look allowed every gradient gives up: the call ends, rows with a gradient and the loss are NaN, rewards
    # and rows without one are as ever; with one look each row is right or NaN; with the default all are right
    lens, lead, tail, v = [600, 810, 0, 900, 340, 700, 650, 450], 3, 400, 50257
    x, t, off, ref = big_pref(torch, lens, lead, tail, v, "bf16", v, 7)
    n, seqs = x.shape[0], len(lens)
    assert x.numel() * 2 > 400 << 20
    polls = C.c_int.in_dll(M.load(), "muon_preference_max_polls")

    def call(most):
        before, polls.value = polls.value, most
        try:
            loss, rew, d = torch.full((1,), 9.0, device=DEV), torch.full((seqs,), 9.0, device=DEV), torch.full_like(x, 9.0)
            M.preference_loss(x, t, off, ref, loss, rew, d, poisoned(torch, M.preference_loss_workspace_bytes(n, seqs // 2)))
            torch.cuda.synchronize()
            return loss, rew, d
        finally:
            polls.value = before
    loss, rew, d = call(polls.value)
    assert not loss.isnan().any() and not d.isnan().any()
    at = torch.arange(n, device=DEV)
    live = (t >= 0) & (at >= lead) & (at < n - tail)
    none, rew0, d0 = call(-1)
    assert none.isnan().all() and torch.equal(rew0, rew)
    assert d0[live].isnan().all() and not d0[~live].any()
    one, rew1, d1 = call(0)
    bad = d1.isnan().all(1)
    assert torch.equal(rew1, rew) and torch.equal(d1[~bad], d[~bad]) and not (bad & ~live).any()
    assert bool(one.isnan()) == bool(bad.any()) and (bad.any() or torch.equal(one, loss))
    again = call(polls.value)
    assert all(torch.equal(a, b) for a, b in zip(again, (loss, rew, d)))


def test_preference_of_more_pairs_than_a_launch_has_workgroups(torch):
    # no rows at all: every pair is empty, its margin is its references'
    pairs, v = (1 << 22) + 5, 8
    g = torch.Generator(DEV).manual_seed(3)
    ref = torch.randn(2 * pairs, generator=g, device=DEV)
    gain = -ref.double()
    m = 0.1 * (gain[:pairs] - gain[pairs:])
    want = float(torch.nn.functional.softplus(-m).mean())
    x, t = torch.empty((0, v), device=DEV), torch.empty(0, dtype=torch.int64, device=DEV)
    off = torch.zeros(2 * pairs + 1, dtype=torch.int32, device=DEV)
    loss, rew = torch.full((1,), 9.0, device=DEV), torch.full((2 * pairs,), 9.0, device=DEV)
    M.preference_loss(x, t, off, ref, loss, rew, torch.empty_like(x),
                      poisoned(torch, M.preference_loss_workspace_bytes(0, pairs)), beta=0.1)
    assert bool(((rew.double() - 0.1 * gain).abs() <= 2 * E * 0.1 * gain.abs() + TINY).all())
    within(f64(loss), [want], 2 * E * want, "loss")


@pytest.mark.parametrize("v", [2000, 6000, 70000])
def test_fp32_gradients_without_a_bias_in_the_exponent(torch, v):
    # Away from its target a gradient is dlogp exp(x - lse).  The relative error may be up to (2 |d| + 8) e an
    # element, but of either sign: fitted to d = x - max over 10^6 elements its slope is 0 within the noise, whose
    # deviation is below e (|d| + 4) / (10^3 std(d)) = 3.3e-10 (logits of deviation 4, |d| around 18; six of those
    # are 2e-9).  log2(e) rounded to fp32 alone is low by 1.3e-8 of itself, and that is the slope without its rest.
    n = 1 + 10 ** 6 // v
    g = torch.Generator(DEV).manual_seed(v)
    x = torch.empty((n, v), device=DEV).normal_(0.0, 4.0, generator=g)
    t = np.zeros(n, dtype=np.int64)
    z = x.double()
    want = torch.log_softmax(z, 1)
    shift = z - z.max(1, keepdim=True).values
    seqs = 2 * (n // 2)
    off = np.arange(seqs + 1)
    lp = want[:, 0].float()

    def slope(d, rows):
        # ratios of the elements to the first one after the target take the row's own factor (and its rounding) out
        rel = (d[:rows, 1:].double().abs().log() - want[:rows, 1:])
        s = shift[:rows, 1:]
        rel, s = rel - rel.mean(1, keepdim=True), s - s.mean(1, keepdim=True)
        keep = want[:rows, 1:] > -60.0  # away from the smallest numbers
        return float((rel * s)[keep].sum() / (s * s)[keep].sum())
    d, stats, logp = torch.empty_like(x), torch.empty(4, device=DEV), torch.empty(n, device=DEV)
    M.policy_loss(x, vec(torch, t, "int64"), torch.ones(n, device=DEV), torch.ones(n, device=DEV), stats, logp, d,
                  poisoned(torch, M.policy_loss_workspace_bytes(n)))
    assert abs(slope(d, n)) < 2e-9, "policy loss"
    loss, rew = torch.empty(1, device=DEV), torch.empty(seqs, device=DEV)
    M.preference_loss(x, vec(torch, t, "int64"), vec(torch, off, "int64"), lp[:seqs].contiguous(), loss, rew, d,
                      poisoned(torch, M.preference_loss_workspace_bytes(n, seqs // 2)), beta=1.0)
    assert abs(slope(d, seqs)) < 2e-9, "preference loss"


@pytest.mark.parametrize("n,e", [(5, 8), (3000, 8), (100, 256)])
def test_balance_of_a_valid_token_with_everything_masked(torch, n, e):
    # it has no softmax, and says so: NaN in its gradient and the sums; the same token without its mark counts nowhere
    x = torch.zeros((n, e), device=DEV)
    x[2] = -INF
    ch = torch.zeros((n, 1), dtype=torch.int64, device=DEV)
    for counted in (True, False):
        valid = torch.ones(n, dtype=torch.bool, device=DEV)
        valid[2] = counted
        counts, stats = torch.empty(e, dtype=torch.int32, device=DEV), torch.empty(3, device=DEV)
        d = torch.full_like(x, 9.0)
        M.balance_loss(x, ch, counts, stats, d, poisoned(torch, M.balance_loss_workspace_bytes(n, e)), valid=valid,
                       coef=0.1, z_coef=0.01)
        got = f64(stats)
        assert int(counts[0]) == n - 1 + counted and not counts[1:].any()
        assert not d[:2].isnan().any() and not d[3:].isnan().any()
        if counted:
            assert d[2].isnan().all() and np.isnan(got[0]) and np.isnan(got[1]) and got[2] == INF
        else:
            assert not d[2].any() and np.isfinite(got).all()
