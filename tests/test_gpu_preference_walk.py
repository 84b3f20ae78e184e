"""The preference loss where it walks pair by pair: over several launches, with more pairs than workgroups of a
launch, with bad offsets; and which calls do.  Definitions and tolerances are those of test_gpu_train_ops.py."""

from __future__ import annotations

import ctypes as C

import numpy as np
import pytest

import muon_newton_schulz_step_amd as M
import oracle.train_ops as T
from test_gpu_train_ops import (DEV, E, TINY, around_untouched, big_pref, dt, f64, grad_tol, poisoned,  # noqa: F401
                                row_tol, strided, torch, vec, within)
from test_gpu_train_ops import test_preference_loss_in_one_walk as one_walk

pytestmark = pytest.mark.gpu


def test_preference_walk_in_several_launches(torch):
    # more rows than one launch takes, so that most gradients are written by the later ones; a target in one row of 64
    n, v, beta, smooth = (1 << 21) + 5, 3, 1e-2, 0.1
    g = torch.Generator(DEV).manual_seed(8)
    x = torch.randn(n, v, generator=g, device=DEV)
    t = torch.where(torch.rand(n, generator=g, device=DEV) < 1 / 64, torch.randint(0, v, (n,), generator=g, device=DEV), -1)
    o = [2, n // 3, n // 2, n - 70, n - 1]
    z = torch.log_softmax(x.double(), 1)
    has = t >= 0
    lp = torch.where(has, z.gather(1, t.clamp(min=0)[:, None])[:, 0], 0.0)
    sums = np.array([float(lp[a:b].sum()) for a, b in zip(o, o[1:])])
    ref = torch.tensor(np.round(sums + [40.0, -30.0, 25.0, 10.0]), device=DEV, dtype=torch.float32)
    loss, rew, d = torch.full((1,), 9.0, device=DEV), torch.full((4,), 9.0, device=DEV), torch.full_like(x, 9.0)
    M.preference_loss(x, t.int(), torch.tensor(o, device=DEV, dtype=torch.int32), ref, loss, rew, d,
                      poisoned(torch, M.preference_loss_workspace_bytes(n, 2)), beta=beta, label_smoothing=smooth)
    # three terms a row: the sum's relative error is below (2 |d| + 68) e with |d| < 16
    tol = torch.where(has, 100 * E * (1 + lp.abs()), 0.0)
    err = beta * np.array([float(tol[a:b].sum()) for a, b in zip(o, o[1:])])
    gain = sums - f64(ref)
    within(f64(rew), beta * gain, err + 4 * E * beta * np.abs(gain), "rewards")
    m, pair_tol = beta * (gain[:2] - gain[2:]), err[:2] + err[2:] + 4 * E
    want = ((1 - smooth) * np.logaddexp(0, -m) + smooth * np.logaddexp(0, m)).mean()
    within(f64(loss), [want], pair_tol.mean() + 4 * E * (1 + want), "loss")
    c = beta / 2 * (smooth / (1 + np.exp(-m)) - (1 - smooth) / (1 + np.exp(m)))
    a, dd = torch.zeros(n, dtype=torch.float64, device=DEV), torch.zeros(n, dtype=torch.float64, device=DEV)
    for s in range(4):
        a[o[s]:o[s + 1]] = c[s] if s < 2 else -c[s - 2]
        dd[o[s]:o[s + 1]] = beta / 2 / 4 * pair_tol[s % 2]
    a, dd = torch.where(has, a, 0.0)[:, None], torch.where(has, dd, 0.0)[:, None]
    one = torch.zeros_like(z).scatter_(1, t.clamp(min=0)[:, None], 1.0)
    wd = a * (one - z.exp())
    assert bool(((d.double() - wd).abs() <= 300 * E * a.abs() + dd + TINY).all())
    assert not d[~has].any() and not d[:2].any() and not d[n - 1:].any()


@pytest.mark.parametrize("dtype,idt", [("fp32", "int32"), ("bf16", "int64")])
def test_preference_of_few_rows_in_many_pairs(torch, dtype, idt):
    # as many pairs as only the walk takes, all but two of them empty; the offsets' ends lie outside the rows
    pairs, v, n, beta = (1 << 21) + 1, 40, 7, 0.5
    rng = np.random.default_rng(4)
    x, _ = strided(torch, rng.standard_normal((n, v)), dtype, v + 2, 1)
    t = rng.integers(0, v, n)
    t[3] = -1
    seqs, far = 2 * pairs, 2 ** 31 - 1 if idt == "int32" else 2 ** 40
    off = torch.full((seqs + 1,), 2, dtype=dt(torch, idt), device=DEV)
    off[0], off[pairs + 1:seqs], off[seqs] = -far, 4, far  # rows 0, 1: chosen 0; 2, 3: rejected 0; 4 to 6: the last rejected
    ref = torch.zeros(seqs, device=DEV)
    ref[0] = -4.0
    loss, rew, d = torch.full((1,), 9.0, device=DEV), torch.full((seqs,), 9.0, device=DEV), torch.full((n, v), 9.0, dtype=x.dtype, device=DEV)
    M.preference_loss(x, vec(torch, t, idt), off, ref, loss, rew, d,
                      poisoned(torch, M.preference_loss_workspace_bytes(n, pairs)), beta=beta)
    x64 = f64(x)
    lp, _ = T.token_logprob(x64, t)
    _, _, tol = row_tol(x64, t)
    gains = {0: lp[0:2].sum() + 4.0, pairs: lp[2:4].sum(), seqs - 1: lp[4:7].sum()}
    err = beta * tol.sum() + 4 * E * beta * max(abs(g) for g in gains.values())
    got = f64(rew)
    for s, g in gains.items():
        within(got[s], beta * g, err, f"reward {s}")
        got[s] = 0.0
    assert not got.any()
    m = np.array([beta * (gains[0] - gains[pairs]), -beta * gains[seqs - 1]])
    want = (np.logaddexp(0, -m).sum() + (pairs - 2) * np.log(2)) / pairs
    within(f64(loss), [want], err + 4 * E * (1 + want), "loss")
    c = -beta / pairs / (1 + np.exp(m))
    dlogp = np.array([c[0], c[0], -c[0], 0.0, -c[1], -c[1], -c[1]])
    wd = T.logit_grad(x64, t, dlogp)
    gt = grad_tol(x64, t, dlogp, np.abs(dlogp), wd, dtype)
    within(f64(d), wd, gt + 2 * err * beta / pairs * (np.exp(T.log_softmax(x64)[0]) + (np.arange(v) == t[:, None])), "dlogits")


def test_preference_walk_of_bad_offsets_touches_no_row_outside(torch):
    # decreasing and out-of-range offsets: results unspecified, but the call ends and the buffers around stay
    pairs, n = (1 << 21) + 1, 6
    rng = np.random.default_rng(9)
    x, _ = strided(torch, rng.standard_normal((n, 40)), "fp32", 44, 2)
    dl, dbuf = strided(torch, np.zeros((n, 40)), "fp32", 43, 5)
    t = vec(torch, rng.integers(0, 40, n), "int64")
    for k in range(3):
        g = torch.Generator(DEV).manual_seed(k)
        off = torch.randint(-3, 9, (2 * pairs + 1,), generator=g, device=DEV)
        if k:
            off[torch.rand(off.shape, generator=g, device=DEV) < 0.3] = 2 ** 62 if k == 1 else -2 ** 62
        loss, rew = torch.empty(1, device=DEV), torch.empty(2 * pairs, device=DEV)
        M.preference_loss(x, t, off, torch.zeros(2 * pairs, device=DEV), loss, rew, dl,
                          poisoned(torch, M.preference_loss_workspace_bytes(n, pairs)))
        torch.cuda.synchronize()
        assert around_untouched(torch, dl, dbuf)


# (a call takes the walk from 400 MB of logits on, as test_which_way pins)
@pytest.mark.parametrize("lens,lead,tail,v,dtype,ld", [
    # ragged pairs, an empty sequence and an empty pair, rows before and after them
    ([600, 0, 0, 1011, 40, 1000, 633, 0, 820, 1], 3, 650, 50257, "bf16", 50257),
    ([300, 400, 260, 10, 400, 320, 290, 350, 290, 310, 250, 300], 0, 0, 32001, "fp32", 32003)])
def test_preference_walk_of_large_logits(torch, lens, lead, tail, v, dtype, ld):
    one_walk(torch, lens, lead, tail, v, dtype, ld)


def test_preference_walk_of_large_logits_in_a_graph(torch):
    v, lens = 50257, [500, 610, 700, 340, 650, 650, 450, 400]
    x, t, off, ref = big_pref(torch, lens, 0, 0, v, "bf16", v, 1)
    ws = poisoned(torch, M.preference_loss_workspace_bytes(x.shape[0], 4))

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


@pytest.mark.parametrize("n,v,pairs,dtype,walk", [
    (34000, 4000, 40, "bf16", False),    # 272 MB of short rows
    (14000, 16000, 18, "bf16", False),   # 448 MB of 32 KB rows: the tickets would take longer than the rows
    (3000, 50257, 4, "bf16", False),     # 302 MB: the second read is half out of the cache anyway
    (4500, 50257, 6, "bf16", True),      # 452 MB of 100 KB rows
    (7000, 32000, 9, "bf16", True),      # 448 MB of 64 KB rows
    (2400, 50257, 30, "fp32", True),     # 482 MB of 200 KB rows in short pairs
    (2400, 50257, 3, "fp32", False),     # the same in long ones, which the cache does not hold
    (1700, 131072, 17, "bf16", False)])  # nor these rows
def test_which_way(torch, n, v, pairs, dtype, walk):
    # with no look allowed at its pair a gradient of the walk is given up, so its loss is NaN; three launches wait
    # for nothing
    g = torch.Generator(DEV).manual_seed(n)
    x = torch.empty((n, v), dtype=dt(torch, dtype), device=DEV).normal_(0.0, 2.0, generator=g)
    t = torch.randint(0, v, (n,), generator=g, device=DEV)
    off = torch.arange(2 * pairs + 1, device=DEV) * n // (2 * pairs)
    loss, rew, d = torch.full((1,), 9.0, device=DEV), torch.empty(2 * pairs, device=DEV), torch.empty_like(x)
    polls = C.c_int.in_dll(M.load(), "muon_preference_max_polls")
    before, polls.value = polls.value, -1
    try:
        M.preference_loss(x, t, off, torch.zeros(2 * pairs, device=DEV), loss, rew, d,
                          poisoned(torch, M.preference_loss_workspace_bytes(n, pairs)))
        torch.cuda.synchronize()
    finally:
        polls.value = before
    assert bool(loss.isnan()) == walk
