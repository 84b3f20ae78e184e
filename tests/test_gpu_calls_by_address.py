"""The operators' entry points by name, on addresses, against the calls on tensors."""

from __future__ import annotations

import numpy as np
import pytest

import muon_newton_schulz_step_amd as M
from test_gpu_train_ops import _all_operators, torch, vec  # noqa: F401

pytestmark = pytest.mark.gpu


def test_calls_by_address(torch):
    # the entry points by name, on addresses and strides, give what the calls on tensors give
    inp, out, ws, calls = _all_operators(torch, 0)
    calls()
    ids, tab, x, t, adv, w, old, ref, scores, picks = inp
    n, vocab, dim, e = x.shape[0], tab.shape[0], tab.shape[1], scores.shape[1]
    off = vec(torch, np.array([0, 100, 300, 450, 700]), "int64")
    sref = vec(torch, np.array([-500.0, -900.0, -700.0, -1100.0], dtype=np.float32))
    o = [torch.full_like(a, 9) for a in out]
    size = [a.numel() for a in ws]
    M.muon_embed_forward(tab, vocab, dim, dim, "bf16", ids, "int64", n, 2.0, o[0], dim)
    M.muon_embed_backward(ids, "int64", n, o[0], "bf16", dim, 2.0, o[1], vocab, dim, dim, True, ws[0], size[0])
    lo = M.muon_logits(x.data_ptr(), t.data_ptr(), n, vocab, vocab, 1, 1)
    M.muon_token_logprob(lo, o[2], o[3])
    M.muon_policy_loss(lo, adv, w, old, ref, M.muon_policy_options(0.2, 0.2, 0.1), o[4], o[5], o[6], vocab, ws[1], size[1])
    M.muon_preference_loss(lo, off, "int64", 2, sref, M.muon_preference_options(0.1, 0.0), o[7], o[8], o[9], vocab, ws[2], size[2])
    M.muon_balance_loss(scores, n, e, e, "fp32", picks, "int32", 2, None, M.muon_balance_options(0.01, 0.001), o[10], o[11],
                        o[12], e, ws[3], size[3])
    assert all(torch.equal(a, b) for a, b in zip(o, out))
    for f, a in ((M.muon_embed_forward, (tab, vocab, dim, dim - 1, "bf16", ids, "int64", n, 2.0, o[0], dim)),
                 (M.muon_embed_backward, (ids, "int64", n, o[0], "bf16", dim, 2.0, o[1], vocab, dim, dim, True, ws[0], 8)),
                 (M.muon_token_logprob, (lo, None)),
                 (M.muon_policy_loss, (lo, adv, w, old, ref, M.muon_policy_options(0.2, 0.2, 0.1), o[4], o[5], o[6], 1, ws[1], size[1])),
                 (M.muon_preference_loss, (lo, off, "int64", 0, sref, M.muon_preference_options(0.1, 0.0), o[7], o[8], o[9], vocab,
                                           ws[2], size[2])),
                 (M.muon_balance_loss, (scores, n, e, e, "fp32", picks, "int32", 0, None, M.muon_balance_options(0.01, 0.001), o[10],
                                        o[11], o[12], e, ws[3], size[3]))):
        with pytest.raises(M.MuonError, match=f.__name__):
            f(*a)
