"""Limits of the operators of a trained layer, where one begins to refuse (nothing reaches a device)."""

from __future__ import annotations

from test_layer_ops_host import _route_opt
from test_train_ops_host import BASE, BIG, _expect


def test_route_refuses_from_its_limit_of_tokens_on():
    far = 1 << 50  # apart from each other at any of these sizes
    for n, e, k in ((1 << 26, 257, 1), (1 << 30, 8, 2), (1 << 31, 1, 1)):
        _expect("muon_route", "MUON_ERR_UNSUPPORTED", BASE, n, e, e, 0, None, None, _route_opt(groups=1), BASE + far, 0, k,
                BASE + 2 * far, None)
        _expect("muon_route_backward", "MUON_ERR_UNSUPPORTED", BASE, n, e, e, 0, None, _route_opt(groups=1), BASE + far, 0, k,
                BASE + 2 * far, BASE + 3 * far, e, 1, None)
    assert BIG < far
