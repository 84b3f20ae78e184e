"""The example runs, and what it trains improves."""

from __future__ import annotations

import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    spec = importlib.util.spec_from_file_location("align_tokens", os.path.join(ROOT, "examples", "align_tokens.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def test_training_improves(example):
    out = example.main(steps=6, log=lambda *_: None)
    assert out["preference"][-1] < out["preference"][0]
    assert out["fit"][1] > out["fit"][0]
    assert out["reward"][-1] > out["reward"][0]


def test_backward_against_differences(example):
    # the loss's change along a direction in all parameters, with the router's picks held (across a change of them
    # the loss jumps), against the accumulated gradients
    import torch
    model = example.Model(64, 32, 4, 3)
    g = torch.Generator(example.DEV).manual_seed(4)
    batch = example.preference_batch(64, 4, 20, g)
    start = model.flat.clone()
    choice = model.forward(batch[0])["choice"]
    example.prefer(model, *batch, True, beta=0.1)
    grads = [a.clone() for a in model.acc]
    u = [torch.randn(p.shape, generator=g, device=example.DEV) for p in model.params]

    def loss(eps):
        model.flat.copy_(start)
        for p, d in zip(model.params, u):
            p.add_(d, alpha=eps)
        # the balance loss that backward() adds, with its coefficients
        scores, e = model.forward(batch[0], choice)["scores"].double(), model.experts
        f = torch.bincount(choice[:, 0], minlength=e).double() / choice.shape[0]
        balance = e * (f * scores.softmax(1).mean(0)).sum()
        return float(example.prefer(model, *batch, True, beta=0.1, choice=choice)) + float(
            0.01 * balance + 1e-3 * scores.logsumexp(1).square().mean())
    h = 1e-3
    diff = (loss(h) - loss(-h)) / (2 * h)
    got = sum(float((a.double() * d.double()).sum()) for a, d in zip(grads, u))
    size = sum(float((a.double() * d.double()).norm()) for a, d in zip(grads, u))
    # h^2 curvature 1e-6 and the loss's rounding 1e-6 / h = 1e-3, both against slopes of order `size`
    assert got == pytest.approx(diff, abs=0.02 * size + 2e-3)
    model.group.close()
