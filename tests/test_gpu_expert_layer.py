"""A layer of experts as a training program runs it: routing, order, gather, the experts' two products with an
activation between them, the weighted sum, dropout into the residual stream, and all the way back, against the fp64
definitions; the same captured into a graph and on another stream; and the entry points by name, on addresses."""

from __future__ import annotations

import importlib.util
import os

import numpy as np
import pytest

import muon_newton_schulz_step_amd as M
import oracle.layer_ops as L
import oracle.train_ops as T
from test_gpu_train_ops import DEV, E, dt, f64, poisoned, torch, vec, within  # noqa: F401

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SEED, P = 12345, 0.25


class Layer:
    """Buffers of a layer for t tokens; run() enqueues a forward and a backward pass."""

    def __init__(self, torch, t, dim, ffn, experts, k, dtype, seed):
        g = torch.Generator(DEV).manual_seed(seed)
        d = dt(torch, dtype)

        def normal(*shape, std=1.0, kind=None):
            return torch.empty(*shape, dtype=kind or d, device=DEV).normal_(0.0, std, generator=g)

        def empty(*shape, kind=None):
            return torch.full(shape, 7, dtype=kind or d, device=DEV)
        self.t, self.k, self.shape = t, k, (dim, ffn, experts)
        self.x, self.dout = normal(t, dim), normal(t, dim)
        self.router = normal(dim, experts, std=dim ** -0.5)
        self.w1, self.b1 = normal(experts, dim, ffn, std=dim ** -0.5), normal(experts, ffn, std=0.1)
        self.w2, self.b2 = normal(experts, dim, ffn, std=ffn ** -0.5).transpose(1, 2), normal(experts, dim, std=0.1)
        self.bias = normal(experts, std=0.1, kind=torch.float32)
        self.step = torch.zeros(1, dtype=torch.int64, device=DEV)
        n, i32, f32 = t * k, torch.int32, torch.float32
        self.scores, self.dscores = empty(t, experts), empty(t, experts)
        self.choices, self.gate, self.dgate = empty(t, k, kind=i32), empty(t, k, kind=f32), empty(t, k, kind=f32)
        self.tokens, self.offsets, self.place = empty(n, kind=i32), empty(experts + 1, kind=i32), empty(t, k, kind=i32)
        self.xs, self.pre, self.mid, self.z = empty(n, dim), empty(n, ffn), empty(n, ffn), empty(n, dim)
        self.sum, self.out, self.dsum, self.dz, self.dpre = empty(t, dim), empty(t, dim), empty(t, dim), empty(n, dim), empty(n, ffn)
        self.dxs, self.dx = empty(n, dim), empty(t, dim)
        self.dw1, self.db1 = empty(experts, dim, ffn, kind=f32), empty(experts, ffn, kind=f32)
        self.dw2, self.db2 = empty(experts, ffn, dim, kind=f32), empty(experts, dim, kind=f32)
        self.drouter = empty(dim, experts, kind=f32)
        sizes = [M.expert_order_workspace_bytes(t, k, experts), M.linear_workspace_bytes(t, dim, experts, 1), M.linear_workspace_bytes(t, experts, dim, 1),
                 M.linear_workspace_bytes(n, dim, ffn, experts), M.linear_workspace_bytes(n, ffn, dim, experts),
                 M.linear_weight_grad_workspace_bytes(n, dim, ffn, experts), M.linear_weight_grad_workspace_bytes(n, ffn, dim, experts),
                 M.linear_weight_grad_workspace_bytes(t, dim, experts, 1)]
        self.ws = poisoned(torch, max(sizes))
        self.outputs = ("scores", "choices", "gate", "tokens", "offsets", "place", "out", "dx", "dw1", "db1", "dw2", "db2", "drouter")

    def run(self):
        how = dict(scoring="sigmoid", scale=2.0)
        M.linear_forward(self.x, self.router, self.scores, self.ws)
        M.route_experts(self.scores, self.choices, self.gate, bias=self.bias, **how)
        M.expert_order(self.choices, self.tokens, self.offsets, self.place, self.ws)
        M.embed_forward(self.x, self.tokens, self.xs)
        M.linear_forward(self.xs, self.w1, self.mid, self.ws, bias=self.b1, activation="silu", pre=self.pre, offsets=self.offsets)
        M.linear_forward(self.mid, self.w2, self.z, self.ws, bias=self.b2, offsets=self.offsets)
        M.expert_combine(self.z, self.place, self.sum, weights=self.gate)
        M.dropout(self.sum, self.out, P, SEED, site=3, step=self.step, residual=self.x)
        M.dropout(self.dout, self.dsum, P, SEED, site=3, step=self.step)
        M.expert_combine_backward(self.dsum, self.place, self.dz, weights=self.gate, y=self.z, dweights=self.dgate)
        M.linear_weight_grad(self.mid, self.dz, self.dw2, True, self.ws, dbias=self.db2, offsets=self.offsets)
        M.linear_input_grad(self.dz, self.w2, self.dpre, self.ws, pre=self.pre, activation="silu", offsets=self.offsets)
        M.linear_weight_grad(self.xs, self.dpre, self.dw1, True, self.ws, dbias=self.db1, offsets=self.offsets)
        M.linear_input_grad(self.dpre, self.w1, self.dxs, self.ws, offsets=self.offsets)
        M.expert_combine(self.dxs, self.place, self.dx, residual=self.dout)
        M.route_backward(self.scores, self.choices, self.dgate, self.dscores, True, **how)
        M.linear_weight_grad(self.x, self.dscores, self.drouter, True, self.ws)
        M.linear_input_grad(self.dscores, self.router, self.dx, self.ws, residual=self.dx)

    def results(self):
        return {name: getattr(self, name).clone() for name in self.outputs}


def test_expert_layer_against_the_definition(torch):
    # fp32 throughout: what a pass hands to the next one carries some e of its size, which the sums behind average
    a = Layer(torch, 90, 40, 72, 6, 2, "fp32", 1)
    a.step.fill_(17)
    a.run()
    got = {k: f64(v) for k, v in a.results().items()}
    x, dout = f64(a.x), f64(a.dout)
    scores = x @ f64(a.router)
    choices, gate = L.route(scores, 2, "sigmoid", bias=f64(a.bias), scale=2.0)
    assert np.array_equal(got["choices"], choices)
    tokens, offsets, place = L.expert_order(choices, 6)
    assert np.array_equal(got["tokens"], tokens) and np.array_equal(got["offsets"], offsets) and np.array_equal(got["place"], place)
    xs = x[tokens]
    mid, pre = L.linear_forward(xs, f64(a.w1), f64(a.b1), "silu", offsets=offsets)
    z, _ = L.linear_forward(mid, f64(a.w2), f64(a.b2), offsets=offsets)
    keep = L.dropout_keep(90, 40, P, SEED, 3, 17)
    out = L.dropout(L.expert_combine(z, place, gate), keep, P, x)
    dsum = L.dropout(dout, keep, P)
    dz, dgate = L.expert_combine_backward(dsum, z, place, np.zeros(z.shape), gate)
    dw2, db2 = L.linear_weight_grad(mid, dz, offsets)
    dpre = L.linear_input_grad(dz, f64(a.w2), "silu", pre, offsets=offsets)
    dw1, db1 = L.linear_weight_grad(xs, dpre, offsets)
    dx = L.expert_combine(L.linear_input_grad(dpre, f64(a.w1), offsets=offsets), place, residual=dout)
    dscores = L.route_backward(scores, choices, dgate, "sigmoid", scale=2.0)
    dx = dx + dscores @ f64(a.router).T
    want = dict(scores=scores, gate=gate, out=out, dx=dx, dw1=dw1, db1=db1, dw2=dw2, db2=db2, drouter=x.T @ dscores)
    for name, w in want.items():
        # ten passes of at most (72 + 90 + 60) e of a sum of magnitudes, which is at most 20 times the largest result
        within(got[name], w, 10 * 222 * E * 20 * np.abs(w).max(), name)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_expert_layer_in_a_graph_and_on_another_stream(torch, dtype):
    a = Layer(torch, 300, 64, 136, 8, 3, dtype, 2)
    a.run()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a.run()
    for k in range(4):
        a.step.fill_(k)
        a.x.normal_(generator=torch.Generator(DEV).manual_seed(10 + k))
        graph.replay()
        torch.cuda.synchronize()
        replayed = a.results()
        for v in a.outputs:
            getattr(a, v).fill_(7)
        a.ws.fill_(0xFF)
        if k % 2:
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                a.run()
            torch.cuda.current_stream().wait_stream(s)
        else:
            a.run()
        torch.cuda.synchronize()
        for name, v in a.results().items():
            assert torch.equal(v, replayed[name]), (k, name)


def test_two_layers_at_once(torch):
    # two layers on two streams, each with its own workspace, give what each gives alone
    a, b = Layer(torch, 257, 72, 128, 7, 2, "bf16", 3), Layer(torch, 511, 64, 200, 5, 4, "bf16", 4)
    a.run()
    b.run()
    torch.cuda.synchronize()
    alone = [a.results(), b.results()]
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(3):
        for st, layer in ((s, a), (t, b)):
            st.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(st):
                layer.run()
        torch.cuda.synchronize()
        for layer, want in zip((a, b), alone):
            assert all(torch.equal(v, want[name]) for name, v in layer.results().items())


def test_calls_by_address(torch):
    # the entry points by name, on addresses and strides, give what the calls on tensors give
    a = Layer(torch, 130, 48, 80, 6, 2, "bf16", 5)
    a.run()
    torch.cuda.synchronize()
    want = a.results()
    want.update(dz=a.dz.clone(), dgate=a.dgate.clone(), dscores=a.dscores.clone(), sum=a.sum.clone(), dpre=a.dpre.clone())
    t, k, (dim, ffn, n), slots = a.t, a.k, a.shape, a.t * a.k
    ws = a.ws.numel()
    o = M.muon_route_options(1, 1, 1, 1, 1, 0, 2.0)
    p = {name: getattr(a, name).data_ptr() for name in vars(a) if hasattr(getattr(a, name), "data_ptr")}
    for name in ("choices", "gate", "tokens", "offsets", "place", "sum", "out", "dz", "dgate", "dscores", "dw1", "db1", "dpre", "mid", "pre"):
        getattr(a, name).fill_(7)
    M.muon_route(p["scores"], t, n, n, "bf16", p["bias"], None, o, p["choices"], "int32", k, p["gate"])
    M.muon_expert_order(p["choices"], "int32", t, k, n, p["tokens"], p["offsets"], p["place"], p["ws"], ws)
    w1 = M.muon_weights(p["w1"], dim, ffn, ffn, dim * ffn, 0, n, p["offsets"], 0, 1)
    w2 = M.muon_weights(p["w2"], ffn, dim, ffn, dim * ffn, 1, n, p["offsets"], 0, 1)
    M.muon_linear_forward(p["xs"], slots, dim, w1, p["b1"], "silu", p["pre"], ffn, None, 0, p["mid"], ffn, p["ws"], ws)
    M.muon_linear_forward(p["mid"], slots, ffn, w2, p["b2"], "none", None, 0, None, 0, p["z"], dim, p["ws"], ws)
    M.muon_expert_combine(p["z"], slots, dim, dim, "bf16", p["place"], t, k, p["gate"], None, 0, p["sum"], dim)
    M.muon_dropout(p["sum"], t, dim, dim, "bf16", P, SEED, 3, 99, p["step"], p["x"], dim, p["out"], dim)
    M.muon_expert_combine_backward(p["dsum"], t, dim, dim, "bf16", p["place"], k, p["gate"], p["z"], dim, slots, p["dz"], dim, p["dgate"])
    M.muon_linear_input_grad(p["dz"], slots, dim, w2, "silu", p["pre"], ffn, None, 0, p["dpre"], ffn, p["ws"], ws)
    M.muon_linear_weight_grad(p["xs"], slots, dim, dim, p["dpre"], ffn, ffn, "bf16", p["offsets"], "int32", n, p["dw1"], ffn, dim * ffn, "in_out",
                              p["db1"], True, p["ws"], ws)
    M.muon_route_backward(p["scores"], t, n, n, "bf16", None, o, p["choices"], "int32", k, p["dgate"], p["dscores"], n, True)
    torch.cuda.synchronize()
    for name in ("choices", "gate", "tokens", "offsets", "place", "sum", "out", "dz", "dgate", "dscores", "dw1", "db1", "dpre"):
        assert torch.equal(getattr(a, name), want[name]), name
    half = torch.empty_like(a.dpre)
    M.muon_activation_grad(p["dpre"], slots, ffn, ffn, "bf16", "gelu", p["pre"], ffn, half, ffn)
    other = torch.empty_like(half)
    M.activation_grad(a.dpre, a.pre, other, "gelu")
    assert torch.equal(half, other)
    for f, args in ((M.muon_dropout, (p["sum"], t, dim, dim, "bf16", 1.5, SEED, 3, 0, None, None, 0, p["out"], dim)),
                    (M.muon_route, (p["scores"], t, n, n, "bf16", None, None, o, p["choices"], "int32", 0, p["gate"])),
                    (M.muon_route_backward, (p["scores"], t, n, n, "bf16", None, o, p["choices"], "int32", 0, p["dgate"], p["dscores"], n, True)),
                    (M.muon_expert_order, (p["choices"], "int32", t, k, n, p["tokens"], p["offsets"], p["place"], p["ws"], 8)),
                    (M.muon_expert_combine, (p["z"], slots, 0, dim, "bf16", p["place"], t, k, p["gate"], None, 0, p["sum"], dim)),
                    (M.muon_expert_combine_backward, (p["dsum"], t, dim, 1, "bf16", p["place"], k, None, None, 0, slots, p["dz"], dim, None)),
                    (M.muon_linear_forward, (p["xs"], slots, 1, w1, None, "none", None, 0, None, 0, p["mid"], ffn, p["ws"], ws)),
                    (M.muon_linear_input_grad, (p["dz"], slots, 1, w2, "none", None, 0, None, 0, p["dpre"], ffn, p["ws"], ws)),
                    (M.muon_linear_weight_grad, (p["xs"], slots, dim, 1, p["dpre"], ffn, ffn, "bf16", None, "int32", 1, p["dw1"], ffn, 0, "in_out", None,
                                                 True, p["ws"], ws)),
                    (M.muon_activation_grad, (p["dpre"], slots, 0, ffn, "bf16", "gelu", p["pre"], ffn, p["mid"], ffn))):
        with pytest.raises(M.MuonError, match=f.__name__):
            f(*args)


def test_example_with_dropout_runs_and_differentiates(torch):
    spec = importlib.util.spec_from_file_location("align_tokens", os.path.join(ROOT, "examples", "align_tokens.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    out = example.main(steps=2, vocab=96, dim=64, experts=4, dropout=0.2, log=lambda *_: None)
    assert np.isfinite(out["preference"] + out["reward"] + out["fit"]).all()
    # the gradient of a fixed mask: the calls' number set back before every pass
    model = example.Model(64, 32, 4, 3, dropout=0.3)
    g = torch.Generator(DEV).manual_seed(4)
    batch = example.preference_batch(64, 4, 20, g)
    start, choice = model.flat.clone(), model.forward(batch[0])["choice"]

    def loss(eps, u=None):
        model.flat.copy_(start)
        if u is not None:
            for p, d in zip(model.params, u):
                p.add_(d, alpha=eps)
        model.calls.zero_()
        return float(example.prefer(model, *batch, True, beta=0.1, choice=choice)), model.forward(batch[0], choice, train=False)
    loss(0.0)
    grads = [a.clone() for a in model.acc]
    # by the output matrix alone: what the router's balance loss adds does not depend on it
    u = [torch.zeros_like(p) for p in model.params]
    u[2].normal_(generator=g)
    h = 1e-2
    diff = (loss(h, u)[0] - loss(-h, u)[0]) / (2 * h)
    got = float((grads[2].double() * u[2].double()).sum())
    # the loss is of order 1 with a rounding of 1e-6 / h = 1e-4, its third derivatives h^2 of the slope
    assert got == pytest.approx(diff, rel=2e-3, abs=1e-3)
    model.group.close()
