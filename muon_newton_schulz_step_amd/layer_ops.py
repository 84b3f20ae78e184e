"""The operators of a trained layer of experts, on torch tensors: dropout, a
router's choice of experts, the order of the tokens by expert and the weighted
sum of what the experts return, and the product with a weight matrix or with
one a group of rows, each with its gradient (include/muon.h states each
formula).

Outputs, checks, streams and errors are as in ``train_ops``: every output is
the caller's tensor, ``ValueError`` comes before anything is enqueued, nothing
is allocated and nothing synchronises the host.
"""

from __future__ import annotations

import ctypes as C

from . import _lib
from .train_ops import _launch, _matrix, _refuse, _same, _vector, _workspace

__all__ = ["dropout", "route_experts", "route_backward", "expert_order", "expert_order_workspace_bytes",
           "expert_combine", "expert_combine_backward", "linear_forward", "linear_input_grad", "linear_weight_grad",
           "linear_workspace_bytes", "linear_weight_grad_workspace_bytes", "activation_grad"]

expert_order_workspace_bytes = _lib.muon_expert_order_workspace_bytes
linear_workspace_bytes = _lib.muon_linear_workspace_bytes
linear_weight_grad_workspace_bytes = _lib.muon_linear_weight_grad_workspace_bytes


def _like(x, what, rows, cols, dt):
    """(address, ld) of an optional matrix of that shape and type."""
    if x is None:
        return None, 0
    r, c, ld, _ = _matrix(x, what, dt)
    _same(what, (r, c), (rows, cols))
    return x.data_ptr(), ld


def _p(x):
    return None if x is None else x.data_ptr()


def dropout(x, out, p: float, seed: int, site: int = 0, step=0, residual=None, stream=None) -> None:
    """out = residual + (kept ? x / (1 - p) : 0); an element is kept or not by its row, its column, seed, site and
    step alone, so the gradient by x is the same call on the gradient by out.

    x, out, residual (None: none): rows x cols of one type; out may be x or the residual.  seed: 64 bits; site (a
    layer's number) and step: 32 bits.  step may be an int64 tensor of one element, read on the device."""
    rows, cols, ld, dt = _matrix(x, "x")
    op, old = _like(out, "out", rows, cols, dt)
    rp, rld = _like(residual, "residual", rows, cols, dt)
    device_step = None
    if not isinstance(step, int):
        _vector(step, "step", 1, dtype="int64")
        device_step, step = step, 0
    if not 0 <= seed < 1 << 64 or not 0 <= site < 1 << 32 or not 0 <= step < 1 << 32:
        _refuse("dropout", "seed is not of 64 bits, or site or step not of 32")
    f = _lib.load().muon_dropout
    _launch("dropout", lambda s: f(x.data_ptr(), rows, cols, ld, dt, p, seed, site, step, _p(device_step), rp, rld, op,
                                   old, s), stream, (x, out, residual, device_step))


def _choices(choices, tokens):
    if choices.dim() != 2 or choices.shape[0] != tokens or choices.shape[1] < 1:
        _refuse("choices", f"shape {tuple(choices.shape)}, expected ({tokens}, k)")
    return choices.shape[1], _vector(choices, "choices", choices.numel(), index=True)


def _scoring(name):
    if name not in _lib.SCORING:
        _refuse("scoring", f"{name!r}, expected one of {', '.join(_lib.SCORING)}")
    return _lib.SCORING[name]


def route_experts(logits, choices, weights, scoring: str = "softmax", bias=None, valid=None, groups: int = 1,
                  keep_groups: int = 1, group_top: int = 1, renormalize: bool = True, scale: float = 1.0,
                  stream=None) -> None:
    """choices[t]: the k experts of highest rank, highest first, where rank = score + bias, score = the softmax or
    sigmoid of logits[t]; weights[t] = scale * their scores, divided by the scores' sum if renormalize.

    logits: tokens x E; choices: tokens x k, int32 or int64; weights: fp32, tokens x k; bias: fp32[E] or None;
    valid: bool, one a token, or None.  With groups > 1 only experts of the keep_groups groups with the highest sum
    of their group_top (1 or 2) best ranks can be chosen.  -1 and weight 0 where there is no expert to choose."""
    tokens, experts, ld, dt = _matrix(logits, "logits")
    k, ct = _choices(choices, tokens)
    _vector(weights, "weights", tokens * k)
    if bias is not None:
        _vector(bias, "bias", experts)
    if valid is not None:
        _vector(valid, "valid", tokens, dtype="bool")
    o = _lib.muon_route_options(_scoring(scoring), 1 if renormalize else 0, groups, keep_groups, group_top, 0, scale)
    f = _lib.load().muon_route
    _launch("route", lambda s: f(logits.data_ptr(), tokens, experts, ld, dt, _p(bias), _p(valid), C.byref(o),
                                 choices.data_ptr(), ct, k, weights.data_ptr(), s), stream,
            (logits, choices, weights, bias, valid))


def route_backward(logits, choices, dweights, dlogits, first: bool, scoring: str = "softmax", valid=None,
                   renormalize: bool = True, scale: float = 1.0, stream=None) -> None:
    """dlogits = (0 if first else dlogits) + the gradient by the logits for the gradient dweights (fp32, tokens x k)
    by the weights of route_experts; choices as it gave them, scoring, valid, renormalize and scale as it took them.
    dlogits: like logits."""
    tokens, experts, ld, dt = _matrix(logits, "logits")
    k, ct = _choices(choices, tokens)
    _vector(dweights, "dweights", tokens * k)
    if valid is not None:
        _vector(valid, "valid", tokens, dtype="bool")
    dp, dld = _like(dlogits, "dlogits", tokens, experts, dt)
    o = _lib.muon_route_options(_scoring(scoring), 1 if renormalize else 0, 1, 1, 1, 0, scale)
    f = _lib.load().muon_route_backward
    _launch("route_backward", lambda s: f(logits.data_ptr(), tokens, experts, ld, dt, _p(valid), C.byref(o),
                                          choices.data_ptr(), ct, k, dweights.data_ptr(), dp, dld, 1 if first else 0,
                                          s), stream, (logits, choices, dweights, dlogits, valid))


def expert_order(choices, tokens, offsets, place, ws, stream=None) -> None:
    """Sorts the choices (T x k, int32 or int64) by expert, in the order of their tokens: expert e has the slots
    [offsets[e], offsets[e + 1]), slot s belongs to token tokens[s] (-1 behind the last), and choice (t, j) has the
    slot place[t, j] (-1 if it is outside [0, E)).

    tokens: int32[T * k]; offsets: int32[E + 1]; place: int32, T x k; ws: at least
    expert_order_workspace_bytes(T, k, E) bytes, 256-byte aligned."""
    if choices.dim() != 2 or choices.shape[1] < 1:
        _refuse("choices", f"shape {tuple(choices.shape)}, expected (tokens, k)")
    t, k = choices.shape
    ct = _vector(choices, "choices", t * k, index=True)
    _vector(tokens, "tokens", t * k, dtype="int32")
    _vector(place, "place", t * k, dtype="int32")
    experts = offsets.numel() - 1
    _vector(offsets, "offsets", experts + 1, dtype="int32")
    wp, wb = _workspace(ws)
    f = _lib.load().muon_expert_order
    _launch("expert_order", lambda s: f(choices.data_ptr(), ct, t, k, experts, tokens.data_ptr(), offsets.data_ptr(),
                                        place.data_ptr(), wp, wb, s), stream, (choices, tokens, offsets, place, ws))


def _place(place, tokens):
    if place.dim() != 2 or place.shape[0] != tokens or place.shape[1] < 1:
        _refuse("place", f"shape {tuple(place.shape)}, expected ({tokens}, k)")
    _vector(place, "place", place.numel(), dtype="int32")
    return place.shape[1]


def expert_combine(y, place, out, weights=None, residual=None, stream=None) -> None:
    """out[t] = residual[t] + sum_j weights[t, j] * y[place[t, j]]; a place outside y's rows adds nothing.
    place: int32, T x k; weights: fp32, T x k, or None (1 each); residual: like out, may be out, or None."""
    rows, dim, yld, dt = _matrix(y, "y")
    tokens, cols, old, _ = _matrix(out, "out", dt)
    _same("out columns", cols, dim)
    k = _place(place, tokens)
    if weights is not None:
        _vector(weights, "weights", tokens * k)
    rp, rld = _like(residual, "residual", tokens, dim, dt)
    f = _lib.load().muon_expert_combine
    _launch("expert_combine", lambda s: f(y.data_ptr(), rows, dim, yld, dt, place.data_ptr(), tokens, k, _p(weights),
                                          rp, rld, out.data_ptr(), old, s), stream, (y, place, out, weights, residual))


def expert_combine_backward(dout, place, dy=None, weights=None, y=None, dweights=None, stream=None) -> None:
    """dy[place[t, j]] = weights[t, j] * dout[t] (rows of no place are kept) and dweights[t, j] = the sum of dout[t] *
    y[place[t, j]] (0 for a place outside); either may be None.  y is needed for dweights only; dy may be y."""
    if dy is None and dweights is None:
        _refuse("expert_combine_backward", "neither dy nor dweights is asked for")
    tokens, dim, dold, dt = _matrix(dout, "dout")
    k = _place(place, tokens)
    rows = yld = dyld = 0
    if dweights is not None:
        if y is None:
            _refuse("dweights", "needs y")
        rows, cols, yld, _ = _matrix(y, "y", dt)
        _same("y columns", cols, dim)
        _vector(dweights, "dweights", tokens * k)
    if dy is not None:
        n, cols, dyld, _ = _matrix(dy, "dy", dt)
        _same("dy columns", cols, dim)
        if dweights is not None:
            _same("dy rows", n, rows)
        rows = n
    if weights is not None:
        _vector(weights, "weights", tokens * k)
    f = _lib.load().muon_expert_combine_backward
    _launch("expert_combine_backward",
            lambda s: f(dout.data_ptr(), tokens, dim, dold, dt, place.data_ptr(), k, _p(weights), _p(y), yld, rows,
                        _p(dy), dyld, _p(dweights), s), stream, (dout, place, dy, weights, y, dweights))


def _weights(w, what, offsets, dtype=None):
    """(groups, in, out, ld, stride, layout, muon_dtype, index type) of a matrix, in x out, or of one a group, groups x
    in x out; either of in and out may be the adjacent one in memory."""
    if w.dim() != (2 if offsets is None else 3):
        _refuse(what, f"{w.dim()} dimensions, expected " + ("2 without offsets" if offsets is None else "3 with offsets"))
    one = w if offsets is None else w[0] if w.shape[0] > 0 else _refuse(what, "no groups")
    a, b = one.shape
    layout = 0 if one.stride(1) == 1 or b == 1 else 1
    _, _, ld, dt = _matrix(one if layout == 0 else one.t(), what, dtype)
    groups = 1 if offsets is None else w.shape[0]
    it = 0
    if offsets is not None:
        it = _vector(offsets, "offsets", groups + 1, index=True)
    return groups, a, b, ld, 0 if groups == 1 else w.stride(0), layout, dt, it


def _activation(name):
    if name not in _lib.ACTIVATION:
        _refuse("activation", f"{name!r}, expected one of {', '.join(_lib.ACTIVATION)}")
    return _lib.ACTIVATION[name]


def linear_forward(x, w, out, ws, bias=None, activation: str = "none", pre=None, residual=None, offsets=None,
                   stream=None) -> None:
    """out = act(x w + bias) + residual, and pre = x w + bias if asked for.

    x: rows x in; w: in x out (a transposed view of out x in will do), or with offsets groups x in x out: group g has
    the rows [offsets[g], offsets[g + 1]), rows of no group are left alone; out, pre, residual (may be out): rows x
    out; bias: out or groups x out numbers; all of one type.  offsets: int32 or int64, groups + 1, on the device.
    activation: none, relu, silu, gelu or gelu_tanh.  ws: at least linear_workspace_bytes(rows, in, out, groups)
    bytes, 256-byte aligned."""
    groups, a, b, ld, stride, layout, dt, it = _weights(w, "w", offsets)
    rows, cols, xld, _ = _matrix(x, "x", dt)
    _same("x columns", cols, a)
    op, old = _like(out, "out", rows, b, dt)
    pp, pld = _like(pre, "pre", rows, b, dt)
    rp, rld = _like(residual, "residual", rows, b, dt)
    if bias is not None:
        _vector(bias, "bias", groups * b, dtype="bfloat16" if dt else "float32")
    act = _activation(activation)
    wp, wb = _workspace(ws)
    o = _lib.muon_weights(w.data_ptr(), a, b, ld, stride, layout, groups, _p(offsets), it, dt)
    f = _lib.load().muon_linear_forward
    _launch("linear_forward", lambda s: f(x.data_ptr(), rows, xld, C.byref(o), _p(bias), act, pp, pld, rp, rld, op, old,
                                          wp, wb, s), stream, (x, w, out, ws, bias, pre, residual, offsets))


def linear_input_grad(dy, w, dx, ws, pre=None, activation: str = "none", residual=None, offsets=None,
                      stream=None) -> None:
    """dx = (dy w') act'(pre) + residual: the gradient by the product's input, through the activation that made it
    (pre: what that took, rows x in), with a gradient that joins (residual, may be dx).

    dy: rows x out; w, offsets: as linear_forward took them; ws: at least linear_workspace_bytes(rows, out, in,
    groups) bytes, 256-byte aligned."""
    groups, a, b, ld, stride, layout, dt, it = _weights(w, "w", offsets)
    rows, cols, yld, _ = _matrix(dy, "dy", dt)
    _same("dy columns", cols, b)
    act = _activation(activation)
    if act and pre is None:
        _refuse("pre", "an activation needs it")
    if not act:
        pre = None
    xp, xld = _like(dx, "dx", rows, a, dt)
    pp, pld = _like(pre, "pre", rows, a, dt)
    rp, rld = _like(residual, "residual", rows, a, dt)
    wp, wb = _workspace(ws)
    o = _lib.muon_weights(w.data_ptr(), a, b, ld, stride, layout, groups, _p(offsets), it, dt)
    f = _lib.load().muon_linear_input_grad
    _launch("linear_input_grad", lambda s: f(dy.data_ptr(), rows, yld, C.byref(o), act, pp, pld, rp, rld, xp, xld, wp,
                                             wb, s), stream, (dy, w, dx, ws, pre, residual, offsets))


def linear_weight_grad(x, dy, dw, first: bool, ws, dbias=None, offsets=None, stream=None) -> None:
    """dw = (0 if first else dw) + x' dy and dbias = (0 if first else dbias) + the sums of dy's columns, a group of
    rows each if there are offsets.

    x: rows x in; dy: rows x out, of one type; dw: fp32, in x out or groups x in x out, either adjacent; dbias: fp32,
    out or groups x out numbers; ws: at least linear_weight_grad_workspace_bytes(rows, in, out, groups) bytes,
    256-byte aligned."""
    groups, a, b, ld, stride, layout, _, it = _weights(dw, "dw", offsets, 0)
    rows, cols, xld, dt = _matrix(x, "x")
    _same("x columns", cols, a)
    n, cols, yld, _ = _matrix(dy, "dy", dt)
    _same("dy", (n, cols), (rows, b))
    if dbias is not None:
        _vector(dbias, "dbias", groups * b)
    wp, wb = _workspace(ws)
    f = _lib.load().muon_linear_weight_grad
    _launch("linear_weight_grad", lambda s: f(x.data_ptr(), rows, a, xld, dy.data_ptr(), b, yld, dt, _p(offsets), it,
                                              groups, dw.data_ptr(), ld, stride, layout, _p(dbias), 1 if first else 0,
                                              wp, wb, s), stream, (x, dy, dw, ws, dbias, offsets))


def activation_grad(dy, pre, dpre, activation: str, stream=None) -> None:
    """dpre = dy act'(pre), for an activation that no product follows; dpre may be dy or pre."""
    rows, cols, yld, dt = _matrix(dy, "dy")
    pp, pld = _like(pre, "pre", rows, cols, dt)
    op, old = _like(dpre, "dpre", rows, cols, dt)
    act = _activation(activation)
    f = _lib.load().muon_activation_grad
    _launch("activation_grad", lambda s: f(dy.data_ptr(), rows, cols, yld, dt, act, pp, pld, op, old, s), stream,
            (dy, pre, dpre))
