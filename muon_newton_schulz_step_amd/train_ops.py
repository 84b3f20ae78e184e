"""The operators around the Muon step, on torch tensors: embedding lookup and
its gradient, token log-probabilities, the clipped policy loss, the preference
loss and a router's balance loss, the losses with their gradients by the
logits (include/muon.h states each formula).

Every output is the caller's: results are written into the tensors given, as
``MuonGroup`` does, and a loss's gradient by the logits may be written over
the logits themselves.  Matrices may have any row stride; their elements in a
row have to be adjacent.  The calls check every tensor (device, type, shape,
strides) and raise ``ValueError`` before anything is enqueued; what the
library itself refuses raises ``MuonError``.  Work is ordered on ``stream``
(the current one of the tensors' device by default); on another stream than a
tensor's own, keeping the tensor until the work is done is the caller's part
(``Tensor.record_stream``).  Nothing synchronises the host, and nothing is
allocated, so the calls can be captured into a graph.
"""

from __future__ import annotations

import ctypes as C

from . import _lib

__all__ = ["embed_forward", "embed_backward", "embed_backward_workspace_bytes", "token_logprob", "policy_loss",
           "policy_loss_workspace_bytes", "preference_loss", "preference_loss_workspace_bytes", "balance_loss",
           "balance_loss_workspace_bytes"]

embed_backward_workspace_bytes = _lib.muon_embed_backward_workspace_bytes
policy_loss_workspace_bytes = _lib.muon_policy_loss_workspace_bytes
preference_loss_workspace_bytes = _lib.muon_preference_loss_workspace_bytes
balance_loss_workspace_bytes = _lib.muon_balance_loss_workspace_bytes

_torch = None
_DT: dict = {}     # torch dtype -> muon_dtype
_INDEX: dict = {}  # torch dtype -> muon_index_type


def _init():
    global _torch
    import torch
    _DT.update({torch.float32: 0, torch.bfloat16: 1})
    _INDEX.update({torch.int32: 0, torch.int64: 1})
    _torch = torch


def _refuse(what, why):
    raise ValueError(f"{what}: {why}")


def _matrix(x, what, dtype=None):
    """(rows, columns, row stride, muon_dtype) of a 2-D fp32 or bf16 tensor on the GPU."""
    if _torch is None:
        _init()
    dt = _DT.get(x.dtype)
    if dt is None or (dtype is not None and dt != dtype):
        _refuse(what, f"dtype {x.dtype}, expected " + ("float32 or bfloat16" if dtype is None else
                                                       "bfloat16" if dtype else "float32"))
    shape = x.shape
    if len(shape) != 2:
        _refuse(what, f"{len(shape)} dimensions, expected 2")
    rows, cols = shape
    ld, inner = x.stride()
    if inner != 1 and cols > 1 and rows > 0:
        _refuse(what, "the elements of a row are not adjacent (a transposed view?)")
    if rows <= 1:
        ld = max(ld, cols)
    elif ld < cols:
        _refuse(what, f"row stride {ld} is below the row length {cols} (an expanded view?)")
    if not x.is_cuda:
        _refuse(what, "a host tensor; the library needs device memory")
    return rows, cols, ld, dt


def _vector(x, what, n, index=False, dtype="float32"):
    """Checks a dense tensor of n elements on the GPU; the muon_index_type of an index vector."""
    if _torch is None:
        _init()
    t = None
    if index:
        t = _INDEX.get(x.dtype)
        if t is None:
            _refuse(what, f"dtype {x.dtype}, expected int32 or int64")
    elif x.dtype is not getattr(_torch, dtype):
        _refuse(what, f"dtype {x.dtype}, expected {dtype}")
    if x.numel() != n:
        _refuse(what, f"{x.numel()} elements, expected {n}")
    if not x.is_contiguous():
        _refuse(what, "not contiguous")
    if not x.is_cuda:
        _refuse(what, "a host tensor; the library needs device memory")
    return t


def _workspace(ws):
    if not ws.is_contiguous():
        _refuse("workspace", "not contiguous")
    if not ws.is_cuda:
        _refuse("workspace", "a host tensor; the library needs device memory")
    return ws.data_ptr(), ws.numel() * ws.element_size()


def _same(what, got, want):
    if got != want:
        _refuse(what, f"{got}, expected {want}")


def _launch(name, call, stream, tensors):
    """call(stream) on the device that all the tensors are on."""
    dev = tensors[0].get_device()
    for t in tensors:
        if t is not None and t.get_device() != dev:
            _refuse(name, "the tensors are on different devices")
    if stream is None:  # the handle alone: a Stream object costs a microsecond
        s = _torch._C._cuda_getCurrentRawStream(dev)
    else:
        s = stream if isinstance(stream, int) else stream.cuda_stream
    if _torch._C._cuda_getDevice() == dev:
        st = call(s)
    else:
        with _torch.cuda.device(dev):
            st = call(s)
    if st:
        _lib._check(st, "muon_" + name)


def embed_forward(table, ids, out, scale: float = 1.0, stream=None) -> None:
    """out[t] = scale * table[ids[t]]; zeros for an id outside the table.
    table: vocab x dim, ids: int32 or int64 of any shape, out: ids.numel() x dim of the table's type."""
    vocab, dim, table_ld, dt = _matrix(table, "table")
    tokens = ids.numel()
    it = _vector(ids, "ids", tokens, index=True)
    rows, cols, out_ld, _ = _matrix(out, "out", dt)
    _same("out", (rows, cols), (tokens, dim))
    f = _lib.load().muon_embed_forward
    _launch("embed_forward", lambda s: f(table.data_ptr(), vocab, dim, table_ld, dt, ids.data_ptr(), it, tokens,
                                         scale, out.data_ptr(), out_ld, s), stream, (table, ids, out))


def embed_backward(ids, dout, acc, first: bool, ws, scale: float = 1.0, stream=None) -> None:
    """acc[v] = (0 if first else acc[v]) + scale * the sum of dout[t] over the tokens t with ids[t] = v.
    dout: ids.numel() x dim, fp32 or bf16; acc: vocab x dim, fp32; ws: at least
    embed_backward_workspace_bytes(tokens, vocab, dim) bytes, 256-byte aligned."""
    tokens = ids.numel()
    it = _vector(ids, "ids", tokens, index=True)
    rows, dim, dout_ld, dt = _matrix(dout, "dout")
    _same("dout rows", rows, tokens)
    vocab, cols, acc_ld, _ = _matrix(acc, "acc", 0)
    _same("acc columns", cols, dim)
    wp, wb = _workspace(ws)
    f = _lib.load().muon_embed_backward
    _launch("embed_backward", lambda s: f(ids.data_ptr(), it, tokens, dout.data_ptr(), dt, dout_ld, scale,
                                          acc.data_ptr(), vocab, dim, acc_ld, 1 if first else 0, wp, wb, s),
            stream, (ids, dout, acc, ws))


def _logits(logits, targets):
    rows, vocab, ld, dt = _matrix(logits, "logits")
    it = _vector(targets, "targets", rows, index=True)
    return _lib.muon_logits(logits.data_ptr(), targets.data_ptr(), rows, vocab, ld, dt, it)


def _dlogits(dlogits, x):
    rows, vocab, ld, _ = _matrix(dlogits, "dlogits", x.dtype)
    _same("dlogits", (rows, vocab), (x.rows, x.vocab))
    return ld


def token_logprob(logits, targets, logp, lse=None, stream=None) -> None:
    """logp[r] = logits[r, targets[r]] - lse[r], lse[r] = log sum exp logits[r]; both 0 in a row whose target is
    outside the vocabulary (that row is not read).  logp, lse: fp32, one a row."""
    x = _logits(logits, targets)
    _vector(logp, "logp", x.rows)
    if lse is not None:
        _vector(lse, "lse", x.rows)
    f = _lib.load().muon_token_logprob
    _launch("token_logprob", lambda s: f(C.byref(x), logp.data_ptr(), None if lse is None else lse.data_ptr(), s),
            stream, (logits, targets, logp, lse))


def policy_loss(logits, targets, advantages, weights, stats, logp, dlogits, ws, old_logp=None, ref_logp=None,
                clip_low: float = 0.2, clip_high: float = 0.2, kl_coef: float = 0.0, stream=None) -> None:
    """The clipped policy loss sum_r weights[r] (-min(ratio A, clip(ratio) A) + kl_coef (exp(d) - 1 - d)) with
    ratio = exp(logp - old_logp) and d = ref_logp - logp, and its gradient by the logits.

    stats: fp32[4], receives the loss, its policy part, the weighted KL term and the weight of the clipped rows;
    logp: fp32, one a row; dlogits: like logits, may be the logits.  Rows of weight 0 or without a target (outside
    the vocabulary) are not read and get a zero gradient.  old_logp None: the rows' own log-probabilities.
    ws: at least policy_loss_workspace_bytes(rows) bytes, 256-byte aligned."""
    x = _logits(logits, targets)
    n = x.rows
    for t, what in ((advantages, "advantages"), (weights, "weights"), (logp, "logp"), (old_logp, "old_logp"),
                    (ref_logp, "ref_logp")):
        if t is not None:
            _vector(t, what, n)
    _vector(stats, "stats", 4)
    dld = _dlogits(dlogits, x)
    wp, wb = _workspace(ws)
    o = _lib.muon_policy_options(clip_low, clip_high, kl_coef)
    f = _lib.load().muon_policy_loss
    _launch("policy_loss", lambda s: f(C.byref(x), advantages.data_ptr(), weights.data_ptr(),
                                       None if old_logp is None else old_logp.data_ptr(),
                                       None if ref_logp is None else ref_logp.data_ptr(), C.byref(o),
                                       stats.data_ptr(), logp.data_ptr(), dlogits.data_ptr(), dld, wp, wb, s),
            stream, (logits, targets, advantages, weights, stats, logp, dlogits, ws, old_logp, ref_logp))


def preference_loss(logits, targets, offsets, ref_logp, loss, rewards, dlogits, ws, beta: float = 0.1,
                    label_smoothing: float = 0.0, stream=None) -> None:
    """The preference loss of pairs of sequences packed into the rows, and its gradient by the logits.

    Sequence s has the rows [offsets[s], offsets[s + 1]); of the 2 * pairs sequences, i is the chosen and pairs + i
    the rejected one of pair i.  gain = sum of logp - ref_logp, m = beta (gain_chosen - gain_rejected); the loss is
    the mean of -(1 - label_smoothing) log sigmoid(m) - label_smoothing log sigmoid(-m), and rewards = beta gain.
    loss: fp32[1]; ref_logp, rewards: fp32, one a sequence; dlogits: like logits, may be the logits.
    ws: at least preference_loss_workspace_bytes(rows, pairs) bytes, 256-byte aligned."""
    x = _logits(logits, targets)
    seqs = ref_logp.numel()
    if seqs < 2 or seqs % 2:
        _refuse("ref_logp", f"{seqs} sequences, expected a positive even number")
    _vector(ref_logp, "ref_logp", seqs)
    ot = _vector(offsets, "offsets", seqs + 1, index=True)
    _vector(loss, "loss", 1)
    _vector(rewards, "rewards", seqs)
    dld = _dlogits(dlogits, x)
    wp, wb = _workspace(ws)
    o = _lib.muon_preference_options(beta, label_smoothing)
    f = _lib.load().muon_preference_loss
    _launch("preference_loss", lambda s: f(C.byref(x), offsets.data_ptr(), ot, seqs // 2, ref_logp.data_ptr(),
                                           C.byref(o), loss.data_ptr(), rewards.data_ptr(), dlogits.data_ptr(), dld,
                                           wp, wb, s),
            stream, (logits, targets, offsets, ref_logp, loss, rewards, dlogits, ws))


def balance_loss(logits, experts, counts, stats, dlogits, ws, valid=None, coef: float = 0.01, z_coef: float = 0.0,
                 stream=None) -> None:
    """A router's balance loss coef E sum_e f_e mean_t p[t, e] + z_coef mean_t lse[t]^2 over the valid tokens, its
    gradient by the router's logits, and the tokens each expert gets.

    logits: tokens x E; experts: tokens x k, each token's choices, int32 or int64 (a choice outside [0, E) is counted
    nowhere); valid: bool, one a token, or None; counts: int32[E]; stats: fp32[3], the loss, its balance and its z
    term; dlogits: like logits, may be the logits.  ws: at least balance_loss_workspace_bytes(tokens, E) bytes,
    256-byte aligned."""
    tokens, n_experts, ld, dt = _matrix(logits, "logits")
    if experts.dim() != 2 or experts.shape[0] != tokens or experts.shape[1] < 1:
        _refuse("experts", f"shape {tuple(experts.shape)}, expected ({tokens}, k)")
    k = experts.shape[1]
    it = _vector(experts, "experts", tokens * k, index=True)
    _vector(counts, "counts", n_experts, dtype="int32")
    _vector(stats, "stats", 3)
    if valid is not None:
        _vector(valid, "valid", tokens, dtype="bool")
    rows, cols, dld, _ = _matrix(dlogits, "dlogits", dt)
    _same("dlogits", (rows, cols), (tokens, n_experts))
    wp, wb = _workspace(ws)
    o = _lib.muon_balance_options(coef, z_coef)
    f = _lib.load().muon_balance_loss
    _launch("balance_loss", lambda s: f(logits.data_ptr(), tokens, n_experts, ld, dt, experts.data_ptr(), it, k,
                                        None if valid is None else valid.data_ptr(), C.byref(o), counts.data_ptr(),
                                        stats.data_ptr(), dlogits.data_ptr(), dld, wp, wb, s),
            stream, (logits, experts, counts, stats, dlogits, ws, valid))
