#!/usr/bin/env python
"""A small token model aligned on one GPU: the operators around the step and the step itself, as a training program
calls them.

The model reads a token and scores the next one: an embedding lookup, a layer of experts of which a router picks one
per token (routing, the tokens sorted by expert, a product for each group of rows, the gated sum), and an output
matrix.  It is trained on synthetic sequences that follow a rule (the next token is a * token + b): first by preference
between sequences that follow it and ones that do not, then by policy gradient on tokens it samples itself.  Each update
accumulates two micro-batches and takes one Muon step over all matrices.

    python examples/align_tokens.py [--steps 12] [--vocab 512] [--dim 256] [--experts 8] [--dropout 0.0]
"""

from __future__ import annotations

import argparse
import math
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import torch  # noqa: E402

import muon_newton_schulz_step_amd as M  # noqa: E402

DEV = "cuda:0"
MICRO = 2


def scratch(nbytes):
    return torch.empty(nbytes, dtype=torch.uint8, device=DEV)


class Model:
    """Parameters as views of one flat fp32 partition, which the Muon step updates."""

    def __init__(self, vocab, dim, experts, seed, dropout=0.0):
        self.vocab, self.dim, self.experts, self.dropout, self.seed = vocab, dim, experts, dropout, seed
        shapes = [(vocab, dim), (dim, experts), (dim, vocab)] + [(dim, dim)] * experts
        self.group = M.MuonGroup(shapes, precision="bf16", grad_dtype="fp32")
        g = torch.Generator(DEV).manual_seed(seed)
        self.flat = torch.zeros(self.group.partition_numel, device=DEV)
        self.params = [self.flat[o:o + r * c].view(r, c) for (r, c), o in zip(shapes, self.group.offsets)]
        for p in self.params:
            p.normal_(0.0, 1.0 / math.sqrt(dim), generator=g)
        # the experts' matrices as one tensor: they lie one behind the other in the partition, and so do their gradients
        first = self.group.offsets[3]
        self.mix = torch.as_strided(self.flat, (experts, dim, dim), (dim * dim, dim, 1), first)
        assert all(o == first + e * dim * dim for e, o in enumerate(self.group.offsets[3:]))
        self.a_mix = torch.empty(experts, dim, dim, device=DEV)
        self.update = torch.zeros_like(self.flat)
        self.acc = [torch.empty(s, device=DEV) for s in shapes[:3]] + list(self.a_mix)
        self.momenta = [torch.zeros(s, device=DEV) for s in shapes]
        self.ws = torch.empty(self.group.workspace_bytes, dtype=torch.uint8, device=DEV)
        self.scale = math.sqrt(dim)
        self.calls = torch.zeros(1, dtype=torch.int64, device=DEV)  # of the dropout: each draws another mask

    def forward(self, ids, choice=None, train=False):
        """choice: the router's picks, if they are to be held."""
        table, router, out, *_ = self.params
        n, d, e = ids.numel(), self.dim, self.experts
        h, xs, z, y = (torch.empty(n, d, device=DEV) for _ in range(4))
        M.embed_forward(table, ids, h, scale=self.scale)
        step = None
        if train and self.dropout > 0.0:
            self.calls += 1
            step = self.calls.clone()  # what the backward pass draws the same mask from
            M.dropout(h, h, self.dropout, self.seed, step=step)
        scores, logits = torch.empty(n, e, device=DEV), torch.empty(n, self.vocab, device=DEV)
        ws = scratch(max(M.linear_workspace_bytes(n, d, e, 1), M.linear_workspace_bytes(n, d, d, e),
                         M.linear_workspace_bytes(n, d, self.vocab, 1), M.expert_order_workspace_bytes(n, 1, e)))
        M.linear_forward(h, router, scores, ws)
        if choice is None:
            choice, gate = torch.empty(n, 1, dtype=torch.int64, device=DEV), torch.empty(n, 1, device=DEV)
            M.route_experts(scores, choice, gate, renormalize=False)
        else:
            gate = scores.softmax(1).gather(1, choice)
        # the tokens by expert, through their experts, and back to their places
        tokens, place = torch.empty(n, dtype=torch.int32, device=DEV), torch.empty(n, 1, dtype=torch.int32, device=DEV)
        offsets = torch.empty(e + 1, dtype=torch.int32, device=DEV)
        M.expert_order(choice, tokens, offsets, place, ws)
        M.embed_forward(h, tokens, xs)
        M.linear_forward(xs, self.mix, z, ws, offsets=offsets)
        M.expert_combine(z, place, y, weights=gate, residual=h)
        M.linear_forward(y, out, logits, ws)
        return {"ids": ids, "h": h, "scores": scores, "choice": choice, "gate": gate, "place": place, "offsets": offsets,
                "xs": xs, "z": z, "y": y, "logits": logits, "step": step}

    def backward(self, s, dlogits, first, coef=0.01):
        """Adds the gradients of a micro-batch, the router's balance loss among them; returns that loss's terms."""
        table, router, out, *_ = self.params
        a_table, a_router, a_out, *_ = self.acc
        n, d, e = s["ids"].numel(), self.dim, self.experts
        ws = scratch(max([M.linear_workspace_bytes(n, self.vocab, d, 1), M.linear_workspace_bytes(n, e, d, 1),
                          M.linear_workspace_bytes(n, d, d, e), M.balance_loss_workspace_bytes(n, e),
                          M.embed_backward_workspace_bytes(n, self.vocab, d)] +
                         [M.linear_weight_grad_workspace_bytes(n, d, c, g) for c, g in ((self.vocab, 1), (e, 1), (d, e))]))
        dy, dz, dxs, dh = (torch.empty(n, d, device=DEV) for _ in range(4))
        dgate = torch.empty(n, 1, device=DEV)
        M.linear_weight_grad(s["y"], dlogits, a_out, first, ws)
        M.linear_input_grad(dlogits, out, dy, ws)
        M.expert_combine_backward(dy, s["place"], dz, weights=s["gate"], y=s["z"], dweights=dgate)
        M.linear_weight_grad(s["xs"], dz, self.a_mix, first, ws, offsets=s["offsets"])
        M.linear_input_grad(dz, self.mix, dxs, ws, offsets=s["offsets"])
        M.expert_combine(dxs, s["place"], dh, residual=dy)
        # the router: its balance loss, and the chosen gate through the softmax
        counts = torch.empty(e, dtype=torch.int32, device=DEV)
        stats, dscores = torch.empty(3, device=DEV), torch.empty_like(s["scores"])
        M.balance_loss(s["scores"], s["choice"], counts, stats, dscores, ws, coef=coef, z_coef=1e-3)
        M.route_backward(s["scores"], s["choice"], dgate, dscores, False, renormalize=False)
        M.linear_weight_grad(s["h"], dscores, a_router, first, ws)
        M.linear_input_grad(dscores, router, dh, ws, residual=dh)
        if s["step"] is not None:
            M.dropout(dh, dh, self.dropout, self.seed, step=s["step"])
        M.embed_backward(s["ids"], dh, a_table, first, ws, scale=self.scale)
        return stats, counts

    def step(self, lr):
        self.group.step(self.acc, self.momenta, [self.update], self.ws)
        self.group.apply_update([self.flat], [self.update], lr, 0.0, 1e6, self.ws)

    def logprobs(self, ids, targets):
        s = self.forward(ids)
        logp = torch.empty(ids.numel(), device=DEV)
        M.token_logprob(s["logits"], targets, logp)
        return logp


def rule(ids, vocab):
    return (5 * ids + 3) % vocab


def preference_batch(vocab, pairs, length, g):
    """Ragged pairs packed into rows: chosen sequences follow the rule, rejected ones are random; the first two
    tokens of each are its prompt and no targets."""
    lengths = torch.randint(length // 2, length + 1, (2 * pairs,), generator=g, device=DEV).tolist()
    ids, targets, offsets = [], [], [0]
    for s, n in enumerate(lengths):
        x = torch.randint(0, vocab, (n,), generator=g, device=DEV)
        y = rule(x, vocab) if s < pairs else torch.randint(0, vocab, (n,), generator=g, device=DEV)
        y[:2] = -100
        ids.append(x)
        targets.append(y)
        offsets.append(offsets[-1] + n)
    return torch.cat(ids), torch.cat(targets), torch.tensor(offsets, device=DEV)


def prefer(model, ids, targets, offsets, first, beta, choice=None):
    """One micro-batch of the preference loss, against the uniform model as the reference."""
    seqs = offsets.numel() - 1
    s = model.forward(ids, choice, train=True)
    rows = offsets[1:] - offsets[:-1] - 2
    ref = -math.log(model.vocab) * rows.float()
    loss, rewards = torch.empty(1, device=DEV), torch.empty(seqs, device=DEV)
    ws = torch.empty(M.preference_loss_workspace_bytes(ids.numel(), seqs // 2), dtype=torch.uint8, device=DEV)
    M.preference_loss(s["logits"], targets, offsets, ref, loss, rewards, s["logits"], ws, beta=beta)
    model.backward(s, s["logits"], first)  # the gradient has taken the logits' place
    return loss


def reinforce(model, ids, g, first, old_logits, ref_logp_of):
    """One micro-batch of the policy loss on tokens drawn from the policy before the update."""
    n = ids.numel()
    drawn = torch.multinomial(old_logits.softmax(1), 1, generator=g)[:, 0]
    reward = (drawn == rule(ids, model.vocab)).float()
    adv = (reward - reward.mean()) / (reward.std() + 1e-3)
    old = torch.empty(n, device=DEV)
    M.token_logprob(old_logits, drawn, old)
    s = model.forward(ids, train=True)
    stats, logp = torch.empty(4, device=DEV), torch.empty(n, device=DEV)
    weights = torch.full((n,), 1.0 / n, device=DEV)
    ws = torch.empty(M.policy_loss_workspace_bytes(n), dtype=torch.uint8, device=DEV)
    M.policy_loss(s["logits"], drawn, adv, weights, stats, logp, s["logits"], ws, old_logp=old, ref_logp=ref_logp_of(ids, drawn),
                  clip_low=0.2, clip_high=0.28, kl_coef=0.02)
    model.backward(s, s["logits"], first)
    return reward.mean()


def main(steps=12, vocab=512, dim=256, experts=8, seed=0, dropout=0.0, lr=0.05, log=print):
    g = torch.Generator(DEV).manual_seed(seed)
    model = Model(vocab, dim, experts, seed, dropout)
    every = torch.arange(vocab, device=DEV)

    def fit():
        return float(model.logprobs(every, rule(every, vocab)).mean())
    out = {"fit": [fit()], "preference": [], "reward": []}
    for k in range(steps):
        losses = [prefer(model, *preference_batch(vocab, 16, 64, g), i == 0, beta=0.1) for i in range(MICRO)]
        model.step(lr)
        out["preference"].append(float(sum(losses)) / MICRO)
        log(f"preference step {k}: loss {out['preference'][-1]:.4f}")
    out["fit"].append(fit())
    frozen = model.flat.clone()

    def ref_logp(ids, targets):
        now = model.flat.clone()
        model.flat.copy_(frozen)
        logp = model.logprobs(ids, targets)
        model.flat.copy_(now)
        return logp
    for k in range(steps):
        rewards = []
        batch = torch.randint(0, vocab, (MICRO, 1024), generator=g, device=DEV)
        old = [model.forward(ids)["logits"] for ids in batch]
        for i, ids in enumerate(batch):
            rewards.append(reinforce(model, ids, g, i == 0, old[i], ref_logp))
        model.step(lr / 4)
        out["reward"].append(float(sum(rewards)) / MICRO)
        log(f"policy step {k}: reward {out['reward'][-1]:.4f}")
    out["fit"].append(fit())
    log("mean log-probability of the rule's token: start %.3f, after preferences %.3f, after the policy steps %.3f"
        % tuple(out["fit"]))
    model.group.close()
    return out


if __name__ == "__main__":
    p = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, default in (("steps", 12), ("vocab", 512), ("dim", 256), ("experts", 8), ("seed", 0)):
        p.add_argument("--" + name, type=int, default=default)
    p.add_argument("--dropout", type=float, default=0.0)
    main(**vars(p.parse_args()))
