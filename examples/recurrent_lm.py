#!/usr/bin/env python3
"""A small recurrent language model on this package's operators: trained on packed
sequences, then generating one token a call from a pool of states.

  python examples/recurrent_lm.py [--steps N] [--layers L] [--width D] [--quiet]

A layer is  x + W_out recurrence(W_in layer_norm(x)):  the input and both gates come from
one fused projection and go to the recurrence as slices of its rows.  The loss is the mean
negative log probability of the next token, from token_logprobs.  Generation keeps one
fp32 state a layer for each request in a pool, moves it with recurrence_step, and reports
each token with its most likely alternatives.  The matrix products are torch's.

The data is synthetic: documents that count upwards modulo the vocabulary by a step that
is the document's own, so the model has to remember something of what it read.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import stream_compaction_decoupled_gb300 as gb  # noqa: E402
from stream_compaction_decoupled_gb300 import autograd  # noqa: E402


class Model:
    def __init__(self, vocab: int, width: int, layers: int, seed: int = 0, dtype=torch.bfloat16):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def normal(shape, std):
            return (torch.randn(shape, generator=g, device="cuda") * std).requires_grad_()

        def ones(n, value=1.0):
            return torch.full((n,), value, device="cuda").requires_grad_()

        self.dtype, self.width, self.vocab = dtype, width, vocab
        self.embed = normal((vocab, width), 1.0)
        self.layers = [{"norm_w": ones(width), "norm_b": ones(width, 0.0), "w_in": normal((3 * width, width), width ** -0.5),
                        "b_in": torch.cat([torch.zeros(width), torch.full((width,), 2.0), torch.zeros(width)]).cuda().requires_grad_(),
                        "w_out": normal((width, width), 0.5 * width ** -0.5)} for _ in range(layers)]
        self.norm_w, self.norm_b = ones(width), ones(width, 0.0)
        self.head = normal((vocab, width), width ** -0.5)

    def parameters(self):
        return [self.embed, self.norm_w, self.norm_b, self.head] + [p for q in self.layers for p in q.values()]

    def _project(self, q, y):
        p = torch.nn.functional.linear(y, q["w_in"].to(self.dtype), q["b_in"].to(self.dtype))
        return p.split(self.width, dim=-1)  # x, f, i: slices of each row

    def hidden(self, tokens, starts):
        """(batch, length) tokens to the final normalised hidden rows."""
        x = self.embed[tokens].to(self.dtype)
        for q in self.layers:
            u, f, i = self._project(q, autograd.layer_norm(x, q["norm_w"], q["norm_b"]))
            h, _ = autograd.recurrence(u, f, i, None, starts)
            x = x + torch.nn.functional.linear(h, q["w_out"].to(self.dtype))
        return autograd.layer_norm(x, self.norm_w, self.norm_b)

    def loss(self, tokens, targets, starts):
        y = self.hidden(tokens, starts)
        logits = torch.nn.functional.linear(y, self.head.to(self.dtype)).view(-1, self.vocab)
        logprob, entropy = autograd.token_logprobs(logits, targets.reshape(-1))
        return -logprob.sum() / (targets >= 0).sum(), entropy.mean()

    @torch.no_grad()
    def logits_step(self, tokens, states, slots):
        """One token of each request: moves the states, returns the logits."""
        x = self.embed[tokens].to(self.dtype)
        for q, state in zip(self.layers, states):
            y, _, _ = gb.layer_norm(x, q["norm_w"], q["norm_b"])
            u, f, i = self._project(q, y)
            x = x + torch.nn.functional.linear(gb.recurrence_step(u, f, state, i, slots=slots), q["w_out"].to(self.dtype))
        y, _, _ = gb.layer_norm(x, self.norm_w, self.norm_b)
        return torch.nn.functional.linear(y, self.head.to(self.dtype))

    @torch.no_grad()
    def generate(self, prompts, length: int, top: int = 4):
        """Greedy continuation of (requests, prompt) tokens: tokens, their log
        probabilities, and the alternatives at each position."""
        n = prompts.shape[0]
        states = [torch.zeros((n + 2, self.width), device="cuda") for _ in self.layers]
        slots = torch.arange(n, device="cuda", dtype=torch.int32) + 1  # anywhere in the pool
        logits = None
        for t in range(prompts.shape[1]):
            logits = self.logits_step(prompts[:, t], states, slots)
        out, scores, others = [], [], []
        for _ in range(length):
            # The most likely token is the first alternative; scoring it is one more look.
            r = gb.token_logprobs(logits, torch.full((n,), -1, device="cuda"), top=top)
            tok = r.top_ids[:, 0].long()
            out.append(tok)
            scores.append(r.top_values[:, 0])
            others.append(r.top_ids)
            logits = self.logits_step(tok, states, slots)
        return torch.stack(out, 1), torch.stack(scores, 1), torch.stack(others, 1)


def batch(rows: int, length: int, vocab: int, g):
    """Documents of 12 to 60 tokens packed into rows: tokens, next-token targets (-1 across a
    document's end), and the start flags."""
    tokens = torch.empty((rows, length + 1), dtype=torch.int64)
    starts = torch.zeros((rows, length + 1), dtype=torch.uint8)
    for r in range(rows):
        t = 0
        while t <= length:
            n = int(torch.randint(12, 61, (1,), generator=g))
            a, s = (int(v) for v in torch.randint(1, vocab, (2,), generator=g))
            s = s % 5 + 1
            n = min(n, length + 1 - t)
            tokens[r, t:t + n] = (a + s * torch.arange(n)) % vocab
            starts[r, t] = 1
            t += n
    targets = tokens[:, 1:].clone()
    targets[starts[:, 1:] != 0] = -1
    return tokens[:, :-1].cuda(), targets.cuda(), starts[:, :-1].contiguous().cuda()


def train(model: Model, steps: int, rows: int = 16, length: int = 256, lr: float = 3e-3, seed: int = 1, report=None):
    opt = torch.optim.AdamW(model.parameters(), lr=lr, weight_decay=0.0)
    g = torch.Generator().manual_seed(seed)
    losses = []
    for k in range(steps):
        loss, entropy = model.loss(*batch(rows, length, model.vocab, g))
        opt.zero_grad(set_to_none=True)
        loss.backward()
        opt.step()
        if k % 20 == 0 or k == steps - 1:
            losses.append(float(loss.detach()))
            if report:
                report("step %4d  loss %.3f  mean entropy %.3f" % (k, losses[-1], float(entropy.detach())))
    return losses


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=200)
    ap.add_argument("--layers", type=int, default=2)
    ap.add_argument("--width", type=int, default=256)
    ap.add_argument("--vocab", type=int, default=101)
    ap.add_argument("--quiet", action="store_true")
    a = ap.parse_args()
    model = Model(a.vocab, a.width, a.layers)
    losses = train(model, a.steps, report=None if a.quiet else print)
    prompts = torch.stack([(7 + s * torch.arange(10)) % a.vocab for s in (1, 2, 3)]).cuda()
    tokens, scores, others = model.generate(prompts, 8)
    for p, t, s, o in zip(prompts.tolist(), tokens.tolist(), scores.tolist(), others.tolist()):
        print("%s -> %s" % (p, t))
        print("   log probabilities %s; alternatives of the first %s" % (["%.2f" % v for v in s], o[0]))
    print("loss %.3f -> %.3f" % (losses[0], losses[-1]))


if __name__ == "__main__":
    main()
