"""GPU: the language-model operators joined by autograd, against torch's own operators in
64 bits, and the example that trains a small recurrent model and generates with it."""
import os
import sys

import pytest
import torch

import lm_reference as ref
import stream_compaction_decoupled_gb300 as gb
from stream_compaction_decoupled_gb300 import autograd

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def leaf(g, shape, scale=1.0):
    return (torch.randn(shape, generator=g) * scale).cuda().requires_grad_()


def wide(t):
    return None if t is None else t.detach().double().requires_grad_()


def close(got, want, rel):
    """Within `rel` of the gradient's own largest magnitude: fp32 sums of a few hundred
    terms, each product a few roundings (a few hundred times 2^-24)."""
    assert got.dtype == torch.float32
    assert (got.double() - want).abs().max() <= rel * want.abs().max()


def test_a_block_against_torch_in_64_bits():
    """layer norm -> fused projection -> recurrence -> logits -> log probability and entropy:
    every gradient against autograd of the plain formulas in 64 bits."""
    g = torch.Generator().manual_seed(1)
    b, t, d, v = 2, 45, 40, 57
    x, nw, nb = leaf(g, (b, t, d)), leaf(g, (d,)), leaf(g, (d,))
    w_in, head, h0 = leaf(g, (3 * d, d), d ** -0.5), leaf(g, (v, d), d ** -0.5), leaf(g, (b, d))
    starts = (torch.rand((b, t), generator=g) < 0.1).to(torch.uint8).cuda()
    targets = torch.randint(-1, v, (b * t,), generator=g).cuda()
    ce, cl = torch.randn(b * t, generator=g).cuda(), torch.randn((b, d), generator=g).cuda()

    def ours():
        y = autograd.layer_norm(x, nw, nb)
        u, f, i = torch.nn.functional.linear(y, w_in).split(d, -1)
        h, last = autograd.recurrence(u, f, i, h0, starts)
        lp, ent = autograd.token_logprobs(torch.nn.functional.linear(h, head).view(-1, v), targets)
        return (lp * ce).sum() + 0.3 * (ent * ce).sum() + (last * cl).sum()

    leaves = [x, nw, nb, w_in, head, h0]
    torch.backends.cuda.matmul.allow_tf32 = False
    grads = torch.autograd.grad(ours(), leaves)

    xw, nww, nbw, ww, hw, h0w = (wide(p) for p in leaves)
    c = xw - xw.mean(-1, keepdim=True)
    y = c / torch.sqrt((c * c).mean(-1, keepdim=True) + 1e-5) * nww + nbw
    u, f, i = (y @ ww.t()).split(d, -1)
    state, hs = h0w, []
    for k in range(t):
        keep = (starts[:, k] == 0).double()[:, None]
        state = torch.sigmoid(f[:, k]) * keep * state + torch.sigmoid(i[:, k]) * u[:, k]
        hs.append(state)
    logits = (torch.stack(hs, 1) @ hw.t()).view(-1, v)
    logp = torch.log_softmax(logits, -1)
    lp = torch.where(targets < 0, 0.0, logp.gather(1, targets.clamp(min=0)[:, None])[:, 0])
    ent = -(logp.exp() * logp).sum(-1)
    total = (lp * ce.double()).sum() + 0.3 * (ent * ce.double()).sum() + (state * cl.double()).sum()
    for got, want in zip(grads, torch.autograd.grad(total, [xw, nww, nbw, ww, hw, h0w])):
        close(got, want, 2e-5)


def test_only_some_outputs_have_gradients():
    g = torch.Generator().manual_seed(2)
    x, f, h0 = leaf(g, (2, 9, 16)), leaf(g, (2, 9, 16)), leaf(g, (2, 16))
    h, last = autograd.recurrence(x, f, None, h0)
    only_last = torch.autograd.grad(last.sum(), [x, f, h0])
    h, last = autograd.recurrence(x, f, None, h0)
    same = torch.autograd.grad(h[:, -1].sum(), [x, f, h0])
    assert all(torch.equal(p, q) for p, q in zip(only_last, same))
    y = autograd.layer_norm(x, None, torch.zeros(16, device="cuda", requires_grad=True))
    assert torch.autograd.grad(y.square().sum(), x)[0].shape == x.shape
    bias = torch.zeros(16, device="cuda", requires_grad=True)
    db, = torch.autograd.grad(autograd.layer_norm(x, None, bias).sum(), bias)
    assert torch.equal(db, torch.full((16,), 18.0, device="cuda"))
    lg = leaf(g, (3, 20))
    lp, ent = autograd.token_logprobs(lg, torch.tensor([1, -1, 3], device="cuda"))
    d, = torch.autograd.grad(ent.sum(), lg)
    assert d.abs().sum() > 0


def test_broadcast_gradient():
    """An expanded gradient (stride 0) reaches the kernels."""
    g = torch.Generator().manual_seed(3)
    x = leaf(g, (4, 32))
    d, = torch.autograd.grad(autograd.layer_norm(x).sum(), x)
    assert d.abs().max() < 1e-5  # a constant gradient is orthogonal to the normalisation


def test_example_learns_and_generates():
    import recurrent_lm
    model = recurrent_lm.Model(vocab=31, width=128, layers=2, seed=3)
    losses = recurrent_lm.train(model, 160, rows=8, length=160)
    # Uniform guessing costs log 31 = 3.43; the first two tokens of a document of 12 to 60
    # cannot be guessed, which leaves about 0.1 to 0.3.
    assert losses[0] > 3.0 and losses[-1] < 1.0
    prompts = torch.stack([(3 + s * torch.arange(12)) % 31 for s in (1, 2)]).cuda()
    tokens, scores, others = model.generate(prompts, 5)
    assert tokens.shape == (2, 5) and others.shape == (2, 5, 4)
    assert torch.equal(tokens, others[:, :, 0].long()) and (scores <= 0).all()
    # The step form continues what the sequence form computes: same last logits.
    starts = torch.zeros(prompts.shape, dtype=torch.uint8, device="cuda")
    with torch.no_grad():
        y = model.hidden(prompts, starts)
        logits = torch.nn.functional.linear(y[:, -1], model.head.to(model.dtype))
    assert torch.equal(logits.argmax(-1), tokens[:, 0])
    assert gb.device_error() == gb.OK
