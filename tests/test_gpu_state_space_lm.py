"""GPU: the state space operators joined: a layer trained through autograd against torch's own
operators in 64 bits, and a model that reads a prompt, generates token by token from pools of
states, and does the same with drafted tokens."""
import pytest
import torch

import stream_compaction_decoupled_gb300 as gb
from stream_compaction_decoupled_gb300 import autograd

pytestmark = pytest.mark.gpu

linear = torch.nn.functional.linear


def leaf(g, shape, scale=1.0, shift=0.0):
    return (torch.randn(shape, generator=g) * scale + shift).cuda().requires_grad_()


def parameters(g, d, inner, n, rank, taps, vocab):
    return {"embed": leaf(g, (vocab, d)), "norm_w": leaf(g, (d,), 0.2, 1.0), "norm_b": leaf(g, (d,), 0.1),
            "w_in": leaf(g, (2 * inner, d), d ** -0.5), "conv_w": leaf(g, (inner, taps), taps ** -0.5),
            "conv_b": leaf(g, (inner,), 0.1), "w_x": leaf(g, (rank + 2 * n, inner), inner ** -0.5),
            "w_dt": leaf(g, (inner, rank), rank ** -0.5), "dt_bias": leaf(g, (inner,), 0.5, -2.0),
            "log_a": leaf(g, (inner, n), 0.5), "d": leaf(g, (inner,), 0.1, 1.0),
            "w_out": leaf(g, (d, inner), inner ** -0.5), "head": leaf(g, (vocab, d), 3.0 * d ** -0.5)}


def rows(p, tokens, starts=None, states=None):
    """Logits of (batch, length) tokens and the states behind them; states: (conv, scan) to start from."""
    x = p["embed"][tokens]
    conv0, h0 = states if states is not None else (None, None)
    inner, n, rank = p["conv_w"].shape[0], p["log_a"].shape[1], p["w_dt"].shape[1]
    u, z = linear(autograd.layer_norm(x, p["norm_w"], p["norm_b"]), p["w_in"]).split(inner, -1)
    c, conv1 = autograd.causal_conv(u, p["conv_w"], p["conv_b"], conv0, starts)
    low, bm, cm = linear(c, p["w_x"]).split((rank, n, n), -1)
    y, h1 = autograd.selective_scan(c, linear(low, p["w_dt"]), -torch.exp(p["log_a"]), bm, cm, p["d"], z, p["dt_bias"], h0, starts)
    return linear(x + linear(y, p["w_out"]), p["head"]), (conv1, h1)


def rows64(p, tokens, starts):
    """The same from the formulas."""
    x = p["embed"][tokens]
    inner, n, rank, taps = p["conv_w"].shape[0], p["log_a"].shape[1], p["w_dt"].shape[1], p["conv_w"].shape[1]
    m = x - x.mean(-1, keepdim=True)
    v = m / torch.sqrt((m * m).mean(-1, keepdim=True) + 1e-5) * p["norm_w"] + p["norm_b"]
    u, z = (v @ p["w_in"].t()).split(inner, -1)
    b, t, _ = x.shape
    a = -torch.exp(p["log_a"])
    out = []
    window = [torch.zeros_like(u[:, 0])] * taps
    h = torch.zeros((b, inner, n), dtype=u.dtype, device=u.device)
    for k in range(t):
        keep = (starts[:, k] == 0).to(u.dtype)[:, None]
        window = [w * keep for w in window[1:]] + [u[:, k]]
        h = h * keep[..., None]
        s = p["conv_b"] + sum(w * p["conv_w"][:, j] for j, w in enumerate(window))
        s = s * torch.sigmoid(s)
        low, bm, cm = (s @ p["w_x"].t()).split((rank, n, n), -1)
        step = torch.nn.functional.softplus(low @ p["w_dt"].t() + p["dt_bias"])
        h = torch.exp(step[..., None] * a) * h + (step * s)[..., None] * bm[:, None]
        y = (h * cm[:, None]).sum(-1) + p["d"] * s
        y = y * z[:, k] * torch.sigmoid(z[:, k])
        out.append((x[:, k] + y @ p["w_out"].t()) @ p["head"].t())
    return torch.stack(out, 1)


def test_a_layer_against_torch_in_64_bits():
    g = torch.Generator().manual_seed(3)
    b, t, vocab = 2, 60, 31
    p = parameters(g, 24, 40, 16, 5, 4, vocab)
    tokens = torch.randint(0, vocab, (b, t), generator=g).cuda()
    starts = (torch.rand((b, t), generator=g) < 0.08).to(torch.uint8).cuda()
    targets = torch.randint(-1, vocab, (b * t,), generator=g).cuda()
    weight = torch.randn(b * t, generator=g).cuda()
    torch.backends.cuda.matmul.allow_tf32 = False
    logits, _ = rows(p, tokens, starts)
    logprob, entropy = autograd.token_logprobs(logits.reshape(-1, vocab), targets)
    grads = torch.autograd.grad((logprob * weight).sum() + 0.2 * (entropy * weight).sum(), list(p.values()))
    q = {k: v.detach().double().requires_grad_() for k, v in p.items()}
    lp = torch.log_softmax(rows64(q, tokens, starts).reshape(-1, vocab), -1)
    at = targets.clamp(min=0)[:, None]
    loss = (torch.where(targets < 0, 0.0, lp.gather(1, at)[:, 0]) * weight).sum() - 0.2 * ((lp.exp() * lp).sum(-1) * weight).sum()
    # fp32 sums of some hundred terms through five operators: a few hundred times 2^-24 of the largest.
    for name, got, want in zip(p, grads, torch.autograd.grad(loss, list(q.values()))):
        assert got.dtype == torch.float32
        assert (got.double() - want).abs().max() <= 5e-5 * want.abs().max(), name


class Generator:
    """One token a call for each request, states in pools; or several at once from a request's
    states, without moving them."""

    def __init__(self, p, pool):
        self.p = {k: v.detach() for k, v in p.items()}
        inner, taps = p["conv_w"].shape
        self.conv = torch.zeros((pool, taps - 1, inner), device="cuda")
        self.scan = torch.zeros((pool, inner, p["log_a"].shape[1]), device="cuda")
        self.a = -torch.exp(self.p["log_a"])

    def several(self, tokens, slots):
        at = slots.long()
        return rows(self.p, tokens, states=(self.conv[at], self.scan[at]))

    def take(self, tokens, slots):
        logits, (conv, scan) = self.several(tokens, slots)
        self.conv[slots.long()], self.scan[slots.long()] = conv, scan
        return logits

    def step(self, tokens, slots):
        p = self.p
        inner, n, rank = p["conv_w"].shape[0], self.a.shape[1], p["w_dt"].shape[1]
        x = p["embed"][tokens]
        v, _, _ = gb.layer_norm(x, p["norm_w"], p["norm_b"])
        u, z = linear(v, p["w_in"]).split(inner, -1)
        c = gb.causal_conv_step(u, self.conv, p["conv_w"], p["conv_b"], slots=slots)
        low, bm, cm = linear(c, p["w_x"]).split((rank, n, n), -1)
        y = gb.selective_scan_step(c, linear(low, p["w_dt"]), self.a, bm, cm, self.scan, p["d"], z, p["dt_bias"], slots=slots)
        return linear(x + linear(y, p["w_out"]), p["head"])


@torch.no_grad()
def test_prompt_then_tokens_then_drafts():
    """Greedy: the prompt at once and then token by token; the same with drafts, right ones and
    wrong ones, verified against the most likely tokens."""
    g = torch.Generator().manual_seed(5)
    vocab, n, length, more, k = 29, 3, 17, 24, 4
    p = parameters(g, 24, 64, 16, 8, 4, vocab)
    prompts = torch.randint(0, vocab, (n, length), generator=g).cuda()
    slots = torch.tensor([4, 0, 2], dtype=torch.int32, device="cuda")
    torch.backends.cuda.matmul.allow_tf32 = False
    one = Generator(p, 5)
    logits = one.take(prompts, slots)[:, -1]
    plain = []
    for _ in range(more + k + 1):
        plain.append(logits.argmax(-1))
        logits = one.step(plain[-1], slots)
    plain = torch.stack(plain, 1)

    two = Generator(p, 5)
    last = two.take(prompts[:, :-1], slots)[:, -1:] if length > 1 else None
    assert last is not None
    token = prompts[:, -1].clone()
    out = [[] for _ in range(n)]
    calls = 0
    while min(len(o) for o in out) < more:
        # Drafts: what is known to come, spoilt at a random place.
        drafts = torch.stack([torch.as_tensor((plain[r].tolist() + [0] * k)[len(out[r]):len(out[r]) + k]) for r in range(n)])
        spoil = torch.randint(0, k + 2, (n,), generator=g)
        for r in range(n):
            if spoil[r] < k:
                drafts[r, spoil[r]] = (drafts[r, spoil[r]] + 1) % vocab
        drafts = drafts.cuda()
        logits, _ = two.several(torch.cat([token[:, None], drafts], 1), slots)
        sure = torch.nn.functional.one_hot(logits.argmax(-1), vocab).float()
        r = gb.verify_drafts(drafts, sure, None, torch.rand((n, k), generator=g).cuda(), torch.rand((n,), generator=g).cuda())
        for row in range(n):
            a = int(r.accepted[row])
            new = r.tokens[row, :a + 1].tolist()
            assert r.tokens[row, a + 1:].tolist() == [-1] * (k - a)
            # What was accepted moves the request's states on; its last token comes first next time.
            one_slot = slots[row:row + 1]
            two.take(torch.cat([token[row:row + 1], drafts[row, :a]])[None], one_slot)
            token[row] = new[-1]
            out[row] += new
        calls += 1
    for row in range(n):
        assert out[row][:more] == plain[row, :more].tolist()
    assert calls < more


@torch.no_grad()
def test_a_step_of_the_whole_layer_in_a_graph():
    """The single-token forms captured once and replayed: the states move as they do eagerly."""
    g = torch.Generator().manual_seed(6)
    p = parameters(g, 24, 64, 16, 8, 4, 29)
    slots = torch.tensor([1, 3, -1], dtype=torch.int32, device="cuda")
    eager, graphed = Generator(p, 4), Generator(p, 4)
    tokens = torch.randint(0, 29, (6, 3), generator=g).cuda()
    want = [eager.step(tokens[i], slots) for i in range(6)]
    held = tokens[0].clone()
    graphed.step(held, slots)
    graphed.conv.zero_(), graphed.scan.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        logits = graphed.step(held, slots)
    graphed.conv.zero_(), graphed.scan.zero_()
    for i in range(6):
        held.copy_(tokens[i])
        graph.replay()
        assert torch.equal(logits, want[i])
    assert torch.equal(graphed.scan, eager.scan) and torch.equal(graphed.conv, eager.conv)
