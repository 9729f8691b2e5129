"""GPU: calls of the state space operators at the edges of what they allow: offsets past 32 bits,
two calls at once, a training step captured and replayed, outputs in place of inputs, rows on
4-byte boundaries, one group with and without its dimension."""
import pytest
import torch

import lm_reference as lm
import ssm_reference as ref
import stream_compaction_decoupled_gb300 as gb
import test_gpu_causal_conv as conv
import test_gpu_selective_scan as scan
from stream_compaction_decoupled_gb300 import autograd

pytestmark = pytest.mark.gpu


def rand(shape, dtype=torch.float32, scale=1.0, shift=0.0, seed=0):
    g = torch.Generator("cuda").manual_seed(seed)
    return (torch.empty(shape, dtype=dtype, device="cuda").normal_(generator=g).mul_(scale).add_(shift))


def close(got, want):
    """Two roundings to bf16, each off by half a step (2^-8 relative), and states that two ways to
    split the tokens leave a few units of 2^-24 apart: 16 of them, weighted, stay below 2^-12 of
    the largest output."""
    got, want = got.float(), want.float()
    assert ((got - want).abs() <= 2.0 ** -7 * want.abs() + 2.0 ** -12 * want.abs().max()).all()


def test_offsets_past_32_bits():
    """A row of more than 2^31 values: its end as the same tokens give alone, from the state before."""
    if torch.cuda.mem_get_info()[0] < 64 << 30:
        pytest.skip("needs 64 GB")
    t, d, n, tail = (1 << 20) + 5000, 2048, 16, 4096
    head = t - tail
    x, dy = rand((1, t, d), torch.bfloat16, seed=1), rand((1, t, d), torch.bfloat16, seed=2)
    w, bias = rand((d, 4), torch.bfloat16, 0.5), rand((d,), torch.bfloat16, 0.1)
    end = slice(head, None)
    y, last = gb.causal_conv(x, w, bias)
    want, want_last = gb.causal_conv(x[:, end], w, bias, state=x[:, head - 3:head].contiguous())
    assert torch.equal(y[:, end], want) and torch.equal(last, want_last)
    dx = gb.causal_conv_backward(dy, x, w, bias)[0]
    want = gb.causal_conv_backward(dy[:, end], x[:, end], w, bias, state=x[:, head - 3:head].contiguous())[0]
    assert torch.equal(dx[:, end], want)
    del y, dx

    dt, a = rand((1, t, d), torch.bfloat16, 0.5, seed=3), -torch.exp(rand((d, n), scale=0.5, seed=4))
    b, c, skip = rand((1, t, n), torch.bfloat16, seed=5), rand((1, t, n), torch.bfloat16, seed=6), rand((d,), seed=7)
    y, last, kept = gb.selective_scan(x, dt, a, b, c, skip, keep=True)
    assert kept.numel() > 1 << 31
    h0 = gb.selective_scan(x[:, :head], dt[:, :head], a, b[:, :head], c[:, :head], skip)[1]
    want, want_last, tail_kept = gb.selective_scan(x[:, end], dt[:, end], a, b[:, end], c[:, end], skip, h0=h0, keep=True)
    close(y[:, end], want)
    assert ((last - want_last).abs() <= 2.0 ** -18 * want_last.abs().max()).all()
    del y
    g = gb.selective_scan_backward(dy, x, dt, a, b, c, kept, skip)
    del kept
    want = gb.selective_scan_backward(dy[:, end], x[:, end], dt[:, end], a, b[:, end], c[:, end], tail_kept, skip)
    for k in ("dx", "ddt", "db", "dc"):
        close(getattr(g, k)[:, end], getattr(want, k))


def test_pools_past_32_bits():
    """States whose places are past 2^31 values, by the forms for one token."""
    if torch.cuda.mem_get_info()[0] < 64 << 30:
        pytest.skip("needs 64 GB")
    d, n, small = 4096, 16, 6
    pool = (1 << 31) // (d * n) + 10
    high = [pool - 1, 3, pool - 7, -1, pool // 2 + 1, pool - 2]
    slots = torch.tensor(high, dtype=torch.int32, device="cuda")
    low = torch.tensor([0, 1, 2, -1, 4, 5], dtype=torch.int32, device="cuda")
    x, dt, z = rand((small, d), torch.bfloat16, seed=1), rand((small, d), torch.bfloat16, seed=2), rand((small, d), torch.bfloat16, seed=3)
    b, c = rand((small, n), torch.bfloat16, seed=4), rand((small, n), torch.bfloat16, seed=5)
    a, start = -torch.exp(rand((d, n), scale=0.5, seed=6)), rand((small, d, n), seed=7)
    states = torch.zeros((pool, d, n), device="cuda")
    for k, s in enumerate(high):
        if s >= 0:
            states[s] = start[k]
    want_states = start.clone()
    want = gb.selective_scan_step(x, dt, a, b, c, want_states, z=z, slots=low)
    got = gb.selective_scan_step(x, dt, a, b, c, states, z=z, slots=slots)
    assert torch.equal(got, want)
    for k, s in enumerate(high):
        if s >= 0:
            assert torch.equal(states[s], want_states[k])
            states[s] = 0
    assert not states.any()
    del states
    pool = (1 << 31) // (3 * d) + 10
    high = [pool - 1, 3, pool - 7, -1, pool // 2 + 1, pool - 2]
    slots = torch.tensor(high, dtype=torch.int32, device="cuda")
    w, start = rand((d, 4), torch.bfloat16, 0.5), rand((small, 3, d), torch.bfloat16, seed=8)
    windows = torch.zeros((pool, 3, d), dtype=torch.bfloat16, device="cuda")
    for k, s in enumerate(high):
        if s >= 0:
            windows[s] = start[k]
    want_windows = start.clone()
    want = gb.causal_conv_step(x, want_windows, w, slots=low)
    got = gb.causal_conv_step(x, windows, w, slots=slots)
    assert torch.equal(got, want)
    for k, s in enumerate(high):
        if s >= 0:
            assert torch.equal(windows[s], want_windows[k])


@pytest.mark.parametrize("drafter", [True, False])
def test_vocabularies_past_32_bits(drafter):
    """More than 2^31 probabilities, rows at odd offsets."""
    if torch.cuda.mem_get_info()[0] < 64 << 30:
        pytest.skip("needs 64 GB")
    n, k, v = 4, 4, (1 << 27) + 3
    g = torch.Generator("cuda").manual_seed(1)
    target = torch.rand((n, k + 1, v), generator=g, device="cuda")
    draft = torch.rand((n, k, v), generator=g, device="cuda") if drafter else None
    drafts = torch.randint(0, v, (n, k), generator=g, device="cuda")
    accept = torch.zeros((n, k), device="cuda")
    accept[0, 1] = accept[1, 3] = accept[3, 2] = 0.999
    for row, i in ((0, 1), (1, 3), (3, 2)):  # refused there
        target[row, i, drafts[row, i]] = 0.0
    sample = torch.tensor([0.999, 0.5, 0.25, 0.75], device="cuda")
    got = gb.verify_drafts(drafts, target, draft, accept, sample)
    assert got.accepted.tolist() == [1, 3, 4, 2]
    for row, i in enumerate((1, 3, 4, 2)):
        rest = target[row, i].double()
        if i < k:
            if drafter:
                rest = (rest - draft[row, i].double()).clamp(min=0)
            else:
                rest[drafts[row, i]] = 0.0
        sums = rest.cumsum(0)
        token = int(got.tokens[row, i])
        # Within what 64-bit sums of 2^27 values leave open: 2^27 roundings of 2^-53 of the total.
        limit, slack = sample[row].double() * sums[-1], 2.0 ** -25 * sums[-1]
        assert sums[token] > limit - slack and (token == 0 or sums[token - 1] <= limit + slack) and rest[token] > 0


def layer(size, dtype, seed):
    b, t, d, n = size
    leaves = [rand((b, t, d), dtype, seed=seed), rand((d, 4), dtype, 0.5, seed=seed + 1), rand((d,), dtype, 0.1, seed=seed + 2),
              rand((b, t, d), dtype, 0.5, -1.0, seed=seed + 3), rand((d, n), scale=0.5, seed=seed + 4),
              rand((b, t, n), dtype, seed=seed + 5), rand((b, t, n), dtype, seed=seed + 6), rand((d,), seed=seed + 7),
              rand((b, t, d), dtype, seed=seed + 8), rand((d,), scale=0.3, seed=seed + 9)]
    return [v.requires_grad_() for v in leaves]


def train(leaves):
    x, w, bias, dt, log_a, b, c, d, z, dt_bias = leaves
    u, _ = autograd.causal_conv(x, w, bias)
    y, last = autograd.selective_scan(u, dt, -torch.exp(log_a), b, c, d, z, dt_bias)
    loss = y.float().square().mean() + last.mean()
    return (loss.detach(), *torch.autograd.grad(loss, leaves))


@pytest.mark.parametrize("size", [(2, 100, 96, 16), (1, 1500, 72, 8)])
def test_a_training_step_in_a_graph(size):
    """Captured, replayed with other inputs and again with the first.  (No eager graph of the leaves is
    alive: torch would run their end of the backward pass on that graph's stream.)"""
    leaves, other = layer(size, torch.bfloat16, 10), layer(size, torch.bfloat16, 50)
    want = train(leaves)
    with torch.no_grad():
        keep = [v.clone() for v in leaves]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = train(leaves)
    graph.replay()
    for u, v in zip(got, want):
        assert torch.equal(u, v)
    with torch.no_grad():
        for v, w in zip(leaves, other):
            v.copy_(w)
    graph.replay()
    for u, v in zip(got, train(other)):
        assert torch.equal(u, v)
    with torch.no_grad():
        for v, w in zip(leaves, keep):
            v.copy_(w)
    graph.replay()
    for u, v in zip(got, want):
        assert torch.equal(u, v)


def test_two_training_steps_at_once():
    """On two streams, over and over: each as alone."""
    size = (2, 900, 160, 16)
    many = [layer(size, torch.bfloat16, 10), layer(size, torch.bfloat16, 90)]
    want = [train(v) for v in many]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(4):
        for k in range(2):
            with torch.cuda.stream(streams[k]):
                got[k].append(train(many[k]))
    torch.cuda.synchronize()
    for k in range(2):
        for run in got[k]:
            for u, v in zip(run, want[k]):
                assert torch.equal(u, v)


def test_nothing_of_the_convolution_in_place():
    x, w = rand((2, 40, 64)), rand((64, 4))
    with pytest.raises(ValueError):
        gb.causal_conv(x, w, out=x)
    dy = rand((2, 40, 64), seed=1)
    for out in (x, dy):
        with pytest.raises(ValueError):
            gb.causal_conv_backward(dy, x, w, out=out)


def test_one_group_with_its_dimension_beside_one_without():
    size = (2, 40, 64, 16)
    leaves = layer(size, torch.float32, 3)
    want = train(leaves)
    x, w, bias, dt, log_a, b, c, d, z, dt_bias = leaves
    u, _ = autograd.causal_conv(x, w, bias)
    y, last = autograd.selective_scan(u, dt, -torch.exp(log_a), b[:, :, None], c, d, z, dt_bias)
    loss = y.square().mean() + last.mean()
    for u, v in zip((loss, *torch.autograd.grad(loss, leaves)), want):
        assert torch.equal(u, v)


def test_a_gradient_of_broadcast_inputs():
    """Inputs that all rows share get the sum of the rows' gradients (in 64 bits, rounded: each row's
    is off by 2^-24 or so of the largest, the sum of 3 by less than 2^-20)."""
    b, t, d, n = 3, 50, 64, 16
    x, dt, z = rand((1, t, d), seed=1), rand((1, t, d), seed=2), rand((1, t, d), seed=3)
    bm, cm = rand((1, t, n), seed=4), rand((1, t, n), seed=5)
    a, h0, dy = -torch.exp(rand((d, n), scale=0.5, seed=6)), rand((b, d, n), seed=7), rand((b, t, d), seed=8)
    shared = [v.requires_grad_() for v in (x, dt, z, bm, cm)]
    e = [v.expand(b, -1, -1) for v in shared]
    y, _ = autograd.selective_scan(e[0], e[1], a, e[3], e[4], None, e[2], h0=h0)
    got = torch.autograd.grad(y, shared, dy)
    full = [v.detach().expand(b, -1, -1).contiguous().requires_grad_() for v in shared]
    y2, _ = autograd.selective_scan(full[0], full[1], a, full[3], full[4], None, full[2], h0=h0)
    assert torch.equal(y, y2)
    for u, v in zip(got, torch.autograd.grad(y2, full, dy)):
        v = v.double().sum(0, keepdim=True)
        assert ((u.double() - v).abs() <= 2.0 ** -20 * v.abs().max()).all()


@pytest.mark.parametrize("dt", list(scan.DT))
@pytest.mark.parametrize("size", [(2, 45, 46, 6, 1), (1, 150, 130, 18, 1), (2, 33, 60, 10, 3), (1, 700, 34, 14, 1),
                                  (2, 20, 30, 44, 1), (1, 40, 2, 2, 1), (3, 18, 66, 16, 1)], ids=str)
def test_scans_of_rows_on_4_byte_boundaries(size, dt):
    scan.run(*size, scan.DT[dt], True, seed=sum(size))
    scan.run(*size, scan.DT[dt], False, seed=sum(size), pad=2)


@pytest.mark.parametrize("dt", list(conv.DT))
@pytest.mark.parametrize("taps", [2, 3, 4, 6])
@pytest.mark.parametrize("size", [(2, 70, 66), (1, 513, 130), (3, 40, 2046), (1, 30, 2)], ids=str)
def test_convolutions_of_rows_on_4_byte_boundaries(size, taps, dt):
    conv.run(*size, taps, conv.DT[dt], True, seed=sum(size) + taps)
    conv.run(*size, taps, conv.DT[dt], False, seed=sum(size) + taps, pad=2)


@pytest.mark.parametrize("dt", list(scan.DT))
@pytest.mark.parametrize("n", [13, 16, 40])
@pytest.mark.parametrize("d", [2050, 4097])
def test_single_tokens_of_many_rows(d, n, dt):
    """More rows and channels than fill the device: four rows a thread, the last of them alone; with a
    row of padding and a slot past the pool among them."""
    rows = 21
    q, _, _, _ = scan.inputs(rows, 1, d, n, 2 if d % 2 == 0 else 1, scan.DT[dt], True, d + n, pad=2)
    one = {k: v[:, 0] if k in ("x", "dt", "b", "c", "z") else v for k, v in q.items()}
    g = torch.Generator().manual_seed(n)
    pool = scan.rand(g, (30, d, n))
    before = pool.clone()
    slots = torch.randperm(30, generator=g)[:rows].int().cuda()
    slots[6], slots[17] = -1, 30
    y = gb.selective_scan_step(state=pool, slots=slots, **one)
    assert gb.device_error() == gb.ERR_RANGE and gb.device_error() == gb.OK
    assert not y[6].any() and not y[17].any()
    live = [r for r in range(rows) if r not in (6, 17)]
    at = slots[live].long()
    part = {k: v[live] if k in ("x", "dt", "b", "c", "z") else v for k, v in q.items()}
    want, last, bound, blast = ref.scan(**part, h0=before[at], starts=None)
    lm.check(y[live].unsqueeze(1), want, bound, "y")
    lm.check(pool[at], last, blast, "state")
    rest = [s for s in range(30) if s not in at.tolist()]
    assert torch.equal(pool[rest], before[rest])


@pytest.mark.parametrize("dt", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("offset", [0, 1, 2])
def test_taps_of_fp32_and_at_odd_places(offset, dt):
    """The single-token convolution's four taps: fp32 beside 16-bit inputs, and not where one access
    could read them."""
    b, d = 6, 264
    for pd in {scan.DT[dt], torch.float32}:
        g = torch.Generator().manual_seed(offset)
        x, bias = conv.rand(g, (b, d), scan.DT[dt]), conv.rand(g, (d,), pd)
        w = conv.rand(g, (d * 4 + 8,), pd, 0.5)[offset:offset + d * 4].view(d, 4)
        pool = conv.rand(g, (b, 3, d), scan.DT[dt])
        before = pool.clone()
        y = gb.causal_conv_step(x, pool, w, bias)
        want, last, bound, _ = ref.conv(x.unsqueeze(1), w, bias, before, None)
        lm.check(y.unsqueeze(1), want, bound, "y")
        assert torch.equal(lm.wide(pool), last)
        y, last = gb.causal_conv(x.unsqueeze(1), w, bias, state=before)
        lm.check(y, want, bound, "y")
        assert torch.equal(last, pool)


@pytest.mark.parametrize("dt", list(scan.DT))
@pytest.mark.parametrize("size", [(28, 20, 1024, 16), (28, 20, 1022, 14), (28, 20, 1023, 13), (4, 260, 2046, 6),
                                  (4, 260, 2047, 7)], ids=str)
def test_scans_that_fill_the_device(size, dt):
    """Enough rows and channels that two lanes share a pair of them: one part, or several."""
    b, t, d, n = size
    q, more, _, _ = scan.inputs(b, t, d, n, 1, scan.DT[dt], True, sum(size))
    scan.check_forward(q, more, gb.selective_scan(**q, **more))


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("size", [(28, 20, 512, 16), (28, 20, 510, 14), (28, 20, 511, 13), (20, 40, 448, 8),
                                  (13, 20, 510, 18)], ids=str)
def test_gradients_that_fill_the_device(size, dt):
    scan.run(*size, 1, scan.DT[dt], True, seed=sum(size))
