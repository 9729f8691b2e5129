"""GPU: the causal convolution, its gradient and its single-token form against the definition in
64 bits, with tolerances from a first-order error analysis (ssm_reference.py)."""
import pytest
import torch

import lm_reference as lm
import ssm_reference as ref
import stream_compaction_decoupled_gb300 as gb
from stream_compaction_decoupled_gb300 import autograd

pytestmark = pytest.mark.gpu

DT = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}


def rand(g, shape, dtype, std=1.0):
    return (torch.randn(shape, generator=g) * std).to(dtype).cuda()


def inputs(b, t, d, taps, dtype, extras, seed, pad=None, wide=False, p_start=0.15):
    g = torch.Generator().manual_seed(seed)
    x, dy = rand(g, (b, t, d), dtype), rand(g, (b, t, d), dtype)
    if pad is not None:  # a slice of longer rows
        buf = torch.full((b, t, d + pad), float("nan"), dtype=dtype, device="cuda")
        buf[..., pad:] = x
        x = buf[..., pad:]
    pd = torch.float32 if wide else dtype
    w, bias = rand(g, (d, taps), pd, taps ** -0.5), rand(g, (d,), pd, 0.3) if extras else None
    state = rand(g, (b, taps - 1, d), dtype) if extras else None
    starts = (torch.rand((b, t), generator=g) < p_start).cuda() if extras else None
    dlast = rand(g, (b, taps - 1, d), dtype) if extras else None
    return x, dy, w, bias, state, starts, dlast


def run(b, t, d, taps, dtype, extras, seed=1, silu=True, **kw):
    x, dy, w, bias, state, starts, dlast = inputs(b, t, d, taps, dtype, extras, seed, **kw)
    y, last = gb.causal_conv(x, w, bias, state=state, starts=starts, silu=silu)
    want, wlast, bound, _ = ref.conv(x, w, bias, state, starts, silu)
    lm.check(y, want, bound, "y")
    assert last.dtype == dtype and torch.equal(lm.wide(last), wlast)
    got = gb.causal_conv_backward(dy, x, w, bias, state=state, starts=starts, dlast=dlast, silu=silu)
    wants, bounds = ref.conv_grad(dy, x, w, bias, state, starts, dlast, silu)
    for name, q, v, e in zip(("dx", "dw", "db", "dstate"), got, wants, bounds):
        if (name == "db" and bias is None) or (name == "dstate" and state is None):
            assert q is None
        else:
            lm.check(q, v, e, name)


SIZES = [(1, 1, 1), (2, 1, 8), (1, 2, 33), (3, 7, 64), (5, 31, 8), (2, 129, 72), (1, 513, 40), (2, 1000, 33),
         (3, 70, 1001), (40, 20, 520)]


@pytest.mark.parametrize("extras", [False, True], ids=["plain", "starts_state"])
@pytest.mark.parametrize("taps", [1, 2, 3, 4, 7, 8])
@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_conv(size, dt, taps, extras):
    run(*size, taps, DT[dt], extras, seed=sum(size) + taps)


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("pad", [0, 1, 2, 3, 4, 7, 8])
def test_row_strides_of_every_alignment(dt, pad):
    run(2, 70, 64, 4, DT[dt], True, seed=pad, pad=pad)
    run(2, 70, 64, 8, DT[dt], True, seed=pad, pad=pad)


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
def test_fp32_parameters_and_no_activation(dt):
    run(2, 90, 96, 4, DT[dt], True, wide=True)
    run(2, 90, 96, 3, DT[dt], True, silu=False)


def test_a_long_row_and_many_rows():
    """Runs of many lengths; more batch rows than rows of partial sums."""
    run(1, 20000, 64, 4, torch.bfloat16, True, p_start=0.01)
    run(300, 9, 4096, 4, torch.float32, True)


@pytest.mark.parametrize("t", [0, 1, 2, 3, 4])
def test_rows_shorter_than_the_window(t):
    run(2, t, 40, 4, torch.float32, True, p_start=0.0) if t else None
    x, dy, w, bias, state, starts, dlast = inputs(2, t, 40, 4, torch.float32, True, 3, p_start=0.0)
    y, last = gb.causal_conv(x, w, bias, state=state)
    assert y.shape == x.shape
    if t == 0:
        assert torch.equal(last, state)
        dx, dw, db, dstate = gb.causal_conv_backward(dy, x, w, bias, state=state, dlast=dlast)
        assert torch.equal(dstate, dlast) and not dw.any() and not db.any()


def test_in_pieces_and_token_by_token():
    """A row in three pieces, and one token a call, leave the same state and the same outputs."""
    b, t, d, taps = 3, 40, 48, 4
    x, _, w, bias, state, _, _ = inputs(b, t, d, taps, torch.bfloat16, True, 5)
    whole, end = gb.causal_conv(x, w, bias, state=state)
    at, s = 0, state
    for n in (1, 25, 14):
        y, s = gb.causal_conv(x[:, at:at + n], w, bias, state=s)
        assert torch.equal(y, whole[:, at:at + n])
        at += n
    assert torch.equal(s, end)
    pool = torch.zeros((7, taps - 1, d), dtype=x.dtype, device="cuda")
    slots = torch.tensor([5, 0, 3], dtype=torch.int32, device="cuda")
    pool[slots.long()] = state
    for k in range(t):
        y = gb.causal_conv_step(x[:, k], pool, w, bias, slots=slots)
        assert torch.equal(y, whole[:, k])
    assert torch.equal(pool[slots.long()], end)
    assert not pool[[1, 2, 4, 6]].any()


@pytest.mark.parametrize("taps", [1, 2, 4, 8])
@pytest.mark.parametrize("d", [1, 7, 64, 96, 1001])
@pytest.mark.parametrize("dt", list(DT))
def test_step(dt, d, taps):
    g = torch.Generator().manual_seed(d)
    x, w, bias = rand(g, (5, 2 * d), DT[dt])[:, :d], rand(g, (d, taps), DT[dt], 0.5), rand(g, (d,), DT[dt])
    pool = rand(g, (9, taps - 1, d), DT[dt])
    before = pool.clone()
    slots = torch.tensor([8, -1, 2, 0, -5], dtype=torch.int32, device="cuda")
    y = gb.causal_conv_step(x, pool, w, bias, slots=slots)
    for r, s in enumerate(slots.tolist()):
        if s < 0:
            assert not y[r].any()
            continue
        want, last, bound, _ = ref.conv(x[r].view(1, 1, d), w, bias, before[s].unsqueeze(0), None)
        lm.check(y[r].view(1, 1, d), want, bound, "y")
        assert torch.equal(lm.wide(pool[s]), last[0])
    rest = [1, 3, 4, 5, 6, 7]
    assert torch.equal(pool[rest], before[rest])
    y = gb.causal_conv_step(x, pool[:4].contiguous(), w, bias, slots=torch.tensor([0, 4, 1, 2, 3], dtype=torch.int32,
                                                                                 device="cuda"))
    assert not y[1].any() and gb.device_error() == gb.ERR_RANGE and gb.device_error() == gb.OK


def test_a_start_drops_infinities_and_nans():
    b, t, d = 1, 12, 64
    x, dy, w, bias, state, _, _ = inputs(b, t, d, 4, torch.float32, True, 2)
    starts = torch.zeros((b, t), dtype=torch.uint8, device="cuda")
    starts[0, 0] = starts[0, 6] = 1
    x[0, 5] = float("inf")
    state[:] = float("nan")
    y, last = gb.causal_conv(x, w, bias, state=state, starts=starts)
    want, _, bound, _ = ref.conv(x, w, bias, state, starts)
    lm.check(y[:, :5], want[:, :5], bound[:, :5])
    lm.check(y[:, 6:], want[:, 6:], bound[:, 6:])
    assert torch.isfinite(last).all()
    dx, dw, _, dstate = gb.causal_conv_backward(dy, x, w, bias, state=state, starts=starts)
    assert torch.isfinite(dx[:, 6:]).all() and not dstate.any()


def test_gradients_against_differences():
    """Each gradient against central differences of the forward kernel in fp32: a step of 2^-7 on
    smooth functions is off by its third derivative, some 1e-5 of the sum's scale, and by the
    forward's roundings, 1e-6 over the step."""
    b, t, d, taps = 2, 9, 16, 4
    x, dy, w, bias, state, starts, dlast = inputs(b, t, d, taps, torch.float32, True, 9)
    args = [x, w, bias, state]

    def loss(v):
        y, last = gb.causal_conv(v[0], v[1], v[2], state=v[3], starts=starts)
        return float((y.double() * dy.double()).sum() + (last.double() * dlast.double()).sum())

    grads = gb.causal_conv_backward(dy, *args[:3], state=state, starts=starts, dlast=dlast)
    g = torch.Generator().manual_seed(0)
    for k, grad in enumerate(grads):
        for _ in range(3):
            way = torch.randn(args[k].shape, generator=g).cuda()
            way /= way.norm()
            h = 2.0 ** -7
            up, down = list(args), list(args)
            up[k], down[k] = args[k] + h * way, args[k] - h * way
            slope = (loss(up) - loss(down)) / (2 * h)
            assert abs(slope - float((grad.double() * way.double()).sum())) < 2e-3 * max(1.0, float(grad.norm()))


def test_the_same_from_run_to_run_on_streams_and_in_graphs():
    x, dy, w, bias, state, starts, dlast = inputs(4, 300, 128, 4, torch.bfloat16, True, 4)

    def call(stream=None):
        return (*gb.causal_conv(x, w, bias, state=state, starts=starts, stream=stream),
                *gb.causal_conv_backward(dy, x, w, bias, state=state, starts=starts, dlast=dlast, stream=stream))

    want = call()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = call(side)
    side.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = call()
    for v in held:
        v.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(held, want))


def test_outputs_into_slices_and_refusals():
    x, dy, w, bias, state, starts, dlast = inputs(2, 30, 64, 4, torch.bfloat16, True, 6)
    buf = torch.zeros((2, 30, 200), dtype=x.dtype, device="cuda")
    y, _ = gb.causal_conv(x, w, bias, out=buf[..., 64:128])
    want, _ = gb.causal_conv(x, w, bias)
    assert torch.equal(buf[..., 64:128], want) and not buf[..., :64].any() and not buf[..., 128:].any()
    dx = gb.causal_conv_backward(dy, x, w, bias, out=buf[..., :64])[0]
    assert torch.equal(dx, gb.causal_conv_backward(dy, x, w, bias)[0])
    assert gb.causal_conv_backward(dy, x, w, bias, dparams=False)[1:] == (None, None, None)
    for bad in (dict(weight=w.float().double()), dict(bias=bias.float())):
        with pytest.raises(TypeError):
            gb.causal_conv(**{**dict(x=x, weight=w, bias=bias), **bad})
    for bad in (dict(weight=w[:32]), dict(weight=w[:, :0]), dict(weight=torch.zeros((64, 9), dtype=x.dtype, device="cuda")),
                dict(state=state[:, :2]), dict(starts=starts[:, :5]), dict(x=x[..., ::2]), dict(x=x.cpu()), dict(bias=bias[:8])):
        with pytest.raises(ValueError):
            gb.causal_conv(**{**dict(x=x, weight=w, bias=bias), **bad})
    with pytest.raises(ValueError):
        gb.causal_conv_step(x[:, 0], state[:1], w, bias)


def test_autograd_and_frozen_parameters():
    x, dy, w, bias, state, starts, dlast = inputs(2, 40, 32, 4, torch.float32, True, 7)
    leaves = [v.clone().requires_grad_() for v in (x, w, bias, state)]
    y, last = autograd.causal_conv(*leaves, starts)
    got = torch.autograd.grad((y * dy).sum() + (last * dlast).sum(), leaves)
    want = gb.causal_conv_backward(dy, x, w, bias, state=state, starts=starts, dlast=dlast)
    assert all(torch.equal(p, q) for p, q in zip(got, want))
    y, _ = autograd.causal_conv(leaves[0], w, bias, None, None)
    (dx,) = torch.autograd.grad((y * dy).sum(), [leaves[0]])
    assert torch.equal(dx, gb.causal_conv_backward(dy, x, w, bias)[0])
