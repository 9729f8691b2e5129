"""GPU: a document start drops the state before it, whatever that state is.  Infinities and
NaNs of one document, or of the state that a row starts from, do not reach the next one,
nor does a gradient of a later document reach an earlier one."""
import pytest
import torch

import stream_compaction_decoupled_gb300 as gb

pytestmark = pytest.mark.gpu

DT = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
NAN, INF = float("nan"), float("inf")
# (batch, length, channels): one block, blocks in clusters, odd widths, many strips alone.
SIZES = [(2, 50, 64), (1, 3000, 64), (1, 1500, 57), (40, 300, 520)]


def make(b, t, d, dtype, gate, seed):
    g = torch.Generator().manual_seed(seed)
    x, f, i, dh = (torch.randn((b, t, d), generator=g).to(dtype).cuda() for _ in range(4))
    h0, dlast = (torch.randn((b, d), generator=g).cuda() for _ in range(2))
    return x, f, (i if gate else None), h0, dh, dlast


def marks(b, t, *at):
    s = torch.zeros((b, t), dtype=torch.uint8, device="cuda")
    s[:, list(at)] = 1
    return s


def poison(t, value):
    """Every second channel."""
    t[..., ::2] = value


def same(p, q, where=slice(None)):
    assert torch.equal(p[:, where], q[:, where])


@pytest.mark.parametrize("value", [NAN, INF, -INF])
@pytest.mark.parametrize("gate", [False, True], ids=["tied", "gated"])
@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_a_start_drops_any_state(size, dt, gate, value):
    b, t, d = size
    x, f, i, h0, _, _ = make(*size, DT[dt], gate, t)
    first, second = t // 3 + 1, t // 2 + 2
    starts = marks(b, t, 0, first, second)
    want, wlast = gb.recurrence(x, f, i, h0=h0, starts=starts)
    assert torch.isfinite(want).all()
    # The state that the rows start from, and documents after it.
    bad = h0.clone()
    poison(bad, value)
    h, last = gb.recurrence(x, f, i, h0=bad, starts=starts)
    same(h, want)
    assert torch.equal(last, wlast)
    # Tokens of the first two documents; those after them are as they were.
    for at in (0, first - 1, first, second - 1):
        x2, f2 = x.clone(), f.clone()
        poison(x2[:, at], value)
        h, last = gb.recurrence(x2, f, i, h0=h0, starts=starts)
        assert not torch.isfinite(h[:, at, ::2]).any()
        same(h, want, slice(first if at < first else second, t))
        if at >= first:
            same(h, want, slice(0, first))
        assert torch.equal(last, wlast)
        poison(f2[:, at], value)
        h, last = gb.recurrence(x, f2, i, h0=h0, starts=starts)
        same(h, want, slice(first if at < first else second, t))
        assert torch.equal(last, wlast)


@pytest.mark.parametrize("value", [NAN, INF])
@pytest.mark.parametrize("gate", [False, True], ids=["tied", "gated"])
@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_a_start_stops_any_gradient(size, dt, gate, value):
    b, t, d = size
    x, f, i, h0, dh, dlast = make(*size, DT[dt], gate, t + 1)
    first, second = t // 3 + 1, t // 2 + 2
    starts = marks(b, t, first, second)
    h, _ = gb.recurrence(x, f, i, h0=h0, starts=starts)
    want = gb.recurrence_backward(dh, x, f, h, i, h0=h0, starts=starts, dlast=dlast)
    assert all(torch.isfinite(q).all() for q in want if q is not None)
    bad = dlast.clone()
    poison(bad, value)
    got = gb.recurrence_backward(dh, x, f, h, i, h0=h0, starts=starts, dlast=bad)
    for p, q in zip(got[:3], want):
        if q is not None:
            same(p, q, slice(0, second))
    assert torch.equal(got[3], want[3])
    assert not torch.isfinite(got[0][:, t - 1, ::2]).any()
    for at in (first, second - 1, second, t - 1):
        dh2 = dh.clone()
        poison(dh2[:, at], value)
        got = gb.recurrence_backward(dh2, x, f, h, i, h0=h0, starts=starts, dlast=dlast)
        for p, q in zip(got[:3], want):
            if q is not None:
                same(p, q, slice(0, first if at < second else second))
                same(p, q, slice(at + 1, t))
        assert torch.equal(got[3], want[3])
    # The states of a document that overflowed are not those before the next one's start.
    h2, bad0 = h.clone(), h0.clone()
    poison(h2[:, first - 1], value)
    poison(bad0, value)
    all_starts = starts.clone()
    all_starts[:, 0] = 1
    clean = gb.recurrence_backward(dh, x, f, h, i, h0=h0, starts=all_starts, dlast=dlast)
    got = gb.recurrence_backward(dh, x, f, h2, i, h0=bad0, starts=all_starts, dlast=dlast)
    for p, q in zip(got, clean):
        if q is not None:
            assert torch.equal(p, q)


@pytest.mark.parametrize("dt", list(DT))
def test_without_a_start_it_stays(dt):
    """The same values with no start between them reach everything after them."""
    x, f, i, h0, dh, dlast = make(1, 3000, 64, DT[dt], True, 5)
    f = f + 3
    poison(h0, NAN)
    h, last = gb.recurrence(x, f, i, h0=h0, starts=marks(1, 3000))
    assert torch.isnan(h[..., ::2]).all() and torch.isnan(last[:, ::2]).all()
    assert torch.isfinite(h[..., 1::2]).all()


@pytest.mark.parametrize("gate", [False, True], ids=["tied", "gated"])
@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_what_is_not_finite_stays_to_the_end_of_its_document(size, dt, gate):
    b, t, d = size
    x, f, i, h0, _, _ = make(*size, DT[dt], gate, t + 2)
    first, second = t // 3 + 1, t // 2 + 2
    starts = marks(b, t, first, second)
    want, wlast = gb.recurrence(x, f, i, h0=h0, starts=starts)
    x2 = x.clone()
    poison(x2[:, first + 3], NAN)
    poison(x2[:, t - 1], NAN)
    h, last = gb.recurrence(x2, f, i, h0=h0, starts=starts)
    nan = torch.zeros_like(h, dtype=torch.bool)
    nan[:, first + 3:second, ::2] = True
    nan[:, t - 1, ::2] = True
    assert torch.equal(torch.isnan(h), nan) and torch.equal(h[~nan], want[~nan])
    assert torch.isnan(last[:, ::2]).all() and torch.equal(last[:, 1::2], wlast[:, 1::2])


@pytest.mark.parametrize("gate", [False, True], ids=["tied", "gated"])
@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("often", [0.05, 0.3, 0.7])
@pytest.mark.parametrize("t,d", [(5, 8), (9, 16), (40, 40), (70, 72), (257, 260), (300, 303)])
def test_every_token_and_every_placing_of_starts(t, d, often, dt, gate):
    """Channel j has a NaN at token j (of x, then of dh): what follows it, or comes before it, to
    the next start is not finite, and everything else is as without."""
    b = 4
    x, f, i, h0, dh, dlast = make(b, t, d, DT[dt], gate, t + d)
    g = torch.Generator().manual_seed(d)
    starts = (torch.rand((b, t), generator=g) < often).to(torch.uint8).cuda()
    document = starts.long().cumsum(1)  # of each token
    n = min(t, d)
    token, at = torch.arange(t, device="cuda")[:, None], torch.arange(n, device="cuda")
    same_document = document[:, :, None] == document[:, None, :n]  # (batch, token, channel's token)
    want, wlast = gb.recurrence(x, f, i, h0=h0, starts=starts)
    x2 = x.clone()
    x2[:, at, at] = NAN
    h, last = gb.recurrence(x2, f, i, h0=h0, starts=starts)
    nan = torch.zeros_like(h, dtype=torch.bool)
    nan[:, :, :n] = same_document & (token >= at)
    assert torch.equal(torch.isnan(h), nan) and torch.equal(h[~nan], want[~nan])
    assert torch.equal(torch.isnan(last), nan[:, -1]) and torch.equal(last[~nan[:, -1]], wlast[~nan[:, -1]])
    wants = gb.recurrence_backward(dh, x, f, want, i, h0=h0, starts=starts, dlast=dlast)
    dh2 = dh.clone()
    dh2[:, at, at] = NAN
    grads = gb.recurrence_backward(dh2, x, f, want, i, h0=h0, starts=starts, dlast=dlast)
    nan[:, :, :n] = same_document & (token <= at)
    for p, q in zip(grads[:3], wants):
        if q is not None:
            assert torch.equal(torch.isnan(p), nan) and torch.equal(p[~nan], q[~nan])
    first = nan[:, 0] & (starts[:, 0] == 0)[:, None]
    assert torch.equal(torch.isnan(grads[3]), first) and torch.equal(grads[3][~first], wants[3][~first])
