"""GPU: infinities in the selective scan and its gradient.  What is infinite by the definition stays
an infinity of its sign, in every number of states, channels and tokens; what does not depend on
one keeps its value."""
import math

import pytest
import torch

import lm_reference as lm
import ssm_reference as ref
import stream_compaction_decoupled_gb300 as gb
import test_gpu_selective_scan as scan

pytestmark = pytest.mark.gpu

INF = math.inf


def inputs(t, d, n, dtype, seed, rates=1.0):
    """Everything positive but the rates, so that no infinity of y or a state meets one of the other
    sign; step sizes of 0.1 to 1."""
    g = torch.Generator().manual_seed(seed)

    def some(shape, dtype, lo, hi):
        return (torch.rand(shape, generator=g) * (hi - lo) + lo).to(dtype).cuda()

    q = {"x": some((1, t, d), dtype, 0.25, 1.5), "dt": some((1, t, d), dtype, -2.0, 0.5),
         "a": -some((d, n), torch.float32, 0.1 * rates, rates), "b": some((1, t, 1, n), dtype, 0.25, 1.5),
         "c": some((1, t, 1, n), dtype, 0.25, 1.5), "d": some((d,), torch.float32, 0.25, 1.5),
         "z": some((1, t, d), dtype, 0.25, 1.5), "dt_bias": some((d,), torch.float32, -0.2, 0.0)}
    more = {"h0": some((1, d, n), torch.float32, 0.25, 1.5), "starts": None}
    return q, more, some((1, t, d), dtype, 0.25, 1.5), some((1, d, n), torch.float32, 0.25, 1.5)


def check_gradient(q, more, dy, dlast, same=None, skip=()):
    """All gradients but `skip` against the definition's, of `same` in place of a."""
    kept = gb.selective_scan(**q, **more, keep=True)[2]
    got = gb.selective_scan_backward(dy, **q, kept=kept, dlast=dlast)
    wants, bounds = ref.scan_grad(dy, **{**q, "a": q["a"] if same is None else same}, **more, dlast=dlast)
    for name, v, w, e in zip(scan.NAMES, got, wants, bounds):
        if name not in skip:
            lm.check(v, w, e, name)
    return got, wants, bounds


@pytest.mark.parametrize("dt", list(scan.DT))
@pytest.mark.parametrize("n", [1, 6, 8, 13, 16, 18, 40])
@pytest.mark.parametrize("t", [21, 24, 300])
@pytest.mark.parametrize("where", ["x", "dt"])
def test_states_past_the_last_stay_zero(where, t, n, dt):
    """An infinite input or step size in some channels: their y and last are infinite from there on."""
    q, more, _, _ = inputs(t, 24, n, scan.DT[dt], t + n)
    q[where][0, 5, ::2] = INF
    y, last, _ = gb.selective_scan(**q, **more)
    assert (y[0, 5:, ::2] == INF).all() and (last[0, ::2] == INF).all()
    want, wlast, bound, blast = ref.scan(**q, **more)
    bound, blast = bound.nan_to_num(0.0), blast.nan_to_num(0.0)  # (of infinities)
    lm.check(y, want, bound, "y")
    lm.check(last, wlast, blast, "last")


@pytest.mark.parametrize("dt", list(scan.DT))
@pytest.mark.parametrize("size", [(1, 24, 16), (7, 24, 16), (21, 24, 16), (21, 5, 13), (24, 24, 16), (300, 33, 40)], ids=str)
def test_tokens_behind_the_end_leave_states_of_infinite_rates(size, dt):
    """A rate of -infinity: its state keeps nothing from token to token, wherever the row ends."""
    t, d, n = size
    q, more, _, _ = inputs(t, d, n, scan.DT[dt], sum(size))
    q["a"][::3, 1] = -INF
    same = q["a"].clone()
    same[::3, 1] = -1e30
    got = gb.selective_scan(**q, **more)
    want, wlast, bound, blast = ref.scan(**{**q, "a": same}, **more)
    lm.check(got[0], want, bound, "y")
    lm.check(got[1], wlast, blast, "last")


@pytest.mark.parametrize("dt", list(scan.DT))
@pytest.mark.parametrize("where", ["b", "x"])
@pytest.mark.parametrize("t", [1, 7, 21])
def test_an_infinite_last_token_with_others_behind_it(t, where, dt):
    q, more, _, _ = inputs(t, 24, 16, scan.DT[dt], t)
    q[where][0, t - 1] = INF
    y, last, _ = gb.selective_scan(**q, **more)
    assert (last == INF).all() and (y[0, t - 1] == INF).all() and torch.isfinite(y[0, :t - 1]).all()


@pytest.mark.parametrize("dt", list(scan.DT))
def test_an_infinite_state_goes_through_parts(dt):
    """Rates that bring a part's decay below fp32's range, but no token's: an infinity lasts."""
    q, more, dy, dlast = inputs(600, 24, 16, scan.DT[dt], 3, rates=40.0)
    q["x"][0, 5, ::2] = INF
    y, last, _ = gb.selective_scan(**q, **more)
    want, wlast, bound, blast = ref.scan(**q, **more)
    assert (y[0, 5:, ::2] == INF).all() and (last[0, ::2] == INF).all()
    lm.check(y, want, bound, "y")
    lm.check(last, wlast, blast, "last")


@pytest.mark.parametrize("dt", list(scan.DT))
def test_an_infinite_gradient_goes_through_parts(dt):
    q, more, dy, dlast = inputs(600, 24, 16, scan.DT[dt], 3, rates=40.0)
    dy[0, -5, ::2] = INF
    got, _, _ = check_gradient(q, more, dy, dlast)
    assert (got.dx[0, :-4, ::2] == INF).all() and (got.dh0[0, ::2] == INF).all()


SIZES = [(32, 64, 6), (32, 64, 13), (304, 64, 40), (304, 64, 8)]


@pytest.mark.parametrize("dt", list(scan.DT))
@pytest.mark.parametrize("at", [5, -1])
@pytest.mark.parametrize("where", ["x", "dy"])
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_gradient_with_states_past_the_last(size, where, at, dt):
    t, d, n = size
    q, more, dy, dlast = inputs(t, d, n, scan.DT[dt], sum(size))
    (dy if where == "dy" else q["x"])[0, at, ::4] = INF
    check_gradient(q, more, dy, dlast)


@pytest.mark.parametrize("dt", list(scan.DT))
@pytest.mark.parametrize("where", ["a", "b", "c", "x", "dy"])
@pytest.mark.parametrize("t", [1, 15, 21, 300])
def test_gradient_with_tokens_behind_the_end(t, where, dt):
    q, more, dy, dlast = inputs(t, 64, 16, scan.DT[dt], t)
    if where != "a":
        (dy if where == "dy" else q[where])[0, -1] = INF
        check_gradient(q, more, dy, dlast)
        return
    q["a"][::3, 1] = -INF
    same = q["a"].clone()
    same[::3, 1] = -1e30
    # (the step size's gradient has the product of that rate and a decay of 0)
    got, wants, bounds = check_gradient(q, more, dy, dlast, same, skip=("ddt", "ddt_bias"))
    lm.check(got.ddt[..., 1::3].contiguous(), wants[1][..., 1::3], bounds[1][..., 1::3], "ddt")
    lm.check(got.ddt_bias[1::3].contiguous(), wants[7][1::3], bounds[7][1::3], "ddt_bias")


@pytest.mark.parametrize("dt", list(scan.DT))
@pytest.mark.parametrize("at", [5, -1])
@pytest.mark.parametrize("where", ["b", "c"])
@pytest.mark.parametrize("size", [(32, 24, 16), (32, 5, 16), (32, 33, 13), (21, 1, 32), (300, 70, 16), (32, 20, 40)], ids=str)
def test_gradient_with_channels_past_the_last(size, where, at, dt):
    t, d, n = size
    q, more, dy, dlast = inputs(t, d, n, scan.DT[dt], sum(size))
    q[where][0, at] = INF
    check_gradient(q, more, dy, dlast)


@pytest.mark.parametrize("dt", list(scan.DT))
@pytest.mark.parametrize("size", [(21, 24, 13), (40, 10, 16), (40, 66, 40), (300, 34, 6), (300, 64, 16)], ids=str)
def test_infinities_of_one_document_among_others(size, dt):
    """Two rows, two groups of channels; an infinite input in one row's first document, dropped by the
    next document's start, in the same tile or in another."""
    t, d, n = size
    q, _, dy, _ = inputs(2 * t, d, 2 * n, scan.DT[dt], sum(size))
    q = {k: v.unflatten(1, (2, t)).squeeze(0) if k in ("x", "dt", "z", "b", "c") else v for k, v in q.items()}
    q["b"], q["c"] = (q[k].squeeze(2).unflatten(-1, (2, n)) for k in ("b", "c"))
    q["a"] = q["a"][:, :n].contiguous()
    dy = dy.unflatten(1, (2, t)).squeeze(0)
    starts = torch.zeros((2, t), dtype=torch.uint8, device="cuda")
    starts[:, 9] = starts[0, t - 2] = starts[1, 0] = 1
    q["x"][1, 5, ::2] = INF
    more = {"h0": None, "starts": starts}
    y, last, kept = gb.selective_scan(**q, **more, keep=True)
    want, wlast, bound, blast = ref.scan(**q, **more)
    lm.check(y, want, bound, "y")
    lm.check(last, wlast, blast, "last")
    assert (y[1, 5:9, ::2] == INF).all() and torch.isfinite(y[1, 9:]).all() and torch.isfinite(last).all()
    got = gb.selective_scan_backward(dy, **q, kept=kept, starts=starts)
    wants, bounds = ref.scan_grad(dy, **q, **more, dlast=None)
    for name, v, w, e in zip(scan.NAMES, got, wants, bounds):
        lm.check(v, w, e, name)
