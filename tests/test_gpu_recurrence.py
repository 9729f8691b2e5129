"""GPU: the gated linear recurrence, its gradient and its single-token form against the
definition in 64 bits, with tolerances from a first-order error analysis (lm_reference.py),
and the gradient against differences of the forward kernel."""
import pytest
import torch

import lm_reference as ref
import stream_compaction_decoupled_gb300 as gb

pytestmark = pytest.mark.gpu

DT = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}


def rand(g, shape, dtype, mean=0.0, std=1.0):
    return (torch.randn(shape, generator=g) * std + mean).to(dtype).cuda()


def inputs(b, t, d, dtype, gate, extras, seed, fused=True, pad=0):
    """x, f, i as slices of one buffer whose rows are `pad` values longer (odd pads make
    the rows start at every alignment), or as arrays of their own."""
    g = torch.Generator().manual_seed(seed)
    k = 3 if gate else 2
    x = rand(g, (b, t, d), dtype)
    f = rand(g, (b, t, d), dtype, 1.5, 2.0).clamp_(-8, 8)
    i = rand(g, (b, t, d), dtype, 0.0, 2.0).clamp_(-8, 8) if gate else None
    if fused:
        buf = torch.zeros((b, t, k * d + pad), dtype=dtype, device="cuda")
        views = [buf[..., n * d:(n + 1) * d] for n in range(k)]
        for v, src in zip(views, (x, f, i)):
            v.copy_(src)
        x, f, i = views[0], views[1], views[2] if gate else None
    h0 = rand(g, (b, d), torch.float32) if extras else None
    starts = (torch.rand((b, t), generator=g) < 0.05).cuda() if extras else None
    dh, dlast = rand(g, (b, t, d), dtype), rand(g, (b, d), torch.float32) if extras else None
    return x, f, i, h0, starts, dh, dlast


def run(b, t, d, dtype, gate, extras, seed=1, **kw):
    x, f, i, h0, starts, dh, dlast = inputs(b, t, d, dtype, gate, extras, seed, **kw)
    h, last = gb.recurrence(x, f, i, h0=h0, starts=starts)
    want, wlast, bound, blast = ref.recurrence(x, f, i, h0, starts)
    ref.check(h, want, bound, "h")
    ref.check(last, wlast, blast, "last")
    got = gb.recurrence_backward(dh, x, f, h, i, h0=h0, starts=starts, dlast=dlast)
    wants, bounds = ref.recurrence_grad(dh, x, f, h, i, h0, starts, dlast)
    for name, q, w, e in zip(("dx", "df", "di", "dh0"), got, wants, bounds):
        if w is None:
            assert q is None
        else:
            ref.check(q, w, e, name)


SIZES = [(1, 1, 1), (2, 1, 8), (1, 2, 33), (3, 7, 64), (5, 31, 8), (2, 129, 72), (1, 513, 40), (2, 1000, 33),
         (1, 5000, 16), (4, 300, 1001), (1, 2050, 256), (40, 20, 520)]


@pytest.mark.parametrize("extras", [False, True], ids=["plain", "starts_h0"])
@pytest.mark.parametrize("gate", [False, True], ids=["tied", "gated"])
@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_recurrence(size, dt, gate, extras):
    run(*size, DT[dt], gate, extras, seed=sum(size))


@pytest.mark.parametrize("dt", ["fp32", "bf16"])
@pytest.mark.parametrize("strips", [8, 32, 40, 45, 52, 62, 80, 120, 155, 200])
def test_clusters_of_every_size(strips, dt):
    """Few 64-channel strips are shared by clusters of up to 8 blocks, more by fewer, and
    many by none; lengths that end in the first, a middle and the last block's tile."""
    for t in (450, 1025) if strips < 100 else (130,):
        run(strips, t, 64, DT[dt], True, True, seed=strips)


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("pad", [1, 2, 3, 4, 7, 8])
def test_row_strides_of_every_alignment(dt, pad):
    run(2, 70, 64, DT[dt], True, True, seed=pad, pad=pad)


@pytest.mark.parametrize("dt", list(DT))
def test_arrays_of_their_own(dt):
    run(2, 200, 96, DT[dt], True, True, seed=5, fused=False)


def test_time_major_layout():
    """(time, batch, channel) memory seen as (batch, time, channel)."""
    x, f, i, h0, starts, dh, _ = inputs(3, 50, 64, torch.bfloat16, True, True, 3, fused=False)
    want = gb.recurrence(x, f, i, h0=h0, starts=starts)
    tm = [v.transpose(0, 1).contiguous().transpose(0, 1) for v in (x, f, i)]
    out = torch.empty((50, 3, 64), dtype=x.dtype, device="cuda").transpose(0, 1)
    got = gb.recurrence(*tm, h0=h0, starts=starts, out=out)
    assert got[0] is out and torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_broadcast_input():
    """An expanded input (stride 0 over batch) is read in place."""
    x, f, i, _, _, _, _ = inputs(1, 40, 64, torch.float32, True, False, 4, fused=False)
    xe = x.expand(3, -1, -1)
    fe, ie = f.repeat(3, 1, 1), i.repeat(3, 1, 1)
    h, last = gb.recurrence(xe, fe, ie)
    one, _ = gb.recurrence(x, f, i)
    assert all(torch.equal(h[k], one[0]) for k in range(3))


@pytest.mark.parametrize("gate", [False, True])
def test_starts_everywhere_and_saturated_gates(gate):
    """Every token a start: h = u x.  Gates at +-100 and infinite are 0 and 1 exactly
    enough; nothing overflows into a NaN."""
    b, t, d = 2, 130, 48
    x, f, i, h0, _, dh, _ = inputs(b, t, d, torch.float32, gate, True, 9)
    ones = torch.ones((b, t), dtype=torch.uint8, device="cuda")
    h, last = gb.recurrence(x, f, i, h0=h0, starts=ones)
    want, wlast, bound, blast = ref.recurrence(x, f, i, h0, ones)
    ref.check(h, want, bound)
    dx, df, di, dh0 = gb.recurrence_backward(dh, x, f, h, i, h0=h0, starts=ones)
    assert torch.equal(dh0, torch.zeros_like(dh0))
    if gate:
        assert torch.equal(df, torch.zeros_like(df))
    for big in (100.0, float("inf")):
        f2 = torch.where(torch.arange(d, device="cuda") % 2 == 0, big, -big).expand(b, t, d).contiguous()
        h, last = gb.recurrence(x, f2, f2 if gate else None, h0=h0)
        assert torch.isfinite(h).all()
        odd = x[..., 1::2] * (0.0 if gate else 1.0)  # forgotten at once
        assert (h[..., 1::2] - odd).abs().max() <= 1e-6 * 8
        if not gate:  # kept for ever
            assert torch.equal(h[..., 0::2], h0[:, None, 0::2].expand(b, t, d // 2))
        grads = gb.recurrence_backward(dh, x, f2, h, f2 if gate else None, h0=h0)
        assert all(torch.isfinite(q).all() for q in grads if q is not None)


def test_nan_stays_in_its_channel_and_after_its_token():
    x, f, i, _, _, _, _ = inputs(1, 300, 64, torch.float32, True, False, 2)
    clean, _ = gb.recurrence(x, f, i)
    x[0, 100, 5] = float("nan")
    h, last = gb.recurrence(x, f, i)
    assert torch.isnan(h[0, 100:, 5]).all() and torch.isnan(last[0, 5])
    h[0, 100:, 5] = clean[0, 100:, 5]
    assert torch.equal(h, clean)


@pytest.mark.parametrize("shape", [(0, 5, 8), (2, 0, 8), (2, 5, 0)], ids=str)
def test_empty(shape):
    b, t, d = shape
    x = torch.zeros(shape, device="cuda", dtype=torch.bfloat16)
    h0 = torch.ones((b, d), device="cuda")
    h, last = gb.recurrence(x, x, x, h0=h0)
    assert h.shape == shape and last.shape == (b, d)
    grads = gb.recurrence_backward(x, x, x, h, x, h0=h0, dlast=2 * h0)
    assert all(q.shape == shape for q in grads[:3])
    if t == 0:
        assert torch.equal(last, h0) and torch.equal(grads[3], 2 * h0)
        assert torch.equal(gb.recurrence(x, x)[1], torch.zeros((b, d), device="cuda"))


def test_pieces_equal_the_whole():
    """A sequence fed in pieces through `last` and h0 gives the whole's states."""
    x, f, i, h0, starts, _, _ = inputs(2, 777, 40, torch.float32, True, True, 8)
    whole, last = gb.recurrence(x, f, i, h0=h0, starts=starts)
    state, parts = h0, []
    for a, b in ((0, 1), (1, 130), (130, 500), (500, 777)):
        h, state = gb.recurrence(x[:, a:b], f[:, a:b], i[:, a:b], h0=state, starts=starts[:, a:b].contiguous())
        parts.append(h)
    want, wlast, bound, blast = ref.recurrence(x, f, i, h0, starts)
    ref.check(torch.cat(parts, 1), want, bound)
    ref.check(state, wlast, blast)


def test_results_do_not_vary():
    x, f, i, h0, starts, dh, dlast = inputs(1, 6000, 128, torch.bfloat16, True, True, 12)
    first = gb.recurrence(x, f, i, h0=h0, starts=starts)
    for _ in range(5):
        again = gb.recurrence(x, f, i, h0=h0, starts=starts)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_offsets_past_32_bits():
    """Rows more than 2^31 values from the first."""
    stride = (1 << 30) + 64
    buf = torch.zeros(3 * stride, dtype=torch.bfloat16, device="cuda")
    x = buf.as_strided((3, 2, 64), (stride, 64, 1))
    g = torch.Generator().manual_seed(3)
    x.copy_(rand(g, (3, 2, 64), torch.bfloat16))
    h, _ = gb.recurrence(x, x)
    want, _, bound, _ = ref.recurrence(x, x, None, None, None)
    ref.check(h, want, bound)


@pytest.mark.parametrize("gate", [False, True], ids=["tied", "gated"])
def test_gradient_against_differences(gate):
    """<grad, v> against a central difference of the forward kernel along v.  The step's
    truncation is what it is in 64 bits; the rest is the forward's rounding over the step."""
    b, t, d, eps = 2, 60, 24, 2.0 ** -5
    x, f, i, h0, starts, dh, dlast = inputs(b, t, d, torch.float32, gate, True, 21, fused=False)
    g = torch.Generator().manual_seed(22)
    vs = [rand(g, (b, t, d), torch.float32) if v is not None else None for v in (x, f, i)] + \
        [rand(g, (b, d), torch.float32)]
    h, _ = gb.recurrence(x, f, i, h0=h0, starts=starts)
    grads = gb.recurrence_backward(dh, x, f, h, i, h0=h0, starts=starts, dlast=dlast)

    def moved(k):
        return [None if p is None else p + k * v for p, v in zip((x, f, i, h0), vs)]

    def loss(h, last):
        return float((ref.wide(h) * ref.wide(dh)).sum() + (ref.wide(last) * ref.wide(dlast)).sum())

    def kernel(k):
        return loss(*gb.recurrence(*moved(k)[:3], h0=moved(k)[3], starts=starts))

    def exact(k):
        h, last, bound, blast = ref.recurrence(*moved(k), starts)
        return loss(h, last), float((bound * ref.wide(dh).abs()).sum() + (blast * ref.wide(dlast).abs()).sum())

    (up, e1), (down, e2) = exact(eps), exact(-eps)
    wants, bounds = ref.recurrence_grad(dh, x, f, ref.recurrence(x, f, i, h0, starts)[0], i, h0, starts, dlast)
    along = sum(float((ref.wide(q) * ref.wide(v)).sum()) for q, v in zip(grads, vs) if q is not None)
    along64 = sum(float((q * ref.wide(v)).sum()) for q, v in zip(wants, vs) if q is not None)
    slack = sum(float((e * ref.wide(v).abs()).sum()) for e, v in zip(bounds, vs) if e is not None)
    truncation = abs((up - down) / (2 * eps) - along64)
    # The gradient read h rounded to fp32; df's share of that is within 2 u of its magnitude
    # and covered by the bounds' 40 u.
    assert abs((kernel(eps) - kernel(-eps)) / (2 * eps) - along) <= truncation + (e1 + e2) / (2 * eps) + slack


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("gate", [False, True], ids=["tied", "gated"])
@pytest.mark.parametrize("b,d,pool", [(1, 1, 1), (3, 40, 7), (64, 256, 70), (5, 1001, 5)])
def test_step(b, d, pool, gate, dt):
    dtype, g = DT[dt], torch.Generator().manual_seed(b + d)
    k = 3 if gate else 2
    proj = rand(g, (b, k * d), dtype).clamp_(-8, 8)
    x, f, i = proj[:, :d], proj[:, d:2 * d], proj[:, 2 * d:] if gate else None
    state = rand(g, (pool, d), torch.float32)
    slots = torch.randperm(pool, generator=g)[:b].to(torch.int32)
    if b > 2:
        slots[1] = -1
    want = state.clone()
    h = gb.recurrence_step(x, f, state, i, slots=slots.cuda())
    for r in range(b):
        s = int(slots[r])
        if s < 0:
            assert torch.equal(h[r], torch.zeros_like(h[r]))
            continue
        hr, last, bound, blast = ref.recurrence(x[r][None, None], f[r][None, None],
                                                i[r][None, None] if gate else None, want[s][None], None)
        ref.check(h[r], hr[0, 0], bound[0, 0])
        ref.check(state[s], last[0], blast[0])
    untouched = [s for s in range(pool) if s not in slots.tolist()]
    assert torch.equal(state[untouched], want[untouched])
    assert gb.device_error() == gb.OK


def test_step_equals_the_sequence():
    """T steps of one token give the sequence's outputs within both bounds."""
    x, f, i, h0, _, _, _ = inputs(4, 30, 64, torch.float32, True, True, 31)
    want, wlast, bound, blast = ref.recurrence(x, f, i, h0, None)
    state = h0.clone()
    hs = torch.stack([gb.recurrence_step(x[:, k], f[:, k], state, i[:, k]) for k in range(30)], 1)
    ref.check(hs, want, bound)
    ref.check(state, wlast, blast)


def test_step_slot_past_the_pool_is_reported():
    x = torch.ones((2, 16), device="cuda")
    state = torch.ones((3, 16), device="cuda")
    before = state.clone()
    slots = torch.tensor([3, -1], dtype=torch.int32, device="cuda")
    h = gb.recurrence_step(x, x, state, slots=slots)
    assert gb.device_error() == gb.ERR_RANGE and gb.device_error() == gb.OK
    assert torch.equal(h, torch.zeros_like(h)) and torch.equal(state, before)


def test_another_stream():
    """Inputs made on a side stream, the call given that stream, results used there."""
    s = torch.cuda.Stream()
    x, f, i, h0, starts, dh, dlast = inputs(2, 500, 64, torch.bfloat16, True, True, 41)
    want = gb.recurrence(x, f, i, h0=h0, starts=starts)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        x2, f2, i2 = x.clone(), f.clone(), i.clone()
    h, last = gb.recurrence(x2, f2, i2, h0=h0, starts=starts, stream=s)
    del x2, f2, i2
    s.synchronize()
    assert torch.equal(h, want[0]) and torch.equal(last, want[1])


def test_capture_in_a_graph():
    x, f, i, h0, starts, dh, dlast = inputs(2, 300, 64, torch.bfloat16, True, True, 43)
    want = gb.recurrence(x, f, i, h0=h0, starts=starts)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        h, last = gb.recurrence(x, f, i, h0=h0, starts=starts)
    h.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(h, want[0]) and torch.equal(last, want[1])


def test_refusals():
    x = torch.zeros((2, 4, 8), device="cuda")
    state = torch.zeros((2, 8), device="cuda")
    for bad, err in [
        (lambda: gb.recurrence(x.double(), x.double()), TypeError),
        (lambda: gb.recurrence(x, x.half()), TypeError),
        (lambda: gb.recurrence(x[0], x[0]), ValueError),
        (lambda: gb.recurrence(x, x[:, :3]), ValueError),
        (lambda: gb.recurrence(x.transpose(1, 2), x.transpose(1, 2)), ValueError),
        (lambda: gb.recurrence(x, x, h0=state.double()), TypeError),
        (lambda: gb.recurrence(x, x, h0=state[:1]), ValueError),
        (lambda: gb.recurrence(x, x, starts=torch.zeros((2, 5), dtype=torch.uint8, device="cuda")), ValueError),
        (lambda: gb.recurrence(x, x, out=x[:1].expand(2, 4, 8)), ValueError),
        (lambda: gb.recurrence(x.cpu(), x.cpu()), ValueError),
        (lambda: gb.recurrence(x, x.cpu()), ValueError),
        (lambda: gb.recurrence_backward(x, x, x, x[:1]), ValueError),
        (lambda: gb.recurrence_step(x[:, 0], x[:, 0], state[:1]), ValueError),
        (lambda: gb.recurrence_step(x[:, 0], x[:, 0], state.half()), TypeError),
        (lambda: gb.recurrence_step(x[:, 0], x[:, 0], state, slots=torch.zeros(2, device="cuda").long()), TypeError),
    ]:
        with pytest.raises(err):
            bad()
