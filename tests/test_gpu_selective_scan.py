"""GPU: the selective scan, its gradient and its single-token form against the definition in 64
bits, with tolerances from a first-order error analysis (ssm_reference.py)."""
import pytest
import torch

import lm_reference as lm
import ssm_reference as ref
import stream_compaction_decoupled_gb300 as gb
from stream_compaction_decoupled_gb300 import autograd

pytestmark = pytest.mark.gpu

DT = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
NAMES = "dx ddt da db dc dd dz ddt_bias dh0".split()


def rand(g, shape, dtype=torch.float32, std=1.0, mean=0.0):
    return (torch.randn(shape, generator=g) * std + mean).to(dtype).cuda()


def inputs(b, t, d, n, groups, dtype, extras, seed, pad=0, p_start=0.05):
    """A dict of arguments; x, dt, z and b, c are slices of rows `pad` values longer."""
    g = torch.Generator().manual_seed(seed)

    def rows(width):
        return rand(g, (b, t, width + pad), dtype)[..., pad:]

    q = {"x": rows(d), "dt": rows(d), "a": -torch.exp(rand(g, (d, n), std=0.5)),
         "b": rows(groups * n).unflatten(-1, (groups, n)), "c": rows(groups * n).unflatten(-1, (groups, n)),
         "d": rand(g, (d,), mean=1.0, std=0.2) if extras else None, "z": rows(d) if extras else None,
         "dt_bias": rand(g, (d,), mean=-2.0) if extras else None}
    more = {"h0": rand(g, (b, d, n)) if extras else None,
            "starts": (torch.rand((b, t), generator=g) < p_start).cuda() if extras else None}
    dy, dlast = rows(d), rand(g, (b, d, n)) if extras else None
    return q, more, dy, dlast


def check_forward(q, more, got, softplus=True):
    want, wlast, bound, blast = ref.scan(**q, **more, softplus=softplus)
    lm.check(got[0], want, bound, "y")
    lm.check(got[1], wlast, blast, "last")


def run(b, t, d, n, groups, dtype, extras, seed=1, softplus=True, **kw):
    q, more, dy, dlast = inputs(b, t, d, n, groups, dtype, extras, seed, **kw)
    if not softplus:
        q["dt"] = q["dt"].abs() * 0.1
        q["dt_bias"] = None
    y, last, kept = gb.selective_scan(**q, **more, softplus=softplus, keep=True)
    check_forward(q, more, (y, last), softplus)
    y2, last2, none = gb.selective_scan(**q, **more, softplus=softplus)
    assert none is None and torch.equal(y, y2) and torch.equal(last, last2)
    got = gb.selective_scan_backward(dy, **q, kept=kept, starts=more["starts"], dlast=dlast, softplus=softplus)
    wants, bounds = ref.scan_grad(dy, **q, **more, dlast=dlast, softplus=softplus)
    for name, v, w, e in zip(NAMES, got, wants, bounds):
        if w is None:
            assert v is None, name
        else:
            lm.check(v, w, e, name)


SIZES = [(1, 1, 1, 1, 1), (2, 1, 8, 16, 1), (1, 2, 33, 3, 1), (3, 16, 64, 16, 1), (2, 17, 72, 13, 2), (1, 129, 40, 8, 4),
         (2, 100, 130, 16, 1), (1, 33, 65, 16, 1), (2, 40, 12, 32, 1), (1, 50, 20, 61, 2), (1, 20, 6, 128, 1),
         (3, 35, 300, 5, 3)]


@pytest.mark.parametrize("extras", [False, True], ids=["plain", "all"])
@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_scan(size, dt, extras):
    run(*size, DT[dt], extras, seed=sum(size))


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("pad", [1, 2, 3, 4, 8])
def test_row_strides_of_every_alignment(dt, pad):
    run(2, 37, 64, 16, 2, DT[dt], True, seed=pad, pad=pad)


@pytest.mark.parametrize("t", [64, 200, 500, 1025])
def test_long_rows_in_parts(t):
    """Few channels and many tokens: the row is split into parts, which start from each other's
    ends; lengths that end in the first, a middle and the last token of a tile."""
    run(1, t, 48, 16, 1, torch.float32, True, seed=t, p_start=0.01)
    run(2, t, 7, 20, 1, torch.bfloat16, True, seed=t, p_start=0.0)


def test_steps_as_they_are():
    run(2, 50, 40, 16, 1, torch.float32, True, softplus=False)
    run(2, 50, 40, 16, 1, torch.bfloat16, False, softplus=False)


def test_positive_and_zero_rates():
    """exp(D a) above and at 1 (growing states, plain sums)."""
    q, more, _, _ = inputs(1, 20, 32, 16, 1, torch.float32, True, 3)
    q["a"] = q["a"] * torch.tensor([0.0, -0.5]).cuda().repeat(8)
    got = gb.selective_scan(**q, **more)
    check_forward(q, more, got)


def test_one_group_without_its_dimension_and_time_major_rows():
    q, more, dy, dlast = inputs(2, 40, 64, 16, 1, torch.bfloat16, True, 4)
    want = gb.selective_scan(**q, **more, keep=True)
    flat = {**q, "b": q["b"].squeeze(2), "c": q["c"].squeeze(2)}
    got = gb.selective_scan(**flat, **more)
    assert torch.equal(got[0], want[0])
    wg = gb.selective_scan_backward(dy, **q, kept=want[2], starts=more["starts"], dlast=dlast)
    gg = gb.selective_scan_backward(dy, **flat, kept=want[2], starts=more["starts"], dlast=dlast)
    assert gg.db.shape == flat["b"].shape and torch.equal(gg.db, wg.db.squeeze(2)) and torch.equal(gg.dc, wg.dc.squeeze(2))
    tm = {k: v.transpose(0, 1).contiguous().transpose(0, 1) if k in ("x", "dt", "z", "b", "c") else v for k, v in q.items()}
    got = gb.selective_scan(**tm, **more)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_a_broadcast_input():
    """b and c of one row for the whole batch (stride 0) are read in place."""
    q, more, _, _ = inputs(1, 30, 64, 16, 1, torch.float32, False, 5)
    wide = {k: (v.repeat(3, 1, 1) if k in ("x", "dt") else v.expand(3, -1, -1, -1) if k in ("b", "c") else v)
            for k, v in q.items()}
    one, many = gb.selective_scan(**q), gb.selective_scan(**wide)
    assert all(torch.equal(many[0][k], one[0][0]) for k in range(3))


@pytest.mark.parametrize("t", [30, 700])
def test_a_start_drops_infinities_and_nans(t):
    q, more, dy, _ = inputs(1, t, 64, 16, 1, torch.float32, True, 6, p_start=0.0)
    starts = torch.zeros((1, t), dtype=torch.uint8, device="cuda")
    at = [0, 13, t - 7]
    starts[0, at] = 1
    more["starts"] = starts
    more["h0"][:] = float("nan")
    q["x"][0, 12] = float("inf")
    q["x"][0, t - 8] = float("nan")
    y, last, kept = gb.selective_scan(**q, **more, keep=True)
    clean = q["x"].clone()
    clean[0, 12] = clean[0, t - 8] = 0.0
    want, wlast, bound, blast = ref.scan(**{**q, "x": clean}, **{**more, "h0": torch.zeros_like(more["h0"])})
    fine = [k for k in range(t) if k not in (12, t - 8)]
    lm.check(y[:, fine], want[:, fine], bound[:, fine], "y")
    lm.check(last, wlast, blast, "last")
    g = gb.selective_scan_backward(dy, **q, kept=kept, starts=starts)
    assert torch.isfinite(g.dx[:, fine]).all() and torch.isfinite(g.db[:, fine]).all() and not g.dh0.any()


@pytest.mark.parametrize("t", [1, 7, 21])
def test_an_infinity_in_the_last_token_stays_one(t):
    """Rows end inside a tile: what is behind the last token takes no part."""
    q, more, dy, _ = inputs(1, t, 24, 16, 1, torch.float32, True, 13, p_start=0.0)
    more["starts"] = None
    q["x"][0, t - 1] = float("inf")
    q["b"][0, t - 1] = 1.0
    _, last, _ = gb.selective_scan(**q, **more)
    assert torch.isinf(last).all()


def test_in_pieces_and_token_by_token():
    """A row in pieces and one token a call: the same as at once, up to the roundings that the
    bounds of both allow."""
    b, t, d, n = 3, 50, 40, 16
    q, more, _, _ = inputs(b, t, d, n, 2, torch.float32, True, 7, p_start=0.0)
    more["starts"] = None
    want, wlast, bound, blast = ref.scan(**q, **more)
    h, at, ys = more["h0"], 0, []
    for k in (1, 16, 33):
        part = {key: v[:, at:at + k] if key in ("x", "dt", "b", "c", "z") else v for key, v in q.items()}
        y, h, _ = gb.selective_scan(**part, h0=h)
        ys.append(y)
        at += k
    lm.check(torch.cat(ys, 1), want, bound, "y")
    lm.check(h, wlast, blast, "last")
    pool = torch.full((6, d, n), 7.0, device="cuda")
    slots = torch.tensor([4, 0, 2], dtype=torch.int32, device="cuda")
    pool[slots.long()] = more["h0"]
    for k in range(t):
        tok = {key: v[:, k] if key in ("x", "dt", "b", "c", "z") else v for key, v in q.items()}
        y = gb.selective_scan_step(state=pool, slots=slots, **tok)
        lm.check(y, want[:, k], bound[:, k], "step %d" % k)
    lm.check(pool[slots.long()], wlast, blast, "state")
    assert (pool[[1, 3, 5]] == 7.0).all()


@pytest.mark.parametrize("n", [1, 3, 4, 16, 30, 64, 128])
@pytest.mark.parametrize("d", [1, 6, 64, 130])
@pytest.mark.parametrize("dt", list(DT))
def test_step(dt, d, n):
    groups = 2 if d % 2 == 0 else 1
    q, _, _, _ = inputs(5, 1, d, n, groups, DT[dt], True, d + n, pad=1)
    tok = {k: v[:, 0] if k in ("x", "dt", "b", "c", "z") else v for k, v in q.items()}
    g = torch.Generator().manual_seed(n)
    pool = rand(g, (9, d, n))
    before = pool.clone()
    slots = torch.tensor([8, -1, 2, 0, -9], dtype=torch.int32, device="cuda")
    y = gb.selective_scan_step(state=pool, slots=slots, **tok)
    for r, s in enumerate(slots.tolist()):
        if s < 0:
            assert not y[r].any()
            continue
        one = {k: v[r:r + 1] if k in ("x", "dt", "b", "c", "z") else v for k, v in q.items()}
        want, last, bound, blast = ref.scan(**one, h0=before[s:s + 1], starts=None)
        lm.check(y[r].view(1, 1, d), want, bound, "y")
        lm.check(pool[s:s + 1], last, blast, "state")
    rest = [1, 3, 4, 5, 6, 7]
    assert torch.equal(pool[rest], before[rest])
    y = gb.selective_scan_step(state=pool[:4].contiguous(), slots=torch.tensor([0, 4, 1, 2, 3], dtype=torch.int32, device="cuda"),
                               **tok)
    assert not y[1].any() and gb.device_error() == gb.ERR_RANGE and gb.device_error() == gb.OK


def test_empty_rows():
    q, more, dy, dlast = inputs(2, 0, 24, 16, 1, torch.bfloat16, True, 8)
    y, last, kept = gb.selective_scan(**q, h0=more["h0"], keep=True)
    assert y.shape == (2, 0, 24) and torch.equal(last, more["h0"])
    g = gb.selective_scan_backward(dy, **q, kept=kept, dlast=dlast)
    assert torch.equal(g.dh0, dlast) and not g.da.any() and not g.dd.any() and not g.ddt_bias.any()
    q, more, dy, dlast = inputs(0, 5, 24, 16, 1, torch.bfloat16, True, 8)
    y, last, kept = gb.selective_scan(**q, keep=True)
    g = gb.selective_scan_backward(dy, **q, kept=kept)
    assert y.shape == (0, 5, 24) and not g.da.any()


def test_gradients_against_differences():
    """Each gradient against central differences of the forward kernel in fp32: a step of 2^-7 is
    off by the third derivative and the forward's roundings over the step, some 1e-4 of the scale."""
    q, more, dy, dlast = inputs(2, 21, 16, 5, 2, torch.float32, True, 11)
    q = {k: v.contiguous() for k, v in q.items()}
    keys = ["x", "dt", "a", "b", "c", "d", "z", "dt_bias", "h0"]

    def loss(v):
        y, last, _ = gb.selective_scan(**{k: v[k] for k in keys[:-1]}, h0=v["h0"], starts=more["starts"])
        return float((y.double() * dy.double()).sum() + (last.double() * dlast.double()).sum())

    base = {**q, "h0": more["h0"]}
    kept = gb.selective_scan(**q, **more, keep=True)[2]
    grads = gb.selective_scan_backward(dy, **q, kept=kept, starts=more["starts"], dlast=dlast)
    g = torch.Generator().manual_seed(0)
    for key, grad in zip(keys, (grads.dx, grads.ddt, grads.da, grads.db, grads.dc, grads.dd, grads.dz, grads.ddt_bias,
                                grads.dh0)):
        for _ in range(3):
            way = torch.randn(base[key].shape, generator=g).cuda()
            way /= way.norm()
            h = 2.0 ** -7
            slope = (loss({**base, key: base[key] + h * way}) - loss({**base, key: base[key] - h * way})) / (2 * h)
            assert abs(slope - float((grad.double() * way.double()).sum())) < 3e-3 * max(1.0, float(grad.norm())), key


@pytest.mark.parametrize("t", [50, 600])
def test_the_same_from_run_to_run_on_streams_and_in_graphs(t):
    q, more, dy, dlast = inputs(2, t, 96, 16, 1, torch.bfloat16, True, 9)

    def call(stream=None):
        y, last, kept = gb.selective_scan(**q, **more, keep=True, stream=stream)
        if stream is not None:
            stream.synchronize()
        return y, last, *gb.selective_scan_backward(dy, **q, kept=kept, starts=more["starts"], dlast=dlast, stream=stream)

    want = call()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = call(side)
    side.synchronize()
    assert all(torch.equal(p, w) for p, w in zip(got, want))
    graphs = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()]
    held = []
    for graph in graphs:
        with torch.cuda.graph(graph):
            held.append(call())
    for out in held:
        for v in out:
            v.zero_()
    for graph in graphs:
        graph.replay()
    torch.cuda.synchronize()
    for out in held:
        assert all(torch.equal(p, w) for p, w in zip(out, want))


def test_outputs_into_slices_and_refusals():
    q, more, dy, dlast = inputs(2, 30, 64, 16, 1, torch.bfloat16, True, 10)
    want = gb.selective_scan(**q, **more, keep=True)
    buf = torch.zeros((2, 30, 3 * 64 + 10), dtype=torch.bfloat16, device="cuda")
    gb.selective_scan(**q, **more, out=buf[..., 64:128])
    assert torch.equal(buf[..., 64:128], want[0]) and not buf[..., :64].any() and not buf[..., 128:].any()
    g = gb.selective_scan_backward(dy, **q, kept=want[2], starts=more["starts"])
    views = tuple(buf[..., k * 64:(k + 1) * 64] for k in range(3))
    s = gb.selective_scan_backward(dy, **q, kept=want[2], starts=more["starts"], out=views)
    assert all(torch.equal(p, w) for p, w in zip(s, g) if p is not None) and not buf[..., 192:].any()
    for bad in (dict(a=q["a"].to(torch.bfloat16)), dict(d=q["d"].half()), dict(b=q["b"].float()), dict(z=q["z"].float())):
        with pytest.raises(TypeError):
            gb.selective_scan(**{**q, **bad})
    for bad in (dict(a=q["a"][:, :8].contiguous()), dict(b=q["b"][..., :8]), dict(dt=q["dt"][:, :4]), dict(dt=q["dt"].cpu()),
                dict(a=torch.zeros((64, 129), device="cuda")), dict(a=q["a"][:, :0]),
                dict(b=q["b"].expand(-1, -1, 3, -1), c=q["c"].expand(-1, -1, 3, -1)), dict(h0=more["h0"][:1]),
                dict(x=q["x"][..., ::2]), dict(out=q["x"][:, :1].expand(-1, 30, -1))):
        with pytest.raises(ValueError):
            gb.selective_scan(**{**q, **bad})
    with pytest.raises(ValueError):
        gb.selective_scan_backward(dy, **q, kept=want[2][:, :1])
    with pytest.raises(gb.GbError):
        gb.selective_scan_backward(dy, **q, kept=want[2], temp=torch.empty(16, dtype=torch.uint8, device="cuda"))


def test_autograd():
    q, more, dy, dlast = inputs(2, 40, 32, 16, 2, torch.float32, True, 12)
    keys = ["x", "dt", "a", "b", "c", "d", "z", "dt_bias"]
    leaves = [q[k].clone().requires_grad_() for k in keys] + [more["h0"].clone().requires_grad_()]
    y, last = autograd.selective_scan(*leaves, more["starts"])
    got = torch.autograd.grad((y * dy).sum() + (last * dlast).sum(), leaves)
    kept = gb.selective_scan(**q, **more, keep=True)[2]
    g = gb.selective_scan_backward(dy.contiguous(), **q, kept=kept, starts=more["starts"], dlast=dlast)
    want = (g.dx, g.ddt, g.da, g.db, g.dc, g.dd, g.dz, g.ddt_bias, g.dh0)
    assert all(torch.equal(p, w) for p, w in zip(got, want))
    y, _ = autograd.selective_scan(*(v.detach() for v in leaves[:5]))  # nothing asks for a gradient
    assert not y.requires_grad
