"""GPU: layer norm and its gradient against the definition in 64 bits (lm_reference.py),
with tolerances from the number of roundings along a sum, and against differences."""
import pytest
import torch

import lm_reference as ref
import stream_compaction_decoupled_gb300 as gb

pytestmark = pytest.mark.gpu

DT = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
# Roundings along a row's sum: at most 32 values of a thread, 5 steps of a warp, 16 warps;
# past the registers' reach a thread adds up to cols / 512 values.
DEPTH = 80


def rand(g, shape, dtype, mean=0.0, std=1.0):
    return (torch.randn(shape, generator=g) * std + mean).to(dtype).cuda()


def case(n, d, dtype, wdtype, seed, offset=0, pad=0):
    g = torch.Generator().manual_seed(seed)
    buf = torch.zeros(n * (d + pad) + offset, dtype=dtype, device="cuda")
    x = buf[offset:].view(n, d + pad)[:, :d]
    x.copy_(rand(g, (n, d), dtype, 0.7, 1.5))
    w = None if wdtype is None else rand(g, (d,), wdtype, 1.0, 0.3)
    b = None if wdtype is None else rand(g, (d,), wdtype, 0.0, 0.3)
    return x, w, b, rand(g, (n, d), dtype)


def run(n, d, dtype, wdtype, seed, eps=1e-5, **kw):
    x, w, b, dy = case(n, d, dtype, wdtype, seed, **kw)
    depth = DEPTH + d // 512
    y, mean, rstd = gb.layer_norm(x, w, b, eps=eps)
    wy, wm, wr, by, bm, br = ref.layer_norm(x, w, b, eps, depth)
    ref.check(mean, wm, bm, "mean")
    ref.check(rstd, wr, br, "rstd")
    ref.check(y, wy, by, "y")
    dx, dw, db = gb.layer_norm_backward(dy, x, mean, rstd, w)
    wants, bounds = ref.layer_norm_grad(dy, x, mean, rstd, w, n, depth)
    ref.check(dx, wants[0], bounds[0], "dx")
    if w is None:
        assert dw is None and db is None
    else:
        assert dw.dtype == db.dtype == w.dtype
        ref.check(dw, wants[1], bounds[1], "dw")
        ref.check(db, wants[2], bounds[2], "db")


SIZES = [(1, 1), (3, 2), (1, 7), (5, 33), (9, 64), (17, 255), (40, 512), (700, 96), (33, 1000), (12, 1025), (7, 2048),
         (300, 2047), (5, 4096), (11, 4099), (6, 8192), (3, 8200), (4, 16384), (3, 16385), (2, 33000)]


@pytest.mark.parametrize("wdt", ["none", "same", "fp32"])
@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_layer_norm(size, dt, wdt):
    run(*size, DT[dt], {"none": None, "same": DT[dt], "fp32": torch.float32}[wdt], sum(size))


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("offset,pad", [(0, 8), (1, 0), (1, 8), (3, 5), (8, 1), (2, 3)])
def test_alignments_and_strides(dt, offset, pad):
    """Rows at every offset from a 16-byte boundary, the same for x and y or not."""
    run(37, 250, DT[dt], DT[dt], offset + pad, offset=offset, pad=pad)


@pytest.mark.parametrize("dt", list(DT))
def test_many_rows(dt):
    run(5000, 136, DT[dt], DT[dt], 3)
    run(2600, 1021, DT[dt], DT[dt], 4)


def test_leading_dimensions_and_last_token_rows():
    g = torch.Generator().manual_seed(5)
    x = rand(g, (3, 20, 64), torch.bfloat16)
    y, mean, rstd = gb.layer_norm(x)
    y2, _, _ = gb.layer_norm(x.view(60, 64))
    assert y.shape == x.shape and torch.equal(y.view(60, 64), y2) and mean.shape == (60,)
    y3, _, _ = gb.layer_norm(x[:, -1])
    assert torch.equal(y3, y[:, -1])
    out = torch.empty_like(x)
    assert gb.layer_norm(x, out=out)[0] is out and torch.equal(out, y)


def test_constant_rows_and_large_means():
    """A constant row has variance 0: y = b, and rstd = 1 / sqrt(eps).  A mean far above the
    deviations does not swallow them."""
    x = torch.full((4, 300), 3.25, device="cuda")
    w, b = torch.full((300,), 2.0, device="cuda"), torch.linspace(-1, 1, 300, device="cuda")
    y, mean, rstd = gb.layer_norm(x, w, b)
    assert torch.equal(mean, x[:, 0]) and torch.equal(y, b.expand(4, 300))
    assert (rstd - 1e-5 ** -0.5).abs().max() < 1e-4 * 1e-5 ** -0.5
    g = torch.Generator().manual_seed(6)
    x = (1000.0 + torch.randn((8, 1000), generator=g)).cuda()
    y, mean, rstd = gb.layer_norm(x)
    wy, wm, wr, by, bm, br = ref.layer_norm(x, None, None, 1e-5, DEPTH)
    ref.check(y, wy, by)


def test_nan_and_infinity_stay_in_their_row():
    g = torch.Generator().manual_seed(7)
    x = rand(g, (6, 513), torch.float32)
    clean, _, _ = gb.layer_norm(x)
    x[2, 100], x[4, 3] = float("nan"), float("inf")
    y, _, _ = gb.layer_norm(x)
    assert torch.isnan(y[2]).all() and not torch.isfinite(y[4]).any()
    assert torch.equal(y[[0, 1, 3, 5]], clean[[0, 1, 3, 5]])


def test_empty():
    x = torch.zeros((0, 16), device="cuda", dtype=torch.bfloat16)
    w = torch.ones(16, device="cuda", dtype=torch.bfloat16)
    y, mean, rstd = gb.layer_norm(x, w, w)
    assert y.shape == (0, 16) and mean.shape == (0,)
    dx, dw, db = gb.layer_norm_backward(x, x, mean, rstd, w)
    assert dx.shape == (0, 16) and torch.equal(dw, torch.zeros_like(w)) and torch.equal(db, torch.zeros_like(w))


def test_results_do_not_vary():
    x, w, b, dy = case(3000, 1024, torch.bfloat16, torch.bfloat16, 8)
    y, mean, rstd = gb.layer_norm(x, w, b)
    first = gb.layer_norm_backward(dy, x, mean, rstd, w)
    for _ in range(4):
        assert all(torch.equal(p, q) for p, q in zip(first, gb.layer_norm_backward(dy, x, mean, rstd, w)))


def test_scratch_of_the_caller_and_none():
    x, w, b, dy = case(50, 200, torch.float32, torch.float32, 9)
    y, mean, rstd = gb.layer_norm(x, w, b)
    want = gb.layer_norm_backward(dy, x, mean, rstd, w)
    nbytes = gb.load().gb_layer_norm_temp_bytes(50, 200)
    temp = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
    got = gb.layer_norm_backward(dy, x, mean, rstd, w, temp=temp)
    assert all(torch.equal(p, q) for p, q in zip(want, got))
    with pytest.raises(gb.GbError):
        gb.layer_norm_backward(dy, x, mean, rstd, w, temp=temp[:256])
    dw, dx = torch.empty_like(w), torch.empty_like(x)
    rc = gb.load().gb_layer_norm_backward(gb.F32, gb.F32, 50, 200, dy.data_ptr(), 200, x.data_ptr(), 200,
                                          mean.data_ptr(), rstd.data_ptr(), w.data_ptr(), dx.data_ptr(), 200,
                                          dw.data_ptr(), None, None, 0, torch.cuda.current_stream().cuda_stream)
    assert rc == gb.OK and torch.equal(dw, want[1]) and torch.equal(dx, want[0])


def test_another_stream():
    s = torch.cuda.Stream()
    x, w, b, dy = case(900, 512, torch.bfloat16, torch.bfloat16, 10)
    y, mean, rstd = gb.layer_norm(x, w, b)
    want = gb.layer_norm_backward(dy, x, mean, rstd, w)
    torch.cuda.synchronize()
    y2, mean2, rstd2 = gb.layer_norm(x, w, b, stream=s)
    got = gb.layer_norm_backward(dy, x, mean2, rstd2, w, stream=s)
    s.synchronize()
    assert torch.equal(y, y2) and all(torch.equal(p, q) for p, q in zip(want, got))


def test_gradient_against_differences():
    """<grad, v> against a central difference of the forward kernel along v: the truncation
    as it is in 64 bits, and the forward's rounding bound over the step."""
    n, d, eps = 6, 200, 2.0 ** -5
    x, w, b, dy = case(n, d, torch.float32, torch.float32, 11)
    g = torch.Generator().manual_seed(12)
    vs = [rand(g, (n, d), torch.float32), rand(g, (d,), torch.float32), rand(g, (d,), torch.float32)]
    _, mean, rstd = gb.layer_norm(x, w, b)
    grads = gb.layer_norm_backward(dy, x, mean, rstd, w)

    def moved(k):
        return [p + k * v for p, v in zip((x, w, b), vs)]

    def kernel(k):
        return float((ref.wide(gb.layer_norm(*moved(k))[0]) * ref.wide(dy)).sum())

    def exact(k):
        y, _, _, bound, _, _ = ref.layer_norm(*moved(k), 1e-5, DEPTH)
        return float((y * ref.wide(dy)).sum()), float((bound * ref.wide(dy).abs()).sum())

    (up, e1), (down, e2) = exact(eps), exact(-eps)
    wants, bounds = ref.layer_norm_grad(dy, x, mean, rstd, w, n, DEPTH)
    along = sum(float((ref.wide(q) * ref.wide(v)).sum()) for q, v in zip(grads, vs))
    along64 = sum(float((q * ref.wide(v)).sum()) for q, v in zip(wants, vs))
    slack = sum(float((e * ref.wide(v).abs()).sum()) for e, v in zip(bounds, vs))
    truncation = abs((up - down) / (2 * eps) - along64)
    assert abs((kernel(eps) - kernel(-eps)) / (2 * eps) - along) <= truncation + (e1 + e2) / (2 * eps) + slack


def test_refusals():
    x = torch.zeros((4, 8), device="cuda", dtype=torch.bfloat16)
    w = torch.zeros(8, device="cuda", dtype=torch.bfloat16)
    m = torch.zeros(4, device="cuda")
    for bad, err in [
        (lambda: gb.layer_norm(x.double()), TypeError),
        (lambda: gb.layer_norm(x, w.half()), TypeError),
        (lambda: gb.layer_norm(x, w, w.float()), TypeError),
        (lambda: gb.layer_norm(x, w[:4]), ValueError),
        (lambda: gb.layer_norm(x.t()), ValueError),
        (lambda: gb.layer_norm(x.cpu()), ValueError),
        (lambda: gb.layer_norm(x, w.cpu()), ValueError),
        (lambda: gb.layer_norm(x, eps=-1.0), gb.GbError),
        (lambda: gb.layer_norm(x, eps=float("nan")), gb.GbError),
        (lambda: gb.layer_norm(torch.zeros((4, 0), device="cuda")), ValueError),
        (lambda: gb.layer_norm(x, out=x[:1].expand(4, 8)), ValueError),
        (lambda: gb.layer_norm_backward(x, x, m[:3], m, w), ValueError),
        (lambda: gb.layer_norm_backward(x[:3], x, m, m, w), ValueError),
        (lambda: gb.layer_norm_backward(x.float(), x, m, m, w), TypeError),
    ]:
        with pytest.raises(err):
            bad()
