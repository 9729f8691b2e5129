"""GPU: token log probabilities, entropy and top alternatives, and their gradient, against
the definition in 64 bits (lm_reference.py) and against differences.  Ids are compared
exactly, ties included."""
import pytest
import torch

import lm_reference as ref
import stream_compaction_decoupled_gb300 as gb

pytestmark = pytest.mark.gpu

DT = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
U = ref.U
NEG = float("-inf")


def bounds(logits, want, lp):
    """Bounds of 32-bit results: the sum of exponentials has at most V / 256 / 8 + 40
    roundings along any path (a thread's share of a row at one CTA a row is V / 256 values),
    each exponential is off by (4 + |d|) u relative with d = x - max <= 0, whose weight is
    at most e^-|d| |d| < 1; the entropy's sum carries a factor |d| more."""
    depth = logits.shape[1] / 256 + 60
    mean_d = want[1].abs() + 2  # sum p |x - max| = entropy - log s + ..., log s >= 0 bounded below
    fin = torch.where(torch.isfinite(want[2]), want[2].abs(), torch.zeros_like(want[2]))
    b_lse = U * (depth + 8 + 2 * fin)
    lim = torch.where(torch.isfinite(lp), lp.abs(), torch.zeros_like(lp))
    return b_lse, U * (depth + 16) * (1 + mean_d), b_lse, lim


def check(logits, targets, top):
    got = gb.token_logprobs(logits, targets, top=top)
    want = ref.token_logprobs(logits, targets, top)
    b_lp, b_ent, b_lse, _ = bounds(logits, want, want[6])
    ref.check(got.lse, want[2], b_lse, "lse")
    ref.check(got.logprob, want[0], b_lp, "logprob")
    ref.check(got.entropy, want[1], b_ent, "entropy")
    if top:
        assert got.top_ids.dtype == torch.int32 and torch.equal(got.top_ids.cpu().long(), want[4]), "top ids"
        ref.check(got.top_values, want[3], b_lse[:, None].expand_as(want[3]), "top values")
    else:
        assert got.top_values is None and got.top_ids is None
    return got


def check_grad(logits, targets, got, seed=0):
    n = logits.shape[0]
    g = torch.Generator().manual_seed(seed)
    dl, de = torch.randn(n, generator=g).cuda(), torch.randn(n, generator=g).cuda()
    for a, b in ((dl, de), (dl, None), (None, de)):
        d = gb.token_logprobs_backward(logits, targets, got.lse, got.entropy, a, b)
        want, bound = ref.token_logprobs_grad(logits, targets, a, b)
        # entropy and lse enter as computed: their own errors, twice, times the weights.
        depth = logits.shape[1] / 256 + 60
        bound = bound + (0 if a is None else ref.wide(a).abs()[:, None]) * ref.token_logprobs(logits, targets, 0)[5] \
            * U * depth * 2
        if b is not None:
            _, ent, _, _, _, p, lp = ref.token_logprobs(logits, targets, 0)
            lim = torch.where(p > 0, lp.abs(), torch.zeros_like(lp)) + ent[:, None] + 2
            bound = bound + ref.wide(b).abs()[:, None] * p * lim * U * depth * 4
        ref.check(d, want, bound, "dlogits")


def make(n, v, dtype, seed, std=3.0):
    g = torch.Generator().manual_seed(seed)
    logits = (torch.randn((n, v), generator=g) * std).to(dtype).cuda()
    return logits, torch.randint(0, v, (n,), generator=g).cuda()


SIZES = [(1, 1), (2, 3), (5, 31), (3, 64), (1, 1000), (4, 4097), (7, 8191), (2, 8192), (3, 20011), (1, 50021),
         (400, 1003), (2, 131072), (1, 200000)]


@pytest.mark.parametrize("top", [0, 1, 7, 20, 32])
@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_token_logprobs(size, dt, top):
    logits, targets = make(*size, DT[dt], sum(size))
    got = check(logits, targets, min(top, size[1]))
    if top == 7:
        check_grad(logits, targets, got)


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("offset,pad", [(0, 8), (1, 0), (3, 1), (7, 5), (2, 2)])
def test_alignments_and_strides(dt, offset, pad):
    n, v = 9, 5000
    src, targets = make(n, v, DT[dt], offset)
    buf = torch.full((n * (v + pad) + offset,), 1e4, dtype=DT[dt], device="cuda")  # neighbours that would win
    logits = buf[offset:].view(n, v + pad)[:, :v]
    logits.copy_(src)
    got = check(logits, targets.to(torch.int32), 20)
    check_grad(logits, targets, got)


@pytest.mark.parametrize("dt", list(DT))
def test_equal_values_take_the_lowest_ids(dt):
    n, v = 4, 40000
    logits = torch.zeros((n, v), dtype=DT[dt], device="cuda")
    logits[1, ::3] = 1.0
    logits[2, 5:] = -0.0
    logits[3, 17000:17010] = 2.0
    check(logits, torch.zeros(n, dtype=torch.int64, device="cuda"), 32)


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("v", [37, 5000, 100003])
def test_masked_rows(dt, v):
    """Rows with everything, almost everything and one half masked; masks of the type's
    lowest finite value; a masked target."""
    logits, targets = make(8, v, DT[dt], v)
    low = torch.finfo(DT[dt]).min
    logits[0] = NEG
    logits[1, 1:] = NEG
    logits[2, : v - 3] = NEG
    logits[3, v // 2:] = NEG
    logits[4] = low
    logits[5, : v - 5] = low
    targets[3] = v - 1
    targets[6] = -1
    targets[7] = -100
    got = check(logits, targets, 20)
    assert got.logprob[0] == NEG and got.entropy[0] == 0 and got.logprob[6] == 0 and got.logprob[7] == 0
    assert got.top_ids[0].tolist() == list(range(20))
    check_grad(logits, targets, got)
    d = gb.token_logprobs_backward(logits, targets, got.lse, got.entropy, torch.ones_like(got.lse), got.lse)
    assert torch.equal(d[0], torch.zeros_like(d[0]))


@pytest.mark.parametrize("order", ["rising", "falling", "blocks"])
@pytest.mark.parametrize("dt", list(DT))
def test_sorted_rows(order, dt):
    """Orders that fill the candidate buffer over and over (values that rise along the row)
    or never."""
    v = 60000
    base = torch.linspace(-20, 20, v)
    if order == "falling":
        base = base.flip(0)
    if order == "blocks":
        base = base.view(-1, 100).flip(1).reshape(-1)
    logits = base.to(DT[dt]).cuda().repeat(2, 1)
    check(logits, torch.tensor([0, v - 1], device="cuda"), 32)
    check(logits.repeat(200, 1), torch.zeros(400, dtype=torch.int64, device="cuda"), 32)


def test_confident_and_flat_rows():
    """Entropy near 0 and near log V, without cancellation."""
    v = 30000
    logits = torch.zeros((3, v), device="cuda")
    logits[0, 77] = 60.0
    logits[1, 77] = 20.0
    check(logits, torch.tensor([77, 77, 5], device="cuda"), 5)


def test_large_values():
    logits, targets = make(4, 3000, torch.float32, 3)
    logits[0] *= 1e30
    logits[1] = -1e38
    logits[1, 5] = 1e38
    logits[2] = 3e38
    got = check(logits, targets, 3)


def test_nan_and_infinity_stay_in_their_row():
    logits, targets = make(4, 9000, torch.float32, 4)
    clean = gb.token_logprobs(logits, targets, top=4)
    logits[1, 8000] = float("nan")
    logits[2, 10] = float("inf")
    got = gb.token_logprobs(logits, targets, top=4)
    for r in (1, 2):
        assert all(torch.isnan(q[r]).all() for q in (got.logprob, got.entropy, got.lse, got.top_values))
    assert got.top_ids[1, 0] == 8000 and got.top_ids[2, 0] == 10
    for q, c in zip(got, clean):
        assert torch.equal(q[[0, 3]], c[[0, 3]])


def test_targets_past_the_vocabulary_are_reported():
    logits, targets = make(3, 100, torch.float32, 5)
    targets[1] = 100
    got = gb.token_logprobs(logits, targets)
    assert gb.device_error() == gb.ERR_RANGE and gb.device_error() == gb.OK
    assert got.logprob[1] == 0
    d = gb.token_logprobs_backward(logits, targets, got.lse, dlogprob=torch.ones(3, device="cuda"))
    assert torch.equal(d[1], torch.zeros_like(d[1])) and gb.device_error() == gb.OK


def test_empty():
    for n, v in ((0, 10), (3, 0)):
        logits = torch.zeros((n, v), device="cuda", dtype=torch.bfloat16)
        targets = torch.full((n,), -1, device="cuda")
        got = gb.token_logprobs(logits, targets)
        assert got.lse.shape == (n,) and torch.equal(got.entropy, torch.zeros(n, device="cuda"))
        assert gb.token_logprobs_backward(logits, targets, got.lse, dlogprob=got.lse).shape == (n, v)


def test_gradient_in_place():
    logits, targets = make(5, 7001, torch.bfloat16, 6)
    got = gb.token_logprobs(logits, targets)
    w = torch.randn(5, device="cuda")
    want = gb.token_logprobs_backward(logits, targets, got.lse, got.entropy, w, w)
    out = gb.token_logprobs_backward(logits, targets, got.lse, got.entropy, w, w, out=logits)
    assert out is logits and torch.equal(out, want)


def test_gradient_into_rows_of_another_alignment():
    logits, targets = make(5, 701, torch.bfloat16, 7)
    got = gb.token_logprobs(logits, targets)
    w = torch.randn(5, device="cuda")
    want = gb.token_logprobs_backward(logits, targets, got.lse, got.entropy, w, w)
    out = torch.zeros((5, 704), dtype=logits.dtype, device="cuda")[:, 1:702]
    gb.token_logprobs_backward(logits, targets, got.lse, got.entropy, w, w, out=out)
    assert torch.equal(out, want)


def test_gradient_against_differences():
    """<grad, v> against a central difference of the forward kernel along v: the truncation
    as it is in 64 bits, and the forward's rounding bound over the step."""
    n, v, eps = 4, 600, 2.0 ** -4
    logits, targets = make(n, v, torch.float32, 8, std=2.0)
    g = torch.Generator().manual_seed(9)
    dirn = torch.randn((n, v), generator=g).cuda()
    dl, de = torch.randn(n, generator=g).cuda(), torch.randn(n, generator=g).cuda()
    got = gb.token_logprobs(logits, targets)
    grad = gb.token_logprobs_backward(logits, targets, got.lse, got.entropy, dl, de)

    def loss(lp, ent):
        return float((ref.wide(lp) * ref.wide(dl) + ref.wide(ent) * ref.wide(de)).sum())

    def kernel(k):
        r = gb.token_logprobs(logits + k * dirn, targets)
        return loss(r.logprob, r.entropy)

    def exact(k):
        moved = logits + k * dirn
        w = ref.token_logprobs(moved, targets, 0)
        b_lp, b_ent, _, _ = bounds(moved, w, w[6])
        return loss(w[0], w[1]), float(((b_lp + U * w[0].abs()) * ref.wide(dl).abs() + b_ent * ref.wide(de).abs()).sum())

    (up, e1), (down, e2) = exact(eps), exact(-eps)
    want, bound = ref.token_logprobs_grad(logits, targets, dl, de)
    along, along64 = float((ref.wide(grad) * ref.wide(dirn)).sum()), float((want * ref.wide(dirn)).sum())
    truncation = abs((up - down) / (2 * eps) - along64)
    slack = float((bound * ref.wide(dirn).abs()).sum()) + 400 * U * float((want.abs() * ref.wide(dirn).abs()).sum())
    assert abs((kernel(eps) - kernel(-eps)) / (2 * eps) - along) <= truncation + (e1 + e2) / (2 * eps) + slack


def test_results_do_not_vary():
    logits, targets = make(3, 100000, torch.bfloat16, 10)
    first = gb.token_logprobs(logits, targets, top=20)
    for _ in range(5):
        assert all(torch.equal(p, q) for p, q in zip(first, gb.token_logprobs(logits, targets, top=20)))


def test_another_stream():
    s = torch.cuda.Stream()
    logits, targets = make(9, 40000, torch.bfloat16, 11)
    want = gb.token_logprobs(logits, targets, top=10)
    torch.cuda.synchronize()
    got = gb.token_logprobs(logits, targets, top=10, stream=s)
    s.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(want, got))


def test_refusals():
    x = torch.zeros((4, 100), device="cuda", dtype=torch.bfloat16)
    t = torch.zeros(4, device="cuda", dtype=torch.int64)
    lse = torch.zeros(4, device="cuda")
    for bad, err in [
        (lambda: gb.token_logprobs(x.double(), t), TypeError),
        (lambda: gb.token_logprobs(x, t.float()), TypeError),
        (lambda: gb.token_logprobs(x, t[:3]), ValueError),
        (lambda: gb.token_logprobs(x, t, top=33), ValueError),
        (lambda: gb.token_logprobs(x, t, top=-1), ValueError),
        (lambda: gb.token_logprobs(x[:, :5], t, top=6), ValueError),
        (lambda: gb.token_logprobs(x.t(), t), ValueError),
        (lambda: gb.token_logprobs(x.cpu(), t), ValueError),
        (lambda: gb.token_logprobs(x, t.cpu()), ValueError),
        (lambda: gb.token_logprobs_backward(x, t, lse, dentropy=lse), ValueError),
        (lambda: gb.token_logprobs_backward(x, t, lse[:2]), ValueError),
        (lambda: gb.token_logprobs_backward(x, t, lse.double()), TypeError),
        (lambda: gb.token_logprobs_backward(x, t, lse, out=x[:1].expand(4, 100)), ValueError),
    ]:
        with pytest.raises(err):
            bad()
