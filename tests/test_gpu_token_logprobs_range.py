"""GPU: token log probabilities of confident rows, whose entropy is the small difference of
two sums, and of logits far from 0, whose log of a sum is lost beside the maximum."""
import pytest
import torch

import lm_reference as ref
import stream_compaction_decoupled_gb300 as gb

pytestmark = pytest.mark.gpu

DT = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
U = ref.U


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("vocab", [20000, 128000])
def test_entropy_of_confident_rows(vocab, dt):
    """One value 4 to 7 nats over another that its thread meets first, the rest far below.
    s = 1 + r: the largest term is exact in fp32 (off by 2 u in 16 bits, and 2 u more from its
    reference), 1 + r takes one rounding, t / s is a few roundings of the entropy's size."""
    dtype, rows = DT[dt], 96
    per = 2048 if dtype is not torch.float32 else 1024  # values between a thread's packs
    g = torch.Generator().manual_seed(vocab)
    logits = torch.full((rows, vocab), -20.0)
    high = 4.0 + 3.0 * torch.rand(rows, generator=g)
    at = torch.arange(rows) % (vocab // per - 1) + 1
    col = torch.randint(0, 64, (rows,), generator=g)
    k = torch.arange(rows)
    logits[k, col] = 2 * torch.rand(rows, generator=g) - 1
    logits[k, at * per + col] = logits[k, col] + high
    logits = logits.to(dtype).cuda()
    targets = (at * per + col).cuda()
    got = gb.token_logprobs(logits, targets)
    want = ref.token_logprobs(logits, targets, 0)
    assert (want[1] < 0.12).all() and (want[1] > 0.004).all()
    room = U * ((2 if dt == "fp32" else 7) + 24 * want[1])
    ref.check(got.entropy, want[1], room, "entropy")
    ref.check(got.logprob, want[0], room, "logprob")


@pytest.mark.parametrize("top", [0, 5])
@pytest.mark.parametrize("offset", [0.0, 100.0, -3000.0, 5e4, -9e5, 1e6, 3e6, -1e7, 1e9, -3e9, 1e12, 1e20, -1e30, 3e37])
@pytest.mark.parametrize("dt", ["fp32", "bf16"])
def test_logits_far_from_zero(dt, offset, top):
    n, v = 12, 3001
    g = torch.Generator().manual_seed(3)
    logits = (torch.randn((n, v), generator=g) * 3 * max(1.0, abs(offset) * 2.0 ** -7)).double() + offset
    logits = logits.to(DT[dt]).cuda()
    logits[::3, 1000:] = float("-inf")
    logits[1::3, 2000:] = -1e9 if abs(offset) < 1e8 else torch.finfo(DT[dt]).min
    targets = torch.randint(0, v, (n,), generator=g).cuda()
    got = gb.token_logprobs(logits, targets, top=top)
    want = ref.token_logprobs(logits, targets, top)
    assert torch.isfinite(got.lse).all() and (got.lse >= logits.float().max(1).values - 4 * U).all()
    # 72 roundings along a sum's path at most; differences, and their sum with the log, round once each.
    ref.check(got.lse, want[2], U * (80 + want[2].abs()), "lse")
    ref.check(got.logprob, want[0], U * (80 + 2 * want[0].abs().nan_to_num(0.0, 0.0, 0.0)), "logprob")
    ref.check(got.entropy, want[1], U * 96 * (3 + want[1]), "entropy")
    if top:
        assert torch.equal(got.top_ids.cpu().long(), want[4])
        ref.check(got.top_values, want[3], U * (80 + 2 * want[3].abs().nan_to_num(0.0, 0.0, 0.0)), "top values")


@pytest.mark.parametrize("dt", list(DT))
def test_masks_of_every_depth(dt):
    """Masked values that a thread meets before any other do not spoil its sums."""
    v = 30000
    g = torch.Generator().manual_seed(4)
    low = torch.finfo(DT[dt]).min
    depths = [d for d in (-50.0, -1e3, -6e4, -1e5, -1e6, -2e6, -1e9, -1e13, -1e30, low, float("-inf")) if d >= low]
    logits = torch.randn((len(depths), v), generator=g).to(DT[dt])
    for r, d in enumerate(depths):
        logits[r, :v - 700] = d
    logits = logits.cuda()
    targets = torch.full((len(depths),), v - 3, device="cuda")
    got = gb.token_logprobs(logits, targets, top=3)
    want = ref.token_logprobs(logits, targets, 3)
    assert torch.equal(got.top_ids.cpu().long(), want[4])
    ref.check(got.lse, want[2], U * (180 + want[2].abs()), "lse")
    ref.check(got.entropy, want[1], U * 180 * (3 + want[1]), "entropy")
