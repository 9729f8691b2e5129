"""GPU: the gradient of token log probabilities where logits, or the entropy's weight, are so
large that a product with a difference of logits overflows: what has no probability gets 0."""
import pytest
import torch

import lm_reference as ref
import stream_compaction_decoupled_gb300 as gb

pytestmark = pytest.mark.gpu

DT = {"fp32": torch.float32, "bf16": torch.bfloat16}


@pytest.mark.parametrize("weight", [5.0, 1e20, -1e30])
@pytest.mark.parametrize("top", [1e19, 1e38, 3e38])
@pytest.mark.parametrize("dt", list(DT))
def test_logits_near_the_top_of_the_range(dt, top, weight):
    g = torch.Generator().manual_seed(1)
    logits = torch.randn((4, 3000), generator=g).to(DT[dt]).cuda()
    logits[0, 7] = top
    logits[1, :] = -top
    logits[1, 5] = top
    logits[2, 5:9] = top
    logits[2, 100:] = float("-inf")
    targets = torch.tensor([7, 9, 5, 0], device="cuda")
    got = gb.token_logprobs(logits, targets)
    w, h = torch.ones(4, device="cuda"), torch.full((4,), weight, device="cuda")
    for a, b in ((w, h), (None, h), (w, None)):
        d = gb.token_logprobs_backward(logits, targets, got.lse, got.entropy, a, b)
        want, _ = ref.token_logprobs_grad(logits, targets, a, b)
        assert torch.isfinite(d).all()
        # Without a probability of its own a logit has no gradient but the target's.
        p = ref.token_logprobs(logits, targets, 0)[5]
        gone = p == 0
        assert torch.equal(ref.wide(d)[gone], want[gone].to(DT[dt]).double())


@pytest.mark.parametrize("weight", [3e18, 1e25])
@pytest.mark.parametrize("dt", list(DT))
def test_a_large_weight_and_masked_logits(dt, weight):
    g = torch.Generator().manual_seed(2)
    logits = torch.randn((2, 500), generator=g).to(DT[dt]).cuda()
    logits[:, 300:] = float("-inf")
    logits[1, :200] = torch.finfo(DT[dt]).min
    targets = torch.tensor([3, -1], device="cuda")
    got = gb.token_logprobs(logits, targets)
    h = torch.full((2,), weight, device="cuda")
    d = gb.token_logprobs_backward(logits, targets, got.lse, got.entropy, None, h)
    want, bound = ref.token_logprobs_grad(logits, targets, None, h)
    _, ent, _, _, _, p, lp = ref.token_logprobs(logits, targets, 0)
    # The entropy and lse enter as computed: their sums have 62 roundings along a path at most.
    lim = torch.where(p > 0, lp.abs(), torch.zeros_like(lp)) + ent[:, None] + 2
    ref.check(d, want, bound + weight * p * lim * ref.U * 62 * 4, "dlogits")
    assert torch.equal(d[:, 300:], torch.zeros_like(d[:, 300:]))
