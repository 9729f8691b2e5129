"""GPU: in fp32 the gradient's small probabilities keep their relative accuracy."""
import pytest
import torch

import lm_reference as ref
import stream_compaction_decoupled_gb300 as gb

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("pad", [0, 1], ids=["whole_packs", "values"])
def test_tails(pad):
    """With lse = 0 the log probabilities are the logits themselves, exactly, and dlogits =
    -exp(logit): the exponential's two units in the last place, a product's half, the output's."""
    v = 40000
    g = torch.Generator().manual_seed(1)
    logits = (-80.0 * torch.rand((3, v), generator=g)).cuda()
    targets = torch.full((3,), -1, device="cuda")
    zero, one = torch.zeros(3, device="cuda"), torch.ones(3, device="cuda")
    out = torch.empty((3, v + 4), device="cuda")[:, pad:v + pad]
    gb.token_logprobs_backward(logits, targets, zero, zero, None, one, out=out)
    x = ref.wide(logits)
    want = -x.exp() * x  # -p (log p + 0)
    assert ((ref.wide(out) - want).abs() <= 8 * ref.U * want.abs()).all()
    gb.token_logprobs_backward(logits, targets.zero_(), zero, zero, one, None, out=out)
    want = -x.exp()
    want[:, 0] += 1
    assert ((ref.wide(out) - want).abs()[:, 1:] <= 6 * ref.U * want.abs()[:, 1:]).all()
