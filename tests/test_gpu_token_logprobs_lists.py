"""GPU: rows whose candidate lists take several passes to expand: equal values, a masked
beginning of the row or of each block's slice, vocabularies barely above the number of
candidates a pass takes.  Each is run many times: the selection must not depend on which
warp comes first."""
import pytest
import torch

import lm_reference as ref
import stream_compaction_decoupled_gb300 as gb

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
NEG = float("-inf")


def same_every_time(logits, top, times=30):
    """The ids of the definition (equal values in rising order of index), every time."""
    targets = torch.zeros(logits.shape[0], dtype=torch.int64, device="cuda")
    want = torch.sort(logits.float(), dim=1, descending=True, stable=True).indices[:, :top].int()
    first = gb.token_logprobs(logits, targets, top=top)
    assert torch.equal(first.top_ids, want)
    for _ in range(times):
        got = gb.token_logprobs(logits, targets, top=top)
        assert torch.equal(got.top_ids, want)
        assert torch.equal(got.top_values, first.top_values) and torch.equal(got.lse, first.lse)
    # lse's sum has V / 256 + 60 roundings along a path at most, 572 for the longest row here.
    few = ref.token_logprobs(logits[:2], targets[:2], top)
    ref.check(first.top_values[:2], few[3], 600 * ref.U * (1 + few[2].abs()[:, None]).nan_to_num(0.0, 0.0), "top values")


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("top", [20, 32])
@pytest.mark.parametrize("rows,vocab", [(600, 4096), (600, 10000), (3, 50000), (40, 128000)])
def test_rows_of_equal_values(rows, vocab, top, dt):
    same_every_time(torch.zeros((rows, vocab), dtype=DT[dt], device="cuda"), top)


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("top", [20, 32])
@pytest.mark.parametrize("rows,vocab", [(600, 20000), (3, 131072)])
def test_only_late_ids_are_allowed(rows, vocab, top, dt):
    """The first tile of the row, and of every block's eighth of it, is masked throughout."""
    g = torch.Generator().manual_seed(rows + top)
    logits = torch.randn((rows, vocab), generator=g).to(DT[dt]).cuda()
    slices = 8 if rows < 38 else 1  # of a row that blocks share
    for k in range(slices):
        first = k * (vocab // slices)
        logits[:, max(0, first - 64):first + 8300] = NEG
    same_every_time(logits, top)
    logits[:, :vocab - 40] = NEG
    same_every_time(logits, top)


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("top", [20, 32])
@pytest.mark.parametrize("vocab", [513, 600, 777, 990, 1000, 1024])
def test_small_vocabularies(vocab, top, dt):
    g = torch.Generator().manual_seed(vocab)
    same_every_time(torch.randn((600, vocab), generator=g).to(DT[dt]).cuda(), top)


@pytest.mark.parametrize("dt", list(DT))
def test_values_that_rise_in_steps(dt):
    """The list overflows in the first tile and in later ones."""
    base = (torch.arange(40000) // 64 * 0.05).to(DT[dt]).cuda()
    same_every_time(base.repeat(304, 1), 32)
