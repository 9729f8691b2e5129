"""GPU: what the convolution's sums over tokens may be off by on average, in fp32.

u = 2^-24.  Adding n values of one sign one after another leaves 0.425 u sqrt(n / 3) of the whole (root
mean square: the k-th addition is off by up to half a unit of the last place of a sum of k values).
8 x 2048 tokens go in some 72 to 112 runs of 152 to 232 tokens, 3.7 u / sqrt(72) = 0.4 u at most; the runs'
sums to 16 warps in chains of 5 to 7, 0.65 u / sqrt(16), and those in a chain of 16, 1.0 u: 1.1 u in all.
The limit is 2 u; one chain of all tokens would be off by 31 u.
"""
import pytest
import torch

import stream_compaction_decoupled_gb300 as gb
from lm_reference import U

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [2048, 2047])
def test_sums_over_tokens_are_not_one_chain(d):
    g = torch.Generator("cuda").manual_seed(d)
    x, dy = (torch.empty((8, 2048, d), device="cuda").uniform_(0.5, 1.5, generator=g) for _ in range(2))
    w, bias = torch.ones((d, 4), device="cuda"), torch.ones((d,), device="cuda")
    _, dw, db, _ = gb.causal_conv_backward(dy, x, w, bias, silu=False)
    assert float((db.double() / dy.double().sum((0, 1)) - 1).square().mean().sqrt()) < 2 * U
    for tap in range(4):
        back = 3 - tap
        want = (dy[:, back:].double() * x[:, :2048 - back].double()).sum((0, 1))
        assert float((dw[:, tap].double() / want - 1).square().mean().sqrt()) < 2 * U
