"""GPU: what layer norm takes and refuses beyond its operands' shapes and types."""
import pytest
import torch

import stream_compaction_decoupled_gb300 as gb

pytestmark = pytest.mark.gpu


def test_scratch_that_the_kernels_cannot_use_is_refused():
    x = torch.randn((50, 200), device="cuda")
    w = torch.ones(200, device="cuda")
    _, mean, rstd = gb.layer_norm(x, w)
    want = gb.layer_norm_backward(x, x, mean, rstd, w)
    nbytes = gb.load().gb_layer_norm_temp_bytes(50, 200)
    for temp in (torch.empty(nbytes, dtype=torch.uint8), torch.empty(nbytes, dtype=torch.uint8).pin_memory(),
                 torch.empty(2 * nbytes, dtype=torch.uint8, device="cuda")[::2]):
        with pytest.raises(ValueError):
            gb.layer_norm_backward(x, x, mean, rstd, w, temp=temp)
    with pytest.raises(gb.GbError):  # not 256-byte aligned
        gb.layer_norm_backward(x, x, mean, rstd, w, temp=torch.empty(nbytes + 1, dtype=torch.uint8, device="cuda")[1:])
    temp = torch.empty(nbytes // 4, device="cuda")  # of any type
    assert all(torch.equal(p, q) for p, q in zip(want, gb.layer_norm_backward(x, x, mean, rstd, w, temp=temp)))
