"""GPU: the recurrence's gates alone.  With one token and x or the state 1 its output is the
gate itself, sigmoid(f), sigmoid(i) or 1 - sigmoid(f), accurate where it is small too."""
import pytest
import torch

import lm_reference as ref
import stream_compaction_decoupled_gb300 as gb

pytestmark = pytest.mark.gpu

U = ref.U
DT = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}


def units(dt, z):
    """fp32: the exponential's 4 units, 1 of 1 + e, 2 of the reciprocal, 1 of the product.  16
    bits: the instructions' 2.5 and 2, two roundings, and the exponent's, which is 0.72 units
    for each of its |z| log2(e), and log2(e)'s own 0.22 |z|."""
    return 8.0 if dt == "fp32" else 8 + 1.3 * z.abs()


@pytest.mark.parametrize("step", [False, True], ids=["sequence", "step"])
@pytest.mark.parametrize("channels", [20000, 20001])
@pytest.mark.parametrize("dt", list(DT))
def test_gates(dt, channels, step):
    g = torch.Generator().manual_seed(channels)
    z = (160 * torch.rand(channels, generator=g) - 80).to(DT[dt]).cuda()
    z[:3] = torch.tensor([0.0, 80.0, -80.0])
    one, zero = torch.ones_like(z), torch.zeros_like(z)
    ones, zeros = torch.ones((1, channels), device="cuda"), torch.zeros((1, channels), device="cuda")

    def last(x, f, i, h0):
        if step:
            state = h0.clone()
            gb.recurrence_step(x[None], f[None], state, None if i is None else i[None])
            return state[0]
        return gb.recurrence(x[None, None], f[None, None], None if i is None else i[None, None], h0=h0)[1][0]

    zw = ref.wide(z)
    a, c = torch.sigmoid(zw), torch.sigmoid(-zw)
    for what, got, want in (("a tied", last(zero, z, None, ones), a), ("a gated", last(zero, z, zero, ones), a),
                            ("1 - a", last(one, z, None, zeros), c), ("u", last(one, zero, z, zeros), a)):
        off = (ref.wide(got) - want).abs() / want
        assert (off <= U * units(dt, zw)).all(), "%s: %.1f units" % (what, float(off.max() / U))


@pytest.mark.parametrize("gate", [False, True], ids=["tied", "gated"])
@pytest.mark.parametrize("big", [float("inf"), 104.0, 200.0, 1e30])
def test_closed_gates_are_zero_in_fp32(big, gate):
    x, f = torch.full((1, 5, 64), 2.0, device="cuda"), torch.full((1, 5, 64), -big, device="cuda")
    h0 = torch.full((1, 64), 1e38, device="cuda")
    h, last = gb.recurrence(x, f, -f if gate else None, h0=h0)
    assert torch.equal(h, x) and torch.equal(last, x[:, 0])
    h, last = gb.recurrence(x, -f, f if gate else None, h0=h0)
    assert torch.equal(last, h0)


@pytest.mark.parametrize("dt", list(DT))
def test_nan_gates(dt):
    x = torch.ones((1, 3, 64), dtype=DT[dt], device="cuda")
    f = torch.zeros_like(x)
    f[0, 1, 5] = float("nan")
    for args in ((x, f, None), (x, f, x), (x, x, f)):
        h, _ = gb.recurrence(*args)
        nan = torch.zeros_like(h, dtype=torch.bool)
        nan[0, 1:, 5] = True
        assert torch.equal(torch.isnan(h), nan)
