"""GPU: what decays and sums over many tokens may be off by on average, in fp32: limits that a decay
which is always low, or a sum over all tokens in one chain, would not keep.

u = 2^-24.  Decays.  The base-2 exponential of an argument of -0.003 to -0.03 is low by 0.3 to 0.45 u
on average where its argument is taken as it is, and off by 0.1 u at most with 2^-25 added to it.  A
state's share of an input of age k is a product of k decays, so the mean of all states' relative errors
is about 0.37 u or 0.1 u times their mean age; the limit is 0.2 u.  (Roundings to nearest are off to
both sides: over 4096 states and more their mean is below 0.1 u.)

Sums.  Adding n values of one sign one after another, the k-th addition's error is uniform within half
a unit of the last place of a sum of k values: relative to that sum 0.425 u (root mean square over
where the sum lies between two powers of two).  All of them: 0.425 u sqrt(n / 3) of the whole.
  d's gradient: each of 4 lanes adds a quarter of the tokens, then the lanes are added.  2048 tokens
  in chains of 512: 5.6 u / sqrt(4) = 2.8 u.  In chains of 16 and then 32: 1.0 u / sqrt(32) and 1.4 u,
  1.4 u / sqrt(4) = 0.7 u; with the last additions and the product's rounding 0.9 u.  The limit is 1.7 u.
  a's gradient: a chain of 2048 would be off by 11.1 u; chains of 64 and then 32 by 2.0 u / sqrt(32)
  and 1.4 u.  Decays of e^-1 to e^-4 make the terms themselves off by a few units, of which the
  mean (1 u or so for each of the two decays that matter) stays: below 3 u.  The limit is 5.5 u.
"""
import pytest
import torch

import stream_compaction_decoupled_gb300 as gb
from lm_reference import U

pytestmark = pytest.mark.gpu


def some(seed, shape, lo, hi):
    g = torch.Generator("cuda").manual_seed(seed)
    return torch.empty(shape, device="cuda").uniform_(lo, hi, generator=g)


def relative(got, want):
    return (got.double() - want) / want


@pytest.mark.parametrize("n", [16, 13, 32])
def test_decays_are_not_low_on_average(n):
    """112 tokens: one part, whatever the rest."""
    t, d = 112, 512
    x, dt = some(1, (1, t, d), 0.5, 1.5), some(2, (1, t, d), 0.5, 1.5)
    a, b, c = -some(3, (d, n), 0.006, 0.02), some(4, (1, t, n), 0.5, 1.5), some(5, (1, t, n), 0.5, 1.5)
    dy = some(6, (1, t, d), 0.5, 1.5)
    _, last, kept = gb.selective_scan(x, dt, a, b, c, softplus=False, keep=True)
    got = gb.selective_scan_backward(dy, x, dt, a, b, c, kept, softplus=False)
    x, dt, a, b, c, dy = (v.double() for v in (x, dt, a, b, c, dy))
    h = aged = torch.zeros((d, n), dtype=torch.float64, device="cuda")  # a state, and it by the age of its parts
    before, older = [], []
    for k in range(t):
        before.append(h), older.append(aged)
        decay = torch.exp(dt[0, k, :, None] * a)
        aged, h = decay * (aged + h), decay * h + (dt[0, k] * x[0, k])[:, None] * b[0, k]
    assert abs(float(relative(last[0], h).mean())) < 0.2 * U * float((aged / h).mean())
    g = aging = torch.zeros_like(h)
    da = age = torch.zeros_like(h)
    for k in range(t - 1, -1, -1):
        g = g + dy[0, k][:, None] * c[0, k]
        decay = torch.exp(dt[0, k, :, None] * a)
        g, aging = decay * g, decay * (aging + g)
        da = da + g * before[k] * dt[0, k, :, None]
        age = age + (g * older[k] + aging * before[k]) * dt[0, k, :, None]
    assert abs(float(relative(got.da, da).mean())) < 0.2 * U * float((age / da).mean())


def test_sums_over_tokens_are_not_one_chain():
    """More blocks of channels than fill the device twice: rows of one part."""
    t, d = 2048, 64 * 640
    x, dt = some(1, (1, t, d), 0.5, 1.5), some(2, (1, t, d), 0.8, 1.25)
    a, b, c = -some(3, (d, 1), 1.25, 3.2), some(4, (1, t, 1), 0.5, 1.5), some(5, (1, t, 1), 0.5, 1.5)
    skip, dy = some(6, (d,), 0.5, 1.5), some(7, (1, t, d), 0.5, 1.5)
    kept = gb.selective_scan(x, dt, a, b, c, skip, softplus=False, keep=True)[2]
    got = gb.selective_scan_backward(dy, x, dt, a, b, c, kept, skip, softplus=False)
    dd = torch.zeros(d, dtype=torch.float64, device="cuda")
    h, before = dd, []
    for k in range(t):
        before.append(h)
        dd = dd + dy[0, k].double() * x[0, k].double()
        h = torch.exp(dt[0, k].double() * a[:, 0].double()) * h + dt[0, k].double() * x[0, k].double() * b[0, k].double()
    assert float(relative(got.dd, dd).square().mean().sqrt()) < 1.7 * U
    g = da = torch.zeros_like(dd)
    for k in range(t - 1, -1, -1):
        g = torch.exp(dt[0, k].double() * a[:, 0].double()) * (g + dy[0, k].double() * c[0, k].double())
        da = da + g * before[k] * dt[0, k].double()
    assert float(relative(got.da[:, 0], da).square().mean().sqrt()) < 5.5 * U
