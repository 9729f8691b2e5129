"""GPU: the recurrence's waits between the blocks of a cluster end at the limit.  A block
that never sends one of its maps makes the others' waits run out; the call reports
GB_ERR_TIMEOUT, soon, and the next call is right.  No fault, trap or hang is involved: the
limit is a few milliseconds of the GPU's global timer."""
import time

import pytest
import torch

import stream_compaction_decoupled_gb300 as gb

pytestmark = pytest.mark.gpu

DT = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}


@pytest.fixture
def quiet():
    gb.device_error()
    yield
    gb.set_stalled_tile(-1)
    gb.set_wait_limit_ns(0)
    torch.cuda.synchronize()
    gb.device_error()


def calls(dtype, gate, channels, length, batch=1):
    g = torch.Generator().manual_seed(channels + length)
    x, f, i, dh = (torch.randn((batch, length, channels), generator=g).to(dtype).cuda() for _ in range(4))
    i = i if gate else None
    h, _ = gb.recurrence(x, f, i)
    return (lambda: gb.recurrence(x, f, i)), (lambda: gb.recurrence_backward(dh, x, f, h, i))


@pytest.mark.parametrize("tile", [0, 3, 21])
@pytest.mark.parametrize("channels", [64, 100, 57], ids=["even", "two_strips", "odd"])
@pytest.mark.parametrize("gate", [False, True], ids=["tied", "gated"])
@pytest.mark.parametrize("dt", list(DT))
def test_a_map_that_is_never_sent(quiet, dt, gate, channels, tile):
    length = 32 * 24 if dt == "fp32" else 64 * 24  # 24 tiles of a strip: three rounds of 8 blocks
    for call in calls(DT[dt], gate, channels, length):
        want = call()
        assert gb.device_error() == gb.OK
        gb.set_wait_limit_ns(3_000_000)
        gb.set_stalled_tile(tile)
        torch.cuda.synchronize()
        t0 = time.perf_counter()
        call()
        torch.cuda.synchronize()
        took = time.perf_counter() - t0
        assert gb.device_error() == gb.ERR_TIMEOUT and gb.device_error() == gb.OK
        # A thread waits out one limit at most; a peer that has had the map goes on for a round,
        # so a cluster's waits follow one another for two or three limits.
        assert took < 0.25
        gb.set_stalled_tile(-1)
        gb.set_wait_limit_ns(0)
        again = call()
        assert gb.device_error() == gb.OK
        assert all(torch.equal(p, q) for p, q in zip(want, again) if p is not None)


@pytest.mark.parametrize("dt", list(DT))
def test_many_clusters_stop_at_once(quiet, dt):
    for call in calls(DT[dt], True, 1024, 2048, 2):
        want = call()
        gb.set_wait_limit_ns(2_000_000)
        gb.set_stalled_tile(9)
        call()
        assert gb.device_error() == gb.ERR_TIMEOUT
        gb.set_stalled_tile(-1)
        gb.set_wait_limit_ns(0)
        assert all(torch.equal(p, q) for p, q in zip(want, call()) if p is not None)
        assert gb.device_error() == gb.OK


@pytest.mark.parametrize("limit", [1, 100, 1000, 10000])
def test_short_limits(quiet, limit):
    """Waits that may or may not run out, in any block and round."""
    for call in calls(torch.bfloat16, True, 200, 6000):
        want = call()
        for _ in range(20):
            gb.set_wait_limit_ns(limit)
            call()
            assert gb.device_error() in (gb.OK, gb.ERR_TIMEOUT)
        gb.set_wait_limit_ns(0)
        assert all(torch.equal(p, q) for p, q in zip(want, call()) if p is not None)
        assert gb.device_error() == gb.OK


def test_a_stalled_tile_does_not_concern_a_block_alone(quiet):
    """One tile a strip: no cluster, no wait."""
    for call in calls(torch.float32, False, 64, 20):
        want = call()
        gb.set_stalled_tile(0)
        assert all(torch.equal(p, q) for p, q in zip(want, call()) if p is not None)
        assert gb.device_error() == gb.OK
