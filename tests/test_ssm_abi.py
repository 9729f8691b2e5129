"""CPU-only checks of the state space entry points: argument errors are reported before any CUDA
call, sizes of scratch, and the bounds that keep every launch in range."""
import ctypes

import pytest

import stream_compaction_decoupled_gb300 as gb
from stream_compaction_decoupled_gb300 import _build

P = ctypes.c_void_p(256)
ODD = ctypes.c_void_p(257)
HALF = ctypes.c_void_p(258)


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return gb.load()


def strides(*v):
    return (ctypes.c_int64 * len(v))(*v)


def conv(lib, dtype=gb.BF16, pdt=gb.BF16, b=2, t=4, d=8, taps=4, x=P, s=None, w=P, bias=P, silu=1, state=None, starts=None,
         y=P, last=P):
    return lib.gb_causal_conv(dtype, pdt, b, t, d, taps, x, s, w, bias, silu, state, starts, y, last, None)


def test_causal_conv(lib):
    assert conv(lib, b=-1) == conv(lib, t=-1) == conv(lib, d=-1) == conv(lib, taps=0) == conv(lib, silu=2) == gb.ERR_INVALID
    assert conv(lib, dtype=gb.F64) == conv(lib, pdt=gb.F16) == conv(lib, taps=9) == gb.ERR_UNSUPPORTED
    for k in ("x", "w", "y"):
        assert conv(lib, **{k: None}) == conv(lib, **{k: ODD}) == gb.ERR_INVALID
    assert conv(lib, bias=ODD) == conv(lib, state=ODD) == conv(lib, last=ODD) == conv(lib, pdt=gb.F32, w=HALF) == gb.ERR_INVALID
    assert conv(lib, s=strides(-1, 8, 32, 8)) == conv(lib, s=strides(1 << 60, 8, 32, 8)) == gb.ERR_INVALID
    assert conv(lib, d=(1 << 28) + 1) == conv(lib, t=(1 << 30) + 1) == conv(lib, b=1 << 40) == gb.ERR_RANGE
    assert conv(lib, b=0) == conv(lib, d=0) == conv(lib, t=0, last=None) == conv(lib, t=0, taps=1) == gb.OK


def test_causal_conv_backward(lib):
    def call(dtype=gb.F32, pdt=gb.F32, b=2, t=4, d=8, taps=4, dy=P, x=P, s=None, w=P, bias=None, dlast=None, dx=P, dw=P, db=P,
             dstate=None, temp=None, tb=0):
        return lib.gb_causal_conv_backward(dtype, pdt, b, t, d, taps, dy, x, s, w, bias, 1, None, None, dlast, dx, dw, db,
                                           dstate, temp, tb, None)
    assert call(dtype=gb.I32) == call(pdt=gb.BF16) == gb.ERR_UNSUPPORTED
    for k in ("dy", "x", "w", "dx"):
        assert call(**{k: None}) == call(**{k: HALF}) == gb.ERR_INVALID
    for k in ("dw", "db", "dlast", "dstate"):
        assert call(**{k: HALF}) == gb.ERR_INVALID
    assert call(s=strides(32, 8, 32, 8, -32, 8)) == gb.ERR_INVALID
    assert call(d=0) == gb.OK
    need = lib.gb_causal_conv_temp_bytes
    assert need(0, 4, 8, 4) == need(2, 4, 0, 4) == need(2, 4, 8, 0) == need(2, 4, 8, 9) == 0
    assert need(1, 0, 1, 1) > 0
    # A row of sums for each run of tokens, not for each of many short rows.
    assert need(1 << 20, 4, 4096, 4) < 1 << 26 and need(1, 1 << 20, 64, 4) < 1 << 22


def ssc(lib, dtype=gb.BF16, b=2, t=4, d=8, n=16, g=1, x=P, dt=P, a=P, bm=P, c=P, dd=None, z=None, bias=None, sp=1, s=None,
        h0=None, y=P, last=None, kept=None):
    return lib.gb_selective_scan(dtype, b, t, d, n, g, x, dt, a, bm, c, dd, z, bias, sp, s, h0, None, y, last, kept, None, 0,
                                 None)


def test_selective_scan(lib):
    for k in ("b", "t", "d"):
        assert ssc(lib, **{k: -1}) == gb.ERR_INVALID
    assert ssc(lib, n=0) == ssc(lib, g=0) == ssc(lib, g=3) == ssc(lib, sp=2) == gb.ERR_INVALID
    assert ssc(lib, dtype=gb.F64) == gb.ERR_UNSUPPORTED
    assert ssc(lib, n=129) == ssc(lib, d=(1 << 28) + 1) == ssc(lib, t=(1 << 30) + 1) == ssc(lib, b=1 << 33) == gb.ERR_RANGE
    for k in ("x", "dt", "a", "bm", "c", "y"):
        assert ssc(lib, **{k: None}) == ssc(lib, **{k: ODD}) == gb.ERR_INVALID
    for k in ("a", "dd", "bias", "h0", "last", "kept"):
        assert ssc(lib, **{k: HALF}) == gb.ERR_INVALID
    assert ssc(lib, z=ODD) == gb.ERR_INVALID
    good = [32, 8, 32, 8, 0, 0, 32, 8, 64, 16, 16, 64, 16, 16]
    for k in (0, 3, 7, 8, 10, 13):
        assert ssc(lib, s=strides(*good[:k], -1, *good[k + 1:])) == gb.ERR_INVALID
    assert ssc(lib, b=0) == ssc(lib, d=0) == ssc(lib, t=0) == gb.OK


def test_selective_scan_backward(lib):
    names = ("dy", "x", "dt", "a", "bm", "c", "kept", "dx", "ddt", "da", "db", "dc")

    def call(dtype=gb.F32, b=2, t=4, d=8, n=16, g=1, z=None, dz=None, s=None, dh0=None, **p):
        v = {k: p.get(k, P) for k in names}
        return lib.gb_selective_scan_backward(dtype, b, t, d, n, g, v["dy"], v["x"], v["dt"], v["a"], v["bm"], v["c"], None, z,
                                              None, 1, s, v["kept"], None, None, v["dx"], v["ddt"], v["da"], v["db"],
                                              v["dc"], None, dz, None, dh0, None, 0, None)
    assert call(dtype=gb.U32) == gb.ERR_UNSUPPORTED
    for k in names:
        assert call(**{k: None}) == call(**{k: HALF}) == gb.ERR_INVALID
    assert call(z=P) == call(dh0=HALF) == call(s=strides(*[8] * 25, -1)) == gb.ERR_INVALID
    assert call(d=0) == gb.OK
    need = lib.gb_selective_scan_temp_bytes
    assert need(0, 4, 8, 16, 1, 1) == need(2, 4, 8, 0, 1, 1) == need(2, 4, 8, 16, 3, 1) == need(2, 4, 8, 129, 1, 0) == 0
    assert need(64, 2048, 2048, 16, 1, 0) == 0 < need(1, 2048, 64, 16, 1, 0) < need(1, 2048, 64, 16, 1, 1)


def test_selective_scan_step(lib):
    def call(dtype=gb.F16, b=2, d=8, n=16, g=1, x=P, dt=P, a=P, bm=P, c=P, z=None, s=None, state=P, pool=2, slots=None, y=P):
        return lib.gb_selective_scan_step(dtype, b, d, n, g, x, dt, a, bm, c, None, z, None, 1, s, state, pool, slots, y, None)
    assert call(dtype=gb.I64) == gb.ERR_UNSUPPORTED
    assert call(pool=1) == call(pool=-1) == call(g=3) == call(n=0) == gb.ERR_INVALID
    for k in ("x", "dt", "a", "bm", "c", "state", "y"):
        assert call(**{k: None}) == call(**{k: ODD}) == gb.ERR_INVALID
    assert call(state=HALF) == call(slots=HALF) == call(z=ODD) == call(s=strides(8, 8, 8, -8, 16, 16, 16, 16)) == gb.ERR_INVALID
    assert call(n=129) == gb.ERR_RANGE
    assert call(b=0, pool=0) == call(d=0) == gb.OK


def test_causal_conv_step(lib):
    def call(dtype=gb.F16, pdt=gb.F16, b=2, d=8, taps=4, x=P, s=None, w=P, state=P, pool=2, slots=None, y=P):
        return lib.gb_causal_conv_step(dtype, pdt, b, d, taps, x, s, w, None, 1, state, pool, slots, y, None)
    assert call(dtype=gb.I64) == call(pdt=gb.BF16) == call(taps=9) == gb.ERR_UNSUPPORTED
    assert call(pool=1) == call(pool=-1) == call(taps=0) == call(s=strides(8, -8)) == gb.ERR_INVALID
    for k in ("x", "w", "state", "y"):
        assert call(**{k: None}) == call(**{k: ODD}) == gb.ERR_INVALID
    assert call(b=0, pool=0) == call(d=0) == gb.OK


def test_verify_drafts(lib):
    def call(dtype=gb.F32, b=2, k=3, v=10, tok=P, tdt=gb.I64, target=P, draft=P, s=None, acc=P, sam=P, lens=None, n=P, out=P):
        return lib.gb_verify_drafts(dtype, b, k, v, tok, tdt, target, draft, s, acc, sam, lens, n, out, None)
    assert call(b=-1) == call(k=-1) == call(v=-1) == call(tdt=gb.F32) == gb.ERR_INVALID
    assert call(dtype=gb.F64) == gb.ERR_UNSUPPORTED
    assert call(v=(1 << 30) + 1) == call(b=1 << 40) == call(k=1 << 31) == gb.ERR_RANGE
    for k in ("tok", "target", "acc", "sam", "n", "out"):
        assert call(**{k: None}) == call(**{k: ODD}) == gb.ERR_INVALID
    assert call(tok=ctypes.c_void_p(260)) == call(draft=HALF) == call(lens=HALF) == gb.ERR_INVALID
    assert call(s=strides(40, -10, 30, 10)) == call(s=strides(40, 10, 30, -10)) == gb.ERR_INVALID
    assert call(b=0) == gb.OK


def test_valid_calls_without_gpu_fail_loudly(lib):
    import torch
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    assert conv(lib) == ssc(lib) == gb.ERR_CUDA
    x, w = torch.zeros(1, 2, 8), torch.zeros(8, 4)
    with pytest.raises(ValueError):
        gb.causal_conv(x, w)
    with pytest.raises(ValueError):
        gb.selective_scan(x, x, torch.zeros(8, 16), torch.zeros(1, 2, 16), torch.zeros(1, 2, 16))
    with pytest.raises(ValueError):
        gb.verify_drafts(torch.zeros((1, 2), dtype=torch.int64), torch.zeros(1, 3, 5), None, torch.zeros(1, 2), torch.zeros(1))


@pytest.mark.parametrize("mode,keep", [("enable_grad", True), ("no_grad", False), ("inference_mode", False)])
def test_states_are_kept_only_for_a_gradient(monkeypatch, mode, keep):
    """Parameters require gradients while a model generates, too: without a graph nothing is kept."""
    torch = pytest.importorskip("torch")
    from stream_compaction_decoupled_gb300 import autograd, ssm

    asked = []

    def scan(x, *args, keep, **kw):
        asked.append(keep)
        return x.clone(), x.new_zeros(1), x.new_zeros(1) if keep else None

    monkeypatch.setattr(ssm, "selective_scan", scan)
    x, a = torch.zeros(1, 4, 2), torch.zeros(2, 3, requires_grad=True)
    bc = torch.zeros(1, 4, 3)
    with getattr(torch, mode)():
        autograd.selective_scan(x, x, a, bc, bc)
        autograd.selective_scan(x, x, a.detach(), bc, bc)
    assert asked == [keep, False]
