"""CPU-only checks of the language-model entry points: argument errors are reported before
any CUDA call, sizes of scratch, and the bounds that keep every launch in range."""
import ctypes

import pytest

import stream_compaction_decoupled_gb300 as gb
from stream_compaction_decoupled_gb300 import _build

P = ctypes.c_void_p(256)
ODD = ctypes.c_void_p(257)


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return gb.load()


def strides(*v):
    return (ctypes.c_int64 * len(v))(*v)


def rec(lib, dtype=None, b=2, t=4, d=8, x=P, f=P, i=None, s=None, h0=None, starts=None, h=P, last=None):
    return lib.gb_recurrence(gb.BF16 if dtype is None else dtype, b, t, d, x, f, i, s, h0, starts, h, last, None)


def test_recurrence(lib):
    assert rec(lib, b=-1) == rec(lib, t=-1) == rec(lib, d=-1) == gb.ERR_INVALID
    for dt in (gb.I32, gb.F64, gb.U64, 8, -1):
        assert rec(lib, dtype=dt) == gb.ERR_UNSUPPORTED
    assert rec(lib, x=None) == rec(lib, f=None) == rec(lib, h=None) == gb.ERR_INVALID
    assert rec(lib, x=ODD) == rec(lib, h=ODD) == rec(lib, h0=ODD) == rec(lib, last=ODD) == gb.ERR_INVALID
    assert rec(lib, dtype=gb.F32, f=ctypes.c_void_p(258)) == gb.ERR_INVALID
    assert rec(lib, s=strides(-1, 8, 32, 8, 0, 0, 32, 8)) == gb.ERR_INVALID
    assert rec(lib, s=strides(1 << 60, 8, 32, 8, 0, 0, 32, 8)) == gb.ERR_INVALID
    assert rec(lib, d=(1 << 28) + 1) == rec(lib, t=(1 << 30) + 1) == gb.ERR_RANGE
    assert rec(lib, b=1 << 40) == gb.ERR_RANGE
    assert rec(lib, b=1 << 20, d=1 << 30) == gb.ERR_RANGE
    assert rec(lib, b=0) == rec(lib, d=0) == rec(lib, t=0) == gb.OK


def test_recurrence_backward(lib):
    def call(dtype=gb.F32, b=2, t=4, d=8, dh=P, x=P, f=P, i=None, h=P, s=None, dx=P, df=P, di=None, dh0=None):
        return lib.gb_recurrence_backward(dtype, b, t, d, dh, x, f, i, h, s, None, None, None, dx, df, di, dh0, None)
    assert call(dtype=gb.F64) == gb.ERR_UNSUPPORTED
    for k in ("dh", "x", "f", "h", "dx", "df"):
        assert call(**{k: None}) == gb.ERR_INVALID
        assert call(**{k: ODD}) == gb.ERR_INVALID
    assert call(i=P) == gb.ERR_INVALID  # i without di
    assert call(s=strides(*[32, 8] * 6, -32, 8, 32, 8)) == gb.ERR_INVALID
    assert call(b=0) == call(t=0) == call(d=0) == gb.OK


def test_recurrence_step(lib):
    def call(dtype=gb.F16, b=2, d=8, x=P, f=P, i=None, s=None, state=P, pool=2, slots=None, h=P):
        return lib.gb_recurrence_step(dtype, b, d, x, f, i, s, state, pool, slots, h, None)
    assert call(dtype=gb.I64) == gb.ERR_UNSUPPORTED
    assert call(pool=1) == call(pool=-1) == call(state=None) == call(x=None) == call(h=ODD) == gb.ERR_INVALID
    assert call(state=ctypes.c_void_p(258)) == call(slots=ctypes.c_void_p(258)) == gb.ERR_INVALID
    assert call(s=strides(8, 8, 8, -8)) == gb.ERR_INVALID
    assert call(b=0, pool=0) == call(d=0) == gb.OK


def test_layer_norm(lib):
    def call(dtype=gb.BF16, pdt=gb.BF16, n=4, d=8, x=P, xs=8, w=P, b=P, eps=1e-5, y=P, ys=8, mean=P, rstd=P):
        return lib.gb_layer_norm(dtype, pdt, n, d, x, xs, w, b, eps, y, ys, mean, rstd, None)
    assert call(dtype=gb.F64) == call(pdt=gb.F16) == call(dtype=gb.F32, pdt=gb.BF16) == gb.ERR_UNSUPPORTED
    assert call(n=-1) == call(d=-1) == call(xs=-1) == call(ys=-1) == call(eps=-1.0) == gb.ERR_INVALID
    assert call(eps=float("nan")) == gb.ERR_INVALID
    for k in ("x", "y", "mean", "rstd"):
        assert call(**{k: None}) == call(**{k: ODD}) == gb.ERR_INVALID
    assert call(w=ODD) == call(pdt=gb.F32, b=ctypes.c_void_p(258)) == gb.ERR_INVALID
    assert call(d=(1 << 28) + 1) == gb.ERR_RANGE
    assert call(n=0) == call(d=0) == gb.OK


def test_layer_norm_backward(lib):
    def call(dtype=gb.BF16, pdt=gb.F32, n=4, d=8, dy=P, x=P, mean=P, rstd=P, w=P, dx=P, dw=P, db=P, dxs=8):
        return lib.gb_layer_norm_backward(dtype, pdt, n, d, dy, 8, x, 8, mean, rstd, w, dx, dxs, dw, db, None, 0, None)
    assert call(dtype=gb.U32) == call(pdt=gb.F16) == gb.ERR_UNSUPPORTED
    for k in ("dy", "x", "mean", "rstd", "dx"):
        assert call(**{k: None}) == gb.ERR_INVALID
    assert call(dw=ctypes.c_void_p(258)) == call(dxs=-1) == gb.ERR_INVALID
    assert call(d=0) == gb.OK
    assert lib.gb_layer_norm_temp_bytes(0, 8) == lib.gb_layer_norm_temp_bytes(8, 0) == 0
    assert lib.gb_layer_norm_temp_bytes(1, 1) > 0 and lib.gb_layer_norm_temp_bytes(1 << 40, 64) < 1 << 20


def test_token_logprobs(lib):
    def call(dtype=gb.F32, n=2, v=10, x=P, s=10, t=P, tdt=gb.I64, lp=P, ent=P, lse=P, top=0, tv=None, ti=None):
        return lib.gb_token_logprobs(dtype, n, v, x, s, t, tdt, lp, ent, lse, top, tv, ti, None)
    assert call(dtype=gb.F64) == gb.ERR_UNSUPPORTED
    assert call(n=-1) == call(v=-1) == call(s=-1) == call(tdt=gb.F32) == call(tdt=gb.U32) == gb.ERR_INVALID
    assert call(top=-1) == call(top=33, v=100) == call(top=11) == call(top=3) == gb.ERR_INVALID
    for k in ("x", "t", "lp", "ent", "lse"):
        assert call(**{k: None}) == gb.ERR_INVALID
    assert call(x=ctypes.c_void_p(258)) == call(t=ctypes.c_void_p(260)) == gb.ERR_INVALID
    assert call(v=(1 << 30) + 1) == call(n=1 << 40) == gb.ERR_RANGE
    assert call(n=0) == gb.OK


def test_token_logprobs_backward(lib):
    def call(dtype=gb.F32, n=2, v=10, x=P, s=10, t=P, tdt=gb.I32, lse=P, ent=P, dl=P, de=P, dx=P, ds=10):
        return lib.gb_token_logprobs_backward(dtype, n, v, x, s, t, tdt, lse, ent, dl, de, dx, ds, None)
    assert call(dtype=gb.I32) == gb.ERR_UNSUPPORTED
    assert call(ent=None) == call(x=None) == call(lse=None) == call(dx=None) == call(t=None) == gb.ERR_INVALID
    assert call(ds=12) == gb.ERR_INVALID  # in place with another stride
    assert call(s=-1) == call(tdt=gb.F16) == gb.ERR_INVALID
    assert call(n=1 << 30, v=1 << 20) == gb.ERR_RANGE
    assert call(n=0) == call(v=0) == gb.OK


def test_valid_calls_without_gpu_fail_loudly(lib):
    import torch
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    assert rec(lib) == gb.ERR_CUDA
    with pytest.raises(ValueError):
        gb.recurrence(torch.zeros(1, 2, 8), torch.zeros(1, 2, 8))
    with pytest.raises(ValueError):
        gb.layer_norm(torch.zeros(2, 8))
    with pytest.raises(ValueError):
        gb.token_logprobs(torch.zeros(2, 8), torch.zeros(2, dtype=torch.int64))


def test_the_scans_refuse_the_16_bit_types(lib):
    assert lib.gb_scan_inclusive(gb.BF16, 1, gb.ADD, P, P, 10, None, 0, None) == gb.ERR_INVALID
    assert lib.gb_temp_storage_bytes(gb.KIND_SCAN, gb.F16, 1, 10, 0) == 0
