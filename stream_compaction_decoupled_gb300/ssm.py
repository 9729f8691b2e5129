"""Operators of state space language models: a short causal convolution and the selective
state space scan, each with its gradient and its form for one token a call, and the
verification of drafted tokens.

The functions marshal torch tensors into the ``gb_*`` entry points of the same names
(include/gbscan.h, where the formulas are), by the same rules as lm.py: fp32, bf16 or fp16
CUDA tensors with unit stride along their last dimension and any strides along the others
(slices of a fused projection need no copy), states of the scan in fp32, a call on `stream`
or the current stream.  ``autograd`` wraps the convolution and the scan for training.
"""
from __future__ import annotations

import functools
import struct
from collections import namedtuple

import torch

from . import I32, I64, _check, load
from .lm import _DTYPES, _dense, _first, _out, _p, _param, _rows_like, _run, _starts

SelectiveScanGrads = namedtuple("SelectiveScanGrads", "dx ddt da db dc dd dz ddt_bias dh0")
Verified = namedtuple("Verified", "accepted tokens")

_empty = torch.empty  # (Tensor.new_empty() costs a call 2 to 3 us more)
_KEPT = 16  # tokens from one kept state to the next
_pack = {n: struct.Struct("%dq" % n).pack for n in (2, 4, 6, 8, 14, 26)}


# ------------------------------------------------------------ causal convolution ------

def _taps(weight, bias, dtype, d, index):
    """Checks the convolution's parameters: (type code, taps)."""
    if weight.dim() != 2:
        raise ValueError("weight must be (channels, taps)")
    if weight.dtype is not dtype and weight.dtype is not torch.float32:
        raise TypeError("weight must be %s or fp32, not %s" % (dtype, weight.dtype))
    taps = weight.shape[1]
    if not 1 <= taps <= 8:
        raise ValueError("weight must have between 1 and 8 taps, not %d" % taps)
    _dense(weight, "weight", (d, taps), weight.dtype, index)
    code = _DTYPES[weight.dtype]
    if bias is not None and _param(bias, "bias", dtype, d, index) != code:
        raise TypeError("weight and bias must have the same type")
    return code, taps


def _apart(out, x):
    """Tokens need their neighbours' inputs, so nothing is computed in place."""
    if out.data_ptr() == x.data_ptr() and x.numel():
        raise ValueError("out must not be an input")


def causal_conv(x, weight, bias=None, state=None, starts=None, silu: bool = True, out=None, stream=None):
    """Causal convolution of each channel over dim 1 of a (batch, length, channels) tensor,
    then silu (or, silu=False, as it is): y_t = silu(bias + sum_k weight[:, k] x_{t-taps+1+k}).
    weight (channels, taps), 1 to 8 taps, of x's type or fp32, as bias (channels).  state
    (batch, taps - 1, channels) of x's type holds the inputs before the first, the newest last;
    starts as in recurrence().  Returns (y, last): last is the state after the last token."""
    code = _first(x, "x", 3, "(batch, length, channels)")
    (b, t, d), dtype, index = x.shape, x.dtype, x.get_device()
    pcode, taps = _taps(weight, bias, dtype, d, index)
    if state is not None:
        _dense(state, "state", (b, taps - 1, d), dtype, index)
    if starts is not None:
        starts = _starts(starts, (b, t), index)
    if out is not None:
        _out(out, "out", x.shape, dtype, index)
        _apart(out, x)
    return _run(_causal_conv, x, stream, (code, pcode, taps, x, weight, bias, state, starts, silu, out))


def _causal_conv(s, code, pcode, taps, x, weight, bias, state, starts, silu, out):
    b, t, d = x.shape
    if out is None:
        out = _empty((b, t, d), dtype=x.dtype, device=x.device)
    last = _empty((b, taps - 1, d), dtype=x.dtype, device=x.device)
    sx, sy = x.stride(), out.stride()
    rc = load().gb_causal_conv(code, pcode, b, t, d, taps, x.data_ptr(), _pack[4](sx[0], sx[1], sy[0], sy[1]),
                               weight.data_ptr(), _p(bias), 1 if silu else 0, _p(state), _p(starts), out.data_ptr(),
                               last.data_ptr(), s)
    if rc:
        _check(rc, "gb_causal_conv")
    return out, last


def causal_conv_backward(dy, x, weight, bias=None, state=None, starts=None, dlast=None, silu: bool = True,
                         dparams: bool = True, out=None, temp=None, stream=None):
    """Gradient of causal_conv() from its inputs, the gradient dy of y and dlast (like the state,
    or None) of the last state.  Returns (dx, dweight, dbias, dstate): dbias None without bias,
    dstate without state, dweight and dbias where `dparams` is False.  `out` gives dx."""
    code = _first(x, "x", 3, "(batch, length, channels)")
    (b, t, d), dtype, index = x.shape, x.dtype, x.get_device()
    _rows_like(dy, "dy", x.shape, dtype, index)
    pcode, taps = _taps(weight, bias, dtype, d, index)
    for v, what in ((state, "state"), (dlast, "dlast")):
        if v is not None:
            _dense(v, what, (b, taps - 1, d), dtype, index)
    if starts is not None:
        starts = _starts(starts, (b, t), index)
    if out is not None:
        _out(out, "out", x.shape, dtype, index)
        _apart(out, x)
        _apart(out, dy)
    _scratch(temp, index)
    return _run(_causal_conv_backward, x, stream,
                (code, pcode, taps, dy, x, weight, bias, state, starts, dlast, silu, dparams, out, temp))


def _causal_conv_backward(s, code, pcode, taps, dy, x, weight, bias, state, starts, dlast, silu, dparams, out, temp):
    (b, t, d), dev, lib = x.shape, x.device, load()
    if out is None:
        out = _empty((b, t, d), dtype=x.dtype, device=x.device)
    dw = db = dstate = None
    tb = 0
    if dparams:
        dw = torch.empty_like(weight)
        db = None if bias is None else torch.empty_like(bias)
        temp, tb = _temp(temp, lib.gb_causal_conv_temp_bytes(b, t, d, taps), dev)
    else:
        temp = None
    if state is not None:
        dstate = torch.empty_like(state)
    rc = lib.gb_causal_conv_backward(
        code, pcode, b, t, d, taps, dy.data_ptr(), x.data_ptr(),
        _pack[6](*dy.stride()[:2], *x.stride()[:2], *out.stride()[:2]), weight.data_ptr(), _p(bias), 1 if silu else 0,
        _p(state), _p(starts), _p(dlast), out.data_ptr(), _p(dw), _p(db), _p(dstate), _p(temp), tb, s)
    if rc:
        _check(rc, "gb_causal_conv_backward")
    return out, dw, db, dstate


def causal_conv_step(x, state, weight, bias=None, slots=None, silu: bool = True, out=None, stream=None):
    """One token for each row of a (batch, channels) tensor: the convolution with the inputs in
    state[slots[b]] ((pool, taps - 1, channels) of x's type), which is updated in place.  slots as
    in recurrence_step().  Returns y."""
    code = _first(x, "x", 2, "(batch, channels)")
    (b, d), dtype, index = x.shape, x.dtype, x.get_device()
    pcode, taps = _taps(weight, bias, dtype, d, index)
    if state.dim() != 3:
        raise ValueError("state must be (pool, taps - 1, channels)")
    _dense(state, "state", (state.shape[0], taps - 1, d), dtype, index)
    _slots(slots, b, state, index)
    if out is not None:
        _out(out, "out", x.shape, dtype, index)
    return _run(_causal_conv_step, x, stream, (code, pcode, taps, x, state, weight, bias, slots, silu, out))


def _causal_conv_step(s, code, pcode, taps, x, state, weight, bias, slots, silu, out):
    b, d = x.shape
    if out is None:
        out = _empty((b, d), dtype=x.dtype, device=x.device)
    rc = load().gb_causal_conv_step(code, pcode, b, d, taps, x.data_ptr(), _pack[2](x.stride()[0], out.stride()[0]),
                                    weight.data_ptr(), _p(bias), 1 if silu else 0, state.data_ptr(), state.shape[0],
                                    _p(slots), out.data_ptr(), s)
    if rc:
        _check(rc, "gb_causal_conv_step")
    return out


def _slots(slots, b, state, index):
    if slots is not None:
        _dense(slots, "slots", (b,), torch.int32, index)
    elif b > state.shape[0]:
        raise ValueError("state has %d rows for a batch of %d" % (state.shape[0], b))


def _scratch(temp, index):
    if temp is not None and (temp.get_device() != index or not temp.is_contiguous()):
        raise ValueError("temp must be a contiguous CUDA tensor on device %d" % index)


def _temp(temp, need, dev):
    """The call's scratch and its bytes: the caller's, or new."""
    if temp is not None:
        return temp, temp.numel() * temp.element_size()
    return (torch.empty((need,), dtype=torch.uint8, device=dev), need) if need else (None, 0)


# ------------------------------------------------------------ selective scan ------

def _vectors(m, what, lead, states, dtype, index):
    """Checks b or c, (*lead, groups, states) or (*lead, states): (groups, its strides but the last,
    with a group's stride of 0 where it has no such dimension)."""
    shape, strides, dims = m.shape, m.stride(), len(lead)
    grouped = len(shape) == dims + 2
    if not grouped and len(shape) != dims + 1:
        raise ValueError("%s must be (%s, groups, states), or without groups" % (what, "batch, length" if dims == 2 else "batch"))
    if m.dtype is not dtype or shape[:dims] != lead or m.get_device() != index or (strides[-1] != 1 and shape[-1] > 1):
        _rows_like(m, what, lead + shape[dims:], dtype, index)
    if shape[-1] != states:
        raise ValueError("%s must have %d states, not %d" % (what, states, shape[-1]))
    return (shape[-2], strides[:-1]) if grouped else (1, strides[:-1] + (0,))


def _ssm(x, dt, a, b, c, d, z, dt_bias):
    """Checks what the forms of the scan share: (groups, strides of b, strides of c)."""
    shape, dtype, index = x.shape, x.dtype, x.get_device()
    width = shape[-1]
    if dt.dtype is not dtype or dt.shape != shape or dt.get_device() != index or dt.stride()[-1] != 1:
        _rows_like(dt, "dt", shape, dtype, index)
    if z is not None and (z.dtype is not dtype or z.shape != shape or z.get_device() != index or z.stride()[-1] != 1):
        _rows_like(z, "z", shape, dtype, index)
    if a.dim() != 2:
        raise ValueError("a must be (channels, states)")
    states = a.shape[1]
    if not 1 <= states <= 128:
        raise ValueError("a must have between 1 and 128 states, not %d" % states)
    _dense(a, "a", (width, states), torch.float32, index)
    groups, sb = _vectors(b, "b", shape[:-1], states, dtype, index)
    also, sc = _vectors(c, "c", shape[:-1], states, dtype, index)
    if groups != also:
        raise ValueError("b and c must have the same groups")
    if groups < 1 or width % groups:
        raise ValueError("%d channels do not divide into %d groups" % (width, groups))
    if d is not None:
        _dense(d, "d", (width,), torch.float32, index)
    if dt_bias is not None:
        _dense(dt_bias, "dt_bias", (width,), torch.float32, index)
    return groups, sb, sc


@functools.lru_cache(maxsize=512)
def _scan_scratch(rows, t, width, states, groups, backward):
    return load().gb_selective_scan_temp_bytes(rows, t, width, states, groups, backward)


def selective_scan(x, dt, a, b, c, d=None, z=None, dt_bias=None, h0=None, starts=None, softplus: bool = True,
                   keep: bool = False, out=None, temp=None, stream=None):
    """Selective state space scan over dim 1 of a (batch, length, channels) tensor, for each
    channel with `states` (1 to 128) states h:
        D_t = softplus(dt_t + dt_bias),  h_t = exp(D_t a) h_{t-1} + D_t x_t b_t,
        y_t = (c_t . h_t + d x_t) silu(z_t).
    dt, z like x; a (channels, states), d and dt_bias (channels) fp32; b, c (batch, length,
    groups, states) of x's type, or (batch, length, states) for one group.  Without d, z and
    dt_bias their parts fall away; softplus=False takes dt + dt_bias as it is.  h0 (batch,
    channels, states) fp32 is the state to start from; starts as in recurrence().
    Returns (y, last, kept): last the state after the last token, kept (with keep=True; else
    None) what selective_scan_backward() needs: the state before every 16th token, fp32."""
    code = _first(x, "x", 3, "(batch, length, channels)")
    vectors = _ssm(x, dt, a, b, c, d, z, dt_bias)
    (rows, t, width), index = x.shape, x.get_device()
    if h0 is not None:
        _dense(h0, "h0", (rows, width, a.shape[1]), torch.float32, index)
    if starts is not None:
        starts = _starts(starts, (rows, t), index)
    if out is not None:
        _out(out, "out", x.shape, x.dtype, index)
    _scratch(temp, index)
    return _run(_selective_scan, x, stream, (code, vectors, x, dt, a, b, c, d, z, dt_bias, h0, starts, softplus, keep, out, temp))


def _selective_scan(s, code, vectors, x, dt, a, b, c, d, z, dt_bias, h0, starts, softplus, keep, out, temp):
    (rows, t, width), dev, lib = x.shape, x.device, load()
    (groups, sb, sc), states = vectors, a.shape[1]
    if out is None:
        out = _empty((rows, t, width), dtype=x.dtype, device=x.device)
    last = _empty((rows, width, states), dtype=torch.float32, device=x.device)
    kept = _empty((rows, -(-t // _KEPT), width, states), dtype=torch.float32, device=x.device) if keep else None
    temp, tb = _temp(temp, _scan_scratch(rows, t, width, states, groups, 0), dev)
    sx, sd, sz, sy = x.stride(), dt.stride(), (0, 0) if z is None else z.stride(), out.stride()
    rc = lib.gb_selective_scan(
        code, rows, t, width, states, groups, x.data_ptr(), dt.data_ptr(), a.data_ptr(), b.data_ptr(), c.data_ptr(),
        _p(d), _p(z), _p(dt_bias), 1 if softplus else 0,
        _pack[14](sx[0], sx[1], sd[0], sd[1], sz[0], sz[1], sy[0], sy[1], sb[0], sb[1], sb[2], sc[0], sc[1], sc[2]),
        _p(h0), _p(starts), out.data_ptr(), last.data_ptr(), _p(kept), _p(temp), tb, s)
    if rc:
        _check(rc, "gb_selective_scan")
    return out, last, kept


def selective_scan_backward(dy, x, dt, a, b, c, kept, d=None, z=None, dt_bias=None, starts=None, dlast=None,
                            softplus: bool = True, out=None, temp=None, stream=None):
    """Gradient of selective_scan() from its inputs, what it kept, the gradient dy of y and dlast
    (fp32, or None) of the last state.  Returns a SelectiveScanGrads (dx, ddt, da, db, dc, dd, dz,
    ddt_bias, dh0): None for what the call had no input for, dh0 always, da, dd, ddt_bias and dh0
    fp32.  `out` gives the tensors for (dx, ddt, dz) or, without z, (dx, ddt)."""
    code = _first(x, "x", 3, "(batch, length, channels)")
    vectors = _ssm(x, dt, a, b, c, d, z, dt_bias)
    (rows, t, width), dtype, index = x.shape, x.dtype, x.get_device()
    _rows_like(dy, "dy", x.shape, dtype, index)
    _dense(kept, "kept", (rows, -(-t // _KEPT), width, a.shape[1]), torch.float32, index)
    if dlast is not None:
        _dense(dlast, "dlast", (rows, width, a.shape[1]), torch.float32, index)
    if starts is not None:
        starts = _starts(starts, (rows, t), index)
    dx = ddt = dz = None
    if out is not None:
        dx, ddt, dz = out if z is not None else (*out[:2], None)
        for v, what in ((dx, "dx"), (ddt, "ddt"), (dz, "dz")):
            if what != "dz" or z is not None:
                _out(v, what, x.shape, dtype, index)
    _scratch(temp, index)
    return _run(_selective_scan_backward, x, stream,
                (code, vectors, dy, x, dt, a, b, c, kept, d, z, dt_bias, starts, dlast, softplus, dx, ddt, dz, temp))


def _selective_scan_backward(s, code, vectors, dy, x, dt, a, b, c, kept, d, z, dt_bias, starts, dlast, softplus, dx, ddt,
                             dz, temp):
    (rows, t, width), dtype, dev, lib = x.shape, x.dtype, x.device, load()
    (groups, sb, sc), states = vectors, a.shape[1]
    if dx is None:
        dx = _empty((rows, t, width), dtype=x.dtype, device=x.device)
        ddt = _empty((rows, t, width), dtype=x.dtype, device=x.device)
        if z is not None:
            dz = _empty((rows, t, width), dtype=x.dtype, device=x.device)
    db = _empty(b.shape, dtype=x.dtype, device=x.device)
    dc = _empty(c.shape, dtype=x.dtype, device=x.device)
    da = _empty((width, states), dtype=torch.float32, device=x.device)
    dd = None if d is None else _empty((width,), dtype=torch.float32, device=x.device)
    dbias = None if dt_bias is None else _empty((width,), dtype=torch.float32, device=x.device)
    dh0 = _empty((rows, width, states), dtype=torch.float32, device=x.device)
    temp, tb = _temp(temp, _scan_scratch(rows, t, width, states, groups, 1), dev)
    sz, sdz = ((0, 0), (0, 0)) if z is None else (z.stride()[:2], dz.stride()[:2])
    rc = lib.gb_selective_scan_backward(
        code, rows, t, width, states, groups, dy.data_ptr(), x.data_ptr(), dt.data_ptr(), a.data_ptr(), b.data_ptr(),
        c.data_ptr(), _p(d), _p(z), _p(dt_bias), 1 if softplus else 0,
        _pack[26](*dy.stride()[:2], *x.stride()[:2], *dt.stride()[:2], *sz, *dx.stride()[:2], *ddt.stride()[:2], *sdz,
                  *sb, *sc, t * groups * states, groups * states, states, t * groups * states, groups * states, states),
        kept.data_ptr(), _p(starts), _p(dlast), dx.data_ptr(), ddt.data_ptr(), da.data_ptr(), db.data_ptr(),
        dc.data_ptr(), _p(dd), _p(dz), _p(dbias), dh0.data_ptr(), _p(temp), tb, s)
    if rc:
        _check(rc, "gb_selective_scan_backward")
    return SelectiveScanGrads(dx, ddt, da, db, dc, dd, dz, dbias, dh0)


def selective_scan_step(x, dt, a, b, c, state, d=None, z=None, dt_bias=None, slots=None, softplus: bool = True, out=None,
                        stream=None):
    """One token for each row of (batch, channels) tensors: the scan from state[slots[b]] (fp32,
    (pool, channels, states)), which is updated in place.  b, c (batch, groups, states) or (batch,
    states); slots as in recurrence_step().  Returns y."""
    code = _first(x, "x", 2, "(batch, channels)")
    vectors = _ssm(x, dt, a, b, c, d, z, dt_bias)
    (rows, width), index = x.shape, x.get_device()
    if state.dim() != 3:
        raise ValueError("state must be (pool, channels, states)")
    _dense(state, "state", (state.shape[0], width, a.shape[1]), torch.float32, index)
    _slots(slots, rows, state, index)
    if out is not None:
        _out(out, "out", x.shape, x.dtype, index)
    return _run(_selective_scan_step, x, stream, (code, vectors, x, dt, a, b, c, state, d, z, dt_bias, slots, softplus, out))


def _selective_scan_step(s, code, vectors, x, dt, a, b, c, state, d, z, dt_bias, slots, softplus, out):
    rows, width = x.shape
    if out is None:
        out = _empty((rows, width), dtype=x.dtype, device=x.device)
    groups, sb, sc = vectors
    rc = load().gb_selective_scan_step(
        code, rows, width, a.shape[1], groups, x.data_ptr(), dt.data_ptr(), a.data_ptr(), b.data_ptr(), c.data_ptr(),
        _p(d), _p(z), _p(dt_bias), 1 if softplus else 0,
        _pack[8](x.stride()[0], dt.stride()[0], 0 if z is None else z.stride()[0], out.stride()[0], sb[0], sb[1], sc[0], sc[1]),
        state.data_ptr(), state.shape[0], _p(slots), out.data_ptr(), s)
    if rc:
        _check(rc, "gb_selective_scan_step")
    return out


# ------------------------------------------------------------ drafted tokens ------

def verify_drafts(drafts, target, draft, accept, sample, lengths=None, stream=None):
    """Which of the drafted tokens (batch, k) (int32 or int64) the target's probabilities
    (batch, k + 1, vocab) accept, and the token after them.  draft (batch, k, vocab) holds the
    drafter's probabilities, of target's type; None: the drafts are certain (looked up).  accept
    (batch, k) and sample (batch) are fp32 random numbers in [0, 1); lengths (batch) int32 says
    how many drafts a row has (None: k).  Draft i is accepted while accept_i q_i < p_i; the token
    after the accepted ones is drawn with `sample` from max(p - q, 0) where a draft was refused
    (without `draft`: from p but for the refused token), else from the next row of target.
    Returns (accepted, tokens): (batch) int32, and (batch, k + 1) int32: the accepted drafts, the
    token drawn (-1 where no probability is positive), and -1 behind it."""
    code = _first(target, "target", 3, "(batch, drafts + 1, vocab)")
    n, k, v = target.shape
    k, dtype, index = k - 1, target.dtype, target.get_device()
    if k < 0:
        raise ValueError("target must have one row more than there are drafts")
    if drafts.dtype is not torch.int64 and drafts.dtype is not torch.int32:
        raise TypeError("drafts must be int32 or int64, not %s" % drafts.dtype)
    _dense(drafts, "drafts", (n, k), drafts.dtype, index)
    if draft is not None:
        _rows_like(draft, "draft", (n, k, v), dtype, index)
    _dense(accept, "accept", (n, k), torch.float32, index)
    _dense(sample, "sample", (n,), torch.float32, index)
    if lengths is not None:
        _dense(lengths, "lengths", (n,), torch.int32, index)
    return _run(_verify_drafts, target, stream, (code, drafts, target, draft, accept, sample, lengths))


def _verify_drafts(s, code, drafts, target, draft, accept, sample, lengths):
    n, k, v = target.shape
    accepted = _empty((n,), dtype=torch.int32, device=sample.device)
    tokens = _empty((n, k), dtype=torch.int32, device=sample.device)
    st, sd = target.stride(), (0, 0) if draft is None else draft.stride()
    rc = load().gb_verify_drafts(code, n, k - 1, v, drafts.data_ptr(), I64 if drafts.dtype is torch.int64 else I32,
                                 target.data_ptr(), _p(draft), _pack[4](st[0], st[1], sd[0], sd[1]), accept.data_ptr(),
                                 sample.data_ptr(), _p(lengths), accepted.data_ptr(), tokens.data_ptr(), s)
    if rc:
        _check(rc, "gb_verify_drafts")
    return Verified(accepted, tokens)
