"""Language-model operators: a gated linear recurrence (a scan of affine maps over time),
layer norm, and log probabilities of given tokens, each with its gradient.

The functions marshal torch tensors into the ``gb_*`` entry points of the same names
(declared at the end of include/gbscan.h, where the formulas are), as the rest of the
binding does.  Inputs are fp32, bf16 or fp16 CUDA tensors with unit stride along their
last dimension and any strides along the others (slices of a fused projection need no
copy); states and statistics are fp32.  ``autograd`` wraps the same calls for training.

A call runs on `stream`, or the current stream.  With an explicit stream its outputs are
allocated there and its inputs are kept from reuse until the call's kernels have run, but
ordering the call after whatever wrote the inputs is the caller's part.
"""
from __future__ import annotations

import struct
from collections import namedtuple

import torch

from . import BF16, F16, F32, I32, I64, _check, _torch_stream, load

_DTYPES = {torch.float32: F32, torch.bfloat16: BF16, torch.float16: F16}
_current_device = torch.cuda.current_device


def _raw_stream(index):
    return torch.cuda.current_stream(index).cuda_stream


if hasattr(torch._C, "_cuda_getCurrentRawStream"):  # the same handle, without a Stream object
    _raw_stream = torch._C._cuda_getCurrentRawStream

TokenLogprobs = namedtuple("TokenLogprobs", "logprob entropy lse top_values top_ids")


def _wrong(t, what, shape, dtype, device):
    """Raises what is wrong with an operand."""
    if t.dtype is not dtype:
        raise TypeError("%s must be %s, not %s" % (what, dtype, t.dtype))
    if t.shape != shape:
        raise ValueError("%s must have shape %s, not %s" % (what, tuple(shape), tuple(t.shape)))
    if not t.is_cuda or t.device != device:
        raise ValueError("%s must be a CUDA tensor on %s" % (what, device))
    raise ValueError("%s must have unit stride along its last dimension" % what)


def _rows_like(t, what, shape, dtype, device):
    """Checks an operand of any leading strides: its type, shape, device and last stride."""
    if t.dtype is not dtype or t.shape != shape or t.device != device or \
            (t.stride(-1) != 1 and shape[-1] > 1):
        _wrong(t, what, shape, dtype, device)


def _dense(t, what, shape, dtype, device):
    """Checks a contiguous operand."""
    if t.dtype is not dtype or t.shape != shape or t.device != device:
        _wrong(t, what, shape, dtype, device)
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % what)


def _first(x, what, dims, names):
    """Checks the operand that sets the type, shape and device of a call; its type's code."""
    if x.dim() != dims:
        raise ValueError("%s must be %s" % (what, names))
    code = _DTYPES.get(x.dtype)
    if code is None:
        raise TypeError("%s must be fp32, bf16 or fp16, not %s" % (what, x.dtype))
    if not x.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % what)
    if x.stride(-1) != 1 and x.shape[-1] > 1:
        raise ValueError("%s must have unit stride along its last dimension" % what)
    return code


def _out(t, what, shape, dtype, device):
    """Checks an output tensor of the caller's: its rows must not lie on each other (as an
    expanded tensor's do)."""
    _rows_like(t, what, shape, dtype, device)
    if any(s == 0 and n > 1 for s, n in zip(t.stride(), t.shape)):
        raise ValueError("%s must not be an expanded tensor" % what)


class _On:
    """Where a call runs: the stream handle, with allocation on that stream and the
    tensor's device current inside the block."""

    __slots__ = ("handle", "guards")

    def __init__(self, x, stream, inputs):
        self.guards = ()
        if x.device.index != _current_device():
            self.guards = (torch.cuda.device(x.device),)
        if stream is None:
            self.handle = _raw_stream(x.device.index)
        else:
            s = _torch_stream(x, stream)
            self.handle = s.cuda_stream
            self.guards += (torch.cuda.stream(s),)
            for t in inputs:
                if t is not None:
                    t.record_stream(s)

    def __enter__(self):
        for g in self.guards:
            g.__enter__()
        return self.handle

    def __exit__(self, *exc):
        for g in reversed(self.guards):
            g.__exit__(*exc)
        return False


class _Here:
    """The common case of _On, the current stream of the current device: nothing to set up."""

    __slots__ = ("handle",)

    def __init__(self, handle):
        self.handle = handle

    def __enter__(self):
        return self.handle

    def __exit__(self, *exc):
        return False


def _on(x, stream, *inputs):
    index = x.device.index
    if stream is None and index == _current_device():
        return _Here(_raw_stream(index))
    return _On(x, stream, inputs)


# Host arrays of strides, as the bytes of 64-bit integers.
_int64s = {n: struct.Struct("%dq" % n).pack for n in (4, 8, 16)}


def _starts(starts, shape, device):
    if starts.dtype is torch.bool:
        starts = starts.view(torch.uint8)
    _dense(starts, "starts", shape, torch.uint8, device)
    return starts


def recurrence(x, f, i=None, h0=None, starts=None, out=None, stream=None):
    """Gated linear recurrence h_t = a_t h_{t-1} + u_t x_t over dim 1 of (batch, length,
    channels) tensors; a = sigmoid(f), u = sigmoid(i), or 1 - a without i.  h0 (batch,
    channels) fp32 is the state to start from, starts (batch, length) uint8 or bool marks
    tokens before which the state is dropped.  Returns (h, last): h like x, last the fp32
    state after the final token."""
    code = _first(x, "x", 3, "(batch, length, channels)")
    shape, dtype, dev = x.shape, x.dtype, x.device
    b, t, d = shape
    _rows_like(f, "f", shape, dtype, dev)
    i_ptr = h0_ptr = starts_ptr = None
    si = (0, 0, 0)
    if i is not None:
        _rows_like(i, "i", shape, dtype, dev)
        i_ptr, si = i.data_ptr(), i.stride()
    if h0 is not None:
        _dense(h0, "h0", (b, d), torch.float32, dev)
        h0_ptr = h0.data_ptr()
    if starts is not None:
        starts = _starts(starts, (b, t), dev)
        starts_ptr = starts.data_ptr()
    if out is not None:
        _out(out, "out", shape, dtype, dev)
    with _on(x, stream, x, f, i, h0, starts, out) as s:
        if out is None:
            out = torch.empty(shape, dtype=dtype, device=dev)
        last = torch.empty((b, d), dtype=torch.float32, device=dev)
        sx, sf, sh = x.stride(), f.stride(), out.stride()
        rc = load().gb_recurrence(code, b, t, d, x.data_ptr(), f.data_ptr(), i_ptr,
                                  _int64s[8](sx[0], sx[1], sf[0], sf[1], si[0], si[1], sh[0], sh[1]), h0_ptr,
                                  starts_ptr, out.data_ptr(), last.data_ptr(), s)
    if rc:
        _check(rc, "gb_recurrence")
    return out, last


def recurrence_backward(dh, x, f, h, i=None, h0=None, starts=None, dlast=None, out=None, stream=None):
    """Gradient of recurrence() from its inputs, its output h and the gradients dh of h
    and dlast (fp32, or None) of the last state.  Returns (dx, df, di, dh0), di None
    without i.  `out` gives the tensors for (dx, df, di), such as slices of one buffer."""
    code = _first(x, "x", 3, "(batch, length, channels)")
    shape, dtype, dev = x.shape, x.dtype, x.device
    b, t, d = shape
    _rows_like(dh, "dh", shape, dtype, dev)
    _rows_like(f, "f", shape, dtype, dev)
    _rows_like(h, "h", shape, dtype, dev)
    if i is not None:
        _rows_like(i, "i", shape, dtype, dev)
    if h0 is not None:
        _dense(h0, "h0", (b, d), torch.float32, dev)
    if dlast is not None:
        _dense(dlast, "dlast", (b, d), torch.float32, dev)
    if starts is not None:
        starts = _starts(starts, (b, t), dev)
    dx = df = di = None
    if out is not None:
        dx, df, di = out if i is not None else (*out[:2], None)
        for v, what in ((dx, "dx"), (df, "df"), (di, "di")):
            if what != "di" or i is not None:
                _out(v, what, shape, dtype, dev)
    with _on(x, stream, dh, x, f, h, i, h0, starts, dlast, dx, df, di) as s:
        if out is None:
            dx = torch.empty(shape, dtype=dtype, device=dev)
            df = torch.empty(shape, dtype=dtype, device=dev)
            if i is not None:
                di = torch.empty(shape, dtype=dtype, device=dev)
        dh0 = torch.empty((b, d), dtype=torch.float32, device=dev)
        none = (0, 0)
        si, sdi = (none, none) if i is None else (i.stride()[:2], di.stride()[:2])
        rc = load().gb_recurrence_backward(
            code, b, t, d, dh.data_ptr(), x.data_ptr(), f.data_ptr(), _p(i), h.data_ptr(),
            _int64s[16](*dh.stride()[:2], *x.stride()[:2], *f.stride()[:2], *si, *h.stride()[:2], *dx.stride()[:2],
                        *df.stride()[:2], *sdi),
            _p(h0), _p(starts), _p(dlast), dx.data_ptr(), df.data_ptr(), _p(di), dh0.data_ptr(), s)
    if rc:
        _check(rc, "gb_recurrence_backward")
    return dx, df, di, dh0


def recurrence_step(x, f, state, i=None, slots=None, out=None, stream=None):
    """One token for each row of (batch, channels) tensors: the recurrence from
    state[slots[b]] (fp32, (pool, channels)), which is updated in place.  slots int32;
    None: row b uses state b; negative: padding, whose output is zero.  Returns h."""
    code = _first(x, "x", 2, "(batch, channels)")
    shape, dtype, dev = x.shape, x.dtype, x.device
    b, d = shape
    _rows_like(f, "f", shape, dtype, dev)
    i_ptr, si, slots_ptr = None, 0, None
    if i is not None:
        _rows_like(i, "i", shape, dtype, dev)
        i_ptr, si = i.data_ptr(), i.stride(0)
    if state.dim() != 2:
        raise ValueError("state must be (pool, channels)")
    pool = state.shape[0]
    _dense(state, "state", (pool, d), torch.float32, dev)
    if slots is not None:
        _dense(slots, "slots", (b,), torch.int32, dev)
        slots_ptr = slots.data_ptr()
    elif b > pool:
        raise ValueError("state has %d rows for a batch of %d" % (pool, b))
    if out is not None:
        _out(out, "out", shape, dtype, dev)
    with _on(x, stream, x, f, i, state, slots, out) as s:
        if out is None:
            out = torch.empty(shape, dtype=dtype, device=dev)
        rc = load().gb_recurrence_step(code, b, d, x.data_ptr(), f.data_ptr(), i_ptr,
                                       _int64s[4](x.stride(0), f.stride(0), si, out.stride(0)), state.data_ptr(),
                                       pool, slots_ptr, out.data_ptr(), s)
    if rc:
        _check(rc, "gb_recurrence_step")
    return out


def _p(t):
    return None if t is None else t.data_ptr()


def _rows(t, what):
    """A tensor as rows: 2-D as it is, other shapes as a (rows, cols) view."""
    if t.dim() == 2:
        return t
    if t.dim() == 0:
        raise ValueError("%s must have at least one dimension" % what)
    try:
        return t.view(-1, t.shape[-1]) if t.numel() else t.reshape(0, t.shape[-1])
    except RuntimeError:
        raise ValueError("%s must be 2-D, or have leading dimensions that merge into rows" % what) from None


def _param(p, what, dtype, d, dev):
    if p.dtype is not dtype and p.dtype is not torch.float32:
        raise TypeError("%s must be %s or fp32, not %s" % (what, dtype, p.dtype))
    _dense(p, what, (d,), p.dtype, dev)


def layer_norm(x, weight=None, bias=None, eps: float = 1e-5, out=None, stream=None):
    """Layer norm over the last dimension: (y, mean, rstd), mean and rstd fp32 with one
    entry a row.  weight and bias: of x's type or fp32, or None."""
    x2 = _rows(x, "x")
    code = pcode = _first(x2, "x", 2, "rows")
    n, d = x2.shape
    dtype, dev = x.dtype, x.device
    w_ptr = b_ptr = None
    if weight is not None:
        _param(weight, "weight", dtype, d, dev)
        pcode, w_ptr = _DTYPES[weight.dtype], weight.data_ptr()
    if bias is not None:
        _param(bias, "bias", dtype, d, dev)
        pcode, b_ptr = _DTYPES[bias.dtype], bias.data_ptr()
        if weight is not None and weight.dtype is not bias.dtype:
            raise TypeError("weight and bias must have the same type")
    if d == 0 and n:
        raise ValueError("x must have at least one column")
    if out is not None:
        _out(out, "out", x.shape, dtype, dev)
    with _on(x, stream, x, weight, bias, out) as s:
        if out is None:
            out = torch.empty(x.shape, dtype=dtype, device=dev)
            y_stride = d
        else:
            y_stride = _rows(out, "out").stride(0)
        mean = torch.empty((n,), dtype=torch.float32, device=dev)
        rstd = torch.empty((n,), dtype=torch.float32, device=dev)
        rc = load().gb_layer_norm(code, pcode, n, d, x2.data_ptr(), x2.stride(0), w_ptr, b_ptr, eps, out.data_ptr(),
                                  y_stride, mean.data_ptr(), rstd.data_ptr(), s)
    if rc:
        _check(rc, "gb_layer_norm")
    return out, mean, rstd


def layer_norm_backward(dy, x, mean, rstd, weight=None, bias: bool = True, temp=None, stream=None):
    """Gradient of layer_norm() from its input and its mean and rstd: (dx, dweight,
    dbias), the last two of weight's type (None without a weight; dbias None too with
    bias=False)."""
    x2, dy2 = _rows(x, "x"), _rows(dy, "dy")
    code = pcode = _first(x2, "x", 2, "rows")
    n, d = x2.shape
    dtype, dev = x.dtype, x.device
    _rows_like(dy2, "dy", x2.shape, dtype, dev)
    _dense(mean, "mean", (n,), torch.float32, dev)
    _dense(rstd, "rstd", (n,), torch.float32, dev)
    if weight is not None:
        _param(weight, "weight", dtype, d, dev)
        pcode = _DTYPES[weight.dtype]
    dw = db = tp = None
    tb = 0
    lib = load()
    with _on(x, stream, dy, x, mean, rstd, weight, temp) as s:
        dx = torch.empty(x.shape, dtype=dtype, device=dev)
        if weight is not None:
            dw = torch.empty((d,), dtype=weight.dtype, device=dev)
            if bias:
                db = torch.empty((d,), dtype=weight.dtype, device=dev)
            if temp is None:
                tb = lib.gb_layer_norm_temp_bytes(n, d)
                temp = torch.empty((max(tb, 1),), dtype=torch.uint8, device=dev)
            else:
                tb = temp.numel() * temp.element_size()
            tp = temp.data_ptr()
        rc = lib.gb_layer_norm_backward(code, pcode, n, d, dy2.data_ptr(), dy2.stride(0), x2.data_ptr(),
                                        x2.stride(0), mean.data_ptr(), rstd.data_ptr(), _p(weight), dx.data_ptr(),
                                        d, _p(dw), _p(db), tp, tb, s)
    if rc:
        _check(rc, "gb_layer_norm_backward")
    return dx, dw, db


def _targets(targets, n, device):
    if targets.dtype is not torch.int64 and targets.dtype is not torch.int32:
        raise TypeError("targets must be int32 or int64, not %s" % targets.dtype)
    _dense(targets, "targets", (n,), targets.dtype, device)
    return I64 if targets.dtype is torch.int64 else I32


def token_logprobs(logits, targets, top: int = 0, stream=None):
    """Of each row of (rows, vocab) logits: the log probability of its target (int32 or
    int64; negative: ignored, 0), the entropy, the log of the sum of exponentials, and the
    `top` (0 .. 32) most likely tokens' log probabilities and int32 ids, in falling order,
    ties to the lower id (None, None for top=0).  A logit of -inf is masked."""
    code = _first(logits, "logits", 2, "(rows, vocab)")
    (n, v), dev = logits.shape, logits.device
    tcode = _targets(targets, n, dev)
    if not 0 <= top <= min(32, v):
        raise ValueError("top must be between 0 and 32, and at most the vocabulary")
    values = ids = values_ptr = ids_ptr = None
    with _on(logits, stream, logits, targets) as s:
        logprob = torch.empty((n,), dtype=torch.float32, device=dev)
        entropy = torch.empty((n,), dtype=torch.float32, device=dev)
        lse = torch.empty((n,), dtype=torch.float32, device=dev)
        if top:
            values = torch.empty((n, top), dtype=torch.float32, device=dev)
            ids = torch.empty((n, top), dtype=torch.int32, device=dev)
            values_ptr, ids_ptr = values.data_ptr(), ids.data_ptr()
        rc = load().gb_token_logprobs(code, n, v, logits.data_ptr(), logits.stride(0), targets.data_ptr(), tcode,
                                      logprob.data_ptr(), entropy.data_ptr(), lse.data_ptr(), top, values_ptr,
                                      ids_ptr, s)
    if rc:
        _check(rc, "gb_token_logprobs")
    return TokenLogprobs(logprob, entropy, lse, values, ids)


def token_logprobs_backward(logits, targets, lse, entropy=None, dlogprob=None, dentropy=None, out=None, stream=None):
    """Gradient of token_logprobs()'s logprob and entropy with respect to the logits, from
    its lse and entropy: dlogits like logits.  dlogprob, dentropy: (rows) fp32 or None for
    zero.  out may be logits itself, which is then overwritten."""
    code = _first(logits, "logits", 2, "(rows, vocab)")
    (n, v), dev = logits.shape, logits.device
    tcode = _targets(targets, n, dev)
    _dense(lse, "lse", (n,), torch.float32, dev)
    for t, what in ((entropy, "entropy"), (dlogprob, "dlogprob"), (dentropy, "dentropy")):
        if t is not None:
            _dense(t, what, (n,), torch.float32, dev)
    if dentropy is not None and entropy is None:
        raise ValueError("dentropy needs the entropy")
    if out is not None:
        _out(out, "out", logits.shape, logits.dtype, dev)
    with _on(logits, stream, logits, targets, lse, entropy, dlogprob, dentropy, out) as s:
        if out is None:
            out = torch.empty((n, v), dtype=logits.dtype, device=dev)
        rc = load().gb_token_logprobs_backward(code, n, v, logits.data_ptr(), logits.stride(0), targets.data_ptr(),
                                               tcode, lse.data_ptr(), _p(entropy), _p(dlogprob), _p(dentropy),
                                               out.data_ptr(), out.stride(0), s)
    if rc:
        _check(rc, "gb_token_logprobs_backward")
    return out
