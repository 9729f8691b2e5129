"""Language-model operators: a gated linear recurrence (a scan of affine maps over time),
layer norm, and log probabilities of given tokens, each with its gradient.

The functions marshal torch tensors into the ``gb_*`` entry points of the same names
(declared at the end of include/gbscan.h, where the formulas are), as the rest of the
binding does.  Inputs are fp32, bf16 or fp16 CUDA tensors with unit stride along their
last dimension and any strides along the others (slices of a fused projection need no
copy; what layer norm copies, it says); states and statistics are fp32.  ``autograd`` wraps the same calls for training.

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


# The same numbers without their wrappers, where torch has them.
if hasattr(torch._C, "_cuda_getCurrentRawStream") and hasattr(torch._C, "_cuda_getDevice"):
    _raw_stream, _current_device = torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice

TokenLogprobs = namedtuple("TokenLogprobs", "logprob entropy lse top_values top_ids")


def _wrong(t, what, shape, dtype, index):
    """Raises what is wrong with an operand."""
    if t.dtype is not dtype:
        raise TypeError("%s must be %s, not %s" % (what, dtype, t.dtype))
    if t.shape != shape:
        raise ValueError("%s must have shape %s, not %s" % (what, tuple(shape), tuple(t.shape)))
    if t.get_device() != index:
        raise ValueError("%s must be a CUDA tensor on device %d" % (what, index))
    raise ValueError("%s must have unit stride along its last dimension" % what)


def _rows_like(t, what, shape, dtype, index):
    """Checks an operand of any leading strides: its type, shape, device (a CUDA index, which
    no CPU tensor has) and last stride."""
    if t.dtype is not dtype or t.shape != shape or t.get_device() != index or \
            (t.stride(-1) != 1 and shape[-1] > 1):
        _wrong(t, what, shape, dtype, index)


def _dense(t, what, shape, dtype, index):
    """Checks a contiguous operand."""
    if t.dtype is not dtype or t.shape != shape or t.get_device() != index:
        _wrong(t, what, shape, dtype, index)
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


def _out(t, what, shape, dtype, index):
    """Checks an output tensor of the caller's: its rows must not lie on each other (as an
    expanded tensor's do)."""
    _rows_like(t, what, shape, dtype, index)
    if any(s == 0 and n > 1 for s, n in zip(t.stride(), t.shape)):
        raise ValueError("%s must not be an expanded tensor" % what)


class _On:
    """Where a call runs: the stream handle, with allocation on that stream and the
    tensor's device current inside the block."""

    __slots__ = ("handle", "guards")

    def __init__(self, x, stream, inputs):
        self.guards = ()
        if x.get_device() != _current_device():
            self.guards = (torch.cuda.device(x.device),)
        if stream is None:
            self.handle = _raw_stream(x.get_device())
        else:
            s = _torch_stream(x, stream)
            self.handle = s.cuda_stream
            self.guards += (torch.cuda.stream(s),)
            for t in inputs:
                if torch.is_tensor(t):
                    t.record_stream(s)

    def __enter__(self):
        for g in self.guards:
            g.__enter__()
        return self.handle

    def __exit__(self, *exc):
        for g in reversed(self.guards):
            g.__exit__(*exc)
        return False


def _run(call, x, stream, args):
    """call(stream handle, *args) where x's call runs: directly on the current stream of the
    current device, which is the common case and the quick one."""
    if stream is None:
        index = x.get_device()
        if index == _current_device():
            return call(_raw_stream(index), *args)
    with _On(x, stream, args) as s:
        return call(s, *args)


# Host arrays of strides, as the bytes of 64-bit integers.
_int64s = {n: struct.Struct("%dq" % n).pack for n in (4, 8, 16)}


def _starts(starts, shape, index):
    if starts.dtype is torch.bool:
        starts = starts.view(torch.uint8)
    _dense(starts, "starts", shape, torch.uint8, index)
    return starts


def recurrence(x, f, i=None, h0=None, starts=None, out=None, stream=None):
    """Gated linear recurrence h_t = a_t h_{t-1} + u_t x_t over dim 1 of (batch, length,
    channels) tensors; a = sigmoid(f), u = sigmoid(i), or 1 - a without i.  h0 (batch,
    channels) fp32 is the state to start from, starts (batch, length) uint8 or bool marks
    tokens before which the state is dropped.  Returns (h, last): h like x, last the fp32
    state after the final token."""
    code = _first(x, "x", 3, "(batch, length, channels)")
    shape, dtype, index = x.shape, x.dtype, x.get_device()
    _rows_like(f, "f", shape, dtype, index)
    if i is not None:
        _rows_like(i, "i", shape, dtype, index)
    if h0 is not None:
        _dense(h0, "h0", (shape[0], shape[2]), torch.float32, index)
    if starts is not None:
        starts = _starts(starts, shape[:2], index)
    if out is not None:
        _out(out, "out", shape, dtype, index)
    return _run(_recurrence, x, stream, (code, x, f, i, h0, starts, out))


def _recurrence(s, code, x, f, i, h0, starts, out):
    b, t, d = x.shape
    if out is None:
        out = torch.empty((b, t, d), dtype=x.dtype, device=x.device)
    last = torch.empty((b, d), dtype=torch.float32, device=x.device)
    sx, sf, sh = x.stride(), f.stride(), out.stride()
    si = (0, 0) if i is None else i.stride()
    rc = load().gb_recurrence(code, b, t, d, x.data_ptr(), f.data_ptr(), _p(i),
                              _int64s[8](sx[0], sx[1], sf[0], sf[1], si[0], si[1], sh[0], sh[1]), _p(h0), _p(starts),
                              out.data_ptr(), last.data_ptr(), s)
    if rc:
        _check(rc, "gb_recurrence")
    return out, last


def recurrence_backward(dh, x, f, h, i=None, h0=None, starts=None, dlast=None, out=None, stream=None):
    """Gradient of recurrence() from its inputs, its output h and the gradients dh of h
    and dlast (fp32, or None) of the last state.  Returns (dx, df, di, dh0), di None
    without i.  `out` gives the tensors for (dx, df, di), such as slices of one buffer."""
    code = _first(x, "x", 3, "(batch, length, channels)")
    shape, dtype, index = x.shape, x.dtype, x.get_device()
    _rows_like(dh, "dh", shape, dtype, index)
    _rows_like(f, "f", shape, dtype, index)
    _rows_like(h, "h", shape, dtype, index)
    if i is not None:
        _rows_like(i, "i", shape, dtype, index)
    if h0 is not None:
        _dense(h0, "h0", (shape[0], shape[2]), torch.float32, index)
    if dlast is not None:
        _dense(dlast, "dlast", (shape[0], shape[2]), torch.float32, index)
    if starts is not None:
        starts = _starts(starts, shape[:2], index)
    dx = df = di = None
    if out is not None:
        dx, df, di = out if i is not None else (*out[:2], None)
        for v, what in ((dx, "dx"), (df, "df"), (di, "di")):
            if what != "di" or i is not None:
                _out(v, what, shape, dtype, index)
    return _run(_recurrence_backward, x, stream, (code, dh, x, f, h, i, h0, starts, dlast, dx, df, di))


def _recurrence_backward(s, code, dh, x, f, h, i, h0, starts, dlast, dx, df, di):
    b, t, d = x.shape
    dtype, dev = x.dtype, x.device
    if dx is None:
        dx = torch.empty((b, t, d), dtype=dtype, device=dev)
        df = torch.empty((b, t, d), dtype=dtype, device=dev)
        if i is not None:
            di = torch.empty((b, t, d), dtype=dtype, device=dev)
    dh0 = torch.empty((b, d), dtype=torch.float32, device=dev)
    si, sdi = ((0, 0), (0, 0)) if i is None else (i.stride()[:2], di.stride()[:2])
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
    shape, dtype, index = x.shape, x.dtype, x.get_device()
    _rows_like(f, "f", shape, dtype, index)
    if i is not None:
        _rows_like(i, "i", shape, dtype, index)
    if state.dim() != 2:
        raise ValueError("state must be (pool, channels)")
    _dense(state, "state", (state.shape[0], shape[1]), torch.float32, index)
    if slots is not None:
        _dense(slots, "slots", shape[:1], torch.int32, index)
    elif shape[0] > state.shape[0]:
        raise ValueError("state has %d rows for a batch of %d" % (state.shape[0], shape[0]))
    if out is not None:
        _out(out, "out", shape, dtype, index)
    return _run(_recurrence_step, x, stream, (code, x, f, state, i, slots, out))


def _recurrence_step(s, code, x, f, state, i, slots, out):
    b, d = x.shape
    if out is None:
        out = torch.empty((b, d), dtype=x.dtype, device=x.device)
    rc = load().gb_recurrence_step(code, b, d, x.data_ptr(), f.data_ptr(), _p(i),
                                   _int64s[4](x.stride(0), f.stride(0), 0 if i is None else i.stride(0), out.stride(0)),
                                   state.data_ptr(), state.shape[0], _p(slots), out.data_ptr(), s)
    if rc:
        _check(rc, "gb_recurrence_step")
    return out


def _p(t):
    return None if t is None else t.data_ptr()


def _rows(t, what):
    """A tensor as rows: 2-D as it is, other shapes as a (rows, cols) view, or None where the
    leading dimensions do not merge into rows of one stride."""
    if t.dim() == 2:
        return t
    if t.dim() == 0:
        raise ValueError("%s must have at least one dimension" % what)
    try:
        return t.view(-1, t.shape[-1]) if t.numel() else t.reshape(0, t.shape[-1])
    except RuntimeError:
        return None


def _laid_out(t, t2):
    """The rows t2 of t, copied where t has none (on the stream that is current)."""
    return t.contiguous().view(-1, t.shape[-1]) if t2 is None else t2


def _param(p, what, dtype, d, index):
    if p.dtype is not dtype and p.dtype is not torch.float32:
        raise TypeError("%s must be %s or fp32, not %s" % (what, dtype, p.dtype))
    _dense(p, what, (d,), p.dtype, index)
    return _DTYPES[p.dtype]


def layer_norm(x, weight=None, bias=None, eps: float = 1e-5, out=None, stream=None):
    """Layer norm over the last dimension: (y, mean, rstd), mean and rstd fp32 with one
    entry a row.  weight and bias: of x's type or fp32, or None.  x may have any leading
    dimensions: where they do not merge into rows of one stride (x[:, 1:] of three
    dimensions) it is copied first.  Those of `out` must merge."""
    x2 = _rows(x, "x")
    code = pcode = _first(x, "x", x.dim(), "rows")
    d, index = x.shape[-1], x.get_device()
    if weight is not None:
        pcode = _param(weight, "weight", x.dtype, d, index)
    if bias is not None:
        pcode = _param(bias, "bias", x.dtype, d, index)
        if weight is not None and weight.dtype is not bias.dtype:
            raise TypeError("weight and bias must have the same type")
    if d == 0 and (x2 is None or x2.shape[0]):
        raise ValueError("x must have at least one column")
    if out is not None:
        _out(out, "out", x.shape, x.dtype, index)
        if _rows(out, "out") is None:
            raise ValueError("out must be 2-D, or have leading dimensions that merge into rows")
    return _run(_layer_norm, x, stream, (code, pcode, x, x2, weight, bias, eps, out))


def _layer_norm(s, code, pcode, x, x2, weight, bias, eps, out):
    x2 = _laid_out(x, x2)
    (n, d), dev = x2.shape, x2.device
    if out is None:
        out, y_stride = torch.empty(x.shape, dtype=x.dtype, device=dev), d
    else:
        y_stride = _rows(out, "out").stride(0)
    mean = torch.empty((n,), dtype=torch.float32, device=dev)
    rstd = torch.empty((n,), dtype=torch.float32, device=dev)
    rc = load().gb_layer_norm(code, pcode, n, d, x2.data_ptr(), x2.stride(0), _p(weight), _p(bias), eps, out.data_ptr(),
                              y_stride, mean.data_ptr(), rstd.data_ptr(), s)
    if rc:
        _check(rc, "gb_layer_norm")
    return out, mean, rstd


def layer_norm_backward(dy, x, mean, rstd, weight=None, bias: bool = True, temp=None, stream=None,
                        dweight: bool = True):
    """Gradient of layer_norm() from its input and its mean and rstd: (dx, dweight,
    dbias), the last two of weight's type (None without a weight, and each None
    where `bias` or `dweight` is False; without both there are no sums over rows).  x and dy may have any leading dimensions, as layer_norm()'s x."""
    x2, dy2 = _rows(x, "x"), _rows(dy, "dy")
    code = pcode = _first(x, "x", x.dim(), "rows")
    d, index = x.shape[-1], x.get_device()
    n = x.numel() // d if x2 is None else x2.shape[0]
    if dy2 is None:  # checked as rows that it does not have: by its own shape
        _rows_like(dy, "dy", x.shape, x.dtype, index)
    else:
        _rows_like(dy2, "dy", torch.Size((n, d)), x.dtype, index)
    _dense(mean, "mean", (n,), torch.float32, index)
    _dense(rstd, "rstd", (n,), torch.float32, index)
    if weight is not None:
        pcode = _param(weight, "weight", x.dtype, d, index)
    if temp is not None and (temp.get_device() != index or not temp.is_contiguous()):
        raise ValueError("temp must be a contiguous CUDA tensor on device %d" % index)
    return _run(_layer_norm_backward, x, stream, (code, pcode, dy, dy2, x, x2, mean, rstd, weight, bias, temp, dweight))


def _layer_norm_backward(s, code, pcode, dy, dy2, x, x2, mean, rstd, weight, bias, temp, dweight):
    x2, dy2 = _laid_out(x, x2), _laid_out(dy, dy2)
    (n, d), dev, lib = x2.shape, x2.device, load()
    dx = torch.empty(x.shape, dtype=x.dtype, device=dev)
    dw = db = None
    tb = 0
    if weight is None or not (dweight or bias):
        temp = None
    else:
        if dweight:
            dw = torch.empty((d,), dtype=weight.dtype, device=dev)
        if bias:
            db = torch.empty((d,), dtype=weight.dtype, device=dev)
        if temp is None:
            tb = lib.gb_layer_norm_temp_bytes(n, d)
            temp = torch.empty((max(tb, 1),), dtype=torch.uint8, device=dev)
        else:
            tb = temp.numel() * temp.element_size()
    rc = lib.gb_layer_norm_backward(code, pcode, n, d, dy2.data_ptr(), dy2.stride(0), x2.data_ptr(), x2.stride(0),
                                    mean.data_ptr(), rstd.data_ptr(), _p(weight), dx.data_ptr(), d, _p(dw), _p(db),
                                    _p(temp), tb, s)
    if rc:
        _check(rc, "gb_layer_norm_backward")
    return dx, dw, db


def _targets(targets, n, index):
    if targets.dtype is not torch.int64 and targets.dtype is not torch.int32:
        raise TypeError("targets must be int32 or int64, not %s" % targets.dtype)
    _dense(targets, "targets", (n,), targets.dtype, index)
    return I64 if targets.dtype is torch.int64 else I32


def token_logprobs(logits, targets, top: int = 0, stream=None):
    """Of each row of (rows, vocab) logits: the log probability of its target (int32 or
    int64; negative: ignored, 0), the entropy, the log of the sum of exponentials, and the
    `top` (0 .. 32) most likely tokens' log probabilities and int32 ids, in falling order,
    ties to the lower id (None, None for top=0).  A logit of -inf is masked."""
    code = _first(logits, "logits", 2, "(rows, vocab)")
    n, v = logits.shape
    tcode = _targets(targets, n, logits.get_device())
    if not 0 <= top <= min(32, v):
        raise ValueError("top must be between 0 and 32, and at most the vocabulary")
    return _run(_token_logprobs, logits, stream, (code, tcode, logits, targets, top))


def _token_logprobs(s, code, tcode, logits, targets, top):
    (n, v), dev = logits.shape, logits.device
    logprob = torch.empty((n,), dtype=torch.float32, device=dev)
    entropy = torch.empty((n,), dtype=torch.float32, device=dev)
    lse = torch.empty((n,), dtype=torch.float32, device=dev)
    values = ids = None
    if top:
        values = torch.empty((n, top), dtype=torch.float32, device=dev)
        ids = torch.empty((n, top), dtype=torch.int32, device=dev)
    rc = load().gb_token_logprobs(code, n, v, logits.data_ptr(), logits.stride(0), targets.data_ptr(), tcode,
                                  logprob.data_ptr(), entropy.data_ptr(), lse.data_ptr(), top, _p(values), _p(ids), s)
    if rc:
        _check(rc, "gb_token_logprobs")
    return TokenLogprobs(logprob, entropy, lse, values, ids)


def token_logprobs_backward(logits, targets, lse, entropy=None, dlogprob=None, dentropy=None, out=None, stream=None):
    """Gradient of token_logprobs()'s logprob and entropy with respect to the logits, from
    its lse and entropy: dlogits like logits.  dlogprob, dentropy: (rows) fp32 or None for
    zero.  out may be logits itself, which is then overwritten."""
    code = _first(logits, "logits", 2, "(rows, vocab)")
    n, index = logits.shape[0], logits.get_device()
    tcode = _targets(targets, n, index)
    _dense(lse, "lse", (n,), torch.float32, index)
    for t, what in ((entropy, "entropy"), (dlogprob, "dlogprob"), (dentropy, "dentropy")):
        if t is not None:
            _dense(t, what, (n,), torch.float32, index)
    if dentropy is not None and entropy is None:
        raise ValueError("dentropy needs the entropy")
    if out is not None:
        _out(out, "out", logits.shape, logits.dtype, index)
    return _run(_token_logprobs_backward, logits, stream,
                (code, tcode, logits, targets, lse, entropy, dlogprob, dentropy, out))


def _token_logprobs_backward(s, code, tcode, logits, targets, lse, entropy, dlogprob, dentropy, out):
    n, v = logits.shape
    if out is None:
        out = torch.empty((n, v), dtype=logits.dtype, device=logits.device)
    rc = load().gb_token_logprobs_backward(code, n, v, logits.data_ptr(), logits.stride(0), targets.data_ptr(), tcode,
                                           lse.data_ptr(), _p(entropy), _p(dlogprob), _p(dentropy), out.data_ptr(),
                                           out.stride(0), s)
    if rc:
        _check(rc, "gb_token_logprobs_backward")
    return out
