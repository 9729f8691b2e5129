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

import ctypes
from collections import namedtuple

import torch

from . import BF16, F16, F32, I32, I64, _check, _torch_stream, load

_DTYPES = {torch.float32: F32, torch.bfloat16: BF16, torch.float16: F16}
_raw_stream = torch._C._cuda_getCurrentRawStream if hasattr(torch._C, "_cuda_getCurrentRawStream") else None

TokenLogprobs = namedtuple("TokenLogprobs", "logprob entropy lse top_values top_ids")


def _code(t, what):
    code = _DTYPES.get(t.dtype)
    if code is None:
        raise TypeError("%s must be fp32, bf16 or fp16, not %s" % (what, t.dtype))
    return code


def _like(t, what, shape, dtype, device):
    """Checks an optional operand: its shape, type, device and unit last stride."""
    if t.dtype != dtype:
        raise TypeError("%s must be %s, not %s" % (what, dtype, t.dtype))
    if t.shape != shape:
        raise ValueError("%s must have shape %s, not %s" % (what, tuple(shape), tuple(t.shape)))
    if t.device != device:
        raise ValueError("%s must be on %s" % (what, device))
    if t.stride(-1) != 1 and shape[-1] > 1:
        raise ValueError("%s must have unit stride along its last dimension" % what)


def _dense(t, what, shape, dtype, device):
    """Checks an optional contiguous operand."""
    _like(t, what, shape, dtype, device)
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % what)


def _cuda(t, what):
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % what)
    if t.stride(-1) != 1 and t.shape[-1] > 1:
        raise ValueError("%s must have unit stride along its last dimension" % what)


def _own_rows(t, what):
    """Checks that an output's rows do not lie on each other (as an expanded tensor's do)."""
    if any(s == 0 and n > 1 for s, n in zip(t.stride(), t.shape)):
        raise ValueError("%s must not be an expanded tensor" % what)


def _p(t):
    return None if t is None else t.data_ptr()


class _On:
    """Where a call runs: the stream handle, with allocation on that stream and the
    tensor's device current inside the block."""

    __slots__ = ("handle", "guards")

    def __init__(self, x, stream, inputs=()):
        self.guards = ()
        if x.device.index != torch.cuda.current_device():
            self.guards = (torch.cuda.device(x.device),)
        if stream is None:
            self.handle = _raw_stream(x.device.index) if _raw_stream else torch.cuda.current_stream(x.device).cuda_stream
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


def _strides(*ts):
    """The leading strides of each tensor, as a host array (0 for a missing one)."""
    lead = next(t for t in ts if t is not None).dim() - 1
    flat = []
    for t in ts:
        flat += t.stride()[:lead] if t is not None else (0,) * lead
    return (ctypes.c_int64 * len(flat))(*flat)


def _starts(starts, shape, device):
    if starts.dtype == torch.bool:
        starts = starts.view(torch.uint8)
    _dense(starts, "starts", shape, torch.uint8, device)
    return starts


def recurrence(x, f, i=None, h0=None, starts=None, out=None, stream=None):
    """Gated linear recurrence h_t = a_t h_{t-1} + u_t x_t over dim 1 of (batch, length,
    channels) tensors; a = sigmoid(f), u = sigmoid(i), or 1 - a without i.  h0 (batch,
    channels) fp32 is the state to start from, starts (batch, length) uint8 or bool marks
    tokens before which the state is dropped.  Returns (h, last): h like x, last the fp32
    state after the final token."""
    if x.dim() != 3:
        raise ValueError("x must be (batch, length, channels)")
    _cuda(x, "x")
    code, shape, dev = _code(x, "x"), x.shape, x.device
    _like(f, "f", shape, x.dtype, dev)
    if i is not None:
        _like(i, "i", shape, x.dtype, dev)
    b, t, d = shape
    if h0 is not None:
        _dense(h0, "h0", (b, d), torch.float32, dev)
    if starts is not None:
        starts = _starts(starts, (b, t), dev)
    if out is not None:
        _like(out, "out", shape, x.dtype, dev)
        _own_rows(out, "out")
    with _On(x, stream, (x, f, i, h0, starts, out)) as s:
        if out is None:
            out = torch.empty(shape, dtype=x.dtype, device=dev)
        last = torch.empty((b, d), dtype=torch.float32, device=dev)
        rc = load().gb_recurrence(code, b, t, d, x.data_ptr(), f.data_ptr(), _p(i), _strides(x, f, i, out), _p(h0),
                                  _p(starts), out.data_ptr(), last.data_ptr(), s)
    if rc:
        _check(rc, "gb_recurrence")
    return out, last


def recurrence_backward(dh, x, f, h, i=None, h0=None, starts=None, dlast=None, out=None, stream=None):
    """Gradient of recurrence() from its inputs, its output h and the gradients dh of h
    and dlast (fp32, or None) of the last state.  Returns (dx, df, di, dh0), di None
    without i.  `out` gives the tensors for (dx, df, di), such as slices of one buffer."""
    if x.dim() != 3:
        raise ValueError("x must be (batch, length, channels)")
    _cuda(x, "x")
    code, shape, dev = _code(x, "x"), x.shape, x.device
    for t, what in ((dh, "dh"), (f, "f"), (h, "h"), (i, "i")):
        if t is not None or what != "i":
            _like(t, what, shape, x.dtype, dev)
    b, t, d = shape
    for v, what in ((h0, "h0"), (dlast, "dlast")):
        if v is not None:
            _dense(v, what, (b, d), torch.float32, dev)
    if starts is not None:
        starts = _starts(starts, (b, t), dev)
    dx = df = di = None
    if out is not None:
        dx, df, di = out
        for v, what in ((dx, "dx"), (df, "df"), (di, "di")):
            if what != "di" or i is not None:
                _like(v, what, shape, x.dtype, dev)
                _own_rows(v, what)
    with _On(x, stream, (dh, x, f, h, i, h0, starts, dlast, dx, df, di)) as s:
        if out is None:
            dx = torch.empty(shape, dtype=x.dtype, device=dev)
            df = torch.empty(shape, dtype=x.dtype, device=dev)
            di = torch.empty(shape, dtype=x.dtype, device=dev) if i is not None else None
        dh0 = torch.empty((b, d), dtype=torch.float32, device=dev)
        rc = load().gb_recurrence_backward(code, b, t, d, dh.data_ptr(), x.data_ptr(), f.data_ptr(), _p(i),
                                           h.data_ptr(), _strides(dh, x, f, i, h, dx, df, di if i is not None else None),
                                           _p(h0), _p(starts), _p(dlast), dx.data_ptr(), df.data_ptr(), _p(di),
                                           dh0.data_ptr(), s)
    if rc:
        _check(rc, "gb_recurrence_backward")
    return dx, df, di if i is not None else None, dh0


def recurrence_step(x, f, state, i=None, slots=None, out=None, stream=None):
    """One token for each row of (batch, channels) tensors: the recurrence from
    state[slots[b]] (fp32, (pool, channels)), which is updated in place.  slots int32;
    None: row b uses state b; negative: padding, whose output is zero.  Returns h."""
    if x.dim() != 2 or state.dim() != 2:
        raise ValueError("x must be (batch, channels) and state (pool, channels)")
    _cuda(x, "x")
    code, shape, dev = _code(x, "x"), x.shape, x.device
    _like(f, "f", shape, x.dtype, dev)
    if i is not None:
        _like(i, "i", shape, x.dtype, dev)
    b, d = shape
    pool = state.shape[0]
    _dense(state, "state", (pool, d), torch.float32, dev)
    if slots is not None:
        _dense(slots, "slots", (b,), torch.int32, dev)
    elif b > pool:
        raise ValueError("state has %d rows for a batch of %d" % (pool, b))
    if out is not None:
        _like(out, "out", shape, x.dtype, dev)
        _own_rows(out, "out")
    with _On(x, stream, (x, f, i, state, slots, out)) as s:
        if out is None:
            out = torch.empty(shape, dtype=x.dtype, device=dev)
        rc = load().gb_recurrence_step(code, b, d, x.data_ptr(), f.data_ptr(), _p(i), _strides(x, f, i, out),
                                       state.data_ptr(), pool, _p(slots), out.data_ptr(), s)
    if rc:
        _check(rc, "gb_recurrence_step")
    return out


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


def _param(p, what, x, d):
    if p.dtype != x.dtype and p.dtype != torch.float32:
        raise TypeError("%s must be %s or fp32, not %s" % (what, x.dtype, p.dtype))
    _dense(p, what, (d,), p.dtype, x.device)


def layer_norm(x, weight=None, bias=None, eps: float = 1e-5, out=None, stream=None):
    """Layer norm over the last dimension: (y, mean, rstd), mean and rstd fp32 with one
    entry a row.  weight and bias: of x's type or fp32, or None."""
    x2 = _rows(x, "x")
    _cuda(x2, "x")
    code, (n, d) = _code(x, "x"), x2.shape
    pcode = code
    for p, what in ((weight, "weight"), (bias, "bias")):
        if p is not None:
            _param(p, what, x, d)
            pcode = _DTYPES[p.dtype]
    if weight is not None and bias is not None and weight.dtype != bias.dtype:
        raise TypeError("weight and bias must have the same type")
    if d == 0 and n:
        raise ValueError("x must have at least one column")
    if out is not None:
        _like(out, "out", x.shape, x.dtype, x.device)
        _own_rows(out, "out")
    with _On(x, stream, (x, weight, bias, out)) as s:
        if out is None:
            out = torch.empty(x.shape, dtype=x.dtype, device=x.device)
        y2 = out if out.dim() == 2 else _rows(out, "out")
        mean, rstd = torch.empty((2, n), dtype=torch.float32, device=x.device).unbind(0)
        rc = load().gb_layer_norm(code, pcode, n, d, x2.data_ptr(), x2.stride(0), _p(weight), _p(bias), eps,
                                  y2.data_ptr(), y2.stride(0), mean.data_ptr(), rstd.data_ptr(), s)
    if rc:
        _check(rc, "gb_layer_norm")
    return out, mean, rstd


def layer_norm_backward(dy, x, mean, rstd, weight=None, bias: bool = True, temp=None, stream=None):
    """Gradient of layer_norm() from its input and its mean and rstd: (dx, dweight,
    dbias), the last two of weight's type (None without a weight; dbias None too with
    bias=False)."""
    x2, dy2 = _rows(x, "x"), _rows(dy, "dy")
    _cuda(x2, "x")
    code, (n, d) = _code(x, "x"), x2.shape
    _like(dy2, "dy", x2.shape, x.dtype, x.device)
    for v, what in ((mean, "mean"), (rstd, "rstd")):
        _dense(v, what, (n,), torch.float32, x.device)
    pcode = code
    if weight is not None:
        _param(weight, "weight", x, d)
        pcode = _DTYPES[weight.dtype]
    dw = db = None
    with _On(x, stream, (dy, x, mean, rstd, weight, temp)) as s:
        dx = torch.empty(x.shape, dtype=x.dtype, device=x.device)
        tp, tb = None, 0
        if weight is not None:
            if bias:
                dw, db = torch.empty((2, d), dtype=weight.dtype, device=x.device).unbind(0)
            else:
                dw = torch.empty((d,), dtype=weight.dtype, device=x.device)
            if temp is None:
                tb = load().gb_layer_norm_temp_bytes(n, d)
                temp = torch.empty(max(tb, 1), dtype=torch.uint8, device=x.device)
            else:
                tb = temp.numel() * temp.element_size()
            tp = temp.data_ptr()
        rc = load().gb_layer_norm_backward(code, pcode, n, d, dy2.data_ptr(), dy2.stride(0), x2.data_ptr(),
                                           x2.stride(0), mean.data_ptr(), rstd.data_ptr(), _p(weight), dx.data_ptr(),
                                           d, _p(dw), _p(db), tp, tb, s)
    if rc:
        _check(rc, "gb_layer_norm_backward")
    return dx, dw, db


def _targets(targets, n, device):
    if targets.dtype not in (torch.int32, torch.int64):
        raise TypeError("targets must be int32 or int64, not %s" % targets.dtype)
    _dense(targets, "targets", (n,), targets.dtype, device)
    return I64 if targets.dtype == torch.int64 else I32


def token_logprobs(logits, targets, top: int = 0, stream=None):
    """Of each row of (rows, vocab) logits: the log probability of its target (int32 or
    int64; negative: ignored, 0), the entropy, the log of the sum of exponentials, and the
    `top` (0 .. 32) most likely tokens' log probabilities and int32 ids, in falling order,
    ties to the lower id (None, None for top=0).  A logit of -inf is masked."""
    if logits.dim() != 2:
        raise ValueError("logits must be (rows, vocab)")
    _cuda(logits, "logits")
    code, (n, v), dev = _code(logits, "logits"), logits.shape, logits.device
    tcode = _targets(targets, n, dev)
    if not 0 <= top <= min(32, v):
        raise ValueError("top must be between 0 and 32, and at most the vocabulary")
    values = ids = None
    with _On(logits, stream, (logits, targets)) as s:
        logprob, entropy, lse = torch.empty((3, n), dtype=torch.float32, device=dev).unbind(0)
        if top:
            values = torch.empty((n, top), dtype=torch.float32, device=dev)
            ids = torch.empty((n, top), dtype=torch.int32, device=dev)
        rc = load().gb_token_logprobs(code, n, v, logits.data_ptr(), logits.stride(0), targets.data_ptr(), tcode,
                                      logprob.data_ptr(), entropy.data_ptr(), lse.data_ptr(), top, _p(values),
                                      _p(ids), s)
    if rc:
        _check(rc, "gb_token_logprobs")
    return TokenLogprobs(logprob, entropy, lse, values, ids)


def token_logprobs_backward(logits, targets, lse, entropy=None, dlogprob=None, dentropy=None, out=None, stream=None):
    """Gradient of token_logprobs()'s logprob and entropy with respect to the logits, from
    its lse and entropy: dlogits like logits.  dlogprob, dentropy: (rows) fp32 or None for
    zero.  out may be logits itself, which is then overwritten."""
    if logits.dim() != 2:
        raise ValueError("logits must be (rows, vocab)")
    _cuda(logits, "logits")
    code, (n, v), dev = _code(logits, "logits"), logits.shape, logits.device
    tcode = _targets(targets, n, dev)
    for t, what in ((lse, "lse"), (entropy, "entropy"), (dlogprob, "dlogprob"), (dentropy, "dentropy")):
        if t is not None:
            _dense(t, what, (n,), torch.float32, dev)
    if dentropy is not None and entropy is None:
        raise ValueError("dentropy needs the entropy")
    if out is not None:
        _like(out, "out", logits.shape, logits.dtype, dev)
        _own_rows(out, "out")
    with _On(logits, stream, (logits, targets, lse, entropy, dlogprob, dentropy, out)) as s:
        if out is None:
            out = torch.empty((n, v), dtype=logits.dtype, device=dev)
        rc = load().gb_token_logprobs_backward(code, n, v, logits.data_ptr(), logits.stride(0), targets.data_ptr(),
                                               tcode, lse.data_ptr(), _p(entropy), _p(dlogprob), _p(dentropy),
                                               out.data_ptr(), out.stride(0), s)
    if rc:
        _check(rc, "gb_token_logprobs_backward")
    return out
