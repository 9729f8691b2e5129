"""The language-model operators as differentiable torch functions: the forward and
gradient calls of lm.py and ssm.py joined, so that they can stand in a module's forward pass.

    h, last = autograd.recurrence(x, f, i, h0, starts)
    y = autograd.layer_norm(x, weight, bias)
    logprob, entropy = autograd.token_logprobs(logits, targets)
    y, last = autograd.causal_conv(x, weight, bias, state, starts)
    y, last = autograd.selective_scan(x, dt, a, b, c, d, z, dt_bias, h0, starts)

All compute is in the library's kernels, forward and backward; gradients are
deterministic, and cannot be differentiated again.  The gradients of a recurrence's inputs
come from one pass together, as those of a selective scan, and layer norm's and the
convolution's dx always; their weight's and bias's only where they are asked for.  The
backward calls run on the stream that torch's autograd makes current, which is the forward
call's.

A forward and backward pass can be captured into a CUDA graph while no eager graph of the same
leaves is alive (a loss that was kept is one): torch accumulates a leaf's gradient on the stream
of the graph that used it first, and a capture that meets another stream is void, which
loss.backward() does not survive.  Capture before the first eager pass, or delete its results.
"""
from __future__ import annotations

import torch
from torch.autograd.function import once_differentiable

from . import lm, ssm


def _unit(t):
    """A gradient as the kernels read it: unit stride along the last dimension."""
    return t if t.stride(-1) == 1 or t.shape[-1] <= 1 else t.contiguous()


class _Recurrence(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, f, i, h0, starts):
        h, last = lm.recurrence(x, f, i, h0=h0, starts=starts)
        ctx.save_for_backward(x, f, i, h0, starts, h)
        ctx.set_materialize_grads(False)
        return h, last

    @staticmethod
    @once_differentiable
    def backward(ctx, dh, dlast):
        x, f, i, h0, starts, h = ctx.saved_tensors
        if dh is None and dlast is None:
            return None, None, None, None, None
        dh = torch.zeros_like(h) if dh is None else _unit(dh)
        dlast = None if dlast is None else dlast.contiguous()
        dx, df, di, dh0 = lm.recurrence_backward(dh, x, f, h, i, h0=h0, starts=starts, dlast=dlast)
        return dx, df, di, dh0 if h0 is not None else None, None


class _LayerNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, eps):
        y, mean, rstd = lm.layer_norm(x, weight, bias, eps=eps)
        ctx.save_for_backward(x, weight, bias, mean, rstd)
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        x, weight, bias, mean, rstd = ctx.saved_tensors
        dy = dy if dy.is_contiguous() else dy.contiguous()
        _, dweight, dbias, _ = ctx.needs_input_grad  # frozen parameters cost no sums over rows
        scale = weight if weight is not None or not dbias else torch.ones_like(bias)
        dx, dw, db = lm.layer_norm_backward(dy, x, mean, rstd, scale, bias=dbias, dweight=dweight)
        return dx, dw, db, None


class _TokenLogprobs(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, targets):
        r = lm.token_logprobs(logits, targets)
        ctx.save_for_backward(logits, targets, r.lse, r.entropy)
        ctx.set_materialize_grads(False)
        return r.logprob, r.entropy

    @staticmethod
    @once_differentiable
    def backward(ctx, dlogprob, dentropy):
        logits, targets, lse, entropy = ctx.saved_tensors
        if dlogprob is None and dentropy is None:
            return None, None
        dlogprob = None if dlogprob is None else dlogprob.contiguous()
        dentropy = None if dentropy is None else dentropy.contiguous()
        return lm.token_logprobs_backward(logits, targets, lse, entropy, dlogprob, dentropy), None


class _CausalConv(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, state, starts, silu):
        y, last = ssm.causal_conv(x, weight, bias, state=state, starts=starts, silu=silu)
        ctx.save_for_backward(x, weight, bias, state, starts)
        ctx.silu = silu
        ctx.set_materialize_grads(False)
        return y, last

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, dlast):
        x, weight, bias, state, starts = ctx.saved_tensors
        if dy is None and dlast is None:
            return (None,) * 6
        dy = torch.zeros(x.shape, dtype=x.dtype, device=x.device) if dy is None else _unit(dy)
        dlast = None if dlast is None else dlast.contiguous()
        _, dw, db, _, _, _ = ctx.needs_input_grad  # frozen parameters cost no sums over tokens
        dx, dweight, dbias, dstate = ssm.causal_conv_backward(dy, x, weight, bias, state=state, starts=starts, dlast=dlast,
                                                              silu=ctx.silu, dparams=dw or db)
        return dx, dweight, dbias, dstate, None, None


class _SelectiveScan(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, dt, a, b, c, d, z, dt_bias, h0, starts, softplus, grads):
        # needs_input_grad says what requires a gradient, with gradients switched off too.
        y, last, kept = ssm.selective_scan(x, dt, a, b, c, d, z, dt_bias, h0=h0, starts=starts, softplus=softplus,
                                           keep=grads and any(ctx.needs_input_grad))
        ctx.save_for_backward(x, dt, a, b, c, d, z, dt_bias, h0, starts, kept)
        ctx.softplus = softplus
        ctx.set_materialize_grads(False)
        return y, last

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, dlast):
        x, dt, a, b, c, d, z, dt_bias, h0, starts, kept = ctx.saved_tensors
        if dy is None and dlast is None:
            return (None,) * 12
        dy = torch.zeros(x.shape, dtype=x.dtype, device=x.device) if dy is None else _unit(dy)
        dlast = None if dlast is None else dlast.contiguous()
        g = ssm.selective_scan_backward(dy, x, dt, a, b, c, kept, d, z, dt_bias, starts=starts, dlast=dlast,
                                        softplus=ctx.softplus)
        return g.dx, g.ddt, g.da, g.db, g.dc, g.dd, g.dz, g.ddt_bias, g.dh0 if h0 is not None else None, None, None, None


def recurrence(x, f, i=None, h0=None, starts=None):
    """lm.recurrence(): (h, last), differentiable in x, f, i and h0."""
    return _Recurrence.apply(x, f, i, h0, starts)


def layer_norm(x, weight=None, bias=None, eps: float = 1e-5):
    """lm.layer_norm()'s y, differentiable in x, weight and bias."""
    return _LayerNorm.apply(x, weight, bias, eps)


def token_logprobs(logits, targets):
    """lm.token_logprobs()'s (logprob, entropy), differentiable in the logits."""
    return _TokenLogprobs.apply(logits, targets)


def causal_conv(x, weight, bias=None, state=None, starts=None, silu: bool = True):
    """ssm.causal_conv(): (y, last), differentiable in x, weight, bias and state."""
    return _CausalConv.apply(x, weight, bias, state, starts, silu)


def selective_scan(x, dt, a, b, c, d=None, z=None, dt_bias=None, h0=None, starts=None, softplus: bool = True):
    """ssm.selective_scan(): (y, last), differentiable in x, dt, a, b, c, d, z, dt_bias and h0."""
    return _SelectiveScan.apply(x, dt, a, b, c, d, z, dt_bias, h0, starts, softplus, torch.is_grad_enabled())
