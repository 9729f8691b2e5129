"""The language-model operators as differentiable torch functions: the forward and
gradient calls of lm.py joined, so that they can stand in a module's forward pass.

    h, last = autograd.recurrence(x, f, i, h0, starts)
    y = autograd.layer_norm(x, weight, bias)
    logprob, entropy = autograd.token_logprobs(logits, targets)

All compute is in the library's kernels, forward and backward; gradients are
deterministic, and cannot be differentiated again.  The gradients of a recurrence's inputs
come from one pass together, and layer norm's dx always; its weight's and bias's only where
they are asked for.  The backward calls run on the stream that torch's autograd makes current,
which is the forward call's.
"""
from __future__ import annotations

import torch
from torch.autograd.function import once_differentiable

from . import lm


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


def recurrence(x, f, i=None, h0=None, starts=None):
    """lm.recurrence(): (h, last), differentiable in x, f, i and h0."""
    return _Recurrence.apply(x, f, i, h0, starts)


def layer_norm(x, weight=None, bias=None, eps: float = 1e-5):
    """lm.layer_norm()'s y, differentiable in x, weight and bias."""
    return _LayerNorm.apply(x, weight, bias, eps)


def token_logprobs(logits, targets):
    """lm.token_logprobs()'s (logprob, entropy), differentiable in the logits."""
    return _TokenLogprobs.apply(logits, targets)
