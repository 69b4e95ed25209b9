"""A mixture-of-experts layer through the library's operators: the router's choices,
tokens sorted by expert, the expert layer, and the weighted sum back.

    out[t] = sum_j w[t, j] * ffn_{e[t, j]}(x[t]),   (e, w) the k largest of the token's logits and their weights

``moe_ffn`` has gradients by the tokens, the logits and the experts' weights;
``moe_ffn_fp8`` is the serving form with 8-bit experts.  The logits are the caller's
(a product of the tokens with the router's weight, say), so that masks (-inf) and biases
are too.  Choices and weights come from the same logits: a bias that is to move the
choices alone has no place here.
"""
from __future__ import annotations

import functools

import torch

from . import (rgg_combine, rgg_combine_backward, rgg_dispatch, rgg_moe_swiglu_fp8_block, rgg_route_topk,
               rgg_route_topk_backward, rgg_sort_by_expert)
from .expert_layer import expert_ffn

__all__ = ["route_topk", "dispatch", "combine", "moe_ffn", "moe_ffn_fp8"]


class _NoSecondDerivative(torch.autograd.Function):
    @staticmethod
    def forward(ctx, t):
        return t.view_as(t)

    @staticmethod
    def backward(ctx, _):
        raise RuntimeError("trying to differentiate twice through a function that has first derivatives only")


def _first_derivatives(backward):
    """A backward pass whose results raise where they are differentiated again.  (once_differentiable does so only
    where the incoming gradient depends on something; these results depend on the saved tensors too.)"""
    @functools.wraps(backward)
    def wrapped(ctx, *grads):
        with torch.no_grad():
            out = backward(ctx, *grads)
        if not torch.is_grad_enabled():  # no graph of the backward pass is wanted
            return out
        return tuple(t if t is None else _NoSecondDerivative.apply(t.detach().requires_grad_()) for t in out)
    return wrapped


class _RouteTopk(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, k, score, renormalize, scale):
        experts, weights = rgg_route_topk(logits, k, score=score, renormalize=renormalize, scale=scale)
        ctx.save_for_backward(logits, experts)
        ctx.rule = {"score": score, "renormalize": renormalize, "scale": scale}
        ctx.mark_non_differentiable(experts)
        return experts, weights

    @staticmethod
    @_first_derivatives
    def backward(ctx, _, dweights):
        logits, experts = ctx.saved_tensors
        return rgg_route_topk_backward(logits, experts, dweights.contiguous(), **ctx.rule), None, None, None, None


def route_topk(logits, k, *, score="softmax", renormalize=True, scale=1.0):
    """``rgg_route_topk`` with the weights' gradient by the logits (first derivatives)."""
    return _RouteTopk.apply(logits, k, score, renormalize, scale)


class _Dispatch(torch.autograd.Function):
    @staticmethod
    def forward(ctx, X, position):
        ctx.save_for_backward(position)
        return rgg_dispatch(X, position)

    @staticmethod
    @_first_derivatives
    def backward(ctx, dXs):
        return rgg_combine(dXs.contiguous(), ctx.saved_tensors[0]), None


def dispatch(X, position):
    """``rgg_dispatch`` of bf16 tokens with its gradient by them; rows of no choice hold unspecified values, and what
    comes back for them is not read."""
    if X.is_cuda and X.dtype is not torch.bfloat16:
        raise TypeError("X must be bf16, as its gradient is, not %s (rgg_dispatch takes any type)" % X.dtype)
    return _Dispatch.apply(X, position)


class _Combine(torch.autograd.Function):
    @staticmethod
    def forward(ctx, Y, position, weights, whole):
        ctx.save_for_backward(Y, position, weights)
        ctx.whole = whole
        return rgg_combine(Y, position, weights)

    @staticmethod
    @_first_derivatives
    def backward(ctx, dout):
        Y, position, weights = ctx.saved_tensors
        dY = False
        if ctx.needs_input_grad[0]:
            # rows of no choice: zero, or unspecified where nobody looks at them (anomaly mode looks for NaN)
            dY = torch.zeros_like(Y) if ctx.whole or torch.is_anomaly_enabled() else None
        dY, dweights = rgg_combine_backward(dout.contiguous(), Y, position, weights, dY,
                                            None if ctx.needs_input_grad[2] else False)
        return dY, None, dweights, None


def combine(Y, position, weights):
    """``rgg_combine`` with its gradients by Y (zero for rows of no choice) and the weights."""
    if not isinstance(weights, torch.Tensor):
        raise TypeError("weights must be a tensor [T, k] (rgg_combine takes None, for sums without weights)")
    return _Combine.apply(Y, position, weights, True)


def moe_ffn(X, logits, W13, W2, k, *, score="softmax", renormalize=True, scale=1.0):
    """The layer's output for tokens X, with gradients by X, logits, W13 and W2 (first derivatives).

    X: bf16 CUDA [T, K]; logits: bf16, fp16 or fp32 CUDA [T, E]; W13: bf16 CUDA [E, K, 2N] (gate columns first);
    W2: bf16 CUDA [E, N, K_out]; k, score, renormalize, scale: as for ``rgg_route_topk``.  A token whose logits
    are all -inf gets zeros."""
    if logits.dim() != 2 or logits.shape[1] != W13.shape[0]:
        raise ValueError("logits must be [T, E] with E = %d experts, not %s" % (W13.shape[0], tuple(logits.shape)))
    experts, weights = route_topk(logits, k, score=score, renormalize=renormalize, scale=scale)
    group_offsets, _, position = rgg_sort_by_expert(experts, W13.shape[0])
    Y = expert_ffn(dispatch(X, position), W13, W2, group_offsets)
    # whose backward pass reads the experts' rows alone: the others' gradient need not be filled with zeros
    return _Combine.apply(Y, position, weights, False)


def moe_ffn_fp8(X, logits, experts, k, *, score="softmax", renormalize=True, scale=1.0):
    """The layer's output for tokens X with 8-bit experts (``expert_layer.quantize_experts_fp8``), for serving: a token
    is quantised once and goes to its experts in 8 bits.  X: bf16 CUDA [T, K], K a multiple of 16.  One call of the
    library: ``rgg_moe_swiglu_fp8_block``."""
    w13, w2 = experts
    return rgg_moe_swiglu_fp8_block(X, logits, *w13, *w2, k, score=score, renormalize=renormalize, scale=scale)
