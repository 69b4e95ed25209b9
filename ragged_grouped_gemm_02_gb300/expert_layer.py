"""One expert layer through the library's operators: forward and backward for
training, and its 4-bit and 8-bit forms for serving.

The layer is ``Y_e = (silu(X_e . W13_e[:, :N]) * (X_e . W13_e[:, N:])) . W2_e`` on rows
grouped by expert.  Its backward pass keeps nothing of the forward pass but the
inputs: ``rgg_grouped_gemm_swiglu_backward`` computes gate and up again.
"""
from __future__ import annotations

import torch
from torch.autograd.function import once_differentiable

from . import (rgg_fp8_block_quantize, rgg_fp8_block_quantize_weights, rgg_grouped_gemm, rgg_grouped_gemm_dgrad,
               rgg_grouped_gemm_fp8_block, rgg_grouped_gemm_mxfp4, rgg_grouped_gemm_swiglu,
               rgg_grouped_gemm_swiglu_backward, rgg_grouped_gemm_swiglu_fp8_block, rgg_grouped_gemm_swiglu_mxfp4,
               rgg_grouped_gemm_wgrad, rgg_mxfp4_quantize, rgg_mxfp4_quantize_weights)

__all__ = ["expert_ffn", "quantize_experts", "expert_ffn_mxfp4", "quantize_experts_fp8", "expert_ffn_fp8"]


class _ExpertFFN(torch.autograd.Function):
    @staticmethod
    def forward(ctx, X, W13, W2, group_offsets):
        ctx.save_for_backward(X, W13, W2, group_offsets)
        H = rgg_grouped_gemm_swiglu(X, W13, group_offsets)
        Y = torch.zeros(X.shape[0], W2.shape[2], dtype=X.dtype, device=X.device)  # rows of no expert: zero
        return rgg_grouped_gemm(H, W2, group_offsets, Y)

    @staticmethod
    @once_differentiable
    def backward(ctx, dY):
        X, W13, W2, group_offsets = ctx.saved_tensors
        dY = dY.contiguous()
        dH = rgg_grouped_gemm_dgrad(dY, W2, group_offsets)
        dGU, H = rgg_grouped_gemm_swiglu_backward(X, W13, group_offsets, dH,
                                                  H=None if ctx.needs_input_grad[2] else False)
        dX = dW13 = dW2 = None
        if ctx.needs_input_grad[2]:
            dW2 = rgg_grouped_gemm_wgrad(H, dY, group_offsets)
        if ctx.needs_input_grad[1]:
            dW13 = rgg_grouped_gemm_wgrad(X, dGU, group_offsets)
        if ctx.needs_input_grad[0]:
            dX = rgg_grouped_gemm_dgrad(dGU, W13, group_offsets, torch.zeros_like(X))
        return dX, dW13, dW2, None


def expert_ffn(X, W13, W2, group_offsets):
    """Y for routed rows X, with gradients by X, W13 and W2 (first derivatives: the
    gradients cannot be differentiated again, and autograd raises if asked to).

    X: bf16 CUDA [M_tot, K], rows grouped by expert; W13: bf16 CUDA [E, K, 2N]
    (gate columns first); W2: bf16 CUDA [E, N, K_out]; group_offsets: int32
    CUDA [E+1].  Rows of no expert get zeros, in Y and in the gradient."""
    return _ExpertFFN.apply(X, W13, W2, group_offsets)


def _whole_blocks(W13, W2):
    """The weights detached, of a width N of whole 128s: zero columns of gate and up and zero rows of W2 behind the others."""
    W13, W2 = W13.detach(), W2.detach()
    N = W2.shape[1] if W2.dim() == 3 else 0
    if W13.dim() != 3 or N == 0 or W13.shape[2] != 2 * N:
        raise ValueError("W13 must be [E, K, 2N] and W2 [E, N, K_out], not %s and %s" % (tuple(W13.shape), tuple(W2.shape)))
    fill = -N % 128
    if fill:
        W13 = torch.cat([torch.nn.functional.pad(half, (0, fill)) for half in W13.split(N, 2)], 2)
        W2 = torch.nn.functional.pad(W2, (0, 0, 0, fill))
    return W13, W2


def quantize_experts(W13, W2):
    """The layer's weights in MXFP4, laid out once: what ``expert_ffn_mxfp4`` takes.

    The gate-up product takes widths N of whole 128s, so other widths are filled
    up with zero columns of gate and up and zero rows of W2: their activations are
    0 and add nothing.  (A width of 1344 becomes 1408: 5 % more weight.)"""
    W13, W2 = _whole_blocks(W13, W2)
    return rgg_mxfp4_quantize_weights(W13), rgg_mxfp4_quantize_weights(W2)


def expert_ffn_mxfp4(X, experts, group_offsets):
    """Y for routed rows X with 4-bit weights (``quantize_experts``) and
    activations quantised on the way.  K must be a multiple of 32, K_out of 8.
    Rows of no expert hold unspecified values.

    What to expect of 4 bits: one rounding of normally distributed values is off
    by 0.115 of their root mean square.  The layer rounds four times (X, W13, H
    and W2); on random normal inputs and weights Y is off by 0.30 of its own, 0.20
    of it from the weights alone."""
    w13, w2 = experts
    H = rgg_grouped_gemm_swiglu_mxfp4(*rgg_mxfp4_quantize(X, group_offsets), *w13, group_offsets)
    return rgg_grouped_gemm_mxfp4(*rgg_mxfp4_quantize(H, group_offsets), *w2, group_offsets)


def quantize_experts_fp8(W13, W2):
    """The layer's weights in 8 bits with a scale per 128 x 128, laid out once: what ``expert_ffn_fp8`` takes.

    Widths N that are not whole 128s are filled up with zeros, as for ``quantize_experts``.  Weights that are in
    this form already (codes [E, 2N, K] and [E, K_out, N] with their scales) need no call: pass them as they are."""
    W13, W2 = _whole_blocks(W13, W2)
    return rgg_fp8_block_quantize_weights(W13), rgg_fp8_block_quantize_weights(W2)


def expert_ffn_fp8(X, experts, group_offsets):
    """Y for routed rows X with 8-bit weights (``quantize_experts_fp8``) and activations quantised on the way.

    X: bf16 CUDA [M_tot, K], or the ``(codes, scales)`` of ``rgg_fp8_block_quantize``; K must be a multiple of 16,
    K_out of 8.  The activation between the two products never leaves 8 bits.  Rows of no expert hold unspecified
    values."""
    w13, w2 = experts
    if isinstance(X, torch.Tensor):
        X = rgg_fp8_block_quantize(X)
    H = rgg_grouped_gemm_swiglu_fp8_block(*X, *w13, group_offsets)
    return rgg_grouped_gemm_fp8_block(*H, *w2, group_offsets)
