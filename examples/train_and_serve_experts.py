"""Train one expert layer for a few steps, then serve it in 4 bits.

Routed rows go through the fused gate-up product and the down projection; the
backward pass runs the grouped gradients, the gradients are clipped by their
global norm, and plain SGD updates fp32 master weights.  The target is another
layer's output plus noise.  At the end the weights are quantised to MXFP4 and the
4-bit layer is compared with the bf16 one on a decode-sized batch.

    python examples/train_and_serve_experts.py [--steps N]
"""
import argparse
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import ragged_grouped_gemm_02_gb300 as rgg  # noqa: E402
from ragged_grouped_gemm_02_gb300 import workloads as wl  # noqa: E402
from ragged_grouped_gemm_02_gb300.expert_layer import expert_ffn, expert_ffn_mxfp4, quantize_experts  # noqa: E402


def main(steps=20, E=16, K=512, N=1024, rows=4096, seed=0):
    """Returns the losses of the steps and the 4-bit layer's relative error."""
    gen = torch.Generator().manual_seed(seed)
    offsets = torch.from_numpy(wl.offsets_from_counts(
        wl.power_law_counts_largest_remainder(rows, E, 1.2, gen))).cuda()

    def layer():
        return [(torch.randn(E, K, 2 * N, generator=gen) * K ** -0.5).cuda(),
                (torch.randn(E, N, K, generator=gen) * N ** -0.5).cuda()]

    target = [w.bfloat16() for w in layer()]
    master = layer()
    X = torch.randn(rows, K, generator=gen).cuda().bfloat16()
    want = expert_ffn(X, *target, offsets).float()

    losses = []
    for step in range(steps):
        params = [w.bfloat16().requires_grad_() for w in master]
        Y = expert_ffn(X, *params, offsets)
        loss = (Y.float() - want).square().mean()
        loss.backward()
        grads = [p.grad for p in params]
        norm = rgg.rgg_clip_grad_norm(grads, 0.03)
        for w, g in zip(master, grads):
            w.add_(g.float(), alpha=-20.0)
        losses.append(float(loss.detach()))
        print("step %2d  loss %.5f  gradient norm %.4f" % (step, losses[-1], float(norm)))

    trained = [w.bfloat16() for w in master]
    experts = quantize_experts(*trained)
    decode = torch.from_numpy(wl.offsets_from_counts(np.full(E, 4))).cuda()
    x = torch.randn(4 * E, K, generator=gen).cuda().bfloat16()
    full, four = expert_ffn(x, *trained, decode).float(), expert_ffn_mxfp4(x, experts, decode).float()
    error = float((four - full).norm() / full.norm())
    print("4-bit layer: relative error %.3f, weights %.2f MB instead of %.2f MB" % (
        error, sum(t.numel() for pair in experts for t in pair) / 1e6, sum(2 * w.numel() for w in trained) / 1e6))
    return losses, error


if __name__ == "__main__":
    parser = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    parser.add_argument("--steps", type=int, default=20)
    main(steps=parser.parse_args().steps)
