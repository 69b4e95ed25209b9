"""The expert layer of expert_layer.py: its gradients through autograd, its 4-bit form, and the example, on a GB300."""
import importlib.util
import os

import numpy as np
import pytest
import torch

import expert_refs as refs
import ragged_grouped_gemm_02_gb300 as rgg
from ragged_grouped_gemm_02_gb300 import _build
from ragged_grouped_gemm_02_gb300.expert_layer import expert_ffn, expert_ffn_mxfp4, quantize_experts

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available(), "the gpu tests need a CUDA device"
    _build.build()


def _layer(counts, K, N, seed, lead=0, spare=0):
    gen = torch.Generator().manual_seed(seed)
    off, M = refs.ragged(counts, lead, spare)
    E = len(counts)
    return (refs.normal(gen, M, K), refs.normal(gen, E, K, 2 * N, std=K ** -0.5),
            refs.normal(gen, E, N, K, std=N ** -0.5), off, refs.normal(gen, M, K))


def _reference(X, W13, W2, off, dY):
    """Y and the gradients in 64 bits, rows of no expert zero."""
    X, W13, W2, dY = (t.double() for t in (X, W13, W2, dY))
    gu = refs.gate_up(X, W13, off)[0]
    H = refs.swiglu(gu)
    Y, dX = torch.zeros_like(dY), torch.zeros_like(X)
    for e, (a, b) in enumerate(refs.spread(off)):
        Y[a:b] = H[a:b] @ W2[e]
    dH = refs.dgrad(dY, W2, off)[0]
    dGU, _ = refs.swiglu_backward(gu, dH)
    for e, (a, b) in enumerate(refs.spread(off)):
        dX[a:b] = dGU[a:b] @ W13[e].t()
    return Y, dX, refs.wgrad(X, dGU, off)[0], refs.wgrad(H, dY, off)[0]


def _close(got, ref, what):
    # a chain of up to three products with bf16 between them: each rounding is 2^-9 of a value of the chain, so the
    # result is off by a few times that of its root mean square
    rel = float((got.double().cpu() - ref).norm() / ref.norm())
    assert rel < 4 * 2.0 ** -8, "%s: relative error %.4g" % (what, rel)


@pytest.mark.parametrize("counts,lead,spare", [([70, 0, 200, 1, 130], 0, 0), ([16] * 8, 2, 3), ([600, 300], 0, 1)])
def test_gradients(counts, lead, spare):
    X, W13, W2, off, dY = _layer(counts, 256, 136, 1, lead, spare)
    x, w13, w2 = (t.cuda().requires_grad_() for t in (X, W13, W2))
    Y = expert_ffn(x, w13, w2, torch.from_numpy(off).cuda())
    Y.backward(dY.cuda())
    ref = _reference(X, W13, W2, off, dY)
    for got, r, what in zip((Y.detach(), x.grad, w13.grad, w2.grad), ref, ("Y", "dX", "dW13", "dW2")):
        _close(got, r, what)
    for t in (Y.detach(), x.grad):
        outside = torch.cat([t[: off[0]], t[off[-1]:]])
        assert not bool(outside.any()), "rows of no expert are zero"
    if 0 in counts:
        assert not bool(w13.grad[counts.index(0)].any())


def test_only_what_is_asked_for():
    X, W13, W2, off, dY = _layer([40, 60], 64, 128, 2)
    x = X.cuda().requires_grad_()
    w13, w2 = W13.cuda(), W2.cuda()
    expert_ffn(x, w13, w2, torch.from_numpy(off).cuda()).backward(dY.cuda())
    _close(x.grad, _reference(X, W13, W2, off, dY)[1], "dX")
    assert w13.grad is None and w2.grad is None


def test_four_bit_layer():
    # each of the three roundings to 4 bits (weights, rows, H) is about 0.1 of a value, and the products' errors add up
    X, W13, W2, off, _ = _layer([16] * 8, 256, 256, 3)
    offg = torch.from_numpy(off).cuda()
    experts = quantize_experts(W13.cuda(), W2.cuda())
    got = expert_ffn_mxfp4(X.cuda(), experts, offg).float().cpu()
    # against the same roundings in 64 bits
    x = rgg.rgg_mxfp4_dequantize(*rgg.rgg_mxfp4_quantize(X.cuda(), offg), offg).cpu().double()
    w13 = rgg.rgg_mxfp4_dequantize_weights(*experts[0]).cpu().double().transpose(1, 2)
    w2 = rgg.rgg_mxfp4_dequantize_weights(*experts[1]).cpu().double()
    H = refs.swiglu(refs.gate_up(x, w13, off)[0]).to(torch.bfloat16)
    h = rgg.rgg_mxfp4_dequantize(*rgg.rgg_mxfp4_quantize(H.cuda(), offg), offg).cpu().double()
    want = torch.cat([h[a:b] @ w2[e].t() for e, (a, b) in enumerate(refs.spread(off))])
    assert float((got - want).norm() / want.norm()) < 0.02  # H's rounding to bf16 may move a code now and then


def test_example_trains_and_serves(capsys):
    spec = importlib.util.spec_from_file_location("example", os.path.join(ROOT, "examples", "train_and_serve_experts.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    losses, error = module.main(steps=6, E=4, K=128, N=128, rows=512)
    assert all(np.isfinite(losses)) and losses[-1] < losses[0]
    assert 0 < error < 0.5
    assert "4-bit layer" in capsys.readouterr().out
