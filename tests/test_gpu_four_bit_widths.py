"""The 4-bit expert layer at widths that are no multiple of 128, on a GB300: against the definition's roundings of the
layer as it is, in 64 bits."""
import pytest
import torch

import expert_refs as refs
import ragged_grouped_gemm_02_gb300 as rgg
from ragged_grouped_gemm_02_gb300 import _build
from ragged_grouped_gemm_02_gb300.expert_layer import expert_ffn, expert_ffn_mxfp4, quantize_experts

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available(), "the gpu tests need a CUDA device"
    _build.build()


def _mx(x):
    """What MXFP4 holds of x (fp64 [..., K]), the last block filled up with zeros."""
    K = x.shape[-1]
    b = torch.nn.functional.pad(x, (0, -K % 32)).reshape(*x.shape[:-1], -1, 32)
    top = b.abs().amax(-1, keepdim=True)
    exponent = torch.frexp(top).exponent - 1
    scale = torch.where(top > 0, 2.0 ** torch.clamp(exponent - 2, min=-127).double(), 1.0)
    v = (b / scale).abs().clamp(max=6.0)
    step = torch.where(v < 2, 0.5, torch.where(v < 4, 1.0, 2.0)).double()
    return (torch.sign(b) * torch.round(v / step) * step * scale).flatten(-2)[..., :K]


def _layer(counts, K, N, K_out, seed):
    gen = torch.Generator().manual_seed(seed)
    off, M = refs.ragged(counts)
    E = len(counts)
    return (refs.normal(gen, M, K), refs.normal(gen, E, K, 2 * N, std=K ** -0.5),
            refs.normal(gen, E, N, K_out, std=N ** -0.5), off)


# 1344: half of the 2688 gate-up columns of the repository's workloads
@pytest.mark.parametrize("K,N,K_out", [(64, 1344, 72), (1024, 1344, 1024), (64, 8, 64), (96, 136, 104), (32, 200, 8),
                                       (64, 128, 64)])
def test_widths(K, N, K_out):
    X, W13, W2, off = _layer([5, 0, 130, 33], K, N, K_out, seed=N)
    experts = quantize_experts(W13.cuda(), W2.cuda())
    got = expert_ffn_mxfp4(X.cuda(), experts, torch.from_numpy(off).cuda())
    assert rgg.rgg_query_status(0) == rgg.RGG_OK and got.shape == (X.shape[0], K_out)
    x, w13 = _mx(X.double()), _mx(W13.double().transpose(1, 2))
    w2 = _mx(W2.double().transpose(1, 2))
    want = torch.empty(X.shape[0], K_out, dtype=torch.float64)
    for e, (a, b) in enumerate(refs.spread(off)):
        if a == b:
            continue
        h = refs.swiglu(x[a:b] @ w13[e].t()).to(torch.bfloat16)
        want[a:b] = _mx(h.double()) @ w2[e].t()
    # H's rounding to bf16 may move a code now and then
    assert float((got.cpu().double() - want).norm() / want.norm()) < 0.02


def test_the_layer_that_was_trained_is_served():
    # a trained layer's weights go straight to the 4-bit form; each of its three roundings to 4 bits is about 0.1 of a value
    X, W13, W2, off = _layer([16] * 8, 1024, 1344, 1024, seed=1)
    w13, w2, offg = W13.cuda().requires_grad_(), W2.cuda().requires_grad_(), torch.from_numpy(off).cuda()
    full = expert_ffn(X.cuda(), w13, w2, offg)
    full.float().square().mean().backward()
    four = expert_ffn_mxfp4(X.cuda(), quantize_experts(w13, w2), offg)
    assert 0 < float((four - full.detach()).float().norm() / full.detach().float().norm()) < 0.5


def test_refusals():
    X, W13, W2, off = _layer([5], 64, 136, 64, seed=2)
    with pytest.raises(ValueError):
        quantize_experts(W13.cuda(), W2[:, :128].contiguous().cuda())
    with pytest.raises(ValueError):
        quantize_experts(W13[:, :, :256].contiguous().cuda(), W2.cuda())
    with pytest.raises(ValueError):
        quantize_experts(W13[0].cuda(), W2.cuda())
    with pytest.raises(ValueError):
        quantize_experts(W13.cuda(), W2[0, 0].cuda())
