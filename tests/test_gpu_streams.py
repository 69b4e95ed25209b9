"""Calls of the expert layer's operators on a stream that is not the current one, on a GB300: their outputs come from
that stream's memory, so work that the current stream has still to do keeps its own."""
import numpy as np
import pytest
import torch

import ragged_grouped_gemm_02_gb300 as rgg
from ragged_grouped_gemm_02_gb300 import _build

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available(), "the gpu tests need a CUDA device"
    _build.build()


E, K, N, ROWS = 4, 256, 512, 1024


def _calls():
    gen = torch.Generator(device="cuda").manual_seed(0)

    def normal(*shape):
        return torch.empty(shape, dtype=torch.bfloat16, device="cuda").normal_(generator=gen)

    off = torch.from_numpy(np.arange(0, ROWS + 1, ROWS // E, dtype=np.int32)).cuda()
    X, dY, W, dH = normal(ROWS, K), normal(ROWS, N), normal(E, K, N), normal(ROWS, N // 2)
    xq, wq = rgg.rgg_mxfp4_quantize(X, off), rgg.rgg_mxfp4_quantize_weights(W)
    grads = [normal(E, K, N)]
    return {
        "dgrad": lambda s: rgg.rgg_grouped_gemm_dgrad(dY, W, off, stream=s),
        "wgrad": lambda s: rgg.rgg_grouped_gemm_wgrad(X, dY, off, stream=s),
        "swiglu_backward": lambda s: rgg.rgg_grouped_gemm_swiglu_backward(X, W, off, dH, stream=s),
        "clip": lambda s: rgg.rgg_clip_grad_norm(grads, 1e9, stream=s),
        "quantize": lambda s: rgg.rgg_mxfp4_quantize(X, off, stream=s),
        "dequantize": lambda s: rgg.rgg_mxfp4_dequantize(*xq, off, stream=s),
        "quantize_weights": lambda s: rgg.rgg_mxfp4_quantize_weights(W, stream=s),
        "dequantize_weights": lambda s: rgg.rgg_mxfp4_dequantize_weights(*wq, stream=s),
        "mxfp4": lambda s: rgg.rgg_grouped_gemm_mxfp4(*xq, *wq, off, stream=s),
    }


def _tensors(result):
    return [result] if isinstance(result, torch.Tensor) else list(result)


@pytest.mark.parametrize("name", ["clip", "dequantize", "dequantize_weights", "dgrad", "mxfp4", "quantize",
                                  "quantize_weights", "swiglu_backward", "wgrad"])
def test_outputs_are_the_streams_own(name):
    call = _calls()[name]
    want = [t.clone() for t in _tensors(call(None))]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    # blocks of the outputs' sizes, freed while the current stream has still to read them
    torch.cuda.empty_cache()
    held = [torch.full((t.numel() * t.element_size(),), 7, dtype=torch.uint8, device="cuda")
            for t in want for _ in (0, 1)]
    torch.cuda.synchronize()
    torch.cuda._sleep(50_000_000)
    copies = [t.clone() for t in held]
    del held
    got = _tensors(call(side))
    side.synchronize()
    torch.cuda.synchronize()
    for t in copies:
        assert bool((t == 7).all()), "%s wrote memory that the current stream had still to read" % name
    for g, w in zip(got, want):
        if name == "quantize" and g.dim() == 3:
            continue  # scales of rows that are not there are not written
        assert torch.equal(g, w), name
