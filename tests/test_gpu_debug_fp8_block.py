"""The bounds-checked debug build on the block-scaled 8-bit products, on a GB300: no check of their boxes, accumulator columns
and stores may fire on the ragged edges, and the results are those of the release build."""
import pytest
import torch

import expert_refs as refs
import ragged_grouped_gemm_02_gb300 as rgg
from ragged_grouped_gemm_02_gb300 import _build

pytestmark = pytest.mark.gpu

EDGE = [0, 1, 15, 31, 32, 33, 63, 64, 65, 96, 97, 127, 128, 129, 255, 256, 257, 300, 385]


@pytest.fixture(scope="module")
def debug_lib():
    assert torch.cuda.is_available(), "the gpu tests need a CUDA device"
    _build.build()
    lib = rgg.open_library(rgg.debug_library_path())
    handles = {}
    yield lib, handles
    for h in handles.values():
        lib.rgg_destroy(h)


def _inputs(K, cols, seed):
    gen = torch.Generator().manual_seed(seed)
    off, M = refs.ragged(EDGE, 3, 2)
    X, W = refs.normal(gen, M, K), refs.normal(gen, len(EDGE), K, cols, std=K ** -0.5)
    return rgg.rgg_fp8_block_quantize(X.cuda()), rgg.rgg_fp8_block_quantize_weights(W.cuda()), torch.from_numpy(off).cuda(), off


def _both(debug_lib, call):
    """call's result from the release build and from the debug build, whose status must be clean."""
    want = call()
    saved = rgg._lib, rgg._handles
    rgg._lib, rgg._handles = debug_lib
    try:
        return want, call()
    finally:
        rgg._lib, rgg._handles = saved


@pytest.mark.parametrize("opts", [dict(bm=128, bn=128), dict(bm=128, bn=256), dict(bm=256),
                                  dict(bm=128, bn=256, stages=2, max_ctas=3), dict(bm=256, stages=2, max_ctas=4)], ids=str)
@pytest.mark.parametrize("K,N", [(272, 136), (528, 392), (16, 8), (1024, 264)])
def test_product_edges(debug_lib, K, N, opts):
    x, w, off, bounds = _inputs(K, N, K)
    want, got = _both(debug_lib, lambda: rgg.rgg_grouped_gemm_fp8_block(*x, *w, off, check=True, **opts))
    a, b = int(bounds[0]), int(bounds[-1])
    assert torch.equal(want[a:b], got[a:b])


@pytest.mark.parametrize("opts", [dict(bm=128), dict(bm=256), dict(bm=128, stages=2, max_ctas=3),
                                  dict(bm=256, stages=2, max_ctas=4)], ids=str)
@pytest.mark.parametrize("K,N", [(272, 128), (528, 384), (16, 256)])
def test_gate_up_edges(debug_lib, K, N, opts):
    x, w, off, bounds = _inputs(K, 2 * N, K)
    want, got = _both(debug_lib, lambda: rgg.rgg_grouped_gemm_swiglu_fp8_block(*x, *w, off, check=True, **opts))
    a, b = int(bounds[0]), int(bounds[-1])
    assert torch.equal(want[0][a:b].view(torch.uint8), got[0][a:b].view(torch.uint8)) and torch.equal(want[1][a:b], got[1][a:b])
