"""The bounds-checked debug build on the MXFP4 gate-up product, on a GB300: no check of its boxes, scales, accumulator
columns and stores may fire on the ragged edges, and H is right to the bounds of test_gpu_mxfp4.py."""
import pytest
import torch

import expert_refs as refs
import ragged_grouped_gemm_02_gb300 as rgg
from ragged_grouped_gemm_02_gb300 import _build

pytestmark = pytest.mark.gpu

EDGE = [0, 1, 15, 16, 17, 63, 64, 65, 127, 128, 129, 255, 256, 257, 300, 385]


@pytest.fixture(scope="module", autouse=True)
def debug_lib():
    assert torch.cuda.is_available(), "the gpu tests need a CUDA device"
    _build.build()
    lib = rgg.open_library(rgg.debug_library_path())
    saved_lib, saved_handles = rgg._lib, rgg._handles
    rgg._lib, rgg._handles = lib, {}
    yield lib
    for h in rgg._handles.values():
        lib.rgg_destroy(h)
    rgg._lib, rgg._handles = saved_lib, saved_handles


# one output tile, several, and one and a half of the wide ones
@pytest.mark.parametrize("opts", [dict(bn=128), dict(bn=256), dict(bn=128, stages=2, max_ctas=3),
                                  dict(bn=256, stages=2, max_ctas=4)], ids=str)
@pytest.mark.parametrize("K,N", [(288, 128), (544, 384), (32, 256)])
def test_gate_up_edges(K, N, opts):
    gen = torch.Generator().manual_seed(K)
    off, M = refs.ragged(EDGE, 3, 2)
    X, W13 = refs.normal(gen, M, K), refs.normal(gen, len(EDGE), K, 2 * N, std=K ** -0.5)
    offg = torch.from_numpy(off).cuda()
    xq, wq = rgg.rgg_mxfp4_quantize(X.cuda(), offg, check=True), rgg.rgg_mxfp4_quantize_weights(W13.cuda())
    x = rgg.rgg_mxfp4_dequantize(*xq, offg, check=True).cpu().double()
    w = rgg.rgg_mxfp4_dequantize_weights(*wq).cpu().double()
    H = rgg.rgg_grouped_gemm_swiglu_mxfp4(*xq, *wq, offg, check=True, **opts)
    for e, (a, b) in enumerate(refs.spread(off)):
        gu, mag = x[a:b] @ w[e].t(), x[a:b].abs() @ w[e].abs().t()
        g, u, eps = gu[:, :N], gu[:, N:], K * 2.0 ** -23 * mag
        ref = refs.swiglu(gu)
        limit = refs.ROUND_BF16 * ref.abs() + g.abs() * eps[:, N:] + 1.1 * u.abs() * eps[:, :N] + \
            2.0 ** -18 * (g * u).abs() + refs.TINY
        if a < b:
            refs.assert_close(H[a:b], ref, limit, "H of expert %d" % e)
