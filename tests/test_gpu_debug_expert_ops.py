"""The bounds-checked debug build on the backward products and the MXFP4 product, on a GB300: no check may fire on the
ragged edges, and the results are those of the release build's tests."""
import numpy as np
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


def _case(K, N, seed):
    gen = torch.Generator().manual_seed(seed)
    off, M = refs.ragged(EDGE, 3, 2)
    return (refs.normal(gen, M, K), refs.normal(gen, M, N), refs.normal(gen, len(EDGE), K, N, std=K ** -0.5), off,
            torch.from_numpy(off).cuda())


OPTS = [dict(), dict(bm=64, bn=128), dict(bm=128, bn=192), dict(bm=256, bn=128), dict(bm=256, bn=256), dict(mixed=1),
        dict(mixed=2), dict(mixed=1, mixed_pair_sms=2)]


@pytest.mark.parametrize("opts", OPTS, ids=[str(o) for o in OPTS])
def test_dgrad_edges(opts):
    X, dY, W, off, offg = _case(264, 520, 1)
    dX = rgg.rgg_grouped_gemm_dgrad(dY.cuda(), W.cuda(), offg, check=True, **opts)
    ref, limit = refs.dgrad(dY, W, off)
    a, b = int(off[0]), int(off[-1])
    refs.assert_close(dX[a:b], ref[a:b], limit[a:b], "dX")


@pytest.mark.parametrize("bn", [128, 256])
@pytest.mark.parametrize("accumulate", [False, True])
def test_wgrad_edges(bn, accumulate):
    X, dY, W, off, offg = _case(264, 520, 2)
    dW = torch.zeros(len(EDGE), 264, 520, device="cuda")
    rgg.rgg_grouped_gemm_wgrad(X.cuda(), dY.cuda(), offg, dW, bn=bn, accumulate=accumulate, check=True)
    ref, mag = refs.wgrad(X, dY, off)
    n = torch.from_numpy(np.diff(off).astype(np.float64))[:, None, None]
    refs.assert_close(dW, ref, (n + 1) * 2.0 ** -23 * mag + refs.TINY, "dW")


@pytest.mark.parametrize("opts", [o for o in OPTS if o.get("bn") != 192],
                         ids=[str(o) for o in OPTS if o.get("bn") != 192])
def test_swiglu_backward_edges(opts):
    X, dH, _, off, offg = _case(264, 264, 3)
    W13 = refs.normal(torch.Generator().manual_seed(4), len(EDGE), 264, 528, std=264 ** -0.5)
    dGU, H = rgg.rgg_grouped_gemm_swiglu_backward(X.cuda(), W13.cuda(), offg, dH.cuda(), check=True, **opts)
    gu, mag = refs.gate_up(X, W13, off)
    ref, act = refs.swiglu_backward(gu, dH.double())
    limit, act_limit = refs.swiglu_backward_bound(gu, mag, dH.double(), 264)
    a, b = int(off[0]), int(off[-1])
    refs.assert_close(dGU[a:b], ref[a:b], limit[a:b], "dGU")
    refs.assert_close(H[a:b], act[a:b], act_limit[a:b], "H")


@pytest.mark.parametrize("bn", [128, 256])
@pytest.mark.parametrize("K,N", [(288, 520), (544, 384), (32, 8)])
def test_mxfp4_edges(K, N, bn):
    X, _, W, off, offg = _case(K, N, 5)
    xq, wq = rgg.rgg_mxfp4_quantize(X.cuda(), offg, check=True), rgg.rgg_mxfp4_quantize_weights(W.cuda())
    x = rgg.rgg_mxfp4_dequantize(*xq, offg, check=True).cpu().double()
    w = rgg.rgg_mxfp4_dequantize_weights(*wq).cpu().double()
    Y = rgg.rgg_grouped_gemm_mxfp4(*xq, *wq, offg, bn=bn, check=True)
    for e, (a, b) in enumerate(refs.spread(off)):
        ref, mag = x[a:b] @ w[e].t(), x[a:b].abs() @ w[e].abs().t()
        refs.assert_close(Y[a:b], ref, refs.bound(ref, K, mag), "Y of expert %d" % e)
    if N % 256 == 0:
        H = rgg.rgg_grouped_gemm_swiglu_mxfp4(*xq, *wq, offg, bn=bn, check=True)
        assert H.shape == (X.shape[0], N // 2)
