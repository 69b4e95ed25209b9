"""How results leave the grouped products, on a GB300: outputs on and off a 32-byte boundary hold the same bits,
and the groups of epilogue warps that take a CTA's tiles in turn keep to their own tiles on walks of any length."""
import numpy as np
import pytest
import torch

import expert_refs as refs
import ragged_grouped_gemm_02_gb300 as rgg
from ragged_grouped_gemm_02_gb300 import _build

pytestmark = pytest.mark.gpu

CANARY = 0x7FC1
COUNTS = [0, 1, 63, 64, 65, 0, 127, 128, 129, 300, 17]


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available(), "the gpu tests need a CUDA device"
    _build.build()


def _out(M, N, shift):
    """bf16 [M, N], its first element `shift` elements after a 256-byte boundary, and the memory around it."""
    whole = torch.full((M * N + 64,), CANARY, dtype=torch.int16, device="cuda")
    return whole[shift:shift + M * N].view(torch.bfloat16).view(M, N), whole


def _inputs(K, N, seed):
    gen = torch.Generator().manual_seed(seed)
    off, M = refs.ragged(COUNTS, 3, 5)
    E = len(COUNTS)
    return (refs.normal(gen, M, K).cuda(), refs.normal(gen, E, K, N, std=K ** -0.5).cuda(),
            refs.normal(gen, M, N).cuda(), torch.from_numpy(off).cuda(), off, M)


def _same_bits(run, M, N, outputs=1):
    """run(outputs...) on and 16 bytes off a 32-byte boundary: the same bits, none written around them."""
    got = []
    for shift in (0, 8):
        outs = [_out(M, n, shift) for n in ([N] if outputs == 1 else N)]
        run(*[o for o, _ in outs])
        torch.cuda.synchronize()
        for (o, whole) in outs:
            assert bool((whole[:shift] == CANARY).all()) and bool((whole[shift + o.numel():] == CANARY).all())
        got.append([o.view(torch.int16).cpu().clone() for o, _ in outs])
    for a, b in zip(*got):
        assert torch.equal(a, b)


@pytest.mark.parametrize("bm,bn", [(0, 0), (64, 128), (64, 256), (128, 128), (128, 256), (256, 128), (256, 256)])
@pytest.mark.parametrize("K,N", [(272, 80), (528, 16)])
def test_off_a_boundary(K, N, bm, bn):
    X, W, dY, offg, _, M = _inputs(K, N, seed=K + bm)
    _same_bits(lambda Y: rgg.rgg_grouped_gemm(X, W, offg, Y, bm=bm, bn=bn, check=True), M, N)
    _same_bits(lambda dX: rgg.rgg_grouped_gemm_dgrad(dY, W, offg, dX, bm=bm, bn=bn, check=True), M, K)


@pytest.mark.parametrize("bm,bn", [(0, 0), (64, 256), (128, 128), (256, 256)])
def test_gate_up_off_a_boundary(bm, bn):
    K, N = 264, 80
    X, W13, _, offg, _, M = _inputs(K, 2 * N, seed=bm + bn)
    dH = refs.normal(torch.Generator().manual_seed(5), M, N).cuda()
    _same_bits(lambda H: rgg.rgg_grouped_gemm_swiglu(X, W13, offg, H, bm=bm, bn=bn, check=True), M, N)
    _same_bits(lambda dGU, H: rgg.rgg_grouped_gemm_swiglu_backward(X, W13, offg, dH, dGU, H, bm=bm, bn=bn, check=True),
               M, [2 * N, N], outputs=2)


@pytest.mark.parametrize("bn", [128, 256])
def test_mxfp4_off_a_boundary(bn):
    K = 544
    X, W, _, offg, _, M = _inputs(K, 272, seed=bn)
    x = rgg.rgg_mxfp4_quantize(X, offg, check=True)
    w = rgg.rgg_mxfp4_quantize_weights(W)
    _same_bits(lambda Y: rgg.rgg_grouped_gemm_mxfp4(*x, *w, offg, Y, bn=bn, check=True), M, 272)
    W13 = refs.normal(torch.Generator().manual_seed(7), len(COUNTS), K, 512, std=K ** -0.5).cuda()
    w = rgg.rgg_mxfp4_quantize_weights(W13)
    _same_bits(lambda H: rgg.rgg_grouped_gemm_swiglu_mxfp4(*x, *w, offg, H, bn=bn, check=True), M, 256)


@pytest.mark.parametrize("max_ctas", [2, 4, 6])
@pytest.mark.parametrize("bm,bn", [(64, 128), (128, 256), (256, 128), (256, 256)])
def test_dgrad_long_walks(bm, bn, max_ctas):
    # odd and even numbers of tiles a CTA, one to three reduction stages
    for N in (8, 72, 136):
        _, W, dY, offg, off, M = _inputs(264, N, seed=N)
        dX = torch.full((M, 264), float("nan"), dtype=torch.bfloat16, device="cuda")
        rgg.rgg_grouped_gemm_dgrad(dY, W, offg, dX, bm=bm, bn=bn, max_ctas=max_ctas, check=True)
        ref, limit = refs.dgrad(dY.cpu(), W.cpu(), off)
        a, b = int(off[0]), int(off[-1])
        refs.assert_close(dX.cpu()[a:b], ref[a:b], limit[a:b], "dX")


@pytest.mark.parametrize("counts", [[3], [533], [5, 5], [0, 0, 9, 0], [1] * 20, [64] * 8])
def test_few_tiles(counts):
    # calls whose tiles one wave holds
    gen = torch.Generator().manual_seed(len(counts))
    off, M = refs.ragged(counts, 2, 3)
    offg, (a, b) = torch.from_numpy(off).cuda(), (int(off[0]), int(off[-1]))
    K, N = 264, 400
    X, W, dY = refs.normal(gen, M, K), refs.normal(gen, len(counts), K, N, std=K ** -0.5), refs.normal(gen, M, N)
    dX = rgg.rgg_grouped_gemm_dgrad(dY.cuda(), W.cuda(), offg, check=True)
    ref, limit = refs.dgrad(dY, W, off)
    refs.assert_close(dX.cpu()[a:b], ref[a:b], limit[a:b], "dX")
    dH = dY[:, :N // 2]
    dGU, H = rgg.rgg_grouped_gemm_swiglu_backward(X.cuda(), W.cuda(), offg, dH.contiguous().cuda(), check=True)
    gu, mag = refs.gate_up(X, W, off)
    want, act = refs.swiglu_backward(gu, dH.double())
    limit, act_limit = refs.swiglu_backward_bound(gu, mag, dH.double(), K)
    refs.assert_close(dGU.cpu()[a:b], want[a:b], limit[a:b], "dGU")
    refs.assert_close(H.cpu()[a:b], act[a:b], act_limit[a:b], "H")
