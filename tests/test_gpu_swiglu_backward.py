"""rgg_grouped_gemm_swiglu_backward against the formulas in 64 bits, on a GB300."""
import numpy as np
import pytest
import torch

import expert_refs as refs
import ragged_grouped_gemm_02_gb300 as rgg
from ragged_grouped_gemm_02_gb300 import _build

pytestmark = pytest.mark.gpu

CANARY = 0x7FC1
COUNTS = [0, 1, 63, 64, 65, 127, 128, 129, 300, 17, 0, 513]
SHAPES = [(64, 128), (64, 256), (128, 128), (128, 256), (256, 128), (256, 256)]


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available(), "the gpu tests need a CUDA device"
    _build.build()


def _case(counts, K, N, seed, lead=3, spare=5):
    gen = torch.Generator().manual_seed(seed)
    off, M = refs.ragged(counts, lead, spare)
    # gates from about -12 to 12, so that the sigmoid saturates on both sides
    return (refs.normal(gen, M, K, std=3.0), refs.normal(gen, len(counts), K, 2 * N, std=K ** -0.5), off,
            refs.normal(gen, M, N))


def _canaries(*shape):
    return torch.full(shape, CANARY, dtype=torch.int16, device="cuda").view(torch.bfloat16)


def _run(X, W13, off, dH, H=None, **opts):
    M, N = dH.shape
    dGU, H = _canaries(M, 2 * N), _canaries(M, N) if H is None else H
    got = rgg.rgg_grouped_gemm_swiglu_backward(X.cuda(), W13.cuda(), torch.from_numpy(off).cuda(), dH.cuda(), dGU, H,
                                               check=True, **opts)
    assert got[0] is dGU
    return dGU.cpu(), None if got[1] is None else got[1].cpu()


def _check(X, W13, off, dH, dGU, H):
    gu, mag = refs.gate_up(X, W13, off)
    ref, act = refs.swiglu_backward(gu, dH.double())
    limit, act_limit = refs.swiglu_backward_bound(gu, mag, dH.double(), X.shape[1])
    a, b = int(off[0]), int(off[-1])
    for got, r, lim, what in ((dGU, ref, limit, "dGU"), (H, act, act_limit, "H")):
        if got is not None:
            refs.assert_close(got[a:b], r[a:b], lim[a:b], what)
            bits = got.view(torch.int16)
            assert bool((bits[:a] == CANARY).all()) and bool((bits[b:] == CANARY).all())


@pytest.mark.parametrize("bm,bn", SHAPES)
@pytest.mark.parametrize("K,N", [(264, 520), (64, 128), (8, 8), (72, 200)])
def test_tile_shapes_and_tails(bm, bn, K, N):
    case = _case(COUNTS, K, N, seed=bm + bn + K)
    _check(*case, *_run(*case, bm=bm, bn=bn))


@pytest.mark.parametrize("mixed", [1, 2])
@pytest.mark.parametrize("psms", [0, -1, 2, 76])
def test_mixed_launch(mixed, psms):
    case = _case(COUNTS + [700, 1000], 136, 264, seed=mixed)
    _check(*case, *_run(*case, mixed=mixed, mixed_pair_sms=psms, host_counts=np.diff(case[2])))


@pytest.mark.parametrize("counts", [[1], [0, 0, 1], [2048], [16] * 32, [100] * 8, [1024] * 3])
def test_planned(counts):
    case = _case(counts, 328, 264, seed=len(counts), lead=0, spare=0)
    _check(*case, *_run(*case))


def test_without_the_activation():
    case = _case([100, 0, 30], 64, 72, seed=5)
    dGU, H = _run(*case, H=False)
    assert H is None
    _check(*case, dGU, None)


def test_no_rows():
    case = _case([0, 0], 64, 64, seed=6)
    _check(*case, *_run(*case))


def test_saturated_gates():
    # gates of +-200: exp(-g) overflows or vanishes, the formulas stay finite
    X = torch.ones(4, 8, dtype=torch.bfloat16)
    X[1::2] = -1
    W13 = torch.full((1, 8, 16), 25.0, dtype=torch.bfloat16)
    off = np.array([0, 4], dtype=np.int32)
    dH = torch.full((4, 8), 0.5, dtype=torch.bfloat16)
    dGU, H = _run(X, W13, off, dH)
    up = torch.where(torch.arange(4) % 2 == 0, 200.0, -200.0)[:, None].expand(4, 8)
    pos = up > 0
    assert torch.equal(H.float(), torch.where(pos, 40000.0, 0.0).to(torch.bfloat16).float())
    assert torch.equal(dGU[:, :8].float(), torch.where(pos, 100.0, 0.0))
    assert torch.equal(dGU[:, 8:].float(), torch.where(pos, 100.0, 0.0))


def test_matches_the_forward_call():
    X, W13, off, dH = _case([70, 5, 200], 256, 136, seed=7)
    _, H = _run(X, W13, off, dH)
    fwd = _canaries(*dH.shape)
    rgg.rgg_grouped_gemm_swiglu(X.cuda(), W13.cuda(), torch.from_numpy(off).cuda(), fwd, check=True)
    gu, mag = refs.gate_up(X, W13, off)
    a, b = int(off[0]), int(off[-1])
    limit = refs.swiglu_backward_bound(gu, mag, dH.double(), X.shape[1])[1][a:b]
    refs.assert_close(fwd.cpu()[a:b], H[a:b].double(), 2 * limit, "forward and recomputed H")


def test_refusals():
    X, W13, off, dH = _case([5, 6], 64, 72, seed=8, lead=0, spare=0)
    X, W13, off, dH = X.cuda(), W13.cuda(), torch.from_numpy(off).cuda(), dH.cuda()
    with pytest.raises(TypeError):
        rgg.rgg_grouped_gemm_swiglu_backward(X, W13, off, dH.float())
    with pytest.raises(ValueError):
        rgg.rgg_grouped_gemm_swiglu_backward(X, W13, off, dH[:, :64])
    with pytest.raises(ValueError):
        rgg.rgg_grouped_gemm_swiglu_backward(X, W13, off, dH[:, :64].contiguous())
    with pytest.raises(ValueError):
        rgg.rgg_grouped_gemm_swiglu_backward(X, W13[:, :, :143], off, dH)
    with pytest.raises(rgg.RggError) as ei:
        rgg.rgg_grouped_gemm_swiglu_backward(X, W13, off, dH, bn=192)
    assert ei.value.status == rgg.RGG_ERR_INVALID_ARG
    dGU, H = _canaries(11, 144), _canaries(11, 72)
    bad = torch.tensor([0, 6, 5], dtype=torch.int32, device="cuda")
    with pytest.raises(rgg.RggError) as ei:
        rgg.rgg_grouped_gemm_swiglu_backward(X, W13, bad, dH, dGU, H, check=True)
    assert ei.value.status == rgg.RGG_ERR_BAD_OFFSETS
    assert bool((dGU.view(torch.int16) == CANARY).all()) and bool((H.view(torch.int16) == CANARY).all())
