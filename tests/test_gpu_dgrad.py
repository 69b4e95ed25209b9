"""rgg_grouped_gemm_dgrad (dX_e = dY_e . W_e^T) against 64-bit products, on a GB300."""
import numpy as np
import pytest
import torch

import expert_refs as refs
import ragged_grouped_gemm_02_gb300 as rgg
from ragged_grouped_gemm_02_gb300 import _build

pytestmark = pytest.mark.gpu

CANARY = 0x7FC1
COUNTS = [0, 1, 63, 64, 65, 127, 128, 129, 300, 17, 0, 513]


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available(), "the gpu tests need a CUDA device"
    _build.build()


def _case(counts, K, N, seed, lead=3, spare=5):
    gen = torch.Generator().manual_seed(seed)
    off, M = refs.ragged(counts, lead, spare)
    return refs.normal(gen, M, N), refs.normal(gen, len(counts), K, N, std=N ** -0.5), off


def _run(dY, W, off, **opts):
    dX = torch.full((dY.shape[0], W.shape[1]), CANARY, dtype=torch.int16, device="cuda").view(torch.bfloat16)
    rgg.rgg_grouped_gemm_dgrad(dY.cuda(), W.cuda(), torch.from_numpy(off).cuda(), dX, check=True, **opts)
    return dX.cpu()


def _check(dY, W, off, dX):
    ref, limit = refs.dgrad(dY, W, off)
    a, b = int(off[0]), int(off[-1])
    refs.assert_close(dX[a:b], ref[a:b], limit[a:b], "dX")
    bits = dX.view(torch.int16)
    assert bool((bits[:a] == CANARY).all()) and bool((bits[b:] == CANARY).all())


@pytest.mark.parametrize("bm,bn", [(64, 128), (64, 192), (64, 256), (128, 128), (128, 192), (128, 256), (256, 128),
                                   (256, 256)])
@pytest.mark.parametrize("K,N", [(264, 520), (512, 64), (8, 8), (200, 1032)])
def test_tile_shapes_and_tails(bm, bn, K, N):
    dY, W, off = _case(COUNTS, K, N, seed=bm + bn + K)
    _check(dY, W, off, _run(dY, W, off, bm=bm, bn=bn))


@pytest.mark.parametrize("mixed", [1, 2])
@pytest.mark.parametrize("psms", [0, -1, 2, 76])
def test_mixed_launch(mixed, psms):
    dY, W, off = _case(COUNTS + [700, 1000], 392, 136, seed=mixed)
    _check(dY, W, off, _run(dY, W, off, mixed=mixed, mixed_pair_sms=psms, host_counts=np.diff(off)))
    if psms == 0:
        _check(dY, W, off, _run(dY, W, off, mixed=mixed))


@pytest.mark.parametrize("counts", [[1], [0, 0, 1], [2048], [16] * 32, [100] * 8, [1024] * 3])
def test_planned(counts):
    dY, W, off = _case(counts, 520, 328, seed=len(counts), lead=0, spare=0)
    _check(dY, W, off, _run(dY, W, off))
    _check(dY, W, off, _run(dY, W, off, host_counts=counts))


def test_no_rows():
    dY, W, off = _case([0, 0, 0], 64, 64, seed=1, lead=2, spare=2)
    _check(dY, W, off, _run(dY, W, off))


def test_rows_of_no_expert_do_not_reach_a_result():
    dY, W, off = _case([50, 0, 70], 128, 192, seed=2)
    dY[: off[0]] = float("nan")
    dY[off[-1]:] = float("inf")
    _check(dY, W, off, _run(dY, W, off))


def test_refusals():
    dY, W, off = (t.cuda() if isinstance(t, torch.Tensor) else torch.from_numpy(t).cuda()
                  for t in _case([5, 6], 64, 72, seed=3, lead=0, spare=0))
    with pytest.raises(TypeError):
        rgg.rgg_grouped_gemm_dgrad(dY.float(), W, off)
    with pytest.raises(TypeError):
        rgg.rgg_grouped_gemm_dgrad(dY, W, off.long())
    with pytest.raises(ValueError):
        rgg.rgg_grouped_gemm_dgrad(dY[:, :64], W, off)
    with pytest.raises(ValueError):
        rgg.rgg_grouped_gemm_dgrad(dY, W.transpose(1, 2), off)
    with pytest.raises(ValueError):
        rgg.rgg_grouped_gemm_dgrad(dY.cpu(), W, off)
    with pytest.raises(ValueError):
        rgg.rgg_grouped_gemm_dgrad(dY, W, off, torch.empty(11, 72, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(rgg.RggError) as ei:
        rgg.rgg_grouped_gemm_dgrad(dY, W, off, bm=32)
    assert ei.value.status == rgg.RGG_ERR_INVALID_ARG
    dX = torch.full((11, 64), CANARY, dtype=torch.int16, device="cuda").view(torch.bfloat16)
    with pytest.raises(rgg.RggError) as ei:
        rgg.rgg_grouped_gemm_dgrad(dY, W, torch.tensor([0, 6, 5], dtype=torch.int32, device="cuda"), dX, check=True)
    assert ei.value.status == rgg.RGG_ERR_BAD_OFFSETS
    assert bool((dX.view(torch.int16) == CANARY).all())
