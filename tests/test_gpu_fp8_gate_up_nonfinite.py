"""NaN and Inf in the 8-bit gate-up product's H: the whole block of 128 columns comes back as NaN, and nothing else does.  On
a GB300."""
import pytest
import torch

import ragged_grouped_gemm_02_gb300 as rgg
from ragged_grouped_gemm_02_gb300 import _build

pytestmark = pytest.mark.gpu

COUNTS, K, N = [40, 300, 5], 256, 384


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available(), "the gpu tests need a CUDA device"
    _build.build()


def _case():
    gen = torch.Generator().manual_seed(3)
    X = torch.randn(sum(COUNTS), K, generator=gen).to(torch.bfloat16).cuda()
    W = (torch.randn(len(COUNTS), K, 2 * N, generator=gen) * K ** -0.5).to(torch.bfloat16).cuda()
    offsets = torch.tensor([0] + COUNTS).cumsum(0).to(torch.int32).cuda()
    return rgg.rgg_fp8_block_quantize(X), rgg.rgg_fp8_block_quantize_weights(W), offsets


def _check(got, want, bad):
    """bad: [rows, N / 128], the blocks that have to be NaN; the others are as they were, bit for bit."""
    wide = bad.repeat_interleave(128, 1)
    back = rgg.rgg_fp8_block_dequantize(*got)
    assert bool(back[wide].isnan().all())
    assert torch.equal(got[0].view(torch.uint8)[~wide], want[0].view(torch.uint8)[~wide])
    assert torch.equal(got[1][~bad], want[1][~bad])


@pytest.mark.parametrize("bm", [128, 256])
@pytest.mark.parametrize("column", [7, 127, 200, N + 0, N + 290, 2 * N - 1])
def test_one_column_of_nan(column, bm):
    x, w, offsets = _case()
    want = rgg.rgg_grouped_gemm_swiglu_fp8_block(*x, *w, offsets, bm=bm)
    codes = w[0].clone()
    codes.view(torch.uint8)[1, column, 77] = 0x7F
    got = rgg.rgg_grouped_gemm_swiglu_fp8_block(*x, codes, w[1], offsets, bm=bm, check=True)
    bad = torch.zeros(sum(COUNTS), N // 128, dtype=torch.bool, device="cuda")
    bad[int(offsets[1]) : int(offsets[2]), column % N // 128] = True
    _check(got, want, bad)


@pytest.mark.parametrize("bm", [128, 256])
def test_rows_that_overflow(bm):
    # gate and up near 2^66: their product passes fp32's range where the gate is positive
    x, w, offsets = _case()
    want = rgg.rgg_grouped_gemm_swiglu_fp8_block(*x, *w, offsets, bm=bm)
    scales, bad = x[1].clone(), torch.zeros(sum(COUNTS), N // 128, dtype=torch.bool, device="cuda")
    for row in (3, 41, 200, 344):
        scales[row] *= 2.0 ** 66
        bad[row] = True
    got = rgg.rgg_grouped_gemm_swiglu_fp8_block(x[0], scales, *w, offsets, bm=bm, check=True)
    assert bool(got[1][bad].isinf().all())
    _check(got, want, bad)
