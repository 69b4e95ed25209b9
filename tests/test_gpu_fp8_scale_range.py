"""Where the range of the block-scaled 8-bit product's scales ends, on a GB300: the product of a row's scale and a weight's at
either end of fp32's normal numbers."""
import pytest
import torch

import ragged_grouped_gemm_02_gb300 as rgg
from ragged_grouped_gemm_02_gb300 import _build

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available(), "the gpu tests need a CUDA device"
    _build.build()


@pytest.mark.parametrize("opts", [dict(bm=128, bn=128), dict(bm=128, bn=256), dict(bm=256)], ids=str)
@pytest.mark.parametrize("row,weight", [(-63, -63), (-108, -18), (0, -126), (-126, 0), (60, 60), (100, 27), (0, 127), (127, -126)])
def test_ends_of_the_range(row, weight, opts):
    M, K, N = 140, 128, 136
    gen = torch.Generator().manual_seed(0)
    x, w = (torch.randint(-4, 5, shape, generator=gen).double() for shape in ((M, K), (1, N, K)))
    x[5] = 0.0
    offsets = torch.tensor([0, M], dtype=torch.int32, device="cuda")
    eight = [t.float().to(torch.float8_e4m3fn).cuda() for t in (x, w)]
    Y = rgg.rgg_grouped_gemm_fp8_block(eight[0], torch.full((M, 1), 2.0 ** row, device="cuda"), eight[1],
                                       torch.full((1, 2, 1), 2.0 ** weight, device="cuda"), offsets, check=True, **opts)
    want = (x @ w[0].t()) * 2.0 ** (row + weight)  # whole numbers times a power of two: exact, Inf past the largest
    assert torch.equal(Y.cpu(), want.to(torch.bfloat16))
    assert bool((Y[5] == 0).all())
