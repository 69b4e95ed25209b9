"""The block-scaled 8-bit product over many short tiles on few CTAs: the scales' products and the tiles' coordinates go
round their places in shared memory hundreds of times, and every stage has scales of its own.  On a GB300."""
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
@pytest.mark.parametrize("blocks", [1, 2, 3, 4, 5, 8, 9])
def test_every_stage_has_its_own_scales(blocks, opts):
    # codes of 1 and scales that are small whole numbers: sums of fewer than 24 bits, exact in fp32
    counts, N = [300, 1, 129, 64, 257, 500], 1160
    E, K, M = len(counts), 128 * blocks, sum(counts)
    gen = torch.Generator().manual_seed(blocks)
    offsets = torch.tensor([0] + counts).cumsum(0).to(torch.int32).cuda()
    sx = torch.randint(1, 12, (M, blocks), generator=gen).float().cuda()
    sw = torch.randint(1, 12, (E, -(-N // 128), blocks), generator=gen).float().cuda()
    ones = torch.ones(M, K, device="cuda").to(torch.float8_e4m3fn), torch.ones(E, N, K, device="cuda").to(torch.float8_e4m3fn)
    owner = torch.repeat_interleave(torch.arange(E), torch.tensor(counts)).cuda()
    sums = 128 * torch.einsum("mb,mnb->mn", sx.double(), sw.double()[owner])
    want = sums.repeat_interleave(128, 1)[:, :N].to(torch.bfloat16)
    for max_ctas in (2, 6, 0):
        for stages in (2, 0):
            Y = rgg.rgg_grouped_gemm_fp8_block(ones[0], sx, ones[1], sw, offsets, max_ctas=max_ctas, stages=stages,
                                               check=True, **opts)
            assert torch.equal(Y, want), (max_ctas, stages)
