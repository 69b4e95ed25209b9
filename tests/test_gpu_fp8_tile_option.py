"""The tile that bn asks the block-scaled 8-bit product for, on a GB300.  Results do not tell the tiles apart, but what fits in
shared memory does: six stages of 128 x 128 tiles, and four of 128 x 256."""
import pytest
import torch

import ragged_grouped_gemm_02_gb300 as rgg
from ragged_grouped_gemm_02_gb300 import _build

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available(), "the gpu tests need a CUDA device"
    _build.build()


@pytest.mark.parametrize("rows", [16, 200])  # per expert: below and above 128, where the choice by the sizes differs
@pytest.mark.parametrize("N", [128, 136])
@pytest.mark.parametrize("bm", [0, 128])
def test_bn_sets_the_tile(rows, N, bm):
    E, K = 2, 1024
    gen = torch.Generator().manual_seed(rows)
    X = torch.randn(E * rows, K, generator=gen).to(torch.bfloat16).cuda()
    W = torch.randn(E, K, N, generator=gen).to(torch.bfloat16).cuda()
    offsets = (torch.arange(E + 1) * rows).to(torch.int32).cuda()
    args = (*rgg.rgg_fp8_block_quantize(X), *rgg.rgg_fp8_block_quantize_weights(W), offsets)

    def call(**opts):  # one CTA: no pairs
        return rgg.rgg_grouped_gemm_fp8_block(*args, bm=bm, max_ctas=1, check=True, **opts)

    want = call()
    assert torch.equal(call(bn=128, stages=6), want)
    assert torch.equal(call(bn=256), want) and torch.equal(call(bn=256, stages=4), want)
    with pytest.raises(rgg.RggError) as error:
        call(bn=256, stages=6)
    assert error.value.status == rgg.RGG_ERR_UNSUPPORTED
