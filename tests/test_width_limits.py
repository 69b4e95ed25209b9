"""The widest K and N: 2^31 - 1024, as tiles end past the last column and columns are counted in 32 bits.  Wider calls
are refused before anything is launched."""
import ctypes

import pytest

import ragged_grouped_gemm_02_gb300 as rgg
from ragged_grouped_gemm_02_gb300 import _build

LIMIT = 2 ** 31 - 1024
WIDE = [LIMIT + 8, 2 ** 31 - 256, 2 ** 31 - 8]


@pytest.fixture(scope="module", autouse=True)
def built():
    _build.build()


def test_the_planner_takes_the_limit():
    assert rgg.rgg_plan(1, 1, 8, LIMIT)["max_tiles"] > 0
    assert rgg.rgg_plan(1, 1, LIMIT, 8)["max_tiles"] > 0
    assert rgg.rgg_plan(1, 1, 8, LIMIT // 2, op="swiglu")["max_tiles"] > 0


@pytest.mark.parametrize("width", WIDE)
@pytest.mark.parametrize("op", ["gemm", "fp8", "gather"])
def test_the_planner_refuses_wider(width, op):
    wide = max(width // 16 * 16, LIMIT + 16) if op == "fp8" else width  # FP8 widths are multiples of 16
    for K, N in ((16, wide), (wide, 16)):
        with pytest.raises(rgg.RggError) as ei:
            rgg.rgg_plan(1, 1, K, N, op=op)
        assert ei.value.status == rgg.RGG_ERR_INVALID_ARG


@pytest.mark.parametrize("op", ["swiglu", "swiglu_gather"])
@pytest.mark.parametrize("width", [LIMIT // 2 + 8, 2 ** 30])
def test_the_planner_refuses_wider_gate_up(width, op):
    with pytest.raises(rgg.RggError) as ei:
        rgg.rgg_plan(1, 1, 8, width, op=op)
    assert ei.value.status == rgg.RGG_ERR_INVALID_ARG


@pytest.mark.gpu
@pytest.mark.parametrize("wide", WIDE)
def test_the_calls_refuse_wider(wide):
    import torch
    lib, handle = rgg.load_library(), rgg._handle(0)
    p = ctypes.c_void_p(torch.zeros(64, device="cuda").data_ptr())  # never read
    blocks, half = wide // 32 * 32, (wide // 2 + 127) // 128 * 128
    assert half > LIMIT // 2
    refused = [lib.rgg_grouped_gemm(handle, p, p, p, p, 1, 1, 8, wide, None, None),
               lib.rgg_grouped_gemm_swiglu(handle, p, p, p, p, 1, 1, 8, half, None, None),
               lib.rgg_grouped_gemm_swiglu_backward(handle, p, p, p, p, p, p, 1, 1, 8, half, None, None),
               lib.rgg_grouped_gemm_dgrad(handle, p, p, p, p, 1, 1, wide, 8, None, None),
               lib.rgg_grouped_gemm_dgrad(handle, p, p, p, p, 1, 1, 8, wide, None, None),
               lib.rgg_grouped_gemm_wgrad(handle, p, p, p, p, 1, 1, wide, 8, 0, None, None),
               lib.rgg_grouped_gemm_wgrad(handle, p, p, p, p, 1, 1, 8, wide, 0, None, None),
               lib.rgg_mxfp4_quantize_weights(handle, p, p, p, 1, 32, wide, None),
               lib.rgg_mxfp4_dequantize_weights(handle, p, p, p, 1, 32, wide, None),
               lib.rgg_grouped_gemm_mxfp4(handle, p, p, p, p, p, p, 1, 1, 32, wide, None, None),
               lib.rgg_grouped_gemm_swiglu_mxfp4(handle, p, p, p, p, p, p, 1, 1, 32, half, None, None)]
    if blocks > LIMIT:
        refused += [lib.rgg_mxfp4_quantize(handle, p, p, p, p, 1, 1, blocks, None),
                    lib.rgg_mxfp4_dequantize(handle, p, p, p, p, 1, 1, blocks, None)]
    assert refused == [rgg.RGG_ERR_INVALID_ARG] * len(refused)
    assert lib.rgg_grouped_gemm_wgrad_workspace(handle, 1, 1, wide, 8, 0) == 0
