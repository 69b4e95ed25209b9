"""What the router, the sort, the row kernels and the block-scaled 8-bit operators refuse: decided on the host, without a GPU."""
import ctypes

import pytest
import torch

import ragged_grouped_gemm_02_gb300 as rgg
from ragged_grouped_gemm_02_gb300 import _build
from ragged_grouped_gemm_02_gb300.expert_layer import quantize_experts_fp8
from ragged_grouped_gemm_02_gb300.moe_layer import moe_ffn, moe_ffn_fp8

BF16, FP32, I32, FP8 = torch.bfloat16, torch.float32, torch.int32, torch.float8_e4m3fn


def _t(*shape, dtype=BF16):
    return torch.zeros(*shape, dtype=FP32).to(dtype)


@pytest.mark.parametrize("call", [
    lambda: rgg.rgg_route_topk(_t(4, 8), 2),
    lambda: rgg.rgg_route_topk_backward(_t(4, 8), _t(4, 2, dtype=I32), _t(4, 2, dtype=FP32)),
    lambda: rgg.rgg_sort_by_expert(_t(4, 2, dtype=I32), 8),
    lambda: rgg.rgg_dispatch(_t(4, 8), _t(4, 2, dtype=I32)),
    lambda: rgg.rgg_combine(_t(8, 8), _t(4, 2, dtype=I32)),
    lambda: rgg.rgg_combine_backward(_t(4, 8), _t(8, 8), _t(4, 2, dtype=I32), _t(4, 2, dtype=FP32)),
    lambda: rgg.rgg_fp8_block_quantize(_t(4, 16)),
    lambda: rgg.rgg_fp8_block_dequantize(_t(4, 16, dtype=FP8), _t(4, 1, dtype=FP32)),
    lambda: rgg.rgg_fp8_block_quantize_weights(_t(2, 16, 8)),
    lambda: rgg.rgg_fp8_block_dequantize_weights(_t(2, 8, 16, dtype=FP8), _t(2, 1, 1, dtype=FP32)),
    lambda: rgg.rgg_grouped_gemm_fp8_block(_t(4, 16, dtype=FP8), _t(4, 1, dtype=FP32), _t(2, 8, 16, dtype=FP8),
                                           _t(2, 1, 1, dtype=FP32), _t(3, dtype=I32)),
])
def test_cpu_tensors(call):
    with pytest.raises(ValueError, match="CUDA"):
        call()


@pytest.mark.parametrize("call,error", [
    (lambda: rgg.rgg_route_topk(_t(8), 2), ValueError),
    (lambda: rgg.rgg_route_topk(_t(4, 8, dtype=torch.float64), 2), TypeError),
    (lambda: rgg.rgg_route_topk(_t(4, 8, dtype=I32), 2), TypeError),
    (lambda: rgg.rgg_sort_by_expert(_t(8, dtype=I32), 4), ValueError),
    (lambda: rgg.rgg_sort_by_expert(torch.zeros(4, 0, dtype=I32), 4), ValueError),
    (lambda: rgg.rgg_dispatch(_t(8), _t(4, 2, dtype=I32)), ValueError),
    (lambda: rgg.rgg_combine(_t(8, 8), _t(4, dtype=I32)), ValueError),
    (lambda: rgg.rgg_combine(_t(8), _t(4, 2, dtype=I32)), ValueError),
    (lambda: rgg.rgg_fp8_block_quantize(_t(16)), ValueError),
    (lambda: rgg.rgg_fp8_block_quantize_weights(_t(16, 8)), ValueError),
    (lambda: quantize_experts_fp8(_t(2, 16, 24), _t(2, 8, 16)), ValueError),
    (lambda: moe_ffn(_t(4, 16), _t(4, 3), _t(2, 16, 16), _t(2, 8, 16), 1), ValueError),
    (lambda: moe_ffn_fp8(_t(4, 16), _t(4, 2, dtype=I32), ((_t(2, 256, 16), None), (_t(2, 16, 128), None)), 1), TypeError),
])
def test_shapes_and_types(call, error):
    with pytest.raises(error):
        call()


def test_score_names():
    with pytest.raises(ValueError):
        rgg._route_flags("relu", True)
    assert {rgg._route_flags(s, r) for s in ("softmax", "sigmoid") for r in (True, False)} == {0, 1, 2, 3}


# The C entries check a call before they touch its handle or the GPU: a handle that is not NULL will do.
HANDLE = ctypes.c_void_p(8)
P = 4096  # a well-aligned address that is never read


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return rgg.load_library()


INVALID, UNSUPPORTED = rgg.RGG_ERR_INVALID_ARG, rgg.RGG_ERR_UNSUPPORTED
BIG = 1 << 31


@pytest.mark.parametrize("handle,logits,dtype,T,E,k,flags,scale,want", [
    (None, P, 1, 4, 8, 2, 0, 1.0, INVALID), (HANDLE, None, 1, 4, 8, 2, 0, 1.0, INVALID),
    (HANDLE, P + 2, 1, 4, 8, 2, 0, 1.0, INVALID), (HANDLE, P + 1, 0, 4, 8, 2, 0, 1.0, INVALID),
    (HANDLE, P, 3, 4, 8, 2, 0, 1.0, INVALID), (HANDLE, P, 1, -1, 8, 2, 0, 1.0, INVALID),
    (HANDLE, P, 1, BIG, 8, 2, 0, 1.0, INVALID), (HANDLE, P, 1, 4, 0, 1, 0, 1.0, INVALID),
    (HANDLE, P, 1, 4, 8, 0, 0, 1.0, INVALID), (HANDLE, P, 1, 4, 8, 9, 0, 1.0, INVALID),
    (HANDLE, P, 1, 4, 8, 2, 4, 1.0, INVALID), (HANDLE, P, 1, 4, 8, 2, 0, float("nan"), INVALID),
    (HANDLE, P, 1, 4, 4097, 2, 0, 1.0, UNSUPPORTED), (HANDLE, P, 1, 4, 64, 33, 0, 1.0, UNSUPPORTED),
    (HANDLE, P, 1, 0, 8, 2, 0, 1.0, rgg.RGG_OK),
])
def test_route_arguments(lib, handle, logits, dtype, T, E, k, flags, scale, want):
    assert lib.rgg_route_topk(handle, logits, dtype, T, E, k, flags, scale, P, P, None) == want
    assert lib.rgg_route_topk_backward(handle, logits, dtype, P, P, P, T, E, k, flags, scale, None) == want


def test_route_outputs(lib):
    for experts, weights in ((None, P), (P, None), (P + 2, P), (P, P + 1)):
        assert lib.rgg_route_topk(HANDLE, P, 1, 4, 8, 2, 0, 1.0, experts, weights, None) == INVALID
    for e, dw, dl in ((None, P, P), (P, None, P), (P, P, None), (P + 1, P, P), (P, P + 2, P), (P, P, P + 2)):
        assert lib.rgg_route_topk_backward(HANDLE, P, 1, e, dw, dl, 4, 8, 2, 0, 1.0, None) == INVALID


@pytest.mark.parametrize("args,want", [
    ((None, P, 4, 2, 8, P, P, P, None, 0), INVALID), ((HANDLE, None, 4, 2, 8, P, P, P, None, 0), INVALID),
    ((HANDLE, P, 4, 2, 8, None, P, P, None, 0), INVALID), ((HANDLE, P, 4, 2, 8, P, None, P, None, 0), INVALID),
    ((HANDLE, P, 4, 2, 8, P, P, None, None, 0), INVALID), ((HANDLE, P + 2, 4, 2, 8, P, P, P, None, 0), INVALID),
    ((HANDLE, P, -1, 2, 8, P, P, P, None, 0), INVALID), ((HANDLE, P, 4, 0, 8, P, P, P, None, 0), INVALID),
    ((HANDLE, P, 4, 2, 0, P, P, P, None, 0), INVALID), ((HANDLE, P, 4, 2, 4097, P, P, P, None, 0), UNSUPPORTED),
    ((HANDLE, P, 1 << 30, 2, 8, P, P, P, P, 1 << 30), INVALID),
    ((HANDLE, P, 100000, 2, 8, P, P, P, None, 0), INVALID), ((HANDLE, P, 100000, 2, 8, P, P, P, P, 64), INVALID),
])
def test_sort_arguments(lib, args, want):
    assert lib.rgg_sort_by_expert(*args, None) == want


def test_sort_workspace(lib):
    assert lib.rgg_sort_by_expert_workspace(0, 8) == 0
    assert lib.rgg_sort_by_expert_workspace(4096, 8) == 0
    assert lib.rgg_sort_by_expert_workspace(4097, 8) > 0
    assert lib.rgg_sort_by_expert_workspace(-1, 8) == lib.rgg_sort_by_expert_workspace(10 ** 6, 0) == 0
    assert lib.rgg_sort_by_expert_workspace(2 ** 31 - 1, 4096) < 1 << 24


@pytest.mark.parametrize("T,k,rows,size", [(-1, 1, 4, 8), (BIG, 1, 4, 8), (4, 0, 4, 8), (4, 1, -1, 8), (4, 1, BIG, 8),
                                           (4, 1, 4, 0), (4, 1, 4, BIG), (4, 1, 4, 1 << 30), (1 << 30, 2, 4, 8)])
def test_row_sizes(lib, T, k, rows, size):
    assert lib.rgg_dispatch(HANDLE, P, P, T, k, rows, size, P, None) == INVALID
    assert lib.rgg_combine(HANDLE, P, P, P, T, k, rows, size, P, None) == INVALID
    assert lib.rgg_combine_backward(HANDLE, P, P, P, P, T, k, rows, size, P, P, None) == INVALID


def test_row_pointers(lib):
    for X, p, out in ((None, P, P), (P, None, P), (P, P, None), (P, P + 2, P)):
        assert lib.rgg_dispatch(HANDLE, X, p, 4, 2, 8, 16, out, None) == INVALID
    assert lib.rgg_dispatch(None, P, P, 4, 2, 8, 16, P, None) == INVALID
    for Y, p, w, out in ((None, P, P, P), (P, None, P, P), (P, P, P, None), (P + 1, P, P, P), (P, P + 1, P, P),
                         (P, P, P + 2, P), (P, P, P, P + 1)):
        assert lib.rgg_combine(HANDLE, Y, p, w, 4, 2, 8, 16, out, None) == INVALID
    for d, Y, p, w, dY, dw in ((None, P, P, P, P, P), (P, None, P, P, P, P), (P, P, None, P, P, P), (P, P, P, None, P, P),
                               (P + 1, P, P, P, P, P), (P, P, P, P, P + 1, P), (P, P, P, P, P, P + 2)):
        assert lib.rgg_combine_backward(HANDLE, d, Y, p, w, 4, 2, 8, 16, dY, dw, None) == INVALID
    assert lib.rgg_combine_backward(HANDLE, P, P, P, P, 4, 2, 8, 16, None, None, None) == rgg.RGG_OK


@pytest.mark.parametrize("T,k,rows,K,position", [(4, 2, 8, 24, P), (4, 2, 8, 0, P), (-1, 2, 8, 16, P), (4, 0, 8, 16, P),
                                                 (4, 2, -1, 16, P), (4, 1, 5, 16, None), (1 << 30, 2, 8, 16, P),
                                                 (4, 2, 8, 16, P + 2)])
def test_quantize_sizes(lib, T, k, rows, K, position):
    assert lib.rgg_fp8_block_quantize(HANDLE, P, position, T, k, rows, K, P, P, None) == INVALID


def test_quantize_pointers(lib):
    for X, c, s in ((None, P, P), (P, None, P), (P, P, None), (P + 8, P, P), (P, P + 8, P), (P, P, P + 2)):
        assert lib.rgg_fp8_block_quantize(HANDLE, X, None, 4, 1, 4, 32, c, s, None) == INVALID
        assert lib.rgg_fp8_block_dequantize(HANDLE, c, s, X, 4, 32, None) == INVALID
        assert lib.rgg_fp8_block_quantize_weights(HANDLE, X, c, s, 2, 32, 8, None) == INVALID
        assert lib.rgg_fp8_block_dequantize_weights(HANDLE, c, s, X, 2, 32, 8, None) == INVALID
    for E, K, N in ((0, 32, 8), (2, 24, 8), (2, 32, 12), (2, 8, 8)):
        assert lib.rgg_fp8_block_quantize_weights(HANDLE, P, P, P, E, K, N, None) == INVALID
        assert lib.rgg_fp8_block_dequantize_weights(HANDLE, P, P, P, E, K, N, None) == INVALID
    assert lib.rgg_fp8_block_quantize_weights(HANDLE, P, P, P, 4097, 32, 8, None) == UNSUPPORTED


@pytest.mark.parametrize("gate_up", [False, True])
def test_product_arguments(lib, gate_up):
    def call(x=P, sx=P, w=P, sw=P, off=P, out=P, hs=P, E=2, M=64, K=128, N=128, opt=None, h=HANDLE):
        if gate_up:
            return lib.rgg_grouped_gemm_swiglu_fp8_block(h, x, sx, w, sw, off, out, hs, E, M, K, N, None, opt)
        return lib.rgg_grouped_gemm_fp8_block(h, x, sx, w, sw, off, out, E, M, K, N, None, opt)

    for bad in ({"x": None}, {"sx": None}, {"w": None}, {"sw": None}, {"off": None}, {"out": None}, {"h": None}, {"x": P + 8},
                {"sx": P + 2}, {"w": P + 8}, {"sw": P + 1}, {"out": P + 8}, {"off": P + 2}, {"E": 0}, {"M": -1}, {"M": BIG},
                {"K": 8}, {"K": 24}, {"N": 12}, {"N": 0}, {"K": 2 ** 31 - 8}):
        assert call(**bad) == INVALID, bad
    assert call(E=4097) == UNSUPPORTED
    if gate_up:
        assert call(N=64) == call(hs=None) == call(hs=P + 2) == call(N=2 ** 30) == INVALID
    for kw in ({"bn": 64}, {"bm": 256, "bn": 128}, {"bm": 64}, {"bm": 192}, {"max_ctas": -1}, {"stages": 1}, {"stages": 17}):
        assert call(opt=ctypes.byref(rgg._options(**kw)[0])) == INVALID, kw


def test_moe_arguments(lib):
    def call(h=HANDLE, X=P, lg=P, dt=1, a=P, b=P, c=P, d=P, out=P, T=4, E=4, k=2, K=32, N=128, K_out=32, flags=0, scale=1.0,
             ws=P, nbytes=1 << 30):
        return lib.rgg_moe_swiglu_fp8_block(h, X, lg, dt, a, b, c, d, out, T, E, k, K, N, K_out, flags, scale, ws, nbytes, None)

    for bad in ({"h": None}, {"X": None}, {"lg": None}, {"dt": 3}, {"a": None}, {"b": None}, {"c": None}, {"d": None},
                {"out": None}, {"T": -1}, {"E": 0}, {"k": 0}, {"k": 5}, {"K": 24}, {"N": 64}, {"K_out": 12}, {"flags": 4},
                {"scale": float("nan")}, {"ws": None}, {"ws": P + 16}, {"nbytes": 100}, {"X": P + 8}, {"lg": P + 2},
                {"a": P + 8}, {"b": P + 1}, {"c": P + 8}, {"d": P + 2}, {"out": P + 1}, {"T": 1 << 30}):
        assert call(**bad) == INVALID, bad
    assert call(E=4097) == call(E=64, k=33) == UNSUPPORTED
    assert call(T=0) == rgg.RGG_OK
    size = lib.rgg_moe_swiglu_fp8_block_workspace
    assert size(4, 4, 5, 32, 128, 32) == size(4, 4, 2, 24, 128, 32) == 0
    assert 0 < size(4, 4, 2, 32, 128, 32) < size(4000, 4, 2, 32, 128, 32)
