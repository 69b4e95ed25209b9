"""The 8-bit form with a scale per block of 128, and its grouped products, against their definition in 64 bits, on a GB300."""
import pytest
import torch

import expert_refs
import moe_refs as refs
import ragged_grouped_gemm_02_gb300 as rgg
from ragged_grouped_gemm_02_gb300 import _build

pytestmark = pytest.mark.gpu

CANARY = 0x7FC1
COUNTS = [0, 1, 31, 32, 33, 127, 128, 129, 300, 17, 0, 257]


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available(), "the gpu tests need a CUDA device"
    _build.build()


def _acts(M, K, seed):
    """Rows whose blocks of 32 differ in size by up to 2^12."""
    gen = torch.Generator().manual_seed(seed)
    size = torch.exp2(torch.randint(-6, 7, (M, -(-K // 32)), generator=gen).float()).repeat_interleave(32, 1)[:, :K]
    return (torch.randn(M, K, generator=gen) * size).to(torch.bfloat16)


def _equal(got, want):
    return torch.equal(got.cpu().double(), want.double())


@pytest.mark.parametrize("K", [16, 32, 112, 128, 144, 256, 512, 528, 1040, 2688])
def test_quantize_rows(K):
    X = _acts(67, K, K)
    codes, scales = rgg.rgg_fp8_block_quantize(X.cuda(), check=True)
    want, s, value = refs.fp8_rows(X)
    assert _equal(codes.float(), want) and _equal(scales, s)
    assert _equal(rgg.rgg_fp8_block_dequantize(codes, scales), value.float().to(torch.bfloat16))


def test_every_value_against_every_largest():
    # all bf16 mantissas as the block's largest, beside all mantissas in the exponents below: every tie of the division
    mantissa = 1 + torch.arange(128) / 128
    X = torch.zeros(128, 8 * 128)
    for j in range(8):
        X[:, 128 * j : 128 * j + 127] = (mantissa * 2.0 ** (-2 * j))[:127] * (-1.0) ** torch.arange(127)
        X[:, 128 * j + 127] = 2 * mantissa
    X = (X * torch.exp2(torch.arange(128) % 60 - 30.0)[:, None]).to(torch.bfloat16)
    codes, scales = rgg.rgg_fp8_block_quantize(X.cuda())
    want, s, _ = refs.fp8_rows(X)
    assert _equal(codes.float(), want) and _equal(scales, s)


def test_extreme_values():
    X = torch.zeros(9, 256)
    X[1, 5] = 2.0 ** -133
    X[2, :128] = 2.0 ** -126 * torch.arange(128)
    X[3, 7], X[3, 8] = 3.3895e38, -1e38
    X[4, 0], X[4, 1] = 2.0 ** -100, 2.0 ** -104
    X[5, 0], X[5, 1] = 2.0 ** -101, -2.0 ** -107
    X[6, 3] = float("inf")
    X[7, 200] = float("-inf")
    X[8, 64] = float("nan")
    X[6:9, 10] = 1.0
    X = X.to(torch.bfloat16)
    codes, scales = rgg.rgg_fp8_block_quantize(X.cuda())
    want, s, value = refs.fp8_rows(X[:6])
    assert _equal(codes[:6].float(), want) and _equal(scales[:6], s)
    back = rgg.rgg_fp8_block_dequantize(codes, scales).cpu()
    assert bool(back[6, :128].isnan().all()) and bool(back[7, 128:].isnan().all()) and bool(back[8, :128].isnan().all())
    assert bool(back[6, 128:].isfinite().all()) and bool(back[7, :128].isfinite().all())
    eight = torch.cat([X[:6], X[:2]])  # columns come in eights
    cw, sw = rgg.rgg_fp8_block_quantize_weights(eight.t().contiguous()[None].cuda())
    want, s, _ = refs.fp8_weights(eight[None])
    assert _equal(cw.float(), want) and _equal(sw, s)
    cw, sw = rgg.rgg_fp8_block_quantize_weights(X[6:, :128].t().contiguous().repeat(1, 3)[None, :, :8].contiguous().cuda())
    assert bool(rgg.rgg_fp8_block_dequantize_weights(cw, sw).isnan().all())


@pytest.mark.parametrize("T,k,K", [(1, 1, 16), (5, 3, 144), (40, 4, 512), (130, 2, 1040)])
def test_quantize_to_the_rows_of_the_choices(T, k, K):
    gen = torch.Generator().manual_seed(T)
    experts = refs.choices(gen, T, k, 8, 0.2)
    _, row_index, position = refs.sort(experts, 8)
    rows = int((experts >= 0).sum())
    X = _acts(T, K, 1).cuda()
    codes = torch.full((T * k + 2, K), 0x77, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    scales = torch.full((T * k + 2, -(-K // 128)), 77.0, device="cuda")
    rgg.rgg_fp8_block_quantize(X, position.cuda(), codes, scales, check=True)
    want = rgg.rgg_fp8_block_quantize(X)
    at = row_index[:rows].long().cuda()
    assert torch.equal(codes[:rows].view(torch.uint8), want[0].view(torch.uint8)[at])
    assert torch.equal(scales[:rows], want[1][at])
    assert bool((codes[rows:].view(torch.uint8) == 0x77).all()) and bool((scales[rows:] == 77).all())
    position[0, 0] = T * k + 2
    with pytest.raises(rgg.RggError, match="BAD_ROW_INDEX"):
        rgg.rgg_fp8_block_quantize(X, position.cuda(), codes, scales, check=True)


@pytest.mark.parametrize("E,K,N", [(1, 16, 8), (2, 128, 128), (3, 144, 136), (2, 1040, 264), (1, 256, 1000), (2, 112, 120)])
def test_quantize_weights(E, K, N):
    W = _acts(E * K, N, E + K).view(E, K, N)
    codes, scales = rgg.rgg_fp8_block_quantize_weights(W.cuda())
    want, s, value = refs.fp8_weights(W.transpose(1, 2))
    assert _equal(codes.float(), want) and _equal(scales, s)
    assert _equal(rgg.rgg_fp8_block_dequantize_weights(codes, scales), value.float().to(torch.bfloat16))


def _product_case(counts, K, cols, seed, lead=3, spare=5):
    gen = torch.Generator().manual_seed(seed)
    off, M = expert_refs.ragged(counts, lead, spare)
    X = _acts(M, K, seed)
    W = (torch.randn(len(counts), K, cols, generator=gen) * K ** -0.5).to(torch.bfloat16)
    x, w = rgg.rgg_fp8_block_quantize(X.cuda()), rgg.rgg_fp8_block_quantize_weights(W.cuda())
    return x, w, off, torch.from_numpy(off).cuda()


def _reference(x, w, off):
    """Products of the values that codes and scales stand for, and the sums of their magnitudes; on the GPU, fp64."""
    K = x[0].shape[1]
    xv = x[0].double() * x[1].double().repeat_interleave(128, 1)[:, :K]
    E, N = w[0].shape[:2]
    wv = w[0].double() * w[1].double().repeat_interleave(128, 2)[:, :, :K].repeat_interleave(128, 1)[:, :N]
    ref = torch.full((len(xv), N), float("nan"), dtype=torch.float64, device="cuda")
    mag = torch.zeros_like(ref)
    for e, (a, b) in enumerate(expert_refs.spread(off)):
        ref[a:b] = xv[a:b] @ wv[e].t()
        mag[a:b] = xv[a:b].abs() @ wv[e].abs().t()
    return ref, mag


def _sum_error(mag, K):
    """128 products a block, the blocks one after the other, two roundings of the scales' product."""
    return (128 + -(-K // 128) + 2) * 2.0 ** -23 * mag


def _check(Y, ref, mag, off, K):
    a, b = int(off[0]), int(off[-1])
    limit = refs.rounding(ref, torch.bfloat16) * 1.01 + _sum_error(mag, K)
    error = (Y.double() - ref).abs()
    assert bool((error <= limit)[a:b].all()), float((error - limit)[a:b].max())
    bits = Y.view(torch.int16)
    assert bool((bits[:a] == CANARY).all()) and bool((bits[b:] == CANARY).all())


def _canary(M, N):
    return torch.full((M, N), CANARY, dtype=torch.int16, device="cuda").view(torch.bfloat16)


@pytest.mark.parametrize("K,N,bm", [(16, 8, 128), (16, 8, 256), (128, 128, 128), (256, 256, 256), (144, 264, 128),
                                    (144, 264, 256), (528, 392, 256), (1040, 200, 128), (1024, 512, 256), (2688, 648, 0),
                                    (2048, 1032, 128)])
def test_product(K, N, bm):
    x, w, off, offg = _product_case(COUNTS, K, N, seed=K + N)
    Y = _canary(len(x[0]), N)
    rgg.rgg_grouped_gemm_fp8_block(*x, *w, offg, Y, bm=bm, check=True)
    _check(Y, *_reference(x, w, off), off, K)


def _check_gate_up(h, x, w, off, K):
    gu, mag = _reference(x, w, off)
    a, b = int(off[0]), int(off[-1])
    N = gu.shape[1] // 2
    g, u = gu[a:b, :N], gu[a:b, N:]
    eps = _sum_error(mag, K)[a:b]
    ref = g * torch.sigmoid(g) * u
    # |silu'| <= 1.1, |silu(g)| <= |g|; the exponential's argument error grows with |g| (at most 64 here): 2^-16 of the value
    off_by = 1.1 * eps[:, :N] * u.abs() + (g.abs() + eps[:, :N]) * eps[:, N:] + 2.0 ** -16 * ref.abs()
    top = ref.abs().view(len(ref), -1, 128).amax(-1).clamp(min=2.0 ** -100)
    top_off = off_by.view(len(ref), -1, 128).amax(-1)
    scales = h[1][a:b].double()
    assert bool(((scales - top / 448).abs() <= (top_off + top * 2.0 ** -22) / 448).all())
    wide = scales.repeat_interleave(128, 1)
    error = (h[0][a:b].double() * wide - ref).abs()
    # half a step of E4M3: 2^-4 of the value, or half the spacing of its smallest values
    limit = (ref.abs() + off_by) * 2.0 ** -4 + wide * 2.0 ** -10 + off_by + wide * 448 * 2.0 ** -22
    assert bool((error <= limit).all()), float((error - limit).max())


@pytest.mark.parametrize("bm", [128, 256])
@pytest.mark.parametrize("K,N", [(16, 128), (144, 256), (1040, 384), (512, 128)])
def test_gate_up(K, N, bm):
    x, w, off, offg = _product_case(COUNTS, K, 2 * N, seed=K + N)
    M = len(x[0])
    codes = torch.full((M, N), 0x77, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    scales = torch.full((M, N // 128), 77.0, device="cuda")
    h = rgg.rgg_grouped_gemm_swiglu_fp8_block(*x, *w, offg, codes, scales, bm=bm, check=True)
    _check_gate_up(h, x, w, off, K)
    a, b = int(off[0]), int(off[-1])
    bits = codes.view(torch.uint8)
    assert bool((bits[:a] == 0x77).all()) and bool((bits[b:] == 0x77).all())
    assert bool((scales[:a] == 77).all()) and bool((scales[b:] == 77).all())


@pytest.mark.parametrize("K,N", [(16, 8), (144, 264), (528, 392), (1040, 200), (256, 512)])
@pytest.mark.parametrize("bn", [128, 256])
def test_single_cta_tiles(K, N, bn):
    x, w, off, offg = _product_case(COUNTS, K, N, seed=K + N)
    Y = _canary(len(x[0]), N)
    rgg.rgg_grouped_gemm_fp8_block(*x, *w, offg, Y, bm=128, bn=bn, check=True)
    _check(Y, *_reference(x, w, off), off, K)


@pytest.mark.parametrize("gate_up", [False, True])
@pytest.mark.parametrize("counts", [[1], [0, 0, 5], [1] * 70, [600], [256] * 4, [3, 1500, 2, 90]])
def test_routings(counts, gate_up):
    K, N = 272, 256
    x, w, off, offg = _product_case(counts, K, 2 * N if gate_up else N, seed=len(counts), lead=0, spare=0)
    results = []
    for bm in (0, 128, 256):
        if gate_up:
            h = rgg.rgg_grouped_gemm_swiglu_fp8_block(*x, *w, offg, bm=bm, check=True)
            _check_gate_up(h, x, w, off, K)
            results.append(h[0].view(torch.uint8))
        else:
            Y = rgg.rgg_grouped_gemm_fp8_block(*x, *w, offg, bm=bm, check=True)
            _check(Y, *_reference(x, w, off), off, K)
            results.append(Y)
    assert all(torch.equal(results[0], r) for r in results[1:]), "the tile shape does not change a result"


def test_long_walks_on_few_ctas():
    # many tiles for each CTA: stages, accumulators and magnitudes go round many times
    x, w, off, offg = _product_case([700, 3, 260, 129], 656, 512, seed=3)
    for bm, max_ctas in ((128, 1), (128, 3), (256, 2), (256, 6)):
        for stages in (2, 3, 0):
            Y = _canary(len(x[0]), 512)
            rgg.rgg_grouped_gemm_fp8_block(*x, *w, offg, Y, bm=bm, max_ctas=max_ctas, stages=stages, check=True)
            _check(Y, *_reference(x, w, off), off, 656)
            h = rgg.rgg_grouped_gemm_swiglu_fp8_block(*x, *w, offg, bm=bm, max_ctas=max_ctas, stages=stages, check=True)
            _check_gate_up(h, x, w, off, 656)


def test_rows_of_no_expert_and_neighbours_do_not_matter():
    # NaN in rows of no expert, and in the rows of one expert, stay out of all other rows
    x, w, off, offg = _product_case([40, 7, 100], 256, 256, seed=6)
    for bm in (128, 256):
        want = rgg.rgg_grouped_gemm_fp8_block(*x, *w, offg, _canary(len(x[0]), 256), bm=bm)
        codes, scales = x[0].clone(), x[1].clone()
        a, b = int(off[0]), int(off[-1])
        codes.view(torch.uint8)[:a] = 0x7F
        codes.view(torch.uint8)[b:] = 0x7F
        scales[b:] = float("nan")
        codes.view(torch.uint8)[int(off[1]) : int(off[2])] = 0x7F
        got = rgg.rgg_grouped_gemm_fp8_block(codes, scales, *w, offg, _canary(len(x[0]), 256), bm=bm, check=True)
        bad = slice(int(off[1]), int(off[2]))
        assert bool(got[bad].isnan().all())
        keep = torch.ones(len(got), dtype=torch.bool, device="cuda")
        keep[bad] = False
        assert torch.equal(got.view(torch.int16)[keep], want.view(torch.int16)[keep])


def test_inputs_with_nan_and_inf_come_out_as_nan():
    X = _acts(6, 256, 1)
    X[1, 3], X[4, 200] = float("nan"), float("inf")
    W = torch.randn(1, 256, 64, generator=torch.Generator().manual_seed(0)).to(torch.bfloat16)
    off = torch.tensor([0, 6], dtype=torch.int32, device="cuda")
    Y = rgg.rgg_grouped_gemm_fp8_block(*rgg.rgg_fp8_block_quantize(X.cuda()), *rgg.rgg_fp8_block_quantize_weights(W.cuda()),
                                       off, check=True)
    assert Y.isnan().all(1).tolist() == [False, True, False, False, True, False]
    assert bool(Y[[0, 2, 3, 5]].isfinite().all())


def test_bad_offsets_write_nothing():
    x, w, off, offg = _product_case([5, 9], 128, 128, seed=1)
    bad = offg.clone()
    bad[1] = bad[2] + 1
    Y = _canary(len(x[0]), 128)
    with pytest.raises(rgg.RggError, match="BAD_OFFSETS"):
        rgg.rgg_grouped_gemm_fp8_block(*x, *w, bad, Y, check=True)
    assert bool((Y.view(torch.int16) == CANARY).all())


@pytest.mark.parametrize("gate_up", [False, True])
@pytest.mark.parametrize("bm", [128, 256])
def test_a_stalled_pipeline_is_reported(bm, gate_up):
    x, w, off, offg = _product_case([300, 9], 512, 256, seed=1)
    call = rgg.rgg_grouped_gemm_swiglu_fp8_block if gate_up else rgg.rgg_grouped_gemm_fp8_block
    with pytest.raises(rgg.RggError, match="TIMEOUT"):
        call(*x, *w, offg, bm=bm, timeout_ns=20_000_000, debug_flags=rgg.RGG_DEBUG_PRODUCER_STALL, check=True)
    if not gate_up:  # and the handle works on
        _check(rgg.rgg_grouped_gemm_fp8_block(*x, *w, offg, _canary(len(x[0]), 256), bm=bm, check=True),
               *_reference(x, w, off), off, 512)


def test_no_rows():
    x, w, off, offg = _product_case([4], 128, 128, seed=1)
    none = torch.zeros(2, dtype=torch.int32, device="cuda")
    assert rgg.rgg_grouped_gemm_fp8_block(x[0][:0], x[1][:0], *w, none, check=True).shape == (0, 128)
    assert rgg.rgg_fp8_block_quantize(torch.empty(0, 32, dtype=torch.bfloat16, device="cuda"))[0].shape == (0, 32)
    Y = _canary(len(x[0]), 128)
    rgg.rgg_grouped_gemm_fp8_block(*x, *w, none, Y, check=True)
    assert bool((Y.view(torch.int16) == CANARY).all())
