"""MXFP4 quantisers and grouped product against their definition in 64 bits, on a GB300."""
import numpy as np
import pytest
import torch

import expert_refs as refs
import ragged_grouped_gemm_02_gb300 as rgg
from ragged_grouped_gemm_02_gb300 import _build

pytestmark = pytest.mark.gpu

CANARY = 0x7FC1
MAGNITUDES = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)
COUNTS = [0, 1, 31, 32, 33, 127, 128, 129, 300, 17, 0, 257]


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available(), "the gpu tests need a CUDA device"
    _build.build()


def mx(x):
    """What MXFP4 holds of x (bf16 [..., K]) in fp64, and its scale bytes: the nearest of the magnitudes, ties to the
    even code; blocks with Inf or NaN are NaN."""
    b = x.double().reshape(*x.shape[:-1], -1, 32)
    top = b.abs().amax(-1, keepdim=True)
    bad = ~torch.isfinite(b).all(-1, keepdim=True)
    b = torch.where(bad, torch.zeros_like(b), b)
    exponent = torch.frexp(torch.where(bad, torch.ones_like(top), top)).exponent - 1
    exponent = torch.clamp(torch.where(b.abs().amax(-1, keepdim=True) > 0, exponent, -1000) - 2, min=-127)
    scale = torch.pow(torch.tensor(2.0, dtype=torch.float64), exponent.double())
    dist = ((b / scale).abs().unsqueeze(-1) - MAGNITUDES).abs()
    best = dist.amin(-1, keepdim=True)
    near = dist == best  # one code, or two neighbours at a tie: the even one
    code = torch.where(near.sum(-1) == 2, (near * torch.arange(8) * (torch.arange(8) % 2 == 0)).sum(-1),
                       near.to(torch.int64).argmax(-1))
    value = torch.sign(b) * MAGNITUDES[code] * scale
    value = torch.where(bad, torch.full_like(value, float("nan")), value)
    byte = torch.where(bad, 255, exponent + 127)[..., 0]
    return value.reshape(x.shape), byte.to(torch.uint8)


def _acts(counts, K, seed, lead=3, spare=5):
    gen = torch.Generator().manual_seed(seed)
    off, M = refs.ragged(counts, lead, spare)
    X = refs.normal(gen, M, K) * torch.exp2(torch.randint(-6, 7, (M, K // 32), generator=gen).repeat_interleave(32, 1))
    return X.to(torch.bfloat16), off


def _scale_at(scales, off, e, r, K):
    """Scale bytes of row r of expert e, from the documented layout."""
    blocks = scales[int(off[e]) // 128 + e + r // 128]
    return torch.stack([blocks[s // 4, (r % 32) * 16 + (r % 128) // 32 * 4 + s % 4] for s in range(K // 32)])


@pytest.mark.parametrize("K", [32, 64, 96, 160, 256, 1024, 1056, 2080])
def test_quantize_rows(K):
    X, off = _acts(COUNTS, K, seed=K)
    codes = torch.full((X.shape[0], K // 2), 0x77, dtype=torch.uint8, device="cuda")
    codes, scales = rgg.rgg_mxfp4_quantize(X.cuda(), torch.from_numpy(off).cuda(), codes, check=True)
    value, byte = mx(X)
    c = codes.cpu()
    got = torch.stack((c & 15, c >> 4), -1).reshape(X.shape)
    a, b = int(off[0]), int(off[-1])
    signed = torch.cat([MAGNITUDES, -MAGNITUDES])
    scales = scales.cpu()
    scale = torch.pow(torch.tensor(2.0, dtype=torch.float64), byte.double() - 127).repeat_interleave(32, 1)
    assert torch.equal((signed[got.long()] * scale)[a:b], value[a:b])
    for e, (lo, hi) in enumerate(refs.spread(off)):
        for r in {0, 1, 31, 32, 127, 128, 200, hi - lo - 1} & set(range(hi - lo)):
            assert torch.equal(_scale_at(scales, off, e, r, K), byte[lo + r])
            if K % 128:
                row = scales[lo // 128 + e + r // 128, -1]
                first = (r % 32) * 16 + (r % 128) // 32 * 4
                assert not bool(row[first + (K % 128) // 32:first + 4].any()), "scales past K are 0"
    assert bool((c[:a] == 0x77).all()) and bool((c[b:] == 0x77).all())
    back = torch.full(X.shape, CANARY, dtype=torch.int16, device="cuda").view(torch.bfloat16)
    rgg.rgg_mxfp4_dequantize(codes, scales.cuda(), torch.from_numpy(off).cuda(), back, check=True)
    assert torch.equal(back.cpu().double()[a:b], value[a:b])
    bits = back.cpu().view(torch.int16)
    assert bool((bits[:a] == CANARY).all()) and bool((bits[b:] == CANARY).all())


@pytest.mark.parametrize("E,K,N", [(1, 32, 8), (2, 64, 128), (3, 160, 136), (2, 1056, 264), (1, 256, 1000)])
def test_quantize_weights(E, K, N):
    gen = torch.Generator().manual_seed(E + K + N)
    W = refs.normal(gen, E, K, N, std=K ** -0.5)
    codes, scales = rgg.rgg_mxfp4_quantize_weights(W.cuda())
    value, byte = mx(W.transpose(1, 2).contiguous())
    assert torch.equal(rgg.rgg_mxfp4_dequantize_weights(codes, scales).cpu().double(), value)
    s = scales.cpu()
    for e in range(E):
        for n in {0, 7, N // 2, N - 1}:
            got = torch.stack([s[e, n // 128, k // 4, (n % 32) * 16 + (n % 128) // 32 * 4 + k % 4]
                               for k in range(K // 32)])
            assert torch.equal(got, byte[e, n])


def test_every_code_and_tie():
    # every bf16 between 4 and 8 as the block's largest beside a sweep of values over all codes and their midpoints
    sweep = torch.tensor([0.0, 0.25, 0.5, 0.75, 1.0, 1.25, 1.5, 1.75, 2.0, 2.5, 3.0, 3.5, 4.0, 4.99, 5.0, 5.01])
    rows = []
    for i in range(128):
        row = torch.cat([sweep, -sweep]).clone()
        row[31] = 4.0 + i / 32
        rows.append(row * 2.0 ** (i % 40 - 20))
    X = torch.stack(rows).to(torch.bfloat16)
    off = torch.tensor([0, 128], dtype=torch.int32, device="cuda")
    codes, scales = rgg.rgg_mxfp4_quantize(X.cuda(), off, check=True)
    assert torch.equal(rgg.rgg_mxfp4_dequantize(codes, scales, off).cpu().double(), mx(X)[0])


def test_extremes():
    # zeros, bf16's smallest and largest values, Inf and NaN
    X = torch.zeros(8, 64)
    X[1, 5] = 2.0 ** -133
    X[2, :32] = 2.0 ** -126 * torch.arange(32)
    X[3, 7] = 3.3895e38
    X[3, 8] = -1e38
    X[4, 3] = float("inf")
    X[5, 40] = float("-inf")
    X[6, 63] = float("nan")
    X[7, 0] = -2.0 ** -127
    X[4:7, 10] = 1.0
    X = X.to(torch.bfloat16)
    off = torch.tensor([0, 3, 8], dtype=torch.int32, device="cuda")
    codes, scales = rgg.rgg_mxfp4_quantize(X.cuda(), off, check=True)
    got = rgg.rgg_mxfp4_dequantize(codes, scales, off).cpu().double()
    want = mx(X)[0]
    assert torch.equal(got.nan_to_num(nan=7.0), want.nan_to_num(nan=7.0))
    assert torch.equal(got.isnan(), want.isnan()) and bool(want[4, :32].isnan().all())
    cw, sw = rgg.rgg_mxfp4_quantize_weights(X.t().contiguous()[None].cuda())
    back = rgg.rgg_mxfp4_dequantize_weights(cw, sw).cpu().double()[0]
    assert torch.equal(back.nan_to_num(nan=7.0), want.nan_to_num(nan=7.0))


def _product_case(counts, K, cols, seed, lead=3, spare=5):
    X, off = _acts(counts, K, seed, lead, spare)
    W = refs.normal(torch.Generator().manual_seed(seed + 1), len(counts), K, cols, std=K ** -0.5)
    offg = torch.from_numpy(off).cuda()
    xq = rgg.rgg_mxfp4_quantize(X.cuda(), offg, check=True)
    wq = rgg.rgg_mxfp4_quantize_weights(W.cuda())
    return X, W, off, offg, xq, wq


def _reference(X, W, off):
    """Products of the values and the sums of their magnitudes."""
    x, w = mx(X)[0], mx(W.transpose(1, 2).contiguous())[0]
    ref = torch.full((X.shape[0], w.shape[1]), float("nan"), dtype=torch.float64)
    mag = torch.zeros_like(ref)
    for e, (a, b) in enumerate(refs.spread(off)):
        ref[a:b] = x[a:b] @ w[e].t()
        mag[a:b] = x[a:b].abs() @ w[e].abs().t()
    return ref, mag


def _canary_out(M, N):
    return torch.full((M, N), CANARY, dtype=torch.int16, device="cuda").view(torch.bfloat16)


def _check_rows(got, ref, limit, off):
    a, b = int(off[0]), int(off[-1])
    refs.assert_close(got[a:b], ref[a:b], limit[a:b], "Y")
    bits = got.cpu().view(torch.int16)
    assert bool((bits[:a] == CANARY).all()) and bool((bits[b:] == CANARY).all())


@pytest.mark.parametrize("K,N,bn", [(32, 8, 128), (32, 8, 256), (64, 128, 128), (256, 256, 256), (96, 264, 128),
                                    (96, 264, 256), (544, 392, 256), (1056, 200, 128), (1024, 512, 256),
                                    (2080, 648, 0)])
def test_product(K, N, bn):
    X, W, off, offg, xq, wq = _product_case(COUNTS, K, N, seed=K + N)
    Y = _canary_out(X.shape[0], N)
    rgg.rgg_grouped_gemm_mxfp4(*xq, *wq, offg, Y, bn=bn, check=True)
    ref, mag = _reference(X, W, off)
    _check_rows(Y, ref, refs.bound(ref, K, mag), off)


@pytest.mark.parametrize("bn", [128, 256])
@pytest.mark.parametrize("K,N", [(32, 128), (544, 128), (256, 384), (1056, 256)])
def test_gate_up(K, N, bn):
    X, W, off, offg, xq, wq = _product_case(COUNTS, K, 2 * N, seed=K + N)
    H = _canary_out(X.shape[0], N)
    rgg.rgg_grouped_gemm_swiglu_mxfp4(*xq, *wq, offg, H, bn=bn, check=True)
    gu, mag = _reference(X, W, off)
    g, u = gu[:, :N], gu[:, N:]
    eps = K * 2.0 ** -23 * mag
    ref = g * torch.sigmoid(g) * u
    limit = refs.ROUND_BF16 * ref.abs() + g.abs() * eps[:, N:] + 1.1 * u.abs() * eps[:, :N] + \
        2.0 ** -18 * (g * u).abs() + refs.TINY
    _check_rows(H, ref, limit, off)


@pytest.mark.parametrize("stages,max_ctas", [(2, 2), (3, 3), (0, 6)])
def test_long_walks(stages, max_ctas):
    # many tiles a CTA: the accumulators, their shared columns and the ring go round
    X, W, off, offg, xq, wq = _product_case(COUNTS, 800, 712, seed=stages)
    ref, mag = _reference(X, W, off)
    for bn in (128, 256):
        Y = _canary_out(X.shape[0], 712)
        rgg.rgg_grouped_gemm_mxfp4(*xq, *wq, offg, Y, bn=bn, stages=stages, max_ctas=max_ctas, check=True)
        _check_rows(Y, ref, refs.bound(ref, 800, mag), off)


@pytest.mark.parametrize("counts", [[1], [0, 0, 1], [700], [16] * 32, [100] * 8, [512] * 3, [1] * 200])
def test_planned(counts):
    X, W, off, offg, xq, wq = _product_case(counts, 288, 264, seed=len(counts), lead=0, spare=0)
    ref, mag = _reference(X, W, off)
    Y = _canary_out(X.shape[0], 264)
    rgg.rgg_grouped_gemm_mxfp4(*xq, *wq, offg, Y, check=True)
    _check_rows(Y, ref, refs.bound(ref, 288, mag), off)


def test_a_bad_row_stays_alone():
    # Inf and NaN activations spoil their own rows, not their tile's others
    X, off = _acts([70, 60], 96, seed=5, lead=0, spare=0)
    W = refs.normal(torch.Generator().manual_seed(6), 2, 96, 136)
    X[3, 40], X[100, 0] = float("inf"), float("nan")
    offg = torch.from_numpy(off).cuda()
    xq, wq = rgg.rgg_mxfp4_quantize(X.cuda(), offg), rgg.rgg_mxfp4_quantize_weights(W.cuda())
    Y = rgg.rgg_grouped_gemm_mxfp4(*xq, *wq, offg, check=True).cpu()
    good = [i for i in range(130) if i not in (3, 100)]
    X[3], X[100] = 0, 0
    ref, mag = _reference(X, W, off)
    refs.assert_close(Y[good], ref[good], refs.bound(ref, 96, mag)[good], "Y")
    assert bool(Y[3].isnan().all()) and bool(Y[100].isnan().all())


def test_no_rows():
    X, W, off, offg, xq, wq = _product_case([0, 0], 64, 128, seed=7)
    Y = _canary_out(X.shape[0], 128)
    rgg.rgg_grouped_gemm_mxfp4(*xq, *wq, offg, Y, check=True)
    assert bool((Y.cpu().view(torch.int16) == CANARY).all())


def test_graph():
    X, W, off, offg, xq, wq = _product_case([40, 3, 200], 352, 256, seed=8, lead=0, spare=0)
    want = rgg.rgg_grouped_gemm_mxfp4(*xq, *wq, offg, check=True)
    graph = torch.cuda.CUDAGraph()
    Xg = X.cuda()
    with torch.cuda.graph(graph):
        c, s = rgg.rgg_mxfp4_quantize(Xg, offg)
        Y = rgg.rgg_grouped_gemm_mxfp4(c, s, *wq, offg)
    Y.fill_(7)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(Y, want)


def test_producer_stall_is_reported():
    X, W, off, offg, xq, wq = _product_case([40, 3], 64, 128, seed=9)
    with pytest.raises(rgg.RggError) as ei:
        rgg.rgg_grouped_gemm_mxfp4(*xq, *wq, offg, check=True, timeout_ns=20_000_000,
                                   debug_flags=rgg.RGG_DEBUG_PRODUCER_STALL)
    assert ei.value.status == rgg.RGG_ERR_DEVICE_TIMEOUT


def test_refusals():
    X, W, off, offg, xq, wq = _product_case([5, 6], 64, 264, seed=10, lead=0, spare=0)
    Xg, Wg = X.cuda(), W.cuda()
    for call, error in ((lambda: rgg.rgg_mxfp4_quantize(Xg.float(), offg), TypeError),
                        (lambda: rgg.rgg_mxfp4_quantize(Xg, offg.long()), TypeError),
                        (lambda: rgg.rgg_mxfp4_quantize(X, offg), ValueError),
                        (lambda: rgg.rgg_mxfp4_quantize(Xg.t(), offg), ValueError),
                        (lambda: rgg.rgg_mxfp4_quantize_weights(Wg[0]), ValueError),
                        (lambda: rgg.rgg_mxfp4_dequantize(xq[0], xq[1][:1], offg), ValueError),
                        (lambda: rgg.rgg_grouped_gemm_mxfp4(xq[0].float(), xq[1], *wq, offg), TypeError),
                        (lambda: rgg.rgg_grouped_gemm_mxfp4(*xq, wq[0][:, :, :16], wq[1], offg), ValueError),
                        (lambda: rgg.rgg_grouped_gemm_mxfp4(*xq, *wq, offg[:2]), ValueError)):
        with pytest.raises(error):
            call()
    # K of no whole blocks; a gate-up width of no whole blocks of scales; a tile that is not there
    for call in (lambda: rgg.rgg_mxfp4_quantize(Xg[:, :48].contiguous(), offg),
                 lambda: rgg.rgg_mxfp4_quantize_weights(Wg[:, :48].contiguous()),
                 lambda: rgg.rgg_mxfp4_quantize_weights(Wg[:, :, :12].contiguous()),
                 lambda: rgg.rgg_grouped_gemm_swiglu_mxfp4(*xq, *wq, offg),
                 lambda: rgg.rgg_grouped_gemm_mxfp4(*xq, *wq, offg, bn=192),
                 lambda: rgg.rgg_grouped_gemm_mxfp4(*xq, *wq, offg, bn=256, max_ctas=1)):
        with pytest.raises(rgg.RggError) as ei:
            call()
        assert ei.value.status == rgg.RGG_ERR_INVALID_ARG
    bad = torch.tensor([0, 6, 5], dtype=torch.int32, device="cuda")
    Y = _canary_out(11, 264)
    codes = torch.full((11, 32), 0x77, dtype=torch.uint8, device="cuda")
    for call in (lambda: rgg.rgg_grouped_gemm_mxfp4(*xq, *wq, bad, Y, check=True),
                 lambda: rgg.rgg_mxfp4_quantize(Xg, bad, codes, check=True),
                 lambda: rgg.rgg_mxfp4_dequantize(*xq, bad, Xg.fill_(5), check=True)):
        with pytest.raises(rgg.RggError) as ei:
            call()
        assert ei.value.status == rgg.RGG_ERR_BAD_OFFSETS
    assert bool((Y.view(torch.int16) == CANARY).all()) and bool((codes == 0x77).all()) and bool((Xg == 5).all())
