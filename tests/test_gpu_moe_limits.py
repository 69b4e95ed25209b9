"""Sorting, moving rows and the block-scaled 8-bit product at the sizes where 32 bits end, on a GB300."""
import gc

import pytest
import torch

import ragged_grouped_gemm_02_gb300 as rgg
from ragged_grouped_gemm_02_gb300 import _build

pytestmark = pytest.mark.gpu

ROWS = 2 ** 31 - 1


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available(), "the gpu tests need a CUDA device"
    _build.build()
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 120e9:
        pytest.skip("needs 120 GB of device memory")
    yield
    gc.collect()
    torch.cuda.empty_cache()


def test_sort_of_the_most_choices():
    experts = torch.empty(ROWS, 1, dtype=torch.int32, device="cuda")
    for e in range(3):  # token i goes to expert i % 3
        experts[e::3] = e
    offsets, row_index, position = rgg.rgg_sort_by_expert(experts, 3, check=True)
    each = [len(range(e, ROWS, 3)) for e in range(3)]
    assert offsets.tolist() == [0, each[0], each[0] + each[1], ROWS]
    for e in range(3):
        lo = int(offsets[e])
        want = torch.arange(each[e], device="cuda")
        assert torch.equal(position[e::3, 0], (lo + want).to(torch.int32))
        assert torch.equal(row_index[lo : lo + each[e]], (3 * want + e).to(torch.int32))


def test_rows_past_four_gigabytes():
    # 400,000 rows of 6,146 values: 4.9 GB, of an even and of an odd number of 16-byte blocks
    T, k = 50_000, 8
    gen = torch.Generator(device="cuda").manual_seed(0)
    order = torch.randperm(T * k, generator=gen, device="cuda").to(torch.int32).view(T, k)
    back = torch.empty(T * k, dtype=torch.long, device="cuda")
    back[order.view(-1).long()] = torch.arange(T * k, device="cuda") // k
    for K in (6144, 6147):
        X = torch.randint(-8, 9, (T, K), generator=gen, device="cuda").to(torch.bfloat16)
        rows = rgg.rgg_dispatch(X, order, check=True)
        for a in range(0, T * k, 50_000):
            assert torch.equal(rows[a : a + 50_000], X[back[a : a + 50_000]])
        w = torch.full((T, k), 0.125, device="cuda")
        out = rgg.rgg_combine(rows, order, w, check=True)
        assert torch.equal(out, X)  # eighths of eight equal rows: exact
        dY, dw = rgg.rgg_combine_backward(X, rows, order, w, check=True)
        for a in range(0, T * k, 50_000):
            assert torch.equal(dY[a : a + 50_000], rows[a : a + 50_000] * 0.125)
        norms = X.float().square().sum(1, keepdim=True).expand(T, k)
        assert torch.equal(dw, norms)  # sums of whole numbers below 2^24: exact
        if K % 16 == 0:
            codes, scales = rgg.rgg_fp8_block_quantize(X, order, check=True)
            want = rgg.rgg_fp8_block_quantize(X)
            for a in range(0, T * k, 50_000):
                at = back[a : a + 50_000]
                assert torch.equal(codes[a : a + 50_000].view(torch.uint8), want[0].view(torch.uint8)[at])
                assert torch.equal(scales[a : a + 50_000], want[1][at])
            del codes, scales, want
        del X, rows, out, dY, dw


@pytest.mark.parametrize("opts", [dict(), dict(bm=128, bn=128), dict(bm=128, bn=256), dict(bm=256)], ids=str)
def test_product_of_the_most_rows(opts):
    base = 2 ** 20  # the rows repeat after so many
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randint(-4, 5, (base, 16), generator=gen, device="cuda").float()
    w = torch.randint(-4, 5, (1, 8, 16), generator=gen, device="cuda").float()
    want = (x @ w[0].t()).to(torch.bfloat16)  # exact
    codes = torch.empty(ROWS, 16, dtype=torch.uint8, device="cuda")
    n = ROWS // base
    codes[: n * base].view(n, base, 16).copy_(x.to(torch.float8_e4m3fn).view(torch.uint8))
    codes[n * base :].copy_(codes[: ROWS - n * base])
    y = torch.full((ROWS, 8), float("nan"), dtype=torch.bfloat16, device="cuda")
    rgg.rgg_grouped_gemm_fp8_block(codes.view(torch.float8_e4m3fn), torch.ones(ROWS, 1, device="cuda"),
                                   w.to(torch.float8_e4m3fn), torch.ones(1, 1, 1, device="cuda"),
                                   torch.tensor([0, ROWS], dtype=torch.int32, device="cuda"), y, check=True, **opts)
    whole = y[: n * base].view(n, base, 8)
    for i in range(n):
        if not torch.equal(whole[i], want):
            raise AssertionError("rows from %d" % (i * base))
    assert torch.equal(y[n * base :], want[: ROWS - n * base])


def test_product_of_the_most_experts():
    E, K, N = 4096, 32, 128
    gen = torch.Generator(device="cuda").manual_seed(2)
    counts = torch.randint(0, 4, (E,), generator=gen, device="cuda")
    off = torch.cat([torch.zeros(1, device="cuda"), counts.cumsum(0)]).to(torch.int32)
    M = int(off[-1])
    x = torch.randint(-4, 5, (M, K), generator=gen, device="cuda").float()
    w = torch.randint(-4, 5, (E, 2 * N, K), generator=gen, device="cuda").float()
    owner = torch.repeat_interleave(torch.arange(E, device="cuda"), counts)
    want = torch.einsum("mk,mnk->mn", x, w[owner])
    args = (x.to(torch.float8_e4m3fn), torch.ones(M, 1, device="cuda"), w.to(torch.float8_e4m3fn),
            torch.ones(E, 2, 1, device="cuda"), off)
    for opts in (dict(), dict(bm=128, bn=256), dict(bm=256)):
        assert torch.equal(rgg.rgg_grouped_gemm_fp8_block(*args, check=True, **opts), want.to(torch.bfloat16))
    codes, scales = rgg.rgg_grouped_gemm_swiglu_fp8_block(*args, check=True)
    h = torch.nn.functional.silu(want[:, :N].double()) * want[:, N:].double()
    top = h.abs().amax(1, keepdim=True).clamp(min=2.0 ** -100)
    # half a step of E4M3, or of its smallest values' spacing; 2^-16 for the exponential and the scale
    limit = h.abs() * 2.0 ** -4 + top / 448 * 2.0 ** -10 + top * 2.0 ** -16
    assert bool(((codes.double() * scales.double() - h).abs() <= limit).all())
