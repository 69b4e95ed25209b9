"""rgg_grouped_gemm_wgrad (dW_e = X_e^T . dY_e) against 64-bit products, on a GB300."""
import numpy as np
import pytest
import torch

import expert_refs as refs
import ragged_grouped_gemm_02_gb300 as rgg
from ragged_grouped_gemm_02_gb300 import _build

pytestmark = pytest.mark.gpu

# every remainder of the 64-row stage and of its 16-row steps, among them one row and whole stages
COUNTS = [0, 1, 15, 16, 17, 31, 48, 63, 64, 65, 127, 128, 129, 300, 0, 513]
SIZES = [(264, 520), (512, 64), (8, 8), (136, 256), (256, 392)]


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available(), "the gpu tests need a CUDA device"
    _build.build()


def _case(counts, K, N, seed, lead=3, spare=5):
    gen = torch.Generator().manual_seed(seed)
    off, M = refs.ragged(counts, lead, spare)
    X, dY = refs.normal(gen, M, K), refs.normal(gen, M, N)
    # rows of no expert hold what must not reach a result
    X[: off[0]] = float("nan")
    dY[: off[0]] = float("inf")
    X[off[-1]:] = float("inf")
    dY[off[-1]:] = float("nan")
    return X, dY, off


def _run(X, dY, off, dW=None, **opts):
    if dW is None:
        shape = (len(off) - 1, X.shape[1], dY.shape[1])
        dW = torch.full(shape, float("nan"), dtype=opts.get("dtype") or torch.bfloat16, device="cuda")
    got = rgg.rgg_grouped_gemm_wgrad(X.cuda(), dY.cuda(), torch.from_numpy(off).cuda(), dW, check=True, **opts)
    assert got is dW
    return got.cpu()


def _limit(ref, mag, off, dtype, old=None):
    """n * 2^-23 of the summed magnitudes (and of the value added to), plus half a bf16 unit for a bf16 result."""
    n = torch.from_numpy(np.diff(off).astype(np.float64))[:, None, None]
    extra = 0 if old is None else old.double().abs()
    limit = (n + 1) * 2.0 ** -23 * (mag + extra) + refs.TINY
    return limit + (refs.ROUND_BF16 * ref.abs() if dtype == torch.bfloat16 else 0)


def _check(X, dY, off, dW):
    ref, mag = refs.wgrad(X, dY, off)
    refs.assert_close(dW, ref, _limit(ref, mag, off, dW.dtype), "dW")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("bn", [128, 256])
@pytest.mark.parametrize("K,N", SIZES)
def test_tile_shapes_and_tails(K, N, bn, dtype):
    X, dY, off = _case(COUNTS, K, N, seed=K + bn)
    _check(X, dY, off, _run(X, dY, off, bn=bn, dtype=dtype))


@pytest.mark.parametrize("stages,max_ctas", [(2, 2), (3, 4), (2, 0), (0, 6)])
def test_small_rings_and_grids(stages, max_ctas):
    # tails reuse the ring's slots many times over
    X, dY, off = _case(COUNTS * 3, 264, 264, seed=stages)
    _check(X, dY, off, _run(X, dY, off, stages=stages, max_ctas=max_ctas, bn=128))
    _check(X, dY, off, _run(X, dY, off, stages=stages, max_ctas=max_ctas, bn=256))


@pytest.mark.parametrize("counts", [[1], [0, 0, 1], [2048], [16] * 32, [100] * 8, [1024] * 3, [1] * 300, [0] * 5])
def test_planned(counts):
    X, dY, off = _case(counts, 328, 200, seed=len(counts), lead=0, spare=0)
    _check(X, dY, off, _run(X, dY, off))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("N", [264, 256])
def test_accumulate(dtype, N):
    X, dY, off = _case(COUNTS, 136, N, seed=9)
    old = torch.randn(len(COUNTS), 136, N, generator=torch.Generator().manual_seed(10)).to(dtype)
    got = _run(X, dY, off, old.cuda(), accumulate=True)
    ref, mag = refs.wgrad(X, dY, off)
    refs.assert_close(got, ref + old.double(), _limit(ref + old.double(), mag, off, dtype, old), "dW")
    for e in (0, 14):
        assert torch.equal(got[e], old[e]), "an expert without rows is left alone"


SPLIT = [[4096], [15000, 0, 3603], [2, 9000], [9000, 9001, 8999, 1]]


def _splits(counts, K, N):
    return rgg.load_library().rgg_grouped_gemm_wgrad_workspace(rgg._handle(0), len(counts), sum(counts), K, N, 0) > 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("counts", SPLIT)
def test_rows_split_where_tiles_are_few(counts, dtype):
    assert _splits(counts, 136, 264)
    X, dY, off = _case(counts, 136, 264, seed=len(counts), lead=0, spare=0)
    got = _run(X, dY, off, dtype=dtype)
    _check(X, dY, off, got)
    assert torch.equal(_run(X, dY, off, dtype=dtype), got), "equal calls give equal bits"
    old = torch.randn(len(counts), 136, 264, generator=torch.Generator().manual_seed(21)).to(dtype)
    old[counts.index(0) if 0 in counts else 0, 0, 0] = -0.0
    added = _run(X, dY, off, old.cuda(), accumulate=True)
    ref, mag = refs.wgrad(X, dY, off)
    refs.assert_close(added, ref + old.double(), _limit(ref + old.double(), mag, off, dtype, old), "dW")
    if 0 in counts:
        e, bits = counts.index(0), torch.int16 if dtype == torch.bfloat16 else torch.int32
        assert not bool(got[e].any()) and torch.equal(added[e].view(bits), old[e].view(bits))


def test_split_rows_with_bad_offsets_write_nothing():
    X, dY, _ = _case([4096, 4096], 64, 72, seed=22, lead=0, spare=0)
    assert _splits([4096, 4096], 64, 72)
    dW = torch.full((2, 64, 72), 3.0, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(rgg.RggError) as ei:
        rgg.rgg_grouped_gemm_wgrad(X.cuda(), dY.cuda(), torch.tensor([0, 5000, 4000], dtype=torch.int32, device="cuda"),
                                   dW, check=True)
    assert ei.value.status == rgg.RGG_ERR_BAD_OFFSETS
    assert bool((dW == 3).all())


def test_workspace_too_small():
    X, dY, off = _case([4096], 64, 72, seed=23, lead=0, spare=0)
    X, dY, off = X.cuda(), dY.cuda(), torch.from_numpy(off).cuda()
    dW = torch.empty(1, 64, 72, dtype=torch.bfloat16, device="cuda")
    opt, _ = rgg._options()
    rgg._set_workspace(opt, torch.empty(64, device="cuda"))
    s = rgg.load_library().rgg_grouped_gemm_wgrad(rgg._handle(0), X.data_ptr(), dY.data_ptr(), off.data_ptr(),
                                                  dW.data_ptr(), 1, 4096, 64, 72, 0,
                                                  torch.cuda.current_stream().cuda_stream, opt)
    assert s == rgg.RGG_ERR_INVALID_ARG


def test_neighbours_may_hold_anything():
    # each expert's sums stay finite while its neighbours' rows are Inf and NaN
    counts = [5, 16, 21, 64, 77, 3]
    X, dY, off = _case(counts, 136, 264, seed=11)
    for poisoned in range(len(counts)):
        Xp, dYp = X.clone(), dY.clone()
        a, b = int(off[poisoned]), int(off[poisoned + 1])
        Xp[a:b], dYp[a:b] = float("inf"), float("nan")
        got = _run(Xp, dYp, off)
        keep = [e for e in range(len(counts)) if e != poisoned]
        ref, mag = refs.wgrad(X, dY, off)
        limit = _limit(ref, mag, off, torch.bfloat16)
        refs.assert_close(got[keep], ref[keep], limit[keep], "dW beside expert %d" % poisoned)
        assert bool(got[poisoned].isnan().all())


def test_no_rows_at_all():
    X, dY = torch.empty(0, 64, dtype=torch.bfloat16), torch.empty(0, 72, dtype=torch.bfloat16)
    got = _run(X, dY, np.zeros(4, dtype=np.int32))
    assert got.shape == (3, 64, 72) and not bool(got.any())


def test_equal_calls_give_equal_bits():
    X, dY, off = _case(COUNTS, 264, 520, seed=12)
    first = _run(X, dY, off, dtype=torch.float32)
    for _ in range(3):
        assert torch.equal(_run(X, dY, off, dtype=torch.float32), first)


def test_graph_and_other_stream():
    X, dY, off = (t.cuda() if isinstance(t, torch.Tensor) else torch.from_numpy(t).cuda()
                  for t in _case(COUNTS, 264, 136, seed=13))
    want = rgg.rgg_grouped_gemm_wgrad(X, dY, off, check=True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    dW = torch.empty_like(want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        rgg.rgg_grouped_gemm_wgrad(X, dY, off, dW)
    dW.fill_(7)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(dW, want)


def test_producer_stall_is_reported():
    X, dY, off = _case([70, 5], 64, 64, seed=14)
    with pytest.raises(rgg.RggError) as ei:
        _run(X, dY, off, debug_flags=rgg.RGG_DEBUG_PRODUCER_STALL, timeout_ns=20_000_000)
    assert ei.value.status == rgg.RGG_ERR_DEVICE_TIMEOUT
    _check(X, dY, off, _run(X, dY, off))


def test_refusals():
    X, dY, off = (t.cuda() if isinstance(t, torch.Tensor) else torch.from_numpy(t).cuda()
                  for t in _case([5, 6], 64, 72, seed=15, lead=0, spare=0))
    wgrad = rgg.rgg_grouped_gemm_wgrad
    with pytest.raises(TypeError):
        wgrad(X.float(), dY, off)
    with pytest.raises(TypeError):
        wgrad(X, dY, off, dtype=torch.float16)
    with pytest.raises(TypeError):
        wgrad(X, dY, off.long())
    with pytest.raises(ValueError):
        wgrad(X[:10], dY, off)
    with pytest.raises(ValueError):
        wgrad(X, dY[:, :64], off)
    with pytest.raises(ValueError):
        wgrad(X, dY, off, accumulate=True)
    with pytest.raises(ValueError):
        wgrad(X, dY, off, torch.empty(2, 72, 64, dtype=torch.bfloat16, device="cuda"))
    for opts in (dict(bn=192), dict(stages=1), dict(max_ctas=1)):
        with pytest.raises(rgg.RggError) as ei:
            wgrad(X, dY, off, **opts)
        assert ei.value.status == rgg.RGG_ERR_INVALID_ARG
    with pytest.raises(rgg.RggError) as ei:
        wgrad(X[:, :60].contiguous(), dY, off)
    assert ei.value.status == rgg.RGG_ERR_INVALID_ARG
    dW = torch.full((2, 64, 72), 3.0, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(rgg.RggError) as ei:
        wgrad(X, dY, torch.tensor([0, 6, 5], dtype=torch.int32, device="cuda"), dW, check=True)
    assert ei.value.status == rgg.RGG_ERR_BAD_OFFSETS
    assert bool((dW == 3).all())
