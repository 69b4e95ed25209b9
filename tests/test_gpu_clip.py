"""rgg_clip_grad_norm against 64-bit norms, on a GB300.

The norm: fp32 sums of at most 128 squares, so relative error at most 128 * 2^-24 of the sum of squares, half of
that in its root, and one rounding to fp32: 64 * 2^-24 + 2^-24 < 2^-17.  Outputs: the factor is rounded to fp32 and the
product is rounded once to the type: 2^-17 plus half a unit (2^-23 fp32, 2^-8 bf16, 2^-10 fp16, as bounds)."""
import math

import pytest
import torch

import ragged_grouped_gemm_02_gb300 as rgg
from ragged_grouped_gemm_02_gb300 import _build

pytestmark = pytest.mark.gpu

NORM_RTOL = 2.0 ** -17
UNIT = {torch.float32: 2.0 ** -23, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -10}
TINY = {torch.float32: 2.0 ** -149, torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -24}


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available(), "the gpu tests need a CUDA device"
    _build.build()


def _grads(sizes, dtypes, seed=0, std=1.0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return [(torch.randn(n, generator=gen, device="cuda") * std).to(dtypes[i % len(dtypes)])
            for i, n in enumerate(sizes)]


def _norm64(grads):
    return math.sqrt(sum(float(g.double().square().sum()) for g in grads))


def _check(grads, max_norm, norm, got):
    want = _norm64(grads)
    assert abs(float(norm) - want) <= NORM_RTOL * want
    scale = min(1.0, max_norm / (want + 1e-6))
    for g, o in zip(grads, got):
        ref = g.double() * scale
        err = (o.double() - ref).abs()
        limit = (NORM_RTOL + UNIT[g.dtype]) * ref.abs() + TINY[g.dtype]
        assert o.dtype == g.dtype and bool((err <= limit).all()), (g.numel(), g.dtype, float((err - limit).max()))


SIZES = [1, 0, 7, 8, 9, 255, 4096, 16383, 16384, 16385, 32767, 32768, 32769, 100003]


@pytest.mark.parametrize("dtypes", [[torch.bfloat16], [torch.float32], [torch.float16],
                                    [torch.bfloat16, torch.float32, torch.float16]])
@pytest.mark.parametrize("max_norm", [0.0, 1.0, 1e9, math.inf])
def test_lists(dtypes, max_norm):
    grads = _grads(SIZES, dtypes, seed=len(dtypes))
    out = [torch.full_like(g, 7) for g in grads]
    _check(grads, max_norm, rgg.rgg_clip_grad_norm(grads, max_norm, out=out), out)
    same = [g.clone() for g in grads]
    _check(grads, max_norm, rgg.rgg_clip_grad_norm(same, max_norm), same)


@pytest.mark.parametrize("count", [1, 63, 64, 65, 959, 960, 961, 2500])
def test_many_tensors(count):
    grads = _grads([17 + (i * 37) % 5000 for i in range(count)], [torch.bfloat16, torch.float32], seed=count)
    out = [torch.empty_like(g) for g in grads]
    _check(grads, 2.0, rgg.rgg_clip_grad_norm(grads, 2.0, out=out), out)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32, torch.float16])
@pytest.mark.parametrize("shift_in,shift_out", [(1, 1), (3, 0), (0, 5), (2, 7), (7, 7)])
def test_any_alignment(dtype, shift_in, shift_out):
    n = 70001
    flat = _grads([n + 16], [dtype], seed=shift_in)[0]
    target = torch.full((n + 16,), 7, dtype=dtype, device="cuda")
    g, o = flat[shift_in:shift_in + n], target[shift_out:shift_out + n]
    _check([g], 1.0, rgg.rgg_clip_grad_norm([g], 1.0, out=[o]), [o])
    assert bool((target[:shift_out] == 7).all()) and bool((target[shift_out + n:] == 7).all())


@pytest.mark.parametrize("std", [1e-30, 1e-22, 1e-16, 1e16, 1e22, 1e30])
def test_squares_outside_fp32(std):
    grads = _grads([5000, 40001], [torch.float32, torch.bfloat16], seed=3, std=std)
    out = [torch.empty_like(g) for g in grads]
    max_norm = 1e-3 * std
    norm = rgg.rgg_clip_grad_norm(grads, max_norm, out=out)
    want = _norm64(grads)
    assert abs(float(norm) - want) <= NORM_RTOL * want
    _check(grads, max_norm, norm, out)


def test_mixed_magnitudes():
    # one large tensor beside many tiny ones, and zeros
    grads = [torch.full((100000,), 1e-25, device="cuda"), torch.full((3,), 1e25, device="cuda"),
             torch.zeros(50000, device="cuda")]
    norm = rgg.rgg_clip_grad_norm(grads, math.inf)
    assert abs(float(norm) - 3 ** 0.5 * 1e25) <= NORM_RTOL * 1e26


def test_all_zero():
    grads = [torch.zeros(40000, dtype=torch.bfloat16, device="cuda")]
    assert float(rgg.rgg_clip_grad_norm(grads, 1.0)) == 0.0 and not bool(grads[0].any())


@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
def test_a_norm_that_is_not_finite(bad):
    grads = _grads([70000, 33], [torch.bfloat16, torch.float32], seed=4)
    grads[0][12345] = bad
    out = [torch.zeros_like(g) for g in grads]
    norm = float(rgg.rgg_clip_grad_norm(grads, 1.0, out=out))
    assert math.isnan(norm) if math.isnan(bad) else norm == math.inf
    for g, o in zip(grads, out):
        bits = torch.int16 if g.dtype == torch.bfloat16 else torch.int32
        assert torch.equal(g.view(bits), o.view(bits))


def test_equal_calls_give_equal_bits():
    grads = _grads([3000000, 70001], [torch.bfloat16, torch.float32], seed=5)
    first = rgg.rgg_clip_grad_norm(grads, math.inf)
    for _ in range(4):
        assert torch.equal(rgg.rgg_clip_grad_norm(grads, math.inf), first)


def test_graph_and_other_stream():
    grads = _grads([100000, 500], [torch.bfloat16, torch.float32], seed=6)
    out = [torch.empty_like(g) for g in grads]
    want = rgg.rgg_clip_grad_norm(grads, 1.0, out=out).clone()
    kept = [o.clone() for o in out]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    norm = rgg.rgg_clip_grad_norm(grads, 1.0, out=out, stream=side)
    side.synchronize()
    assert torch.equal(norm, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        norm = rgg.rgg_clip_grad_norm(grads, 1.0, out=out)
    for o in out:
        o.fill_(7)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(norm, want) and all(torch.equal(a, b) for a, b in zip(out, kept))


def test_refusals():
    g = torch.ones(8, 8, device="cuda")
    for call in (lambda: rgg.rgg_clip_grad_norm([], 1.0), lambda: rgg.rgg_clip_grad_norm([g], -1.0),
                 lambda: rgg.rgg_clip_grad_norm([g], math.nan), lambda: rgg.rgg_clip_grad_norm([g.t()[1:]], 1.0),
                 lambda: rgg.rgg_clip_grad_norm([g], 1.0, out=[]),
                 lambda: rgg.rgg_clip_grad_norm([g], 1.0, out=[torch.ones(8, device="cuda")]),
                 lambda: rgg.rgg_clip_grad_norm([g.cpu()], 1.0), lambda: rgg.rgg_clip_grad_norm([g, g.cpu()], 1.0)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: rgg.rgg_clip_grad_norm([g.double()], 1.0),
                 lambda: rgg.rgg_clip_grad_norm([g], 1.0, out=[g.bfloat16()])):
        with pytest.raises(TypeError):
            call()
    assert bool((g == 1).all())
