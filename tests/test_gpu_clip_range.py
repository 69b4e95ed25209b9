"""rgg_clip_grad_norm at the ends of fp32's range, on a GB300: norms that fp32 does not hold, and factors below its
normal range.  Bounds as in test_gpu_clip.py: the norm is right to 2^-17, results to that and half a unit."""
import math

import pytest
import torch

import ragged_grouped_gemm_02_gb300 as rgg
from ragged_grouped_gemm_02_gb300 import _build

pytestmark = pytest.mark.gpu

NORM_RTOL = 2.0 ** -17


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available(), "the gpu tests need a CUDA device"
    _build.build()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n", [4, 100001])
def test_finite_values_whose_norm_fp32_does_not_hold(dtype, n):
    # the caller is told Inf, so the values must come unscaled, as for any norm that is not finite
    grads = [torch.full((n,), 2e38, dtype=dtype, device="cuda"), torch.ones(33, device="cuda")]
    kept = [g.clone() for g in grads]
    out = [torch.zeros_like(g) for g in grads]
    assert float(rgg.rgg_clip_grad_norm(grads, 1.0, out=out)) == math.inf
    assert all(torch.equal(o, k) for o, k in zip(out, kept))
    assert float(rgg.rgg_clip_grad_norm(grads, 1.0)) == math.inf
    assert all(torch.equal(g, k) for g, k in zip(grads, kept))


def test_the_largest_norm_that_is_finite():
    grads = [torch.full((4,), 1.7e38, device="cuda")]  # the norm is 3.4e38
    norm = float(rgg.rgg_clip_grad_norm(grads, 3.4e38 / 4))
    assert abs(norm - 3.4e38) <= NORM_RTOL * 3.4e38
    assert bool(((grads[0] - 1.7e38 / 4).abs() <= 2 * NORM_RTOL * 1.7e38 / 4).all())


@pytest.mark.parametrize("dtype,unit,tiny", [(torch.float32, 2.0 ** -23, 2.0 ** -149),
                                             (torch.bfloat16, 2.0 ** -8, 2.0 ** -133)])
@pytest.mark.parametrize("max_norm", [1e-38, 1e-20, 1e-3, 0.3, 1.0, 30.0])
@pytest.mark.parametrize("shift", [0, 1])
def test_factors_below_the_normal_range(dtype, unit, tiny, max_norm, shift):
    # max_norm over a norm of 1e38 is subnormal in fp32, or less: the results have all their bits all the same
    gen = torch.Generator(device="cuda").manual_seed(3)
    flat = (torch.randn(5002, generator=gen, device="cuda") * 1e36).to(dtype)
    flat[::7] *= 1e-30
    grads = [flat[:5001]]
    out = [torch.empty(5002, dtype=dtype, device="cuda")[shift:5001 + shift]]
    norm = rgg.rgg_clip_grad_norm(grads, max_norm, out=out)
    want = math.sqrt(float(grads[0].double().square().sum()))
    assert abs(float(norm) - want) <= NORM_RTOL * want
    ref = grads[0].double() * (torch.tensor(max_norm).double().item() / (want + 1e-6))
    err = (out[0].double() - ref).abs()
    assert bool((err <= (NORM_RTOL + unit) * ref.abs() + tiny).all())
