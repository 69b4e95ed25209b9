"""The router's gradient where a weight is close to 1, on a GB300: against the formulas in 64 bits, written as sums of
differences, with limits relative to the terms of those sums (u = 2^-24 a rounding).

expf is off by at most 2 units in the last place (4 u) and by the rounding of its argument, |difference| u; a division and
a product by u each; a sum of n terms by n u of their magnitudes.
"""
import pytest
import torch

import ragged_grouped_gemm_02_gb300 as rgg
from ragged_grouped_gemm_02_gb300 import _build

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available(), "the gpu tests need a CUDA device"
    _build.build()


def _backward(z, experts, g, score, renormalize, scale):
    return rgg.rgg_route_topk_backward(z.cuda(), experts.to(torch.int32).cuda(), g.cuda(), score=score,
                                       renormalize=renormalize, scale=scale, check=True).cpu().double()


def _check(got, want, limit):
    worst = ((got - want).abs() / (limit + 2.0 ** -126)).max()
    assert bool(((got - want).abs() <= limit + 2.0 ** -126).all()), float(worst)


def test_sigmoid():
    gen = torch.Generator().manual_seed(0)
    z = torch.cat([torch.linspace(-60, 60, 240), 8 + 32 * torch.rand(240, generator=gen)]).view(60, 8)
    experts, g, scale = torch.topk(z, 3, dim=1).indices, torch.randn(60, 3, generator=gen), 2.5
    l = z.double().gather(1, experts)
    want = torch.zeros(60, 8, dtype=torch.float64).scatter(1, experts, scale * g.double() * torch.sigmoid(l) * torch.sigmoid(-l))
    # both sigmoids 6 u, four products
    _check(_backward(z, experts, g, "sigmoid", False, scale), want, want.abs() * 16 * U)
