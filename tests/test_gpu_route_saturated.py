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
EPS = 1e-20


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


def _choices(z, k, shuffled, gen):
    """The k largest of each row, in their order or in another."""
    experts = torch.topk(z, k, dim=1).indices
    return experts.gather(1, torch.rand(experts.shape, generator=gen).argsort(1)) if shuffled else experts


def test_sigmoid():
    gen = torch.Generator().manual_seed(0)
    z = torch.cat([torch.linspace(-60, 60, 240), 8 + 32 * torch.rand(240, generator=gen)]).view(60, 8)
    experts, g, scale = torch.topk(z, 3, dim=1).indices, torch.randn(60, 3, generator=gen), 2.5
    l = z.double().gather(1, experts)
    want = torch.zeros(60, 8, dtype=torch.float64).scatter(1, experts, scale * g.double() * torch.sigmoid(l) * torch.sigmoid(-l))
    # both sigmoids 6 u, four products
    _check(_backward(z, experts, g, "sigmoid", False, scale), want, want.abs() * 16 * U)


def _pairs(w, g):
    """For each choice i: sum over j of w_j (g_i - g_j), and of the magnitudes."""
    d = g.unsqueeze(2) - g.unsqueeze(1)
    return (w.unsqueeze(1) * d).sum(2), (w.unsqueeze(1) * d.abs()).sum(2)


@pytest.mark.parametrize("shuffled", [False, True])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("k", [1, 2, 3, 8, 16, 20])
def test_renormalized(k, score, shuffled):
    gen = torch.Generator().manual_seed(k)
    T, E, scale = 41, 24, 1.5
    z = torch.randn(T, E, generator=gen)
    z[:, 5] += torch.linspace(0, 30, T)  # one expert takes more and more of the weight
    z = z[:, torch.randperm(E, generator=gen)] if score == "softmax" else z - 12
    experts, g = _choices(z, k, shuffled, gen), torch.randn(T, k, generator=gen)
    l = z.double().gather(1, experts)
    if score == "softmax":
        w, rest, factor = torch.softmax(l, 1), 0.0, torch.softmax(l, 1)
    else:
        s = torch.sigmoid(l)
        total = s.sum(1, keepdim=True) + EPS
        w, rest, factor = s / total, EPS / total, s * torch.sigmoid(-l) / total
    diff, size = _pairs(w, g.double())
    want = scale * factor * (diff + rest * g.double())
    # with r the largest weight's choice, (g_i - g_r) - sum w_j (g_j - g_r): |g_i - g_r| <= k size_i as w_r >= 1 / k, so the
    # terms sum to at most (2 k + 1) size_i; each is off by the weights' 24 u, their arguments' and the sums' k u
    spread = l.amax(1, keepdim=True) - l.amin(1, keepdim=True)
    units = (24 + 2 * k + 2 * spread) * U
    limit = scale * factor * ((2 * k + 1) * size + 2 * rest * g.double().abs()) * units
    got = _backward(z, experts, g, score, True, scale)
    _check(got.gather(1, experts), want, limit)
    assert bool((got.scatter(1, experts, 0.0) == 0).all())


@pytest.mark.parametrize("E", [6, 40, 128, 200, 256, 300])
def test_softmax_over_all(E):
    gen = torch.Generator().manual_seed(E)
    T, k, scale = 31, 4, 2.5
    z = torch.randn(T, E, generator=gen)
    z[:, 3] += torch.linspace(8, 30, T)  # more than half of the weight in each row
    experts, g = _choices(z, k, True, gen), torch.randn(T, k, generator=gen).double()
    s = torch.softmax(z.double(), 1)
    all_g = torch.zeros(T, E, dtype=torch.float64).scatter(1, experts, g)
    want = scale * s * _pairs(s, all_g)[0]
    assert bool((s[:, 3] > 0.5).all()) and bool((experts == 3).any(1).all())
    # with r the largest: (g_i - g_r) - (sum over the other choices of s_j g_j - g_r sum over j != r of s_j)
    g_r, others = all_g[:, 3:4], s.clone()
    others[:, 3] = 0.0
    terms = (all_g - g_r).abs() + (others * (all_g.abs() + g_r.abs())).sum(1, keepdim=True)
    plain = (s * all_g.abs()).sum(1, keepdim=True).expand(T, E)  # experts of no choice
    chosen = torch.zeros(T, E, dtype=torch.bool).scatter(1, experts, True)
    spread = z.double().amax(1, keepdim=True) - z.double().amin(1, keepdim=True)
    limit = scale * s * torch.where(chosen, terms, plain) * (24 + 2 * E + 2 * spread) * U
    _check(_backward(z, experts, g.float(), "softmax", False, scale), want, limit)
