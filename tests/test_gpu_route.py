"""The router against its definition in 64 bits, on a GB300."""
import pytest
import torch

import moe_refs as refs
import ragged_grouped_gemm_02_gb300 as rgg
from ragged_grouped_gemm_02_gb300 import _build

pytestmark = pytest.mark.gpu

TYPES = [torch.float32, torch.bfloat16, torch.float16]
RULES = [("softmax", True, 1.0), ("softmax", False, 2.5), ("sigmoid", True, 2.5), ("sigmoid", False, 1.0)]
SIZES = [(1, 1, 1), (1, 2, 2), (7, 5, 3), (33, 32, 8), (64, 64, 4), (65, 100, 6), (40, 128, 8), (19, 257, 7), (9, 513, 32),
         (5, 1024, 8), (3, 1025, 2), (2, 4096, 32)]


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available(), "the gpu tests need a CUDA device"
    _build.build()


def _logits(T, E, dtype, seed, masked=0.0):
    gen = torch.Generator().manual_seed(seed)
    z = 2.0 * torch.randn(T, E, generator=gen)
    z[torch.rand(T, E, generator=gen) < masked] = float("-inf")
    return z.to(dtype)


def _check(logits, k, rule):
    score, renormalize, scale = rule
    experts, weights = rgg.rgg_route_topk(logits.cuda(), k, score=score, renormalize=renormalize, scale=scale)
    want, w, limit = refs.route(logits, k, *rule)
    assert torch.equal(experts.cpu().long(), want)
    assert bool(((weights.cpu().double() - w).abs() <= limit).all()), float((weights.cpu().double() - w).abs().max())
    return experts, weights


@pytest.mark.parametrize("rule", RULES)
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,E,k", SIZES)
def test_choices_and_weights(T, E, k, dtype, rule):
    _check(_logits(T, E, dtype, seed=T + E), k, rule)


@pytest.mark.parametrize("rule", RULES)
@pytest.mark.parametrize("dtype", TYPES)
def test_masked_experts(dtype, rule):
    # from none to all experts masked, a row of nothing, a row of one
    logits = _logits(64, 40, dtype, seed=3, masked=0.9)
    logits[0] = float("-inf")
    logits[1] = float("-inf")
    logits[1, 39] = -3.0
    logits[2] = torch.finfo(dtype).min  # the type's lowest value is no mask
    _check(logits, 8, rule)


@pytest.mark.parametrize("dtype", TYPES)
def test_ties_go_to_the_lower_expert(dtype):
    gen = torch.Generator().manual_seed(5)
    logits = torch.randint(-2, 3, (50, 300), generator=gen).to(dtype)
    logits[0] = 0.0
    logits[1, ::2] = -0.0
    logits[1, 1::2] = 0.0  # minus zero equals zero
    _check(logits, 9, ("softmax", True, 1.0))


@pytest.mark.parametrize("dtype", TYPES)
def test_extreme_logits(dtype):
    big = torch.finfo(dtype).max
    logits = torch.tensor([[big, -big, 0.0, 1.0], [-big, -big, -big, -big], [-200.0, -300.0, -250.0, -1e4],
                           [100.0, 99.0, 98.0, -big], [1e-6, -1e-6, 0.0, 2e-6]]).to(dtype)
    for rule in RULES:
        _check(logits, 3, rule)


def test_nan_and_inf_show_in_the_weights():
    logits = torch.zeros(3, 8, device="cuda")
    logits[0, 5] = float("nan")
    logits[1, 2] = float("inf")
    experts, weights = rgg.rgg_route_topk(logits, 2)
    assert experts[0, 0] == 5 and bool(weights[0].isnan().all())
    assert experts[1, 0] == 2 and bool(weights[1].isnan().any())
    assert experts[2].tolist() == [0, 1] and weights[2].tolist() == [0.5, 0.5]
    back = rgg.rgg_route_topk_backward(logits, experts, torch.ones(3, 2, device="cuda"), renormalize=False)
    assert bool(back[0].isnan().any()) and bool(back[2].isfinite().all())


@pytest.mark.parametrize("rule", RULES)
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,E,k", SIZES)
def test_gradient(T, E, k, dtype, rule):
    score, renormalize, scale = rule
    logits = _logits(T, E, dtype, seed=T + 7 * E, masked=0.2)
    dweights = torch.randn(T, k, generator=torch.Generator().manual_seed(1))
    experts = refs.route(logits, k, *rule)[0]
    out = torch.full((T, E), 7.0, dtype=dtype, device="cuda")
    got = rgg.rgg_route_topk_backward(logits.cuda(), experts.to(torch.int32).cuda(), dweights.cuda(), out, score=score,
                                      renormalize=renormalize, scale=scale, check=True)
    want, size = refs.route_gradient(logits, experts, dweights, *rule)
    # the terms' weights are off by at most that many units (see refs.route), the sums over E and k by as many roundings
    limit = refs.rounding(want, dtype) + size * (2 * 12 + 24 + 4 * E) * 2.0 ** -23
    error = (got.cpu().double() - want).abs()
    assert bool((error <= limit).all()), float((error - limit).max())


def test_gradient_against_differences():
    # central differences of the kernel's own weights: step 2^-6, curvature at most 1 in weights of at most 1
    logits = _logits(16, 12, torch.float32, seed=9).cuda()
    g = torch.randn(16, 3, generator=torch.Generator().manual_seed(2)).cuda()
    for score, renormalize, scale in RULES:
        rule = {"score": score, "renormalize": renormalize, "scale": scale}
        experts, _ = rgg.rgg_route_topk(logits, 3, **rule)
        got = rgg.rgg_route_topk_backward(logits, experts, g, **rule)
        step = 2.0 ** -6
        for e in range(12):
            sides = []
            for sign in (1, -1):
                moved = logits.clone()
                moved[:, e] += sign * step
                other, w = rgg.rgg_route_topk(moved, 3, **rule)
                same = (other == experts).all(1)
                sides.append(((w * g).sum(1), same))
            diff = (sides[0][0] - sides[1][0]) / (2 * step)
            ok = sides[0][1] & sides[1][1]
            # third derivative of a weight at most 1: step^2 / 6 of sum |g| scale; fp32 noise 2^-20 / step
            limit = g.abs().sum(1) * scale * (step ** 2 + 2.0 ** -20 / step)
            assert bool(((diff - got[:, e]).abs() <= limit)[ok].all())


def test_an_expert_named_twice_gets_both_gradients():
    logits = _logits(4, 6, torch.float32, seed=2).cuda()
    experts = torch.tensor([[1, 1], [2, 5], [-1, 3], [0, 0]], dtype=torch.int32)
    g = torch.tensor([[1.0, 2.0], [3.0, 4.0], [5.0, 6.0], [-1.0, 1.0]])
    for rule in RULES:
        score, renormalize, scale = rule
        got = rgg.rgg_route_topk_backward(logits, experts.cuda(), g.cuda(), score=score, renormalize=renormalize, scale=scale)
        want, size = refs.route_gradient(logits.cpu(), experts.long(), g, *rule)
        assert bool(((got.cpu().double() - want).abs() <= size * 2.0 ** -16).all())


def test_experts_out_of_range_are_reported():
    logits = torch.randn(4, 6, device="cuda")
    experts = torch.tensor([[1, 6], [2, 5], [-7, 3], [0, 2 ** 31 - 1]], dtype=torch.int32, device="cuda")
    g = torch.ones(4, 2, device="cuda")
    with pytest.raises(rgg.RggError, match="BAD_ROW_INDEX"):
        rgg.rgg_route_topk_backward(logits, experts, g, check=True)
    none = torch.where(experts >= 6, -1, experts)
    a = rgg.rgg_route_topk_backward(logits, experts, g)
    assert rgg.rgg_query_status() == rgg.RGG_ERR_BAD_ROW_INDEX
    assert torch.equal(a, rgg.rgg_route_topk_backward(logits, none, g, check=True))


def test_no_tokens():
    logits = torch.empty(0, 8, device="cuda")
    experts, weights = rgg.rgg_route_topk(logits, 2)
    assert experts.shape == weights.shape == (0, 2)
    assert rgg.rgg_route_topk_backward(logits, experts, weights).shape == (0, 8)


def test_many_tokens():
    # past what one wave of blocks holds; the same rows give the same results
    logits = _logits(64, 96, torch.bfloat16, seed=8).cuda()
    a = rgg.rgg_route_topk(logits, 5)
    b = rgg.rgg_route_topk(logits.repeat(700, 1), 5)
    for x, y in zip(a, b):
        assert torch.equal(x.repeat(700, 1), y)
