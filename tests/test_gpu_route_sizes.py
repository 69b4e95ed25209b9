"""The router at 129 to 256 experts and at 9 to 16 choices, aligned and not, on a GB300."""
import pytest
import torch

import moe_refs as refs
import ragged_grouped_gemm_02_gb300 as rgg
from ragged_grouped_gemm_02_gb300 import _build

pytestmark = pytest.mark.gpu

TYPES = [torch.float32, torch.bfloat16, torch.float16]
RULES = [("softmax", True, 1.0), ("softmax", False, 2.5), ("sigmoid", True, 2.5), ("sigmoid", False, 1.0)]


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available(), "the gpu tests need a CUDA device"
    _build.build()


def _logits(T, E, dtype, seed, masked):
    gen = torch.Generator().manual_seed(seed)
    z = 2.0 * torch.randn(T, E, generator=gen)
    z[torch.rand(T, E, generator=gen) < masked] = float("-inf")
    return z.to(dtype)


def _place(t, shift):
    """t on the GPU, `shift` elements behind a 16-byte boundary."""
    out = torch.empty(t.numel() + shift, dtype=t.dtype, device="cuda")[shift:].view(t.shape)
    return out.copy_(t)


def _forward(logits, k, rule, shift=0):
    score, renormalize, scale = rule
    experts, weights = rgg.rgg_route_topk(_place(logits, shift), k, score=score, renormalize=renormalize, scale=scale)
    want, w, limit = refs.route(logits, k, *rule)
    assert torch.equal(experts.cpu().long(), want)
    error = (weights.cpu().double() - w).abs()
    assert bool((error <= limit).all()), float((error - limit).max())


def _gradient(logits, k, rule, shift=0):
    score, renormalize, scale = rule
    T, E = logits.shape
    dweights = torch.randn(T, k, generator=torch.Generator().manual_seed(1))
    experts = refs.route(logits, k, *rule)[0]
    out = _place(torch.full((T, E), 7.0, dtype=logits.dtype), shift)
    got = rgg.rgg_route_topk_backward(_place(logits, shift), experts.to(torch.int32).cuda(), dweights.cuda(), out, score=score,
                                      renormalize=renormalize, scale=scale, check=True)
    want, size = refs.route_gradient(logits, experts, dweights, *rule)
    # a row without an expert has weights of 0 whatever its logits (the reference's softmax makes NaN of it)
    want[logits.isneginf().all(1)] = 0.0
    # a weight is off by at most 12 units, and twice that by the logits' rounding; the sums over E and k by as many roundings
    limit = refs.rounding(want, logits.dtype) + size * (2 * 12 + 24 + 4 * E) * 2.0 ** -23
    error = (got.cpu().double() - want).abs()
    assert bool((error <= limit).all()), float((error - limit).max())


@pytest.mark.parametrize("rule", RULES)
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,E,k", [(33, 256, 8), (5, 256, 32), (9, 255, 8), (19, 200, 7), (11, 160, 12), (7, 129, 3)])
def test_up_to_256_experts(T, E, k, dtype, rule):
    for masked in (0.0, 0.3, 0.98):
        logits = _logits(T, E, dtype, T + E, masked)
        _forward(logits, k, rule)
        _gradient(logits, k, rule)


@pytest.mark.parametrize("rule", RULES)
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("E", [128, 256])
def test_logits_off_a_wide_boundary(E, dtype, rule):
    logits = _logits(21, E, dtype, E, 0.1)
    _forward(logits, 8, rule, shift=1)
    _gradient(logits, 8, rule, shift=1)


@pytest.mark.parametrize("rule", RULES)
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,E,k", [(1, 16, 16), (3, 20, 9), (17, 64, 12), (33, 48, 15), (64, 256, 16), (35, 300, 10), (2, 17, 17)])
def test_nine_to_sixteen_choices(T, E, k, dtype, rule):
    logits = _logits(T, E, dtype, T + k, 0.2)
    _forward(logits, k, rule)
    _gradient(logits, k, rule)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("E", [129, 250, 256])
def test_ties_go_to_the_lower_expert(E, dtype):
    logits = torch.randint(-2, 3, (40, E), generator=torch.Generator().manual_seed(5)).to(dtype)
    logits[0] = 0.0
    logits[1, ::2] = -0.0
    logits[1, 1::2] = 0.0  # minus zero equals zero
    _forward(logits, 20, ("softmax", True, 1.0))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("E", [8, 200, 256])
def test_nan_and_inf(E, dtype):
    logits = torch.zeros(4, E)
    logits[0, 5] = float("nan")
    logits[1, 2], logits[1, 6] = float("inf"), torch.finfo(dtype).max
    logits[2, 3], logits[2, 7] = float("inf"), float("nan")
    logits = logits.to(dtype).cuda()
    for score in ("softmax", "sigmoid"):
        experts, weights = rgg.rgg_route_topk(logits, 2, score=score)
        assert experts.tolist() == [[5, 0], [2, 6], [7, 3], [0, 1]]
        assert bool(weights[0].isnan().all()) and bool(weights[2].isnan().any())
        assert weights[3].tolist() == [0.5, 0.5]
        assert bool(weights[1].isnan().any()) == (score == "softmax")
        back = rgg.rgg_route_topk_backward(logits, experts, torch.ones(4, 2, device="cuda"), score=score, renormalize=False)
        assert bool(back[0].isnan().any()) and bool(back[2].isnan().any()) and bool(back[3].isfinite().all())
