"""rgg_clip_grad_norm refuses lists whose results would depend on the order in which memory is written, on a GB300."""
import math

import pytest
import torch

import ragged_grouped_gemm_02_gb300 as rgg
from ragged_grouped_gemm_02_gb300 import _build

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available(), "the gpu tests need a CUDA device"
    _build.build()


def _refused(grads, max_norm=1.0, **kw):
    before = [g.clone() for g in grads]
    with pytest.raises(rgg.RggError) as ei:
        rgg.rgg_clip_grad_norm(grads, max_norm, **kw)
    assert ei.value.status == rgg.RGG_ERR_INVALID_ARG
    assert all(torch.equal(g, b) for g, b in zip(grads, before))


@pytest.mark.parametrize("more", [0, 100])
def test_overlapping_tensors(more):
    flat = torch.ones(40000, device="cuda")
    other = [torch.ones(17, device="cuda") for _ in range(more)]
    _refused([flat, flat] + other)
    _refused(other + [flat[:20000], flat[19999:]])
    _refused([flat] + other + [flat[100:200]])
    _refused([flat[100:200]] + other + [flat])
    _refused([flat, flat.view(torch.bfloat16)[:8]] + other)
    # results over what is read elsewhere, or shifted over their own input
    outs = [torch.empty_like(t) for t in other]
    _refused([flat[:100], flat[200:300]] + other, out=[flat[200:300], torch.empty(100, device="cuda")] + outs)
    _refused([flat[:1000]] + other, out=[flat[1:1001]] + outs)
    _refused([flat[:100], flat[200:300]] + other, out=[torch.empty(100, device="cuda")] * 2 + outs)


@pytest.mark.parametrize("more", [0, 100])
def test_lists_that_share_no_written_memory(more):
    flat = torch.ones(30000, device="cuda")
    other = [torch.ones(10, device="cuda") for _ in range(more)]
    total = math.sqrt(30000 + 10 * more)
    # neighbouring views, and an empty tensor inside one
    norm = rgg.rgg_clip_grad_norm([flat[10000:], flat[5:5], flat[:10000]] + other, total / 2)
    assert abs(float(norm) - total) < 1e-4 * total and bool(((flat - 0.5).abs() < 1e-5).all())
    # an input read twice
    flat.fill_(1.0)
    outs = [torch.empty_like(flat) for _ in (0, 1)]
    norm = rgg.rgg_clip_grad_norm([flat, flat], 1.0, out=outs)
    assert abs(float(norm) - math.sqrt(60000)) < 1e-2 and torch.equal(*outs)
    # the norm alone writes no tensor
    assert abs(float(rgg.rgg_clip_grad_norm([flat, flat] + other, math.inf)) ** 2 - 60000 - sum(
        float(t.square().sum()) for t in other)) < 10
