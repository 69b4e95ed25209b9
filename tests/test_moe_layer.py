"""moe_layer.py's autograd functions on the CPU, plain sums standing in for the kernels: what they promise about
derivatives does not depend on them."""
import pytest
import torch

import moe_refs as refs
from ragged_grouped_gemm_02_gb300 import moe_layer


def _route(logits, k, score, renormalize, scale):
    experts = refs.route(logits, k, score, renormalize, scale)[0]
    return experts, refs.weights_of(logits, experts, score, renormalize, scale)


def _route_backward(logits, experts, dweights, score, renormalize, scale):
    return refs.route_gradient(logits, experts, dweights, score, renormalize, scale)[0]


def _dispatch(X, position):
    out = X.new_zeros(position.numel(), X.shape[1])
    for j in range(position.shape[1]):
        kept = position[:, j] >= 0
        out[position[kept, j].long()] = X[kept]
    return out


def _combine(Y, position, weights=None):
    kept = (position >= 0).to(Y.dtype)
    w = kept if weights is None else weights * kept
    return (Y[position.long().clamp(min=0)] * w.unsqueeze(-1)).sum(1)


def _combine_backward(dout, Y, position, weights, dY, dweights):
    kept = position >= 0
    if dY is not False:
        dY[position[kept].long()] = (weights.unsqueeze(-1) * dout.unsqueeze(1))[kept]
    dw = (Y[position.long().clamp(min=0)] * dout.unsqueeze(1)).sum(-1) * kept
    return None if dY is False else dY, None if dweights is False else dw


@pytest.fixture
def plain(monkeypatch):
    for name, fn in (("rgg_route_topk", _route), ("rgg_route_topk_backward", _route_backward), ("rgg_dispatch", _dispatch),
                     ("rgg_combine", _combine), ("rgg_combine_backward", _combine_backward)):
        monkeypatch.setattr(moe_layer, name, fn)


def _inputs():
    gen = torch.Generator().manual_seed(0)
    experts = refs.choices(gen, 5, 2, 4, 0.2)
    position = refs.sort(experts, 4)[2]
    X, w = (torch.randn(5, n, generator=gen, dtype=torch.float64).requires_grad_() for n in (3, 2))
    Y = torch.randn(10, 3, generator=gen, dtype=torch.float64).requires_grad_()
    logits = torch.randn(5, 4, generator=gen, dtype=torch.float64).requires_grad_()
    return X, Y, w, logits, position


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [True, False])
def test_route_gradient(plain, score, renormalize):
    logits = _inputs()[3]
    rule = {"score": score, "renormalize": renormalize, "scale": 1.5}
    assert torch.autograd.gradcheck(lambda z: moe_layer.route_topk(z, 2, **rule)[1], logits)
    assert not moe_layer.route_topk(logits, 2, **rule)[0].requires_grad


def test_dispatch_and_combine_gradients(plain):
    X, Y, w, _, position = _inputs()
    assert torch.autograd.gradcheck(lambda x: moe_layer.dispatch(x, position), X)
    assert torch.autograd.gradcheck(lambda y, v: moe_layer.combine(y, position, v), (Y, w))
    assert torch.autograd.gradcheck(lambda y: moe_layer.combine(y, position, w.detach()), Y)
    assert torch.autograd.gradcheck(lambda v: moe_layer.combine(Y.detach(), position, v), w)


@pytest.mark.parametrize("which", ["route", "dispatch", "combine Y", "combine w"])
@pytest.mark.parametrize("linear", [True, False])
def test_second_derivatives_are_refused(plain, which, linear):
    # also where the incoming gradient is a constant: the results depend on the saved tensors all the same
    X, Y, w, logits, position = _inputs()
    out = (moe_layer.route_topk(logits, 2)[1] if which == "route" else moe_layer.dispatch(X, position)
           if which == "dispatch" else moe_layer.combine(Y, position, w))
    by = {"route": logits, "dispatch": X, "combine Y": Y, "combine w": w}[which]
    loss = (out if linear else out.square()).sum()
    g, = torch.autograd.grad(loss, by, create_graph=True)
    with pytest.raises(RuntimeError, match="first derivatives only"):
        (loss + g.square().sum()).backward()
