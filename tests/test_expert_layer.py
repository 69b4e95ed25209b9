"""expert_layer.py's autograd function on the CPU, plain products standing in for the kernels: what it promises about
derivatives does not depend on them."""
import pytest
import torch

from ragged_grouped_gemm_02_gb300 import expert_layer


def _spread(off):
    return [(int(a), int(b)) for a, b in zip(off[:-1], off[1:])]


def _product(X, W, off, out=None):
    out = X.new_zeros(X.shape[0], W.shape[2]) if out is None else out
    for e, (a, b) in enumerate(_spread(off)):
        out[a:b] = X[a:b] @ W[e]
    return out


def _swiglu(X, W13, off):
    g, u = _product(X, W13, off).chunk(2, 1)
    return torch.nn.functional.silu(g) * u


def _swiglu_backward(X, W13, off, dH, H=None):
    g, u = _product(X, W13, off).chunk(2, 1)
    s = torch.sigmoid(g)
    return torch.cat([dH * u * s * (1 + g * (1 - s)), dH * g * s], 1), None if H is False else g * s * u


@pytest.fixture
def plain(monkeypatch):
    for name, fn in (("rgg_grouped_gemm", _product), ("rgg_grouped_gemm_swiglu", _swiglu),
                     ("rgg_grouped_gemm_dgrad", lambda dY, W, off, dX=None: _product(dY, W.transpose(1, 2), off, dX)),
                     ("rgg_grouped_gemm_swiglu_backward", _swiglu_backward),
                     ("rgg_grouped_gemm_wgrad", lambda X, dY, off: torch.stack(
                         [X[a:b].t() @ dY[a:b] for a, b in _spread(off)]))):
        monkeypatch.setattr(expert_layer, name, fn)


def _layer():
    gen = torch.Generator().manual_seed(0)
    return [torch.randn(*s, generator=gen, dtype=torch.float64).requires_grad_()
            for s in ((6, 4), (3, 4, 10), (3, 5, 4))], torch.tensor([0, 2, 2, 6])


def test_first_derivatives(plain):
    leaves, off = _layer()
    assert torch.autograd.gradcheck(lambda *t: expert_layer.expert_ffn(*t, off), leaves)


@pytest.mark.parametrize("by", [0, 1, 2])
def test_second_derivatives_are_refused(plain, by):
    # a penalty on the gradient must not come back as if it did not depend on the inputs
    leaves, off = _layer()
    loss = expert_layer.expert_ffn(*leaves, off).square().sum()
    g, = torch.autograd.grad(loss, leaves[by], create_graph=True)
    assert g.requires_grad
    with pytest.raises(RuntimeError, match="once_differentiable"):
        (loss + g.square().sum()).backward()
