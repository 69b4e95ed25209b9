"""The 64-bit gradient references against central differences of the forward product (CPU)."""
import torch

import expert_refs as refs


def _layer(seed=0):
    gen = torch.Generator().manual_seed(seed)
    counts, K, N = [3, 0, 4, 1], 8, 8
    off, M = refs.ragged(counts)
    X = refs.normal(gen, M, K)
    W13 = refs.normal(gen, len(counts), K, 2 * N)
    dH = refs.normal(gen, M, N)
    return X.double(), W13.double(), off, dH.double()


def _difference(f, x, at, h=1e-5):
    up, down = x.clone(), x.clone()
    up[at] += h
    down[at] -= h
    return (f(up) - f(down)) / (2 * h)


def test_gradients_agree_with_differences():
    X, W13, off, dH = _layer()
    loss = lambda x, w: float((refs.swiglu(refs.gate_up(x, w, off)[0]) * dH).sum())  # noqa: E731
    dGU, _ = refs.swiglu_backward(refs.gate_up(X, W13, off)[0], dH)
    dX = refs.dgrad(dGU, W13, off)[0]
    dW = refs.wgrad(X, dGU, off)[0]
    for at in [(0, 0), (2, 7), (3, 1), (6, 4), (7, 3)]:
        assert abs(_difference(lambda x: loss(x, W13), X, at) - float(dX[at])) < 1e-6
    for at in [(0, 0, 0), (0, 3, 15), (2, 5, 9), (3, 7, 2)]:
        assert abs(_difference(lambda w: loss(X, w), W13, at) - float(dW[at])) < 1e-6
    assert not bool(dW[1].any()), "an expert without rows has a zero gradient"
