"""64-bit references of the expert layer's backward products, shared by the GPU tests.

Error bounds.  The kernels sum exact products of bf16 values in fp32 and round
once to bf16.  Over n products whose magnitudes sum to S, an fp32 sum that
truncates at every step is off by at most n * 2^-23 * S; rounding to bf16 adds
half a unit in the last place, 2^-9 of the value (2^-8 leaves room for the sum's
own error moving it over a rounding boundary).  Values below bf16's normal range
round in units of 2^-133.
"""
import numpy as np
import torch

ROUND_BF16 = 2.0 ** -8
TINY = 2.0 ** -133


def spread(offsets):
    return [(int(a), int(b)) for a, b in zip(offsets[:-1], offsets[1:])]


def bound(ref, n, magnitude):
    """The largest error an output may have: ref and sum of |products| (fp64), n products."""
    return ROUND_BF16 * ref.abs() + n * 2.0 ** -23 * magnitude + TINY


def dgrad(dY, W, offsets):
    """dX and its error bound, fp64 [M_tot, K]; NaN on rows of no expert."""
    M, (E, K, N) = dY.shape[0], W.shape
    ref = torch.full((M, K), float("nan"), dtype=torch.float64)
    mag = torch.zeros(M, K, dtype=torch.float64)
    for e, (a, b) in enumerate(spread(offsets)):
        w = W[e].double()
        ref[a:b] = dY[a:b].double() @ w.t()
        mag[a:b] = dY[a:b].double().abs() @ w.abs().t()
    return ref, bound(ref, N, mag)


def wgrad(X, dY, offsets):
    """dW, and the sums of |products|, fp64 [E, K, N]."""
    parts = [(X[a:b].double().t() @ dY[a:b].double(), X[a:b].double().abs().t() @ dY[a:b].double().abs())
             for a, b in spread(offsets)]
    return torch.stack([p[0] for p in parts]), torch.stack([p[1] for p in parts])


def gate_up(X, W13, offsets):
    """[gate | up] and the sums of |products|, fp64 [M_tot, 2N]; NaN on rows of no expert."""
    M, (E, K, N2) = X.shape[0], W13.shape
    gu = torch.full((M, N2), float("nan"), dtype=torch.float64)
    mag = torch.zeros(M, N2, dtype=torch.float64)
    for e, (a, b) in enumerate(spread(offsets)):
        gu[a:b] = X[a:b].double() @ W13[e].double()
        mag[a:b] = X[a:b].double().abs() @ W13[e].double().abs()
    return gu, mag


def swiglu(gu):
    N = gu.shape[1] // 2
    g, u = gu[:, :N], gu[:, N:]
    return g * torch.sigmoid(g) * u


def swiglu_backward(gu, dH):
    """dGU and H from the gate-up product (all fp64)."""
    N = gu.shape[1] // 2
    g, u = gu[:, :N], gu[:, N:]
    s = torch.sigmoid(g)
    return torch.cat([dH * u * s * (1 + g * (1 - s)), dH * g * s], 1), g * s * u


def swiglu_backward_bound(gu, mag, dH, K):
    """Error bounds of dGU and H.  The accumulators are off by eps = K * 2^-23 * mag each; |silu'| <= 1.1,
    |silu''| <= 0.5, |silu(g)| <= |g|; the fp32 evaluation of the formulas adds at most 2^-18 of the terms'
    magnitudes (a dozen operations, the exponential's argument error growing with |g| <= 64)."""
    N = gu.shape[1] // 2
    ref, act = swiglu_backward(gu, dH)
    eps = K * 2.0 ** -23 * mag
    g, u, eg, eu, d = gu[:, :N].abs(), gu[:, N:].abs(), eps[:, :N], eps[:, N:], dH.abs()
    bg = d * (1.1 * eu + 0.5 * u * eg) + 2.0 ** -18 * d * u * (1 + g)
    bu = d * 1.1 * eg + 2.0 ** -18 * d * g
    bh = g * eu + 1.1 * u * eg + 2.0 ** -18 * g * u
    return ROUND_BF16 * ref.abs() + torch.cat([bg, bu], 1) + TINY, ROUND_BF16 * act.abs() + bh + TINY


def ragged(counts, lead=0, spare=0):
    """Offsets of the counts, the first expert starting at row `lead`; and the row total with `spare` rows after."""
    off = lead + np.concatenate([[0], np.cumsum(counts)])
    return off.astype(np.int32), int(off[-1]) + spare


def normal(gen, *shape, std=1.0):
    return (torch.randn(shape, generator=gen) * std).to(torch.bfloat16)


def assert_close(got, ref, limit, what):
    err = (got.double().cpu() - ref).abs()
    bad = ~(err <= limit)
    assert not bool(bad.any()), "%s: %d of %d out of bounds, first %s: got %r, reference %r" % (
        what, int(bad.sum()), bad.numel(), bad.nonzero()[0].tolist(), float(got.cpu()[tuple(bad.nonzero()[0])]),
        float(ref[tuple(bad.nonzero()[0])]))
