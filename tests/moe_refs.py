"""64-bit references of routing, sorting by expert, combining and the 8-bit form with a scale per block of 128.

Rounding to a type is off by at most half a step, eps / 2 of the value (bf16 2^-8, fp16 2^-11, fp32 2^-24, e4m3 2^-4)
or half the spacing of its smallest values.  An fp32 sum of n terms whose magnitudes sum to S is off by at most
n * 2^-23 * S, however it is ordered and whether it rounds or truncates.
"""
import math

import torch

TINY = {torch.float32: 2.0 ** -149, torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -24}


def rounding(t, dtype):
    """The most that rounding t to dtype can change it."""
    return t.abs() * (torch.finfo(dtype).eps / 2) + TINY[dtype]


# ------------------------------------------------------------------- router


def route(logits, k, score, renormalize, scale):
    """experts (int64 [T, k], -1: none), weights and their error bound."""
    z = logits.double()
    T, E = z.shape
    experts = torch.full((T, k), -1, dtype=torch.int64)
    for t in range(T):
        row = z[t].tolist()
        order = sorted((e for e in range(E) if row[e] != -math.inf), key=lambda e: (-row[e], e))[:k]
        experts[t, : len(order)] = torch.tensor(order, dtype=torch.int64)
    w = weights_of(z, experts, score, renormalize, scale)
    # exp of a difference d: the difference is off by 2^-24 |d|, expf by 2 units in the last place, the division and the
    # scale by one rounding each; a sum of E exponentials by E * 2^-23 of itself; sigmoid's argument is exact
    spread = torch.where(z.isinf(), 0.0, z).abs().amax(1, keepdim=True)
    return experts, w, w.abs() * (2 * spread + 12 + 2 * E) * 2.0 ** -23 + 2.0 ** -126


def weights_of(z, experts, score, renormalize, scale):
    """The weights of these choices, differentiable by z (fp64)."""
    chosen = experts >= 0
    s = torch.sigmoid(z) if score == "sigmoid" else torch.nan_to_num(torch.softmax(z, 1))
    w = torch.where(chosen, s.gather(1, experts.clamp(min=0)), 0.0)
    if renormalize:
        w = w / (w.sum(1, keepdim=True) + 1e-20)
    return w * scale


def route_gradient(logits, experts, dweights, score, renormalize, scale):
    """dlogits (fp64) and a magnitude that its fp32 terms do not pass."""
    with torch.enable_grad():
        z = logits.detach().double().requires_grad_()
        w = weights_of(z, experts, score, renormalize, scale)
        (d,) = torch.autograd.grad(w, z, dweights.double())
    # every term is a weight or a score (at most 1) times a dweight times scale; a row's terms sum to at most this
    size = (dweights.double().abs().sum(1, keepdim=True) * abs(scale)).expand_as(d)
    return d, size


# ----------------------------------------------------------------- sorting


def sort(experts, E):
    """group_offsets, row_index and position of [T, k] choices, by counting."""
    T, k = experts.shape
    flat = experts.reshape(-1).tolist()
    rows = [[] for _ in range(E)]
    for i, e in enumerate(flat):
        if 0 <= e < E:
            rows[e].append(i)
    offsets, order = [0], []
    for r in rows:
        order += r
        offsets.append(len(order))
    position = torch.full((T * k,), -1, dtype=torch.int32)
    position[torch.tensor(order, dtype=torch.int64)] = torch.arange(len(order), dtype=torch.int32)
    row_index = torch.full((T * k,), -1, dtype=torch.int32)
    row_index[: len(order)] = torch.tensor([i // k for i in order], dtype=torch.int32)
    return torch.tensor(offsets, dtype=torch.int32), row_index, position.view(T, k)


def choices(gen, T, k, E, dropped=0.0):
    """k different experts for each token, some of them dropped."""
    e = torch.rand(T, E, generator=gen).argsort(1)[:, :k].to(torch.int32)
    e[torch.rand(T, k, generator=gen) < dropped] = -1
    return e.contiguous()


def combine(Y, position, weights):
    """out and its error bound."""
    at = position.long().clamp(min=0)
    kept = (position >= 0).unsqueeze(-1)
    terms = torch.where(kept, weights.double().unsqueeze(-1) * Y.double()[at], 0.0) if len(Y) else torch.zeros(
        *position.shape, Y.shape[1], dtype=torch.float64)
    out = terms.sum(1)
    return out, rounding(out, torch.bfloat16) + position.shape[1] * 2.0 ** -23 * terms.abs().sum(1)


# ------------------------------------------------------- 8 bits, blocks of 128


def _e4m3(v):
    """The nearest E4M3 value of each v of at most 448, ties to the even one."""
    exponent = torch.clamp(torch.frexp(v).exponent - 1, min=-6)
    step = torch.pow(torch.tensor(2.0, dtype=torch.float64), (exponent - 3).double())
    return torch.round(v / step) * step


def fp8_rows(x):
    """What the 8-bit form holds of x (bf16 [rows, K]): codes' values, scales (the fp32 quotients) and values, fp64."""
    rows, K = x.shape
    blocks = -(-K // 128)
    b = torch.zeros(rows, blocks * 128, dtype=torch.float64)
    b[:, :K] = x.double()
    return _fp8(b.view(rows, blocks, 128), (2,), lambda t: t.reshape(rows, -1)[:, :K])


def fp8_weights(w):
    """The same of a weight [E, N, K], one scale per 128 x 128."""
    E, N, K = w.shape
    nb, kb = -(-N // 128), -(-K // 128)
    b = torch.zeros(E, nb * 128, kb * 128, dtype=torch.float64)
    b[:, :N, :K] = w.double()
    return _fp8(b.view(E, nb, 128, kb, 128), (2, 4), lambda t: t.reshape(E, nb * 128, kb * 128)[:, :N, :K])


def _fp8(b, dims, shaped):
    top = torch.clamp(b.abs().amax(dims, keepdim=True), min=2.0 ** -100)
    codes = _e4m3(b * 448.0 / top)
    scales = (top.float() / 448.0).double()
    return shaped(codes), scales.flatten(dims[0]).reshape([s for i, s in enumerate(b.shape) if i not in dims]), shaped(codes * scales)
