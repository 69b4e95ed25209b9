"""What stands around the expert products in a mixture-of-experts layer, and their 8-bit form, as cases that can be timed
and compared.

* ``route``     the k largest of a token's E logits (ties to the lower expert; -inf is a masked expert, never chosen: such a
  slot holds expert -1 and weight 0) and the choices' weights: softmax over all experts or sigmoid of the logit, optionally
  divided by their sum over the choices (sigmoid: + 1e-20), times ``scale``.  Training adds the gradient by the logits;
* ``dispatch``  the choices sorted by expert, stably (offsets, the token of each row, the row of each choice), and the
  tokens' rows copied in that order;
* ``combine``   out[t] = sum_j weight[t, j] * Y[position[t, j]]; training adds dY and dweight;
* ``quantize``  8-bit E4M3 codes with one fp32 scale per 128 values of a row (sorted by expert on the way) or per 128 x 128
  values of a weight: with a = max(max |x|, 2^-100), the scale is a / 448 and a code is 448 x / a rounded to nearest even;
* ``fp8``       the ragged grouped product of such rows and weights, the sums in 32 bits;
* ``layer``     quantise, gate-up product, SiLU, quantise, down product;
* ``moe``       a whole serving step: route, dispatch, layer, combine.

``own`` selects the framework's kernels; otherwise ``run`` computes the plain form in 32 bits.
"""
import math

import numpy as np
import torch

own = False

DEVICE = "cuda"


# --------------------------------------------------------------------- cases


def listed():
    return [
        # the router of one decode step: 64 tokens, latency
        {"name": "route decode", "op": "route", "T": 64, "E": 64, "k": 4, "dtype": "float32", "score": "softmax",
         "renormalize": True, "scale": 1.0, "masked": 0, "train": False},
        # the router of a training batch of 32,768 tokens over many experts, forward and backward
        {"name": "route train", "op": "route", "T": 32768, "E": 256, "k": 8, "dtype": "bfloat16", "score": "sigmoid",
         "renormalize": True, "scale": 2.5, "masked": 0, "train": True},
        # 512 rows for 32 experts: the rows of the repository's decode workload
        {"name": "dispatch decode", "op": "dispatch", "T": 128, "E": 32, "k": 4, "K": 6144, "skew": 0.0},
        # 32,768 rows on 32 experts: those of its prefill workload
        {"name": "dispatch prefill", "op": "dispatch", "T": 8192, "E": 32, "k": 4, "K": 6144, "skew": 0.0},
        # the same steps on their way back
        {"name": "combine decode", "op": "combine", "T": 128, "E": 32, "k": 4, "K": 6144, "dropped": 0.0, "train": False},
        # a training batch with a width that no wide load divides, some choices dropped for want of capacity
        {"name": "combine train", "op": "combine", "T": 8192, "E": 64, "k": 6, "K": 2693, "dropped": 0.05, "train": True},
        # a prefill's tokens to 8 bits, each to the rows of its four experts
        {"name": "quantize prefill rows", "op": "quantize", "what": "rows", "T": 8192, "E": 32, "k": 4, "K": 6144},
        # a whole expert weight, once at load time
        {"name": "quantize weights", "op": "quantize", "what": "weights", "E": 32, "K": 6144, "N": 4096},
        # decode: 16 rows per expert, bound by the weights' bytes
        {"name": "fp8 decode", "op": "fp8", "E": 32, "K": 6144, "N": 4096, "routing": "uniform", "rows": 512},
        {"name": "fp8 prefill", "op": "fp8", "E": 32, "K": 6144, "N": 4096, "routing": "multinomial", "rows": 32768},
        # rank^-1.2 routing over 64 experts: from 4,800 rows down to 32 per expert
        {"name": "layer skew16k", "op": "layer", "E": 64, "K": 1024, "N": 1408, "routing": "skew", "rows": 16384},
        # one serving step of 16 tokens through a layer of 64 experts
        {"name": "moe decode", "op": "moe", "T": 16, "E": 64, "k": 4, "K": 1024, "N": 1408},
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _odd(rng, lo, hi):
    """An odd number; sizes are odd multiples of their alignment, so that they end inside tiles."""
    return min(_log_uniform(rng, lo, hi) | 1, hi - 1 if hi % 2 == 0 else hi)


def draw(rng):
    op = rng.choice(["route", "dispatch", "combine", "quantize", "fp8", "layer", "moe"])
    if op == "route":
        E = _log_uniform(rng, 2, 256)
        c = {"op": op, "T": _log_uniform(rng, 1, 32768), "E": E, "k": rng.randint(1, min(E, 8)),
             "dtype": rng.choice(["float32", "bfloat16", "float16"]), "score": rng.choice(["softmax", "sigmoid"]),
             "renormalize": rng.random() < 0.5, "scale": rng.choice([1.0, 2.5]),
             "masked": rng.choice([0, rng.randint(0, E - 1)]), "train": rng.random() < 0.5}
        if c["train"] and c["renormalize"]:  # a single choice's weight is 1, whatever its logit
            c["k"], c["masked"] = max(c["k"], 2), min(c["masked"], E - 2)
        return c
    if op == "moe":
        E = _log_uniform(rng, 2, 64)
        return {"op": op, "T": _log_uniform(rng, 1, 64), "E": E, "k": rng.randint(1, min(E, 6)), "K": 16 * _odd(rng, 8, 64),
                "N": 128 * _log_uniform(rng, 1, 11)}
    if op in ("fp8", "layer") or (op == "quantize" and rng.random() < 0.5):
        c = {"op": op, "E": _log_uniform(rng, 1, 64), "K": 16 * _odd(rng, 16, 128 if op == "layer" else 384)}
        c["N"] = 128 * _log_uniform(rng, 1, 16) if op == "layer" else 8 * _odd(rng, 16, 512)
        while c["E"] * c["K"] * c["N"] > 32 * 6144 * 4096:
            c["E"] = max(1, c["E"] // 2)
        if op == "quantize":
            return {**c, "what": "weights"}
        c["routing"] = rng.choice(["uniform", "skew", "multinomial"])
        c["rows"] = _odd(rng, 1, 16384 if op == "layer" else 32768)
        if c["routing"] == "uniform":
            c["rows"] = max(1, c["rows"] // c["E"]) * c["E"]
        return c
    E = _log_uniform(rng, 1, 256)
    c = {"op": op, "T": _log_uniform(rng, 1, 8192), "E": E, "k": rng.randint(1, min(E, 6))}
    if op == "quantize":
        return {**c, "what": "rows", "k": min(c["k"], 4), "K": 16 * _odd(rng, 16, 384)}
    c["K"] = rng.choice([_log_uniform(rng, 64, 2693), 8 * _odd(rng, 8, 336)])
    if op == "dispatch":
        return {**c, "skew": rng.choice([0.0, 1.2])}
    return {**c, "dropped": rng.choice([0.0, 0.05, 0.3]), "train": rng.random() < 0.5}


# ------------------------------------------------------------------- routing


def _counts(case, seed):
    """Rows of each expert."""
    r = np.random.RandomState(seed % (1 << 31))
    E, M = case["E"], case["rows"]
    if case["routing"] == "multinomial":
        return np.bincount(r.randint(0, E, M), minlength=E).astype(np.int64)
    counts = _even_counts(case)
    return counts[r.permutation(E)] if case["routing"] == "skew" else counts


def _even_counts(case):
    part = (np.arange(case["E"]) + 1.0) ** (-1.2 if case["routing"] == "skew" else 0.0)
    share = part / part.sum() * case["rows"]
    counts = np.floor(share).astype(np.int64)
    counts[np.argsort(counts - share, kind="stable")[: case["rows"] - int(counts.sum())]] += 1
    return counts


def _busy(case, rows):
    """How many experts have rows, for the bytes of their weights."""
    if case.get("routing", "multinomial") == "multinomial":
        return case["E"] * (1.0 - (1.0 - 1.0 / case["E"]) ** rows)
    return int((_even_counts(case) > 0).sum())


def _choices(g, T, E, k, skew):
    """k different experts for each token; skew: how the experts' shares fall with their rank."""
    gumbel = -torch.log(torch.empty(T, E, device=DEVICE).exponential_(generator=g))
    share = -skew * torch.log(torch.arange(1, E + 1, device=DEVICE, dtype=torch.float32))
    return torch.topk(gumbel + share, k, dim=1).indices.to(torch.int32)


def _sort(experts, E):
    """Offsets by expert, the token of each sorted row and the row of each choice (experts < 0: -1, behind the last row)."""
    T, k = experts.shape
    key = torch.where(experts < 0, E, experts).reshape(-1).long()
    order = torch.sort(key, stable=True).indices
    counts = torch.bincount(key, minlength=E + 1)[:E]
    offsets = torch.zeros(E + 1, dtype=torch.int32, device=key.device)
    offsets[1:] = torch.cumsum(counts, 0)
    rank = torch.arange(T * k, device=key.device)
    position = torch.empty_like(rank)
    position[order] = rank
    dropped = key == E
    row_index = torch.where(dropped[order], -1, order // k)
    return offsets, row_index.to(torch.int32), torch.where(dropped, -1, position).to(torch.int32).view(T, k)


# ----------------------------------------------------------------- prepare


def _normal(g, *shape, std=1.0, dtype=torch.bfloat16):
    return torch.empty(shape, dtype=dtype, device=DEVICE).normal_(0.0, std, generator=g)


def _activations(g, rows, K):
    """Hidden states: normal, with a spread of scales between channels as normed activations have."""
    channel = torch.exp(0.5 * torch.empty(K, device=DEVICE).normal_(generator=g))
    return (torch.empty(rows, K, device=DEVICE).normal_(generator=g) * channel).to(torch.bfloat16)


def _weight(g, E, N, K):
    """A weight's codes [E, N, K] and scales [E, ceil(N / 128), ceil(K / 128)], as a checkpoint holds them."""
    codes, scales = [], []
    for _ in range(E):
        c, s = _quantize_weight(_normal(g, N, K, std=K ** -0.5, dtype=torch.float32))
        codes.append(c)
        scales.append(s)
    return torch.stack([c.view(torch.uint8) for c in codes]).view(torch.float8_e4m3fn), torch.stack(scales)


def prepare(case, seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(int(seed))
    op, E = case["op"], case["E"]
    s = dict(case)
    if op in ("route", "moe"):
        T = case["T"]
        logits = _normal(g, T, E, std=1.5, dtype=torch.float32) + _normal(g, E, std=0.5, dtype=torch.float32)
        if op == "route":
            if case["masked"]:  # experts that a token may not take, others for each token
                score = torch.empty(T, E, device=DEVICE).uniform_(generator=g)
                logits.scatter_(1, score.topk(case["masked"], dim=1).indices, float("-inf"))
            s["logits"] = logits.to(getattr(torch, case["dtype"]))
            s["dweights"] = _normal(g, T, case["k"], dtype=torch.float32)
            return s
        s["logits"] = logits
        s["X"] = _activations(g, T, case["K"])
    if op in ("dispatch", "combine") or case.get("what") == "rows":
        T, k, K = case["T"], case["k"], case["K"]
        experts = _choices(g, T, E, k, case.get("skew", 0.0))
        if op == "combine" and case["dropped"]:
            drop = torch.empty(T * k, device=DEVICE).uniform_(generator=g).argsort()[: int(T * k * case["dropped"])]
            experts.view(-1)[drop] = -1
        s["experts"] = experts
        if op != "dispatch":
            s["position"] = _sort(experts, E)[2]
        if op != "combine":
            s["X"] = _activations(g, T, K)
            return s
        rows = int((experts >= 0).sum())
        s["Y"] = _normal(g, rows, K)
        s["weights"] = torch.softmax(_normal(g, T, k, dtype=torch.float32), 1)
        s["dout"] = _normal(g, T, K, std=1e-2)
        return s
    K, N = case["K"], case["N"]
    if op == "quantize":
        s["W"] = _normal(g, E, K, N, std=K ** -0.5)
        return s
    if op == "fp8":
        s["w"] = _weight(g, E, N, K)
    else:
        s["experts"] = (_weight(g, E, 2 * N, K), _weight(g, E, K, N))
    if op == "moe":
        return s
    offsets = np.concatenate([[0], np.cumsum(_counts(case, seed))])
    s["bounds"] = [int(v) for v in offsets]  # the host's copy, for the plain form's slices
    s["offsets"] = torch.from_numpy(offsets.astype(np.int32)).to(DEVICE)
    x = _activations(g, case["rows"], K)
    if op == "fp8":
        s["x"] = _quantize_rows(x.float())
    else:
        s["X"] = x
    return s


# --------------------------------------------------------------------- run


def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_own(s):
    import ragged_grouped_gemm_02_gb300 as rgg
    from ragged_grouped_gemm_02_gb300.expert_layer import expert_ffn_fp8
    from ragged_grouped_gemm_02_gb300.moe_layer import moe_ffn_fp8

    op = s["op"]
    if op == "route":
        rule = {"score": s["score"], "renormalize": s["renormalize"], "scale": s["scale"]}
        experts, weights = rgg.rgg_route_topk(s["logits"], s["k"], **rule)
        if not s["train"]:
            return experts, weights
        return experts, weights, rgg.rgg_route_topk_backward(s["logits"], experts, s["dweights"], **rule)
    if op == "dispatch":
        offsets, row_index, position = rgg.rgg_sort_by_expert(s["experts"], s["E"])
        return offsets, row_index, position, rgg.rgg_dispatch(s["X"], position)
    if op == "combine":
        out = rgg.rgg_combine(s["Y"], s["position"], s["weights"])
        if not s["train"]:
            return out
        return (out, *rgg.rgg_combine_backward(s["dout"], s["Y"], s["position"], s["weights"]))
    if op == "quantize":
        if s["what"] == "weights":
            return rgg.rgg_fp8_block_dequantize_weights(*rgg.rgg_fp8_block_quantize_weights(s["W"]))
        return rgg.rgg_fp8_block_dequantize(*rgg.rgg_fp8_block_quantize(s["X"], s["position"]))
    if op == "fp8":
        return rgg.rgg_grouped_gemm_fp8_block(*s["x"], *s["w"], s["offsets"])
    if op == "layer":
        return expert_ffn_fp8(s["X"], s["experts"], s["offsets"])
    return moe_ffn_fp8(s["X"], s["logits"], s["experts"], s["k"])


def _blocks(x):
    """The last dimension in blocks of 128, zeros behind its end."""
    x = torch.nn.functional.pad(x, (0, -x.shape[-1] % 128))
    return x.view(*x.shape[:-1], -1, 128)


def _spread(scales, n):
    """Each scale 128 times along the last dimension, n in all."""
    return scales.repeat_interleave(128, -1)[..., :n]


def _codes(x, top):
    # 448 = 0.4375 * 2^10: of a bf16 x the product is exact, so the one rounding of the division leaves ties as they are
    return (x * 0.4375 / top * 1024.0).to(torch.float8_e4m3fn)


def _quantize_rows(x):
    """x: fp32 [rows, K].  Codes [rows, K] and scales [rows, ceil(K / 128)]."""
    top = torch.clamp(_blocks(x).abs().amax(-1), min=2.0 ** -100)
    return _codes(x, _spread(top, x.shape[-1])), top / 448.0


def _quantize_weight(w):
    """w: fp32 [..., N, K].  Codes of that shape and scales [..., ceil(N / 128), ceil(K / 128)]."""
    N, K = w.shape[-2:]
    top = _blocks(_blocks(w).abs().amax(-1).transpose(-1, -2)).amax(-1).transpose(-1, -2)
    top = torch.clamp(top, min=2.0 ** -100)
    return _codes(w, _spread_weight(top, N, K)), top / 448.0


def _spread_weight(scales, N, K):
    return _spread(_spread(scales, K).transpose(-1, -2), N).transpose(-1, -2)


def _row_values(codes, scales):
    return codes.float() * _spread(scales, codes.shape[-1])


def _weight_values(codes, scales):
    return codes.float() * _spread_weight(scales, *codes.shape[-2:])


def _route(logits, k, score, renormalize, scale):
    """experts, weights, and what the gradient reads: the scores of all experts and the chosen ones' before the scale."""
    z = logits.float()
    value, index = torch.sort(z, dim=1, descending=True, stable=True)
    index, chosen = index[:, :k], value[:, :k] > -math.inf
    if score == "sigmoid":
        p = 1.0 / (1.0 + torch.exp(-z))
    else:
        top = value[:, :1]
        p = torch.exp(z - torch.where(top > -math.inf, top, 0.0))
        p = p / torch.clamp(p.sum(1, keepdim=True), min=1e-30)
    w = torch.where(chosen, p.gather(1, index), 0.0)
    if renormalize:
        w = w / (w.sum(1, keepdim=True) + 1e-20)
    return torch.where(chosen, index, -1).to(torch.int32), w * scale, p, w


def _route_gradient(s, p, w, experts):
    chosen = experts >= 0
    index = torch.clamp(experts, min=0).long()
    g = torch.where(chosen, s["dweights"] * s["scale"], 0.0)
    q = p.gather(1, index)
    if s["renormalize"]:
        g = g - (g * w).sum(1, keepdim=True)
        if s["score"] == "sigmoid":  # by the chosen scores, then by their logits
            g = g / (torch.where(chosen, q, 0.0).sum(1, keepdim=True) + 1e-20) * q * (1.0 - q)
        else:
            g = g * w
    elif s["score"] == "sigmoid":
        g = g * q * (1.0 - q)
    g = torch.where(chosen, g, 0.0)
    d = torch.zeros_like(p).scatter_add_(1, index, g)
    if s["score"] == "softmax" and not s["renormalize"]:  # every expert's logit is in every weight
        d = p * (d - (g * q).sum(1, keepdim=True))
    return d.to(s["logits"].dtype)


def _products(x, w, bounds, rows, N):
    """One fp32 product per expert, as the experts' row counts differ and no single product holds them all."""
    y = torch.empty(rows, N, device=DEVICE)
    for e in range(len(bounds) - 1):
        if bounds[e] < bounds[e + 1]:
            y[bounds[e] : bounds[e + 1]] = x[bounds[e] : bounds[e + 1]] @ _weight_values(w[0][e], w[1][e]).t()
    return y


def _silu_up(gu):
    g, u = gu.chunk(2, -1)
    return g / (1.0 + torch.exp(-g)) * u


def _run_plain(s):
    op = s["op"]
    if op == "route":
        experts, weights, p, w = _route(s["logits"], s["k"], s["score"], s["renormalize"], s["scale"])
        return (experts, weights, _route_gradient(s, p, w, experts)) if s["train"] else (experts, weights)
    if op == "dispatch":
        offsets, row_index, position = _sort(s["experts"], s["E"])
        return offsets, row_index, position, s["X"][row_index.long()]
    if op == "combine":
        kept = s["position"] >= 0
        at = torch.clamp(s["position"], min=0).long()
        w = torch.where(kept, s["weights"], 0.0)
        rows = s["Y"][at].float()
        out = (rows * w.unsqueeze(-1)).sum(1).to(torch.bfloat16)
        if not s["train"]:
            return out
        d = s["dout"].float().unsqueeze(1)
        dY = torch.empty_like(s["Y"])
        dY[at[kept]] = (w.unsqueeze(-1) * d).to(torch.bfloat16)[kept]
        return out, dY, torch.where(kept, (rows * d).sum(-1), 0.0)
    if op == "quantize":
        if s["what"] == "weights":
            return _weight_values(*_quantize_weight(s["W"].float().transpose(1, 2))).to(torch.bfloat16)
        token = torch.empty(s["position"].numel(), dtype=torch.long, device=DEVICE)
        token[s["position"].reshape(-1).long()] = torch.arange(s["T"], device=DEVICE).repeat_interleave(s["k"])
        return _row_values(*_quantize_rows(s["X"].float())).to(torch.bfloat16)[token]
    if op == "fp8":
        return _products(_row_values(*s["x"]), s["w"], s["bounds"], s["rows"], s["N"]).to(torch.bfloat16)
    w13, w2 = s["experts"]
    x = _row_values(*_quantize_rows(s["X"].float()))
    if op == "layer":
        h = _silu_up(_products(x, w13, s["bounds"], s["rows"], 2 * s["N"]))
        h = _row_values(*_quantize_rows(h))
        return _products(h, w2, s["bounds"], s["rows"], s["K"]).to(torch.bfloat16)
    # a few tokens: every expert on every token, and the router's weights, zero where it was not chosen
    experts, weights, _, _ = _route(s["logits"], s["k"], "softmax", True, 1.0)
    h = _silu_up(x @ _weight_values(*w13).transpose(1, 2))
    y = (_row_values(*_quantize_rows(h)) @ _weight_values(*w2).transpose(1, 2)).to(torch.bfloat16).float()
    dense = torch.zeros(s["T"], s["E"], device=DEVICE).scatter_(1, experts.long(), weights)
    return (dense.t().unsqueeze(-1) * y).sum(0).to(torch.bfloat16)


# -------------------------------------------------------------------- work


def work(case):
    op, E = case["op"], case["E"]
    if op == "route":
        T, k, width = case["T"], case["k"], 4 if case["dtype"] == "float32" else 2
        b = T * E * width + 8 * T * k
        f = T * E * (3 + k)
        if case["train"]:  # the logits are there already; dweights read, dlogits written
            b, f = b + T * E * width + 4 * T * k, f + 4 * T * E
        return {"bytes": b, "flops": f}
    if "T" in case:
        T, k, K = case["T"], case["k"], case["K"]
        rows = T * k
        if op == "dispatch":
            return {"bytes": 2 * T * K + 2 * rows * K + 12 * rows + 4 * (E + 1), "flops": rows}
        if op == "combine":
            b, f = 2 * rows * K + 2 * T * K + 8 * rows, 2 * rows * K
            if case["train"]:  # dout read, dY and dweights written
                b, f = b + 2 * T * K + 2 * rows * K + 4 * rows, f + 3 * rows * K
            return {"bytes": b, "flops": f}
        if op == "quantize":  # read, and the rows' values written
            return {"bytes": 2 * T * K + 2 * rows * K + 4 * rows, "flops": 2 * T * K}
    K, N = case["K"], case["N"]
    if op == "quantize":
        return {"bytes": 4 * E * K * N, "flops": 2 * E * K * N}
    if op == "fp8":
        M = case["rows"]
        scales = 4 * M * -(-K // 128) + 4 * E * -(-K // 128) * -(-N // 128)
        return {"bytes": M * K + _busy(case, M) * K * N + scales + 2 * M * N + 4 * (E + 1), "flops": 2 * M * K * N}
    M = case["rows"] if op == "layer" else case["T"] * case["k"]
    held = 3 * _busy(case, M) * K * N * (1 + 4 / 128 ** 2)
    if op == "layer":
        return {"bytes": 4 * M * K + held + 4 * (E + 1), "flops": 6 * M * K * N}
    return {"bytes": 4 * case["T"] * K + held + 4 * case["T"] * E, "flops": 6 * M * K * N}


# ------------------------------------------------------------------- exact


def _e4m3_64(v):
    """The nearest E4M3 value of each v in [-448, 448], ties to the even one."""
    exponent = torch.clamp(torch.frexp(v).exponent - 1, min=-6)
    step = torch.ldexp(torch.ones_like(v), exponent - 3)
    return torch.clamp(torch.round(v / step) * step, -448.0, 448.0)


def _held_rows_64(x, one_scale=False):
    """What the 8-bit form holds of x (fp64 [rows, K]), block by block along K; one_scale: of all rows of a block together."""
    out = torch.empty_like(x)
    for k0 in range(0, x.shape[1], 128):
        b = x[:, k0 : k0 + 128]
        top = b.abs().max() if one_scale else b.abs().amax(1, keepdim=True)
        top = torch.clamp(top, min=2.0 ** -100)
        out[:, k0 : k0 + 128] = _e4m3_64(b * 448.0 / top) * (top / 448.0)
    return out


def _weight_64(w, e):
    """The values of expert e's weight in 64 bits, [N, K]."""
    codes = w[0][e].double()
    n = torch.arange(codes.shape[0], device=DEVICE) // 128
    k = torch.arange(codes.shape[1], device=DEVICE) // 128
    return codes * w[1][e].double()[n[:, None], k[None, :]]


def _ffn_64(x, experts, e):
    gu = x @ _weight_64(experts[0], e).t()
    N = gu.shape[1] // 2
    h = gu[:, :N] * torch.sigmoid(gu[:, :N]) * gu[:, N:]
    return _held_rows_64(h) @ _weight_64(experts[1], e).t()


def _route_64(logits, k, score, renormalize, scale):
    """experts and weights, chosen one after the other: the largest logit that is left, the first of equal ones."""
    z = logits.double().clone()
    p = torch.sigmoid(z) if score == "sigmoid" else torch.nan_to_num(torch.softmax(z, 1), nan=0.0)
    experts, weights, rows = [], [], torch.arange(z.shape[0], device=DEVICE)
    for _ in range(k):
        best = z.amax(1, keepdim=True)
        e = torch.where(z == best, torch.arange(z.shape[1], device=DEVICE), z.shape[1]).amin(1)
        ok = best[:, 0] > -math.inf
        experts.append(torch.where(ok, e, -1))
        weights.append(torch.where(ok, p[rows, e], 0.0))
        z[rows, e] = -math.inf
    experts, w = torch.stack(experts, 1).to(torch.int32), torch.stack(weights, 1)
    if renormalize:
        w = w / (w.sum(1, keepdim=True) + 1e-20)
    return experts, w * scale


def exact(case, seed):
    s = prepare(case, seed)
    op, E = case["op"], case["E"]
    if op == "route":
        rule = (case["score"], case["renormalize"], case["scale"])
        if not case["train"]:
            return _route_64(s["logits"], case["k"], *rule)
        with torch.enable_grad():
            z = s["logits"].double().requires_grad_()
            experts, _ = _route_64(z.detach(), case["k"], *rule)
            chosen, at = experts >= 0, torch.clamp(experts, min=0).long()
            p = torch.sigmoid(z) if case["score"] == "sigmoid" else torch.softmax(z, 1)
            w = torch.where(chosen, p.gather(1, at), 0.0)
            if case["renormalize"]:
                w = w / (w.sum(1, keepdim=True) + 1e-20)
            w = w * case["scale"]
            (d,) = torch.autograd.grad(w, z, s["dweights"].double())
        return experts, w.detach(), d
    if op == "dispatch":
        e = s["experts"].cpu().numpy().reshape(-1)
        T, k = case["T"], case["k"]
        row_index, position, offsets, at = np.empty(T * k, np.int32), np.empty(T * k, np.int32), [0], 0
        for i in range(E):
            mine = np.nonzero(e == i)[0]
            row_index[at : at + len(mine)], position[mine] = mine // k, np.arange(at, at + len(mine))
            at += len(mine)
            offsets.append(at)
        token = torch.from_numpy(row_index.astype(np.int64)).to(DEVICE)
        return np.array(offsets, np.int32), row_index, position.reshape(T, k), s["X"].index_select(0, token).double()
    if op == "combine":
        T, k, K = case["T"], case["k"], case["K"]
        out = torch.zeros(T, K, dtype=torch.float64, device=DEVICE)
        dY = torch.zeros(*s["Y"].shape, dtype=torch.float64, device=DEVICE)
        dw = torch.zeros(T, k, dtype=torch.float64, device=DEVICE)
        for j in range(k):
            t = torch.nonzero(s["position"][:, j] >= 0)[:, 0]
            at = s["position"][t, j].long()
            y, w, d = s["Y"][at].double(), s["weights"][t, j].double()[:, None], s["dout"][t].double()
            out[t] += w * y
            dY[at] = w * d
            dw[t, j] = torch.einsum("tk,tk->t", y, d)
        return (out, dY, dw) if case["train"] else out
    if op == "quantize":
        if case["what"] == "rows":
            held = _held_rows_64(s["X"].double())
            out = torch.empty(case["T"] * case["k"], case["K"], dtype=torch.float64, device=DEVICE)
            for j in range(case["k"]):
                out[s["position"][:, j].long()] = held
            return out
        out = torch.empty(E, case["N"], case["K"], dtype=torch.float64, device=DEVICE)
        for e in range(E):
            w = s["W"][e].double().t()
            for n0 in range(0, case["N"], 128):
                out[e, n0 : n0 + 128] = _held_rows_64(w[n0 : n0 + 128], one_scale=True)
        return out
    if op == "moe":
        experts, weights = _route_64(s["logits"], case["k"], "softmax", True, 1.0)
        x = _held_rows_64(s["X"].double())
        out = torch.zeros(case["T"], case["K"], dtype=torch.float64, device=DEVICE)
        for e in range(E):
            t, j = torch.nonzero(experts == e, as_tuple=True)
            if len(t):
                out.index_add_(0, t, weights[t, j][:, None] * _ffn_64(x[t], s["experts"], e))
        return out
    parts = []
    b = s["bounds"]
    if op == "fp8":
        scale = s["x"][1].double()[:, torch.arange(case["K"], device=DEVICE) // 128]
        x = s["x"][0].double() * scale
    else:
        x = _held_rows_64(s["X"].double())
    for e in range(E):
        rows = x[b[e] : b[e + 1]]
        parts.append(rows @ _weight_64(s["w"], e).t() if op == "fp8" else _ffn_64(rows, s["experts"], e))
    return torch.cat(parts)
