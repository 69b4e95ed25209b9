"""The expert layer's training and 4-bit operators, as cases that can be timed and compared.

Six operators around the ragged grouped product Y_e = X_e . W_e (expert e owns rows
[off[e], off[e+1]) of X, W is [E, K, N]):

* ``dgrad``   dX_e = dY_e . W_e^T, the gradient by the activations;
* ``wgrad``   dW_e = X_e^T . dY_e, the gradient by the weights (zeros for an expert without rows);
* ``swiglu_backward``  with g = X_e . W13_e[:, :N], u = X_e . W13_e[:, N:] computed again from X, the gradient
  [dH * u * silu'(g) | dH * silu(g)] and the activation H = silu(g) * u that the down projection's wgrad reads;
* ``clip``    the global 2-norm of a list of gradients, and the gradients scaled by min(1, max_norm / (norm + 1e-6));
* ``quantize``  MXFP4: blocks of 32 values along K, 4-bit E2M1 codes with a power-of-two scale per block,
  2^(floor(log2(max |x|)) - 2); rows as the activations of a call, or a [E, K, N] weight laid out once at load time;
* ``mxfp4``   bf16 activations quantised on the fly, times MXFP4 weights: plain, or the gate-up projection with SiLU.

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
        # four experts with an empty one and ragged tails: the smallest call, where latency counts
        {"name": "dgrad tiny", "op": "dgrad", "E": 4, "K": 256, "N": 512, "routing": "ragged", "rows": 256},
        # prefill-scale training batch: 32,768 tokens on 32 experts, K and N of the repository's prefill workload
        {"name": "dgrad prefill", "op": "dgrad", "E": 32, "K": 6144, "N": 4096, "routing": "multinomial", "rows": 32768},
        # rank^-1.2 routing over 64 experts: from 4,800 rows down to 32 per expert
        {"name": "wgrad skew16k", "op": "wgrad", "E": 64, "K": 1024, "N": 2688, "routing": "skew", "rows": 16384},
        {"name": "wgrad prefill", "op": "wgrad", "E": 32, "K": 6144, "N": 4096, "routing": "multinomial", "rows": 32768},
        # a small skewed batch whose experts have 4 to 600 rows; N is half of the gate-up weight's 2,688 columns
        {"name": "swiglu_bwd skew2k", "op": "swiglu_backward", "E": 64, "K": 1024, "N": 1344, "routing": "skew",
         "rows": 2048},
        {"name": "swiglu_bwd prefill", "op": "swiglu_backward", "E": 32, "K": 6144, "N": 2048,
         "routing": "multinomial", "rows": 32768},
        # the gradients of one tiny layer: five tensors, two types, latency
        {"name": "clip tiny", "op": "clip", "layers": 1, "E": 4, "K": 256, "N": 256},
        # the gradients of six expert layers: 30 tensors, 3.2 GB
        {"name": "clip six layers", "op": "clip", "layers": 6, "E": 64, "K": 1024, "N": 1344},
        # the activations of a decode step, 16 rows for each of 32 experts
        {"name": "quantize decode rows", "op": "quantize", "what": "rows", "E": 32, "K": 6144, "routing": "uniform",
         "rows": 512},
        # a whole expert weight, once at load time
        {"name": "quantize weights", "op": "quantize", "what": "weights", "E": 32, "K": 6144, "N": 4096},
        # decode: gate-up projection of 16 rows per expert, bound by the weights' bytes
        {"name": "mxfp4 decode gate-up", "op": "mxfp4", "swiglu": True, "E": 32, "K": 6144, "N": 2048,
         "routing": "uniform", "rows": 512},
        {"name": "mxfp4 prefill", "op": "mxfp4", "swiglu": False, "E": 32, "K": 6144, "N": 4096,
         "routing": "multinomial", "rows": 32768},
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _odd(rng, lo, hi):
    """An odd number; sizes are odd multiples of their alignment, so that they end inside tiles."""
    return min(_log_uniform(rng, lo, hi) | 1, hi - 1 if hi % 2 == 0 else hi)


def draw(rng):
    op = rng.choice(["dgrad", "wgrad", "swiglu_backward", "clip", "quantize", "mxfp4"])
    while True:
        if op == "clip":
            c = {"op": op, "layers": _log_uniform(rng, 1, 12), "E": _log_uniform(rng, 1, 64),
                 "K": 8 * _odd(rng, 8, 768), "N": 8 * _odd(rng, 8, 256)}
            if c["layers"] * c["E"] * c["K"] * c["N"] <= 6 * 64 * 1024 * 1344:
                return c
            continue
        c = _draw_product(rng, op, 32 if op in ("quantize", "mxfp4") else 8)
        # no more weights than the largest listed case has
        if c["E"] * c["K"] * c.get("N", 1) <= 32 * 6144 * (2048 if op == "swiglu_backward" or c.get("swiglu") else 4096):
            return c


def _draw_product(rng, op, unit):
    c = {"op": op, "E": _log_uniform(rng, 1, 64), "K": unit * _odd(rng, 256 // unit, 6144 // unit)}
    c["routing"] = rng.choice(["uniform", "skew", "multinomial"])
    c["rows"] = _odd(rng, 1, 32768)
    if c["routing"] == "uniform":
        c["rows"] = _odd(rng, 1, max(1, 32768 // c["E"])) * c["E"]
    c["N"] = 8 * _odd(rng, 32, 512)
    if op == "quantize":
        c["what"] = rng.choice(["rows", "weights"])
        for key in ("N",) if c["what"] == "rows" else ("routing", "rows"):
            del c[key]
    if op == "swiglu_backward":
        c["N"] = 8 * _odd(rng, 16, 256)
    if op == "mxfp4":
        c["swiglu"] = rng.random() < 0.5
        if c["swiglu"]:
            c["N"] = 128 * _odd(rng, 1, 16)
    return c


# ------------------------------------------------------------------- routing


def _shares(case):
    """Row counts by rank: the multiset is the same for every seed (multinomial routing: its mean)."""
    E, M = case["E"], case["rows"]
    if case["routing"] == "ragged":  # 37, 0, 64, 155 of 256 on four experts
        part = np.array([37.0, 0.0, 64.0, 155.0] * (-(-E // 4)))[:E]
    elif case["routing"] == "skew":
        part = (np.arange(E) + 1.0) ** -1.2
    else:
        part = np.ones(E)
    share = part / part.sum() * M
    counts = np.floor(share).astype(np.int64)
    counts[np.argsort(counts - share, kind="stable")[: M - int(counts.sum())]] += 1
    return counts


def _counts(case, seed):
    r = np.random.RandomState(seed % (1 << 31))
    if case["routing"] == "multinomial":
        return np.bincount(r.randint(0, case["E"], case["rows"]), minlength=case["E"]).astype(np.int64)
    counts = _shares(case)
    return counts[r.permutation(case["E"])] if case["routing"] == "skew" else counts


def _busy(case):
    """How many experts have rows, for the bytes of their weights."""
    if case["routing"] == "multinomial":
        return case["E"] * (1.0 - (1.0 - 1.0 / case["E"]) ** case["rows"])
    return int((_shares(case) > 0).sum())


# --------------------------------------------------------------------- MXFP4

# The values of the 16 codes of E2M1 (bit 3 the sign, two exponent bits, one mantissa bit).
E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0]


def _quantize(x):
    """x: fp32 [..., K].  Codes (uint8 [..., K]) and scale bytes (uint8 [..., K / 32], 2^(byte - 127))."""
    blocks = x.reshape(*x.shape[:-1], -1, 32)
    top = blocks.abs().amax(-1)
    byte = torch.clamp((top.view(torch.int32) >> 23) - 2, min=0)  # top's exponent field, less E2M1's largest exponent
    v = blocks * ((254 - byte) << 23).view(torch.float32).unsqueeze(-1)  # times 2^(127 - byte)
    a = v.abs()
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    code = code + 8 * (v < 0)
    return code.reshape(x.shape).to(torch.uint8), byte.to(torch.uint8)


def _values(code, byte):
    """fp32 values of codes [..., K] with scale bytes [..., K / 32]."""
    table = torch.tensor(E2M1, dtype=torch.float32, device=code.device)
    v = table[code.long()].reshape(*code.shape[:-1], -1, 32)
    b = byte.int()
    scale = torch.where(b == 0, 1 << 22, b << 23).view(torch.float32)  # 2^(byte - 127), subnormal for byte 0
    return (v * scale.unsqueeze(-1)).reshape(code.shape)


def _pack(code):
    """Two codes a byte, the even column in the low half."""
    return code[..., 0::2] | (code[..., 1::2] << 4)


def _unpack(packed):
    return torch.stack((packed & 15, packed >> 4), -1).reshape(*packed.shape[:-1], -1)


def _tile_scales(byte):
    """Scale bytes [E, N, K / 32] in the layout the products read: blocks of 128 rows by 4 scales, 512 bytes each, where
    row r and scale s of a block are at (r % 32) * 16 + (r / 32) * 4 + s; [E, N / 128, K / 128, 512], zeros in the padding."""
    E, N, S = byte.shape
    pad = torch.zeros(E, -(-N // 128) * 128, -(-S // 4) * 4, dtype=torch.uint8, device=byte.device)
    pad[:, :N, :S] = byte
    t = pad.view(E, -(-N // 128), 4, 32, -(-S // 4), 4)  # n-block, r / 32, r % 32, k-block, s
    return t.permute(0, 1, 4, 3, 2, 5).contiguous().view(E, -(-N // 128), -(-S // 4), 512)


def _untile_scales(tiled, N, K):
    E, nb, kb, _ = tiled.shape
    t = tiled.view(E, nb, kb, 32, 4, 4).permute(0, 1, 4, 3, 2, 5).reshape(E, nb * 128, kb * 4)
    return t[:, :N, : K // 32]


# ----------------------------------------------------------------- prepare


def _normal(g, *shape, std=1.0, dtype=torch.bfloat16):
    t = torch.empty(shape, dtype=dtype, device=DEVICE)
    return t.normal_(0.0, std, generator=g)


def _activations(g, rows, K):
    """Hidden states: normal, with a spread of scales between channels as normed activations have."""
    channel = torch.exp(0.5 * torch.empty(K, device=DEVICE).normal_(generator=g))
    return (torch.empty(rows, K, device=DEVICE).normal_(generator=g) * channel).to(torch.bfloat16)


def prepare(case, seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(int(seed))
    op = case["op"]
    s = dict(case)
    if op == "clip":
        E, K, N = case["E"], case["K"], case["N"]
        grads = []
        for _ in range(case["layers"]):
            # gate-up, down (bf16); router, a norm's weight, the routing bias (fp32)
            grads += [_normal(g, E, K, 2 * N, std=1e-3), _normal(g, E, N, K, std=2e-3),
                      _normal(g, E, K, std=1e-2, dtype=torch.float32), _normal(g, K, std=1e-2, dtype=torch.float32),
                      _normal(g, E, std=1e-2, dtype=torch.float32)]
        s["grads"] = grads
        s["clipped"] = [torch.empty_like(t) for t in grads]
        return s
    E, K = case["E"], case["K"]
    if op == "quantize" and case["what"] == "weights":
        s["W"] = _normal(g, E, K, case["N"], std=K ** -0.5)
        return s
    counts = _counts(case, seed)
    offsets = np.concatenate([[0], np.cumsum(counts)])
    s["bounds"] = [int(v) for v in offsets]  # the host's copy, for the plain form's slices
    s["offsets"] = torch.from_numpy(offsets.astype(np.int32)).to(DEVICE)
    M = case["rows"]
    if op == "quantize":
        s["X"] = _activations(g, M, K)
        return s
    N = case["N"]
    if op == "dgrad":
        s["dY"], s["W"] = _normal(g, M, N, std=1e-2), _normal(g, E, K, N, std=K ** -0.5)
    elif op == "wgrad":
        s["X"], s["dY"] = _activations(g, M, K), _normal(g, M, N, std=1e-2)
    elif op == "swiglu_backward":
        s["X"], s["W13"] = _normal(g, M, K), _normal(g, E, K, 2 * N, std=K ** -0.5)
        s["dH"] = _normal(g, M, N, std=1e-2)
    else:
        s["X"] = _activations(g, M, K)
        cols = 2 * N if case["swiglu"] else N
        codes, bytes_ = [], []
        for _ in range(E):
            code, byte = _quantize(_normal(g, cols, K, std=K ** -0.5, dtype=torch.float32))
            codes.append(_pack(code))
            bytes_.append(byte)
        s["W_codes"], s["W_scales"] = torch.stack(codes), _tile_scales(torch.stack(bytes_))
    return s


# --------------------------------------------------------------------- run


def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_own(s):
    import ragged_grouped_gemm_02_gb300 as rgg

    op = s["op"]
    if op == "dgrad":
        return rgg.rgg_grouped_gemm_dgrad(s["dY"], s["W"], s["offsets"])
    if op == "wgrad":
        return rgg.rgg_grouped_gemm_wgrad(s["X"], s["dY"], s["offsets"])
    if op == "swiglu_backward":
        return rgg.rgg_grouped_gemm_swiglu_backward(s["X"], s["W13"], s["offsets"], s["dH"])
    if op == "clip":
        norm = rgg.rgg_clip_grad_norm(s["grads"], 1.0, out=s["clipped"])
        return {"norm": norm, "clipped": s["clipped"]}
    if op == "quantize":
        if s["what"] == "weights":
            codes, scales = rgg.rgg_mxfp4_quantize_weights(s["W"])
            return rgg.rgg_mxfp4_dequantize_weights(codes, scales)
        codes, scales = rgg.rgg_mxfp4_quantize(s["X"], s["offsets"])
        return rgg.rgg_mxfp4_dequantize(codes, scales, s["offsets"])
    codes, scales = rgg.rgg_mxfp4_quantize(s["X"], s["offsets"])
    product = rgg.rgg_grouped_gemm_swiglu_mxfp4 if s["swiglu"] else rgg.rgg_grouped_gemm_mxfp4
    return product(codes, scales, s["W_codes"], s["W_scales"], s["offsets"])


def _silu(z):
    return z / (1.0 + torch.exp(-z))


def _run_plain(s):
    op = s["op"]
    if op == "clip":
        norm = torch.sqrt(torch.stack([t.float().square().sum() for t in s["grads"]]).sum())
        scale = torch.clamp(1.0 / (norm + 1e-6), max=1.0)
        for t, out in zip(s["grads"], s["clipped"]):
            out.copy_(t.float() * scale)
        return {"norm": norm, "clipped": s["clipped"]}
    if op == "quantize":
        x = s["X"] if s["what"] == "rows" else s["W"].transpose(1, 2)
        return _values(*_quantize(x.float().contiguous())).to(torch.bfloat16)
    if op == "wgrad":
        out = torch.empty(s["E"], s["K"], s["N"], dtype=torch.bfloat16, device=DEVICE)
    elif op == "dgrad":
        out = torch.empty(s["rows"], s["K"], dtype=torch.bfloat16, device=DEVICE)
    elif op == "swiglu_backward":
        out = torch.empty(s["rows"], 2 * s["N"], dtype=torch.bfloat16, device=DEVICE)
        H = torch.empty(s["rows"], s["N"], dtype=torch.bfloat16, device=DEVICE)
    else:
        out = torch.empty(s["rows"], s["N"], dtype=torch.bfloat16, device=DEVICE)
        X = _values(*_quantize(s["X"].float()))
        byte = _untile_scales(s["W_scales"], s["W_codes"].shape[1], s["K"])
    N = s["N"]
    # one fp32 product per expert: the experts' row counts differ, so no single product holds them all
    for e in range(s["E"]):
        rows = slice(s["bounds"][e], s["bounds"][e + 1])
        if op == "wgrad":
            out[e] = s["X"][rows].float().t() @ s["dY"][rows].float()
        elif rows.start == rows.stop:
            continue
        elif op == "dgrad":
            out[rows] = (s["dY"][rows].float() @ s["W"][e].float().t()).to(torch.bfloat16)
        elif op == "swiglu_backward":
            gu = s["X"][rows].float() @ s["W13"][e].float()
            g, u, dH = gu[:, :N], gu[:, N:], s["dH"][rows].float()
            sig = 1.0 / (1.0 + torch.exp(-g))
            H[rows] = (g * sig * u).to(torch.bfloat16)
            out[rows, :N] = (dH * u * sig * (1.0 + g * (1.0 - sig))).to(torch.bfloat16)
            out[rows, N:] = (dH * g * sig).to(torch.bfloat16)
        else:
            y = X[rows] @ _values(_unpack(s["W_codes"][e]), byte[e]).t()
            out[rows] = (_silu(y[:, :N]) * y[:, N:] if s["swiglu"] else y).to(torch.bfloat16)
    return (out, H) if op == "swiglu_backward" else out


# -------------------------------------------------------------------- work


def work(case):
    op, E, K = case["op"], case["E"], case["K"]
    if op == "clip":
        per = 3 * E * K * case["N"] * 2 + (E * K + K + E) * 4
        n = 3 * E * K * case["N"] + E * K + K + E
        return {"bytes": 2 * case["layers"] * per + 4, "flops": 3 * case["layers"] * n}
    if op == "quantize":
        n = E * K * case["N"] if case["what"] == "weights" else case["rows"] * K
        return {"bytes": 4 * n, "flops": 2 * n}
    M, N, busy = case["rows"], case["N"], _busy(case)
    cols = 2 * N if op == "swiglu_backward" or case.get("swiglu") else N
    flops = 2 * M * K * cols
    if op == "dgrad":
        moved = 2 * (M * N + busy * K * N + M * K)
    elif op == "wgrad":
        moved = 2 * (M * K + M * N + E * K * N)
    elif op == "swiglu_backward":
        moved = 2 * (M * K + busy * K * cols + M * N + M * cols + M * N)
    else:
        moved = 2 * M * K + busy * cols * K * (0.5 + 1 / 32) + 2 * M * N
    return {"bytes": moved + 4 * (E + 1), "flops": flops}


# ------------------------------------------------------------------- exact


def _power_of_two(n):
    """2^n in fp64, from its bits."""
    return ((n.to(torch.int64) + 1023) << 52).view(torch.float64)


def _mx64(x):
    """What MXFP4 holds of x (fp64 [..., K]), from the definition: nearest of the eight magnitudes, ties to the even one."""
    b = x.reshape(*x.shape[:-1], -1, 32)
    exponent = torch.frexp(b.abs().amax(-1, keepdim=True)).exponent - 1  # floor(log2), as frexp's fraction is in [0.5, 1)
    scale = _power_of_two(torch.clamp(exponent - 2, min=-127))
    v = torch.clamp((b / scale).abs(), max=6.0)
    step = torch.where(v < 2, 0.5, torch.where(v < 4, 1.0, 2.0))  # spacing of E2M1 around v
    return (torch.sign(b) * torch.round(v / step) * step * scale).reshape(x.shape)


def exact(case, seed):
    s = prepare(case, seed)
    op, E, K = case["op"], case["E"], case["K"]
    if op == "clip":
        norm = math.sqrt(math.fsum(float(t.double().square().sum()) for t in s["grads"]))
        scale = min(1.0, 1.0 / (norm + 1e-6))
        return {"norm": torch.tensor(norm, dtype=torch.float64), "clipped": [t.double() * scale for t in s["grads"]]}
    if op == "quantize":
        if case["what"] == "rows":
            return _mx64(s["X"].double())
        return torch.stack([_mx64(s["W"][e].double().t().contiguous()) for e in range(E)])
    N, b = case["N"], s["bounds"]
    parts, more = [], []
    for e in range(E):
        r0, r1 = b[e], b[e + 1]
        if op == "dgrad":
            parts.append(torch.einsum("mn,kn->mk", s["dY"][r0:r1].double(), s["W"][e].double()))
        elif op == "wgrad":
            parts.append(torch.einsum("mk,mn->kn", s["X"][r0:r1].double(), s["dY"][r0:r1].double()))
        elif op == "swiglu_backward":
            x = s["X"][r0:r1].double()
            g, u = x @ s["W13"][e, :, :N].double(), x @ s["W13"][e, :, N:].double()
            silu = g * torch.sigmoid(g)
            slope = torch.sigmoid(g) + silu * torch.sigmoid(-g)
            dH = s["dH"][r0:r1].double()
            parts.append(torch.cat([dH * u * slope, dH * silu], 1))
            more.append(silu * u)
        else:
            w = s["W_codes"][e]
            rows = w.shape[0]
            mag = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64, device=w.device)
            values = torch.empty(rows, K, dtype=torch.float64, device=w.device)
            for half in (0, 1):
                c = (w >> (4 * half)) & 15
                values[:, half::2] = mag[(c & 7).long()] * (1.0 - 2.0 * (c >> 3).double())
            n, k = torch.arange(rows, device=w.device)[:, None], torch.arange(K // 32, device=w.device)[None, :]
            byte = s["W_scales"][e][n // 128, k // 4, (n % 32) * 16 + (n % 128) // 32 * 4 + k % 4]
            values *= _power_of_two(byte.int() - 127).repeat_interleave(32, 1)
            y = _mx64(s["X"][r0:r1].double()) @ values.t()
            parts.append(y[:, :N] * torch.sigmoid(y[:, :N]) * y[:, N:] if case["swiglu"] else y)
    if op == "wgrad":
        return torch.stack(parts)
    return (torch.cat(parts), torch.cat(more)) if op == "swiglu_backward" else torch.cat(parts)
