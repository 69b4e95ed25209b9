"""The mixture-of-experts layer: its operators together, gradients, graphs and streams, on a GB300."""
import pytest
import torch

import moe_refs as refs
import ragged_grouped_gemm_02_gb300 as rgg
from ragged_grouped_gemm_02_gb300 import _build
from ragged_grouped_gemm_02_gb300.expert_layer import expert_ffn_fp8, quantize_experts_fp8
from ragged_grouped_gemm_02_gb300.moe_layer import combine, dispatch, moe_ffn, moe_ffn_fp8

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available(), "the gpu tests need a CUDA device"
    _build.build()


def _layer(T=150, E=7, K=256, N=192, seed=0, dtype=torch.bfloat16):
    gen = torch.Generator().manual_seed(seed)
    X = torch.randn(T, K, generator=gen).to(torch.bfloat16)
    logits = (1.5 * torch.randn(T, E, generator=gen)).to(dtype)
    W13 = (torch.randn(E, K, 2 * N, generator=gen) * K ** -0.5).to(torch.bfloat16)
    W2 = (torch.randn(E, N, K, generator=gen) * N ** -0.5).to(torch.bfloat16)
    return [t.cuda() for t in (X, logits, W13, W2)]


def _plain(X, logits, W13, W2, k, score="softmax", renormalize=True, scale=1.0):
    """The layer in 64 bits, differentiable."""
    experts = refs.route(logits.detach().cpu(), k, score, renormalize, scale)[0].cuda()
    w = refs.weights_of(logits, experts, score, renormalize, scale)
    out = torch.zeros(X.shape[0], W2.shape[2], dtype=torch.float64, device=X.device)
    for e in range(W13.shape[0]):
        t, j = torch.nonzero(experts == e, as_tuple=True)
        g, u = (X[t] @ W13[e]).chunk(2, 1)
        out = out.index_add(0, t, w[t, j].unsqueeze(1) * ((torch.nn.functional.silu(g) * u) @ W2[e]))
    return out


def _off(a, b):
    a, b = a.detach().double(), b.detach().double()
    return float((a - b).norm() / b.norm())


@pytest.mark.parametrize("score,renormalize", [("softmax", True), ("softmax", False), ("sigmoid", True)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_training(score, renormalize, dtype):
    rule = {"score": score, "renormalize": renormalize, "scale": 1.5}
    leaves = [t.requires_grad_() for t in _layer(dtype=dtype)]
    out = moe_ffn(*leaves, 3, **rule)
    dout = torch.randn(out.shape, generator=torch.Generator().manual_seed(5)).to(torch.bfloat16).cuda()
    grads = torch.autograd.grad(out, leaves, dout)
    same = [t.detach().double().requires_grad_() for t in leaves]
    want = _plain(*same, 3, **rule)
    ref = torch.autograd.grad(want, same, dout.double())
    # bf16 roundings (each 2^-8 / sqrt 3 of the root mean square at most): H and Y forward; dY, dH, dGU, H, dX backward
    for got, exact in zip((out, *grads), (want, *ref)):
        assert _off(got, exact) < 6 * 2.0 ** -8 / 3 ** 0.5
    assert rgg.rgg_query_status() == rgg.RGG_OK


def test_dispatch_and_combine_gradients_leave_rows_of_no_choice_zero():
    gen = torch.Generator().manual_seed(1)
    experts = refs.choices(gen, 40, 3, 6, 0.3)
    position = refs.sort(experts, 6)[2].cuda()
    rows = int((experts >= 0).sum())
    X = torch.randn(40, 64, generator=gen).to(torch.bfloat16).cuda().requires_grad_()
    w = torch.rand(40, 3, generator=gen).cuda().requires_grad_()
    Xs = dispatch(X, position)
    (dX,) = torch.autograd.grad(Xs[:rows].sum(), X)
    assert torch.equal(dX, (position >= 0).sum(1, keepdim=True).expand(40, 64).to(torch.bfloat16))
    Y = torch.randn(120, 64, generator=gen).to(torch.bfloat16).cuda().requires_grad_()
    dY, dw = torch.autograd.grad(combine(Y, position, w).sum(), (Y, w))
    assert bool((dY[rows:] == 0).all()) and bool((dw[position < 0] == 0).all())
    assert bool((dY[:rows] != 0).all())
    (dw2,) = torch.autograd.grad(combine(Y.detach(), position, w).sum(), w)
    assert torch.equal(dw, dw2)


def test_masked_tokens_get_zeros():
    X, logits, W13, W2 = _layer(T=20)
    logits[3] = float("-inf")
    logits[5, 1:] = float("-inf")
    leaves = [t.requires_grad_() for t in (X, logits, W13, W2)]
    out = moe_ffn(*leaves, 2)
    assert bool((out[3] == 0).all())
    grads = torch.autograd.grad(out.float().sum(), leaves)
    assert all(bool(g.isfinite().all()) for g in grads)
    assert bool((grads[0][3] == 0).all()) and bool((grads[1][3] == 0).all())
    experts = quantize_experts_fp8(W13, W2)
    assert bool((moe_ffn_fp8(X.detach(), logits.detach(), experts, 2)[3] == 0).all())


@pytest.mark.parametrize("T,N", [(1, 128), (150, 192), (600, 256)])
def test_serving(T, N):
    X, logits, W13, W2 = _layer(T=T, N=N)
    experts = quantize_experts_fp8(W13, W2)
    out = moe_ffn_fp8(X, logits, experts, 3)
    chosen, w = rgg.rgg_route_topk(logits, 3)
    offsets, _, position = rgg.rgg_sort_by_expert(chosen, 7, check=True)
    rows = rgg.rgg_dispatch(X, position)
    assert torch.equal(out, rgg.rgg_combine(expert_ffn_fp8(rows, experts, offsets), position, w))
    # each rounding to E4M3 is off by at most 2^-4 / sqrt 3 of the root mean square; X and W13 are in gate and in up
    # (whose errors add in H, with |silu'| <= 1.1), then H and W2
    exact = _plain(*(t.double() for t in (X, logits, W13, W2)), 3)
    assert _off(out, exact) < (2.1 * 2 + 2) * 2.0 ** -4 / 3 ** 0.5
    assert rgg.rgg_query_status() == rgg.RGG_OK


def test_graphs_that_share_nothing_replay_together():
    # two captured serving steps and one training step, replayed on streams of their own, give what eager calls give
    serve = [_layer(T=40, seed=s) for s in (1, 2)]
    experts = [quantize_experts_fp8(c[2], c[3]) for c in serve]
    want = [moe_ffn_fp8(c[0], c[1], e, 2) for c, e in zip(serve, experts)]
    train = [t.requires_grad_() for t in _layer(T=60, seed=3)]

    def step():
        return torch.autograd.grad(moe_ffn(*train, 2).float().sum(), train)

    ref = [g.clone() for g in step()]
    torch.cuda.synchronize()
    graphs, outs, streams = [], [], [torch.cuda.Stream() for _ in range(3)]
    for i in range(3):
        with torch.cuda.stream(streams[i]):
            (step if i == 2 else lambda: moe_ffn_fp8(serve[i][0], serve[i][1], experts[i], 2))()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=streams[i]):
            outs.append(step() if i == 2 else moe_ffn_fp8(serve[i][0], serve[i][1], experts[i], 2))
        graphs.append(g)
    for _ in range(5):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want[0]) and torch.equal(outs[1], want[1])
    assert all(torch.equal(a, b) for a, b in zip(outs[2], ref))
    # new inputs in the captured buffers
    serve[0][1].copy_(serve[1][1])
    serve[0][0].copy_(serve[1][0])
    with torch.cuda.stream(streams[0]):
        graphs[0].replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], moe_ffn_fp8(serve[1][0], serve[1][1], experts[0], 2))


def test_calls_on_another_stream():
    X, logits, W13, W2 = _layer(T=80)
    experts = quantize_experts_fp8(W13, W2)
    want = moe_ffn_fp8(X, logits, experts, 2)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    chosen, w = rgg.rgg_route_topk(logits, 2, stream=s)
    offsets, _, position = rgg.rgg_sort_by_expert(chosen, 7, stream=s)
    x = rgg.rgg_fp8_block_quantize(X, position, stream=s)
    h = rgg.rgg_grouped_gemm_swiglu_fp8_block(*x, *experts[0], offsets, stream=s)
    y = rgg.rgg_grouped_gemm_fp8_block(*h, *experts[1], offsets, stream=s)
    out = rgg.rgg_combine(y, position, w, stream=s)
    s.synchronize()
    assert torch.equal(out, want)


def test_equal_calls_give_equal_bits():
    leaves = [t.requires_grad_() for t in _layer(T=500, seed=4)]
    runs = []
    for _ in range(3):
        out = moe_ffn(*leaves, 4, renormalize=False)
        runs.append([out, *torch.autograd.grad(out.float().square().sum(), leaves)])
    for r in runs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(runs[0], r))


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16])
def test_dispatch_with_a_gradient_takes_bf16(dtype):
    # the gradient is a sum of bf16 rows: refused at the call, not in the backward pass
    X = torch.zeros(4, 8, dtype=dtype, device="cuda", requires_grad=True)
    with pytest.raises(TypeError, match="bf16"):
        dispatch(X, torch.zeros(4, 2, dtype=torch.int32, device="cuda"))


def test_rows_of_no_choice_do_not_reach_gradients(monkeypatch):
    # tokens with fewer experts than k, or none: rows behind the last expert's hold NaN on the way forward and back
    from ragged_grouped_gemm_02_gb300 import moe_layer
    X, logits, W13, W2 = _layer(T=90, E=5)
    logits[::4, 1:] = float("-inf")
    logits[::7] = float("-inf")
    leaves = [t.requires_grad_() for t in (X, logits, W13, W2)]

    def grads():
        return torch.autograd.grad(moe_ffn(*leaves, 3).float().square().sum(), leaves)

    want = grads()
    dispatch_, backward_, passed = rgg.rgg_dispatch, rgg.rgg_combine_backward, []

    def nan_dispatch(X, position):
        return dispatch_(X, position, torch.full((position.numel(), X.shape[1]), float("nan"), dtype=X.dtype, device="cuda"))

    def nan_backward(dout, Y, position, weights, dY=None, dweights=None):
        passed.append(dY)
        return backward_(dout, Y, position, weights, torch.full_like(Y, float("nan")), dweights)

    monkeypatch.setattr(moe_layer, "rgg_dispatch", nan_dispatch)
    monkeypatch.setattr(moe_layer, "rgg_combine_backward", nan_backward)
    got = grads()
    assert passed == [None]
    assert all(torch.equal(a, b) and bool(torch.isfinite(a).all()) for a, b in zip(got, want))
    assert rgg.rgg_query_status() == rgg.RGG_OK
