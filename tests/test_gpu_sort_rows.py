"""Sorting by expert, dispatch and combine against counting and 64-bit sums, on a GB300."""
import pytest
import torch

import moe_refs as refs
import ragged_grouped_gemm_02_gb300 as rgg
from ragged_grouped_gemm_02_gb300 import _build

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available(), "the gpu tests need a CUDA device"
    _build.build()


def _gen(seed):
    return torch.Generator().manual_seed(seed)


@pytest.mark.parametrize("T,k,E", [(0, 2, 4), (1, 1, 1), (1, 3, 3), (5, 2, 40), (31, 1, 2), (33, 3, 7), (512, 4, 32),
                                   (1023, 4, 64), (1024, 4, 33), (1025, 4, 64), (4097, 1, 5), (3000, 6, 256),
                                   (700, 8, 1000), (1500, 3, 4096), (20000, 8, 64), (200000, 1, 3)])
def test_sort(T, k, E):
    experts = torch.randint(-1, E, (T, k), generator=_gen(T + E), dtype=torch.int32)
    got = rgg.rgg_sort_by_expert(experts.cuda(), E, check=True)
    for a, b in zip(got, refs.sort(experts, E)):
        assert torch.equal(a.cpu(), b)


@pytest.mark.parametrize("T", [40, 3000])
@pytest.mark.parametrize("kind", ["one expert", "none", "first and last", "descending"])
def test_sort_uneven(T, kind):
    E = 37
    experts = torch.full((T, 2), 5, dtype=torch.int32)
    if kind == "none":
        experts[:] = -3
    elif kind == "first and last":
        experts[:, 0], experts[:, 1] = E - 1, 0
    elif kind == "descending":
        experts = (E - 1 - torch.arange(2 * T, dtype=torch.int32).view(T, 2) * E // (2 * T)).to(torch.int32)
    for a, b in zip(rgg.rgg_sort_by_expert(experts.cuda(), E, check=True), refs.sort(experts, E)):
        assert torch.equal(a.cpu(), b)


@pytest.mark.parametrize("T", [10, 4000])
def test_sort_reports_experts_out_of_range(T):
    experts = torch.randint(0, 8, (T, 2), generator=_gen(1), dtype=torch.int32)
    experts[T // 2, 1] = 8
    experts[T - 1, 0] = 2 ** 31 - 1
    with pytest.raises(rgg.RggError, match="BAD_ROW_INDEX"):
        rgg.rgg_sort_by_expert(experts.cuda(), 8, check=True)
    got = rgg.rgg_sort_by_expert(experts.cuda(), 8)
    assert rgg.rgg_query_status() == rgg.RGG_ERR_BAD_ROW_INDEX
    for a, b in zip(got, refs.sort(experts, 8)):
        assert torch.equal(a.cpu(), b)


@pytest.mark.parametrize("K", [1, 2, 3, 7, 8, 60, 128, 500, 513, 1024, 2693])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32, torch.uint8, torch.float64])
def test_dispatch(K, dtype):
    T, k, E = 37, 3, 9
    experts = refs.choices(_gen(K), T, k, E, dropped=0.2)
    _, row_index, position = refs.sort(experts, E)
    X = torch.randint(0, 200, (T, K), generator=_gen(K)).to(dtype)
    out = torch.full((T * k + 3, K), 77, dtype=dtype, device="cuda")
    rgg.rgg_dispatch(X.cuda(), position.cuda(), out, check=True)
    rows = int((experts >= 0).sum())
    assert torch.equal(out.cpu()[:rows], X[row_index[:rows].long()])
    assert bool((out[rows:] == 77).all()), "rows of no choice are left alone"


@pytest.mark.parametrize("shift", [1, 2, 4, 8])
def test_dispatch_and_combine_of_unaligned_tensors(shift):
    # views that start off a wide boundary, of rows that would take wide loads
    T, k, K = 20, 2, 512
    experts = refs.choices(_gen(1), T, k, 4)
    _, row_index, position = refs.sort(experts, 4)
    flat = torch.randn(T * K + shift, generator=_gen(2)).to(torch.bfloat16).cuda()
    X = flat[shift:].view(T, K)
    out = torch.zeros(T * k * K + shift, dtype=torch.bfloat16, device="cuda")[shift:].view(T * k, K)
    rgg.rgg_dispatch(X, position.cuda(), out, check=True)
    assert torch.equal(out.cpu(), X.cpu()[row_index.long()])
    w = torch.rand(T, k, generator=_gen(3))
    back = torch.zeros(T * K + shift, dtype=torch.bfloat16, device="cuda")[shift:].view(T, K)
    rgg.rgg_combine(out, position.cuda(), w.cuda(), back, check=True)
    want, limit = refs.combine(out.cpu(), position, w)
    assert bool(((back.cpu().double() - want).abs() <= limit).all())
    d = torch.randn(T * K + shift, generator=_gen(4)).to(torch.bfloat16).cuda()[shift:].view(T, K)
    dY, dw = rgg.rgg_combine_backward(d, out, position.cuda(), w.cuda(), check=True)
    _check_backward(d, out, position, w, dY, dw)


def _case(T, k, N, dropped, seed=0):
    gen = _gen(seed + T + k + N)
    E = max(k, 5)
    position = refs.sort(refs.choices(gen, T, k, E, dropped), E)[2]
    rows = int((position >= 0).sum())
    Y = torch.randn(rows + 2, N, generator=gen).to(torch.bfloat16)
    return Y, position, torch.rand(T, k, generator=gen), torch.randn(T, N, generator=gen).to(torch.bfloat16), rows


def _check_backward(d, Y, position, w, dY, dw):
    d, Y, dY = d.cpu(), Y.cpu(), dY.cpu()
    kept = position >= 0
    at = position.long().clamp(min=0)
    want = w.double().unsqueeze(-1) * d.double().unsqueeze(1)
    assert bool(((dY.double()[at] - want).abs() <= refs.rounding(want, torch.bfloat16))[kept].all())
    terms = Y.double()[at] * d.double().unsqueeze(1)
    want = torch.where(kept, terms.sum(-1), 0.0)
    limit = Y.shape[1] * 2.0 ** -23 * terms.abs().sum(-1)
    assert bool(((dw.cpu().double() - want).abs() <= limit).all())


@pytest.mark.parametrize("dropped", [0.0, 0.4])
@pytest.mark.parametrize("T,k,N", [(1, 1, 1), (3, 2, 7), (5, 4, 8), (17, 8, 100), (9, 9, 256), (6, 33, 257), (40, 6, 1344),
                                   (11, 5, 2693), (300, 1, 6), (2, 70, 130), (257, 3, 2050)])
def test_combine_and_gradients(T, k, N, dropped):
    Y, position, w, d, rows = _case(T, k, N, dropped)
    out = rgg.rgg_combine(Y.cuda(), position.cuda(), w.cuda(), check=True)
    want, limit = refs.combine(Y, position, w)
    assert bool(((out.cpu().double() - want).abs() <= limit).all())
    plain = rgg.rgg_combine(Y.cuda(), position.cuda(), check=True)
    want, limit = refs.combine(Y, position, torch.ones_like(w))
    assert bool(((plain.cpu().double() - want).abs() <= limit).all())
    dY = torch.full(Y.shape, 77.0, dtype=torch.bfloat16, device="cuda")
    _, dw = rgg.rgg_combine_backward(d.cuda(), Y.cuda(), position.cuda(), w.cuda(), dY, check=True)
    _check_backward(d, Y, position, w, dY, dw)
    assert bool((dY[rows:] == 77).all()), "rows of no choice are left alone"
    alone = rgg.rgg_combine_backward(d.cuda(), Y.cuda(), position.cuda(), w.cuda(), False, check=True)
    assert alone[0] is None and torch.equal(alone[1], dw)
    alone = rgg.rgg_combine_backward(d.cuda(), Y.cuda(), position.cuda(), w.cuda(), None, False, check=True)
    assert alone[1] is None and torch.equal(alone[0][:rows], dY[:rows])


def test_rows_of_no_choice_do_not_reach_a_sum():
    Y, position, w, d, rows = _case(30, 4, 264, 0.3)
    out = rgg.rgg_combine(Y.cuda(), position.cuda(), w.cuda())
    grads = rgg.rgg_combine_backward(d.cuda(), Y.cuda(), position.cuda(), w.cuda())
    bad = Y.clone()
    bad[rows:] = float("nan")
    w2 = torch.where(position >= 0, w, float("nan"))
    assert torch.equal(rgg.rgg_combine(bad.cuda(), position.cuda(), w2.cuda()), out)
    again = rgg.rgg_combine_backward(d.cuda(), bad.cuda(), position.cuda(), w2.cuda())
    assert torch.equal(again[0][:rows], grads[0][:rows]) and torch.equal(again[1], grads[1])


@pytest.mark.parametrize("call", ["dispatch", "combine", "backward"])
def test_positions_out_of_range_are_reported(call):
    Y, position, w, d, rows = _case(20, 3, 64, 0.0)
    position[4, 1] = Y.shape[0]
    position[19, 0] = 2 ** 31 - 1
    position[7, 2] = -5
    none = torch.where(position >= Y.shape[0], -1, position)
    args = [t.cuda() for t in (Y, w, d)]

    def run(p):
        out = torch.zeros_like(args[0])
        if call == "dispatch":
            return rgg.rgg_dispatch(args[2], p.cuda(), out)
        if call == "combine":
            return rgg.rgg_combine(args[0], p.cuda(), args[1])
        return torch.cat([t.flatten().float() for t in rgg.rgg_combine_backward(args[2], args[0], p.cuda(), args[1], out)])

    a = run(position)
    assert rgg.rgg_query_status() == rgg.RGG_ERR_BAD_ROW_INDEX
    assert torch.equal(a, run(none))
    assert rgg.rgg_query_status() == rgg.RGG_OK


def test_empty_batches():
    position = torch.empty(0, 2, dtype=torch.int32, device="cuda")
    assert rgg.rgg_dispatch(torch.empty(0, 8, device="cuda"), position).shape == (0, 8)
    Y = torch.empty(0, 8, dtype=torch.bfloat16, device="cuda")
    assert rgg.rgg_combine(Y, position).shape == (0, 8)
    # tokens without a single row
    none = torch.full((3, 2), -1, dtype=torch.int32, device="cuda")
    assert bool((rgg.rgg_combine(Y, none, torch.ones(3, 2, device="cuda"), check=True) == 0).all())
    dY, dw = rgg.rgg_combine_backward(torch.ones(3, 8, dtype=torch.bfloat16, device="cuda"), Y, none,
                                      torch.ones(3, 2, device="cuda"), check=True)
    assert dY.shape == (0, 8) and bool((dw == 0).all())


def test_sort_feeds_the_gather_products():
    # row_index and group_offsets as the gather product reads them: the same rows as dispatch then the product
    T, k, E, K, N = 90, 2, 6, 256, 128
    gen = _gen(4)
    X = torch.randn(T, K, generator=gen).to(torch.bfloat16).cuda()
    W = (torch.randn(E, K, N, generator=gen) / 16).to(torch.bfloat16).cuda()
    offsets, row_index, position = rgg.rgg_sort_by_expert(refs.choices(gen, T, k, E, 0.1).cuda(), E, check=True)
    rows = int(offsets[-1])
    a = rgg.rgg_grouped_gemm(rgg.rgg_dispatch(X, position), W, offsets, check=True)
    b = rgg.rgg_grouped_gemm_gather(X, row_index, W, offsets, check=True)
    assert torch.equal(a[:rows], b[:rows])


def test_sorts_of_two_threads():
    # tables of 70 KB and 221 KB of shared memory by turns: neither thread's call takes room from the other's
    import threading
    cases = [torch.randint(-1, E, (1024, 4), generator=_gen(E), dtype=torch.int32) for E in (512, 2048)]
    want = [refs.sort(c, E) for c, E in zip(cases, (512, 2048))]
    errors = []

    def work(i, E):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                experts = cases[i].cuda()
                for _ in range(300):
                    got = rgg.rgg_sort_by_expert(experts, E)
            stream.synchronize()
            assert all(torch.equal(a.cpu(), b) for a, b in zip(got, want[i]))
        except BaseException as e:  # shown by the test's thread
            errors.append(e)

    threads = [threading.Thread(target=work, args=a) for a in ((0, 512), (1, 2048))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    assert rgg.rgg_query_status() == rgg.RGG_OK
