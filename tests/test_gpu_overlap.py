"""Launches with claims that overlap on a GB300 (two streams, two graphs of one capturing stream) on the package's one
handle: each has tile counters of its own, so every tile of every call is computed once, as in calls that follow each
other.  And a handle whose counters are all taken."""
import ctypes
import threading

import pytest
import torch

import expert_refs as refs
import ragged_grouped_gemm_02_gb300 as rgg
from ragged_grouped_gemm_02_gb300 import _build

pytestmark = pytest.mark.gpu

E, K, N = 8, 512, 1024
COUNTS = [[300, 5, 900, 0, 130, 257, 64, 700], [1, 800, 16, 333, 0, 512, 40, 256]]
HALF = dict(mixed=1, max_ctas=70)  # two such launches fit the GPU side by side


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available(), "the gpu tests need a CUDA device"
    _build.build()


def _case(seed):
    gen = torch.Generator().manual_seed(seed)
    off, M = refs.ragged(COUNTS[seed])
    x, dy, w = refs.normal(gen, M, K), refs.normal(gen, M, N), refs.normal(gen, E, K, N, std=K ** -0.5)
    return x.cuda(), dy.cuda(), w.cuda(), torch.from_numpy(off).cuda()


def _call(name, case, out, **kw):
    x, dy, w, off = case
    if name == "forward":
        return rgg.rgg_grouped_gemm(x, w, off, out[0], **HALF, **kw)
    if name == "gate_up":
        return rgg.rgg_grouped_gemm_swiglu(x, w, off, out[0], **HALF, **kw)
    if name == "dgrad":
        return rgg.rgg_grouped_gemm_dgrad(dy, w, off, out[0], **HALF, **kw)
    return rgg.rgg_grouped_gemm_swiglu_backward(x, w, off, dy[:, : N // 2].contiguous(), out[0], out[1], **HALF, **kw)


WIDTHS = {"forward": [N], "gate_up": [N // 2], "dgrad": [K], "gate_up_backward": [N, N // 2]}


def _outs(name, case):
    return [torch.empty(case[0].shape[0], n, dtype=torch.bfloat16, device="cuda") for n in WIDTHS[name]]


@pytest.mark.parametrize("name", sorted(WIDTHS))
def test_two_streams(name):
    cases = [_case(0), _case(1)]
    want = [_outs(name, c) for c in cases]
    for c, w in zip(cases, want):
        _call(name, c, w, check=True)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    rounds = 20
    got = [[_outs(name, c) for _ in range(rounds)] for c in cases]
    for side in got:
        for outs in side:
            for o in outs:
                o.fill_(7)
    torch.cuda.synchronize()
    for i in range(rounds):
        for c, side, s in zip(cases, got, streams):
            with torch.cuda.stream(s):
                _call(name, c, side[i])
    torch.cuda.synchronize()
    assert rgg.rgg_query_status(0) == rgg.RGG_OK
    for side, w in zip(got, want):
        for i, outs in enumerate(side):
            for o, r in zip(outs, w):
                assert torch.equal(o, r), "call %d of %s" % (i, name)


def test_two_graphs_of_one_stream():
    cases = [_case(0), _case(1)]
    want = [_outs("dgrad", c) for c in cases]
    for c, w in zip(cases, want):
        _call("dgrad", c, w, check=True)
    got = [_outs("dgrad", c) for c in cases]
    capturing = torch.cuda.Stream()
    graphs = []
    for c, o in zip(cases, got):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1], stream=capturing):
            for _ in range(10):
                _call("dgrad", c, o)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        for o in got:
            o[0].fill_(7)
        eager = _outs("dgrad", cases[0])
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        with torch.cuda.stream(capturing):  # and calls on the stream they were captured from, beside them
            _call("dgrad", cases[0], eager)
        torch.cuda.synchronize()
        assert rgg.rgg_query_status(0) == rgg.RGG_OK
        for o, w in zip(got + [eager], want + want[:1]):
            assert torch.equal(o[0], w[0])


def test_no_counters_left():
    # each capture takes a set for good; past the last one launches go without claims, with the same results
    lib = rgg.load_library()
    handle = ctypes.c_void_p()
    assert lib.rgg_create(ctypes.byref(handle), 0) == rgg.RGG_OK
    try:
        x, dy, w, off = _case(0)
        want = rgg.rgg_grouped_gemm_dgrad(dy, w, off, mixed=-1, check=True)
        dx = torch.empty_like(want)
        opt, _ = rgg._options(mixed=1)

        def call(stream):
            s = lib.rgg_grouped_gemm_dgrad(handle, dy.data_ptr(), w.data_ptr(), off.data_ptr(), dx.data_ptr(), E,
                                           dy.shape[0], K, N, stream.cuda_stream, opt)
            assert s == rgg.RGG_OK

        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            for _ in range(4096):
                graph = torch.cuda.CUDAGraph()
                graph.capture_begin()
                call(side)
                graph.capture_end()
            dx.fill_(7)
            graph.replay()
            side.synchronize()
            assert torch.equal(dx, want)
            dx.fill_(7)
            call(side)  # no set for the stream itself
            side.synchronize()
            assert torch.equal(dx, want)
        assert lib.rgg_query_status(handle, side.cuda_stream) == rgg.RGG_OK
    finally:
        torch.cuda.synchronize()
        lib.rgg_destroy(handle)


def test_calls_beside_a_capture():
    # calls on streams that the handle sees for the first time, while another stream is being captured
    cases = [_case(0), _case(1)]
    want = [_outs("dgrad", c) for c in cases]
    for c, w in zip(cases, want):
        _call("dgrad", c, w, check=True)
    got, eager = _outs("dgrad", cases[0]), [_outs("dgrad", cases[1]) for _ in range(3)]
    others = [torch.cuda.Stream() for _ in eager]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for o, s in zip(eager, others):
            _call("dgrad", cases[0], got)
            _call("dgrad", cases[1], o, stream=s)
    for s in others:
        s.synchronize()
    got[0].fill_(7)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0][0])
    for o in eager:
        assert torch.equal(o[0], want[1][0])


def test_per_thread_default_streams():
    # one handle stands for the default stream of each thread: its calls run beside those of other threads
    per_thread = torch.cuda.ExternalStream(2)
    cases = [_case(0), _case(1)]
    want = [_outs("dgrad", c) for c in cases]
    for c, w in zip(cases, want):
        _call("dgrad", c, w, check=True)
    got = [[_outs("dgrad", c) for _ in range(20)] for c in cases]
    torch.cuda.synchronize()
    failures = []

    def work(i):
        try:
            torch.cuda.set_device(0)
            for outs in got[i]:
                _call("dgrad", cases[i], outs, stream=per_thread)
            per_thread.synchronize()
        except Exception as e:  # shown by the test's own thread
            failures.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in (0, 1)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failures, failures
    assert rgg.rgg_query_status(0) == rgg.RGG_OK
    for side, w in zip(got, want):
        for outs in side:
            assert torch.equal(outs[0], w[0])
    # and captured
    out, graph = _outs("dgrad", cases[0]), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=per_thread):
        _call("dgrad", cases[0], out)
    out[0].fill_(7)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out[0], want[0][0])
