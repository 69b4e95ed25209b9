"""rgg_grouped_gemm_wgrad's workspace on a GB300: the queried size is enough for every option, no call writes past the
workspace, and options do not keep the Python function from splitting the rows.  Sums: as in test_gpu_wgrad.py."""
import numpy as np
import pytest
import torch

import expert_refs as refs
import ragged_grouped_gemm_02_gb300 as rgg
from ragged_grouped_gemm_02_gb300 import _build

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available(), "the gpu tests need a CUDA device"
    _build.build()


def _case(counts, K, N, seed):
    gen = torch.Generator().manual_seed(seed)
    off, M = refs.ragged(counts)
    return refs.normal(gen, M, K), refs.normal(gen, M, N), off


# sizes at which some tile width or grid wants more parts than the query's
@pytest.mark.parametrize("flags", [0, 1, 2, 3])
@pytest.mark.parametrize("counts,K,N", [([6353, 6353, 6353, 6354, 6354], 152, 664), ([8192], 720, 1440),
                                        ([32768], 104, 488), ([8000, 192], 240, 432)])
def test_the_queried_size_is_enough(counts, K, N, flags):
    X, dY, off = _case(counts, K, N, seed=N)
    E, M = len(counts), X.shape[0]
    lib, handle = rgg.load_library(), rgg._handle(0)
    need = lib.rgg_grouped_gemm_wgrad_workspace(handle, E, M, K, N, flags)
    assert need > 0
    Xg, dYg, offg = X.cuda(), dY.cuda(), torch.from_numpy(off).cuda()
    dtype = torch.float32 if flags & 1 else torch.bfloat16
    ref, mag = refs.wgrad(X, dY, off)
    # n products, and one more addition for dW's old value or a part's sum
    n = torch.from_numpy(np.diff(off).astype(np.float64))[:, None, None] + 33
    limit = n * 2.0 ** -23 * mag + refs.TINY + (0 if flags & 1 else refs.ROUND_BF16 * ref.abs())
    for opts in (dict(), dict(bn=128), dict(bn=256), dict(max_ctas=64), dict(bn=256, max_ctas=64), dict(max_ctas=2),
                 dict(stages=2), dict(timeout_ns=1_000_000_000)):
        space = torch.full((need + 4096,), 0x5A, dtype=torch.uint8, device="cuda")
        dW = torch.zeros(E, K, N, dtype=dtype, device="cuda")
        opt, _ = rgg._options(**opts)
        rgg._set_workspace(opt, space[:need])
        s = lib.rgg_grouped_gemm_wgrad(handle, Xg.data_ptr(), dYg.data_ptr(), offg.data_ptr(), dW.data_ptr(), E, M, K,
                                       N, flags, torch.cuda.current_stream().cuda_stream, opt)
        assert s == rgg.RGG_OK, (opts, rgg.rgg_status_string(s))
        assert rgg.rgg_query_status(0) == rgg.RGG_OK
        refs.assert_close(dW, ref, limit, "dW with %s" % opts)
        assert bool((space[need:] == 0x5A).all()), opts


def test_options_keep_the_split():
    # the order of the sums depends on the sizes alone: an option that changes none of it changes no bit
    X, dY, off = _case([4096], 136, 264, seed=1)
    args = X.cuda(), dY.cuda(), torch.from_numpy(off).cuda()
    assert rgg.load_library().rgg_grouped_gemm_wgrad_workspace(rgg._handle(0), 1, 4096, 136, 264, 1) > 0
    want = rgg.rgg_grouped_gemm_wgrad(*args, dtype=torch.float32, check=True)
    got = rgg.rgg_grouped_gemm_wgrad(*args, dtype=torch.float32, timeout_ns=1_000_000_000, check=True)
    assert torch.equal(got, want)
