"""One expert with 2^31 - 1 rows, the most the library takes, on a GB300: nothing on the way from the offsets to the
tiles may pass 32 bits.  The widths are the smallest (8), so that inputs and outputs take 34 GB each."""
import gc

import pytest
import torch

import ragged_grouped_gemm_02_gb300 as rgg
from ragged_grouped_gemm_02_gb300 import _build

pytestmark = pytest.mark.gpu

ROWS = 2 ** 31 - 1
BASE = 2 ** 20  # the rows repeat after so many


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available(), "the gpu tests need a CUDA device"
    _build.build()
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 100e9:
        pytest.skip("needs 100 GB of device memory")
    yield
    gc.collect()
    torch.cuda.empty_cache()


def _offsets():
    return torch.tensor([0, ROWS], dtype=torch.int32, device="cuda")


def _whole(x):
    """x as its whole repetitions of BASE rows, and the rest."""
    n = x.shape[0] // BASE
    return x[: n * BASE].view(n, BASE, x.shape[1]), x[n * BASE:]


@pytest.mark.parametrize("opts", [dict(), dict(bm=64, bn=128), dict(bm=128, bn=128), dict(bm=256, bn=128, walk_order=4)],
                         ids=str)
@pytest.mark.parametrize("call", ["forward", "dgrad"])
def test_products(call, opts):
    gen = torch.Generator(device="cuda").manual_seed(1)
    base = torch.randint(-4, 5, (BASE, 8), generator=gen, device="cuda").to(torch.bfloat16)
    w = torch.randint(-4, 5, (1, 8, 8), generator=gen, device="cuda").to(torch.bfloat16)
    want = (base.float() @ (w[0].float() if call == "forward" else w[0].float().t())).to(torch.bfloat16)  # exact
    x = torch.empty(ROWS, 8, dtype=torch.bfloat16, device="cuda")
    whole, rest = _whole(x)
    whole.copy_(base)
    rest.copy_(base[: rest.shape[0]])
    y = torch.empty_like(x).fill_(float("nan"))
    product = rgg.rgg_grouped_gemm if call == "forward" else rgg.rgg_grouped_gemm_dgrad
    product(x, w, _offsets(), y, check=True, **opts)
    del x, whole, rest
    whole, rest = _whole(y)
    assert torch.equal(rest, want[: rest.shape[0]])
    for i in range(whole.shape[0]):
        if not torch.equal(whole[i], want):
            raise AssertionError("rows from %d" % (i * BASE))


@pytest.mark.parametrize("accumulate", [False, True])
def test_wgrad(accumulate):
    # rows at the ends and around the parts' first rows; whole numbers, so the sums are exact
    at = sorted({r for part in range(33) for d in (-65, -64, -1, 0, 1, 63, 64) for r in [part * (ROWS // 32) + d]
                 if 0 <= r < ROWS} | {ROWS - 1, ROWS - 2, ROWS - 64})
    gen = torch.Generator(device="cuda").manual_seed(2)
    X, dY = (torch.zeros(ROWS, 8, dtype=torch.bfloat16, device="cuda") for _ in (0, 1))
    rows = torch.tensor(at, device="cuda")
    x, dy = (torch.randint(-4, 5, (len(at), 8), generator=gen, device="cuda").to(torch.bfloat16) for _ in (0, 1))
    X[rows], dY[rows] = x, dy
    want = x.float().t() @ dy.float()
    old = torch.full((1, 8, 8), 3.0, device="cuda")
    got = rgg.rgg_grouped_gemm_wgrad(X, dY, _offsets(), old.clone(), accumulate=accumulate, check=True)
    assert torch.equal(got[0], want + 3.0 if accumulate else want)
