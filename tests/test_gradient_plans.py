"""The planner on dgrad and the gate-up backward: the configuration that the calls run."""
import pytest

import ragged_grouped_gemm_02_gb300 as rgg
from ragged_grouped_gemm_02_gb300 import _build


@pytest.fixture(scope="module", autouse=True)
def built():
    _build.build()


def _tile(*args, **kw):
    p = rgg.rgg_plan(*args, **kw)
    return p["bm"], p["bn"]


def test_few_tiles_take_the_smallest():
    # 64 x 128 tiles where one wave of 152 holds them, every expert's last tile counted as partial
    assert _tile(4, 256, 256, 512, op="dgrad") == (64, 128)          # (4 + 4) x 2 tiles
    assert _tile(1, 533, 504, 1768, op="dgrad") == (64, 128)
    assert _tile(2, 10, 3048, 280, op="swiglu_backward") == (64, 128)
    # 152 tiles of 128 columns, and 153
    assert _tile(1, 1, 128 * 152, 512, op="dgrad") == (64, 128)
    assert _tile(1, 1, 128 * 153, 512, op="dgrad") == (64, 256)
    assert _tile(1, 1, 512, 64 * 152, op="swiglu_backward") == (64, 128)
    assert _tile(1, 1, 512, 64 * 153, op="swiglu_backward") == (64, 256)
    # fewer CTAs, fewer tiles
    assert _tile(4, 256, 256, 512, op="dgrad", max_ctas=15) == _tile(4, 256, 512, 256, max_ctas=15)
    assert _tile(4, 256, 256, 512, op="dgrad", max_ctas=16) == (64, 128)
    assert _tile(4, 256, 256, 512, op="dgrad", num_sms=15) == _tile(4, 256, 512, 256, num_sms=15)


@pytest.mark.parametrize("opts", [dict(bm=128), dict(bn=256), dict(bm=256, bn=128), dict(mixed=1), dict(mixed=-1)], ids=str)
def test_options_come_first(opts):
    assert rgg.rgg_plan(4, 256, 256, 512, op="dgrad", **opts) == dict(rgg.rgg_plan(4, 256, 512, 256, **opts), threads=320)
    assert rgg.rgg_plan(4, 256, 256, 512, op="swiglu_backward", **opts) == rgg.rgg_plan(4, 256, 256, 512, op="swiglu",
                                                                                         **opts)


@pytest.mark.parametrize("E,M,K,N", [(64, 16384, 1024, 2688), (32, 32768, 6144, 4096), (64, 2048, 1024, 2688),
                                     (32, 512, 6144, 2048)])
def test_otherwise_as_the_forward_products(E, M, K, N):
    # dgrad with K and N exchanged; eight epilogue warps
    assert rgg.rgg_plan(E, M, K, N, op="dgrad") == dict(rgg.rgg_plan(E, M, N, K), threads=320)
    assert rgg.rgg_plan(E, M, K, N, op="swiglu_backward") == rgg.rgg_plan(E, M, K, N, op="swiglu")


def test_refusals():
    for kw in (dict(K=12), dict(N=100), dict(M_tot=-1), dict(E=0)):
        args = dict(E=4, M_tot=256, K=256, N=512)
        args.update(kw)
        for op in ("dgrad", "swiglu_backward"):
            with pytest.raises(rgg.RggError) as ei:
                rgg.rgg_plan(**args, op=op)
            assert ei.value.status == rgg.RGG_ERR_INVALID_ARG
    opt, _ = rgg._options(op=7)
    assert rgg.load_library().rgg_plan(0, 0, 4, 256, 256, 512, opt, rgg._PlanInfo()) == rgg.RGG_ERR_INVALID_ARG
    with pytest.raises(rgg.RggError):
        rgg.rgg_plan(4, 256, 256, 512, op="swiglu_backward", bn=192)
