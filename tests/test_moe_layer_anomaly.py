"""moe_layer.py under autograd's anomaly mode, on the CPU with plain sums for the kernels."""
import torch

from ragged_grouped_gemm_02_gb300 import moe_layer
from test_moe_layer import _combine_backward, _inputs, plain  # noqa: F401 (a fixture)


def test_rows_of_no_choice_under_anomaly_mode(plain, monkeypatch):  # noqa: F811
    # a gradient that the call leaves unwritten holds whatever lay in its memory: NaN here
    def backward(dout, Y, position, weights, dY, dweights):
        dY = torch.full_like(Y, float("nan")) if dY is None else dY
        return _combine_backward(dout, Y, position, weights, dY, dweights)

    monkeypatch.setattr(moe_layer, "rgg_combine_backward", backward)
    _, Y, w, _, position = _inputs()
    assert bool((position < 0).any())

    def gradient():
        return torch.autograd.grad(moe_layer._Combine.apply(Y, position, w, False).sum(), Y)[0]

    rows = position[position >= 0].long()
    want = gradient()
    with torch.autograd.set_detect_anomaly(True):
        got = gradient()  # and raises no error
    assert torch.equal(got[rows], want[rows]) and bool(torch.isfinite(got).all())
