"""Arguments that moe_layer.py's functions with gradients refuse at the call, on the CPU."""
import pytest
import torch

from ragged_grouped_gemm_02_gb300 import moe_layer


@pytest.mark.parametrize("weights", [None, 1.0])
def test_combine_with_a_gradient_wants_weights(weights):
    # rgg_combine takes None, for sums without weights; its gradient has no such form
    Y = torch.zeros(6, 4, dtype=torch.bfloat16, requires_grad=True)
    with pytest.raises(TypeError, match="weights"):
        moe_layer.combine(Y, torch.zeros(3, 2, dtype=torch.int32), weights)
