"""The Python binding of the few-token layer and the 4-bit weight calls, no GPU:
arguments that the C calls never see are refused by name."""
import pytest
import torch

import combine_moe_route_histogram_amd as M


@pytest.mark.parametrize("w", [[1.0] * 256, 1.0, "w"])
def test_mx_weights_that_are_no_tensor(w):
    mx = torch.zeros(136, dtype=torch.uint8)
    with pytest.raises(TypeError, match="w must be a torch.Tensor"):
        M.moe_mx_quantize(1, 32, 8, w, mx)
    with pytest.raises(TypeError, match="w must be a torch.Tensor"):
        M.moe_mx_dequantize(1, 32, 8, mx, w)
