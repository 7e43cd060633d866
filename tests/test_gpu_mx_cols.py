"""moe_mx_dequantize's cols: what the codes' bytes do not hold is refused, whatever the number."""
import pytest
import torch

import mixture_experts_routing_top_amd as moe

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", ["fp4", "fp6", "fp8"])
@pytest.mark.parametrize("width", [0, 1, 3])
@pytest.mark.parametrize("cols", [2 ** 61, 2 ** 62, 2 ** 63 - 1, 2 ** 60, 2 ** 40, 0, -1, -2 ** 61, -2 ** 63])
def test_cols_the_codes_do_not_hold(cols, width, fmt):
    q, s = (torch.zeros((3, n), dtype=torch.uint8, device="cuda") for n in (width, 1))
    with pytest.raises(ValueError, match="do not hold"):
        moe.moe_mx_dequantize(q, s, fmt, cols=cols)


def test_codes_of_nothing():
    q = torch.zeros((3, 0), dtype=torch.uint8, device="cuda")
    with pytest.raises(ValueError, match="do not hold"):
        moe.moe_mx_dequantize(q, q, "fp8")
    with pytest.raises(ValueError):
        moe.moe_mx_quantize(torch.zeros((3, 0), device="cuda"), "fp8")
