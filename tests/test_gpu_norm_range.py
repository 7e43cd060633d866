"""The norm at the ends of float32's range: a row's sum is taken in float32."""
import pytest
import torch

import mixture_experts_routing_top_amd as moe

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("H", [64, 512, 1024, 2048, 4096, 8192, 16384])
def test_norm_of_rows_at_the_end_of_the_range(H, dtype):
    """A constant row whose elements add up to just below the largest float is normed
    exactly (H is a power of two: no sum is rounded) to the bias; one beyond gives NaN in
    that row alone, and the rows beside both keep their bits."""
    gen = torch.Generator().manual_seed(H)
    x = torch.randn((9, H), generator=gen).to(dtype).cuda()
    dy = torch.randn((9, H), generator=gen).to(dtype).cuda()
    w, b = torch.randn(H, generator=gen).cuda(), torch.randn(H, generator=gen).cuda()
    want, _ = moe.moe_layer_norm(x, w, b)
    grad = moe.moe_layer_norm_backward(dy, x, w, b)["d_x"]
    x[2] = 1.5 * 2.0 ** 127 / H       # adds up to 1.5 * 2^127
    x[5] = -1.5 * 2.0 ** 127 / H
    x[7] = 2.0 ** 128 / H             # adds up to 2^128
    y, _ = moe.moe_layer_norm(x, w, b)
    d = moe.moe_layer_norm_backward(dy, x, w, b)["d_x"]
    assert torch.equal(y[2], b.to(dtype)) and torch.equal(y[5], b.to(dtype))
    assert torch.all(torch.isfinite(d[[2, 5]].float()))
    assert torch.all(torch.isnan(y[7])) and torch.all(torch.isnan(d[7]))
    beside = [0, 1, 3, 4, 6, 8]
    assert torch.equal(y[beside], want[beside]) and torch.equal(d[beside], grad[beside])
