"""moe_combine_backward from rows kept in 8 bits, at the ends of float32's range: a block's
largest code lies in 224 .. 448 whatever its values are, and the sums are those of the
values, not of the codes.

The bar is the sum's own, n = 9 ceil(H / 512) + 12 roundings of 2^-24 of sum |d y|, and where
a product is subnormal half of 2^-149 for each term.
"""
import math

import numpy as np
import pytest
import torch

import mixture_experts_routing_top_amd as moe
from oracle import mx as om
from test_gpu_mx import DTYPES, _f64, _np, _places

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T", [5, 4100])   # a block a token, a wave a token
@pytest.mark.parametrize("d,y", [(2e36, 1.0), (3e37, 0.02), (2.0 ** 126, 2.0 ** -126), (2.0 ** -142, 2.0 ** 100),
                                 (2.0 ** -130, 2.0 ** 118)])
def test_sums_of_values_not_of_codes(dtype, T, d, y):
    k, H = 2, 72
    gen = torch.Generator().manual_seed(T)
    rnd = lambda *s: torch.rand(s, generator=gen) * 2 - 1  # noqa: E731
    d_out, rows = (rnd(T, H) * d).to(dtype).cuda(), (rnd(T * k, H) * y).to(dtype).cuda()
    rows[0] = y   # a block of one value: its code is a power of two
    kept = moe.moe_mx_quantize(rows, "fp8")
    yv = om.dequantize(_np(kept[0]), _np(kept[1]), "fp8", H)
    inv, w = _places(T, k, T * k, 1).cuda(), torch.ones((T, k), device="cuda")
    _, d_w = moe.moe_combine_backward(d_out, kept, inv, w)
    terms = _f64(d_out)[:, None, :] * yv[_np(inv)]
    assert np.abs(terms).sum(-1).max() < 3e38
    bar = (9 * math.ceil(H / 512) + 12) * 2.0 ** -24 * np.abs(terms).sum(-1) + H * 2.0 ** -150
    assert np.all(np.abs(_f64(d_w) - terms.sum(-1)) <= bar)
    # at the values that the blocks stand for, the form on rows in the dtype sums the same (bf16 holds them here too)
    back = moe.moe_mx_dequantize(*kept, "fp8", dtype)
    if np.array_equal(_f64(back), yv):
        assert torch.equal(d_w, moe.moe_combine_backward(d_out, back, inv, w)[1])
