"""The 4-bit FFN's GELU by itself: pre-activations that float32 sums hold exactly, and a
down product that hands Q(h) out.

x is made of values that e2m3 (or e2m1) holds at scale 1, a weight row has one scale, so
z = Q(x) w is a whole multiple of its smallest step and below 2^24 of them: exact in any
order.  Down weights of ones on the diagonal return Q(h) in float32 unrounded.  What is
left is h = z Phi(z) in float32 beside float64.

The bar, in units of 2^-24 |h|, for z below 0, where h = -|z| R(t) 2^(-z^2 log2(e) / 2):
R's fit 2.5; t = 1 / (1 + p |z|) 1 and 2, R' t / R being 1 at most; its polynomial's last
steps and products 5; the exponent's two roundings 2 ln 2 log2(e) / 2 z^2 = z^2; the power
2; |z| times it, and the last rounding, 2: 14.5 + z^2, rounded up to 16 + z^2.  For z above 0
h is z less that, and off by no more.  Q(h) may differ from the oracle's only where h within
this bar rounds otherwise.  A power below 2^-126 may come as zero, |z| R being at most 1/2 where
z^2 passes 170: 2^-126 beside it.
"""
import numpy as np
import pytest
import torch
from scipy.special import ndtr

import mixture_experts_routing_top_amd as moe
from oracle import mx as om
from test_gpu_mx import X_FORMATS, _f64, _rounded_apart, _table, _wide

pytestmark = pytest.mark.gpu

H, I = 128, 512


def _codes(w, byte):
    """Codes and scales of w, e2m1 values, under the rows' scale bytes."""
    index = np.searchsorted(om.GRID["fp4"], np.abs(w)) + 8 * (w < 0)
    q = (index[:, 0::2] + 16 * index[:, 1::2]).astype(np.uint8)
    s = np.repeat(byte[:, None], w.shape[1] // 32, 1).astype(np.uint8)
    return torch.from_numpy(q)[None].cuda(), torch.from_numpy(s)[None].cuda()


# rows for the stream, and 64-, 128- and 256-row tiles (these from 2^19 rows * H on: more columns, of zeros)
@pytest.mark.parametrize("M,pad", [(16, 0), (60, 0), (125, 0), (500, 1920)])
@pytest.mark.parametrize("fmt", X_FORMATS)
def test_gelu_in_float32(fmt, M, pad):
    rng = np.random.default_rng(M)
    x = rng.choice(om.GRID[fmt], (M, H))
    x[:, ::32] = om.GRID[fmt][-1]
    w = rng.choice(om.GRID["fp4"][1:], (I, H))
    # of 32 columns in a row: mixed signs, or all negative; z from a hundredth to some tens
    mixed = np.arange(I) // 32 % 2 == 0
    w = np.where(mixed[:, None], w * rng.choice([-1.0, 1.0], (I, H)), -w)
    byte = np.where(mixed, 116 + np.arange(I) // 64 % 8, 114 + np.arange(I) // 64 % 8)
    z = x @ (w * 2.0 ** (byte[:, None] - 127.0)).T
    h = z * ndtr(z)
    eye = np.zeros((H + pad, I))
    y = np.zeros((M, I))
    xs = torch.from_numpy(np.pad(x, ((0, 0), (0, pad)))).float().cuda()
    up = _codes(np.pad(w, ((0, 0), (0, pad))), byte)
    assert np.array_equal(om.values(_f64(xs), fmt)[:, :H], x)
    for c in range(0, I, H):   # 128 columns of h at a time
        eye[:] = 0
        eye[np.arange(H), c + np.arange(H)] = 1
        down = _codes(eye, np.full(H + pad, 127))
        assert np.array_equal(_wide(down, 0), eye)
        y[:, c:c + H] = _f64(moe.moe_mx_expert_ffn(xs, *_table([M]), up, None, down, "gelu", fmt))[:, :H]
    apart = _rounded_apart(h, (16 + z * z) * 2.0 ** -24 * np.abs(h) + 2.0 ** -126, fmt)
    assert (apart > 0)[np.abs(h) > 2.0 ** -100].mean() < 0.01   # (the bar leaves a code open next to a border alone)
    off = np.abs(y - om.values(h, fmt))
    assert np.all(off <= apart), (int((off > apart).sum()), z[off > apart][:8])
