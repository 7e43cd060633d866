"""Scales at the ends of their range.  x times 2^s beside weights times 2^-s gives the same
products, so the same bits of y, for every s that neither x nor the scale bytes leave; and a
weight block marked NaN makes NaN of its own outputs alone."""
import numpy as np
import pytest
import torch

import mixture_experts_routing_top_amd as moe
from oracle import mx as om
from test_gpu_mx import DTYPES, X_FORMATS, _f64, _rows, _table, _weights

pytestmark = pytest.mark.gpu

TILES = [([5], 128), ([40, 64], 384), ([130, 90], 256), ([300, 270], 2176)]   # the stream, 64-, 128- and 256-row tiles


@pytest.mark.parametrize("fmt", X_FORMATS)
@pytest.mark.parametrize("act", ["swiglu", "gelu"])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("counts,H", TILES)
def test_x_and_weights_by_inverse_powers(fmt, act, dtype, counts, H):
    E, M, I = len(counts), sum(counts), 128
    gen = torch.Generator().manual_seed(H)
    grid = torch.from_numpy(om.GRID[fmt]).float()
    x = grid[torch.randint(0, len(grid), (M, H), generator=gen)] * torch.sign(torch.randn((M, H), generator=gen))
    x[:, ::32] = grid[-1]
    wts = (_weights(E, I, H, 1), _weights(E, I, H, 2) if act == "swiglu" else None, _weights(E, H, I, 3))
    table = _table(counts)
    want = moe.moe_mx_expert_ffn(x.to(dtype).cuda(), *table, *wts, act, fmt)
    assert bool(want.isfinite().all()) and bool(want.any(1).all())
    both = [w for w in wts[:2] if w is not None]
    low, high = min(int(w[1].min()) for w in both), max(int(w[1].max()) for w in both)
    assert 100 < low and high <= 127
    for s in (-127, -126, -60, 60, low):
        moved = [None if w is None else (w[0], (w[1].int() - s).to(torch.uint8)) for w in wts[:2]]
        got = moe.moe_mx_expert_ffn((x * 2.0 ** s).to(dtype).cuda(), *table, *moved, wts[2], act, fmt)
        assert torch.equal(got, want), s


@pytest.mark.parametrize("fmt", X_FORMATS)
@pytest.mark.parametrize("counts,H", TILES)
def test_blocks_marked_nan(fmt, counts, H):
    """Of w_down: its column of y, in its expert's rows.  Of w_gate or w_up: a value of h and with it that block of h, so
    its expert's rows whole."""
    E, M, I = len(counts), sum(counts), 256
    wts = [_weights(E, I, H, 1), _weights(E, I, H, 2), _weights(E, H, I, 3)]
    x, table = _rows((M, H), torch.bfloat16, 5), _table(counts)
    want = moe.moe_mx_expert_ffn(x, *table, *wts, x_format=fmt)
    assert bool(want.isfinite().all())
    off = np.cumsum([0] + counts)
    for which in (0, 1, 2):
        for e in range(E):
            scale = wts[which][1].clone()
            row, block = scale.shape[1] - 3, scale.shape[2] - 1
            scale[e, row, block] = 255
            broken = list(wts)
            broken[which] = (wts[which][0], scale)
            y = moe.moe_mx_expert_ffn(x, *table, *broken, x_format=fmt)
            bad = np.zeros((M, H), bool)
            bad[off[e]:off[e + 1], slice(row, row + 1) if which == 2 else slice(None)] = True
            assert np.array_equal(np.isnan(_f64(y)), bad)
            good = torch.from_numpy(~bad).cuda()
            assert torch.equal(y[good], want[good])


@pytest.mark.parametrize("act", ["swiglu", "gelu"])
@pytest.mark.parametrize("fmt", X_FORMATS)
@pytest.mark.parametrize("counts,H", TILES)
def test_h_past_the_range(fmt, act, counts, H):
    """Sums or an h that float32 does not hold: that row of y is NaN, the others as they were, and x is clean."""
    E, M, I = len(counts), sum(counts), 128
    wts = (_weights(E, I, H, 1), _weights(E, I, H, 2) if act == "swiglu" else None, _weights(E, H, I, 3))
    x, table = _rows((M, H), torch.float32, 5), _table(counts)
    x[1] = 0
    want = moe.moe_mx_expert_ffn(x, *table, *wts, act, fmt)
    x[1] = 3e38 * torch.sign(x[2])
    check = moe.new_check_word()
    y = moe.moe_mx_expert_ffn(x, *table, *wts, act, fmt, check=check)
    assert moe.moe_check_device_error(check) == 0
    others = torch.arange(M, device="cuda") != 1
    assert bool(y[1].isnan().all()) and torch.equal(y[others], want[others])
