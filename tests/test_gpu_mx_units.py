"""Large calls of moe_mx_quantize and moe_mx_dequantize, which take two or four units of a row
a lane (from 2^19 units of eight values and 2^20 of four on): all bits as the oracle's, on
whole rows and rows that end inside a block, narrow and wide, and by a map with rows out of
range."""
import numpy as np
import pytest
import torch

import mixture_experts_routing_top_amd as moe
from oracle import mx as om
from test_gpu_mx import DTYPES, FMT, _f64, _np, _rows

pytestmark = pytest.mark.gpu

# K in whole blocks and the last thread block ragged; wide rows (more units than a thread block) that end inside a
# block and one value into it; narrow rows, one of several thread blocks
SHAPES = [(4101, 2080), (4099, 2079), (1031, 8193), (70001, 65), (140003, 33)]


def _chunks(R, K):
    """Rows that make calls below the limit, which the oracle's own tests cover."""
    step = max(1, 1_500_000 // K)
    return [(a, min(R, a + step)) for a in range(0, R, step)]


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("R,K", SHAPES)
def test_many_units(R, K, dtype, fmt):
    lane = 8 if dtype == torch.bfloat16 or fmt == "fp6" else 4
    assert R * -(-K // 32) * (32 // lane) >= 256 * 256 * 4 * (16 // lane)
    x = _rows((R, K), dtype, R)
    x[R // 2, K // 2], x[R - 1, K - 1] = float("nan"), float("inf")
    q, s = moe.moe_mx_quantize(x, fmt)
    back = {dt: moe.moe_mx_dequantize(q, s, fmt, dt, cols=K) for dt in DTYPES}
    for a, b in _chunks(R, K):
        cq, cs = moe.moe_mx_quantize(x[a:b], fmt)
        assert torch.equal(q[a:b], cq) and torch.equal(s[a:b], cs)
        for dt in DTYPES:
            part = moe.moe_mx_dequantize(cq, cs, fmt, dt, cols=K)
            assert torch.equal(back[dt][a:b].nan_to_num(9.0), part.nan_to_num(9.0))
    # the oracle at rows from all over
    some = np.unique(np.concatenate([np.arange(0, R, R // 97), [1, R // 2, R - 2, R - 1]]))
    rq, rs = om.quantize(_f64(x[torch.from_numpy(some).cuda()]), fmt)
    assert np.array_equal(_np(q)[some], rq) and np.array_equal(_np(s)[some], rs)
    want = np.nan_to_num(om.dequantize(rq, rs, fmt, K), nan=9.0)
    for dt in DTYPES:
        assert np.array_equal(np.nan_to_num(_f64(back[dt][torch.from_numpy(some).cuda()]), nan=9.0), want)


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("R,K,n", [(900, 2080, 4500), (1100, 2079, 4400), (40, 8193, 1100), (5000, 65, 80000)])
def test_many_units_by_rows(R, K, n, dtype, fmt):
    x = _rows((R, K), dtype, R)
    q, s = moe.moe_mx_quantize(x, fmt)
    rows = torch.randint(0, R, (n,), generator=torch.Generator().manual_seed(n), dtype=torch.int32)
    rows[::501], rows[7], rows[n - 1] = -1, R, 2 ** 31 - 1
    check = moe.new_check_word()
    out = moe.moe_mx_dequantize(q, s, fmt, dtype, cols=K, rows=rows.cuda(), check=check)
    with pytest.raises(moe.MoEError, match="outside"):
        moe.moe_check_device_error(check)
    ref = moe.moe_mx_dequantize(q, s, fmt, dtype, cols=K)
    assert np.array_equal(_f64(ref), om.dequantize(_np(q), _np(s), fmt, K))
    there = (rows >= 0) & (rows < R)
    want = torch.where(there.cuda()[:, None], ref[rows.clamp(0, R - 1).long().cuda()], torch.zeros((), dtype=dtype, device="cuda"))
    assert torch.equal(out, want)
    clean = moe.new_check_word()
    moe.moe_mx_dequantize(q, s, fmt, dtype, cols=K, rows=rows[there].cuda(), check=clean)
    assert moe.moe_check_device_error(clean) == 0
