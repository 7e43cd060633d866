"""Experts' weights past twice the last-level cache, whose lone row tiles are read with a hint: the
same bits as the same rows with the live experts' weights alone, below that size and without it.
64- and 128-row tiles, both activations' formats, types and functions, experts of one tile and of
several; and one expert whose codes end near 2^31 bytes."""
import pytest
import torch
from scipy.special import ndtr

import mixture_experts_routing_top_amd as moe
from oracle import mx as om
from test_gpu_mx import _f64, _rows, _sums, _table, _wide

pytestmark = pytest.mark.gpu

E, H, I = 160, 2048, 2048


def _bytes(experts, act):
    return experts * H * I * (3 if act == "swiglu" else 2) * 17 / 32


@pytest.mark.parametrize("act,fmt,dtype", [("swiglu", "fp6", torch.bfloat16), ("swiglu", "fp4", torch.float32),
                                           ("gelu", "fp6", torch.float32), ("gelu", "fp4", torch.bfloat16)])
@pytest.mark.parametrize("rows", [64, 128])
def test_lone_tiles_past_the_cache(rows, act, fmt, dtype):
    if rows == 128:   # more than 64 rows an expert over all 160, and fewer than 2^19 / H over the 76 that have rows
        live = list(range(3, 155, 2))
        counts = [128, 100, 70, 257, 129][:5] * 15 + [200]
    else:
        live, counts = [3, 50, 51, 159], [7, 64, 90, 30]
    M = sum(counts)
    assert (M // E > 64) == (rows == 128) and (64 < M // len(live) < 2 ** 19 // H) == (rows == 128) and M > 24
    assert _bytes(E, act) > 2 ** 29 >= _bytes(len(live), act)
    gen = torch.Generator(device="cuda").manual_seed(rows)
    raw = lambda n, k: (torch.randint(0, 256, (E, n, k // 2), generator=gen, device="cuda", dtype=torch.uint8),  # noqa: E731
                        torch.randint(116, 121, (E, n, k // 32), generator=gen, device="cuda", dtype=torch.uint8))
    wts = [raw(I, H), raw(I, H) if act == "swiglu" else None, raw(H, I)]
    few = [None if w is None else tuple(t[live].contiguous() for t in w) for w in wts]
    x = _rows((M, H), dtype, 3)
    all_counts = [0] * E
    for e, c in zip(live, counts):
        all_counts[e] = c
    y = moe.moe_mx_expert_ffn(x, *_table(all_counts), *wts, act, fmt)
    assert bool(y.isfinite().all())
    assert torch.equal(y, moe.moe_mx_expert_ffn(x, *_table(counts), *few, act, fmt))


@pytest.mark.parametrize("M", [5, 30])   # the stream, and 64-row tiles
@pytest.mark.parametrize("wide", ["H", "I"])
def test_codes_that_end_near_2_31_bytes(M, wide):
    """GELU's two matrices of 2.11e9 bytes of codes, zero but for 128 rows and columns at either end: as the small
    matrices of these alone.  x holds values of e2m3 at scale 1 and the weights have one scale, so that z is exact in any
    order, and Q(h) the same; y's sums are off by E of the other tests."""
    big, side, n = 32256, 130944, 128
    h, i = (side, big) if wide == "H" else (big, side)
    assert 0x7d000000 < h * i // 2 < 0x7e000000 and h % 128 == i % 128 == 0
    gen = torch.Generator(device="cuda").manual_seed(M)
    at = lambda size: torch.cat([torch.arange(n), torch.arange(size - n, size)]).cuda()  # noqa: E731
    wts, few = [], []
    for rows, cols in ((i, h), (h, i)):
        q = torch.randint(0, 256, (2 * n, n), generator=gen, device="cuda", dtype=torch.uint8)
        codes = torch.zeros((rows, cols // 2), dtype=torch.uint8, device="cuda")
        scale = torch.full((rows, cols // 32), 120, dtype=torch.uint8, device="cuda")
        codes[at(rows), :n // 2], codes[at(rows), -(n // 2):] = q[:, :n // 2], q[:, n // 2:]
        few.append((q[None], torch.full((1, 2 * n, n // 16), 120, dtype=torch.uint8, device="cuda")))
        wts.append((codes[None], scale[None]))
    xs = torch.from_numpy(om.GRID["fp6"]).float().cuda()[torch.randint(0, 32, (M, 2 * n), generator=gen, device="cuda")]
    xs[:, ::32] = -7.5
    x = torch.zeros((M, h), device="cuda")
    x[:, :n], x[:, -n:] = xs[:, :n], xs[:, n:]
    table = _table([M])
    y = moe.moe_mx_expert_ffn(x, *table, wts[0], None, wts[1], "gelu")
    assert not bool(y[:, n:-n].any())
    want = _f64(moe.moe_mx_expert_ffn(xs, *table, few[0], None, few[1], "gelu"))
    z = _f64(xs) @ _wide(few[0], 0).T
    bar = 2 * _sums(om.values(z * ndtr(z), "fp6"), _wide(few[1], 0))
    assert bool((abs(want).max(1) > 100 * bar.max(1)).all())
    assert bool((abs(_f64(y[:, at(h)]) - want) <= bar).all())
