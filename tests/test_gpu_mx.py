"""Microscaled blocks, the 4-bit expert FFN and the combine's gradient against the
float64 oracle.

Codes and scales are compared bit for bit (powers of two and one rounding, which
float64 does the same), the values that come back too: they are exact in float32.

FFN tolerances.  The products of e2m1 by e2m1 or e2m3 are exact; their sums take at
most K / 8 + K / 64 float32 additions in a row, and whether these round or cut each
is off by at most 2^-23 of the sum of the magnitudes: E(a, w) = K / 6 2^-23 sum_k
|a_k w_k|.  h = act(g, u) follows: |silu'| <= 1.1 and |gelu'| <= 1.13, so dh = 1.13
(E_g |u| + |silu(g)| E_u) + 1.1 E_g E_u, + 2^-20 |h| for the activation in float32
(the fast exponential's argument g log2 e is off by 2^-24 |g|, for |g| <= 8 some
2^-20; beyond, silu(g) is g or next to nothing).  Q(h) may differ from the oracle's
where h +- dh rounds differently, by that difference (the whole block where its scale
may differ); y by the sum of these times |Wd|, plus E(Q(h), Wd), plus half a step of
its type.

combine_backward: d_y is one float32 product, rounded once: 2^-24 and half a step of
the type.  d_w's sum goes over 9 roundings a chunk of eight and lane, ceil(H / 512)
chunks, then 6 + 4: n = 9 ceil(H / 512) + 12 times 2^-24 times the sum of |d y|.
"""
import math

import numpy as np
import pytest
import torch

import mixture_experts_routing_top_amd as moe
from oracle import mx as om

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
FMT = ["fp4", "fp6", "fp8"]
X_FORMATS = ["fp6", "fp4"]
DTYPES = [torch.float32, torch.bfloat16]


def _f64(t):
    return t.detach().double().cpu().numpy()


def _np(t):
    return t.detach().cpu().numpy()


def _rows(shape, dtype, seed, scale=1.0):
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn(shape, generator=gen) * scale
    x[..., shape[-1] // 3] *= 30.0
    return x.to(dtype).cuda()


def _same_blocks(x, fmt):
    q, s = moe.moe_mx_quantize(x, fmt)
    rq, rs = om.quantize(_f64(x), fmt)
    assert q.shape == rq.shape and s.shape == rs.shape
    assert np.array_equal(_np(s), rs)
    assert np.array_equal(_np(q), rq)
    return q, s


# ----------------------------------------------------------------- quantised rows
@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shape", [(1, 1), (1, 31), (3, 32), (5, 33), (9, 7), (7, 100), (2, 4095), (130, 256), (3, 2, 65),
                                   (2100, 1056), (64,)])
def test_quantize_is_the_oracles(fmt, dtype, shape):
    q, s = _same_blocks(_rows(shape, dtype, sum(shape)), fmt)
    for dt in DTYPES:
        back = moe.moe_mx_dequantize(q, s, fmt, dt, cols=shape[-1])
        assert back.shape == shape and back.dtype == dt
        assert np.array_equal(_f64(back), om.dequantize(_np(q), _np(s), fmt, shape[-1]))


@pytest.mark.parametrize("fmt", FMT)
def test_quantize_borders(fmt):
    """Ties of every step, block maxima on both sides of where the scale changes, zeros, the smallest and largest floats."""
    grid = om.GRID[fmt]
    ties = np.concatenate([grid, (grid[1:] + grid[:-1]) / 2, np.nextafter((grid[1:] + grid[:-1]) / 2, 0, dtype=np.float32)])
    rows = []
    for e in (-130, -126, -20, 0, 3, 100, 118):
        for lead in (grid[-1], grid[-1] * 0.51):
            v = np.concatenate([np.full((len(ties) + 30) // 31, 0.0)[:, None] + lead,
                                np.resize(ties, ((len(ties) + 30) // 31, 31))], 1)
            rows.append(np.minimum(v, lead) * 2.0 ** e)
    border = {"fp4": 7.0, "fp6": 7.75, "fp8": 464.0}[fmt]
    for e in (-134, -127, -100, 0, 100, 115):
        for top in (border, np.nextafter(np.float32(border), np.float32(0)), np.nextafter(np.float32(border), np.float32(1e9)),
                    border / 2, grid[-1], 2 * border):
            v = np.resize(ties, 32) * 0.5
            v[5] = float(top)
            rows.append(np.minimum(np.abs(v), float(top))[None] * 2.0 ** e)
    rows.append(np.zeros((1, 32)))
    rows.append(np.full((1, 32), -0.0))
    rows.append(np.full((1, 32), 2.0 ** -149))
    rows.append(np.full((1, 32), float(np.finfo(np.float32).max)))
    x = np.concatenate(rows)
    x[:, ::2] *= -1
    _same_blocks(torch.from_numpy(x.astype(np.float32)).cuda(), fmt)
    _same_blocks(torch.from_numpy(x.astype(np.float32)).bfloat16().cuda(), fmt)


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("dtype", DTYPES)
def test_not_finite_blocks(fmt, dtype):
    x = _rows((6, 128), dtype, 3)
    x[1, 40], x[2, 127], x[4, 0] = math.nan, math.inf, -math.inf
    check = moe.new_check_word()
    q, s = moe.moe_mx_quantize(x, fmt, check=check)
    with pytest.raises(moe.MoEError, match="quantised block"):
        moe.moe_check_device_error(check)
    bad = np.zeros((6, 4), bool)
    bad[1, 1] = bad[2, 3] = bad[4, 0] = True
    assert np.array_equal(_np(s) == 255, bad)
    _same_blocks(x, fmt)
    back = _f64(moe.moe_mx_dequantize(q, s, fmt, dtype))
    assert np.array_equal(np.isnan(back), np.repeat(bad, 32, 1))
    clean = moe.new_check_word()
    moe.moe_mx_quantize(x[3:4], fmt, check=clean)
    assert moe.moe_check_device_error(clean) == 0


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("R,K", [(5, 64), (40, 1000), (3, 33)])
def test_dequantize_by_rows(fmt, dtype, R, K):
    x = _rows((R, K), torch.float32, R + K)
    q, s = moe.moe_mx_quantize(x, fmt)
    rows = torch.tensor([R - 1, 0, 0, -1, 2, R, 1, -2 ** 31, 2 ** 31 - 1] + list(range(R)), dtype=torch.int32).cuda()
    check = moe.new_check_word()
    out = _f64(moe.moe_mx_dequantize(q, s, fmt, dtype, cols=K, rows=rows, check=check))
    ref = om.dequantize(_np(q), _np(s), fmt, K)
    for i, r in enumerate(rows.tolist()):
        assert np.array_equal(out[i], ref[r] if 0 <= r < R else np.zeros(K))
    with pytest.raises(moe.MoEError):
        moe.moe_check_device_error(check)
    none = moe.moe_mx_dequantize(q, s, fmt, dtype, cols=K, rows=rows[:0])
    assert none.shape == (0, K)


def test_every_code_and_scale():
    """All codes under all scales, as float32 and bf16 hold them (subnormal values rounded once)."""
    for fmt in FMT:
        n = om.BITS[fmt]
        codes = np.resize(np.arange(1 << n, dtype=np.uint8), (max(1, (1 << n) // 32), 32))
        bits = np.unpackbits(codes[..., None], axis=-1, bitorder="little")[..., :n].reshape(len(codes), -1)
        q = np.tile(np.packbits(bits, axis=-1, bitorder="little"), (256, 1))
        s = np.repeat(np.arange(256, dtype=np.uint8), len(codes))[:, None]
        ref = om.dequantize(q, s, fmt)
        for dt in DTYPES:
            out = moe.moe_mx_dequantize(torch.from_numpy(q).cuda(), torch.from_numpy(s).cuda(), fmt, dt)
            want = torch.from_numpy(ref).float().to(dt)
            a, b = _f64(out), want.double().numpy()
            assert np.array_equal(np.isnan(a), np.isnan(b))
            assert np.array_equal(a[~np.isnan(a)], b[~np.isnan(b)])


def test_quantize_past_32_bit_offsets():
    R, K = 525000, 4100
    x = torch.empty((R, K), dtype=torch.bfloat16, device="cuda")
    x.fill_(1.0)
    x[-3:] = _rows((3, K), torch.bfloat16, 1)
    assert x.numel() > 2 ** 31
    q, s = moe.moe_mx_quantize(x, "fp8")
    rq, rs = moe.moe_mx_quantize(x[-3:], "fp8")
    assert torch.equal(q[-3:], rq) and torch.equal(s[-3:], rs)
    rows = torch.tensor([R - 1, 0, R - 3], dtype=torch.int32, device="cuda")
    back = moe.moe_mx_dequantize(q, s, "fp8", torch.bfloat16, rows=rows)
    ref = moe.moe_mx_dequantize(rq, rs, "fp8", torch.bfloat16)
    assert torch.equal(back[0], ref[2]) and torch.equal(back[2], ref[0]) and bool((back[1] == 1).all())


# ------------------------------------------------------------- the combine's gradient
def _places(T, k, M, seed):
    gen = torch.Generator().manual_seed(seed)
    return torch.randperm(M, generator=gen)[:T * k].view(T, k).int()


@pytest.mark.parametrize("kept", [False, True])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,k,H,more", [(1, 1, 8, 0), (1, 8, 8192, 0), (61, 2, 1024, 3), (7, 3, 72, 0), (33, 6, 520, 5),
                                        (4096, 2, 40, 0), (5003, 5, 64, 7)])
def test_combine_backward(kept, dtype, T, k, H, more):
    M = T * k + more
    d_out, y = _rows((T, H), dtype, T + H, 0.01), _rows((M, H), dtype, k + H)
    inv = _places(T, k, M, T).cuda()
    w = torch.softmax(torch.randn((T, k), generator=torch.Generator().manual_seed(5)), 1).cuda()
    given = moe.moe_mx_quantize(y, "fp8") if kept else y
    yv = om.dequantize(_np(given[0]), _np(given[1]), "fp8", H) if kept else _f64(y)
    filled = torch.full((M, H), 7.0, dtype=dtype, device="cuda")
    d_y, d_w = moe.moe_combine_backward(d_out, given, inv, w, d_y=filled)
    assert d_y is filled
    ref_y, ref_w = om.combine_backward(_f64(d_out), yv, _np(inv), _f64(w))
    left = np.isnan(ref_y)
    got = _f64(d_y)
    assert np.all(got[left] == 7.0)
    ref = np.where(left, 0.0, ref_y)
    assert np.all(np.abs(got - ref)[~left] <= ((HALF[dtype] + 2 * U) * np.abs(ref) + 2.0 ** -133)[~left])
    mag = np.stack([(np.abs(_f64(d_out)) * np.abs(yv[_np(inv)[:, i]])).sum(1) for i in range(k)], 1)
    assert np.all(np.abs(_f64(d_w) - ref_w) <= (9 * math.ceil(H / 512) + 12) * U * mag + 1e-37)


def test_combine_backward_is_the_combines_gradient():
    """Against differences of moe_combine along random directions: it is linear in both."""
    T, k, H = 40, 3, 64
    M = T * k
    y, inv = _rows((M, H), torch.float32, 1), _places(T, k, M, 2).cuda()
    gen = torch.Generator().manual_seed(3)
    w, d_out = torch.rand((T, k), generator=gen).cuda(), torch.randn((T, H), generator=gen).cuda()
    d_y, d_w = moe.moe_combine_backward(d_out, y, inv, w)
    dy, dw = torch.randn((M, H), generator=gen).cuda(), torch.randn((T, k), generator=gen).cuda()
    for a, b, lin in ((y + dy, w, (_f64(d_y) * _f64(dy)).sum()), (y, w + dw, (_f64(d_w) * _f64(dw)).sum())):
        diff = (_f64(moe.moe_combine(a, inv, b)) - _f64(moe.moe_combine(y, inv, w))) * _f64(d_out)
        # each output is off by (k + 1) U of its terms, and so is the gradient's side
        mag = sum((np.abs(_f64(v)[_np(inv)[:, i]]) * np.abs(_f64(u)[:, i:i + 1]) * np.abs(_f64(d_out))).sum()
                  for v, u in ((a, b), (y, w)) for i in range(k))
        assert abs(diff.sum() - lin) <= 24 * U * mag


def test_combine_backward_skips_rows_out_of_range():
    T, k, H = 9, 2, 64
    M = T * k
    y, d_out, w = _rows((M, H), torch.float32, 1), _rows((T, H), torch.float32, 2), torch.ones((T, k), device="cuda")
    inv = _places(T, k, M, 1)
    inv[3, 1], inv[5, 0], inv[8, 0] = -1, M, 2 ** 31 - 1
    check = moe.new_check_word()
    d_y, d_w = moe.moe_combine_backward(d_out, y, inv.cuda(), w, d_y=torch.zeros((M, H), device="cuda"), check=check)
    with pytest.raises(moe.MoEError, match="inv_pos"):
        moe.moe_check_device_error(check)
    assert d_w[3, 1] == 0 and d_w[5, 0] == 0 and d_w[8, 0] == 0
    ref, _ = om.combine_backward(_f64(d_out), _f64(y), inv.numpy(), _f64(w))
    assert np.array_equal(_f64(d_y), np.nan_to_num(ref))


def test_combine_backward_of_nothing():
    e = torch.empty((0, 64), device="cuda")
    d_y, d_w = moe.moe_combine_backward(e, e, torch.empty((0, 2), dtype=torch.int32, device="cuda"),
                                        torch.empty((0, 2), device="cuda"))
    assert d_y.shape == (0, 64) and d_w.shape == (0, 2)


# ------------------------------------------------------------------- the experts' FFN
def _weights(E, N, K, seed):
    gen = torch.Generator().manual_seed(seed)
    return moe.moe_mx_quantize((torch.randn((E, N, K), generator=gen) / math.sqrt(K)).cuda(), "fp4")


def _wide(w, e):
    return om.dequantize(_np(w[0][e]), _np(w[1][e]), "fp4")


def _table(counts, experts=None, max_slots=None):
    experts = list(range(len(counts))) if experts is None else experts
    n, m = len(counts), max_slots or len(counts)
    off = [0]
    for c in counts:
        off.append(off[-1] + c)
    off += [off[-1]] * (m - n)
    dev = dict(dtype=torch.int32, device="cuda")
    return torch.tensor(off, **dev), torch.tensor(experts + [0] * (m - n), **dev), torch.tensor([n], **dev)


def _rounded_apart(h, dh, fmt):
    """How far the quantised h may be from the oracle's for h within dh."""
    lo, hi = np.sign(h) * np.maximum(np.abs(h) - dh, 0.0), h + np.sign(h) * dh
    q = om.values(h, fmt)
    b = np.abs(om._blocks(h)).max(-1)
    bh, bl = np.abs(om._blocks(hi)).max(-1), np.abs(om._blocks(lo)).max(-1)
    s = om.scale_bytes(b, fmt)
    moved = (om.scale_bytes(bh, fmt) != s) | (om.scale_bytes(bl, fmt) != s)
    # in the nominal scale: the nearest values of lo and hi
    scale = np.repeat(2.0 ** (s - 127.0), om.BLOCK, -1).reshape(h.shape)
    last = len(om.GRID[fmt]) - 1
    grid = lambda v: np.sign(v) * om.GRID[fmt][np.minimum(om._nearest(np.abs(v) / scale, fmt), last)] * scale  # noqa: E731
    apart = np.maximum(np.abs(grid(lo) - q), np.abs(grid(hi) - q))
    # a scale that may be twice or half: every value of the block by half a step of either
    top = om.GRID[fmt][-1] - om.GRID[fmt][-2]
    whole = np.repeat(moved, om.BLOCK, -1).reshape(h.shape)
    return np.where(whole, np.maximum(apart, 2 * top * scale), apart)


def _sums(a, w):
    """E(a, w) of the header."""
    return a.shape[1] / 6 * 2.0 ** -23 * (np.abs(a) @ np.abs(w).T)


def _assert_ffn(y, xv, rows, table, wts, act, fmt, dtype):
    """xv: the quantised x in float64; rows: the row of x that each row takes (None: zero)."""
    got = _f64(y)
    off, experts, n = (_np(t) for t in table)
    for s in range(int(n[0])):
        lo, hi = off[s], off[s + 1]
        if lo == hi:
            continue
        wg, wd = _wide(wts[0], experts[s]), _wide(wts[2], experts[s])
        wu = None if wts[1] is None else _wide(wts[1], experts[s])
        a = np.stack([xv[r] if r is not None else np.zeros(xv.shape[1]) for r in rows[lo:hi]])
        h, ref = om.ffn(a, wg, wu, wd, fmt)
        eg = _sums(a, wg)
        if wu is None:
            dh = 1.13 * eg
        else:
            g, u, eu = a @ wg.T, a @ wu.T, _sums(a, wu)
            dh = 1.13 * (eg * np.abs(u) + np.abs(om.act(g, 1.0)) * eu) + 1.1 * eg * eu
        dh = dh + 2.0 ** -20 * np.abs(h)
        tol = _rounded_apart(h, dh, fmt) @ np.abs(wd).T + _sums(om.values(h, fmt), wd)
        tol = tol + HALF[dtype] * (np.abs(ref) + tol) + 1e-37
        err = np.abs(got[lo:hi] - ref)
        assert np.all(err <= tol), (s, float((err / tol).max()))


CASES = [
    # counts, H, I: few rows (single ones, 16, 17; short and long sums, many columns), the edges of 64-, 128- and
    # 256-row tiles, odd counts of K steps, columns that do not fill a tile
    ([1], 128, 128),
    ([1, 0, 2, 0], 256, 384),
    ([16, 17, 1, 0, 33], 640, 128),
    ([40, 64, 65, 1, 0], 384, 256),
    ([130, 128, 1, 120], 512, 384),
    ([300, 256, 511, 0], 128, 640),
    ([257], 1152, 128),
    ([3, 0, 1], 2176, 2048),
    ([16] * 8, 2048, 128),
    ([126, 125, 130, 123], 2944, 384),
    ([300, 256, 511, 0], 2176, 640),
    ([257, 300], 2048, 128),
    ([16, 0, 7, 1], 640, 256),
    ([18, 5], 2048, 128),
    ([1, 0, 3, 1] * 8, 256, 384),
    ([64, 50, 65, 77], 1152, 256),
]


@pytest.mark.parametrize("fmt", X_FORMATS)
@pytest.mark.parametrize("act", ["swiglu", "gelu"])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("counts,H,I", CASES)
def test_ffn(fmt, act, dtype, counts, H, I):
    E, M = len(counts), sum(counts)
    x = _rows((M, H), dtype, M + H)
    wts = (_weights(E, I, H, 1), _weights(E, I, H, 2) if act == "swiglu" else None, _weights(E, H, I, 3))
    table = _table(counts)
    check = moe.new_check_word()
    y = moe.moe_mx_expert_ffn(x, *table, *wts, act=act, x_format=fmt, check=check)
    assert y.dtype == dtype and moe.moe_check_device_error(check) == 0
    _assert_ffn(y, om.values(_f64(x), fmt), list(range(M)), table, wts, act, fmt, dtype)


@pytest.mark.parametrize("act,fmt,dtype", [("swiglu", "fp6", torch.bfloat16), ("gelu", "fp4", torch.float32),
                                           ("gelu", "fp6", torch.bfloat16), ("swiglu", "fp4", torch.float32)])
def test_ffn_whole_and_quartered_tiles(act, fmt, dtype):
    """256-row tiles, 9 of rows: 261 of SwiGLU's h (a round of 256, the rest in quarters), 135 of GELU's (the last
    columns half a tile) and 144 of y."""
    counts, H, I = [300, 300, 300, 300, 140], 4096, 3712
    wts = (_weights(5, I, H, 1), _weights(5, I, H, 2) if act == "swiglu" else None, _weights(5, H, I, 3))
    x = _rows((sum(counts), H), dtype, 5)
    table = _table(counts)
    y = moe.moe_mx_expert_ffn(x, *table, *wts, act, fmt)
    _assert_ffn(y, om.values(_f64(x), fmt), range(sum(counts)), table, wts, act, fmt, dtype)


@pytest.mark.parametrize("act", ["swiglu", "gelu"])
def test_ffn_of_experts_past_the_cache(act):
    """160 experts, 1.07 GB of them (GELU 0.71), of which four have rows (one and two tiles): as the four alone."""
    E, H, I, counts, live = 160, 2048, 2048, [7, 0, 90, 30], [3, 50, 51, 159]
    gen = torch.Generator(device="cuda").manual_seed(1)
    raw = lambda n, k: (torch.randint(0, 256, (E, n, k // 2), generator=gen, device="cuda", dtype=torch.uint8),  # noqa: E731
                        torch.randint(116, 121, (E, n, k // 32), generator=gen, device="cuda", dtype=torch.uint8))
    wts = [raw(I, H), raw(I, H) if act == "swiglu" else None, raw(H, I)]
    few = [None if w is None else tuple(t[live].contiguous() for t in w) for w in wts]
    x = _rows((sum(counts), H), torch.bfloat16, 3)
    off, experts, n = _table(counts)
    all_counts = [0] * E
    for e, c in zip(live, counts):
        all_counts[e] = c
    y = moe.moe_mx_expert_ffn(x, *_table(all_counts), *wts, act)
    assert bool(y.isfinite().all()) and torch.equal(y, moe.moe_mx_expert_ffn(x, off, experts, n, *few, act))


@pytest.mark.parametrize("fmt", X_FORMATS)
@pytest.mark.parametrize("counts", [[3, 0, 5, 9], [30, 2, 21, 50], [70, 2, 31, 90], [60, 100, 70, 50], [200, 150, 300, 129]])
def test_ffn_gathers_rows(fmt, counts):
    """Rows by a map: repeated, unordered, out of range (zero rows); replica slots and spare slots; y whole."""
    M, T = sum(counts), 50
    H, I, E = 2176 if M > 300 else 384, 256, 2
    x = _rows((T, H), torch.bfloat16, 4)
    src = torch.randint(0, T, (M,), generator=torch.Generator().manual_seed(1)).int()
    src[1], src[M // 2], src[M - 1] = -1, T, 2 ** 31 - 1
    wts = (_weights(E, I, H, 1), _weights(E, I, H, 2), _weights(E, H, I, 3))
    table = _table(counts, [0, 0, 1, 1], 7)
    y = moe.moe_mx_expert_ffn(x, *table, *wts, x_format=fmt, row_src=src.cuda())
    rows = [r if 0 <= r < T else None for r in src.tolist()]
    _assert_ffn(y, om.values(_f64(x), fmt), rows, table, wts, "swiglu", fmt, torch.bfloat16)


@pytest.mark.parametrize("fmt", X_FORMATS)
@pytest.mark.parametrize("counts", [[5, 4], [60, 50], [150, 120], [260, 270]])
def test_ffn_rows_stand_alone(fmt, counts):
    """A NaN in x leaves the other rows as they were; a row of zeros gives zeros."""
    M = sum(counts)
    H, I = 256 if M < 500 else 2176, 128
    wts = (_weights(2, I, H, 1), _weights(2, I, H, 2), _weights(2, H, I, 3))
    x = _rows((M, H), torch.bfloat16, 8)
    x[2] = 0
    table = _table(counts)
    y = moe.moe_mx_expert_ffn(x, *table, *wts, x_format=fmt)
    assert bool((y[2] == 0).all())
    x[1, 7], x[M - 2, 200] = math.nan, math.inf
    check = moe.new_check_word()
    z = moe.moe_mx_expert_ffn(x, *table, *wts, x_format=fmt, check=check)
    with pytest.raises(moe.MoEError, match="quantised block"):
        moe.moe_check_device_error(check)
    bad = torch.zeros(M, dtype=torch.bool, device="cuda")
    bad[1] = bad[M - 2] = True
    assert bool(z[bad].isnan().all()) and torch.equal(z[~bad], y[~bad])


def test_ffn_of_no_rows():
    wts = (_weights(2, 128, 128, 1), _weights(2, 128, 128, 2), _weights(2, 128, 128, 3))
    y = moe.moe_mx_expert_ffn(torch.empty((0, 128), device="cuda"), *_table([0, 0]), *wts)
    assert y.shape == (0, 128)


def test_ffn_flags_a_broken_slot_table():
    """Ranges are clamped to the rows, experts outside [0, E) skipped."""
    H = I = 128
    wts = (_weights(2, I, H, 1), _weights(2, I, H, 2), _weights(2, H, I, 3))
    x = _rows((20, H), torch.bfloat16, 8)
    for off, experts, n in (([0, 10, 25], [0, 1], 2), ([-4, 10, 20], [0, 1], 2), ([0, 12, 8], [0, 1], 2), ([0, 10, 20], [0, 2], 2),
                            ([0, 10, 20], [-1, 1], 2), ([0, 10, 20], [0, 1], 3), ([0, 10, 20], [0, 1], -1)):
        dev = dict(dtype=torch.int32, device="cuda")
        check = moe.new_check_word()
        moe.moe_mx_expert_ffn(x, torch.tensor(off, **dev), torch.tensor(experts, **dev), torch.tensor([n], **dev), *wts,
                              check=check)
        with pytest.raises(moe.MoEError, match="slot table"):
            moe.moe_check_device_error(check)


def test_ffn_on_streams_and_in_graphs():
    """Two calls on two streams with workspaces of their own; a captured call replayed between eager ones."""
    H, I, counts = 512, 256, [30, 50, 9]
    M = sum(counts)
    wts = (_weights(3, I, H, 1), _weights(3, I, H, 2), _weights(3, H, I, 3))
    table = _table(counts)
    xs = [_rows((M, H), torch.bfloat16, s) for s in (1, 2)]
    want = [moe.moe_mx_expert_ffn(x, *table, *wts) for x in xs]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [moe.moe_mx_expert_ffn(x, *table, *wts, stream=s) for x, s in zip(xs, streams)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    x, y = xs[0].clone(), torch.empty_like(xs[0])
    ws = torch.empty(moe.moe_mx_expert_ffn_workspace_bytes(M, H, I, 3), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q, s = moe.moe_mx_quantize(x, "fp8")
        back = moe.moe_mx_dequantize(q, s, "fp8", torch.bfloat16)
        moe.moe_mx_expert_ffn(x, *table, *wts, y_perm=y, workspace=ws)
    for r in (1, 0, 1):
        x.copy_(xs[r])
        y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want[r])
        assert torch.equal(back, moe.moe_mx_dequantize(*moe.moe_mx_quantize(xs[r], "fp8"), "fp8", torch.bfloat16))
