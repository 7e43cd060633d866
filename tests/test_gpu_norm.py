"""moe_layer_norm and moe_layer_norm_backward against the float64 oracle.

Tolerances, with u = 2^-24.  A row's sum in float32 goes over at most 16 values
a thread, 6 steps of a wave and 16 waves, or 32 values, 6 steps and 8 waves: n = 46
roundings at most (38 in the forward pass).  The mean's error is
made good by the sum of the deviations, which itself errs by n u mean|d|.  So
n^ = (x - mean) rstd errs by at most (n/2 + 8) u |n^| + 2 n u: y = n^ w + b by
64 u ((|n^| + 1) |w| + |b|), plus half a step of the type.  The deviations are
taken from a mean off by delta <= n u mean|x|, which the variance's correction
cancels at the cost of a factor 1 + (delta / sigma)^2.
d_x = rstd (g - c1 - n^ c2) has such errors in each term, c1 and c2 being means
over the row: 128 u rstd (|g| + mean|g| + (|n^| + 1) (mean|g n^| + mean|g|)),
plus half a step.  A column's sum over T rows adds at most T / 512 + 56 terms in
sequence: (64 + T / 512 + 56) u times the sum of |d_y| (|n^| + 1), plus half a
step.
"""
import math

import numpy as np
import pytest
import torch

import mixture_experts_routing_top_amd as moe
from oracle import operators as oo

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
TINY = 2.0 ** -133


def _rows(T, H, dtype, seed, scale=1.0, shift=0.25):
    gen = torch.Generator().manual_seed(seed)
    x = (torch.randn((T, H), generator=gen) + shift) * scale
    if H > 40:
        x[:, H // 3] *= 40.0     # a channel far larger than the others
    return x.to(dtype).cuda()


def _vec(H, dtype, seed, one):
    gen = torch.Generator().manual_seed(seed)
    return (one + 0.1 * torch.randn(H, generator=gen)).to(dtype).cuda()


def _f64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def _hat(x, eps):
    m = x.mean(1, keepdims=True)
    sd = np.sqrt(((x - m) ** 2).mean(1, keepdims=True) + eps)
    delta = 38 * U * np.abs(x).mean(1, keepdims=True)
    return (x - m) / sd, 1.0 / sd, 1.0 + (delta / sd) ** 2


def _assert_forward(y, x, w, b, eps, dtype):
    xd, wd, bd = _f64(x), _f64(w), _f64(b)
    ref = oo.layer_norm(xd, wd, bd, eps)
    hat, _, factor = _hat(xd, eps)
    aw = 1.0 if wd is None else np.abs(wd)
    ab = 0.0 if bd is None else np.abs(bd)
    tol = 64 * U * factor * ((np.abs(hat) + 1) * aw + ab) + HALF[dtype] * np.abs(ref) * 1.01 + TINY
    err = np.abs(_f64(y) - ref)
    assert np.all(err <= tol), float((err / tol).max())


def _assert_backward(d, dy, x, w, b, eps, skip, dtype):
    xd, gd, wd, sd = _f64(x), _f64(dy), _f64(w), _f64(skip)
    ref = oo.layer_norm_backward(gd, xd, wd, eps, sd)
    hat, rstd, factor = _hat(xd, eps)
    g = np.abs(gd if wd is None else gd * wd)
    mg, mgh = g.mean(1, keepdims=True), (g * np.abs(hat)).mean(1, keepdims=True)
    tol = 128 * U * factor * rstd * (g + mg + (np.abs(hat) + 1) * (mgh + mg)) + \
        (HALF[dtype] * 1.01 + U) * (np.abs(ref["d_x"]) + (0 if sd is None else U * np.abs(sd))) + TINY
    err = np.abs(_f64(d["d_x"]) - ref["d_x"])
    assert np.all(err <= tol), float((err / tol).max())
    T = xd.shape[0]
    n = 64 + T / 512 + 56
    for key, given, mass in (("d_weight", w, (np.abs(gd) * (np.abs(hat) + 1) * factor).sum(0)),
                             ("d_bias", b, np.abs(gd).sum(0))):
        if given is None:
            assert d[key] is None
            continue
        assert d[key].dtype == given.dtype
        tol = n * U * mass + HALF[given.dtype] * np.abs(ref[key]) * 1.01 + TINY
        err = np.abs(_f64(d[key]) - ref[key])
        assert np.all(err <= tol), (key, float((err / tol).max()))


WIDTHS = [1, 2, 7, 8, 9, 63, 64, 65, 511, 512, 513, 1000, 1023, 1024, 1025, 2047, 2048, 2056, 4095, 4096, 4097, 5120,
          8191, 8192, 8193, 12289, 16383, 16384]


@pytest.mark.parametrize("dtype,wdtype", [(torch.float32, torch.float32), (torch.bfloat16, torch.float32),
                                          (torch.bfloat16, torch.bfloat16)])
@pytest.mark.parametrize("H", WIDTHS)
def test_norm_widths(H, dtype, wdtype):
    """Every width class, its borders and odd widths; each combination of weight,
    bias, residual and skip somewhere."""
    for n, T in enumerate((1, 5, 19)):
        x, r = _rows(T, H, dtype, H + n), _rows(T, H, dtype, H + n + 50, 2.0)
        w = _vec(H, wdtype, 1, 1.0) if (n + H) % 4 != 1 else None
        b = _vec(H, wdtype, 2, 0.0) if (n + H) % 3 != 1 else None
        residual = r if n != 1 else None
        y, s = moe.moe_layer_norm(x, w, b, residual=residual)
        if residual is None:
            assert s is None
            s = x
        else:
            assert torch.equal(s, (x.float() + r.float()).to(dtype))
        _assert_forward(y, s, w, b, 1e-5, dtype)
        dy = _rows(T, H, dtype, H + n + 70, 0.01, 0.0)
        skip = _rows(T, H, dtype, H + n + 90, 0.02, 0.0) if n != 0 else None
        d = moe.moe_layer_norm_backward(dy, s, w, b, d_skip=skip)
        _assert_backward(d, dy, s, w, b, 1e-5, skip, dtype)


@pytest.mark.parametrize("T,H,dtype", [(4099, 96, torch.float32), (8200, 64, torch.bfloat16), (2500, 1023, torch.float32),
                                       (1100, 4096, torch.bfloat16), (1031, 4096, torch.float32),
                                       (700, 8192, torch.bfloat16), (601, 16384, torch.float32)])
def test_norm_many_rows(T, H, dtype):
    """More rows than the launch has blocks: each walks several, the last is ragged."""
    x, w, b = _rows(T, H, dtype, 1), _vec(H, torch.float32, 1, 1.0), _vec(H, torch.float32, 2, 0.0)
    y, _ = moe.moe_layer_norm(x, w, b)
    _assert_forward(y, x, w, b, 1e-5, dtype)
    dy = _rows(T, H, dtype, 3, 0.01, 0.0)
    d = moe.moe_layer_norm_backward(dy, x, w, b, d_skip=x)
    _assert_backward(d, dy, x, w, b, 1e-5, x, dtype)
    # the order of the sums is fixed: the same bits again
    again = moe.moe_layer_norm_backward(dy, x, w, b, d_skip=x)
    assert all(torch.equal(d[key], again[key]) for key in d)


@pytest.mark.parametrize("H", [8, 100, 1024, 4096])
def test_norm_large_mean_small_spread(H):
    """A mean of ten thousand deviations: the variance is not lost to cancellation."""
    gen = torch.Generator().manual_seed(H)
    x = (1e4 + torch.randn((9, H), generator=gen)).cuda()
    y, _ = moe.moe_layer_norm(x)
    _assert_forward(y, x, None, None, 1e-5, torch.float32)
    dy = torch.randn((9, H), generator=gen).cuda()
    d = moe.moe_layer_norm_backward(dy, x)
    _assert_backward(d, dy, x, None, None, 1e-5, None, torch.float32)


def test_norm_constant_zero_and_bad_rows():
    H = 777
    x = _rows(6, H, torch.float32, 5)
    x[1] = 3.0
    x[2] = 0.0
    x[3, 10] = math.nan
    x[4, 700] = math.inf
    w, b = _vec(H, torch.float32, 1, 1.0), _vec(H, torch.float32, 2, 0.0)
    y, _ = moe.moe_layer_norm(x, w, b)
    assert torch.equal(y[1], b) and torch.equal(y[2], b)
    assert torch.all(torch.isnan(y[3])) and torch.all(torch.isnan(y[4]))   # each in its own row
    good = [0, 5]
    _assert_forward(y[good], x[good], w, b, 1e-5, torch.float32)
    dy = _rows(6, H, torch.float32, 6, 1.0, 0.0)
    d = moe.moe_layer_norm_backward(dy, x, w)
    _assert_backward(moe.moe_layer_norm_backward(dy[good], x[good], w), dy[good], x[good], w, None, 1e-5, None,
                     torch.float32)
    assert torch.equal(d["d_x"][good], moe.moe_layer_norm_backward(dy[good], x[good], w)["d_x"])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("H", [63, 1024, 1023, 4096])
def test_norm_unaligned_rows_and_what_lies_around(H, dtype):
    T = 11
    n = T * H
    flat = torch.full((n + 9,), 7.0, dtype=dtype, device="cuda")
    x = flat[1:1 + n].view(T, H)
    x.copy_(_rows(T, H, dtype, 8))
    r = _rows(T, H, dtype, 9)
    fy, fs = torch.full_like(flat, 5.0), torch.full_like(flat, 5.0)
    wflat = torch.full((H + 3,), 1.5, device="cuda")
    w = wflat[1:1 + H]
    y, s = moe.moe_layer_norm(x, w, residual=r, y=fy[3:3 + n].view(T, H), x_sum=fs[1:1 + n].view(T, H))
    assert torch.all(fy[:3] == 5) and torch.all(fy[3 + n:] == 5) and fs[0] == 5 and torch.all(fs[1 + n:] == 5)
    _assert_forward(y, s, w, None, 1e-5, dtype)
    fd = torch.full_like(flat, 5.0)
    dw = torch.full((H + 3,), 5.0, device="cuda")
    d = moe.moe_layer_norm_backward(r, s, w, out={"d_x": fd[1:1 + n].view(T, H), "d_weight": dw[1:1 + H]})
    assert fd[0] == 5 and torch.all(fd[1 + n:] == 5) and dw[0] == 5 and torch.all(dw[1 + H:] == 5)
    _assert_backward(d, r, s, w, None, 1e-5, None, dtype)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,H", [(3, 64), (4000, 512), (2600, 4096)])
def test_norm_in_place(T, H, dtype):
    x, r = _rows(T, H, dtype, 1), _rows(T, H, dtype, 2)
    w, b = _vec(H, torch.float32, 1, 1.0), _vec(H, torch.float32, 2, 0.0)
    y, s = moe.moe_layer_norm(x, w, b, residual=r)
    x2, r2 = x.clone(), r.clone()
    moe.moe_layer_norm(x2, w, b, residual=r2, y=x2, x_sum=r2)
    assert torch.equal(x2, y) and torch.equal(r2, s)
    x3 = s.clone()
    moe.moe_layer_norm(x3, w, b, y=x3)
    assert torch.equal(x3, y)
    dy, skip = _rows(T, H, dtype, 3, 0.01), _rows(T, H, dtype, 4, 0.01)
    d = moe.moe_layer_norm_backward(dy, s, w, b, d_skip=skip)
    dy2, skip2 = dy.clone(), skip.clone()
    d2 = moe.moe_layer_norm_backward(dy2, s, w, b, d_skip=skip, out={"d_x": dy2})
    d3 = moe.moe_layer_norm_backward(dy, s, w, b, d_skip=skip2, out={"d_x": skip2})
    s4 = s.clone()
    d4 = moe.moe_layer_norm_backward(dy, s4, w, b, d_skip=skip, out={"d_x": s4})
    for key in d:
        assert all(torch.equal(d[key], other[key]) for other in (d2, d3, d4)), key


def test_norm_backward_against_differences():
    """Central differences of the kernel's own forward pass, weighted by d_y and summed
    in float64: the step 2^-7 errs by h^2/6 of a third derivative below 40 here
    (unit spread, |d_y| <= 2), the forward's rounding by 64 u sum|d_y| 4 / h."""
    T, H, h = 2, 24, 2.0 ** -7
    x, dy = _rows(T, H, torch.float32, 1), _rows(T, H, torch.float32, 2, 0.5, 0.0).clamp(-2, 2)
    w, b = _vec(H, torch.float32, 1, 1.0), _vec(H, torch.float32, 2, 0.0)
    d = moe.moe_layer_norm_backward(dy, x, w, b)

    def loss(*a):
        return float((moe.moe_layer_norm(*a)[0].double() * dy.double()).sum())

    tol = h * h / 6 * 40 + 64 * U * float(dy.abs().sum()) * 4 / h
    for t, i in ((0, 0), (0, 23), (1, 7), (1, 12)):
        up, down = x.clone(), x.clone()
        up[t, i] += h
        down[t, i] -= h
        assert abs((loss(up, w, b) - loss(down, w, b)) / (2 * h) - float(d["d_x"][t, i])) <= tol
    for i in (0, 8, 23):
        for key, at in (("d_weight", 1), ("d_bias", 2)):
            args = [[x, w, b], [x, w, b]]
            for a, sign in zip(args, (h, -h)):
                a[at] = a[at].clone()
                a[at][i] += sign
            assert abs((loss(*args[0]) - loss(*args[1])) / (2 * h) - float(d[key][i])) <= tol


def test_norm_offsets_beyond_32_bits():
    T, H = (1 << 19) + 3, 4096 + 1
    x = torch.zeros((T, H), dtype=torch.bfloat16, device="cuda")
    tail = _rows(5, H, torch.bfloat16, 3)
    x[-5:] = tail
    y, _ = moe.moe_layer_norm(x)
    assert torch.equal(y[-5:], moe.moe_layer_norm(tail)[0]) and not torch.any(y[:-5])
    d = moe.moe_layer_norm_backward(x, x, out={"d_x": y})
    assert torch.equal(d["d_x"][-5:], moe.moe_layer_norm_backward(tail, tail)["d_x"])
    del x, y, d
    torch.cuda.empty_cache()


def test_norm_empty_and_refusals():
    x = _rows(4, 32, torch.bfloat16, 1)
    w = _vec(32, torch.bfloat16, 1, 1.0)
    y, s = moe.moe_layer_norm(x[:0], w, residual=x[:0])
    assert y.shape == s.shape == (0, 32)
    d = moe.moe_layer_norm_backward(x[:0], x[:0], w, w)
    assert not torch.any(d["d_weight"]) and not torch.any(d["d_bias"]) and d["d_x"].shape == (0, 32)
    with pytest.raises(TypeError):
        moe.moe_layer_norm(x.half())
    with pytest.raises(TypeError):
        moe.moe_layer_norm(x, w.half())
    with pytest.raises(TypeError):
        moe.moe_layer_norm(x.float(), w)
    with pytest.raises(ValueError):
        moe.moe_layer_norm(x, w, w.float())
    with pytest.raises(ValueError):
        moe.moe_layer_norm(x, w[:31])
    with pytest.raises(ValueError):
        moe.moe_layer_norm(x, residual=x[:3])
    with pytest.raises(ValueError):
        moe.moe_layer_norm(x, x_sum=x)
    with pytest.raises(ValueError):
        moe.moe_layer_norm(x.t())
    with pytest.raises(ValueError):
        moe.moe_layer_norm(x.view(2, 2, 32))
    with pytest.raises(moe.MoEError):
        moe.moe_layer_norm(x, eps=0.0)
    with pytest.raises(moe.MoEError):
        moe.moe_layer_norm(torch.zeros((1, 16392), device="cuda"))
    with pytest.raises(ValueError):
        moe.moe_layer_norm_backward(x, x, w, workspace=torch.empty(4, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        moe.moe_layer_norm_backward(x, x, out={"d_weight": w})
