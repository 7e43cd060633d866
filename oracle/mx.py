"""Microscaled blocks, the 4-bit expert FFN and the combine's gradient in plain numpy
float64 -- TEST INFRASTRUCTURE ONLY.

Written from the formulas in include/moe.h; it shares no code with the HIP library
and never imports it.
"""
from __future__ import annotations

import math

import numpy as np

BLOCK = 32
BITS = {"fp4": 4, "fp6": 6, "fp8": 8}
GRID = {"fp4": np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]),
        "fp6": np.array([m / 8 if e == 0 else (1 + m / 8) * 2.0 ** (e - 1) for e in range(4) for m in range(8)]),
        "fp8": np.array([(m / 8 * 2.0 ** -6) if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
                         for e in range(16) for m in range(8)][:127])}


def _nearest(a, fmt):
    """Index of the grid's value nearest to each magnitude a (past the largest: one more), ties to the even index."""
    grid = GRID[fmt]
    nxt = 480.0 if fmt == "fp8" else 8.0     # the value after the largest, were there one
    full = np.append(grid, nxt)
    hi = np.minimum(np.searchsorted(full, a), len(full) - 1)
    lo = np.maximum(hi - 1, 0)
    up, down = full[hi] - a, a - full[lo]
    return np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)


def scale_bytes(top, fmt):
    """The smallest byte with which each magnitude rounds to the largest value or less; 255 where it is not finite."""
    out = np.zeros(top.shape, dtype=np.int64)
    ok = np.isfinite(top)
    last = len(GRID[fmt]) - 1
    with np.errstate(divide="ignore"):
        guess = np.where(ok & (top > 0), np.floor(np.log2(np.where(top > 0, top, 1.0))), -200.0)
    b = np.clip(guess.astype(np.int64) + 127 - 10, 0, 254)
    while True:
        past = ok & (b < 254) & (_nearest(np.where(ok, top, 0.0) * 2.0 ** (127.0 - b), fmt) > last)
        if not past.any():
            break
        b = np.where(past, b + 1, b)
    out[:] = np.where(ok, b, 255)
    return out


def _blocks(x):
    K = x.shape[-1]
    pad = -K % BLOCK
    return np.pad(x, [(0, 0)] * (x.ndim - 1) + [(0, pad)]).reshape(*x.shape[:-1], -1, BLOCK)


def quantize(x, fmt):
    """(codes uint8 [..., bytes of K codes], scale uint8 [..., K / 32]) of float64 rows."""
    K = x.shape[-1]
    v = _blocks(x)
    byte = scale_bytes(np.abs(v).max(-1), fmt)
    nan = byte == 255
    a = np.where(nan[..., None], 0.0, v) * 2.0 ** (127.0 - np.where(nan, 127, byte))[..., None]
    code = np.where(nan[..., None], 0, np.minimum(_nearest(np.abs(a), fmt), len(GRID[fmt]) - 1))
    sign = np.where(nan[..., None], False, np.signbit(v))
    code = (code + sign * (1 << BITS[fmt] - 1)).astype(np.uint8).reshape(*x.shape[:-1], -1)[..., :K]
    bits = np.unpackbits(code[..., None], axis=-1, bitorder="little")[..., :BITS[fmt]]
    return np.packbits(bits.reshape(*x.shape[:-1], -1), axis=-1, bitorder="little"), byte.astype(np.uint8)


def dequantize(codes, scale, fmt, K=None):
    n = BITS[fmt]
    bits = np.unpackbits(codes, axis=-1, bitorder="little")
    K = bits.shape[-1] // n if K is None else K
    bits = bits[..., :K * n].reshape(*codes.shape[:-1], K, n)
    codes = np.packbits(bits, axis=-1, bitorder="little")[..., 0]
    grid = np.append(GRID[fmt], math.nan)
    top = 1 << n - 1
    v = grid[codes & (top - 1)] * np.where(codes & top, -1.0, 1.0)
    s = np.where(scale == 255, math.nan, 2.0 ** (scale.astype(np.float64) - 127.0))
    return v * np.repeat(s, BLOCK, -1)[..., :K]


def values(x, fmt):
    return dequantize(*quantize(x, fmt), fmt, x.shape[-1])


def act(g, u=None):
    if u is None:
        return 0.5 * g * (1.0 + np.vectorize(math.erf)(g / math.sqrt(2.0)))
    with np.errstate(over="ignore"):
        return g / (1.0 + np.exp(-g)) * u


def ffn(xq, wg, wu, wd, fmt):
    """(h, y) of one expert for rows xq that are quantised already; weights float64 [I, H] and [H, I]."""
    h = act(xq @ wg.T, None if wu is None else xq @ wu.T)
    return h, values(h, fmt) @ wd.T


def combine_backward(d_out, y, inv_pos, w):
    """(d_y [M, H] with NaN rows where no entry points, d_topk_w [T, k])."""
    d_y = np.full(y.shape, np.nan)
    d_w = np.zeros(w.shape)
    for t in range(w.shape[0]):
        for i in range(w.shape[1]):
            r = inv_pos[t, i]
            if 0 <= r < y.shape[0]:
                d_y[r] = w[t, i] * d_out[t]
                d_w[t, i] = d_out[t] @ y[r]
    return d_y, d_w
