"""moe_gate and moe_gate_backward against the float64 oracle (oracle/operators.py).

Tolerances.  The experts must be the oracle's.  Forward weights are formed in
double and rounded once: 2^-24 of the value (1 % more for double's own errors).
The backward pass runs in float32.  With R the row's range of live logits, an
exponential's relative error is at most (R + 4) u (u = 2^-24: the argument's
rounding, two ulps of exp and one of the sum's term), a sum's over E <= 256
terms 8 u more, a ratio's 2 (R + 13) u; s (g - sum g s) then errs by at most
2 G (4 (R + 13) + k + 4) u with G the largest |scale d_w| (every s is at most 1,
the inner sum at most G in size and k terms long), plus half a step of the
output's type.  Renormalised sigmoids have ratios of the same form.  The dense
row's exponentials are 2^x of a product rounded once, (1.5 R + 2) u each: their
2 G (4.5 R + 19.5 + k/2) u in all is less than the above up to R = 73.
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
LOWEST = {torch.float32: float(np.finfo(np.float32).min), torch.bfloat16: -3.3895313892515355e38}


def _logits(T, E, dtype, seed, spread=1.0):
    rng = np.random.default_rng(seed)
    lg = spread * (rng.standard_normal((T, E)) - np.log1p(rng.permutation(E)))
    return torch.from_numpy(lg.astype(np.float32)).to(dtype).cuda()


def _f64(t):
    return t.detach().double().cpu().numpy()


def _check_gate(lg, k, bias=None, **kw):
    idx, w = moe.moe_gate(lg, k, bias=bias, **kw)
    ref_idx, ref_w = oo.gate(_f64(lg), k, bias=None if bias is None else _f64(bias), **kw)
    assert np.array_equal(idx.cpu().numpy(), ref_idx)
    got = _f64(w)
    assert np.all(np.abs(got - ref_w) <= 1.01 * U * np.abs(ref_w) + 2.0 ** -149), np.max(np.abs(got - ref_w))
    return idx, w


# E, n_groups, keep, k: one expert to 256, group sizes that divide nothing evenly
SHAPES = [(1, 1, 1, 1), (2, 1, 1, 2), (8, 1, 1, 2), (9, 3, 2, 4), (16, 1, 1, 4), (31, 1, 1, 8), (64, 64, 8, 8),
          (64, 8, 3, 6), (65, 5, 2, 8), (96, 3, 1, 5), (128, 2, 1, 8), (160, 8, 3, 6), (160, 1, 1, 6), (203, 7, 4, 3),
          (255, 5, 5, 7), (256, 8, 4, 8), (256, 1, 1, 1), (256, 32, 2, 8), (8, 1, 1, 8), (16, 16, 8, 8), (144, 9, 4, 8),
          (208, 13, 5, 8), (256, 16, 3, 8), (256, 2, 1, 8), (252, 3, 2, 7), (240, 6, 1, 5)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_gate_against_oracle(shape, dtype):
    E, G, keep, k = shape
    rng = np.random.default_rng(E * 10 + k)
    bias = torch.from_numpy((0.1 * rng.standard_normal(E)).astype(np.float32)).cuda()
    n = 0
    for score in ("softmax", "sigmoid"):
        for renorm in (False, True):
            for b in (None, bias):
                n += 1
                _check_gate(_logits((1, 2, 5, 67)[n % 4], E, dtype, n), k, bias=b, score=score, n_groups=G,
                            keep_groups=keep, group_score=("max", "top2")[(n + E) % 2], renorm=renorm,
                            scale=(1.0, 2.5)[n % 2])
    _check_gate(_logits(130, E, dtype, 99), k, bias=bias, score="sigmoid", n_groups=G, keep_groups=keep,
                group_score="top2")
    _check_gate(_logits(131, E, dtype, 98), k, n_groups=G, keep_groups=keep, group_score="top2")


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("with_bias", [False, True])
def test_gate_masks(score, dtype, with_bias):
    """-inf, the lowest values and NaN mask an expert, up to whole groups and rows;
    +inf is the largest logit there is."""
    T, E, k = 96, 24, 4
    lg = _logits(T, E, torch.float32, 5).cpu()
    rng = np.random.default_rng(3)
    lg[torch.from_numpy(rng.random((T, E)) < 0.4)] = -math.inf
    lg[torch.from_numpy(rng.random((T, E)) < 0.1)] = LOWEST[dtype]
    lg[torch.from_numpy(rng.random((T, E)) < 0.05)] = math.nan
    lg[0] = -math.inf                      # nothing left
    lg[1] = LOWEST[dtype]
    lg[2] = math.nan
    lg[3, 1:] = -math.inf                  # one expert left
    lg[4, 6:] = -math.inf                  # one group left (of four)
    lg[5, :18] = -math.inf                 # the last group alone
    lg[6, 3] = math.inf
    lg[7, 3] = lg[7, 20] = math.inf
    lg = lg.to(dtype).cuda()
    # biases that would lift a masked expert over every other one
    bias = torch.linspace(3.0, -3.0, E, device="cuda") if with_bias else None
    for G, keep, gs in ((1, 1, "max"), (4, 2, "max"), (4, 2, "top2"), (4, 1, "top2"), (6, 6, "max")):
        for renorm in (False, True):
            idx, w = _check_gate(lg, k, bias=bias, score=score, n_groups=G, keep_groups=keep, group_score=gs,
                                 renorm=renorm, scale=1.5)
            assert torch.all(w[0:3] == 0) and torch.all((idx >= 0) & (idx < E))


def test_gate_bias_extremes_keep_the_order_defined():
    lg = _logits(33, 16, torch.float32, 6)
    bias = torch.zeros(16, device="cuda")
    bias[3], bias[7], bias[9] = -math.inf, math.nan, math.inf
    idx, w = moe.moe_gate(lg, 8, score="sigmoid", bias=bias)
    assert torch.all(idx[:, 0] == 9) and not torch.any((idx == 3) | (idx == 7)) and torch.all(torch.isfinite(w))
    # with two finite-biased experts left, the lowest follow in index order
    lg[:, [i for i in range(16) if i not in (1, 2, 3, 7)]] = -math.inf
    idx, _ = moe.moe_gate(lg, 5, score="sigmoid", bias=bias)
    assert torch.all(idx[:, 2:] == torch.tensor([3, 7, 0], device="cuda"))


@pytest.mark.parametrize("scale", [1e3, 1e8, 1e25, 1e34])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_gate_wide_biases_and_logits(score, scale):
    """Biases and logits whose spread leaves no float between close scores."""
    T, E = 41, 72
    rng = np.random.default_rng(int(math.log10(scale)))
    small = (0.01 * rng.standard_normal(E)).astype(np.float32)
    for bias in (small + np.float32(scale), np.where(np.arange(E) % 5 == 0, np.float32(scale), small),
                 np.where(np.arange(E) % 7 == 0, np.float32(-scale), small)):
        b = torch.from_numpy(bias.astype(np.float32)).cuda()
        for G, keep, gs in ((1, 1, "max"), (8, 3, "max"), (8, 3, "top2")):
            _check_gate(_logits(T, E, torch.float32, 3), 6, bias=b, score=score, n_groups=G, keep_groups=keep,
                        group_score=gs, renorm=False)
    wide = _logits(T, E, torch.float32, 4)
    wide[:, ::3] *= -scale
    wide[:, 1] += scale
    for G, keep, gs in ((1, 1, "max"), (6, 2, "max"), (6, 2, "top2")):
        for bias in (None, torch.from_numpy(small).cuda()):
            for renorm in (False, True):
                _check_gate(wide, 8, bias=bias, score=score, n_groups=G, keep_groups=keep, group_score=gs,
                            renorm=renorm)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("E,G,keep", [(64, 1, 1), (256, 8, 4), (48, 3, 1)])
def test_gate_ties_go_to_the_lower_index(E, G, keep, dtype):
    rng = np.random.default_rng(E)
    lg = torch.from_numpy((rng.integers(-3, 4, (150, E)) * 0.5).astype(np.float32)).to(dtype).cuda()
    zero = torch.zeros(E, device="cuda")
    for score in ("softmax", "sigmoid"):
        for bias in (None, zero):
            for gs in ("max", "top2"):
                _check_gate(lg, 8, bias=bias, score=score, n_groups=G, keep_groups=keep, group_score=gs)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_gate_orders_scores_closer_than_a_float(score, dtype):
    """Biases that cancel the scores up to their own rounding: all experts of a row lie
    within some 6e-8, and which come first is decided far below a float's step."""
    E, k = 128, 8
    for seed in range(24):
        lg = _logits(1, E, dtype, 100 + seed)
        s = oo._row_scores(_f64(lg)[0], score)[2]
        bias = torch.from_numpy((0.75 - s).astype(np.float32)).cuda()
        for G, keep, gs in ((1, 1, "max"), (8, 2, "top2"), (8, 2, "max")):
            _check_gate(lg.expand(3, E).contiguous(), k, bias=bias, score=score, n_groups=G, keep_groups=keep,
                        group_score=gs)


@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,G,keep,k", [(8, 4, 2, 3), (40, 2, 1, 4), (64, 8, 1, 2), (64, 8, 2, 5), (24, 3, 2, 8),
                                        (33, 1, 1, 2), (256, 32, 2, 8)])
def test_gate_biases_without_a_spread(E, G, keep, k, score, renorm):
    """Infinite and NaN biases and ones beyond 1e30, in whole groups, in all but a few
    experts and throughout: they rank as +-1e299 (NaN lowest), ties by index."""
    rng = np.random.default_rng(E + k)
    size = E // G
    small = (0.1 * rng.standard_normal(E)).astype(np.float32)
    cases = []
    for odd in (math.inf, -math.inf, math.nan, 2e30, -3e38):
        last, few, all_ = small.copy(), np.full(E, odd, np.float32), np.full(E, odd, np.float32)
        last[-size:] = odd
        few[[0, E // 2, E - 1]] = small[[0, E // 2, E - 1]]
        mixed = small.copy()
        mixed[::3] = odd
        cases += [last, few, all_, mixed]
    for b in cases:
        exact = b.astype(np.float64)
        exact = np.clip(np.where(np.isnan(exact), -math.inf, exact), -1e299, 1e299)
        lg = _logits(19, E, torch.float32, 8)
        for gs in ("max", "top2"):
            kw = dict(score=score, n_groups=G, keep_groups=keep, group_score=gs, renorm=renorm)
            idx, w = moe.moe_gate(lg, k, bias=torch.from_numpy(b).cuda(), **kw)
            ref_idx, ref_w = oo.gate(_f64(lg), k, bias=exact, **kw)
            assert np.array_equal(idx.cpu().numpy(), ref_idx), (b, gs)
            assert np.all(np.abs(_f64(w) - ref_w) <= 1.01 * U * np.abs(ref_w) + 2.0 ** -149)


@pytest.mark.parametrize("E,G,keep,k", [(16, 4, 2, 4), (16, 4, 1, 3), (64, 8, 2, 8), (24, 3, 2, 8)])
def test_gate_without_a_bias_saturated_sigmoids_go_by_logit(E, G, keep, k):
    """From 37 on a sigmoid is 1 in double too, and the experts' order still the logits'."""
    rng = np.random.default_rng(E)
    size = E // G
    lg = rng.standard_normal((21, E)) - 5.0
    for row in lg:
        for g in rng.permutation(G)[:keep]:
            row[g * size:(g + 1) * size] = 40.0 + rng.permutation(size)
    _check_gate(torch.from_numpy(lg.astype(np.float32)).cuda(), k, score="sigmoid", n_groups=G, keep_groups=keep,
                group_score="top2")


@pytest.mark.parametrize("E,G,keep,k", [(64, 1, 1, 6), (160, 8, 3, 6), (256, 8, 4, 8), (24, 1, 1, 8), (20, 4, 2, 8)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_gate_pairs_closer_than_a_float(score, E, G, keep, k):
    """In every row some pairs (or triples) of experts whose values differ by about a
    float's step or less, among otherwise spread ones: logits a few steps apart without a
    bias, and with one logits that make up for the bias as well as a float can."""
    T = 700
    rng = np.random.default_rng(E)
    lg = (2.0 * rng.standard_normal((T, E)) + 1.0).astype(np.float32)
    plain = lg.copy()
    for t in range(T):
        order = np.argsort(-plain[t])
        for at in rng.integers(0, k + 2, 3):     # the partner of a high one: anywhere in the row
            other = rng.integers(0, E)
            steps = int(rng.integers(-3, 4))
            v = plain[t, order[min(at, E - 1)]]
            plain[t, other] = v + steps * np.spacing(v)
    opts = dict(score=score, n_groups=G, keep_groups=keep)
    for gs in ("max", "top2"):
        _check_gate(torch.from_numpy(plain).cuda(), k, group_score=gs, **opts)
    if score == "softmax":
        bias = np.zeros(E, np.float32)       # (the scores hang on the whole row: equal logits, ties by index)
        _check_gate(torch.from_numpy(plain).cuda(), k, bias=torch.from_numpy(bias).cuda(), group_score="top2", **opts)
        return
    bias = (0.2 * rng.standard_normal(E)).astype(np.float32)
    for t in range(T):
        value = 1.0 / (1.0 + np.exp(-lg[t].astype(np.float64))) + bias
        order = np.argsort(-value)
        for at in rng.integers(0, k + 2, 3):
            other = int(rng.integers(0, E))
            s = value[order[min(at, E - 1)]] - bias[other]
            if 1e-3 < s < 1 - 1e-3:
                lg[t, other] = np.float32(np.log(s / (1.0 - s)))
                value[other] = 1.0 / (1.0 + np.exp(-np.float64(lg[t, other]))) + bias[other]
    b = torch.from_numpy(bias).cuda()
    for gs in ("max", "top2"):
        _check_gate(torch.from_numpy(lg).cuda(), k, bias=b, group_score=gs, **opts)


def test_gate_equals_moe_route_where_they_mean_the_same():
    lg = _logits(1000, 160, torch.float32, 8)
    idx, w = moe.moe_gate(lg, 6)
    ridx, rw = moe.moe_route(lg, 6)
    assert torch.equal(idx, ridx)
    # both are softmaxes over the same six logits: moe_route's runs in float32 (a few u)
    assert float((w - rw).abs().max()) <= 16 * U


def test_gate_check_word():
    lg = _logits(70, 40, torch.float32, 9)
    check = moe.new_check_word()
    lg[3, 5] = -math.inf
    moe.moe_gate(lg, 2, check=check)
    assert moe.moe_check_device_error(check) == 0
    for bad in (math.nan, math.inf):
        lg2 = lg.clone()
        lg2[69, 39] = bad
        check.zero_()
        moe.moe_gate(lg2, 2, check=check)
        with pytest.raises(moe.MoEError):
            moe.moe_check_device_error(check)
        assert int(check.item()) == moe.CHECK_BITS["logits"]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("E", [20, 33, 256])
def test_gate_unaligned_views_and_what_lies_around(E, dtype):
    """Logits that begin one element into a buffer; outputs inside larger buffers
    whose other rows stay as they were."""
    T, k = 37, 5
    flat = torch.empty(T * E + 8, dtype=dtype, device="cuda").fill_(50.0)
    lg = flat[1:1 + T * E].view(T, E)
    lg.copy_(_logits(T, E, dtype, 11))
    idx = torch.full((T + 2, k), -7, dtype=torch.int32, device="cuda")
    w = torch.full((T + 2, k), -7.0, device="cuda")
    moe.moe_gate(lg, k, topk_idx=idx[1:T + 1], topk_w=w[1:T + 1])
    ref_idx, _ = oo.gate(_f64(lg), k)
    assert np.array_equal(idx[1:T + 1].cpu().numpy(), ref_idx)
    assert torch.all(idx[[0, T + 1]] == -7) and torch.all(w[[0, T + 1]] == -7)
    d_flat = torch.full((T * E + 8,), 3.0, dtype=dtype, device="cuda")
    g = torch.randn(T, k, device="cuda")
    moe.moe_gate_backward(lg, idx[1:T + 1], g, renorm=False, d_logits=d_flat[1:1 + T * E].view(T, E))
    assert torch.all(d_flat[[0, -7, -6, -5, -4, -3, -2, -1]] == 3.0)
    assert torch.equal(d_flat[1:1 + T * E].view(T, E), moe.moe_gate_backward(lg, idx[1:T + 1], g, renorm=False))


def test_gate_offsets_beyond_32_bits():
    """2^23 + 5 tokens of 256 experts: more than 2^31 logits."""
    T, E, k = (1 << 23) + 5, 256, 8
    lg = torch.zeros((T, E), dtype=torch.bfloat16, device="cuda")
    tail = _logits(7, E, torch.bfloat16, 12)
    lg[-7:] = tail
    opts = dict(score="sigmoid", n_groups=8, keep_groups=4, group_score="top2")
    idx, w = moe.moe_gate(lg, k, **opts)
    ref_idx, ref_w = oo.gate(_f64(tail), k, **opts)
    assert np.array_equal(idx[-7:].cpu().numpy(), ref_idx)
    assert np.allclose(_f64(w[-7:]), ref_w, rtol=2 * U)
    assert torch.all(idx[:-7] == torch.arange(k, device="cuda", dtype=torch.int32))
    g = torch.randn(T, k, device="cuda")
    d = moe.moe_gate_backward(lg, idx, g, score="softmax", renorm=False)
    small = moe.moe_gate_backward(tail, idx[-7:], g[-7:], score="softmax", renorm=False)
    assert torch.equal(d[-7:], small)
    del lg, d
    torch.cuda.empty_cache()


def _bound(lg, d_w, scale, k, dtype, ref):
    live = np.where(np.isfinite(lg) & (lg > -1e38), lg, np.nan)
    R = float(np.nanmax(live) - np.nanmin(live)) if np.isfinite(live).any() else 0.0
    G = float(np.abs(scale * d_w[np.isfinite(d_w)]).max()) if d_w.size else 0.0
    return 2 * G * (4 * (R + 13) + k + 4) * U + HALF[dtype] * np.abs(ref) * 1.01 + 2.0 ** -133


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("shape", [s for s in SHAPES if s[0] not in (31, 96)], ids=str)
def test_gate_backward_against_oracle(shape, dtype):
    E, _, _, k = shape
    rng = np.random.default_rng(E + k)
    for n, T in enumerate((1, 3, 70)):
        lg = _logits(T, E, dtype, 20 + n)
        g = torch.from_numpy(rng.standard_normal((T, k)).astype(np.float32)).cuda()
        for score in ("softmax", "sigmoid"):
            idx, _ = moe.moe_gate(lg, k, score=score)
            for renorm in (False, True):
                d = moe.moe_gate_backward(lg, idx, g, score=score, renorm=renorm, scale=2.5)
                ref = oo.gate_backward(_f64(lg), idx.cpu().numpy(), _f64(g), score, renorm, 2.5)
                assert d.dtype == dtype
                assert np.all(np.abs(_f64(d) - ref) <= _bound(_f64(lg), _f64(g), 2.5, k, dtype, ref)), (T, score, renorm)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_gate_backward_masks_repeats_and_bad_indices(score, renorm, dtype):
    T, E, k = 12, 20, 3
    lg = _logits(T, E, torch.float32, 31).cpu()
    lg[:, 4] = -math.inf
    lg[0] = -math.inf
    lg[1] = LOWEST[dtype]
    lg[2, 7] = math.nan
    lg = lg.to(dtype).cuda()
    rng = np.random.default_rng(4)
    idx = torch.from_numpy(rng.integers(0, E, (T, k)).astype(np.int32)).cuda()
    idx[5] = torch.tensor([6, 6, 9])       # the same expert twice
    idx[6] = torch.tensor([6, 6, 6])
    g = torch.from_numpy(rng.standard_normal((T, k)).astype(np.float32)).cuda()
    idx[7] = torch.tensor([4, 2, 3])
    g[7, 0] = math.inf                     # a gradient at a masked expert counts for nothing
    idx[8] = torch.tensor([4, 2, 3])
    g[8, 0] = math.nan
    check = moe.new_check_word()
    d = moe.moe_gate_backward(lg, idx, g, score=score, renorm=renorm, check=check)
    assert moe.moe_check_device_error(check) == 0
    ref = oo.gate_backward(_f64(lg), idx.cpu().numpy(), _f64(g), score, renorm)
    assert np.all(np.abs(_f64(d) - ref) <= _bound(_f64(lg), _f64(g), 1.0, k, dtype, ref))
    assert torch.all(d[0:2] == 0) and torch.all(d[:, 4] == 0) and d[2, 7] == 0
    # an index outside the experts is skipped, and flagged
    idx2 = idx.clone()
    idx2[9] = torch.tensor([-1, 2, E])
    d2 = moe.moe_gate_backward(lg, idx2, g, score=score, renorm=renorm, check=check)
    with pytest.raises(moe.MoEError):
        moe.moe_check_device_error(check)
    assert int(check.item()) == moe.CHECK_BITS["index"]
    ref = oo.gate_backward(_f64(lg), idx2.cpu().numpy(), _f64(g), score, renorm)
    assert np.all(np.abs(_f64(d2) - ref) <= _bound(_f64(lg), _f64(g), 1.0, k, dtype, ref))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_gate_backward_against_differences_of_the_kernel(score, renorm):
    """Central differences of moe_gate's own weights.  The step h = 2^-6 errs by
    h^2/6 times the third derivative of sum g w (at most 6 G k in size for softmax
    and sigmoid ratios), the weights' rounding by k G u / h."""
    T, E, k, h = 1, 10, 3, 2.0 ** -6
    lg = torch.tensor([[2.0, -1.0, 1.5, 0.5, -2.0, 0.25, -0.75, 3.0, -3.0, 0.0]], device="cuda")
    g = torch.tensor([[0.5, -1.0, 0.75]], device="cuda")
    idx, _ = moe.moe_gate(lg, k, score=score, renorm=renorm)
    d = moe.moe_gate_backward(lg, idx, g, score=score, renorm=renorm)
    tol = h * h / 6 * 6 * 1.0 * k + 2 * k * U / h + 1e-6
    for e in range(E):
        v = []
        for sign in (h, -h):
            moved = lg.clone()
            moved[0, e] += sign
            i2, w2 = moe.moe_gate(moved, k, score=score, renorm=renorm)
            assert torch.equal(i2, idx)
            v.append(float((w2.double() * g.double()).sum()))
        assert abs((v[0] - v[1]) / (2 * h) - float(d[0, e])) <= tol, e


def test_gate_refuses_what_it_cannot_take():
    lg = _logits(8, 16, torch.float32, 1)
    with pytest.raises(TypeError):
        moe.moe_gate(lg.half(), 2)
    with pytest.raises(ValueError):
        moe.moe_gate(lg.t(), 2)                                    # not contiguous
    with pytest.raises(ValueError):
        moe.moe_gate(lg, 2, bias=torch.zeros(15, device="cuda"))
    with pytest.raises(ValueError):
        moe.moe_gate(lg, 2, bias=torch.zeros(16, device="cuda", dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        moe.moe_gate(lg, 2, topk_w=torch.zeros((8, 3), device="cuda"))
    with pytest.raises(KeyError):
        moe.moe_gate(lg, 2, score="relu")
    with pytest.raises(moe.MoEError):
        moe.moe_gate(lg, 2, n_groups=3)
    idx, w = moe.moe_gate(lg, 2)
    with pytest.raises(ValueError):
        moe.moe_gate_backward(lg, idx.long(), w)
    with pytest.raises(ValueError):
        moe.moe_gate_backward(lg, idx, w[:4])
    empty = moe.moe_gate(lg[:0], 2)
    assert empty[0].shape == (0, 2) and moe.moe_gate_backward(lg[:0], *empty).shape == (0, 16)
