"""Cases for the operators around the expert layer: the gate, layer norm, gradient clipping.

    gate           router logits -> experts and weights: softmax or sigmoid scores, a selection
                   bias, expert groups, top-k, renormalised or scaled weights
    gate_backward  the gradient of the weights, back to the router logits
    norm           layer norm of the rows of x, or of x + residual (the sum is returned too)
    norm_backward  its gradients: rows, weight and bias
    clip           the global norm of many gradients, and the gradients scaled to at most max_norm

A case is a dict of plain values; prepare() draws its inputs on the GPU, run() makes one pass (plain torch,
or the library's calls where `own` is set) and exact() evaluates the definition in float64.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
MASK_BELOW = -1e38     # a router logit at or below this (or NaN) is a masked expert
F32_MAX = torch.finfo(torch.float32).max


# ------------------------------------------------------------------------------------------- cases
def listed():
    return [
        # one decoded token of a sequence being served: 256 experts in 8 groups, sigmoid scores and a
        # balance bias; latency is all that counts
        dict(name="gate_token", op="gate", T=1, E=256, k=8, dtype="f32", score="sigmoid", bias=True, groups=8, keep=4,
             group_score="top2", renorm=True, scale=2.5, masked=0),
        # a training batch of the 160-expert workload: softmax scores, group-limited by the best expert,
        # weights not renormalised
        dict(name="gate_softmax_groups", op="gate", T=16384, E=160, k=6, dtype="f32", score="softmax", bias=False,
             groups=8, keep=3, group_score="max", renorm=False, scale=16.0, masked=0),
        # the largest batch of long prompts: bf16 logits, biased sigmoid scores, a few experts switched off
        dict(name="gate_sigmoid_bias", op="gate", T=65536, E=256, k=8, dtype="bf16", score="sigmoid", bias=True,
             groups=8, keep=4, group_score="top2", renorm=True, scale=2.5, masked=5),
        # its gradients in training: dense through the softmax over all experts ...
        dict(name="gate_bwd_softmax", op="gate_backward", T=16384, E=160, k=6, dtype="f32", score="softmax",
             renorm=False, scale=16.0),
        # ... and sparse through renormalised sigmoid scores, on a ragged number of tokens
        dict(name="gate_bwd_sigmoid", op="gate_backward", T=60013, E=256, k=8, dtype="bf16", score="sigmoid",
             renorm=True, scale=2.5),
        # one decoded token before an expert layer of hidden size 4096
        dict(name="norm_token", op="norm", T=1, H=4096, dtype="bf16", wdtype="bf16", weight=True, bias=True,
             residual=True),
        # a training batch: the sum with the residual stream and its norm
        dict(name="norm_residual", op="norm", T=8192, H=4096, dtype="bf16", wdtype="f32", weight=True, bias=True,
             residual=True),
        # ragged: an odd number of tokens of an odd row width
        dict(name="norm_odd", op="norm", T=15001, H=1023, dtype="f32", wdtype="f32", weight=True, bias=True,
             residual=False),
        # the training batch's backward pass, with the gradient that reaches the sum past the norm
        dict(name="norm_bwd_skip", op="norm_backward", T=8192, H=4096, dtype="bf16", wdtype="f32", weight=True,
             bias=True, skip=True),
        # many short float rows: the reduction over the tokens weighs more
        dict(name="norm_bwd_short", op="norm_backward", T=16384, H=1024, dtype="f32", wdtype="f32", weight=True,
             bias=True, skip=False),
        # the small parameters of 12 layers (norms and routers), views of one flat buffer
        dict(name="clip_small", op="clip", layers=12, E=32, H=1023, I=0, gated=False, dtype="bf16", flat=True,
             max_norm=1.0),
        # one layer of 32 GELU experts, 1024 x 4096 each, in float32: about a gigabyte
        dict(name="clip_layer", op="clip", layers=1, E=32, H=1024, I=4096, gated=False, dtype="f32", flat=False,
             max_norm=1.0),
    ]


def _spread(rng, low, high):
    """A whole number between low and high, spread evenly over its logarithm."""
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["gate", "gate", "gate_backward", "norm", "norm_backward", "clip"])
    dtype = rng.choice(["f32", "bf16"])
    if op in ("gate", "gate_backward"):
        groups = rng.choice([1, 1, 2, 4, 8])
        size = rng.randint(max(1, 8 // groups), 256 // groups)
        E, k = groups * size, rng.randint(1, 8)
        case = dict(op=op, T=_spread(rng, 1, 65536), E=E, k=k, dtype=dtype, score=rng.choice(["softmax", "sigmoid"]),
                    renorm=rng.random() < 0.5, scale=rng.choice([1.0, 2.5, 16.0]))
        if op == "gate":
            need = -(-k // size)
            case.update(bias=rng.random() < 0.6, groups=groups, keep=rng.randint(need, groups),
                        group_score=rng.choice(["max", "top2"]), masked=rng.choice([0, 0, rng.randint(1, E // 4 + 1)]))
        return case
    if op in ("norm", "norm_backward"):
        H = _spread(rng, 64, 16384)
        T = _spread(rng, 1, max(1, min(65536, 8192 * 4096 // (H * (2 if dtype == "f32" else 1)))))
        weight = rng.random() < 0.8
        case = dict(op=op, T=T, H=H, dtype=dtype, wdtype=rng.choice([dtype, "f32"]), weight=weight,
                    bias=weight and rng.random() < 0.7)
        case["residual" if op == "norm" else "skip"] = rng.random() < 0.5
        return case
    H, I, E = _spread(rng, 64, 4096), rng.choice([0, _spread(rng, 64, 4096)]), rng.choice([8, 16, 32])
    gated = rng.random() < 0.5
    per_layer = E * H * I * (3 if gated else 2) + E * H + 2 * H + E
    layers = max(1, min(_spread(rng, 1, 24), 200_000_000 // per_layer))
    while E * H * I * (3 if gated else 2) > 200_000_000:
        I //= 2
    return dict(op=op, layers=layers, E=E, H=H, I=I, gated=gated, dtype=dtype, flat=rng.random() < 0.5,
                max_norm=rng.choice([1.0, 1.0, 1e6]))


# ------------------------------------------------------------------------------------------ inputs
def _randn(gen, *shape):
    return torch.randn(shape, generator=gen, device=gen.device, dtype=torch.float32)


def _router_logits(gen, T, E, dtype, masked=0):
    """Noise plus a popularity bias of -ln(rank + 1): a few experts are hot."""
    rank = torch.randperm(E, generator=gen, device=gen.device).float()
    lg = _randn(gen, T, E) - torch.log(rank + 1.0)
    if masked:
        lg[:, torch.randperm(E, generator=gen, device=gen.device)[:masked]] = -math.inf
    return lg.to(dtype)


def _rows(gen, T, H, dtype):
    """Hidden states: a shifted mean, and a few channels far larger than the others."""
    channel = 1.0 + 29.0 * (torch.rand(H, generator=gen, device=gen.device) < 0.003).float()
    return ((_randn(gen, T, H) + 0.25) * channel).to(dtype)


def _grad_shapes(case):
    """The gradients of `layers` layers: norm weight and bias, router weight and bias, expert weights."""
    E, H, I, dt = case["E"], case["H"], case["I"], DTYPES[case["dtype"]]
    layer = [((H,), dt), ((H,), dt), ((E, H), torch.float32), ((E,), torch.float32)]
    if I:
        layer += [((E, I, H), dt)] * (2 if case["gated"] else 1) + [((E, H, I), dt)]
    return layer * case["layers"]


def _views(flat, shapes):
    """Tensors of the given shapes one after the other in a flat buffer."""
    ends = [0]
    for shape in shapes:
        ends.append(ends[-1] + math.prod(shape))
    return [flat[a:b].view(shape) for a, b, shape in zip(ends, ends[1:], shapes)]


def _gradients(gen, case):
    shapes = _grad_shapes(case)
    if not case["flat"]:
        return [(_randn(gen, *shape) * 0.01).to(dt) for shape, dt in shapes]
    grads = [None] * len(shapes)
    for dt in sorted({dt for _, dt in shapes}, key=str):
        at = [i for i, (_, d) in enumerate(shapes) if d == dt]
        flat = (_randn(gen, sum(math.prod(shapes[i][0]) for i in at)) * 0.01).to(dt)
        for i, view in zip(at, _views(flat, [shapes[i][0] for i in at])):
            grads[i] = view
    return grads


def prepare(case, seed):
    gen = torch.Generator(device="cuda" if torch.cuda.is_available() else "cpu").manual_seed(seed)
    dev, op, st = gen.device, case["op"], dict(case=case)
    if op in ("gate", "gate_backward"):
        T, E, k = case["T"], case["E"], case["k"]
        st["logits"] = _router_logits(gen, T, E, DTYPES[case["dtype"]], case.get("masked", 0))
        if op == "gate":
            st["bias"] = 0.05 * _randn(gen, E) if case["bias"] else None
        else:
            noisy = st["logits"].float() + 0.1 * _randn(gen, T, E)
            st["idx"] = torch.topk(noisy, k, dim=1).indices.to(torch.int32).contiguous()
            st["d_w"] = _randn(gen, T, k)
    elif op in ("norm", "norm_backward"):
        T, H, wdt = case["T"], case["H"], DTYPES[case["wdtype"]]
        st["x"] = _rows(gen, T, H, DTYPES[case["dtype"]])
        st["weight"] = (1.0 + 0.1 * _randn(gen, H)).to(wdt) if case["weight"] else None
        st["bias"] = (0.1 * _randn(gen, H)).to(wdt) if case["bias"] else None
        if op == "norm":
            st["residual"] = _rows(gen, T, H, st["x"].dtype) if case["residual"] else None
        else:
            st["d_y"] = (0.01 * _randn(gen, T, H)).to(st["x"].dtype)
            st["d_skip"] = (0.01 * _randn(gen, T, H)).to(st["x"].dtype) if case["skip"] else None
    else:
        st["grads"] = _gradients(gen, case)
        st["clipped"] = [torch.empty_like(g) for g in st["grads"]]
    st["eps"] = 1e-5
    if dev.type == "cuda":
        torch.cuda.synchronize()
    return st


# ------------------------------------------------------------------------------------ plain forms
def _masked_logits(logits, dtype):
    lg = logits.to(dtype)
    live = lg > MASK_BELOW                       # false for NaN too
    return torch.where(live, lg.clamp(max=F32_MAX), torch.full_like(lg, -math.inf)), live


def _scores(lg, live, score):
    """Scores in [0, 1]; a masked expert's is zero."""
    if score == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-lg))
    top = torch.where(live.any(1, keepdim=True), lg.amax(1, keepdim=True), torch.zeros_like(lg[:, :1]))
    e = torch.exp(lg - top)
    return e / e.sum(1, keepdim=True).clamp(min=1.0)


def _gate_plain(st):
    """In 64 bits: which experts are taken hangs on scores next to each other."""
    c = st["case"]
    T, E, k, G = c["T"], c["E"], c["k"], c["groups"]
    lg, live = _masked_logits(st["logits"], torch.float64)
    s = _scores(lg, live, c["score"])
    # without a bias the experts' order is the logits' own
    key = lg if st["bias"] is None else torch.where(live, s + st["bias"].double(), torch.full_like(s, -math.inf))
    key = torch.where(live, key, torch.full_like(key, -1e300))    # masked: after every other expert
    if c["keep"] < G:
        if c["group_score"] == "max":
            group = key.view(T, G, E // G).amax(2)
        else:
            value = s if st["bias"] is None else s + st["bias"].double()
            value = torch.where(live, value, torch.full_like(value, -math.inf)).view(T, G, E // G)
            two = torch.sort(value, dim=2, descending=True).values[:, :, :2]
            group = two[:, :, 0] + torch.where(torch.isfinite(two), two, torch.zeros_like(two))[:, :, 1:].sum(2)
        order = torch.sort(group, dim=1, descending=True, stable=True).indices
        kept = torch.zeros((T, G), dtype=torch.bool, device=key.device).scatter_(1, order[:, :c["keep"]], True)
        key = torch.where(kept.repeat_interleave(E // G, 1), key, torch.full_like(key, -math.inf))
    idx = torch.sort(key, dim=1, descending=True, stable=True).indices[:, :k]
    w = torch.gather(s, 1, idx)
    if c["renorm"]:
        total = w.sum(1, keepdim=True)
        w = torch.where(total > 0, w / total, torch.zeros_like(w))
    return idx.to(torch.int32), (c["scale"] * w).float()


def _gate_backward_plain(st):
    c = st["case"]
    lg, live = _masked_logits(st["logits"], torch.float32)
    idx, g = st["idx"].long(), st["d_w"] * c["scale"]
    s = _scores(lg, live, c["score"])
    sk = torch.gather(s, 1, idx)
    if c["renorm"]:
        total = sk.sum(1, keepdim=True)
        w = torch.where(total > 0, sk / total, torch.zeros_like(sk))
        slot = w * (g - (g * w).sum(1, keepdim=True))
        slot = slot * (1.0 - sk) if c["score"] == "sigmoid" else slot
        d = torch.zeros_like(s).scatter_add_(1, idx, slot)
    elif c["score"] == "sigmoid":
        d = torch.zeros_like(s).scatter_add_(1, idx, g * sk * (1.0 - sk))
    else:
        d = torch.zeros_like(s).scatter_add_(1, idx, g * sk) - s * (g * sk).sum(1, keepdim=True)
    return d.to(st["logits"].dtype)


def _norm_plain(st):
    x = st["x"]
    if st["residual"] is not None:
        x = (x.float() + st["residual"].float()).to(x.dtype)
    v = x.float()
    centred = v - v.mean(1, keepdim=True)
    y = centred / torch.sqrt((centred * centred).mean(1, keepdim=True) + st["eps"])
    y = y if st["weight"] is None else y * st["weight"].float()
    y = y if st["bias"] is None else y + st["bias"].float()
    return [y.to(x.dtype)] + ([] if st["residual"] is None else [x])


def _norm_backward_plain(st):
    x, g = st["x"].float(), st["d_y"].float()
    centred = x - x.mean(1, keepdim=True)
    rstd = 1.0 / torch.sqrt((centred * centred).mean(1, keepdim=True) + st["eps"])
    xhat = centred * rstd
    gw = g if st["weight"] is None else g * st["weight"].float()
    dx = rstd * (gw - gw.mean(1, keepdim=True) - xhat * (gw * xhat).mean(1, keepdim=True))
    dx = dx if st["d_skip"] is None else dx + st["d_skip"].float()
    out = {"d_x": dx.to(st["x"].dtype)}
    if st["weight"] is not None:
        out["d_weight"] = (g * xhat).sum(0).to(st["weight"].dtype)
    if st["bias"] is not None:
        out["d_bias"] = g.sum(0).to(st["bias"].dtype)
    return out


def _clip_plain(st):
    """The sum of squares in 64 bits: it is a long one."""
    squares = torch.stack([g.float().square().sum(dtype=torch.float64) for g in st["grads"]])
    norm = torch.sqrt(squares.sum())
    factor = torch.clamp(st["case"]["max_norm"] / (norm + 1e-6), max=1.0).float()
    return [norm.float().reshape(1)] + [(g.float() * factor).to(g.dtype) for g in st["grads"]]


# ------------------------------------------------------------------------------------------- a pass
def _library(st):
    import mixture_experts_routing_top_amd as moe
    c = st["case"]
    if c["op"] == "gate":
        return moe.moe_gate(st["logits"], c["k"], score=c["score"], bias=st["bias"], n_groups=c["groups"],
                            keep_groups=c["keep"], group_score=c["group_score"], renorm=c["renorm"], scale=c["scale"])
    if c["op"] == "gate_backward":
        return moe.moe_gate_backward(st["logits"], st["idx"], st["d_w"], score=c["score"], renorm=c["renorm"],
                                     scale=c["scale"])
    if c["op"] == "norm":
        y, x_sum = moe.moe_layer_norm(st["x"], st["weight"], st["bias"], eps=st["eps"], residual=st["residual"])
        return [y] + ([] if st["residual"] is None else [x_sum])
    if c["op"] == "norm_backward":
        d = moe.moe_layer_norm_backward(st["d_y"], st["x"], st["weight"], st["bias"], eps=st["eps"],
                                        d_skip=st["d_skip"])
        return {key: v for key, v in d.items() if v is not None}
    norm, clipped = moe.moe_clip_grads(st["grads"], c["max_norm"], out=st["clipped"])
    return [norm] + clipped


def run(state):
    if own:
        return _library(state)
    plain = {"gate": _gate_plain, "gate_backward": _gate_backward_plain, "norm": _norm_plain,
             "norm_backward": _norm_backward_plain, "clip": _clip_plain}
    return plain[state["case"]["op"]](state)


def work(case):
    """Every input read once, every output written once; the operations of the formulas."""
    size = {"f32": 4, "bf16": 2}
    op, s = case["op"], size[case["dtype"]]
    if op == "gate":
        T, E, k = case["T"], case["E"], case["k"]
        return {"bytes": T * E * s + T * k * 8 + (4 * E if case["bias"] else 0), "flops": T * E * 4}
    if op == "gate_backward":
        T, E, k = case["T"], case["E"], case["k"]
        dense = case["score"] == "softmax" and not case["renorm"]
        return {"bytes": (2 if dense else 1) * T * E * s + T * k * (8 + (0 if dense else s)),
                "flops": T * (4 * E if dense else 6 * k)}
    if op == "norm":
        n, vectors = case["T"] * case["H"], case["H"] * size[case["wdtype"]] * (case["weight"] + case["bias"])
        return {"bytes": n * s * (4 if case["residual"] else 2) + vectors, "flops": n * 8}
    if op == "norm_backward":
        n = case["T"] * case["H"]
        vectors = case["H"] * size[case["wdtype"]] * (2 * case["weight"] + case["bias"])
        return {"bytes": n * s * (4 if case["skip"] else 3) + vectors, "flops": n * 16}
    counts = [(math.prod(shape), 4 if dt == torch.float32 else 2) for shape, dt in _grad_shapes(case)]
    return {"bytes": sum(2 * n * b for n, b in counts) + 4, "flops": sum(3 * n for n, _ in counts)}


# ----------------------------------------------------------------------- the definitions in float64
def _exact_gate(st):
    """One expert after the other, by score and then by index."""
    c = st["case"]
    T, E, G = c["T"], c["E"], c["groups"]
    lg = st["logits"].double()
    dead = torch.isnan(lg) | (lg <= MASK_BELOW)
    if c["score"] == "softmax":
        lowest = lg.masked_fill(dead, -math.inf)
        s = torch.exp(lowest - torch.logsumexp(lowest, 1, keepdim=True)).masked_fill(dead, 0.0)
    else:
        s = torch.sigmoid(lg).masked_fill(dead, 0.0)
    biased = s if st["bias"] is None else s + st["bias"].double()
    order = (lg if st["bias"] is None else biased).masked_fill(dead, -1e300)
    column = torch.arange(E, device=lg.device)
    if c["keep"] < G:
        inside = (order if c["group_score"] == "max" else biased.masked_fill(dead, -math.inf)).reshape(T, G, -1)
        value = inside.amax(2)
        if c["group_score"] == "top2" and E > G:
            second = torch.topk(inside, 2, dim=2).values[:, :, 1]
            value = value + second.masked_fill(torch.isinf(second), 0.0)
        # a group is kept if fewer than `keep` groups come before it
        before = (value[:, None, :] > value[:, :, None])
        ties = (value[:, None, :] == value[:, :, None]) & (torch.arange(G, device=lg.device)[None, :]
                                                           < torch.arange(G, device=lg.device)[:, None])[None]
        out = (before | ties).sum(2) >= c["keep"]
        order = order.masked_fill(out.repeat_interleave(E // G, 1), -math.inf)
    w = torch.empty((T, c["k"]), dtype=torch.float64, device=lg.device)
    for i in range(c["k"]):
        best = order.amax(1, keepdim=True)
        first = torch.where(order == best, column, E).amin(1, keepdim=True)
        w[:, i] = s.gather(1, first)[:, 0]
        order = order.scatter(1, first, -math.inf)
    if c["renorm"]:
        w = torch.nan_to_num(w / w.sum(1, keepdim=True))
    return None, c["scale"] * w


def _exact_gate_backward(st):
    """By the Jacobian of the weights with respect to the kept scores."""
    c = st["case"]
    lg, idx, g = st["logits"].double(), st["idx"].long(), st["d_w"].double()
    p = torch.softmax(lg, 1) if c["score"] == "softmax" else torch.sigmoid(lg)
    kept = p.gather(1, idx)
    if c["renorm"]:
        total = kept.sum(1, keepdim=True)
        d_kept = c["scale"] * (g / total - (g * kept).sum(1, keepdim=True) / total ** 2)
    else:
        d_kept = c["scale"] * g
    d_p = torch.zeros_like(p).scatter_add(1, idx, d_kept)
    if c["score"] == "sigmoid":
        return d_p * p * (1.0 - p)
    return p * (d_p - (d_p * p).sum(1, keepdim=True))


def _exact_norm(st):
    x = st["x"]
    summed = x.double() if st["residual"] is None else x.double() + st["residual"].double()
    # the norm is of the sum as it is kept, in the rows' own type (one rounding of the float32 sum)
    v = x.double() if st["residual"] is None else (x.float() + st["residual"].float()).to(x.dtype).double()
    var, mean = torch.var_mean(v, dim=1, correction=0, keepdim=True)
    y = (v - mean) * torch.rsqrt(var + st["eps"])
    y = y if st["weight"] is None else y * st["weight"].double()
    y = y if st["bias"] is None else y + st["bias"].double()
    return [y] + ([] if st["residual"] is None else [summed])


def _exact_norm_backward(st):
    """Through the variance and the mean, as the chain rule has them."""
    x, g = st["x"].double(), st["d_y"].double()
    H = x.shape[1]
    var, mean = torch.var_mean(x, dim=1, correction=0, keepdim=True)
    inv = (var + st["eps"]) ** -0.5
    d_hat = g if st["weight"] is None else g * st["weight"].double()
    d_var = (d_hat * (x - mean)).sum(1, keepdim=True) * -0.5 * inv ** 3
    d_x = d_hat * inv + d_var * 2.0 * (x - mean) / H - (d_hat * inv).sum(1, keepdim=True) / H
    out = {"d_x": d_x if st["d_skip"] is None else d_x + st["d_skip"].double()}
    if st["weight"] is not None:
        out["d_weight"] = (g * (x - mean) * inv).sum(0)
    if st["bias"] is not None:
        out["d_bias"] = g.sum(0)
    return out


def _exact_clip(st):
    norm = math.sqrt(sum(float(torch.linalg.vector_norm(g.double())) ** 2 for g in st["grads"]))
    factor = min(1.0, st["case"]["max_norm"] / (norm + 1e-6))
    first = torch.full((1,), norm, dtype=torch.float64, device=st["grads"][0].device)
    return [first] + [g.double() * factor for g in st["grads"]]


def exact(case, seed):
    st = prepare(case, seed)
    forms = {"gate": _exact_gate, "gate_backward": _exact_gate_backward, "norm": _exact_norm,
             "norm_backward": _exact_norm_backward, "clip": _exact_clip}
    return forms[case["op"]](st)
