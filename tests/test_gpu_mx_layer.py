"""A layer held in few bits, through moe_layer_forward and moe_layer_backward: 4-bit
expert weights when it serves, activations kept in 8 bits when it trains.

moe_backward_mx is moe_backward_gated at the values that the blocks stand for: those are
exact in both types (e4m3 has 4 significant bits), and the two share their products, so
d_x and the weights' gradients are the same bits; d_topk_w is summed in another order,
each off by n = 9 ceil(H / 512) + 12 roundings of 2^-24 at most of sum |d y| (and
moe_backward_gated's by no more).  Against float64 the bars are the layer's own (float32
products 1e-4 of the norm, 4 stored bf16 roundings 2e-2).
"""
import numpy as np
import pytest
import torch

import mixture_experts_routing_top_amd as moe
from oracle import backward as ob
from oracle import mx as om
from _util import REL_FP32_GEMM, REL_BF16

pytestmark = pytest.mark.gpu

GATE = dict(score="sigmoid", renorm=True, n_groups=2, keep_groups=1, group_score="top2", scale=1.5)
# T, E, H, I, k: one token, ragged ones, experts without rows, more experts than rows
SIZES = [(1, 4, 64, 64, 1), (37, 6, 128, 192, 2), (150, 16, 192, 128, 6), (5, 24, 64, 320, 3), (700, 8, 576, 64, 8)]


def _case(T, E, H, I, k, dtype=torch.float32, act="swiglu", seed=0):
    gen = torch.Generator().manual_seed(seed)
    rnd = lambda *s, f=1.0: (f * torch.randn(s, generator=gen)).to(dtype).cuda()  # noqa: E731
    return dict(x=rnd(T, H), logits=torch.randn((T, E), generator=gen).cuda(), k=k, act=act,
                wts=[rnd(E, I, H, f=H ** -0.5), rnd(E, I, H, f=H ** -0.5) if act == "swiglu" else None,
                     rnd(E, H, I, f=I ** -0.5)], d_out=rnd(T, H, f=0.1))


def _forward(c, **kw):
    return moe.moe_layer_forward(c["x"], c["logits"], c["k"], *c["wts"], c["act"], **kw)


def _backward(c, f, **kw):
    return moe.moe_layer_backward(f, c["logits"], *c["wts"], c["d_out"], c["act"], **kw)


def _f64(t):
    return t.detach().double().cpu().numpy()


def _rel(a, b):
    return np.linalg.norm(a - b) / max(np.linalg.norm(b), 1e-300)


@pytest.mark.parametrize("act", ["swiglu", "gelu"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("size", SIZES)
def test_backward_is_the_gated_one_at_the_kept_values(size, dtype, act):
    c = _case(*size, dtype, act)
    T, E, H, _, k = size
    check = moe.new_check_word()
    f = _forward(c, keep="fp8", check=check)
    x_perm = moe.moe_mx_dequantize(*f["kept_x"], "fp8", dtype, rows=f["perm_src"])
    y_perm = moe.moe_mx_dequantize(*f["kept_y"], "fp8", dtype)
    want = moe.moe_backward_gated(x_perm, y_perm, f["idx"], f["w"], f["inv_pos"], f["expert_off"], *c["wts"], c["d_out"],
                                  act)
    got = moe.moe_backward_mx(f["kept_x"], f["kept_y"], f["perm_src"], f["w"], f["inv_pos"], f["expert_off"], *c["wts"],
                              c["d_out"], act, check=check)
    assert moe.moe_check_device_error(check) == 0
    assert set(got) == set(want)
    for name in set(got) - {"d_topk_w"}:
        assert torch.equal(got[name], want[name]), name
    inv, d, y = _f64(f["inv_pos"]).astype(int), _f64(c["d_out"]), _f64(y_perm)
    terms = d[:, None, :] * y[inv]
    bar = (9 * -(-H // 512) + 12) * 2.0 ** -24 * np.abs(terms).sum(-1)
    assert np.all(np.abs(_f64(got["d_topk_w"]) - terms.sum(-1)) <= bar)
    # what is kept is the oracle's blocks of x and of the outputs
    plain = _forward(c)
    for pair, t in ((f["kept_x"], c["x"]), (f["kept_y"], plain["y_perm"])):
        for part, ref in zip(pair, om.quantize(_f64(t), "fp8")):
            assert np.array_equal(part.cpu().numpy(), ref)
    assert torch.equal(f["out"], plain["out"])
    assert f.get("x_perm") is None and "y_perm" not in f


@pytest.mark.parametrize("act", ["swiglu", "gelu"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_layer_backward_is_the_formulas(dtype, act):
    """Against the chain rule in float64 at x's kept values, and d_logits from y's kept ones."""
    c = _case(61, 6, 128, 192, 2, dtype, act, seed=3)
    f = _forward(c, keep="fp8")
    b = _backward(c, f)
    x = om.dequantize(*(t.cpu().numpy() for t in f["kept_x"]), "fp8", 128)
    y = om.dequantize(*(t.cpu().numpy() for t in f["kept_y"]), "fp8", 128)
    idx, w, d = f["idx"].cpu().numpy(), _f64(f["w"]), _f64(c["d_out"])
    ref = ob.layer_backward(x, idx, w, [None if t is None else _f64(t) for t in c["wts"]], act, d)
    bar = REL_FP32_GEMM if dtype == torch.float32 else 4 * REL_BF16
    for name in ("d_x", "d_w_gate", "d_w_down") + (("d_w_up",) if act == "swiglu" else ()):
        assert _rel(_f64(b[name]), ref[name]) <= bar, name
    dw = (d[:, None, :] * y[_f64(f["inv_pos"]).astype(int)]).sum(-1)
    d_logits = np.zeros((61, 6))
    np.put_along_axis(d_logits, idx.astype(int), w * (dw - (w * dw).sum(1, keepdims=True)), 1)
    assert _rel(_f64(b["d_logits"]), d_logits) <= REL_FP32_GEMM


def test_layer_backward_against_differences():
    """<grad, dir> against a central difference in float64, x being values that 8 bits hold.  A
    gradient is off by 1e-4 of its norm (its products), d_logits also by y's rounding (2^-4 of
    a value, 2^-10 of its block's scale); the difference, taken at two steps h and h / 2, is off
    by less than their distance (its error falls with h^2)."""
    T, E, H, I, k = 23, 5, 64, 128, 2
    c = _case(T, E, H, I, k, seed=5)
    c["x"] = moe.moe_mx_dequantize(*moe.moe_mx_quantize(c["x"], "fp8"), "fp8", torch.float32)
    f = _forward(c, keep="fp8")
    b = _backward(c, f)
    assert torch.equal(moe.moe_mx_dequantize(*f["kept_x"], "fp8", torch.float32), c["x"])
    idx = f["idx"].long().cpu()
    at = {"d_x": c["x"], "d_logits": c["logits"], "d_w_gate": c["wts"][0], "d_w_up": c["wts"][1], "d_w_down": c["wts"][2]}
    at = {name: t.double().cpu() for name, t in at.items()}
    d = c["d_out"].double().cpu()

    def outputs(p):
        w = torch.softmax(torch.gather(p["d_logits"], 1, idx), 1)
        ys = torch.stack([torch.stack([p["d_w_down"][e] @ (torch.nn.functional.silu(p["d_w_gate"][e] @ p["d_x"][t]) *
                                                           (p["d_w_up"][e] @ p["d_x"][t])) for e in idx[t]])
                          for t in range(T)])
        return w, ys

    def loss(p):
        w, ys = outputs(p)
        return float((w[:, :, None] * ys * d[:, None, :]).sum())

    w, ys = outputs(at)
    scale = moe.moe_mx_dequantize(torch.full_like(f["kept_y"][0], 0x38), f["kept_y"][1], "fp8", torch.float32)
    inv = f["inv_pos"].long().cpu()
    off = torch.maximum(ys.abs() * 2.0 ** -4, scale.double().cpu()[inv] * 2.0 ** -10) + 1e-4 * ys.abs()
    d_dw = (d.abs()[:, None, :] * off).sum(-1)
    gen = torch.Generator().manual_seed(9)
    for name, t in at.items():
        step = torch.randn(t.shape, generator=gen, dtype=torch.float64)
        diff = [(loss({**at, name: t + h * step}) - loss({**at, name: t - h * step})) / (2 * h) for h in (2e-4, 1e-4)]
        got = float((b[name].double().cpu() * step).sum())
        bar = 1e-4 * float(b[name].double().norm()) * float(step.norm()) + abs(diff[0] - diff[1]) + 1e-9
        if name == "d_logits":
            s = torch.gather(step, 1, idx).abs()
            bar += float((s * w * (d_dw + (w * d_dw).sum(1, keepdim=True))).sum())
        assert abs(got - diff[1]) <= bar, name


@pytest.mark.parametrize("gated", [False, True])
def test_layers_share_buffers_between_their_passes(gated):
    """Two layers on one set of buffers, as a step runs them: each backward pass finds what its forward kept."""
    norm = dict(weight=torch.linspace(0.5, 1.5, 128).cuda(), bias=torch.linspace(-1, 1, 128).cuda())
    opts = dict(norm=norm, gate=GATE if gated else None)
    cs = [_case(90, 8, 128, 192, 2, torch.bfloat16, seed=s) for s in (1, 2)]

    def step(shared):
        bufs, fs, x = {}, [], cs[0]["x"]
        for c in cs:
            f = moe.moe_layer_forward(x, c["logits"], 2, *c["wts"], residual=x, keep="fp8",
                                      bufs=bufs if shared else None, **opts)
            fs.append(f)
            x = f["normed"]
        grads = []
        for c, f in zip(cs, fs):
            grads.append(_backward(c, f, d_x_sum=c["d_out"], max_norm=0.5, **opts))
        return grads

    for a, b in zip(step(True), step(False)):
        assert set(a) == set(b) and "grad_norm" in a
        for name in a:
            assert torch.equal(a[name], b[name]), name


def test_keep_with_replicas_and_statistics():
    """Replica slots are the experts' parts of the same rows: the same gradients without them."""
    c = _case(200, 8, 128, 128, 2, seed=7)
    state = torch.empty(moe.moe_stats_state_bytes(1, 8, 4), dtype=torch.uint8, device="cuda")
    moe.moe_stats_init(state, 1, 8, 4)
    a = _backward(c, _forward(c, keep="fp8"))
    b = _backward(c, _forward(c, keep="fp8", replica_budget=5, stats_state=state, stats_dims=(1, 8, 4)))
    for name in a:
        assert torch.equal(a[name], b[name]), name


def _quantised(wts):
    return [None if w is None else moe.moe_mx_quantize(w, "fp4") for w in wts]


@pytest.mark.parametrize("x_format", ["fp6", "fp4"])
@pytest.mark.parametrize("size,act", [((1, 4, 128, 128, 1), "swiglu"), ((61, 8, 256, 128, 2), "gelu"),
                                      ((700, 6, 128, 384, 3), "swiglu")])
def test_layer_on_quantised_weights(size, act, x_format):
    """The layer is its calls, one after the other; cached buffers change nothing, nor does the copying dispatch."""
    c = _case(*size, torch.bfloat16, act)
    T, E, H, I, k = size
    wq = _quantised(c["wts"])
    check, bufs = moe.new_check_word(), {}
    run = lambda **kw: moe.moe_layer_forward(c["x"], c["logits"], k, *wq, act, x_format=x_format, check=check,  # noqa: E731
                                             **kw)
    f = run()
    y = moe.moe_mx_expert_ffn(c["x"], f["slot_off"], f["slot_expert"], f["n_slots"], *wq, act, x_format,
                              row_src=f["perm_src"])
    assert torch.equal(f["y_perm"], y)
    assert torch.equal(f["out"], moe.moe_combine(y, f["inv_pos"], f["w"]))
    for g in (run(bufs=bufs), run(bufs=bufs), run(copy_rows=True)):
        assert torch.equal(g["out"], f["out"])
    # float weights on the same buffers, and back
    moe.moe_layer_forward(c["x"], c["logits"], k, *c["wts"], act, bufs=bufs)
    assert torch.equal(run(bufs=bufs)["out"], f["out"])
    assert moe.moe_check_device_error(check) == 0


def test_layer_on_quantised_weights_with_options():
    """Gate, replicas, statistics, residual and norm as with float weights."""
    c = _case(333, 8, 128, 256, 2, torch.bfloat16, seed=4)
    wq = _quantised(c["wts"])
    state = torch.empty(moe.moe_stats_state_bytes(2, 8, 4), dtype=torch.uint8, device="cuda")
    moe.moe_stats_init(state, 2, 8, 4)
    f = moe.moe_layer_forward(c["x"], c["logits"], 2, *wq, replica_budget=4, stats_state=state, stats_dims=(2, 8, 4),
                              gate=GATE, residual=c["x"], norm={})
    y = moe.moe_mx_expert_ffn(c["x"], f["slot_off"], f["slot_expert"], f["n_slots"], *wq, row_src=f["perm_src"])
    assert int(f["n_slots"]) > 8 and torch.equal(f["y_perm"], y)
    normed, _ = moe.moe_layer_norm(moe.moe_combine(y, f["inv_pos"], f["w"]), residual=c["x"])
    assert torch.equal(f["normed"], normed)
    with pytest.raises(ValueError, match="no backward"):
        moe.moe_layer_backward(f, c["logits"], *c["wts"], c["d_out"], gate=GATE, norm={})


def test_training_then_serving():
    """All of it in a row: forward that keeps 8 bits, backward, clipped step, weights to 4 bits, a served layer;
    eager, captured and replayed, and on two streams at once."""
    cs = [_case(90, 8, 128, 256, 2, torch.bfloat16, seed=s) for s in (1, 2)]

    def run(c, stream=None):
        f = _forward(c, keep="fp8", stream=stream)
        b = _backward(c, f, max_norm=1.0, stream=stream)
        with torch.cuda.stream(stream) if stream is not None else torch.cuda.stream(torch.cuda.current_stream()):
            wts = [w - 0.1 * b[n] for w, n in zip(c["wts"], ("d_w_gate", "d_w_up", "d_w_down"))]
        wq = [moe.moe_mx_quantize(w, "fp4", stream=stream) for w in wts]
        s = moe.moe_layer_forward(c["x"], c["logits"], 2, *wq, stream=stream)
        return [b["d_x"], b["d_logits"], b["grad_norm"], s["out"]] + [t for q in wq for t in q]

    want = [run(c) for c in cs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [run(c, s) for c, s in zip(cs, streams)]
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        assert all(torch.equal(a, b) for a, b in zip(g, w))
    live = {key: cs[0][key].clone() for key in ("x", "logits", "d_out")}
    c = {**cs[0], **live, "wts": [w.clone() for w in cs[0]["wts"]]}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run(c)
    for r in (1, 0, 1):
        for key in live:
            c[key].copy_(cs[r][key])
        for w, new in zip(c["wts"], cs[r]["wts"]):
            w.copy_(new)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want[r]))
        assert all(torch.equal(a, b) for a, b in zip(run(cs[r]), want[r]))


def test_backward_mx_flags_rows_out_of_range():
    """A token outside the batch reads as a zero row, an expert row outside [0, M) is left out."""
    c = _case(12, 4, 64, 64, 2)
    f = _forward(c, keep="fp8")
    for name, at, bad in (("perm_src", 3, 12), ("perm_src", 0, -1), ("inv_pos", 5, 24), ("inv_pos", 0, -2)):
        check = moe.new_check_word()
        rows = {"perm_src": f["perm_src"].clone(), "inv_pos": f["inv_pos"].clone()}
        rows[name].view(-1)[at] = bad
        moe.moe_backward_mx(f["kept_x"], f["kept_y"], rows["perm_src"], f["w"], rows["inv_pos"], f["expert_off"], *c["wts"],
                            c["d_out"], check=check)
        with pytest.raises(moe.MoEError, match="out of range|outside"):
            moe.moe_check_device_error(check)


def test_backward_mx_of_nothing():
    c = _case(0, 4, 64, 64, 2)
    b = _backward(c, _forward(c, keep="fp8"))
    assert b["d_x"].shape == (0, 64) and not b["d_w_gate"].any() and not b["d_w_down"].any()


def test_layer_refusals():
    c = _case(8, 4, 128, 128, 2)
    wq = _quantised(c["wts"])
    x, lg = c["x"], c["logits"]
    for kw, msg in ((dict(keep="fp8"), "backward"), (dict(path="dense"), "path"), (dict(ffn_events=[1, 2, 3]), "ffn_events")):
        with pytest.raises(ValueError, match=msg):
            moe.moe_layer_forward(x, lg, 2, *wq, **kw)
    for kw, msg in ((dict(keep="fp4"), "fp8"), (dict(keep="fp8", copy_rows=True), "copy_rows"),
                    (dict(x_format="fp6"), "not quantised")):
        with pytest.raises(ValueError, match=msg):
            moe.moe_layer_forward(x, lg, 2, *c["wts"], **kw)
    with pytest.raises(ValueError, match="4-bit"):
        moe.moe_layer_forward_pipelined(x, lg, 2, *wq)
    f = moe.moe_layer_forward(x, lg, 2, *c["wts"], keep="fp8")
    with pytest.raises(ValueError, match="no backward"):
        moe.moe_layer_backward(f, lg, *wq, c["d_out"])
    run = lambda **kw: moe.moe_backward_mx(**{**dict(  # noqa: E731
        x=f["kept_x"], y_perm=f["kept_y"], perm_src=f["perm_src"], topk_w=f["w"], inv_pos=f["inv_pos"],
        expert_off=f["expert_off"], w_gate=c["wts"][0], w_up=c["wts"][1], w_down=c["wts"][2], d_out=c["d_out"]), **kw})
    assert set(run()) == {"d_x", "d_topk_w", "d_w_gate", "d_w_up", "d_w_down"}
    q, s = f["kept_x"]
    for kw in (dict(x=q), dict(x=(q, None)), dict(x=(q[:4], s)), dict(x=(q, s[:, :2])), dict(x=(c["x"], s)),
               dict(y_perm=f["kept_x"]), dict(perm_src=f["perm_src"][:3]), dict(perm_src=f["perm_src"].long()),
               dict(topk_w=f["w"].double()), dict(inv_pos=f["inv_pos"][:4]), dict(expert_off=f["expert_off"][:4]),
               dict(w_gate=c["wts"][0].bfloat16()), dict(w_down=c["wts"][2][:, :, :64]), dict(perm_src=None),
               dict(w_down=None), dict(workspace=torch.empty(16, dtype=torch.uint8, device="cuda")),
               dict(out=dict(d_x=torch.empty((8, 64), device="cuda"))), dict(check=torch.zeros(1, device="cuda"))):
        with pytest.raises(ValueError):
            run(**kw)
