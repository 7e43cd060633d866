"""The stream argument of every call: a torch stream, its integer handle, or an object
with a `cuda_stream`; with the call's own workspaces and outputs."""
import pytest
import torch

import mixture_experts_routing_top_amd as moe

pytestmark = pytest.mark.gpu


class Handle:
    def __init__(self, raw):
        self.cuda_stream = raw


def _forms(s):
    return {"stream": s, "integer": s.cuda_stream, "object": Handle(s.cuda_stream),
            "external": torch.cuda.ExternalStream(s.cuda_stream), "default": 0}


@pytest.mark.parametrize("form", ["stream", "integer", "object", "external", "default"])
def test_operators_take_every_form_of_a_stream(form):
    gen = torch.Generator().manual_seed(5)
    rnd = lambda *s: torch.randn(s, generator=gen).cuda()  # noqa: E731
    x, dy, w, lg = rnd(300, 512), rnd(300, 512), rnd(512), rnd(300, 64)
    grads = [rnd(5000), rnd(77)]
    runs = [lambda s: moe.moe_gate(lg, 4, score="sigmoid", stream=s),
            lambda s: (moe.moe_gate_backward(lg, idx, g, stream=s),),
            lambda s: moe.moe_layer_norm(x, w, w, residual=dy, stream=s),
            lambda s: tuple(moe.moe_layer_norm_backward(dy, x, w, w, stream=s).values()),
            lambda s: (moe.moe_grad_norm(grads, stream=s),),
            lambda s: (moe.moe_clip_grads(grads, 0.5, out=[torch.empty_like(g) for g in grads], stream=s)[0],)]
    idx, _ = moe.moe_gate(lg, 4)
    g = rnd(300, 4)
    want = [r(None) for r in runs]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for run, ref in zip(runs, want):
        got = run(_forms(s)[form])
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, ref))


def test_a_stream_that_is_none_is_refused():
    x = torch.randn(8, 64, device="cuda")
    for bad in ("stream", 1.5, object()):
        with pytest.raises(TypeError):
            moe.moe_layer_norm(x, stream=bad)


@pytest.mark.parametrize("form", ["stream", "integer", "object", "external", "default"])
def test_the_profiled_ffn_takes_every_form_of_a_stream(form):
    """Its events, whose handles do not exist before the call, are of that stream too."""
    gen = torch.Generator().manual_seed(6)
    rnd = lambda *s: torch.randn(s, generator=gen).cuda()  # noqa: E731
    x, lg = rnd(60, 128), rnd(60, 8)
    wts = [rnd(8, 192, 128), rnd(8, 192, 128), rnd(8, 128, 192)]
    want = moe.moe_layer_forward(x, lg, 2, *wts)["out"]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    events = [torch.cuda.Event(enable_timing=True) for _ in range(3)]
    got = moe.moe_layer_forward(x, lg, 2, *wts, ffn_events=events, stream=_forms(s)[form])["out"]
    torch.cuda.synchronize()
    assert torch.equal(got, want) and events[0].elapsed_time(events[2]) >= 0
