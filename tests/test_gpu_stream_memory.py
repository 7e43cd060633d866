"""Calls on a stream beside the current one, with work pending on both: neither stream's
memory is handed to the other while it is in use."""
import pytest
import torch

import mixture_experts_routing_top_amd as moe
from test_gpu_train_step import _case

pytestmark = pytest.mark.gpu

WAIT = 20_000_000     # cycles of a waiting kernel: some milliseconds


def _forms(s):
    return [s, s.cuda_stream]


def _step(c, stream):
    f = moe.moe_layer_forward(c["x"], c["logits"], c["k"], *c["wts"], gate=c["gate"], norm=c["norm"],
                              residual=c["x"], copy_rows=True, stream=stream)
    b = moe.moe_layer_backward(f, c["logits"], *c["wts"], c["d_normed"], gate=c["gate"], norm=c["norm"],
                               d_x_sum=c["d_x_sum"], max_norm=0.5, stream=stream)
    return [f["out"], f["normed"], f["x_sum"], f["w"]] + list(b.values())


@pytest.mark.parametrize("form", [0, 1], ids=["stream", "handle"])
def test_a_layer_on_another_stream_keeps_what_it_dropped(form):
    """Everything the step does not return is dropped while the step still waits on its
    stream, and the current stream allocates and fills meanwhile."""
    c = _case("sigmoid", torch.float32, T=700)
    ref = [t.clone() for t in _step(c, None)]
    sizes = [4 * n for n in (150, 700, 2100, 8192, 70_000, 500_000, 3_000_000)]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for _ in range(3):
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            torch.cuda._sleep(WAIT)
        got = _step(c, _forms(s)[form])
        junk = [torch.full((n // 4,), 1e9, device="cuda") for n in sizes for _ in range(4)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, ref))
        del got, junk


@pytest.mark.parametrize("form", [0, 1], ids=["stream", "handle"])
def test_pending_work_of_the_current_stream_does_not_meet_a_calls_outputs(form):
    """Tensors dropped on the current stream with a fill still to run there: a call on
    another stream, which has no reason to wait for it, gets other memory."""
    grads = [torch.randn(9000, device="cuda")]
    x, w = torch.randn(64, 512, device="cuda"), torch.randn(512, device="cuda")
    lg = torch.randn(64, 16, device="cuda")
    calls = [lambda s: (moe.moe_grad_norm(grads, stream=s),), lambda s: moe.moe_gate(lg, 4, stream=s),
             lambda s: moe.moe_route(lg, 4, stream=s), lambda s: moe.moe_layer_norm(x, w, residual=x, stream=s),
             lambda s: tuple(t for t in moe.moe_layer_norm_backward(x, x, w, stream=s).values() if t is not None)]
    ref = [c(None) for c in calls]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for call, want in zip(calls, ref):
        dropped = [torch.empty_like(t) for t in want for _ in range(3)]
        torch.cuda._sleep(WAIT)
        for t in dropped:
            t.fill_(7)
        del dropped, t
        got = call(_forms(s)[form])
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_a_call_on_another_stream_inside_a_capture():
    """A second stream of a capture: what the call allocates stays with the graph."""
    c = _case("softmax", torch.float32, T=90)
    side = torch.cuda.Stream()
    ref = [t.clone() for t in _step(c, None)]
    warm = torch.cuda.Stream()
    with torch.cuda.stream(warm):
        _step(c, None)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        got = _step(c, side)
        torch.cuda.current_stream().wait_stream(side)
    for rep in range(3):
        for t in got:
            t.fill_(-7.0)
        junk = [torch.full((n,), 1e9, device="cuda") for n in (300, 9000, 70_000, 900_000)]
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, ref)), rep
        del junk
