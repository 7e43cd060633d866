"""What a call on a stream other than the current one allocates belongs to that stream:
torch's allocator gives memory that a call drops back to the stream it was allocated on,
and a workspace of another stream could be handed out while its kernels still run.

On the CPU, with the library calls recorded instead of made and torch's streams and
allocations replaced by ones that say which stream is current."""
import contextlib

import pytest
import torch

import mixture_experts_routing_top_amd as moe


class FakeStream:
    def __init__(self, raw):
        self.cuda_stream = raw

    def wait_event(self, event):
        pass


class FakeEvent:
    def record(self, stream):
        pass


CURRENT, SIDE, OTHER = FakeStream(1), FakeStream(2), FakeStream(3)


@pytest.fixture
def allocations(monkeypatch):
    """[(stream, bytes)] of every allocation, as the calls make them."""
    now, log = [CURRENT], []

    @contextlib.contextmanager
    def on(stream):
        now.append(stream)
        try:
            yield
        finally:
            now.pop()

    def logged(fn):
        def run(*a, **kw):
            t = fn(*a, **kw)
            log.append((now[-1], t.numel() * t.element_size()))
            return t
        return run

    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: now[-1])
    monkeypatch.setattr(torch.cuda, "default_stream", lambda *a: FakeStream(0))
    monkeypatch.setattr(torch.cuda, "ExternalStream",
                        lambda raw, device=None: {s.cuda_stream: s for s in (CURRENT, SIDE, OTHER)}[raw])
    monkeypatch.setattr(torch.cuda, "Event", FakeEvent)
    monkeypatch.setattr(torch, "empty", logged(torch.empty))
    monkeypatch.setattr(torch, "empty_like", logged(torch.empty_like))
    monkeypatch.setattr(moe, "_ptr", lambda t: None)
    monkeypatch.setattr(moe, "_call", lambda name, *a: None)
    return log


T, E, K, H, I = 12, 8, 2, 64, 64


def _inputs():
    x, lg = torch.zeros((T, H)), torch.zeros((T, E))
    wts = [torch.zeros((E, I, H)), torch.zeros((E, I, H)), torch.zeros((E, H, I))]
    return x, lg, wts


def _i32(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def _calls():
    x, lg, wts = _inputs()
    idx, w, y = _i32(T, K), torch.zeros((T, K)), torch.zeros((T * K, H))
    state = torch.zeros(64, dtype=torch.uint8)
    return {
        "moe_route": lambda s: moe.moe_route(lg, K, stream=s),
        "moe_stats_load_state": lambda s: moe.moe_stats_load_state(state, 1, E, 4, 0, 0, stream=s),
        "moe_plan_replicas": lambda s: moe.moe_plan_replicas(torch.zeros(E), T * K, 4, stream=s),
        "moe_prediction_quality": lambda s: moe.moe_prediction_quality(torch.zeros(E), _i32(E), stream=s),
        "moe_dispatch": lambda s: moe.moe_dispatch(x, idx, E, stream=s),
        "moe_expert_ffn": lambda s: moe.moe_expert_ffn(y, _i32(E + 1), _i32(E), _i32(1), *wts, stream=s),
        "moe_combine": lambda s: moe.moe_combine(y, idx, w, stream=s),
        "moe_backward": lambda s: moe.moe_backward(y, y, idx, w, idx, _i32(E + 1), *wts, x, stream=s),
        "moe_layer_forward": lambda s: moe.moe_layer_forward(x, lg, K, *wts, stream=s),
        "moe_layer_forward, statistics": lambda s: moe.moe_layer_forward(
            x, lg, K, *wts, replica_budget=2, stats_state=state, stats_dims=(2, E, 4), stream=s),
    }


@pytest.mark.parametrize("form", ["stream", "handle"])
@pytest.mark.parametrize("call", list(_calls()))
def test_allocations_belong_to_the_calls_stream(allocations, call, form):
    run = _calls()[call]
    run(None)
    assert allocations and all(s is CURRENT for s, _ in allocations)
    sizes = sorted(n for _, n in allocations)
    allocations.clear()
    run(SIDE if form == "stream" else SIDE.cuda_stream)
    assert all(s is SIDE for s, _ in allocations)
    assert sorted(n for _, n in allocations) == sizes


@pytest.mark.parametrize("compute", [CURRENT, SIDE])
def test_pipelined_allocations_belong_to_a_stream_that_waits_for_their_use(allocations, compute):
    """What the compute stream's products use belongs to either stream of the call (each
    waits for the other's uses); with a compute stream that is not the current one,
    nothing belongs to the current one."""
    x, lg, wts = _inputs()
    bufs = {}
    moe.moe_layer_forward_pipelined(x, lg, K, *wts, n_chunks=3, compute_stream=None if compute is CURRENT else compute,
                                    memory_stream=OTHER, bufs=bufs)
    assert allocations and all(s in (compute, OTHER) for s, _ in allocations)
    need = moe.moe_expert_ffn_workspace_bytes(torch.float32, T // 3 * K, H, I, E)
    assert (compute, need) in allocations


@pytest.mark.parametrize("bad", [1.5, "7", b"7", None.__class__, object()])
def test_what_is_no_stream_is_refused(bad):
    """A number that is not whole is no handle: cut to one, it would name memory."""
    with pytest.raises(TypeError):
        moe._stream(bad)
    assert moe._stream(12).value == 12 and moe._stream(SIDE).value == 2 and moe._stream(0).value is None
