"""Refusals of the microscaled-block calls, on the CPU: every one is reported before
anything reaches the GPU.  Workspace sizes."""
import ctypes

import pytest
import torch

import mixture_experts_routing_top_amd as moe
from mixture_experts_routing_top_amd import _native
from test_stream_memory import SIDE, allocations  # noqa: F401

N, P, BIG = None, 16, 1 << 40


def _ffn(x=P, rows=N, n_src=8, dt=1, M=8, H=128, I=256, E=4, off=P, se=P, ns=P, slots=4, wg=P, sg=P, wu=P, su=P, wd=P,
         sd=P, act=0, fmt=2, y=P, ws=P, wb=BIG):
    return ("moe_mx_expert_ffn", (x, rows, n_src, dt, M, H, I, E, off, se, ns, slots, wg, sg, wu, su, wd, sd, act, fmt, y, ws,
                                  wb, N, N))


def _combine(d_out=P, dt=1, y=P, ys=P, M=16, inv=P, w=P, T=8, k=2, H=64, d_y=P, d_w=P):
    return ("moe_combine_backward", (d_out, dt, y, ys, M, inv, w, T, k, H, d_y, d_w, N, N))


def _backward(x=P, xs=P, y=P, ys=P, dt=1, T=8, k=2, H=64, I=64, E=4, src=P, w=P, inv=P, off=P, wg=P, wu=P, wd=P, act=0,
              d_out=P, d_x=P, d_w=P, dg=P, du=P, dd=P, ws=P, size=1 << 50):
    return "moe_backward_mx", (x, xs, y, ys, dt, T, k, H, I, E, src, w, inv, off, wg, wu, wd, act, d_out, d_x, d_w, dg, du,
                               dd, ws, size, N, N)


@pytest.mark.parametrize("call,status,msg", [
    (_backward(dt=2), -1, "dtype"), (_backward(act=2), -1, "activation"), (_backward(E=0), -1, "E=0"),
    (_backward(E=300), -2, "E=300"), (_backward(k=5), -1, "k=5"), (_backward(k=0), -1, "k=0"), (_backward(T=-1), -1, "T"),
    (_backward(H=96), -2, "multiples of 64"), (_backward(I=32), -2, "multiples of 64"),
    (_ffn(M=(1 << 14) - 1, I=1 << 22, slots=1 << 20), -2, "tiles in one launch"),
    (_combine(T=(1 << 25) + 1, M=1 << 27), -2, "2\\^25 tokens"),
    (_backward(T=(1 << 25) + 1, k=1, dt=0), -2, "too large|2\\^25"),
    (_backward(T=1 << 20, k=2, H=1 << 17), -2, "2\\^30 blocks"),
    (_backward(wu=N), -1, "w_up"), (_backward(act=1), -1, "GELU"), (_backward(size=100), -3, "workspace"),
    (_backward(ws=N), -1, "null"), (_backward(x=N), -1, "null"), (_backward(xs=N), -1, "null"), (_backward(y=N), -1, "null"),
    (_backward(ys=N), -1, "null"), (_backward(src=N), -1, "null"), (_backward(w=N), -1, "null"),
    (_backward(inv=N), -1, "null"), (_backward(off=N), -1, "null"), (_backward(d_out=N), -1, "null"),
    (_backward(d_x=N), -1, "null"), (_backward(d_w=N), -1, "null"), (_backward(dg=N), -1, "null"),
    (_backward(dd=N), -1, "null"), (_backward(du=N), -1, "null"), (_backward(y=P + 8), -1, "aligned"),
    (_backward(d_out=P + 4), -1, "aligned"),
    (("moe_mx_quantize", (P, 2, 4, 64, 0, P, P, N, N)), -1, "dtype"),
    (("moe_mx_quantize", (P, 1, 4, 64, 3, P, P, N, N)), -1, "format"),
    (("moe_mx_quantize", (P, 1, -1, 64, 0, P, P, N, N)), -1, "rows"),
    (("moe_mx_quantize", (P, 1, 4, 0, 0, P, P, N, N)), -1, "K=0"),
    (("moe_mx_quantize", (P, 1, 4, 1 << 29, 0, P, P, N, N)), -1, "K="),
    (("moe_mx_quantize", (P, 1, 1 << 32, 64, 0, P, P, N, N)), -2, "2\\^30 blocks"),
    (("moe_mx_quantize", (N, 1, 4, 64, 0, P, P, N, N)), -1, "null"),
    (("moe_mx_quantize", (P, 1, 4, 64, 0, P, N, N, N)), -1, "null"),
    (("moe_mx_quantize", (N, 1, 0, 64, 0, N, N, N, N)), 0, ""),
    (("moe_mx_dequantize", (P, P, 5, 4, 64, N, 0, 1, P, N, N)), -1, "format"),
    (("moe_mx_dequantize", (P, P, 0, 4, 64, N, 0, 7, P, N, N)), -1, "dtype"),
    (("moe_mx_dequantize", (P, P, 0, 4, 64, P, -3, 1, P, N, N)), -1, "rows"),
    (("moe_mx_dequantize", (P, P, 0, 4, 64, P, 1 << 33, 1, P, N, N)), -2, "blocks"),
    (("moe_mx_dequantize", (N, P, 0, 4, 64, N, 0, 1, P, N, N)), -1, "null"),
    (("moe_mx_dequantize", (P, P, 0, 4, 64, N, 0, 1, N, N, N)), -1, "null"),
    (("moe_mx_dequantize", (N, N, 0, 4, 64, P, 0, 1, N, N, N)), 0, ""),
    (_combine(dt=3), -1, "dtype"),
    (_combine(k=9), -1, "k=9"),
    (_combine(k=0), -1, "k=0"),
    (_combine(T=-1), -1, "T or M"),
    (_combine(T=1 << 30), -1, "T or M"),
    (_combine(H=60), -1, "multiple of 8"),
    (_combine(H=0), -1, "multiple of 8"),
    (_combine(inv=N), -1, "null"),
    (_combine(d_y=N), -1, "null"),
    (_combine(y=8), -1, "aligned"),
    (_combine(d_out=24), -1, "aligned"),
    (_combine(T=0, d_out=N, y=N, inv=N, w=N, d_y=N, d_w=N), 0, ""),
    (_ffn(dt=2), -1, "dtype"),
    (_ffn(act=2), -1, "activation"),
    (_ffn(fmt=1), -1, "x_format"),
    (_ffn(M=-1), -1, "M out of range"),
    (_ffn(M=1 << 31), -1, "M out of range"),
    (_ffn(rows=P, n_src=-1), -1, "n_src"),
    (_ffn(H=192), -2, "multiples of 128"),
    (_ffn(I=64), -2, "multiples of 128"),
    (_ffn(H=1 << 16, I=1 << 16), -2, "32-bit offsets"),
    (_ffn(H=1 << 23, I=128), -2, "32-bit offsets"),
    (_ffn(M=1 << 29), -2, "2\\^36 values"),
    (_ffn(E=0), -1, "E <= max_slots"),
    (_ffn(E=5), -1, "E <= max_slots"),
    (_ffn(wu=N), -1, "w_up"),
    (_ffn(su=N), -1, "w_up"),
    (_ffn(act=1), -1, "GELU"),
    (_ffn(sd=N), -1, "null"),
    (_ffn(off=N), -1, "null"),
    (_ffn(y=N), -1, "null"),
    (_ffn(x=N), -1, "null"),
    (_ffn(wd=24), -1, "aligned"),
    (_ffn(wb=1000), -3, "workspace"),
    (_ffn(M=0, x=N, y=N), 0, ""),
])
def test_refusals(call, status, msg):
    import re
    lib = _native.lib()
    name, args = call
    assert getattr(lib, name)(*args) == status, lib.moe_last_error()
    if status:
        assert re.search(msg, lib.moe_last_error().decode()), lib.moe_last_error()


@pytest.mark.parametrize("M,H,I,slots", [(0, 128, 128, 1), (6, 5120, 1536, 160), (2048, 256, 384, 12)])
def test_workspace_holds_what_the_call_keeps(M, H, I, slots):
    for fmt, bits in (("fp4", 4), ("fp6", 6)):
        held = M * (H + I) * bits // 8 + M * (H + I) // 32 + 16 * min(M, slots) + 4
        got = moe.moe_mx_expert_ffn_workspace_bytes(M, H, I, slots, fmt)
        assert held <= got <= held + 16 * (M // 16) + 8 * 256
    assert _native.lib().moe_mx_expert_ffn_workspace_bytes(-1, 128, 128, 1, 0) == 0
    assert _native.lib().moe_mx_expert_ffn_workspace_bytes(8, 128, 128, 1, 1) == 0


def test_the_binding_checks_its_arguments():
    x = torch.zeros((4, 64))
    for call in (lambda: moe.moe_mx_quantize(x), lambda: moe.moe_mx_dequantize(x.byte(), x.byte()),
                 lambda: moe.moe_combine_backward(x, x, x.int(), x)):
        with pytest.raises(ValueError, match="GPU"):
            call()
    with pytest.raises(TypeError):
        moe.moe_mx_quantize(x.half())
    with pytest.raises(TypeError):
        moe.moe_mx_quantize([1.0])
    with pytest.raises(KeyError):
        moe.moe_mx_quantize(x, "fp5")
    with pytest.raises(TypeError, match="float32 or bfloat16"):
        moe.moe_mx_dequantize(x.byte(), x.byte(), dtype=torch.float16)


def test_backward_mx_workspace():
    """moe_backward's and x_perm."""
    for dt, size in ((torch.float32, 4), (torch.bfloat16, 2)):
        base = moe.moe_backward_workspace_bytes(dt, 100, 2, 128, 192, 8)
        got = moe.moe_backward_mx_workspace_bytes(dt, 100, 2, 128, 192, 8)
        assert base + 200 * 128 * size <= got <= base + 200 * 128 * size + 256
    assert _native.lib().moe_backward_mx_workspace_bytes(2, 8, 2, 64, 64, 4, 0) == 0


@pytest.mark.parametrize("form", ["stream", "handle"])
def test_backward_mx_allocates_on_its_stream(allocations, form):
    T, E, k, H, I = 12, 8, 2, 64, 64
    x, inv = torch.zeros((T, H)), torch.zeros((T, k), dtype=torch.int32)
    wts = [torch.zeros((E, I, H)), torch.zeros((E, I, H)), torch.zeros((E, H, I))]
    kept = [(torch.zeros((n, H), dtype=torch.uint8), torch.zeros((n, H // 32), dtype=torch.uint8)) for n in (T, T * k)]
    allocations.clear()
    moe.moe_backward_mx(*kept, inv.view(-1), torch.zeros((T, k)), inv, torch.zeros(E + 1, dtype=torch.int32), *wts, x,
                        stream=SIDE if form == "stream" else SIDE.cuda_stream)
    assert len(allocations) == 6 and all(s is SIDE for s, _ in allocations)


def test_layer_refusals_need_no_gpu():
    x, lg = torch.zeros((4, 128)), torch.zeros((4, 4))
    w = torch.zeros((4, 128, 128))
    pair = (torch.zeros((4, 128, 64), dtype=torch.uint8), torch.zeros((4, 128, 4), dtype=torch.uint8))
    for wts, kw in (((pair, pair, pair), dict(keep="fp8")), ((pair, pair, pair), dict(path="dense")), ((w, w, w), dict(keep="fp6")),
                    ((w, w, w), dict(keep="fp8", copy_rows=True)), ((w, w, w), dict(x_format="fp4"))):
        with pytest.raises(ValueError):
            moe.moe_layer_forward(x, lg, 2, *wts, **kw)
    with pytest.raises(ValueError, match="no backward"):
        moe.moe_layer_backward({"x_format": "fp6", "x_perm": x}, lg, w, w, w, x)
    with pytest.raises(ValueError, match="keep="):
        moe.moe_layer_backward({}, lg, w, w, w, x)
