"""What a workspace, an output or a CU's LDS held before changes no result of the calls on
microscaled blocks: bit for bit the same over buffers of zeros, of ones (NaN codes, scales
and floats) and after products of NaN on every CU."""
import pytest
import torch

import mixture_experts_routing_top_amd as moe
from test_gpu_mx import X_FORMATS, _rows, _table, _weights
from test_gpu_mx_layer import _case, _forward

pytestmark = pytest.mark.gpu


# the stream, 64-, 128- and 256-row tiles, whole and ragged, even and odd K steps; spare slots
@pytest.mark.parametrize("counts,H,I", [([1, 0, 2], 640, 384), ([40, 64, 9, 0], 384, 1152), ([130, 90, 128], 1024, 640),
                                        ([400, 300, 261], 2176, 384)])
@pytest.mark.parametrize("act", ["swiglu", "gelu"])
@pytest.mark.parametrize("fmt", X_FORMATS)
def test_ffn_reads_only_what_it_wrote(fmt, act, counts, H, I):
    E, M = len(counts), sum(counts)
    x = _rows((M + 3, H), torch.bfloat16, H)
    rows = torch.randperm(M + 3, generator=torch.Generator().manual_seed(1))[:M].int().cuda()
    wts = (_weights(E, I, H, 1), _weights(E, I, H, 2) if act == "swiglu" else None, _weights(E, H, I, 3))
    table = _table(counts, max_slots=E + 2)
    ws = torch.empty(moe.moe_mx_expert_ffn_workspace_bytes(M, H, I, E + 2, fmt), dtype=torch.uint8, device="cuda")
    y = torch.empty((M, H), dtype=torch.bfloat16, device="cuda")
    nan = torch.full_like(x, float("nan"))
    got = []
    for byte in (0, 0xFF, 0x7F, 0xFF):
        if byte == 0xFF:
            moe.moe_mx_expert_ffn(nan, *table, *wts, act, fmt, row_src=rows)
        ws.fill_(byte)
        y.view(torch.uint8).fill_(byte)
        moe.moe_mx_expert_ffn(x, *table, *wts, act, fmt, y_perm=y, workspace=ws, row_src=rows)
        got.append(y.clone())
    assert bool(got[0].isfinite().all())
    assert all(torch.equal(got[0].view(torch.int16), g.view(torch.int16)) for g in got[1:])


# rows before the first slot, behind the last one and (from an expert out of range on) of a slot that is skipped
@pytest.mark.parametrize("off,H,tail", [([2, 5, 9], 384, 4), ([3, 40, 41], 384, 30), ([70, 150, 290], 640, 60),
                                        ([5, 300, 520], 2176, 290)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("fmt", X_FORMATS)
def test_ffn_leaves_rows_of_no_slot(fmt, dtype, off, H, tail):
    I, M = 256, off[-1] + tail
    x = _rows((M, H), dtype, H)
    wts = (_weights(2, I, H, 1), _weights(2, I, H, 2), _weights(2, H, I, 3))
    dev = dict(dtype=torch.int32, device="cuda")
    for experts in ([1, 0], [1, 2]):
        table = torch.tensor(off, **dev), torch.tensor(experts, **dev), torch.tensor([2], **dev)
        want = moe.moe_mx_expert_ffn(x, *table, *wts, x_format=fmt)
        there = torch.zeros(M, dtype=torch.bool, device="cuda")
        there[off[0]:off[2] if experts[1] == 0 else off[1]] = True
        rows = torch.where(there[:, None], x, torch.full_like(x, float("nan")))   # (their x is nobody's)
        y = moe.moe_mx_expert_ffn(rows, *table, *wts, x_format=fmt, y_perm=torch.full_like(x, 7.0))
        assert bool(want[there].isfinite().all())
        assert torch.equal(y[there], want[there]) and bool((y[~there] == 7).all())


@pytest.mark.parametrize("act", ["swiglu", "gelu"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("size", [(1, 4, 64, 64, 1), (37, 6, 128, 192, 2), (700, 8, 576, 64, 8)])
def test_backward_mx_reads_only_what_it_wrote(size, dtype, act):
    c = _case(*size, dtype, act)
    f = _forward(c, keep="fp8")
    T, E, H, I, k = size
    ws = torch.empty(moe.moe_backward_mx_workspace_bytes(dtype, T, k, H, I, E, act), dtype=torch.uint8, device="cuda")
    got = []
    for byte in (0, 0xFF, 0x7F):
        ws.fill_(byte)
        out = moe.moe_backward_mx(f["kept_x"], f["kept_y"], f["perm_src"], f["w"], f["inv_pos"], f["expert_off"], *c["wts"],
                                  c["d_out"], act, workspace=ws)
        got.append(out)
    assert all(bool(t.isfinite().all()) for t in got[0].values())
    for g in got[1:]:
        assert all(torch.equal(got[0][name], g[name]) for name in got[0])


@pytest.mark.parametrize("fmt", ["fp4", "fp6", "fp8"])
@pytest.mark.parametrize("shape", [(3, 33), (130, 256), (7, 4095)])
def test_every_byte_of_the_outputs_is_written(fmt, shape):
    x = _rows(shape, torch.float32, 2)
    q, s = moe.moe_mx_quantize(x, fmt)
    for byte in (0, 0xFF):
        pair = moe.moe_mx_quantize(x, fmt, q=torch.full_like(q, byte), scale=torch.full_like(s, byte))
        assert torch.equal(pair[0], q) and torch.equal(pair[1], s)
        out = torch.empty_like(x)
        out.view(torch.uint8).fill_(byte)
        back = moe.moe_mx_dequantize(q, s, fmt, torch.float32, cols=shape[1], out=out)
        assert torch.equal(back, moe.moe_mx_dequantize(q, s, fmt, torch.float32, cols=shape[1]))
