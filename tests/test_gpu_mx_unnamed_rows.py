"""moe_backward_mx where no entry of inv_pos names a row: the row counts as zero, whatever the
workspace held before.  A pair (token, slot) left out that way has the gradients of one whose
weight is 0, bit for bit: its row of d_y is zero in both."""
import pytest
import torch

import mixture_experts_routing_top_amd as moe
from test_gpu_mx_layer import _case, _forward

pytestmark = pytest.mark.gpu


def _run(c, f, act, w=None, inv=None, src=None, fill=0xFF, check=None):
    T, H = c["x"].shape
    E, I = c["wts"][0].shape[:2]
    ws = torch.full((moe.moe_backward_mx_workspace_bytes(c["x"].dtype, T, c["k"], H, I, E, act),), fill, dtype=torch.uint8,
                    device="cuda")
    return moe.moe_backward_mx(f["kept_x"], f["kept_y"], f["perm_src"] if src is None else src, f["w"] if w is None else w,
                               f["inv_pos"] if inv is None else inv, f["expert_off"], *c["wts"], c["d_out"], act,
                               workspace=ws, check=check)


@pytest.mark.parametrize("act", ["swiglu", "gelu"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("size", [(12, 4, 64, 64, 2), (301, 6, 192, 128, 3), (70, 3, 576, 64, 1)])
def test_left_out_is_weight_zero(size, dtype, act):
    c = _case(*size, dtype, act)
    f = _forward(c, keep="fp8")
    M = size[0] * size[4]
    at = torch.tensor([3, M - 1, M // 2])
    inv, w = f["inv_pos"].clone(), f["w"].clone()
    inv.view(-1)[at] = torch.tensor([-1, M, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    w.view(-1)[at] = 0
    check = moe.new_check_word()
    want = _run(c, f, act, w=w, fill=0)
    for fill in (0xFF, 0x7F, 0):
        got = _run(c, f, act, inv=inv, fill=fill, check=check)
        for name in set(want) - {"d_topk_w"}:
            assert torch.equal(got[name], want[name]), name
        named = torch.ones(M, dtype=torch.bool)
        named[at] = False
        a, b = got["d_topk_w"].view(-1), want["d_topk_w"].view(-1)
        assert torch.equal(a[named], b[named]) and not a[~named].any()
    with pytest.raises(moe.MoEError, match="outside"):
        moe.moe_check_device_error(check)


def test_tables_that_disagree_leave_nothing_stale():
    """Two entries with one row (another is named by none), and a perm_src of other tokens: still no row of the workspace
    as it was; rows that an entry names are its own whatever perm_src says."""
    c = _case(40, 4, 64, 64, 2)
    f = _forward(c, keep="fp8")
    inv = f["inv_pos"].clone()
    inv.view(-1)[7] = inv.view(-1)[6]
    a, b = (_run(c, f, "swiglu", inv=inv, fill=fill) for fill in (0xFF, 0))
    assert all(bool(t.isfinite().all()) for t in a.values())
    for name in ("d_topk_w", "d_w_gate", "d_w_up", "d_w_down", "d_x"):
        assert torch.equal(a[name], b[name]), name
    # perm_src moves x's rows alone: d_topk_w has no x in it, d_x is finite
    src = f["perm_src"].roll(1)
    a, b = _run(c, f, "swiglu", src=src), _run(c, f, "swiglu")
    assert torch.equal(a["d_topk_w"], b["d_topk_w"]) and all(bool(t.isfinite().all()) for t in a.values())
    src[5] = -1
    check = moe.new_check_word()
    assert all(bool(t.isfinite().all()) for t in _run(c, f, "swiglu", src=src, check=check).values())
    with pytest.raises(moe.MoEError, match="outside"):
        moe.moe_check_device_error(check)
