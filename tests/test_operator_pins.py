"""The float64 oracle of the gate, layer norm and clipping, pinned on the CPU by
worked values, torch autograd and differences; and the library's refusals,
which reach no GPU."""
import ctypes
import math

import numpy as np
import pytest
import torch

from mixture_experts_routing_top_amd import _native
from oracle import operators as oo


def test_gate_worked_example():
    # groups {0,1} {2,3} {4,5}; sigmoid scores 0.5 0.8 0.9 0.1 0.75 0.76; the bias
    # lifts expert 0; top2 sums 1.8, 1.0, 1.51: groups 0 and 2 stay
    s = np.array([0.5, 0.8, 0.9, 0.1, 0.75, 0.76])
    row = np.log(s / (1 - s))
    bias = np.array([0.5, 0, 0, 0, 0, 0.0])
    idx, w = oo.gate_row(row, 3, score="sigmoid", bias=bias, n_groups=3, keep_groups=2, group_score="top2", scale=2.0)
    assert idx.tolist() == [0, 1, 5]
    assert np.allclose(w, 2.0 * np.array([0.5, 0.8, 0.76]) / 2.06)
    # by the best expert alone: 1.0, 0.9, 0.76
    idx, w = oo.gate_row(row, 3, score="sigmoid", bias=bias, n_groups=3, keep_groups=2, renorm=False)
    assert idx.tolist() == [0, 2, 1] and np.allclose(w, [0.5, 0.9, 0.8])


def test_gate_masks_ties_and_empty_rows():
    idx, w = oo.gate_row(np.array([-math.inf, 1.0, 1.0, math.nan]), 4)
    assert idx.tolist() == [1, 2, 0, 3] and w.tolist() == [0.5, 0.5, 0, 0]
    idx, w = oo.gate_row(np.full(4, -3.4e38), 2, score="sigmoid", n_groups=2, keep_groups=1)
    assert idx.tolist() == [0, 1] and w.tolist() == [0, 0]
    # sigmoids that underflow keep their ratios under renormalisation
    _, w = oo.gate_row(np.array([-900.0, -901.0, -2000.0]), 2, score="sigmoid")
    assert np.allclose(w, [1 / (1 + math.exp(-1)), math.exp(-1) / (1 + math.exp(-1))])


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_gate_backward_against_autograd_and_differences(score, renorm):
    rng = np.random.default_rng(1)
    lg = rng.standard_normal((5, 12))
    idx, _ = oo.gate(lg, 4, score=score, renorm=renorm, scale=1.5)
    g = rng.standard_normal((5, 4))
    t = torch.tensor(lg, requires_grad=True)
    s = torch.softmax(t, 1) if score == "softmax" else torch.sigmoid(t)
    k = torch.gather(s, 1, torch.tensor(idx).long())
    w = 1.5 * (k / k.sum(1, keepdim=True) if renorm else k)
    (w * torch.tensor(g)).sum().backward()
    d = oo.gate_backward(lg, idx, g, score, renorm, 1.5)
    assert np.allclose(d, t.grad.numpy(), rtol=1e-12, atol=1e-14)
    h = 1e-6
    for t0, e in ((0, int(idx[0, 0])), (3, int(idx[3, 2])), (4, 7)):
        v = []
        for sign in (1, -1):
            moved = lg.copy()
            moved[t0, e] += sign * h
            i2, w2 = oo.gate(moved, 4, score=score, renorm=renorm, scale=1.5)
            assert np.array_equal(i2, idx)
            v.append(float((w2 * g).sum()))
        assert abs((v[0] - v[1]) / (2 * h) - d[t0, e]) < 1e-7


def test_layer_norm_backward_against_autograd_and_differences():
    rng = np.random.default_rng(2)
    x, dy, w, b = rng.standard_normal((6, 9)), rng.standard_normal((6, 9)), rng.standard_normal(9), rng.standard_normal(9)
    t, tw, tb = (torch.tensor(a, requires_grad=True) for a in (x, w, b))
    y = torch.nn.functional.layer_norm(t, (9,), tw, tb, 1e-3)
    assert np.allclose(oo.layer_norm(x, w, b, 1e-3), y.detach().numpy(), rtol=1e-12)
    (y * torch.tensor(dy)).sum().backward()
    d = oo.layer_norm_backward(dy, x, w, 1e-3)
    for key, ref in (("d_x", t.grad), ("d_weight", tw.grad), ("d_bias", tb.grad)):
        assert np.allclose(d[key], ref.numpy(), rtol=1e-11, atol=1e-13), key
    h = 1e-6
    up, down = x.copy(), x.copy()
    up[2, 4] += h
    down[2, 4] -= h
    slope = ((oo.layer_norm(up, w, b, 1e-3) - oo.layer_norm(down, w, b, 1e-3)) * dy).sum() / (2 * h)
    assert abs(slope - d["d_x"][2, 4]) < 1e-7


def test_clip_worked_example():
    norm, out = oo.clip([np.array([3.0, 0.0]), np.array([[4.0]])], 1.0, eps=5.0)
    assert norm == 5.0 and out[0].tolist() == [0.30000000000000004, 0.0] and out[1].tolist() == [[0.4]]
    assert oo.clip([np.array([3.0, 4.0])], 100.0)[1][0].tolist() == [3.0, 4.0]


N = None
F32, BF16 = 0, 1


def _list(n, ptrs, counts, types):
    return (ctypes.c_void_p * n)(*ptrs), (ctypes.c_int64 * n)(*counts), (ctypes.c_int * n)(*types)


@pytest.mark.parametrize("call,args,status,msg", [
    ("moe_gate", (16, 2, 4, 8, 2, 0, N, 1, 1, 0, 1, 1.0, 16, 16, N, N), -1, "dtype"),
    ("moe_gate", (16, F32, 4, 0, 1, 0, N, 1, 1, 0, 1, 1.0, 16, 16, N, N), -1, "E=0"),
    ("moe_gate", (16, F32, 4, 257, 2, 0, N, 1, 1, 0, 1, 1.0, 16, 16, N, N), -2, "E=257"),
    ("moe_gate", (16, F32, 4, 64, 9, 0, N, 1, 1, 0, 1, 1.0, 16, 16, N, N), -1, "k=9"),
    ("moe_gate", (16, F32, 4, 4, 5, 0, N, 1, 1, 0, 1, 1.0, 16, 16, N, N), -1, "k=5"),
    ("moe_gate", (16, F32, 4, 8, 2, 2, N, 1, 1, 0, 1, 1.0, 16, 16, N, N), -1, "score 2"),
    ("moe_gate", (16, F32, 4, 8, 2, 0, N, 1, 1, 2, 1, 1.0, 16, 16, N, N), -1, "group score 2"),
    ("moe_gate", (16, F32, 4, 8, 2, 0, N, 3, 1, 0, 1, 1.0, 16, 16, N, N), -1, "n_groups=3"),
    ("moe_gate", (16, F32, 4, 8, 2, 0, N, 0, 1, 0, 1, 1.0, 16, 16, N, N), -1, "n_groups=0"),
    ("moe_gate", (16, F32, 4, 130, 2, 0, N, 65, 2, 0, 1, 1.0, 16, 16, N, N), -2, "n_groups=65"),
    ("moe_gate", (16, F32, 4, 8, 3, 0, N, 4, 1, 0, 1, 1.0, 16, 16, N, N), -1, "keep_groups=1"),
    ("moe_gate", (16, F32, 4, 8, 2, 0, N, 2, 3, 0, 1, 1.0, 16, 16, N, N), -1, "keep_groups=3"),
    ("moe_gate", (16, F32, -1, 8, 2, 0, N, 1, 1, 0, 1, 1.0, 16, 16, N, N), -1, "T=-1"),
    ("moe_gate", (16, F32, 1 << 30, 8, 2, 0, N, 1, 1, 0, 1, 1.0, 16, 16, N, N), -1, "out of range"),
    ("moe_gate", (16, F32, 4, 8, 2, 0, N, 1, 1, 0, 1, math.nan, 16, 16, N, N), -1, "scale"),
    ("moe_gate", (N, F32, 4, 8, 2, 0, N, 1, 1, 0, 1, 1.0, 16, 16, N, N), -1, "null"),
    ("moe_gate", (16, F32, 4, 8, 2, 0, N, 1, 1, 0, 1, 1.0, 16, N, N, N), -1, "null"),
    ("moe_gate_backward", (16, F32, 4, 8, 2, 3, 1, 1.0, 16, 16, 16, N, N), -1, "score 3"),
    ("moe_gate_backward", (16, F32, 4, 8, 2, 0, 1, math.inf, 16, 16, 16, N, N), -1, "scale"),
    ("moe_gate_backward", (16, F32, 4, 8, 2, 0, 1, 1.0, 16, N, 16, N, N), -1, "null"),
    ("moe_layer_norm", (16, N, 2, 4, 8, N, N, 0, 1e-5, N, 16, N), -1, "dtype"),
    ("moe_layer_norm", (16, N, F32, 4, 8, 16, N, BF16, 1e-5, N, 16, N), -1, "float32 or of the rows"),
    ("moe_layer_norm", (16, N, F32, 4, 0, N, N, F32, 1e-5, N, 16, N), -1, "H=0"),
    ("moe_layer_norm", (16, N, F32, 4, 16385, N, N, F32, 1e-5, N, 16, N), -2, "H=16385"),
    ("moe_layer_norm", (16, N, F32, -4, 8, N, N, F32, 1e-5, N, 16, N), -1, "T=-4"),
    ("moe_layer_norm", (16, N, F32, 4, 8, N, N, F32, 0.0, N, 16, N), -1, "eps"),
    ("moe_layer_norm", (16, N, F32, 4, 8, N, N, F32, math.nan, N, 16, N), -1, "eps"),
    ("moe_layer_norm", (16, 32, F32, 4, 8, N, N, F32, 1e-5, N, 16, N), -1, "x_sum"),
    ("moe_layer_norm", (16, N, F32, 4, 8, N, N, F32, 1e-5, 32, 16, N), -1, "x_sum"),
    ("moe_layer_norm", (16, 32, F32, 4, 8, N, N, F32, 1e-5, 64, 64, N), -1, "same buffer"),
    ("moe_layer_norm", (18, N, F32, 4, 8, N, N, F32, 1e-5, N, 16, N), -1, "misaligned"),
    ("moe_layer_norm", (16, N, F32, 4, 8, N, N, F32, 1e-5, N, N, N), -1, "null"),
    ("moe_layer_norm_backward", (16, N, F32, 4, 8, N, F32, 1e-5, N, 16, N, N, N, 0, N), -1, "null"),
    ("moe_layer_norm_backward", (16, 16, F32, 4, 8, 16, F32, 1e-5, N, 32, 16, N, N, 0, N), -3, "workspace"),
    ("moe_layer_norm_backward", (16, 16, F32, 4, 8, 16, F32, 1e-5, N, 32, 16, N, 16, 4, N), -3, "workspace"),
    ("moe_layer_norm_backward", (16, 16, F32, 4, 8, 16, F32, 1e-5, N, 32, 16, N, 24, 1 << 20, N), -1, "16-byte"),
    ("moe_layer_norm_backward", (16, 16, BF16, 4, 8, 16, F32, 1e-5, N, 33, 16, N, 16, 1 << 20, N), -1, "misaligned"),
    ("moe_grad_norm", (N, N, N, 2, 16, 16, 8192, N, N), -1, "null list"),
    ("moe_grad_norm", (*_list(1, [16], [4], [7]), 1, 16, 16, 8192, N, N), -1, "dtype 7"),
    ("moe_grad_norm", (*_list(1, [16], [-4], [0]), 1, 16, 16, 8192, N, N), -1, "size -4"),
    ("moe_grad_norm", (*_list(1, [N], [4], [0]), 1, 16, 16, 8192, N, N), -1, "null tensor"),
    ("moe_grad_norm", (*_list(1, [18], [4], [0]), 1, 16, 16, 8192, N, N), -1, "misaligned"),
    ("moe_grad_norm", (*_list(1, [16], [4], [0]), 1, N, 16, 8192, N, N), -1, "null norm"),
    ("moe_grad_norm", (*_list(1, [16], [4], [0]), 1, 16, 16, 100, N, N), -3, "workspace"),
    ("moe_grad_norm", (*_list(1, [16], [4], [0]), -1, 16, 16, 8192, N, N), -1, "n=-1"),
])
def test_operators_refuse_bad_arguments_before_any_hip_call(call, args, status, msg):
    lib = _native.lib()
    rc = getattr(lib, call)(*args)
    assert rc == status, (rc, lib.moe_last_error())
    assert msg in lib.moe_last_error().decode()


@pytest.mark.parametrize("ptrs,outs,counts,types,max_norm,msg", [
    ([4096, 4096], [4096, 4096], [8, 8], [0, 0], 1.0, "overlaps"),              # one tensor twice
    ([4096, 8192], [4096, 4112], [8, 8], [0, 0], 1.0, "overlaps"),              # outputs overlap
    ([4096, 8192], [16384, 4100], [8, 8], [0, 0], 1.0, "overlaps"),             # an output in another gradient
    ([4096], [4100], [8], [0], 1.0, "overlaps"),                                # shifted on itself
    ([4096, 4128], [4096, 4128], [8, 8], [0, 0], -1.0, "max_norm"),
    ([4096], [4096], [8], [0], math.inf, "max_norm"),
    ([4096], [None], [8], [0], 1.0, "null output"),
    ([4096], [4098], [8], [0], 1.0, "misaligned"),
])
def test_clip_refuses_overlaps(ptrs, outs, counts, types, max_norm, msg):
    lib = _native.lib()
    n = len(ptrs)
    p, c, t = _list(n, ptrs, counts, types)
    rc = lib.moe_clip_grads(p, (ctypes.c_void_p * n)(*outs), c, t, n, max_norm, 1e-6, 16, 16, 8192, None, None)
    assert rc == -1 and msg in lib.moe_last_error().decode()


def test_operator_workspace_queries():
    lib = _native.lib()
    assert lib.moe_layer_norm_backward_workspace_bytes(0, 64) == 0
    assert lib.moe_layer_norm_backward_workspace_bytes(1, 63) >= 2 * 63 * 4
    assert lib.moe_layer_norm_backward_workspace_bytes(4, 20000) == 0
    assert 0 < lib.moe_grad_norm_workspace_bytes() <= 8192


def test_empty_batches_return_at_once():
    lib = _native.lib()
    assert lib.moe_gate(None, F32, 0, 8, 2, 0, None, 1, 1, 0, 1, 1.0, None, None, None, None) == 0
    assert lib.moe_gate_backward(None, F32, 0, 8, 2, 0, 1, 1.0, None, None, None, None, None) == 0
    assert lib.moe_layer_norm(None, None, F32, 0, 8, None, None, F32, 1e-5, None, None, None) == 0


def test_binding_refuses_host_tensors():
    import mixture_experts_routing_top_amd as moe
    x = torch.zeros((4, 8))
    with pytest.raises((ValueError, RuntimeError)):
        moe.moe_gate(x, 2)
    with pytest.raises((ValueError, RuntimeError)):
        moe.moe_layer_norm(x)
    with pytest.raises(ValueError):
        moe.moe_clip_grads([x], 1.0)
    with pytest.raises(ValueError):
        moe.moe_grad_norm([])
