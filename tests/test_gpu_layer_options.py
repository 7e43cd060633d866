"""moe_layer_backward takes the gate and the norm that the forward pass ran, and refuses
others: their gradients would be those of another layer."""
import pytest
import torch

import mixture_experts_routing_top_amd as moe
from test_gpu_train_step import _case

pytestmark = pytest.mark.gpu


def _forward(c, **kw):
    return moe.moe_layer_forward(c["x"], c["logits"], c["k"], *c["wts"], copy_rows=True, **kw)


def _backward(c, f, **kw):
    return moe.moe_layer_backward(f, c["logits"], *c["wts"], c["d_normed"], **kw)


def test_layer_backward_refuses_another_gate():
    c = _case("sigmoid", torch.float32, T=20)
    same = {"score": moe.SIGMOID, "renorm": 1, "scale": 1.5}       # what the gradient hangs on, otherwise spelt
    f = _forward(c, gate=c["gate"])
    for gate in (None, {}, {**c["gate"], "score": "softmax"}, {**c["gate"], "renorm": False},
                 {**c["gate"], "scale": 1.0}):
        with pytest.raises(ValueError, match="gate"):
            _backward(c, f, gate=gate)
    a, b = _backward(c, f, gate=c["gate"]), _backward(c, f, gate=same)
    assert all(torch.equal(a[key], b[key]) for key in a)
    plain = _forward(c)
    with pytest.raises(ValueError, match="gate"):
        _backward(c, plain, gate=c["gate"])
    _backward(c, plain, gate={})          # moe_route's own formula
    _backward(c, _forward(c, gate={}))


def test_layer_backward_refuses_another_norm():
    c = _case("softmax", torch.float32, T=20)
    f = _forward(c, norm=c["norm"], residual=c["x"])
    for norm in (None, {**c["norm"], "eps": 1e-3}, {**c["norm"], "weight": None}, {"eps": 1e-5}):
        with pytest.raises(ValueError, match="norm"):
            _backward(c, f, norm=norm)
    a = _backward(c, f, norm=c["norm"])
    b = _backward(c, f, norm={**c["norm"], "bias": None})      # its gradient is not asked for
    assert "d_bias" in a and "d_bias" not in b and all(torch.equal(a[key], b[key]) for key in b)
    # eps left out is its default
    _backward(c, _forward(c, norm={}), norm={"eps": 1e-5})


def test_layer_backward_of_a_result_put_together_by_hand():
    """A dict without the record of its options is taken at the caller's word."""
    c = _case("sigmoid", torch.float32, T=20)
    f = _forward(c, gate=c["gate"], norm=c["norm"])
    keys = ("idx", "w", "x_perm", "y_perm", "inv_pos", "expert_off", "out", "normed", "x_sum")
    a = _backward(c, f, gate=c["gate"], norm=c["norm"])
    b = _backward(c, {key: f[key] for key in keys}, gate=c["gate"], norm=c["norm"])
    assert all(torch.equal(a[key], b[key]) for key in a)
