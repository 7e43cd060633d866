"""A token's experts and weights do not hang on the tokens beside it in the batch."""
import numpy as np
import pytest
import torch

import mixture_experts_routing_top_amd as moe

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("E,k", [(64, 8), (256, 8), (8, 2)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_gate_rows_are_independent(score, renorm, E, k):
    """Every other row replaced by one whose sigmoids all underflow, or that is masked:
    the rows between keep their bits."""
    T = 40000
    rng = np.random.default_rng(E)
    lg = torch.from_numpy((1.5 * rng.standard_normal((T, E)) - 6.0).astype(np.float32)).cuda()
    idx, w = moe.moe_gate(lg, k, score=score, renorm=renorm)
    for other in (-700.0, -1e6, -float("inf"), 30.0):
        lg2 = lg.clone()
        lg2[1::2] = other
        idx2, w2 = moe.moe_gate(lg2, k, score=score, renorm=renorm)
        assert torch.equal(idx[0::2], idx2[0::2])
        assert torch.equal(w[0::2], w2[0::2]), int((w[0::2] != w2[0::2]).sum())
