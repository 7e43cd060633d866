"""The gate under biases with a large common part: s + b in double then keeps little or
nothing of the scores, and experts and groups that this makes equal go by index.  The
experts must be the oracle's and the weights within the bound of test_gpu_gate.py."""
import numpy as np
import pytest
import torch

from test_gpu_gate import _check_gate

pytestmark = pytest.mark.gpu

# E, n_groups, keep, k: fewer than 16 experts kept, and more
SHAPES = [(64, 8, 1, 8), (32, 4, 1, 3), (24, 6, 2, 4), (96, 16, 2, 5), (160, 8, 3, 6), (256, 8, 4, 8), (40, 1, 1, 5)]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("group_score", ["max", "top2"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_gate_biases_with_a_large_common_part(shape, group_score, score):
    E, G, keep, k = shape
    rng = np.random.default_rng(E + keep)
    for power in (4, 9, 10, 11, 13, 20, 28, 32, 34, 40, 50, 60, 90, 99):
        common = np.float32((-1.0) ** power * 2.0 ** power)
        for jitter in (0.0, 0.1):
            bias = torch.from_numpy((common + jitter * rng.standard_normal(E)).astype(np.float32)).cuda()
            # scores over the whole range, and ones near the bottom of the keys' units
            for shift in (0.0, -9.0):
                lg = torch.from_numpy((1.5 * rng.standard_normal((23, E)) + shift).astype(np.float32)).cuda()
                _check_gate(lg, k, bias=bias, score=score, n_groups=G, keep_groups=keep, group_score=group_score,
                            renorm=power % 3 == 0)


@pytest.mark.parametrize("group_score", ["max", "top2"])
def test_gate_groups_of_one_live_expert_under_a_common_bias(group_score):
    """A group with one unmasked expert has its score alone, others a sum of two."""
    E, G = 48, 8
    rng = np.random.default_rng(1)
    lg = rng.standard_normal((64, E)).astype(np.float32)
    for t in range(64):
        for g in rng.permutation(G)[:3]:
            lg[t, g * 6:(g + 1) * 6][np.arange(6) != rng.integers(6)] = -np.inf
    for common in (-0.5, 0.5, -3.0, 7.0, -100.0, 1000.0, -2.0 ** 20, 2.0 ** 30, -2.0 ** 60):
        bias = torch.from_numpy((common + 0.05 * rng.standard_normal(E)).astype(np.float32)).cuda()
        _check_gate(torch.from_numpy(lg).cuda(), 6, bias=bias, score="sigmoid", n_groups=G, keep_groups=2,
                    group_score=group_score)
