"""Equal logits under biases that differ by less than the float32 keys resolve: the
biases decide, not the index."""
import numpy as np
import pytest
import torch

from test_gpu_gate import _check_gate

pytestmark = pytest.mark.gpu

SHAPES = [(8, 1, 1, 2), (40, 1, 1, 5), (64, 8, 3, 8), (88, 8, 6, 6), (160, 8, 3, 6), (256, 8, 4, 8), (256, 1, 1, 8)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_gate_equal_logits_go_by_close_biases(shape, score, dtype):
    E, G, keep, k = shape
    rng = np.random.default_rng(E + k)
    for spread in (0.05, 1.0, 6.0):
        # values a few steps apart, so that each comes several times, some of them +inf
        lg = (spread * np.round(4 * rng.standard_normal((200, E))) / 4).astype(np.float32)
        lg[::7, ::5] = np.inf
        lg = torch.from_numpy(lg).to(dtype).cuda()
        for size in (1e-9, 1e-7, 1e-6, 1e-5, 1e-4):
            bias = torch.from_numpy((size * rng.standard_normal(E)).astype(np.float32)).cuda()
            _check_gate(lg, k, bias=bias, score=score, n_groups=G, keep_groups=keep, group_score="max", renorm=False)


def test_gate_two_equal_logits_apart_from_the_rest():
    """One pair of equal logits in each row, at every place among the best, its biases in
    both orders; every other expert clearly apart."""
    E, k = 32, 8
    rng = np.random.default_rng(3)
    for place in range(k + 1):
        lg, bias = np.zeros((64, E), np.float32), np.zeros(E, np.float32)
        bias[:16] = 1e-7 * (1 + np.arange(16))           # the higher index has the higher bias
        for t in range(64):
            order = rng.permutation(E)
            lg[t, order] = 3.0 - 0.25 * np.arange(E)
            i, j = sorted(rng.permutation(16)[:2])
            for e, at in ((i, place), (j, place + 1)):    # the two at `place` and the one after
                other = order[at]
                lg[t, e], lg[t, other] = lg[t, other], lg[t, e]
                order[np.nonzero(order == e)[0][0]], order[at] = other, e
            lg[t, j] = lg[t, i]
        for score in ("softmax", "sigmoid"):
            _check_gate(torch.from_numpy(lg).cuda(), k, bias=torch.from_numpy(bias).cuda(), score=score)
