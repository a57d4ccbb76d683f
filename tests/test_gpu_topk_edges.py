"""Router on the GPU at the edges of its 32-bit evaluation, against the definition in 64 bits."""
import math

import numpy as np
import pytest

from tests._cases import say
from tests.test_gpu_topk import check, logits

pytestmark = pytest.mark.gpu


# ---- groups whose best values cancel ---------------------------------------------

@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E, n_group", [(4, 2), (16, 2), (64, 8), (256, 8), (1024, 32), (60, 4)])
def test_group_scores_that_cancel(score, E, n_group):
    """A bias of +b on one expert of every group and -b on another, the rest banned by -4 b: a group's score is the sum of
    two scores, of which the biased values hold only what the rounding of b leaves.  The chosen experts themselves
    lie far apart."""
    run = E // n_group
    for b in (1e2, 1e4, 1e6, 3e38 / 4):
        bias = np.full((n_group, run), -4 * b, np.float32)
        bias[:, 0] = b
        bias[:, 1] = -b
        say(f"[topk] cancelling groups {score} E={E} groups={n_group} bias={b:g}")
        for seed, std in ((1, 1.5), (2, 1e-4)):
            for keep, k in ((1, 1), (1, 2)):
                check(logits(2000, E, seed, std), k, "f32", score, bias.reshape(-1), n_group, keep, 2, renorm=False)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_group_scores_that_cancel_to_neighbours(score):
    """Two groups whose sums differ by less than 2^-18 while the biased values are off by as much."""
    rng = np.random.default_rng(3)
    bias = np.array([100, -100, 0, 0], np.float32)
    l = rng.standard_normal((4000, 4)).astype(np.float32)
    l[:, 2:] = l[:, :2] + rng.uniform(-4e-6, 4e-6, (4000, 2)).astype(np.float32)
    check(l, 1, "f32", score, bias, 2, 1, 2, renorm=False)
    check(l, 2, "f32", score, bias, 2, 1, 2)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_group_scores_past_the_range_of_32_bits(score):
    """Biases whose sum is infinite in 32 bits and finite in 64; groups without an available expert beside them."""
    l = logits(50, 16, 4)
    l[::3, 4:8] = -math.inf
    l[1::3, 1:4] = -math.inf
    for b in (3e38, -3e38):
        bias = np.repeat(np.float32([b, b / 2, b, b / 4]), 4)
        check(l, 3, "f32", score, bias.astype(np.float32), 4, 2, 2, renorm=False)
        check(l, 3, "f32", score, bias.astype(np.float32), 4, 2, 1, renorm=False)
