"""Router on the GPU at the edges of its 32-bit evaluation, against the definition in 64 bits."""
import math

import numpy as np
import pytest
import torch

from quantized_moe_expert_quantize_amd import ftq
from tests._cases import say
from tests.test_gpu_topk import balance, check, logits, topk64

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


# ---- groups without an available expert -------------------------------------------

def route(l, k, bias=None, n_group=1, topk_group=1, group_top=1, score="sigmoid", renorm=False):
    ids, gates = ftq.moe_topk(torch.from_numpy(l).cuda(), k, score=ftq.SCORE_SOFTMAX if score == "softmax" else ftq.SCORE_SIGMOID,
                              bias=None if bias is None else torch.from_numpy(bias).cuda(), n_group=n_group,
                              topk_group=topk_group, group_top=group_top, renorm=renorm)
    return ids.cpu().numpy(), gates.cpu().numpy()


@pytest.mark.parametrize("E, n_group, alive", [(256, 8, 3), (256, 8, 1), (64, 8, 2), (1024, 16, 5), (8, 4, 1)])
def test_masked_groups_cost_nothing(E, n_group, alive):
    """Fewer groups with an available expert than are kept: the choice is that of the same rows without groups, and so
    are the gates' bits, which the evaluation in 64 bits would round otherwise in some row of many."""
    T, run = 3000, E // n_group
    l = logits(T, E, E + alive).reshape(T, n_group, run)
    rng = np.random.default_rng(E)
    for t in range(T):
        l[t, rng.permutation(n_group)[alive:]] = -math.inf
    l = l.reshape(T, E)
    k = min(4, alive * run)
    for group_top in (1, 2):
        for bias in (None, np.zeros(E, np.float32)):
            check(l[:200], k, "f32", "sigmoid", bias, n_group, alive + 1, group_top)
            got = route(l, k, bias, n_group, alive + 1, group_top)
            want = route(l, k, bias)
            assert np.array_equal(got[0], want[0]) and np.array_equal(got[1], want[1]), (group_top, bias is None)


def test_groups_that_tie_at_minus_infinity():
    """One available expert in each group, two wanted for a group's score: all groups score -inf, the lower ones stay."""
    l = np.full((40, 32), -math.inf, np.float32)
    x = logits(40, 8, 3)
    l[:, ::4] = x
    for bias in (None, np.zeros(32, np.float32)):
        for score in ("softmax", "sigmoid"):
            gi, _ = check(l, 3, "f32", score, bias, 8, 4, 2)
            assert (gi < 16).all()


# ---- gates to a few units in the last place ----------------------------------------

# Roundings that a gate goes through, in units of 2^-24 relative: softmax: exponential 3 (one unit in the last place, 2,
# and a product), divisor 3 + 10 (a tree of at most 1024), its reciprocal, the product, the scale: 19; renormalised 3 + (3
# + 6) + 2 = 14.  Sigmoid: exponential 3, sum 1, reciprocal 2 (one unit in the last place): 6; renormalised 6 + (6 + 6)
# + 2 = 20.  One more for the products of these.
GATE_UNITS = 21


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E, k", [(8, 2), (64, 6), (100, 8), (128, 8), (256, 8), (384, 8), (1000, 16), (1024, 64)])
def test_gates_hold_their_last_places(score, E, k):
    """Whatever the size of the logits, a gate is within a constant number of roundings."""
    say(f"[topk] gates {score} E={E} k={k}")
    for i, (mean, std) in enumerate(((0, 1.5), (0, 12), (-12, 1), (-35, 3), (-60, 1), (1000, 5), (1e6, 3), (17, 0.01))):
        l = (mean + logits(300, E, 10 * E + i, std)).astype(np.float32)
        for renorm in (True, False):
            for bias in (None, np.linspace(-0.5, 0.5, E).astype(np.float32)):
                gi, gg = check(l, k, "f32", score, bias, renorm=renorm, scale=2.5)
                _, want = topk64(l, bias, k, score, 1, 1, 1, renorm, 2.5)
                off = np.abs(gg - want) / np.maximum(want, 2.0 ** -100)
                assert off.max() <= GATE_UNITS * 2.0 ** -24, (mean, std, renorm, bias is not None, off.max() * 2 ** 24)


# ---- a row's bits and the number of rows ---------------------------------------------

@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E, k, n_group", [(128, 8, 1), (256, 8, 1), (256, 8, 8), (100, 8, 1), (130, 5, 1), (100, 20, 1), (255, 9, 1), (384, 8, 4),
                                           (511, 3, 1), (64, 6, 1)])
def test_rows_do_not_depend_on_the_number_of_rows(score, E, k, n_group):
    """Few rows and many are laid out otherwise over the lanes; a row's ids and gates keep their bits."""
    l, b = logits(5001, E, E), balance(E, E)
    for bias in (None, b):
        for renorm in (False, True):
            whole = route(l, k, bias, n_group, max(1, n_group // 2), 1, score, renorm)
            for a, z in ((0, 1), (0, 4095), (17, 300), (5000, 5001)):
                part = route(l[a:z], k, bias, n_group, max(1, n_group // 2), 1, score, renorm)
                assert np.array_equal(part[0], whole[0][a:z]) and np.array_equal(part[1], whole[1][a:z]), (a, z, renorm)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_offsets_past_32_bits(score):
    """Logits whose element and byte offsets pass 2^32: by their rows' stride, and by their number."""
    E, k = 64, 4
    kw = dict(score=ftq.SCORE_SOFTMAX if score == "softmax" else ftq.SCORE_SIGMOID, bias=torch.from_numpy(balance(E, 1)).cuda())
    x = torch.from_numpy(logits(6, E, 8)).bfloat16().cuda()
    want = ftq.moe_topk(x, k, **kw)
    far = torch.empty(5 * (1 << 30) + E, dtype=torch.bfloat16, device="cuda")
    rows = far.as_strided((6, E), (1 << 30, 1))
    rows.copy_(x)
    say(f"[topk] far rows by stride {score}")
    got = ftq.moe_topk(rows, k, **kw)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    T = (1 << 26) + 6
    many = far[: T * E].view(T, E)
    many.zero_()
    many[-6:] = x
    say(f"[topk] far rows by number {score}")
    got = ftq.moe_topk(many, k, **kw)
    assert torch.equal(got[0][-6:], want[0]) and torch.equal(got[1][-6:], want[1])
    first = ftq.moe_topk(many[:1], k, **kw)
    assert (got[0][:-6] == first[0]).all() and (got[1][:-6] == first[1]).all()
