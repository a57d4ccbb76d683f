"""Router on the GPU against its definition in 64 bits (numpy): ids equal, gates
within the fp32 evaluation's error, on every type, layout, group form and edge."""
import math

import numpy as np
import pytest
import torch

from quantized_moe_expert_quantize_amd import ftq
from tests._cases import say
from tests._fp8 import DTYPES

pytestmark = pytest.mark.gpu


def topk64(l, bias, k, score, n_group, topk_group, group_top, renorm, scale):
    """The definition, row by row in 64 bits; l is what the logits' type holds."""
    T, E = l.shape
    ids = np.full((T, k), -1, np.int32)
    gates = np.zeros((T, k))
    for t in range(T):
        x = l[t].astype(np.float64)
        if np.isnan(x).any() or (score == "softmax" and (x == math.inf).any()):
            gates[t] = math.nan
            continue
        m = x.max() if x.max() > -math.inf else 0.0
        with np.errstate(over="ignore", under="ignore"):
            s = np.exp(x - m) / max(np.exp(x - m).sum(), 1e-300) if score == "softmax" else 1 / (1 + np.exp(-x))
        c = x.copy() if bias is None else np.where(x == -math.inf, -math.inf, s + bias.astype(np.float64))
        if n_group > 1:
            by = np.where(x == -math.inf, -math.inf, s) if bias is None and group_top == 2 else c
            g = -np.sort(-by.reshape(n_group, -1), axis=1)[:, :group_top].sum(1)
            keep = np.argsort(-g, kind="stable")[:topk_group]
            mask = np.zeros(n_group, bool)
            mask[keep] = True
            c = np.where(np.repeat(mask, E // n_group), c, -math.inf)
        order = np.argsort(-c, kind="stable")[:k]
        order = order[c[order] > -math.inf]
        ids[t, : len(order)] = order
        v = s[order]
        if renorm:
            v = v / v.sum() if v.sum() > 0 else np.zeros_like(v)
        gates[t, : len(order)] = v * scale
    return ids, gates


def tolerance(l, score):
    """Relative error of a gate: the exponent's argument l - max is rounded once (2^-24 of it, up to the row's
    range R), the exponential, the quotients, the sum over up to 1024 experts (a tree of 6 levels over 16 serial
    terms) and the products are a few units each: (2 R + 48) 2^-23."""
    x = l.astype(np.float64)
    x = x[np.isfinite(x)]
    R = float(x.max() - x.min()) if x.size and score == "softmax" else 0.0
    return (2 * min(R, 200.0) + 48) * 2.0 ** -23


def check(l, k, dtype="f32", score="softmax", bias=None, n_group=1, topk_group=1, group_top=1, renorm=True, scale=1.0, ld=None):
    T, E = l.shape
    buf = torch.full((T, ld or E), 7.0, dtype=DTYPES[dtype], device="cuda")
    buf[:, :E] = torch.from_numpy(l).to(DTYPES[dtype]).cuda()
    x = buf[:, :E]
    held = x.double().cpu().numpy()
    b = None if bias is None else torch.from_numpy(bias).cuda()
    ids = torch.full((T + 1, k), 77, dtype=torch.int32, device="cuda")
    gates = torch.full((T + 1, k), 7.0, device="cuda")
    ftq.moe_topk(x, k, score=ftq.SCORE_SOFTMAX if score == "softmax" else ftq.SCORE_SIGMOID, bias=b, n_group=n_group,
                 topk_group=topk_group, group_top=group_top, renorm=renorm, scale=scale, ids=ids[:T], gates=gates[:T])
    torch.cuda.synchronize()
    assert (ids[T] == 77).all() and (gates[T] == 7.0).all(), "rows behind the last were written"
    ri, rg = topk64(held, bias, k, score, n_group, topk_group, group_top, renorm, scale)
    gi, gg = ids[:T].cpu().numpy(), gates[:T].double().cpu().numpy()
    bad = np.nonzero((gi != ri).any(1))[0]
    assert not len(bad), f"row {bad[0]} of {len(bad)}: {gi[bad[0]]} instead of {ri[bad[0]]}"
    assert np.array_equal(np.isnan(gg), np.isnan(rg))
    d = np.abs(gg - rg)
    lim = tolerance(held, score) * np.abs(rg) + 2.0 ** -126 * abs(scale)
    assert not (d > lim).any(), f"gates off by {np.nanmax(d - lim):.3e} over the bound"
    return gi, gg


def logits(T, E, seed, std=1.5):
    return (np.random.default_rng(seed).standard_normal((T, E)) * std).astype(np.float32)


def balance(E, seed, std=0.1):
    return (np.random.default_rng(seed + 1).standard_normal(E) * std).astype(np.float32)


# every lane count per row and experts per lane, odd numbers of both
SIZES = [(1, 8, 2), (33, 3, 3), (5, 1, 1), (64, 8, 8), (9, 16, 4), (17, 12, 5), (10, 32, 6), (7, 31, 31), (3, 60, 4), (70, 64, 6),
         (5, 64, 64), (11, 128, 8), (6, 100, 64), (3, 160, 6), (4, 256, 8), (3, 255, 9), (2, 384, 8), (3, 512, 10), (2, 1000, 16), (2, 1024, 64)]


@pytest.mark.parametrize("size", SIZES, ids=lambda s: "T{}E{}k{}".format(*s))
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_sizes_and_types(size, dtype):
    T, E, k = size
    say(f"[topk] T={T} E={E} k={k} {dtype}")
    for score in ("softmax", "sigmoid"):
        for bias in (None, balance(E, T)):
            for renorm in (True, False):
                check(logits(T, E, T * E + k), k, dtype, score, bias, renorm=renorm, scale=2.5 if renorm else 1.0)


# runs that fill whole lanes and ones that do not
GROUPS = [(256, 8, 8, 4), (128, 8, 4, 2), (64, 4, 8, 3), (160, 6, 8, 3), (56, 3, 8, 4), (28, 4, 4, 2), (8, 2, 4, 2), (8, 2, 2, 1),
          (384, 8, 4, 4), (1024, 16, 32, 5), (192, 8, 64, 7), (64, 8, 64, 9), (24, 2, 8, 2), (512, 8, 2, 1)]


@pytest.mark.parametrize("g", GROUPS, ids=lambda g: "E{}k{}g{}of{}".format(g[0], g[1], g[3], g[2]))
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_groups(g, dtype):
    E, k, n_group, topk_group = g
    say(f"[topk] groups E={E} k={k} {topk_group} of {n_group} {dtype}")
    for score in ("softmax", "sigmoid"):
        for bias in (None, balance(E, E)):
            for group_top in (1, 2):
                if group_top <= E // n_group:
                    check(logits(37, E, E + k), k, dtype, score, bias, n_group, topk_group, group_top, scale=2.5)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_row_strides(score):
    for E, ld in ((64, 65), (256, 260), (8, 11), (100, 128), (256, 1024)):
        say(f"[topk] stride {ld} of {E}")
        check(logits(9, E, ld), 4, "bf16", score, balance(E, 3), ld=ld)
        check(logits(9, E, ld), 4, "f32", score, None, ld=ld)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_equal_scores_go_to_the_lowest_id(score):
    for E, n_group in ((8, 1), (64, 1), (256, 8), (100, 4)):
        flat = np.zeros((5, E), np.float32)
        flat[1] = -3.0
        flat[2, ::2] = -0.0
        flat[3, E // 2:] = 1.0
        flat[4] = np.round(logits(1, E, 3)[0] * 2) / 2
        for bias in (None, np.zeros(E, np.float32), np.full(E, -0.25, np.float32)):
            check(flat, 4, "f32", score, bias, n_group, max(1, n_group // 2), 1)
            if n_group > 1:
                check(flat, 4, "bf16", score, bias, n_group, n_group // 2, 2)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_scores_closer_than_32_bits_hold(score):
    """Experts whose order fp32 scores do not settle: neighbours by one unit in the last place, saturated
    sigmoids, tiny probabilities, a bias that nearly cancels the difference."""
    rng = np.random.default_rng(5)
    for E, n_group in ((64, 1), (256, 8), (16, 2)):
        l = np.full((12, E), 1.0, np.float32)
        for e in range(E):
            l[0, e] = np.nextafter(np.float32(1.0), np.float32(2.0)) if e % 3 else 1.0
        l[1] = 20 + rng.standard_normal(E)          # sigmoid: all within 2^-28 of 1
        l[2] = -25 + rng.standard_normal(E)         # sigmoid: all below 2^-34
        l[3] = rng.standard_normal(E) * 1e-7
        l[4] = rng.standard_normal(E) * 30          # softmax: most probabilities far below fp32's resolution of 1
        l[5:] = 1 + rng.standard_normal((7, E)) * 1e-6
        for bias in (None, np.zeros(E, np.float32), (rng.standard_normal(E) * 1e-7).astype(np.float32), np.full(E, 0.5, np.float32)):
            for gt in ((1,) if n_group == 1 else (1, 2)):
                check(l, 4, "f32", score, bias, n_group, max(1, n_group // 2), gt)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_far_apart_logits(score):
    """Scores that underflow in 32 bits, chosen for their bias; sums of them."""
    E = 32
    l = np.zeros((4, E), np.float32)
    l[:, 8:] = -95.0
    l[1, 8:] = -300.0 + np.arange(24)
    l[2] = -1e30
    l[3] = np.linspace(-3e38, 3e38, E)
    b = np.zeros(E, np.float32)
    b[20:] = 10.0 + np.arange(12, dtype=np.float32)
    check(l[:1], 4, "f32", score, b, renorm=True)
    check(l[:1], 4, "f32", score, b, renorm=False)
    check(l, 4, "f32", score, None)
    check(l, 4, "f32", score, b, renorm=False)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_masked_and_undefined_rows(score, dtype):
    """-inf logits are not chosen, rows without enough experts end in -1, rows with a NaN (or, for softmax, +inf) are undefined."""
    for E, n_group in ((8, 1), (8, 2), (256, 8), (100, 4)):
        say(f"[topk] masks E={E} groups={n_group} {dtype}")
        l = logits(12, E, 17)
        l[0, :] = -math.inf
        l[1, 1:] = -math.inf
        l[2, : E - 1] = -math.inf
        l[3, ::2] = -math.inf
        l[4, 3] = math.nan
        l[5, E - 1] = math.inf
        l[6, :3] = -math.inf
        l[6, 4] = math.nan
        l[7, : E // 2] = -math.inf
        l[8, : E - 2] = -math.inf
        l[9, :] = -65504.0 if dtype == "f16" else -3e38      # the lowest finite values are no mask
        l[10, 1::3] = -65504.0 if dtype == "f16" else -3e38
        for bias in (None, balance(E, 4)):
            for gt in ((1,) if n_group == 1 else (1, 2)):
                gi, gg = check(l, 4, dtype, score, bias, n_group, max(1, n_group // 2), gt)
                assert (gi[0] == -1).all() and (gg[0] == 0).all()
                assert (gi[4] == -1).all() and np.isnan(gg[4]).all()


def test_bias_masks_an_expert():
    b = np.zeros(64, np.float32)
    b[::2] = -math.inf
    gi, _ = check(logits(20, 64, 2), 6, "f32", "sigmoid", b)
    assert (gi % 2 == 1).all()


@pytest.mark.parametrize("case", [(8191, 128, 8, "bf16", "softmax", False, 1, 1, 1), (4099, 256, 8, "f32", "sigmoid", True, 8, 4, 2),
                                  (20001, 8, 2, "f32", "softmax", False, 1, 1, 1)], ids=str)
def test_many_rows(case):
    T, E, k, dtype, score, bias, ng, tg, gt = case
    say(f"[topk] {case}")
    check(logits(T, E, 1), k, dtype, score, balance(E, 1) if bias else None, ng, tg, gt)


def test_rows_do_not_depend_on_the_batch():
    x = torch.from_numpy(logits(301, 128, 9)).cuda()
    b = torch.from_numpy(balance(128, 9)).cuda()
    ids, gates = ftq.moe_topk(x, 8, score=ftq.SCORE_SIGMOID, bias=b, n_group=4, topk_group=2, group_top=2)
    for cut in (1, 100, 299):
        for part, rows in ((x[:cut], slice(0, cut)), (x[cut:], slice(cut, 301))):
            i2, g2 = ftq.moe_topk(part, 8, score=ftq.SCORE_SIGMOID, bias=b, n_group=4, topk_group=2, group_top=2)
            assert torch.equal(i2, ids[rows]) and torch.equal(g2, gates[rows])


def test_binding_refuses():
    x = torch.zeros(4, 16, device="cuda")
    with pytest.raises(ValueError):
        ftq.moe_topk(x.t(), 2)
    with pytest.raises(ValueError):
        ftq.moe_topk(x.double(), 2)
    with pytest.raises(ValueError):
        ftq.moe_topk(x, 2, bias=torch.zeros(15, device="cuda"))
    with pytest.raises(ValueError):
        ftq.moe_topk(x, 2, ids=torch.zeros(4, 3, dtype=torch.int32, device="cuda"))
    with pytest.raises(ftq.FtqError):
        ftq.moe_topk(x, 17)
    assert ftq.moe_topk(x[:0], 2)[0].shape == (0, 2)
