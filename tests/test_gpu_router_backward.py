"""Balance loss with counts, the gradient of gates and losses with respect to the
logits, and the combine's gradient, against definitions in 64 bits and against
differences."""
import pytest
import torch

from quantized_moe_expert_quantize_amd import ftq
from tests import _train as t

pytestmark = pytest.mark.gpu
INF = float("inf")


def _inputs(T, E, k, dtype, seed, spread=1.5):
    g = torch.Generator().manual_seed(seed)
    logits = (spread * torch.randn(T, E, generator=g) + 0.5 * torch.randn(E, generator=g)).to(t.DTYPES[dtype])
    ids = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)]).to(torch.int32) if T else torch.zeros(0, k, dtype=torch.int32)
    return g, logits, ids


def _cuts(g, T, S, before=0, behind=0):
    cuts = torch.sort(torch.randint(before, T - behind + 1, (S - 1,), generator=g)).values
    return torch.cat([torch.tensor([before]), cuts, torch.tensor([T - behind])]).to(torch.int32)


def _cuda(*a):
    return [v.cuda() if isinstance(v, torch.Tensor) else v for v in a]


SOFT = {ftq.SCORE_SOFTMAX: True, ftq.SCORE_SIGMOID: False}


def _check_loss(logits, ids, score, offsets=None, valid=None):
    T, E = logits.shape
    k = ids.shape[1]
    loss, counts, tokens = ftq.moe_balance(*_cuda(logits, ids), score=score, offsets=None if offsets is None else offsets.cuda(),
                                           valid=None if valid is None else valid.cuda())
    seqs = t.sequences(T, offsets, valid)
    assert tokens.tolist() == [len(r) for r in seqs]
    for s, r in enumerate(seqs):
        assert torch.equal(counts[s].cpu(), t.counts_of(ids, r, E).to(torch.int32)), f"sequence {s}"
    ref = t.losses(logits.double(), ids, E, k, seqs, SOFT[score])
    # all terms are positive.  A share: an exponential (|x| + 2 units of 2^-24, |x| <= 20 here, or the share is lost beside
    # the row's others), the score's reciprocal and products (6), the row's sum (16 + 6) and the division (2), below 60; the
    # sum over rows: 64 in fp32 and a tree, then fp64 and one rounding.  Together below 200 units, 100 steps
    off = (loss.double().cpu() - ref).abs()
    assert (off <= 2 * t.U * 100 * ref).all(), (off / ref).max()
    return loss, counts, tokens


@pytest.mark.parametrize("score", [ftq.SCORE_SOFTMAX, ftq.SCORE_SIGMOID])
@pytest.mark.parametrize("T,E,k,dtype", [
    (1, 1, 1, "f32"), (1, 8, 2, "bf16"), (3, 7, 7, "f32"), (65, 60, 4, "f16"), (200, 64, 6, "bf16"), (129, 97, 5, "f32"), (130, 128, 8, "bf16"),
    (300, 256, 8, "f32"), (70, 200, 64, "f16"), (66, 255, 3, "f32"), (40, 511, 2, "bf16"), (33, 512, 8, "f32"), (37, 1023, 8, "f16"), (35, 1024, 9, "f32"),
])
def test_loss_of_one_sequence(T, E, k, dtype, score):
    print(f"[balance] T={T} E={E} k={k} {dtype} score={score}", flush=True)
    _, logits, ids = _inputs(T, E, k, dtype, seed=T + E)
    _check_loss(logits, ids, score)


@pytest.mark.parametrize("score", [ftq.SCORE_SOFTMAX, ftq.SCORE_SIGMOID])
@pytest.mark.parametrize("T,E,k", [(20, 1024, 64), (32, 1023, 8), (1024, 32, 64), (1025, 32, 64), (300, 28, 64)])
def test_layouts_of_the_most_lds(T, E, k, score):
    """Loss by one workgroup over rows of up to 1024 experts, gradients of 128 rows at a time with 64 choices each."""
    g, logits, _ = _inputs(T, E, 1, "f32", seed=T + E)
    ids = torch.randint(-1, E + 1, (T, k), generator=g).to(torch.int32)
    offsets = _cuts(g, T, 4)
    d_gates, d_loss = torch.randn(T, k, generator=g), torch.randn(4, generator=g)
    _check_loss(logits, ids, score)
    _check_loss(logits, ids, score, offsets)
    _check_grad(logits, ids, score, True, 1.0, d_gates, d_loss, offsets)


@pytest.mark.parametrize("score", [ftq.SCORE_SOFTMAX, ftq.SCORE_SIGMOID])
@pytest.mark.parametrize("T,S,before,behind,padded", [(500, 1, 3, 70, 0.0), (700, 5, 0, 0, 0.2), (1000, 40, 5, 130, 0.1), (130, 300, 0, 0, 0.5), (64, 2, 0, 0, 1.0)])
def test_loss_of_packed_sequences(T, S, before, behind, padded, score):
    g, logits, ids = _inputs(T, 64, 4, "f32", seed=S)
    ids[torch.rand(T, 4, generator=g) < 0.1] = -1
    ids[torch.rand(T, 4, generator=g) < 0.05] = 64            # no expert either
    ids[:, 1] = torch.where(torch.rand(T, generator=g) < 0.1, ids[:, 0], ids[:, 1])   # the same expert twice
    valid = torch.rand(T, generator=g) >= padded
    logits[~valid] = float("nan")                             # padding may hold anything
    logits[:before] = float("nan")
    if behind:
        logits[T - behind:] = float("nan")
    offsets = _cuts(g, T, S, before, behind)
    _check_loss(logits, ids, score, offsets, valid)


@pytest.mark.parametrize("T,S", [(5000, 5000), (300, 20000), (3000, 64), (3000, 63), (3000, 65), (9000, 130)])
def test_many_sequences(T, S):
    """Sequences of one row, long runs of empty ones, and numbers of them around a wave's lanes: loss and gradient."""
    g, logits, ids = _inputs(T, 16, 2, "f32", seed=S)
    offsets = torch.arange(S + 1, dtype=torch.int32) if T == S else _cuts(g, T, S, 2, 3)
    loss, counts, tokens = _check_loss(logits, ids, ftq.SCORE_SIGMOID, offsets)
    d_loss = torch.randn(S, generator=g)
    got = ftq.moe_topk_backward(*_cuda(logits, ids), score=ftq.SCORE_SIGMOID, d_loss=d_loss.cuda(), counts=counts, tokens=tokens,
                                offsets=offsets.cuda()).cpu()
    row = torch.arange(T)
    seq = torch.searchsorted(offsets[1:].contiguous(), row.to(torch.int32), right=True)
    inside = (row >= offsets[0]) & (row < offsets[-1])
    at = seq.clamp_max(S - 1)
    n = tokens.cpu().double()[at].clamp_min(1)
    v = counts.cpu().double()[at] * (d_loss.double()[at] * 16 / (2 * n * n))[:, None] * inside[:, None]
    s, p = scores_and_shares(logits.double(), False)
    t.close(got, p * (1 - s) * (v - (p * v).sum(1, keepdim=True)), p * (v.abs() + (p * v.abs()).sum(1, keepdim=True)), 144, "d_logits")


def test_offsets_that_descend_end():
    """Offsets that are not ascending have no defined losses, but the call ends and leaves the next one right."""
    g, logits, ids = _inputs(9000, 16, 2, "f32", seed=2)
    for cuts in ([0, 9000, 4000, 100, 9000], [9000, 0, 9000, 0, 5], [-5, 20000, -7, 3, 20000], [7, 7, 5, 7, 6]):
        for more in (0, 200):
            offsets = torch.tensor(cuts + cuts[1:] * (more // 4), dtype=torch.int32).cuda()
            _, counts, tokens = ftq.moe_balance(*_cuda(logits, ids), offsets=offsets)
            ftq.moe_topk_backward(*_cuda(logits, ids), d_loss=torch.ones(len(offsets) - 1).cuda(), counts=counts, tokens=tokens, offsets=offsets)
    torch.cuda.synchronize()
    _check_loss(logits, ids, ftq.SCORE_SOFTMAX, _cuts(g, 9000, 5))


def test_loss_of_strange_rows():
    _, logits, ids = _inputs(300, 64, 4, "f32", seed=1)
    logits[5, :60] = -INF                                      # few experts left
    logits[6] = -INF                                           # none
    logits[7] = -300.0 + logits[7]                             # sigmoids that 32 bits cannot hold
    logits[8] *= 60.0
    for score in SOFT:
        _check_loss(logits, ids, score)
    offsets = torch.tensor([0, 100, 200, 300], dtype=torch.int32)
    logits[150, 3] = float("nan")
    logits[250, 4] = INF
    soft = ftq.moe_balance(*_cuda(logits, ids), offsets=offsets.cuda())[0]
    assert soft.isnan().tolist() == [False, True, True]
    sig = ftq.moe_balance(*_cuda(logits, ids), score=ftq.SCORE_SIGMOID, offsets=offsets.cuda())[0]
    assert sig.isnan().tolist() == [False, True, False]


def test_loss_of_nothing_and_strides():
    _, logits, ids = _inputs(0, 16, 2, "f32", seed=1)
    off = torch.zeros(4, dtype=torch.int32)
    loss, counts, tokens = ftq.moe_balance(logits.cuda(), ids.cuda(), offsets=off.cuda())
    assert not loss.any() and not counts.any() and not tokens.any() and counts.shape == (3, 16)
    _, wide, ids = _inputs(100, 80, 3, "bf16", seed=2)
    ids %= 30
    view = wide[:, 7:37]
    a = ftq.moe_balance(wide.cuda()[:, 7:37], ids.cuda())
    b = ftq.moe_balance(view.contiguous().cuda(), ids.cuda())
    assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_loss_of_many_rows_and_again():
    g, logits, ids = _inputs(1, 128, 8, "f32", seed=3)
    T = 70001
    logits = torch.randn(T, 128, generator=g)
    ids = logits.topk(8, dim=1).indices.to(torch.int32)
    offsets = torch.tensor([0, 1, 1, 40000, T], dtype=torch.int32)
    a = _check_loss(logits, ids, ftq.SCORE_SOFTMAX, offsets)
    b = ftq.moe_balance(*_cuda(logits, ids), offsets=offsets.cuda())
    assert all(torch.equal(p, q) for p, q in zip(a, b))


# ---- gradient of the logits -------------------------------------------------------

def _grad_ref(logits, ids, d_gates, score, renorm, scale, d_loss, offsets, valid):
    """The gradient by differentiating the definition, and the magnitudes of what it is a sum of."""
    T, E = logits.shape
    k, soft = ids.shape[1], SOFT[score]
    l = logits.double().requires_grad_()
    live = torch.ones(T, dtype=torch.bool) if valid is None else valid
    seqs = t.sequences(T, offsets, valid)
    total = l.sum() * 0
    mag = torch.zeros(T, E, dtype=torch.float64)
    s, p = scores_and_shares(l.detach(), soft)
    tail = 1.0 if soft else (1 - s)
    ok = (ids >= 0) & (ids < E)
    if d_gates is not None:
        w = d_gates.double() * live[:, None]
        total = total + (t.gates_of(l, ids, soft, renorm, scale) * w).sum()
        gate = t.gates_of(l.detach(), ids, soft, renorm, scale)
        at = ids.long().clamp(0, E - 1)
        if renorm:
            whole = (gate * w.abs()).sum(1, keepdim=True) / scale
            mag.scatter_add_(1, at, gate * (w.abs() + whole) * ok)
            mag *= tail
        elif soft:
            mag += s * (gate * w.abs()).sum(1, keepdim=True)
            mag.scatter_add_(1, at, gate * w.abs())
        else:
            mag.scatter_add_(1, at, gate * w.abs())
    if d_loss is not None:
        total = total + (t.losses(l, ids, E, k, seqs, soft) * d_loss.double()).sum()
        for q, rows in enumerate(seqs):
            if len(rows):
                v = t.counts_of(ids, rows, E).double() * abs(float(d_loss[q])) * E / (k * len(rows) ** 2)
                pr = p[rows]
                mag[rows] += pr * (v + (pr * v).sum(1, keepdim=True)) * (1.0 if soft else tail[rows])
    return torch.autograd.grad(total, l)[0], mag


def scores_and_shares(l, soft):
    return t.scores(l, soft), t.shares(l, soft)


def _check_grad(logits, ids, score, renorm, scale=1.0, d_gates=None, d_loss=None, offsets=None, valid=None, check=True):
    dev = dict(d_gates=d_gates, d_loss=d_loss, offsets=offsets, valid=valid)
    dev = {n: None if v is None else v.cuda() for n, v in dev.items()}
    if d_loss is not None:
        _, dev["counts"], dev["tokens"] = ftq.moe_balance(*_cuda(logits, ids), score=score, offsets=dev["offsets"], valid=dev["valid"])
    got = ftq.moe_topk_backward(*_cuda(logits, ids), score=score, renorm=renorm, scale=scale, **dev)
    if check:
        ref, mag = _grad_ref(logits, ids, d_gates, score, renorm, scale, d_loss, offsets, valid)
        # in steps of two units: the shares' 60 units twice (p and the sum over the row), a sum over at most 64 choices (64
        # units), products and differences: below 144 steps
        t.close(got, ref, mag, 34 * 2 + 64 + 12, "d_logits")
    return got


@pytest.mark.parametrize("score", [ftq.SCORE_SOFTMAX, ftq.SCORE_SIGMOID])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("T,E,k,dtype", [(1, 1, 1, "f32"), (1, 8, 2, "bf16"), (40, 60, 4, "f16"), (65, 97, 5, "f32"), (33, 128, 8, "bf16"),
                                         (50, 256, 8, "f32"), (9, 200, 64, "f32"), (20, 511, 3, "f16"), (17, 1023, 8, "f32"), (18, 1024, 8, "f32")])
def test_gradient(T, E, k, dtype, renorm, score):
    print(f"[topk_backward] T={T} E={E} k={k} {dtype} renorm={renorm} score={score}", flush=True)
    g, logits, ids = _inputs(T, E, k, dtype, seed=T + E)
    d_gates, d_loss = torch.randn(T, k, generator=g), torch.rand(1, generator=g) + 0.5
    _check_grad(logits, ids, score, renorm, 2.5, d_gates=d_gates)
    _check_grad(logits, ids, score, renorm, 2.5, d_loss=d_loss)
    _check_grad(logits, ids, score, renorm, 2.5, d_gates=d_gates, d_loss=d_loss)


@pytest.mark.parametrize("score", [ftq.SCORE_SOFTMAX, ftq.SCORE_SIGMOID])
@pytest.mark.parametrize("renorm", [True, False])
def test_gradient_of_packed_sequences(renorm, score):
    T, E, k, S = 700, 64, 6, 60
    g, logits, ids = _inputs(T, E, k, "f32", seed=4)
    ids[torch.rand(T, k, generator=g) < 0.1] = -1
    ids[torch.rand(T, k, generator=g) < 0.05] = E
    ids[:, 1] = torch.where(torch.rand(T, generator=g) < 0.1, ids[:, 0], ids[:, 1])
    ids[9] = -1
    valid = torch.rand(T, generator=g) >= 0.1
    offsets = _cuts(g, T, S, 5, 60)
    d_gates, d_loss = torch.randn(T, k, generator=g), torch.randn(S, generator=g)
    _check_grad(logits, ids, score, renorm, 0.7, d_gates, d_loss, offsets, valid)
    only = _check_grad(logits, ids, score, renorm, 0.7, None, d_loss, offsets, valid)
    assert not only[:5].any() and not only[-60:].any() and not only[~valid.cuda()].any()
    dirty = logits.clone()
    dirty[~valid] = float("nan")                               # padding holds anything and stays out
    a = _check_grad(dirty, ids, score, renorm, 0.7, d_gates, d_loss, offsets, valid, check=False)
    b = _check_grad(logits, ids, score, renorm, 0.7, d_gates, d_loss, offsets, valid, check=False)
    assert torch.equal(a, b)


@pytest.mark.parametrize("E,k", [(2, 64), (31, 64), (8, 9), (100, 33)])
def test_gradient_of_many_choices(E, k):
    """More choices than lanes of a row, and than experts: every expert several times."""
    g, logits, _ = _inputs(200, E, 1, "f32", seed=E)
    ids = torch.randint(-1, E, (200, k), generator=g).to(torch.int32)
    d_gates, d_loss = torch.randn(200, k, generator=g), torch.rand(1, generator=g)
    for score in SOFT:
        _check_loss(logits, ids, score)
        for renorm in (True, False):
            _check_grad(logits, ids, score, renorm, 1.0, d_gates, d_loss)


@pytest.mark.parametrize("score", [ftq.SCORE_SOFTMAX, ftq.SCORE_SIGMOID])
def test_gradient_of_strange_rows(score):
    T, E, k = 12, 64, 4
    g, logits, ids = _inputs(T, E, k, "f32", seed=5)
    logits[1, ids[1, 0].long()] = -INF                         # a choice that is not available
    logits[2] = -INF
    logits[4] *= 100.0                                         # scores that 32 bits cannot hold beside their row's largest
    logits[5, 10:] = -INF
    d_gates, d_loss = torch.randn(T, k, generator=g), torch.rand(1, generator=g)
    for renorm in (True, False):
        got = _check_grad(logits, ids, score, renorm, 1.0, d_gates, d_loss, check=False)
        assert got[1, ids[1, 0].long()] == 0 and not got[2].any() and not got[5, 10:].any() and got.isfinite().all()
    rows = torch.tensor([0, 3, 4, 6, 7])
    _check_grad(logits[rows], ids[rows], score, True, 1.0, d_gates[rows])
    bad = logits.clone()
    bad[7, 2] = float("nan")
    noids = ids.clone()
    noids[7] = -1                                              # as the router leaves such a row
    got = _check_grad(bad, noids, score, True, 1.0, d_gates, check=False)
    assert not got[7].any()
    loss = ftq.moe_balance(logits.cuda(), noids.cuda(), score=score)
    got = ftq.moe_topk_backward(bad.cuda(), noids.cuda(), d_loss=d_loss.cuda(), counts=loss[1], tokens=loss[2], score=score)
    assert got[7].isnan().all() and not got[:7].isnan().any() and not got[8:].isnan().any()


@pytest.mark.parametrize("score", [ftq.SCORE_SOFTMAX, ftq.SCORE_SIGMOID])
@pytest.mark.parametrize("renorm", [True, False])
def test_gradient_against_differences(renorm, score):
    T, E, k, S = 60, 40, 4, 3
    g, logits, ids = _inputs(T, E, k, "f32", seed=6)
    offsets = _cuts(g, T, S)
    d_gates, d_loss = torch.randn(T, k, generator=g), torch.rand(S, generator=g)
    got = _check_grad(logits, ids, score, renorm, 1.5, d_gates, d_loss, offsets).double().cpu()
    seqs = t.sequences(T, offsets, None)

    def value(l):
        return float((t.gates_of(l, ids, SOFT[score], renorm, 1.5) * d_gates.double()).sum()
                     + (t.losses(l, ids, E, k, seqs, SOFT[score]) * d_loss.double()).sum())
    for seed in range(5):
        v = torch.randn(T, E, generator=g).double()
        e = 1e-5                                               # error e^2 * third derivative (about 1) and 1e-16 * value / e
        want = (value(logits.double() + e * v) - value(logits.double() - e * v)) / (2 * e)
        assert abs(want - float((got * v).sum())) <= 1e-6 * float((got * v).abs().sum()) + 1e-8


def test_gradient_strides_and_refusals():
    T, E, k = 50, 30, 3
    g, wide, ids = _inputs(T, 48, k, "bf16", seed=7)
    ids %= E
    d_gates = torch.randn(T, k, generator=g).cuda()
    out = torch.full((T, 40), 7.0, dtype=torch.bfloat16, device="cuda")
    a = ftq.moe_topk_backward(wide.cuda()[:, 5:35], ids.cuda(), d_gates, out=out[:, 3:33])
    b = ftq.moe_topk_backward(wide[:, 5:35].contiguous().cuda(), ids.cuda(), d_gates)
    assert torch.equal(a, b) and (out[:, :3] == 7).all() and (out[:, 33:] == 7).all()
    l = wide[:, :E].contiguous().cuda()
    for kw in (dict(), dict(d_loss=torch.ones(1, device="cuda")), dict(d_gates=d_gates.half()), dict(d_gates=d_gates[:, :2].contiguous()),
               dict(d_gates=d_gates, valid=torch.ones(T, device="cuda")), dict(d_gates=d_gates, out=torch.empty(T, E, device="cuda"))):
        with pytest.raises((ValueError, ftq.FtqError)):
            ftq.moe_topk_backward(l, ids.cuda(), **kw)
    assert ftq.moe_topk_backward(l[:0], ids[:0].cuda(), d_gates[:0]).shape == (0, E)


# ---- the combine ---------------------------------------------------------------------

@pytest.mark.parametrize("T,k,N,dtype", [(1, 1, 1, "f32"), (1, 2, 4096, "bf16"), (7, 8, 100, "f16"), (33, 3, 257, "bf16"), (20, 64, 1030, "f32"), (5, 2, 9001, "f16")])
def test_combine_gradient(T, k, N, dtype):
    print(f"[combine_backward] T={T} k={k} N={N} {dtype}", flush=True)
    g = torch.Generator().manual_seed(N)
    d_out, y, gates = torch.randn(T, N, generator=g), torch.randn(T * k, N, generator=g), torch.randn(T, k, generator=g)
    d_y, d_gates = ftq.combine_topk_backward(d_out.cuda(), y.cuda(), gates.cuda(), d_y_dtype=t.DTYPES[dtype])
    prod = (gates[:, :, None].double() * d_out[:, None, :].double()).view(T * k, N)
    # one rounding to fp32, one to the type (for fp16 the hardware may round the exact product at once: within the same bound,
    # but not the same bits as the two roundings)
    t.close(d_y, prod, prod.abs(), 1, "d_y")
    terms = y.view(T, k, N).double() * d_out[:, None, :].double()
    t.close(d_gates, terms.sum(2), terms.abs().sum(2), N + 2, "d_gates")
    # one of the two alone: the same bits; and rows by themselves too
    L, P = ftq.lib(), lambda v: v.data_ptr() if v is not None else None
    a, b, c = d_out.cuda(), y.cuda(), gates.cuda()
    only_y, only_g = torch.empty_like(d_y), torch.empty_like(d_gates)
    dt = ftq._DTYPE[d_y.dtype]
    assert L.ftq_moe_combine_topk_backward(P(a), None, P(c), P(only_y), dt, None, T, k, N, None) == ftq.OK
    assert L.ftq_moe_combine_topk_backward(P(a), P(b), None, None, dt, P(only_g), T, k, N, None) == ftq.OK
    torch.cuda.synchronize()
    assert torch.equal(only_y, d_y) and torch.equal(only_g, d_gates)
    last = ftq.combine_topk_backward(a[-1:].clone(), b[-k:].clone(), c[-1:].clone(), d_y_dtype=t.DTYPES[dtype])
    assert torch.equal(last[0], d_y[-k:]) and torch.equal(last[1], d_gates[-1:])


def test_combine_gradient_against_differences():
    T, k, N = 6, 3, 40
    g = torch.Generator().manual_seed(1)
    d_out, y, gates = torch.randn(T, N, generator=g), torch.randn(T * k, N, generator=g), torch.randn(T, k, generator=g)
    d_y, d_gates = ftq.combine_topk_backward(d_out.cuda(), y.cuda(), gates.cuda())

    def value(y, gates):                                       # bilinear: differences are exact but for roundings
        return float(((gates[:, :, None] * y.view(T, k, N)).sum(1) * d_out.double()).sum())
    for _ in range(3):
        vy, vg = torch.randn(T * k, N, generator=g).double(), torch.randn(T, k, generator=g).double()
        y0, g0 = y.double(), gates.double()
        want = (value(y0 + vy, g0) - value(y0 - vy, g0)) / 2 + (value(y0, g0 + vg) - value(y0, g0 - vg)) / 2
        got = float((d_y.cpu().double() * vy).sum() + (d_gates.cpu().double() * vg).sum())
        assert abs(want - got) <= 1e-5 * (1 + abs(want))


# ---- offsets past 32 bits -------------------------------------------------------------

def test_router_offsets_past_32_bits():
    T, E, k = (1 << 21) + 300, 1024, 2                         # 2.1e9 logits
    logits = torch.empty(T, E, dtype=torch.bfloat16, device="cuda").normal_()
    ids = torch.randint(0, E, (T, k), dtype=torch.int32, device="cuda")
    offsets = torch.tensor([0, T - 77, T], dtype=torch.int32, device="cuda")
    loss, counts, tokens = ftq.moe_balance(logits, ids, offsets=offsets)
    assert tokens.tolist() == [T - 77, 77]
    assert torch.equal(counts[0], torch.bincount(ids[:-77].reshape(-1).long(), minlength=E).to(torch.int32))
    tail = [logits[-77:].clone(), ids[-77:].clone()]
    few = ftq.moe_balance(*tail)
    assert torch.equal(counts[1], few[1][0]) and abs(float(loss[1]) / float(few[0][0]) - 1) <= 2 * t.U * 100
    # evenly spread pairs: the loss is 1 but for the spread of counts and probabilities over 2e6 rows
    assert abs(float(loss[0]) - 1) < 1e-3
    d_gates, d_loss = torch.randn(T, k, device="cuda"), torch.rand(2, device="cuda")
    got = ftq.moe_topk_backward(logits, ids, d_gates, d_loss=d_loss, counts=counts, tokens=tokens, offsets=offsets)
    want = ftq.moe_topk_backward(*tail, d_gates[-77:].clone(), d_loss=d_loss[1:].clone(), counts=counts[1:].clone(), tokens=tokens[1:].clone())
    assert torch.equal(got[-77:], want)


def test_combine_offsets_past_32_bits():
    T, k, N = 33000, 2, 33000                                  # 2.2e9 values of y
    y = torch.zeros(T * k, N, device="cuda")
    y[-6:] = torch.randn(6, N, device="cuda")
    d_out, gates = torch.zeros(T, N, device="cuda"), torch.rand(T, k, device="cuda")
    d_out[-3:] = torch.randn(3, N, device="cuda")
    d_y, d_gates = ftq.combine_topk_backward(d_out, y, gates, d_y_dtype=torch.bfloat16)
    few = ftq.combine_topk_backward(d_out[-3:].clone(), y[-6:].clone(), gates[-3:].clone(), d_y_dtype=torch.bfloat16)
    assert torch.equal(d_y[-6:], few[0]) and torch.equal(d_gates[-3:], few[1])
    assert not d_y[:-6].any() and not d_gates[:-3].any()
