"""Shared helpers of the tests of what trains beside frozen experts: definitions in
64 bits on the host, and comparisons that count roundings."""
from __future__ import annotations

import torch

U = 2.0 ** -24                                   # half a step of fp32, relative
DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
TINY = {torch.float32: 2.0 ** -149, torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -133}   # half a step near 0


def close(got, ref, mag, terms, what=""):
    """|got - ref| within `terms` fp32 roundings (a step each, whatever way they go) of the terms' magnitudes and one
    rounding to got's type; and in norm within four times what as many roundings of random sign make."""
    half = torch.finfo(got.dtype).eps / 2 if got.dtype != torch.float32 else U
    got, ref, mag = got.cpu(), ref.cpu(), mag.cpu()
    off = (got.double() - ref).abs()
    # the reference's own roundings: sums in 64 bits (up to 2^13 terms of at most mag's largest, 2^-53 each) that
    # cancel exactly in the definition, as a renormalised gate's do for the experts not chosen, leave their remainders
    own = 2.0 ** -40 * mag.max() if mag.numel() else 0.0
    tol = 2 * U * terms * mag + half * (1 + 2 * U * terms) * ref.abs() + TINY[got.dtype] + own
    bad = ~(off <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off, worst {float((off / tol.clamp_min(1e-300)).max()):.3g} of the bound"
    norm = 4 * (2 * U * terms ** 0.5 * mag.norm() + half * ref.norm()) + (TINY[got.dtype] + own) * ref.numel() ** 0.5
    assert off.norm() <= norm, f"{what}: norm {float(off.norm()):.3g}, at most {float(norm):.3g}"


# ---- router --------------------------------------------------------------------

def sequences(T, offsets, valid):
    """Counted rows of each sequence."""
    cuts = [0, T] if offsets is None else [int(v) for v in offsets]
    ok = torch.ones(T, dtype=torch.bool) if valid is None else valid.cpu()
    return [torch.tensor([t for t in range(max(b, 0), min(e, T)) if ok[t]], dtype=torch.long) for b, e in zip(cuts, cuts[1:])]


def scores(l, softmax):
    if softmax:
        s = torch.exp(l - l.amax(1, keepdim=True).clamp_min(-1e300))
        total = s.sum(1, keepdim=True)
        return s / torch.where(total == 0, torch.ones_like(total), total)
    return torch.sigmoid(l)


def shares(l, softmax):
    s = scores(l, softmax)
    if softmax:
        return s
    total = s.sum(1, keepdim=True)
    return s / torch.where(total == 0, torch.ones_like(total), total)


def counts_of(ids, rows, E):
    flat = ids[rows].reshape(-1).long()
    return torch.bincount(flat[(flat >= 0) & (flat < E)], minlength=E)


def losses(l, ids, E, top_k, seqs, softmax):
    out = []
    for rows in seqs:
        n = max(len(rows), 1)
        out.append(E / (top_k * n * n) * (counts_of(ids, rows, E).double() * shares(l[rows], softmax).sum(0)).sum())
    return torch.stack(out)


def gates_of(l, ids, softmax, renorm, scale):
    """Gates of the chosen experts (0 for ids that name none), differentiable."""
    E = l.shape[1]
    ok = (ids >= 0) & (ids < E)
    s = scores(l, softmax).gather(1, ids.long().clamp(0, E - 1)) * ok
    if renorm:
        total = s.sum(1, keepdim=True)
        s = s / torch.where(total == 0, torch.ones_like(total), total)
    return scale * s


# ---- adapters --------------------------------------------------------------------

def row_of(ids, per_pair):
    T, k = ids.shape
    p = torch.arange(T * k)
    return p if per_pair else p // k


def lora_forward(x, a, b, ids, scale, base, per_pair):
    """(out, h, magnitude of out's terms, magnitude of h's terms) in 64 bits."""
    L, R, K = a.shape
    N = b.shape[1]
    flat, row = ids.reshape(-1).cpu(), row_of(ids, per_pair)
    x, a, b = x.cpu().double(), a.cpu().double(), b.cpu().double()
    out = base.cpu().double().clone() if base is not None else torch.zeros(len(flat), N, dtype=torch.float64)
    h = torch.zeros(len(flat), R, dtype=torch.float64)
    mo, mh = out.abs(), torch.zeros_like(h)
    for l in range(L):
        p = (flat == l).nonzero()[:, 0]
        if len(p):
            s = 1.0 if scale is None else float(scale[l])
            h[p] = x[row[p]] @ a[l].t()
            mh[p] = x[row[p]].abs() @ a[l].abs().t()
            out[p] += s * (h[p] @ b[l].t())
            mo[p] += abs(s) * (mh[p] @ b[l].abs().t())
    return out, h, mo, mh


def lora_backward(dy, x, a, b, ids, h, scale, base, per_pair):
    """{name: (gradient, magnitude of its terms)} in 64 bits."""
    L, R, K = a.shape
    flat, row = ids.reshape(-1).cpu(), row_of(ids, per_pair)
    dy, x, a, b, h = (t.cpu().double() for t in (dy, x, a, b, h))
    dx = base.cpu().double().clone() if base is not None else torch.zeros_like(x)
    mx = dx.abs()
    da, db = torch.zeros_like(a), torch.zeros_like(b)
    ma, mb = torch.zeros_like(a), torch.zeros_like(b)
    for l in range(L):
        p = (flat == l).nonzero()[:, 0]
        if len(p):
            s = 1.0 if scale is None else float(scale[l])
            g, mg = s * (dy[p] @ b[l]), abs(s) * (dy[p].abs() @ b[l].abs())
            dx.index_add_(0, row[p], g @ a[l])
            mx.index_add_(0, row[p], mg @ a[l].abs())
            da[l], ma[l] = g.t() @ x[row[p]], mg.t() @ x[row[p]].abs()
            db[l], mb[l] = s * (dy[p].t() @ h[p]), abs(s) * (dy[p].abs().t() @ h[p].abs())
    return {"d_x": (dx, mx), "d_a": (da, ma), "d_b": (db, mb)}
