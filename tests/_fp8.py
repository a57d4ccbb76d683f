"""Shared helpers of the 8-bit floating-point and router tests: the formats and
definitions in 64 bits, on the host (numpy) or, for the large products, as plain
64-bit torch products."""
from __future__ import annotations

import math

import numpy as np
import torch

BLOCK = 128
U32 = 2.0 ** -24
DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def e4m3_table() -> np.ndarray:
    """The value of each of the 256 e4m3 codes: sign, four exponent bits (bias 7), three mantissa bits."""
    v = np.empty(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        x = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        if e == 15 and m == 7:
            x = math.nan
        v[c] = -x if c & 128 else x
    return v


TABLE = e4m3_table()


def e4m3_codes(q: np.ndarray) -> np.ndarray:
    """fp32 quotients to codes: nearest value, ties to the even code, saturated; NaN to 0x7f (sign ignored)."""
    mag = np.minimum(np.abs(q.astype(np.float64)), 448.0)
    grid = TABLE[:127]                                  # ascending, codes 0 .. 126
    hi = np.searchsorted(grid, np.where(np.isnan(mag), 0.0, mag)).clip(1, 126)
    lo = hi - 1
    dl, dh = mag - grid[lo], grid[hi] - mag
    code = np.where(dl < dh, lo, np.where(dh < dl, hi, np.where(lo % 2 == 0, lo, hi)))
    code = np.where(mag == 0, 0, code) | (np.signbit(q).astype(np.int64) << 7)
    return np.where(np.isnan(q), 0x7f, code).astype(np.uint8)


def block_scales(x: np.ndarray, axes) -> np.ndarray:
    with np.errstate(all="ignore"):
        return (np.abs(x).max(axis=axes) / np.float32(448.0)).astype(np.float32)


def quantize_rows(x: np.ndarray):
    """fp32 [T, K] -> (codes, scales) by the definition, in the fp32 steps it names."""
    T, K = x.shape
    nb = -(-K // BLOCK)
    v = np.zeros((T, nb * BLOCK), np.float32)
    v[:, :K] = x
    v = v.reshape(T, nb, BLOCK)
    s = block_scales(v, 2)
    with np.errstate(all="ignore"):
        q = np.where(s[..., None] == 0, np.float32(0), v / s[..., None]).astype(np.float32)
    return e4m3_codes(q).reshape(T, nb * BLOCK)[:, :K], s


def quantize_weight(w: np.ndarray):
    E, N, K = w.shape
    nr, nb = -(-N // BLOCK), -(-K // BLOCK)
    v = np.zeros((E, nr * BLOCK, nb * BLOCK), np.float32)
    v[:, :N, :K] = w
    v = v.reshape(E, nr, BLOCK, nb, BLOCK)
    s = block_scales(v, (2, 4))
    with np.errstate(all="ignore"):
        q = np.where(s[:, :, None, :, None] == 0, np.float32(0), v / s[:, :, None, :, None]).astype(np.float32)
    return e4m3_codes(q).reshape(E, nr * BLOCK, nb * BLOCK)[:, :N, :K], s


def _act64(name, g):
    if name == "silu":
        return g / (1 + torch.exp(-g))
    return 0.5 * g * (1 + torch.tanh(math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3)))


def moe64(w, ws, a, as_, ids, per_pair, act=None, coarse=False):
    """(result, bound) of the expert matmul in 64 bits for fp32 results.

    bound: an element's fp32 error.  Within a block of 128 the products are exact
    and their sum is off by at most 128 roundings or truncations (2^-23 each); the
    scales' product is one rounding, each block's FMA one, the sum over up to 8
    waves' parts 8 (2^-24 each), all relative to the sum of the terms' magnitudes.
    coarse (16-bit results of the grouped path): the 8-bit matrix instructions drop, of
    seven products in eight, what lies below 2^-13 of the eighth: 7 * 2^-13 of the sum
    of magnitudes more.
    An activation adds: |act'| <= 1.13, 9 roundings of act and one product."""
    T, k = ids.shape
    E, N, K = w.shape
    flat = ids.reshape(-1)
    nb = -(-K // BLOCK)
    cols = N if act is None else N // 2
    out = torch.zeros(flat.numel(), cols, dtype=torch.float64, device=w.device)
    bound = torch.zeros_like(out)
    kb = torch.arange(K, device=w.device) // BLOCK
    rb = torch.arange(N, device=w.device) // BLOCK
    rel = 128 * 2 * U32 + (1 + nb + 8) * U32 + (7 * 2.0 ** -13 if coarse else 0.0)
    for e in range(E):
        p = (flat == e).nonzero()[:, 0]
        if not len(p):
            continue
        r = p if per_pair else p // k
        x = a.view(torch.uint8)[r].view(a.dtype).double() * as_[r].double()[:, kb]
        we = w[e].double() * ws[e].double()[rb][:, kb]
        y, mag = x @ we.t().contiguous(), x.abs() @ we.abs().t().contiguous()
        d = rel * mag
        if act is None:
            out[p], bound[p] = y, d
        else:
            g, u, dg, du = y[:, :cols], y[:, cols:], d[:, :cols], d[:, cols:]
            f = _act64(act, g)
            out[p] = f * u
            bound[p] = 1.13 * dg * (u.abs() + du) + f.abs() * du + 9 * U32 * (f.abs() + 1.13 * dg + g.abs() + dg) * (u.abs() + du)
    return out, bound


def assert_close(got, ref, bound, what=""):
    """got (fp32, fp16 or bf16) within the fp32 bound plus one rounding to its type (half a step, or half the
    smallest subnormal step)."""
    eps = torch.finfo(got.dtype).eps / 2 if got.dtype != torch.float32 else 0.0
    tiny = {torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134, torch.float32: 0.0}[got.dtype]
    d = (got.double() - ref).abs()
    lim = bound + eps * (ref.abs() + bound) + tiny
    bad = ~(d <= lim)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {d.numel()} off, worst {float((d - lim).max()):.3e} over its bound"
