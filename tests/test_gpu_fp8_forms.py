"""The two forms of the 8-bit floating-point products on the GPU: exact ones for 16-bit results when
they are asked for; what the fast one loses, and that a row keeps its bits in it."""
import math

import pytest
import torch

from quantized_moe_expert_quantize_amd import ftq, inputs
from tests._cases import say
from tests._fp8 import DTYPES, _act64, assert_close, moe64
from tests.test_gpu_fp8 import Experts

pytestmark = pytest.mark.gpu

ACTS = {None: 0, "silu": ftq.ACT_SILU, "gelu": ftq.ACT_GELU_TANH}
# tiles of 32, 64 and 256 pairs, ragged in pairs, rows and columns
SHAPES = [(8, 96, 272, 20, 2), (8, 320, 512, 150, 2), (2, 544, 400, 300, 2), (1, 224, 1152, 700, 1), (16, 32, 16, 5, 3)]


def call(c, path, act, dtype, exact):
    return ftq.moe_fp8(c.w, c.ws, c.a, c.as_, c.ids, c.E, c.N, c.K, per_pair=c.per_pair, act=ACTS[act], path=path, out_dtype=DTYPES[dtype],
                       exact=exact)


def assert_rounded(got, full, product):
    """got is the fp32 result rounded to its type.  product: the last step of the result is a product p of two fp32
    values, which an instruction may round to fp16 in one step.  That differs from rounding it to fp32 and then to
    fp16 only if the fp32 rounding of p crosses or reaches a border between two fp16 results; such a border, having 12
    significant bits, is an fp32 number, and rounding to fp32, being monotonic, reaches it but does not cross it: the fp32
    result is then exactly midway between the two fp16 ones."""
    want = full.to(got.dtype)
    d = got != want
    assert product or not d.any()
    v, g, w = full[d].double(), got[d].double(), want[d].double()
    assert ((v - g).abs() == (v - w).abs()).all() and (g != w).all()


@pytest.mark.parametrize("path", [ftq.PATH_GEMV, ftq.PATH_GROUPED])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("act", [None, "silu", "gelu"])
def test_exact_16_bit_results_are_the_rounded_fp32_ones(path, dtype, act):
    for shape in SHAPES:
        for per_pair in (False, True):
            say(f"[fp8] exact {shape} path={path} {dtype} {act} per_pair={per_pair}")
            c = Experts(*shape, per_pair=per_pair, seed=sum(shape), masked=5)
            got = call(c, path, act, dtype, True)
            assert_rounded(got, call(c, path, act, "f32", False), act is not None and dtype == "f16")
            assert_close(got, *moe64(c.w, c.ws, c.a, c.as_, c.ids, per_pair, act), "exact")
            if path == ftq.PATH_GEMV:
                assert torch.equal(got, call(c, path, act, dtype, False))


@pytest.mark.parametrize("T", [40, 200, 600])
def test_exact_products_of_terms_that_cancel(T):
    """Every eight terms: two of +-2^16 and six of +-4, which are the result and lie below 2^-13 of the largest."""
    E, N, K = 2, 64, 512
    w = torch.full((E, N, K), 2.0, device="cuda")
    a = torch.full((T, K), 2.0, device="cuda")
    w[:, :, ::8], w[:, :, 1::8] = 256.0, 256.0
    a[:, ::8], a[:, 1::8] = 256.0, -256.0
    w[:, ::3, 2::8] = -2.0
    w, a = w.to(ftq.FP8), a.to(ftq.FP8)
    ws, as_ = torch.ones(E, 1, 4, device="cuda"), torch.ones(T, 4, device="cuda")
    ids = (torch.arange(T, device="cuda") % 2).to(torch.int32)[:, None].contiguous()
    want = torch.full((T, N), 64 * 6 * 4.0, device="cuda")
    want[:, ::3] = 64 * (5 - 1) * 4.0
    # in whatever order, the sums of a block stay below 16 * 2^16, so that an addition in 32 bits is off by 2^-3 at
    # most; both results are numbers of every type
    for dtype in ("f32", "f16", "bf16"):
        for path in (ftq.PATH_GEMV, ftq.PATH_GROUPED):
            out = ftq.moe_fp8(w, ws, a, as_, ids, E, N, K, path=path, out_dtype=DTYPES[dtype], exact=True)
            assert (out.double() - want.double()).abs().max() <= K * 2.0 ** -3, (dtype, path)


def test_exact_on_routed_pairs():
    c = Experts(8, 320, 512, 150, 2, seed=1)
    ws = torch.empty(ftq.fp8_workspace_bytes(8, 320, 512, 150, 2, ftq.PATH_GROUPED), dtype=torch.uint8, device="cuda")
    ftq.moe_fp8_route(c.ids, 8, ws, ftq.PATH_GROUPED)
    for act in (None, "silu"):
        out = torch.empty(300, 320 if act is None else 160, dtype=torch.bfloat16, device="cuda")
        ftq.moe_fp8_routed(c.w, c.ws, c.a, c.as_, c.ids, 8, 320, 512, out, ws, ftq.PATH_GROUPED, act=ACTS[act], exact=True)
        assert torch.equal(out, call(c, ftq.PATH_GROUPED, act, "bf16", True))


# What the fast form loses of a result's norm on normal values is given as 1.5e-5; twice that is allowed.
FAST = 3e-5


@pytest.mark.parametrize("act", [None, "silu", "gelu"])
@pytest.mark.parametrize("T", [60, 300, 1300], ids=["tiles of 32", "tiles of 64", "tiles of 256"])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_fast_products_lose_little_of_the_norm(dtype, T, act):
    """Against the 64-bit results rounded to the type, in norm.

    With d the fast form's error of an element and u the step of the type there, the rounded results differ by u with
    probability |d| / u (the 64-bit results lie anywhere between two numbers of the type), so that the squares add up to
    sum |d| u <= |d| |u| in norms.  u is at most 2^-10 (fp16) or 2^-7 (bf16) of the element.  A dropped
    product or three more lost bits do not pass."""
    E, N, K, k = 8, 320, 2048, 2
    g = torch.Generator().manual_seed(T)
    w, ws = ftq.quantize_fp8_weight((torch.randn(E, N, K, generator=g) / math.sqrt(K)).cuda())
    a, as_ = ftq.quantize_fp8(torch.randn(T, K, generator=g).cuda())
    ids = torch.from_numpy(inputs.routing(T, E, k, seed=T)).cuda()
    got = ftq.moe_fp8(w, ws, a, as_, ids, E, N, K, act=ACTS[act], path=ftq.PATH_GROUPED, out_dtype=DTYPES[dtype])
    y, _ = moe64(w, ws, a, as_, ids, False)
    loss = FAST * y.square().mean().sqrt()               # of an element without activation
    if act is None:
        ref, d = y, torch.full_like(y, loss)
    else:
        gate, up = y[:, : N // 2], y[:, N // 2:]
        ref = _act64(act, gate) * up
        slope = (_act64(act, gate + 1e-6) - _act64(act, gate - 1e-6)) / 2e-6
        d = loss * ((slope * up).square() + _act64(act, gate).square()).sqrt()
    step = {"f16": 2.0 ** -10, "bf16": 2.0 ** -7}[dtype]
    off = (got.double() - ref.to(DTYPES[dtype]).double()).norm()
    lim = (d.norm() * step * ref.norm() + d.norm() ** 2).sqrt()
    say(f"[fp8] fast {dtype} T={T} {act}: {float(off / ref.norm()):.2e} of {float(lim / ref.norm()):.2e}")
    assert off <= lim


@pytest.mark.parametrize("act", [None, "silu"])
@pytest.mark.parametrize("exact", [False, True])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_a_16_bit_row_does_not_depend_on_the_batch(dtype, exact, act):
    """A pair's bits alone, in a part and in the whole batch, by kernels of every tile height."""
    E, N, K, k = 8, 224, 1424, 2
    for T in (60, 300, 1300):
        c = Experts(E, N, K, T, k, seed=T)
        whole = call(c, ftq.PATH_GROUPED, act, dtype, exact)
        for a, b in ((0, 1), (0, 7), (T // 3, T // 3 + 200), (T // 2, T), (T - 1, T)):
            part = ftq.moe_fp8(c.w, c.ws, c.a[a:b], c.as_[a:b], c.ids[a:b].contiguous(), E, N, K, path=ftq.PATH_GROUPED, act=ACTS[act],
                               out_dtype=DTYPES[dtype], exact=exact)
            assert torch.equal(part, whole[a * k: min(b, T) * k]), (T, a, b)


def test_quantiser_offsets_past_32_bits():
    """Activations by rows and by their stride, and weights, whose offsets pass 2^32."""
    g = torch.Generator().manual_seed(2)
    x = torch.randn(6, 272, generator=g).bfloat16().cuda()
    q, s = ftq.quantize_fp8(x)
    far = torch.empty(5 * (1 << 30) + 272, dtype=torch.bfloat16, device="cuda")
    rows = far.as_strided((6, 272), (1 << 30, 1))
    rows.copy_(x)
    say("[fp8] quantise far rows by stride")
    q2, s2 = ftq.quantize_fp8(rows)
    assert torch.equal(q2.view(torch.uint8), q.view(torch.uint8)) and torch.equal(s2, s)
    T = (1 << 24) + 6
    many = far[: T * 272].view(T, 272)
    many.zero_()
    many[-6:] = x
    say("[fp8] quantise far rows by number")
    q2, s2 = ftq.quantize_fp8(many)
    assert torch.equal(q2[-6:].view(torch.uint8), q.view(torch.uint8)) and torch.equal(s2[-6:], s)
    assert not q2[:-6].view(torch.uint8).any() and not s2[:-6].any()
    del q2, s2
    E, N, K = 17, 16384, 16400
    w = far[: E * N * K].view(E, N, K)
    w.zero_()
    w[-1, -6:, -272:] = x
    say("[fp8] quantise far weights")
    q2, s2 = ftq.quantize_fp8_weight(w)
    alone = torch.zeros(1, 128, K, dtype=torch.bfloat16, device="cuda")
    alone[0, -6:, -272:] = x
    q1, s1 = ftq.quantize_fp8_weight(alone)
    assert torch.equal(q2[-1, -128:].view(torch.uint8), q1[0].view(torch.uint8)) and torch.equal(s2[-1, -1], s1[0, 0])
    q2[-1, -6:, -272:] = 0
    assert not q2.view(torch.uint8).any() and not s2[:-1].any() and not s2[-1, :-1].any()
