"""The two forms of the 8-bit floating-point products on the GPU: exact ones for 16-bit results when
they are asked for."""
import pytest
import torch

from quantized_moe_expert_quantize_amd import ftq
from tests._cases import say
from tests._fp8 import DTYPES, assert_close, moe64
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
