"""8-bit floating-point quantisers and expert matmul on the GPU: codes and scales
bit for bit, products against 64 bits within the fp32 evaluation's bound, at the
sizes, types and masks where they can go wrong; and the whole expert layer."""
import math

import numpy as np
import pytest
import torch

from quantized_moe_expert_quantize_amd import ftq, inputs
from tests import _fp8
from tests._cases import say
from tests._fp8 import DTYPES, assert_close, moe64

pytestmark = pytest.mark.gpu


# ---- quantisers ----------------------------------------------------------------

def _values(shape, seed):
    g = np.random.default_rng(seed)
    x = g.standard_normal(shape).astype(np.float32) * np.exp(2 * g.standard_normal(shape[-1])).astype(np.float32)
    return x


def _codes(t):
    return t.view(torch.uint8).cpu().numpy()


def _same_codes(got, want):
    nan = (got & 0x7F) == 0x7F
    return np.array_equal(np.where(nan, 0x7F, got), np.where((want & 0x7F) == 0x7F, 0x7F, want))


def _check_rows(x, ld=None):
    """x: CPU tensor [T, K] of its own type."""
    T, K = x.shape
    buf = torch.full((T, ld or K), 9.0, dtype=x.dtype, device="cuda")
    buf[:, :K] = x.cuda()
    q = torch.full((T + 1, K), 3.0, device="cuda").to(ftq.FP8)
    s = torch.full((T + 1, -(-K // 128)), 7.0, device="cuda")
    ftq.quantize_fp8(buf[:, :K], out=q[:T], scales=s[:T])
    torch.cuda.synchronize()
    assert (q[T].float() == 3.0).all() and (s[T] == 7.0).all(), "rows behind the last were written"
    rq, rs = _fp8.quantize_rows(x.float().numpy())
    assert np.array_equal(s[:T].cpu().numpy(), rs, equal_nan=True)
    assert _same_codes(_codes(q[:T]), rq)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_quantize_rows(dtype):
    for T, K, ld in ((1, 16, None), (1, 128, None), (3, 144, None), (5, 112, 128), (2, 256, 512), (17, 2816, None), (33, 1040, 1072), (4, 4096, None),
                     (700, 1408, None)):
        say(f"[fp8] quantize {dtype} T={T} K={K} ld={ld}")
        _check_rows(torch.from_numpy(np.clip(_values((T, K), T + K), -6e4, 6e4)).to(DTYPES[dtype]), ld)


def test_quantize_extremes():
    """Zero blocks, ties, subnormal blocks, the largest values, NaN and infinities."""
    K = 128
    x = np.zeros((16, K), np.float32)
    x[1, 5] = -0.0
    x[2, :] = 448.0
    x[3, :] = np.linspace(-448, 448, K)
    x[4, 0] = 448.0
    x[4, 1:127] = ((_fp8.TABLE[:126] + _fp8.TABLE[1:127]) / 2).astype(np.float32)      # midpoints of neighbours
    x[5, 0] = -448.0
    x[5, 1:127] = -((_fp8.TABLE[:126] + _fp8.TABLE[1:127]) / 2).astype(np.float32)
    x[6, :] = np.float32(1e-45)
    x[7, :] = np.linspace(-1e-38, 1e-38, K)
    x[8, :] = np.linspace(-1e-43, 1e-43, K)
    x[9, :] = np.linspace(-3.4e38, 3.4e38, K)
    x[10, 3] = math.nan
    x[10, 4] = 1.0
    x[11, 7] = math.inf
    x[11, 8] = -2.0
    x[12, 1] = -math.inf
    x[12, 2] = math.nan
    x[13, :] = np.float32(3.0) * np.float32(2.0) ** np.arange(-100, 28)
    x[14, 9] = 1.17549435e-38 * 448
    x[14, 10] = 1e-40
    x[15, :] = np.nextafter(np.float32(448), np.float32(0))
    _check_rows(torch.from_numpy(x))


def test_quantize_every_quotient_of_a_wide_range():
    """A million quotients over the whole range of codes."""
    g = np.random.default_rng(1)
    _check_rows(torch.from_numpy((g.standard_normal((512, 2048)) * np.exp(4 * g.standard_normal((512, 1)))).astype(np.float32)))


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_quantize_weight(dtype):
    for E, N, K in ((1, 1, 16), (2, 128, 128), (3, 130, 144), (2, 100, 272), (1, 257, 512), (5, 64, 1040), (8, 300, 400)):
        say(f"[fp8] weight {dtype} E={E} N={N} K={K}")
        w = torch.from_numpy(_values((E, N, K), E + N + K) * 0.02).to(DTYPES[dtype])
        q = torch.full((E + 1, N, K), 3.0, device="cuda").to(ftq.FP8)
        s = torch.full((E + 1, -(-N // 128), -(-K // 128)), 7.0, device="cuda")
        ftq.quantize_fp8_weight(w.cuda(), out=q[:E], scales=s[:E])
        torch.cuda.synchronize()
        assert (q[E].float() == 3.0).all() and (s[E] == 7.0).all()
        rq, rs = _fp8.quantize_weight(w.float().numpy())
        assert np.array_equal(s[:E].cpu().numpy(), rs)
        assert _same_codes(_codes(q[:E]), rq)


def test_quantize_weight_undefined_blocks():
    w = torch.from_numpy(_values((1, 300, 272), 4))
    w[0, 130, 3] = math.nan
    w[0, 5, 200] = math.inf
    w[0, 256:, 128:256] = 0.0
    q, s = ftq.quantize_fp8_weight(w.cuda())
    rq, rs = _fp8.quantize_weight(w.numpy())
    assert np.array_equal(s.cpu().numpy(), rs, equal_nan=True) and _same_codes(_codes(q), rq)


# ---- matmul ----------------------------------------------------------------------

class Experts:
    """Random codes (every finite one) and scales, and routed rows."""

    def __init__(self, E, N, K, T, k, per_pair=False, seed=0, kind="uniform", masked=0):
        g = np.random.default_rng(seed)
        self.E, self.N, self.K, self.T, self.k, self.per_pair = E, N, K, T, k, per_pair
        rows, nb = T * k if per_pair else T, -(-K // 128)

        def codes(*shape):
            c = g.integers(0, 256, shape, dtype=np.uint8)
            c[(c & 0x7F) == 0x7F] = 0x42
            return torch.from_numpy(c).cuda().view(ftq.FP8)
        self.w, self.a = codes(E, N, K), codes(rows, K)
        self.ws = torch.from_numpy(g.uniform(1e-4, 3e-4, (E, -(-N // 128), nb)).astype(np.float32)).cuda()
        self.as_ = torch.from_numpy(g.uniform(1e-3, 2e-2, (rows, nb)).astype(np.float32)).cuda()
        ids = inputs.routing(T, E, k, seed=seed, kind=kind)
        if masked:
            ids[::masked, 0] = -1
            ids[1::masked + 1, -1] = E + 3
        self.ids = torch.from_numpy(ids).cuda()

    def run(self, path, act=None, dtype="f32"):
        cols = self.N if act is None else self.N // 2
        buf = torch.full((self.T * self.k + 1, cols), 5.0, dtype=DTYPES[dtype], device="cuda")
        ftq.moe_fp8(self.w, self.ws, self.a, self.as_, self.ids, self.E, self.N, self.K, per_pair=self.per_pair,
                    act={None: 0, "silu": ftq.ACT_SILU, "gelu": ftq.ACT_GELU_TANH}[act], path=path, out=buf[:-1])
        torch.cuda.synchronize()
        assert (buf[-1] == 5.0).all(), "rows behind the last were written"
        return buf[:-1]

    def check(self, path, act=None, dtype="f32"):
        if path == ftq.PATH_AUTO:
            path = ftq.fp8_select_path(self.E, self.N, self.K, self.T, self.k)
        coarse = path == ftq.PATH_GROUPED and dtype != "f32"
        ref, bound = moe64(self.w, self.ws, self.a, self.as_, self.ids, self.per_pair, act, coarse)
        out = self.run(path, act, dtype)
        assert_close(out, ref, bound, f"path {path} {act} {dtype}")
        return out


# (E, N, K, T, k): one value, ragged N and K (a partial scale block, a partial row tile), one expert, many experts,
# more pairs than experts and fewer, every tile height of the grouped path
SHAPES = [(1, 1, 16, 1, 1), (2, 5, 16, 3, 1), (8, 64, 256, 4, 2), (8, 100, 144, 5, 2), (4, 130, 400, 7, 3), (8, 257, 512, 33, 2),
          (128, 48, 272, 3, 8), (128, 96, 128, 40, 8), (3, 300, 1040, 50, 2), (8, 192, 384, 300, 2), (2, 513, 640, 200, 1),
          (16, 260, 1408, 90, 4), (1, 256, 1152, 300, 1), (4095, 16, 32, 9, 5),
          (4, 70, 208, 270, 2), (2, 300, 96, 400, 1), (8, 600, 2048, 480, 2), (1, 33, 4112, 513, 1)]


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "E{}N{}K{}T{}k{}".format(*s))
@pytest.mark.parametrize("path", [ftq.PATH_GEMV, ftq.PATH_GROUPED])
def test_shapes(shape, path):
    E, N, K, T, k = shape
    for per_pair in (False, True):
        say(f"[fp8] {shape} path={path} per_pair={per_pair}")
        c = Experts(*shape, per_pair=per_pair, seed=N + T, masked=3 if T > 2 else 0)
        c.check(path)


@pytest.mark.parametrize("path", [ftq.PATH_GEMV, ftq.PATH_GROUPED])
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_activations(path, act):
    for shape in ((8, 32, 128, 4, 2), (4, 96, 272, 50, 2), (8, 544, 512, 300, 2), (16, 256, 384, 100, 4), (128, 352, 256, 5, 8), (2, 1120, 144, 260, 1), (3, 1056, 640, 500, 2)):
        say(f"[fp8] act {shape} path={path} {act}")
        Experts(*shape, seed=shape[1], masked=5).check(path, act)


@pytest.mark.parametrize("path", [ftq.PATH_GEMV, ftq.PATH_GROUPED])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_output_types(path, dtype):
    for shape in ((8, 99, 256, 20, 2), (8, 320, 512, 300, 2), (16, 96, 144, 120, 4), (4, 544, 400, 257, 2), (2, 70, 96, 640, 2), (1, 257, 2064, 700, 1)):
        say(f"[fp8] {shape} path={path} {dtype}")
        Experts(*shape, seed=3).check(path, None, dtype)
        if shape[1] % 32 == 0:
            Experts(*shape, seed=4).check(path, "silu", dtype)


@pytest.mark.parametrize("path", [ftq.PATH_GEMV, ftq.PATH_GROUPED])
def test_unaligned_outputs(path):
    """Output rows that start at any element."""
    c = Experts(8, 68, 256, 200, 2, seed=6)
    for dtype in ("f32", "bf16"):
        ref, bound = moe64(c.w, c.ws, c.a, c.as_, c.ids, False, None, path == ftq.PATH_GROUPED and dtype != "f32")
        buf = torch.full((400 * 68 + 3,), 5.0, dtype=DTYPES[dtype], device="cuda")
        for off in (1, 2, 3):
            buf.fill_(5.0)
            out = buf[off: off + 400 * 68].view(400, 68)
            ftq.moe_fp8(c.w, c.ws, c.a, c.as_, c.ids, 8, 68, 256, path=path, out=out)
            torch.cuda.synchronize()
            assert_close(out, ref, bound, f"{dtype} at {off}")
            assert (buf[:off] == 5.0).all() and (buf[off + 400 * 68:] == 5.0).all()


@pytest.mark.parametrize("path", [ftq.PATH_GEMV, ftq.PATH_GROUPED])
def test_every_pair_on_one_expert_and_repeated_ids(path):
    c = Experts(8, 100, 272, 70, 3, seed=8)
    c.ids.fill_(5)
    c.check(path)
    c.ids[:, 1] = 2
    c.ids[3] = -7
    c.check(path)
    c.ids.fill_(-1)
    assert (c.run(path) == 0).all()
    c.ids.fill_(2 ** 31 - 1)
    assert (c.run(path, "silu") == 0).all() if c.N % 32 == 0 else (c.run(path) == 0).all()


@pytest.mark.parametrize("path", [ftq.PATH_GEMV, ftq.PATH_GROUPED])
def test_nan_reaches_only_its_results(path):
    """NaN codes and scales stay in the rows and columns that they are terms of, also next to ragged ends."""
    c = Experts(4, 70, 144, 9, 2, seed=9)
    clean = c.run(path).clone()
    flat = c.ids.reshape(-1).cpu()
    for what in ("w", "ws", "a", "as_"):
        d = Experts(4, 70, 144, 9, 2, seed=9)
        hit = torch.zeros(18, 70, dtype=torch.bool)
        if what == "w":
            d.w.view(torch.uint8)[1, 69, 143] = 0x7F
            d.w.view(torch.uint8)[2, 0, 0] = 0xFF
            hit[flat == 1, 69] = True
            hit[flat == 2, 0] = True
        elif what == "ws":
            d.ws[3, 0, 1] = math.nan
            hit[flat == 3] = True
        elif what == "a":
            d.a.view(torch.uint8)[8, 143] = 0x7F
            d.a.view(torch.uint8)[0, 0] = 0x7F
            hit[16:] = True
            hit[:2] = True
        else:
            d.as_[4, 0] = math.nan
            hit[8:10] = True
        out = d.run(path)
        assert torch.equal(torch.isnan(out).cpu(), hit), what
        assert torch.equal(out[~hit.cuda()], clean[~hit.cuda()]), what


@pytest.mark.parametrize("path", [ftq.PATH_GEMV, ftq.PATH_GROUPED])
def test_a_row_does_not_depend_on_the_batch(path):
    """Each forced path gives a pair the same bits alone, in a part and in the whole batch (every tile height)."""
    E, N, K, k = 8, 200, 1408, 2
    for T in ((60,) if path == ftq.PATH_GEMV else (60, 300, 900)):
        c = Experts(E, N, K, T, k, seed=T)
        whole = c.run(path)
        for a, b in ((0, 1), (0, 7), (T // 2, T), (T - 1, T)):
            part = ftq.moe_fp8(c.w, c.ws, c.a[a:b], c.as_[a:b], c.ids[a:b].contiguous(), E, N, K, path=path)
            assert torch.equal(part, whole[a * k: b * k]), (T, a, b)


def test_auto_takes_the_selected_path():
    for T in (1, 8, 64, 300):
        c = Experts(8, 96, 256, T, 2, seed=T)
        assert torch.equal(c.run(ftq.PATH_AUTO), c.run(ftq.fp8_select_path(8, 96, 256, T, 2)))


def test_one_routing_serves_both_layers():
    c = Experts(16, 256, 256, 120, 4, seed=2)
    ws = torch.empty(ftq.fp8_workspace_bytes(16, 256, 256, 120, 4, ftq.PATH_GROUPED), dtype=torch.uint8, device="cuda")
    ftq.moe_fp8_route(c.ids, 16, ws, ftq.PATH_GROUPED)
    h = torch.empty(480, 128, device="cuda")
    ftq.moe_fp8_routed(c.w, c.ws, c.a, c.as_, c.ids, 16, 256, 256, h, ws, act=ftq.ACT_SILU, path=ftq.PATH_GROUPED)
    assert torch.equal(h, c.run(ftq.PATH_GROUPED, "silu"))
    d = Experts(16, 300, 128, 120, 4, per_pair=True, seed=3)
    y = torch.empty(480, 300, device="cuda")
    ftq.moe_fp8_routed(d.w, d.ws, d.a, d.as_, c.ids, 16, 300, 128, y, ws, per_pair=True, path=ftq.PATH_GROUPED)
    d.ids = c.ids
    assert torch.equal(y, d.run(ftq.PATH_GROUPED))


@pytest.mark.parametrize("shape", [(128, 1408, 2816, 1, 8), (8, 1000, 4096, 8, 2), (128, 704, 2816, 300, 8), (128, 512, 1408, 2500, 8)], ids=str)
def test_workload_sizes(shape):
    E, N, K, T, k = shape
    say(f"[fp8] {shape}")
    Experts(*shape, seed=1, kind="zipf").check(ftq.PATH_AUTO)


def test_offsets_past_32_bits():
    """Weights, activations and outputs whose byte offsets pass 2^32."""
    E, N, K = 40, 8192, 16384                       # 5.4 GB of codes
    w = torch.zeros(E, N, K, dtype=torch.uint8, device="cuda")
    w[-1, -40:] = 0x38                              # 1.0
    ws = torch.ones(E, 64, 128, device="cuda")
    for path, T in ((ftq.PATH_GEMV, 3), (ftq.PATH_GROUPED, 270000)):
        say(f"[fp8] far offsets path={path} T={T}")
        a = torch.zeros(T, K, dtype=torch.uint8, device="cuda")
        a[-2:, 8] = 0x40                            # 2.0
        as_ = torch.ones(T, 128, device="cuda")
        ids = torch.full((T, 1), -1, dtype=torch.int32, device="cuda")
        ids[-2:] = E - 1
        out = torch.full((T, N), 5.0, dtype=torch.bfloat16, device="cuda")
        ftq.moe_fp8(w.view(ftq.FP8), ws, a.view(ftq.FP8), as_, ids, E, N, K, path=path, out=out)
        torch.cuda.synchronize()
        assert (out[-2:, -40:] == 2.0).all() and (out[-2:, :-40] == 0).all() and (out[:-2] == 0).all()
        del a, out


@pytest.mark.parametrize("E", [4095, 4094], ids=["by_pair", "by_expert"])
def test_gemv_of_more_workgroups_than_a_launch_takes(E):
    """4096 pairs times 2049 column tiles: more than 2^32 work-items."""
    T, N, K = 4096, 65568, 16
    say(f"[fp8] gemv work-items past 2^32 E={E}")
    w = torch.zeros(E, N, K, dtype=torch.uint8, device="cuda")
    a = torch.zeros(T, K, dtype=torch.uint8, device="cuda")
    w[:, :2] = w[:, -3:] = 0x38                     # 1.0
    a[:, 5] = 0x40                                  # 2.0
    ws, as_ = torch.ones(E, 513, 1, device="cuda"), torch.ones(T, 1, device="cuda")
    ids = torch.full((T, 1), -1, dtype=torch.int32, device="cuda")
    live = {0: 0, 2047: 17, 2048: 17, 3000: 2049, T - 1: E - 1}
    for p, e in live.items():
        ids[p] = e
    out = torch.full((T, N), 5.0, dtype=torch.bfloat16, device="cuda")
    ftq.moe_fp8(w.view(ftq.FP8), ws, a.view(ftq.FP8), as_, ids, E, N, K, path=ftq.PATH_GEMV, out=out)
    torch.cuda.synchronize()
    p = list(live)
    assert (out[p, :2] == 2.0).all() and (out[p, -3:] == 2.0).all() and (out[p, 2:-3] == 0).all()
    out[p] = 0
    assert (out == 0).all()


# ---- streams, graphs, the whole layer ----------------------------------------------

def _layer(x, logits, w13, s13, w2, s2, bias, k, E, N2, K, act, path, bufs=None):
    """Expert FFN of one layer: router, quantise, first layer, quantise, second layer, combine."""
    T = x.shape[0]
    ids, gates = ftq.moe_topk(logits, k, score=ftq.SCORE_SIGMOID, bias=bias, n_group=4, topk_group=2, group_top=2, scale=2.5)
    a, as_ = ftq.quantize_fp8(x)
    h = ftq.moe_fp8(w13, s13, a, as_, ids, E, 2 * N2, K, act=act, path=path, out_dtype=torch.bfloat16)
    q, qs = ftq.quantize_fp8(h)
    y = ftq.moe_fp8(w2, s2, q, qs, ids, E, K, N2, per_pair=True, path=path)
    return ids, gates, h, y, ftq.combine_topk(y, gates)


def _layer_inputs(T, E, N2, K, seed=0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, K, generator=g).bfloat16().cuda()
    logits = torch.randn(T, E, generator=g).cuda() * 2
    bias = torch.randn(E, generator=g).cuda() * 0.1
    w13, s13 = ftq.quantize_fp8_weight((torch.randn(E, 2 * N2, K, generator=g) * 0.05).bfloat16().cuda())
    w2, s2 = ftq.quantize_fp8_weight((torch.randn(E, K, N2, generator=g) * 0.05).bfloat16().cuda())
    return x, logits, w13, s13, w2, s2, bias


@pytest.mark.parametrize("T", [1, 13, 400])
@pytest.mark.parametrize("path", [ftq.PATH_AUTO, ftq.PATH_GEMV, ftq.PATH_GROUPED])
def test_expert_layer(T, path):
    """The operators as they are used together, each step against the definition on the step's own inputs."""
    E, N2, K, k = 16, 208, 400, 4
    x, logits, w13, s13, w2, s2, bias = _layer_inputs(T, E, N2, K, T)
    ids, gates, h, y, out = _layer(x, logits, w13, s13, w2, s2, bias, k, E, N2, K, ftq.ACT_SILU, path)
    from tests.test_gpu_topk import topk64
    ri, rg = topk64(logits.double().cpu().numpy(), bias.cpu().numpy(), k, "sigmoid", 4, 2, 2, True, 2.5)
    assert np.array_equal(ids.cpu().numpy(), ri)
    a, as_ = (torch.from_numpy(t).cuda() for t in _fp8.quantize_rows(x.float().cpu().numpy()))
    grouped = (path or ftq.fp8_select_path(E, 2 * N2, K, T, k)) == ftq.PATH_GROUPED
    assert_close(h, *moe64(w13, s13, a.view(ftq.FP8), as_, ids, False, "silu", grouped), "first layer")
    q, qs = (torch.from_numpy(t).cuda() for t in _fp8.quantize_rows(h.float().cpu().numpy()))
    assert_close(y, *moe64(w2, s2, q.view(ftq.FP8), qs, ids, True), "second layer")
    ref = (gates.double()[:, :, None] * y.double().view(T, k, K)).sum(1)
    mag = (gates.double()[:, :, None] * y.double().view(T, k, K)).abs().sum(1)
    assert ((out.double() - ref).abs() <= (k + 1) * 2.0 ** -24 * mag).all()
    assert np.allclose(gates.cpu().numpy(), rg, rtol=1e-5)


@pytest.mark.parametrize("T", [3, 200])
def test_expert_layer_in_a_graph(T):
    """Captured once, replayed with other inputs and eager work between the replays."""
    E, N2, K, k = 16, 128, 256, 4
    args = _layer_inputs(T, E, N2, K, 1)
    _layer(*args, k, E, N2, K, ftq.ACT_GELU_TANH, ftq.PATH_AUTO)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = _layer(*args, k, E, N2, K, ftq.ACT_GELU_TANH, ftq.PATH_AUTO)
    for seed in range(4):
        x, logits = _layer_inputs(T, E, N2, K, 10 + seed)[:2]
        args[0].copy_(x)
        args[1].copy_(logits)
        want = _layer(*args, k, E, N2, K, ftq.ACT_GELU_TANH, ftq.PATH_AUTO)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_two_streams_at_once():
    """Two layers at once on two streams, each with its own buffers."""
    cases = [Experts(8, 256, 512, 200, 2, seed=s) for s in (1, 2)]
    want = [c.run(ftq.PATH_GROUPED).clone() for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(3):
        got = [ftq.moe_fp8(c.w, c.ws, c.a, c.as_, c.ids, 8, 256, 512, path=ftq.PATH_GROUPED, stream=s) for c, s in zip(cases, streams)]
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_the_layer_on_another_stream():
    """Every call on a stream that is not the current one, or that was made current."""
    E, N2, K, k, T = 16, 128, 256, 4, 150
    args = _layer_inputs(T, E, N2, K, 5)
    want = _layer(*args, k, E, N2, K, ftq.ACT_SILU, ftq.PATH_AUTO)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        got = _layer(*args, k, E, N2, K, ftq.ACT_SILU, ftq.PATH_AUTO)
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    x, logits, w13, s13 = args[:4]
    ids, gates = ftq.moe_topk(logits, k, score=ftq.SCORE_SIGMOID, bias=args[6], n_group=4, topk_group=2, group_top=2, scale=2.5, stream=s)
    a, as_ = ftq.quantize_fp8(x, stream=s)
    h = ftq.moe_fp8(w13, s13, a, as_, ids, E, 2 * N2, K, act=ftq.ACT_SILU, out_dtype=torch.bfloat16, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(ids, want[0]) and torch.equal(gates, want[1]) and torch.equal(h, want[2])


def test_no_tokens():
    c = Experts(8, 64, 256, 4, 2)
    z = torch.zeros(0, 2, dtype=torch.int32, device="cuda")
    for path in (ftq.PATH_AUTO, ftq.PATH_GEMV, ftq.PATH_GROUPED):
        assert ftq.moe_fp8(c.w, c.ws, c.a[:0], c.as_[:0], z, 8, 64, 256, path=path).shape == (0, 64)
    assert ftq.quantize_fp8(torch.zeros(0, 256, device="cuda"))[1].shape == (0, 2)
    assert ftq.quantize_fp8_weight(torch.zeros(0, 4, 256, device="cuda"))[0].shape == (0, 4, 256)


def test_two_graphs_with_a_workspace_each():
    """Two captured matmuls replayed in turn, with other routings than the ones they were captured with."""
    cases = [Experts(8, 256, 384, 300, 2, seed=s) for s in (1, 2)]
    graphs, outs = [], []
    for c in cases:
        ws = torch.empty(ftq.fp8_workspace_bytes(8, 256, 384, 300, 2, ftq.PATH_GROUPED), dtype=torch.uint8, device="cuda")
        out = torch.empty(600, 256, device="cuda")
        call = lambda c=c, ws=ws, out=out: ftq.moe_fp8(c.w, c.ws, c.a, c.as_, c.ids, 8, 256, 384, path=ftq.PATH_GROUPED, out=out, workspace=ws)  # noqa: E731
        call()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call()
        graphs.append((g, ws))
        outs.append(out)
    for seed in range(4):
        want = []
        for i, c in enumerate(cases):
            c.ids.copy_(torch.from_numpy(inputs.routing(300, 8, 2, seed=10 * seed + i, kind="zipf")))
            want.append(c.run(ftq.PATH_GROUPED))
        for g, _ in graphs:
            g.replay()
        torch.cuda.synchronize()
        for a, b in zip(outs, want):
            assert torch.equal(a, b)


def test_binding_refuses():
    c = Experts(8, 64, 256, 4, 2)
    call = lambda **kw: ftq.moe_fp8(**{**dict(w=c.w, w_scale=c.ws, a=c.a, a_scale=c.as_, topk_ids=c.ids, E=8, N=64, K=256), **kw})  # noqa: E731
    for kw in (dict(w=c.w[:7]), dict(w_scale=c.ws[:, :0]), dict(a=c.a[:3]), dict(a_scale=c.as_[:, :1]), dict(per_pair=True), dict(topk_ids=c.ids.long()),
               dict(out=torch.empty(8, 63, device="cuda")), dict(out=torch.empty(8, 64, device="cuda", dtype=torch.float64)),
               dict(w=c.w.view(torch.uint8)), dict(a=c.a.float()), dict(w=c.w.cpu())):
        with pytest.raises(ValueError):
            call(**kw)
    with pytest.raises(ftq.FtqError):
        call(path=9)
    with pytest.raises(ValueError):
        ftq.quantize_fp8(torch.zeros(4, 4, 128, device="cuda"))
    with pytest.raises(ftq.FtqError):
        ftq.quantize_fp8(torch.zeros(4, 24, device="cuda"))
