"""Low-rank adapters and their gradients against definitions in 64 bits and against
differences: ids that name no adapter, tiles that many adapters share, ranks and
lengths that end inside a tile, strides, types, paths."""
import pytest
import torch

from quantized_moe_expert_quantize_amd import ftq
from tests import _train as t

pytestmark = pytest.mark.gpu
PATHS = [ftq.PATH_GEMV, ftq.PATH_GROUPED]


def make(L, R, K, N, T, k, dtype, out, seed=0, per_pair=False, runs=None, none=0.1, base=True):
    """Inputs on the GPU; runs: rows of an adapter lie together in about so many runs (None: at random)."""
    g = torch.Generator().manual_seed(seed + 7 * K + 13 * N + R)
    dt = t.DTYPES[dtype]
    rows = T * k if per_pair else T
    c = dict(x=torch.randn(rows, K, generator=g).to(dt), a=(torch.randn(L, R, K, generator=g) / K ** 0.5).to(dt),
             b=(torch.randn(L, N, R, generator=g) / R ** 0.5).to(dt), scale=torch.rand(L, generator=g) + 0.5)
    if runs:
        request = torch.sort(torch.randint(0, runs, (T,), generator=g)).values
        ids = torch.randint(0, L, (runs,), generator=g)[request].view(T, 1).repeat(1, k)
    else:
        ids = torch.randint(0, L, (T, k), generator=g)
    drop = torch.rand(T, k, generator=g)
    ids[drop < none] = -1
    ids[drop < none / 3] = L                                   # out of range on the other side
    c["ids"] = ids.to(torch.int32)
    c["base"] = torch.randn(T * k, N, generator=g).to(t.DTYPES[out]) if base else None
    c["dy"] = torch.randn(T * k, N, generator=g).to(dt)
    return {n: v.cuda() if v is not None else None for n, v in c.items()}


def forward(c, out, path, per_pair=False, **kw):
    pairs, R = c["ids"].numel(), c["a"].shape[1]
    h = torch.full((pairs, R), float("nan"), device="cuda")
    y = ftq.lora(c["x"], c["a"], c["b"], c["ids"], scale=c["scale"], base=c["base"], per_pair=per_pair, path=path,
                 out_dtype=t.DTYPES[out], h=h, **kw)
    return y, h


def check_forward(c, out, path, per_pair=False):
    y, h = forward(c, out, path, per_pair)
    assert y.dtype == t.DTYPES[out]
    ro, rh, mo, mh = t.lora_forward(c["x"], c["a"], c["b"], c["ids"], c["scale"], c["base"], per_pair)
    L, R, K = c["a"].shape
    t.close(h, rh, mh, K + 4, "h")
    t.close(y, ro, mo, K + R + 8, "out")
    return y, h


CASES = [
    # L, R, K, N, T, top_k, per_pair, runs
    (1, 8, 8, 8, 1, 1, False, None), (3, 8, 64, 72, 5, 1, False, None), (8, 16, 512, 256, 16, 1, False, None), (2, 16, 520, 264, 1, 1, False, None),
    (5, 24, 200, 328, 63, 1, False, 4), (4, 32, 1000, 520, 200, 1, False, 6), (2, 64, 256, 640, 129, 1, False, 2), (3, 128, 328, 1032, 70, 1, False, 3),
    (3, 120, 136, 136, 37, 1, False, None), (12, 16, 264, 136, 90, 4, False, None), (40, 8, 136, 264, 70, 6, True, None), (100, 40, 72, 200, 33, 8, False, None),
]


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("dtype,out", [("f32", "f32"), ("bf16", "bf16"), ("f16", "f16"), ("bf16", "f32"), ("f16", "f32"), ("f32", "bf16"), ("bf16", "f16")])
@pytest.mark.parametrize("L,R,K,N,T,k,per_pair,runs", CASES)
def test_forward(L, R, K, N, T, k, per_pair, runs, dtype, out, path):
    print(f"[lora] L={L} R={R} K={K} N={N} T={T} k={k} per_pair={per_pair} runs={runs} {dtype}->{out} path={path}", flush=True)
    c = make(L, R, K, N, T, k, dtype, out, per_pair=per_pair, runs=runs)
    check_forward(c, out, path, per_pair)


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_forward_of_long_rows(dtype, path):
    c = make(6, 16, 4104, 3000, 150, 1, dtype, dtype, runs=9)
    check_forward(c, dtype, path)


@pytest.mark.parametrize("path", PATHS)
def test_forward_in_place_without_base_and_strided(path):
    c = make(4, 16, 264, 136, 77, 1, "bf16", "bf16", runs=6)
    want, h = check_forward(c, "bf16", path)
    wide = torch.full((77, 400), 3.0, dtype=torch.bfloat16, device="cuda")
    wide[:, 128:264] = c["base"]
    xs = torch.zeros(77, 512, dtype=torch.bfloat16, device="cuda")
    xs[:, 64:328] = c["x"]
    got = ftq.lora(xs[:, 64:328], c["a"], c["b"], c["ids"], scale=c["scale"], base=wide[:, 128:264], out=wide[:, 128:264], path=path)
    assert torch.equal(got, want) and (wide[:, :128] == 3).all() and (wide[:, 264:] == 3).all()
    c["base"] = None
    check_forward(c, "f32", path)
    c["scale"] = None
    check_forward(c, "f32", path)
    c["ids"].fill_(-1)
    y, h = forward(c, "f32", path)
    assert not y.any() and not h.any()


def test_in_place_with_another_stride_is_refused():
    """out at base's address with a stride of its own would be another tensor than base."""
    x, a, b, ids = torch.ones(4, 8).cuda(), torch.ones(1, 8, 8).cuda(), torch.ones(1, 8, 8).cuda(), torch.zeros(4, 1, dtype=torch.int32).cuda()
    buf = torch.full((4, 16), 2.0).cuda()
    with pytest.raises(ftq.FtqError):
        ftq.lora(x, a, b, ids, base=buf[:, :8], out=buf.view(8, 8)[:4])
    assert (buf == 2.0).all()
    ftq.lora(x[:1], a, b, ids[:1], base=buf[:1, :8], out=buf.view(8, 8)[:1])   # one row: the same tensor
    assert (buf[0, :8] == 66.0).all() and (buf[0, 8:] == 2.0).all()


def test_an_out_dtype_that_base_or_out_has_not_is_refused():
    x, a, b, ids = (torch.ones(4, 8).bfloat16().cuda(), torch.ones(1, 8, 8).bfloat16().cuda(), torch.ones(1, 8, 8).bfloat16().cuda(),
                    torch.zeros(4, 1, dtype=torch.int32).cuda())
    base = torch.ones(4, 8).bfloat16().cuda()
    for kw in (dict(base=base), dict(out=base.clone()), dict(base=base, out=base)):
        with pytest.raises(ValueError):
            ftq.lora(x, a, b, ids, out_dtype=torch.float32, **kw)
        assert ftq.lora(x, a, b, ids, out_dtype=torch.bfloat16, **kw).dtype == torch.bfloat16
    assert ftq.lora(x, a, b, ids, out_dtype=torch.float32).dtype == torch.float32 and ftq.lora(x, a, b, ids).dtype == torch.bfloat16


@pytest.mark.parametrize("path", PATHS)
def test_rows_depend_on_their_own_inputs_alone(path):
    """NaN and infinities of one adapter or row stay with the pairs that use them; a pair alone has the same bits."""
    c = make(5, 16, 520, 264, 61, 1, "bf16", "f32", none=0.1)
    want, h = forward(c, "f32", path)
    dirty = {n: v.clone() for n, v in c.items()}
    dirty["a"][2, 3, 7] = float("nan")
    dirty["b"][3, 5] = float("inf")
    row = int((c["ids"][:, 0] == 1).nonzero()[0])
    dirty["x"][row, 11] = float("inf")
    got, hd = forward(dirty, "f32", path)
    ids = c["ids"][:, 0]
    clean = (ids != 2) & (ids != 3)
    clean[row] = False
    assert torch.equal(got[clean], want[clean]) and torch.equal(hd[clean], h[clean])
    assert hd[ids == 2][:, 3].isnan().all() and got[ids == 2].isnan().all()
    three = got[ids == 3]
    assert not three[:, 5].isfinite().any() and torch.equal(three[:, :5], want[ids == 3][:, :5])
    assert not hd[row].isfinite().any()


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_both_paths_have_the_same_bits(dtype):
    for L, R, K, N, T, k, per_pair, runs in CASES:
        c = make(L, R, K, N, T, k, dtype, "f32", per_pair=per_pair, runs=runs)
        a, b = (forward(c, "f32", p, per_pair) for p in PATHS)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]), (L, R, K, N, T, k)


def test_magnitudes_of_h():
    """h far from 1 in both directions: its pieces keep their bits."""
    for dtype, size in (("bf16", 1e20), ("bf16", 1e-20), ("f16", 300.0), ("f16", 1e-4), ("f32", 1e15)):
        c = make(3, 16, 264, 136, 40, 1, dtype, "f32", none=0.0, base=False)
        c["x"] = (c["x"].float() * size).to(t.DTYPES[dtype])
        c["b"] = (c["b"].float() / min(size, 1e4) if size > 1 else c["b"].float()).to(t.DTYPES[dtype])
        for path in PATHS:
            check_forward(c, "f32", path)
    # a row whose h differ by far in size
    c = make(1, 16, 264, 136, 20, 1, "f16", "f32", none=0.0, base=False)
    c["a"][0, :8] *= 1e-3
    c["x"] = (c["x"].float() * 100).half()
    check_forward(c, "f32", ftq.PATH_GEMV)


# ---- gradients --------------------------------------------------------------------------

def backward(c, h, per_pair=False, base=None, **kw):
    return dict(zip(("d_x", "d_a", "d_b"), ftq.lora_backward(c["dy"], c["x"], c["a"], c["b"], c["ids"], h, scale=c["scale"], base=base,
                                                             per_pair=per_pair, **kw)))


def check_backward(c, per_pair=False, base=None):
    L, R, K = c["a"].shape
    N, (T, k) = c["b"].shape[1], c["ids"].shape
    h = t.lora_forward(c["x"], c["a"], c["b"], c["ids"], c["scale"], None, per_pair)[1].float().cuda()
    got = backward(c, h, per_pair, base)
    ref = t.lora_backward(c["dy"], c["x"], c["a"], c["b"], c["ids"], h, c["scale"], base, per_pair)
    flat = c["ids"].reshape(-1)
    most = int(torch.bincount(flat[(flat >= 0) & (flat < L)].long(), minlength=1).max()) if flat.numel() else 0
    terms = {"d_x": N + k * R + 10, "d_a": N + most + 10, "d_b": most + 10}
    for n, v in got.items():
        t.close(v, *ref[n], terms[n], n)
    return got


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("L,R,K,N,T,k,per_pair,runs", CASES)
def test_backward(L, R, K, N, T, k, per_pair, runs, dtype):
    print(f"[lora_backward] L={L} R={R} K={K} N={N} T={T} k={k} per_pair={per_pair} runs={runs} {dtype}", flush=True)
    c = make(L, R, K, N, T, k, dtype, "f32", per_pair=per_pair, runs=runs)
    got = check_backward(c, per_pair)
    used = set(c["ids"].reshape(-1).tolist())
    for l in range(L):
        if l not in used:
            assert not got["d_a"][l].any() and not got["d_b"][l].any()


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_backward_of_many_rows(dtype):
    c = make(3, 16, 136, 264, 2500, 1, dtype, "f32", runs=4)
    check_backward(c)
    c = make(1, 64, 264, 136, 1500, 1, dtype, "f32", none=0.0)
    check_backward(c)


@pytest.mark.parametrize("dtype,R", [("bf16", 8), ("f16", 16), ("f32", 8), ("bf16", 128), ("f16", 64)])
def test_backward_of_long_runs(dtype, R):
    """Runs of more than 32 tiles of 32 pairs, whose rows are listed 32 tiles at a time, with data in all of them: an adapter that ends inside a
    list, one that ends with it, one over several lists and runs, one pair, none."""
    K = N = 2048
    counts = [20 * 32 + 5, 11 * 32, 500 * 32 + 7, 0, 1, 32 * 32, 44000]
    T, L, g = sum(counts), len(counts), torch.Generator().manual_seed(R)
    item = 512 // (4 if dtype == "f32" else 2)
    assert (T // 32) * (K // item + N // item) > 33 * 512      # the workgroups that share the tiles: longer than 32 each
    dt = t.DTYPES[dtype]
    ids = torch.repeat_interleave(torch.arange(L), torch.tensor(counts))[torch.randperm(T, generator=g)].to(torch.int32).cuda()
    torch.manual_seed(R)
    x, dy, h = torch.randn(T, K, device="cuda").to(dt), torch.randn(T, N, device="cuda").to(dt), torch.randn(T, R, device="cuda")
    a, b, scale = (torch.randn(L, R, K, device="cuda") / 45).to(dt), (torch.randn(L, N, R, device="cuda") / 45).to(dt), torch.rand(L, device="cuda") + 0.5
    _, d_a, d_b = ftq.lora_backward(dy, x, a, b, ids.view(T, 1), h, scale=scale)
    for l, n in enumerate(counts):
        p = (ids == l).nonzero()[:, 0]
        xl, dl, hl, s = x[p].double(), dy[p].double(), h[p].double(), float(scale[l])
        gl, ml = s * (dl @ b[l].double()), s * (dl.abs() @ b[l].double().abs())
        t.close(d_a[l], gl.t().contiguous() @ xl, ml.t().contiguous() @ xl.abs(), N + n + 10, f"d_a of {n} pairs")
        t.close(d_b[l], s * (dl.t().contiguous() @ hl), s * (dl.abs().t().contiguous() @ hl.abs()), n + 10, f"d_b of {n} pairs")


@pytest.mark.parametrize("per_pair", [False, True])
def test_backward_base_strides_and_parts(per_pair):
    k = 3
    c = make(6, 16, 264, 136, 50, k, "bf16", "f32", per_pair=per_pair)
    base = torch.randn(c["x"].shape, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    want = check_backward(c, per_pair, base)
    h = t.lora_forward(c["x"], c["a"], c["b"], c["ids"], c["scale"], None, per_pair)[1].float().cuda()
    wide_dy = torch.zeros(150, 200, dtype=torch.bfloat16, device="cuda")
    wide_dy[:, 32:168] = c["dy"]
    wide_x = torch.zeros(c["x"].shape[0], 400, dtype=torch.bfloat16, device="cuda")
    wide_x[:, 8:272] = c["x"]
    keep = base.clone()
    got = ftq.lora_backward(wide_dy[:, 32:168], wide_x[:, 8:272], c["a"], c["b"], c["ids"], h, scale=c["scale"], base=keep, d_x=keep, per_pair=per_pair)
    assert all(torch.equal(p, q) for p, q in zip(got, want.values()))
    # each gradient by itself, without what it does not need
    L, R, K = c["a"].shape
    N, T = 136, 50
    P = lambda v: v.data_ptr() if v is not None else None  # noqa: E731
    need = ftq.lora_backward_workspace_bytes(L, R, K, N, T, k, torch.bfloat16)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    for name, (x, a, b, hh, bs) in dict(d_x=(None, c["a"], c["b"], None, base), d_a=(c["x"], None, c["b"], None, None),
                                        d_b=(None, None, None, h, None)).items():
        out = {n: torch.empty_like(v) if n == name else None for n, v in want.items()}
        st = ftq.lib().ftq_lora_backward(P(c["dy"]), N, P(x), K, P(a), P(b), P(c["scale"]), P(c["ids"]), P(hh), P(bs), P(out["d_x"]), P(out["d_a"]),
                                         P(out["d_b"]), ftq.BF16, L, R, K, N, T, k, int(per_pair), P(ws), need, None)
        assert st == ftq.OK, ftq.last_error()
        torch.cuda.synchronize()
        assert torch.equal(out[name], want[name]), name


def test_backward_of_nothing():
    c = make(4, 8, 64, 72, 3, 2, "f32", "f32")
    got = ftq.lora_backward(c["dy"][:0], c["x"][:0], c["a"], c["b"], c["ids"][:0], torch.empty(0, 8, device="cuda"))
    assert got[0].shape == (0, 64) and not got[1].any() and not got[2].any()
    c["ids"].fill_(-1)
    got = check_backward(c)
    assert not any(v.any() for v in got.values())


def test_backward_keeps_rows_apart():
    """NaN of one row or adapter reaches only what it is a term of."""
    c = make(5, 16, 264, 136, 61, 1, "bf16", "f32", none=0.1)
    h = t.lora_forward(c["x"], c["a"], c["b"], c["ids"], c["scale"], None, False)[1].float().cuda()
    want = backward(c, h)
    ids = c["ids"][:, 0]
    dirty = {n: v.clone() if v is not None else None for n, v in c.items()}
    dirty["a"][2, 3, 7] = float("nan")
    row = int((ids == 1).nonzero()[0])
    dirty["x"][row, 11] = float("nan")
    none = int(((ids < 0) | (ids >= 5)).nonzero()[0])
    dirty["x"][none] = float("nan")
    dirty["dy"][none] = float("inf")
    hd = h.clone()
    hd[none] = float("nan")
    got = backward(dirty, hd)
    other = ids != 2
    assert torch.equal(got["d_x"][other], want["d_x"][other]) and got["d_x"][~other][:, 7].isnan().all()
    assert torch.equal(got["d_x"][~other][:, :7], want["d_x"][~other][:, :7])
    assert torch.equal(got["d_a"][[0, 2, 3, 4]], want["d_a"][[0, 2, 3, 4]]) and got["d_a"][1][:, 11].isnan().all()
    assert torch.equal(got["d_a"][1][:, :11], want["d_a"][1][:, :11]) and torch.equal(got["d_b"], want["d_b"])


@pytest.mark.parametrize("per_pair", [False, True])
def test_backward_against_differences(per_pair):
    c = make(3, 8, 24, 40, 20, 2, "f32", "f32", per_pair=per_pair, base=False)
    _, h = forward(c, "f32", ftq.PATH_AUTO, per_pair)
    got = backward(c, h, per_pair)
    dy, g = c["dy"].cpu().double(), torch.Generator().manual_seed(1)

    def value(x, a, b):
        return float((t.lora_forward(x, a, b, c["ids"].cpu(), c["scale"].cpu(), None, per_pair)[0] * dy).sum())
    at = [c[n].cpu().double() for n in ("x", "a", "b")]
    for i, n in enumerate(("d_x", "d_a", "d_b")):              # linear in each: differences are exact but for roundings
        v = torch.randn(at[i].shape, generator=g).double()
        up, down = ([w + s * v if j == i else w for j, w in enumerate(at)] for s in (1, -1))
        want = (value(*up) - value(*down)) / 2
        terms = got[n].cpu().double() * v
        assert abs(want - float(terms.sum())) <= 1e-5 * float(terms.abs().sum()), n


# ranks (or pairs) in four classes of far different size; values of 16 bits hold 2^-24 beside 1 only with fewer bits, so that
# those of a, b and x are a factor of 2^24 apart at most and fp32's h further
FAR = (2.0 ** 12, 2.0 ** 4, 2.0 ** -4, 2.0 ** -12)
FAR_H = (1.0, 2.0 ** -20, 2.0 ** -24, 2.0 ** -30)


def by_class(n, factors):
    return torch.tensor([factors[i % 4] for i in range(n)], device="cuda")


def apart(n, m):
    """[n, m] of ones where both indices are of one class, else zeros."""
    return (torch.arange(n, device="cuda")[:, None] % 4 == torch.arange(m, device="cuda")[None] % 4).float()


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_results_of_ranks_of_far_different_size(dtype, path):
    """A result owes nothing to the ranks that its own weights leave out, however large their values in h."""
    for R in (8, 32, 64, 128):
        c = make(2, R, 136, 264, 70, 1, dtype, "f32", none=0.1, base=False)
        c["a"] = (c["a"].float() * by_class(R, FAR)[:, None]).to(t.DTYPES[dtype])
        c["b"] = (c["b"].float() * apart(264, R)).to(t.DTYPES[dtype])
        y, h = forward(c, "f32", path)
        ro, rh, mo, mh = t.lora_forward(c["x"], c["a"], c["b"], c["ids"], c["scale"], None, False)
        for q in range(4):
            t.close(h[:, q::4], rh[:, q::4], mh[:, q::4], 136 + 4, f"h of class {q}")
            t.close(y[:, q::4], ro[:, q::4], mo[:, q::4], 136 + R + 8, f"out of class {q}")


def backward_by_class(c, h, ways, per_pair=False):
    """Gradients compared class by class, where ways[name] is the dimension that the classes lie along."""
    K, N, most = c["a"].shape[2], c["b"].shape[1], c["ids"].numel()
    got = backward(c, h, per_pair)
    ref = t.lora_backward(c["dy"], c["x"], c["a"], c["b"], c["ids"], h, c["scale"], None, per_pair)
    terms = {"d_x": N + c["ids"].shape[1] * c["a"].shape[1] + 10, "d_a": N + most + 10, "d_b": most + 10}
    for n, dim in ways.items():
        for q in range(4):
            at = [slice(None)] * ref[n][0].dim()
            at[dim] = slice(q, None, 4)
            at = tuple(at)
            t.close(got[n][at], ref[n][0][at], ref[n][1][at], terms[n], f"{n} of class {q}")


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("R", [8, 24, 64, 128])
def test_gradients_of_ranks_of_far_different_size(R, dtype):
    """A rank's gradient is a sum of its own values of g or h: however small beside the other ranks', they keep fp32's bits."""
    c = make(2, R, 136, 264, 90, 1, dtype, "f32", none=0.1)
    c["b"] = (c["b"].float() * by_class(R, FAR)).to(t.DTYPES[dtype])
    c["a"] = (c["a"].float() * apart(R, 136)).to(t.DTYPES[dtype])
    h = torch.randn(90, R, generator=torch.Generator().manual_seed(R)).cuda() * by_class(R, FAR_H)
    backward_by_class(c, h, {"d_x": 1, "d_a": 1, "d_b": 2})


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_gradients_of_pairs_of_far_different_size(dtype):
    """The columns that only small pairs reach, beside large pairs of the same adapter."""
    c = make(1, 16, 136, 264, 90, 1, dtype, "f32", none=0.0)
    c["dy"] = (c["dy"].float() * by_class(90, FAR)[:, None]).to(t.DTYPES[dtype])
    c["x"] = (c["x"].float() * apart(90, 136)).to(t.DTYPES[dtype])
    h = torch.randn(90, 16, generator=torch.Generator().manual_seed(1)).cuda()
    backward_by_class(c, h, {"d_a": 2})
    c = make(1, 16, 136, 264, 90, 1, dtype, "f32", none=0.0)
    c["dy"] = (c["dy"].float() * apart(90, 264)).to(t.DTYPES[dtype])
    backward_by_class(c, h * by_class(90, FAR_H)[:, None], {"d_b": 1})


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_infinity_of_one_rank_stays_in_it(dtype):
    c = make(3, 16, 136, 264, 61, 1, dtype, "f32", none=0.1)
    h = torch.randn(61, 16, generator=torch.Generator().manual_seed(1)).cuda() * by_class(16, (1e5, 1.0, 1e-3, 1e-6))
    want = backward(c, h)
    dirty, hd = {n: v.clone() for n, v in c.items()}, h.clone()
    hd[int((c["ids"][:, 0] == 1).nonzero()[0]), 5] = float("inf")
    dirty["b"][1, 7, 3] = float("inf")
    got = backward(dirty, hd)
    ranks = torch.arange(16, device="cuda")
    assert not got["d_b"][1][:, 5].isfinite().any() and torch.equal(got["d_b"][1][:, ranks != 5], want["d_b"][1][:, ranks != 5])
    assert not got["d_a"][1][3].isfinite().any() and torch.equal(got["d_a"][1][ranks != 3], want["d_a"][1][ranks != 3])
    assert torch.equal(got["d_a"][[0, 2]], want["d_a"][[0, 2]]) and torch.equal(got["d_b"][[0, 2]], want["d_b"][[0, 2]])


@pytest.mark.parametrize("size", [3.4e38, 2.0 ** -100])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_r_vectors_at_the_ends_of_32_bits(dtype, size):
    c = make(2, 8, 64, 72, 40, 1, dtype, "f32", none=0.1)
    c["dy"] = (c["dy"].float() * 2.0 ** -12).to(t.DTYPES[dtype])
    h = size * (0.5 + 0.5 * torch.rand(40, 8, generator=torch.Generator().manual_seed(1))).cuda()
    got = backward(c, h)["d_b"]
    assert got.isfinite().all()
    ref, mag = t.lora_backward(c["dy"], c["x"], c["a"], c["b"], c["ids"], h, c["scale"], None, False)["d_b"]
    t.close(got, ref, mag, 40 + 10, "d_b")


def test_same_bits_again():
    c = make(3, 16, 264, 136, 700, 2, "bf16", "f32")
    first, h = forward(c, "f32", ftq.PATH_AUTO)
    grads = backward(c, h)
    for _ in range(3):
        y, h2 = forward(c, "f32", ftq.PATH_AUTO)
        assert torch.equal(y, first) and torch.equal(h, h2)
        assert all(torch.equal(v, grads[n]) for n, v in backward(c, h).items())


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("L,T,k", [(4095, 300, 8), (4095, 7, 1), (2048, 2000, 2)])
def test_as_many_adapters_as_a_sort_takes(L, T, k, dtype):
    c = make(L, 8, 64, 72, T, k, dtype, "f32", per_pair=k > 1)
    c["ids"][0, 0], c["ids"][-1, 0], c["ids"][T // 2, 0] = L - 1, 2 ** 31 - 1, -2 ** 31
    a, b = (check_forward(c, "f32", p, k > 1) for p in PATHS)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    check_backward(c, k > 1)


def test_offsets_past_32_bits():
    """Rows of x and out, and adapters, whose byte and element offsets pass 2^31 and 2^32."""
    L, R, K, N, T = 2, 8, 65536, 8, 33000                      # x: 2.16e9 elements
    x = torch.zeros(T, K, dtype=torch.bfloat16, device="cuda")
    x[-40:] = torch.randn(40, K, device="cuda").bfloat16()
    a, b = (torch.randn(L, R, K, device="cuda") / 256).bfloat16(), torch.randn(L, N, R, device="cuda").bfloat16()
    ids = (torch.arange(T, device="cuda") % L).to(torch.int32).view(T, 1)
    for path in PATHS:
        out = ftq.lora(x, a, b, ids, path=path, out_dtype=torch.float32)
        small = ftq.lora(x[-40:], a, b, ids[-40:], path=path, out_dtype=torch.float32)
        assert not out[:-40].any()
        ref, _, mag, _ = t.lora_forward(x[-40:], a, b, ids[-40:], None, None, False)
        t.close(out[-40:], ref, mag, K + R + 8)
        t.close(small, ref, mag, K + R + 8)
    g = ftq.lora_backward(torch.ones(T, N, dtype=torch.bfloat16, device="cuda"), x, a, b, ids, torch.zeros(T, R, device="cuda"))
    tail = ftq.lora_backward(torch.ones(40, N, dtype=torch.bfloat16, device="cuda"), x[-40:], a, b, ids[-40:], torch.zeros(40, R, device="cuda"))
    assert torch.equal(g[0][-40:], tail[0])
    ref = t.lora_backward(torch.ones(40, N), x[-40:], a, b, ids[-40:], torch.zeros(40, R), None, None, False)["d_a"]
    t.close(g[1], *ref, T + N + 10, "d_a")
    del x, g
    L, R, K, N = 4100, 64, 16384, 8                            # a: 4.3e9 elements, more adapters than a sort takes
    a = torch.zeros(L, R, K, dtype=torch.float16, device="cuda")
    a[-1] = torch.randn(R, K, device="cuda") / 128
    b = torch.randn(L, N, R, device="cuda").half()
    x = torch.randn(3, K, device="cuda").half()
    ids = torch.tensor([[L - 1], [0], [L]], dtype=torch.int32, device="cuda")
    out = ftq.lora(x, a, b, ids, out_dtype=torch.float32)
    assert not out[1:].any()
    ref, _, mag, _ = t.lora_forward(x[:1], a[-1:], b[-1:], torch.zeros(1, 1, dtype=torch.int32), None, None, False)
    t.close(out[:1], ref, mag, K + R + 8)


def test_wide_rows_past_32_bits():
    """Results, their base and gradients of more than 2^31 elements and 2^32 bytes."""
    L, R, K, N, T = 2, 8, 8, 65536, 33000
    x, a, b = torch.randn(T, K, device="cuda").bfloat16(), torch.randn(L, R, K, device="cuda").bfloat16(), torch.randn(L, N, R, device="cuda").bfloat16()
    ids = (torch.arange(T, device="cuda") % L).to(torch.int32).view(T, 1)
    for path in PATHS:
        out = torch.ones(T, N, dtype=torch.bfloat16, device="cuda")
        h = torch.empty(T, R, device="cuda")
        ftq.lora(x, a, b, ids, base=out, out=out, h=h, path=path)
        few = ftq.lora(x[-40:], a, b, ids[-40:], base=torch.ones(40, N, dtype=torch.bfloat16, device="cuda"), path=path)
        assert torch.equal(out[-40:], few)
    out.zero_()
    out[-40:] = torch.randn(40, N, device="cuda")              # now the gradient
    _, d_a, d_b = ftq.lora_backward(out, x, a, b, ids, h)
    ref = t.lora_backward(out[-40:], x[-40:], a, b, ids[-40:], h[-40:], None, None, False)
    t.close(d_a, *ref["d_a"], N + T + 10, "d_a")
    t.close(d_b, *ref["d_b"], T + 10, "d_b")
