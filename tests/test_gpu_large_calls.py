"""Calls of more workgroups than one launch takes: sequences, pairs and rows up to
the documented limits.  Most rows are zeros, so that what the others give can be told
from a call on those alone."""
import pytest
import torch

from quantized_moe_expert_quantize_amd import ftq
from tests import _train as t

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def memory():
    torch.cuda.empty_cache()
    yield
    torch.cuda.empty_cache()


def spread(n, more=2000):
    """Ascending indices below n: the first ones, the last ones and some between."""
    g = torch.Generator().manual_seed(n)
    at = torch.cat([torch.arange(40), torch.randint(0, n, (more,), generator=g), torch.arange(n - 40, n)])
    return torch.unique(at).cuda()


def nonzero_rows(v, step=1 << 26):
    return sum(int((part != 0).any(1).sum()) for part in v.split(step))


def adapters(L, R, K, N, pairs):
    g = torch.Generator().manual_seed(1)
    at = spread(pairs)
    a, b = torch.randn(L, R, K, generator=g).half().cuda(), torch.randn(L, N, R, generator=g).half().cuda()
    ids = torch.randint(-1, L, (len(at), 1), generator=g).to(torch.int32).cuda()
    all_ids = (torch.arange(pairs, dtype=torch.int32, device="cuda") % L).view(pairs, 1)
    all_ids[at] = ids
    return g, at, a, b, ids, all_ids


def scattered(pairs, columns, at, rows):
    v = torch.zeros(pairs, columns, dtype=rows.dtype, device="cuda")
    v[at] = rows
    return v


@pytest.mark.parametrize("path", [ftq.PATH_GEMV, ftq.PATH_GROUPED])
def test_adapters_of_a_thousand_million_pairs(path):
    L, R, K, N, pairs = 3, 8, 8, 8, (1 << 30) + 5000
    print(f"[lora] pairs={pairs} path={path}", flush=True)
    g, at, a, b, ids, all_ids = adapters(L, R, K, N, pairs)
    few = torch.randn(len(at), K, generator=g).half().cuda()
    x = scattered(pairs, K, at, few)
    out = ftq.lora(x, a, b, all_ids, path=path)
    want = ftq.lora(few, a, b, ids, path=path)
    assert torch.equal(out[at], want) and nonzero_rows(out) == nonzero_rows(want)


def test_gradients_of_hundreds_of_millions_of_pairs():
    L, R, K, N, pairs = 3, 8, 8, 8, (1 << 28) + 5000
    print(f"[lora_backward] pairs={pairs}", flush=True)
    g, at, a, b, ids, all_ids = adapters(L, R, K, N, pairs)
    dy, x = (torch.randn(len(at), c, generator=g).half().cuda() for c in (N, K))
    h = torch.randn(len(at), R, generator=g).cuda()
    d_x, d_a, d_b = ftq.lora_backward(scattered(pairs, N, at, dy), scattered(pairs, K, at, x), a, b, all_ids, scattered(pairs, R, at, h))
    want = ftq.lora_backward(dy, x, a, b, ids, h)
    assert torch.equal(d_x[at], want[0]) and nonzero_rows(d_x) == nonzero_rows(want[0])
    ref = t.lora_backward(dy, x, a, b, ids, h, None, None, False)
    t.close(d_a, *ref["d_a"], N + len(at) + 10, "d_a")
    t.close(d_b, *ref["d_b"], len(at) + 10, "d_b")


def test_gradients_of_rows_that_pairs_share():
    """d_x alone, of 64 slices of columns and more than 2^20 tokens."""
    L, R, K, N, T, k = 2, 8, 32768, 8, (1 << 20) + 300, 2
    print(f"[lora_backward] T={T} K={K}", flush=True)
    g = torch.Generator().manual_seed(1)
    at = spread(T)
    a, b = (torch.randn(L, R, K, generator=g) / 8).bfloat16().cuda(), torch.randn(L, N, R, generator=g).bfloat16().cuda()
    ids = torch.randint(-1, L, (T, k), generator=g).to(torch.int32).cuda()
    few_ids = ids[at].contiguous()
    few = torch.randn(len(at), k, N, generator=g).bfloat16().cuda()
    dy = torch.zeros(T, k, N, dtype=torch.bfloat16, device="cuda")
    dy[at] = few

    def call(dy, ids):
        T = len(ids)
        d_x = torch.full((T, K), float("nan"), dtype=torch.bfloat16, device="cuda")
        need = ftq.lora_backward_workspace_bytes(L, R, K, N, T, k, torch.bfloat16)
        ws = torch.empty(need, dtype=torch.uint8, device="cuda")
        st = ftq.lib().ftq_lora_backward(dy.data_ptr(), N, None, K, a.data_ptr(), b.data_ptr(), None, ids.data_ptr(), None, None, d_x.data_ptr(),
                                         None, None, ftq.BF16, L, R, K, N, T, k, 0, ws.data_ptr(), need, None)
        assert st == ftq.OK, ftq.last_error()
        torch.cuda.synchronize()
        return d_x
    want, got = call(few, few_ids), call(dy, ids)
    assert torch.equal(got[at], want) and nonzero_rows(got, 1 << 17) == nonzero_rows(want)


@pytest.mark.parametrize("T", [40, 3000])
def test_millions_of_sequences(T):
    S, E, k = (1 << 22) + 500, 3, 2
    print(f"[balance] T={T} S={S}", flush=True)
    g = torch.Generator().manual_seed(T)
    logits, ids = torch.randn(T, E, generator=g), torch.randint(0, E, (T, k), generator=g).to(torch.int32)
    cuts = torch.sort(torch.randint(0, T, (S + 1,), generator=g)).values.to(torch.int32)
    cuts[0], cuts[-300:] = 0, T - 1                            # sequences of the last launch are empty but for one row, the last one's
    cuts[-1] = T
    loss, counts, tokens = ftq.moe_balance(logits.cuda(), ids.cuda(), offsets=cuts.cuda())
    used = torch.unique(torch.searchsorted(cuts[1:].contiguous(), torch.arange(T, dtype=torch.int32), right=True))
    few = torch.cat([cuts[used], cuts[-1:]])                   # the same rows in the sequences that hold any
    want = ftq.moe_balance(logits.cuda(), ids.cuda(), offsets=few.cuda())
    assert used[-1] == S - 1 and used[0] < S
    at = used.cuda()
    assert torch.equal(tokens[at], want[2]) and torch.equal(counts[at], want[1]) and int(tokens.sum()) == T and int(counts.sum()) == T * k
    # sums cut into other chunks: the shares' roundings of either side, below 100 steps each
    assert ((loss[at] - want[0]).abs() <= 2 * 2 * t.U * 100 * want[0]).all()
    tokens[at] = 0
    assert not tokens.any() and int((loss != 0).sum()) == len(used)


def apart(v):
    """The first, last and some other columns of v, which are the only ones that are not zero."""
    v[..., spread(v.shape[-1])] = torch.randn(*v.shape[:-1], len(spread(v.shape[-1])), device="cuda").to(v.dtype)
    return v


def test_rows_of_more_than_2_26_elements():
    wide, L, R, small, T = (1 << 26) + 1048, 2, 8, 64, 5
    print(f"[lora] K, N of {wide} and {small}", flush=True)
    ids, at = torch.tensor([[0], [1], [-1], [1], [0]], dtype=torch.int32, device="cuda"), spread(wide)
    zeros = lambda *shape: torch.zeros(*shape, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    # wide rows: x and a
    x, a, b = apart(zeros(T, wide)), apart(zeros(L, R, wide)), torch.randn(L, small, R, device="cuda").bfloat16()
    h = torch.empty(T, R, device="cuda")
    out = ftq.lora(x, a, b, ids, out_dtype=torch.float32, h=h)
    few_x, few_a = x[:, at].contiguous(), a[:, :, at].contiguous()
    ro, rh, mo, mh = t.lora_forward(few_x, few_a, b, ids, None, None, False)
    t.close(h, rh, mh, len(at) + 4, "h")
    t.close(out, ro, mo, len(at) + R + 8, "out")
    dy = torch.randn(T, small, device="cuda").bfloat16()
    d_x, d_a, d_b = ftq.lora_backward(dy, x, a, b, ids, h)
    ref = t.lora_backward(dy, few_x, few_a, b, ids, h, None, None, False)
    t.close(d_x[:, at], *ref["d_x"], small + R + 10, "d_x")
    t.close(d_a[:, :, at], *ref["d_a"], small + T + 10, "d_a")
    t.close(d_b, *ref["d_b"], T + 10, "d_b")
    for v in (d_x, d_a):
        v[..., at] = 0
        assert not v.any()
    del x, a, few_x, few_a, d_x, d_a
    # wide results: b and d_out
    x, a, b = torch.randn(T, small, device="cuda").bfloat16(), torch.randn(L, R, small, device="cuda").bfloat16(), zeros(L, wide, R)
    b[:, at] = torch.randn(L, len(at), R, device="cuda").bfloat16()
    out = ftq.lora(x, a, b, ids, h=h)
    few_b, dy = b[:, at].contiguous(), apart(zeros(T, wide))
    want = ftq.lora(x, a, torch.nn.functional.pad(few_b, (0, 0, 0, -len(at) % 8)), ids)[:, :len(at)]
    assert torch.equal(out[:, at], want)
    out[:, at] = 0
    assert not out.any()
    d_x, d_a, d_b = ftq.lora_backward(dy, x, a, b, ids, h)
    ref = t.lora_backward(dy[:, at], x, a, few_b, ids, h, None, None, False)
    t.close(d_x, *ref["d_x"], len(at) + R + 10, "d_x")
    t.close(d_a, *ref["d_a"], len(at) + T + 10, "d_a")
    t.close(d_b[:, at], *ref["d_b"], T + 10, "d_b")
    d_b[:, at] = 0
    assert not d_b.any()
