"""Calls on a stream that is not the current one: what they allocate belongs to that stream."""
import pytest
import torch

from quantized_moe_expert_quantize_amd import ftq, inputs

pytestmark = pytest.mark.gpu

E, N, K, T, TOP_K = 8, 64, 256, 80, 2


def calls():
    """name -> call(stream) of every entry that allocates, on its path with a workspace."""
    g = torch.Generator().manual_seed(0)
    x = torch.randn(T, K, generator=g).cuda()
    xp = torch.randn(T * TOP_K, K, generator=g).cuda()
    w32 = (torch.randn(E, N, K, generator=g) * 0.05).cuda()
    logits = torch.randn(T, E, generator=g).cuda()
    ids = torch.from_numpy(inputs.routing(T, E, TOP_K, seed=1)).cuda()
    gates = torch.from_numpy(inputs.gates(T, TOP_K, seed=1)).cuda()
    w, a, ap = ftq.quantize_q4_0(w32), ftq.quantize_q8_1(x), ftq.quantize_q8_1(xp)
    w8 = torch.from_numpy(inputs.gguf_blocks(ftq.W_Q8_0, E, N, K)).cuda()
    w5 = torch.from_numpy(inputs.gguf_blocks(ftq.W_Q5_0, E, N, K)).cuda()
    f, fs = ftq.quantize_fp8_weight(w32)
    b, bs = ftq.quantize_fp8(x)
    y = torch.randn(T * TOP_K, N, generator=g).cuda()
    P = ftq.PATH_GROUPED
    return {
        "quantize_q8_1": lambda s: ftq.quantize_q8_1(x, stream=s),
        "quantize_q4_0": lambda s: ftq.quantize_q4_0(w32, stream=s),
        "moe": lambda s: ftq.moe(w, a, ids, E, N, K, path=P, stream=s),
        "moe_partials": lambda s: ftq.moe_partials(w, a, ids, E, N, K, path=P, stream=s),
        "moe_pairs": lambda s: ftq.moe_pairs(w, ap, ids, E, N, K, path=P, stream=s),
        "moe_pairs_partials": lambda s: ftq.moe_pairs_partials(w, ap, ids, E, N, K, path=P, stream=s),
        "moe_act": lambda s: ftq.moe_act(w, a, ids, E, N, K, ftq.ACT_SILU, path=P, stream=s),
        "moe_gguf": lambda s: ftq.moe_gguf(w8, ftq.W_Q8_0, a, ids, E, N, K, path=P, stream=s),
        "moe_gguf_gemv": lambda s: ftq.moe_gguf(w5, ftq.W_Q5_0, a, ids, E, N, K, stream=s),
        "moe_gguf_partials": lambda s: ftq.moe_gguf_partials(w8, ftq.W_Q8_0, a, ids, E, N, K, path=P, stream=s),
        "combine_topk": lambda s: ftq.combine_topk(y, gates, stream=s),
        "moe_topk": lambda s: ftq.moe_topk(logits, TOP_K, stream=s),
        "quantize_fp8": lambda s: ftq.quantize_fp8(x, stream=s),
        "quantize_fp8_weight": lambda s: ftq.quantize_fp8_weight(w32, stream=s),
        "moe_fp8": lambda s: ftq.moe_fp8(f, fs, b, bs, ids, E, N, K, path=P, stream=s),
    }


NAMES = ["quantize_q8_1", "quantize_q4_0", "moe", "moe_partials", "moe_pairs", "moe_pairs_partials", "moe_act", "moe_gguf", "moe_gguf_gemv",
         "moe_gguf_partials", "combine_topk", "moe_topk", "quantize_fp8", "quantize_fp8_weight", "moe_fp8"]


def same(a, b):
    a, b = (t if isinstance(t, tuple) else (t,) for t in (a, b))
    return all(torch.equal(p.view(torch.uint8), q.view(torch.uint8)) for p, q in zip(a, b))


@pytest.mark.parametrize("name", NAMES)
def test_memory_of_a_call_on_another_stream(name, monkeypatch):
    call = calls()[name]
    want = call(None)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    seen = []
    empty = torch.empty

    def spy(*args, **kw):
        seen.append(torch.cuda.current_stream())
        return empty(*args, **kw)
    monkeypatch.setattr(torch, "empty", spy)
    current = torch.cuda.current_stream()
    got = call(s)
    monkeypatch.undo()
    assert torch.cuda.current_stream() == current
    torch.cuda.synchronize()
    assert seen and all(t == s for t in seen)
    assert same(got, want)


def test_a_chain_beside_work_of_the_current_stream():
    """A chain on one stream while the current one fills and frees memory of the same sizes: neither disturbs the other."""
    s = torch.cuda.Stream()
    g = torch.Generator().manual_seed(3)
    x, logits = torch.randn(600, K, generator=g).cuda(), torch.randn(600, E, generator=g).cuda()
    w, ws = ftq.quantize_fp8_weight((torch.randn(E, N, K, generator=g) * 0.05).cuda())

    def chain(stream):
        ids, gates = ftq.moe_topk(logits, TOP_K, stream=stream)
        a, as_ = ftq.quantize_fp8(x, stream=stream)
        y = ftq.moe_fp8(w, ws, a, as_, ids, E, N, K, path=ftq.PATH_GROUPED, stream=stream)
        out = ftq.combine_topk(y, gates, stream=stream)
        if stream is not None:
            for t in (ids, gates, a, as_, y):   # freed here, still to be read there
                t.record_stream(stream)
        return out
    want = chain(None)
    torch.cuda.synchronize()
    for i in range(20):
        mine = [torch.full((600 * TOP_K, N), float(i), device="cuda") for _ in range(4)]
        total = sum(mine)
        del mine
        got = chain(s)
        torch.cuda.synchronize()
        assert torch.equal(got, want) and (total == 4.0 * i).all()


@pytest.mark.parametrize("tokens", [3, 600])
def test_a_captured_chain_on_a_forked_stream(tokens):
    """A graph whose calls run on a stream forked from the captured one and joined again, replayed with other inputs and
    eager work between the replays."""
    g = torch.Generator().manual_seed(4)
    x, logits = torch.randn(tokens, K, generator=g).cuda(), torch.randn(tokens, E, generator=g).cuda()
    w, ws = ftq.quantize_fp8_weight((torch.randn(E, N, K, generator=g) * 0.05).cuda())
    s = torch.cuda.Stream()

    def chain(stream):
        ids, gates = ftq.moe_topk(logits, TOP_K, stream=stream)
        a, as_ = ftq.quantize_fp8(x, stream=stream)
        y = ftq.moe_fp8(w, ws, a, as_, ids, E, N, K, out_dtype=torch.float32, stream=stream)
        return ids, gates, y, ftq.combine_topk(y, gates, stream=stream)
    chain(None)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.wait_stream(torch.cuda.current_stream())
        got = chain(s)
        torch.cuda.current_stream().wait_stream(s)
    for seed in range(4):
        g.manual_seed(10 + seed)
        x.copy_(torch.randn(tokens, K, generator=g))
        logits.copy_(torch.randn(tokens, E, generator=g))
        want = chain(None)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
