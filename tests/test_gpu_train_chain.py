"""The operators that train a router and adapters beside frozen experts, as they are
used together: one expert layer with its loss and gradients, on other streams, in
graphs that share or have their own workspaces, on two streams at once, and on a
padded batch whose padding is left out."""
import pytest
import torch

from quantized_moe_expert_quantize_amd import ftq
from tests import _train as t

pytestmark = pytest.mark.gpu

E, H, F, K = 8, 256, 128, 2          # experts, hidden size, expert width, choices
L, R = 2 * E, 16                     # two fine-tunes' adapters of each expert's second layer


class Layer:
    """Router -> experts (e4m3, frozen) -> adapters on the second layer -> combine, and back."""

    def __init__(self, T, seed=0):
        g = torch.Generator().manual_seed(seed)
        self.T = T
        self.x = torch.randn(T, H, generator=g).cuda()
        self.logits = torch.randn(T, E, generator=g).cuda()
        self.tune = torch.randint(0, 2, (T, 1), generator=g).to(torch.int32).cuda()
        self.w1, self.s1 = ftq.quantize_fp8_weight((torch.randn(E, 2 * F, H, generator=g) / 16).cuda())
        self.w2, self.s2 = ftq.quantize_fp8_weight((torch.randn(E, H, F, generator=g) / 11).cuda())
        self.a = (torch.randn(L, R, F, generator=g) / 11).bfloat16().cuda()
        self.b = (torch.randn(L, H, R, generator=g) / 4).bfloat16().cuda()
        self.scale = (torch.rand(L, generator=g) + 0.5).cuda()
        self.offsets = torch.tensor([0, T // 3, T], dtype=torch.int32).cuda()
        self.valid = torch.ones(T, dtype=torch.bool).cuda()
        self.d_out = torch.randn(T, H, generator=g).cuda()
        self.d_loss = torch.tensor([0.1, 0.2]).cuda()

    def run(self, stream=None):
        """Loss, output and all gradients; the memory of what lies between stays referenced."""
        ids, gates = ftq.moe_topk(self.logits, K, stream=stream)
        loss, counts, tokens = ftq.moe_balance(self.logits, ids, offsets=self.offsets, valid=self.valid, stream=stream)
        q, qs = ftq.quantize_fp8(self.x, stream=stream)
        h = ftq.moe_fp8(self.w1, self.s1, q, qs, ids, E, 2 * F, H, act=ftq.ACT_SILU, out_dtype=torch.bfloat16, stream=stream)
        hq, hs = ftq.quantize_fp8(h, stream=stream)
        y = ftq.moe_fp8(self.w2, self.s2, hq, hs, ids, E, H, F, per_pair=True, stream=stream)
        with torch.cuda.stream(stream or torch.cuda.current_stream()):
            ad = (self.tune * E + ids).contiguous()
            hidden = torch.empty(self.T * K, R, device="cuda")
        ftq.lora(h, self.a, self.b, ad, scale=self.scale, base=y, per_pair=True, out=y, h=hidden, stream=stream)
        out = ftq.combine_topk(y, gates, stream=stream)
        d_y, d_gates = ftq.combine_topk_backward(self.d_out, y, gates, d_y_dtype=torch.bfloat16, stream=stream)
        d_h, d_a, d_b = ftq.lora_backward(d_y, h, self.a, self.b, ad, hidden, scale=self.scale, per_pair=True, stream=stream)
        d_logits = ftq.moe_topk_backward(self.logits, ids, d_gates, d_loss=self.d_loss, counts=counts, tokens=tokens, offsets=self.offsets,
                                         valid=self.valid, stream=stream)
        self.keep = (q, qs, hq, hs, ad)
        return dict(ids=ids, gates=gates, loss=loss, counts=counts, h=h, y=y, hidden=hidden, out=out, d_y=d_y, d_gates=d_gates, d_h=d_h, d_a=d_a,
                    d_b=d_b, d_logits=d_logits)


def same(a, b):
    return [n for n in a if not torch.equal(a[n], b[n])]


@pytest.mark.parametrize("T", [3, 200, 1500])
def test_layer_against_64_bits(T):
    """Each step against its definition on what the step before gave, and the gradients against differences of the loss."""
    m = Layer(T)
    r = {n: v.cpu() for n, v in m.run().items()}
    seqs = t.sequences(T, m.offsets.tolist(), None)
    l = m.logits.cpu().double()
    want = t.losses(l, r["ids"], E, K, seqs, True)
    assert ((r["loss"].double() - want).abs() <= 2 * t.U * 100 * want).all()
    ad = (m.tune.cpu() * E + r["ids"])
    base = torch.zeros(T * K, H)
    delta, hid, md, mh = t.lora_forward(r["h"], m.a, m.b, ad, m.scale.cpu(), base, True)
    t.close(r["hidden"], hid, mh, F + 4, "hidden")
    y = r["y"].double()
    t.close(r["out"], (r["gates"].double()[:, :, None] * y.view(T, K, H)).sum(1), (r["gates"][:, :, None] * y.view(T, K, H).abs()).sum(1), K + 2, "out")
    ref = t.lora_backward(r["d_y"], r["h"], m.a, m.b, ad, r["hidden"], m.scale.cpu(), None, True)
    for n, terms in (("h", H + R + 10), ("a", H + T * K + 10), ("b", T * K + 10)):
        t.close(r["d_" + n], *ref["d_x" if n == "h" else "d_" + n], terms, n)

    # differences of <d_out, out> + <d_loss, losses> along random directions of logits, A and B, the choices held fixed
    y0 = y - delta                                             # what the frozen experts give (to y's rounding)

    def value(l, a, b):
        y = y0 + t.lora_forward(r["h"], a, b, ad, m.scale.cpu(), None, True)[0]
        out = (t.gates_of(l, r["ids"], True, True, 1.0)[:, :, None] * y.view(T, K, H)).sum(1)
        return float((out * m.d_out.cpu().double()).sum() + (t.losses(l, r["ids"], E, K, seqs, True) * m.d_loss.cpu().double()).sum())
    g, e = torch.Generator().manual_seed(1), 1e-4
    at = [l, m.a.cpu().double(), m.b.cpu().double()]
    for i, n in enumerate(("d_logits", "d_a", "d_b")):
        v = torch.randn(at[i].shape, generator=g).double()
        up, down = ([w + s * e * v if j == i else w for j, w in enumerate(at)] for s in (1, -1))
        diff = (value(*up) - value(*down)) / (2 * e)
        terms = r[n].double() * v
        # d_y passed through bf16 (2^-8 of each term, random sign), the rest in fp32; differences to e^2
        bound = 4 * 2.0 ** -8 * float(terms.norm()) * (1 if n != "d_logits" else 2.0 ** -8) + 1e-5 * float(terms.abs().sum()) + 1e-6
        assert abs(diff - float(terms.sum())) <= bound, (n, diff, float(terms.sum()), bound)


def test_layer_on_another_stream():
    m = Layer(300)
    want = m.run()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        noise = [torch.full((300 * K, H), float("nan"), device="cuda") for _ in range(3)]
        del noise
        got = m.run(s)
        torch.cuda.synchronize()
        assert not same(got, want)


def test_two_layers_at_once():
    """Two streams with calls of their own, each with its own workspaces."""
    layers = [Layer(700, seed=1), Layer(90, seed=2)]
    want = [m.run() for m in layers]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(5):
        got = [m.run(s) for m, s in zip(layers, streams)]
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert not same(a, b)


@pytest.mark.parametrize("T", [5, 600])
def test_captured_layer(T):
    """A graph of the whole layer, replayed with other inputs, eager work and synchronisations between the replays."""
    m = Layer(T)
    m.run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = m.run()
    kept = m.keep
    g = torch.Generator().manual_seed(3)
    for _ in range(4):
        for name in ("x", "logits", "d_out"):
            v = getattr(m, name)
            v.copy_(torch.randn(v.shape, generator=g))
        m.valid.copy_(torch.rand(T, generator=g) < 0.8)
        want = m.run()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert not same(got, want)
    del kept


def test_two_graphs_share_workspaces():
    """Calls of different sizes captured into two graphs with the same workspaces: each replay has its own results."""
    ws = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in (1 << 22, 1 << 24, 1 << 20)]
    graphs, results, wants = [], [], []
    for T, seed in ((400, 1), (37, 2)):
        g = torch.Generator().manual_seed(seed)
        x, a, b = torch.randn(T, 64, generator=g).half().cuda(), torch.randn(5, 8, 64, generator=g).half().cuda(), torch.randn(5, 72, 8, generator=g).half().cuda()
        ids = torch.randint(-1, 5, (T, 2), generator=g).to(torch.int32).cuda()
        dy, logits = torch.randn(2 * T, 72, generator=g).half().cuda(), torch.randn(T, 5, generator=g).cuda()
        hidden = torch.empty(2 * T, 8, device="cuda")

        def call(x=x, a=a, b=b, ids=ids, dy=dy, logits=logits, hidden=hidden):
            out = ftq.lora(x, a, b, ids, h=hidden, path=ftq.PATH_GROUPED, workspace=ws[0])
            grads = ftq.lora_backward(dy, x, a, b, ids, hidden, workspace=ws[1])
            return (out, *grads, *ftq.moe_balance(logits, ids, workspace=ws[2]))
        wants.append([v.clone() for v in call()])
        torch.cuda.synchronize()
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            results.append(call())
    for i in (0, 1, 1, 0, 1, 0):
        for w in ws:
            w.fill_(0xff)                                      # what a workspace holds on entry does not matter
        graphs[i].replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(results[i], wants[i]))


def test_padding_stays_out():
    """A batch with padded rows, whatever they hold, gives what the batch without them gives."""
    m = Layer(120)
    r = m.run()
    p = Layer(120)
    pad = 40
    for name in ("x", "logits", "d_out"):
        v = getattr(m, name)
        setattr(p, name, torch.cat([v, torch.full((pad, v.shape[1]), float("nan"), device="cuda")]))
    p.T, p.tune = 160, torch.cat([m.tune, torch.zeros(pad, 1, dtype=torch.int32, device="cuda")])
    p.valid = torch.cat([m.valid, torch.zeros(pad, dtype=torch.bool, device="cuda")])
    p.offsets = torch.tensor([0, 40, 160], dtype=torch.int32).cuda()
    ids, gates = ftq.moe_topk(p.logits, K)
    assert (ids[120:] == -1).all()                             # rows of NaN choose nothing
    loss, counts, tokens = ftq.moe_balance(p.logits, ids, offsets=p.offsets, valid=p.valid)
    assert torch.equal(loss, r["loss"]) and torch.equal(counts, r["counts"]) and tokens.tolist() == [40, 80]
    ad = torch.where(ids >= 0, p.tune * E + ids, -1).contiguous()
    h = torch.cat([r["h"], torch.full((pad * K, F), float("nan"), dtype=torch.bfloat16, device="cuda")])
    hidden = torch.cat([r["hidden"], torch.full((pad * K, R), float("nan"), device="cuda")])
    d_y = torch.cat([r["d_y"], torch.full((pad * K, H), float("nan"), dtype=torch.bfloat16, device="cuda")])
    _, d_a, d_b = ftq.lora_backward(d_y, h, p.a, p.b, ad, hidden, scale=p.scale, per_pair=True)
    for got, want in ((d_a, r["d_a"]), (d_b, r["d_b"])):
        assert got.isfinite().all()
        # the same sums of at most 240 terms, cut into other runs of tiles: as many roundings of random sign
        assert (got - want).norm() <= 4 * 2 * t.U * 240 ** 0.5 * want.norm()
    d_logits = ftq.moe_topk_backward(p.logits, ids, torch.cat([r["d_gates"], torch.ones(pad, K, device="cuda")]), d_loss=p.d_loss, counts=counts,
                                     tokens=tokens, offsets=p.offsets, valid=p.valid)
    assert torch.equal(d_logits[:120], r["d_logits"]) and not d_logits[120:].any()


def _allocating_calls():
    g = torch.Generator().manual_seed(5)
    x, a, b = torch.randn(300, 64, generator=g).cuda(), torch.randn(5, 8, 64, generator=g).cuda(), torch.randn(5, 72, 8, generator=g).cuda()
    ids = torch.randint(-1, 5, (300, 2), generator=g).to(torch.int32).cuda()
    hidden, dy, y = torch.randn(600, 8, generator=g).cuda(), torch.randn(600, 72, generator=g).cuda(), torch.randn(600, 72, generator=g).cuda()
    logits, gates, d_out = torch.randn(300, 5, generator=g).cuda(), torch.rand(300, 2, generator=g).cuda(), torch.randn(300, 72, generator=g).cuda()
    return {
        "moe_balance": lambda s: ftq.moe_balance(logits, ids, stream=s),
        "moe_topk_backward": lambda s: ftq.moe_topk_backward(logits, ids, gates, stream=s),
        "combine_topk_backward": lambda s: ftq.combine_topk_backward(d_out, y, gates, stream=s),
        "lora": lambda s: ftq.lora(x, a, b, ids, path=ftq.PATH_GROUPED, stream=s),
        "lora_backward": lambda s: ftq.lora_backward(dy, x, a, b, ids, hidden, stream=s),
    }


@pytest.mark.parametrize("name", ["moe_balance", "moe_topk_backward", "combine_topk_backward", "lora", "lora_backward"])
def test_memory_of_a_call_on_another_stream(name, monkeypatch):
    """What a call allocates comes from the memory of the stream it works on."""
    call = _allocating_calls()[name]
    want = call(None)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    seen, empty = [], torch.empty

    def spy(*args, **kw):
        seen.append(torch.cuda.current_stream())
        return empty(*args, **kw)
    monkeypatch.setattr(torch, "empty", spy)
    got = call(s)
    monkeypatch.undo()
    torch.cuda.synchronize()
    assert seen and all(v == s for v in seen)
    got, want = ((v,) if isinstance(v, torch.Tensor) else v for v in (got, want))
    assert all(torch.equal(p, q) for p, q in zip(got, want))
