"""What the operators that train a router and low-rank adapters beside frozen experts are measured on.

Five kinds of call, each in a plain form (elementary torch operations in 32 bits,
64 for long sums) and as the calls a user makes of the package:

  balance           router logits and choices -> per-expert counts and balance loss of every packed sequence;
  router_backward   gradients of gates and balance losses -> gradient of the logits;
  combine_backward  gradient of a layer's output -> gradients of the experts' rows and of the gates;
  lora              rows of requests with an adapter each, or of (token, expert) pairs -> shared projection's result
                    plus the low-rank product of the row's own adapter;
  lora_backward     gradient of that -> gradients of the rows and of every adapter's two factors.
"""
import math

import torch

own = False

DEVICE = "cuda"
DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "f16": 2, "bf16": 2}


# ---- cases -------------------------------------------------------------------

def listed():
    return [
        # the loss of a small batch: latency of one call
        dict(name="balance_batch", kind="balance", T=256, E=64, top_k=6, dtype="bf16", score="softmax", seqs=1, padded=0.0, tail=0),
        # a training step's packed sequences of different lengths, some rows padding
        dict(name="balance_packed", kind="balance", T=32768, E=256, top_k=8, dtype="f32", score="sigmoid", seqs=37, padded=0.03, tail=0),
        # gradients of one prompt's gates, no balance loss
        dict(name="router_backward_gates", kind="router_backward", T=1000, E=128, top_k=8, dtype="bf16", score="softmax", renorm=True,
             scale=1.0, balance=False, seqs=1, padded=0.0, tail=0),
        # gates and balance losses of a training step's packed sequences
        dict(name="router_backward_packed", kind="router_backward", T=32768, E=256, top_k=8, dtype="f32", score="sigmoid", renorm=True,
             scale=2.5, balance=True, seqs=37, padded=0.03, tail=0),
        # a short sequence through 2 of 8 experts
        dict(name="combine_backward_short", kind="combine_backward", T=64, top_k=2, N=4096, out="bf16"),
        # a long batch through 8 of 128 experts
        dict(name="combine_backward_long", kind="combine_backward", T=8191, top_k=8, N=2816, out="bf16"),
        # a decode step: 16 requests, one token each, on 8 adapters (some requests have none)
        dict(name="lora_decode", kind="lora", L=8, R=16, K=4096, N=4096, T=16, top_k=1, per_pair=False, requests=16, without=0.1,
             dtype="bf16", out="bf16", keep=False),
        # a prefill of requests of different lengths
        dict(name="lora_prefill", kind="lora", L=8, R=32, K=4096, N=4096, T=8191, top_k=1, per_pair=False, requests=20, without=0.1,
             dtype="bf16", out="bf16", keep=False),
        # second layer of the experts: an adapter for each of 4 fine-tunes x 128 experts, one row a pair, added to fp32 results
        dict(name="lora_experts", kind="lora", L=512, R=16, K=1408, N=2816, T=2048, top_k=8, per_pair=True, requests=0, without=0.0,
             dtype="bf16", out="f32", keep=False),
        # a short batch of three small adapters
        dict(name="lora_backward_short", kind="lora_backward", L=3, R=8, K=1024, N=1000, T=500, top_k=1, per_pair=False, requests=5,
             without=0.1, dtype="f16"),
        # a training step of a few wide adapters
        dict(name="lora_backward_long", kind="lora_backward", L=4, R=64, K=4096, N=4096, T=8192, top_k=1, per_pair=False, requests=8,
             without=0.0, dtype="bf16"),
        # first layer of the experts: one adapter an expert, a token's row shared by its pairs
        dict(name="lora_backward_experts", kind="lora_backward", L=128, R=16, K=2816, N=2816, T=1024, top_k=8, per_pair=False, requests=0,
             without=0.0, dtype="bf16"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["balance", "router_backward", "combine_backward", "lora", "lora", "lora_backward", "lora_backward"])
    dtype = rng.choice(["f32", "f16", "bf16", "bf16"])
    if kind in ("balance", "router_backward"):
        E = rng.choice([8, 16, 60, 64, 100, 128, 160, 256, 384])
        T = _log_int(rng, 16, 32768 * 256 // max(E, 256))
        case = dict(kind=kind, T=T, E=E, top_k=rng.randint(1, 8), dtype=dtype, score=rng.choice(["softmax", "sigmoid"]),
                    seqs=rng.choice([1, 1, _log_int(rng, 2, min(64, T // 4))]), padded=rng.choice([0.0, 0.0, 0.1]),
                    tail=rng.choice([0, 0, T // 9]))
        if kind == "router_backward":
            case.update(renorm=rng.random() < 0.6, scale=rng.choice([1.0, 2.5]), balance=rng.random() < 0.7)
        return case
    if kind == "combine_backward":
        top_k, N = rng.randint(1, 8), _log_int(rng, 100, 4100)
        return dict(kind=kind, T=_log_int(rng, 1, 8191 * 8 * 2816 // (8 * 4100)), top_k=top_k, N=N, out=dtype)
    R, K, N = rng.choice([8, 16, 16, 24, 32, 64, 96]), 8 * _log_int(rng, 16, 512), 8 * _log_int(rng, 16, 512)
    wide = 2 if dtype == "f32" else 1
    most = 8191 * 16 // (max(R, 16) * wide)                      # rows, so that no drawn case outgrows the listed ones
    if rng.random() < 0.6:                                       # requests of adapters
        T = _log_int(rng, 1, most)
        case = dict(kind=kind, L=rng.choice([1, 2, 5, 8, 16, 32]), R=R, K=K, N=N, T=T, top_k=1, per_pair=False,
                    requests=rng.choice([T, max(1, T // 7), 1 + min(20, T // 2)]) if T <= 256 else _log_int(rng, 1, 32),
                    without=rng.choice([0.0, 0.1, 0.3]), dtype=dtype)
    else:                                                        # adapters of experts
        top_k = rng.choice([2, 4, 6, 8])
        case = dict(kind=kind, L=rng.choice([8, 16, 60, 64, 128]), R=min(R, 32), K=K, N=N, T=_log_int(rng, 1, max(2, most // (2 * top_k))),
                    top_k=top_k, per_pair=rng.random() < 0.5, requests=0, without=rng.choice([0.0, 0.1]), dtype=dtype)
    if kind == "lora":
        case.update(out=rng.choice([dtype, "f32"]), keep=rng.random() < 0.4)
    return case


# ---- inputs ------------------------------------------------------------------

def _generator(seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(seed)
    return g


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device=DEVICE)


def _uniform(g, *shape):
    return torch.rand(*shape, generator=g, device=DEVICE)


def _distinct(g, T, E, top_k):
    """top_k distinct experts per token, evenly spread but for some more popular ones."""
    gumbel = -torch.log((-torch.log(_uniform(g, T, E).clamp(1e-20, 1 - 1e-7))))
    return (gumbel + 0.3 * _normal(g, E)).topk(top_k, dim=1).indices.to(torch.int32)


def _cuts(g, total, parts):
    """Ascending offsets [parts + 1] of `parts` runs of different lengths (some may be empty) that fill `total`."""
    w = torch.cumsum(0.1 + _uniform(g, parts), 0)
    ends = (w / w[-1] * total).round().to(torch.int32)
    return torch.cat([torch.zeros(1, dtype=torch.int32, device=DEVICE), ends])


def _adapters(g, case, state):
    L, R, K, N, T, top_k = (case[k] for k in ("L", "R", "K", "N", "T", "top_k"))
    dt = DTYPES[case["dtype"]]
    rows = T * top_k if case["per_pair"] else T
    state["x"] = (_normal(g, rows, K) * torch.exp(0.5 * _normal(g, K))).to(dt)
    state["a"] = (_normal(g, L, R, K) / math.sqrt(K)).to(dt)
    state["b"] = (_normal(g, L, N, R) / math.sqrt(R)).to(dt)
    state["lora_scale"] = 0.5 + _uniform(g, L)
    if case["requests"]:                                         # the rows of a request lie together and share its adapter
        cuts = _cuts(g, T, case["requests"])
        request = torch.searchsorted(cuts[1:].contiguous(), torch.arange(T, device=DEVICE, dtype=torch.int32), right=True)
        adapter = torch.randint(0, L, (case["requests"],), generator=g, device=DEVICE, dtype=torch.int32)
        adapter = torch.where(_uniform(g, case["requests"]) < case["without"], -1, adapter)
        state["topk_ids"] = adapter[request.clamp_max(case["requests"] - 1)].reshape(T, 1).contiguous()
    else:
        ids = _distinct(g, T, L, top_k)
        state["topk_ids"] = torch.where(_uniform(g, T, top_k) < case["without"], torch.full_like(ids, -1), ids).contiguous()
    flat = state["topk_ids"].reshape(-1).long()
    state["cap"] = max(1, int(torch.bincount(flat[flat >= 0], minlength=L).max()))   # rows of the fullest adapter


def prepare(case, seed):
    g = _generator(seed)
    kind, state = case["kind"], dict(case)
    if kind in ("balance", "router_backward"):
        T, E, S = case["T"], case["E"], case["seqs"]
        logits = 1.5 * _normal(g, T, E) + 0.5 * _normal(g, E)
        state["logits"] = logits.to(DTYPES[case["dtype"]])
        state["topk_ids"] = state["logits"].float().topk(case["top_k"], dim=1).indices.to(torch.int32).contiguous()
        state["valid"] = _uniform(g, T) >= case["padded"] if case["padded"] else None
        state["offsets"] = _cuts(g, T - case["tail"], S) if S > 1 or case["tail"] else None
        if kind == "router_backward":
            state["d_gates"] = _normal(g, T, case["top_k"])
            state["d_loss"] = (0.01 * (1 + _uniform(g, S))) if case["balance"] else None
            state["counts"], state["tokens"] = _counts(state) if case["balance"] else (None, None)
            state["d_logits"] = torch.empty_like(state["logits"])
    elif kind == "combine_backward":
        T, top_k, N = case["T"], case["top_k"], case["N"]
        state["y"] = _normal(g, T * top_k, N)
        state["gates"] = torch.softmax(_normal(g, T, top_k), 1)
        state["d_out"] = _normal(g, T, N)
        state["d_y"] = torch.empty(T * top_k, N, dtype=DTYPES[case["out"]], device=DEVICE)
        state["d_gates"] = torch.empty(T, top_k, device=DEVICE)
    else:
        _adapters(g, case, state)
        pairs = case["T"] * case["top_k"]
        if kind == "lora":
            state["base"] = _normal(g, pairs, case["N"]).to(DTYPES[case["out"]])
            state["out_buffer"] = torch.empty_like(state["base"])
            state["h"] = torch.empty(pairs, case["R"], device=DEVICE) if case["keep"] else None
        else:
            state["d_out"] = _normal(g, pairs, case["N"]).to(DTYPES[case["dtype"]])
            state["h"] = _lora_plain(state)[1]                   # as the forward pass kept it
            state["d_x"] = torch.empty_like(state["x"])
            state["d_a"] = torch.empty(state["a"].shape, device=DEVICE)
            state["d_b"] = torch.empty(state["b"].shape, device=DEVICE)
    return state


# ---- the passes --------------------------------------------------------------

def run(state):
    kind = state["kind"]
    if own:
        return _own(kind, state)
    if kind == "balance":
        return _balance_plain(state)
    if kind == "router_backward":
        return _router_backward_plain(state)
    if kind == "combine_backward":
        return _combine_backward_plain(state)
    if kind == "lora":
        out, h = _lora_plain(state)
        return (out, h) if state["keep"] else out
    return _lora_backward_plain(state)


def _own(kind, state):
    from quantized_moe_expert_quantize_amd import ftq
    if kind in ("balance", "router_backward"):
        score = ftq.SCORE_SOFTMAX if state["score"] == "softmax" else ftq.SCORE_SIGMOID
    if kind == "balance":
        if "workspace" not in state:   # a program keeps one workspace for its shapes
            state["workspace"] = torch.empty(ftq.balance_workspace_bytes(state["T"], state["E"], state["top_k"], state["seqs"]),
                                             dtype=torch.uint8, device=DEVICE)
        return ftq.moe_balance(state["logits"], state["topk_ids"], score=score, offsets=state["offsets"], valid=state["valid"],
                               workspace=state["workspace"])
    if kind == "router_backward":
        return ftq.moe_topk_backward(state["logits"], state["topk_ids"], d_gates=state["d_gates"], score=score, renorm=state["renorm"],
                                     scale=state["scale"], d_loss=state["d_loss"], counts=state["counts"], tokens=state["tokens"],
                                     offsets=state["offsets"], valid=state["valid"], out=state["d_logits"])
    if kind == "combine_backward":
        return ftq.combine_topk_backward(state["d_out"], state["y"], state["gates"], d_y=state["d_y"], d_gates=state["d_gates"])
    L, R, K, N, T, top_k = (state[k] for k in ("L", "R", "K", "N", "T", "top_k"))
    if "workspace" not in state:
        size = ftq.lora_workspace_bytes if kind == "lora" else ftq.lora_backward_workspace_bytes
        state["workspace"] = torch.empty(size(L, R, K, N, T, top_k, state["x"].dtype), dtype=torch.uint8, device=DEVICE)
    if kind == "lora":
        out = ftq.lora(state["x"], state["a"], state["b"], state["topk_ids"], scale=state["lora_scale"], base=state["base"],
                       per_pair=state["per_pair"], out=state["out_buffer"], h=state["h"], workspace=state["workspace"])
        return (out, state["h"]) if state["keep"] else out
    return ftq.lora_backward(state["d_out"], state["x"], state["a"], state["b"], state["topk_ids"], state["h"],
                             scale=state["lora_scale"], per_pair=state["per_pair"], d_x=state["d_x"], d_a=state["d_a"],
                             d_b=state["d_b"], workspace=state["workspace"])


# ---- plain forms -------------------------------------------------------------

def _sequence_of(state):
    """(sequence of each row, number of sequences); rows that count nowhere belong to one more."""
    T, S = state["T"], state["seqs"]
    row = torch.arange(T, device=DEVICE, dtype=torch.int32)
    seq = torch.zeros(T, dtype=torch.long, device=DEVICE)
    if state["offsets"] is not None:
        seq = torch.searchsorted(state["offsets"][1:].contiguous(), row, right=True)   # S behind the last one
    if state["valid"] is not None:
        seq = torch.where(state["valid"], seq, S)
    return seq, S


def _counts(state):
    """Pairs of every sequence sent to every expert, and its counted tokens."""
    E, (seq, S) = state["E"], _sequence_of(state)
    at = (seq[:, None] * E + state["topk_ids"].long()).reshape(-1)
    counts = torch.zeros((S + 1) * E, dtype=torch.int32, device=DEVICE).scatter_add_(0, at, torch.ones_like(at, dtype=torch.int32))
    return counts.view(S + 1, E)[:S].contiguous(), _by_sequence(torch.ones(state["T"], 1, device=DEVICE), state)[:, 0].to(torch.int32)


def _by_sequence(rows, state):
    """Sums of the counted rows of every sequence, in 64 bits: products with their membership, 128 rows each, then their sum."""
    seq, S = _sequence_of(state)
    blocks, more = -(-len(seq) // 128), -len(seq) % 128
    member = torch.nn.functional.pad((seq[:, None] == torch.arange(S, device=DEVICE)).double(), (0, 0, 0, more))
    rows = torch.nn.functional.pad(rows.double(), (0, 0, 0, more))
    return torch.bmm(member.view(blocks, 128, S).transpose(1, 2).contiguous(), rows.view(blocks, 128, -1)).sum(0)


def _probabilities(logits, score):
    """(scores, their share of the row's sum)."""
    if score == "softmax":
        e = torch.exp(logits - logits.amax(1, keepdim=True))
        p = e / e.sum(1, keepdim=True)
        return p, p
    s = 1 / (1 + torch.exp(-logits))
    return s, s / s.sum(1, keepdim=True)


def _balance_plain(state):
    _, p = _probabilities(state["logits"].float(), state["score"])
    counts, tokens = _counts(state)
    n = tokens.double().clamp_min(1)
    total = (counts.double() * _by_sequence(p, state)).sum(1)
    return (total * state["E"] / (state["top_k"] * n * n)).float(), counts, tokens


def _router_backward_plain(state):
    E, top_k = state["E"], state["top_k"]
    seq, S = _sequence_of(state)
    s, p = _probabilities(state["logits"].float(), state["score"])
    ids = state["topk_ids"].long()
    ds = torch.zeros_like(s)
    if state["renorm"]:
        chosen = s.gather(1, ids)
        q = chosen / chosen.sum(1, keepdim=True)
        d = state["scale"] * q * (state["d_gates"] - (q * state["d_gates"]).sum(1, keepdim=True))   # d_s times s
        ds.scatter_(1, ids, d)
        grad = ds if state["score"] == "softmax" else ds * (1 - s)
    else:
        ds.scatter_(1, ids, state["scale"] * state["d_gates"])
        if state["score"] == "softmax":
            grad = s * (ds - (ds * s).sum(1, keepdim=True))
        else:
            grad = s * (1 - s) * ds
    if state["balance"]:
        n = state["tokens"].float().clamp_min(1)
        v = state["counts"].float() * (state["d_loss"] * E / (top_k * n * n))[:, None]
        v = torch.cat([v, torch.zeros(1, E, device=DEVICE)])[seq]
        add = p * (v - (p * v).sum(1, keepdim=True))
        grad = grad + (add if state["score"] == "softmax" else add * (1 - s))
    if state["valid"] is not None:
        grad = torch.where(state["valid"][:, None], grad, 0.0)
    return grad.to(state["logits"].dtype)


def _combine_backward_plain(state):
    T, top_k, N = state["T"], state["top_k"], state["N"]
    d_out, y = state["d_out"][:, None, :], state["y"].view(T, top_k, N)
    d_y = (state["gates"][:, :, None] * d_out).to(DTYPES[state["out"]]).view(T * top_k, N)
    return d_y, (y * d_out).sum(2)


def _slots(state):
    """Where each pair lies when the pairs are sorted by adapter and every adapter's padded to the fullest one's."""
    L, cap = state["L"], state["cap"]
    flat = state["topk_ids"].reshape(-1).long()
    pair = torch.arange(flat.numel(), device=DEVICE)
    bucket = torch.where(flat < 0, L, flat)
    order = torch.argsort(bucket, stable=True)
    first = torch.searchsorted(bucket[order].contiguous(), torch.arange(L + 1, device=DEVICE))
    slot = torch.empty_like(pair)
    slot[order] = bucket[order] * cap + pair - first[bucket[order]]
    return torch.where(flat < 0, L * cap, slot), flat < 0, pair if state["per_pair"] else pair // state["top_k"]


def _spread(rows, slot, state):
    """Rows of the pairs -> [L, cap, columns], zeros in the padding."""
    out = torch.zeros(state["L"] * state["cap"] + 1, rows.shape[1], device=DEVICE)
    out[slot] = rows
    return out[:-1].view(state["L"], state["cap"], -1)


def _gather(blocks, slot, none):
    flat = blocks.reshape(-1, blocks.shape[2])
    return flat[slot.clamp_max(flat.shape[0] - 1)].masked_fill(none[:, None], 0.0)


def _lora_plain(state):
    slot, none, row = _slots(state)
    h = torch.bmm(_spread(state["x"].float()[row], slot, state), state["a"].float().transpose(1, 2))
    y = torch.bmm(h, state["b"].float().transpose(1, 2)) * state["lora_scale"][:, None, None]
    out = _gather(y, slot, none)
    if "base" in state:
        out = (state["base"].float() + out).to(DTYPES[state["out"]])
    return out, _gather(h, slot, none)


def _lora_backward_plain(state):
    T, top_k = state["T"], state["top_k"]
    slot, none, row = _slots(state)
    dy = _spread(state["d_out"].float(), slot, state) * state["lora_scale"][:, None, None]
    x, h = _spread(state["x"].float()[row], slot, state), _spread(state["h"], slot, state)
    g = torch.bmm(dy, state["b"].float())
    d_x = _gather(torch.bmm(g, state["a"].float()), slot, none)
    if not state["per_pair"]:
        d_x = d_x.view(T, top_k, -1).sum(1)
    d_a, d_b = torch.bmm(g.transpose(1, 2), x), torch.bmm(dy.transpose(1, 2), h)
    return d_x.to(state["x"].dtype), d_a, d_b


# ---- work --------------------------------------------------------------------

def work(case):
    kind = case["kind"]
    if kind == "combine_backward":
        T, top_k, N = case["T"], case["top_k"], case["N"]
        return {"bytes": T * top_k * (N * (4 + BYTES[case["out"]]) + 8) + T * N * 4, "flops": 3 * T * top_k * N}
    if kind in ("balance", "router_backward"):
        T, E, top_k, S = case["T"], case["E"], case["top_k"], case["seqs"]
        rows = T * E * BYTES[case["dtype"]]
        if kind == "balance":
            return {"bytes": rows + T * top_k * 4 + S * (E + 2) * 4, "flops": 6 * T * E}
        return {"bytes": 2 * rows + T * top_k * 8 + (S * (E + 2) * 4 if case["balance"] else 0), "flops": 12 * T * E}
    L, R, K, N, T, top_k = (case[k] for k in ("L", "R", "K", "N", "T", "top_k"))
    pairs = T * top_k
    rows = pairs if case["per_pair"] else T
    es = BYTES[case["dtype"]]
    share = 1 - case["without"]
    takers = (case["requests"] or pairs) * share
    used = L * (1 - (1 - 1 / L) ** takers) if L > 1 else 1       # adapters that some row takes
    weights = int(used * R * (K + N))
    if kind == "lora":
        return {"bytes": rows * K * es + weights * es + pairs * 4 + 2 * pairs * N * BYTES[case["out"]] + (pairs * R * 4 if case["keep"] else 0),
                "flops": int(2 * pairs * share * R * (K + N))}
    return {"bytes": 2 * rows * K * es + pairs * (N * es + R * 4 + 4) + weights * es + L * R * (K + N) * 4,
            "flops": int(4 * pairs * share * R * (K + N))}


# ---- the definitions in 64 bits ----------------------------------------------

def _rows_by_sequence(case, state):
    """The counted rows of each sequence."""
    cuts = [0, case["T"]] if state["offsets"] is None else state["offsets"].tolist()
    valid = torch.ones(case["T"], dtype=torch.bool, device=DEVICE) if state["valid"] is None else state["valid"]
    return [b + valid[b:e].nonzero()[:, 0] for b, e in zip(cuts, cuts[1:])]


def _share64(l, score):
    if score == "softmax":
        return torch.exp(l - torch.logsumexp(l, 1, keepdim=True))
    s = 1 / (1 + torch.exp(-l))
    return s / s.sum(1, keepdim=True)


def _loss64(l, ids, case, rows):
    """The balance loss of one sequence's rows, and its counts."""
    E, n = case["E"], len(rows)
    c = torch.bincount(ids[rows].reshape(-1).long(), minlength=E)
    return E * ((c.double() / (max(n, 1) * case["top_k"])) * (_share64(l[rows], case["score"]).sum(0) / max(n, 1))).sum(), c


def exact(case, seed):
    state = prepare(case, seed)
    kind = case["kind"]
    if kind == "balance":
        l = state["logits"].double()
        rows = _rows_by_sequence(case, state)
        both = [_loss64(l, state["topk_ids"], case, r) for r in rows]
        return (torch.stack([b[0] for b in both]), torch.stack([b[1] for b in both]).to(torch.int32),
                torch.tensor([len(r) for r in rows], dtype=torch.int32, device=DEVICE))
    if kind == "router_backward":                                # by differentiating the definition
        l = state["logits"].double().requires_grad_()
        s = torch.softmax(l, 1) if case["score"] == "softmax" else torch.sigmoid(l)
        gates = s.gather(1, state["topk_ids"].long())
        if case["renorm"]:
            gates = gates / gates.sum(1, keepdim=True)
        weight = state["d_gates"].double()
        if state["valid"] is not None:
            weight = weight * state["valid"][:, None]
        total = (case["scale"] * gates * weight).sum()
        if case["balance"]:
            for q, r in enumerate(_rows_by_sequence(case, state)):
                if len(r):
                    total = total + state["d_loss"][q].double() * _loss64(l, state["topk_ids"], case, r)[0]
        return torch.autograd.grad(total, l)[0]
    if kind == "combine_backward":
        T, top_k, N = case["T"], case["top_k"], case["N"]
        d_y = torch.empty(T * top_k, N, dtype=torch.float64, device=DEVICE)
        d_gates = torch.empty(T, top_k, dtype=torch.float64, device=DEVICE)
        d_out = state["d_out"].double()
        for j in range(top_k):
            d_y[j::top_k] = state["gates"][:, j, None].double() * d_out
            d_gates[:, j] = (state["y"][j::top_k].double() * d_out).sum(1)
        return d_y, d_gates
    L, R, K, N, T, top_k = (case[k] for k in ("L", "R", "K", "N", "T", "top_k"))
    flat = state["topk_ids"].reshape(-1)
    back = kind == "lora_backward"
    if back:
        d_x = torch.zeros(state["x"].shape, dtype=torch.float64, device=DEVICE)
        d_a = torch.zeros(L, R, K, dtype=torch.float64, device=DEVICE)
        d_b = torch.zeros(L, N, R, dtype=torch.float64, device=DEVICE)
    else:
        out = state["base"].double()
        hs = torch.zeros(T * top_k, R, dtype=torch.float64, device=DEVICE)
    for l in range(L):
        p = (flat == l).nonzero()[:, 0]
        if not len(p):
            continue
        r = p if case["per_pair"] else p // top_k
        x, a, b, scale = state["x"][r].double(), state["a"][l].double(), state["b"][l].double(), state["lora_scale"][l].double()
        if back:
            dy = state["d_out"][p].double() * scale
            g = dy @ b
            d_x.index_add_(0, r, g @ a)
            d_a[l] = g.t() @ x
            d_b[l] = dy.t() @ state["h"][p].double()
        else:
            h = x @ a.t()
            hs[p] = h
            out[p] += scale * (h @ b.t())
    if back:
        return d_x, d_a, d_b
    return (out, hs) if case["keep"] else out
