"""Operators over the paged latent cache of a batch of sequences, as cases to be measured: attention for a
tree of drafted tokens over each sequence's cached rows, the attention weight that every cached row has
gathered, and eviction of the rows that gathered least.  Each has a plain form (elementary torch operations
in 32 bits, rounded once), the call of the library (`own`), and its definition in 64 bits (`exact`).

A row of 8 bits stands for bf16(code * scale): that is what the library's attention multiplies, and the
weights belong to the probabilities of that attention."""

import math

import torch

own = False

DEV = "cuda"
LATENT, ROW = 512, 576
FP8_ROW = 656
PAGE = 64
SCALE = ROW ** -0.5


def listed():
    return [
        # one sequence verifies 8 drafted tokens over a short context: latency
        {"name": "tree one sequence", "op": "tree", "seqs": 1, "context": 1000, "drafted": 8, "heads": 8, "format": "bf16", "ragged": False},
        # a decode batch of 32 sequences, trees of 16 tokens, 8 heads of a rank
        {"name": "tree batch", "op": "tree", "seqs": 32, "context": 16384, "drafted": 16, "heads": 8, "format": "bf16", "ragged": True},
        # an odd batch of small ragged trees over rows of 8 bits
        {"name": "tree odd fp8", "op": "tree", "seqs": 37, "context": 8191, "drafted": 5, "heads": 16, "format": "fp8", "ragged": True},
        # few sequences with very long contexts, one token each: the plain decode step
        {"name": "tree long one token", "op": "tree", "seqs": 4, "context": 65536, "drafted": 1, "heads": 16, "format": "bf16", "ragged": False},
        # wide trees at 64 heads
        {"name": "tree wide", "op": "tree", "seqs": 8, "context": 8192, "drafted": 64, "heads": 64, "format": "bf16", "ragged": False},
        # the weights of one short sequence: latency
        {"name": "weights one sequence", "op": "weights", "seqs": 1, "context": 1000, "drafted": 1, "heads": 8, "format": "bf16", "ragged": False},
        # the decode batch of above
        {"name": "weights batch", "op": "weights", "seqs": 32, "context": 16384, "drafted": 16, "heads": 8, "format": "bf16", "ragged": True},
        # the odd batch in rows of 8 bits
        {"name": "weights odd fp8", "op": "weights", "seqs": 37, "context": 8191, "drafted": 5, "heads": 16, "format": "fp8", "ragged": True},
        # a prompt's last 64 tokens at 64 heads, whose weights choose what is kept of the prompt
        {"name": "weights wide", "op": "weights", "seqs": 8, "context": 8192, "drafted": 64, "heads": 64, "format": "bf16", "ragged": False},
        # one short sequence cut to half: latency
        {"name": "evict one sequence", "op": "evict", "seqs": 1, "context": 1000, "budget": 500, "sinks": 4, "recent": 64, "format": "bf16", "ragged": False},
        # a batch of long prompts cut to 4096 rows each
        {"name": "evict batch", "op": "evict", "seqs": 32, "context": 16384, "budget": 4096, "sinks": 4, "recent": 512, "format": "bf16", "ragged": True},
        # 128 sequences in rows of 8 bits, an odd budget
        {"name": "evict fp8", "op": "evict", "seqs": 128, "context": 8191, "budget": 2001, "sinks": 0, "recent": 128, "format": "fp8", "ragged": True},
    ]


def _spread(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(max(low, high))))))


def draw(rng):
    op = rng.choice(["tree", "weights", "evict"])
    fmt = rng.choice(["bf16", "fp8"])
    if op == "evict":
        seqs = _spread(rng, 1, 128)
        context = _spread(rng, 256, min(65536, 32 * 16384 // seqs))
        budget = _spread(rng, 64, context)
        return {"op": op, "seqs": seqs, "context": context, "budget": budget, "sinks": rng.choice([0, 4]),
                "recent": rng.randrange(1 + budget // 4), "format": fmt, "ragged": rng.random() < 0.7}
    heads, drafted, seqs = rng.choice([8, 16, 32, 64]), _spread(rng, 1, 64), _spread(rng, 1, 64)
    most = min(65536, 32 * 16384 // seqs, 8 * 8192 * 64 * 64 // (seqs * heads * drafted))
    return {"op": op, "seqs": seqs, "context": _spread(rng, 256, most), "drafted": drafted, "heads": heads, "format": fmt,
            "ragged": rng.random() < 0.7}


# ------------------------------------------------------------------------------------- inputs

def _parts(case):
    """0 .. 1 for each sequence: how much of the range its sizes leave out."""
    return [(i * 0.61803398875) % 1.0 if case["ragged"] else 0.0 for i in range(case["seqs"])]


def _lengths(case):
    """Cached rows of each sequence, between half the context and all of it."""
    return [case["context"] - int(x * (case["context"] // 2)) for x in _parts(case)]


def _drafted(case):
    """Drafted tokens of each sequence, between one and all."""
    return [case["drafted"] - int((1 - x) * (case["drafted"] - 1)) if case["ragged"] else case["drafted"] for x in _parts(case)]


def _pack_fp8(x):
    """Rows [n, 576] as cache rows of 656 bytes."""
    tiles = x[:, :LATENT].float().reshape(-1, 4, 128)
    amax = tiles.abs().amax(dim=2, keepdim=True)
    scale = torch.where(amax > 0, amax / 448.0, torch.ones_like(amax))
    rows = torch.empty((x.shape[0], FP8_ROW), dtype=torch.uint8, device=x.device)
    rows[:, :LATENT] = (tiles / scale).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).reshape(-1, LATENT).view(torch.uint8)
    rows[:, LATENT:528] = scale.reshape(-1, 4).view(torch.uint8)
    rows[:, 528:] = x[:, LATENT:].to(torch.bfloat16).contiguous().view(torch.uint8)
    return rows


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)

    def ints(values):
        return torch.tensor(values, dtype=torch.int32, device=DEV)

    B, lengths = case["seqs"], _lengths(case)
    drafted = _drafted(case) if case["op"] != "evict" else [0] * B
    blocks = max(-(-(n + d) // PAGE) for n, d in zip(lengths, drafted))
    new_blocks = -(-case["budget"] // PAGE) if case["op"] == "evict" else 0
    old = B * blocks
    pages = old + B * new_blocks
    cache = torch.randn(pages * PAGE, ROW, generator=g, device=DEV, dtype=torch.bfloat16) * 0.5
    if case["format"] == "fp8":
        cache = torch.cat([_pack_fp8(part) for part in cache.split(65536)])
    state = {"case": dict(case), "cache": cache, "host_lengths": lengths, "host_drafted": drafted, "lengths": ints(lengths),
             "tables": torch.randperm(old, generator=g, device=DEV).int().reshape(B, blocks)}
    if case["op"] != "tree":  # what earlier steps gathered
        state["weights"] = torch.empty((B, blocks * PAGE), device=DEV).exponential_(1.0, generator=g)
    if case["op"] == "evict":
        cache[old * PAGE:] = 0
        state.update(new_tables=(old + torch.randperm(B * new_blocks, generator=g, device=DEV)).int().reshape(B, new_blocks), first_new=old * PAGE)
        return state
    starts = [0]
    for d in drafted:
        starts.append(starts[-1] + d)
    T, most = starts[-1], case["drafted"]
    # random trees: token j hangs on one of the eight before it, and sees itself and its ancestors
    parent = [(torch.rand(B, generator=g, device=DEV) * min(j, 8)).long() + max(0, j - 8) for j in range(most)]
    sees = torch.zeros((B, most, -(-most // 32) * 32), dtype=torch.bool, device=DEV)
    every = torch.arange(B, device=DEV)
    for j in range(most):
        if j:
            sees[:, j] = sees[every, parent[j]]
        sees[:, j, j] = True
    bits = (sees.reshape(B, most, -1, 32).long() << torch.arange(32, device=DEV)).sum(dim=3)
    bits = torch.where(bits >= 2 ** 31, bits - 2 ** 32, bits).int()
    seq, index = _tokens(state)
    state.update(starts=ints(starts), mask=bits[seq, index].contiguous(),
                 q=torch.randn(T, case["heads"], ROW, generator=g, device=DEV, dtype=torch.bfloat16))
    if case["op"] == "weights":
        state.update(lse=_plain_tree(state)[1], decay=0.95)
    return state


# ------------------------------------------------------------------------------------- the plain forms

def _tokens(s):
    """Sequence and index in its tree of every token."""
    counts = torch.tensor(s["host_drafted"], device=DEV)
    T = sum(s["host_drafted"])
    seq = torch.repeat_interleave(torch.arange(len(counts), device=DEV), counts, output_size=T)
    return seq, torch.arange(T, device=DEV) - (counts.cumsum(0) - counts)[seq]


def _rows(s, slots, dtype):
    """The values of cache rows."""
    rows = s["cache"][slots]
    if s["case"]["format"] == "bf16":
        return rows.to(dtype)
    latent = rows[..., :LATENT].view(torch.float8_e4m3fn).to(dtype).unflatten(-1, (4, 128))
    scale = rows[..., LATENT:528].contiguous().view(torch.float32).to(dtype)
    rope = rows[..., 528:].contiguous().view(torch.bfloat16).to(dtype)
    return torch.cat([(latent * scale[..., None]).flatten(-2).to(torch.bfloat16).to(dtype), rope], dim=-1)


def _plain_logits(s):
    """Logits [B, tokens, heads, keys] of every sequence's tokens, -inf where a key takes no part, and the rows."""
    c = s["case"]
    B, h, most = c["seqs"], c["heads"], c["drafted"]
    keys = max(n + d for n, d in zip(s["host_lengths"], s["host_drafted"]))
    at = torch.arange(keys, device=DEV)
    rows = _rows(s, s["tables"][:, at // PAGE].long() * PAGE + at % PAGE, torch.float32)
    seq, index = _tokens(s)
    q = torch.zeros((B, most, h, ROW), device=DEV)
    q[seq, index] = s["q"].float()
    words = torch.zeros((B, most, s["mask"].shape[1]), dtype=torch.int32, device=DEV)
    words[seq, index] = s["mask"]
    node = at - s["lengths"][:, None]  # [B, keys]: which drafted token a key is
    word = (node >> 5).clamp(0, words.shape[2] - 1).long()
    seen = (words.gather(2, word[:, None].expand(-1, most, -1)) >> (node & 31)[:, None]) & 1
    drafted = torch.tensor(s["host_drafted"], device=DEV)[:, None, None]
    sees = (node < 0)[:, None] | ((seen == 1) & (node[:, None] < drafted))
    logits = torch.matmul(q.reshape(B, most * h, ROW), rows.transpose(1, 2)).mul_(SCALE).reshape(B, most, h, keys)
    return logits.masked_fill_(~sees[:, :, None], -math.inf), rows


def _plain_tree(s):
    logits, rows = _plain_logits(s)
    B, most, h, _ = logits.shape
    top = logits.amax(dim=3, keepdim=True)
    p = torch.exp(logits.sub_(top.clamp(min=-1e30)))
    total = p.sum(dim=3, keepdim=True)
    out = torch.matmul(p.reshape(B, most * h, -1), rows[..., :LATENT]).reshape(B, most, h, LATENT) / total
    seq, index = _tokens(s)
    return out[seq, index].to(torch.bfloat16), (top + torch.log(total))[seq, index, :, 0]


def _plain_weights(s):
    logits, _ = _plain_logits(s)
    B, most, h, keys = logits.shape
    seq, index = _tokens(s)
    lse = torch.full((B, most, h), math.inf, device=DEV)
    lse[seq, index] = s["lse"]
    out = torch.where(torch.arange(s["weights"].shape[1], device=DEV) < s["lengths"][:, None], s["decay"] * s["weights"], 0.0)
    out[:, :keys] += torch.exp(logits.sub_(lse[..., None])).reshape(B, most * h, keys).sum(dim=1)
    return out


def _plain_evict(s):
    c = s["case"]
    B, budget, width = c["seqs"], c["budget"], s["weights"].shape[1]
    n = s["lengths"][:, None]
    at = torch.arange(width, device=DEV)
    rank = torch.where((at < c["sinks"]) | (at >= n - c["recent"]), math.inf, s["weights"])
    order = torch.sort(torch.where(at < n, rank, -1.0), dim=1, descending=True, stable=True).indices[:, :budget]
    place = torch.arange(budget, device=DEV)
    if budget > width:
        order = torch.nn.functional.pad(order, (0, budget - width))
    some = n.clamp(max=budget)
    kept = torch.sort(torch.where(place < some, order, width), dim=1).values
    live = place < some
    kept = torch.where(live, kept, -1)
    new_weights = torch.zeros((B, s["new_tables"].shape[1] * PAGE), device=DEV)
    new_weights[:, :budget] = torch.where(live, s["weights"].gather(1, kept.clamp(min=0)), 0.0)
    source = s["tables"].long().gather(1, kept.clamp(min=0) // PAGE) * PAGE + kept % PAGE
    target = s["new_tables"].long()[:, place // PAGE] * PAGE + place % PAGE
    s["cache"][target[live]] = s["cache"][source[live]]
    return kept.int(), some[:, 0].int(), new_weights, s["cache"][s["first_new"]:]


def run(state):
    s, c = state, state["case"]
    if own:
        import token_sparse_mla_gb300 as smla
        if c["op"] == "tree":
            return smla.sparse_mla_tree(s["q"], s["cache"], s["tables"], s["lengths"], s["starts"], SCALE, mask=s["mask"], kv_format=c["format"])
        if c["op"] == "weights":
            return smla.sparse_mla_weights(s["q"], s["cache"], s["tables"], s["lengths"], s["starts"], s["lse"], SCALE, mask=s["mask"],
                                           weights=s["weights"], decay=s["decay"], kv_format=c["format"])
        kept, lengths, weights = smla.sparse_mla_evict(s["cache"], s["tables"], s["lengths"], s["weights"], s["new_tables"], c["budget"],
                                                       sinks=c["sinks"], recent=c["recent"], kv_format=c["format"])
        return kept, lengths, weights, s["cache"][s["first_new"]:]
    if c["op"] == "tree":
        return _plain_tree(s)
    if c["op"] == "weights":
        return _plain_weights(s)
    return _plain_evict(s)


def work(case):
    row = 2 * ROW if case["format"] == "bf16" else FP8_ROW
    lengths = _lengths(case)
    B, context = case["seqs"], sum(lengths)
    if case["op"] == "evict":
        kept = sum(min(n, case["budget"]) for n in lengths)
        return {"bytes": 2 * kept * row + 4 * (context + kept + B * (case["budget"] + 2 + -(-case["budget"] // PAGE) * PAGE)), "flops": context}
    drafted, h = _drafted(case), case["heads"]
    T, keys = sum(drafted), context + sum(drafted)
    pairs = sum(d * h * (n + d) for n, d in zip(lengths, drafted))
    small = T * 4 * -(-case["drafted"] // 32) + 4 * (keys // PAGE + 3 * B)
    if case["op"] == "tree":
        return {"bytes": keys * row + T * h * (2 * ROW + 2 * LATENT + 4) + small, "flops": 2 * pairs * (ROW + LATENT)}
    return {"bytes": keys * (row + 4) + 4 * context + T * h * (2 * ROW + 4) + small, "flops": 2 * pairs * ROW}


# ------------------------------------------------------------------------------------- 64 bits

def _exact_sequence(s, b, first):
    """One sequence: its rows, and for every token a list of which of them it sees, in 64 bits."""
    n, d = s["host_lengths"][b], s["host_drafted"][b]
    table = s["tables"][b].long()
    rows = _rows(s, (table[:, None] * PAGE + torch.arange(PAGE, device=DEV)).flatten()[:n + d], torch.float64)
    words = s["mask"][first:first + d].long()
    bits = (words[:, :, None] >> torch.arange(32, device=DEV) & 1).flatten(1)[:, :d].bool()
    return rows, torch.cat([torch.ones((d, n), dtype=torch.bool, device=DEV), bits], dim=1)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "evict":
        width = s["new_tables"].shape[1] * PAGE
        kept = torch.full((case["seqs"], case["budget"]), -1, dtype=torch.int32)
        weights = torch.zeros((case["seqs"], width), dtype=torch.float64)
        for b, n in enumerate(s["host_lengths"]):
            w = s["weights"][b, :n].double().cpu()
            value = w.tolist()
            always = [i for i in range(n) if i < case["sinks"] or i >= n - case["recent"]]
            held = set(always)
            rest = sorted((i for i in range(n) if i not in held), key=lambda i: (-value[i], i)) if n > case["budget"] else []
            chosen = sorted(always + rest[:case["budget"] - len(always)]) if n > case["budget"] else list(range(n))
            kept[b, :len(chosen)] = torch.tensor(chosen, dtype=torch.int32)
            weights[b, :len(chosen)] = w[chosen]
            target = s["new_tables"][b].long().repeat_interleave(PAGE) * PAGE + torch.arange(width, device=DEV) % PAGE
            at = torch.tensor(chosen, device=DEV)
            s["cache"][target[:len(chosen)]] = s["cache"][s["tables"][b].long()[at // PAGE] * PAGE + at % PAGE]
        return kept, torch.tensor([min(n, case["budget"]) for n in s["host_lengths"]], dtype=torch.int32), weights, s["cache"][s["first_new"]:].clone()
    T, h = s["q"].shape[:2]
    first = 0
    out = torch.empty((T, h, LATENT), dtype=torch.float64, device=DEV)
    lse = torch.empty((T, h), dtype=torch.float64, device=DEV)
    if case["op"] == "weights":
        gathered = s["weights"].double() * s["decay"]
    for b, d in enumerate(s["host_drafted"]):
        rows, sees = _exact_sequence(s, b, first)
        if case["op"] == "weights":
            gathered[b, s["host_lengths"][b]:] = 0
        for t in range(d):
            k = rows[sees[t]]
            logits = torch.einsum("hd,kd->hk", s["q"][first + t].double(), k) * SCALE
            if case["op"] == "weights":
                at = sees[t].nonzero()[:, 0]
                gathered[b].index_add_(0, at, torch.exp(logits - s["lse"][first + t].double()[:, None]).sum(dim=0))
            else:
                lse[first + t] = torch.logsumexp(logits, dim=1)
                out[first + t] = torch.einsum("hk,kd->hd", torch.softmax(logits, dim=1), k[:, :LATENT])
        first += d
    return gathered if case["op"] == "weights" else (out, lse)
