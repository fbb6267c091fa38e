"""The operators around the sparse attention, as cases to be measured: appending rows to the paged
latent cache, the query's way into the latent space, and attention over a prefix that a whole batch
shares.  Each has a plain form (elementary torch operations in 32 bits, rounded once), the call of
the library (`own`), and its definition in 64 bits (`exact`)."""

import math

import torch

own = False

DEV = "cuda"
LATENT, ROPE, ROW = 512, 64, 576
FP8_ROW = 656
PAGE = 64
MAX_POS = 65536
EPS = 1e-6


def listed():
    return [
        # one new token for each of 32 sequences, as a decode step appends them
        {"name": "append decode bf16", "op": "append", "tokens": 32, "format": "bf16", "norm": True,
         "interleaved": True, "chunk": False, "padded": 0, "pages": 512},
        # a captured decode step of 128 slots with 27 of them unused, rows of 8 bits
        {"name": "append decode fp8 padded", "op": "append", "tokens": 128, "format": "fp8", "norm": True,
         "interleaved": True, "chunk": False, "padded": 27, "pages": 512},
        # a prefill chunk of 16384 tokens
        {"name": "append chunk bf16", "op": "append", "tokens": 16384, "format": "bf16", "norm": True,
         "interleaved": True, "chunk": True, "padded": 0, "pages": 512},
        # the tokens of a mixed batch of 32768, rows of 8 bits, the latent normed before the call
        {"name": "append mixed fp8", "op": "append", "tokens": 32768, "format": "fp8", "norm": False,
         "interleaved": False, "chunk": True, "padded": 0, "pages": 1024},
        # the queries of a decode step: 32 tokens, 8 heads of a rank
        {"name": "q_up decode", "op": "q_up", "tokens": 32, "heads": 8, "nope": 128, "interleaved": True},
        # an odd number of tokens at 64 heads and a nope part of 192
        {"name": "q_up 1001 tokens", "op": "q_up", "tokens": 1001, "heads": 64, "nope": 192, "interleaved": False},
        # the queries of a prefill chunk: 16384 tokens at 64 heads
        {"name": "q_up chunk", "op": "q_up", "tokens": 16384, "heads": 64, "nope": 128, "interleaved": True},
        # one token, a short prefix that ends inside a page: latency
        {"name": "prefix one token", "op": "prefix", "tokens": 1, "heads": 16, "prefix": 1000, "format": "bf16"},
        # a decode batch of 32 sequences that share a prompt of 16384 tokens
        {"name": "prefix decode", "op": "prefix", "tokens": 32, "heads": 8, "prefix": 16384, "format": "bf16"},
        # an odd batch over a shared prompt in rows of 8 bits
        {"name": "prefix odd fp8", "op": "prefix", "tokens": 37, "heads": 16, "prefix": 8191, "format": "fp8"},
        # 128 sequences over a long shared document, 64 heads
        {"name": "prefix batch", "op": "prefix", "tokens": 128, "heads": 64, "prefix": 32768, "format": "bf16"},
        # 128 sequences over the longest document of an 8-bit cache
        {"name": "prefix long fp8", "op": "prefix", "tokens": 128, "heads": 8, "prefix": 65536, "format": "fp8"},
    ]


def _spread(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["append", "q_up", "prefix", "prefix"])
    if op == "append":
        tokens = _spread(rng, 1, 32768)
        chunk = tokens > 256 or rng.random() < 0.3
        return {"op": op, "tokens": tokens, "format": rng.choice(["bf16", "fp8"]), "norm": rng.random() < 0.7,
                "interleaved": rng.random() < 0.5, "chunk": chunk, "padded": rng.randrange(tokens) if rng.random() < 0.3 else 0,
                "pages": max(512, tokens // PAGE + 2)}
    if op == "q_up":
        heads = rng.choice([8, 16, 32, 64])
        return {"op": op, "tokens": _spread(rng, 1, 16384 * 64 // heads // 2), "heads": heads,
                "nope": rng.choice([128, 192, 256]), "interleaved": rng.random() < 0.5}
    heads = rng.choice([8, 16, 32, 64])
    tokens = _spread(rng, 1, 8192 // heads)
    return {"op": op, "tokens": tokens, "heads": heads, "prefix": _spread(rng, 64, min(65536, 8192 * 32768 // (tokens * heads))),
            "format": rng.choice(["bf16", "fp8"])}


# ------------------------------------------------------------------------------------- inputs

def _table(device):
    """cos and sin of position times frequency, angles in 64 bits."""
    freq = 10000.0 ** (-torch.arange(0, ROPE, 2, dtype=torch.float64, device=device) / ROPE)
    angle = torch.arange(MAX_POS, dtype=torch.float64, device=device)[:, None] * freq
    return torch.cat([angle.cos(), angle.sin()], dim=1).float().contiguous()


def _pack_fp8(x):
    """Rows [n, 576] in 32 bits as cache rows of 656 bytes."""
    tiles = x[:, :LATENT].reshape(-1, 4, 128)
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

    def randn(*shape, sd=0.5):
        return (torch.randn(*shape, generator=g, device=DEV) * sd).to(torch.bfloat16)

    op, T = case["op"], case["tokens"]
    state = {"case": dict(case)}
    if op == "append":
        pages = case["pages"]
        if case["chunk"]:  # consecutive positions of one sequence, from inside a page on
            first = int(torch.randint(0, PAGE, (1,), generator=g, device=DEV))
            table = torch.randperm(pages, generator=g, device=DEV)
            at = first + torch.arange(T, device=DEV)
            slots, positions = table[at // PAGE] * PAGE + at % PAGE, at
        else:  # one token each of T sequences
            slots = torch.randperm(pages, generator=g, device=DEV)[:T] * PAGE + torch.randint(0, PAGE, (T,), generator=g, device=DEV)
            positions = torch.randint(0, MAX_POS, (T,), generator=g, device=DEV)
        if case["padded"]:
            slots[T - case["padded"]:] = -1
        # the fused projection's output: latent, rotated part and the query's latent side by side
        fused = randn(T, ROW + 1536, sd=1.0)
        state.update(kv=fused[:, :ROW], slots=slots.int(), positions=positions.int(), table=_table(DEV),
                     weight=(1 + 0.1 * torch.randn(LATENT, generator=g, device=DEV)).to(torch.bfloat16) if case["norm"] else None,
                     cache=torch.zeros((pages * PAGE, ROW), dtype=torch.bfloat16, device=DEV) if case["format"] == "bf16"
                     else torch.zeros((pages * PAGE, FP8_ROW), dtype=torch.uint8, device=DEV))
    elif op == "q_up":
        h, nope = case["heads"], case["nope"]
        state.update(q=randn(T, h, nope + ROPE), w=randn(h, nope, LATENT, sd=nope ** -0.5),
                     positions=torch.randint(0, MAX_POS, (T,), generator=g, device=DEV).int(), table=_table(DEV))
    else:
        h, P = case["heads"], case["prefix"]
        used = -(-P // PAGE)
        pages = used + 16  # other sequences' pages lie between the prefix's
        cache = randn(pages * PAGE, ROW)
        state.update(q=randn(T, h, ROW), cache=cache if case["format"] == "bf16" else _pack_fp8(cache.float()),
                     pages=torch.randperm(pages, generator=g, device=DEV)[:used].int().contiguous(), scale=ROW ** -0.5)
    return state


# ------------------------------------------------------------------------------------- the plain forms

def _rotate(x, positions, table, interleaved):
    """Pairs of the last 64 values turned by their position's angles: (2i, 2i + 1), or (i, i + 32)."""
    cs = table[positions.long()]
    cos, sin = cs[:, :32], cs[:, 32:]
    while cos.dim() < x.dim():
        cos, sin = cos[:, None], sin[:, None]
    if interleaved:
        a, b = x[..., 0::2], x[..., 1::2]
        return torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)
    a, b = x[..., :32], x[..., 32:]
    return torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)


def _cache_outputs(cache, fmt):
    if fmt == "bf16":
        return [cache]
    return [cache[:, :LATENT].view(torch.float8_e4m3fn), cache[:, LATENT:528].view(torch.float32), cache[:, 528:].view(torch.bfloat16)]


def _plain_append(s):
    c, x = s["case"], s["kv"].float()
    latent = x[:, :LATENT]
    if s["weight"] is not None:
        latent = latent * torch.rsqrt((latent * latent).mean(dim=1, keepdim=True) + EPS) * s["weight"].float()
    row = torch.cat([latent, _rotate(x[:, LATENT:], s["positions"], s["table"], c["interleaved"])], dim=1)
    row = row.to(torch.bfloat16) if c["format"] == "bf16" else _pack_fp8(row)
    keep = s["slots"] >= 0
    s["cache"][s["slots"][keep].long()] = row[keep]


def _plain_q_up(s):
    q, nope = s["q"].float(), s["case"]["nope"]
    latent = torch.matmul(q[..., :nope].transpose(0, 1), s["w"].float()).transpose(0, 1)
    rope = _rotate(q[..., nope:], s["positions"], s["table"], s["case"]["interleaved"])
    return torch.cat([latent, rope], dim=-1).to(torch.bfloat16)


def _prefix_rows(s, dtype):
    P = s["case"]["prefix"]
    at = torch.arange(P, device=DEV)
    rows = s["cache"][s["pages"].long()[at // PAGE] * PAGE + at % PAGE]
    if s["case"]["format"] == "bf16":
        return rows.to(dtype)
    latent = rows[:, :LATENT].view(torch.float8_e4m3fn).to(dtype).reshape(P, 4, 128)
    scale = rows[:, LATENT:528].contiguous().view(torch.float32).to(dtype)
    rope = rows[:, 528:].contiguous().view(torch.bfloat16).to(dtype)
    return torch.cat([(latent * scale[:, :, None]).reshape(P, LATENT), rope], dim=1)


def _plain_prefix(s):
    T, h, _ = s["q"].shape
    rows = _prefix_rows(s, torch.float32)
    logits = torch.matmul(s["q"].reshape(T * h, ROW).float(), rows.t()) * s["scale"]
    top = logits.amax(dim=1, keepdim=True)
    p = torch.exp(logits - top)
    total = p.sum(dim=1, keepdim=True)
    out = torch.matmul(p, rows[:, :LATENT]) / total
    return out.to(torch.bfloat16).reshape(T, h, LATENT), (top + torch.log(total)).reshape(T, h)


def run(state):
    c = state["case"]
    if own:
        import token_sparse_mla_gb300 as smla
        if c["op"] == "append":
            smla.sparse_mla_append(state["kv"], state["positions"], state["slots"], state["cache"], state["table"],
                                   norm_weight=state["weight"], eps=EPS, interleaved=c["interleaved"], kv_format=c["format"])
            return _cache_outputs(state["cache"], c["format"])
        if c["op"] == "q_up":
            return smla.sparse_mla_q_up(state["q"], state["w"], state["positions"], state["table"], interleaved=c["interleaved"])
        return smla.sparse_mla_prefix(state["q"], state["cache"], state["pages"], c["prefix"], state["scale"], kv_format=c["format"])
    if c["op"] == "append":
        _plain_append(state)
        return _cache_outputs(state["cache"], c["format"])
    if c["op"] == "q_up":
        return _plain_q_up(state)
    return _plain_prefix(state)


def work(case):
    T = case["tokens"]
    if case["op"] == "append":
        rows = T - case["padded"]
        row = 1152 if case["format"] == "bf16" else FP8_ROW
        return {"bytes": rows * (1152 + row + 4 + 256) + 4 * T + (1024 if case["norm"] else 0), "flops": rows * (4 * LATENT + 3 * ROPE)}
    if case["op"] == "q_up":
        h, nope = case["heads"], case["nope"]
        return {"bytes": T * h * ((nope + ROPE) * 2 + 1152) + h * nope * 1024 + T * 260, "flops": T * h * (2 * LATENT * nope + 3 * ROPE)}
    h, P = case["heads"], case["prefix"]
    row = 1152 if case["format"] == "bf16" else FP8_ROW
    return {"bytes": T * h * (1152 + 1024 + 4) + P * row + 4 * -(-P // PAGE), "flops": 2 * T * h * P * (ROW + LATENT)}


# ------------------------------------------------------------------------------------- 64 bits

def _turn(x, positions, table, interleaved):
    """The rotation as products with complex numbers, in 64 bits."""
    z = torch.complex(table[positions.long(), :32].double(), table[positions.long(), 32:].double())
    z = z.reshape(z.shape[0], *([1] * (x.dim() - 2)), 32)
    pairs = x.double().unflatten(-1, (32, 2)) if interleaved else x.double().unflatten(-1, (2, 32)).transpose(-1, -2)
    turned = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * z)
    return (turned if interleaved else turned.transpose(-1, -2)).flatten(-2)


def _to_e4m3(x):
    """Nearest value of 4 bits of precision, exponents from -6 on, ties to even, at most 448."""
    size = x.abs()
    power = torch.floor(torch.log2(size.clamp(min=2.0 ** -60))).clamp(min=-6.0)
    step = torch.exp2(power - 3.0)
    return torch.sign(x) * (torch.round(size / step) * step).clamp(max=448.0)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "append":
        x = s["kv"].double()
        latent = x[:, :LATENT]
        if case["norm"]:
            latent = latent / (latent.pow(2).sum(dim=1, keepdim=True) / LATENT + EPS).sqrt() * s["weight"].double()
        rope = _turn(x[:, LATENT:], s["positions"], s["table"], case["interleaved"])
        n, real = s["cache"].shape[0], case["tokens"] - case["padded"]
        slots = s["slots"][:real].long()

        def placed(values):
            whole = torch.zeros((n, values.shape[1]), dtype=torch.float64, device=DEV)
            return whole.index_copy_(0, slots, values[:real])

        if case["format"] == "bf16":
            return [placed(torch.cat([latent, rope], dim=1))]
        tiles = latent.reshape(-1, 4, 128)
        scale = tiles.abs().amax(dim=2) / 448.0
        scale = torch.where(scale > 0, scale, torch.ones_like(scale))
        return [placed(_to_e4m3(tiles / scale[:, :, None]).reshape(-1, LATENT)), placed(scale), placed(rope)]
    if case["op"] == "q_up":
        nope = case["nope"]
        latent = torch.einsum("thd,hdn->thn", s["q"][..., :nope].double(), s["w"].double())
        return torch.cat([latent, _turn(s["q"][..., nope:], s["positions"], s["table"], case["interleaved"])], dim=-1)
    T, h, _ = s["q"].shape
    rows = _prefix_rows(s, torch.float64)
    q = s["q"].double().reshape(T * h, ROW)
    out = torch.empty((T * h, LATENT), dtype=torch.float64, device=DEV)
    lse = torch.empty(T * h, dtype=torch.float64, device=DEV)
    for r in range(0, T * h, 1024):
        logits = torch.einsum("rd,pd->rp", q[r:r + 1024], rows) * s["scale"]
        lse[r:r + 1024] = torch.logsumexp(logits, dim=1)
        out[r:r + 1024] = torch.einsum("rp,pd->rd", torch.softmax(logits, dim=1), rows[:, :LATENT])
    return out.reshape(T, h, LATENT), lse.reshape(T, h)
