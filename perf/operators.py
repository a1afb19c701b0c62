"""The operators of a served step over a block-paged 8-bit KV cache, as they are measured.

  plan       block tables, slot map, positions and lengths of a step from request lengths
  append     new K/V rows into the 8-bit blocks, one scale per block and KV head
  attention  queries of many requests (one new token, several, or a prompt chunk each) over such a cache
  rules      repetition / presence / frequency penalties, logit biases and grammar masks

``run`` computes them in plain torch operations, or, where ``own`` is true, with this repository's operators.  The shapes
are those of the 3.7B model (32 query heads over 8 KV heads of 128, vocabulary 250624) and of the medium test model (8
over 2 heads of 64); block sizes 16 to 128 are the usual ones of paged caches.

The 8-bit codes of int8 blocks are returned as they are, next to their scales: both sides use the same IEEE operations
(maximum, division, round to nearest even), so the codes, and with the scales the values they stand for, have to be
equal.  Codes in E4M3 are returned as float8 tensors, next to their scales.
"""
import math

import torch

own = False

QMAX = {"i8": 127.0, "f8": 448.0}
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
CODES = {"i8": torch.int8, "f8": torch.float8_e4m3fn}


# ---- cases -----------------------------------------------------------------------------------------------------------

def listed():
    return [
        # a decode step's tables: 64 running requests of any length, one new token each, some finished
        {"name": "plan decode 64", "op": "plan", "requests": 64, "lo": 1, "hi": 8192, "new": 1, "chunk_every": 0, "done_every": 16,
         "block": 16, "pad": 0},
        # a large mixed step: 1024 requests, every 64th a prompt chunk of 2048 tokens, padded for a captured graph
        {"name": "plan mixed 1024", "op": "plan", "requests": 1024, "lo": 1, "hi": 32768, "new": 2048, "chunk_every": 64,
         "done_every": 32, "block": 16, "pad": 1000},
        # the K/V rows of one decode step of 64 requests, most of them into half-filled blocks
        {"name": "append decode 64 i8", "op": "append", "requests": 64, "new": 1, "block": 16, "kv_heads": 8, "dim": 128,
         "cache": "i8", "type": "bf16"},
        # four prompt chunks of 2048 tokens, the rows taken out of packed q|k|v rows
        {"name": "append prompt 8192 f8", "op": "append", "requests": 4, "new": 2048, "block": 32, "kv_heads": 8, "dim": 128,
         "cache": "f8", "type": "f16"},
        # one conversation of moderate length: latency counts
        {"name": "attend 1 x 1000 i8", "op": "attention", "requests": 1, "lo": 1000, "hi": 1000, "new": 1, "chunk_every": 1,
         "block": 16, "heads": 32, "kv_heads": 8, "dim": 128, "cache": "i8", "type": "bf16"},
        # the batch of the batched-decode benchmark
        {"name": "attend 16 x 8192 i8", "op": "attention", "requests": 16, "lo": 8192, "hi": 8192, "new": 1, "chunk_every": 1,
         "block": 16, "heads": 32, "kv_heads": 8, "dim": 128, "cache": "i8", "type": "bf16"},
        # many requests of very different lengths, E4M3 blocks of 64
        {"name": "attend 48 ragged f8", "op": "attention", "requests": 48, "lo": 1, "hi": 32768, "new": 1, "chunk_every": 1,
         "block": 64, "heads": 32, "kv_heads": 8, "dim": 128, "cache": "f8", "type": "f16"},
        # a prompt chunk of 2048 tokens behind 8192 cached ones
        {"name": "attend chunk 2048+8192 i8", "op": "attention", "requests": 1, "lo": 8192, "hi": 8192, "new": 2048,
         "chunk_every": 1, "block": 16, "heads": 32, "kv_heads": 8, "dim": 128, "cache": "i8", "type": "f16"},
        # a mixed step of the medium model: every fourth request a prompt chunk, the others one token each
        {"name": "attend mixed 12 d64 f8", "op": "attention", "requests": 12, "lo": 37, "hi": 5000, "new": 509, "chunk_every": 4,
         "block": 32, "heads": 8, "kv_heads": 2, "dim": 64, "cache": "f8", "type": "bf16"},
        # one conversation under a grammar
        {"name": "rules 1 row", "op": "rules", "rows": 1, "vocab": 250624, "history": 600, "bias": 20, "masks": 1, "allowed": 0.02},
        # a full batch: long histories, a few grammars shared by the rows, biases
        {"name": "rules 64 rows", "op": "rules", "rows": 64, "vocab": 250624, "history": 8192, "bias": 300, "masks": 4,
         "allowed": 0.5},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["plan", "append", "attention", "attention", "rules"])
    if op == "plan":
        return {"op": op, "requests": _log(rng, 1, 1024), "lo": 1, "hi": _log(rng, 16, 32768), "new": _log(rng, 1, 2048),
                "chunk_every": rng.choice([0, 32, 64]), "done_every": rng.choice([0, 3, 10, 32]), "block": rng.choice([16, 32, 64, 128]),
                "pad": rng.choice([0, 77])}
    if op == "append":
        requests = _log(rng, 1, 256)
        return {"op": op, "requests": requests, "new": _log(rng, 1, max(1, 8192 // requests)), "block": rng.choice([16, 32, 64, 128]),
                "kv_heads": rng.choice([1, 2, 8]), "dim": rng.choice([64, 128]), "cache": rng.choice(["i8", "f8"]),
                "type": rng.choice(["bf16", "f16"])}
    if op == "attention":
        requests = _log(rng, 1, 64)
        rep = rng.choice([1, 2, 4, 8])
        kv_heads = rng.choice([2, 4, 8])
        chunk = rng.random() < 0.4
        hi = _log(rng, 2, 8192 if chunk else 32768)
        return {"op": op, "requests": min(requests, 8) if chunk else requests, "lo": _log(rng, 1, hi), "hi": hi,
                "new": _log(rng, 2, 1024) if chunk else rng.choice([1, 1, 2, 5]), "chunk_every": rng.choice([2, 4]) if chunk else 1,
                "block": rng.choice([16, 32, 64, 128]), "heads": kv_heads * rep, "kv_heads": kv_heads, "dim": rng.choice([64, 128]),
                "cache": rng.choice(["i8", "f8"]), "type": rng.choice(["bf16", "f16"])}
    return {"op": op, "rows": _log(rng, 1, 64), "vocab": rng.choice([512, 1000, 32001, 128256, 250624]), "history": _log(rng, 1, 8192),
            "bias": rng.choice([0, 7, 300]), "masks": rng.choice([0, 1, 4]), "allowed": rng.choice([0.001, 0.5, 0.99])}


def _spread(n, lo, hi):
    """n lengths spread evenly over the logarithm of [lo, hi]."""
    return [int(round(lo * (hi / lo) ** (i / max(1, n - 1)))) for i in range(n)]


def _lengths(case):
    """(cached, new) of every request, in an order that the seed shuffles; new = -1: the request is finished."""
    every, done = case["chunk_every"], case.get("done_every", 0)
    got = []
    for i, cached in enumerate(_spread(case["requests"], case["lo"], case["hi"])):
        new = case["new"] if every and i % every == 0 else 1
        got.append((cached, -1 if done and i % done == done - 1 else new))
    return got


def work(case):
    if case["op"] == "plan":
        n, b = _lengths(case), case["block"]
        tokens = sum(max(f, 0) for _, f in n)
        blocks = sum(-(-(c + f) // b) - -(-c // b) for c, f in n if f > 0) + sum(-(-c // b) for c, f in n if f < 0)
        # lengths read and written, blocks moved between the stack and the tables, a slot and a position per token
        return {"bytes": 4 * (4 * len(n) + 2 * blocks + 2 * (tokens + case["pad"])), "flops": 0}
    if case["op"] == "append":
        rows = case["requests"] * case["new"] * case["kv_heads"] * 2
        return {"bytes": rows * case["dim"] * 3, "flops": rows * case["dim"] * 3}
    if case["op"] == "attention":
        n, d, h, g = _lengths(case), case["dim"], case["heads"], case["kv_heads"]
        keys = sum(c + f for c, f in n)
        blocks = sum(-(-(c + f) // case["block"]) for c, f in n)
        pairs = sum(f * c + f * (f + 1) // 2 for c, f in n)
        return {"bytes": keys * g * d * 2 + blocks * (8 * g + 4) + sum(f for _, f in n) * h * d * 4, "flops": 4 * pairs * h * d}
    rows, v = case["rows"], case["vocab"]
    return {"bytes": rows * v * 8 + case["masks"] * -(-v // 32) * 4 + rows * (case["history"] * 4 + case["bias"] * 8),
            "flops": rows * v}


# ---- inputs ----------------------------------------------------------------------------------------------------------

def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return {"plan": _prepare_plan, "append": _prepare_append, "attention": _prepare_attention, "rules": _prepare_rules}[case["op"]](case, gen)


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _shuffled(pairs, gen):
    order = torch.randperm(len(pairs), device="cuda", generator=gen)
    return _ints([a for a, _ in pairs])[order], _ints([b for _, b in pairs])[order]


def _tables(owned, stride, pool, gen):
    """A table of `stride` columns whose row r names owned[r] blocks of a pool in random order (the rest -1), and the other blocks."""
    perm = torch.randperm(pool, device="cuda", generator=gen).int()
    first = torch.cumsum(owned, 0) - owned
    col = torch.arange(stride, device="cuda")
    at = first[:, None] + col
    table = torch.where(col < owned[:, None], perm[at.clamp(max=pool - 1).long()], -1)
    return table.int().contiguous(), perm[int(owned.sum()):]


def _prepare_plan(case, gen):
    b = case["block"]
    n = _lengths(case)
    cached, fresh = _shuffled(n, gen)
    stride = max(-(-(c + max(f, 0)) // b) for c, f in n) + 3
    owned = (cached + b - 1) // b
    need = sum(-(-(c + f) // b) - -(-c // b) for c, f in n if f > 0)
    pool = int(owned.sum()) + need + 11
    table, free = _tables(owned, stride, pool, gen)
    stack = torch.full((pool,), -1, dtype=torch.int32, device="cuda")
    stack[:free.numel()] = free
    tokens = sum(max(f, 0) for _, f in n) + case["pad"]
    new = lambda m: torch.zeros(m, dtype=torch.int32, device="cuda")  # noqa: E731
    return {"op": "plan", "block": b, "cached": cached, "fresh": fresh, "table": table, "free": stack, "free_count": _ints([free.numel()]),
            "free_count_out": new(1), "kv_len": new(len(n)), "cu_new": new(len(n) + 1), "slots": new(tokens), "positions": new(tokens),
            "status": new(4)}


def _codes(shape, cache, gen):
    x = torch.randn(shape, device="cuda", generator=gen)
    return (x * 42).round_().clamp_(-127, 127).to(torch.int8) if cache == "i8" else (x * 110).clamp_(-448, 448).to(torch.float8_e4m3fn)


def _pool(case, blocks, gen):
    g, b, d = case["kv_heads"], case["block"], case["dim"]
    unit = 0.024 if case["cache"] == "i8" else 0.009
    scale = lambda: (torch.randn(blocks, g, device="cuda", generator=gen) * 0.4).exp_() * unit  # noqa: E731
    return {"k": _codes((blocks, g, b, d), case["cache"], gen), "v": _codes((blocks, g, b, d), case["cache"], gen), "k_scale": scale(),
            "v_scale": scale()}


def _prepare_append(case, gen):
    r, n, b, g, d = case["requests"], case["new"], case["block"], case["kv_heads"], case["dim"]
    before = torch.randint(0, 4 * b, (r,), device="cuda", generator=gen, dtype=torch.int32)
    stride = -(-(4 * b + n) // b)
    table, _ = _tables(torch.full((r,), stride, dtype=torch.int32, device="cuda"), stride, r * stride + 5, gen)
    at = before[:, None] + torch.arange(n, device="cuda", dtype=torch.int32)
    slots = (table.gather(1, (at // b).long()) * b + at % b).int().reshape(-1)
    # rows of a packed q|k|v product: K and V are slices of it
    packed = torch.randn(r * n, 3 * g, d, device="cuda", generator=gen)
    packed *= (torch.randn(3 * g, 1, device="cuda", generator=gen) * 0.5).exp_()
    packed = packed.to(TYPES[case["type"]])
    return {"op": "append", "cache": case["cache"], "new_k": packed[:, g:2 * g], "new_v": packed[:, 2 * g:], "slots": slots,
            **_pool(case, r * stride + 5, gen)}


def _prepare_attention(case, gen):
    b = case["block"]
    n = _lengths(case)
    cached, fresh = _shuffled(n, gen)
    kv_len = cached + fresh
    owned = (kv_len + b - 1) // b
    stride = max(-(-(c + f) // b) for c, f in n)
    blocks = sum(-(-(c + f) // b) for c, f in n) + 7
    table, _ = _tables(owned, stride, blocks, gen)
    cu = torch.zeros(len(n) + 1, dtype=torch.int32, device="cuda")
    cu[1:] = torch.cumsum(fresh, 0)
    q = torch.randn(sum(f for _, f in n), case["heads"], case["dim"], device="cuda", generator=gen) * 1.5
    q = q.to(TYPES[case["type"]])
    return {"op": "attention", "cache": case["cache"], "q": q, "out": torch.zeros_like(q), "cu_q": cu, "kv_len": kv_len, "table": table,
            "max_q": max(f for _, f in n), "scale": case["dim"] ** -0.5, **_pool(case, blocks, gen)}


def _prepare_rules(case, gen):
    rows, v, h = case["rows"], case["vocab"], case["history"]
    rand = lambda *shape: torch.rand(*shape, device="cuda", generator=gen)  # noqa: E731
    logits = torch.randn(rows, v, device="cuda", generator=gen) * 3
    # token histories are skewed: a few ids come back often
    ids = (rand(rows, h) ** 3 * v).int().clamp_(max=v - 1)
    length = (h * (0.5 + 0.5 * rand(rows))).int().clamp_(min=1)
    length[0] = h
    s = {"op": "rules", "logits": logits, "out": torch.zeros_like(logits), "ids": ids, "ids_len": length, "prompt_len": (length * rand(rows)).int(),
         "repetition": 1 + 0.3 * rand(rows), "presence": 0.6 * rand(rows), "frequency": 0.2 * rand(rows), "bias": None, "mask": None,
         "mask_row": None}
    if case["bias"]:
        n = case["bias"]
        each = torch.randint(0, v, (rows, n), device="cuda", generator=gen, dtype=torch.int32)
        s["bias"] = (torch.arange(rows + 1, device="cuda", dtype=torch.int32) * n, each.reshape(-1),
                     torch.randn(rows * n, device="cuda", generator=gen) * 4)
    if case["masks"]:
        m, words = case["masks"], -(-v // 32)
        bits = rand(m, words * 32) < case["allowed"]
        s["mask"] = (bits.view(m, words, 32).long() << torch.arange(32, device="cuda")).sum(-1).to(torch.uint32).view(torch.int32)
        s["mask_row"] = torch.randint(-1 if rows > 1 else 0, m, (rows,), device="cuda", generator=gen, dtype=torch.int32)
    return s


# ---- one pass --------------------------------------------------------------------------------------------------------

def run(state):
    if own:
        return {"plan": _own_plan, "append": _own_append, "attention": _own_attention, "rules": _own_rules}[state["op"]](state)
    return {"plan": _plan, "append": _append, "attention": _attention, "rules": _rules}[state["op"]](state)


def _own_cache(s):
    """The handle that a program keeps for its pool."""
    if "handle" not in s:
        from dense_gqa_decoder_gb300 import k2
        s["handle"] = k2.PagedCache.of(s["k"], s["v"], s["k_scale"], s["v_scale"])
    return s["handle"]


def _own_plan(s):
    from dense_gqa_decoder_gb300 import k2
    k2.paged_plan(s["cached"], s["fresh"], s["table"], s["free"], s["free_count"], s["block"], kv_len=s["kv_len"], cu_new=s["cu_new"],
                  slots=s["slots"], positions=s["positions"], status=s["status"], free_count_out=s["free_count_out"])
    return [s[n] for n in ("table", "free", "free_count_out", "kv_len", "cu_new", "slots", "positions", "status")]


def _own_append(s):
    from dense_gqa_decoder_gb300 import k2
    k2.paged_append(_own_cache(s), s["new_k"], s["new_v"], s["slots"])
    return [s[n] for n in ("k", "v", "k_scale", "v_scale")]


def _own_attention(s):
    from dense_gqa_decoder_gb300 import k2
    cache = _own_cache(s)
    if "workspace" not in s:
        s["workspace"] = k2.paged_workspace()
    k2.paged_attention(cache, s["q"], s["out"], s["cu_q"], s["kv_len"], s["table"], s["max_q"], s["workspace"], scale=s["scale"])
    return s["out"]


def _own_rules(s):
    from dense_gqa_decoder_gb300 import k2
    k2.adjust_logits(s["logits"], s["out"], repetition=s["repetition"], presence=s["presence"], frequency=s["frequency"], ids=s["ids"],
                     ids_len=s["ids_len"], prompt_len=s["prompt_len"], bias=s["bias"], mask=s["mask"], mask_row=s["mask_row"])
    return s["out"]


def _plan(s):
    b, cached, fresh, table, free = s["block"], s["cached"].long(), s["fresh"].long(), s["table"], s["free"]
    dev = table.device
    live = fresh >= 0
    new = fresh.clamp(min=0)
    old = (cached + b - 1) // b
    total = (cached + new + b - 1) // b
    take, give = torch.where(live, total - old, 0), torch.where(live, 0, old)
    count = s["free_count"].long()
    # the stack with the finished requests' blocks on top
    cap = free.numel()
    col = torch.arange(table.shape[1], device=dev)
    at = torch.where(~live[:, None] & (col < old[:, None]), count + (torch.cumsum(give, 0) - give)[:, None] + col, cap)
    stack = torch.cat([free, free.new_zeros(1)])
    stack[at.reshape(-1)] = table.reshape(-1)
    top = count + give.sum()
    # the new blocks of each request, taken from the top
    fresh_col = live[:, None] & (col >= old[:, None]) & (col < total[:, None])
    k = (torch.cumsum(take, 0) - take)[:, None] + col - old[:, None]
    table.copy_(torch.where(fresh_col, stack[(top - 1 - k).clamp(0, cap)], table))
    left = top - take.sum()
    i = torch.arange(cap, device=dev)
    free.copy_(torch.where(i < left, stack[:cap], free))
    cu = torch.cat([new.new_zeros(1), torch.cumsum(new, 0)])
    t = torch.arange(s["slots"].numel(), device=dev)
    r = torch.searchsorted(cu[1:].contiguous(), t, right=True).clamp(max=cached.numel() - 1)
    pos = cached[r] + t - cu[r]
    inside = t < cu[-1]
    pos = torch.where(inside, pos, 0)
    slot = torch.where(inside, table[r, pos // b].long() * b + pos % b, -1)
    status = torch.stack([cu[-1], take.sum(), give.sum(), cu.new_zeros(())])
    return [x.int() for x in (table, free, left, torch.where(live, cached + new, 0), cu, slot, pos, status)]


def _quantise(x, scale, cache):
    """Codes of x under `scale` (broadcast): nearest, ties to even; NaN and everything under a zero scale become 0."""
    y = torch.where(scale > 0, x / scale, 0.0)
    y = torch.where(torch.isnan(y), 0.0, y).clamp(-QMAX[cache], QMAX[cache])
    return torch.round(y).to(torch.int8) if cache == "i8" else y.to(torch.float8_e4m3fn)


def _append_one(codes, scale, rows, slots, cache):
    n_blocks, g, b, _ = codes.shape
    rows = rows.float()
    block, at = slots // b, slots % b
    # dividing by a tensor on the device is a division; by a Python number it would be a product with the reciprocal
    qmax = torch.full((), QMAX[cache], device=rows.device)
    a = torch.where(torch.isfinite(rows), rows.abs(), 0.0).amax(-1)
    a = torch.zeros(n_blocks, g, device=rows.device).scatter_reduce_(0, block[:, None].expand(-1, g), a, "amax")
    start = torch.full((n_blocks,), b, device=rows.device).scatter_reduce_(0, block, at, "amin")
    old = torch.where((start > 0)[:, None], scale, 0.0)
    new = torch.maximum(old, a / qmax)
    ratio = torch.where(new > old, old / new, 1.0)
    raw = codes.view(torch.uint8)
    if block.numel() * b <= n_blocks * b:  # few rows: only their blocks
        prior = (torch.arange(b, device=rows.device) < start[block][:, None])[:, None, :, None]
        was = codes.view(torch.uint8)[block].view(codes.dtype)
        again = _quantise(was.float() * ratio[block][:, :, None, None], torch.ones((), device=rows.device), cache)
        raw[block] = torch.where(prior, again.view(torch.uint8), was.view(torch.uint8))
    else:
        touched = (start < b)[:, None] & (torch.arange(b, device=rows.device) < start[:, None])
        again = _quantise(codes.float() * ratio[:, :, None, None], torch.ones((), device=rows.device), cache)
        raw.copy_(torch.where(touched[:, None, :, None], again.view(torch.uint8), raw))
    scale.copy_(torch.where((start < b)[:, None], new, scale))
    raw[block, :, at] = _quantise(rows, scale[block][:, :, None], cache).view(torch.uint8)


def _append(s):
    slots = s["slots"].long()
    _append_one(s["k"], s["k_scale"], s["new_k"], slots, s["cache"])
    _append_one(s["v"], s["v_scale"], s["new_v"], slots, s["cache"])
    return [s[n] for n in ("k", "v", "k_scale", "v_scale")]


def _rows_of(codes, scale, table):
    """[requests, KV heads, keys, dim] values in fp32."""
    n = table.clamp(min=0).long()
    x = codes.view(torch.uint8)[n].view(codes.dtype).float() * scale[n][..., None, None]
    r, nb, g, b, d = x.shape
    return x.permute(0, 2, 1, 3, 4).reshape(r, g, nb * b, d)


def _attention(s):
    q, table, kv_len, cu = s["q"], s["table"], s["kv_len"].long(), s["cu_q"].long()
    r, g = table.shape[0], s["k"].shape[1]
    (t, h, d), m = q.shape, s["max_q"]
    k = _rows_of(s["k"], s["k_scale"], table)
    keys = torch.arange(k.shape[2], device=q.device)
    scored = torch.arange(m, device=q.device)
    count = cu[1:] - cu[:-1]
    row = (cu[:-1, None] + scored).clamp(max=t - 1)
    x = q[row].float().view(r, m, g, h // g, d).permute(0, 2, 3, 1, 4).reshape(r, g, -1, d)
    w = torch.matmul(x * s["scale"], k.transpose(2, 3)).view(r, g, h // g, m, -1)
    del k
    last = kv_len[:, None] - count[:, None] + scored
    seen = keys <= last[:, :, None]
    w = torch.where(seen[:, None, None], w, -math.inf)
    top = w.amax(-1, keepdim=True)
    w = torch.exp(w - torch.where(top > -math.inf, top, 0.0))
    total = w.sum(-1, keepdim=True)
    v = _rows_of(s["v"], s["v_scale"], table)
    v = torch.where((keys < kv_len[:, None])[:, None, :, None], v, 0.0)
    o = torch.matmul(w.view(r, g, -1, w.shape[-1]), v).view(r, g, h // g, m, d)
    o = torch.where(total > 0, o / total, 0.0).permute(0, 3, 1, 2, 4).reshape(r, m, h, d)
    return torch.zeros_like(q).index_put_((row[scored < count[:, None]],), o[scored < count[:, None]].to(q.dtype))


def _rules(s):
    logits, ids, v = s["logits"], s["ids"].long(), s["logits"].shape[1]
    at = torch.arange(ids.shape[1], device=ids.device)
    inside = at < s["ids_len"][:, None]
    answered = (inside & (at >= s["prompt_len"][:, None])).float()
    count = torch.zeros_like(logits).scatter_add_(1, ids, answered)
    seen = torch.zeros_like(logits).scatter_add_(1, ids, inside.float()) > 0
    rep = s["repetition"][:, None]
    x = torch.where(seen, torch.where(logits > 0, logits / rep, logits * rep), logits)
    x = torch.where(count > 0, x - s["frequency"][:, None] * count - s["presence"][:, None], x)
    if s["bias"] is not None:
        offset, bias_ids, values = s["bias"]
        rows = torch.searchsorted(offset[1:].contiguous(), torch.arange(values.numel(), device=ids.device, dtype=torch.int32), right=True)
        x = x.index_put_((rows, bias_ids.long()), values, accumulate=True)
    if s["mask"] is not None:
        bits = (s["mask"][..., None] >> torch.arange(32, device=ids.device, dtype=torch.int32)) & 1
        allowed = bits.reshape(s["mask"].shape[0], -1)[:, :v] > 0
        x = torch.where(allowed[s["mask_row"].clamp(min=0).long()] | (s["mask_row"] < 0)[:, None], x, -math.inf)
    return x


# ---- in 64 bits ------------------------------------------------------------------------------------------------------

def exact(case, seed):
    if case["op"] == "plan":
        return None  # whole numbers
    s = prepare(case, seed)
    if case["op"] == "append":
        return [None, None] + [_exact_scale(s[a], s["new_" + a[0]], s["slots"], s["k"].shape[2], QMAX[case["cache"]])
                               for a in ("k_scale", "v_scale")]
    return _exact_attention(s, case["block"]) if case["op"] == "attention" else _exact_rules(s)


def _exact_scale(scale, rows, slots, block, qmax):
    """Largest magnitude of a block's rows over the largest code; a block entered at its first row starts afresh."""
    got = scale.double()
    first = {}
    for i, slot in enumerate(slots.tolist()):
        first.setdefault(slot // block, []).append((i, slot % block))
    top = rows.double().abs().amax(-1) / qmax
    for at, members in first.items():
        m = top[[i for i, _ in members]].amax(0)
        got[at] = m if min(o for _, o in members) == 0 else torch.maximum(got[at], m)
    return got


def _exact_attention(s, block):
    q, cu = s["q"], s["cu_q"].tolist()
    g = s["k"].shape[1]
    rep = q.shape[1] // g
    out = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    for r, n in enumerate(s["kv_len"].tolist()):
        own_blocks = s["table"][r, :-(-n // block)].long()
        values = []
        for name in ("k", "v"):
            x = s[name].view(torch.uint8)[own_blocks].view(s[name].dtype).double() * s[name + "_scale"].double()[own_blocks][:, :, None, None]
            values.append(x.transpose(0, 1).flatten(1, 2)[:, :n])
        k, v = values
        for lo in range(cu[r], cu[r + 1], 128):
            hi = min(lo + 128, cu[r + 1])
            behind = cu[r + 1] - torch.arange(lo, hi, device=q.device)  # 1 for the request's last query
            hidden = torch.arange(n, device=q.device) > (n - behind)[:, None]
            for j in range(g):
                x = q[lo:hi, j * rep:(j + 1) * rep].double() * s["scale"]
                w = torch.einsum("thd,kd->thk", x, k[j]).masked_fill(hidden[:, None], -math.inf)
                out[lo:hi, j * rep:(j + 1) * rep] = torch.einsum("thk,kd->thd", torch.softmax(w, -1), v[j])
    return out


def _exact_rules(s):
    out = s["logits"].double()
    v = out.shape[1]
    ids, length, prompt = s["ids"].tolist(), s["ids_len"].tolist(), s["prompt_len"].tolist()
    for r in range(out.shape[0]):
        mine = torch.tensor(ids[r][:length[r]], device=out.device)
        x, rep = out[r], s["repetition"][r].double()
        before = torch.unique(mine)
        x[before] = torch.where(x[before] > 0, x[before] / rep, x[before] * rep)
        again, times = torch.unique(mine[prompt[r]:], return_counts=True)
        x[again] -= s["frequency"][r].double() * times + s["presence"][r].double()
        if s["bias"] is not None:
            offset, bias_ids, values = s["bias"]
            lo, hi = int(offset[r]), int(offset[r + 1])
            x += torch.bincount(bias_ids[lo:hi].long(), weights=values[lo:hi].double(), minlength=v)
        if s["mask"] is not None and int(s["mask_row"][r]) >= 0:
            words = s["mask"][int(s["mask_row"][r])].long() & 0xFFFFFFFF
            token = torch.arange(v, device=out.device)
            x[(words[token // 32] >> (token % 32)) & 1 == 0] = -math.inf
    return out
