"""Oracle of the operators over a block-paged 8-bit KV cache and of the logit rules.

TEST INFRASTRUCTURE ONLY: imported by ``tests/`` alone; no code shared with the
library.  Plain numpy, one request / row / block at a time.

The pages decode one sequence over a preallocated cache (k2-burn README, "KV
cache storage": symmetric int8 with scales per block, sampling knobs under
"Sampling + greedy generation"); many requests over shared blocks, and rules that
differ per request, are this library's own, so the definitions are those of the
C header: what is an integer or a code is computed exactly as stated there
(float32 maxima, divisions and products), values in float64.
"""
import numpy as np

from oracle.k2_fp8 import E4M3_VALUES, e4m3_encode

F32 = np.float32
QMAX = {"i8": F32(127.0), "f8": F32(448.0)}

BAD_LENGTH, TABLE_FULL, NO_BLOCKS, TOKENS_FULL = 1, 2, 4, 8


def plan(cached, fresh, table, free, count, block, max_tokens):
    """One step's tables.  Returns a dict of the arrays after the step."""
    cached, fresh = [int(c) for c in cached], [int(f) for f in fresh]
    table, free = np.array(table), np.array(free)
    nb = lambda n: -(-n // block)  # noqa: E731
    bad = 0
    if count < 0 or count > free.size:
        bad |= NO_BLOCKS
    ok = []
    for c, f in zip(cached, fresh):
        if c < 0 or f < -1:
            bad |= BAD_LENGTH
        elif c + max(f, 0) > min(table.shape[1] * block, 2 ** 31 - 1):
            bad |= TABLE_FULL
        else:
            ok.append((c, f))
    taken = sum(nb(c + f) - nb(c) for c, f in ok if f >= 0)
    given = sum(nb(c) for c, f in ok if f < 0)
    tokens = sum(f for c, f in ok if f > 0)
    if taken > count + given or count + given - taken > free.size:
        bad |= NO_BLOCKS
    if tokens > max_tokens:
        bad |= TOKENS_FULL
    slots, positions = np.full(max_tokens, -1), np.zeros(max_tokens, dtype=np.int64)
    if bad:
        return {"table": table, "free": free, "count": count, "kv_len": np.maximum(cached, 0),
                "cu": np.zeros(len(cached) + 1, dtype=np.int64), "slots": slots, "positions": positions,
                "status": np.array([0, taken, given, bad])}
    stack = list(free[:count])
    for r, (c, f) in enumerate(ok):
        if f < 0:
            stack += list(table[r, :nb(c)])
    cu, t = [0], 0
    for r, (c, f) in enumerate(ok):
        if f >= 0:
            for j in range(nb(c), nb(c + f)):
                table[r, j] = stack.pop()
            for pos in range(c, c + f):
                slots[t], positions[t] = int(table[r, pos // block]) * block + pos % block, pos
                t += 1
        cu.append(t)
    free[:len(stack)] = stack
    return {"table": table, "free": free, "count": len(stack),
            "kv_len": np.array([c + f if f >= 0 else 0 for c, f in ok]), "cu": np.array(cu), "slots": slots,
            "positions": positions, "status": np.array([t, taken, given, 0])}


def values(codes, cache):
    """float64 values (in units of the scale) of uint8-stored codes."""
    return codes.view(np.int8).astype(np.float64) if cache == "i8" else E4M3_VALUES[codes]


def _round(y, cache):
    y = np.where(np.isnan(y), F32(0.0), y).astype(F32)
    y = np.clip(y, -QMAX[cache], QMAX[cache])
    return np.rint(y).astype(np.int8).view(np.uint8) if cache == "i8" else e4m3_encode(y)


def append(codes, scale, rows, slots, cache):
    """Rows [tokens][heads][dim] float32 into codes [blocks][heads][block][dim]
    (uint8-stored) under scale [blocks][heads] float32; both changed in place."""
    block = codes.shape[2]
    todo = {}
    for t, s in enumerate(slots):
        if 0 <= s < codes.shape[0] * block:
            todo.setdefault(int(s) // block, []).append((int(s) % block, t))
    for b, members in todo.items():
        members.sort()
        o = members[0][0]
        for h in range(codes.shape[1]):
            x = np.stack([rows[t, h] for _, t in members]).astype(F32)
            finite = np.abs(x[np.isfinite(x)])
            a = finite.max() if finite.size else F32(0.0)
            was = scale[b, h] if o > 0 else F32(0.0)
            now = np.maximum(was, F32(a / QMAX[cache]))
            if now > was and o > 0:
                y = values(codes[b, h, :o], cache).astype(F32) * F32(was / now)
                codes[b, h, :o] = _round(y, cache)
            scale[b, h] = now
            with np.errstate(over="ignore", invalid="ignore", divide="ignore"):
                y = x / now if now > 0 else np.zeros_like(x)
            for (at, _), c in zip(members, _round(y, cache)):
                codes[b, h, at] = c


def attention(q, cu, kv_len, table, k, ks, v, vs, cache, scale):
    """(out, mass, score) float64 for queries [tokens][heads][dim]: out the
    attention output; mass[t][h][d] = sum_j p_j |v_jd| and score[t][h] = the largest
    sum_d |q_d k_jd| * scale over the visible keys, from which error bounds follow.
    Rows of no request are NaN."""
    q = q.astype(np.float64)
    block, g = k.shape[2], k.shape[1]
    rep = q.shape[1] // g
    out, mass = np.full(q.shape, np.nan), np.zeros(q.shape)
    score = np.zeros(q.shape[:2])
    for r, n in enumerate(kv_len):
        n, lo, hi = int(n), int(cu[r]), int(cu[r + 1])
        if hi == lo:
            continue
        ids = table[r, :-(-n // block)]
        kk = (values(k[ids], cache) * ks[ids].astype(np.float64)[:, :, None, None]).transpose(1, 0, 2, 3)
        vv = (values(v[ids], cache) * vs[ids].astype(np.float64)[:, :, None, None]).transpose(1, 0, 2, 3)
        kk, vv = kk.reshape(g, -1, k.shape[3])[:, :n], vv.reshape(g, -1, k.shape[3])[:, :n]
        for t in range(lo, hi):
            seen = n - (hi - t) + 1
            if seen <= 0:
                out[t] = 0.0
                continue
            for h in range(q.shape[1]):
                kh, vh = kk[h // rep, :seen], vv[h // rep, :seen]
                s = kh @ q[t, h] * scale
                p = np.exp(s - s.max())
                p /= p.sum()
                out[t, h] = p @ vh
                mass[t, h] = p @ np.abs(vh)
                score[t, h] = (np.abs(kh) @ np.abs(q[t, h])).max() * abs(scale)
    return out, mass, score


def rules(logits, repetition=None, presence=None, frequency=None, ids=None, ids_len=None, prompt_len=None, bias=None,
          mask=None, mask_row=None):
    """The adjusted rows in float64."""
    x = logits.astype(np.float64)
    rows, vocab = x.shape
    for r in range(rows):
        if ids is not None:
            mine = [int(i) for i in ids[r, :max(0, min(int(ids_len[r]), ids.shape[1]))]]
            answer = mine[max(0, int(prompt_len[r])) if prompt_len is not None else 0:]
            for i in {i for i in mine if 0 <= i < vocab}:
                if repetition is not None:
                    x[r, i] = x[r, i] / repetition[r] if x[r, i] > 0 else x[r, i] * repetition[r]
                c = answer.count(i)
                if c:
                    x[r, i] -= (0.0 if frequency is None else float(frequency[r])) * c
                    x[r, i] -= 0.0 if presence is None else float(presence[r])
        if bias is not None:
            for j in range(max(int(bias[0][r]), 0), min(int(bias[0][r + 1]), len(bias[1]))):
                if 0 <= bias[1][j] < vocab:
                    x[r, bias[1][j]] += float(bias[2][j])
        if mask is not None:
            m = int(mask_row[r]) if mask_row is not None else r
            if 0 <= m < mask.shape[0]:
                i = np.arange(vocab)
                x[r, (mask[m].view(np.uint32)[i // 32] >> (i % 32).astype(np.uint32)) & 1 == 0] = -np.inf
    return x


class PagedModel:
    """An ``oracle.k2_oracle.OracleModel``'s layers over rows of many requests, with K/V in block pools of the given
    code format (float32 rows appended, as the library rounds them) and attention over their values in float64."""

    def __init__(self, model, n_blocks, block, cache):
        s = model.s
        self.m, self.cache = model, cache
        shape = (n_blocks, s.n_kv_heads, block, s.head_dim)
        self.pools = [[np.zeros(shape, np.uint8), np.zeros(shape[:2], F32), np.zeros(shape, np.uint8), np.zeros(shape[:2], F32)]
                      for _ in range(s.n_layers)]

    def step(self, tokens, positions, slots, cu, kv_len, table):
        """Logits after each request's last new token ([requests][vocab]; zeros for a request without one)."""
        from oracle.k2_oracle import rope_split_half, silu
        m, s = self.m, self.m.s
        n = int(cu[-1])
        if n == 0:
            return np.zeros((len(kv_len), s.vocab))
        x = m.embed(np.asarray(tokens)[:n])
        pos = np.asarray(positions)[:n]
        for l, (k, ks, v, vs) in enumerate(self.pools):
            xn = m._norm(x, m._w("attn_norm", l))
            rows = [(xn @ m._w(w, l).T).reshape(n, -1, s.head_dim) for w in ("wq", "wk", "wv")]
            q, kr = (rope_split_half(r, pos, s.rope_theta) for r in rows[:2])
            append(k, ks, kr.astype(F32), slots[:n], self.cache)
            append(v, vs, rows[2].astype(F32), slots[:n], self.cache)
            o, _, _ = attention(q, cu, kv_len, table, k, ks, v, vs, self.cache, s.head_dim ** -0.5)
            x = x + o.reshape(n, -1) @ m._w("wo", l).T
            xn = m._norm(x, m._w("mlp_norm", l))
            x = x + (silu(xn @ m._w("w_gate", l).T) * (xn @ m._w("w_up", l).T)) @ m._w("w_down", l).T
        out = np.zeros((len(kv_len), s.vocab))
        for r in range(len(kv_len)):
            if cu[r + 1] > cu[r]:
                out[r] = m.head(x[cu[r + 1] - 1:cu[r + 1]])[0]
        return out
