"""The operators over a block-paged 8-bit KV cache (k2_paged.cu, k2_paged_attn.cu) and the logit rules (k2_rules.cu)
against their plain oracle (oracle/k2_paged.py): tables and codes exactly, values within bounds that follow from the
roundings the header names."""
import numpy as np
import pytest
import torch

from oracle import k2_paged as P

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


@pytest.fixture(scope="module")
def k2():
    from dense_gqa_decoder_gb300 import k2 as mod
    return mod


def dev(x, dtype=torch.int32):
    return torch.tensor(np.asarray(x), dtype=dtype, device="cuda")


def host(x):
    return x.detach().cpu().numpy()


def raw(t):
    """The codes of a pool tensor as numpy uint8 (a copy)."""
    return host(t.view(torch.uint8)).copy()


# ---- plan ------------------------------------------------------------------------------------

def plan_state(cached, stride, blocks, block, seed, free_extra=0):
    rng = np.random.default_rng(seed)
    ids = rng.permutation(blocks)
    table, at = np.full((len(cached), stride), -7), 0
    for r, c in enumerate(cached):
        n = -(-c // block)
        table[r, :n] = ids[at:at + n]
        at += n
    free = np.full(blocks + free_extra, -3)
    free[:blocks - at] = ids[at:]
    return table, free, blocks - at


def run_plan(k2, cached, fresh, table, free, count, block, max_tokens, in_place=True):
    c, f, t, fr, n = dev(cached), dev(fresh), dev(table), dev(free), dev([count])
    z = lambda m: torch.full((m,), 99, dtype=torch.int32, device="cuda")  # noqa: E731
    kv, out, cu, slots, pos, st = (c if in_place else z(len(cached))), (n if in_place else z(1)), z(len(cached) + 1), \
        z(max_tokens), z(max_tokens), z(4)
    k2.paged_plan(c, f, t, fr, n, block, kv_len=kv, cu_new=cu, slots=slots, positions=pos, status=st,
                  free_count_out=out)
    if not in_place:
        assert host(c).tolist() == list(cached) and int(n) == count
    return {"table": host(t), "free": host(fr), "count": int(out), "kv_len": host(kv), "cu": host(cu),
            "slots": host(slots), "positions": host(pos), "status": host(st)}


def check_plan(k2, cached, fresh, table, free, count, block, max_tokens, in_place=True):
    want = P.plan(cached, fresh, table, free, count, block, max_tokens)
    got = run_plan(k2, cached, fresh, table, free, count, block, max_tokens, in_place)
    for n, w in want.items():
        assert np.array_equal(got[n], w), n
    return got


@pytest.mark.parametrize("requests,block,max_new,max_tokens", [
    (1, 16, 1, 1), (1, 128, 300, 300), (3, 16, 40, 200), (33, 32, 3, 100), (64, 16, 1, 64), (1024, 16, 9, 9500),
    (1025, 64, 2, 5000), (2048, 16, 30, 70000)])
@pytest.mark.parametrize("in_place", [True, False])
def test_plan_matches_the_oracle(k2, requests, block, max_new, max_tokens, in_place):
    rng = np.random.default_rng(requests + block)
    cached = rng.integers(0, 5 * block, requests)
    fresh = rng.integers(-1 if requests > 2 else 1, max_new + 1, requests)
    stride = 5 + -(-max_new // block) + 1
    blocks = int((-(-cached // block)).sum() + (-(-(cached + np.maximum(fresh, 0)) // block)).sum()) + 3
    table, free, count = plan_state(cached, stride, blocks, block, 1, free_extra=2)
    got = check_plan(k2, cached, fresh, table, free, count, block, max_tokens, in_place)
    assert got["status"][3] == 0


def test_plan_takes_blocks_that_the_same_step_gives_back(k2):
    cached, fresh = [40, 16, 0, 100], [-1, 33, 64, -1]
    table, free, count = plan_state(cached, 8, 11, 16, 2)
    assert count == 0  # 3 + 1 + 0 + 7 blocks held
    check_plan(k2, cached, fresh, table, free, count, 16, 97)


@pytest.mark.parametrize("cached,fresh,stride,blocks,max_tokens,why", [
    ([16, 3], [1, 1], 2, 2, 8, P.NO_BLOCKS), ([16, 3], [1, 30], 2, 9, 40, P.TABLE_FULL), ([16, 3], [5, 4], 4, 9, 8, P.TOKENS_FULL),
    ([16, -1], [1, 1], 4, 9, 8, P.BAD_LENGTH), ([16, 3], [1, -2], 4, 9, 8, P.BAD_LENGTH),
    ([16, 3], [2 ** 31 - 1, 1], 4, 9, 8, P.TABLE_FULL), ([2 ** 31 - 1, 0], [-1, 0], 4, 9, 8, P.TABLE_FULL),
    ([16, 3], [70, 70], 3, 3, 8, P.TABLE_FULL), ([16, 3], [20, 20], 4, 3, 8, P.NO_BLOCKS | P.TOKENS_FULL)])
def test_a_refused_plan_changes_nothing(k2, cached, fresh, stride, blocks, max_tokens, why):
    held = [c if 0 <= c <= 64 else 0 for c in cached]
    table, free, count = plan_state(held, stride, blocks, 16, 3)
    got = check_plan(k2, cached, fresh, table, free, count, 16, max_tokens)
    assert got["status"][3] == why and np.array_equal(got["table"], table) and np.array_equal(got["free"], free)
    assert (got["slots"] == -1).all() and not got["cu"].any()


def test_a_refused_large_plan_changes_nothing(k2):
    """More tokens than one CTA maps, and a request whose table is full."""
    cached, fresh = np.arange(40), np.full(40, 100)
    cached[7] = 200
    table, free, count = plan_state(cached, 13, 900, 16, 4)
    got = check_plan(k2, cached, fresh, table, free, count, 16, 5000)
    assert got["status"][3] == P.TABLE_FULL and np.array_equal(got["table"], table) and np.array_equal(got["free"], free)
    assert (got["slots"] == -1).all() and not got["cu"].any()


def test_plan_refuses_a_count_outside_the_list(k2):
    for count in (-1, 6):
        got = check_plan(k2, [0], [1], [[0]], [1, 2, 3, 4, 5], count, 16, 4)
        assert got["status"][3] == P.NO_BLOCKS


# ---- append ----------------------------------------------------------------------------------

def new_pool(k2, blocks, block, heads, dim, cache, seed, scale=0.02):
    rng = np.random.default_rng(seed)
    c = k2.PagedCache(blocks, block, heads, dim, cache)
    shape = (blocks, heads, block, dim)
    for codes, s in ((c.k, c.k_scale), (c.v, c.v_scale)):
        if cache == "i8":
            x = rng.integers(-127, 128, shape).astype(np.int8).view(np.uint8)
        else:
            x = rng.integers(0, 256, shape).astype(np.uint8)
            x[(x & 0x7F) == 0x7F] = 0  # no NaN codes
        codes.view(torch.uint8).copy_(torch.from_numpy(x))
        s.copy_(torch.from_numpy((scale * np.exp(0.5 * rng.standard_normal((blocks, heads)))).astype(np.float32)))
    return c


def check_append(k2, c, cache, k, v, slots):
    want = []
    for codes, s, x in ((c.k, c.k_scale, k), (c.v, c.v_scale, v)):
        w, ws = raw(codes), host(s).copy()
        P.append(w, ws, host(x.float()), slots, cache)
        want += [w, ws]
    k2.paged_append(c, k, v, dev(slots))
    for n, w, got in zip(("k", "k_scale", "v", "v_scale"), want, (raw(c.k), host(c.k_scale), raw(c.v), host(c.v_scale))):
        if got.dtype == np.uint8 and cache == "f8":  # +0 and -0 are the same value
            got, w = np.where(got == 0x80, 0, got), np.where(w == 0x80, 0, w)
        assert np.array_equal(got, w), n


def slots_of(runs, block):
    return [b * block + o + i for b, o, n in runs for i in range(n)]


@pytest.mark.parametrize("cache", ["i8", "f8"])
@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("block,heads,dim", [(16, 8, 128), (32, 1, 64), (64, 3, 128), (128, 9, 64)])
def test_append_matches_the_oracle(k2, cache, kind, block, heads, dim):
    rng = np.random.default_rng(block + heads)
    c = new_pool(k2, 9, block, heads, dim, cache, 4)
    # a fresh block filled whole, a whole block that follows it, single rows first / inside / last, a tail, padding
    runs = [(3, 0, block), (5, 0, block), (0, block - 1, 1), (1, 0, 1), (2, 7, 1), (4, 3, block - 3), (6, 0, 5), (7, 9, 2)]
    slots = slots_of(runs, block)
    slots[block:block] = [-1, -1]
    slots += [-1, -5]
    packed = rng.standard_normal((len(slots), 3 * heads, dim)) * np.exp(rng.standard_normal((len(slots), 3 * heads, 1)))
    packed = torch.tensor(packed, dtype=TYPES[kind], device="cuda")
    check_append(k2, c, cache, packed[:, heads:2 * heads], packed[:, 2 * heads:], slots)
    assert int(c.flags) == 0


@pytest.mark.parametrize("cache", ["i8", "f8"])
def test_append_token_by_token(k2, cache):
    """A block filled one row per call: growing rows make every call round the earlier rows again."""
    rng = np.random.default_rng(8)
    c = new_pool(k2, 2, 16, 2, 64, cache, 5)
    for o in range(16):
        x = torch.tensor(rng.standard_normal((1, 2, 64)) * (1.3 ** o if o % 3 else 0.1), dtype=torch.bfloat16, device="cuda")
        check_append(k2, c, cache, x, -x, [16 + o])


@pytest.mark.parametrize("cache", ["i8", "f8"])
def test_append_of_zeros_infinities_and_nan(k2, cache):
    c = new_pool(k2, 4, 16, 2, 64, cache, 6)
    x = torch.randn(4, 2, 64, device="cuda", generator=torch.Generator("cuda").manual_seed(1))
    x[0] = 0.0
    x[1, 0, 3], x[1, 0, 4], x[1, 1, 5] = float("inf"), float("-inf"), float("nan")
    x[2] = float("nan")
    x[3, 0] = 1e-44  # too small for a scale
    x[3, 1] = 3.4e38
    check_append(k2, c, cache, x, x.flip(0).contiguous(), [0, 16, 35, 48])


def test_append_takes_ties_to_even_and_exact_quotients(k2):
    """Rows whose quotients lie on, or one rounding from, the border between two codes."""
    rows = np.zeros((1, 1, 64), np.float32)
    rows[0, 0, 0] = 127.0 * 0.375  # the scale: 0.375
    half = (np.arange(63) - 31 + 0.5).astype(np.float32) * np.float32(0.375)
    rows[0, 0, 1:] = half
    c = new_pool(k2, 1, 16, 1, 64, "i8", 7)
    x = torch.tensor(rows, device="cuda")
    check_append(k2, c, "i8", x, torch.tensor(np.nextafter(rows, np.float32(np.inf)), device="cuda"), [0])
    # E4M3: midpoints of neighbouring codes, and their neighbours
    from oracle.k2_fp8 import E4M3_VALUES
    pos = E4M3_VALUES[:0x7F]
    mid = ((pos[1:] + pos[:-1]) / 2).astype(np.float32)
    rows = np.zeros((6, 1, 64), np.float32)
    for i, m in enumerate((mid, np.nextafter(mid, np.float32(0)), np.nextafter(mid, np.float32(1e9)))):
        rows[2 * i, 0, 1:64], rows[2 * i + 1, 0, 1:64] = m[:63], -m[63:126]
    rows[:, 0, 0] = 448.0
    c = new_pool(k2, 1, 16, 1, 64, "f8", 7)
    check_append(k2, c, "f8", torch.tensor(rows, device="cuda"), torch.tensor(-rows, device="cuda"), list(range(6)))


def test_append_flags_slots_outside_the_pool(k2):
    c = new_pool(k2, 2, 16, 2, 64, "i8", 8)
    x = torch.randn(3, 2, 64, device="cuda").to(torch.float16)
    check_append(k2, c, "i8", x, x, [32, 3, 2 ** 31 - 1])
    assert int(c.flags) == k2.K2_PAGED_BAD_SLOT


# ---- attention -------------------------------------------------------------------------------

def attention_case(k2, pairs, block, heads, kv_heads, dim, cache, kind, seed, q_scale=1.0, spare=2):
    """Pool, tables and queries for requests of (cached, new) tokens.  Rows behind a request's last token hold what
    must not be read: NaN codes (E4M3), and blocks of no request have NaN scales."""
    rng = np.random.default_rng(seed)
    owned = [-(-(c + f) // block) for c, f in pairs]
    blocks = sum(owned) + spare
    c = new_pool(k2, blocks, block, kv_heads, dim, cache, seed, scale=0.01)
    ids = rng.permutation(blocks)
    table, at = np.full((len(pairs), max(owned + [1]) + 1), -1), 0
    for r, n in enumerate(owned):
        table[r, :n] = ids[at:at + n]
        at += n
    junk = torch.tensor(ids[at:].copy(), device="cuda")
    for t, s in ((c.k, c.k_scale), (c.v, c.v_scale)):
        s[junk] = float("nan")
        for r, (a, f) in enumerate(pairs):
            if owned[r] and cache == "f8":
                t.view(torch.uint8)[int(table[r, owned[r] - 1]), :, (a + f - 1) % block + 1:] = 0x7F
    cu = np.concatenate([[0], np.cumsum([f for _, f in pairs])])
    q = torch.tensor(rng.standard_normal((int(cu[-1]) + 3, heads, dim)) * q_scale, dtype=TYPES[kind], device="cuda")
    return c, table, cu, np.array([a + f for a, f in pairs]), q


def bound(out, mass, score, n, dim, kind, vmax):
    """|error| of an output: probabilities rounded to fp16 (2^-11 of each term, plus 2^-36 of the largest value for
    those too small for that), scores accumulated in fp32 by adds that may truncate (2^-23 of the absolute sum each,
    which moves a probability by twice its exponential), the sum and the products over n keys in fp32, and the output's
    own rounding (bf16 2^-8, fp16 2^-11; fp16 values below 2^-14 have a step of 2^-24)."""
    delta = score[..., None] * (dim + 8) * 2.0 ** -23
    rel = 2.0 ** -11 + 2 * np.expm1(delta) + (n + 64) * 2.0 ** -23
    u = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}[kind]
    err = mass * rel + n * 2.0 ** -36 * vmax
    return err + (np.abs(out) + err) * u + (2.0 ** -25 if kind == "f16" else 0.0)


def check_attention(k2, c, table, cu, kv_len, q, cache, kind, scale=None, out=None, max_q=None, workspace=None):
    dim = c.head_dim
    s = dim ** -0.5 if scale is None else scale
    out = torch.full_like(q, 7.0) if out is None else out
    ws = k2.paged_workspace() if workspace is None else workspace
    k2.paged_attention(c, q, out, dev(cu), dev(kv_len), dev(table), int(np.diff(cu).max()) if max_q is None else max_q, ws,
                       scale=scale)
    want, mass, score = P.attention(host(q.float()), cu, kv_len, table, raw(c.k), host(c.k_scale), raw(c.v),
                                    host(c.v_scale), cache, s)
    got = host(out.float()).astype(np.float64)
    rows = ~np.isnan(want[:, 0, 0])
    assert (got[~rows] == 7.0).all()  # rows of no request are left as they were
    vs = host(c.v_scale)
    vmax = float(np.nanmax(np.abs(vs))) * (127 if cache == "i8" else 448)
    room = bound(want, mass, score, int(max(kv_len)), dim, kind, vmax)
    worst = (np.abs(got - want) / room)[rows]
    assert np.isfinite(got[rows]).all() and worst.max(initial=0) <= 1.0, float(worst.max())
    return out


SHORT = [(0, 1), (14, 1), (15, 1), (16, 1), (31, 1), (32, 1), (63, 1), (64, 1), (127, 1), (128, 1), (200, 1)]
DECODE = [
    (SHORT, 16, 8, 2, 128, "i8", "bf16"), (SHORT, 32, 8, 2, 128, "f8", "f16"), (SHORT, 64, 8, 2, 64, "i8", "f16"),
    (SHORT, 128, 4, 1, 64, "f8", "bf16"), ([(0, 1)], 16, 4, 1, 128, "i8", "f16"), ([(1000, 1)], 16, 32, 8, 128, "i8", "bf16"),
    ([(5000, 1), (3, 1), (0, 0), (777, 0), (2500, 1)], 16, 4, 2, 128, "f8", "bf16"),
    ([(4099, 1)], 128, 8, 1, 64, "i8", "f16"),
    ([(300, 1), (40, 1)], 16, 3, 3, 128, "i8", "bf16"), ([(300, 1), (40, 1)], 32, 16, 1, 128, "f8", "f16"),
    ([(300, 1), (40, 1)], 16, 10, 2, 64, "i8", "f16"), ([(333, 1)] * 20, 64, 24, 2, 128, "i8", "bf16"),
]
SEVERAL = [  # a few queries each: speculative steps
    ([(100, 2), (0, 3), (17, 1), (500, 5)], 16, 8, 2, 128, "i8", "bf16"), ([(61, 9), (9, 8), (64, 1)], 32, 8, 2, 128, "f8", "f16"),
    ([(1200, 4), (1, 4)], 64, 4, 1, 64, "i8", "f16"), ([(70, 7), (0, 0), (3, 2)], 16, 12, 4, 128, "f8", "bf16"),
    ([(33, 3)], 128, 16, 1, 64, "f8", "f16"),
]
CHUNKS = [  # prompt chunks, alone and among single tokens
    ([(0, 40)], 16, 8, 2, 128, "i8", "f16"), ([(0, 129), (130, 1), (77, 64)], 16, 4, 1, 128, "i8", "bf16"),
    ([(500, 100), (0, 33), (4000, 1)], 32, 4, 1, 64, "f8", "f16"), ([(64, 64), (63, 65), (65, 63)], 64, 8, 2, 128, "f8", "bf16"),
    ([(10, 200)], 128, 2, 2, 128, "i8", "f16"), ([(31, 70), (0, 0), (5, 20)], 16, 16, 1, 64, "i8", "bf16"),
    ([(100, 300)], 16, 6, 2, 64, "f8", "f16"), ([(129, 100), (0, 1)], 64, 10, 1, 128, "i8", "f16"),
]


@pytest.mark.parametrize("pairs,block,heads,kv_heads,dim,cache,kind", DECODE + SEVERAL + CHUNKS)
def test_attention_matches_the_oracle(k2, pairs, block, heads, kv_heads, dim, cache, kind):
    c, table, cu, kv_len, q = attention_case(k2, pairs, block, heads, kv_heads, dim, cache, kind, len(pairs) + heads)
    check_attention(k2, c, table, cu, kv_len, q, cache, kind)
    assert int(c.flags) == 0


@pytest.mark.parametrize("cache,kind", [("i8", "bf16"), ("f8", "f16")])
@pytest.mark.parametrize("pairs", [[(900, 1), (2000, 1)], [(300, 80), (800, 1)]])
def test_attention_of_peaked_scores(k2, cache, kind, pairs):
    """Queries so large that one key takes nearly all of a row, whose maximum keeps moving."""
    c, table, cu, kv_len, q = attention_case(k2, pairs, 16, 8, 2, 128, cache, kind, 11, q_scale=20.0)
    check_attention(k2, c, table, cu, kv_len, q, cache, kind)


@pytest.mark.parametrize("pairs", [[(900, 1), (100, 1)], [(300, 80)]])
def test_attention_with_block_scales_far_apart(k2, pairs):
    """Blocks whose V scales differ by up to 2^20 (the small ones carry the output: their keys score highest)."""
    c, table, cu, kv_len, q = attention_case(k2, pairs, 16, 4, 1, 128, "i8", "f16", 12)
    rng = np.random.default_rng(1)
    c.v_scale.copy_(torch.tensor(2.0 ** rng.integers(-16, 5, tuple(c.v_scale.shape)), dtype=torch.float32))
    c.k_scale.copy_(torch.tensor(2.0 ** rng.integers(-9, -4, tuple(c.k_scale.shape)), dtype=torch.float32))
    c.v_scale[int(table[0, 3])] = 0.0  # a block of zeros
    check_attention(k2, c, table, cu, kv_len, q, "i8", "f16")


def test_attention_queries_of_any_size(k2):
    """bf16 queries from 2^-60 to 2^60 keep their bits on the way into the products."""
    for e in (-60, -20, 20, 60):
        c, table, cu, kv_len, q = attention_case(k2, [(77, 1), (40, 40)], 16, 4, 1, 128, "i8", "bf16", 13, q_scale=2.0 ** e)
        check_attention(k2, c, table, cu, kv_len, q, "i8", "bf16", scale=0.05 * 2.0 ** -e)


def test_attention_other_scales(k2):
    c, table, cu, kv_len, q = attention_case(k2, [(77, 1), (40, 40)], 16, 4, 1, 64, "i8", "f16", 14)
    for scale in (0.0, -0.2, 1.0):
        check_attention(k2, c, table, cu, kv_len, q, "i8", "f16", scale=scale)


def test_attention_strided_rows(k2):
    pairs = [(50, 1), (0, 70), (300, 3)]
    c, table, cu, kv_len, q = attention_case(k2, pairs, 16, 8, 2, 128, "i8", "bf16", 15)
    packed = torch.full((q.shape[0], 12, 128), 5.0, dtype=q.dtype, device="cuda")
    packed[:, :8] = q
    wide = torch.full((q.shape[0], 9, 128), 7.0, dtype=q.dtype, device="cuda")
    check_attention(k2, c, table, cu, kv_len, packed[:, :8], "i8", "bf16", out=wide[:, :8])
    assert (wide[:, 8] == 7.0).all()


def test_one_row_of_any_stride(k2):
    """The distance between tokens is of no account where there is one."""
    c, table, cu, kv_len, q = attention_case(k2, [(40, 1)], 16, 8, 2, 128, "i8", "bf16", 19)
    one = q[:1].as_strided((1, 8, 128), (3, 128, 1))
    out = torch.full_like(one, 7.0).as_strided((1, 8, 128), (5, 128, 1))
    check_attention(k2, c, table, cu, kv_len, one, "i8", "bf16", out=out)
    k = torch.randn(1, 2, 128, device="cuda")
    again = new_pool(k2, c.n_blocks, 16, 2, 128, "i8", 20)
    other = new_pool(k2, c.n_blocks, 16, 2, 128, "i8", 20)
    k2.paged_append(again, k.as_strided((1, 2, 128), (7, 128, 1)), k, dev([16]))
    k2.paged_append(other, k, k, dev([16]))
    assert np.array_equal(raw(again.k), raw(other.k)) and torch.equal(again.k_scale, other.k_scale)


@pytest.mark.parametrize("pairs,block,heads,kv_heads,dim,cache,kind", [
    ([(40, 1), (0, 1), (300, 2)], 16, 128, 128, 64, "i8", "bf16"), ([(40, 30), (17, 1)], 32, 128, 128, 64, "f8", "f16"),
    ([(33, 1), (5, 3)], 16, 256, 16, 128, "i8", "f16"), ([(20, 1)] * 2047 + [(100, 1)], 16, 4, 1, 64, "f8", "bf16"),
    ([(3, 1), (0, 0)] * 1023 + [(70, 40)], 128, 4, 2, 64, "i8", "f16"), ([(0, 2)] * 700, 16, 16, 1, 128, "f8", "f16")])
def test_attention_of_many_heads_and_requests(k2, pairs, block, heads, kv_heads, dim, cache, kind):
    c, table, cu, kv_len, q = attention_case(k2, pairs, block, heads, kv_heads, dim, cache, kind, 29)
    check_attention(k2, c, table, cu, kv_len, q, cache, kind)
    assert int(c.flags) == 0


def test_append_of_many_heads(k2):
    c = new_pool(k2, 6, 32, 128, 64, "f8", 30)
    x = torch.randn(50, 128, 64, device="cuda", dtype=torch.bfloat16)
    check_append(k2, c, "f8", x, x.flip(0), slots_of([(2, 5, 20), (0, 0, 30)], 32))


def test_two_streams_at_once(k2):
    """Calls that overlap, each with a workspace of its own, give what they give alone."""
    runs = []
    for seed, pairs in ((23, [(9000, 1), (40, 1), (2500, 150)]), (24, [(7000, 2), (1, 70), (3000, 1)])):
        c, table, cu, kv_len, q = attention_case(k2, pairs, 16, 8, 2, 128, "i8", "f16", seed)
        ws = k2.paged_workspace()
        args = (c, q, torch.zeros_like(q), dev(cu), dev(kv_len), dev(table), 150, ws)
        k2.paged_attention(*args)
        runs.append((args, args[2].clone(), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(20):
        for args, _, stream in runs:
            args[2].zero_()
            stream.wait_stream(torch.cuda.current_stream())
            k2.paged_attention(*args, stream=stream)
        for args, want, stream in runs:
            torch.cuda.current_stream().wait_stream(stream)
            assert torch.equal(args[2], want)


def test_a_replayed_mixed_step(k2):
    """Plan, append and attention captured once, for more tokens than a plan's CTA maps, and replayed as requests grow,
    end and begin again, against the same calls made eagerly on buffers of their own."""
    requests, block, heads, kv_heads, dim, most, columns = 5, 32, 8, 2, 64, 1100, 70
    blocks = 200
    i32 = dict(dtype=torch.int32, device="cuda")

    def buffers():
        z = lambda *n: torch.zeros(*n, **i32)  # noqa: E731
        return dict(cached=z(requests), fresh=z(requests), table=torch.full((requests, columns), -1, **i32),
                    free=torch.arange(blocks, **i32), count=torch.full((1,), blocks, **i32), cu=z(requests + 1),
                    slots=z(most), positions=z(most), status=z(4), cache=k2.PagedCache(blocks, block, kv_heads, dim, "f8"),
                    ws=k2.paged_workspace(), q=torch.zeros(most, heads, dim, dtype=torch.float16, device="cuda"),
                    kv=torch.zeros(most, 2 * kv_heads, dim, dtype=torch.float16, device="cuda"),
                    out=torch.zeros(most, heads, dim, dtype=torch.float16, device="cuda"))

    def step(b):
        k2.paged_plan(b["cached"], b["fresh"], b["table"], b["free"], b["count"], block, kv_len=b["cached"], cu_new=b["cu"],
                      slots=b["slots"], positions=b["positions"], status=b["status"])
        k2.paged_append(b["cache"], b["kv"][:, :kv_heads], b["kv"][:, kv_heads:], b["slots"])
        k2.paged_attention(b["cache"], b["q"], b["out"], b["cu"], b["cached"], b["table"], 900, b["ws"])

    mine, eager = buffers(), buffers()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step(mine)  # (nothing to do: every length is 0)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            step(mine)
    side.synchronize()
    gen = torch.Generator("cuda").manual_seed(4)
    for fresh in ([900, 3, 0, 70, 100], [1, 1, 1, 1, 1], [1, 40, 800, -1, 0], [-1, 1, 1, 33, 900], [0, 0, 0, 0, 0], [2, 5, 1, 1, -1]):
        q = torch.randn(most, heads, dim, device="cuda", generator=gen).half()
        kv = torch.randn(most, 2 * kv_heads, dim, device="cuda", generator=gen).half()
        for b in (mine, eager):
            b["fresh"].copy_(dev(fresh))
            b["q"].copy_(q)
            b["kv"].copy_(kv)
            b["out"].fill_(7.0)
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            graph.replay()
        side.synchronize()
        step(eager)
        torch.cuda.synchronize()
        assert int(mine["status"][3]) == 0
        for n in ("cached", "table", "count", "cu", "slots", "positions", "status", "out"):
            assert torch.equal(mine[n], eager[n]), (n, fresh)
        assert np.array_equal(raw(mine["cache"].k), raw(eager["cache"].k))
        tokens = sum(max(f, 0) for f in fresh)
        assert (mine["out"][tokens:] == 7.0).all() and not int(mine["cache"].flags)


def test_attention_is_the_same_every_time(k2):
    """Splits of a long context are joined in one order, whoever finishes last; the workspace is left clean."""
    pairs = [(6000, 1), (300, 2), (2048, 200)]
    c, table, cu, kv_len, q = attention_case(k2, pairs, 16, 8, 2, 128, "i8", "bf16", 16)
    ws = k2.paged_workspace()
    a, b, d = dev(cu), dev(kv_len), dev(table)
    first = torch.empty_like(q)
    k2.paged_attention(c, q, first, a, b, d, 200, ws)
    for _ in range(20):
        out = torch.empty_like(q)
        k2.paged_attention(c, q, out, a, b, d, 200, ws)
        n = int(cu[-1])
        assert torch.equal(out[:n], first[:n])


def test_attention_leaves_out_blocks_outside_the_pool(k2):
    pairs = [(100, 1), (0, 50), (64, 1)]
    c, table, cu, kv_len, q = attention_case(k2, pairs, 16, 4, 1, 128, "i8", "f16", 17)
    out = torch.zeros_like(q)
    bad = table.copy()
    bad[0, 2], bad[1, 1], bad[2, :5] = c.n_blocks, -1, 2 ** 31 - 1
    k2.paged_attention(c, q, out, dev(cu), dev(kv_len), dev(bad), 50, k2.paged_workspace())
    assert int(c.flags) == k2.K2_PAGED_BAD_BLOCK
    assert torch.isfinite(out).all() and not out[cu[2]].any()  # the third request has no key left
    # as if those 16 keys of the first request did not exist
    keep = np.delete(table[0], 2)
    want, _, _ = P.attention(host(q[:1].float()), [0, 1], [101 - 16], keep[None], raw(c.k), host(c.k_scale), raw(c.v),
                             host(c.v_scale), "i8", 128 ** -0.5)
    assert np.allclose(host(out[0].float()), want[0], rtol=2e-3, atol=2e-3)


@pytest.mark.parametrize("cu,kv_len,max_q", [([0, 2, 3], [1, 20], 2), ([0, 2, 3], [20, -4], 2), ([0, 2, 3], [2 ** 31 - 1, 20], 2),
                                             ([0, 2, 900], [20, 900], 900), ([0, 3, 2], [20, 20], 3), ([0, 2, 3], [20, 20], 1),
                                             ([-1, 1, 3], [20, 20], 2)])
def test_attention_flags_lengths_that_contradict(k2, cu, kv_len, max_q):
    c, table, _, _, q = attention_case(k2, [(30, 2), (30, 1)], 16, 4, 1, 64, "i8", "f16", 18)
    out = torch.full_like(q, 7.0)
    k2.paged_attention(c, q, out, dev(cu), dev(kv_len), dev(table), max_q, k2.paged_workspace())
    assert int(c.flags) == k2.K2_PAGED_BAD_LENGTH
    assert torch.isfinite(out).all()


def test_attention_on_another_stream_and_in_a_graph(k2):
    """A captured step is replayed with lengths, tables and queries that changed since."""
    one = [(70, 1), (500, 1), (9, 30)]
    c, table, cu, kv_len, q = attention_case(k2, one, 16, 8, 2, 128, "f8", "bf16", 19)
    a, b, t, ws, out = dev(cu), dev(kv_len), dev(table), k2.paged_workspace(), torch.full_like(q, 7.0)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        k2.paged_attention(c, q, out, a, b, t, 32, ws)
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        k2.paged_attention(c, q, out, a, b, t, 32, ws)
    for n in ([(70, 1), (500, 1), (9, 30)], [(60, 3), (300, 20), (0, 9)], [(0, 0), (17, 32), (0, 0)]):
        cu2, len2 = np.concatenate([[0], np.cumsum([f for _, f in n])]), np.array([x + f for x, f in n])
        a.copy_(dev(cu2))
        b.copy_(dev(len2))
        q.copy_(torch.randn(q.shape, device="cuda").to(q.dtype))
        fill = torch.randint(0, 0x7F, tuple(c.k.shape), dtype=torch.uint8, device="cuda")
        c.k.view(torch.uint8).copy_(fill)
        c.v.view(torch.uint8).copy_(fill.flip(0))
        out.fill_(7.0)
        g.replay()
        want, mass, score = P.attention(host(q.float()), cu2, len2, table, raw(c.k), host(c.k_scale), raw(c.v),
                                        host(c.v_scale), "f8", 128 ** -0.5)
        rows = ~np.isnan(want[:, 0, 0])
        got = host(out.float()).astype(np.float64)
        assert (got[~rows] == 7.0).all()
        room = bound(want, mass, score, 512, 128, "bf16", float(np.nanmax(host(c.v_scale))) * 448)
        assert (np.abs(got - want)[rows] <= room[rows]).all()


def test_a_cache_beyond_4_gib(k2):
    """Code offsets that pass 32 bits."""
    blocks, block, heads, dim = 300_000, 16, 8, 128  # 4.9 GB of K codes
    c = k2.PagedCache(blocks, block, heads, dim, "i8")
    rng = np.random.default_rng(20)
    ids = [blocks - 1, 1, blocks - 7, 262_144, 5, 299_000]
    n = 6 * block - 3
    x = torch.tensor(rng.standard_normal((n, heads, dim)), dtype=torch.bfloat16, device="cuda")
    slots = [ids[i // block] * block + i % block for i in range(n)]
    k2.paged_append(c, x, -x, dev(slots))
    small = k2.PagedCache(6, block, heads, dim, "i8")
    k2.paged_append(small, x, -x, dev(list(range(n))))
    at = torch.tensor(ids, device="cuda")
    assert torch.equal(c.k[at], small.k) and torch.equal(c.v_scale[at], small.v_scale)
    for new in (1, 60):
        q = torch.tensor(rng.standard_normal((new, 32, dim)), dtype=torch.bfloat16, device="cuda")
        got, want = torch.zeros_like(q), torch.zeros_like(q)
        ws = k2.paged_workspace()
        k2.paged_attention(c, q, got, dev([0, new]), dev([n]), dev([ids]), new, ws)
        k2.paged_attention(small, q, want, dev([0, new]), dev([n]), dev([list(range(6))]), new, ws)
        assert torch.equal(got, want) and got.abs().max() > 0


# ---- logit rules -----------------------------------------------------------------------------

def rules_case(rows, vocab, history, n_bias, masks, seed, allowed=0.5):
    rng = np.random.default_rng(seed)
    ids = (rng.random((rows, history)) ** 3 * (vocab + 4)).astype(np.int64) - 2  # some outside the vocabulary
    length = rng.integers(0, history + 1, rows)
    case = {"repetition": (1 + rng.random(rows)).astype(np.float32), "presence": rng.standard_normal(rows).astype(np.float32),
            "frequency": rng.standard_normal(rows).astype(np.float32), "ids": ids, "ids_len": length,
            "prompt_len": rng.integers(0, history + 2, rows)}
    if n_bias:
        cut = np.concatenate([[0], np.sort(rng.integers(0, n_bias + 1, rows - 1)), [n_bias]]) if rows > 1 else np.array([0, n_bias])
        case["bias"] = (cut, rng.integers(-1, vocab + 1, n_bias), rng.standard_normal(n_bias).astype(np.float32))
    if masks:
        bits = rng.random((masks, (vocab + 31) // 32, 32)) < allowed
        case["mask"] = (bits * (1 << np.arange(32, dtype=np.uint64))).sum(-1).astype(np.uint32)
        case["mask_row"] = rng.integers(-1, masks + 1, rows)
    x = (rng.standard_normal((rows, vocab)) * 4).astype(np.float32)
    x[:, ::17] = -np.inf
    x[:, 5 % vocab] = 0.0
    return x, case


def on_device(case):
    got = {}
    for n, v in case.items():
        if n == "bias":
            got[n] = (dev(v[0]), dev(v[1]), dev(v[2], torch.float32))
        elif n == "mask":
            got[n] = dev(v.view(np.int32))
        else:
            got[n] = dev(v, torch.float32 if v.dtype == np.float32 else torch.int32)
    return got


def check_rules(got, x, case):
    want = P.rules(x, **case)
    assert np.array_equal(np.isneginf(got), np.isneginf(want)) and np.array_equal(np.isnan(got), np.isnan(want))
    fine = np.isfinite(want)
    # one fp32 rounding (2^-24) per operation: quotient or product, penalty product, two differences, each bias
    steps = 4 + (0 if "bias" not in case else len(case["bias"][1]))
    count = case["ids"].shape[1] if "ids" in case else 0
    size = np.abs(np.where(np.isfinite(x), x, 0)) * 2 + (4 * (count + 1) if count else 0) + (5 if "bias" in case else 0)
    assert (np.abs(got - np.where(fine, want, 0))[fine] <= (steps * 2.0 ** -24 * (size + np.abs(np.where(fine, want, 0))))[fine]).all()


@pytest.mark.parametrize("rows,vocab,history,n_bias,masks", [
    (1, 1, 1, 1, 1), (1, 512, 30, 5, 1), (3, 1000, 0, 0, 2), (2, 31, 40, 9, 0), (5, 8191, 700, 40, 3), (4, 8192, 33, 0, 0),
    (7, 8193, 1, 100, 1), (2, 250624, 5000, 301, 2), (64, 4097, 256, 64, 4)])
def test_rules_match_the_oracle(k2, rows, vocab, history, n_bias, masks):
    x, case = rules_case(rows, vocab, history, n_bias, masks, rows + vocab)
    d = dev(x, torch.float32)
    out = torch.full_like(d, 9.0)
    k2.adjust_logits(d, out, **on_device(case))
    check_rules(host(out), x, case)
    assert np.array_equal(host(d), x)
    k2.adjust_logits(d, **on_device(case))  # in place
    assert torch.equal(d, out)


@pytest.mark.parametrize("rows,vocab,history,n_bias,masks", [
    (64, 40004, 300, 700, 5), (333, 8192, 40, 0, 2), (400, 4, 3, 50, 2), (40, 65539, 500, 30000, 3), (306, 8195, 0, 0, 1)])
def test_rules_of_many_aligned_rows(k2, rows, vocab, history, n_bias, masks):
    """Steps of many slices, copied ahead: rows that end inside a slice and inside a group of four, long bias lists."""
    x, case = rules_case(rows, vocab, history, n_bias, masks, rows + vocab)
    ld = (vocab + 7) // 4 * 4
    d, out = torch.full((rows, ld), 3.0, device="cuda"), torch.full((rows, ld), 9.0, device="cuda")
    d[:, :vocab] = dev(x, torch.float32)
    given = on_device(case)
    k2.adjust_logits(d[:, :vocab], out[:, :vocab], **given)
    check_rules(host(out[:, :vocab]), x, case)
    assert np.array_equal(host(d[:, :vocab]), x)
    assert (out[:, vocab:] == 9.0).all() and (d[:, vocab:] == 3.0).all()
    k2.adjust_logits(d[:, :vocab], **given)  # in place
    assert torch.equal(d[:, :vocab], out[:, :vocab]) and (d[:, vocab:] == 3.0).all()


@pytest.mark.parametrize("only", ["repetition", "presence", "frequency", "bias", "mask", "none", "ids alone"])
def test_each_rule_alone(k2, only):
    x, case = rules_case(6, 3001, 200, 50, 6, 31)
    keep = {"ids", "ids_len"} if only in ("repetition", "presence", "frequency", "ids alone") else set()
    case = {n: v for n, v in case.items() if n == only or n in keep}
    d = dev(x, torch.float32)
    out = torch.full_like(d, 9.0)
    k2.adjust_logits(d, out, **on_device(case))
    check_rules(host(out), x, case)
    if only in ("none", "ids alone"):
        assert torch.equal(out, d)


def test_rules_on_strided_rows_that_are_not_16_byte_aligned(k2):
    x, case = rules_case(4, 1001, 100, 20, 2, 32)
    wide = torch.full((4, 1101), 3.0, device="cuda")
    wide[:, 7:1008] = dev(x, torch.float32)
    out = torch.full((4, 1013), 9.0, device="cuda")
    k2.adjust_logits(wide[:, 7:1008], out[:, 3:1004], **on_device(case))
    check_rules(host(out[:, 3:1004]), x, case)
    assert (out[:, :3] == 9.0).all() and (out[:, 1004:] == 9.0).all()
    k2.adjust_logits(wide[:, 7:1008], **on_device(case))
    assert torch.equal(wide[:, 7:1008], out[:, 3:1004]) and (wide[:, :7] == 3.0).all() and (wide[:, 1008:] == 3.0).all()


def test_rules_divide_by_any_positive_repetition(k2):
    """Quotients and products round once, for penalties whose reciprocal is not a normal number too."""
    rep = np.array([1e-39, 3e38, 3.0, 1.1], np.float32)
    x = np.array([[1e-3, -1e-3, 7.0, -7.0, 0.0, 30.0, -0.0, 11.0]] * 4, np.float32)
    ids = np.tile(np.arange(7), (4, 1))
    d = dev(x, torch.float32)
    k2.adjust_logits(d, repetition=dev(rep, torch.float32), ids=dev(ids), ids_len=dev([7] * 4))
    with np.errstate(over="ignore"):
        want = np.where(x > 0, x / rep[:, None], x * rep[:, None])
    want[:, 7] = x[:, 7]
    assert np.array_equal(host(d), want)


def test_rules_edge_values(k2):
    """NaN and infinities under a mask, a row whose mask leaves nothing, an id listed many times."""
    x = np.array([[np.nan, np.inf, -np.inf, 1.0, -1.0, 0.0, 2.0, 3.0]] * 3, np.float32)
    case = {"mask": np.array([[0b11111100], [0], [0xFF]], np.uint32), "mask_row": np.array([0, 1, 2]),
            "bias": (np.array([0, 5, 5, 8]), np.array([3, 3, 3, 3, 5, 0, 1, 2]),
                     np.array([1e8, 1.0, -1e8, 0.25, -np.inf, 1.0, 1.0, 1.0], np.float32))}
    d = dev(x, torch.float32)
    out = torch.empty_like(d)
    k2.adjust_logits(d, out, **on_device(case))
    got = host(out)
    assert np.isneginf(got[0, :3]).all() and got[0, 4] == -1.0 and np.isneginf(got[0, 5])
    # in list order: ((1 + 1e8) + 1) - 1e8 + 0.25 in fp32
    v = np.float32(1.0)
    for b in case["bias"][2][:4]:
        v = np.float32(v + b)
    assert got[0, 3] == v
    assert np.isneginf(got[1]).all()
    assert np.isnan(got[2, 0]) and got[2, 1] == np.inf and np.isneginf(got[2, 2])


# ---- together --------------------------------------------------------------------------------

def test_a_served_run(k2):
    """Twelve steps of five requests that come, grow and end over one pool: tables, cache and attention against the
    oracle's at every step, run eagerly and from one captured graph."""
    block, blocks, heads, kv_heads, dim, max_tokens = 16, 24, 8, 2, 64, 48
    rng = np.random.default_rng(40)
    for graph in (False, True):
        c = k2.PagedCache(blocks, block, kv_heads, dim, "i8")
        want = [(np.zeros((blocks, kv_heads, block, dim), np.uint8), np.zeros((blocks, kv_heads), np.float32)) for _ in "kv"]
        table, free, count, lens = np.full((5, 12), -1), np.arange(blocks), blocks, np.zeros(5, dtype=np.int64)
        z = lambda n: torch.zeros(n, dtype=torch.int32, device="cuda")  # noqa: E731
        d_len, d_fresh, d_table, d_free, d_count = z(5), z(5), dev(table), dev(free), dev([count])
        cu, slots, pos, st, ws = z(6), z(max_tokens), z(max_tokens), z(4), k2.paged_workspace()
        rows = torch.zeros(max_tokens, heads + 2 * kv_heads, dim, dtype=torch.bfloat16, device="cuda")
        out = torch.zeros(max_tokens, heads, dim, dtype=torch.bfloat16, device="cuda")

        def step():
            k2.paged_plan(d_len, d_fresh, d_table, d_free, d_count, block, kv_len=d_len, cu_new=cu, slots=slots,
                          positions=pos, status=st)
            k2.paged_append(c, rows[:, heads:heads + kv_heads], rows[:, heads + kv_heads:], slots)
            k2.paged_attention(c, rows[:, :heads], out, cu, d_len, d_table, max_tokens, ws)

        g = None
        if graph:
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                step()
        for i in range(12):
            fresh = np.array([int(rng.choice([0, 1, 1, 2, 20])) if n < 90 else -1 for n in lens])
            if i == 5:
                fresh[:] = 12  # more tokens than the step has rows: refused
            got = P.plan(lens, fresh, table, free, count, block, max_tokens)
            table, free, count, lens = got["table"], got["free"], got["count"], got["kv_len"]
            assert i != 5 or got["status"][3] == P.TOKENS_FULL
            x = rng.standard_normal(tuple(rows.shape)) * np.exp(rng.standard_normal((max_tokens, 1, 1)))
            rows.copy_(torch.tensor(x).to(torch.bfloat16))
            d_fresh.copy_(dev(fresh))
            out.fill_(7.0)
            g.replay() if graph else step()
            for a, b in ((d_table, table), (d_free, free), (d_len, lens), (cu, got["cu"]), (slots, got["slots"]),
                         (pos, got["positions"]), (st, got["status"])):
                assert np.array_equal(host(a), b)
            xf = host(rows.float())
            for (codes, scale), lo in zip(want, (heads, heads + kv_heads)):
                P.append(codes, scale, xf[:, lo:lo + kv_heads], got["slots"], "i8")
            assert np.array_equal(raw(c.k), want[0][0]) and np.array_equal(host(c.v_scale), want[1][1])
            o, mass, score = P.attention(xf[:, :heads], got["cu"], lens, table, want[0][0], want[0][1], want[1][0], want[1][1],
                                         "i8", dim ** -0.5)
            seen, have = ~np.isnan(o[:, 0, 0]), host(out.float()).astype(np.float64)
            assert (have[~seen] == 7.0).all()
            room = bound(o, mass, score, 128, dim, "bf16", float(want[1][1].max()) * 127)
            assert (np.abs(have - o)[seen] <= room[seen]).all()
        assert int(c.flags) == 0


def test_rules_before_the_sampler(k2):
    """Rules, then k2_sample_logits: a grammar that leaves one id gives that id, whatever the logits."""
    from dense_gqa_decoder_gb300 import model_io
    import k2_inputs as ki
    ctx, _ = model_io.build_context(ki.TINY, max_context=32, max_batch=3, kv_dtype="f32")
    ctx.set_sampling(k2.sampling(temperature=0.7, top_p=0.95, seed=3))
    vocab = ki.TINY.vocab
    logits = torch.randn(3, vocab, device="cuda")
    words = np.zeros((2, (vocab + 31) // 32), np.uint32)
    words[0, 300 // 32] = 1 << (300 % 32)
    words[1, 7] = 0b1010
    k2.adjust_logits(logits, mask=dev(words.view(np.int32)), mask_row=dev([0, 1, -1]),
                     bias=(dev([0, 0, 0, 1]), dev([17]), dev([100.0], torch.float32)))
    nxt = torch.full((3,), -1, dtype=torch.int32, device="cuda")
    ctx.sample_logits(logits, 3, dev([1, 2, 3]), nxt)
    got = nxt.tolist()
    assert got[0] == 300 and got[1] in (7 * 32 + 1, 7 * 32 + 3) and got[2] == 17
    assert ctx.sync_status() == k2.K2_OK


def test_wrappers_refuse_tensors_the_calls_cannot_take(k2):
    c = k2.PagedCache(4, 16, 2, 64)
    ws = k2.paged_workspace()
    x = torch.zeros(3, 2, 64, dtype=torch.bfloat16, device="cuda")
    s3 = torch.zeros(3, dtype=torch.int32, device="cuda")
    for k, v, s in ((x.double(), x, s3), (x, x.half(), s3), (x[:, :1], x, s3), (x, x[:2], s3), (x, x, s3.long()), (x, x, s3[:2]),
                    (x.cpu(), x, s3), (x.transpose(0, 1).contiguous().transpose(0, 1), x, s3)):
        with pytest.raises(ValueError):
            k2.paged_append(c, k, v, s)
    q = torch.zeros(3, 4, 64, dtype=torch.float16, device="cuda")
    cu, n, t = s3[:2], s3[:1], torch.zeros(1, 4, dtype=torch.int32, device="cuda")
    for args in ((q.float(), q, cu, n, t), (q, q.bfloat16(), cu, n, t), (q, q[:2], cu, n, t), (q, q, s3, n, t), (q, q, cu, n, t[0]),
                 (q, q, cu, n.cpu(), t), (q[..., :32], q, cu, n, t)):
        with pytest.raises(ValueError):
            k2.paged_attention(c, args[0], args[1], *args[2:], 1, ws)
    with pytest.raises(k2.K2Error):
        k2.paged_attention(c, q, q.clone(), cu, n, t, 1, ws[:0].contiguous())
    with pytest.raises(ValueError):
        k2.PagedCache(4, 16, 2, 64, "f16")
    with pytest.raises(ValueError):
        k2.PagedCache.of(c.k, c.v[:2], c.k_scale, c.v_scale)
    lg = torch.zeros(2, 40, device="cuda")
    for kw in (dict(repetition=torch.ones(3, device="cuda")), dict(ids=torch.zeros(2, 4, dtype=torch.int32, device="cuda")),
               dict(mask=torch.zeros(1, 2, dtype=torch.int32, device="cuda")),
               dict(mask=torch.zeros(2, 1, dtype=torch.int32, device="cuda"))):
        with pytest.raises(ValueError):
            k2.adjust_logits(lg, **kw)
    with pytest.raises(k2.K2Error):
        k2.adjust_logits(lg, torch.zeros(2, 40, device="cuda"), repetition=torch.ones(2, device="cuda"))
