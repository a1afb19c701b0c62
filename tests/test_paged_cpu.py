"""Host-side checks of the operators over a block-paged 8-bit cache and of the logit rules: what the C calls
refuse before they touch a GPU, and pins of their oracle (oracle/k2_paged.py).  No GPU is needed."""
import ctypes as C

import numpy as np
import pytest

from oracle import k2_paged as P


@pytest.fixture(scope="module")
def k2():
    from dense_gqa_decoder_gb300 import build
    build.build()
    from dense_gqa_decoder_gb300 import k2 as mod
    return mod


A = 0x1000  # an aligned non-null address that no refused call reads


def pool(k2, **kw):
    d = dict(k=A, v=A, k_scale=A, v_scale=A, n_blocks=4, block_tokens=16, n_kv_heads=2, head_dim=128, dtype=k2.K2_I8)
    d.update(kw)
    return k2.PagedKv(**d)


BAD_POOLS = [(dict(k=None), "ARG"), (dict(v_scale=None), "ARG"), (dict(v=A + 8), "ARG"), (dict(dtype=2), "UNSUPPORTED"),
             (dict(block_tokens=24), "UNSUPPORTED"), (dict(block_tokens=256), "UNSUPPORTED"),
             (dict(head_dim=96), "UNSUPPORTED"), (dict(n_kv_heads=0), "SHAPE"), (dict(n_blocks=0), "SHAPE"),
             (dict(n_blocks=2 ** 27), "SHAPE")]


@pytest.mark.parametrize("kw,why", BAD_POOLS)
def test_pools_that_are_refused(k2, kw, why):
    kv = pool(k2, **kw)
    want = getattr(k2, "K2_ERR_" + why)
    assert k2.LIB.k2_paged_append(C.addressof(kv), A, A, k2.K2_BF16, 256, 256, A, 1, None) == want
    assert k2.LIB.k2_last_error(None).decode() != ""
    assert k2.LIB.k2_paged_attention(C.addressof(kv), A, k2.K2_BF16, 1024, A, A, A, 4, 1, 1, 8, 1, 0.1, A, 1024, A,
                                     1 << 30, None) == want


def test_append_refusals(k2):
    kv = pool(k2)
    ref = C.addressof(kv)
    f = k2.LIB.k2_paged_append
    assert f(None, A, A, k2.K2_BF16, 256, 256, A, 1, None) == k2.K2_ERR_ARG
    assert f(ref, A, A, k2.K2_I8, 256, 256, A, 1, None) == k2.K2_ERR_UNSUPPORTED
    assert f(ref, A, A, k2.K2_BF16, 256, 256, A, -1, None) == k2.K2_ERR_ARG
    assert f(ref, None, A, k2.K2_BF16, 256, 256, A, 1, None) == k2.K2_ERR_ARG
    assert f(ref, A, A, k2.K2_BF16, 256, 256, None, 1, None) == k2.K2_ERR_ARG
    assert f(ref, A, A + 2, k2.K2_BF16, 256, 256, A, 1, None) == k2.K2_ERR_ARG
    assert f(ref, A, A, k2.K2_BF16, 257, 256, A, 2, None) == k2.K2_ERR_ARG
    assert f(ref, A, A, k2.K2_BF16, 128, 256, A, 2, None) == k2.K2_ERR_ARG
    assert f(ref, None, None, k2.K2_BF16, 0, 0, None, 0, None) == k2.K2_OK  # nothing to store


def test_attention_refusals(k2):
    kv = pool(k2)
    good = dict(kv=C.addressof(kv), q=A, dtype=k2.K2_F16, q_stride=1024, cu=A, kv_len=A, table=A, stride=4, requests=1,
                tokens=2, heads=8, max_q=1, scale=0.1, out=A, out_stride=1024, ws=A, ws_bytes=1 << 30, stream=None)

    def call(**kw):
        return k2.LIB.k2_paged_attention(*{**good, **kw}.values())
    for kw in (dict(kv=None), dict(q=None), dict(cu=None), dict(kv_len=None), dict(table=None), dict(out=None),
               dict(q=A + 4), dict(q_stride=1020), dict(out_stride=512), dict(scale=float("nan")),
               dict(scale=float("inf"))):
        assert call(**kw) == k2.K2_ERR_ARG, kw
    for kw in (dict(heads=7), dict(heads=0), dict(heads=34), dict(requests=-1), dict(requests=2049), dict(tokens=-1),
               dict(max_q=-1), dict(stride=0)):
        assert call(**kw) == k2.K2_ERR_SHAPE, kw
    assert call(dtype=k2.K2_F32) == k2.K2_ERR_UNSUPPORTED
    for kw in (dict(ws=None), dict(ws=A + 16), dict(ws_bytes=16)):
        assert call(**kw) == k2.K2_ERR_WORKSPACE, kw
    for kw in (dict(requests=0), dict(tokens=0), dict(max_q=0)):  # nothing to attend
        assert call(**kw) == k2.K2_OK, kw


def test_plan_refusals(k2):
    good = dict(cached=A, fresh=A, requests=1, block=16, table=A, stride=4, free=A, capacity=4, count=A, count_out=A,
                kv_len=A, cu=A, slots=A, positions=A, max_tokens=4, status=A, stream=None)

    def call(**kw):
        return k2.LIB.k2_paged_plan(*{**good, **kw}.values())
    for n in ("cached", "fresh", "table", "free", "count", "count_out", "kv_len", "cu", "slots", "positions", "status"):
        assert call(**{n: None}) == k2.K2_ERR_ARG, n
    assert call(block=8) == k2.K2_ERR_UNSUPPORTED
    for kw in (dict(requests=0), dict(requests=2049), dict(stride=0), dict(capacity=0), dict(max_tokens=0),
               dict(max_tokens=2 ** 30)):
        assert call(**kw) == k2.K2_ERR_SHAPE, kw


def test_rules_refusals(k2):
    def call(rows=2, vocab=40, ld=40, ld_out=40, x=A, y=A + 4096, **kw):
        u = k2.LogitRules(**kw)
        return k2.LIB.k2_adjust_logits(C.byref(u), x, ld, y, ld_out, rows, vocab, None)
    assert k2.LIB.k2_adjust_logits(None, A, 40, A, 40, 1, 40, None) == k2.K2_ERR_ARG
    for kw in (dict(rows=-1), dict(vocab=0), dict(x=None), dict(y=None), dict(x=A + 2), dict(y=A, ld=48),
               dict(repetition=A), dict(presence=A), dict(frequency=A), dict(ids=A), dict(ids=A, ids_len=A, ids_stride=-1),
               dict(bias_offset=A), dict(bias_offset=A, bias_ids=A, bias=A, n_bias=-1), dict(mask=A),
               dict(mask=A, n_masks=2, mask_stride=1)):
        assert call(**kw) == k2.K2_ERR_ARG, kw
    for kw in (dict(ld=39), dict(ld_out=39), dict(rows=65536)):
        assert call(**kw) == k2.K2_ERR_SHAPE, kw
    assert call(rows=0, x=None, y=None) == k2.K2_OK


def test_further_refusals(k2):
    """Counts that 32-bit indices could not pass, and an output over the queries."""
    ref = C.addressof(pool(k2))
    assert k2.LIB.k2_paged_append(ref, A, A, k2.K2_BF16, 256, 256, A, 2 ** 30 + 1, None) == k2.K2_ERR_ARG

    def attend(tokens, out):
        return k2.LIB.k2_paged_attention(ref, A, k2.K2_F16, 1024, A, A, A, 4, 1, tokens, 8, 1, 0.1, out, 1024, A, 1 << 30, None)
    assert attend(2 ** 30 + 1, 2 * A) == k2.K2_ERR_SHAPE
    assert attend(2, A) == k2.K2_ERR_ARG
    assert "queries" in k2.LIB.k2_last_error(None).decode()
    for kw, vocab in ((dict(ids=A, ids_len=A, ids_stride=2 ** 30 + 1), 40), (dict(), 2 ** 30 + 1),
                      (dict(bias_offset=A, bias_ids=A, bias=A, n_bias=2 ** 30 + 1), 40)):
        u = k2.LogitRules(**kw)
        assert k2.LIB.k2_adjust_logits(C.byref(u), A, vocab, A + 4096, vocab, 2, vocab, None) == k2.K2_ERR_ARG, kw


def test_packed_rules_are_the_structure(k2):
    """adjust_logits hands the call a packed k2_logit_rules: field by field what ctypes lays out."""
    values = [(7 * i + 3) << (20 if dict(k2.LogitRules._fields_)[n] is not C.c_int32 else 0)
              for i, (n, _) in enumerate(k2.LogitRules._fields_)]
    u = k2.LogitRules.from_buffer_copy(k2._RULES(*values).ljust(C.sizeof(k2.LogitRules), b"\0"))
    assert [getattr(u, n) for n, _ in k2.LogitRules._fields_] == values


# ---- the oracle ------------------------------------------------------------------------------

def test_plan_oracle_hands_out_and_takes_back_every_block_once():
    rng = np.random.default_rng(3)
    block, blocks, requests = 16, 40, 6
    table, free, count = np.full((requests, 12), -1), np.arange(blocks), blocks
    cached = np.zeros(requests, dtype=np.int64)
    for _ in range(60):
        fresh = np.array([int(rng.choice([-1, 0, 1, 1, 1, 20, 33])) for _ in range(requests)])
        got = P.plan(cached, fresh, table, free, count, block, 256)
        if got["status"][3]:
            assert np.array_equal(got["table"], table) and got["count"] == count
            fresh[:] = -1
            got = P.plan(cached, fresh, table, free, count, block, 256)
        table, free, count, cached = got["table"], got["free"], got["count"], got["kv_len"]
        held = [b for r in range(requests) for b in table[r, :-(-cached[r] // block)]]
        assert sorted(held + list(free[:count])) == list(range(blocks))
        t = got["slots"][got["slots"] >= 0]
        assert len(set(t)) == t.size == got["cu"][-1]


@pytest.mark.parametrize("cache", ["i8", "f8"])
def test_append_oracle_is_within_half_a_step(cache):
    rng = np.random.default_rng(5)
    codes, scale = np.zeros((2, 1, 16, 64), np.uint8), np.zeros((2, 1), np.float32)
    x = rng.standard_normal((16, 1, 64)).astype(np.float32)
    P.append(codes, scale, x, np.arange(16) + 16, cache)
    back = P.values(codes[1, 0], cache) * scale[1, 0]
    top = np.abs(x).max()
    assert np.isclose(scale[1, 0], top / P.QMAX[cache], rtol=1e-6)
    # int8: half a step of the scale; E4M3: half an ulp (2^-4), or half of the smallest step (2^-10)
    room = scale[1, 0] * 0.5 if cache == "i8" else np.maximum(np.abs(x[:, 0]) * 2.0 ** -4, scale[1, 0] * 2.0 ** -10)
    assert np.all(np.abs(back - x[:, 0]) <= room * (1 + 1e-5))
    assert not codes[0].any() and scale[0, 0] == 0


def test_attention_oracle_against_brute_force():
    rng = np.random.default_rng(7)
    k = rng.integers(0, 256, (3, 1, 16, 64)).astype(np.uint8)
    v = rng.integers(0, 256, (3, 1, 16, 64)).astype(np.uint8)
    ks, vs = np.full((3, 1), 0.01, np.float32), np.full((3, 1), 0.02, np.float32)
    q = rng.standard_normal((3, 2, 64)).astype(np.float32)
    table = np.array([[2, 0]])
    out, mass, _ = P.attention(q, [0, 2], [20], table, k, ks, v, vs, "i8", 0.125)
    kk = np.concatenate([k[2, 0], k[0, 0]]).view(np.int8) * np.float64(ks[0, 0])
    vv = np.concatenate([v[2, 0], v[0, 0]]).view(np.int8) * np.float64(vs[0, 0])
    for t, seen in ((0, 19), (1, 20)):
        for h in range(2):
            e = np.exp(kk[:seen] @ q[t, h].astype(np.float64) * 0.125)
            assert np.allclose(out[t, h], (e / e.sum()) @ vv[:seen], rtol=1e-10, atol=1e-12)
    assert np.all(np.isnan(out[2])) and np.all(mass[:2] >= np.abs(out[:2]) - 1e-12)


def test_rules_oracle_by_hand():
    x = np.array([[2.0, -2.0, 1.0, 0.5, 3.0]], np.float32)
    got = P.rules(x, repetition=np.array([2.0]), presence=np.array([0.25]), frequency=np.array([0.5]),
                  ids=np.array([[0, 1, 1, 9, -1, 1, 2]]), ids_len=np.array([6]), prompt_len=np.array([2]),
                  bias=(np.array([0, 2]), np.array([4, 4]), np.array([1.0, 2.0])), mask=np.array([[0b10111]], np.uint32))
    assert got.tolist() == [[1.0, -4.0 - 2 * 0.5 - 0.25, 1.0, -np.inf, 6.0]]
