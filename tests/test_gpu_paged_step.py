"""k2_paged_step: the model's layers over a block-paged 8-bit cache for many requests at once, against the oracle's
layers with the same paged cache (oracle/k2_paged.py), and in a whole served run with rules and sampling."""
import numpy as np
import pytest
import torch

import k2_inputs as ki
from oracle import k2_oracle as O
from oracle import k2_paged as P

pytestmark = pytest.mark.gpu

BLOCK, BLOCKS, COLS, ROWS = 16, 64, 16, 224


@pytest.fixture(scope="module")
def k2():
    from dense_gqa_decoder_gb300 import k2 as mod
    return mod


@pytest.fixture(scope="module")
def model():
    from dense_gqa_decoder_gb300 import model_io
    return model_io.build_context(ki.MEDIUM, max_context=256, max_batch=6, kv_dtype="f16", gain_scale=0.1, keep_host=True)


def dev(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


class Served:
    """The device side of a served run: pools, tables and the buffers of a step."""

    def __init__(self, k2, ctx, requests, cache, rows=ROWS):
        s = ki.MEDIUM
        z = lambda *n: torch.zeros(*n, dtype=torch.int32, device="cuda")  # noqa: E731
        self.k2, self.ctx = k2, ctx
        self.caches = [k2.PagedCache(BLOCKS, BLOCK, s.n_kv_heads, s.head_dim, cache) for _ in range(s.n_layers)]
        self.len, self.fresh, self.table = z(requests), z(requests), z(requests, COLS)
        self.free, self.count = torch.arange(BLOCKS, dtype=torch.int32, device="cuda"), dev([BLOCKS])
        self.cu, self.status, self.next = z(requests + 1), z(4), z(requests)
        self.tokens, self.slots, self.positions = z(rows), z(rows), z(rows)
        self.logits = torch.zeros(requests, s.vocab, device="cuda")
        self.ws = k2.paged_workspace()

    def step(self, max_new):
        self.k2.paged_plan(self.len, self.fresh, self.table, self.free, self.count, BLOCK, kv_len=self.len, cu_new=self.cu,
                           slots=self.slots, positions=self.positions, status=self.status)
        self.ctx.paged_step(self.caches, self.tokens, self.positions, self.slots, self.cu, self.len, self.table, max_new,
                            self.next, self.ws, logits=self.logits)

    def load(self, fresh, ids):
        self.fresh.copy_(dev(fresh))
        self.tokens.zero_()
        flat = [t for i in ids for t in i]
        if flat:
            self.tokens[:len(flat)] = dev(flat)


def rel(a, b):
    return float(np.linalg.norm(np.asarray(a, np.float64) - b) / np.linalg.norm(b))


# Relative L2 of a row of logits.  Queries, probabilities and outputs are fp16 (2^-11 each, averaged over dims and layers);
# with split 3, the default, all GEMM operands are (ten such roundings, as __graft_entry__'s bar).  What is larger: K and V
# differ from the oracle's in their last bits, so now and then a code falls to the neighbouring step.  For a request of
# one token, whose attention output is its V row, that moves one of 64 elements by up to 1/127 (int8) or 1/8 (E4M3: three
# bits of mantissa) of its magnitude, at most about 2.5 times the elements' root mean square: 2.5 / 8 of the row's norm,
# that is 1/127 * 0.31 = 0.25 % or 1/8 * 0.31 = 4 % of a KV head's output, and over sqrt(2) less of both heads' together:
# 0.17 % and 2.8 %.  So the bars are 1e-2 (five such codes) and 3e-2 (one), and the codes themselves are checked to be
# close to the oracle's.
@pytest.mark.parametrize("cache,split,bar", [("i8", 1, 1e-2), ("f8", 1, 3e-2), ("i8", 3, 1e-2), ("f8", 3, 3e-2)])
def test_prompts_decode_and_mixed_steps_match_the_oracle(k2, model, cache, split, bar):
    ctx, hostw = model
    ctx.set_option(k2.K2_OPT_PREFILL_SPLIT, split)
    s = ki.MEDIUM
    rng = np.random.default_rng(2)
    pm = P.PagedModel(O.OracleModel(s, lambda n, l: hostw[(n, l)], "f32"), BLOCKS, BLOCK, cache)
    sv = Served(k2, ctx, 5, cache)
    table, free, count, lens = np.zeros((5, COLS), int), np.arange(BLOCKS), BLOCKS, np.zeros(5, int)
    prompt = lambda n: [int(t) for t in rng.integers(0, s.vocab, n)]  # noqa: E731
    # prompts together; decode steps; a request ends, another comes while the rest decode; a step of few rows; none
    plan = [[prompt(40), prompt(7), prompt(130), [], []], None, None,
            [None, "end", None, prompt(33), []], None, [None, [], [], None, prompt(1)], [[], [], [], [], []], None]
    nxt = [0] * 5
    for what in plan:
        what = [None if lens[r] else [] for r in range(5)] if what is None else what
        ids = [([nxt[r]] if w is None else [] if w == "end" else w) for r, w in enumerate(what)]
        fresh = [-1 if w == "end" else len(i) for w, i in zip(what, ids)]
        sv.load(fresh, ids)
        before = sv.next.tolist()
        sv.step(max_new=130)
        got = P.plan(lens, fresh, table, free, count, BLOCK, ROWS)
        table, free, count, lens = got["table"], got["free"], got["count"], got["kv_len"]
        assert got["status"][3] == 0 and np.array_equal(sv.slots.cpu().numpy(), got["slots"])
        want = pm.step([t for i in ids for t in i], got["positions"], got["slots"], got["cu"], lens, table)
        have, after = sv.logits.cpu().numpy(), sv.next.tolist()
        for r in range(5):
            if not ids[r]:
                assert after[r] == before[r] and not have[r].any()
                continue
            assert rel(have[r], want[r]) <= bar, (r, rel(have[r], want[r]))
            assert after[r] == int(np.argmax(have[r]))
            nxt[r] = after[r]
    assert ctx.sync_status() == k2.K2_OK and all(int(c.flags) == 0 for c in sv.caches)
    ctx.set_option(k2.K2_OPT_PREFILL_SPLIT, 3)
    # The caches: K and V are linear images of the normalised residual, whose relative error is within `bar`: so a block's
    # largest value (some 2.5 times the root mean square) is within 4 / 2.5 bar, 4 times the root mean square of the errors
    # being the worst of many.  Values in units of the scale, of which the root mean square is some 40 steps of int8 or 180
    # of E4M3's 448: within 4 bar of that, and the rounding (an earlier one too) by a step or, in E4M3, 1/8 of the value.
    for c, pool in zip(sv.caches, pm.pools):
        for have, want, hs, ws in ((c.k, pool[0], c.k_scale, pool[1]), (c.v, pool[2], c.v_scale, pool[3])):
            assert np.allclose(hs.cpu().numpy(), ws, rtol=2 * bar)
            h, w = P.values(have.view(torch.uint8).cpu().numpy(), cache), P.values(want, cache)
            assert (np.abs(h - w) <= (3 if cache == "i8" else 0.25 * np.abs(w) + 448 * 2.0 ** -8 + 180 * 4 * bar)).all()


def test_the_contexts_own_sequences_are_untouched(k2, model):
    ctx, _ = model
    s = ki.MEDIUM
    ctx.kv_reset()
    ctx.prefill(0, torch.randint(0, s.vocab, (30,), dtype=torch.int32, device="cuda"), dev([0]))
    before = ctx.kv_save(0).clone()
    sv = Served(k2, ctx, 3, "i8")
    sv.load([50, 1, 0], [[5] * 50, [7], []])
    sv.step(max_new=50)
    assert torch.equal(ctx.kv_save(0), before) and ctx.kv_view(0, 0)[4] == 30


def test_a_captured_decode_step_feeds_itself(k2, model):
    """Plan, layers, rules and sampling of a decode step in one graph, replayed with the tokens it drew: lengths, tables
    and rules move along, and a replay gives the logits of the same calls made one by one (to the bar of a code or two:
    the GEMMs add their parts in any order)."""
    ctx, _ = model
    s = ki.MEDIUM
    ctx.set_sampling(k2.sampling(temperature=0.8, top_k=40, seed=11))
    try:
        sv = Served(k2, ctx, 4, "i8", rows=64)
        gen = torch.Generator("cuda").manual_seed(3)
        lens = [12, 1, 30, 17]
        ids = torch.randint(0, s.vocab, (60,), device="cuda", generator=gen, dtype=torch.int32)
        sv.load(lens, [i.tolist() for i in ids.split(lens)])
        sv.step(max_new=30)
        hist, ban = torch.zeros(4, 64, dtype=torch.int32, device="cuda"), torch.full((1, 32), -1, dtype=torch.int32, device="cuda")
        ban[0, :8] = 0  # ids below 256 are not allowed
        zero, hlen, rep = dev([0] * 4), dev([1] * 4), torch.full((4,), 1.3, device="cuda")
        small = Served(k2, ctx, 4, "i8", rows=4)
        for n in ("caches", "len", "table", "free", "count", "next"):
            setattr(small, n, getattr(sv, n))
        small.fresh.fill_(1)

        def step():
            small.tokens.copy_(sv.next)
            hist.scatter_(1, hlen[:, None].long(), sv.next[:, None])
            hlen.add_(1)
            small.step(max_new=1)
            k2.adjust_logits(small.logits, repetition=rep, ids=hist, ids_len=hlen, mask=ban, mask_row=zero)
            ctx.sample_logits(small.logits, 4, small.len, sv.next)

        kept = (sv.len, sv.table, sv.free, sv.count, sv.next, hist, hlen)
        step()
        g, state = torch.cuda.CUDAGraph(), [t.clone() for t in kept]
        with torch.cuda.graph(g):
            step()
        step()
        one_by_one = small.logits.clone()
        for t, v in zip(kept, state):
            t.copy_(v)
        g.replay()  # (the rows appended again at the same slots leave the same codes)
        assert torch.equal(torch.isinf(small.logits), torch.isinf(one_by_one)) and torch.isinf(one_by_one[:, :256]).all()
        assert rel(small.logits[:, 256:].cpu().numpy(), one_by_one[:, 256:].cpu().numpy()) <= 1e-2
        for i in range(20):
            g.replay()
            assert all(t >= 256 for t in sv.next.tolist()) and sv.len.tolist() == [n + 3 + i for n in lens]
        assert small.status.tolist()[3] == 0 and ctx.sync_status() == k2.K2_OK
    finally:
        ctx.set_sampling(None)


def test_paged_step_refusals(k2, model):
    ctx, _ = model
    sv = Served(k2, ctx, 3, "i8")
    s = ki.MEDIUM

    def call(status=None, **kw):
        a = dict(caches=sv.caches, tokens=sv.tokens, positions=sv.positions, slots=sv.slots, cu_new=sv.cu, kv_len=sv.len,
                 table=sv.table, max_new=4, next_tokens=sv.next, workspace=sv.ws, **{})
        a.update(kw)
        with pytest.raises(ValueError if status is None else k2.K2Error) as e:
            ctx.paged_step(**a)
        if status is not None:
            assert e.value.status == status and str(e.value)
    call(caches=sv.caches[:2])
    call(tokens=sv.tokens.long())
    call(slots=sv.slots[:5])
    call(logits=torch.zeros(3, 5, device="cuda"))
    other = [k2.PagedCache(4, 16, 1, s.head_dim)] * s.n_layers
    call(k2.K2_ERR_SHAPE, caches=other)
    call(k2.K2_ERR_SHAPE, max_new=0)
    call(k2.K2_ERR_WORKSPACE, workspace=sv.ws[:1024])
    z = lambda *n: torch.zeros(*n, dtype=torch.int32, device="cuda")  # noqa: E731
    call(k2.K2_ERR_SHAPE, tokens=z(257), positions=z(257), slots=z(257))
    call(k2.K2_ERR_SHAPE, cu_new=z(8), kv_len=z(7), table=z(7, 4), next_tokens=z(7))
    from dense_gqa_decoder_gb300 import model_io
    tiny, _ = model_io.build_context(ki.TINY, max_context=32, kv_dtype="f32")
    caches = [k2.PagedCache(4, 16, 2, 64)] * ki.TINY.n_layers
    with pytest.raises(k2.K2Error) as e:
        tiny.paged_step(caches, z(1), z(1), z(1), z(2), z(1), z(1, 1), 1, z(1), sv.ws)
    assert e.value.status == k2.K2_ERR_UNSUPPORTED


def test_a_position_beyond_the_rope_table_raises_the_guard(k2, model):
    ctx, _ = model
    sv = Served(k2, ctx, 2, "i8")
    sv.load([3, 0], [[1, 2, 3], []])
    sv.step(max_new=3)
    assert ctx.sync_status() == k2.K2_OK
    sv.positions.fill_(1 << 20)
    ctx.paged_step(sv.caches, sv.tokens, sv.positions, sv.slots, sv.cu, sv.len, sv.table, 3, sv.next, sv.ws)
    assert ctx.sync_status() == k2.K2_ERR_DEVICE_GUARD
    ctx.clear_status()
    assert ctx.sync_status() == k2.K2_OK
