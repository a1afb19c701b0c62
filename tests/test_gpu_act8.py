"""fp8 weights with E4M3 activations (option K2_OPT_ACT8): prefill blocks and k2_paged_step against the oracle's layers whose
projections round their rows to codes (oracle/k2_linear.py)."""
import numpy as np
import pytest
import torch

import k2_inputs as ki
from oracle import k2_fp8 as Q8
from oracle import k2_linear as L
from oracle import k2_oracle as O
from oracle import k2_paged as P

pytestmark = pytest.mark.gpu

RAGGED = ki.MEDIUM.replace(hidden=640, n_layers=2, intermediate=1664)
ODD = ki.MEDIUM.replace(hidden=200, n_layers=2, n_heads=4, n_kv_heads=1, intermediate=328, vocab=301)
SHAPES = {"medium": ki.MEDIUM, "ragged": RAGGED, "odd": ODD, "layer": ki.K2_LAYER}

# Relative L2 of a row of logits.  The oracle rounds where the library does, but what enters a rounding to codes differs a
# little (1e-6 behind a norm, 2^-11 behind the attention), so some values fall to the neighbouring code; each such step is up to
# 2^-3 of the value, and what follows in later layers is rounded from other numbers altogether.  At worst the two roundings are
# independent: library = exact + n1, oracle = exact + n2 with errors of the same size, and |n1 - n2| = sqrt(2) |n2|.  So the bar
# is 1.5 times the distance of the rounding oracle from the one that rounds nothing, and what the cache and the attention may
# differ by where nothing is rounded to codes: the bars of those tests, 1e-2 (fp16 and int8 pools, five codes of a row), 3e-2
# (E4M3 pools) and 5e-2 (int8 caches).


@pytest.fixture(scope="module")
def k2():
    from dense_gqa_decoder_gb300 import k2 as mod
    return mod


@pytest.fixture(scope="module")
def mio():
    from dense_gqa_decoder_gb300 import model_io
    return model_io


def rel(a, b):
    return float(np.linalg.norm(np.asarray(a, np.float64) - b) / np.linalg.norm(b))


def weights_of(host):
    return Q8.fp8_weights(lambda n, l: host[(n, l)])


def prefill(k2, ctx, ids, vocab, steps=4):
    ctx.kv_reset()
    nxt = torch.zeros(1, dtype=torch.int32, device="cuda")
    logits = torch.empty(vocab, device="cuda")
    ctx.prefill(0, torch.tensor(ids, dtype=torch.int32, device="cuda"), nxt, logits)
    toks, rows = [int(nxt)], [logits.cpu().numpy().copy()]
    for _ in range(steps):
        ctx.decode_step(nxt, 1, nxt, logits)
        toks.append(int(nxt))
        rows.append(logits.cpu().numpy().copy())
    assert ctx.sync_status() == k2.K2_OK
    return toks, np.stack(rows)


@pytest.mark.parametrize("shape,kv,n", [("medium", "f16", 40), ("medium", "i8", 9), ("medium", "f16", 250), ("ragged", "f16", 17),
                                        ("odd", "f16", 70), ("odd", "i8", 33), ("layer", "f16", 300)])
def test_prefill_matches_the_oracle(k2, mio, shape, kv, n):
    s = SHAPES[shape]
    ctx, host = mio.build_context(s, max_context=n + 16, kv_dtype=kv, gain_scale=0.1, keep_host=True, weights="f8")
    assert ctx.info().tc_prefill == 1
    ids = ki.prompt_ids(s.vocab, n, seed=51)
    before = prefill(k2, ctx, ids, s.vocab)
    ctx.set_option(k2.K2_OPT_ACT8, 1)
    toks, got = prefill(k2, ctx, ids, s.vocab)
    # the prompt but its last token on codes, then (over the same cache) what the persistent step computes
    plain = O.OracleModel(s, weights_of(host), kv)
    rounded = L.act8(O.OracleModel(s, weights_of(host), kv), "f16" if kv == "f16" else "bf16")
    cache, exact = plain.new_cache(n + 16), plain.new_cache(n + 16)
    rounded.run(ids[:-1], cache, None)
    plain.run(ids[:-1], exact, None)
    for t, row in zip([ids[-1]] + toks[:-1], got):
        (_, want), (_, without) = plain.run(np.array([t]), cache), plain.run(np.array([t]), exact)
        bar = 1.5 * rel(without[0], want[0]) + (1e-2 if kv == "f16" else 5e-2)
        assert bar < 0.15 and rel(row, want[0]) <= bar, (rel(row, want[0]), bar)
    # the codes cost something, and the option leaves nothing behind
    assert rel(got, before[1]) > 1e-4
    ctx.set_option(k2.K2_OPT_ACT8, 0)
    again = prefill(k2, ctx, ids, s.vocab)
    assert rel(again[1][0], before[1][0]) <= 2e-4  # that path adds shares of K in any order


class Served:
    """The device side of a served run over an fp8 model."""

    def __init__(self, k2, ctx, s, requests, cache, rows=224):
        z = lambda *n: torch.zeros(*n, dtype=torch.int32, device="cuda")  # noqa: E731
        self.k2, self.ctx = k2, ctx
        self.caches = [k2.PagedCache(64, 16, s.n_kv_heads, s.head_dim, cache) for _ in range(s.n_layers)]
        self.len, self.fresh, self.table = z(requests), z(requests), z(requests, 16)
        self.free, self.count = torch.arange(64, dtype=torch.int32, device="cuda"), z(1) + 64
        self.cu, self.status, self.next = z(requests + 1), z(4), z(requests)
        self.tokens, self.slots, self.positions = z(rows), z(rows), z(rows)
        self.logits = torch.zeros(requests, s.vocab, device="cuda")
        self.ws = k2.paged_workspace()

    def load(self, fresh, ids):
        self.fresh.copy_(torch.tensor(fresh, dtype=torch.int32))
        flat = [t for i in ids for t in i]
        self.tokens.zero_()
        self.tokens[:len(flat)] = torch.tensor(flat, dtype=torch.int32, device="cuda")

    def step(self, max_new):
        self.k2.paged_plan(self.len, self.fresh, self.table, self.free, self.count, 16, kv_len=self.len, cu_new=self.cu,
                           slots=self.slots, positions=self.positions, status=self.status)
        self.ctx.paged_step(self.caches, self.tokens, self.positions, self.slots, self.cu, self.len, self.table, max_new,
                            self.next, self.ws, logits=self.logits)


@pytest.mark.parametrize("shape,cache,rows", [("medium", "i8", 224), ("medium", "f8", 224), ("ragged", "i8", 180)])
def test_paged_steps_match_the_oracle(k2, mio, shape, cache, rows):
    s = SHAPES[shape]
    ctx, host = mio.build_context(s, max_context=256, max_batch=6, kv_dtype="f16", gain_scale=0.1, keep_host=True, weights="f8")
    ctx.set_option(k2.K2_OPT_ACT8, 1)
    pm = P.PagedModel(L.act8(O.OracleModel(s, weights_of(host), "f32")), 64, 16, cache)
    exact = P.PagedModel(O.OracleModel(s, weights_of(host), "f32"), 64, 16, cache)
    sv = Served(k2, ctx, s, 5, cache, rows)
    rng = np.random.default_rng(3)
    prompt = lambda n: [int(t) for t in rng.integers(0, s.vocab, n)]  # noqa: E731
    table, free, count, lens, nxt = np.zeros((5, 16), int), np.arange(64), 64, np.zeros(5, int), [0] * 5
    for what in ([prompt(40), prompt(7), prompt(130), [], []], None, None, [None, "end", None, prompt(33), prompt(1)], None):
        what = [None if lens[r] else [] for r in range(5)] if what is None else what
        ids = [([nxt[r]] if w is None else [] if w == "end" else w) for r, w in enumerate(what)]
        fresh = [-1 if w == "end" else len(i) for w, i in zip(what, ids)]
        sv.load(fresh, ids)
        sv.step(max_new=130)
        got = P.plan(lens, fresh, table, free, count, 16, rows)
        table, free, count, lens = got["table"], got["free"], got["count"], got["kv_len"]
        want, without = (m.step([t for i in ids for t in i], got["positions"], got["slots"], got["cu"], lens, table) for m in (pm, exact))
        have = sv.logits.cpu().numpy()
        for r in range(5):
            if not ids[r]:
                assert not have[r].any()
                continue
            bar = 1.5 * rel(without[r], want[r]) + (1e-2 if cache == "i8" else 3e-2)
            assert bar < 0.25 and rel(have[r], want[r]) <= bar, (r, rel(have[r], want[r]), bar)
            nxt[r] = int(sv.next[r])
            assert nxt[r] == int(np.argmax(have[r]))
    assert ctx.sync_status() == k2.K2_OK and all(int(c.flags) == 0 for c in sv.caches)


def test_a_captured_paged_step_equals_eager_ones(k2, mio):
    s = ki.MEDIUM
    ctx, _ = mio.build_context(s, max_context=256, max_batch=6, kv_dtype="f16", gain_scale=0.1, weights="f8")
    ctx.set_option(k2.K2_OPT_ACT8, 1)
    runs = []
    for captured in (False, True):
        sv = Served(k2, ctx, s, 4, "i8", rows=40)
        rng = np.random.default_rng(4)
        ids = [[int(t) for t in rng.integers(0, s.vocab, n)] for n in (20, 3, 9, 1)]
        sv.load([len(i) for i in ids], ids)
        sv.step(max_new=32)
        sv.load([1, 1, 1, 1], [[int(t)] for t in sv.next.tolist()])
        out = []
        if captured:
            side = torch.cuda.Stream()
            side.wait_stream(torch.cuda.current_stream())
            graph = torch.cuda.CUDAGraph()
            keep = [t.clone() for t in (sv.len, sv.table, sv.free, sv.count, sv.next)]
            with torch.cuda.graph(graph, stream=side):
                sv.k2.paged_plan(sv.len, sv.fresh, sv.table, sv.free, sv.count, 16, kv_len=sv.len, cu_new=sv.cu, slots=sv.slots,
                                 positions=sv.positions, status=sv.status)
                ctx.paged_step(sv.caches, sv.tokens, sv.positions, sv.slots, sv.cu, sv.len, sv.table, 32, sv.next, sv.ws,
                               logits=sv.logits, stream=torch.cuda.current_stream())
            for t, k in zip((sv.len, sv.table, sv.free, sv.count, sv.next), keep):
                assert torch.equal(t, k)
        for _ in range(3):
            graph.replay() if captured else sv.step(max_new=32)
            out.append(sv.logits.clone())
            sv.tokens[:4] = sv.next
        assert ctx.sync_status() == k2.K2_OK
        runs.append(out)
    for a, b in zip(*runs):
        assert torch.equal(a, b)


def test_refusals(k2, mio):
    for shape, weights in ((ki.MEDIUM, None), (ki.MEDIUM, "q4"), (ki.TINY, None)):
        ctx, _ = mio.build_context(shape, max_context=32, kv_dtype="f32" if shape is ki.TINY else "f16", weights=weights)
        with pytest.raises(k2.K2Error) as e:
            ctx.set_option(k2.K2_OPT_ACT8, 1)
        assert e.value.status == k2.K2_ERR_UNSUPPORTED
        ctx.set_option(k2.K2_OPT_ACT8, 0)
    ctx, _ = mio.build_context(ki.MEDIUM, max_context=64, max_batch=6, kv_dtype="f16", weights="f8")
    for value in (-1, 2):
        with pytest.raises(k2.K2Error) as e:
            ctx.set_option(k2.K2_OPT_ACT8, value)
        assert e.value.status == k2.K2_ERR_ARG
    sv = Served(k2, ctx, ki.MEDIUM, 2, "i8", rows=20)
    sv.load([3, 0], [[1, 2, 3], []])
    with pytest.raises(k2.K2Error) as e:  # without the option
        sv.step(max_new=3)
    assert e.value.status == k2.K2_ERR_UNSUPPORTED
