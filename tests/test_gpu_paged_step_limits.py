"""k2_paged_step with more requests than one 16-token tile, as decode and as mixed steps, and captured with enough rows
that the layers' matrices are converted beside them.  Against the oracle's layers, to the bars of test_gpu_paged_step.py."""
import numpy as np
import pytest
import torch

import k2_inputs as ki
from oracle import k2_oracle as O
from oracle import k2_paged as P
from test_gpu_paged_step import dev, rel

pytestmark = pytest.mark.gpu

BLOCK, BLOCKS, COLS, REQUESTS = 16, 160, 8, 20


@pytest.fixture(scope="module")
def k2():
    from dense_gqa_decoder_gb300 import k2 as mod
    return mod


@pytest.fixture(scope="module")
def model():
    from dense_gqa_decoder_gb300 import model_io
    return model_io.build_context(ki.MEDIUM, max_context=256, max_batch=24, kv_dtype="f16", gain_scale=0.1, keep_host=True)


class Run:
    """Twenty requests over int8 pools: the device's side and the oracle's."""

    def __init__(self, k2, model, rows):
        (self.ctx, hostw), s = model, ki.MEDIUM
        z = lambda *n: torch.zeros(*n, dtype=torch.int32, device="cuda")  # noqa: E731
        self.k2, self.rows = k2, rows
        self.caches = [k2.PagedCache(BLOCKS, BLOCK, s.n_kv_heads, s.head_dim, "i8") for _ in range(s.n_layers)]
        self.len, self.fresh, self.table = z(REQUESTS), z(REQUESTS), z(REQUESTS, COLS)
        self.free, self.count = torch.arange(BLOCKS, dtype=torch.int32, device="cuda"), dev([BLOCKS])
        self.cu, self.status, self.next = z(REQUESTS + 1), z(4), z(REQUESTS)
        self.tokens, self.slots, self.positions = z(rows), z(rows), z(rows)
        self.logits = torch.zeros(REQUESTS, s.vocab, device="cuda")
        self.ws = k2.paged_workspace()
        self.pm = P.PagedModel(O.OracleModel(s, lambda n, l: hostw[(n, l)], "f32"), BLOCKS, BLOCK, "i8")
        self.state = (np.zeros((REQUESTS, COLS), int), np.arange(BLOCKS), BLOCKS, np.zeros(REQUESTS, int))

    def load(self, ids):
        self.fresh.copy_(dev([len(i) for i in ids]))
        self.tokens.zero_()
        flat = [t for i in ids for t in i]
        self.tokens[:len(flat)] = dev(flat)

    def enqueue(self, max_new):
        self.k2.paged_plan(self.len, self.fresh, self.table, self.free, self.count, BLOCK, kv_len=self.len, cu_new=self.cu,
                           slots=self.slots, positions=self.positions, status=self.status)
        self.ctx.paged_step(self.caches, self.tokens, self.positions, self.slots, self.cu, self.len, self.table, max_new,
                            self.next, self.ws, logits=self.logits)

    def check(self, ids, before, bar=1e-2):
        table, free, count, lens = self.state
        got = P.plan(lens, [len(i) for i in ids], table, free, count, BLOCK, self.rows)
        self.state = got["table"], got["free"], got["count"], got["kv_len"]
        assert got["status"][3] == 0 and np.array_equal(self.slots.cpu().numpy(), got["slots"])
        want = self.pm.step([t for i in ids for t in i], got["positions"], got["slots"], got["cu"], got["kv_len"], got["table"])
        have, after = self.logits.cpu().numpy(), self.next.tolist()
        for r in range(REQUESTS):
            if not ids[r]:
                assert after[r] == before[r] and not have[r].any()
                continue
            assert rel(have[r], want[r]) <= bar, (r, rel(have[r], want[r]))
            assert after[r] == int(np.argmax(have[r]))
        assert self.ctx.sync_status() == self.k2.K2_OK and all(int(c.flags) == 0 for c in self.caches)


def steps(rng):
    """Prompts of 1 to 9 tokens, decode steps, a mixed step, and one where most requests rest."""
    ids = lambda n: [int(t) for t in rng.integers(0, ki.MEDIUM.vocab, n)]  # noqa: E731
    yield [ids(1 + r % 9) for r in range(REQUESTS)]
    yield [ids(1) for _ in range(REQUESTS)]
    yield [ids(30 if r == 4 else r % 2) for r in range(REQUESTS)]
    yield [ids(1 if r in (3, 19) else 0) for r in range(REQUESTS)]


@pytest.mark.parametrize("split", [1, 3])
@pytest.mark.parametrize("graph", [False, True])
def test_twenty_requests(k2, model, split, graph):
    """Run eagerly, and replayed from one capture of a step that every later one fits."""
    run = Run(k2, model, 112)
    run.ctx.set_option(k2.K2_OPT_PREFILL_SPLIT, split)
    try:
        replay = None
        if graph:
            run.enqueue(30)  # (nothing to do: every length is 0)
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                run.enqueue(30)
            replay = g.replay
        for ids in steps(np.random.default_rng(51)):
            run.load(ids)
            before = run.next.tolist()
            replay() if graph else run.enqueue(30)
            run.check(ids, before)
    finally:
        run.ctx.set_option(k2.K2_OPT_PREFILL_SPLIT, 3)


@pytest.mark.parametrize("split", [1, 3])
def test_twenty_requests_decode_without_padding(k2, model, split):
    """As many rows as tokens: a step of single tokens takes the kernel for few rows alone."""
    run = Run(k2, model, REQUESTS)
    run.ctx.set_option(k2.K2_OPT_PREFILL_SPLIT, split)
    try:
        rng = np.random.default_rng(52)
        for _ in range(3):
            ids = [[int(t)] for t in rng.integers(0, ki.MEDIUM.vocab, REQUESTS)]
            run.load(ids)
            before = run.next.tolist()
            run.enqueue(1)
            run.check(ids, before)
    finally:
        run.ctx.set_option(k2.K2_OPT_PREFILL_SPLIT, 3)
