"""The paged operators at the ends of what they accept: block scales of any size, one-signed queries under small
int8 codes, token sums beyond 32 bits, attention whose waits run out.  Against the plain oracle (oracle/k2_paged.py),
with the bounds of test_gpu_paged.py and the terms stated here."""
import numpy as np
import pytest
import torch

from oracle import k2_paged as P
from test_gpu_paged import attention_case, bound, check_plan, dev, host, plan_state, raw

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def k2():
    from dense_gqa_decoder_gb300 import k2 as mod
    return mod


def attend(k2, c, table, cu, kv_len, q, max_q=None, workspace=None, scale=None):
    out = torch.full_like(q, 7.0)
    k2.paged_attention(c, q, out, dev(cu), dev(kv_len), dev(table), int(np.diff(cu).max()) if max_q is None else max_q,
                       k2.paged_workspace() if workspace is None else workspace, scale=scale)
    return out


def oracle(c, table, cu, kv_len, q, cache, scale=None):
    return P.attention(host(q.float()), cu, kv_len, table, raw(c.k), host(c.k_scale), raw(c.v), host(c.v_scale), cache,
                       c.head_dim ** -0.5 if scale is None else scale)


def check(k2, c, table, cu, kv_len, q, cache, kind, **kw):
    """Every row within its bound, those of no request untouched.  bf16 outputs below 2^-126 have a step of 2^-133, of
    which half is lost, and fp32 numbers below it one of 2^-149: the products with the scale and 1 / sum and the joins
    lose less than 2^-140 by that."""
    got = host(attend(k2, c, table, cu, kv_len, q, **kw).float()).astype(np.float64)
    want, mass, score = oracle(c, table, cu, kv_len, q, cache)
    rows = ~np.isnan(want[:, 0, 0])
    assert (got[~rows] == 7.0).all()
    vmax = float(np.nanmax(host(c.v_scale).astype(np.float64))) * (127 if cache == "i8" else 448)
    room = bound(want, mass, score, int(max(kv_len)), c.head_dim, kind, vmax) + 2.0 ** -134 + 2.0 ** -140
    assert np.isfinite(got[rows]).all()
    worst = (np.abs(got - want) / room)[rows].max()
    assert worst <= 1.0, float(worst)


FEW = [[(90, 1), (40, 1), (700, 1)], [(70, 3), (33, 2)]]
CHUNK = [[(100, 60), (300, 1)], [(0, 70), (500, 40)]]
TINY = [1e-45, 1e-40, 1e-36, 4e-35, 1e-30]


def check_v_scales(k2, pairs, cache, kind, size):
    """All V scales about `size`, then blocks of that size before, behind and between blocks of scale about 1."""
    c, table, cu, kv_len, q = attention_case(k2, pairs, 16, 8, 2, 128, cache, kind, 41)
    usual = torch.where(torch.isnan(c.v_scale), 1.0, c.v_scale * 100.0)
    small = (usual.double() * size).clamp(min=1.5e-45).float()
    blocks = -(-int(kv_len[0]) // 16)
    first = torch.tensor(table[:, 0].copy(), device="cuda").long()
    last = torch.tensor([table[r, -(-int(n) // 16) - 1] for r, n in enumerate(kv_len)], device="cuda").long()
    odd = torch.tensor(np.unique(table[:, 1:blocks:2][table[:, 1:blocks:2] >= 0]), device="cuda").long()
    c.v_scale.copy_(small)
    check(k2, c, table, cu, kv_len, q, cache, kind)
    for where in (first, last, odd):
        c.v_scale.copy_(usual)
        c.v_scale[where] = small[where]
        check(k2, c, table, cu, kv_len, q, cache, kind)


@pytest.mark.parametrize("size", TINY)
@pytest.mark.parametrize("cache,kind", [("i8", "bf16"), ("f8", "f16"), ("i8", "f16"), ("f8", "bf16")])
@pytest.mark.parametrize("pairs", FEW)
def test_few_rows_under_v_scales_of_any_size(k2, pairs, cache, kind, size):
    check_v_scales(k2, pairs, cache, kind, size)


@pytest.mark.parametrize("size", TINY)
@pytest.mark.parametrize("cache,kind", [("i8", "bf16"), ("f8", "f16"), ("i8", "f16"), ("f8", "bf16")])
@pytest.mark.parametrize("pairs", CHUNK)
def test_chunks_under_v_scales_of_any_size(k2, pairs, cache, kind, size):
    check_v_scales(k2, pairs, cache, kind, size)


@pytest.mark.parametrize("requests,fresh", [(2, 2 ** 30), (33, 2 ** 26), (4, 2 ** 29)])
@pytest.mark.parametrize("max_tokens", [64, 3000])
@pytest.mark.parametrize("enough", [False, True])
def test_a_plan_whose_tokens_pass_31_bits_is_refused(k2, requests, fresh, max_tokens, enough):
    """New tokens that sum to 2^31 or more although each request's fit its table, and all of them the pool."""
    stride = fresh // 128
    table, free, count = plan_state([0] * requests, stride, requests * stride if enough else 40, 128, 45)
    got = check_plan(k2, [0] * requests, [fresh] * requests, table, free, count, 128, max_tokens)
    assert got["status"][3] == P.TOKENS_FULL | (0 if enough else P.NO_BLOCKS)


def one_signed_case(k2, pairs, dim, kind, outlier):
    """int8 K codes of -1, 0 and 1 under queries of one sign (or with one large dim): a query row's sum of magnitudes
    times a full-scale code is some hundred times any of its scores."""
    c, table, cu, kv_len, q = attention_case(k2, pairs, 16, 8, 2, dim, "i8", kind, 43)
    rng = np.random.default_rng(44)
    c.k.copy_(torch.from_numpy(rng.integers(-1, 2, tuple(c.k.shape)).astype(np.int8)))
    q.copy_((q.float().abs() * 200.0).to(q.dtype))
    if outlier:
        q.mul_(1 / 64)
        q[:, :, 5] = 4000.0
    return c, table, cu, kv_len, q


@pytest.mark.parametrize("outlier", [False, True])
@pytest.mark.parametrize("dim,kind", [(128, "f16"), (64, "bf16"), (64, "f16"), (128, "bf16")])
@pytest.mark.parametrize("pairs", FEW)
def test_few_rows_of_one_signed_queries(k2, pairs, dim, kind, outlier):
    """The scores' error follows what their own products add up to, not the largest code's: the bound's score term is
    the sum of |q_d k_jd| over the visible keys' codes, and every code enters exactly."""
    check(k2, *one_signed_case(k2, pairs, dim, kind, outlier), "i8", kind)


@pytest.mark.parametrize("outlier", [False, True])
@pytest.mark.parametrize("dim,kind", [(128, "f16"), (64, "bf16"), (64, "f16"), (128, "bf16")])
@pytest.mark.parametrize("pairs", CHUNK)
def test_chunks_of_one_signed_queries(k2, pairs, dim, kind, outlier):
    check(k2, *one_signed_case(k2, pairs, dim, kind, outlier), "i8", kind)


@pytest.mark.parametrize("pairs,block,dim,cache", [([(6000, 200), (500, 1), (0, 300)], 16, 128, "i8"),
                                                   ([(9000, 40), (40, 500)], 64, 64, "f8")])
def test_attention_whose_waits_run_out(k2, pairs, block, dim, cache):
    """A wait limit of a microsecond, shorter than a key tile takes from memory to the scores: the call ends, says so, and
    gives each head of a row whole or as NaN.  The next call on the same workspace, with time, is right."""
    c, table, cu, kv_len, q = attention_case(k2, pairs, block, 8, 2, dim, cache, "f16", 46)
    ws = k2.paged_workspace()
    want, mass, score = oracle(c, table, cu, kv_len, q, cache)
    rows = ~np.isnan(want[:, 0, 0])
    vmax = float(np.nanmax(host(c.v_scale))) * (127 if cache == "i8" else 448)
    room = bound(want, mass, score, int(max(kv_len)), dim, "f16", vmax)
    c.desc.wait_limit_us = 1
    got = host(attend(k2, c, table, cu, kv_len, q, workspace=ws).float()).astype(np.float64)
    assert int(c.flags) == k2.K2_PAGED_TIMEOUT
    lost = np.isnan(got).all(-1)
    assert lost[rows].any() and not np.isnan(got[~lost]).any() and (got[~rows] == 7.0).all()
    assert (np.abs(got - want)[rows][~lost[rows]] <= room[rows][~lost[rows]]).all()
    for r, (_, n) in enumerate(pairs):  # single tokens wait for nobody
        assert n > 1 or not lost[cu[r]:cu[r + 1]].any()
    c.desc.wait_limit_us = 0
    c.flags.zero_()
    check(k2, c, table, cu, kv_len, q, cache, "f16", workspace=ws)
    assert int(c.flags) == 0


CONTRADICTIONS = [  # new and cached tokens as given, then the call's lengths and the requests that contradict themselves
    ([(30, 2), (30, 1)], [0, 2, 3], [1, 20], 2, {0}), ([(30, 2), (30, 1)], [0, 2, 3], [20, -4], 2, {1}),
    ([(30, 2), (30, 1)], [0, 2, 3], [2 ** 31 - 1, 20], 2, {0}), ([(30, 2), (30, 1)], [0, 2, 900], [20, 900], 900, {1}),
    ([(30, 2), (30, 1)], [0, 3, 2], [20, 20], 3, {1}), ([(30, 2), (30, 1)], [0, 2, 3], [20, 20], 1, {0}),
    ([(30, 2), (30, 1)], [-1, 1, 3], [20, 20], 2, {0}),
    ([(100, 60), (30, 1), (50, 40)], [0, 60, 61, 101], [160, 31, 39], 60, {2}),
    ([(100, 60), (30, 1), (50, 40)], [0, 60, 61, 101], [59, 31, 90], 60, {0}),
    ([(100, 60), (30, 1), (50, 40)], [0, 60, 61, 101], [160, 0, 90], 60, {1}),
    ([(100, 60), (30, 1), (50, 40)], [0, 60, 61, 101], [160, 31, 90], 40, {0}),
    ([(100, 60), (30, 1), (50, 40)], [0, 60, 61, 101], [160, 31, 2000], 60, {2})]


@pytest.mark.parametrize("pairs,cu,kv_len,max_q,faulty", CONTRADICTIONS)
def test_contradictory_lengths_cost_their_request_alone(k2, pairs, cu, kv_len, max_q, faulty):
    """Zeros in the faulty requests' rows as far as they lie inside the query rows, the others' results as ever, and rows
    of no request untouched."""
    c, table, _, _, q = attention_case(k2, pairs, 16, 4, 1, 64, "i8", "f16", 47)
    got = host(attend(k2, c, table, cu, kv_len, q, max_q=max_q).float()).astype(np.float64)
    assert int(c.flags) == k2.K2_PAGED_BAD_LENGTH
    free = np.ones(q.shape[0], bool)
    for r in range(len(pairs)):
        lo, hi = max(cu[r], 0), min(cu[r + 1], q.shape[0])
        free[lo:hi] = False
        if r in faulty:
            assert not got[lo:hi].any(), r
            continue
        want, mass, score = oracle(c, table[r:r + 1], cu[r:r + 2], kv_len[r:r + 1], q, "i8")
        room = bound(want, mass, score, kv_len[r], 64, "f16", float(np.nanmax(host(c.v_scale))) * 127)
        assert (np.abs(got - want)[lo:hi] <= room[lo:hi]).all(), r
    assert (got[free] == 7.0).all()


def test_outputs_in_other_columns_of_the_inputs_rows(k2):
    """Queries and output, logits and adjusted logits as slices of the same wider rows: nothing of the inputs is written."""
    c, table, cu, kv_len, q = attention_case(k2, [(50, 1), (0, 70), (300, 3)], 16, 8, 2, 128, "i8", "bf16", 48)
    both = torch.full((q.shape[0], 16, 128), 7.0, dtype=q.dtype, device="cuda")
    both[:, :8] = q
    k2.paged_attention(c, both[:, :8], both[:, 8:], dev(cu), dev(kv_len), dev(table), 70, k2.paged_workspace())
    assert torch.equal(both[:, :8], q) and torch.equal(both[:, 8:], attend(k2, c, table, cu, kv_len, q))
    x = torch.randn(5, 333, device="cuda")
    wide = torch.zeros(5, 700, device="cuda")
    wide[:, :333] = x
    bias = (dev([0, 1, 2, 3, 4, 5]), dev([1, 2, 3, 4, 5]), torch.full((5,), 2.0, device="cuda"))
    k2.adjust_logits(wide[:, :333], wide[:, 333:666], bias=bias)
    want = x.clone()
    want[torch.arange(5), torch.arange(1, 6)] += 2.0
    assert torch.equal(wide[:, :333], x) and torch.equal(wide[:, 333:666], want) and not wide[:, 666:].any()


@pytest.mark.parametrize("kw", [dict(), dict(top_k=5), dict(top_p=0.9), dict(min_p=0.1), dict(top_k=5, top_p=0.5)])
def test_a_row_whose_mask_leaves_nothing_raises_the_samplers_guard(k2, kw):
    from dense_gqa_decoder_gb300 import model_io
    import k2_inputs as ki
    ctx, _ = model_io.build_context(ki.TINY, max_context=32, max_batch=3, kv_dtype="f32")
    ctx.set_sampling(k2.sampling(temperature=0.7, seed=5, **kw))
    logits = torch.randn(3, ki.TINY.vocab, device="cuda", generator=torch.Generator("cuda").manual_seed(6))
    mask = torch.full((2, (ki.TINY.vocab + 31) // 32), -1, dtype=torch.int32, device="cuda")
    mask[1] = 0
    nxt = torch.full((3,), -1, dtype=torch.int32, device="cuda")
    k2.adjust_logits(logits, mask=mask, mask_row=dev([0, 0, 0]))
    ctx.sample_logits(logits, 3, dev([1, 2, 3]), nxt)
    assert ctx.sync_status() == k2.K2_OK and all(0 <= t < ki.TINY.vocab for t in nxt.tolist())
    alone = nxt.clone()
    k2.adjust_logits(logits, mask=mask, mask_row=dev([0, 1, 0]))
    ctx.sample_logits(logits, 3, dev([1, 2, 3]), nxt)
    assert torch.isneginf(logits[1]).all() and ctx.sync_status() == k2.K2_ERR_DEVICE_GUARD
    assert nxt[0] == alone[0] and nxt[2] == alone[2] and int(nxt[1]) == 0


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("cache", ["i8", "f8"])
@pytest.mark.parametrize("pairs", FEW + CHUNK)
def test_a_query_that_is_no_number_costs_its_own_row(k2, pairs, cache, value):
    """The head of a token whose query holds a NaN or an infinity gives NaN (zeros if that makes all its scores -inf);
    every other one gives the same bits as without."""
    c, table, cu, kv_len, q = attention_case(k2, pairs, 16, 8, 2, 128, cache, "bf16", 49)
    clean = attend(k2, c, table, cu, kv_len, q)
    bad = [(0, 1, 0), (int(cu[-1]) - 1, 6, len(pairs) - 1)]
    for t, h, _ in bad:
        q[t, h, 17] = value
    got = attend(k2, c, table, cu, kv_len, q)
    for t, h, r in bad:
        seen = int(kv_len[r]) - (int(cu[r + 1]) - t) + 1
        codes = np.concatenate([raw(c.k)[b, h // 4] for b in table[r, :-(-seen // 16)]])[:seen, 17]
        with np.errstate(invalid="ignore"):
            none = (value * P.values(codes, cache) == -np.inf).all()
        assert not got[t, h].any() if none else torch.isnan(got[t, h]).all()
        got[t, h] = clean[t, h]
    assert torch.equal(got, clean)
