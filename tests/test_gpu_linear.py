"""Rows as E4M3 codes (k2_quantize_rows, k2_norm_quantize) and the matrix product with bias, activation and residual
(k2_linear) against their oracle (oracle/k2_linear.py)."""
import numpy as np
import pytest
import torch

from oracle import k2_linear as L
from oracle.k2_fp8 import E4M3_VALUES

pytestmark = pytest.mark.gpu

T = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16, "f8": torch.float8_e4m3fn}
HALF_STEP = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}  # of a value, relative
TINY = {"f32": 2.0 ** -149, "bf16": 2.0 ** -133, "f16": 2.0 ** -24}    # the smallest step


@pytest.fixture(scope="module")
def k2():
    from dense_gqa_decoder_gb300 import k2 as mod
    return mod


def host(t):
    return t.detach().float().cpu().numpy()


def raw(codes):
    return codes.contiguous().view(torch.uint8).cpu().numpy()


def rows(gen, t, n, kind, spread=1.0):
    x = torch.randn(t, n, generator=gen) * torch.exp(spread * torch.randn(t, 1, generator=gen))
    return (x * torch.exp(0.7 * torch.randn(n, generator=gen))).to(T[kind]).cuda()


def wide(x, left=0, right=0):
    """x as a column slice of wider rows, whose other columns hold NaN."""
    fill = lambda n: torch.full((x.shape[0], n), 0x7F, dtype=torch.uint8, device="cuda").view(x.dtype) if x.element_size() == 1 \
        else torch.full((x.shape[0], n), float("nan"), dtype=x.dtype, device="cuda")  # noqa: E731
    if x.element_size() == 1:
        u = torch.cat([fill(left).view(torch.uint8), x.view(torch.uint8), fill(right).view(torch.uint8)], 1)
        return u.view(x.dtype)[:, left:left + x.shape[1]]
    return torch.cat([fill(left), x, fill(right)], 1)[:, left:left + x.shape[1]]


# ---- rows ---------------------------------------------------------------------------------------------------------------

def quantize(k2, x, pad=0, **kw):
    t, n = x.shape
    codes = torch.full((t, n + pad), 0x55, dtype=torch.uint8, device="cuda")
    scales = torch.full((t,), -7.0, device="cuda")
    k2.quantize_rows(x, codes[:, :n], scales, **kw)
    assert (codes[:, n:] == 0x55).all()  # what lies between the rows is left alone
    return codes[:, :n], scales


def check_codes(k2, x, pad=0):
    codes, scales = quantize(k2, x, pad)
    want, scale = L.encode_rows(host(x))
    assert np.array_equal(host(scales), scale, equal_nan=True)
    assert (raw(codes) == want).all()


SHAPES = [(1, 1), (3, 7), (1, 8), (5, 64), (2, 200), (509, 640), (4, 1000), (33, 1664), (64, 2560), (3, 4097), (7, 10240), (2, 20480),
          (1, 49152), (2, 49145), (300, 16)]


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("t,n", SHAPES)
def test_rows_become_the_codes_of_the_definition(k2, t, n, kind):
    check_codes(k2, rows(torch.Generator().manual_seed(t * 7 + n), t, n, kind))


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("n,left,right,pad", [(640, 0, 8, 16), (640, 8, 0, 8), (640, 1, 2, 3), (2560, 16, 16, 4), (37, 3, 0, 11), (8, 8, 8, 8)])
def test_rows_apart_and_at_odd_places(k2, n, left, right, pad, kind):
    check_codes(k2, wide(rows(torch.Generator().manual_seed(n + left), 9, n, kind), left, right), pad)


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("n", [5, 640, 4097])
def test_rows_at_the_ends_of_their_type(k2, n, kind):
    """Zeros, a NaN, infinities, the largest and smallest values, ties between two codes: each row by itself."""
    x = torch.ones(12, n)
    big, small = torch.finfo(T[kind]).max, TINY[kind]
    x[0] = 0
    x[1] = -0.0
    x[2, n // 2] = float("nan")
    x[3, -1] = float("inf")
    x[4, 0] = -float("inf")
    x[5] = big
    x[6] = -big
    x[7] = small
    x[8] = torch.linspace(-448, 448, n)  # a scale of one: the values themselves
    x[9, 0], x[9, 1:] = 448, 17  # half way between 16 and 18
    x[10, 0], x[10, 1:] = big, small
    x[11, 1:] = -1e-3
    check_codes(k2, x.to(T[kind]).cuda())


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("n", [64, 61])
def test_zeros_keep_their_sign(k2, n, kind):
    """Zeros of both signs, and values of both signs that round to zero, beside others."""
    x = torch.randn(9, n, generator=torch.Generator().manual_seed(n))
    x[:, 0::4], x[:, 1::4], x[:, 2::8], x[:, 3::8] = 0.0, -0.0, 1e-5, -1e-5
    x[:, 5] = torch.tensor([1.0, -1.0, 448.0, -3.3, 0.7, 100.0, 5e4, 1e-3, -1.75])
    check_codes(k2, x.to(T[kind]).cuda())


def test_quotients_next_to_the_border_of_two_codes(k2):
    """Rows of values s * B and their neighbours in float32, B half way between two codes: the code is that of the rounded
    quotient, which falls on B, above or below it."""
    gen = np.random.default_rng(23)
    values = np.sort(E4M3_VALUES[:0x7F])
    middles = ((values[1:] + values[:-1]) / 2).astype(np.float32)
    for lo, hi in ((1.0, 2.0), (1e-20, 1e-18), (1e15, 1e16), (2.0 ** -71, 2.0 ** -70)):
        tops = gen.uniform(lo, hi, 300).astype(np.float32)
        scale = (tops / np.float32(448)).astype(np.float32)
        y = (scale[:, None] * middles).astype(np.float32)
        rows = [y, np.nextafter(y, np.float32(np.inf)), np.nextafter(y, np.float32(0)), np.nextafter(np.nextafter(y, np.float32(0)), np.float32(0))]
        x = np.concatenate([np.repeat(tops[:, None], 4, 1)] + rows + [-r for r in rows], 1)
        x = np.minimum(np.abs(x), tops[:, None]) * np.sign(x)
        assert x.shape[1] % 8 == 4  # odd rows too
        check_codes(k2, torch.from_numpy(x).cuda())
        check_codes(k2, torch.from_numpy(np.concatenate([x, x[:, :4]], 1)).cuda())
    # bf16 rows, whose quotients lie on such borders by themselves: every mantissa of the largest value
    x = torch.randn(256, 2560, generator=torch.Generator().manual_seed(5)) * 0.2
    x = x.clamp(-0.99, 0.99)
    x[:, 7] = 1 + torch.arange(256) / 256
    check_codes(k2, x.bfloat16().cuda())
    check_codes(k2, x.half().cuda())


def norm(k2, x, gain, residual=None, groups=1, eps=1e-6, inplace=False, pad=0, **kw):
    t, n = x.shape
    codes = torch.full((t, n + pad), 0x55, dtype=torch.uint8, device="cuda")
    scales = torch.full((t,), -7.0, device="cuda")
    out = None if residual is None else residual if inplace else torch.full_like(residual, 5.0)
    k2.norm_quantize(x, gain, codes[:, :n], scales, residual=residual, residual_out=out, groups=groups, eps=eps, **kw)
    assert (codes[:, n:] == 0x55).all()
    return codes[:, :n], scales, out


def check_norm(k2, x, gain, residual=None, groups=1, eps=1e-6, inplace=False, pad=0, got=None):
    r0 = None if residual is None else residual.clone()
    codes, scales, out = got or norm(k2, x, gain, residual, groups, eps, inplace, pad)
    h, y = L.norm_rows(host(x), None if r0 is None else host(r0), host(gain), groups, eps)
    rel = L.norm_error(x.shape[1] // groups)
    if r0 is not None:
        assert torch.equal(out.cpu(), torch.from_numpy(h).to(r0.dtype))
    top = np.abs(y).max(1) / 448
    s = host(scales).astype(np.float64)
    assert (np.abs(s - top) <= top * (rel + 2 * L.U)).all()
    low, high = L.codes_between(y / np.where(s > 0, s, 1)[:, None], rel + 2 * L.U)  # a row of zeros has no scale
    got = E4M3_VALUES[raw(codes)]
    assert ((low <= got) & (got <= high)).all()


@pytest.mark.parametrize("t,n,groups", [(1, 1, 1), (3, 7, 7), (2, 12, 3), (5, 64, 2), (9, 640, 2), (509, 640, 2), (4, 1000, 4), (3, 2560, 1),
                                        (65, 2560, 2), (2, 2560, 5), (2, 4097, 17), (3, 8192, 4), (1, 16384, 2), (1, 49152, 2), (2, 40000, 8)])
@pytest.mark.parametrize("kinds", [("f32", "f32", "bf16"), ("bf16", None, "f32"), ("f16", "f32", "f16"), ("bf16", "bf16", "bf16"),
                                   ("f32", "f16", "f32"), ("f16", None, "bf16")])
def test_normalised_sums(k2, t, n, groups, kinds):
    gen = torch.Generator().manual_seed(t + n)
    x, gain = rows(gen, t, n, kinds[0]), (1 + 0.3 * torch.randn(n, generator=gen)).to(T[kinds[2]]).cuda()
    check_norm(k2, x, gain, None if kinds[1] is None else rows(gen, t, n, kinds[1]) * 3, groups, inplace=t % 2 == 1)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("n,left,right,pad", [(640, 0, 8, 16), (640, 8, 16, 8), (640, 1, 2, 3), (2560, 16, 16, 4), (38, 3, 0, 11)])
def test_normalised_sums_of_rows_apart(k2, n, left, right, pad, kind):
    gen = torch.Generator().manual_seed(n + left)
    x, r, gain = rows(gen, 9, n, kind), rows(gen, 9, n, kind), torch.randn(n, generator=gen).cuda()
    check_norm(k2, wide(x, left, right), gain, wide(r, right, left), 2, pad=pad)
    check_norm(k2, wide(x, left, right), gain, wide(r, right, left), 2, inplace=True, pad=pad)


@pytest.mark.parametrize("n,groups", [(640, 2), (200, 5), (36, 2), (2560, 1)])
def test_norms_at_the_ends_of_float32(k2, n, groups):
    """Rows whose squares overflow or vanish, zeros, a NaN, an infinity, a sum that overflows: each row by itself."""
    gen = torch.Generator().manual_seed(n)
    x = torch.randn(10, n, generator=gen)
    r = torch.zeros(10, n)
    x[0] *= 1e37
    x[1] *= 1e-30
    x[2] = 0
    x[3, :n // groups] *= 3e37
    x[4] = 3.4e38
    x[5, 3] = 2e25
    gain = torch.ones(n).cuda()
    bad = x.clone()
    bad[6, n - 1], bad[7, 0], bad[8, 1], r[9, 2] = float("nan"), float("inf"), 3e38, -float("inf")
    r[8, 1] = 3e38
    codes, scales, out = norm(k2, bad.cuda(), gain, r.cuda(), groups)
    assert torch.isnan(scales[6:]).all() and (codes[6:] == 0x7F).all()
    assert torch.isnan(out[6, n - 1]) and out[8, 1] == float("inf") and out[9, 2] == -float("inf")
    check_norm(k2, x[:6].cuda(), gain, r[:6].cuda(), groups, got=(codes[:6], scales[:6], out[:6]))
    assert scales[2] == 0 and (codes[2] == 0).all()


def test_eps_is_added_to_the_mean_square(k2):
    x = torch.full((2, 64), 1e-3).cuda()
    for eps in (2.0 ** -126, 1e-6, 1e-2, 10.0, 3e38):
        check_norm(k2, x, torch.ones(64).cuda(), eps=eps)


# ---- the product --------------------------------------------------------------------------------------------------------

def small_numbers(gen, n, k, kind, step):
    """Whole numbers whose sums are exact in float32, rows 16-byte aligned."""
    v = torch.randint(-4, 5, (n, -(-k // step) * step), generator=gen).float().cuda()
    return v.to(T[kind])[:, :k]


def call(k2, w, x, kind, width, pad=0, **kw):
    out = torch.full((x.shape[0] + 3, width + pad), 9.0, dtype=T[kind], device="cuda")
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    k2.linear(w, x, out[:x.shape[0], :width], flags=flags, **kw)
    assert (out[x.shape[0]:] == 9).all() and (out[:, width:] == 9).all() and int(flags) == 0
    return out[:x.shape[0], :width]


TOKENS = [1, 2, 15, 16, 17, 31, 33, 64, 65, 127, 128, 129, 255, 257, 300, 513]


@pytest.mark.parametrize("kind", ["f8", "bf16", "f16"])
@pytest.mark.parametrize("t", TOKENS)
@pytest.mark.parametrize("n,k", [(1, 1), (2, 16), (127, 33), (128, 128), (129, 129), (300, 640), (640, 257), (1000, 64), (255, 2565)])
def test_whole_numbers_are_exact(k2, t, n, k, kind):
    """Every product and sum is a whole number below 2^24, so any order of additions gives the same one."""
    gen = torch.Generator().manual_seed(n + k + t)
    step = 16 if kind == "f8" else 8
    w, x = small_numbers(gen, n, k, kind, step), small_numbers(gen, t, k, kind, step)
    kw = dict(w_scale=torch.ones(n).cuda(), x_scale=torch.ones(t).cuda()) if kind == "f8" else {}
    got = call(k2, w, x, "f32", n, pad=n % 3, **kw)
    assert torch.equal(got, x.float() @ w.float().T)


@pytest.mark.parametrize("kind,t,n,k", [
    ("f8", 70, 700, 300), ("f8", 70, 9730, 1000), ("f8", 333, 9730, 640), ("f8", 431, 6146, 1000), ("f8", 505, 5000, 1500),
    ("f8", 220, 12002, 1500), ("f8", 250, 12002, 2565), ("bf16", 70, 9730, 640), ("f16", 333, 9730, 300), ("bf16", 150, 9730, 1000),
    ("f16", 505, 5000, 640), ("bf16", 220, 12002, 640), ("f16", 250, 12002, 1000)])
def test_every_width_of_tile(k2, kind, t, n, k):
    """Sizes for which tiles of 64, 96, 128, 160, 192, 224 and 256 tokens are chosen, the last of them not full; out = x . w^T + bias +
    residual in whole numbers, at most 16 * 2565 + 2000 of them: exact."""
    gen = torch.Generator().manual_seed(t + n + k)
    step = 16 if kind == "f8" else 8
    w, x = small_numbers(gen, n, k, kind, step), small_numbers(gen, t, k, kind, step)
    kw = dict(w_scale=torch.ones(n).cuda(), x_scale=torch.ones(t).cuda()) if kind == "f8" else {}
    bias, res = (torch.randint(-1000, 1001, shape, generator=gen).float().cuda() for shape in ((n,), (t, n)))
    got = call(k2, w, x, "f32", n, pad=3, bias=bias, residual=res, **kw)
    assert torch.equal(got, x.float() @ w.float().T + bias + res)


def check_product(k2, w, x, kind, pad=0, inplace=False, **kw):
    res = kw.get("residual")
    act = kw.get("activation")
    width = w.shape[0] // 2 if act == "swiglu" else w.shape[0]
    want, off = L.linear(host(w), host(x), *[None if kw.get(a) is None else host(kw[a]) for a in ("w_scale", "x_scale", "bias")], act,
                         None if res is None else host(res))
    if inplace:
        k2.linear(w, x, res, **kw)
        got = res
    else:
        got = call(k2, w, x, kind, width, pad, **kw)
    room = off + (np.abs(want) + off) * HALF_STEP[kind] + TINY[kind]
    err = np.abs(host(got).astype(np.float64) - want)
    assert (err <= room).all(), float((err / room).max())


def operands(gen, t, n, k, kind):
    x, w = rows(gen, t, k, "f32", 0.5), rows(gen, n, k, "f32", 0.2) / k ** 0.5
    kw = {}
    if kind == "f8":
        got = []
        for v in (x, w):
            codes, scale = L.encode_rows(host(v))
            p = np.zeros((v.shape[0], -(-k // 16) * 16), np.uint8)
            p[:, :k] = codes
            got.append((torch.from_numpy(p).cuda().view(torch.float8_e4m3fn)[:, :k], torch.from_numpy(scale).cuda()))
        (x, kw["x_scale"]), (w, kw["w_scale"]) = got
        return x, w, kw
    pad = -(-k // 8) * 8 - k
    return wide(x.to(T[kind]), 0, pad), wide(w.to(T[kind]), 0, pad), kw


@pytest.mark.parametrize("kind", ["f8", "bf16", "f16"])
@pytest.mark.parametrize("act", [None, "relu", "silu", "gelu", "gelu_tanh", "swiglu"])
@pytest.mark.parametrize("t,n,k,out", [(1, 640, 2560, "f32"), (3, 258, 100, "bf16"), (16, 1664, 640, "f16"), (40, 130, 1000, "f32"),
                                       (129, 512, 640, "bf16"), (300, 644, 328, "f16"), (600, 1024, 512, "bf16")])
def test_bias_activation_and_residual(k2, t, n, k, out, act, kind):
    gen = torch.Generator().manual_seed(t + n)
    x, w, kw = operands(gen, t, n, k, kind)
    kw["activation"] = act
    check_product(k2, w, x, out, **kw)
    kw["bias"] = torch.randn(n, generator=gen).cuda()
    check_product(k2, w, x, out, pad=5, **kw)
    width = n // 2 if act == "swiglu" else n
    kw["residual"] = wide(torch.randn(t, width, generator=gen).to(T[out]).cuda(), 3, 2)
    check_product(k2, w, x, out, **kw)
    check_product(k2, w, x, out, inplace=True, **kw)


@pytest.mark.parametrize("t,n,k", [(1, 6144, 2560), (16, 20480, 2560), (64, 2560, 10240), (257, 2560, 4096), (2048, 1280, 2560)])
def test_the_models_sizes(k2, t, n, k):
    x, w, kw = operands(torch.Generator().manual_seed(9), t, n, k, "f8")
    check_product(k2, w, x, "f32", **kw)
    check_product(k2, w, x, "bf16", activation="swiglu", **kw)


@pytest.mark.parametrize("kind", ["f8", "bf16"])
def test_strided_operands(k2, kind):
    gen = torch.Generator().manual_seed(11)
    for t, n, k in ((5, 130, 77), (140, 300, 200), (300, 520, 200)):
        x, w, kw = operands(gen, t, n, k, kind)
        check_product(k2, wide(w, 16, 48 + -(w.shape[1]) % 16), wide(x, 32, 16 + -(x.shape[1]) % 16), "f32", pad=3, **kw)


@pytest.mark.parametrize("t", [1, 20, 130, 300])
@pytest.mark.parametrize("ws,xs", [(1e-22, 1e-20), (1e-30, 1e3), (1e25, 1e-20), (1e-38, 1e-3), (1e15, 1e15), (3e-44, 1e30)])
def test_scales_whose_product_leaves_the_normal_numbers(k2, t, ws, xs):
    """What matters is the result, here between 1e-37 and 1e38."""
    gen = torch.Generator().manual_seed(16)
    n, k = 140, 96
    w, x = small_numbers(gen, n, k, "f8", 16), small_numbers(gen, t, k, "f8", 16)
    sw, sx = torch.full((n,), ws).cuda(), torch.full((t,), xs).cuda()
    z = (x.double() @ w.double().T)
    want = z * sw.double()[0] * sx.double()[0]
    assert want.abs().max() < 3e38
    got = call(k2, w, x, "f32", n, w_scale=sw, x_scale=sx).double()
    # two roundings of numbers that are normal, or of the smallest step
    assert ((got - want).abs() <= want.abs() * 2.0 ** -22 + 2.0 ** -149 * max(1.0, xs)).all()


def test_gates_far_below_zero(k2):
    """silu vanishes slowly against a large factor: gates down to where e^-g overflows."""
    k = 16
    gates = torch.arange(-128, 0, dtype=torch.float32)
    w = torch.zeros(256, k)
    w[0::2, 0] = gates
    w[1::2, 1] = 2.0 ** 100
    x = torch.zeros(3, k)
    x[:, 0] = x[:, 1] = 1
    out = torch.zeros(3, 128, device="cuda")
    k2.linear(w.bfloat16().cuda(), x.bfloat16().cuda(), out, activation="swiglu")
    g = gates.double()
    want = g / (1 + torch.exp(-g)) * 2.0 ** 100
    # e^-g to 2^-23 |g| / ln 2 and two steps; from 88.7 on it is infinite in fp32
    room = want.abs() * (2.0 ** -23 * (g.abs() * 1.5 + 6))
    got = out.double().cpu()
    near = g > -88
    assert ((got - want).abs() <= room)[:, near].all() and (got[:, g < -89].abs() <= want[g < -89].abs().max()).all()


@pytest.mark.parametrize("t", [1, 20, 130, 300])
def test_a_nan_costs_what_it_enters(k2, t):
    gen = torch.Generator().manual_seed(12)
    x, w, kw = operands(gen, t, 260, 200, "f8")
    good = call(k2, w, x, "f32", 260, **kw).clone()
    at, row = t // 2, 131
    xb, wb = wide(x, 0, 8), wide(w, 0, 8)  # copies
    xb.view(torch.uint8)[at, 150], wb.view(torch.uint8)[row, 7] = 0x7F, 0xFF
    lost = torch.zeros(t, 260, dtype=torch.bool, device="cuda")
    lost[at], lost[:, row] = True, True
    for act in (None, "relu", "gelu", "gelu_tanh", "silu"):
        got = call(k2, wb, xb, "f32", 260, activation=act, **kw)
        assert torch.equal(torch.isnan(got), lost)
    got = call(k2, wb, xb, "f32", 260, **kw)
    assert torch.equal(got[~lost], good[~lost])
    kw["x_scale"] = kw["x_scale"].clone()
    kw["x_scale"][at] = float("nan")
    assert torch.isnan(call(k2, w, x, "f32", 260, **kw)[at]).all()
    kw["x_scale"][at] = 0
    assert (call(k2, w, x, "f32", 260, **kw)[at] == 0).all()


@pytest.mark.parametrize("t,n", [(1 << 22, 1), (1 << 22, 130), (65535 * 64 + 1, 3), (70000, 700), (1, 300000), (65, 300000), (40, 1)])
def test_the_most_tokens_and_features(k2, t, n):
    gen = torch.Generator().manual_seed(t + n)
    w, x = small_numbers(gen, n, 24, "bf16", 8), small_numbers(gen, 1000, 24, "bf16", 8).repeat(-(-t // 1000), 1)[:t]
    out = torch.zeros(t, n, dtype=torch.float16, device="cuda")
    k2.linear(w, x, out)
    want = (x[:1000].float() @ w.float().T).half()  # whole numbers up to 384
    for lo in range(0, t, 1000 * 64):
        got = out[lo:lo + 64000]
        assert torch.equal(got, want.repeat(64, 1)[:got.shape[0]])


def test_rows_further_apart_than_32_bits_count(k2):
    """300 rows 8 Mi elements apart: offsets beyond 2^31."""
    far, t, n, k = 1 << 23, 300, 136, 160
    gen = torch.Generator().manual_seed(15)
    for kind, tokens in (("bf16", t), ("f8", t), ("bf16", 60)):
        w, x = small_numbers(gen, n, k, kind, 16), small_numbers(gen, tokens, k, kind, 16)
        xf = torch.empty(tokens * far, dtype=torch.uint8, device="cuda").view(x.dtype).as_strided((tokens, k), (far // x.element_size(), 1))
        xf.copy_(x) if kind != "f8" else xf.view(torch.uint8).copy_(x.view(torch.uint8))
        of = torch.empty(tokens * far, dtype=torch.float16, device="cuda").as_strided((tokens, n), (far, 1))
        kw = dict(w_scale=torch.ones(n).cuda(), x_scale=torch.ones(tokens).cuda()) if kind == "f8" else {}
        k2.linear(w, xf, of, **kw)
        assert torch.equal(of.float(), x.float() @ w.float().T)
        of.fill_(1)
        k2.linear(w, xf, of, residual=of, **kw)
        assert torch.equal(of.float(), x.float() @ w.float().T + 1)
    x = rows(gen, t, 640, "bf16")
    xf = torch.empty(t * far, dtype=torch.bfloat16, device="cuda").as_strided((t, 640), (far, 1))
    xf.copy_(x)
    codes = torch.empty(t * far, dtype=torch.uint8, device="cuda").as_strided((t, 640), (far, 1))
    scales = torch.empty(t, device="cuda")
    k2.quantize_rows(xf, codes, scales)
    want, scale = L.encode_rows(host(x))
    assert (raw(codes) == want).all() and np.array_equal(host(scales), scale)
    k2.norm_quantize(x, torch.ones(640).cuda(), codes, scales, residual=xf)
    check_norm(k2, x, torch.ones(640).cuda(), x, got=(codes, scales, xf))


@pytest.mark.parametrize("t,n,k", [(1, 2560, 10240), (7, 300, 4096), (64, 2560, 2560), (130, 1664, 640), (700, 2560, 640)])
def test_calls_repeat_bit_for_bit(k2, t, n, k):
    x, w, kw = operands(torch.Generator().manual_seed(13), t, n, k, "f8")
    first = call(k2, w, x, "f32", n, **kw).clone()
    for _ in range(5):
        assert torch.equal(call(k2, w, x, "f32", n, **kw), first)


@pytest.mark.parametrize("t,n,k", [(3, 2560, 10240), (130, 640, 2560), (600, 2560, 2560)])
def test_waits_that_run_out(k2, t, n, k):
    """A wait limit of a microsecond, shorter than a tile takes from memory: the call ends, says so, and an output is right or
    NaN.  The next call, with time, is right."""
    x, w, kw = operands(torch.Generator().manual_seed(14), t, n, k, "f8")
    want = call(k2, w, x, "f32", n, **kw).clone()
    torch.empty(1 << 28, dtype=torch.uint8, device="cuda").zero_()  # the operands leave L2
    out = torch.zeros(t, n, device="cuda")
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    k2.linear(w, x, out, flags=flags, wait_limit_us=1, **kw)
    lost = torch.isnan(out)
    assert int(flags) == k2.K2_LINEAR_TIMEOUT and lost.any() and torch.equal(out[~lost], want[~lost])
    assert torch.equal(call(k2, w, x, "f32", n, **kw), want)


def test_no_tokens(k2):
    w = torch.zeros(64, 64, dtype=torch.float8_e4m3fn, device="cuda")
    x, out = w[:0], torch.zeros(0, 64, device="cuda")
    k2.linear(w, x, out, w_scale=torch.ones(64).cuda(), x_scale=torch.ones(0).cuda())
    k2.quantize_rows(out, x, torch.ones(0).cuda())
    k2.norm_quantize(out, torch.ones(64).cuda(), x, torch.ones(0).cuda())


def test_tensors_that_the_binding_refuses(k2):
    w8 = torch.zeros(64, 64, dtype=torch.float8_e4m3fn, device="cuda")
    wb, s, out = torch.zeros(64, 64, dtype=torch.bfloat16, device="cuda"), torch.ones(64).cuda(), torch.zeros(64, 64, device="cuda")
    for args, kw in (((w8, w8, out), {}), ((wb, w8, out), dict(w_scale=s, x_scale=s)), ((wb, wb, out), dict(w_scale=s)),
                     ((wb, wb, out[:, :32]), {}), ((wb, wb[:, :32], out), {}), ((wb, wb, out.t()[::1].t()[:63]), {}),
                     ((wb, wb, out), dict(activation="tanh")), ((wb, wb, out), dict(bias=s.half())), ((wb, wb, out), dict(bias=s[:32])),
                     ((wb, wb, out), dict(residual=out.half())), ((wb, wb.half(), out), {}), ((wb.t().contiguous().t()[:, :], wb, out), {}),
                     ((wb, wb, out), dict(flags=s))):
        with pytest.raises(ValueError):
            k2.linear(*args, **kw)
    with pytest.raises(k2.K2Error):
        k2.linear(wb, wb, wb)  # over its own weights
    with pytest.raises(ValueError):
        k2.norm_quantize(wb, s, w8, s, residual_out=wb)
    with pytest.raises(ValueError):
        k2.quantize_rows(wb, w8[:, :32], s)


# ---- as they are used together ------------------------------------------------------------------------------------------

class Half:
    """The MLP half of a decoder layer over E4M3 weights: its buffers and its four calls."""

    def __init__(self, k2, t, hidden=640, inter=1664, seed=20):
        gen = torch.Generator().manual_seed(seed)
        self.k2, self.groups = k2, 2
        _, self.gu, gu = operands(gen, 1, 2 * inter, hidden, "f8")
        _, self.down, dn = operands(gen, 1, hidden, inter, "f8")
        self.gu_s, self.down_s = gu["w_scale"], dn["w_scale"]
        self.gain = (1 + 0.1 * torch.randn(hidden, generator=gen)).bfloat16().cuda()
        self.x, self.stream = rows(gen, t, hidden, "f32"), rows(gen, t, hidden, "f32")
        e = lambda *s: torch.empty(*s, device="cuda")  # noqa: E731
        self.c1, self.s1, self.act = e(t, hidden).to(torch.float8_e4m3fn), e(t), e(t, inter).bfloat16()
        self.c2, self.s2, self.mid = e(t, inter).to(torch.float8_e4m3fn), e(t), e(t, hidden)

    def run(self, stream=None):
        k2 = self.k2
        k2.norm_quantize(self.x, self.gain, self.c1, self.s1, residual=self.stream, residual_out=self.mid, groups=2, stream=stream)
        k2.linear(self.gu, self.c1, self.act, w_scale=self.gu_s, x_scale=self.s1, activation="swiglu", stream=stream)
        k2.quantize_rows(self.act, self.c2, self.s2, stream=stream)
        k2.linear(self.down, self.c2, self.mid, w_scale=self.down_s, x_scale=self.s2, residual=self.mid, stream=stream)
        return self.mid

    def want(self):
        """Each step's oracle on what the step before left."""
        h, y = L.norm_rows(host(self.x), host(self.stream), host(self.gain), 2, 1e-6)
        x1 = E4M3_VALUES[raw(self.c1)]
        act, _ = L.linear(host(self.gu), x1, host(self.gu_s), host(self.s1), activation="swiglu")
        out, off = L.linear(host(self.down), E4M3_VALUES[raw(self.c2)], host(self.down_s), host(self.s2), residual=h)
        deq1, deq2 = x1 * host(self.s1)[:, None], E4M3_VALUES[raw(self.c2)] * host(self.s2)[:, None]
        return y, deq1, act, deq2, out, off


@pytest.mark.parametrize("t", [1, 5, 70, 300])
def test_a_layers_half(k2, t):
    m = Half(k2, t)
    got = host(m.run()).astype(np.float64)
    y, deq1, act, deq2, out, off = m.want()
    rel = lambda a, b: np.linalg.norm(a - b) / np.linalg.norm(b)  # noqa: E731
    # rounding to E4M3 is off by at most 2^-4 of a value, or of the smallest normal code
    assert rel(deq1, y) < 2.0 ** -4 and rel(deq2, act) < 2.0 ** -4
    assert (np.abs(got - out) <= off + np.abs(out) * 2.0 ** -24).all()


def test_captured_and_replayed(k2):
    """The half in a graph, replayed on other inputs in the same buffers, equals eager calls."""
    m = Half(k2, 33)
    m.run()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        m.run(torch.cuda.current_stream())
    for seed in (31, 32):
        gen = torch.Generator().manual_seed(seed)
        m.x.copy_(rows(gen, 33, 640, "f32"))
        m.stream.copy_(rows(gen, 33, 640, "f32"))
        graph.replay()
        got = m.mid.clone()
        assert torch.equal(m.run(), got) and torch.isfinite(got).all()


def test_two_streams_at_once(k2):
    """Calls that overlap on the GPU share nothing."""
    ms = [Half(k2, t, seed=40 + t) for t in (3, 200)]
    want = [m.run().clone() for m in ms]
    streams = [torch.cuda.Stream() for _ in ms]
    torch.cuda.synchronize()
    for _ in range(10):
        for m, s in zip(ms, streams):
            m.run(s)
    torch.cuda.synchronize()
    for m, w in zip(ms, want):
        assert torch.equal(m.mid, w)


def test_kernels_of_several_streams_share_the_sms(k2):
    """Clusters of few tokens whose K is short (little shared memory), long ones, and pairs of CTAs, on four streams at once:
    all of them hold tensor memory, and each ends with the result that it has alone."""
    cases = []
    for i, (t, n, k) in enumerate([(9, 2560, 200), (300, 2560, 1000), (16, 6000, 384), (40, 2560, 2560), (1, 5000, 256), (513, 640, 640)]):
        gen = torch.Generator().manual_seed(900 + i)
        wq, wqs = L.encode_rows(torch.randn(n, k, generator=gen).numpy())
        xq, xqs = L.encode_rows(torch.randn(t, k, generator=gen).numpy())
        pad = (k + 15) // 16 * 16
        codes = [torch.zeros(len(q), pad, dtype=torch.uint8, device="cuda") for q in (wq, xq)]
        for c, q in zip(codes, (wq, xq)):
            c[:, :k] = torch.from_numpy(q).cuda()
        w, x = (c[:, :k] for c in codes)
        scales = dict(w_scale=torch.from_numpy(wqs).cuda(), x_scale=torch.from_numpy(xqs).cuda())
        alone, flags = torch.empty(t, n, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
        k2.linear(w, x, alone, flags=flags, **scales)
        cases.append((w, x, alone, scales, flags))
    torch.cuda.synchronize()
    streams, outs = [torch.cuda.Stream() for _ in range(4)], []
    for turn in range(40):
        for i, s in enumerate(streams):
            w, x, alone, scales, flags = case = cases[(turn * (i + 1) + i) % len(cases)]
            with torch.cuda.stream(s):
                out = torch.full_like(alone, -7.0)
                k2.linear(w, x, out, flags=flags, **scales)
            outs.append((out, case))
    torch.cuda.synchronize()
    assert all(torch.equal(out, alone) and not flags.item() for out, (_, _, alone, _, flags) in outs)


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("t", [5, 300])
def test_inputs_from_other_streams_copies_and_kernels(k2, t, captured):
    """The kernels start before the one ahead of them on the stream has ended; what they read may come from it, from a copy, a
    fill, or another stream that was joined, each of them slow."""
    gen = torch.Generator().manual_seed(60 + t)
    m = Half(k2, t)
    big = torch.randn(4096, 4096, device="cuda")
    sources = [(rows(gen, t, 640, "f32"), rows(gen, t, 640, "f32")) for _ in range(2)]
    pinned = [(x.cpu().pin_memory(), r.cpu().pin_memory()) for x, r in sources]
    side = torch.cuda.Stream()

    def slow():
        for _ in range(6):
            torch.mm(big, big)

    def passes(i, how):
        here = torch.cuda.current_stream()
        if how == "side":
            side.wait_stream(here)
            with torch.cuda.stream(side):
                slow()
                m.x.copy_(sources[i][0])
                m.stream.copy_(sources[i][1])
            here.wait_stream(side)
        elif how == "kernel":
            slow()
            m.x.copy_(sources[i][0])
            torch.add(sources[i][1], 0, out=m.stream)
        elif how == "copy":
            slow()
            m.x.copy_(pinned[i][0], non_blocking=True)
            m.stream.copy_(pinned[i][1], non_blocking=True)
        else:  # a fill right ahead
            m.x.copy_(sources[i][0])
            m.stream.copy_(sources[i][1])
            slow()
            m.stream.zero_()
        return m.run(here)

    want = {}
    for how in ("side", "kernel", "copy", "fill"):
        for i in range(2):
            m.x.copy_(sources[i][0])
            m.stream.copy_(sources[i][1]) if how != "fill" else m.stream.zero_()
            torch.cuda.synchronize()
            want[how, i] = m.run().clone()
    work = torch.cuda.Stream()
    work.wait_stream(torch.cuda.current_stream())
    for how in ("side", "kernel", "copy", "fill"):
        for i in (0, 1, 0):
            if captured:
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph, stream=work):
                    passes(i, how)
                m.x.fill_(7)
                m.stream.fill_(7)
                graph.replay()
            else:
                with torch.cuda.stream(work):
                    passes(i, how)
            torch.cuda.synchronize()
            assert torch.equal(m.mid, want[how, i]), how
