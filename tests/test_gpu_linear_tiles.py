"""The matrix product where every pair of CTAs works on several tiles: accumulators used again, the ring of stages running on from
tile to tile, and waits that run out in the midst of it."""
import pytest
import torch

pytestmark = pytest.mark.gpu

T = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16, "f8": torch.float8_e4m3fn}


@pytest.fixture(scope="module")
def k2():
    from dense_gqa_decoder_gb300 import k2 as mod
    return mod


def small_numbers(gen, n, k, kind):
    """Whole numbers of -4 .. 4 in rows that are 16-byte aligned."""
    step = 16 if kind == "f8" else 8
    v = torch.randint(-4, 5, (n, -(-k // step) * step), generator=gen, device="cuda")
    return v.to(torch.float32).to(T[kind])[:, :k]


def operands(seed, kind, t, n, k):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    w, x = small_numbers(gen, n, k, kind), small_numbers(gen, t, k, kind)
    kw = dict(w_scale=torch.ones(n, device="cuda"), x_scale=torch.ones(t, device="cuda")) if kind == "f8" else {}
    return gen, w, x, kw


# On 76 pairs: five tiles of 256 x 224 each, of 21 and of 41 steps of K (a ring of seven stages); four of 256 x 160 of 21 steps in
# stages of two, the last of a tile half full (a ring of four); ten of 256 x 224 whose six steps are fewer than the ring's stages
SIZES = [("f8", 1100, 20480, 2565), ("bf16", 1100, 20480, 2565), ("f8", 150, 80000, 2565), ("f16", 150, 80000, 1300),
         ("f8", 2100, 20480, 700), ("bf16", 2100, 20480, 350)]


@pytest.mark.parametrize("kind,t,n,k", SIZES)
def test_several_tiles_a_pair_are_exact(k2, kind, t, n, k):
    """Products, sums, bias and residual are whole numbers below 2^24: any order gives the same."""
    gen, w, x, kw = operands(t + k, kind, t, n, k)
    bias = torch.randint(-1000, 1001, (n,), generator=gen, device="cuda").float()
    res = torch.randint(-1000, 1001, (t, n), generator=gen, device="cuda").float()
    want = x.float() @ w.float().T + bias + res
    out = torch.full((t + 1, n + 3), 9.0, device="cuda")
    for _ in range(2):
        k2.linear(w, x, out[:t, :n], bias=bias, residual=res, **kw)
        assert torch.equal(out[:t, :n], want) and (out[t:] == 9).all() and (out[:, n:] == 9).all()
    k2.linear(w, x, res, bias=bias, residual=res, **kw)
    assert torch.equal(res, want)


@pytest.mark.parametrize("kind,t,n,k", SIZES)
def test_several_tiles_a_pair_with_swiglu(k2, kind, t, n, k):
    """The sums are exact, times a scale of 2^-5; what follows them is off by 2^-23 (1.5 |g| + 6) at most (e^-g that way, the
    rest six steps) and the rounding to bf16 by 2^-8, in its normal range."""
    gen, w, x, kw = operands(t + k + 1, kind, t, n, k)
    if kind == "f8":
        kw["x_scale"] = torch.full((t,), 2.0 ** -5, device="cuda")
    else:
        x *= 2.0 ** -5
    res = torch.randint(-100, 101, (t, n // 2), generator=gen, device="cuda").bfloat16()
    out = torch.zeros(t, n // 2, dtype=torch.bfloat16, device="cuda")
    k2.linear(w, x, out, residual=res, activation="swiglu", **kw)
    z = x.float() @ w.float().T * (2.0 ** -5 if kind == "f8" else 1.0)
    g, u = z[:, 0::2].double(), z[:, 1::2].double()
    y = g / (1 + torch.exp(-g)) * u
    room = y.abs() * (2.0 ** -23 * (1.5 * g.abs() + 6)) + 1e-30
    want = y + res.double()
    room = room + want.abs() * 2.0 ** -24
    assert ((out.double() - want).abs() <= room + (want.abs() + room) * 2.0 ** -8).all()


def whole_tiles(lost):
    """Whether what is lost is whole tiles of 256 outputs x some width of tokens."""
    t, n = lost.shape
    for width in range(64, 257, 32):
        p = torch.nn.functional.pad(lost.float(), (0, -n % 256, 0, -t % width), value=-1)
        p = p.view(p.shape[0] // width, width, p.shape[1] // 256, 256).permute(0, 2, 1, 3).flatten(2)
        if ((p == 1).any(2) & (p == 0).any(2)).sum() == 0:
            return True
    return False


@pytest.mark.parametrize("limit", [1, 2, 3, 4, 6, 9, 14, 25, 60])
@pytest.mark.parametrize("kind,t,n,k", [("f8", 1100, 20480, 2565), ("f8", 150, 80000, 2565), ("bf16", 2100, 20480, 350)])
def test_waits_that_run_out_between_tiles(k2, kind, t, n, k, limit):
    """Limits from below to above what a tile takes: every tile is right throughout or NaN throughout, and the flag says whether
    there is one that is NaN.  The next call, with time, is right."""
    _, w, x, kw = operands(7, kind, t, n, k)
    want = x.float() @ w.float().T
    out = torch.zeros(t, n, device="cuda")
    for _ in range(3):
        torch.empty(1 << 28, dtype=torch.uint8, device="cuda").zero_()  # the operands leave L2
        flags = torch.zeros(1, dtype=torch.int32, device="cuda")
        k2.linear(w, x, out.fill_(9), flags=flags, wait_limit_us=limit, **kw)
        lost = torch.isnan(out)
        assert torch.equal(out[~lost], want[~lost]) and whole_tiles(lost)
        assert not lost.any() or int(flags) == k2.K2_LINEAR_TIMEOUT
    flags.zero_()
    k2.linear(w, x, out, flags=flags, **kw)
    assert torch.equal(out, want) and int(flags) == 0
