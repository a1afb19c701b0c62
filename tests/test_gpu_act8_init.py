"""k2_act8_init: the memory that option K2_OPT_ACT8 needs beside the workspace."""
import pytest
import torch

import k2_inputs as ki

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def k2():
    from dense_gqa_decoder_gb300 import k2 as mod
    return mod


def context(weights="f8", kv="f16", shape=ki.MEDIUM):
    from dense_gqa_decoder_gb300 import model_io
    return model_io.build_context(shape, max_context=128, kv_dtype=kv, gain_scale=0.1, weights=weights)[0]


def logits(k2, ctx, n=70):
    ctx.kv_reset()
    ids = torch.tensor(ki.prompt_ids(ki.MEDIUM.vocab, n, seed=5), dtype=torch.int32, device="cuda")
    out, nxt = torch.empty(ki.MEDIUM.vocab, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    ctx.prefill(0, ids, nxt, out)
    assert ctx.sync_status() == k2.K2_OK
    return out


def test_the_option_needs_its_buffer(k2):
    ctx = context()
    n = k2.LIB.k2_act8_bytes(ctx.ctx)
    # codes of three layers' gates and factors in whole chunks of 512 values, the lm_head in 16 bits, scales of a block's rows
    assert n >= 3 * 2 * 1536 * 512 + 1000 * 512 * 2 + 128 * 4
    assert k2.LIB.k2_set_option(ctx.ctx, k2.K2_OPT_ACT8, 1) == k2.K2_ERR_WORKSPACE
    assert "k2_act8_init" in ctx.last_error()
    assert k2.LIB.k2_set_option(ctx.ctx, k2.K2_OPT_ACT8, 0) == k2.K2_OK
    exact = logits(k2, ctx)
    buffer = torch.full((n + 512,), 0x5A, dtype=torch.uint8, device="cuda")
    stream = torch.cuda.current_stream().cuda_stream
    for at, size in ((0, n), (buffer.data_ptr(), n - 1), (buffer.data_ptr() + 128, n), (buffer.data_ptr(), 0)):
        assert k2.LIB.k2_act8_init(ctx.ctx, at, size, stream) == k2.K2_ERR_WORKSPACE
        assert k2.LIB.k2_set_option(ctx.ctx, k2.K2_OPT_ACT8, 1) == k2.K2_ERR_WORKSPACE
    assert (buffer == 0x5A).all()
    assert k2.LIB.k2_act8_init(ctx.ctx, buffer.data_ptr() + 256, n, stream) == k2.K2_OK
    assert k2.LIB.k2_set_option(ctx.ctx, k2.K2_OPT_ACT8, 1) == k2.K2_OK
    rounded = logits(k2, ctx)
    assert (buffer[:256] == 0x5A).all() and (buffer[256 + n:] == 0x5A).all()
    # through the binding, which allocates it; and in another place
    other = context()
    other.set_option(k2.K2_OPT_ACT8, 1)
    assert other.act8_buffer.numel() == n
    assert torch.equal(logits(k2, other), rounded) and not torch.equal(rounded, exact)
    buffer[:] = 0
    other.act8_init()
    assert torch.equal(logits(k2, other), rounded)
    # without the option nothing of it is read
    other.set_option(k2.K2_OPT_ACT8, 0)
    other.act8_buffer.fill_(0x7F)
    assert torch.equal(logits(k2, other), exact) or (logits(k2, other) - exact).norm() <= 2e-4 * exact.norm()


@pytest.mark.parametrize("weights,kv,shape", [(None, "f16", ki.MEDIUM), ("q4", "f16", ki.MEDIUM), (None, "f32", ki.TINY)])
def test_where_there_is_no_such_option(k2, weights, kv, shape):
    ctx = context(weights, kv, shape)
    assert k2.LIB.k2_act8_bytes(ctx.ctx) == 0
    with pytest.raises(k2.K2Error) as e:
        ctx.act8_init()
    assert e.value.status == k2.K2_ERR_UNSUPPORTED


@pytest.mark.parametrize("eps", [0.0, 1e-39, float("inf")])
def test_a_norm_that_the_rows_calls_refuse(k2, eps):
    """k2_norm_quantize takes no eps below 2^-126, and so the option is refused, ahead of any prompt."""
    ctx = context(shape=ki.MEDIUM.replace(eps=eps))
    with pytest.raises(k2.K2Error) as e:
        ctx.set_option(k2.K2_OPT_ACT8, 1)
    assert e.value.status == k2.K2_ERR_UNSUPPORTED and "eps" in str(e.value)
    assert k2.LIB.k2_act8_bytes(ctx.ctx) == 0
    if eps < 1:
        assert torch.isfinite(logits(k2, ctx)).all()


def test_weights_that_are_still_on_their_way_on_another_stream(k2):
    """The option set right behind a context whose weights are packed on another stream, which is busy."""
    from dense_gqa_decoder_gb300 import model_io
    dev, _ = model_io.device_weights(ki.MEDIUM, gain_scale=0.1)
    cfg = k2.make_config(ki.MEDIUM, max_context=128, kv_dtype="f16", weights="f8")
    rows = []
    for side in (None, torch.cuda.Stream()):
        big = torch.randn(8192, 8192, device="cuda")
        torch.cuda.synchronize()
        if side is not None:
            with torch.cuda.stream(side):
                for _ in range(20):
                    torch.mm(big, big)
        ctx = k2.Context(cfg, dev, stream=side)
        ctx.set_option(k2.K2_OPT_ACT8, 1)
        rows.append(logits(k2, ctx))
    assert torch.equal(*rows)
