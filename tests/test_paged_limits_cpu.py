"""Host-side checks of what test_gpu_paged_limits.py relies on.  No GPU is needed."""
import ctypes as C

import pytest

A = 0x1000  # an aligned non-null address that no refused call reads


@pytest.fixture(scope="module")
def k2():
    from dense_gqa_decoder_gb300 import build
    build.build()
    from dense_gqa_decoder_gb300 import k2 as mod
    return mod


def test_a_negative_wait_limit_is_refused(k2):
    kv = k2.PagedKv(k=A, v=A, k_scale=A, v_scale=A, n_blocks=4, block_tokens=16, n_kv_heads=2, head_dim=128, dtype=k2.K2_I8,
                    wait_limit_us=-1)
    ref = C.addressof(kv)
    assert k2.LIB.k2_paged_append(ref, A, A, k2.K2_BF16, 256, 256, A, 1, None) == k2.K2_ERR_ARG
    assert "wait_limit_us" in k2.LIB.k2_last_error(None).decode()
    assert k2.LIB.k2_paged_attention(ref, A, k2.K2_BF16, 1024, A, A, A, 4, 1, 1, 8, 1, 0.1, 2 * A, 1024, A, 1 << 30, None) == k2.K2_ERR_ARG


def test_the_wait_limit_moves_no_other_field(k2):
    assert C.sizeof(k2.PagedKv) == 64 and k2.PagedKv.flags.offset == 56 and k2.PagedKv.dtype.offset == 48


ATTEND = dict(q=2 ** 20, q_stride=1024, tokens=4, out=2 ** 24, out_stride=1024)


@pytest.mark.parametrize("kw", [dict(out=2 ** 20), dict(out=2 ** 20 + 64), dict(out=2 ** 20 - 64), dict(out=2 ** 20 + 2048 * 3 + 1024),
                                dict(out=2 ** 20 - 2048 * 3 - 1024), dict(q_stride=2048, out_stride=2048, out=2 ** 20 + 2032),
                                dict(q_stride=2048, out_stride=2048, out=2 ** 20 + 2048 + 16), dict(out_stride=2048, out=2 ** 20 + 16),
                                dict(tokens=1, q_stride=0, out_stride=0, out=2 ** 20 + 2032)])
def test_attention_output_over_a_part_of_the_queries_is_refused(k2, kw):
    a = {**ATTEND, **kw}
    kv = k2.PagedKv(k=A, v=A, k_scale=A, v_scale=A, n_blocks=4, block_tokens=16, n_kv_heads=2, head_dim=128, dtype=k2.K2_I8)
    assert k2.LIB.k2_paged_attention(C.addressof(kv), a["q"], k2.K2_F16, a["q_stride"], A, A, A, 4, 1, a["tokens"], 8, 1, 0.1,
                                     a["out"], a["out_stride"], A, 1 << 30, None) == k2.K2_ERR_ARG
    assert "queries" in k2.LIB.k2_last_error(None).decode()


@pytest.mark.parametrize("rows,ld,ld_out,shift", [(3, 40, 40, 4), (3, 40, 40, -4), (3, 40, 40, 4 * 100), (1, 0, 0, 4 * 39),
                                                  (3, 64, 64, 4 * 39), (3, 64, 64, 4 * 25), (2, 40, 48, 4)])
def test_rules_output_over_a_part_of_the_logits_is_refused(k2, rows, ld, ld_out, shift):
    u = k2.LogitRules()
    assert k2.LIB.k2_adjust_logits(C.byref(u), 2 ** 20, ld, 2 ** 20 + shift, ld_out, rows, 40, None) == k2.K2_ERR_ARG
    assert "part" in k2.LIB.k2_last_error(None).decode()
