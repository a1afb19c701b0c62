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
