"""In-place calls of dsa_rope_queries that the kernel cannot do: answered on the host (no GPU)."""
import ctypes

import pytest

import sparse_attention_dsa_gb300 as dsa
from sparse_attention_dsa_gb300 import build as dsa_build

FAKE, OTHER = 0x10000, 0x20000  # aligned non-null addresses; never dereferenced


@pytest.mark.parametrize("dtype,stride,q_idx,refused", [
    (dsa.DSA_BF16, 0, FAKE, False),
    (dsa.DSA_BF16, 64 * 128, FAKE, False),
    (dsa.DSA_BF16, 64 * 128 + 8, FAKE, True),
    (dsa.DSA_FP8_E4M3, 0, FAKE, True),
    (dsa.DSA_MXFP8_E4M3, 0, FAKE, True),
    (dsa.DSA_BF16, 64 * 128 + 8, OTHER, False),
    (dsa.DSA_FP8_E4M3, 0, OTHER, False),
])
def test_only_dense_bf16_rows_are_rotated_in_place(dtype, stride, q_idx, refused):
    dsa_build.build()
    d = dsa.DsaDims(batch=2, total_q=0, max_q_len=1, num_pages=8, page_size=64, max_pages_per_seq=4, idx_heads=64,
                    idx_dim=128, idx_dtype=dtype, top_k=16, attn_heads=128, kv_dim=576, v_dim=512, softmax_scale=1 / 24)
    rope = dsa.DsaRope(table=FAKE, table_len=1024, kv_pairing=1, idx_pairing=0, idx_begin=0)
    status = dsa.lib().dsa_rope_queries(ctypes.byref(d), ctypes.byref(rope), None, 0, 0, None, FAKE, stride, q_idx,
                                        None if dtype == dsa.DSA_BF16 else OTHER, FAKE, FAKE, FAKE, None)
    assert status == (dsa.DSA_ERR_INVALID_ARG if refused else dsa.DSA_OK)
    if refused:
        assert "q_idx" in dsa.lib().dsa_last_error_message().decode()
