"""How a shared-prefix attention call is divided and what workspace it takes, from its sizes alone (host, no GPU)."""
import pytest

import sparse_attention_dsa_gb300 as dsa
from sparse_attention_dsa_gb300 import build as dsa_build

INT_MAX = 2**31 - 1


@pytest.fixture(scope="module", autouse=True)
def _built():
    dsa_build.build()


def _dims(**kw):
    d = dict(batch=2, total_q=2, max_q_len=1, num_pages=4096, page_size=64, max_pages_per_seq=32, idx_heads=64,
             idx_dim=128, idx_dtype=0, top_k=16, attn_heads=128, kv_dim=576, v_dim=512, softmax_scale=1 / 24)
    d.update(kw)
    return dsa.DsaDims(**d)


def _size(prefix=0, **kw):
    return dsa.prefix_attn_workspace_size(_dims(**kw), prefix)


@pytest.mark.parametrize("batch,total,heads", [(1, 1, 128), (1, 1, 16), (3, 7, 128), (64, 64, 16), (5, 1000, 33)])
@pytest.mark.parametrize("most", [2**25, INT_MAX])
def test_no_sequence_is_taken_to_have_more_queries_than_the_batch(batch, total, heads, most):
    """max_q_len may be any bound on the query counts: rows behind the batch's are no items (their numbers would pass 32
    bits, and the items' rows lie in front of the outputs)."""
    for prefix in (0, 2000):
        small = _size(prefix, batch=batch, total_q=total, max_q_len=total, attn_heads=heads)
        assert _size(prefix, batch=batch, total_q=total, max_q_len=most, attn_heads=heads) == small
