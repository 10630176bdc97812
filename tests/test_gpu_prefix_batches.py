"""Shared-prefix attention of batches whose sequences are unlike one another, against the 64-bit form."""
import pytest
import torch

import sparse_attention_dsa_gb300 as dsa  # noqa: F401

from _gpu import ensure_built
from test_gpu_prefix import SHAPES, Call

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    ensure_built()


@pytest.mark.parametrize("where", [0, 63])
def test_a_long_chunk_among_single_queries(where):
    """Between two items of the batch lie hundreds that are empty, so that some warps of a CTA find the next one tiles
    later than others; the tiles before an item's last are ones that every row sees whole."""
    n = [1] * 64
    n[where] = 400
    Call([900 + (i % 9) * 31 for i in range(64)], n, 0, 128, seed=30).run().check()


@pytest.mark.parametrize("name", ["one_row", "two_queries", "ragged_queries_and_none", "packed_many"])
@pytest.mark.parametrize("most", [2**25, 2**31 - 1])
def test_any_bound_on_the_query_counts_may_be_announced(name, most):
    Call(*SHAPES[name], seed=31, max_q_len=most).run().check()
