"""How a shared-prefix attention call is divided and what workspace it takes, from its sizes alone (host, no GPU)."""
import random

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


FAKE = 0x10000  # an aligned non-null address; never dereferenced


@pytest.mark.parametrize("prefix", [2**31 - 256, 2**31 - 128, 64 * (2**25 - 1)])
@pytest.mark.parametrize("heads,dtype", [(16, dsa.DSA_BF16), (128, dsa.DSA_FP8_E4M3)])
def test_a_prefix_that_no_context_can_hold_is_refused(prefix, heads, dtype):
    """Contexts end before 2^31 - 255 positions and every query lies behind the prefix; tiles of a longer prefix would end
    beyond 32 bits."""
    d = _dims(batch=64, total_q=64, max_pages_per_seq=2**25 - 1, attn_heads=heads, kv_dtype=dtype)
    with pytest.raises(dsa.DsaError, match="prefix_len") as e:
        dsa.prefix_attn(d, prefix, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, None, FAKE, stream=0)
    assert e.value.status == dsa.DSA_ERR_UNSUPPORTED
    assert dsa.prefix_attn_workspace_size(d, prefix) == 256
    d.max_pages_per_seq = 1
    assert dsa.prefix_attn_workspace_size(d, 2**31 - 1) == 256


PART = 4 * (128 * 512 + 2 * 128)  # bytes of a partial result


@pytest.mark.parametrize("what,dims,prefix", [
    # one sequence with a chunk of queries among single ones: as the same batch without it
    ("one of 33 queries", dict(batch=64, total_q=96, max_q_len=33, max_pages_per_seq=2048), 0),
    ("one of 512 queries", dict(batch=256, total_q=767, max_q_len=512, max_pages_per_seq=64), 0),
    ("chunk behind a prefix", dict(batch=64, total_q=575, max_q_len=512, max_pages_per_seq=523, attn_heads=16), 32768),
    ("many behind a prefix", dict(batch=2048, total_q=2048, max_pages_per_seq=66, attn_heads=16), 4096),
])
def test_empty_items_do_not_count_against_a_division(what, dims, prefix):
    """A division of the work is seen by the room for its partial results."""
    assert _size(prefix, **dims) > 76 * PART


def _smaller(rng, d):
    """Dims whose sizes are no larger."""
    def at_most(v):
        return rng.choice([v, 1, rng.randint(1, v), max(1, v // rng.choice([2, 3, 7, 50]))])

    return dict(d, batch=at_most(d["batch"]), total_q=at_most(d["total_q"]), max_q_len=at_most(d["max_q_len"]),
                max_pages_per_seq=at_most(d["max_pages_per_seq"]))


@pytest.mark.parametrize("heads", [1, 16, 48, 64, 100, 128])
@pytest.mark.parametrize("dtype", [dsa.DSA_BF16, dsa.DSA_FP8_E4M3])
def test_a_workspace_serves_every_smaller_call(heads, dtype):
    rng = random.Random(heads + 1000 * dtype)
    for _ in range(2000):
        d = dict(batch=rng.choice([1, 2, 8, 38, 64, 76, 128, 300, 2100]), max_q_len=rng.choice([1, 2, 33, 512, 4096]),
                 max_pages_per_seq=rng.choice([1, 4, 16, 17, 32, 33, 40, 520, 2048]), attn_heads=heads, kv_dtype=dtype)
        d["total_q"] = rng.choice([1, d["batch"], rng.randint(1, d["batch"] * d["max_q_len"]), d["batch"] * d["max_q_len"]])
        prefix = rng.choice([0, 0, 1, 100, 64 * d["max_pages_per_seq"], rng.randint(0, 64 * d["max_pages_per_seq"])])
        size = _size(prefix, **d)
        for _ in range(5):
            low = _smaller(rng, d)
            p = min(rng.choice([prefix, 0, rng.randint(0, prefix)]), 64 * low["max_pages_per_seq"])
            assert _size(p, **low) <= size, (d, prefix, low, p)


def test_a_shrinking_batch():
    """Eight sequences of up to 2048 positions are divided, 38 to 128 are not: the larger batch's workspace is enough."""
    sizes = [_size(0, batch=b, total_q=b) for b in (8, 38, 76, 128)]
    assert sizes == sorted(sizes) and sizes[0] > 152 * PART


def test_a_short_workspace_is_refused():
    class Buffer:
        def __init__(self, size):
            self.size = size

        def numel(self):
            return self.size

        def element_size(self):
            return 1

        def data_ptr(self):
            return FAKE

    d = _dims(batch=8, total_q=8)
    need = dsa.prefix_attn_workspace_size(d, 0)
    with pytest.raises(dsa.DsaError, match="workspace") as e:
        dsa.prefix_attn(d, 0, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, None, Buffer(need - 1), stream=0)
    assert e.value.status == dsa.DSA_ERR_INVALID_ARG
    d.total_q = 0  # nothing to do
    dsa.prefix_attn(d, 0, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, None, Buffer(need), stream=0)
