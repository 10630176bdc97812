"""Shared-prefix attention of batches whose sequences are unlike one another, against the 64-bit form."""
import pytest
import torch

import sparse_attention_dsa_gb300 as dsa

from _gpu import ensure_built
from _rope_prefix import Attention
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


MIXED = {
    # name: (seq_lens, q_lens, prefix, heads)
    "chunk_first": ([900 + 31 * (i % 9) for i in range(40)], [70] + [1] * 39, 0, 128),
    "chunk_last": ([900 + 31 * (i % 9) for i in range(40)], [1] * 39 + [70], 0, 128),
    "chunk_between_empty_ones": ([700, 600, 900, 650, 800], [0, 0, 90, 0, 1], 512, 24),
    "few_heads_chunk": ([2600 + 31 * (i % 9) for i in range(30)], [1] * 11 + [45] + [2] * 18, 2500, 16),
    "chunk_of_odd_rows": ([520 + 7 * i for i in range(20)], [1] * 7 + [61, 0, 2] + [1] * 10, 450, 7),
    "thousands_behind_a_prefix": ([1100 + i % 70 for i in range(2100)], [1] * 2100, 1090, 16),
    "one_long_context": ([9000] + [300] * 30, [20] + [1] * 30, 0, 64),
}


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("name", list(MIXED))
def test_chunks_among_single_queries(name, fp8, wide):
    Call(*MIXED[name], fp8=fp8, seed=32, wide=wide).run().check()


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("heads", [16, 128])
def test_inconsistent_sequences_beside_a_chunk(heads, wide):
    """Sequences whose items are found by the rows in front of them: one that is inconsistent, and offsets that do not
    begin at 0, take nothing from the others."""
    n, L = [1, 40, 1, 2, 1, 1, 1, 1], [300, 420, 300, 310, 333, 500, 301, 290]
    c = Call(L, n, 200, heads, seed=33, wide=wide)
    ref = Attention(c.b, c.q, c.cache, False)
    c.b.lens[4] = 200  # its query (token 44) would lie inside the prefix
    c.run()
    assert c.error() == dsa.DSA_DEVERR_SEQ
    assert bool((c.out[44] == 7).all()) and bool((c.lse[44] == 7).all())
    for t in (slice(0, 44), slice(45, 48)):
        ref.check(c.out, c.lse, False, tokens=t)
    dsa.clear_device_error(c.workspace)
    c.out.fill_(7), c.lse.fill_(7)
    c.b.lens[4] = 333
    c.b.cu[0] = 1  # token 0 is nobody's, and sequence 0 has no query
    c.run()
    assert c.error() == dsa.DSA_DEVERR_SEQ
    assert bool((c.out[0] == 7).all()) and bool((c.lse[0] == 7).all())
    ref.check(c.out, c.lse, False, tokens=slice(1, 48))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("heads,prefix", [(16, 0), (16, 2500), (128, 0), (128, 1090)])
def test_one_workspace_for_a_batch_that_shrinks(heads, prefix, fp8):
    """A workspace of the largest step's size, and nothing written behind it by that step or the smaller ones."""
    steps = [([prefix + 1000 + 13 * (i % 40) for i in range(size)], [1] * size) for size in (128, 76, 40, 9, 2, 1)]
    steps.append(([prefix + 700, prefix + 500], [60, 3]))
    calls = [Call(L, n, prefix, heads, fp8=fp8, seed=34) for L, n in steps]
    for c in calls:  # as wide a page table for every step, as a program has
        c.b.pt = torch.nn.functional.pad(c.b.pt, (0, prefix // 64 + 33 - c.b.pt.shape[1]), value=-1)
        c.dims.max_pages_per_seq = c.b.pt.shape[1]
    d = calls[0].dims
    largest = dsa.DsaDims(**{**{n: getattr(d, n) for n, _ in d._fields_}, "max_q_len": 60})
    size = dsa.prefix_attn_workspace_size(largest, prefix)
    room = torch.full((size + (64 << 20),), 0xA5, dtype=torch.uint8, device="cuda")
    room[:256] = 0
    for c in calls:
        c.workspace = room[:size]
        c.run().check()
    assert bool((room[size:] == 0xA5).all())


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("heads,slots,others", [(16, 1, 5), (16, 40, 30), (128, 2, 20), (128, 1, 2)])
def test_padding_slots_in_front_need_no_pages(heads, slots, others, fp8, wide):
    """Slots without a context, the first of the batch among them, and one whose context ends inside the prefix: their
    page tables map nothing of the prefix."""
    prefix = 1090
    L, n = [prefix + 40 + 9 * i for i in range(others)], [1 + i % 2 for i in range(others)]
    c = Call([0] * slots + [70] + L, [0] * (slots + 1) + n, prefix, heads, fp8=fp8, seed=35, wide=wide)
    c.b.pt[:slots] = -1
    c.b.pt[slots, 2:] = -1
    c.run()
    assert c.error() == 0
    want = Call(L, n, prefix, heads, fp8=fp8, seed=35)  # the same batch without them, over the same cache
    pt = c.b.pt[slots + 1:]
    want.b.pt, want.b.pt_host = pt.contiguous(), pt.cpu()
    want.cache, want.q = c.cache, c.q
    Attention(want.b, want.q, want.cache, fp8).check(c.out, c.lse, fp8)


@pytest.mark.parametrize("fp8", [False, True])
def test_captured_between_other_work(fp8):
    """Calls captured behind a memory fill and behind one another, with an input that the step itself writes."""
    c = Call(*SHAPES["full_heads_long_prefix"], fp8=fp8, seed=36)
    d = Call(*SHAPES["packed_many"], fp8=fp8, seed=37, wide=True)
    q = c.q.clone()

    def step():
        c.q.zero_()
        dsa.clear_device_error(c.workspace)
        c.q.add_(q)
        c.run()
        dsa.clear_device_error(d.workspace)
        d.run()
        c.run()

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    c.out.zero_(), d.out.zero_()
    for _ in range(3):
        g.replay()
    c.check()
    d.check()
