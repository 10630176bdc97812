"""Shared-prefix attention on the GPU against its 64-bit form (tolerances: _rope_prefix.Attention.check)."""
import math

import pytest
import torch

import sparse_attention_dsa_gb300 as dsa

from _gpu import ensure_built
from _rope_prefix import KV, LATENT, PAGE, Attention, Batch, latent_fp8_rows, rope_table, rotate

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    ensure_built()


class Call:
    """A batch with its cache and queries, and one call.  wide: its page table has room for contexts so long that the
    work is divided among the CTAs however short the sequences are."""

    def __init__(self, seq_lens, q_lens, prefix, heads, fp8=False, seed=0, gain=1.0, wide=False, **dims):
        self.b = Batch(seq_lens, q_lens, prefix, seed)
        if wide:
            self.b.pt_host = torch.nn.functional.pad(self.b.pt_host, (0, 40), value=-1)
            self.b.pt = self.b.pt_host.cuda()
        g = torch.Generator(device="cuda").manual_seed(seed + 1)
        rows = torch.randn((self.b.pages * PAGE, KV), generator=g, device="cuda").to(torch.bfloat16)
        if prefix % PAGE:  # every sequence's copy of the page in which the prefix ends
            page = self.b.pt[:, prefix // PAGE].long()
            copies = rows.view(-1, PAGE, KV)
            copies[page, :prefix % PAGE] = copies[page[0], :prefix % PAGE].clone()
        self.fp8 = fp8
        self.cache = (latent_fp8_rows(rows) if fp8 else rows).view(self.b.pages, PAGE, -1)
        self.q = (gain * torch.randn((self.b.T, heads, KV), generator=g, device="cuda")).to(torch.bfloat16)
        self.prefix = prefix
        self.dims = self.b.dims(attn_heads=heads, kv_dtype=dsa.DSA_FP8_E4M3 if fp8 else dsa.DSA_BF16, **dims)
        self.workspace = torch.zeros(dsa.prefix_attn_workspace_size(self.dims, prefix), dtype=torch.uint8, device="cuda")
        self.out = torch.full((self.dims.total_q, heads, LATENT), 7.0, dtype=torch.bfloat16, device="cuda")
        self.lse = torch.full((self.dims.total_q, heads), 7.0, device="cuda")

    def run(self, stream=None, lse=True):
        dsa.prefix_attn(self.dims, self.prefix, self.q, self.cache, self.b.pt, self.b.lens, self.b.cu, self.out,
                        self.lse if lse else None, self.workspace, stream)
        return self

    def error(self):
        return dsa.get_device_error(self.workspace)

    def check(self, **kw):
        assert self.error() == 0
        Attention(self.b, self.q, self.cache, self.fp8).check(self.out, self.lse, self.fp8, **kw)


SHAPES = {
    # name: (seq_lens, q_lens, prefix, heads)
    "one_row": ([1], [1], 0, 1),
    "one_token_no_prefix": ([1], [1], 0, 128),
    "prefix_of_one": ([2, 5, 3], [1, 1, 1], 1, 16),
    "own_page_copies": ([100, 101, 163], [1, 1, 1], 99, 16),
    "page_aligned_prefix": ([129, 192, 193, 500], [1, 1, 1, 1], 128, 16),
    "no_prefix_ragged": ([64, 65, 127, 1, 300], [1, 1, 1, 1, 1], 0, 128),
    "two_queries": ([700, 514, 600], [2, 2, 2], 512, 128),
    "ragged_queries_and_none": ([700, 520, 900, 513], [3, 0, 70, 1], 512, 24),
    "odd_heads": ([333, 400], [5, 2], 300, 7),
    "whole_prompt": ([130], [130], 0, 32),
    "whole_prompts_behind_a_prefix": ([330, 201, 457], [130, 1, 257], 200, 16),
    "long_prefix_few_rows": ([20011, 20003], [1, 1], 20000, 8),
    "long_context_each": ([9000, 4000, 8191], [1, 2, 1], 0, 16),
    "packed_many": ([1100 + 7 * i for i in range(40)], [1] * 40, 1090, 16),
    "full_heads_many": ([1100 + 7 * i for i in range(12)], [1] * 12, 1090, 128),
    "full_heads_chunk": ([600, 700], [100, 150], 450, 128),
    "heads_33": ([2100, 2300, 2048], [1, 9, 4], 2000, 33),
    # enough tiles of rows over the prefix that FP8 rows are converted ahead: merged, then packed rows
    "full_heads_long_prefix": ([1100 + 7 * i for i in range(20)], [1] * 20, 1090, 128),
    "packed_ragged": ([900 + 11 * i for i in range(24)], [i % 5 for i in range(24)], 800, 16),
    "packed_long_prefix": ([2510 + 3 * i for i in range(64)], [1] * 64, 2500, 16),
    "packed_thirteen_tiles": ([2510 + i % 90 for i in range(101)], [1] * 101, 2500, 16),
    # more items than are divided evenly: whole items in turn
    "thousands_of_short_ones": ([1 + i % 70 for i in range(2100)], [1] * 2100, 0, 128),
    "many_behind_one_page": ([64 + 1 + i % 5 for i in range(300)], [1] * 300, 64, 32),
}


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("name", list(SHAPES))
def test_attention(name, fp8, wide):
    Call(*SHAPES[name], fp8=fp8, seed=len(name), wide=wide).run().check()


@pytest.mark.parametrize("fp8", [False, True])
def test_peaked_scores(fp8):
    """Scores tens of units apart, so that the running maximum moves and most weights vanish."""
    Call([1500, 1700], [1, 3], 1400, 64, fp8=fp8, seed=2, gain=4.0 if fp8 else 12.0, wide=True).run().check()


def test_rising_and_falling_scores():
    """The largest scores at the far end, or at the start, of a long context."""
    for order in (1, -1):
        c = Call([4000], [1], 0, 32, seed=3)
        ramp = torch.linspace(0, 40, 4000, device="cuda")
        at = torch.arange(4000)
        rows = (c.b.pt_host[0, at // PAGE].long() * PAGE + at % PAGE).cuda()
        c.q.zero_()
        c.q[..., 575] = 24.0  # z = row's last value
        flat = c.cache.view(-1, KV)
        flat[rows, 575] = (ramp if order > 0 else ramp.flip(0)).to(torch.bfloat16)
        c.run().check()


def test_many_small_weights_beside_a_large_one():
    """FP8 rows: one score 24.5 powers of two above all the others, whose weights sum to a share that no rounding
    of single ones may lose."""
    c = Call([60000], [1], 0, 16, fp8=True, seed=22)
    rows = torch.zeros((c.b.pages * PAGE, KV), device="cuda")
    rows[:, :LATENT] = 1.0
    sink = int(c.b.pt_host[0, 777 // PAGE]) * PAGE + 777 % PAGE
    rows[sink] = 0.0
    rows[sink, 575] = 17.0
    c.cache = latent_fp8_rows(rows.to(torch.bfloat16)).view(c.b.pages, PAGE, -1)
    c.q.zero_()
    c.q[..., 575] = 24.0  # z = row's last value
    c.run().check()


@pytest.mark.parametrize("name", ["two_queries", "packed_long_prefix"])
def test_small_fp8_rows(name):
    """Rows of values about 2e-4: their scales are far below what f16 holds."""
    c = Call(*SHAPES[name], fp8=True, seed=23)
    g = torch.Generator(device="cuda").manual_seed(24)
    rows = 2e-4 * torch.randn((c.b.pages * PAGE, KV), generator=g, device="cuda")
    c.cache = latent_fp8_rows(rows.to(torch.bfloat16)).view(c.b.pages, PAGE, -1)
    if c.prefix % PAGE:
        page = c.b.pt[:, c.prefix // PAGE].long()
        c.cache[page, :c.prefix % PAGE] = c.cache[page[0], :c.prefix % PAGE].clone()
    c.run().check()


def test_without_lse():
    a = Call(*SHAPES["two_queries"], seed=4).run()
    kept = a.out.clone()
    a.out.zero_()
    a.run(lse=False)
    assert torch.equal(a.out, kept) and a.error() == 0


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("name", ["own_page_copies", "no_prefix_ragged", "ragged_queries_and_none", "whole_prompt",
                                  "whole_prompts_behind_a_prefix", "packed_many", "full_heads_chunk",
                                  "full_heads_long_prefix", "packed_long_prefix", "packed_ragged"])
def test_what_is_not_visible_does_not_matter(name, fp8, wide):
    """NaN and infinities in rows behind each sequence's end, in spare pages, and in the copies of the prefix's
    last page that are not read, change no bit."""
    c = Call(*SHAPES[name], fp8=fp8, seed=5, wide=wide).run()
    want = c.out.clone(), c.lse.clone()
    used = torch.zeros(c.b.pages * PAGE, dtype=torch.bool)
    for i in range(c.b.B):
        at = torch.arange(c.b.L[i])
        src = torch.where(at < c.prefix, 0, i)
        used[c.b.pt_host[src, at // PAGE].long() * PAGE + at % PAGE] = True
    flat = c.cache.view(-1, c.cache.shape[-1])
    bad = (~used).nonzero().flatten().cuda()
    if fp8:
        flat[bad] = 0x7F  # NaN codes, NaN scales, NaN rotary values
    else:
        flat[bad[0::2]] = math.nan
        flat[bad[1::2]] = math.inf
    c.run()
    assert c.error() == 0
    assert torch.equal(c.out, want[0]) and torch.equal(c.lse, want[1])


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("heads", [16, 128])
@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf])
def test_a_bad_new_row_reaches_only_the_queries_that_see_it(heads, value, wide):
    """Query j of a step must not notice what the later tokens of the step hold."""
    c = Call([205, 100], [5, 5], 90, heads, seed=6, wide=wide).run()
    want = c.out.clone(), c.lse.clone()
    p = 203  # position of sequence 0's fourth query
    c.cache[int(c.b.pt_host[0, p // PAGE]), p % PAGE] = value
    c.run()
    assert c.error() == 0
    assert torch.equal(c.out[:3], want[0][:3]) and torch.equal(c.lse[:3], want[1][:3])
    assert torch.equal(c.out[5:], want[0][5:]) and torch.equal(c.lse[5:], want[1][5:])
    assert bool(c.out[3:5].isnan().all()) and bool(c.lse[3:5].isnan().all())


@pytest.mark.parametrize("wide", [False, True])
def test_a_nan_query_row_stays_alone(wide):
    c = Call([205, 100, 170], [1, 1, 1], 90, 16, seed=7, wide=wide).run()
    want = c.out.clone()
    c.q[1, 3, 10] = math.nan
    c.run()
    keep = torch.ones((3, 16), dtype=torch.bool)
    keep[1, 3] = False
    assert torch.equal(c.out[keep], want[keep]) and bool(c.out[1, 3].isnan().all()) and bool(c.lse[1, 3].isnan())


@pytest.mark.parametrize("wide", [False, True])
def test_scores_of_minus_infinity_have_no_weight(wide):
    """Rows whose rotary part makes every score -inf: out 0, lse -inf; some of them: as if they were not there."""
    c = Call([130, 70], [1, 1], 64, 16, seed=8, wide=wide)
    c.q[..., 575] = 1.0
    c.cache[..., 575] = -math.inf
    c.run()
    assert c.error() == 0
    assert not bool(c.out.any()) and bool((c.lse == -math.inf).all())
    c = Call([130, 70], [1, 1], 64, 16, seed=8, wide=wide)
    c.q[..., 575] = 1.0
    page = int(c.b.pt_host[0, 0])
    c.cache[page, 5:60, 575] = -math.inf
    c.run().check()


@pytest.mark.parametrize("wide", [False, True])
def test_inconsistent_sequences_are_reported_and_left_alone(wide):
    c = Call([300, 300, 300], [1, 1, 1], 200, 16, seed=9, wide=wide, total_q=5)
    c.q = torch.cat([c.q, c.q[:2]])
    ref = Attention(c.b, c.q[:3], c.cache, False)
    c.b.lens[1] = 200  # its query would lie inside the prefix
    c.run()
    assert c.error() == dsa.DSA_DEVERR_SEQ
    assert bool((c.out[1] == 7).all()) and bool((c.lse[1] == 7).all())
    assert bool((c.out[3:] == 7).all()) and bool((c.lse[3:] == 7).all())  # tokens of no sequence
    for t in (0, 2):
        ref.check(c.out[:3], c.lse[:3], False, tokens=slice(t, t + 1))
    dsa.clear_device_error(c.workspace)
    c.b.lens[1] = c.b.pt.shape[1] * PAGE + 1  # beyond its page table
    c.run()
    assert c.error() == dsa.DSA_DEVERR_SEQ and bool((c.out[1] == 7).all())


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("heads", [16, 128])
@pytest.mark.parametrize("fp8", [False, True])
def test_bad_pages_are_reported_and_skipped(heads, fp8, wide):
    c = Call([400, 330], [1, 1], 256, heads, fp8=fp8, seed=10, wide=wide)
    ref = Call([400, 330], [1, 1], 256, heads, fp8=fp8, seed=10, wide=wide).run()
    c.b.pt[0, 5] = c.b.pages  # positions 320..383 of sequence 0
    c.run()
    assert c.error() == dsa.DSA_DEVERR_PAGE
    assert torch.equal(c.out[1], ref.out[1]) and torch.equal(c.lse[1], ref.lse[1])
    assert bool(c.out[0].isfinite().all()) and not torch.equal(c.out[0], ref.out[0])
    # the weights that are left sum to less: the log-sum-exp falls
    assert bool((c.lse[0] < ref.lse[0]).all())


def test_rows_behind_four_gigabytes():
    c = Call([200], [1], 100, 16, seed=11)
    pages = 70000
    big = torch.zeros((pages, PAGE, KV), dtype=torch.bfloat16, device="cuda")
    move = torch.arange(c.b.pages, device="cuda") + pages - c.b.pages
    big[move] = c.cache
    c.cache = big
    c.b.pt = torch.where(c.b.pt >= 0, c.b.pt + pages - c.b.pages, c.b.pt)
    c.b.pt_host = c.b.pt.cpu()
    c.dims.num_pages = pages
    c.run().check()


@pytest.mark.parametrize("wide", [False, True])
def test_the_same_twice_and_on_another_stream(wide):
    c = Call(*SHAPES["packed_many"], seed=12, wide=wide).run()
    want = c.out.clone(), c.lse.clone()
    s = torch.cuda.Stream()
    for stream in (None, s):
        c.out.zero_(), c.lse.zero_()
        s.wait_stream(torch.cuda.current_stream())
        c.run(stream)
        torch.cuda.synchronize()
        assert torch.equal(c.out, want[0]) and torch.equal(c.lse, want[1])


def test_two_calls_at_once_with_their_own_workspaces():
    a = Call(*SHAPES["packed_many"], seed=13, wide=True)
    b = Call(*SHAPES["full_heads_many"], seed=14, wide=True)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(5):
        a.run(s1)
        b.run(s2)
    torch.cuda.synchronize()
    a.check()
    b.check()


def test_two_graphs_of_one_workspace():
    """Two captured calls of different shapes that share a workspace, replayed in turn."""
    a = Call(*SHAPES["packed_long_prefix"], fp8=True, seed=18)
    b = Call(*SHAPES["full_heads_many"], seed=19, wide=True)
    size = max(a.workspace.numel(), b.workspace.numel())
    a.workspace = b.workspace = torch.zeros(size, dtype=torch.uint8, device="cuda")
    graphs = []
    for c in (a, b):
        c.run()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c.run()
        graphs.append(g)
        c.out.zero_(), c.lse.zero_()
    for _ in range(3):
        for g in graphs:
            g.replay()
    a.check()
    b.check()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("name, wide", [("packed_many", True), ("full_heads_chunk", True), ("full_heads_chunk", False),
                                        ("one_token_no_prefix", False)])
def test_waits_give_up_at_their_limit(name, wide, fp8):
    """With a limit of a nanosecond some wait finds its phase incomplete and gives up: the call reports it and ends,
    and the next call, at the default limit, is right."""
    c = Call(*SHAPES[name], fp8=fp8, seed=20, wide=wide)
    old = dsa.set_wait_limit_ns(1)
    try:
        c.run()
        assert c.error() & dsa.DSA_DEVERR_TIMEOUT
    finally:
        dsa.set_wait_limit_ns(old)
    dsa.clear_device_error(c.workspace)
    c.run().check()


def test_a_context_whose_tiles_would_pass_32_bits_is_reported():
    c = Call([300], [1], 0, 16, seed=25)
    pages = (1 << 25) - 1  # the widest page table that a call takes
    c.b.pt = torch.zeros((1, pages), dtype=torch.int32, device="cuda")
    c.dims.max_pages_per_seq = pages
    c.workspace = torch.zeros(dsa.prefix_attn_workspace_size(c.dims, 0), dtype=torch.uint8, device="cuda")
    c.b.lens.fill_(64 * pages)
    c.run()
    assert c.error() == dsa.DSA_DEVERR_SEQ and bool((c.out == 7).all())


def test_more_queries_than_announced_are_reported():
    c = Call([300, 300], [1, 3], 200, 16, seed=21)
    c.dims.max_q_len = 2
    ref = Attention(c.b, c.q, c.cache, False)
    c.run()
    assert c.error() == dsa.DSA_DEVERR_SEQ
    assert bool((c.out[1:] == 7).all())
    ref.check(c.out, c.lse, False, tokens=slice(0, 1))


@pytest.mark.parametrize("wide", [False, True])
def test_a_captured_call_replays_on_new_lengths(wide):
    c = Call([700, 514, 600], [1, 1, 1], 512, 16, seed=15, wide=wide)
    c.b.lens -= 30
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.run()
    g.replay()
    assert c.error() == dsa.DSA_DEVERR_SEQ  # 514 - 30 < 512 + 1: sequence 1's query lies inside the prefix
    dsa.clear_device_error(c.workspace)
    c.b.lens += 30
    g.replay()
    c.check()


def test_a_step_rotated_appended_and_attended():
    """The operators as a serving step uses them: rows rotated into the cache, queries rotated, attention over
    the shared prefix - against the same step in 64 bits."""
    c = Call([700, 514, 600, 530], [2, 1, 3, 1], 512, 32, seed=16)
    b = c.b
    table = rope_table(800, "cuda")
    rope = dsa.DsaRope(table=table.data_ptr(), table_len=800, kv_pairing=dsa.DSA_ROPE_INTERLEAVED,
                       idx_pairing=dsa.DSA_ROPE_HALVES, idx_begin=0)
    g = torch.Generator(device="cuda").manual_seed(5)
    kv_new = torch.randn((b.T, KV), generator=g, device="cuda").to(torch.bfloat16)
    q_raw = c.q.clone()
    dsa.rope_append(c.dims, rope, None, kv_new, b.pt, b.lens, b.cu, None, None, c.cache, c.workspace)
    dsa.rope_queries(c.dims, rope, c.q.data_ptr() + 2 * LATENT, c.q, None, None, None, b.lens, b.cu, c.workspace,
                     q_pe_strides=(32 * KV, KV))
    c.run()
    assert c.error() == 0
    rows = table[torch.tensor(b.pos, device="cuda")]
    turned = rotate(kv_new[:, LATENT:].double(), rows, True)
    cache_rows = c.cache.view(-1, KV)[b.rows]
    assert torch.equal(cache_rows[:, :LATENT], kv_new[:, :LATENT])
    assert bool(((cache_rows[:, LATENT:].double() - turned).abs() <= 2.0 ** -8 * turned.abs() + 1e-6).all())
    turned = rotate(q_raw[..., LATENT:].double(), rows, True)
    assert bool(((c.q[..., LATENT:].double() - turned).abs() <= 2.0 ** -8 * turned.abs() + 1e-6).all())
    Attention(b, c.q, c.cache, False).check(c.out, c.lse, False)


def test_a_rotated_step_feeds_the_sparse_path():
    """rope_append and rope_queries in front of the fused indexer and sparse attention, FP8 caches: with as many
    Top-K as visible positions the selection is everything, and the attention is prefix_attn's."""
    c = Call([200, 130], [1, 1], 64, 128, fp8=True, seed=17)
    b, d = c.b, c.dims
    d.idx_dtype, d.top_k = dsa.DSA_FP8_E4M3, 256
    table = rope_table(256, "cuda")
    rope = dsa.DsaRope(table=table.data_ptr(), table_len=256, kv_pairing=dsa.DSA_ROPE_INTERLEAVED,
                       idx_pairing=dsa.DSA_ROPE_HALVES, idx_begin=0)
    g = torch.Generator(device="cuda").manual_seed(6)

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16)

    k_cache = torch.zeros((b.pages, PAGE, 128), dtype=torch.uint8, device="cuda")
    k_scale = torch.ones((b.pages, PAGE), device="cuda")
    q_idx = torch.zeros((b.T, 64, 128), dtype=torch.uint8, device="cuda")
    q_scale = torch.zeros((b.T, 64), device="cuda")
    w = torch.rand((b.T, 64), generator=g, device="cuda")
    ws = torch.zeros(dsa.workspace_size(d), dtype=torch.uint8, device="cuda")
    topk = torch.zeros((b.T, 256), dtype=torch.int32, device="cuda")
    out, lse = torch.zeros_like(c.out), torch.zeros_like(c.lse)
    dsa.rope_append(d, rope, normal(b.T, 128), normal(b.T, KV), b.pt, b.lens, b.cu, k_cache, k_scale, c.cache, ws)
    dsa.rope_queries(d, rope, normal(b.T, 128, 64), c.q, normal(b.T, 64, 128), q_idx, q_scale, b.lens, b.cu, ws)
    dsa.fused_decode(d, q_idx, q_scale, w, k_cache, k_scale, c.q, c.cache, b.pt, b.lens, b.cu, topk, out, lse, ws)
    assert dsa.get_device_error(ws) == 0
    assert topk[0, :200].tolist() == list(range(200)) and topk[1, :130].tolist() == list(range(130))
    c.run()
    assert c.error() == 0
    # both round the same values to bf16 once more at the end, and their weights to bf16: two half steps each
    assert bool(((out.double() - c.out.double()).abs() <= 4 * 2.0 ** -8 * (c.out.double().abs() + 1)).all())
    assert bool(((lse - c.lse).abs() <= 2.0 ** -8 + 2.0 ** -20).all())
