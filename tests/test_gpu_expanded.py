"""Attention with expanded keys and values on the GPU against 64 bits (tolerances: _latent)."""
import math

import pytest
import torch

import sparse_attention_dsa_gb300 as dsa

from _gpu import ensure_built
from _latent import LATENT, NOPE, ROT, VALUE, Expanded, check_bf16, norm64, normal, weights
from _rope_prefix import KV, PAGE, Batch, latent_fp8_rows, rope_table

pytestmark = pytest.mark.gpu

SCALE = (NOPE + ROT) ** -0.5


@pytest.fixture(scope="module", autouse=True)
def _built():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    ensure_built()


class Call:
    """A batch with its inputs; dense query arrays unless `strided`."""

    def __init__(self, seq_lens, q_lens, heads, fp8=False, seed=0, strided=False, lse=True, std=1.0):
        self.b = Batch(seq_lens, q_lens, seed=seed)
        T = self.b.T
        self.heads, self.fp8 = heads, fp8
        self.rows = normal((self.b.pages * PAGE, KV), seed + 1, std)
        self.kv = (latent_fp8_rows(self.rows).view(self.b.pages, PAGE, -1) if fp8 else
                   self.rows.view(self.b.pages, PAGE, KV))
        self.w = weights(heads, seed + 2)
        self.strides = {}
        if strided:  # as a projection and dsa_rope_queries leave them
            self.q_nope = normal((T, heads, NOPE + ROT), seed + 3)[..., :NOPE]
            self.q_pe = normal((T, heads, KV), seed + 4)[..., LATENT:]
            self.strides = dict(q_nope_strides=self.q_nope.stride()[:2], q_pe_strides=self.q_pe.stride()[:2])
        else:
            self.q_nope, self.q_pe = normal((T, heads, NOPE), seed + 3), normal((T, heads, ROT), seed + 4)
        self.out = torch.full((T, heads, VALUE), 7.0, dtype=torch.bfloat16, device="cuda")
        self.lse = torch.full((T, heads), 7.0, device="cuda") if lse else None
        self.pages = max(1, sum(-(-l // PAGE) for l, n in zip(seq_lens, q_lens) if n))
        self.dims = self.b.dims(attn_heads=heads, kv_dtype=dsa.DSA_FP8_E4M3 if fp8 else dsa.DSA_BF16, softmax_scale=SCALE)
        size = dsa.expanded_attn_workspace_size(self.dims, self.pages)
        # whatever a workspace holds beyond its first 256 bytes
        self.ws = torch.full((size,), 0xFF, dtype=torch.uint8, device="cuda")
        self.ws[:256] = 0

    def run(self, **kw):
        a = dict(self.strides)
        a.update(kw)
        dsa.expanded_attn(self.dims, self.pages, self.q_nope, self.q_pe, self.w, self.kv, self.b.pt, self.b.lens, self.b.cu,
                          self.out, self.lse, self.ws, **a)
        return self

    def check(self, tokens=None, norm=True, error=0):
        assert dsa.get_device_error(self.ws) == error
        Expanded(self.b, self.q_nope, self.q_pe, self.w, self.kv, self.fp8).check(self.out, self.lse, tokens, norm)


BATCHES = [
    # seq_lens, q_lens
    ([1], [1]),
    ([5], [5]),
    ([64], [1]),
    ([127], [127]),
    ([128], [128]),
    ([129], [129]),
    ([300], [257]),
    ([1000], [256]),
    ([513], [513]),
    ([2000], [3]),
    ([777, 1, 130, 64, 900], [130, 1, 2, 64, 600]),
    ([300, 200, 100, 77], [0, 200, 0, 33]),
    ([129, 128, 127, 1, 1, 256, 255], [128, 128, 1, 1, 1, 255, 2]),
]


@pytest.mark.parametrize("seq_lens,q_lens", BATCHES)
@pytest.mark.parametrize("heads,fp8,strided", [(1, False, False), (5, True, True), (16, False, True)])
def test_batches(seq_lens, q_lens, heads, fp8, strided):
    # an average of few values keeps more of its weights' and values' roundings than one of many
    Call(seq_lens, q_lens, heads, fp8, seed=11, strided=strided).run().check()


def test_every_head():
    Call([400, 150], [300, 150], 128, seed=21, strided=True).run().check()


def test_long_context():
    Call([9000], [520], 3, seed=31).run().check()
    Call([20000], [40], 2, True, seed=32).run().check()


@pytest.mark.parametrize("seq_lens,q_lens,heads", [
    ([600, 7, 512, 900, 333], [600, 0, 512, 300, 333], 24),           # more short items than CTAs, of several sequences
    ([1 + 3 * i for i in range(256)], [1] * 256, 1),                  # 256 blocks of queries
    ([1 + 3 * i for i in range(257)], [1 + i % 2 for i in range(257)], 1),
    ([5000, 4700], [520, 500], 40),                                   # long items, fewer than two a CTA
    ([40, 5000, 4000], [40, 1024, 0], 50),
    ([6000], [768], 76),
])
def test_items_whole_and_cut(seq_lens, q_lens, heads):
    c = Call(seq_lens, q_lens, heads, seed=35).run()
    assert dsa.get_device_error(c.ws) == 0
    for h in (0, heads // 2, heads - 1):
        one = slice(h, h + 1)
        Expanded(c.b, c.q_nope[:, one], c.q_pe[:, one], c.w[one], c.kv, False).check(c.out[:, one], c.lse[:, one])
    want = c.out.clone(), c.lse.clone()
    c.out.fill_(7.0)
    c.run()
    assert torch.equal(c.out, want[0]) and torch.equal(c.lse, want[1])


def test_offsets_beyond_32_bits():
    """Keys and values of 128 heads and 70000 positions take 4.6 GB of workspace: the first and the last head's results."""
    c = Call([70000], [300], 128, seed=33, strided=True).run()
    assert dsa.get_device_error(c.ws) == 0
    for h in (0, 127):
        one = slice(h, h + 1)
        Expanded(c.b, c.q_nope[:, one], c.q_pe[:, one], c.w[one], c.kv, False).check(c.out[:, one], c.lse[:, one])


def test_many_sequences():
    g = torch.Generator().manual_seed(5)
    lens = torch.randint(1, 400, (1500,), generator=g).tolist()
    qs = [int(torch.randint(0, min(l, 9) + 1, (1,), generator=g)) for l in lens]
    Call(lens, qs, 2, seed=41).run().check()


def test_without_lse_and_on_another_stream():
    c = Call([500, 90], [200, 90], 8, seed=51, lse=False)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        c.run()
    side.synchronize()
    c.check()


def test_same_bits_again_and_calls_at_once():
    c = Call([1500, 700], [900, 700], 16, seed=61)
    c.run()
    want = c.out.clone(), c.lse.clone()
    other = Call([1500, 700], [900, 700], 16, seed=61)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        c.run()
        with torch.cuda.stream(side):
            other.run()
    torch.cuda.synchronize()
    for x in (c, other):
        assert torch.equal(x.out, want[0]) and torch.equal(x.lse, want[1])
    c.check()


def test_captured_calls_share_a_workspace():
    big, small = Call([1200], [600], 8, seed=71), Call([200, 70], [100, 70], 8, seed=72)
    assert dsa.expanded_attn_workspace_size(small.dims, small.pages) <= big.ws.numel()
    small.ws = big.ws
    graphs = []
    for c in (big, small):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c.run()
        graphs.append(g)
    for c in (big, small):
        c.q_nope.copy_(normal(c.q_nope.shape, 73))
    for i in (0, 1, 0, 1, 1, 0):
        graphs[i].replay()
    torch.cuda.synchronize()
    big.check()
    small.check()


def test_a_captured_call_with_other_lengths():
    """What a graph's call plans by is read anew at each replay (items cut or whole, other tiles, other pages)."""
    lens = [([1500, 40], [700, 40]), ([300, 300], [440, 300]), ([740, 1], [739, 1]), ([1500, 1500], [100, 640])]
    c = Call([1500, 1500], [740, 0], 8, seed=77)
    tokens, pt = 740, c.b.pt_host
    c.pages = 48
    c.ws = torch.zeros(dsa.expanded_attn_workspace_size(c.dims, c.pages), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.run()
    for seq, q in lens * 2:
        q = [q[0], tokens - q[0]] if q[0] + q[1] > tokens else q
        seq = [max(a, b) for a, b in zip(seq, q)]
        b = Batch(seq, q, seed=78)
        b.pt_host = pt
        c.b.lens.copy_(b.lens)
        c.b.cu.copy_(torch.tensor([0, q[0], q[0] + q[1]], dtype=torch.int32))
        c.out.fill_(7)
        c.lse.fill_(7)
        graph.replay()
        owned = q[0] + q[1]
        assert dsa.get_device_error(c.ws) == (0 if owned == tokens else dsa.DSA_DEVERR_SEQ)
        dsa.clear_device_error(c.ws)
        ref = Expanded(b, c.q_nope[:owned], c.q_pe[:owned], c.w, c.kv, False)
        ref.check(c.out[:owned], c.lse[:owned])
        assert bool((c.out[owned:] == 7).all())


@pytest.mark.parametrize("std", [8.0, 0.01])
def test_sharp_and_flat_weights(std):
    """Scores of a few hundred (one weight next to 1, the maximum rises again and again), and of next to nothing."""
    Call([700], [400], 4, seed=81, std=std).run().check(norm=False)


def test_rising_scores():
    """Every tile's scores beyond the ones before, so that sums and outputs are rescaled each time; then falling ones."""
    for order in (1, -1):
        c = Call([1300], [300], 2, seed=91)
        flat = c.kv.flatten(0, 1)
        at = torch.arange(1300)
        row = (c.b.pt_host[0, at // PAGE].long() * PAGE + at % PAGE).cuda()
        lift = torch.arange(1300, device="cuda").double() / 10
        if order < 0:
            lift = lift.flip(0)
        flat[row, LATENT] = lift.to(torch.bfloat16)
        c.q_pe[..., 0] = 8.0
        c.run().check(norm=False)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_hidden_rows_hold_anything(fp8, bad):
    """Rows behind a sequence's last position, in its last page, and pages of no sequence."""
    c = Call([130, 70], [100, 70], 4, fp8, seed=101)
    mine = torch.zeros(c.b.pages * PAGE, dtype=torch.bool, device="cuda")
    for b in range(2):
        at = torch.arange(c.b.L[b])
        mine[(c.b.pt_host[b, at // PAGE].long() * PAGE + at % PAGE).cuda()] = True
    if fp8:
        rows = c.kv.flatten(0, 1)
        rows[~mine] = 0x7F
    else:
        c.kv.flatten(0, 1)[~mine] = bad
    c.run()
    assert dsa.get_device_error(c.ws) == 0
    clean = Call([130, 70], [100, 70], 4, fp8, seed=101)
    clean.run().check()
    assert torch.equal(c.out, clean.out) and torch.equal(c.lse, clean.lse)


@pytest.mark.parametrize("place", [0, 300, 511, LATENT, KV - 1])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_a_row_that_is_not_finite(place, bad):
    """Queries before its position do not see it: bit for bit what they were.  Those from it on are NaN, or, of an infinite
    rotary value, what the formula says: NaN where the score is +inf, without the position where it is -inf."""
    seq, q, at = [300], [260], 180
    clean = Call(seq, q, 3, seed=111).run()
    clean.check()
    c = Call(seq, q, 3, seed=111)
    c.kv[int(c.b.pt_host[0, at // PAGE]), at % PAGE, place] = bad
    c.run()
    assert dsa.get_device_error(c.ws) == 0
    pos = torch.tensor(c.b.pos, device="cuda")
    assert torch.equal(c.out[pos < at], clean.out[pos < at]) and torch.equal(c.lse[pos < at], clean.lse[pos < at])
    after = pos >= at
    if place < LATENT or math.isnan(bad):
        assert bool(c.out[after].isnan().all() and c.lse[after].isnan().all())
        return
    sign = c.q_pe[after, :, place - LATENT].float() * (1 if bad > 0 else -1)
    assert bool(c.out[after][sign > 0].isnan().all() and c.out[after][sign < 0].isfinite().all())
    # with a large number in its place the weight is exactly 0 where the score is below -1000
    c.kv[c.kv == bad] = 3e4 if bad > 0 else -3e4
    ref = Expanded(c.b, c.q_nope, c.q_pe, c.w, c.kv, False)
    far = sign < -0.5
    err = (c.out[after][far].double() - ref.out[after][far]).norm()
    assert err <= 3.3e-3 * ref.out[after][far].norm()
    assert bool(((c.lse[after][far].double() - ref.lse[after][far]).abs() <= 0.05).all())


def test_fp8_rows_and_weights_beyond_range_are_reported():
    """An FP8 row's element, or a weight, beyond f16's range is reported and NaN for those who see it; a scale of infinity or
    NaN is no finite value beyond range: NaN, and no report."""
    clean = Call([300], [260], 2, True, seed=116).run()
    clean.check()
    pos = torch.tensor(clean.b.pos, device="cuda")
    at = 180
    page, place = int(clean.b.pt_host[0, at // PAGE]), at % PAGE
    for scale, error in ((100.0, dsa.DSA_DEVERR_RANGE), (float("inf"), 0), (float("nan"), 0)):
        c = Call([300], [260], 2, True, seed=116)
        c.kv[page, place, :128] = 0x7E  # 448
        c.kv[page, place, LATENT:LATENT + 4].view(torch.float32)[0] = scale
        c.run()
        assert dsa.get_device_error(c.ws) == error
        assert torch.equal(c.out[pos < at], clean.out[pos < at])
        assert bool(c.out[pos >= at].isnan().all() and c.lse[pos >= at].isnan().all())
    c = Call([300], [260], 2, True, seed=116)
    c.w[1, NOPE + 5, 9] = 5000.0
    c.run()
    assert dsa.get_device_error(c.ws) == dsa.DSA_DEVERR_RANGE and bool(c.out[:, 1].isnan().all())


@pytest.mark.parametrize("fp8", [False, True])
def test_values_beyond_range_are_reported(fp8):
    """Head values beyond f16's range: reported, NaN for those who see them; the largest ones within it are exact enough."""
    clean = Call([300], [260], 2, fp8, seed=115).run()
    for size, fits in ((3.0e4, False), (1.2e4, True)):
        c = Call([300], [260], 2, fp8, seed=115)
        at = 180
        page, place = int(c.b.pt_host[0, at // PAGE]), at % PAGE
        row = torch.zeros(1, KV, dtype=torch.bfloat16, device="cuda")
        row[0, 7] = size  # its head values are size times a column of the weights; those of one dim are made 1
        c.w[:, NOPE:, 7] = 0
        c.w[1, NOPE + 3, 7] = 1.0
        c.w[:, :NOPE, 7] = 0
        c.kv[page, place] = latent_fp8_rows(row)[0] if fp8 else row[0]
        clean.w.copy_(c.w)
        clean.run()
        c.run()
        pos = torch.tensor(c.b.pos, device="cuda")
        before, after = pos < at, pos >= at
        assert torch.equal(c.out[before], clean.out[before])
        if fits:
            c.check(norm=False)
        else:
            assert dsa.get_device_error(c.ws) == dsa.DSA_DEVERR_RANGE
            assert bool(c.out[after].isnan().all())


def test_queries_that_are_not_finite():
    clean = Call([300], [200], 3, seed=121).run()
    c = Call([300], [200], 3, seed=121)
    c.q_nope[5, 1, 3] = float("nan")
    c.q_pe[150, 2, 60] = float("inf")
    c.run()
    hit = torch.zeros((200, 3), dtype=torch.bool, device="cuda")
    hit[5, 1] = hit[150, 2] = True
    assert torch.equal(c.out[~hit], clean.out[~hit]) and torch.equal(c.lse[~hit], clean.lse[~hit])
    assert bool(c.out[hit].isnan().all() and c.lse[hit].isnan().all())


def test_every_score_minus_infinity():
    """One dim of every key's rotary part at -inf, the queries' positive there: nothing has a weight."""
    c = Call([200], [150], 2, seed=131)
    c.kv[:, :, KV - 1] = -float("inf")
    c.q_pe[..., ROT - 1] = 1.0
    c.run()
    assert dsa.get_device_error(c.ws) == 0
    assert bool((c.out == 0).all() and (c.lse == -math.inf).all())


def test_bad_pages_are_reported_and_seen_as_nan():
    for bad in (-1, 10 ** 6):
        c = Call([400, 200], [350, 200], 3, seed=141)
        clean = Call([400, 200], [350, 200], 3, seed=141).run()
        c.b.pt[0, 4] = bad
        c.run()
        assert dsa.get_device_error(c.ws) == dsa.DSA_DEVERR_PAGE
        pos, seq = torch.tensor(c.b.pos, device="cuda"), torch.tensor(c.b.seq, device="cuda")
        hit = (seq == 0) & (pos >= 4 * PAGE)
        assert torch.equal(c.out[~hit], clean.out[~hit]) and torch.equal(c.lse[~hit], clean.lse[~hit])
        assert bool(c.out[hit].isnan().all() and c.lse[hit].isnan().all())


def test_entries_of_no_position_are_not_read():
    c = Call([130, 200], [100, 200], 2, seed=151)
    c.b.pt = torch.cat([c.b.pt, torch.full((2, 3), 10 ** 8, dtype=torch.int32, device="cuda")], dim=1)
    c.dims.max_pages_per_seq = c.b.pt.shape[1]
    c.run().check()


def test_inconsistent_sequences_are_left_alone():
    def reported(change, tokens_left):
        c = Call([100, 300, 64, 90], [10, 20, 30, 40], 2, seed=161)
        clean = Call([100, 300, 64, 90], [10, 20, 30, 40], 2, seed=161).run()
        change(c)
        c.run()
        assert dsa.get_device_error(c.ws) == dsa.DSA_DEVERR_SEQ
        left = torch.zeros(100, dtype=torch.bool, device="cuda")
        left[tokens_left] = True
        assert bool((c.out[left] == 7).all() and (c.lse[left] == 7).all())
        assert torch.equal(c.out[~left], clean.out[~left]) and torch.equal(c.lse[~left], clean.lse[~left])

    def length(b, value):
        return lambda c: c.b.lens.__setitem__(b, value)

    reported(length(1, 19), slice(10, 30))  # more queries than positions
    reported(length(1, -5), slice(10, 30))
    reported(length(1, 10 ** 6), slice(10, 30))  # beyond the page table
    reported(length(3, 2 ** 31 - 1), slice(60, 100))


def test_tokens_that_no_sequence_owns():
    c = Call([100, 300, 64, 90], [10, 20, 30, 40], 2, seed=162)
    c.b.cu[4] = 95
    c.run()
    assert dsa.get_device_error(c.ws) == dsa.DSA_DEVERR_SEQ
    assert bool((c.out[95:] == 7).all() and (c.lse[95:] == 7).all())
    short = Call([100, 300, 64, 90], [10, 20, 30, 35], 2, seed=162)
    short.q_nope.copy_(c.q_nope[:95])
    short.q_pe.copy_(c.q_pe[:95])
    short.run().check()
    assert torch.equal(c.out[:95], short.out) and torch.equal(c.lse[:95], short.lse)


def test_fewer_pages_announced():
    """Sequences whose pages do not fit the workspace are reported and left alone; those in front of them are done."""
    c = Call([1000, 2000, 100], [100, 100, 100], 2, seed=171)
    c.pages = 16
    c.run()
    assert dsa.get_device_error(c.ws) == dsa.DSA_DEVERR_SEQ
    clean = Call([1000, 2000, 100], [100, 100, 100], 2, seed=171).run()
    assert torch.equal(c.out[:100], clean.out[:100]) and bool((c.out[100:200] == 7).all())


def test_offsets_that_run_backwards():
    c = Call([200, 200, 200], [100, 0, 100], 2, seed=181)
    c.b.cu.copy_(torch.tensor([0, 200, 0, 200], dtype=torch.int32))
    c.run()  # the first and the last claim all tokens, the second is none
    assert dsa.get_device_error(c.ws) & dsa.DSA_DEVERR_SEQ


def test_short_waits_are_reported():
    c = Call([900, 500], [700, 300], 16, seed=191)
    old = dsa.set_wait_limit_ns(200)
    try:
        c.run()
        torch.cuda.synchronize()
    finally:
        dsa.set_wait_limit_ns(old)
    assert dsa.get_device_error(c.ws) & dsa.DSA_DEVERR_TIMEOUT
    dsa.clear_device_error(c.ws)
    c.run().check()


@pytest.mark.parametrize("fp8", [False, True])
def test_a_layer_in_both_forms(fp8):
    """From a layer's input to its head values: norm, projections, the latent rows' norm and their rotation into the cache,
    then the queries in absorbed form (absorb, rotate, dense attention over latent rows, value heads) and in expanded form,
    whose results are those of one formula."""
    heads, hidden, seq, q = 8, 1024, [333, 128, 40], [200, 128, 1]
    b = Batch(seq, q, seed=3)
    T = b.T
    x, res, w_in = normal((T, hidden), 201), normal((T, hidden), 202, 3.0), (1 + normal((hidden,), 203, 0.1)).to(torch.bfloat16)
    proj_q, proj_kv = normal((heads * (NOPE + ROT), hidden), 204, hidden ** -0.5), normal((KV, hidden), 205, hidden ** -0.5)
    w_latent, w_kv = (1 + normal((LATENT,), 206, 0.1)).to(torch.bfloat16), weights(heads, 207)
    table = rope_table(400, "cuda")
    rope = dsa.DsaRope(table=table.data_ptr(), table_len=400, kv_pairing=dsa.DSA_ROPE_INTERLEAVED,
                       idx_pairing=dsa.DSA_ROPE_HALVES, idx_begin=-1)
    cache = normal((b.pages * PAGE, KV), 208)
    cache = (latent_fp8_rows(cache) if fp8 else cache).view(b.pages, PAGE, -1)
    dims = b.dims(attn_heads=heads, kv_dtype=dsa.DSA_FP8_E4M3 if fp8 else dsa.DSA_BF16, softmax_scale=SCALE)
    ws = b.workspace

    normed, total = torch.empty_like(x), torch.empty_like(x)
    dsa.rms_norm(x, w_in, 1e-6, out=normed, residual=res, sum=total)
    check_bf16(normed, norm64(x, w_in, 1e-6, res)[1])
    q_proj = (normed @ proj_q.T).view(T, heads, NOPE + ROT)
    kv_new = normed @ proj_kv.T
    latent = kv_new[:, :LATENT]
    want = norm64(latent, w_latent, 1e-6)[1]
    dsa.rms_norm(latent, w_latent, 1e-6, out=latent)  # in place, in front of the rotary part
    check_bf16(kv_new[:, :LATENT], want)
    dsa.rope_append(dims, rope, None, kv_new, b.pt, b.lens, b.cu, None, None, cache, ws)
    queries = torch.zeros((T, heads, KV), dtype=torch.bfloat16, device="cuda")
    strides = q_proj.stride()[:2]
    dsa.rope_queries(dims, rope, q_proj[..., NOPE:], queries, None, None, None, b.lens, b.cu, ws, q_pe_strides=strides)

    dsa.absorb_queries(dims, q_proj, w_kv, queries, ws, q_nope_strides=strides)
    latent_out = torch.zeros((T, heads, LATENT), dtype=torch.bfloat16, device="cuda")
    lse = torch.zeros((T, heads), device="cuda")
    ws_prefix = torch.zeros(dsa.prefix_attn_workspace_size(dims, 0), dtype=torch.uint8, device="cuda")
    dsa.prefix_attn(dims, 0, queries, cache, b.pt, b.lens, b.cu, latent_out, lse, ws_prefix)
    absorbed = torch.zeros((T, heads, VALUE), dtype=torch.bfloat16, device="cuda")
    dsa.value_heads(dims, latent_out, w_kv, absorbed, ws)

    pages = sum(-(-l // PAGE) for l in seq)
    ws_expanded = torch.zeros(dsa.expanded_attn_workspace_size(dims, pages), dtype=torch.uint8, device="cuda")
    expanded, lse2 = torch.zeros_like(absorbed), torch.zeros_like(lse)
    dsa.expanded_attn(dims, pages, q_proj, queries[..., LATENT:], w_kv, cache, b.pt, b.lens, b.cu, expanded, lse2, ws_expanded,
                      q_nope_strides=strides, q_pe_strides=queries.stride()[:2])
    for w in (ws, ws_prefix, ws_expanded):
        assert dsa.get_device_error(w) == 0
    ref = Expanded(b, q_proj[..., :NOPE], queries[..., LATENT:], w_kv, cache, fp8)
    ref.check(expanded, lse2)
    # the absorbed form rounds to bf16 (0.0017 each): q, and so its scores, weights, its output and the values
    assert (absorbed.double() - ref.out).norm() <= 5e-3 * ref.out.norm()
    assert (lse.double() - ref.lse).abs().max() <= ref.dz.max() + 2.0 ** -8 * 8
