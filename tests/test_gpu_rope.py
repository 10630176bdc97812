"""Rotating append and query rotation on the GPU against 64-bit forms.

Tolerances: a rotated value is two products and a sum in fp32, each within 2^-24 of the magnitudes, then one
rounding to the stored type (bf16 2^-8 relative, E4M3 2^-4 relative or half of its smallest step 2^-9); an fp32
scale is one division, within 2^-24 of a maximum that is itself within 3 * 2^-24.
"""
import math

import pytest
import torch

import sparse_attention_dsa_gb300 as dsa

from _gpu import ensure_built
from _rope_prefix import KV, LATENT, PAGE, Batch, latent_values, rope_table, rotate

pytestmark = pytest.mark.gpu

BF16, FP8, MX = dsa.DSA_BF16, dsa.DSA_FP8_E4M3, dsa.DSA_MXFP8_E4M3


@pytest.fixture(scope="module", autouse=True)
def _built():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    ensure_built()


def _normal(shape, seed, spread=True):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(shape, generator=g, device="cuda")
    if spread and shape[0]:
        x = x * 2.0 ** torch.randint(-6, 7, (shape[0],) + (1,) * (len(shape) - 1), generator=g, device="cuda")
    return x.to(torch.bfloat16)


def _rope(table, kv=dsa.DSA_ROPE_INTERLEAVED, idx=dsa.DSA_ROPE_HALVES, begin=0):
    return dsa.DsaRope(table=table.data_ptr(), table_len=table.shape[0], kv_pairing=kv, idx_pairing=idx, idx_begin=begin)


def _turn_index(x, rows, pairing, begin):
    y = x.double()
    if begin >= 0:
        y[..., begin:begin + 64] = rotate(y[..., begin:begin + 64].clone(), rows, pairing == dsa.DSA_ROPE_INTERLEAVED)
    return y


def _size(x):
    """Magnitude whose 2^-22 covers the fp32 roundings of a rotated value: the row's largest."""
    return x.double().abs().amax(-1, keepdim=True)


def _check_bf16(got, want, size):
    err = (got.double() - want).abs()
    tol = 2.0 ** -8 * want.abs() + 2.0 ** -22 * size + 1e-38
    assert bool((err <= tol).all()), f"worst {(err / tol).max().item():.3g} of the bound"


def _check_codes(codes, scale, want):
    """codes (bytes) * scale (float64, broadcastable) against values."""
    got = codes.view(torch.float8_e4m3fn).double() * scale
    tol = torch.maximum(2.0 ** -4 * want.abs(), 2.0 ** -10 * scale) * (1 + 2.0 ** -18) + 1e-38
    err = (got - want).abs()
    assert bool((err <= tol).all()), f"worst {(err / tol).max().item():.3g} of the bound"


def _check_index(codes, scale, want, kind, size):
    """Rows [..., Di] of an indexer array as they are stored, against 64-bit values."""
    if kind == BF16:
        _check_bf16(codes, want, size)
        return
    if kind == FP8:
        m = want.abs().amax(-1)
        exact = torch.where(m > 0, m / 448, torch.ones_like(m))
        assert bool(((scale.double() - exact).abs() <= 2.0 ** -21 * exact + 2.0 ** -149).all())
        _check_codes(codes, scale.double()[..., None], want)
        return
    g = want.reshape(*want.shape[:-1], -1, 32)
    m = g.abs().amax(-1)
    e = torch.where(m > 0, torch.frexp(m).exponent - 9, torch.zeros_like(m, dtype=torch.int32)).clamp(-127, 127)
    step = scale.int() - 127 - e
    near = (m > 0) & ((torch.frexp(m).mantissa - 0.5 < 2.0 ** -20) | (1 - torch.frexp(m).mantissa < 2.0 ** -20))
    assert bool(((step == 0) | (near & (step.abs() == 1))).all())
    value = torch.exp2(scale.double() - 127)[..., None]
    got = codes.view(torch.float8_e4m3fn).double().reshape(g.shape) * value
    # above 448 / 512 of the binade the code saturates: at most 448 / 512 of the largest value below it
    tol = torch.maximum(2.0 ** -4 * g.abs(), 2.0 ** -10 * value) * (1 + 2.0 ** -18)
    tol = torch.where(g.abs() > 448 * value, g.abs() - 448 * value + 2.0 ** -18 * g.abs(), tol)
    assert bool(((got - g).abs() <= tol + 1e-38).all())


RAGGED = dict(seq_lens=[300, 129, 64, 1, 2000, 65, 5], q_lens=[1, 3, 2, 1, 4, 65, 0])
CASES = [
    # idx dtype, kv dtype, Di, idx_begin, kv pairing, idx pairing, strided
    (BF16, BF16, 128, 0, 1, 0, False),
    (FP8, FP8, 128, 64, 0, 1, True),
    (MX, FP8, 128, 0, 1, 0, False),
    (MX, BF16, 128, 32, 0, 1, True),
    (BF16, FP8, 64, 0, 1, 1, False),
    (FP8, BF16, 96, 8, 0, 0, True),
    (FP8, FP8, 8, -1, 1, 0, False),
    (MX, FP8, 96, 32, 1, 1, False),
    (BF16, BF16, 72, 8, 0, 1, True),
    (MX, FP8, 32, -1, 0, 0, True),
]


def _caches(b, idx, kv, di, fill=0x5A):
    k = torch.full((b.pages, PAGE, di * (2 if idx == BF16 else 1)), fill, dtype=torch.uint8, device="cuda")
    ks = (None if idx == BF16 else torch.full((b.pages, PAGE), 7.0, device="cuda") if idx == FP8 else
          torch.full((b.pages, PAGE, di // 32), fill, dtype=torch.uint8, device="cuda"))
    kvc = torch.full((b.pages, PAGE, 656 if kv == FP8 else 1152), fill, dtype=torch.uint8, device="cuda")
    return k, ks, kvc


@pytest.mark.parametrize("idx,kv,di,begin,pair_kv,pair_idx,strided", CASES)
def test_append(idx, kv, di, begin, pair_kv, pair_idx, strided):
    b = Batch(**RAGGED, seed=3)
    table = rope_table(2000, "cuda")
    k_new, kv_new = _normal((b.T, di), 11), _normal((b.T, KV), 12)
    k_new[0] = 0
    kv_new[1, 128:256] = 0
    k_in, kv_in = k_new, kv_new
    if strided:
        k_in = torch.cat([k_new, _normal((b.T, 24), 13)], dim=1)[:, :di]
        kv_in = torch.cat([kv_new, _normal((b.T, 136), 14)], dim=1)[:, :KV]
    k, ks, kvc = _caches(b, idx, kv, di)
    before = [None if c is None else c.clone() for c in (k, ks, kvc)]
    dsa.rope_append(b.dims(idx_dim=di, idx_dtype=idx, kv_dtype=kv), _rope(table, pair_kv, pair_idx, begin), k_in, kv_in,
                    b.pt, b.lens, b.cu, k, ks, kvc, b.workspace, k_stride=k_in.stride(0), kv_stride=kv_in.stride(0))
    assert dsa.get_device_error(b.workspace) == 0
    rows = table[torch.tensor(b.pos, device="cuda")]
    want = _turn_index(k_new, rows, pair_idx, begin)
    got = k.flatten(0, 1)[b.rows]
    _check_index(got.view(torch.bfloat16) if idx == BF16 else got, None if ks is None else ks.flatten(0, 1)[b.rows], want,
                 idx, _size(k_new))
    got = kvc.flatten(0, 1)[b.rows]
    rot = rotate(kv_new[:, LATENT:].double(), rows, pair_kv == dsa.DSA_ROPE_INTERLEAVED)
    if kv == BF16:
        got = got.view(torch.bfloat16)
        assert torch.equal(got[:, :LATENT], kv_new[:, :LATENT])
        _check_bf16(got[:, LATENT:], rot, _size(kv_new[:, LATENT:]))
    else:
        scale = got[:, LATENT:LATENT + 16].contiguous().view(torch.float32)
        tiles = kv_new[:, :LATENT].reshape(-1, 4, 128)
        _check_index(got[:, :LATENT].contiguous().reshape(-1, 4, 128), scale, tiles.double(), FP8, None)
        _check_bf16(got[:, LATENT + 16:].contiguous().view(torch.bfloat16), rot, _size(kv_new[:, LATENT:]))
    # every other row is as it was
    for cache, old in zip((k, ks, kvc), before):
        if cache is not None:
            cache.flatten(0, 1)[b.rows] = old.flatten(0, 1)[b.rows]
            assert torch.equal(cache, old)


@pytest.mark.parametrize("idx,kv", [(BF16, BF16), (FP8, FP8)])
def test_without_a_rotation_it_is_the_plain_append(idx, kv):
    b = Batch(**RAGGED, seed=4)
    table = torch.cat([torch.ones(2000, 32), torch.zeros(2000, 32)], dim=1).cuda()
    k_new, kv_new = _normal((b.T, 128), 21), _normal((b.T, KV), 22)
    d = b.dims(idx_dtype=idx, kv_dtype=kv)
    a, c = _caches(b, idx, kv, 128), _caches(b, idx, kv, 128)
    dsa.append_rows(d, k_new, kv_new, b.pt, b.lens, b.cu, a[0], a[1], a[2], b.workspace)
    dsa.rope_append(d, _rope(table), k_new, kv_new, b.pt, b.lens, b.cu, c[0], c[1], c[2], b.workspace)
    assert dsa.get_device_error(b.workspace) == 0
    for x, y in zip(a, c):
        assert x is None or torch.equal(x, y)


def test_quantised_rows_of_every_magnitude_are_the_plain_append_s():
    """Codes and scales are those of correctly rounded divisions, at magnitudes from subnormal to the largest, with
    zeros of both signs, infinities and NaN: byte for byte what the plain append makes."""
    b = Batch([4000], [4000], seed=16)
    kv_new, k_new = _normal((b.T, KV), 93).float(), _normal((b.T, 128), 94).float()
    power = torch.randint(-133, 125, (b.T, 1), generator=torch.Generator().manual_seed(95)).cuda().float()
    power[:2000] = power[:2000] / 16
    kv_new, k_new = kv_new * torch.exp2(power), k_new * torch.exp2(power)
    for x in (kv_new, k_new):
        x[:, 5::64] = 0.0
        x[:, 7::64] = -0.0
        x[100:110, 9] = math.inf
        x[105:115, 300 % x.shape[1]] = math.nan
    kv_new[:, LATENT:] = 0.0
    kv_new, k_new = kv_new.to(torch.bfloat16), k_new.to(torch.bfloat16)
    d = b.dims(idx_dim=128, idx_dtype=FP8, kv_dtype=FP8)
    got, want = _caches(b, FP8, FP8, 128), _caches(b, FP8, FP8, 128)
    dsa.rope_append(d, _rope(rope_table(4000, "cuda"), 0, 0, -1), k_new, kv_new, b.pt, b.lens, b.cu, *got, b.workspace)
    dsa.append_rows(d, k_new, kv_new, b.pt, b.lens, b.cu, *want, b.workspace)
    assert dsa.get_device_error(b.workspace) == 0
    assert torch.equal(got[0], want[0])
    assert torch.equal(got[1].view(torch.int32), want[1].view(torch.int32))
    # (the rotary part, zeros, is left out: rotated by a negative cosine, 0 is -0)
    assert torch.equal(got[2][..., :528], want[2][..., :528])


@pytest.mark.parametrize("which", ["k", "kv"])
def test_append_of_one_cache_alone(which):
    b = Batch(**RAGGED, seed=5)
    table = rope_table(2000, "cuda")
    k, ks, kvc = _caches(b, BF16, BF16, 128)
    old_k, old_kv = k.clone(), kvc.clone()
    dsa.rope_append(b.dims(), _rope(table), _normal((b.T, 128), 1) if which == "k" else None,
                    _normal((b.T, KV), 2) if which == "kv" else None, b.pt, b.lens, b.cu, k if which == "k" else None,
                    None, kvc if which == "kv" else None, b.workspace)
    assert dsa.get_device_error(b.workspace) == 0
    assert torch.equal(k, old_k) == (which == "kv") and torch.equal(kvc, old_kv) == (which == "k")


def test_append_many_sequences_and_a_long_step():
    """More sequences than a warp looks at in one go, and thousands of tokens."""
    for lens, qs in (([70 + i % 5 for i in range(200)], [1] * 200), ([5000], [4999])):
        b = Batch(lens, qs, seed=6)
        table = rope_table(5000, "cuda")
        kv_new = _normal((b.T, KV), 31)
        k, ks, kvc = _caches(b, BF16, BF16, 128)
        dsa.rope_append(b.dims(), _rope(table), None, kv_new, b.pt, b.lens, b.cu, None, None, kvc, b.workspace)
        assert dsa.get_device_error(b.workspace) == 0
        got = kvc.flatten(0, 1)[b.rows].view(torch.bfloat16)
        rot = rotate(kv_new[:, LATENT:].double(), table[torch.tensor(b.pos, device="cuda")], True)
        assert torch.equal(got[:, :LATENT], kv_new[:, :LATENT])
        _check_bf16(got[:, LATENT:], rot, _size(kv_new[:, LATENT:]))


def test_append_behind_four_gigabytes():
    """Rows whose byte offset needs more than 32 bits."""
    b = Batch([64], [64], seed=7)
    pages = 70000
    b.pt[0, 0] = pages - 1
    kvc = torch.zeros((pages, PAGE, KV), dtype=torch.bfloat16, device="cuda")
    kv_new = _normal((64, KV), 41)
    table = rope_table(64, "cuda")
    dsa.rope_append(b.dims(num_pages=pages), _rope(table), None, kv_new, b.pt, b.lens, b.cu, None, None, kvc, b.workspace)
    assert dsa.get_device_error(b.workspace) == 0
    assert torch.equal(kvc[pages - 1, :, :LATENT], kv_new[:, :LATENT])
    assert not bool(kvc[:pages - 1].any())


def test_append_reports_and_skips_what_it_cannot_place():
    b = Batch([300, 129, 70, 700], [1, 1, 1, 1], seed=8)
    kv_new = _normal((6, KV), 51)  # tokens 4 and 5 belong to no sequence
    table = rope_table(600, "cuda")  # sequence 3's position 699 has no angles
    b.pt[1, 2] = b.pages + 3
    b.lens[2] = 0  # one query token, but no cached position
    kvc = _caches(b, BF16, BF16, 128)[2]
    old = kvc.clone()
    d = b.dims(total_q=6)
    dsa.rope_append(d, _rope(table), None, kv_new, b.pt, b.lens, b.cu, None, None, kvc, b.workspace)
    assert dsa.get_device_error(b.workspace) == dsa.DSA_DEVERR_PAGE | dsa.DSA_DEVERR_SEQ | dsa.DSA_DEVERR_ROPE
    changed = (kvc != old).flatten(0, 1).any(dim=1).nonzero().flatten().tolist()
    assert changed == [int(b.rows[0])]


QUERIES = [
    # idx dtype, Hq, Hi, Di, idx_begin, pairings (kv, idx)
    (BF16, 128, 64, 128, 0, 1, 0),
    (FP8, 128, 64, 128, 64, 0, 1),
    (MX, 16, 64, 128, 0, 1, 0),
    (BF16, 7, 4, 64, 0, 0, 1),
    (FP8, 1, 1, 96, 8, 1, 1),
    (MX, 33, 3, 32, -1, 0, 0),
    (FP8, 128, 128, 72, 8, 1, 0),
]


@pytest.mark.parametrize("idx,hq,hi,di,begin,pair_kv,pair_idx", QUERIES)
@pytest.mark.parametrize("strided", [False, True])
def test_queries(idx, hq, hi, di, begin, pair_kv, pair_idx, strided):
    b = Batch(**RAGGED, seed=9)
    table = rope_table(2000, "cuda")
    rows = table[torch.tensor(b.pos, device="cuda")]
    q_pe, x = _normal((b.T, hq, 64), 61), _normal((b.T, hi, di), 62)
    x[0, 0] = 0
    pe_in, x_in = q_pe, x.reshape(b.T, hi * di)
    strides, x_stride = (0, 0), 0
    if strided:
        pe_in = torch.cat([_normal((b.T, hq, 128), 63), q_pe], dim=2)[:, :, 128:]
        x_in = torch.cat([x_in, _normal((b.T, 40), 64)], dim=1)
        strides, x_stride = (pe_in.stride(0), pe_in.stride(1)), x_in.stride(0)
    q = _normal((b.T, hq, KV), 65)
    old = q.clone()
    out = torch.zeros((b.T, hi, di), dtype=torch.bfloat16 if idx == BF16 else torch.uint8, device="cuda")
    scale = {BF16: None, FP8: torch.zeros((b.T, hi), device="cuda"),
             MX: torch.zeros((b.T, hi, max(di // 32, 1)), dtype=torch.uint8, device="cuda")}[idx]
    dsa.rope_queries(b.dims(attn_heads=hq, idx_heads=hi, idx_dim=di, idx_dtype=idx), _rope(table, pair_kv, pair_idx, begin),
                     pe_in, q, x_in, out, scale, b.lens, b.cu, b.workspace, q_pe_strides=strides, q_idx_stride=x_stride)
    assert dsa.get_device_error(b.workspace) == 0
    assert torch.equal(q[:, :, :LATENT], old[:, :, :LATENT])
    _check_bf16(q[:, :, LATENT:], rotate(q_pe.double(), rows, pair_kv == dsa.DSA_ROPE_INTERLEAVED), _size(q_pe))
    _check_index(out, scale, _turn_index(x, rows, pair_idx, begin), idx, _size(x))


def test_queries_in_place():
    b = Batch(**RAGGED, seed=10)
    table = rope_table(2000, "cuda")
    rows = table[torch.tensor(b.pos, device="cuda")]
    q, x = _normal((b.T, 128, KV), 71), _normal((b.T, 64, 128), 72)
    old_q, old_x = q.clone(), x.clone()
    dsa.rope_queries(b.dims(), _rope(table), q.data_ptr() + 2 * LATENT, q, x, x, None, b.lens, b.cu, b.workspace,
                     q_pe_strides=(128 * KV, KV))
    assert dsa.get_device_error(b.workspace) == 0
    assert torch.equal(q[:, :, :LATENT], old_q[:, :, :LATENT])
    _check_bf16(q[:, :, LATENT:], rotate(old_q[:, :, LATENT:].double(), rows, True), _size(old_q[:, :, LATENT:]))
    _check_bf16(x, _turn_index(old_x, rows, 0, 0), _size(old_x))


def test_queries_report_and_skip():
    b = Batch([300, 129], [1, 1], seed=11)
    table = rope_table(200, "cuda")
    q, q_pe = torch.zeros((3, 128, KV), dtype=torch.bfloat16, device="cuda"), _normal((3, 128, 64), 81)
    dsa.rope_queries(b.dims(total_q=3), _rope(table), q_pe, q, None, None, None, b.lens, b.cu, b.workspace)
    assert dsa.get_device_error(b.workspace) == dsa.DSA_DEVERR_ROPE | dsa.DSA_DEVERR_SEQ
    assert not bool(q[0].any()) and not bool(q[2].any()) and bool(q[1].any())


def test_offsets_out_of_range_are_reported():
    """Offsets whose difference passes 32 bits own no token."""
    b = Batch([300], [1], seed=12)
    b.cu.copy_(torch.tensor([-2_000_000_000, 1_000_000_000], dtype=torch.int32))
    table = rope_table(400, "cuda")
    kvc = _caches(b, BF16, BF16, 128)[2]
    old = kvc.clone()
    dsa.rope_append(b.dims(), _rope(table), None, _normal((1, KV), 91), b.pt, b.lens, b.cu, None, None, kvc, b.workspace)
    assert dsa.get_device_error(b.workspace) == dsa.DSA_DEVERR_SEQ and torch.equal(kvc, old)
    dsa.clear_device_error(b.workspace)
    q = torch.zeros((1, 128, KV), dtype=torch.bfloat16, device="cuda")
    dsa.rope_queries(b.dims(), _rope(table), _normal((1, 128, 64), 92), q, None, None, None, b.lens, b.cu, b.workspace)
    assert dsa.get_device_error(b.workspace) == dsa.DSA_DEVERR_SEQ and not bool(q.any())


def test_infinities_and_nan_stay_in_their_groups():
    """A row with an infinity or a NaN leaves other rows and, in the latent part, other tiles as they would be."""
    b = Batch([10, 20], [2, 2], seed=12)
    table = rope_table(64, "cuda")
    kv_new, k_new = _normal((4, KV), 91, spread=False), _normal((4, 128), 92, spread=False)
    clean = _caches(b, FP8, FP8, 128)
    d = b.dims(idx_dtype=FP8, kv_dtype=FP8)
    dsa.rope_append(d, _rope(table), k_new, kv_new, b.pt, b.lens, b.cu, *clean, b.workspace)
    kv_new[1, 130], kv_new[2, 520], k_new[3, 100] = float("inf"), float("nan"), float("nan")
    got = _caches(b, FP8, FP8, 128)
    dsa.rope_append(d, _rope(table), k_new, kv_new, b.pt, b.lens, b.cu, *got, b.workspace)
    assert dsa.get_device_error(b.workspace) == 0
    r = b.rows
    x, y = clean[2].flatten(0, 1)[r], got[2].flatten(0, 1)[r]
    assert torch.equal(x[0], y[0]) and torch.equal(x[3], y[3])
    assert torch.equal(x[1, :128], y[1, :128]) and torch.equal(x[1, 256:512], y[1, 256:512])
    assert torch.equal(x[2, :528], y[2, :528])
    assert latent_values(y[2:3], True)[0, 512:].isnan().any()
    assert torch.equal(clean[0].flatten(0, 1)[r[:3]], got[0].flatten(0, 1)[r[:3]])
    assert got[0].flatten(0, 1)[r[3]].view(torch.float8_e4m3fn).double()[100].isnan()


def test_streams_and_graphs():
    """The calls on a side stream and captured; a replay sees new inputs."""
    b = Batch([300, 129], [2, 1], seed=13)
    table = rope_table(512, "cuda")
    kv_new, q_pe = _normal((b.T, KV), 101), _normal((b.T, 128, 64), 102)
    kvc = torch.zeros((b.pages, PAGE, KV), dtype=torch.bfloat16, device="cuda")
    q = torch.zeros((b.T, 128, KV), dtype=torch.bfloat16, device="cuda")

    def step(stream=None):
        dsa.rope_append(b.dims(), _rope(table), None, kv_new, b.pt, b.lens, b.cu, None, None, kvc, b.workspace, stream)
        dsa.rope_queries(b.dims(), _rope(table), q_pe, q, None, None, None, b.lens, b.cu, b.workspace, stream)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    step(s)
    torch.cuda.synchronize()
    first = kvc.clone(), q.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    kvc.zero_(), q.zero_()
    g.replay()
    assert torch.equal(kvc, first[0]) and torch.equal(q, first[1])
    b.lens += 1  # the next step: the replay reads the new lengths
    kv_new.mul_(2)
    q.zero_()
    g.replay()
    assert dsa.get_device_error(b.workspace) == 0
    pos = torch.tensor(b.pos, device="cuda") + 1
    _check_bf16(q[:, :, LATENT:], rotate(q_pe.double(), table[pos], True), _size(q_pe))
    at = torch.tensor([int(b.pt_host[i, p // PAGE]) * PAGE + p % PAGE for i, p in zip(b.seq, pos.tolist())], device="cuda")
    assert torch.equal(kvc.flatten(0, 1)[at][:, :LATENT], kv_new[:, :LATENT])


def test_queries_take_no_limit_from_the_page_table():
    b = Batch([3000], [2], seed=14)
    table = rope_table(3000, "cuda")
    q, q_pe = torch.zeros((2, 128, KV), dtype=torch.bfloat16, device="cuda"), _normal((2, 128, 64), 111)
    dsa.rope_queries(b.dims(num_pages=1, max_pages_per_seq=1), _rope(table), q_pe, q, None, None, None, b.lens, b.cu,
                     b.workspace)
    assert dsa.get_device_error(b.workspace) == 0
    _check_bf16(q[:, :, LATENT:], rotate(q_pe.double(), table[torch.tensor(b.pos, device="cuda")], True), _size(q_pe))
