"""The range of shared-prefix attention over FP8 rows, whose products take f16 operands (rows times 4, q by 4): finite values
beyond it make the rows that see them NaN and are reported, whatever their signs and wherever the tiles fall; values
within it, and infinities, are what they are."""
import math

import pytest
import torch

import sparse_attention_dsa_gb300 as dsa

from _gpu import ensure_built
from _rope_prefix import KV, LATENT, PAGE, Attention
from test_gpu_prefix import SHAPES, Call

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    ensure_built()


def _row(c, b, pos):
    """The bytes of sequence b's row at a position."""
    src = 0 if pos < c.prefix else b
    return c.cache[int(c.b.pt_host[src, pos // PAGE]), pos % PAGE]


def _set_rotary(c, b, pos, dim, value):
    _row(c, b, pos)[LATENT + 16:].view(torch.bfloat16)[dim] = value


def _set_latent(c, b, pos, tile, scale, code=0x7E):
    row = _row(c, b, pos)
    row[128 * tile:128 * tile + 128] = code
    row[LATENT:LATENT + 16].view(torch.float32)[tile] = scale


BEYOND = {
    "rotary": lambda c, b, pos: _set_rotary(c, b, pos, 63, 16384.0),
    "negative rotary": lambda c, b, pos: _set_rotary(c, b, pos, 0, -3.0e38),
    "element": lambda c, b, pos: _set_latent(c, b, pos, 3, 36.7),  # 448 * 36.7 = 16442
    "negative element": lambda c, b, pos: _set_latent(c, b, pos, 0, 40.0, 0xFE),
    "negative scale": lambda c, b, pos: _set_latent(c, b, pos, 1, -40.0),
    "scale of zeros": lambda c, b, pos: _set_latent(c, b, pos, 2, 64.0, 0),
    "large scale": lambda c, b, pos: _set_latent(c, b, pos, 2, 1.0e30, 0x01),
}
# a context whose row at `pos` lies in a tile that every query sees whole, or in the last one; in the prefix (converted
# ahead, or in passing), or behind it
PLACES = {
    "own tile": (([700, 600], [3, 2], 100, 16), 0, 300),
    "last tile": (([700, 600], [3, 2], 100, 16), 1, 599),
    "no prefix": (([300, 200], [1, 1], 0, 128), 1, 5),
    "prefix": (([700, 600], [3, 2], 300, 16), 0, 20),
    "prefix's end": (([700, 600], [3, 2], 300, 128), 0, 299),
    "converted ahead": (SHAPES["full_heads_long_prefix"], 0, 1000),
    "packed, ahead": (SHAPES["packed_long_prefix"], 0, 2499),
}


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("place", list(PLACES))
@pytest.mark.parametrize("what", list(BEYOND))
def test_rows_beyond_the_range_are_reported_and_nan(what, place, sign, wide):
    shape, b, pos = PLACES[place]
    c = Call(*shape, fp8=True, seed=40, wide=wide)
    c.q.abs_().mul_(sign)  # (every product of the row has one sign)
    c.run()
    assert c.error() == 0
    want = c.out.clone(), c.lse.clone()
    BEYOND[what](c, b, pos)
    c.run()
    assert c.error() == dsa.DSA_DEVERR_RANGE
    seen = torch.tensor([(pos < c.prefix or s == b) and p >= pos for s, p in zip(c.b.seq, c.b.pos)])
    assert bool(seen.any())
    assert bool(c.out[seen].isnan().all()) and bool(c.lse[seen].isnan().all())
    assert torch.equal(c.out[~seen], want[0][~seen]) and torch.equal(c.lse[~seen], want[1][~seen])


@pytest.mark.parametrize("wide", [False, True])
def test_a_row_beyond_the_range_that_only_later_queries_see(wide):
    c = Call([205, 100], [5, 5], 90, 16, fp8=True, seed=41, wide=wide).run()
    want = c.out.clone()
    _set_rotary(c, 0, 203, 7, -20000.0)
    c.run()
    assert c.error() == dsa.DSA_DEVERR_RANGE
    assert bool(c.out[3:5].isnan().all())
    assert torch.equal(c.out[:3], want[:3]) and torch.equal(c.out[5:], want[5:])


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("value", [262144.0, -3.0e38])
def test_a_query_beyond_the_range_is_reported_and_stays_alone(value, wide):
    c = Call([205, 100, 170], [1, 1, 1], 90, 16, fp8=True, seed=42, wide=wide).run()
    want = c.out.clone()
    c.q[1, 3, 10] = value
    c.run()
    assert c.error() == dsa.DSA_DEVERR_RANGE
    keep = torch.ones((3, 16), dtype=torch.bool)
    keep[1, 3] = False
    assert torch.equal(c.out[keep], want[keep])
    assert bool(c.out[1, 3].isnan().all()) and bool(c.lse[1, 3].isnan())


@pytest.mark.parametrize("name", ["two_queries", "own_page_copies", "full_heads_long_prefix", "packed_long_prefix"])
def test_what_no_query_sees_is_not_reported(name):
    """Values beyond the range behind the sequences' ends, in spare pages and in queries of no sequence."""
    c = Call(*SHAPES[name], fp8=True, seed=43)
    used = torch.zeros(c.b.pages * PAGE, dtype=torch.bool)
    for i in range(c.b.B):
        at = torch.arange(c.b.L[i])
        used[c.b.pt_host[torch.where(at < c.prefix, 0, i), at // PAGE].long() * PAGE + at % PAGE] = True
    flat = c.cache.view(-1, c.cache.shape[-1])
    for r in (~used).nonzero().flatten().tolist():
        flat[r, :LATENT] = 0x7E
        flat[r, LATENT:LATENT + 16].view(torch.float32)[:] = 50.0
        flat[r, LATENT + 16:].view(torch.bfloat16)[:] = 30000.0
    c.run().check()


@pytest.mark.parametrize("wide", [False, True])
def test_queries_of_no_sequence_are_not_reported(wide):
    c = Call([300, 300, 300], [1, 1, 1], 200, 16, fp8=True, seed=44, wide=wide, total_q=5)
    tail = c.q[:2] * 1e8
    c.q = torch.cat([c.q, tail])
    c.run()
    assert c.error() == dsa.DSA_DEVERR_SEQ  # (tokens of no sequence)
    Attention(c.b, c.q[:3], c.cache, True).check(c.out[:3], c.lse[:3], True)


@pytest.mark.parametrize("name", ["two_queries", "full_heads_long_prefix", "packed_long_prefix"])
def test_the_largest_values_within_the_range(name):
    """Elements of 448 * 36.5 = 16352 as values, and a rotary value of 16320, where q is 0: the scores are ordinary."""
    c = Call(*SHAPES[name], fp8=True, seed=45)
    c.q[..., 128:256] = 0
    c.q[..., LATENT + 9] = 0
    for pos in (0, 77, c.prefix - 1, c.b.L[0] - 1):
        _set_latent(c, 0, pos, 1, 36.5)
        _set_rotary(c, 0, pos, 9, -16320.0)
    c.q[0, 0, 3] = 2.0 ** -3
    c.run().check()
    c = Call(*SHAPES[name], fp8=True, seed=46)
    c.q[:, :, LATENT + 5] = 261120.0  # the same score for every position
    flat = c.cache.view(-1, c.cache.shape[-1])
    flat[:, LATENT + 16:].view(torch.bfloat16)[:, 5] = 0.0
    c.run().check()


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("place", ["own tile", "last tile", "prefix", "converted ahead", "packed, ahead"])
def test_infinities_are_not_out_of_range(place, wide):
    """A rotary value of infinity makes a score of -inf with q of the other sign: no weight, and no error."""
    shape, b, pos = PLACES[place]
    c = Call(*shape, fp8=True, seed=47, wide=wide)
    c.q[..., KV - 1] = 1.0
    _set_rotary(c, b, pos, 63, -math.inf)
    c.run().check()
