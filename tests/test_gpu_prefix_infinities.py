"""Shared-prefix attention: a row whose infinite value gives a score of -inf makes NaN of that dim wherever the tiles of
positions fall (a weight of 0 times an infinity), and of nothing that does not see it."""
import math

import pytest
import torch

import sparse_attention_dsa_gb300 as dsa  # noqa: F401

from _gpu import ensure_built
from _rope_prefix import PAGE
from test_gpu_prefix import Call

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    ensure_built()


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("heads", [16, 128])
@pytest.mark.parametrize("pos", [0, 127, 128, 199, 200, 260, 383, 384, 500, 694, 697, 699])
def test_an_infinite_value_of_weight_0(pos, heads, wide):
    """Positions in full tiles, in the tiles in which the prefix (200) ends and the sequence's own begin, and in the last
    one, that some of the queries do not see."""
    c = Call([700, 600, 650], [6, 1, 2], 200, heads, seed=60, wide=wide)
    c.q[..., 77] = 1.0
    c.run()
    want = c.out.clone(), c.lse.clone()
    src = c.b.pt_host[0, pos // PAGE]
    c.cache[int(src), pos % PAGE, 77] = -math.inf
    c.run()
    assert c.error() == 0
    seen = torch.tensor([(pos < 200 or s == 0) and p >= pos for s, p in zip(c.b.seq, c.b.pos)])
    assert bool(c.out[seen][..., 77].isnan().all())
    assert torch.equal(c.out[~seen], want[0][~seen]) and torch.equal(c.lse[~seen], want[1][~seen])


@pytest.mark.parametrize("wide", [False, True])
def test_infinite_values_of_every_row(wide):
    c = Call([130, 70], [2, 1], 64, 16, seed=61, wide=wide)
    c.q[..., 300] = -2.0
    c.cache[..., 300] = math.inf
    c.run()
    assert c.error() == 0
    assert bool(c.out[..., 300].isnan().all())
