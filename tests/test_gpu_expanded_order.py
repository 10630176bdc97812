"""Expanded attention where scores are far apart, and where heads go in groups of several with a smaller last one (tolerances:
_latent_stored, whose keys are the kernel's, so that large scores are known as well as small ones)."""
import pytest
import torch

from _latent import LATENT
from _latent_stored import check_call
from _rope_prefix import PAGE
from test_gpu_expanded import Call, _built  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("std", [8.0, 2.0, 0.01])
@pytest.mark.parametrize("fp8", [False, True])
def test_sharp_and_flat_weights(std, fp8):
    """Scores of a few hundred (one weight next to 1, the maximum rises again and again), and of next to nothing."""
    check_call(Call([700], [400], 4, fp8, seed=601, std=std).run())


@pytest.mark.parametrize("step", [0.1, 0.02])
@pytest.mark.parametrize("falling", [False, True])
def test_rising_and_falling_scores(step, falling):
    """Every tile's scores beyond the ones before, so that sums and outputs are rescaled each time, or far below them."""
    c = Call([1300], [300], 2, seed=602)
    at = torch.arange(1300)
    row = (c.b.pt_host[0, at // PAGE].long() * PAGE + at % PAGE).cuda()
    lift = torch.arange(1300, device="cuda").double() * step
    c.kv.flatten(0, 1)[row, LATENT] = (lift.flip(0) if falling else lift).to(torch.bfloat16)
    c.q_pe[..., 0] = 8.0
    check_call(c.run())


@pytest.mark.parametrize("lens,heads,edges", [
    ([1900], 128, (0, 25, 26, 76, 77, 127)),                                 # 15 tiles: groups of 51, 51 and 26 heads, the last first
    ([1900, 1700, 1650, 1900, 1850, 1800, 1910, 1600], 16, (0, 3, 4, 9, 10, 15)),  # 115 tiles: of 6, 6 and 4, longest items first
])
def test_groups_of_heads_with_a_smaller_last_one(lens, heads, edges):
    """Whole items of heads whose keys and values are too many for L2 at once: groups of heads, one after another."""
    check_call(Call(lens, lens, heads, seed=603).run(), heads=edges)
