"""Expanded attention does not depend on how large its numbers are: rows and weights of any magnitude within the documented range
have the relative error of ordinary ones (tolerances: _latent_stored)."""
import pytest
import torch

from _latent import LATENT, NOPE
from _latent_stored import BF16, F16, check_call
from _rope_prefix import PAGE
from test_gpu_expanded import Call, _built  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu

SEQ, Q = [700, 129, 40], [400, 129, 3]


def _rows_of(c, b, at):
    """Cache rows of positions `at` of sequence b."""
    return (c.b.pt_host[b, at // PAGE].long() * PAGE + at % PAGE).cuda()


@pytest.mark.parametrize("power", [6, 10, 12, 13, 16, 20, 27, 40])
def test_small_value_weights(power):
    """Value weights of 2^-power beside ordinary key weights: the output is ordinary but for its scale."""
    c = Call(SEQ, Q, 3, seed=401)
    c.w[:, NOPE:] *= 2.0 ** -power
    check_call(c.run(), half=BF16)


@pytest.mark.parametrize("seq_lens,q_lens,heads", [([5000, 4700], [520, 500], 40), ([2000], [700], 8)])
def test_small_values_in_items_that_are_cut(seq_lens, q_lens, heads):
    c = Call(seq_lens, q_lens, heads, seed=402)
    c.w[:, NOPE:] *= 2.0 ** -24
    check_call(c.run(), half=BF16, heads=(0, heads - 1))


@pytest.mark.parametrize("apart", [1, 17, 32, 100])
def test_small_and_ordinary_values_side_by_side(apart):
    """Positions in runs of `apart` whose latent parts are ordinary, small and next to nothing; queries that see only small ones
    have their own relative error."""
    c = Call([600, 90], [600, 90], 4, seed=403)
    flat = c.kv.flatten(0, 1)
    for b in range(2):
        at = torch.arange(c.b.L[b])
        row = _rows_of(c, b, at)
        size = torch.tensor([2.0 ** -30, 2.0 ** -15, 1.0])[(at // apart) % 3].cuda()
        size[at.cuda() < 150] = 2.0 ** -33
        flat[row, :LATENT] = (flat[row, :LATENT].float() * size[:, None]).to(torch.bfloat16)
    c.run()
    check_call(c, half=BF16)
    check_call(c, torch.tensor(c.b.pos, device="cuda") < 150, half=BF16)


def test_hidden_values_of_any_size_beside_small_ones():
    """What a position that is not seen holds, large as it may be, takes nothing from the small ones in front of it."""
    c = Call([300], [260], 2, seed=404)
    c.kv[..., :LATENT] *= 2.0 ** -30
    row = _rows_of(c, 0, torch.arange(200, 300))
    c.kv.flatten(0, 1)[row, :LATENT] = (c.kv.flatten(0, 1)[row, :LATENT].float() * 2.0 ** 40).to(torch.bfloat16)
    check_call(c.run(), torch.tensor(c.b.pos, device="cuda") < 200, half=BF16)


def test_ordinary_values_keep_eleven_bits():
    for fp8 in (False, True):
        check_call(Call(SEQ, Q, 3, fp8, seed=405).run(), half=F16)
