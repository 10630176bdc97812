"""Expanded attention does not depend on how large its numbers are: rows and weights of any magnitude within the documented range
have the relative error of ordinary ones (tolerances: _latent_stored)."""
import pytest
import torch

import sparse_attention_dsa_gb300 as dsa

from _latent import LATENT, NOPE
from _latent_stored import BF16, F16, check_call
from _rope_prefix import PAGE, latent_fp8_rows
from test_gpu_expanded import Call, _built  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu

SEQ, Q = [700, 129, 40], [400, 129, 3]


def _for_fp8(c):
    """Sizes and workspace of a call whose rows were made FP8 afterwards."""
    c.dims = c.b.dims(attn_heads=c.heads, kv_dtype=dsa.DSA_FP8_E4M3, softmax_scale=c.dims.softmax_scale)
    c.ws = torch.full((dsa.expanded_attn_workspace_size(c.dims, c.pages),), 0xFF, dtype=torch.uint8, device="cuda")
    c.ws[:256] = 0


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


@pytest.mark.parametrize("power", [10, 14, 20, 27, 40])
def test_small_fp8_rows(power):
    """Latent parts of 2^-power beside larger weights and queries, so that the scores are ordinary."""
    c = Call(SEQ, Q, 3, seed=411)
    c.rows[:, :LATENT] *= 2.0 ** -power
    c.kv, c.fp8 = latent_fp8_rows(c.rows).view(c.b.pages, PAGE, -1), True
    _for_fp8(c)
    c.w *= 2.0 ** 9
    c.q_nope *= 2.0 ** (power - 9)
    check_call(c.run(), half=BF16)


@pytest.mark.parametrize("power", [8, 12, 20, 27, 40])
def test_small_weights_with_fp8_rows(power):
    c = Call(SEQ, Q, 3, True, seed=412)
    c.w *= 2.0 ** -power
    c.q_nope *= 2.0 ** power
    check_call(c.run(), half=BF16)


def test_fp8_rows_and_weights_of_many_magnitudes():
    """Every position and every 16 rows of the weights of their own magnitude, and rows within those of somewhat different ones;
    the queries make up for the keys'."""
    c = Call([400, 70], [400, 70], 3, seed=413)
    g = torch.Generator(device="cuda").manual_seed(414)
    c.rows[:, :LATENT] *= (2.0 ** -torch.randint(0, 40, (len(c.rows), 1), generator=g, device="cuda")).to(torch.bfloat16)
    c.kv, c.fp8 = latent_fp8_rows(c.rows).view(c.b.pages, PAGE, -1), True
    _for_fp8(c)
    down = torch.randint(0, 20, (3, 16, 1), generator=g, device="cuda").repeat_interleave(16, dim=1)
    down = down + torch.randint(0, 12, (3, 256, 1), generator=g, device="cuda")
    c.w *= (2.0 ** -down).to(torch.bfloat16)
    c.q_nope *= (2.0 ** down[:, :NOPE, 0])[None].to(torch.bfloat16)
    check_call(c.run(), half=BF16)


def test_fp8_groups_of_zeros_with_any_scale():
    """Codes of 0 are 0 times their scale, whatever finite number that is."""
    c = Call([300], [260], 2, True, seed=415)
    flat = c.kv.flatten(0, 1)
    flat[:, 128:256] = 0
    scales = flat[:, LATENT:LATENT + 16].contiguous().view(torch.float32)
    scales[:, 1] = torch.tensor([3.0e38, 1.0, -2.0e38, 1e-40], device="cuda")[torch.arange(len(flat), device="cuda") % 4]
    flat[:, LATENT:LATENT + 16] = scales.view(torch.uint8)
    check_call(c.run())


@pytest.mark.parametrize("fp8", [False, True])
def test_a_captured_call_with_other_magnitudes(fp8):
    """Which positions are kept in which form, and the rows' powers of two, are found anew at each replay."""
    c = Call([700, 129], [400, 129], 3, fp8, seed=421)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.run()
    w = c.w.clone()
    for power in (0, 24, 0, 12, 30):
        c.w.copy_(w)
        c.w[1:, NOPE:] *= 2.0 ** -power  # (one head keeps its values)
        c.out.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        check_call(c, half=BF16 if power else F16, heads=(0, 1, 2))
