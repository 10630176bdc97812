"""Expanded attention on arrays that begin 16 bytes behind a multiple of 32, as every array may (views of larger buffers, a
pool with pieces of 16 bytes)."""
import pytest
import torch

import sparse_attention_dsa_gb300 as dsa

from test_gpu_expanded import Call, _built  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu


def _behind(t):
    """t's contents 16 bytes behind a multiple of 256."""
    raw = torch.zeros(t.numel() * t.element_size() + 512, dtype=torch.uint8, device="cuda")
    at = -raw.data_ptr() % 256 + 16
    view = raw[at:at + t.numel() * t.element_size()].view(t.dtype).view(t.shape)
    view.copy_(t)
    return view


@pytest.mark.parametrize("names", [("out",), ("ws",), ("out", "ws"), ("q_nope", "q_pe", "w", "kv", "out", "lse", "ws")])
@pytest.mark.parametrize("seq_lens,q_lens,heads,fp8", [
    ([300, 70], [257, 1], 3, False),      # whole items
    ([5000, 4700], [520, 500], 40, False),  # whole items in front of parts
    ([2000], [700], 8, True),             # parts
])
def test_arrays_at_any_multiple_of_16(names, seq_lens, q_lens, heads, fp8):
    want = Call(seq_lens, q_lens, heads, fp8, seed=301).run()
    assert dsa.get_device_error(want.ws) == 0
    c = Call(seq_lens, q_lens, heads, fp8, seed=301)
    for name in names:
        setattr(c, name, _behind(getattr(c, name)))
        assert getattr(c, name).data_ptr() % 32 == 16
    c.run()
    assert dsa.get_device_error(c.ws) == 0
    assert torch.equal(c.out, want.out) and torch.equal(c.lse, want.lse)
