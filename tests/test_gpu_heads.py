"""The products of every head with its weights on the GPU against 64 bits (tolerances: _latent)."""
import pytest
import torch

import sparse_attention_dsa_gb300 as dsa

from _gpu import ensure_built
from _latent import LATENT, NOPE, VALUE, check_product, head_dims, normal, weights
from _rope_prefix import KV

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    ensure_built()


def _workspace():
    return torch.zeros(256, dtype=torch.uint8, device="cuda")


SIZES = [(1, 1), (1, 128), (5, 3), (32, 128), (127, 16), (128, 7), (129, 8), (130, 1), (257, 33), (700, 5), (2048, 16), (4100, 128)]


@pytest.mark.parametrize("tokens,heads", SIZES)
@pytest.mark.parametrize("form", ["dense", "projection", "heads first"])
def test_absorb(tokens, heads, form):
    if form == "dense":
        q_nope = normal((tokens, heads, NOPE), 1)
        strides = (0, 0)
    elif form == "projection":  # the first dims of a projection's 192 a head
        q_nope = normal((tokens, heads, 192), 1)[..., :NOPE]
        strides = q_nope.stride()[:2]
    else:
        q_nope = normal((heads, tokens + 3, NOPE), 1)[:, :tokens].transpose(0, 1)
        strides = q_nope.stride()[:2]
    if tokens == 1 and form == "heads first":
        strides = (8, strides[1])
    w, ws = weights(heads, 2), _workspace()
    q = torch.full((tokens + 1, heads, KV), 7.0, dtype=torch.bfloat16, device="cuda")
    dsa.absorb_queries(head_dims(tokens, heads), q_nope, w, q, ws, q_nope_strides=strides)
    assert dsa.get_device_error(ws) == 0
    check_product(q[:tokens, :, :LATENT], q_nope.double(), w[:, :NOPE].double(), "thd,hdc->thc")
    assert bool((q[:tokens, :, LATENT:] == 7).all() and (q[tokens:] == 7).all())


@pytest.mark.parametrize("tokens,heads", SIZES)
def test_values(tokens, heads):
    o, w, ws = normal((tokens, heads, LATENT), 3), weights(heads, 4), _workspace()
    out = torch.full((tokens + 1, heads, VALUE), 7.0, dtype=torch.bfloat16, device="cuda")
    dsa.value_heads(head_dims(tokens, heads), o, w, out, ws)
    assert dsa.get_device_error(ws) == 0
    check_product(out[:tokens], o.double(), w[:, NOPE:].double(), "thc,hdc->thd")
    assert bool((out[tokens:] == 7).all())


def test_rows_are_independent():
    """An infinity or NaN of one token or head is in no other's result."""
    tokens, heads = 140, 4
    q_nope, o, w, ws = normal((tokens, heads, NOPE), 5), normal((tokens, heads, LATENT), 6), weights(heads, 7), _workspace()
    q, out = torch.zeros((tokens, heads, KV), dtype=torch.bfloat16, device="cuda"), torch.zeros((tokens, heads, VALUE),
                                                                                               dtype=torch.bfloat16, device="cuda")
    dims = head_dims(tokens, heads)

    def both():
        dsa.absorb_queries(dims, q_nope, w, q, ws)
        dsa.value_heads(dims, o, w, out, ws)
        return q.clone(), out.clone()

    clean = both()
    q_nope[3, 1, 7] = o[131, 2, 500] = float("nan")
    q_nope[77, 0, 0] = o[5, 3, 0] = float("inf")
    got = both()
    for a, b, rows in ((clean[0], got[0], ((3, 1), (77, 0))), (clean[1], got[1], ((131, 2), (5, 3)))):
        hit = torch.zeros((tokens, heads), dtype=torch.bool)
        for t, h in rows:
            hit[t, h] = True
        assert torch.equal(a[~hit], b[~hit])
        assert not bool(b[hit][:, :VALUE].isfinite().any())
    assert dsa.get_device_error(ws) == 0


def test_offsets_beyond_32_bits():
    """40000 tokens of 128 heads: the queries' offsets pass 2^31 elements, the last tokens are those of a short call."""
    tokens, heads, last = 40000, 128, 5
    w, ws = weights(heads, 8), _workspace()
    q_nope = torch.zeros((tokens, heads, NOPE), dtype=torch.bfloat16, device="cuda")
    q_nope[-last:] = normal((last, heads, NOPE), 9)
    q = torch.full((tokens, heads, KV), 7.0, dtype=torch.bfloat16, device="cuda")
    dsa.absorb_queries(head_dims(tokens, heads), q_nope, w, q, ws)
    check_product(q[-last:, :, :LATENT], q_nope[-last:].double(), w[:, :NOPE].double(), "thd,hdc->thc")
    assert bool((q[:-last:1000, :, :LATENT] == 0).all() and (q[::1000, :, LATENT:] == 7).all())
    del q_nope
    o = q[..., :LATENT].contiguous()
    out = torch.zeros((tokens, heads, VALUE), dtype=torch.bfloat16, device="cuda")
    dsa.value_heads(head_dims(tokens, heads), o, w, out, ws)
    check_product(out[-last:], o[-last:].double(), w[:, NOPE:].double(), "thc,hdc->thd")
    assert bool((out[:-last:1000] == 0).all()) and dsa.get_device_error(ws) == 0


def test_streams_and_a_graph():
    tokens, heads = 300, 16
    q_nope, w, ws, ws2 = normal((tokens, heads, NOPE), 10), weights(heads, 11), _workspace(), _workspace()
    q = torch.zeros((tokens, heads, KV), dtype=torch.bfloat16, device="cuda")
    q2 = torch.zeros_like(q)
    dims, side = head_dims(tokens, heads), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):  # two calls at once
        dsa.absorb_queries(dims, q_nope, w, q2, ws2)
    dsa.absorb_queries(dims, q_nope, w, q, ws)
    side.synchronize()
    torch.cuda.synchronize()
    assert torch.equal(q, q2)
    out = torch.zeros((tokens, heads, VALUE), dtype=torch.bfloat16, device="cuda")
    o = torch.zeros((tokens, heads, LATENT), dtype=torch.bfloat16, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dsa.absorb_queries(dims, q_nope, w, q, ws)
        o.copy_(q[..., :LATENT])
        dsa.value_heads(dims, o, w, out, ws)
    q_nope.copy_(normal((tokens, heads, NOPE), 12))
    graph.replay()
    torch.cuda.synchronize()
    check_product(q[..., :LATENT], q_nope.double(), w[:, :NOPE].double(), "thd,hdc->thc")
    check_product(out, o.double(), w[:, NOPE:].double(), "thc,hdc->thd")
    assert dsa.get_device_error(ws) == 0


@pytest.mark.parametrize("values", [False, True])
def test_short_waits_are_reported(values):
    tokens, heads = 600, 64
    x, w, ws = normal((tokens, heads, LATENT if values else NOPE), 13), weights(heads, 14), _workspace()
    out = torch.zeros((tokens, heads, VALUE if values else KV), dtype=torch.bfloat16, device="cuda")
    call = dsa.value_heads if values else dsa.absorb_queries
    old = dsa.set_wait_limit_ns(200)
    try:
        call(head_dims(tokens, heads), x, w, out, ws)
        torch.cuda.synchronize()
    finally:
        dsa.set_wait_limit_ns(old)
    assert dsa.get_device_error(ws) & dsa.DSA_DEVERR_TIMEOUT
    dsa.clear_device_error(ws)
    call(head_dims(tokens, heads), x, w, out, ws)
    assert dsa.get_device_error(ws) == 0
    if values:
        check_product(out, x.double(), w[:, NOPE:].double(), "thc,hdc->thd")
    else:
        check_product(out[..., :LATENT], x.double(), w[:, :NOPE].double(), "thd,hdc->thc")
