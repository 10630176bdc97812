"""Refusals of the norm, the per-head products and the expanded attention: answered on the host before any launch (no GPU)."""
import ctypes

import pytest
import torch

import sparse_attention_dsa_gb300 as dsa
from sparse_attention_dsa_gb300 import build as dsa_build

INV, UNS = dsa.DSA_ERR_INVALID_ARG, dsa.DSA_ERR_UNSUPPORTED
FAKE, FAKE2, FAKE3 = 0x10000, 0x20000, 0x30000  # aligned non-null addresses; never dereferenced


@pytest.fixture(scope="module", autouse=True)
def L():
    dsa_build.build()
    return dsa.lib()


def _dims(**kw):
    d = dict(batch=2, total_q=2, max_q_len=1, num_pages=8, page_size=64, max_pages_per_seq=4, idx_heads=64, idx_dim=128,
             idx_dtype=0, top_k=16, attn_heads=128, kv_dim=576, v_dim=512, softmax_scale=192 ** -0.5)
    d.update(kw)
    return dsa.DsaDims(**d)


def _ref(x):
    return ctypes.byref(x) if x is not None else None


def _norm(**a):
    p = dict(rows=4, dim=512, x=FAKE, xs=0, residual=None, sum=None, weight=FAKE, eps=1e-6, out=FAKE2, os=0, dtype=1, group=0,
             codes=None, scale=None)
    p.update(a)
    return dsa.lib().dsa_rms_norm(p["rows"], p["dim"], p["x"], p["xs"], p["residual"], p["sum"], p["weight"], p["eps"],
                                  p["out"], p["os"], p["dtype"], p["group"], p["codes"], p["scale"], None)


def _absorb(d, **a):
    p = dict(q_nope=FAKE, ts=0, hs=0, w=FAKE, q=FAKE2, ws=FAKE)
    p.update(a)
    return dsa.lib().dsa_absorb_queries(_ref(d), p["q_nope"], p["ts"], p["hs"], p["w"], p["q"], p["ws"], None)


def _values(d, **a):
    p = dict(o=FAKE, w=FAKE, out=FAKE2, ws=FAKE)
    p.update(a)
    return dsa.lib().dsa_value_heads(_ref(d), p["o"], p["w"], p["out"], p["ws"], None)


def _expanded(d, pages=8, **a):
    p = dict(q_nope=FAKE, ts=0, hs=0, q_pe=FAKE, pts=0, phs=0, w=FAKE, kv=FAKE, pt=FAKE, lens=FAKE, cu=FAKE, out=FAKE2, lse=None,
             ws=FAKE)
    p.update(a)
    return dsa.lib().dsa_expanded_attn(_ref(d), pages, p["q_nope"], p["ts"], p["hs"], p["q_pe"], p["pts"], p["phs"], p["w"],
                                       p["kv"], p["pt"], p["lens"], p["cu"], p["out"], p["lse"], p["ws"], None)


def _msg():
    return dsa.lib().dsa_last_error_message().decode()


@pytest.mark.parametrize("args,status,word", [
    (dict(rows=-1), INV, "rows"),
    (dict(dim=0), INV, "dim"),
    (dict(dim=20), UNS, "dim"),
    (dict(dim=16392), UNS, "dim"),
    (dict(eps=-1e-6), INV, "eps"),
    (dict(eps=float("nan")), INV, "eps"),
    (dict(eps=float("inf")), INV, "eps"),
    (dict(x=None), INV, "x is NULL"),
    (dict(x=FAKE + 8), INV, "aligned"),
    (dict(xs=504), INV, "x_stride"),
    (dict(xs=516), INV, "x_stride"),
    (dict(xs=-512), INV, "x_stride"),
    (dict(weight=None), INV, "weight"),
    (dict(residual=FAKE + 4), INV, "residual"),
    (dict(sum=FAKE3), INV, "residual"),
    (dict(out=None), INV, "out and codes"),
    (dict(os=260), INV, "out_stride"),
    (dict(out=FAKE, os=520), INV, "stride"),
    (dict(residual=FAKE3, sum=FAKE, xs=520), INV, "dense"),
    (dict(residual=FAKE3, out=FAKE3, os=520), INV, "dense"),
    (dict(residual=FAKE3, sum=FAKE2), INV, "same"),
    (dict(codes=FAKE3, scale=None), INV, "scale"),
    (dict(codes=FAKE3, scale=FAKE, dtype=0), INV, "codes_dtype"),
    (dict(codes=FAKE3, scale=FAKE, dtype=3), INV, "codes_dtype"),
    (dict(codes=FAKE3, scale=FAKE, group=64), INV, "group"),
    (dict(codes=FAKE3, scale=FAKE, group=32), INV, "group"),
    (dict(codes=FAKE3, scale=FAKE, dtype=2, group=0), INV, "group"),
    (dict(codes=FAKE3, scale=FAKE, dtype=2, group=32, dim=520), INV, "group"),
    (dict(codes=FAKE3, scale=FAKE, group=128, dim=576), INV, "group"),
])
def test_norm_is_checked(args, status, word):
    assert _norm(**args) == status and word in _msg()


def test_norm_without_rows():
    assert _norm(rows=0) == dsa.DSA_OK
    assert _norm(rows=0, residual=FAKE3, sum=FAKE3, out=FAKE) == dsa.DSA_OK
    assert _norm(rows=0, x=None, weight=None, out=None) == dsa.DSA_OK  # arrays without elements may have no address
    assert _norm(rows=0, dim=20) == UNS


@pytest.mark.parametrize("call", [_absorb, _values, _expanded])
def test_head_sizes_are_checked(call):
    assert call(None) == INV and "dims" in _msg()
    for kw, status, word in ((dict(total_q=-1), INV, "total_q"), (dict(attn_heads=0), INV, "attn_heads"),
                             (dict(attn_heads=129), UNS, "attn_heads"), (dict(kv_dim=512), UNS, "kv_dim"),
                             (dict(v_dim=256), UNS, "v_dim"), (dict(total_q=2 ** 31 - 5, batch=1), UNS, "total_q")):
        assert call(_dims(**kw)) == status and word in _msg(), kw
    assert call(_dims(total_q=0)) == dsa.DSA_OK


@pytest.mark.parametrize("call,names", [(_absorb, ("q_nope", "w", "q", "ws")), (_values, ("o", "w", "out", "ws")),
                                        (_expanded, ("q_nope", "q_pe", "w", "kv", "pt", "lens", "cu", "out", "ws"))])
def test_pointers_are_checked(call, names):
    for name in names:
        assert call(_dims(), **{name: None}) == INV and "NULL" in _msg()
        assert call(_dims(), **{name: FAKE + 8}) == INV and "aligned" in _msg()


@pytest.mark.parametrize("call,token,head,width", [(_absorb, "ts", "hs", 128), (_expanded, "ts", "hs", 128),
                                                   (_expanded, "pts", "phs", 64)])
def test_query_strides_are_checked(call, token, head, width):
    for t, h in ((0, width), (8192, 0), (-8192, width), (8192, width - 8), (8192, width + 4), (8196, width), (1 << 39, width),
                 (8192, 1 << 39)):
        assert call(_dims(), **{token: t, head: h}) == INV and "stride" in _msg(), (t, h)
    assert call(_dims(total_q=0), **{token: 8192, head: width}) == dsa.DSA_OK


def test_expanded_attention_arguments():
    assert _expanded(_dims(), 0) == INV and "total_pages" in _msg()
    assert _expanded(_dims(), -3) == INV and "total_pages" in _msg()
    assert _expanded(_dims(), 2 ** 31 - 1) == UNS and "total_pages" in _msg()
    assert _expanded(_dims(batch=0)) == INV
    assert _expanded(_dims(page_size=32)) == UNS
    assert _expanded(_dims(num_pages=1 << 26)) == UNS
    assert _expanded(_dims(kv_dtype=2)) == INV and "kv_dtype" in _msg()
    for scale in (0.0, -1.0, float("nan"), float("inf")):
        assert _expanded(_dims(softmax_scale=scale)) == INV and "softmax_scale" in _msg()
    assert _expanded(_dims(), lse=FAKE + 4) == INV
    # the indexer's sizes, top_k and max_q_len play no part
    assert _expanded(_dims(total_q=0, top_k=0, idx_heads=0, idx_dtype=9)) == dsa.DSA_OK


def test_expanded_workspace_size(L):
    assert L.dsa_expanded_attn_workspace_size(None, 4) == 0
    assert dsa.expanded_attn_workspace_size(_dims(), 0) == 0
    assert dsa.expanded_attn_workspace_size(_dims(total_q=0), 4) == 256
    assert dsa.expanded_attn_workspace_size(_dims(), 2 ** 31 - 1) == 256
    size = lambda pages, **kw: dsa.expanded_attn_workspace_size(_dims(**kw), pages)
    tile = 128 * 1152 + 128 * 512 * 128  # 128 positions
    parts = 2 * 152 * 4 * (256 * 128 + 2 * 256)  # two partial results for each SM
    assert parts + 2 * tile <= size(1, total_q=1) < parts + 3 * tile
    # every smaller call fits
    largest = size(200, batch=7, total_q=900)
    for pages in (1, 2, 3, 100, 199, 200):
        for batch in (1, 2, 7):
            for tokens in (1, 5, 899, 900):
                assert size(pages, batch=batch, total_q=tokens) <= largest
    # sequences of one position each take a tile each
    assert size(50, batch=50, total_q=50) >= 50 * tile


def test_wrappers_raise():
    x = torch.zeros((4, 64), dtype=torch.bfloat16)
    for bad in (x.t(), torch.zeros((5, 64), dtype=torch.bfloat16), torch.zeros((4, 128), dtype=torch.bfloat16)[:, ::2]):
        with pytest.raises(dsa.DsaError, match="out must be"):
            dsa.rms_norm(x, x[0], 1e-6, out=bad, stream=0)
    with pytest.raises(dsa.DsaError, match="x must be"):
        dsa.rms_norm(x[0], x[0], 1e-6, out=x, stream=0)
    with pytest.raises(dsa.DsaError, match="x must be"):
        dsa.rms_norm(torch.zeros((4, 128), dtype=torch.bfloat16)[:, ::2], x[0], 1e-6, out=x, stream=0)
    with pytest.raises(dsa.DsaError, match="eps"):
        dsa.rms_norm(x, x[0], -1.0, out=torch.zeros_like(x), stream=0)
    with pytest.raises(dsa.DsaError, match="attn_heads"):
        dsa.absorb_queries(_dims(attn_heads=0), FAKE, FAKE, FAKE, FAKE, stream=0)
    with pytest.raises(dsa.DsaError, match="kv_dim"):
        dsa.value_heads(_dims(kv_dim=512), FAKE, FAKE, FAKE, FAKE, stream=0)
    with pytest.raises(dsa.DsaError, match="too small"):
        dsa.expanded_attn(_dims(), 8, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, None, torch.zeros(256), stream=0)
    with pytest.raises(dsa.DsaError, match="stride"):
        dsa.expanded_attn(_dims(), 8, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, None, FAKE, stream=0, q_pe_strides=(0, 64))
