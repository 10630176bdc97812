"""Refusals of the rotation and shared-prefix entry points: answered on the host before any launch (no GPU)."""
import ctypes

import pytest

import sparse_attention_dsa_gb300 as dsa
from sparse_attention_dsa_gb300 import build as dsa_build

INV, UNS = dsa.DSA_ERR_INVALID_ARG, dsa.DSA_ERR_UNSUPPORTED
FAKE = 0x10000  # an aligned non-null address; never dereferenced


@pytest.fixture(scope="module")
def L():
    dsa_build.build()
    return dsa.lib()


def _dims(**kw):
    d = dict(batch=2, total_q=2, max_q_len=1, num_pages=8, page_size=64, max_pages_per_seq=4, idx_heads=64, idx_dim=128,
             idx_dtype=0, top_k=16, attn_heads=128, kv_dim=576, v_dim=512, softmax_scale=1 / 24)
    d.update(kw)
    return dsa.DsaDims(**d)


def _rope(**kw):
    r = dict(table=FAKE, table_len=1024, kv_pairing=1, idx_pairing=0, idx_begin=0)
    r.update(kw)
    return dsa.DsaRope(**r)


def _ref(x):
    return ctypes.byref(x) if x is not None else None


def _append(d, r, **a):
    p = dict(k_new=FAKE, k_stride=0, kv_new=FAKE, kv_stride=0, pt=FAKE, lens=FAKE, cu=FAKE, k_cache=FAKE, k_scale=None,
             kv_cache=FAKE, ws=FAKE)
    p.update(a)
    return dsa.lib().dsa_rope_append(_ref(d), _ref(r), p["k_new"], p["k_stride"], p["kv_new"], p["kv_stride"], p["pt"],
                                     p["lens"], p["cu"], p["k_cache"], p["k_scale"], p["kv_cache"], p["ws"], None)


def _queries(d, r, **a):
    p = dict(q_pe=FAKE, ts=0, hs=0, q=FAKE, q_idx_in=FAKE, qs=0, q_idx=FAKE, q_scale=None, lens=FAKE, cu=FAKE, ws=FAKE)
    p.update(a)
    return dsa.lib().dsa_rope_queries(_ref(d), _ref(r), p["q_pe"], p["ts"], p["hs"], p["q"], p["q_idx_in"], p["qs"],
                                      p["q_idx"], p["q_scale"], p["lens"], p["cu"], p["ws"], None)


def _prefix(d, prefix_len=64, **a):
    p = dict(q=FAKE, kv=FAKE, pt=FAKE, lens=FAKE, cu=FAKE, out=FAKE, lse=None, ws=FAKE)
    p.update(a)
    return dsa.lib().dsa_prefix_attn(_ref(d), prefix_len, p["q"], p["kv"], p["pt"], p["lens"], p["cu"], p["out"],
                                     p["lse"], p["ws"], None)


def _msg():
    return dsa.lib().dsa_last_error_message().decode()


@pytest.mark.parametrize("call", [_append, _queries])
@pytest.mark.parametrize("rope,status,word", [
    (dict(table=None), INV, "table"),
    (dict(table=FAKE + 4), INV, "aligned"),
    (dict(table_len=0), INV, "table_len"),
    (dict(kv_pairing=2), INV, "kv_pairing"),
    (dict(idx_pairing=-1), INV, "idx_pairing"),
    (dict(idx_begin=-2), INV, "idx_begin"),
    (dict(idx_begin=4), INV, "idx_begin"),
    (dict(idx_begin=72), INV, "idx_begin"),
])
def test_rope_is_checked(L, call, rope, status, word):
    assert call(_dims(), _rope(**rope)) == status and word in _msg()


@pytest.mark.parametrize("call", [_append, _queries])
@pytest.mark.parametrize("dims,status,word", [
    (dict(batch=0), INV, "batch"),
    (dict(total_q=-1), INV, "total_q"),
    (dict(page_size=32), UNS, "page_size"),
    (dict(idx_dim=132), UNS, "idx_dim"),
    (dict(idx_dim=136), UNS, "idx_dim"),
    (dict(idx_dim=56), INV, "idx_begin"),
    (dict(idx_dtype=2, idx_dim=120), UNS, "idx_dim"),
    (dict(idx_dtype=3), INV, "idx_dtype"),
    (dict(idx_dtype=1), INV, "scale"),
    (dict(idx_dtype=2), INV, "scale"),
    (dict(kv_dim=512), UNS, "kv_dim"),
])
def test_dims_are_checked(L, call, dims, status, word):
    assert call(_dims(**dims), _rope()) == status and word in _msg()


def test_append_pointers_and_strides(L):
    assert _append(None, _rope()) == INV and "dims" in _msg()
    assert _append(_dims(), None) == INV and "rope" in _msg()
    assert _append(_dims(kv_dtype=2), _rope()) == INV and "kv_dtype" in _msg()
    for name in ("pt", "lens", "cu", "k_cache", "kv_cache", "ws"):
        assert _append(_dims(), _rope(), **{name: None}) == INV
        assert _append(_dims(), _rope(), **{name: FAKE + 8}) == INV and "aligned" in _msg()
    for name, bad in (("k_stride", (120, 132, -128)), ("kv_stride", (512, 580, -576))):
        for v in bad:
            assert _append(_dims(), _rope(), **{name: v}) == INV and name in _msg()
    assert _append(_dims(num_pages=1 << 26), _rope()) == UNS
    # nothing to do
    assert _append(_dims(total_q=0), _rope()) == dsa.DSA_OK
    assert _append(_dims(), _rope(), k_new=None, kv_new=None, k_cache=None, kv_cache=None) == dsa.DSA_OK


def test_queries_pointers_and_strides(L):
    assert _queries(None, _rope()) == INV and "dims" in _msg()
    assert _queries(_dims(), None) == INV and "rope" in _msg()
    for name in ("q", "q_idx", "lens", "cu", "ws"):
        assert _queries(_dims(), _rope(), **{name: None}) == INV
    assert _queries(_dims(attn_heads=0), _rope()) == INV and "attn_heads" in _msg()
    assert _queries(_dims(attn_heads=129), _rope()) == UNS
    assert _queries(_dims(idx_heads=0), _rope()) == INV and "idx_heads" in _msg()
    assert _queries(_dims(idx_heads=129), _rope()) == UNS
    for ts, hs in ((0, 64), (8192, 0), (-8192, 64), (8192, 56), (8192, 68), (8196, 64)):
        assert _queries(_dims(), _rope(), ts=ts, hs=hs) == INV and "stride" in _msg()
    for qs in (64 * 128 - 8, 64 * 128 + 4, -64 * 128):
        assert _queries(_dims(), _rope(), qs=qs) == INV and "q_idx_stride" in _msg()
    assert _queries(_dims(total_q=0), _rope()) == dsa.DSA_OK
    assert _queries(_dims(), _rope(), q_pe=None, q_idx_in=None, q=None, q_idx=None) == dsa.DSA_OK


def test_prefix_attention_arguments(L):
    assert _prefix(None) == INV and "dims" in _msg()
    assert _prefix(_dims(), -1) == INV and "prefix_len" in _msg()
    assert _prefix(_dims(), 257) == INV and "prefix_len" in _msg()
    assert _prefix(_dims(attn_heads=0)) == INV
    assert _prefix(_dims(attn_heads=129)) == UNS
    assert _prefix(_dims(kv_dim=512)) == UNS
    assert _prefix(_dims(v_dim=600)) == INV
    assert _prefix(_dims(kv_dtype=2)) == INV and "kv_dtype" in _msg()
    for scale in (0.0, -1.0, float("nan"), float("inf")):
        assert _prefix(_dims(softmax_scale=scale)) == INV and "softmax_scale" in _msg()
    for name in ("q", "kv", "pt", "lens", "cu", "out", "ws"):
        assert _prefix(_dims(), **{name: None}) == INV
        assert _prefix(_dims(), **{name: FAKE + 8}) == INV and "aligned" in _msg()
    assert _prefix(_dims(), lse=FAKE + 4) == INV
    assert _prefix(_dims(num_pages=1 << 26)) == UNS
    assert _prefix(_dims(total_q=0)) == dsa.DSA_OK
    # the indexer's sizes and top_k play no part
    assert _prefix(_dims(total_q=0, top_k=0, idx_heads=0, idx_dtype=9)) == dsa.DSA_OK


def test_prefix_workspace_size(L):
    assert L.dsa_prefix_attn_workspace_size(None, 0) == 0
    assert dsa.prefix_attn_workspace_size(_dims(), -1) == 0
    assert dsa.prefix_attn_workspace_size(_dims(), 0) >= 256
    assert dsa.prefix_attn_workspace_size(_dims(), 100) >= 256
    # partial results [128][512] and [128][2] fp32, two for each of 76 pairs, where the work is divided; one for each item
    # and pair where rows are packed; converted rows of 1152 bytes for a long FP8 prefix
    part = 4 * (128 * 512 + 2 * 128)
    short = _dims(batch=8, total_q=8, max_pages_per_seq=8, num_pages=64)
    long = _dims(batch=8, total_q=8, max_pages_per_seq=1000, num_pages=8000)
    assert dsa.prefix_attn_workspace_size(short, 0) < part
    assert 152 * part <= dsa.prefix_attn_workspace_size(long, 0) < 153 * part
    packed = dict(batch=64, total_q=64, max_pages_per_seq=520, num_pages=2000, attn_heads=16)
    assert (64 + 8 + 76) * part <= dsa.prefix_attn_workspace_size(_dims(**packed), 32768) < (64 + 8 + 77) * part
    fp8 = dsa.prefix_attn_workspace_size(_dims(**packed, kv_dtype=dsa.DSA_FP8_E4M3), 32768)
    assert fp8 == dsa.prefix_attn_workspace_size(_dims(**packed), 32768) + 32768 * 1152


def test_wrappers_raise(L):
    with pytest.raises(dsa.DsaError, match="prefix_len"):
        dsa.prefix_attn(_dims(), -1, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, None, FAKE, stream=0)
    with pytest.raises(dsa.DsaError, match="table_len"):
        dsa.rope_append(_dims(), _rope(table_len=0), FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, None, FAKE, FAKE, stream=0)
    with pytest.raises(dsa.DsaError, match="head"):
        dsa.rope_queries(_dims(attn_heads=0), _rope(), FAKE, FAKE, FAKE, FAKE, None, FAKE, FAKE, FAKE, stream=0)
