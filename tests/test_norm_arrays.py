"""rms_norm's arrays are looked at before their addresses are taken: shapes, strides and types that the call would read or
write past, or as something else (no GPU: every call here is refused)."""
import pytest
import torch

import sparse_attention_dsa_gb300 as dsa
from sparse_attention_dsa_gb300 import build as dsa_build

ROWS, DIM = 4, 256


@pytest.fixture(scope="module", autouse=True)
def _built():
    dsa_build.build()


def _zeros(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype)


def _call(eps=1e-6, **kw):
    a = dict(x=_zeros(ROWS, DIM), weight=_zeros(DIM), out=_zeros(ROWS, DIM), residual=_zeros(ROWS, DIM), sum=_zeros(ROWS, DIM),
             codes=_zeros(ROWS, DIM, dtype=torch.uint8), scale=_zeros(ROWS, DIM // 128, dtype=torch.float32), group=128)
    a.update(kw)
    dsa.rms_norm(a.pop("x"), a.pop("weight"), eps, stream=0, **a)


def _wide(rows, dim, dtype=torch.bfloat16):
    return _zeros(rows, dim + 64, dtype=dtype)[:, :dim]


BAD = [
    ("x", _zeros(1, DIM).expand(ROWS, DIM)),                     # one row for all: only that row is there
    ("x", _zeros(ROWS * DIM).as_strided((ROWS, DIM), (DIM // 2, 1))),  # rows that overlap
    ("x", _zeros(ROWS, DIM, dtype=torch.float16)),
    ("x", _zeros(ROWS, DIM, dtype=torch.float32)),
    ("out", _zeros(1, DIM).expand(ROWS, DIM)),
    ("out", _zeros(ROWS, DIM, dtype=torch.float16)),
    ("residual", _wide(ROWS, DIM)),                              # a slice, as x may be
    ("residual", _zeros(1, DIM).expand(ROWS, DIM)),
    ("residual", _zeros(ROWS - 1, DIM)),
    ("residual", _zeros(ROWS, DIM, dtype=torch.float32)),
    ("sum", _wide(ROWS, DIM)),
    ("sum", _zeros(ROWS, DIM + 8)),
    ("sum", _zeros(ROWS, DIM, dtype=torch.float16)),
    ("weight", _zeros(DIM - 8)),
    ("weight", _zeros(DIM + 8)),
    ("weight", _zeros(1, DIM)),
    ("residual", _zeros(ROWS * DIM)),
    ("residual", torch.tensor(0, dtype=torch.bfloat16)),
    ("weight", _zeros(2 * DIM)[::2]),
    ("weight", _zeros(DIM, dtype=torch.float32)),
    ("codes", _zeros(ROWS, DIM // 2, dtype=torch.uint8)),
    ("codes", _wide(ROWS, DIM, torch.uint8)),
    ("codes", _zeros(ROWS, DIM)),
    ("scale", _zeros(ROWS, dtype=torch.float32)),                # a scale a row where a tile has one
    ("scale", _zeros(ROWS, DIM // 128, dtype=torch.uint8)),
    ("scale", _zeros(DIM // 128, ROWS, dtype=torch.float32).t()),
]


@pytest.mark.parametrize("name,t", BAD)
def test_other_arrays_are_refused(name, t):
    with pytest.raises(dsa.DsaError, match=f"^{name} must be") as e:
        _call(**{name: t})
    assert e.value.status == dsa.DSA_ERR_INVALID_ARG


@pytest.mark.parametrize("kw,scale", [
    (dict(group=0), _zeros(ROWS, DIM // 128, dtype=torch.float32)),
    (dict(group=0), _zeros(ROWS - 1, dtype=torch.float32)),
    (dict(group=32, codes_dtype=dsa.DSA_MXFP8_E4M3), _zeros(ROWS, DIM // 128, dtype=torch.uint8)),
    (dict(group=32, codes_dtype=dsa.DSA_MXFP8_E4M3), _zeros(ROWS, DIM // 32, dtype=torch.float32)),
])
def test_scales_of_another_form_are_refused(kw, scale):
    with pytest.raises(dsa.DsaError, match="^scale must be"):
        _call(scale=scale, **kw)


def _passes(**kw):
    """The arrays are taken: the next refusal, of eps, answers."""
    with pytest.raises(dsa.DsaError, match="eps"):
        _call(eps=-1.0, **kw)


def test_arrays_that_are_taken():
    _passes()
    _passes(x=_wide(ROWS, DIM), out=_wide(ROWS, DIM))
    _passes(residual=None, sum=None, codes=None, scale=None)
    _passes(out=None)
    for scale in (_zeros(ROWS, dtype=torch.float32), _zeros(ROWS, 1, dtype=torch.float32)):
        _passes(scale=scale, group=0)
    for dtype in (torch.uint8, torch.float8_e8m0fnu):
        _passes(scale=_zeros(ROWS, DIM // 32, dtype=torch.uint8).view(dtype), group=32, codes_dtype=dsa.DSA_MXFP8_E4M3)
    _passes(codes=_zeros(ROWS, DIM, dtype=torch.uint8).view(torch.float8_e4m3fn))
    _passes(x=_zeros(ROWS, DIM, dtype=torch.int16))  # bf16 bits
    # buffers of more rows than there are
    _passes(residual=_zeros(ROWS + 1, DIM), sum=_zeros(ROWS + 2, DIM), codes=_zeros(ROWS + 1, DIM, dtype=torch.uint8),
            scale=_zeros(ROWS + 3, DIM // 128, dtype=torch.float32))
    _passes(scale=_zeros(ROWS + 3, dtype=torch.float32), group=0)
    # a single row's stride says nothing; bare addresses are taken as they are
    one = {n: _zeros(1, DIM) for n in ("out", "residual", "sum")}
    _passes(x=_zeros(DIM).as_strided((1, DIM), (0, 1)), codes=None, scale=None, **one)
    _passes(residual=0x10000, sum=0x20000, weight=0x30000, codes=0x40000, scale=0x50000)


def test_missing_arrays_are_refused_by_the_call():
    with pytest.raises(dsa.DsaError, match="weight is NULL"):
        _call(weight=None)
    with pytest.raises(dsa.DsaError, match="scale is NULL"):
        _call(scale=None)
