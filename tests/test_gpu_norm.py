"""The root-mean-square norm on the GPU against its formula in 64 bits (tolerances: _latent)."""
import pytest
import torch

import sparse_attention_dsa_gb300 as dsa

from _gpu import ensure_built
from _latent import check_bf16, check_codes, norm64, normal

pytestmark = pytest.mark.gpu

EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def _built():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    ensure_built()


def _rows(rows, dim, seed, wide=0):
    """Rows of magnitudes from 2^-6 to 2^6, as a slice of a wider array where `wide` says so."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    size = 2.0 ** torch.randint(-6, 7, (rows, 1), generator=g, device="cuda")
    x = torch.randn((rows, dim + wide), generator=g, device="cuda") * size
    return x.to(torch.bfloat16)[:, :dim]


def _weight(dim, seed):
    return (1 + 0.3 * torch.randn(dim, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda")).to(torch.bfloat16)


def _scale(rows, dim, form):
    if form == "mx":
        return torch.full((rows, dim // 32), 0x5A, dtype=torch.uint8, device="cuda")
    return torch.full((rows, dim // 128 if form == "tile" else 1), -7.0, device="cuda")


SIZES = [(1, 8), (3, 64), (5, 256), (9, 264), (2, 512), (4, 576), (7, 1024), (3, 1032), (2, 1536), (5, 4096), (3, 4104), (2, 7168),
         (3, 8192), (2, 16376), (2, 16384), (1025, 512), (301, 2048)]


@pytest.mark.parametrize("rows,dim", SIZES)
@pytest.mark.parametrize("residual", [False, True])
def test_bf16(rows, dim, residual):
    x, w = _rows(rows, dim, 1, wide=24 if rows % 2 else 0), _weight(dim, 2)
    res = _rows(rows, dim, 3) if residual else None
    total = torch.zeros((rows, dim), dtype=torch.bfloat16, device="cuda") if residual else None
    whole = torch.full((rows + 1, dim + 8), 7.0, dtype=torch.bfloat16, device="cuda")
    out = whole[:rows, :dim]
    before = x.clone(), None if res is None else res.clone()
    dsa.rms_norm(x, w, EPS, out=out, residual=res, sum=total)
    h, y = norm64(x, w, EPS, res)
    check_bf16(out, y)
    if residual:
        assert torch.equal(total, h.to(torch.float32).to(torch.bfloat16))  # h is exact in 64 bits, one rounding in 32
        assert torch.equal(res, before[1])
    assert torch.equal(x, before[0]) and bool((whole[rows:] == 7).all() and (whole[:, dim:] == 7).all())


@pytest.mark.parametrize("form,group", [("row", 0), ("tile", 128), ("mx", 32)])
@pytest.mark.parametrize("rows,dim", [(1, 128), (3, 256), (9, 512), (5, 640), (3, 1024), (3, 1152), (6, 1536), (3, 4096), (2, 8192),
                                      (2, 16384), (333, 2048)])
@pytest.mark.parametrize("both", [False, True])
def test_codes(form, group, rows, dim, both):
    x, w, res = _rows(rows, dim, 5, wide=64), _weight(dim, 6), _rows(rows, dim, 7) if both else None
    w[:128] = 0  # a tile of zeros: scale 1
    codes = torch.full((rows + 1, dim), 0x33, dtype=torch.uint8, device="cuda")
    scale = _scale(rows, dim, form)
    out = torch.zeros((rows, dim), dtype=torch.bfloat16, device="cuda") if both else None
    dsa.rms_norm(x, w, EPS, out=out, codes=codes, scale=scale, group=group, residual=res,
                 codes_dtype=dsa.DSA_MXFP8_E4M3 if form == "mx" else dsa.DSA_FP8_E4M3)
    _, y = norm64(x, w, EPS, res)
    check_codes(codes[:rows], scale, y, group or dim, form == "mx")
    assert bool((codes[rows:] == 0x33).all())
    if both:
        check_bf16(out, y)


@pytest.mark.parametrize("dim", [8, 24, 200])
def test_row_codes_of_odd_widths(dim):
    x, w = _rows(6, dim, 8), _weight(dim, 9)
    codes, scale = torch.zeros((6, dim), dtype=torch.uint8, device="cuda"), _scale(6, dim, "row")
    dsa.rms_norm(x, w, EPS, codes=codes, scale=scale)
    check_codes(codes, scale, norm64(x, w, EPS)[1], dim)


@pytest.mark.parametrize("dim", [576, 4096])
def test_in_place(dim):
    x, w, res = _rows(33, dim, 10), _weight(dim, 11), _rows(33, dim, 12)
    h, y = norm64(x, w, EPS, res)
    a, b = x.clone(), res.clone()  # the residual stream in place, the result in x
    dsa.rms_norm(a, w, EPS, out=a, residual=b, sum=b)
    check_bf16(a, y)
    assert torch.equal(b, h.to(torch.float32).to(torch.bfloat16))
    a, b = x.clone(), res.clone()  # the sum in x, the result in the residual
    dsa.rms_norm(a, w, EPS, out=b, residual=b, sum=a)
    check_bf16(b, y)
    assert torch.equal(a, h.to(torch.float32).to(torch.bfloat16))
    wide = torch.cat([x, x], dim=1)[:, :dim]  # a slice, in place
    dsa.rms_norm(wide, w, EPS, out=wide)
    check_bf16(wide, norm64(x, w, EPS)[1])


@pytest.mark.parametrize("dim", [512, 4096])
def test_zeros_infinities_and_nan(dim):
    x, w = _rows(6, dim, 13), _weight(dim, 14)
    x[1] = 0
    x[2, 5] = float("inf")
    x[3, 6] = float("nan")
    out = torch.zeros_like(x)
    codes, scale = torch.zeros(x.shape, dtype=torch.uint8, device="cuda"), _scale(6, dim, "tile")
    dsa.rms_norm(x, w, EPS, out=out, codes=codes, scale=scale, group=128)
    _, y = norm64(x, w, EPS)
    good = [0, 1, 4, 5]
    check_bf16(out[good], y[good])
    check_codes(codes[good], scale[good], y[good], 128)
    assert bool((out[1] == 0).all() and (scale[1] == 1).all())
    value = codes.view(torch.float8_e4m3fn).float()
    for got in (out.float(), value):
        assert bool(got[2, 5].isnan()) and bool((got[2, torch.arange(dim) != 5] == 0).all())  # x / inf, inf / inf
        assert bool(got[3].isnan().all())
    # eps alone keeps a row of tiny values finite; without it a row of zeros is 0 / 0
    tiny = (x * 2.0 ** -80)[4:]
    dsa.rms_norm(tiny, w, EPS, out=out[4:])
    check_bf16(out[4:], norm64(tiny, w, EPS)[1])
    dsa.rms_norm(x[1:2], w, 0.0, out=out[1:2])
    assert bool(out[1].isnan().all())


def test_many_long_rows_beyond_32_bits():
    """Element offsets that pass 2^31: the last rows are the ones of a short call."""
    rows, dim = 262200, 8192
    x = torch.zeros((rows, dim), dtype=torch.bfloat16, device="cuda")
    x[-3:] = normal((3, dim), 15)
    w, out = _weight(dim, 16), torch.zeros((rows, dim), dtype=torch.bfloat16, device="cuda")
    dsa.rms_norm(x, w, EPS, out=out)
    check_bf16(out[-3:], norm64(x[-3:], w, EPS)[1])
    assert bool((out[:: 65536][:-1] == 0).all())


def test_another_stream_and_a_graph():
    x, w, out = _rows(50, 4096, 17), _weight(4096, 18), torch.zeros((50, 4096), dtype=torch.bfloat16, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        dsa.rms_norm(x, w, EPS, out=out)
    side.synchronize()
    want = out.clone()
    check_bf16(want, norm64(x, w, EPS)[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dsa.rms_norm(x, w, EPS, out=out)
    x.copy_(_rows(50, 4096, 19))
    graph.replay()
    torch.cuda.synchronize()
    check_bf16(out, norm64(x, w, EPS)[1])
