"""rms_norm of rows whose squares leave fp32's range, large or small: the formula's values all the same."""
import pytest
import torch

import sparse_attention_dsa_gb300 as dsa

from _latent import check_bf16, check_codes, norm64, normal
from test_gpu_norm import _built, _scale, _weight  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu

DIMS = [8, 512, 1024, 4096, 16384]


@pytest.mark.parametrize("dim", DIMS)
@pytest.mark.parametrize("power", [50, 56, 60, 64, 90, 120])
@pytest.mark.parametrize("eps", [0.0, 1e-6, 1e30])
def test_large_rows(dim, power, eps):
    x, res, w = normal((5, dim), 501), normal((5, dim), 502), _weight(dim, 503)
    x, res = x * 2.0 ** power, res * 2.0 ** power  # (powers of two: still bf16)
    x[2], res[2] = 0, 0.5  # an ordinary row, and one with a single large element, between them
    x[3], res[3] = 1.0, 0.0
    x[3, 5] = 2.0 ** (power + 3)
    out, total = torch.zeros_like(x), torch.zeros_like(x)
    dsa.rms_norm(x, w, eps, out=out, residual=res, sum=total)
    h, y = norm64(x, w, eps, res)
    check_bf16(out, y)
    assert torch.equal(total, (x.float() + res.float()).to(torch.bfloat16))


@pytest.mark.parametrize("dim", DIMS)
@pytest.mark.parametrize("power", [45, 60, 64, 70, 100, 125])
@pytest.mark.parametrize("eps", [0.0, 1e-45, 1e-38, 1e-20])
def test_small_rows(dim, power, eps):
    """Down to bf16's subnormal numbers; an eps of 1e-45 is the smallest fp32 number."""
    x, w = (normal((5, dim), 504).float() * 2.0 ** -power).to(torch.bfloat16), _weight(dim, 505)
    x[3] = 1.0
    out = torch.zeros_like(x)
    dsa.rms_norm(x, w, eps, out=out)
    check_bf16(out, norm64(x, w, torch.tensor(eps, dtype=torch.float32).double().item())[1])


@pytest.mark.parametrize("form,group", [("row", 0), ("tile", 128), ("mx", 32)])
@pytest.mark.parametrize("dim", [512, 1024, 4096, 16384])
@pytest.mark.parametrize("power", [100, -100])
def test_codes(form, group, dim, power):
    x, w = (normal((5, dim), 506).float() * 2.0 ** power).to(torch.bfloat16), _weight(dim, 507)
    x[1] = 1.0
    codes, scale = torch.zeros((5, dim), dtype=torch.uint8, device="cuda"), _scale(5, dim, form)
    dsa.rms_norm(x, w, 0.0, codes=codes, scale=scale, group=group,
                 codes_dtype=dsa.DSA_MXFP8_E4M3 if form == "mx" else dsa.DSA_FP8_E4M3)
    check_codes(codes, scale, norm64(x, w, 0.0)[1], group or dim, form == "mx")
