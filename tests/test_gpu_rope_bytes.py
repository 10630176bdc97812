"""The rotation of rope_append and rope_queries, bit for bit: the same rows give the same bytes as a cache row and as a
query, and those of elementary fp32 operations (each product rounded before the sum, IEEE divisions, one rounding at the
end), in every stored type."""
import pytest
import torch

import sparse_attention_dsa_gb300 as dsa

from _gpu import ensure_built
from _rope_prefix import KV, LATENT, PAGE, Batch, rope_table

pytestmark = pytest.mark.gpu

BF16, FP8, MX = dsa.DSA_BF16, dsa.DSA_FP8_E4M3, dsa.DSA_MXFP8_E4M3


@pytest.fixture(scope="module", autouse=True)
def _built():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    ensure_built()


def _rows(shape, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(shape, generator=g, device="cuda")
    x *= 2.0 ** torch.randint(-20, 21, (shape[0],) + (1,) * (len(shape) - 1), generator=g, device="cuda")
    x[..., 1::19] = 0.0
    x[..., 4::23] = -0.0
    return x.to(torch.bfloat16)


def _rotate(x, rows, pairing):
    """x [T, 64] by the table rows [T, 64], one fp32 operation after the other."""
    c, s, x = rows[:, :32], rows[:, 32:], x.float()
    a, b = (x[:, 0::2], x[:, 1::2]) if pairing == dsa.DSA_ROPE_INTERLEAVED else (x[:, :32], x[:, 32:])
    ac, bs, as_, bc = a * c, b * s, a * s, b * c
    y1, y2 = ac - bs, as_ + bc
    return torch.stack([y1, y2], dim=-1).flatten(-2) if pairing == dsa.DSA_ROPE_INTERLEAVED else torch.cat([y1, y2], dim=1)


def _stored(x, kind):
    """fp32 rows [T, Di] as they are stored: (bytes, scales)."""
    if kind == BF16:
        return x.to(torch.bfloat16).view(torch.uint8), None
    if kind == FP8:
        m = x.abs().amax(-1)
        scale = torch.where(m > 0, m / torch.full_like(m, 448.0), torch.ones_like(m))
        y = x / scale[:, None].expand_as(x).contiguous()
        return y.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8), scale
    g = x.unflatten(-1, (-1, 32))
    m = g.abs().amax(-1, keepdim=True)
    e = torch.where(m > 0, torch.frexp(m).exponent - 9, torch.zeros_like(m, dtype=torch.int32)).clamp(-127, 127)
    codes = torch.ldexp(g, -e).clamp(-448, 448).to(torch.float8_e4m3fn).flatten(-2).view(torch.uint8)
    return codes, (e.squeeze(-1) + 127).to(torch.uint8)


@pytest.mark.parametrize("pairing", [dsa.DSA_ROPE_HALVES, dsa.DSA_ROPE_INTERLEAVED])
@pytest.mark.parametrize("kind,di,begin", [(BF16, 128, 0), (BF16, 72, 8), (FP8, 128, 64), (FP8, 96, 16), (MX, 128, 0), (MX, 96, 32)])
def test_keys_and_queries_are_rotated_alike(kind, di, begin, pairing):
    b = Batch([6000, 300], [5900, 1], seed=50)
    table = rope_table(6000, "cuda")
    at = table[torch.tensor(b.pos, device="cuda")]
    x, kv = _rows((b.T, di), 51), _rows((b.T, KV), 52)
    rope = dsa.DsaRope(table=table.data_ptr(), table_len=6000, kv_pairing=pairing, idx_pairing=pairing, idx_begin=begin)
    d = b.dims(attn_heads=1, idx_heads=1, idx_dim=di, idx_dtype=kind)
    bytes_ = di * (2 if kind == BF16 else 1)
    k = torch.zeros((b.pages, PAGE, bytes_), dtype=torch.uint8, device="cuda")
    q_idx = torch.zeros((b.T, bytes_), dtype=torch.uint8, device="cuda")
    shape = {BF16: None, FP8: (), MX: (di // 32,)}[kind]
    dtype = torch.float32 if kind == FP8 else torch.uint8
    k_scale = None if kind == BF16 else torch.zeros((b.pages, PAGE, *shape), dtype=dtype, device="cuda")
    q_scale = None if kind == BF16 else torch.zeros((b.T, *shape), dtype=dtype, device="cuda")
    cache = torch.zeros((b.pages, PAGE, KV), dtype=torch.bfloat16, device="cuda")
    q = torch.zeros((b.T, 1, KV), dtype=torch.bfloat16, device="cuda")
    dsa.rope_append(d, rope, x, kv, b.pt, b.lens, b.cu, k, k_scale, cache, b.workspace)
    dsa.rope_queries(d, rope, kv[:, LATENT:].contiguous(), q, x, q_idx, q_scale, b.lens, b.cu, b.workspace)
    assert dsa.get_device_error(b.workspace) == 0
    turned = _rotate(kv[:, LATENT:], at, pairing).to(torch.bfloat16).view(torch.int16)
    assert torch.equal(cache.flatten(0, 1)[b.rows][:, LATENT:].view(torch.int16), turned)
    assert torch.equal(q[:, 0, LATENT:].view(torch.int16), turned)
    y = x.float()
    y[:, begin:begin + 64] = _rotate(x[:, begin:begin + 64], at, pairing)
    codes, scale = _stored(y, kind)
    assert torch.equal(k.flatten(0, 1)[b.rows], codes)
    assert torch.equal(q_idx, codes)
    if scale is not None:
        assert torch.equal(k_scale.flatten(0, 1)[b.rows], scale)
        assert torch.equal(q_scale, scale)


def test_queries_of_every_magnitude_are_quantised_like_keys():
    """From subnormal to the largest, with zeros of both signs, infinities and NaN (unrotated, so that they stay)."""
    b = Batch([4000], [4000], seed=53)
    x = torch.randn((b.T, 128), generator=torch.Generator(device="cuda").manual_seed(54), device="cuda")
    power = torch.randint(-133, 125, (b.T, 1), generator=torch.Generator().manual_seed(55)).cuda().float()
    power[:2000] = power[:2000] / 16
    x = x * torch.exp2(power)
    x[:, 5::64], x[:, 7::64] = 0.0, -0.0
    x[100:110, 9], x[105:115, 44] = float("inf"), float("nan")
    x = x.to(torch.bfloat16)
    table = rope_table(4000, "cuda")
    rope = dsa.DsaRope(table=table.data_ptr(), table_len=4000, kv_pairing=0, idx_pairing=0, idx_begin=-1)
    for kind, shape, dtype in ((FP8, (), torch.float32), (MX, (4,), torch.uint8)):
        d = b.dims(idx_heads=1, idx_dtype=kind)
        k, q = (torch.zeros((n, 128), dtype=torch.uint8, device="cuda") for n in (b.pages * PAGE, b.T))
        ks, qs = (torch.zeros((n, *shape), dtype=dtype, device="cuda") for n in (b.pages * PAGE, b.T))
        dsa.rope_append(d, rope, x, None, b.pt, b.lens, b.cu, k, ks, None, b.workspace)
        dsa.rope_queries(d, rope, None, None, x, q, qs, b.lens, b.cu, b.workspace)
        assert dsa.get_device_error(b.workspace) == 0
        assert torch.equal(k[b.rows], q)
        assert torch.equal(ks[b.rows].view(torch.uint8), qs.view(torch.uint8))
