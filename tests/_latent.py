"""Plain 64-bit forms of the norm, the per-head products and the expanded attention, with the sums that their tolerances are
made of (torch, float64, on any device)."""
from __future__ import annotations

import math

import torch

import sparse_attention_dsa_gb300 as dsa

from _rope_prefix import KV, LATENT, PAGE, latent_values

NOPE, ROT, VALUE = 128, 64, 128


def normal(shape, seed, std=1.0, device="cuda"):
    g = torch.Generator(device=device).manual_seed(seed)
    return (torch.randn(shape, generator=g, device=device) * std).to(torch.bfloat16)


def weights(heads, seed, device="cuda"):
    return normal((heads, NOPE + VALUE, LATENT), seed, LATENT ** -0.5, device)


def norm64(x, weight, eps, residual=None):
    h = x.double() + (0 if residual is None else residual.double())
    return h, h / torch.sqrt(h.square().mean(-1, keepdim=True) + eps) * weight.double()


# A normalised value: the sum of squares (a chain of at most 24 roundings) enters as its root, then the mean, the
# root and two products are rounded: fewer than 24 * 2^-24 altogether.
NORM_ROUNDING = 2.0 ** -19


def check_bf16(got, want, rounding=NORM_ROUNDING):
    err, tol = (got.double() - want).abs(), (2.0 ** -8 + 2 * rounding) * want.abs() + 1e-38
    assert bool((err <= tol).all()), f"worst {(err / tol).max().item():.3g} of the bound"


def check_codes(codes, scale, want, group, mx=False):
    """E4M3 codes and scales of rows against 64-bit values: codes within half a step (2^-4 relative, or 2^-10 of the scale),
    fp32 scales within the rounding of their maximum; MX scales exact but where the maximum is next to a power of two."""
    g = want.reshape(want.shape[0], -1, group)
    m = g.abs().amax(-1)
    if mx:
        e = torch.where(m > 0, torch.frexp(m).exponent - 9, torch.zeros_like(m, dtype=torch.int32)).clamp(-127, 127)
        step = scale.int() - 127 - e
        near = (m > 0) & ((torch.frexp(m).mantissa - 0.5 < 2.0 ** -18) | (1 - torch.frexp(m).mantissa < 2.0 ** -18))
        assert bool(((step == 0) | (near & (step.abs() == 1))).all())
        value = torch.exp2(scale.double() - 127).reshape(m.shape)[..., None]
    else:
        exact = torch.where(m > 0, m / 448, torch.ones_like(m))
        assert bool(((scale.reshape(m.shape).double() - exact).abs() <= 2 * NORM_ROUNDING * exact).all())
        value = scale.double().reshape(m.shape)[..., None]
    got = codes.view(torch.float8_e4m3fn).double().reshape(g.shape) * value
    tol = torch.maximum(2.0 ** -4 * g.abs(), 2.0 ** -10 * value) * (1 + 2.0 ** -16) + 2 * NORM_ROUNDING * g.abs()
    if mx:  # beyond 448 the code saturates
        tol = torch.where(g.abs() > 448 * value, g.abs() - 448 * value + 2.0 ** -16 * g.abs(), tol)
    assert bool(((got - g).abs() <= tol + 1e-38).all())


def sum_rounding(inner):
    """Products of bf16 are exact in fp32; 16 at a time are added to the accumulator: one rounding a step, and one step's
    alignment of 17 terms (fp32 alignment may truncate), each 2^-23 of the magnitudes summed."""
    return (inner / 16 + 17) * 2.0 ** -23


def check_product(got, x, w, equation):
    want, size = torch.einsum(equation, x, w), torch.einsum(equation, x.abs(), w.abs())
    tol = 2.0 ** -8 * want.abs() * (1 + 2.0 ** -8) + 2 * sum_rounding(x.shape[-1]) * size + 1e-38
    err = (got.double() - want).abs()
    assert bool((err <= tol).all()), f"worst {(err / tol).max().item():.3g} of the bound"


class Expanded:
    """Causal attention of a batch (a _rope_prefix.Batch) with expanded keys and values in 64 bits."""

    def __init__(self, batch, q_nope, q_pe, w_kv, kv_cache, fp8, scale=(NOPE + ROT) ** -0.5):
        flat, heads, dev = kv_cache.reshape(-1, kv_cache.shape[-1]), q_nope.shape[1], q_nope.device
        self.fp8 = fp8
        self.out = torch.zeros((batch.T, heads, VALUE), dtype=torch.float64, device=dev)
        self.lse = torch.full((batch.T, heads), -math.inf, dtype=torch.float64, device=dev)
        self.dz = torch.zeros_like(self.lse)  # how far a visible score may be off
        self.dv = torch.zeros_like(self.out)  # sum_s p_s times how far v_s may be off
        self.weighted = torch.zeros_like(self.out)  # sum_s p_s |v_s|
        w = w_kv.double()
        acc = 2 * sum_rounding(LATENT)
        # a key or value dim: the latent's rounding to f16 (FP8 rows; half a step of 2^-26 of numbers below 2^-16, which the
        # weights, exact from 2^-18 on and half a step of 2^-28 off below, are covered by), the sum's, its own rounding, a
        # key's to bf16, a value's to f16
        rows_off = (2.0 ** -11 if fp8 else 0.0) + acc
        for b in range(batch.B):
            t0, t1 = batch.cu_host[b], batch.cu_host[b + 1]
            if t0 == t1:
                continue
            at = torch.arange(batch.L[b])
            page = batch.pt_host[b, at // PAGE].long()
            r = latent_values(flat[(page * PAGE + at % PAGE).to(dev)], fp8)
            c, rot = r[:, :LATENT], r[:, LATENT:]
            k, size = torch.einsum("sc,hdc->shd", c, w), torch.einsum("sc,hdc->shd", c.abs(), w.abs())
            before = rows_off * size
            if fp8:
                before = before + 2.0 ** -27 * w.abs().sum(-1) + 2.0 ** -29 * c.abs().sum(-1)[:, None, None]
            off = 2.0 ** -8 * k.abs() * (1 + 2.0 ** -8) + (1 + 2.0 ** -8) * before
            off[..., NOPE:] = 2.0 ** -11 * k[..., NOPE:].abs() + (1 + 2.0 ** -8) * before[..., NOPE:] + 2.0 ** -27
            qn, qp = q_nope[t0:t1].double(), q_pe[t0:t1].double()
            z = (torch.einsum("thd,shd->ths", qn, k[..., :NOPE]) + torch.einsum("thd,sd->ths", qp, rot)) * scale
            dz = torch.einsum("thd,shd->ths", qn.abs(), off[..., :NOPE])
            reach = torch.einsum("thd,shd->ths", qn.abs(), k[..., :NOPE].abs()) + torch.einsum("thd,sd->ths", qp.abs(), rot.abs())
            dz = (dz + 2 * sum_rounding(NOPE + ROT) * reach) * scale
            limit = torch.arange(batch.L[b] - (t1 - t0), batch.L[b], device=dev)
            hidden = (at.to(dev)[None, :] > limit[:, None])[:, None, :].expand_as(z)
            z = z.masked_fill(hidden, -math.inf)
            p = torch.softmax(z, dim=-1)
            self.lse[t0:t1] = torch.logsumexp(z, dim=-1)
            self.out[t0:t1] = torch.einsum("ths,shd->thd", p, k[..., NOPE:])
            self.weighted[t0:t1] = torch.einsum("ths,shd->thd", p, k[..., NOPE:].abs())
            self.dv[t0:t1] = torch.einsum("ths,shd->thd", p, off[..., NOPE:])
            self.dz[t0:t1] = dz.masked_fill(hidden, 0).amax(-1)

    def check(self, out, lse, tokens=None, norm=True):
        """Weights: e^(2 dz), exp2 within 2^-22, f16 2^-11 and the sums' 2^-16; the output's own 2^-8.  norm: for standard normal
        data, where a rounding to bf16 is 0.0017 of a value, root mean square, each enters the output's norm by itself: the
        output's (0.0017) and the keys' through the scores (0.0014) make 0.0022, half as much again for a batch of few rows."""
        t = slice(None) if tokens is None else tokens
        rel = torch.expm1(2 * self.dz[t])[..., None] + 2.0 ** -11 + 2.0 ** -16
        tol = rel * (self.weighted[t] + self.dv[t]) + self.dv[t]
        tol = tol + 2.0 ** -8 * (self.out[t].abs() + tol) + 1e-30
        err = (out[t].double() - self.out[t]).abs()
        assert bool((err <= tol).all()), f"worst error {err.max().item():.3g}, {(err / tol).max().item():.3g} of its bound"
        size = self.out[t].norm()
        assert not norm or err.norm() <= 3.3e-3 * size, f"relative error {(err.norm() / size).item():.3g}"
        if lse is not None:
            off = (lse[t].double() - self.lse[t]).abs()
            bound = self.dz[t] + 2.0 ** -18 + 2.0 ** -22 * self.lse[t].abs()
            assert bool((off <= bound).all()), f"lse off by {off.max().item():.3g}"


def head_dims(tokens, heads, **kw):
    d = dict(batch=1, total_q=tokens, max_q_len=max(tokens, 1), num_pages=1, page_size=PAGE, max_pages_per_seq=1, idx_heads=64,
             idx_dim=128, idx_dtype=dsa.DSA_BF16, top_k=64, attn_heads=heads, kv_dim=KV, v_dim=LATENT,
             softmax_scale=(NOPE + ROT) ** -0.5, kv_dtype=dsa.DSA_BF16)
    d.update(kw)
    return dsa.DsaDims(**d)
