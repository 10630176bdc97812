"""Expanded attention in 64 bits from the keys that the kernel stores (rounded to bf16; FP8 rows' elements to f16's 11 bits), so
that a score is known to its fp32 sums, however large it is; errors relative to the magnitudes that are summed, with no absolute
terms."""
from __future__ import annotations

import math

import torch

import sparse_attention_dsa_gb300 as dsa

from _latent import LATENT, NOPE, ROT, VALUE, sum_rounding
from _rope_prefix import PAGE, latent_values

BF16, F16 = 2.0 ** -8, 2.0 ** -11  # half a step


def rounded(x, bits):
    """x (float64) to so many significant bits, ties to even."""
    m, e = torch.frexp(x)
    return torch.ldexp(torch.round(torch.ldexp(m, torch.full_like(e, bits))), e - bits)


class Stored:
    def __init__(self, batch, q_nope, q_pe, w_kv, kv_cache, fp8, scale=(NOPE + ROT) ** -0.5, tokens=None):
        flat, heads, dev = kv_cache.reshape(-1, kv_cache.shape[-1]), q_nope.shape[1], q_nope.device
        self.out = torch.zeros((batch.T, heads, VALUE), dtype=torch.float64, device=dev)
        self.lse = torch.full((batch.T, heads), -math.inf, dtype=torch.float64, device=dev)
        self.dz = torch.zeros_like(self.lse)        # how far a visible score may be off
        self.weighted = torch.zeros_like(self.out)  # sum_s p_s |v_s|
        self.sums = torch.zeros_like(self.out)      # sum_s p_s times how far the fp32 sum of v_s may be off
        w, acc = w_kv.double(), 2 * sum_rounding(LATENT)
        for b in range(batch.B):
            t0, t1 = batch.cu_host[b], batch.cu_host[b + 1]
            if t0 == t1:
                continue
            at = torch.arange(batch.L[b])
            page = batch.pt_host[b, at // PAGE].long()
            r = latent_values(flat[(page * PAGE + at % PAGE).to(dev)], fp8)
            c, rot = r[:, :LATENT], r[:, LATENT:]
            if fp8:
                c = rounded(c, 11)
            exact, off = torch.einsum("sc,hdc->shd", c, w), acc * torch.einsum("sc,hdc->shd", c.abs(), w.abs())
            k = rounded(exact[..., :NOPE], 8)
            # a sum next to the middle of two bf16 values may be rounded to the other one
            flip = torch.maximum((rounded(exact[..., :NOPE] + off[..., :NOPE], 8) - k).abs(),
                                 (rounded(exact[..., :NOPE] - off[..., :NOPE], 8) - k).abs())
            v = exact[..., NOPE:]
            qn, qp = q_nope[t0:t1].double(), q_pe[t0:t1].double()
            z = (torch.einsum("thd,shd->ths", qn, k) + torch.einsum("thd,sd->ths", qp, rot)) * scale
            reach = torch.einsum("thd,shd->ths", qn.abs(), k.abs()) + torch.einsum("thd,sd->ths", qp.abs(), rot.abs())
            # (the scale times log2(e) in fp32: two roundings, and the exponent's own)
            dz = (torch.einsum("thd,shd->ths", qn.abs(), flip) + 2 * sum_rounding(NOPE + ROT) * reach) * scale
            dz = dz + 4 * 2.0 ** -24 * z.abs()
            limit = torch.arange(batch.L[b] - (t1 - t0), batch.L[b], device=dev)
            hidden = (at.to(dev)[None, :] > limit[:, None])[:, None, :].expand_as(z)
            z = z.masked_fill(hidden, -math.inf)
            p = torch.softmax(z, dim=-1)
            # a position without weight cannot change the result, however far its score is off
            dz = torch.where((p > 2.0 ** -60) & ~hidden, dz, torch.zeros_like(dz))
            self.lse[t0:t1] = torch.logsumexp(z, dim=-1)
            self.out[t0:t1] = torch.einsum("ths,shd->thd", p, v)
            self.weighted[t0:t1] = torch.einsum("ths,shd->thd", p, v.abs())
            self.sums[t0:t1] = torch.einsum("ths,shd->thd", p, off[..., NOPE:])
            self.dz[t0:t1] = dz.amax(-1)

    def check(self, out, lse, tokens=slice(None), half=F16):
        """Of an element: weights e^(2 dz) and their rounding (half a step), values' rounding, the output's, and the sums' 2^-16.
        Of the output's norm: a rounding to bf16 is 0.0017 of a value, root mean square, one to f16 0.0002.  The output's, and
        values' and weights' where nothing averages them out, are 0.0017 (f16) or 0.0029 (bf16); half as much again for a batch
        of few rows."""
        assert bool(out[tokens].isfinite().all())
        size, want = self.weighted[tokens], self.out[tokens]
        tol = (torch.expm1(2 * self.dz[tokens])[..., None] + 2 * half + 2.0 ** -16) * (1 + BF16) * size
        tol = tol + (1 + BF16) * self.sums[tokens] + BF16 * want.abs()
        err = (out[tokens].double() - want).abs()
        assert bool((err <= tol).all()), f"worst {(err / tol).max().item():.3g} of the bound"
        whole = (err.norm() / want.norm()).item()
        assert whole <= (2.6e-3 if half == F16 else 4.4e-3), f"relative error {whole:.3g}"
        if lse is not None:
            off = (lse[tokens].double() - self.lse[tokens]).abs()
            bound = self.dz[tokens] + 2.0 ** -18 + 2.0 ** -22 * self.lse[tokens].abs()
            assert bool((off <= bound).all()), f"lse off by {off.max().item():.3g}, {(off / bound).max().item():.3g} of its bound"


def check_call(c, tokens=slice(None), half=F16, heads=None):
    """A test_gpu_expanded.Call that has run, all its heads or some."""
    assert dsa.get_device_error(c.ws) == 0
    for one in [slice(None)] if heads is None else [slice(h, h + 1) for h in heads]:
        Stored(c.b, c.q_nope[:, one], c.q_pe[:, one], c.w[one], c.kv, c.fp8).check(
            c.out[:, one], None if c.lse is None else c.lse[:, one], tokens, half)
