"""Plain 64-bit forms of the position rotation, the quantisations and the shared-prefix attention, and small
batches to run them on (torch, float64, on any device)."""
from __future__ import annotations

import math

import torch

import sparse_attention_dsa_gb300 as dsa

PAGE, KV, LATENT = 64, 576, 512


def rope_table(length, device="cpu", base=10000.0):
    """fp32 [length, 64]: 32 cosines and 32 sines a position."""
    a = torch.arange(length, dtype=torch.float64)[:, None] * base ** (-torch.arange(32, dtype=torch.float64) / 32)
    return torch.cat([a.cos(), a.sin()], dim=1).float().to(device)


def rotate(x, rows, interleaved):
    """x [T, ..., 64] (float64) by the table rows [T, 64] of its tokens."""
    rows = rows.double().reshape(rows.shape[0], *([1] * (x.dim() - 2)), 64)
    c, s = rows[..., :32], rows[..., 32:]
    a, b = (x[..., 0::2], x[..., 1::2]) if interleaved else (x[..., :32], x[..., 32:])
    y = torch.empty_like(x)
    if interleaved:
        y[..., 0::2], y[..., 1::2] = a * c - b * s, a * s + b * c
    else:
        y[..., :32], y[..., 32:] = a * c - b * s, a * s + b * c
    return y


class Batch:
    """Sequences with q_lens new tokens and seq_lens cached ones on shuffled pages, the first prefix positions
    shared.  `spare` pages beyond the ones in use."""

    def __init__(self, seq_lens, q_lens, prefix=0, seed=0, device="cuda", spare=1):
        g = torch.Generator().manual_seed(seed)
        self.n, self.L, self.prefix, self.device = list(q_lens), list(seq_lens), prefix, device
        self.B, self.T = len(self.n), sum(self.n)
        shared = prefix // PAGE
        need = [max(-(-l // PAGE), shared) for l in self.L]
        total = shared + sum(v - shared for v in need)
        ids = torch.randperm(total + spare, generator=g)
        pt = torch.full((self.B, max(max(need), 1)), -1, dtype=torch.int32)
        at = shared
        for b, v in enumerate(need):
            pt[b, :shared] = ids[:shared]
            pt[b, shared:v] = ids[at:at + v - shared]
            at += v - shared
        self.pages = total + spare
        self.pt_host = pt
        self.pt = pt.to(device)
        cu = [0]
        for v in self.n:
            cu.append(cu[-1] + v)
        self.cu_host = cu
        self.cu = torch.tensor(cu, dtype=torch.int32, device=device)
        self.lens = torch.tensor(self.L, dtype=torch.int32, device=device)
        self.seq = [b for b in range(self.B) for _ in range(self.n[b])]
        self.pos = [self.L[b] - self.n[b] + j for b in range(self.B) for j in range(self.n[b])]
        self.rows = torch.tensor([int(pt[b, p // PAGE]) * PAGE + p % PAGE for b, p in zip(self.seq, self.pos)],
                                 dtype=torch.int64, device=device)
        self.workspace = torch.zeros(256, dtype=torch.uint8, device=device)

    def dims(self, **kw):
        d = dict(batch=self.B, total_q=self.T, max_q_len=max(max(self.n), 1), num_pages=self.pages, page_size=PAGE,
                 max_pages_per_seq=self.pt.shape[1], idx_heads=64, idx_dim=128, idx_dtype=dsa.DSA_BF16, top_k=64,
                 attn_heads=128, kv_dim=KV, v_dim=LATENT, softmax_scale=KV ** -0.5, kv_dtype=dsa.DSA_BF16)
        d.update(kw)
        return dsa.DsaDims(**d)


def latent_values(rows, fp8):
    """float64 values of latent-KV rows ([N, 576] bf16, or [N, 656] bytes)."""
    if not fp8:
        return rows.double()
    codes = rows[:, :LATENT].contiguous().view(torch.float8_e4m3fn).double()
    scale = rows[:, LATENT:LATENT + 16].contiguous().view(torch.float32).double()
    rot = rows[:, LATENT + 16:].contiguous().view(torch.bfloat16).double()
    return torch.cat([codes * scale.repeat_interleave(128, dim=1), rot], dim=1)


def latent_fp8_rows(x):
    """bf16 rows [N, 576] in the FP8 row layout."""
    t = x[:, :LATENT].float().reshape(-1, 4, 128)
    m = t.abs().amax(-1, keepdim=True)
    scale = torch.where(m > 0, m / 448, torch.ones_like(m))
    codes = (t / scale).clamp(-448, 448).to(torch.float8_e4m3fn).reshape(-1, LATENT).view(torch.uint8)
    return torch.cat([codes, scale.reshape(-1, 4).contiguous().view(torch.uint8),
                      x[:, LATENT:].contiguous().view(torch.uint8)], dim=1)


class Attention:
    """Dense attention of a batch in 64 bits: out, lse, and per output the sums that its tolerance is made of."""

    def __init__(self, batch, q, kv_cache, fp8, scale=KV ** -0.5):
        flat = kv_cache.reshape(-1, kv_cache.shape[-1])
        H = q.shape[1]
        dev = q.device
        self.out = torch.zeros((batch.T, H, LATENT), dtype=torch.float64, device=dev)
        self.lse = torch.full((batch.T, H), -math.inf, dtype=torch.float64, device=dev)
        self.weighted = torch.zeros_like(self.out)  # sum_s p_s |v_s|
        self.reach = torch.zeros_like(self.lse)  # max_s scale * sum_d |q_d k_d|
        for b in range(batch.B):
            t0, t1 = batch.cu_host[b], batch.cu_host[b + 1]
            if t0 == t1:
                continue
            at = torch.arange(batch.L[b])
            src = torch.where(at < batch.prefix, 0, b)
            page = batch.pt_host[src, at // PAGE].long()
            r = latent_values(flat[(page * PAGE + at % PAGE).to(dev)], fp8)
            qd = q[t0:t1].double()
            z = torch.einsum("thd,sd->ths", qd, r) * scale
            size = torch.einsum("thd,sd->ths", qd.abs(), r.abs()) * scale
            limit = torch.arange(batch.L[b] - (t1 - t0), batch.L[b], device=dev)
            hidden = (at.to(dev)[None, :] > limit[:, None])[:, None, :].expand_as(z)
            z = z.masked_fill(hidden, -math.inf)
            w = torch.softmax(z, dim=-1)
            self.lse[t0:t1] = torch.logsumexp(z, dim=-1)
            self.out[t0:t1] = torch.einsum("ths,sd->thd", w, r[:, :LATENT])
            self.weighted[t0:t1] = torch.einsum("ths,sd->thd", w, r[:, :LATENT].abs())
            self.reach[t0:t1] = size.masked_fill(hidden, 0).amax(-1)

    def check(self, out, lse, fp8, tokens=None):
        """Roundings, each at most half a step (bf16 2^-8, fp32 2^-24 relative):
        * scores: products of bf16 are exact in fp32; 36 steps of 16 products are accumulated, each within
          (1 + 17) * 2^-23 of the magnitudes summed (fp32 alignment may truncate): dz <= 36 * 18 * 2^-23 * reach
          is the worst case, 2^-23 * 53 * reach that of one rounding a step and one group's alignment.
        * FP8 rows are multiplied as f16 (11 bits): their scale and its product with a code are each rounded by
          2^-11, so dz <= 2^-10 * reach.  (q, with 8 bits, is exact in f16.)
        * weights: exp2 within 2^-22 and their rounding, bf16 2^-8, with FP8 rows f16 2^-11; partial sums in fp32;
        * FP8 rows as values: 2^-10; the output's own rounding 2^-8 |out|."""
        t = slice(None) if tokens is None else tokens
        dz = self.reach[t] * (53 * 2.0 ** -23 + (2.0 ** -10 if fp8 else 0.0))
        rel = torch.expm1(2 * dz) + (2.0 ** -11 + 2.0 ** -10 if fp8 else 2.0 ** -8) + 2.0 ** -16
        tol = rel[..., None] * self.weighted[t] * (1 + 2.0 ** -7) + 2.0 ** -8 * self.out[t].abs() + 1e-30
        err = (out[t].double() - self.out[t]).abs()
        assert bool((err <= tol).all()), f"worst error {err.max().item():.3g}, {(err / tol).max().item():.3g} of its bound"
        norm = self.out[t].norm()
        assert (err.norm() <= (3e-3 if fp8 else 4e-3) * norm) or norm == 0, f"relative error {(err.norm() / norm).item():.3g}"
        if lse is not None:
            got = lse[t].double()
            finite = self.lse[t].isfinite()
            assert torch.equal(got.isfinite(), finite)
            bound = dz + 2.0 ** -18 + 2.0 ** -22 * self.lse[t].abs()
            off = (got - self.lse[t]).abs()[finite]
            assert bool((off <= bound[finite]).all()), f"lse off by {off.max().item():.3g}"
