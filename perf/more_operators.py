"""Cases of the normalisation and latent-attention operators: their inputs, their plain forms and their exact values.

Four operators around the attention of sparse_attention_dsa_gb300:

* ``norm``     - the residual's addition and the root-mean-square norm in front of a projection, as bf16 or as codes with
  scales: ``rms_norm``;
* ``absorb``   - the queries' unrotated part through each head's key weights, into the latent space that the paged rows
  live in: ``absorb_queries``;
* ``values``   - attention over latent rows through each head's value weights, back to head values: ``value_heads``;
* ``expanded`` - causal attention of prompts with keys and values of every head, made of the paged latent rows:
  ``expanded_attn``.

``run`` computes them in their plain form, or through the library where ``own`` is true.
"""
import math

import torch

own = False

PAGE, KV, LATENT, ROT = 64, 576, 512, 64  # page size, latent-KV row, its latent part, its rotary part
NOPE, VALUE = 128, 128  # a head's unrotated key dims and value dims
FP8_ROW = 656  # 512 codes, 4 fp32 scales, 64 bf16 rotary values
EPS = 1e-6


# ---------------------------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------------------------
def _norm(name, rows, dim, residual, form, wide=0):
    """form: bf16, row (codes, one scale a row), tile (a scale for 128), mx (E8M0 scales for 32), tile+bf16 (both);
    wide: columns of the array that x is a slice of, beyond its own."""
    return {"name": name, "op": "norm", "rows": rows, "dim": dim, "residual": residual, "form": form, "wide": wide}


def _product(name, op, tokens, heads):
    return {"name": name, "op": op, "tokens": tokens, "heads": heads}


def _expanded(name, batch, tokens, context, heads, kv):
    return {"name": name, "op": "expanded", "batch": batch, "tokens": tokens, "context": context, "heads": heads, "kv": kv}


def listed():
    return [
        # in front of a decode step's projections: nothing but latency
        _norm("norm_decode_32", 32, 4096, True, "bf16"),
        # the latent part of a chunk's new rows, slices of a projection's output, on their way to the cache
        _norm("norm_latent_rows", 4096, 512, False, "bf16", wide=64),
        # query latents of ragged prompts for a product in the microscaling format
        _norm("norm_prompts_mx", 1171, 1536, False, "mx"),
        # prefill chunks in front of an FP8 projection: bandwidth
        _norm("norm_chunk_fp8", 8192, 8192, True, "tile"),
        # the queries of the benchmark's decode step: every head's weights once
        _product("absorb_decode_32", "absorb", 32, 128),
        # a prefill chunk's queries for the sparse path: bandwidth
        _product("absorb_chunk_4096", "absorb", 4096, 128),
        # two tokens a sequence of a batch, heads split over devices
        _product("values_verify_130", "values", 130, 16),
        # an odd number of prompt tokens, every head
        _product("values_prompts_2111", "values", 2111, 128),
        # a few short prompts, heads split over devices: latency
        _expanded("expanded_short_16h", 3, 200, 333, 16, "bf16"),
        # ragged prompts, some behind cached tokens, over the quantised cache
        _expanded("expanded_prompts_fp8", 8, 1171, 1300, 32, "fp8"),
        # a chunk of a long prompt behind what earlier chunks left in the cache, heads split over devices
        _expanded("expanded_chunk_16h", 1, 4096, 16384, 16, "bf16"),
        # a long prompt, every head: matrix products
        _expanded("expanded_prompt_8192", 1, 8192, 8192, 128, "bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("norm", "absorb", "values", "expanded"))
    if op == "norm":
        form = rng.choice(("bf16", "row", "tile", "mx", "tile+bf16"))
        unit = {"bf16": 8, "row": 8, "tile": 128, "mx": 32, "tile+bf16": 128}[form]
        dim = rng.choice((512, 1536, 2048, 4096, 8192, unit * _log(rng, 1, 16384 // unit)))
        rows = max(1, min(_log(rng, 1, 16384), (1 << 26) // dim))
        c = _norm("", rows, dim, rng.random() < 0.5, form, wide=rng.choice((0, 64, 8 * _log(rng, 1, 100))))
    elif op in ("absorb", "values"):
        c = _product("", op, _log(rng, 1, 4096), rng.choice((1, 8, 16, 24, 32, 64, 128)))
    else:
        heads = rng.choice((1, 8, 16, 24, 32, 64, 128))
        tokens = _log(rng, 1, 4096)
        context = tokens + rng.choice((0, _log(rng, 1, 8192)))
        batch = max(1, min(_log(rng, 1, 32), 65536 // context, 2_000_000_000 // (tokens * context * heads)))
        c = _expanded("", batch, tokens, context, heads, rng.choice(("bf16", "fp8")))
    del c["name"]
    return c


def _lengths(case, low, high, salt):
    """One length a sequence, ragged in [low, high], the longest at high; the same for every seed of a case."""
    g = torch.Generator().manual_seed(1009 * case["batch"] + 31 * high + salt)
    n = torch.randint(low, high + 1, (case["batch"],), generator=g)
    n[int(torch.randint(0, case["batch"], (1,), generator=g))] = high
    return n


def _shape(case):
    """(n_b, L_b): query tokens and context of every sequence."""
    n = _lengths(case, (case["tokens"] + 1) // 2, case["tokens"], 1)
    return n, torch.maximum(_lengths(case, (case["context"] + 1) // 2, case["context"], 2), n)


def work(case):
    if case["op"] == "norm":
        n, d = case["rows"], case["dim"]
        made = {"bf16": 2, "row": 1 + 4 / d, "tile": 1 + 4 / 128, "mx": 1 + 1 / 32, "tile+bf16": 3 + 4 / 128}[case["form"]]
        return {"bytes": n * d * (2 + (4 if case["residual"] else 0) + made) + 2 * d, "flops": 5 * n * d}
    h = case["heads"]
    if case["op"] != "expanded":
        t = case["tokens"]
        return {"bytes": t * h * 2 * (NOPE + LATENT) + h * 2 * NOPE * LATENT, "flops": 2 * t * h * NOPE * LATENT}
    n, L = (v.tolist() for v in _shape(case))
    pairs = sum(a * b - a * (a - 1) // 2 for a, b in zip(n, L)) * h
    row = FP8_ROW if case["kv"] == "fp8" else 2 * KV
    return {"bytes": sum(L) * row + h * 2 * (NOPE + VALUE) * LATENT + sum(n) * h * 2 * (NOPE + ROT + VALUE),
            "flops": 2 * (NOPE + ROT + VALUE) * pairs + 2 * sum(L) * h * (NOPE + VALUE) * LATENT}


# ---------------------------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------------------------
def _fp8_rows(x):
    """Latent-KV rows [N, 576] (bf16) in the 656-byte row layout."""
    t = x[:, :LATENT].float().reshape(-1, 4, 128)
    scale = t.abs().amax(-1, keepdim=True) / 448
    codes = (t / scale).clamp(-448, 448).to(torch.float8_e4m3fn).reshape(-1, LATENT).view(torch.uint8)
    return torch.cat([codes, scale.reshape(-1, 4).contiguous().view(torch.uint8),
                      x[:, LATENT:].contiguous().view(torch.uint8)], dim=1)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))

    def normal(*shape, std=1.0):
        return (torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32) * std).to(torch.bfloat16)

    s = {"case": case}
    if case["op"] == "norm":
        n, d = case["rows"], case["dim"]
        s["x"] = normal(n, d + case["wide"])[:, :d]
        s["residual"] = normal(n, d, std=4.0) if case["residual"] else None
        s["sum"] = torch.zeros_like(s["residual"]) if case["residual"] else None
        s["weight"] = (1 + 0.1 * torch.randn(d, generator=gen, device="cuda")).to(torch.bfloat16)
        s["out"] = torch.zeros((n, d), dtype=torch.bfloat16, device="cuda") if "bf16" in case["form"] else None
        s["codes"] = None if case["form"] == "bf16" else torch.zeros((n, d), dtype=torch.uint8, device="cuda")
        s["scale"] = {"bf16": lambda: None, "row": lambda: torch.zeros((n, 1), device="cuda"),
                      "tile": lambda: torch.zeros((n, d // 128), device="cuda"),
                      "tile+bf16": lambda: torch.zeros((n, d // 128), device="cuda"),
                      "mx": lambda: torch.zeros((n, d // 32), dtype=torch.uint8, device="cuda")}[case["form"]]()
        return s
    h = case["heads"]
    s["w_kv"] = normal(h, NOPE + VALUE, LATENT, std=LATENT ** -0.5)
    if case["op"] == "expanded":
        n, L = _shape(case)
        T, B = int(n.sum()), case["batch"]
        cu = torch.zeros(B + 1, dtype=torch.int32)
        cu[1:] = n.cumsum(0)
        s |= {"cu": cu.cuda(), "lens": L.to(torch.int32).cuda(), "T": T, "most": int(n.max())}
        # what the plain form indexes by: each token's sequence, place among its queries, and position
        seq = torch.repeat_interleave(torch.arange(B), n)
        s["seq"] = seq.cuda()
        s["within"] = (torch.arange(T) - cu[seq].long()).cuda()
        s["pos"] = (L[seq] - n[seq]).cuda() + s["within"]
        need = (L + PAGE - 1) // PAGE
        pages = int(need.sum())
        ids = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
        column = torch.arange(int(need.max()))[None, :]
        number = torch.where(column < need[:, None], column + (need.cumsum(0) - need)[:, None], -1).cuda()
        s["pt"] = torch.where(number >= 0, ids[number.clamp(min=0)], -1).to(torch.int32)
        rows = normal(pages * PAGE, KV)
        s["kv_cache"] = (_fp8_rows(rows).view(pages, PAGE, FP8_ROW) if case["kv"] == "fp8"
                         else rows.view(pages, PAGE, KV))
        s["q"] = normal(T, h, NOPE + ROT)
        s["out"] = torch.zeros((T, h, VALUE), dtype=torch.bfloat16, device="cuda")
    else:
        T, B, pages = case["tokens"], 1, 1
        if case["op"] == "absorb":
            # the unrotated part of a projection's output, into the rows whose last dims hold the rotated part
            s["q"] = normal(T, h, NOPE + ROT)
            s["out"] = torch.zeros((T, h, KV), dtype=torch.bfloat16, device="cuda")
        else:
            s["latent"] = normal(T, h, LATENT)
            s["out"] = torch.zeros((T, h, VALUE), dtype=torch.bfloat16, device="cuda")
    if own:
        import sparse_attention_dsa_gb300 as dsa

        s["dims"] = dsa.DsaDims(batch=B, total_q=T, max_q_len=s.get("most", T), num_pages=pages, page_size=PAGE,
                                max_pages_per_seq=s["pt"].shape[1] if "pt" in s else 1, idx_heads=64, idx_dim=128,
                                idx_dtype=dsa.DSA_BF16, top_k=2048, attn_heads=h, kv_dim=KV, v_dim=LATENT,
                                softmax_scale=(NOPE + ROT) ** -0.5,
                                kv_dtype=dsa.DSA_FP8_E4M3 if case.get("kv") == "fp8" else dsa.DSA_BF16)
        s["pages"] = pages
        size = dsa.expanded_attn_workspace_size(s["dims"], pages) if case["op"] == "expanded" else 256
        s["workspace"] = torch.zeros(size, dtype=torch.uint8, device="cuda")
    return s


# ---------------------------------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------------------------------
def run(s):
    return {"norm": _run_norm, "absorb": _run_absorb, "values": _run_values, "expanded": _run_expanded}[s["case"]["op"]](s)


def _coded(y, form):
    """(codes, scales) of rows y: codes as E4M3 numbers, scales in fp32 or as E8M0 bytes."""
    if form == "mx":
        g = y.unflatten(-1, (-1, 32))
        m = g.abs().amax(-1, keepdim=True)
        e = torch.where(m > 0, torch.frexp(m).exponent - 9, torch.zeros_like(m, dtype=torch.int32)).clamp(-127, 127)
        return torch.ldexp(g, -e).clamp(-448, 448).to(torch.float8_e4m3fn).flatten(-2), (e.squeeze(-1) + 127).to(torch.uint8)
    g = y.unflatten(-1, (1, -1) if form == "row" else (-1, 128))
    m = g.abs().amax(-1, keepdim=True)
    scale = torch.where(m > 0, m / 448, torch.ones_like(m))
    return (g / scale).clamp(-448, 448).to(torch.float8_e4m3fn).flatten(-2), scale.squeeze(-1)


def _run_norm(s):
    case = s["case"]
    if own:
        import sparse_attention_dsa_gb300 as dsa

        group = {"bf16": 0, "row": 0, "tile": 128, "tile+bf16": 128, "mx": 32}[case["form"]]
        dsa.rms_norm(s["x"], s["weight"], EPS, out=s["out"], codes=s["codes"], scale=s["scale"],
                     codes_dtype=dsa.DSA_MXFP8_E4M3 if case["form"] == "mx" else dsa.DSA_FP8_E4M3, group=group,
                     residual=s["residual"], sum=s["sum"])
        codes = None if s["codes"] is None else s["codes"].view(torch.float8_e4m3fn)
        scale = s["scale"].view(torch.float8_e8m0fnu) if case["form"] == "mx" else s["scale"]
        return {"sum": s["sum"], "out": s["out"], "codes": codes, "scale": scale}
    x = s["x"].float()
    if s["residual"] is not None:
        x = x + s["residual"].float()
    total = x.to(torch.bfloat16) if s["residual"] is not None else None
    y = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * s["weight"].float()
    codes, scale = (None, None) if case["form"] == "bf16" else _coded(y, case["form"])
    if case["form"] == "mx":
        scale = scale.view(torch.float8_e8m0fnu)
    return {"sum": total, "out": y.to(torch.bfloat16) if s["out"] is not None else None, "codes": codes, "scale": scale}


def _run_absorb(s):
    if own:
        import sparse_attention_dsa_gb300 as dsa

        dsa.absorb_queries(s["dims"], s["q"], s["w_kv"], s["out"], s["workspace"],
                           q_nope_strides=(s["q"].stride(0), s["q"].stride(1)))
        return s["out"]
    q = s["q"][:, :, :NOPE].float().transpose(0, 1)
    s["out"][:, :, :LATENT] = torch.bmm(q, s["w_kv"][:, :NOPE].float()).transpose(0, 1).to(torch.bfloat16)
    return s["out"]


def _run_values(s):
    if own:
        import sparse_attention_dsa_gb300 as dsa

        dsa.value_heads(s["dims"], s["latent"], s["w_kv"], s["out"], s["workspace"])
        return s["out"]
    x = s["latent"].float().transpose(0, 1)
    return torch.bmm(x, s["w_kv"][:, NOPE:].float().transpose(1, 2)).transpose(0, 1).to(torch.bfloat16)


def _run_expanded(s):
    case = s["case"]
    if own:
        import sparse_attention_dsa_gb300 as dsa

        strides = (s["q"].stride(0), s["q"].stride(1))
        dsa.expanded_attn(s["dims"], s["pages"], s["q"], s["q"][:, :, NOPE:], s["w_kv"], s["kv_cache"], s["pt"], s["lens"],
                          s["cu"], s["out"], None, s["workspace"], q_nope_strides=strides, q_pe_strides=strides)
        return s["out"]
    B, H, T, n, m = case["batch"], case["heads"], s["T"], s["most"], case["context"]
    # every sequence's rows, padded to the longest context, in 32 bits
    at = torch.arange(m, device="cuda").expand(B, m)
    page = torch.gather(s["pt"], 1, at // PAGE).clamp(min=0).long()
    rows = s["kv_cache"].flatten(0, 1)[page * PAGE + at % PAGE]
    if case["kv"] == "fp8":
        latent = rows[..., :LATENT].view(torch.float8_e4m3fn).float().unflatten(-1, (4, 128))
        scale = rows[..., LATENT:LATENT + 16].contiguous().view(torch.float32)
        latent = (latent * scale[..., None]).flatten(-2)
        rotary = rows[..., LATENT + 16:].contiguous().view(torch.bfloat16).float()
    else:
        latent, rotary = rows[..., :LATENT].float(), rows[..., LATENT:].float()
    # keys and values of every head: [B, H, m, 128]
    both = (latent.reshape(B * m, LATENT) @ s["w_kv"].float().reshape(-1, LATENT).T).view(B, m, H, NOPE + VALUE)
    both = both.transpose(1, 2)
    k = torch.cat([both[..., :NOPE], rotary[:, None].expand(B, H, m, ROT)], dim=-1)
    q = torch.zeros((B, H, n, NOPE + ROT), device="cuda")
    q[s["seq"], :, s["within"]] = s["q"].float() * (NOPE + ROT) ** -0.5
    z = q @ k.transpose(-1, -2)
    limit = torch.zeros((B, n), dtype=torch.int64, device="cuda")
    limit[s["seq"], s["within"]] = s["pos"]
    z.masked_fill_((torch.arange(m, device="cuda")[None, None, :] > limit[:, :, None])[:, None], -math.inf)
    z = z.sub_(z.amax(-1, keepdim=True)).exp_()
    out = (z @ both[..., NOPE:]) / z.sum(-1, keepdim=True)
    return out[s["seq"], :, s["within"]].to(torch.bfloat16)


# ---------------------------------------------------------------------------------------------------------------
# the same from the definitions, in 64 bits
# ---------------------------------------------------------------------------------------------------------------
def _nearest_e4m3(x):
    """The E4M3 value next to x (ties to even): 3 bits behind the leading one, steps of 2^-9 below 2^-6, at most 448."""
    _, e = torch.frexp(x)
    step = torch.ldexp(torch.ones_like(x), (e - 4).clamp(min=-9))
    return (torch.round(x / step) * step).clamp(-448, 448)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        x = s["x"].double()
        if case["residual"]:
            x = x + s["residual"].double()
        y = x / torch.sqrt((x * x).sum(-1, keepdim=True) / case["dim"] + EPS) * s["weight"].double()
        found = {"sum": x if case["residual"] else None, "out": y if "bf16" in case["form"] else None, "codes": None,
                 "scale": None}
        if case["form"] != "bf16":
            group = {"row": case["dim"], "tile": 128, "tile+bf16": 128, "mx": 32}[case["form"]]
            g = y.reshape(case["rows"], -1, group)
            most = g.abs().amax(-1)
            scale = torch.pow(2.0, torch.floor(torch.log2(most)) - 8) if case["form"] == "mx" else most / 448
            found["codes"] = _nearest_e4m3(g / scale[..., None]).reshape(y.shape)
            found["scale"] = scale
        return found
    h = case["heads"]
    if case["op"] == "absorb":
        out = torch.zeros((case["tokens"], h, KV), dtype=torch.float64, device="cuda")
        out[..., :LATENT] = torch.einsum("thd,hdc->thc", s["q"][..., :NOPE].double(), s["w_kv"][:, :NOPE].double())
        return out
    if case["op"] == "values":
        return torch.einsum("thc,hdc->thd", s["latent"].double(), s["w_kv"][:, NOPE:].double())
    # attention, one sequence and head at a time over all its rows
    n, L = _shape(case)
    out = torch.empty((s["T"], h, VALUE), dtype=torch.float64, device="cuda")
    t0 = 0
    for b in range(case["batch"]):
        nb, lb = int(n[b]), int(L[b])
        at = torch.arange(lb, device="cuda")
        r = s["kv_cache"][s["pt"][b, at // PAGE].long(), at % PAGE]
        if case["kv"] == "fp8":
            codes = r[:, :LATENT].contiguous().view(torch.float8_e4m3fn).double()
            scale = r[:, LATENT:LATENT + 16].contiguous().view(torch.float32).double()
            r = torch.cat([codes * scale.repeat_interleave(128, dim=1),
                           r[:, LATENT + 16:].contiguous().view(torch.bfloat16).double()], dim=1)
        r = r.double()
        seen = at[None, :] <= (lb - nb + torch.arange(nb, device="cuda"))[:, None]
        for i in range(h):
            w = s["w_kv"][i].double()
            key = torch.cat([r[:, :LATENT] @ w[:NOPE].T, r[:, LATENT:]], dim=1)
            z = s["q"][t0:t0 + nb, i].double() @ key.T / math.sqrt(NOPE + ROT)
            z = torch.where(seen, z, torch.full_like(z, -math.inf))
            out[t0:t0 + nb, i] = torch.softmax(z, dim=-1) @ (r[:, :LATENT] @ w[NOPE:].T)
        t0 += nb
    return out
