"""Cases of the rotation and shared-prefix operators: their inputs, their plain forms and their exact values.

Three operators around the paged caches of sparse_attention_dsa_gb300:

* ``append``  - one step's new indexer keys and latent-KV rows go to the caches, rotated by their positions on the
  way (and quantised where the cache is): ``rope_append``;
* ``queries`` - the same rotation of the step's queries, and the quantisation of the indexer's: ``rope_queries``;
* ``attend``  - dense attention of a batch over the latent-KV cache whose sequences share a prefix: ``prefix_attn``.

``run`` computes them in their plain form, or through the library where ``own`` is true.
"""
import math

import torch

own = False

PAGE, KV, LATENT, ROT = 64, 576, 512, 64  # page size, latent-KV row, its latent part (also V), its rotary part
FP8_ROW = 656  # 512 codes, 4 fp32 scales, 64 bf16 rotary values


# ---------------------------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------------------------
def _append(name, batch, tokens, context, idx, kv, idx_dim=128, padded=False):
    return {"name": name, "op": "append", "batch": batch, "tokens": tokens, "context": context, "idx": idx, "kv": kv,
            "idx_dim": idx_dim, "padded": padded}


def _queries(name, batch, tokens, context, heads, idx_heads, idx_dim, idx):
    return {"name": name, "op": "queries", "batch": batch, "tokens": tokens, "context": context, "heads": heads,
            "idx_heads": idx_heads, "idx_dim": idx_dim, "idx": idx}


def _attend(name, batch, tokens, prefix, rest, heads, kv):
    return {"name": name, "op": "attend", "batch": batch, "tokens": tokens, "prefix": prefix, "rest": rest,
            "heads": heads, "kv": kv}


def listed():
    return [
        # a decode step of a few sequences: nothing but latency
        _append("append_decode_4", 4, 1, 1000, "bf16", "bf16"),
        # a speculative-verify step (two tokens a sequence) of a full batch, both caches quantised
        _append("append_verify_256_fp8", 256, 2, 900, "fp8", "fp8"),
        # ragged prompts, keys in the microscaling format; rows are slices of a wider projection
        _append("append_prompts_ragged_mx", 7, 1171, 1300, "mx", "fp8", padded=True),
        # prefill chunks of 4096 tokens of eight prompts: bandwidth
        _append("append_chunks_32k", 8, 4096, 4100, "bf16", "bf16"),
        # the queries of the benchmark's decode step
        _queries("queries_decode_32", 32, 1, 32768, 128, 64, 128, "bf16"),
        # two queries a sequence, the indexer's in FP8
        _queries("queries_verify_fp8", 8, 2, 131072, 128, 64, 128, "fp8"),
        # a prefill chunk: bandwidth
        _queries("queries_chunk_mx", 1, 4096, 65536, 128, 64, 128, "mx"),
        # a few short requests behind one short system prompt: latency
        _attend("attend_short_16h", 3, 1, 333, 70, 16, "bf16"),
        # decode of 32 requests behind one long document, all heads on this device
        _attend("attend_decode_128h", 32, 1, 16384, 1024, 128, "bf16"),
        # decode of 64 requests with the heads split over devices; the prefix ends inside a page
        _attend("attend_decode_16h", 64, 1, 32741, 500, 16, "bf16"),
        # the same over the quantised cache
        _attend("attend_decode_fp8", 32, 1, 16000, 700, 64, "fp8"),
        # prompts continued behind a shared prefix
        _attend("attend_prompts_32h", 8, 257, 4096, 300, 32, "bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("append", "queries", "attend"))
    if op == "append":
        tokens = rng.choice((1, 2, _log(rng, 3, 4096)))
        batch = max(1, min(_log(rng, 1, 256), 28000 // tokens))
        context = tokens + _log(rng, 1, 900)
        c = _append("", batch, tokens, context, rng.choice(("bf16", "fp8", "mx")), rng.choice(("bf16", "fp8")),
                    padded=rng.random() < 0.4)
        if c["idx"] == "bf16" and rng.random() < 0.3:
            c["idx_dim"] = 64
    elif op == "queries":
        tokens = rng.choice((1, 2, _log(rng, 3, 4096)))
        batch = max(1, min(_log(rng, 1, 256), 4096 // tokens))
        idx = rng.choice(("bf16", "fp8", "mx"))
        hi, di = (4, 64) if idx == "bf16" and rng.random() < 0.3 else (64, 128)
        c = _queries("", batch, tokens, tokens + _log(rng, 1, 131072), rng.choice((16, 32, 64, 96, 128)), hi, di, idx)
    else:
        heads = rng.choice((8, 16, 24, 32, 64, 128))
        tokens = rng.choice((1, 1, 2, _log(rng, 3, 300)))
        batch = max(1, min(_log(rng, 1, 64), 65536 // (tokens * heads)))
        prefix = rng.choice((0, _log(rng, 1, 32768), _log(rng, 64, 32768)))
        rest = tokens + _log(rng, 1, 2000)
        most = 215_000_000 // (batch * tokens * heads)  # (row, key) pairs: at most those of the largest listed case
        if prefix + rest > most:
            prefix = max(0, most - rest)
        c = _attend("", batch, tokens, prefix, min(rest, max(tokens, most)), heads, rng.choice(("bf16", "bf16", "fp8")))
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
    if case["tokens"] <= 2:
        n = torch.full((case["batch"],), case["tokens"])
    else:
        n = _lengths(case, (case["tokens"] + 1) // 2, case["tokens"], 1)
    if case["op"] == "attend":
        own_rows = torch.maximum(_lengths(case, 1, case["rest"], 2), n)
        return n, own_rows + case["prefix"]
    return n, torch.maximum(_lengths(case, 1, case["context"], 2), n)


def work(case):
    n, L = (v.tolist() for v in _shape(case))
    T = sum(n)
    if case["op"] == "append":
        di = case["idx_dim"]
        key = {"bf16": 2 * di, "fp8": di + 4, "mx": di + di // 32}[case["idx"]]
        row = FP8_ROW if case["kv"] == "fp8" else 2 * KV
        return {"bytes": T * (2 * di + 2 * KV + 4 * ROT + key + row), "flops": T * 2 * 3 * ROT}
    if case["op"] == "queries":
        hi, di, hq = case["idx_heads"], case["idx_dim"], case["heads"]
        code = {"bf16": 2 * di, "fp8": di + 4, "mx": di + di // 32}[case["idx"]]
        return {"bytes": T * (hq * 4 * ROT + hi * (2 * di + code) + 4 * ROT), "flops": T * 3 * ROT * (hq + hi)}
    pairs = sum(a * b - a * (a - 1) // 2 for a, b in zip(n, L)) * case["heads"]
    rows = case["prefix"] + sum(b - case["prefix"] for b in L)
    row = FP8_ROW if case["kv"] == "fp8" else 2 * KV
    lse = 0 if case["kv"] == "fp8" else 4
    return {"bytes": rows * row + T * case["heads"] * (2 * KV + 2 * LATENT + lse), "flops": 2 * (KV + LATENT) * pairs}


# ---------------------------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------------------------
def _table(length):
    """cos and sin of 32 angles for every position, base 10000, rounded to 32 bits."""
    inv = 10000.0 ** (-torch.arange(ROT // 2, dtype=torch.float64, device="cuda") / (ROT // 2))
    a = torch.arange(length, dtype=torch.float64, device="cuda")[:, None] * inv
    return torch.cat([a.cos(), a.sin()], dim=1).float()


def _pages(case, L, gen):
    """A page table of shuffled pages; with a prefix, every sequence's first pages are the same ones."""
    shared = case.get("prefix", 0) // PAGE
    need = (L + PAGE - 1) // PAGE
    rest = need - shared
    total = shared + int(rest.sum())
    ids = torch.randperm(total, generator=gen, device="cuda").to(torch.int32)
    column = torch.arange(int(need.max()))[None, :]
    number = torch.where(column < shared, column, column + (rest.cumsum(0) - rest)[:, None])
    pt = torch.where(column < need[:, None], number, -1).cuda()
    pt = torch.where(pt >= 0, ids[pt.clamp(min=0)], -1).to(torch.int32)
    return pt, total


def _fp8_rows(x):
    """Latent-KV rows [N, 576] (bf16) in the 656-byte row layout."""
    t = x[:, :LATENT].float().reshape(-1, 4, 128)
    scale = t.abs().amax(-1, keepdim=True) / 448
    codes = (t / scale).clamp(-448, 448).to(torch.float8_e4m3fn).reshape(-1, LATENT).view(torch.uint8)
    return torch.cat([codes, scale.reshape(-1, 4).contiguous().view(torch.uint8),
                      x[:, LATENT:].contiguous().view(torch.uint8)], dim=1)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(torch.bfloat16)

    n, L = _shape(case)
    T, B = int(n.sum()), case["batch"]
    cu = torch.zeros(B + 1, dtype=torch.int32)
    cu[1:] = n.cumsum(0)
    s = {"case": case, "cu": cu.cuda(), "lens": L.to(torch.int32).cuda(), "T": T, "most": int(n.max())}
    # what the plain form indexes by: each token's sequence and position
    seq = torch.repeat_interleave(torch.arange(B), n)
    s["pos"] = (L[seq] - n[seq] + torch.arange(T) - cu[seq].long()).cuda()
    s["seq"] = seq.cuda()
    s["within"] = (torch.arange(T) - cu[seq].long()).cuda()
    if case["op"] == "queries":
        s["table"] = _table(int(L.max()))
        s["q_pe"] = normal(T, case["heads"], ROT)
        s["q"] = normal(T, case["heads"], KV)
        s["q_idx_in"] = normal(T, case["idx_heads"], case["idx_dim"])
        shape = (T, case["idx_heads"], case["idx_dim"])
        s["q_idx"] = torch.zeros(shape, dtype=torch.bfloat16 if case["idx"] == "bf16" else torch.uint8, device="cuda")
        s["q_scale"] = {"bf16": None, "fp8": torch.zeros(shape[:2], device="cuda"),
                        "mx": torch.zeros((*shape[:2], shape[2] // 32), dtype=torch.uint8, device="cuda")}[case["idx"]]
        pages = 1
    else:
        s["pt"], pages = _pages(case, L, gen)
    if case["op"] == "append":
        di = case["idx_dim"]
        s["table"] = _table(int(L.max()))
        # rows of a wider projection's output where the case says so
        s["k_new"] = normal(T, di + 64)[:, :di] if case["padded"] else normal(T, di)
        s["kv_new"] = normal(T, KV + 128)[:, :KV] if case["padded"] else normal(T, KV)
        s["k_cache"] = torch.zeros((pages, PAGE, di), dtype=torch.bfloat16 if case["idx"] == "bf16" else torch.uint8,
                                   device="cuda")
        s["k_scale"] = {"bf16": None, "fp8": torch.zeros((pages, PAGE), device="cuda"),
                        "mx": torch.zeros((pages, PAGE, di // 32), dtype=torch.uint8, device="cuda")}[case["idx"]]
        s["kv_cache"] = (torch.zeros((pages, PAGE, FP8_ROW), dtype=torch.uint8, device="cuda") if case["kv"] == "fp8"
                         else torch.zeros((pages, PAGE, KV), dtype=torch.bfloat16, device="cuda"))
    if case["op"] == "attend":
        rows = normal(pages * PAGE, KV)
        if case["prefix"] % PAGE:  # the page in which the prefix ends is each sequence's own copy
            page = s["pt"][:, case["prefix"] // PAGE].long()
            copies = rows.view(pages, PAGE, KV)
            copies[page, :case["prefix"] % PAGE] = copies[page[0], :case["prefix"] % PAGE]
        s["kv_cache"] = (_fp8_rows(rows).view(pages, PAGE, FP8_ROW) if case["kv"] == "fp8"
                         else rows.view(pages, PAGE, KV))
        s["q"] = normal(T, case["heads"], KV)
        s["out"] = torch.zeros((T, case["heads"], LATENT), dtype=torch.bfloat16, device="cuda")
        # a program that only wants the attention's output asks for no log-sum-exp
        s["lse"] = None if case["kv"] == "fp8" else torch.zeros((T, case["heads"]), device="cuda")
    if own:
        import sparse_attention_dsa_gb300 as dsa

        idx = {"bf16": dsa.DSA_BF16, "fp8": dsa.DSA_FP8_E4M3, "mx": dsa.DSA_MXFP8_E4M3}[case.get("idx", "bf16")]
        s["dims"] = dsa.DsaDims(batch=B, total_q=T, max_q_len=s["most"], num_pages=pages, page_size=PAGE,
                                max_pages_per_seq=s["pt"].shape[1] if "pt" in s else 1,
                                idx_heads=case.get("idx_heads", 64), idx_dim=case.get("idx_dim", 128), idx_dtype=idx,
                                top_k=2048, attn_heads=case.get("heads", 128), kv_dim=KV, v_dim=LATENT,
                                softmax_scale=KV ** -0.5,
                                kv_dtype=dsa.DSA_FP8_E4M3 if case.get("kv") == "fp8" else dsa.DSA_BF16)
        if case["op"] == "attend":
            size = dsa.prefix_attn_workspace_size(s["dims"], case["prefix"])
        else:
            s["rope"] = dsa.DsaRope(table=s["table"].data_ptr(), table_len=s["table"].shape[0],
                                    kv_pairing=dsa.DSA_ROPE_INTERLEAVED, idx_pairing=dsa.DSA_ROPE_HALVES, idx_begin=0)
            size = 256
        s["workspace"] = torch.zeros(size, dtype=torch.uint8, device="cuda")
    return s


# ---------------------------------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------------------------------
def run(s):
    return {"append": _run_append, "queries": _run_queries, "attend": _run_attend}[s["case"]["op"]](s)


def _rotate(x, table, interleaved):
    """x [..., 64] rotated by the positions' angles: pairs (2i, 2i+1), or (i, i+32)."""
    c, z = table[..., :ROT // 2], table[..., ROT // 2:]
    if interleaved:
        a, b = x[..., 0::2], x[..., 1::2]
        return torch.stack([a * c - b * z, a * z + b * c], dim=-1).flatten(-2)
    a, b = x[..., :ROT // 2], x[..., ROT // 2:]
    return torch.cat([a * c - b * z, a * z + b * c], dim=-1)


def _e4m3(x):
    return x.clamp(-448, 448).to(torch.float8_e4m3fn)


def _row_scaled(x):
    """(codes, scale) of groups along the last dim, scale = absmax / 448 (1 for a group of zeros)."""
    m = x.abs().amax(-1, keepdim=True)
    scale = torch.where(m > 0, m / 448, torch.ones_like(m))
    return _e4m3(x / scale), scale.squeeze(-1)


def _microscaled(x):
    """(codes, E8M0 bytes) of groups of 32 along the last dim."""
    g = x.unflatten(-1, (-1, 32))
    m = g.abs().amax(-1, keepdim=True)
    e = torch.where(m > 0, torch.frexp(m).exponent - 9, torch.zeros_like(m, dtype=torch.int32)).clamp(-127, 127)
    return _e4m3(torch.ldexp(g, -e)).flatten(-2), (e.squeeze(-1) + 127).to(torch.uint8)


def _index_part(x, kind):
    """The indexer rows x as their cache holds them, and their scales."""
    if kind == "bf16":
        return x.to(torch.bfloat16), None
    codes, scale = _row_scaled(x) if kind == "fp8" else _microscaled(x)
    return codes.view(torch.uint8), scale


def _index_values(codes, scale, kind):
    """What an indexer array holds, as numbers."""
    if kind == "bf16":
        return [codes]
    return [codes.view(torch.float8_e4m3fn), scale if kind == "fp8" else scale.view(torch.float8_e8m0fnu)]


def _kv_values(cache, kind):
    if kind == "bf16":
        return [cache]
    return [cache[..., :LATENT].view(torch.float8_e4m3fn), cache[..., LATENT:LATENT + 16].view(torch.float32),
            cache[..., LATENT + 16:].view(torch.bfloat16)]


def _run_append(s):
    case = s["case"]
    if own:
        import sparse_attention_dsa_gb300 as dsa

        dsa.rope_append(s["dims"], s["rope"], s["k_new"], s["kv_new"], s["pt"], s["lens"], s["cu"], s["k_cache"],
                        s["k_scale"], s["kv_cache"], s["workspace"], k_stride=s["k_new"].stride(0),
                        kv_stride=s["kv_new"].stride(0))
    else:
        at = s["pt"][s["seq"], s["pos"] // PAGE].long() * PAGE + s["pos"] % PAGE
        angles = s["table"][s["pos"]]
        k = s["k_new"].float()
        k = torch.cat([_rotate(k[:, :ROT], angles, False), k[:, ROT:]], dim=1)
        codes, scale = _index_part(k, case["idx"])
        s["k_cache"].flatten(0, 1)[at] = codes
        if scale is not None:
            s["k_scale"].flatten(0, 1)[at] = scale
        kv = s["kv_new"].float()
        rot = _rotate(kv[:, LATENT:], angles, True).to(torch.bfloat16)
        rows = s["kv_cache"].flatten(0, 1)
        if case["kv"] == "fp8":
            codes, scale = _row_scaled(kv[:, :LATENT].unflatten(-1, (4, 128)))
            rows[at] = torch.cat([codes.flatten(-2).view(torch.uint8), scale.view(torch.uint8),
                                  rot.view(torch.uint8)], dim=1)
        else:
            rows[at] = torch.cat([s["kv_new"][:, :LATENT], rot], dim=1)
    return [*_index_values(s["k_cache"], s["k_scale"], case["idx"]), *_kv_values(s["kv_cache"], case["kv"])]


def _run_queries(s):
    case = s["case"]
    if own:
        import sparse_attention_dsa_gb300 as dsa

        dsa.rope_queries(s["dims"], s["rope"], s["q_pe"], s["q"], s["q_idx_in"], s["q_idx"], s["q_scale"], s["lens"],
                         s["cu"], s["workspace"])
    else:
        angles = s["table"][s["pos"]][:, None, :]
        s["q"][:, :, LATENT:] = _rotate(s["q_pe"].float(), angles, True).to(torch.bfloat16)
        x = s["q_idx_in"].float()
        x = torch.cat([_rotate(x[..., :ROT], angles, False), x[..., ROT:]], dim=-1)
        codes, scale = _index_part(x, case["idx"])
        s["q_idx"].copy_(codes)
        if scale is not None:
            s["q_scale"].copy_(scale)
    return [s["q"], *_index_values(s["q_idx"], s["q_scale"], case["idx"])]


def _rows(s, at):
    """Cache rows at flat row numbers, in 32 bits."""
    r = s["kv_cache"].flatten(0, 1)[at]
    if s["case"]["kv"] == "bf16":
        return r.float()
    latent = r[..., :LATENT].view(torch.float8_e4m3fn).float().unflatten(-1, (4, 128))
    scale = r[..., LATENT:LATENT + 16].contiguous().view(torch.float32)
    rot = r[..., LATENT + 16:].contiguous().view(torch.bfloat16).float()
    return torch.cat([(latent * scale[..., None]).flatten(-2), rot], dim=-1)


def _run_attend(s):
    case = s["case"]
    if own:
        import sparse_attention_dsa_gb300 as dsa

        dsa.prefix_attn(s["dims"], case["prefix"], s["q"], s["kv_cache"], s["pt"], s["lens"], s["cu"], s["out"],
                        s["lse"], s["workspace"])
        return [s["out"]] if s["lse"] is None else [s["out"], s["lse"]]
    B, H, P, T, n = case["batch"], case["heads"], case["prefix"], s["T"], s["most"]
    q = s["q"].float() * KV ** -0.5
    # the prefix: one matrix product of all the batch's rows with the rows that every sequence shares
    at = torch.arange(P, device="cuda")
    shared = _rows(s, s["pt"][0, at // PAGE].long() * PAGE + at % PAGE)
    z = q.reshape(T * H, KV) @ shared.T
    # each sequence's own rows, padded to the longest
    m = case["rest"]
    at = (P + torch.arange(m, device="cuda")).expand(B, m)
    page = torch.gather(s["pt"], 1, (at // PAGE).clamp(max=s["pt"].shape[1] - 1)).clamp(min=0).long()
    mine = _rows(s, page * PAGE + at % PAGE)
    padded = torch.zeros((B, n, H, KV), device="cuda")
    padded[s["seq"], s["within"]] = q
    y = torch.bmm(padded.view(B, n * H, KV), mine.transpose(1, 2)).view(B, n, H, m)[s["seq"], s["within"]]
    hidden = P + torch.arange(m, device="cuda")[None, :] > s["pos"][:, None]
    y.masked_fill_(hidden[:, None, :], -math.inf)
    y = y.view(T * H, m)
    top = y.amax(-1, keepdim=True)
    if P:
        top = torch.maximum(top, z.amax(-1, keepdim=True))
    z = z.sub_(top).exp_()
    y = y.sub_(top).exp_()
    total = z.sum(-1, keepdim=True) + y.sum(-1, keepdim=True)
    out = z @ shared[:, :LATENT]
    padded = torch.zeros((B, n, H, m), device="cuda")
    padded[s["seq"], s["within"]] = y.view(T, H, m)
    out = out.view(T, H, LATENT) + torch.bmm(padded.view(B, n * H, m), mine[:, :, :LATENT]).view(
        B, n, H, LATENT)[s["seq"], s["within"]]
    out = (out / total.view(T, H, 1)).to(torch.bfloat16)
    return [out] if s["lse"] is None else [out, (top + total.log()).view(T, H)]


# ---------------------------------------------------------------------------------------------------------------
# the same from the definitions, in 64 bits
# ---------------------------------------------------------------------------------------------------------------
def _turned(x, pos, pairs):
    """64-bit rotation of x [T, ..., 64]; pairs: the 32 index pairs."""
    first, second = pairs
    table = _table(int(pos.max()) + 1).double()[pos]
    shape = (len(pos),) + (1,) * (x.dim() - 2) + (ROT // 2,)
    c, z = table[:, :ROT // 2].reshape(shape), table[:, ROT // 2:].reshape(shape)
    y = torch.empty_like(x)
    y[..., first] = x[..., first] * c - x[..., second] * z
    y[..., second] = x[..., first] * z + x[..., second] * c
    return y


def _nearest_e4m3(x):
    """The E4M3 value next to x (ties to even): 3 bits behind the leading one, steps of 2^-9 below 2^-6, at most 448."""
    _, e = torch.frexp(x)
    step = torch.ldexp(torch.ones_like(x), (e - 4).clamp(min=-9))
    return (torch.round(x / step) * step).clamp(-448, 448)


def _index_exact(x, kind):
    if kind == "bf16":
        return [x]
    if kind == "fp8":
        scale = x.abs().amax(-1) / 448
        scale = torch.where(scale > 0, scale, torch.ones_like(scale))
        return [_nearest_e4m3(x / scale[..., None]), scale]
    g = x.reshape(*x.shape[:-1], x.shape[-1] // 32, 32)
    scale = torch.pow(2.0, torch.floor(torch.log2(g.abs().amax(-1))) - 8)
    return [_nearest_e4m3(g / scale[..., None]).reshape(x.shape), scale]


def exact(case, seed):
    s = prepare(case, seed)
    halves = (slice(0, 32), slice(32, 64))
    twos = (slice(0, 64, 2), slice(1, 64, 2))
    pos = s["pos"]
    if case["op"] == "queries":
        q = s["q"].double()
        q[..., LATENT:] = _turned(s["q_pe"].double(), pos, twos)
        x = s["q_idx_in"].double()
        x[..., :ROT] = _turned(x[..., :ROT].clone(), pos, halves)
        return [q, *_index_exact(x, case["idx"])]
    if case["op"] == "append":
        where = [s["pt"][s["seq"], pos // PAGE].long(), pos % PAGE]
        x = s["k_new"].double()
        x[:, :ROT] = _turned(x[:, :ROT].clone(), pos, halves)
        kv = s["kv_new"].double()
        rot = _turned(kv[:, LATENT:].clone(), pos, twos)
        pages = s["k_cache"].shape[0]
        found = []

        def put(rows, untouched=0.0):
            whole = torch.full((pages, PAGE, *rows.shape[1:]), untouched, dtype=torch.float64, device="cuda")
            whole[where[0], where[1]] = rows
            found.append(whole)

        for k, rows in enumerate(_index_exact(x, case["idx"])):
            put(rows, 2.0 ** -127 if case["idx"] == "mx" and k == 1 else 0.0)  # the scale byte 0 stands for 2^-127
        if case["kv"] == "bf16":
            put(torch.cat([kv[:, :LATENT], rot], dim=1))
        else:
            tiles = kv[:, :LATENT].reshape(-1, 4, 128)
            scale = tiles.abs().amax(-1) / 448
            put(_nearest_e4m3(tiles / scale[..., None]).reshape(-1, LATENT))
            put(scale)
            put(rot)
        return found
    # attention, one sequence at a time over all its rows
    n, L = _shape(case)
    out = torch.empty((s["T"], case["heads"], LATENT), dtype=torch.float64, device="cuda")
    lse = torch.empty((s["T"], case["heads"]), dtype=torch.float64, device="cuda")
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
        z = torch.einsum("thd,sd->ths", s["q"][t0:t0 + nb].double(), r) / math.sqrt(KV)
        seen = at[None, :] <= (lb - nb + torch.arange(nb, device="cuda"))[:, None]
        z = torch.where(seen[:, None, :], z, torch.full_like(z, -math.inf))
        lse[t0:t0 + nb] = torch.logsumexp(z, dim=-1)
        out[t0:t0 + nb] = torch.einsum("ths,sd->thd", torch.softmax(z, dim=-1), r[:, :LATENT])
        t0 += nb
    return [out] if s["lse"] is None else [out, lse]
