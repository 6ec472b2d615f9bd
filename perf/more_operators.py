"""Timing cases of the operators that take many tokens at once through a decoder layer: the cache
append with a norm of every query and key head, the attention of a chunk of new tokens over the
paged cache, and the product of rows with a packed blob and its epilogue.

``run`` computes them in plain torch operations, or, with ``own`` set, through the library's
entry points.  Shapes are the 7B / 8B decoder shapes of the benchmark (32 query heads of 128, 32
or 8 key heads, widths 4096 and 11008) and generic ones; values are synthetic.
"""

import math

import torch

own = False

TYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16,
         "e4m3": torch.float8_e4m3fn}
BYTES = {"fp32": 4, "fp16": 2, "bf16": 2, "e4m3": 1}
E4M3_MAX = 448.0
INT4_GROUP = 128


# ------------------------------------------------------------------ cases

def _append(name, tokens, kind, heads, kv_heads, dim, rot, pairs, page, src, cache, far, norm,
            weights):
    return dict(name=name, op="append", tokens=tokens, kind=kind, heads=heads, kv_heads=kv_heads,
                dim=dim, rot=rot, pairs=pairs, page=page, src=src, cache=cache, far=far,
                norm=norm, weights=weights)


def _chunk(name, seqs, new, before, lens, heads, kv_heads, dim, page, q, cache, window, order):
    return dict(name=name, op="chunk", seqs=seqs, new=new, before=before, lens=lens, heads=heads,
                kv_heads=kv_heads, dim=dim, page=page, q=q, cache=cache, window=window,
                order=order)


def _gemm(name, rows, d_in, d_out, mats, fmt, form, act, bias, res, out, scale):
    return dict(name=name, op="gemm", rows=rows, d_in=d_in, d_out=d_out, mats=mats, fmt=fmt,
                form=form, act=act, bias=bias, res=res, out=out, scale=scale)


def listed():
    return [
        # one user's next token in a layer whose queries and keys are normed
        _append("normed append 1 token 7b", 1, "decode", 32, 32, 128, 128, "halves", 16, "fp32",
                "fp16", 4096, "rms", "shared"),
        # prompts of three users written at once, half of each head rotated, into an 8-bit cache
        _append("normed append prompts e4m3", 4099, "prompt", 32, 8, 128, 64, "neighbours", 32,
                "fp16", "e4m3", 8192, "rms", "shared"),
        # layer norms with a weight for each head, heads of an odd number of 16-byte pieces
        _append("normed append 997 x 96 layer", 997, "prompt", 20, 4, 96, 96, "halves", 64,
                "bf16", "bf16", 131072, "layer", "own"),
        # a few drafted tokens of one user checked at once against a long conversation
        _chunk("chunk 1 x 5 over 8192 8b", 1, 5, 8192, "even", 32, 8, 128, 16, "fp16", "fp16", 0,
               "heads"),
        # the first prompt of a chat, nothing cached before it
        _chunk("chunk 1 x 509 7b", 1, 509, 0, "even", 32, 32, 128, 16, "fp16", "fp16", 0,
               "heads"),
        # a serving batch: prompts in chunks beside users who decode, rows of a token together
        _chunk("chunk 24 mixed 8b", 24, 512, 4096, "mixed", 32, 8, 128, 64, "bf16", "bf16", 0,
               "tokens"),
        # a whole long prompt
        _chunk("chunk 1 x 8192 8b", 1, 8192, 0, "even", 32, 8, 128, 32, "fp16", "fp16", 0,
               "heads"),
        # chunks of eight long documents over an 8-bit cache
        _chunk("chunk 8 x 512 over 15872 e4m3", 8, 512, 15872, "even", 32, 8, 128, 32, "fp16",
               "e4m3", 0, "heads"),
        # q|k|v of the drafted tokens
        _gemm("gemm 5 x 4096 qkv", 5, 4096, 4096, 3, "fp16", "plain", "silu", False, "none",
              "fp16", 1.0),
        # the down projection of a small batch from a 4-bit base, added to the stream
        _gemm("gemm 61 x 11008 int4", 61, 11008, 4096, 1, "int4", "plain", "silu", False, "fp16",
              "fp16", 1.0),
        # odd sizes with a bias and an activation
        _gemm("gemm 333 x 5003 gelu", 333, 5003, 1344, 1, "fp16", "act", "gelu", True, "fp32",
              "fp32", 0.5),
        # the largest: gate|up of a long prompt
        _gemm("gemm 4096 x 4096 gate up", 4096, 4096, 11008, 2, "fp16", "gated", "silu", False,
              "none", "fp16", 1.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "chunk", "chunk", "chunk", "gemm", "gemm", "gemm"])
    if op == "append":
        kv = rng.choice([1, 2, 4, 8, 32])
        group = rng.choice([1, 4, 5, 8]) if kv < 32 else 1
        dim = rng.choice([64, 96, 128, 192, 256])
        src = rng.choice(["fp32", "fp16", "bf16"])
        low = "fp16" if src == "fp32" else src
        kind = rng.choice(["decode", "prompt"])
        c = _append("", _log(rng, 1, 300) if kind == "decode" else _log(rng, 2, 4000), kind,
                    kv * group, kv, dim, rng.choice([dim, dim, dim // 2, 0]),
                    rng.choice(["halves", "neighbours"]), rng.choice([8, 16, 32, 64, 256]), src,
                    rng.choice([low, low, "e4m3"]), _log(rng, 4096, 1000000),
                    rng.choice(["rms", "rms", "layer"]), rng.choice(["shared", "shared", "own"]))
    elif op == "chunk":
        kv = rng.choice([1, 2, 4, 8, 32])
        group = rng.choice([1, 4, 5, 8, 16, 20]) if kv < 32 else 1
        dim = rng.choice([64, 96, 128, 128, 192, 256])
        q = rng.choice(["fp16", "bf16"])
        seqs, heads = _log(rng, 1, 64), kv * group
        # (rows x keys x heads of the padded plain form stay below the largest listed case's)
        new = _log(rng, 1, max(1, min(4096, 2 ** 24 // (seqs * heads))))
        most = max(64, min(65536, 2 ** 30 // (seqs * heads * new), 2 ** 29 // (seqs * kv * dim)))
        c = _chunk("", seqs, new, rng.choice([0, _log(rng, 1, most)]),
                   rng.choice(["even", "mixed"]), heads, kv, dim, rng.choice([8, 16, 32, 64, 256]),
                   q, rng.choice([q, q, "e4m3"]), rng.choice([0, 0, 0, 1, 100, 1000]),
                   rng.choice(["heads", "tokens"]))
    else:
        fmt = rng.choice(["fp16", "fp16", "int4"])
        form = rng.choice(["plain", "plain", "act", "gated"])
        mats = 2 if form == "gated" else rng.choice([1, 1, 2, 3])
        unit = 128 if fmt == "int4" else 64
        c = _gemm("", _log(rng, 1, 4096), _log(rng, 64, 11008),
                  unit * _log(rng, 1, 11008 // unit), mats, fmt, form,
                  rng.choice(["silu", "gelu"]), rng.choice([True, False]),
                  rng.choice(["none", "fp32", "fp16", "bf16"]),
                  rng.choice(["fp16", "bf16"] if fmt == "int4" else ["fp32", "fp16", "bf16"]),
                  rng.choice([1.0, 1.0, 0.5]))
        while c["rows"] * c["d_in"] * c["d_out"] * mats > 2 ** 37:
            c["rows"] = max(1, c["rows"] // 2)
    del c["name"]
    return c


# ------------------------------------------------------------------ inputs

def _rng(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, shape, dtype, scale=1.0):
    out = torch.empty(shape, dtype=dtype, device="cuda")
    flat = out.view(-1)
    for at in range(0, flat.numel(), 1 << 27):
        part = flat[at:at + (1 << 27)]
        v = torch.randn(part.numel(), generator=g, device="cuda", dtype=torch.float32)
        part.copy_(v.mul_(scale))
    return out


def _segments(c):
    """Prompt cases of the append: (first position, tokens) of up to three sequences."""
    n = c["tokens"]
    cut = [n] if n < 3 else [n // 2, n // 3, n - n // 2 - n // 3]
    return [(min(17 * i, max(0, c["far"] - k)), k) for i, k in enumerate(cut)]


def _spread(i, n, most):
    """The i-th of n lengths from 1 to most, evenly over their logarithm."""
    return max(1, round(most ** (i / max(1, n - 1)))) if most else 0


def _chunks(c):
    """(new tokens, tokens before them) of each sequence (the order is drawn in prepare)."""
    n = c["seqs"]
    if c["lens"] == "even" or n < 3:
        return [(c["new"], c["before"])] * n
    # users who decode, prompts of all lengths, one without new tokens; long and short contexts
    # fall on both
    return [(0, c["before"])] + [(1 if i % 2 else _spread(i, n, c["new"]),
                                  _spread((7 * i) % n, n, c["before"])) for i in range(1, n)]


def _prepare_append(c, g):
    src, cache = TYPES[c["src"]], TYPES[c["cache"]]
    low = torch.float16 if c["src"] == "fp32" else src
    n, hq, hk, dim, page = c["tokens"], c["heads"], c["kv_heads"], c["dim"], c["page"]
    if c["kind"] == "decode":
        positions = torch.randint(0, c["far"], (n,), generator=g, device="cuda",
                                  dtype=torch.int32)
        seq = torch.arange(n, device="cuda", dtype=torch.int32)
        seqs = n
    else:
        parts = _segments(c)
        seqs = len(parts)
        positions = torch.cat([torch.arange(a, a + k, device="cuda", dtype=torch.int32)
                               for a, k in parts])
        seq = torch.cat([torch.full((k,), i, device="cuda", dtype=torch.int32)
                         for i, (a, k) in enumerate(parts)])
    # the pool holds the pages that the tokens land on and a few that stay as they are
    at = seq.long() * (1 << 20) + (positions // page).long()
    used, where = torch.unique(at, return_inverse=True)
    pages = used.numel() + 5
    order = torch.randperm(pages, generator=g, device="cuda")
    table = torch.full((seqs, (c["far"] + page - 1) // page), -1, dtype=torch.int32,
                       device="cuda")
    table[seq.long(), (positions // page).long()] = order[where].int()
    if c["kind"] == "decode" and n > 8:
        positions[torch.randint(0, n, (n // 8,), generator=g, device="cuda")] = -1  # padding
    row = _randn(g, (n, (hq + 2 * hk) * dim), src, 1.5)
    layer, each = c["norm"] == "layer", c["weights"] == "own"

    def weight(heads, mean):
        shape = (heads, dim) if each else (dim,)
        return mean + _randn(g, shape, torch.float32, 0.2)

    s = dict(c=c, seq=seq, positions=positions, table=table, eps=1e-6,
             q=row[:, :hq * dim].view(n, hq, dim),
             k=row[:, hq * dim:(hq + hk) * dim].view(n, hk, dim),
             v=row[:, (hq + hk) * dim:].view(n, hk, dim),
             kc=_randn(g, (pages, hk, page, dim), cache),
             vc=_randn(g, (pages, hk, page, dim), cache),
             q_out=torch.empty((n, hq, dim), dtype=low, device="cuda"),
             inv=(1e4 ** (-torch.arange(0, c["rot"], 2, dtype=torch.float64, device="cuda")
                          / max(1, c["rot"]))).float(),
             qw=weight(hq, 1.0), kw=weight(hk, 1.0), qb=weight(hq, 0.0) if layer else None,
             kb=weight(hk, 0.0) if layer else None, ks=None, vs=None)
    if c["cache"] == "e4m3":
        s["ks"] = torch.rand(hk, generator=g, device="cuda") * 0.05 + 0.01
        s["vs"] = torch.rand(hk, generator=g, device="cuda") * 0.05 + 0.01
    if own:
        import activation_sparse_tiered_amd as spax
        s["cache"] = spax.make_kv_cache(s["kc"], s["vc"], table, k_scale=s["ks"],
                                        v_scale=s["vs"])
        s["plan"] = spax.make_kv_append(s["cache"], s["q"], s["k"], s["v"], positions, s["q_out"],
                                        seq=None if c["kind"] == "decode" else seq,
                                        inv_freq=s["inv"] if c["rot"] else None,
                                        interleaved=c["pairs"] == "neighbours")
        s["norm"] = spax.make_head_norm(s["qw"], s["kw"], q_bias=s["qb"], k_bias=s["kb"],
                                        kind=c["norm"], eps=s["eps"])
    return s


def _prepare_chunk(c, g):
    hq, hk, dim, page, n = c["heads"], c["kv_heads"], c["dim"], c["page"], c["seqs"]
    q_type, cache = TYPES[c["q"]], TYPES[c["cache"]]
    sizes = torch.tensor(_chunks(c), dtype=torch.int32, device="cuda")
    sizes = sizes[torch.randperm(n, generator=g, device="cuda")]
    new, lens = sizes[:, 0], sizes.sum(1, dtype=torch.int32).contiguous()
    starts = torch.zeros(n + 1, dtype=torch.int32, device="cuda")
    starts[1:] = new.cumsum(0, dtype=torch.int32)
    longest = max(a + b for a, b in _chunks(c))
    # a mixed batch has a few rows behind its last sequence
    rows = sum(a for a, b in _chunks(c)) + (3 if c["lens"] == "mixed" else 0)
    need = (lens + page - 1) // page
    width = max(1, (longest + page - 1) // page)
    pages = int(need.sum()) + 3
    held = torch.arange(width, device="cuda")[None, :] < need[:, None]
    table = torch.full((n, width), -1, dtype=torch.int32, device="cuda")
    table[held] = torch.randperm(pages, generator=g, device="cuda")[:pages - 3].int()
    shape = (pages, hk, page, dim) if c["order"] == "heads" else (pages, page, hk, dim)
    s = dict(c=c, lens=lens, starts=starts, table=table, ks=None, vs=None, longest=longest,
             most_new=max(a for a, b in _chunks(c)),
             q=_randn(g, (rows, hq, dim), q_type), kc=_randn(g, shape, cache),
             vc=_randn(g, shape, cache),
             out=torch.zeros((rows, hq, dim), dtype=q_type, device="cuda"),
             lse=torch.zeros((rows, hq), dtype=torch.float32, device="cuda"), scale=dim ** -0.5)
    if c["order"] == "tokens":
        s["kc"], s["vc"] = s["kc"].transpose(1, 2), s["vc"].transpose(1, 2)
    # a cache holds whatever was left in rows that no sequence has reached yet
    last = (lens - 1).clamp(min=0).long()
    ends = (lens > 0) & (lens % page != 0)
    tail_page = table[torch.arange(n, device="cuda"), last // page][ends].long()
    s["vc"][tail_page, :, page - 1] = math.nan
    if c["cache"] == "e4m3":
        s["ks"] = torch.rand(hk, generator=g, device="cuda") * 0.5 + 0.5
        s["vs"] = torch.rand(hk, generator=g, device="cuda") * 0.5 + 0.5
    if own:
        import activation_sparse_tiered_amd as spax
        s["cache"] = spax.make_kv_cache(s["kc"], s["vc"], table, k_scale=s["ks"],
                                        v_scale=s["vs"])
        s["plan"] = spax.make_chunk_attention(s["cache"], s["q"], starts, lens, s["out"],
                                              max_len=longest, scale=s["scale"],
                                              window=c["window"], lse=s["lse"])
        s["ws"] = torch.zeros(spax.spax_chunk_attention_workspace_bytes(s["plan"]),
                              dtype=torch.uint8, device="cuda")
    return s


def _strides(c):
    """Bytes of the packed blob's records: the original columns, and the two-bit ones."""
    n = c["d_out"] * c["mats"]
    original = 2 * n if c["fmt"] == "fp16" else n // 2 + n // INT4_GROUP * 4
    return -(-original // 128) * 128, -(-(n // 4 + n // 64 * 4) // 128) * 128


def _prepare_gemm(c, g):
    rows, d_in, n = c["rows"], c["d_in"], c["d_out"] * c["mats"]
    wide, narrow = _strides(c)
    blob = torch.zeros(d_in * (wide + narrow), dtype=torch.uint8, device="cuda")
    columns = blob[:d_in * wide].view(d_in, wide)
    if c["fmt"] == "fp16":
        columns[:, :2 * n].view(torch.float16).copy_(_randn(g, (d_in, n), torch.float16,
                                                            d_in ** -0.5))
    else:
        columns[:, :n // 2] = torch.randint(0, 256, (d_in, n // 2), generator=g, device="cuda",
                                            dtype=torch.uint8)
        # groups of about normal weights: the smallest value, and a fifteenth of the range
        spread = (torch.rand((d_in, n // INT4_GROUP), generator=g, device="cuda") + 2) * d_in ** -0.5
        scale = columns[:, n // 2:n // 2 + n // INT4_GROUP * 4].view(torch.float16)
        scale[:, 0::2] = (2 * spread / 15).half()
        scale[:, 1::2] = -spread.half()
    # rows of x begin on 16 bytes; what pads them is no part of them
    x = torch.full((rows, -(-d_in // 8) * 8), math.nan, dtype=torch.float16, device="cuda")
    x[:, :d_in] = _randn(g, (rows, d_in), torch.float16)
    width = c["d_out"] if c["form"] == "gated" else n
    s = dict(c=c, blob=blob, x=x[:, :d_in],
             bias=_randn(g, (n,), torch.float32, 0.3) if c["bias"] else None,
             res=None if c["res"] == "none" else _randn(g, (rows, width), TYPES[c["res"]]),
             y=torch.empty((rows, width), dtype=TYPES[c["out"]], device="cuda"))
    if own:
        import activation_sparse_tiered_amd as spax
        fmt = spax.FMT_FP16 if c["fmt"] == "fp16" else spax.FMT_INT4
        s["layout"] = spax.spax_layout_init(d_in, [c["d_out"]] * c["mats"], fmt, INT4_GROUP, 64)
        s["plan"] = spax.make_packed_gemm(s["layout"], blob, s["x"], s["y"], bias=s["bias"],
                                          act=None if c["form"] == "plain" else c["act"],
                                          gated=c["form"] == "gated", residual=s["res"],
                                          scale=c["scale"])
        s["ws"] = torch.zeros(spax.spax_packed_gemm_workspace_bytes(s["plan"]),
                              dtype=torch.uint8, device="cuda")
    return s


def prepare(case, seed):
    return {"append": _prepare_append, "chunk": _prepare_chunk,
            "gemm": _prepare_gemm}[case["op"]](case, _rng(seed))


# ------------------------------------------------------------------ one pass

def _normed(x, kind, w, b, eps):
    """x [tokens, heads, dim], weights [dim] or [heads, dim]."""
    if kind == "layer":
        x = x - x.mean(-1, keepdim=True)
    x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * w
    return x if b is None else x + b


def _turn(x, cos, sin, pairs):
    """The leading 2 * cos.shape[-1] values of each head turned pair by pair."""
    n = cos.shape[-1]
    rest = x[..., 2 * n:]
    if pairs == "halves":
        a, b = x[..., :n], x[..., n:2 * n]
        return torch.cat([a * cos - b * sin, a * sin + b * cos, rest], -1)
    a, b = x[..., 0:2 * n:2], x[..., 1:2 * n:2]
    return torch.cat([torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2), rest],
                     -1)


def _to_cache(x, scale, dtype):
    if scale is not None:
        x = (x / scale[None, :, None]).clamp(-E4M3_MAX, E4M3_MAX)
    return x.to(dtype)


def _run_append(s):
    c = s["c"]
    angle = s["positions"].double()[:, None] * s["inv"].double()
    cos, sin = angle.cos().float()[:, None, :], angle.sin().float()[:, None, :]
    live = (s["positions"] >= 0)
    q = _normed(s["q"].float(), c["norm"], s["qw"], s["qb"], s["eps"])
    q = _turn(q, cos, sin, c["pairs"]) * live[:, None, None]
    s["q_out"].copy_(q)
    k = _normed(s["k"].float(), c["norm"], s["kw"], s["kb"], s["eps"])
    k = _to_cache(_turn(k, cos, sin, c["pairs"]), s["ks"], s["kc"].dtype)
    v = _to_cache(s["v"].float(), s["vs"], s["vc"].dtype)
    at = s["positions"].long()
    page = s["table"][s["seq"].long(), at.clamp(min=0) // c["page"]].long()
    # padding rows write nothing
    live = torch.nonzero(live).squeeze(1)
    page, row = page[live], at[live] % c["page"]
    # (indexing as bytes or halves: every cache type can be stored that way)
    raw = torch.uint8 if c["cache"] == "e4m3" else torch.int16
    s["kc"].view(raw)[page, :, row] = k[live].view(raw)
    s["vc"].view(raw)[page, :, row] = v[live].view(raw)
    return s["q_out"], s["kc"], s["vc"]


def _run_chunk(s):
    c = s["c"]
    hk, dim, page, n = c["kv_heads"], c["dim"], c["page"], c["seqs"]
    group, most = c["heads"] // c["kv_heads"], s["most_new"]
    starts, lens = s["starts"].long(), s["lens"].long()
    new = starts[1:] - starts[:-1]
    # every sequence padded to the most new tokens and to the longest cache
    step = torch.arange(most, device="cuda")[None, :]
    there = step < new[:, None]
    row = torch.where(there, starts[:-1, None] + step, 0)
    place = lens[:, None] - new[:, None] + step                      # [n, most]
    pages = s["table"].long().clamp(min=0)
    length = pages.shape[1] * page
    at = torch.arange(length, device="cuda")
    raw = torch.uint8 if c["cache"] == "e4m3" else torch.int16
    held = at[None, :] < lens[:, None]

    def rows(cache):
        x = cache.view(raw)[pages].view(cache.dtype).float()         # [n, pages, hk, page, dim]
        x = x.permute(0, 2, 1, 3, 4).reshape(n, hk, length, dim)
        return torch.where(held[:, None, :, None], x, 0.0).contiguous()

    k = rows(s["kc"])
    q = s["q"][row].float().view(n, most, hk, group, dim).permute(0, 2, 1, 3, 4)
    q = (q * s["scale"]).reshape(n, hk, most * group, dim).contiguous()
    if s["ks"] is not None:
        q = q * s["ks"][None, :, None, None]
    score = torch.matmul(q, k.transpose(2, 3).contiguous()).view(n, hk, most, group, length)
    del k
    seen = (at <= place[:, :, None]) & there[:, :, None]
    if c["window"]:
        seen = seen & (at > place[:, :, None] - c["window"])
    score.masked_fill_(~seen[:, None, :, None, :], -math.inf)
    top = score.amax(-1, keepdim=True)
    score.sub_(torch.where(top == -math.inf, 0.0, top)).exp_()
    total = score.sum(-1, keepdim=True)
    out = torch.matmul(score.view(n, hk, most * group, length), rows(s["vc"]))
    out = out.view(n, hk, most, group, dim) / torch.where(total == 0, 1.0, total)
    if s["vs"] is not None:
        out = out * s["vs"][None, :, None, None, None]
    lse = (top + total.log()).squeeze(-1).permute(0, 2, 1, 3).reshape(n, most, c["heads"])
    out = out.permute(0, 2, 1, 3, 4).reshape(n, most, c["heads"], dim)
    s["out"][row[there]] = out[there].to(s["out"].dtype)
    s["lse"][row[there]] = lse[there]
    return s["out"], s["lse"]


def _columns(s):
    """The original columns that the blob stands for, fp32 [d_in, d_out_total]."""
    c = s["c"]
    n, wide = c["d_out"] * c["mats"], _strides(c)[0]
    record = s["blob"][:c["d_in"] * wide].view(c["d_in"], wide)
    if c["fmt"] == "fp16":
        return record[:, :2 * n].view(torch.float16).float()
    code = record[:, :n // 2]
    code = torch.stack([code & 15, code >> 4], -1).view(c["d_in"], -1, INT4_GROUP).float()
    pair = record[:, n // 2:n // 2 + n // INT4_GROUP * 4].view(torch.float16).float()
    return (code * pair[:, 0::2, None] + pair[:, 1::2, None]).view(c["d_in"], n)


def _act(x, act):
    if act == "silu":
        return x / (1 + torch.exp(-x))
    return 0.5 * x * (1 + torch.tanh(math.sqrt(2 / math.pi) * (x + 0.044715 * x * x * x)))


def _run_gemm(s):
    c = s["c"]
    t = torch.matmul(s["x"].float(), _columns(s))
    if s["bias"] is not None:
        t = t + s["bias"]
    if c["form"] == "act":
        t = _act(t, c["act"])
    elif c["form"] == "gated":
        t = _act(t[:, :c["d_out"]], c["act"]) * t[:, c["d_out"]:]
    t = t * c["scale"]
    s["y"].copy_(t if s["res"] is None else s["res"].float() + t)
    return s["y"]


def run(state):
    op = state["c"]["op"]
    if own:
        import activation_sparse_tiered_amd as spax
        if op == "append":
            spax.spax_kv_append_normed(state["plan"], state["norm"])
            return state["q_out"], state["kc"], state["vc"]
        if op == "chunk":
            spax.spax_chunk_attention(state["plan"], state["ws"])
            return state["out"], state["lse"]
        spax.spax_packed_gemm(state["plan"], state["ws"])
        return state["y"]
    if op == "append":
        return _run_append(state)
    if op == "chunk":
        return _run_chunk(state)
    return _run_gemm(state)


# ------------------------------------------------------------------ what a pass cannot do without

def _pairs(new, before, window):
    """(token, key) pairs that count, and keys that any token sees."""
    if not window or before + new <= window:
        return new * before + new * (new + 1) // 2, before + new if new else 0
    grow = min(new, max(0, window - before))       # tokens that see all keys before them
    pairs = grow * before + grow * (grow + 1) // 2 + (new - grow) * window
    return pairs, min(before + new, window + new - 1) if new else 0


def work(case):
    c = case
    if c["op"] == "append":
        n, dim, hq, hk = c["tokens"], c["dim"], c["heads"], c["kv_heads"]
        weights = (hq + hk if c["weights"] == "own" else 2) * dim * (2 if c["norm"] == "layer" else 1)
        return {"bytes": BYTES[c["src"]] * n * (hq + 2 * hk) * dim + 2 * n * hq * dim
                + BYTES[c["cache"]] * 2 * n * hk * dim + 12 * n + 4 * weights,
                "flops": n * (hq + hk) * (3 * c["rot"] + 4 * dim)}
    if c["op"] == "chunk":
        both = [_pairs(a, b, c["window"]) for a, b in _chunks(c)]
        pairs, keys = sum(p for p, k in both), sum(k for p, k in both)
        rows = sum(a for a, b in _chunks(c)) * c["heads"]
        return {"bytes": 2 * keys * c["kv_heads"] * c["dim"] * BYTES[c["cache"]]
                + 2 * rows * c["dim"] * BYTES[c["q"]] + 4 * rows + 4 * (keys // c["page"]),
                "flops": 4 * pairs * c["heads"] * c["dim"]}
    n, d_in, rows = c["d_out"] * c["mats"], c["d_in"], c["rows"]
    width = c["d_out"] if c["form"] == "gated" else n
    blob = d_in * (2 * n if c["fmt"] == "fp16" else n // 2 + n // INT4_GROUP * 4)
    res = 0 if c["res"] == "none" else BYTES[c["res"]]
    return {"bytes": blob + 2 * rows * d_in + rows * width * (BYTES[c["out"]] + res)
            + (4 * n if c["bias"] else 0), "flops": 2 * rows * d_in * n}


# ------------------------------------------------------------------ the definitions in 64 bits

def _exact_append(c, s):
    f64 = torch.float64
    q_out = torch.zeros(s["q"].shape, dtype=f64, device="cuda")
    kc, vc = s["kc"].to(f64), s["vc"].to(f64)
    n2 = c["rot"] // 2
    if c["pairs"] == "halves":
        first, second = torch.arange(n2), torch.arange(n2, 2 * n2)
    else:
        first = 2 * torch.arange(n2)
        second = first + 1
    first, second = first.to("cuda"), second.to("cuda")

    def normed(x, w, b):
        x = x.to(f64)
        if c["norm"] == "rms":
            return x * torch.rsqrt(x.square().mean(2, keepdim=True) + s["eps"]) * w.to(f64)
        var, mean = torch.var_mean(x, 2, correction=0, keepdim=True)
        return (x - mean) * torch.rsqrt(var + s["eps"]) * w.to(f64) + b.to(f64)

    def turned(y):
        z = torch.complex(y[..., first], y[..., second])
        phase = s["positions"].to(f64)[:, None] * s["inv"].to(f64)
        z = z * torch.polar(torch.ones_like(phase), phase)[:, None, :]
        y[..., first], y[..., second] = z.real, z.imag
        return y

    use = (s["positions"] >= 0).nonzero()[:, 0]
    q_out[use] = turned(normed(s["q"], s["qw"], s["qb"]))[use]
    p = s["positions"][use].long()
    slot = s["table"][s["seq"][use].long(), p.div(c["page"], rounding_mode="floor")].long()
    for cache, rows, scale in ((kc, turned(normed(s["k"], s["kw"], s["kb"])), s["ks"]),
                               (vc, s["v"].to(f64), s["vs"])):
        rows = rows[use]
        if scale is not None:
            rows = (rows / scale.to(f64).view(1, -1, 1)).clamp(-E4M3_MAX, E4M3_MAX)
        cache[slot, :, p.remainder(c["page"])] = rows
    return q_out, kc, vc


def _exact_chunk(c, s):
    f64 = torch.float64
    out, lse = s["out"].to(f64), s["lse"].to(f64)
    group = c["heads"] // c["kv_heads"]
    raw = torch.uint8 if c["cache"] == "e4m3" else torch.int16
    starts = s["starts"].tolist()
    for i, n in enumerate(s["lens"].tolist()):
        a, b = starts[i], starts[i + 1]
        if a == b:
            continue
        pos = torch.arange(n, device="cuda")
        mine = torch.arange(n - (b - a), n, device="cuda")[:, None]
        hidden = pos > mine
        if c["window"]:
            hidden |= pos <= mine - c["window"]
        page = s["table"][i].long()[pos // c["page"]]
        for h in range(c["kv_heads"]):
            k = s["kc"][:, h].view(raw)[page, pos % c["page"]].view(s["kc"].dtype).to(f64)
            v = s["vc"][:, h].view(raw)[page, pos % c["page"]].view(s["vc"].dtype).to(f64)
            if s["ks"] is not None:
                k, v = k * s["ks"][h].to(f64), v * s["vs"][h].to(f64)
            for y in range(h * group, (h + 1) * group):
                x = (s["q"][a:b, y].to(f64) @ k.t() * s["scale"]).masked_fill_(hidden, -math.inf)
                lse[a:b, y] = torch.logsumexp(x, -1)
                out[a:b, y] = torch.softmax(x, -1) @ v
    return out, lse


def _exact_gemm(c, s):
    f64 = torch.float64
    d_in, n = c["d_in"], c["d_out"] * c["mats"]
    wide = s["blob"].numel() // d_in - _strides(c)[1]
    words = s["blob"][:d_in * wide].view(torch.int16).view(d_in, wide // 2)
    t = torch.zeros((c["rows"], n), dtype=f64, device="cuda")
    for at in range(0, n, INT4_GROUP):
        to = min(n, at + INT4_GROUP)
        if c["fmt"] == "fp16":
            w = words[:, at:to].contiguous().view(torch.float16).to(f64)
        else:
            packed = words[:, at // 4:to // 4].int() & 0xffff
            w = torch.stack([(packed >> (4 * i)) & 15 for i in range(4)], 2).view(d_in, -1).to(f64)
            scales = words[:, n // 4 + at // 64:n // 4 + at // 64 + 2].contiguous()
            scales = scales.view(torch.float16).to(f64)
            w = w * scales[:, :1] + scales[:, 1:]
        t[:, at:to] = s["x"].to(f64) @ w
    if c["bias"]:
        t += s["bias"].to(f64)

    def act(v):
        if c["act"] == "silu":
            return v * torch.sigmoid(v)
        return torch.nn.functional.gelu(v, approximate="tanh")

    if c["form"] == "gated":
        t = act(t[:, :c["d_out"]]) * t[:, c["d_out"]:]
    elif c["form"] == "act":
        t = act(t)
    t = t * c["scale"]
    return t if s["res"] is None else t.add(s["res"].to(f64))


def exact(case, seed):
    s = prepare(case, seed)
    return {"append": _exact_append, "chunk": _exact_chunk,
            "gemm": _exact_gemm}[case["op"]](case, s)
