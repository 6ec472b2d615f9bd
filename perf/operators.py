"""Timing cases of the operators that stand between the projection groups of a decoder step: the
paged cache append with rotation, the attention of one new token per sequence, the gated residual
with its norms, and the gated activation.

``run`` computes them in plain torch operations, or, with ``own`` set, through the library's
entry points.  Shapes are the 7B / 8B decoder shapes of the benchmark (32 query heads of 128, 32
or 8 key heads, widths 4096, 11008 and 14336) and generic ones; values are synthetic.
"""

import math

import torch

own = False

TYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16,
         "e4m3": torch.float8_e4m3fn}
BYTES = {"fp32": 4, "fp16": 2, "bf16": 2, "e4m3": 1}
E4M3_MAX = 448.0


# ------------------------------------------------------------------ cases

def _append(name, tokens, kind, heads, kv_heads, dim, rot, pairs, page, src, cache, far):
    return dict(name=name, op="append", tokens=tokens, kind=kind, heads=heads, kv_heads=kv_heads,
                dim=dim, rot=rot, pairs=pairs, page=page, src=src, cache=cache, far=far)


def _attention(name, seqs, longest, lens, heads, kv_heads, dim, page, q, cache, window, order):
    return dict(name=name, op="attention", seqs=seqs, longest=longest, lens=lens, heads=heads,
                kv_heads=kv_heads, dim=dim, page=page, q=q, cache=cache, window=window,
                order=order)


def _norm(name, rows, d, kind, src, res, out, post, gate, scale):
    return dict(name=name, op="norm", rows=rows, d=d, kind=kind, src=src, res=res, out=out,
                post=post, gate=gate, scale=scale)


def _glu(name, rows, d, act, src, out):
    return dict(name=name, op="glu", rows=rows, d=d, act=act, src=src, out=out)


def listed():
    return [
        # one user's next token in a 7B layer: the q|k|v projection's fp32 row into an fp16 cache
        _append("append 1 token 7b", 1, "decode", 32, 32, 128, 128, "halves", 16, "fp32", "fp16",
                4096),
        # a serving batch of an 8B model, padded, its contexts far along
        _append("append 61 tokens 8b", 61, "decode", 32, 8, 128, 128, "halves", 64, "bf16",
                "bf16", 131072),
        # prompts of three users written at once, half of each head rotated, into an 8-bit cache
        _append("append prompts e4m3", 4099, "prompt", 32, 8, 128, 64, "neighbours", 32, "fp16",
                "e4m3", 8192),
        # the first replies of a chat: a short cache, one head of keys per head of queries
        _attention("attend 1 x 509 7b", 1, 509, "even", 32, 32, 128, 16, "fp16", "fp16", 0,
                   "heads"),
        # one user over a long document: few rows, so the length is what can be shared out
        _attention("attend 1 x 32768 8b", 1, 32768, "even", 32, 8, 128, 16, "fp16", "fp16", 0,
                   "heads"),
        # a serving batch whose lengths spread from none to 8192, rows of a token kept together
        _attention("attend 48 ragged 8b", 48, 8192, "ragged", 32, 8, 128, 64, "bf16", "bf16", 0,
                   "tokens"),
        # the largest: a full batch of long contexts in an 8-bit cache
        _attention("attend 32 x 32768 e4m3", 32, 32768, "even", 32, 8, 128, 32, "fp16", "e4m3", 0,
                   "heads"),
        # between two projections of one token: add to the stream, norm for the next projection
        _norm("norm 1 x 4096", 1, 4096, "rms", "fp32", "fp32", "fp16", False, "none", 1.0),
        # a prompt's rows in a model with norms on both sides and a gate per channel
        _norm("norm 2048 x 4096", 2048, 4096, "rms", "bf16", "bf16", "bf16", True, "channel",
              0.5),
        # an odd width with layer norms and a gate for each row, as in conditioned blocks
        _norm("norm 333 x 5003", 333, 5003, "layer", "fp16", "fp32", "fp16", True, "row", 1.0),
        # one token's gate|up row of the 7B layer
        _glu("glu 1 x 11008", 1, 11008, "silu", "fp32", "fp16"),
        # a prompt's rows of the 8B layer
        _glu("glu 2048 x 14336", 2048, 14336, "gelu", "bf16", "bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "append", "attention", "attention", "attention", "norm", "norm",
                     "glu"])
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
                    rng.choice([low, low, "e4m3"]), _log(rng, 4096, 1000000))
    elif op == "attention":
        kv = rng.choice([1, 2, 4, 8, 32])
        group = rng.choice([1, 4, 5, 8, 16, 20]) if kv < 32 else 1
        dim = rng.choice([64, 96, 128, 128, 192, 256])
        q = rng.choice(["fp16", "bf16"])
        seqs = _log(rng, 1, 128)
        most = max(64, min(65536, 2 ** 29 // (seqs * kv * dim)))
        c = _attention("", seqs, _log(rng, 1, most), rng.choice(["even", "ragged"]), kv * group,
                       kv, dim, rng.choice([8, 16, 32, 64, 256]), q, rng.choice([q, q, "e4m3"]),
                       rng.choice([0, 0, 0, 1, 100, 1000]), rng.choice(["heads", "tokens"]))
    elif op == "norm":
        src = rng.choice(["fp32", "fp16", "bf16"])
        c = _norm("", _log(rng, 1, 3000), _log(rng, 64, 16384), rng.choice(["rms", "layer"]), src,
                  rng.choice([src, "fp32"]), "bf16" if src == "bf16" else "fp16",
                  rng.choice([True, False]), rng.choice(["none", "channel", "row"]),
                  rng.choice([1.0, 0.5, 0.22]))
    else:
        src = rng.choice(["fp32", "fp16", "bf16"])
        c = _glu("", _log(rng, 1, 3000), _log(rng, 64, 16384), rng.choice(["silu", "gelu"]), src,
                 "bf16" if src == "bf16" else "fp16")
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


def _lens(c):
    """How long each sequence is (the same for every seed; the order is not)."""
    if c["lens"] == "even" or c["seqs"] < 3:
        return [c["longest"]] * c["seqs"]
    n = c["seqs"]
    return [0] + [max(1, round(c["longest"] ** (i / (n - 1)))) for i in range(1, n)]


def _segments(c):
    """Prompt cases: (first position, tokens) of up to three sequences."""
    n = c["tokens"]
    cut = [n] if n < 3 else [n // 2, n // 3, n - n // 2 - n // 3]
    return [(min(17 * i, max(0, c["far"] - k)), k) for i, k in enumerate(cut)]


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
    row = _randn(g, (n, (hq + 2 * hk) * dim), src)
    s = dict(c=c, seq=seq, positions=positions, table=table,
             q=row[:, :hq * dim].view(n, hq, dim),
             k=row[:, hq * dim:(hq + hk) * dim].view(n, hk, dim),
             v=row[:, (hq + hk) * dim:].view(n, hk, dim),
             kc=_randn(g, (pages, hk, page, dim), cache),
             vc=_randn(g, (pages, hk, page, dim), cache),
             q_out=torch.empty((n, hq, dim), dtype=low, device="cuda"),
             inv=(1e4 ** (-torch.arange(0, c["rot"], 2, dtype=torch.float64, device="cuda")
                          / max(1, c["rot"]))).float(),
             ks=None, vs=None)
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
    return s


def _prepare_attention(c, g):
    hq, hk, dim, page = c["heads"], c["kv_heads"], c["dim"], c["page"]
    q_type, cache = TYPES[c["q"]], TYPES[c["cache"]]
    lens = torch.tensor(_lens(c), dtype=torch.int32, device="cuda")
    lens = lens[torch.randperm(c["seqs"], generator=g, device="cuda")].contiguous()
    need = (lens + page - 1) // page
    width = max(1, (c["longest"] + page - 1) // page)
    pages = int(need.sum()) + 3
    held = torch.arange(width, device="cuda")[None, :] < need[:, None]
    table = torch.full((c["seqs"], width), -1, dtype=torch.int32, device="cuda")
    table[held] = torch.randperm(pages, generator=g, device="cuda")[:pages - 3].int()
    shape = (pages, hk, page, dim) if c["order"] == "heads" else (pages, page, hk, dim)
    s = dict(c=c, lens=lens, table=table, ks=None, vs=None,
             q=_randn(g, (c["seqs"], hq, dim), q_type),
             kc=_randn(g, shape, cache), vc=_randn(g, shape, cache),
             out=torch.empty((c["seqs"], hq, dim), dtype=q_type, device="cuda"),
             scale=dim ** -0.5)
    if c["order"] == "tokens":
        s["kc"], s["vc"] = s["kc"].transpose(1, 2), s["vc"].transpose(1, 2)
    # a cache holds whatever was left in rows that no sequence has reached yet
    last = (lens - 1).clamp(min=0).long()
    ends = (lens > 0) & (lens % page != 0)
    tail_page = table[torch.arange(c["seqs"], device="cuda"), last // page][ends].long()
    s["vc"][tail_page, :, page - 1] = math.nan
    if c["cache"] == "e4m3":
        s["ks"] = torch.rand(hk, generator=g, device="cuda") * 0.5 + 0.5
        s["vs"] = torch.rand(hk, generator=g, device="cuda") * 0.5 + 0.5
    if own:
        import activation_sparse_tiered_amd as spax
        s["cache"] = spax.make_kv_cache(s["kc"], s["vc"], table, k_scale=s["ks"],
                                        v_scale=s["vs"])
        s["plan"] = spax.make_attention(s["cache"], s["q"], lens, s["out"], max_len=c["longest"],
                                        scale=s["scale"], window=c["window"])
        s["ws"] = torch.zeros(spax.spax_attention_workspace_bytes(s["plan"]), dtype=torch.uint8,
                              device="cuda")
    return s


def _prepare_norm(c, g):
    rows, d = c["rows"], c["d"]
    src, res, out = TYPES[c["src"]], TYPES[c["res"]], TYPES[c["out"]]
    layer = c["kind"] == "layer"

    def weight():
        return 1 + _randn(g, (d,), torch.float32, 0.1)

    s = dict(c=c, eps=1e-5, b=_randn(g, (rows, d), src, 0.7),
             r=_randn(g, (rows, d), res, 2.0),
             h=torch.empty((rows, d), dtype=res, device="cuda"),
             x=torch.empty((rows, d), dtype=out, device="cuda"),
             pre_w=weight(), pre_b=_randn(g, (d,), torch.float32, 0.1) if layer else None,
             post_w=weight() if c["post"] else None,
             post_b=_randn(g, (d,), torch.float32, 0.1) if layer and c["post"] else None,
             gate=None)
    if c["gate"] != "none":
        s["gate"] = _randn(g, (d,) if c["gate"] == "channel" else (rows, d), src, 0.5)
    if own:
        import activation_sparse_tiered_amd as spax
        s["plan"] = spax.make_residual_norm(s["r"], s["b"], s["h"], s["x"], kind=c["kind"],
                                            pre_weight=s["pre_w"], pre_bias=s["pre_b"],
                                            post_weight=s["post_w"], post_bias=s["post_b"],
                                            gate=s["gate"], scale=c["scale"], eps=s["eps"])
    return s


def _prepare_glu(c, g):
    y = _randn(g, (c["rows"], 2 * c["d"]), TYPES[c["src"]], 1.5)
    s = dict(c=c, gate=y[:, :c["d"]], up=y[:, c["d"]:],
             x=torch.empty((c["rows"], c["d"]), dtype=TYPES[c["out"]], device="cuda"))
    if own:
        import activation_sparse_tiered_amd as spax
        s["plan"] = spax.make_glu(s["gate"], s["up"], s["x"], act=c["act"])
    return s


def prepare(case, seed):
    return {"append": _prepare_append, "attention": _prepare_attention, "norm": _prepare_norm,
            "glu": _prepare_glu}[case["op"]](case, _rng(seed))


# ------------------------------------------------------------------ one pass

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
    q = _turn(s["q"].float(), cos, sin, c["pairs"]) * live[:, None, None]
    s["q_out"].copy_(q)
    k = _to_cache(_turn(s["k"].float(), cos, sin, c["pairs"]), s["ks"], s["kc"].dtype)
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


def _run_attention(s):
    c = s["c"]
    hk, dim, page = c["kv_heads"], c["dim"], c["page"]
    n, group = c["seqs"], c["heads"] // c["kv_heads"]
    pages = s["table"].long().clamp(min=0)
    length = pages.shape[1] * page
    at = torch.arange(length, device="cuda")[None, :]
    last = s["lens"].long()[:, None]
    first = (last - c["window"]).clamp(min=0) if c["window"] else torch.zeros_like(last)
    live = (at >= first) & (at < last)
    raw = torch.uint8 if c["cache"] == "e4m3" else torch.int16

    def rows(cache):
        x = cache.view(raw)[pages].view(cache.dtype).float()  # [n, pages, hk, page, dim]
        x = x.permute(0, 2, 1, 3, 4).reshape(n, hk, length, dim)
        return torch.where(live[:, None, :, None], x, 0.0).contiguous()

    k = rows(s["kc"])
    q = s["q"].float().view(n, hk, group, dim) * s["scale"]
    if s["ks"] is not None:
        q = q * s["ks"][None, :, None, None]
    score = torch.matmul(q, k.transpose(2, 3).contiguous())
    del k
    score = torch.where(live[:, None, None, :], score, -math.inf)
    top = score.amax(-1, keepdim=True)
    weight = torch.exp(score - torch.where(top == -math.inf, 0.0, top))
    total = weight.sum(-1, keepdim=True)
    out = torch.matmul(weight, rows(s["vc"])) / torch.where(total == 0, 1.0, total)
    if s["vs"] is not None:
        out = out * s["vs"][None, :, None, None]
    s["out"].copy_(out.reshape(n, c["heads"], dim))
    return s["out"]


def _normed(x, kind, w, b, eps):
    if kind == "layer":
        x = x - x.mean(-1, keepdim=True)
    x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    x = x * w
    return x if b is None else x + b


def _run_norm(s):
    c = s["c"]
    t = s["b"].float()
    if s["post_w"] is not None:
        t = _normed(t, c["kind"], s["post_w"], s["post_b"], s["eps"])
    if s["gate"] is not None:
        t = t * s["gate"].float()
    h = s["r"].float() + c["scale"] * t
    s["h"].copy_(h)
    s["x"].copy_(_normed(h, c["kind"], s["pre_w"], s["pre_b"], s["eps"]))
    return s["h"], s["x"]


def _act(x, act):
    if act == "silu":
        return x / (1 + torch.exp(-x))
    return 0.5 * x * (1 + torch.tanh(math.sqrt(2 / math.pi) * (x + 0.044715 * x * x * x)))


def _run_glu(s):
    s["x"].copy_(_act(s["gate"].float(), s["c"]["act"]) * s["up"].float())
    return s["x"]


def run(state):
    op = state["c"]["op"]
    if own:
        import activation_sparse_tiered_amd as spax
        if op == "append":
            spax.spax_kv_append(state["plan"])
            return state["q_out"], state["kc"], state["vc"]
        if op == "attention":
            spax.spax_paged_attention(state["plan"], state["ws"])
            return state["out"]
        if op == "norm":
            spax.spax_residual_norm(state["plan"])
            return state["h"], state["x"]
        spax.spax_glu(state["plan"])
        return state["x"]
    if op == "append":
        return _run_append(state)
    if op == "attention":
        return _run_attention(state)
    if op == "norm":
        return _run_norm(state)
    return _run_glu(state)


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    c = case
    if c["op"] == "append":
        n, dim, hq, hk = c["tokens"], c["dim"], c["heads"], c["kv_heads"]
        q_bytes = 2 * n * hq * dim
        return {"bytes": BYTES[c["src"]] * n * (hq + 2 * hk) * dim + q_bytes
                + BYTES[c["cache"]] * 2 * n * hk * dim + 12 * n,
                "flops": 3 * n * (hq + hk) * c["rot"]}
    if c["op"] == "attention":
        keys = sum(min(v, c["window"]) if c["window"] else v for v in _lens(c))
        kv = 2 * keys * c["kv_heads"] * c["dim"] * BYTES[c["cache"]]
        return {"bytes": kv + 2 * c["seqs"] * c["heads"] * c["dim"] * BYTES[c["q"]]
                + 4 * (c["seqs"] + keys // c["page"]),
                "flops": 4 * keys * c["heads"] * c["dim"]}
    n = c["rows"] * c["d"]
    if c["op"] == "norm":
        size = n * (BYTES[c["src"]] + 2 * BYTES[c["res"]] + BYTES[c["out"]])
        size += {"none": 0, "channel": c["d"], "row": n}[c["gate"]] * BYTES[c["src"]]
        return {"bytes": size + 4 * c["d"] * (2 if c["post"] else 1), "flops": 12 * n}
    return {"bytes": n * (2 * BYTES[c["src"]] + BYTES[c["out"]]), "flops": 8 * n}


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

    def turned(x):
        z = torch.complex(x[..., first].to(f64), x[..., second].to(f64))
        phase = s["positions"].to(f64)[:, None] * s["inv"].to(f64)
        z = z * torch.polar(torch.ones_like(phase), phase)[:, None, :]
        y = x.to(f64).clone()
        y[..., first], y[..., second] = z.real, z.imag
        return y

    use = (s["positions"] >= 0).nonzero()[:, 0]
    q_out[use] = turned(s["q"])[use]
    p = s["positions"][use].long()
    slot = s["table"][s["seq"][use].long(), p.div(c["page"], rounding_mode="floor")].long()
    for cache, rows, scale in ((kc, turned(s["k"]), s["ks"]), (vc, s["v"].to(f64), s["vs"])):
        rows = rows[use]
        if scale is not None:
            rows = (rows / scale.to(f64).view(1, -1, 1)).clamp(-E4M3_MAX, E4M3_MAX)
        cache[slot, :, p.remainder(c["page"])] = rows
    return q_out, kc, vc


def _exact_attention(c, s):
    f64 = torch.float64
    out = torch.zeros((c["seqs"], c["heads"], c["dim"]), dtype=f64, device="cuda")
    group = c["heads"] // c["kv_heads"]
    for i, n in enumerate(s["lens"].tolist()):
        lo = max(0, n - c["window"]) if c["window"] else 0
        if n <= lo:
            continue
        pos = torch.arange(lo, n, device="cuda")
        page = s["table"][i].long()[pos // c["page"]]
        for h in range(c["kv_heads"]):
            k = s["kc"][:, h].view(torch.uint8 if c["cache"] == "e4m3" else torch.int16)
            v = s["vc"][:, h].view(torch.uint8 if c["cache"] == "e4m3" else torch.int16)
            k = k[page, pos % c["page"]].view(s["kc"].dtype).to(f64)
            v = v[page, pos % c["page"]].view(s["vc"].dtype).to(f64)
            if s["ks"] is not None:
                k, v = k * s["ks"][h].to(f64), v * s["vs"][h].to(f64)
            q = s["q"][i, h * group:(h + 1) * group].to(f64)
            out[i, h * group:(h + 1) * group] = torch.softmax(q @ k.t() * s["scale"], -1) @ v
    return out


def _exact_norm(c, s):
    f64 = torch.float64

    def wide(name):
        return None if s[name] is None else s[name].to(f64)

    def norm(x, w, b):
        if c["kind"] == "rms":
            return x * torch.rsqrt(x.square().mean(1, keepdim=True) + s["eps"]) * w
        var, mean = torch.var_mean(x, 1, correction=0, keepdim=True)
        return (x - mean) * torch.rsqrt(var + s["eps"]) * w + b

    t = wide("b")
    if c["post"]:
        t = norm(t, wide("post_w"), wide("post_b"))
    if c["gate"] != "none":
        t = wide("gate") * t
    h = wide("r").add(t, alpha=c["scale"])
    return h, norm(h, wide("pre_w"), wide("pre_b"))


def _exact_glu(c, s):
    g, u = s["gate"].double(), s["up"].double()
    if c["act"] == "silu":
        return g * torch.sigmoid(g) * u
    return torch.nn.functional.gelu(g, approximate="tanh") * u


def exact(case, seed):
    s = prepare(case, seed)
    return {"append": _exact_append, "attention": _exact_attention, "norm": _exact_norm,
            "glu": _exact_glu}[case["op"]](case, s)
