"""The operators of many tokens at once against the float64 oracle.

Tolerances, per value: half a step of the result's type, as in test_gpu_layer_ops, and the fp32
arithmetic before it:

* normed append: the append's 2^-20 of a pair (the rotation), and the norm: a sum of at most 256
  squares in a thread's chain of 32 and eight steps across threads is off by 40 2^-24 of itself,
  half of that for its root; the mean of a layer norm is off by 40 2^-24 of mean |x|, which is at
  most the root mean square.  With the handful of products 2^-18 of the largest normed value of
  the head covers both, and half a step more the e4m3 value near a middle.
* chunk attention: the error of a score is at most (dim + 4) 2^-24 reach (reach = scale sum
  |q_i k_i|), and it moves a weight and the total by that much each; sums of weights and of
  weighted values run over at most 2048 fp32 additions here; a weight enters rounded to its type:
  half a step of itself (2^-11, 2^-8), and in fp16 2^-39 of the row's largest.  Together mass (2
  (dim + 4) 2^-24 reach + 2048 2^-24 + 2^-16 + half a step), mass = sum softmax |v|.
* product: a column's sum of d_in products passes through at most 16 roundings within a matrix
  instruction, one per 16 k and one per wave and split: mass (16 + d_in / 16 + 32) 2^-23, mass = sum
  |x w|; an int4 weight is rounded to fp16, 2^-11 of itself: mass 2^-11.  The activations are
  steeper than 1 by at most 0.13, and good to 2^-15 of their value.
"""

import numpy as np
import pytest

from oracle import layer as olayer
from oracle import pack as opack
from oracle import prompt as oprompt
from tests.test_gpu_layer_ops import (STEP, TINY, _attention_inputs, _check, _dtype, _f64, _gen,
                                      _randn, env)  # noqa: F401

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ append with normed heads

NORMED = [
    # tokens, heads, kv, dim, rot, pairs, src, out, cache, kind, weights
    (1, 32, 32, 128, 128, "halves", "fp32", "fp16", "fp16", "rms", "shared"),
    (5, 8, 2, 64, 64, "neighbours", "fp16", "fp16", "fp16", "layer", "own"),
    (7, 5, 1, 96, 48, "halves", "bf16", "bf16", "bf16", "rms", "own"),
    (3, 4, 4, 192, 192, "neighbours", "fp32", "bf16", "bf16", "layer", "shared"),
    (9, 16, 2, 256, 128, "halves", "fp16", "fp16", "e4m3", "rms", "shared"),
    (4, 6, 3, 96, 0, "halves", "bf16", "bf16", "e4m3", "layer", "own"),
    (6, 3, 1, 64, 20, "halves", "fp32", "fp16", "fp16", "rms", "shared"),      # pairs one by one
    (6, 3, 2, 256, 2, "neighbours", "fp16", "fp16", "fp16", "layer", "own"),   # 255 items a head
    (6, 3, 2, 192, 90, "halves", "fp16", "fp16", "e4m3", "rms", "own"),
    (700, 5, 2, 64, 64, "halves", "fp16", "fp16", "fp16", "layer", "shared"),  # a prompt
    (700, 11, 3, 96, 24, "halves", "bf16", "bf16", "e4m3", "rms", "own"),
    (5, 0, 2, 128, 128, "halves", "fp16", "fp16", "fp16", "rms", "keys"),      # keys only
    (5, 4, 2, 128, 128, "halves", "fp16", "fp16", "fp16", "rms", "keys"),      # q as it is
    (5, 4, 2, 128, 64, "halves", "fp16", "fp16", "fp16", "layer", "queries"),
]


def _normed_case(env, case, extra=0):
    torch, spax, dev = env
    n, hq, hk, dim, rot, pairs, src, out, cache, kind, weights = case
    g = _gen(torch, n * 1000 + dim + rot)
    page, seqs = 16, min(n, 3)
    width = 64
    pages = seqs * width + 2
    kc, vc = (_randn(torch, g, (pages, hk, page, dim), _dtype(torch, cache)) for _ in range(2))
    table = torch.randperm(pages, generator=g, device=dev)[:seqs * width].int().view(seqs, width)
    table = table.contiguous()
    seq = torch.arange(n, device=dev, dtype=torch.int32) % seqs
    positions = torch.arange(n, device=dev, dtype=torch.int32) // seqs + 3
    if n > 4:
        positions[3] = -7                       # padding
        seq[4] = seqs                           # no such sequence
    row = _randn(torch, g, (n, (hq + 2 * hk) * dim + extra), _dtype(torch, src), 2.0)[:, extra:]
    q = row[:, :hq * dim].unflatten(1, (hq, dim)) if hq else None
    k = row[:, hq * dim:(hq + hk) * dim].unflatten(1, (hk, dim))
    v = row[:, (hq + hk) * dim:].unflatten(1, (hk, dim))
    inv = (1e4 ** (-torch.arange(0, max(rot, 1), 2, device=dev).double() / max(rot, 1))).float()
    scale = [torch.rand(hk, generator=g, device=dev) * 0.1 + 0.01 if cache == "e4m3" else None
             for _ in range(2)]

    def weight(heads, mean):
        shape = (heads, dim) if weights == "own" else (dim,)
        return mean + torch.randn(shape, generator=g, device=dev) * 0.3

    w = dict(q=weight(hq, 1.0) if hq and weights != "keys" else None,
             k=weight(hk, 1.0) if weights != "queries" else None)
    layer = kind == "layer"
    b = {p: None if t is None or not layer else weight(hq if p == "q" else hk, 0.0)
         for p, t in w.items()}
    return dict(q=q, k=k, v=v, kc=kc, vc=vc, table=table, seq=seq, positions=positions, inv=inv,
                scale=scale, w=w, b=b, row=row)


def _normed_ref(s, case, eps):
    n, hq, hk, dim, rot, pairs, src, out, cache, kind, weights = case
    opt = lambda t: None if t is None else _f64(t)  # noqa: E731
    qf = np.zeros((n, 0, dim)) if s["q"] is None else oprompt.head_norm(
        _f64(s["q"]), kind, opt(s["w"]["q"]), opt(s["b"]["q"]), eps)
    kf = oprompt.head_norm(_f64(s["k"]), kind, opt(s["w"]["k"]), opt(s["b"]["k"]), eps)
    vf = _f64(s["v"])
    ks, vs = (np.ones(hk) if t is None else _f64(t) for t in s["scale"])
    kf, vf = kf / ks[None, :, None], vf / vs[None, :, None]
    want_k, want_v = _f64(s["kc"]), _f64(s["vc"])
    ref_q = olayer.kv_append(qf, kf, vf, s["positions"].cpu().numpy(), s["seq"].cpu().numpy(),
                             s["table"].cpu().numpy(), want_k, want_v,
                             _f64(s["inv"]) if rot else np.zeros(0), pairs == "neighbours")
    return qf, kf, vf, ref_q, want_k, want_v


def _normed_call(env, s, case, eps, q_out):
    torch, spax, dev = env
    n, hq, hk, dim, rot, pairs, src, out, cache, kind, weights = case
    c = spax.make_kv_cache(s["kc"], s["vc"], s["table"], *s["scale"])
    a = spax.make_kv_append(c, s["q"], s["k"], s["v"], s["positions"], q_out, seq=s["seq"],
                            inv_freq=s["inv"] if rot else None, interleaved=pairs == "neighbours")
    m = spax.make_head_norm(s["w"]["q"], s["w"]["k"], q_bias=s["b"]["q"], k_bias=s["b"]["k"],
                            kind=kind, eps=eps)
    return a, m


@pytest.mark.parametrize("case", NORMED, ids=[str(c[:5]) for c in NORMED])
@pytest.mark.parametrize("odd", [False, True], ids=["fused", "unaligned"])
def test_normed_append(env, case, odd):  # noqa: F811
    torch, spax, dev = env
    n, hq, hk, dim, rot, pairs, src, out, cache, kind, weights = case
    eps = 1e-3
    s = _normed_case(env, case, 3 if odd else 0)
    qf, kf, vf, ref_q, want_k, want_v = _normed_ref(s, case, eps)
    old_k, old_v = _f64(s["kc"]), _f64(s["vc"])
    q_out = (torch.full((n, hq, dim), float("nan"), dtype=_dtype(torch, out), device=dev)
             if hq else None)
    a, m = _normed_call(env, s, case, eps, q_out)
    print(f"[normed append] {case} odd={odd}", flush=True)
    spax.spax_kv_append_normed(a, m)
    torch.cuda.synchronize()

    def tol(ref, name, big):
        return STEP[name] * np.abs(ref) + TINY[name] + (2.0 ** -20 * 2 + 2.0 ** -18) * big

    if hq:
        _check(_f64(q_out), ref_q, tol(ref_q, out, np.abs(qf).max(axis=-1, keepdims=True)), "q_out")
    for cached, ref, old, rows, name in ((s["kc"], want_k, old_k, kf, "k"),
                                         (s["vc"], want_v, old_v, vf, "v")):
        got = _f64(cached)
        touched = (ref != old).any(axis=-1)
        assert np.array_equal(got[~touched], old[~touched]) and touched.any()
        if cache == "e4m3":
            ref = np.clip(ref, -448, 448)
        _check(got, ref, tol(ref, cache, np.abs(rows).max()), name)


def test_normed_append_in_place(env):  # noqa: F811
    """q_out may be q: a head is read whole before it is written."""
    torch, spax, dev = env
    case = (33, 4, 2, 128, 128, "halves", "bf16", "bf16", "bf16", "layer", "shared")
    s = _normed_case(env, case)
    apart = torch.empty(33, 4, 128, dtype=torch.bfloat16, device=dev)
    spax.spax_kv_append_normed(*_normed_call(env, s, case, 1e-6, apart))
    spax.spax_kv_append_normed(*_normed_call(env, s, case, 1e-6, s["q"]))
    torch.cuda.synchronize()
    assert torch.equal(s["q"].contiguous(), apart)


def test_normed_append_without_size(env):  # noqa: F811
    """A head of zeros: 0 / sqrt(eps), and with eps 0 NaN for that head alone."""
    torch, spax, dev = env
    case = (4, 4, 2, 64, 64, "halves", "fp32", "fp16", "fp16", "rms", "shared")
    s = _normed_case(env, case)
    s["q"][1, 2] = 0
    out = torch.empty(4, 4, 64, dtype=torch.float16, device=dev)
    spax.spax_kv_append_normed(*_normed_call(env, s, case, 1e-6, out))
    torch.cuda.synchronize()
    assert bool((out[1, 2] == 0).all()) and bool(torch.isfinite(out).all())
    spax.spax_kv_append_normed(*_normed_call(env, s, case, 0.0, out))
    torch.cuda.synchronize()
    bad = torch.isnan(out).all(-1)
    assert bool(bad[1, 2]) and int(torch.isnan(out).any(-1).sum()) == 1


# ------------------------------------------------------------------ attention of a chunk

CHUNK = [
    # (new, before) of each sequence, heads, kv, dim, page, type, cache, window, order, max_len
    ([(1, 0)], 1, 1, 128, 4, "fp16", "fp16", 0, "heads", None),
    ([(1, 0), (2, 0), (0, 5), (1, 63), (1, 64), (3, 62), (33, 31)], 4, 2, 64, 16, "fp16", "fp16",
     0, "heads", None),
    ([(130, 0)], 1, 1, 128, 16, "fp16", "fp16", 0, "heads", None),
    ([(127, 0), (0, 0), (128, 1), (129, 200)], 2, 2, 128, 64, "bf16", "bf16", 0, "tokens", None),
    ([(5, 1000)], 8, 2, 128, 16, "fp16", "fp16", 0, "heads", None),             # shared out
    ([(5, 3000), (1, 17), (40, 500)], 8, 1, 128, 32, "bf16", "e4m3", 0, "heads", None),
    ([(50, 100), (3, 40)], 20, 1, 96, 8, "fp16", "fp16", 0, "tokens", None),
    ([(2, 30)], 200, 1, 64, 16, "fp16", "e4m3", 0, "heads", None),              # more heads than rows
    ([(90, 33), (1, 900)], 10, 2, 192, 16, "bf16", "bf16", 0, "heads", None),
    ([(90, 34), (2, 100)], 6, 2, 96, 16, "bf16", "e4m3", 0, "tokens", None),
    ([(70, 34)], 4, 2, 192, 16, "fp16", "e4m3", 0, "heads", None),
    ([(70, 100), (31, 0)], 6, 2, 256, 32, "fp16", "fp16", 0, "heads", None),
    ([(70, 100), (31, 1)], 6, 2, 256, 32, "bf16", "e4m3", 0, "heads", None),
    ([(60, 200), (3, 0)], 8, 2, 128, 16, "fp16", "fp16", 1, "heads", None),     # windows
    ([(60, 200), (3, 0), (2, 700)], 8, 2, 128, 16, "fp16", "fp16", 33, "tokens", None),
    ([(150, 700), (3, 1)], 4, 2, 64, 4, "bf16", "bf16", 130, "heads", None),
    ([(60, 300), (100, 0), (3, -8)], 4, 2, 128, 16, "fp16", "fp16", 0, "heads", 90),  # clamped
]


def _chunk_inputs(env, sizes, hq, hk, dim, page, qt, ct, order, seed, behind=2):
    torch, spax, dev = env
    lens = [a + b for a, b in sizes]
    _, kc, vc, table, ln, scales = _attention_inputs(env, lens, hq, hk, dim, page, qt, ct, order,
                                                     seed)
    starts = np.concatenate([[1], 1 + np.cumsum([a for a, b in sizes])])  # a row before the first
    g = _gen(torch, seed + 1)
    q = _randn(torch, g, (int(starts[-1]) + behind, hq, dim), _dtype(torch, qt))
    return q, kc, vc, table, torch.tensor(starts, dtype=torch.int32, device=dev), ln, scales


def _chunk_check(q, kc, vc, table, starts, ln, scales, out, lse, dim, qt, window, max_len):
    k, v = _f64(kc), _f64(vc)
    if scales[0] is not None:
        k, v = k * _f64(scales[0])[None, :, None, None], v * _f64(scales[1])[None, :, None, None]
    rows, ref, ref_lse, mass, reach = oprompt.chunk_attention(
        _f64(q), k, v, table.cpu().numpy(), starts.cpu().numpy(), ln.cpu().numpy(), dim ** -0.5,
        window, max_len)
    score = (dim + 4) * 2.0 ** -24 * reach
    e = 2 * score[..., None] + 2048 * 2.0 ** -24 + 2.0 ** -16 + STEP[qt]
    tol = STEP[qt] * np.abs(ref) + TINY[qt] + mass * e
    _check(_f64(out)[rows], ref, tol, "out")
    fine = np.where(np.isfinite(ref_lse), np.abs(ref_lse), 0.0)
    _check(_f64(lse)[rows], ref_lse, score + 2048 * 2.0 ** -24 + 2.0 ** -21 * (1 + fine), "lse")
    rest = np.setdiff1d(np.arange(q.shape[0]), rows)
    assert np.isnan(_f64(out)[rest]).all() and np.isnan(_f64(lse)[rest]).all()


@pytest.mark.parametrize("case", CHUNK, ids=[f"{i}-{c[1]}-{c[2]}-{c[3]}-{c[5]}-{c[6]}"
                                             for i, c in enumerate(CHUNK)])
@pytest.mark.parametrize("far", [False, True], ids=["own", "far"])
def test_chunk_attention(env, case, far):  # noqa: F811
    """far: a table with room for more, so the keys are shared out further."""
    torch, spax, dev = env
    sizes, hq, hk, dim, page, qt, ct, window, order, max_len = case
    q, kc, vc, table, starts, ln, scales = _chunk_inputs(
        env, sizes, hq, hk, dim, page, qt, ct, order, sum(a + b for a, b in sizes) + dim)
    if far:
        if max_len is not None:
            pytest.skip("max_len is the case's own")
        wide = torch.full((len(sizes), 20000 // page), -1, dtype=torch.int32, device=dev)
        wide[:, :table.shape[1]] = table
        table = wide
    out = torch.full_like(q, float("nan"))
    lse = torch.full(q.shape[:2], float("nan"), device=dev)
    cache = spax.make_kv_cache(kc, vc, table, *scales)
    a = spax.make_chunk_attention(cache, q, starts, ln, out, max_len=max_len, window=window,
                                  lse=lse)
    need = spax.spax_chunk_attention_workspace_bytes(a)
    ws = torch.full((need + 256,), 0xFF, dtype=torch.uint8, device=dev)
    print(f"[chunk] {case} far={far} workspace {need}", flush=True)
    spax.spax_chunk_attention(a, ws[:need] if need else None)
    torch.cuda.synchronize()
    assert bool((ws[need:] == 0xFF).all())
    _chunk_check(q, kc, vc, table, starts, ln, scales, out, lse, dim, qt, window, max_len)


# more rows for each sequence than small tiles are for, and tables with room for more keys: tiles of 128
# rows, and with 32 key heads of 256
BIG = [
    ([(100, 0), (130, 1500), (101, 37)], 2, 1, 128, 16, "fp16", "fp16", 0, "heads", None),
    ([(100, 0), (130, 1500), (101, 37)], 6, 2, 96, 16, "bf16", "e4m3", 0, "tokens", None),
    ([(140, 900), (300, 0)], 4, 2, 128, 32, "fp16", "e4m3", 0, "heads", None),
    ([(140, 900), (300, 0), (0, 70)], 4, 2, 64, 4, "bf16", "bf16", 700, "heads", None),
    ([(130, 1100), (200, -40)], 2, 2, 192, 16, "fp16", "fp16", 0, "heads", None),
    ([(130, 1100), (200, -40)], 2, 2, 256, 16, "bf16", "e4m3", 0, "heads", None),
    ([(100, 30)] * 6 + [(130, 0), (97, 3000)], 32, 32, 64, 16, "bf16", "bf16", 0, "heads", None),
    ([(100, 100)] * 4 + [(257, 0), (120, 2500)], 32, 32, 128, 16, "fp16", "fp16", 0, "tokens", None),
    ([(100, 100)] * 4 + [(257, 0), (120, 2500)], 32, 32, 96, 64, "fp16", "fp16", 300, "heads", None),
    # more pieces than are joined at once, of small tiles and of large ones
    ([(3, 12000)], 1, 1, 64, 16, "fp16", "fp16", 0, "heads", None),
    ([(130, 12000)], 1, 1, 128, 16, "bf16", "bf16", 0, "heads", None),
]


@pytest.mark.parametrize("case", BIG, ids=[f"{i}-{c[1]}-{c[2]}-{c[3]}-{c[5]}-{c[6]}"
                                           for i, c in enumerate(BIG)])
def test_chunk_attention_in_large_tiles(env, case):  # noqa: F811
    test_chunk_attention(env, case, True)


def test_chunk_many_sequences(env):  # noqa: F811
    """More sequences than a wave has lanes, most of one token, some of none."""
    torch, spax, dev = env
    sizes = [((i * 7) % 5 if i % 3 else 1, i % 40) for i in range(150)]
    sizes = [(a, b if a + b else 1) for a, b in sizes]
    q, kc, vc, table, starts, ln, scales = _chunk_inputs(env, sizes, 4, 2, 64, 8, "fp16", "fp16",
                                                         "heads", 11)
    out = torch.full_like(q, float("nan"))
    lse = torch.full(q.shape[:2], float("nan"), device=dev)
    a = spax.make_chunk_attention(spax.make_kv_cache(kc, vc, table), q, starts, ln, out, lse=lse)
    ws = torch.empty(spax.spax_chunk_attention_workspace_bytes(a), dtype=torch.uint8, device=dev)
    spax.spax_chunk_attention(a, ws)
    torch.cuda.synchronize()
    _chunk_check(q, kc, vc, table, starts, ln, scales, out, lse, 64, "fp16", 0, None)


@pytest.mark.parametrize("kind", ["fp16", "bf16", "e4m3"])
@pytest.mark.parametrize("far", [False, True], ids=["whole", "pieces"])
@pytest.mark.parametrize("others", [0, 3])
def test_chunk_later_tokens_hold_anything(env, kind, far, others):  # noqa: F811
    """NaN and infinities in keys and values of tokens that a row does not see change nothing for it;
    rows that see them get what the formula gives."""
    torch, spax, dev = env
    ct = kind
    qt = "bf16" if kind == "bf16" else "fp16"
    sizes = [(100, 30)] + [(0, 1)] * others      # fewer rows for each sequence: small tiles
    q, kc, vc, table, starts, ln, scales = _chunk_inputs(env, sizes, 2, 1, 64, 16, qt, ct, "heads", 3)
    if far:
        wide = torch.full((1 + others, 1000), -1, dtype=torch.int32, device=dev)
        wide[:, :table.shape[1]] = table
        table = wide
    cache = spax.make_kv_cache(kc, vc, table, *scales)

    def call():
        out = torch.full_like(q, float("nan"))
        a = spax.make_chunk_attention(cache, q, starts, ln, out)
        ws = torch.empty(spax.spax_chunk_attention_workspace_bytes(a), dtype=torch.uint8, device=dev)
        spax.spax_chunk_attention(a, ws)
        torch.cuda.synchronize()
        return _f64(out)[1:101]

    before = call()
    # position 60 is the token of row 30, position 75 that of row 45
    page = table[0].tolist()
    inf, nan = float("inf"), float("nan")
    vc[page[60 // 16], 0, 60 % 16, 5] = nan if ct == "e4m3" else inf
    vc[page[75 // 16], 0, 75 % 16, 5] = nan if ct == "e4m3" else -inf
    vc[page[75 // 16], 0, 75 % 16, 6] = nan
    kc[page[110 // 16], 0, 110 % 16] = nan
    after = call()
    want = before.copy()
    want[30:, :, 5] = nan if ct == "e4m3" else inf
    want[45:, :, 5:7] = nan                      # inf and -inf, and NaN
    want[80:] = nan                              # its scores are NaN
    assert np.array_equal(after, want, equal_nan=True)


def test_chunk_long_tail_under_one_key(env):  # noqa: F811
    """Probabilities far below the row's largest keep their weight in fp16."""
    torch, spax, dev = env
    n, dim = 4096, 64
    kc = torch.zeros(n // 16, 1, 16, dim, dtype=torch.float16, device=dev)
    vc = torch.ones_like(kc)
    kc[0, 0, 0, 0] = 18.0 * 8                     # one key e^18 above the rest, whose value is 0
    vc[0, 0, 0] = 0
    q = torch.zeros(3, 1, dim, dtype=torch.float16, device=dev)
    q[:, 0, 0] = 1.0
    table = torch.arange(n // 16, dtype=torch.int32, device=dev)[None].contiguous()
    starts = torch.tensor([0, 3], dtype=torch.int32, device=dev)
    lens = torch.tensor([n], dtype=torch.int32, device=dev)
    out = torch.empty_like(q)
    a = spax.make_chunk_attention(spax.make_kv_cache(kc, vc, table), q, starts, lens, out)
    ws = torch.empty(spax.spax_chunk_attention_workspace_bytes(a), dtype=torch.uint8, device=dev)
    spax.spax_chunk_attention(a, ws)
    torch.cuda.synchronize()
    tail = np.array([n - 3, n - 2, n - 1]) * np.exp(-18.0)
    ref = (tail / (1 + tail))[:, None]
    # the result is subnormal in fp16 (6e-5): half a step of 2^-24, the weights' 2^-11
    _check(_f64(out)[:, 0], np.broadcast_to(ref, (3, dim)), 2.0 ** -25 + ref * (2.0 ** -11 + 2.0 ** -12), "out")


def test_chunk_of_one_token_is_the_attention_of_one(env):  # noqa: F811
    """One new token per sequence: spax_paged_attention's result within both tolerances."""
    torch, spax, dev = env
    lens = [1, 700, 64, 5]
    q, kc, vc, table, ln, scales = _attention_inputs(env, lens, 8, 2, 128, 16, "fp16", "fp16",
                                                     "heads", 21)
    cache = spax.make_kv_cache(kc, vc, table)
    one, many = torch.empty_like(q), torch.empty_like(q)
    a = spax.make_attention(cache, q, ln, one)
    b = spax.make_chunk_attention(cache, q, torch.arange(5, dtype=torch.int32, device=dev), ln, many)
    for call, need, x in ((spax.spax_paged_attention, spax.spax_attention_workspace_bytes, a),
                          (spax.spax_chunk_attention, spax.spax_chunk_attention_workspace_bytes, b)):
        call(x, torch.empty(need(x), dtype=torch.uint8, device=dev))
    torch.cuda.synchronize()
    # |v| < 5: half a step of each result and of the chunk's weights
    assert float((one.float() - many.float()).abs().max()) <= 5 * 3 * 2.0 ** -11


def _chunk_call(env, q, cache, starts, ln, **kw):
    torch, spax, dev = env
    out = torch.full_like(q, float("nan"))
    lse = torch.full(q.shape[:2], float("nan"), device=dev)
    a = spax.make_chunk_attention(cache, q, starts, ln, out, lse=lse, **kw)
    need = spax.spax_chunk_attention_workspace_bytes(a)
    spax.spax_chunk_attention(a, torch.empty(need, dtype=torch.uint8, device=dev) if need else None)
    torch.cuda.synchronize()
    return out, lse


@pytest.mark.parametrize("far", [False, True], ids=["whole", "pieces"])
@pytest.mark.parametrize("page", [4, 16, 64])
@pytest.mark.parametrize("rows,dim", [(70, 64), (170, 64), (70, 96), (170, 96)])
def test_chunk_pages_that_are_not_there(env, page, far, rows, dim):  # noqa: F811
    """Entries that name no page, in the middle, at the beginning and for all of a token's keys: those
    keys are left out, and a token without any gives zeros and -inf."""
    torch, spax, dev = env
    sizes = [(rows, 300), (5, 0), (3, 200)]
    q, kc, vc, table, starts, ln, scales = _chunk_inputs(env, sizes, 4, 2, dim, page, "fp16", "fp16",
                                                         "heads", 13)
    kc.masked_fill_(torch.isnan(kc), 7.0)
    for s, at in ((0, 100), (0, 260), (0, 345), (2, 0)):
        table[s, at // page] = -1 if at != 260 else kc.shape[0]
    table[1] = -1
    if far:
        wide = torch.full((3, 16384 // page), -1, dtype=torch.int32, device=dev)
        wide[:, :table.shape[1]] = table
        table = wide
    out, lse = _chunk_call(env, q, spax.make_kv_cache(kc, vc, table), starts, ln)
    _chunk_check(q, kc, vc, table, starts, ln, scales, out, lse, dim, "fp16", 0, None)
    first = int(starts[1])
    assert not bool(out[first:first + 5].any()) and bool((lse[first:first + 5] == -float("inf")).all())


@pytest.mark.parametrize("seqs", [250, 300])
def test_chunk_many_sequences_in_pieces(env, seqs):  # noqa: F811
    """More and fewer sequences than those whose steps are counted, some long, one key head."""
    torch, spax, dev = env
    sizes = [((i % 3), 2000 if i % 50 == 0 else 20 + i) for i in range(seqs)]
    q, kc, vc, table, starts, ln, scales = _chunk_inputs(env, sizes, 2, 1, 64, 16, "bf16", "bf16",
                                                         "heads", 17)
    wide = torch.full((seqs, 512), -1, dtype=torch.int32, device=dev)
    wide[:, :table.shape[1]] = table
    out, lse = _chunk_call(env, q, spax.make_kv_cache(kc, vc, wide), starts, ln)
    _chunk_check(q, kc, vc, wide, starts, ln, scales, out, lse, 64, "bf16", 0, None)


@pytest.mark.parametrize("scale", [0.0, -0.125, 3.0])
def test_chunk_scales(env, scale):  # noqa: F811
    """A scale below zero turns the order of the scores, and one of zero makes them equal."""
    torch, spax, dev = env
    q, kc, vc, table, starts, ln, _ = _chunk_inputs(env, [(40, 90)], 4, 2, 64, 16, "fp16", "fp16",
                                                    "heads", 19)
    out, lse = _chunk_call(env, q, spax.make_kv_cache(kc, vc, table), starts, ln, scale=scale)
    k, v = (np.nan_to_num(_f64(t)) for t in (kc, vc))
    rows, ref, ref_lse, mass, reach = oprompt.chunk_attention(
        _f64(q), k, v, table.cpu().numpy(), starts.cpu().numpy(), ln.cpu().numpy(), scale)
    score = 68 * 2.0 ** -24 * reach
    tol = STEP["fp16"] * np.abs(ref) + TINY["fp16"] + mass * (
        2 * score[..., None] + 2048 * 2.0 ** -24 + 2.0 ** -16 + STEP["fp16"])
    _check(_f64(out)[rows], ref, tol, "out")
    _check(_f64(lse)[rows], ref_lse, score + 2048 * 2.0 ** -24 + 2.0 ** -21 * (1 + np.abs(ref_lse)), "lse")


def test_chunk_scores_of_minus_infinity(env):  # noqa: F811
    """Rows whose scores are all -inf give zeros; a single one is left out."""
    torch, spax, dev = env
    kc, vc = (torch.ones(4, 1, 16, 64, dtype=torch.float16, device=dev) for _ in range(2))
    kc[0, 0, 5, 0] = -float("inf")
    vc[0, 0, 5] = 9.0
    q = torch.zeros(40, 2, 64, dtype=torch.float16, device=dev)
    q[:, 0, 0] = 1.0                   # sees -inf at key 5, else 1
    q[:, 1] = 1.0
    q[:, 1, 0] = -float("inf")         # -inf everywhere but at key 5, where it is inf
    table = torch.arange(4, dtype=torch.int32, device=dev)[None].contiguous()
    out, lse = _chunk_call(env, q, spax.make_kv_cache(kc, vc, table),
                           torch.tensor([0, 40], dtype=torch.int32, device=dev),
                           torch.tensor([40], dtype=torch.int32, device=dev), scale=1.0)
    assert bool((out[:, 0] == 1.0).all())
    assert not bool(out[:5, 1].any()) and bool((lse[:5, 1] == -float("inf")).all())
    assert bool(torch.isnan(out[5:, 1]).all())
    seen = torch.tensor([i + 1 - (i >= 5) for i in range(40)], device=dev)
    assert torch.allclose(lse[:, 0], 1.0 + seen.float().log(), atol=1e-5)


def test_chunk_far_in_memory(env):  # noqa: F811
    """Pages more than 2^32 elements into the cache."""
    torch, spax, dev = env
    pages, page, dim = (1 << 22) + 64, 16, 64
    whole = torch.empty(pages, 1, page, dim, dtype=torch.float16, device=dev)
    g = _gen(torch, 23)
    ids = torch.tensor([3, pages - 1, pages - 17, 1 << 21, pages - 2, 9], device=dev)
    near = torch.full((6, 1, page, dim), float("nan"), dtype=torch.float16, device=dev)
    for i in range(6):
        near[i] = _randn(torch, g, (1, page, dim), torch.float16)
        whole[ids[i]] = near[i]
    q = _randn(torch, g, (30, 4, dim), torch.float16)
    starts = torch.tensor([0, 30], dtype=torch.int32, device=dev)
    ln = torch.tensor([91], dtype=torch.int32, device=dev)
    got = []
    for cached, table in ((whole, ids), (near, torch.arange(6, device=dev))):
        cache = spax.make_kv_cache(cached, cached, table.int()[None].contiguous())
        got.append(_chunk_call(env, q, cache, starts, ln))
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
    assert bool(torch.isfinite(got[0][0]).all())


# ------------------------------------------------------------------ product with a packed blob

GEMM = [
    # rows, d_in, d_out, fmt, form, act, bias, residual, y, scale
    (1, 64, [64], "fp16", "plain", "silu", False, None, "fp32", 1.0),
    (3, 1, [64], "fp16", "plain", "silu", True, None, "fp16", 1.0),
    (5, 17, [64, 128], "fp16", "act", "gelu", True, "fp16", "fp16", 0.5),
    (31, 100, [320], "fp16", "act", "silu", False, "fp32", "bf16", 1.0),
    (32, 1024, [256, 64, 64], "fp16", "plain", "silu", True, "bf16", "fp32", 2.0),
    (33, 515, [448], "fp16", "plain", "silu", False, "fp32", "fp32", 1.0),
    (65, 333, [192, 192], "fp16", "gated", "silu", True, None, "fp16", 1.0),
    (2, 2000, [64, 64], "fp16", "gated", "gelu", False, "fp32", "fp32", -1.0),
    (130, 777, [640], "fp16", "plain", "silu", False, None, "fp16", 1.0),
    (257, 130, [576, 576], "fp16", "gated", "silu", False, "fp16", "bf16", 1.0),
    (300, 2051, [832], "fp16", "plain", "silu", True, "fp32", "fp32", 1.0),
    (1, 64, [128], "int4", "plain", "silu", False, None, "fp32", 1.0),
    (7, 129, [128, 384], "int4", "act", "gelu", True, "fp16", "fp16", 0.5),
    (40, 2000, [256], "int4", "plain", "silu", False, "fp32", "fp32", 1.0),
    (100, 300, [384, 384], "int4", "gated", "silu", True, None, "fp16", 1.0),
    (270, 515, [640], "int4", "plain", "silu", False, None, "bf16", 1.0),
]


def _blob(env, d_in, d_out, fmt, seed, scale=None):
    torch, spax, dev = env
    g = _gen(torch, seed)
    Ws = [_randn(torch, g, (d_in, r), torch.float16, d_in ** -0.5 if scale is None else scale)
          for r in d_out]
    kind = spax.FMT_FP16 if fmt == "fp16" else spax.FMT_INT4
    L = spax.spax_layout_init(d_in, d_out, kind, 128, 64)
    packed = torch.empty(int(L.total_bytes), dtype=torch.uint8, device=dev)
    spax.spax_pack_columns(L, Ws, packed)
    O = opack.Layout(d_in, d_out, 0 if fmt == "fp16" else 1, 128, 64)
    torch.cuda.synchronize()
    return L, packed, opack.decode_full_region(O, packed.cpu().numpy())


def _gemm_check(got, x, w, case, bias, residual):
    rows, d_in, d_out, fmt, form, act, _, _, y, scale = case
    opt = lambda t: None if t is None else _f64(t)  # noqa: E731
    ref, t, mass = oprompt.packed_gemm(_f64(x), w, opt(bias), form, act, opt(residual), scale)
    err = mass * ((48 + d_in / 16) * 2.0 ** -23 + (2.0 ** -11 if fmt == "int4" else 0.0))
    err = err + 2.0 ** -23 * np.abs(t)
    if form == "gated":
        half = t.shape[1] // 2
        g, up, eg, eu = t[:, :half], t[:, half:], err[:, :half], err[:, half:]
        a = np.abs(olayer.glu(g, np.ones_like(g), act))
        err = 1.13 * eg * (np.abs(up) + eu) + a * eu + 2.0 ** -15 * a * np.abs(up)
    elif form == "act":
        err = 1.13 * err + 2.0 ** -15 * np.abs(olayer.glu(t, np.ones_like(t), act))
    r = 0.0 if residual is None else np.abs(_f64(residual))
    err = abs(scale) * err + 2.0 ** -23 * (np.abs(ref) + r)
    _check(got, ref, STEP[y] * np.abs(ref) + TINY[y] + err, "y")


def _gemm_case(env, case, seed, pad=0):
    torch, spax, dev = env
    rows, d_in, d_out, fmt, form, act, bias, res, y, scale = case
    L, packed, w = _blob(env, d_in, d_out, fmt, seed)
    g = _gen(torch, seed + 1)
    # what pads a row is NaN
    x = torch.full((rows, (d_in + 7) // 8 * 8 + pad), float("nan"), dtype=torch.float16, device=dev)
    x[:, :d_in] = _randn(torch, g, (rows, d_in), torch.float16)
    x = x[:, :d_in]
    total = sum(d_out)
    width = d_out[0] if form == "gated" else total
    b = _randn(torch, g, (total,), torch.float32, 0.5) if bias else None
    r = None if res is None else _randn(torch, g, (rows, width), _dtype(torch, res))
    out = torch.full((rows, width + 3), float("nan"), dtype=_dtype(torch, y), device=dev)
    return L, packed, w, x, b, r, out


@pytest.mark.parametrize("case", GEMM, ids=[f"{c[0]}x{c[1]}x{sum(c[2])}-{c[3]}-{c[4]}" for c in GEMM])
def test_packed_gemm(env, case):  # noqa: F811
    torch, spax, dev = env
    rows, d_in, d_out, fmt, form, act, bias, res, y, scale = case
    L, packed, w, x, b, r, out = _gemm_case(env, case, rows + d_in, pad=8)
    a = spax.make_packed_gemm(L, packed, x, out[:, 1:-2], bias=b,
                              act=None if form == "plain" else act, gated=form == "gated",
                              residual=r, scale=scale)
    need = spax.spax_packed_gemm_workspace_bytes(a)
    ws = torch.full((need + 256,), 0xFF, dtype=torch.uint8, device=dev)
    print(f"[gemm] {case} workspace {need}", flush=True)
    spax.spax_packed_gemm(a, ws[:need] if need else None)
    torch.cuda.synchronize()
    assert bool((ws[need:] == 0xFF).all())
    got = _f64(out)
    assert np.isnan(got[:, 0]).all() and np.isnan(got[:, -2:]).all()
    _gemm_check(got[:, 1:-2], x, w, case, b, r)


def test_packed_gemm_adds_in_place(env):  # noqa: F811
    """residual may be y itself."""
    torch, spax, dev = env
    case = (70, 256, [192], "fp16", "plain", "silu", False, "fp32", "fp32", 1.0)
    L, packed, w, x, b, r, out = _gemm_case(env, case, 5)
    apart = torch.empty_like(r)
    for y in (apart, r):
        a = spax.make_packed_gemm(L, packed, x, y, residual=r)
        spax.spax_packed_gemm(a, torch.empty(spax.spax_packed_gemm_workspace_bytes(a),
                                             dtype=torch.uint8, device=dev))
    torch.cuda.synchronize()
    assert torch.equal(apart, r)


def test_packed_gemm_rows_are_apart(env):  # noqa: F811
    """NaN and infinities of one row stay in it, and subnormal weights count."""
    torch, spax, dev = env
    d_in, d_out = 96, [128]
    L, packed, w = _blob(env, d_in, d_out, "fp16", 9, scale=2.0 ** -18)
    assert (np.abs(w[w != 0]) < 2.0 ** -14).mean() > 0.99
    x = _randn(torch, _gen(torch, 10), (66, d_in), torch.float16)
    y = torch.empty(66, 128, dtype=torch.float32, device=dev)
    spax.spax_packed_gemm(spax.make_packed_gemm(L, packed, x, y))
    torch.cuda.synchronize()
    ref = _f64(x) @ w
    _check(_f64(y), ref, (np.abs(_f64(x)) @ np.abs(w)) * 60 * 2.0 ** -23, "y")
    x[7, 3] = float("nan")
    x[64, 5] = float("inf")
    z = torch.empty_like(y)
    spax.spax_packed_gemm(spax.make_packed_gemm(L, packed, x, z))
    torch.cuda.synchronize()
    keep = [i for i in range(66) if i not in (7, 64)]
    assert torch.equal(z[keep], y[keep]) and bool(torch.isnan(z[7]).all())
    assert not bool(torch.isfinite(z[64]).any())


@pytest.mark.parametrize("rows,d_in,d_out", [(3, 32768, [65536, 8192]), (70, 32768, [65536, 8192]),
                                             (250, 11000, [10944])])
def test_packed_gemm_far_in_memory(env, rows, d_in, d_out):  # noqa: F811
    """Blobs of more than 2^32 bytes: the last records, and columns at the ends of one.  The last case: k
    cut into pieces between tiles of 256 rows."""
    torch, spax, dev = env
    L = spax.spax_layout_init(d_in, d_out, spax.FMT_FP16, 128, 128 if d_out[0] % 128 == 0 else 64)
    assert L.off_A > 1 << 32 or rows == 250
    packed = torch.zeros(int(L.total_bytes), dtype=torch.uint8, device=dev)
    w = packed[:int(L.off_A)].view(torch.float16).view(d_in, -1)
    used = torch.tensor([0, 5, d_in * 5 // 8, d_in - 17, d_in - 2, d_in - 1], device=dev)
    g = _gen(torch, 29)
    for k in used.tolist():
        w[k] = _randn(torch, g, (w.shape[1],), torch.float16)
    x = torch.zeros(rows, d_in, dtype=torch.float16, device=dev)
    x[:, used] = _randn(torch, g, (rows, 6), torch.float16)
    y = torch.empty(rows, sum(d_out), device=dev)
    a = spax.make_packed_gemm(L, packed, x, y)
    need = spax.spax_packed_gemm_workspace_bytes(a)
    spax.spax_packed_gemm(a, torch.empty(need, dtype=torch.uint8, device=dev) if need else None)
    torch.cuda.synchronize()
    ref = _f64(x[:, used]) @ _f64(w[used, :sum(d_out)])
    mass = np.abs(_f64(x[:, used])) @ np.abs(_f64(w[used, :sum(d_out)]))
    _check(_f64(y), ref, mass * 2.0 ** -20, "y")   # six products, a handful of roundings each


# Sizes at which the rows go by tiles of 128 and of 256, with and without splits of k, with ends of
# every kind inside the last tile.
LARGE = [
    (2000, 130, [2112, 1984], "fp16", "plain", "silu", True, "fp16", "fp16", 1.0),
    (1900, 77, [2112, 2112], "fp16", "gated", "gelu", True, None, "bf16", 1.0),
    (200, 4099, [12224], "fp16", "plain", "silu", False, None, "fp32", 1.0),
    (2000, 200, [2176, 1920], "int4", "act", "silu", False, "fp32", "fp16", 0.5),
    (200, 4099, [12160], "int4", "plain", "silu", True, None, "fp16", 1.0),
    (3001, 130, [4352], "fp16", "plain", "silu", False, "fp32", "fp32", 1.0),
    (3001, 64, [2240, 2240], "fp16", "gated", "silu", False, None, "fp16", 1.0),
    (1000, 4100, [4032], "fp16", "act", "gelu", True, "bf16", "bf16", 1.0),
    (3001, 190, [4352], "int4", "plain", "silu", True, None, "fp16", 1.0),
    (1000, 3000, [2048, 2048], "int4", "gated", "silu", False, None, "fp16", 1.0),
    # k in pieces between tiles of 64 and of 128 rows
    (64, 2000, [2176, 2176], "fp16", "gated", "silu", True, "bf16", "fp16", 1.0),
    (40, 8001, [12032], "int4", "plain", "silu", True, None, "fp16", 1.0),
    (120, 4100, [10240, 10240], "fp16", "gated", "gelu", False, None, "bf16", 1.0),
    (120, 4100, [20480], "int4", "plain", "silu", False, "fp32", "fp32", 1.0),
]


@pytest.mark.parametrize("case", LARGE, ids=[f"{c[0]}x{c[1]}x{sum(c[2])}-{c[3]}-{c[4]}" for c in LARGE])
def test_packed_gemm_of_many_rows(env, case):  # noqa: F811
    """Rows at both ends of every tile, all columns."""
    torch, spax, dev = env
    rows, d_in, d_out, fmt, form, act, bias, res, y, scale = case
    L, packed, w, x, b, r, out = _gemm_case(env, case, rows + d_in)
    out = out[:, :out.shape[1] - 3].contiguous()
    a = spax.make_packed_gemm(L, packed, x, out, bias=b, act=None if form == "plain" else act,
                              gated=form == "gated", residual=r, scale=scale)
    need = spax.spax_packed_gemm_workspace_bytes(a)
    print(f"[gemm] {case} workspace {need}", flush=True)
    spax.spax_packed_gemm(a, torch.full((need,), 0xFF, dtype=torch.uint8, device=dev) if need else None)
    torch.cuda.synchronize()
    assert bool(torch.isfinite(out).all())
    pick = sorted({i for t in range(0, rows, 128) for i in (t, t + 1, t + 31, t + 32, t + 127)
                   if i < rows} | {rows - 1})[:96] + [rows - 2, rows - 1]
    rest = [t[pick] if t is not None else None for t in (x, r, out)]
    _gemm_check(_f64(rest[2]), rest[0], w, case, b, rest[1])
