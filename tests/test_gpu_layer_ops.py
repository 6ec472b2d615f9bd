"""The operators between the projections against the float64 oracle.

Tolerances, per value: half a step of the result's type (2^-11 fp16, 2^-8 bf16, 2^-24 fp32, 2^-4
e4m3 of the value, plus half the smallest subnormal) and the fp32 arithmetic before it:

* append: sine and cosine come from a fraction of a turn held to 2^-25, an angle error of 2 pi
  2^-25 < 2^-22, and their evaluation and the two products and sum add a few 2^-24:
  2^-20 (|x| + |y|) of the pair.  A scaled value adds one division, 2^-24 of the value; a value
  near the middle of two e4m3 values may then go either way, which half a step covers.
* attention: the error of a score is at most (dim + 4) 2^-24 reach (reach = scale sum |q_i k_i|),
  and it moves a weight and the total by that much each; sums of weights and of weighted values
  run over chains of at most 512 fp32 additions (a wave's tiles) and one per piece that is
  joined; a weight enters as two 16-bit values, 2^-17 of it or less.  Together mass * (2 (dim +
  4) 2^-24 reach + (512 + pieces) 2^-24 + 2^-16), mass = sum softmax |v|.
* norms: a sum of d squares in chains of at most 32 additions per thread and 22 across the
  workgroup is off by 54 2^-24 of itself, half of that for its root; 2^-17 covers two norms and
  the handful of products, on top of the error of h carried through the second norm's division
  by the row's root mean square.
* glu: the exponential is good to 2^-22 and its argument to 2^-22 |u|, |u| < 90 where the result
  is not zero: 2^-15 of the value for gelu, 2^-20 for silu.
"""

import numpy as np
import pytest

from oracle import layer as olayer

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def env():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import activation_sparse_tiered_amd as spax
    return torch, spax, torch.device("cuda:0")


STEP = {"fp32": 2.0 ** -24, "fp16": 2.0 ** -11, "bf16": 2.0 ** -8, "e4m3": 2.0 ** -4}
TINY = {"fp32": 2.0 ** -126, "fp16": 2.0 ** -25, "bf16": 2.0 ** -126, "e4m3": 2.0 ** -10}


def _dtype(torch, name):
    return {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16,
            "e4m3": torch.float8_e4m3fn}[name]


def _f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def _check(got, ref, tol, what):
    got = np.asarray(got)
    assert got.shape == ref.shape, what
    same = (got == ref) | (np.isnan(got) & np.isnan(ref))
    bad = ~same & ~(np.abs(got - ref) <= tol)
    if bad.any():
        at = tuple(int(i[0]) for i in np.nonzero(bad))
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.size} values off, first at {at}: "
                             f"{got[at]} for {ref[at]}, allowed {np.broadcast_to(tol, ref.shape)[at]}")


def _gen(torch, seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(torch, g, shape, dtype, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


# ------------------------------------------------------------------ append

APPEND = [
    # tokens, heads, kv, dim, rot, pairs, page, src, out, cache, order
    (1, 32, 32, 128, 128, "halves", 16, "fp32", "fp16", "fp16", "heads"),
    (5, 8, 2, 64, 64, "neighbours", 4, "fp16", "fp16", "fp16", "tokens"),
    (7, 5, 1, 96, 48, "halves", 8, "bf16", "bf16", "bf16", "heads"),
    (3, 4, 4, 192, 192, "neighbours", 32, "fp32", "bf16", "bf16", "tokens"),
    (9, 16, 2, 256, 128, "halves", 64, "fp16", "fp16", "e4m3", "heads"),
    (4, 6, 3, 96, 0, "halves", 16, "bf16", "bf16", "e4m3", "tokens"),
    (6, 3, 1, 64, 20, "halves", 16, "fp32", "fp16", "fp16", "heads"),       # pairs one by one
    (6, 3, 1, 64, 20, "neighbours", 16, "fp16", "fp16", "e4m3", "heads"),
    (700, 5, 2, 64, 64, "halves", 16, "fp16", "fp16", "fp16", "heads"),     # a prompt
    (5, 0, 2, 128, 128, "halves", 16, "fp16", "fp16", "fp16", "heads"),     # keys and values only
]


@pytest.mark.parametrize("case", APPEND, ids=[str(c[:7]) for c in APPEND])
@pytest.mark.parametrize("odd", [False, True], ids=["fused", "unaligned"])
def test_append(env, case, odd):
    torch, spax, dev = env
    n, hq, hk, dim, rot, pairs, page, src, out, cache, order = case
    g = _gen(torch, n * 1000 + dim)
    seqs, width = max(3, min(n, 8)), 40
    pages = 50
    shape = (pages, hk, page, dim) if order == "heads" else (pages, page, hk, dim)
    kc, vc = (_randn(torch, g, shape, _dtype(torch, cache)) for _ in range(2))
    if order == "tokens":
        kc, vc = kc.transpose(1, 2), vc.transpose(1, 2)
    table = torch.full((seqs, width), -1, dtype=torch.int32, device=dev)
    order_ = torch.randperm(pages, generator=g, device=dev).int()
    if n > 100:                                    # one sequence's prompt, and its neighbours'
        seq = torch.zeros(n, dtype=torch.int32, device=dev)
        positions = torch.arange(n, dtype=torch.int32, device=dev) - 3   # three rows of padding
        table[0, :40] = order_[:40]
        positions[-1] = width * page               # past the table
        seq[-2], positions[-2] = seqs, 0           # no such sequence
        seq[-3], positions[-3] = -1, 0
    else:
        seq = torch.arange(n, dtype=torch.int32, device=dev) % seqs
        positions = torch.randint(0, width * page, (n,), generator=g, device=dev).int()
        positions[0] = 0
        slots = seq.long() * width + (positions // page).long()
        table.view(-1)[slots] = order_[torch.unique(slots, return_inverse=True)[1]]
        if n > 4:
            positions[3] = -7                      # padding
            table[seq[4].long(), positions[4].long() // page] = pages   # no such page
    extra = 3 if odd else 0
    row = _randn(torch, g, (n, (hq + 2 * hk) * dim + extra), _dtype(torch, src))
    row = row[:, extra:]
    q = row[:, :hq * dim].unflatten(1, (hq, dim)) if hq else None
    k = row[:, hq * dim:(hq + hk) * dim].unflatten(1, (hk, dim))
    v = row[:, (hq + hk) * dim:].unflatten(1, (hk, dim))
    q_out = torch.full((n, hq, dim), float("nan"), dtype=_dtype(torch, out), device=dev) if hq else None
    inv = (1e4 ** (-torch.arange(0, max(rot, 1), 2, device=dev).double() / max(rot, 1))).float()
    scale = [torch.rand(hk, generator=g, device=dev) * 0.1 + 0.01 for _ in range(2)]
    if cache != "e4m3":
        scale = [None, None]
    want_k, want_v = _f64(kc), _f64(vc)
    ks, vs = (np.ones(hk) if s is None else _f64(s) for s in scale)
    kf, vf = _f64(k) / ks[None, :, None], _f64(v) / vs[None, :, None]
    c = spax.make_kv_cache(kc, vc, table, *scale)
    a = spax.make_kv_append(c, q, k, v, positions, q_out, seq=seq,
                            inv_freq=inv if rot else None, interleaved=pairs == "neighbours")
    print(f"[append] {case} odd={odd}", flush=True)
    spax.spax_kv_append(a)
    torch.cuda.synchronize()
    before = want_k.copy(), want_v.copy()
    pos, tab = positions.cpu().numpy(), table.cpu().numpy()
    freq = _f64(inv) if rot else np.zeros(0)
    qf = _f64(q) if hq else np.zeros((n, 0, dim))
    ref_q = olayer.kv_append(qf, kf, vf, pos, seq.cpu().numpy(), tab, want_k, want_v, freq,
                             pairs == "neighbours")

    def tol(ref, name, pair):
        return STEP[name] * np.abs(ref) + TINY[name] + 2.0 ** -20 * pair

    if hq:
        biggest = np.abs(qf).max(axis=-1, keepdims=True) * 2
        _check(_f64(q_out), ref_q, tol(ref_q, out, biggest), "q_out")
    for got, ref, old, src_rows, name in ((kc, want_k, before[0], kf, "k"),
                                          (vc, want_v, before[1], vf, "v")):
        got = _f64(got)
        if cache == "e4m3":
            ref = np.clip(ref, -448, 448)
        touched = ref != old
        # rows that no token names keep their bits
        rows_touched = touched.any(axis=-1)
        assert np.array_equal(got[~rows_touched], old[~rows_touched])
        assert rows_touched.any()
        _check(got, ref, tol(ref, cache, 2 * np.abs(src_rows).max()), name)


def test_append_far_positions(env):
    """A million tokens in, an angle in 32 bits would be off by 2^-4."""
    torch, spax, dev = env
    g = _gen(torch, 5)
    page, dim = 16, 128
    positions = torch.tensor([1048575, 999999, 524289], dtype=torch.int32, device=dev)
    table = torch.full((3, 65536), -1, dtype=torch.int32, device=dev)
    for s, p in enumerate(positions.tolist()):
        table[s, p // page] = s
    kc = torch.zeros(3, 1, page, dim, dtype=torch.float16, device=dev)
    vc = torch.zeros_like(kc)
    k = _randn(torch, g, (3, 1, dim), torch.float32)
    inv = (5e5 ** (-torch.arange(0, dim, 2, device=dev).double() / dim)).float()
    a = spax.make_kv_append(spax.make_kv_cache(kc, vc, table), None, k, k, positions, None,
                            inv_freq=inv)
    spax.spax_kv_append(a)
    torch.cuda.synchronize()
    for s, p in enumerate(positions.tolist()):
        ref = olayer.rotate(_f64(k)[s, 0], p, _f64(inv), False)
        _check(_f64(kc)[s, 0, p % page], ref, 2.0 ** -11 * np.abs(ref) + 2.0 ** -20 * 8, f"at {p}")


def test_append_e4m3_range_and_specials(env):
    """Past the range: +-448; NaN stays NaN; 16-bit caches keep infinities."""
    torch, spax, dev = env
    nan, inf = float("nan"), float("inf")
    x = torch.zeros(1, 1, 64, device=dev)
    x[0, 0, :10] = torch.tensor([448, 449, -1e9, inf, -inf, nan, 0.0, -0.0, 2.0 ** -9, 2.0 ** -11],
                                device=dev)
    table = torch.zeros(1, 1, dtype=torch.int32, device=dev)
    zero = torch.zeros(1, dtype=torch.int32, device=dev)
    want = np.array([448, 448, -448, 448, -448, nan, 0, 0, 2.0 ** -9, 0])
    for name in ("e4m3", "fp16"):
        kc = torch.zeros(1, 1, 4, 64, device=dev).to(_dtype(torch, name))
        vc = kc.clone()
        spax.spax_kv_append(spax.make_kv_append(spax.make_kv_cache(kc, vc, table), None, x, x, zero,
                                                None))
        torch.cuda.synchronize()
        got = _f64(kc)[0, 0, 0, :10]
        ref = want if name == "e4m3" else _f64(x.half())[0, 0, :10]
        assert np.array_equal(got, ref, equal_nan=True), got
        assert np.array_equal(_f64(vc)[0, 0, 0], _f64(kc)[0, 0, 0], equal_nan=True)
        assert not _f64(kc)[0, 0, 1:].any()


def test_append_rotates_in_place(env):
    """q_out may be q: in a fused row of the cache's type, k and v lie beside it."""
    torch, spax, dev = env
    g = _gen(torch, 8)
    n, hq, hk, dim, page = 5, 4, 2, 64, 8
    row = _randn(torch, g, (n, (hq + 2 * hk) * dim), torch.bfloat16)
    q = row[:, :hq * dim].unflatten(1, (hq, dim))
    k = row[:, hq * dim:(hq + hk) * dim].unflatten(1, (hk, dim))
    v = row[:, (hq + hk) * dim:].unflatten(1, (hk, dim))
    kc = torch.zeros(n, hk, page, dim, dtype=torch.bfloat16, device=dev)
    vc = torch.zeros_like(kc)
    table = torch.arange(n, dtype=torch.int32, device=dev)[:, None].contiguous()
    positions = torch.arange(n, dtype=torch.int32, device=dev)
    inv = torch.rand(dim // 2, generator=g, device=dev)
    apart = torch.empty(n, hq, dim, dtype=torch.bfloat16, device=dev)
    cache = spax.make_kv_cache(kc, vc, table)
    spax.spax_kv_append(spax.make_kv_append(cache, q, k, v, positions, apart, inv_freq=inv))
    kept = row[:, hq * dim:].clone()
    spax.spax_kv_append(spax.make_kv_append(cache, q, k, v, positions, q, inv_freq=inv))
    torch.cuda.synchronize()
    assert torch.equal(q.contiguous(), apart) and torch.equal(row[:, hq * dim:], kept)


# ------------------------------------------------------------------ attention

ATTENTION = [
    # lens, heads, kv, dim, page, type, cache, window, order, max_len
    ([1], 1, 1, 128, 4, "fp16", "fp16", 0, "heads", None),
    ([0, 1, 2, 31, 32, 33, 63, 64, 65], 4, 2, 64, 16, "fp16", "fp16", 0, "heads", None),
    ([0, 127, 128, 129, 500], 32, 32, 128, 16, "fp16", "fp16", 0, "heads", None),
    ([700, 5, 0, 256], 8, 2, 128, 64, "bf16", "bf16", 0, "tokens", None),
    ([4000], 8, 2, 128, 16, "fp16", "fp16", 0, "heads", None),             # shared out
    ([4001, 17, 0, 1030], 8, 1, 128, 32, "bf16", "e4m3", 0, "heads", None),
    ([2500, 40], 20, 1, 96, 8, "fp16", "fp16", 0, "tokens", None),         # two groups of heads
    ([300, 1000], 36, 2, 64, 16, "fp16", "e4m3", 0, "heads", None),
    ([900, 33], 10, 2, 192, 16, "bf16", "bf16", 0, "heads", None),
    ([900, 33], 6, 2, 96, 16, "bf16", "e4m3", 0, "tokens", None),
    ([900, 34], 4, 2, 192, 16, "fp16", "e4m3", 0, "heads", None),
    ([1500, 70], 16, 2, 256, 32, "fp16", "fp16", 0, "heads", None),
    ([1500, 71], 16, 2, 256, 32, "bf16", "e4m3", 0, "heads", None),
    ([1500, 70, 3], 8, 2, 128, 16, "fp16", "fp16", 1, "heads", None),      # windows
    ([1500, 70, 3], 8, 2, 128, 16, "fp16", "fp16", 33, "tokens", None),
    ([5000, 70, 3, 1000], 8, 2, 64, 16, "bf16", "bf16", 1000, "heads", None),
    ([5000, 70, 3, 1000], 8, 8, 64, 16, "bf16", "e4m3", 1001, "heads", None),
    ([600, 100, -5], 8, 2, 128, 16, "fp16", "fp16", 0, "heads", 200),      # clamped
]


def _attention_inputs(env, lens, hq, hk, dim, page, qt, ct, order, seed):
    torch, spax, dev = env
    g = _gen(torch, seed)
    n = len(lens)
    width = max(1, (max(lens) + page - 1) // page)
    used = [max(0, (v + page - 1) // page) for v in lens]
    pages = sum(used) + 2
    ids = torch.randperm(pages, generator=g, device=dev).int().tolist()
    table = torch.full((n, width), -1, dtype=torch.int32)
    at = 0
    for s, u in enumerate(used):
        table[s, :u] = torch.tensor(ids[at:at + u], dtype=torch.int32)
        at += u
    shape = (pages, hk, page, dim) if order == "heads" else (pages, page, hk, dim)
    kc, vc = (_randn(torch, g, shape, _dtype(torch, ct)) for _ in range(2))
    if order == "tokens":
        kc, vc = kc.transpose(1, 2), vc.transpose(1, 2)
    # rows past each sequence's end and unused pages hold NaN and infinities
    for s, v in enumerate(lens):
        if v > 0 and v % page:
            p = int(table[s, v // page])
            kc[p, :, v % page:] = float("nan")
            vc[p, :, v % page:] = float("nan") if s % 2 or ct == "e4m3" else float("inf")
    for p in ids[at:]:
        kc[p] = float("nan")
        vc[p] = float("nan")
    scales = [None, None]
    if ct == "e4m3":
        scales = [torch.rand(hk, generator=g, device=dev) + 0.5 for _ in range(2)]
    q = _randn(torch, g, (n, hq, dim), _dtype(torch, qt))
    return q, kc, vc, table.to(dev), torch.tensor(lens, dtype=torch.int32, device=dev), scales


def _attention_ref(q, kc, vc, table, lens, scales, **kw):
    k, v = _f64(kc), _f64(vc)
    if scales[0] is not None:
        k, v = k * _f64(scales[0])[None, :, None, None], v * _f64(scales[1])[None, :, None, None]
    return olayer.attention(_f64(q), k, v, table.cpu().numpy(), lens.cpu().numpy(), **kw)


def _attention_tol(ref, mass, reach, dim, kind, pieces):
    e = 2 * (dim + 4) * 2.0 ** -24 * reach[..., None] + (512 + pieces) * 2.0 ** -24 + 2.0 ** -16
    return STEP[kind] * np.abs(ref) + TINY[kind] + mass * e


@pytest.mark.parametrize("case", ATTENTION, ids=[f"{i}-{c[1]}-{c[2]}-{c[3]}-{c[5]}-{c[6]}"
                                                 for i, c in enumerate(ATTENTION)])
@pytest.mark.parametrize("far", [False, True], ids=["own", "far"])
def test_attention(env, case, far):
    """far: a max_len well past the longest sequence, as a table with room for more has."""
    torch, spax, dev = env
    lens, hq, hk, dim, page, qt, ct, window, order, max_len = case
    q, kc, vc, table, ln, scales = _attention_inputs(env, lens, hq, hk, dim, page, qt, ct, order,
                                                     sum(lens) + dim)
    if far:
        if max_len is not None:
            pytest.skip("max_len is the case's own")
        wide = torch.full((len(lens), 20000 // page), -1, dtype=torch.int32, device=dev)
        wide[:, :table.shape[1]] = table
        table = wide
    out = torch.full_like(q, float("nan"))
    lse = torch.full((len(lens), hq), float("nan"), device=dev)
    cache = spax.make_kv_cache(kc, vc, table, *scales)
    a = spax.make_attention(cache, q, ln, out, max_len=max_len, window=window, lse=lse)
    need = spax.spax_attention_workspace_bytes(a)
    ws = torch.full((need + 256,), 0xFF, dtype=torch.uint8, device=dev)
    print(f"[attention] {case} far={far} workspace {need}", flush=True)
    spax.spax_paged_attention(a, ws[:need] if need else None)
    torch.cuda.synchronize()
    assert bool((ws[need:] == 0xFF).all())
    ref, ref_lse, mass, reach = _attention_ref(q, kc, vc, table, ln, scales, scale=dim ** -0.5,
                                               window=window, max_len=max_len)
    _check(_f64(out), ref, _attention_tol(ref, mass, reach, dim, qt, 4000), "out")
    tol = (dim + 4) * 2.0 ** -24 * reach + 5000 * 2.0 ** -24 + 2.0 ** -22 * np.where(
        np.isfinite(ref_lse), np.abs(ref_lse), 0)
    _check(_f64(lse), ref_lse, tol, "lse")
    again = torch.full_like(q, float("nan"))
    spax.spax_paged_attention(spax.make_attention(cache, q, ln, again, max_len=max_len,
                                                  window=window),
                              ws[:need] if need else None)
    torch.cuda.synchronize()
    assert torch.equal(out, again)


def _many(n, longest, seed):
    r = np.random.default_rng(seed)
    lens = np.exp(r.uniform(0, np.log(longest), n)).astype(int)
    lens[r.random(n) < 0.15] = 0
    return [int(v) for v in lens]


@pytest.mark.parametrize("n,longest,hq,hk,dim,window,ct", [
    (64, 700, 4, 2, 64, 0, "fp16"), (65, 700, 4, 2, 64, 0, "fp16"), (130, 300, 2, 1, 128, 0, "fp16"),
    (200, 2000, 4, 4, 64, 50, "fp16"), (257, 90, 8, 8, 64, 0, "fp16"), (70, 900, 3, 1, 96, 0, "e4m3"),
    (300, 40, 2, 1, 256, 0, "fp16"), (129, 1500, 2, 2, 192, 400, "fp16"), (90, 500, 34, 2, 64, 0, "fp16"),
])
def test_attention_many_sequences(env, n, longest, hq, hk, dim, window, ct):
    """More sequences than a wave has lanes, of all lengths and in any order: some go to one wave
    each, some are cut, some are empty."""
    torch, spax, dev = env
    for seed in range(2):
        lens = _many(n, longest, seed * 1000 + n)
        if seed:
            lens = [0] * 70 + lens[70:] if n > 70 else [0] * (n - 1) + [longest]
        q, kc, vc, table, ln, scales = _attention_inputs(env, lens, hq, hk, dim, 16, "fp16", ct,
                                                         "heads", seed + n)
        out = torch.full_like(q, float("nan"))
        lse = torch.full((n, hq), float("nan"), device=dev)
        a = spax.make_attention(spax.make_kv_cache(kc, vc, table, *scales), q, ln, out,
                                window=window, lse=lse)
        need = spax.spax_attention_workspace_bytes(a)
        print(f"[attention] {n} sequences up to {longest}, workspace {need}", flush=True)
        spax.spax_paged_attention(a, torch.empty(max(1, need), dtype=torch.uint8, device=dev))
        torch.cuda.synchronize()
        ref, ref_lse, mass, reach = _attention_ref(q, kc, vc, table, ln, scales, scale=dim ** -0.5,
                                                   window=window)
        _check(_f64(out), ref, _attention_tol(ref, mass, reach, dim, "fp16", 300), "out")
        assert np.array_equal(np.isfinite(_f64(lse)), np.isfinite(ref_lse))


@pytest.mark.parametrize("n", [40, 4000])
def test_attention_scores_at_the_edges(env, n):
    """Large scores of both signs, a negative and a zero scale, keys that are -inf, entries that
    name no page."""
    torch, spax, dev = env
    hq, hk, dim, page = 4, 2, 64, 16
    q, kc, vc, table, ln, scales = _attention_inputs(env, [n, n], hq, hk, dim, page, "fp16", "fp16",
                                                     "heads", 77 + n)
    q *= 30
    q[1, :, 0] = 1.0
    p = int(table[1, 1])
    kc[p, :, 3, 0] = float("-inf")      # two keys of sequence 1 whose score is -inf
    kc[p, 0, 5, 0] = float("-inf")
    table[0, 1] = -3                    # pages of sequence 0 that do not exist
    table[0, 2] = kc.shape[0]
    for scale in (0.125, -0.125, 0.0):
        if scale <= 0:                  # -inf * 0 and +inf scores have no finite answer
            kc[p, :, 3, 0] = 0.0
            kc[p, 0, 5, 0] = 0.0
        out = torch.empty_like(q)
        a = spax.make_attention(spax.make_kv_cache(kc, vc, table), q, ln, out, scale=scale)
        need = spax.spax_attention_workspace_bytes(a)
        spax.spax_paged_attention(a, torch.empty(max(1, need), dtype=torch.uint8, device=dev))
        torch.cuda.synchronize()
        ref, _, mass, reach = _attention_ref(q, kc, vc, table, ln, scales, scale=scale)
        reach = np.where(np.isfinite(reach), reach, np.abs(scale) * 30 * 16 * dim)
        _check(_f64(out), ref, _attention_tol(ref, mass, reach, dim, "fp16", 4000), f"scale {scale}")


@pytest.mark.parametrize("n", [40, 4000])
def test_attention_of_nothing(env, n):
    """Every key at -inf, or on no page: zeros and -inf, whatever way the keys are shared out."""
    torch, spax, dev = env
    q, kc, vc, table, ln, _ = _attention_inputs(env, [n, n], 4, 2, 64, 16, "fp16", "fp16",
                                                "heads", 5)
    q[:] = 0.5
    kc[:] = float("-inf")
    table[1] = -1
    out = torch.full_like(q, float("nan"))
    lse = torch.full((2, 4), float("nan"), device=dev)
    a = spax.make_attention(spax.make_kv_cache(kc, vc, table), q, ln, out, lse=lse)
    need = spax.spax_attention_workspace_bytes(a)
    spax.spax_paged_attention(a, torch.empty(max(1, need), dtype=torch.uint8, device=dev))
    torch.cuda.synchronize()
    assert not out.any() and bool((lse == float("-inf")).all())


def test_attention_strided_rows_are_left_alone(env):
    """q and out inside wider rows; what lies between them stays."""
    torch, spax, dev = env
    hq, hk, dim, page = 8, 2, 64, 16
    q, kc, vc, table, ln, scales = _attention_inputs(env, [100, 3000, 0], hq, hk, dim, page, "fp16",
                                                     "fp16", "heads", 9)
    wide = torch.full((3, hq, dim + 16), 7.0, dtype=torch.float16, device=dev)
    row = torch.empty(3, hq * dim + 64, dtype=torch.float16, device=dev)
    row[:, 64:] = q.flatten(1)
    a = spax.make_attention(spax.make_kv_cache(kc, vc, table), row[:, 64:].unflatten(1, (hq, dim)),
                            ln, wide[..., :dim])
    need = spax.spax_attention_workspace_bytes(a)
    spax.spax_paged_attention(a, torch.empty(need, dtype=torch.uint8, device=dev))
    torch.cuda.synchronize()
    ref, _, mass, reach = _attention_ref(q, kc, vc, table, ln, scales, scale=dim ** -0.5)
    _check(_f64(wide[..., :dim]), ref, _attention_tol(ref, mass, reach, dim, "fp16", 4000), "out")
    assert bool((wide[..., dim:] == 7.0).all())


def test_attention_cache_past_32_bit_offsets(env):
    """Pages beyond 2^31 elements (and 2^32 bytes) of one cache tensor."""
    torch, spax, dev = env
    hk, page, dim = 8, 64, 128
    pages = 2 ** 31 // (hk * page * dim) + 40
    kc = torch.empty(pages, hk, page, dim, dtype=torch.float16, device=dev)
    vc = torch.empty_like(kc)
    g = _gen(torch, 3)
    ids = [pages - 1, 0, pages - 20, 1, pages - 3]
    for p in ids:
        kc[p] = _randn(torch, g, kc[p].shape, kc.dtype)
        vc[p] = _randn(torch, g, kc[p].shape, kc.dtype)
    table = torch.tensor([ids], dtype=torch.int32, device=dev)
    ln = torch.tensor([300], dtype=torch.int32, device=dev)
    q = _randn(torch, g, (1, 32, dim), torch.float16)
    out = torch.empty_like(q)
    cache = spax.make_kv_cache(kc, vc, table)
    # the newest key arrives by append
    k = _randn(torch, g, (1, hk, dim), torch.float16)
    spax.spax_kv_append(spax.make_kv_append(cache, None, k, k, ln - 1, None))
    a = spax.make_attention(cache, q, ln, out)
    need = spax.spax_attention_workspace_bytes(a)
    spax.spax_paged_attention(a, torch.empty(max(1, need), dtype=torch.uint8, device=dev))
    torch.cuda.synchronize()
    assert torch.equal(kc[ids[4], :, 299 % page], k[0])
    few_k, few_v = kc[torch.tensor(ids, device=dev)], vc[torch.tensor(ids, device=dev)]
    del kc, vc, cache, a
    ref, _, mass, reach = _attention_ref(q, few_k, few_v,
                                         torch.arange(5, dtype=torch.int32)[None], ln, [None, None],
                                         scale=dim ** -0.5)
    _check(_f64(out), ref, _attention_tol(ref, mass, reach, dim, "fp16", 100), "out")
    torch.cuda.empty_cache()


# ------------------------------------------------------------------ norms

NORM = [
    # rows, d, kind, block, residual, x, post, gate, scale
    (1, 4096, "rms", "fp32", "fp32", "fp16", False, None, 1.0),
    (5, 4096, "rms", "bf16", "bf16", "bf16", True, "channel", 0.5),
    (3, 1, "rms", "fp32", "fp32", "fp32", True, "row", 1.0),
    (3, 7, "layer", "fp16", "fp16", "fp16", True, "row", 2.0),
    (4, 63, "layer", "fp32", "fp16", "bf16", False, "channel", 1.0),
    (4, 64, "rms", "fp16", "fp32", "fp16", True, None, 1.0),
    (2, 5003, "layer", "fp16", "fp32", "fp16", True, "row", 1.0),
    (2, 8192, "layer", "bf16", "fp32", "bf16", True, "channel", 0.3),
    (3, 8200, "rms", "fp32", "bf16", "fp32", True, "row", 1.0),
    (2, 11008, "layer", "bf16", "fp32", "fp16", False, None, 1.0),
    (2, 16385, "rms", "fp16", "fp16", "fp16", True, "row", 1.0),
    (2, 20000, "layer", "fp32", "fp32", "fp32", True, "row", 1.0),
    (2, 32768, "layer", "fp32", "fp32", "fp16", True, "channel", -1.0),
    (1000, 257, "rms", "bf16", "bf16", "bf16", False, "row", 1.0),
    (1200, 1024, "layer", "bf16", "bf16", "bf16", True, "row", 1.0),
]


@pytest.mark.parametrize("case", NORM, ids=[str(c[:6]) for c in NORM])
@pytest.mark.parametrize("layout", ["plain", "padded", "odd"])
def test_norm(env, case, layout):
    torch, spax, dev = env
    rows, d, kind, bt, rt, xt, post, gate, scale = case
    g = _gen(torch, rows * 7 + d)
    extra = {"plain": 0, "padded": 8, "odd": 3}[layout]

    def mat(kind_, s=1.0, value=None):
        t = torch.full((rows, (d + 7) // 8 * 8 + extra), 7.0, dtype=_dtype(torch, kind_), device=dev)
        t = t[:, :d] if layout != "plain" else t[:, :d].contiguous()
        if value is None:
            t.copy_(_randn(torch, g, (rows, d), t.dtype, s))
        return t

    def vec():
        return 1 + 0.1 * torch.randn(d, generator=g, device=dev)

    layer = kind == "layer"
    b, r, h, x = mat(bt, 0.7), mat(rt, 2.0), mat(rt, value=0), mat(xt, value=0)
    r += 0.5
    gt = None if gate is None else mat(bt, 0.5) if gate == "row" else vec().to(_dtype(torch, bt))
    pw, pb = (vec(), vec() if layer else None) if post else (None, None)
    qw, qb = vec(), vec() if layer else None
    print(f"[norm] {case} {layout}", flush=True)
    spax.spax_residual_norm(spax.make_residual_norm(
        r, b, h, x, kind=kind, pre_weight=qw, pre_bias=qb, post_weight=pw, post_bias=pb, gate=gt,
        scale=scale, eps=1e-5))
    torch.cuda.synchronize()

    def np_(t):
        return None if t is None else _f64(t)

    rh, rx = olayer.residual_norm(np_(r), np_(b), kind, np_(qw), np_(qb), np_(pw), np_(pb), np_(gt),
                                  scale, 1e-5)
    # the branch's own size bounds its error: the norm is within 2^-17, the rest a few 2^-24
    branch = np.abs(rh - np_(r))
    if post and layer:
        branch = branch + abs(scale) * np.abs(np_(pb)) * (1 if gt is None else np.abs(np_(gt)))
    eh = 2.0 ** -17 * branch + 2.0 ** -22 * np.abs(np_(r))
    if post and layer:   # subtracting the mean of values near each other
        eh = eh + 2.0 ** -17 * abs(scale) * (1 if gt is None else np.abs(np_(gt)))
    _check(np_(h), rh, STEP[rt] * np.abs(rh) + TINY[rt] + eh, "residual_out")
    c = rh - rh.mean(axis=-1, keepdims=True) if layer else rh
    rms = np.sqrt((c * c).mean(axis=-1, keepdims=True) + 1e-5)
    worst = eh.max(axis=-1, keepdims=True) + 2.0 ** -20 * np.abs(rh).max(axis=-1, keepdims=True)
    ex = np.abs(np_(qw)) * (2 * worst / rms) + 2.0 ** -17 * (np.abs(rx) + (0 if qb is None else
                                                                       np.abs(np_(qb))))
    _check(np_(x), rx, STEP[xt] * np.abs(rx) + TINY[xt] + ex, "x")
    for t, name in ((h, "residual_out"), (x, "x")):
        if layout != "plain":
            whole = t.as_strided((rows, t.stride(0)), (t.stride(0), 1))
            assert bool((whole[:, d:] == 7.0).all()), f"{name}: wrote past its rows"


def test_norm_parts_left_out(env):
    """No block (the first norm of a stack), no residual, no x, no residual_out, no weight."""
    torch, spax, dev = env
    g = _gen(torch, 4)
    r, b = _randn(torch, g, (3, 100), torch.float32), _randn(torch, g, (3, 100), torch.float16)
    w = 1 + _randn(torch, g, (100,), torch.float32, 0.1)
    x, h = torch.empty(3, 100, device=dev), torch.empty(3, 100, device=dev)
    tol = 2.0 ** -16

    def run(*a, **kw):
        spax.spax_residual_norm(spax.make_residual_norm(*a, **kw))
        torch.cuda.synchronize()

    run(r, None, None, x, pre_weight=w)
    assert np.allclose(_f64(x), olayer.norm(_f64(r), "rms", _f64(w), None, 1e-5), rtol=tol, atol=tol)
    run(None, b, h, x, scale=0.5)
    assert np.array_equal(_f64(h), 0.5 * _f64(b))
    assert np.allclose(_f64(x), olayer.norm(0.5 * _f64(b), "rms", None, None, 1e-5), rtol=tol, atol=tol)
    run(r, b, h, None)
    assert np.allclose(_f64(h), _f64(r) + _f64(b), rtol=2.0 ** -23, atol=0)
    run(r, b, None, x, kind="layer")
    assert np.allclose(_f64(x), olayer.norm(_f64(r) + _f64(b), "layer", None, None, 1e-5), rtol=tol,
                       atol=tol)
    # in place: the stream over itself, x over the block
    want_h, want_x = olayer.residual_norm(_f64(r), _f64(b), "rms", _f64(w), None, None, None, None,
                                          1.0, 1e-5)
    run(r, b, r, b, pre_weight=w)
    assert np.allclose(_f64(r), want_h, rtol=2.0 ** -23, atol=0)
    assert np.allclose(_f64(b), want_x, rtol=2.0 ** -11 + tol, atol=2.0 ** -20)
    run(r[:0], b[:0], h[:0], x[:0])   # no rows


def test_norm_keeps_large_offsets_and_specials(env):
    """A layer norm of a row far from zero, rows of zeros, infinities and NaN."""
    torch, spax, dev = env
    g = _gen(torch, 6)
    d = 1000
    r = _randn(torch, g, (5, d), torch.float32)
    r[0] += 4096.0
    r[1] = 0.0
    r[2, 5] = float("inf")
    r[3, 7] = float("nan")
    x = torch.empty_like(r)
    spax.spax_residual_norm(spax.make_residual_norm(r, None, None, x, kind="layer", eps=1e-5))
    torch.cuda.synchronize()
    ref = olayer.norm(_f64(r)[[0, 1, 4]], "layer", None, None, 1e-5)
    # row 0: a mean of 4096 in 32 bits is within 54 * 2^-24 * 4096 = 2^-6.2 of its sum's error bound
    _check(_f64(x)[[0, 1, 4]], ref, np.array([[2.0 ** -6], [0.0], [2.0 ** -16]]) + 2.0 ** -16 * np.abs(ref),
           "layer norm")
    assert torch.isnan(x[2]).all() and torch.isnan(x[3]).all()


# ------------------------------------------------------------------ gated activation

@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("rows,d,src,xt,extra", [
    (1, 11008, "fp32", "fp16", 0), (3, 1, "fp32", "fp32", 0), (3, 7, "bf16", "bf16", 0),
    (2, 2049, "fp16", "fp16", 0), (5, 2048, "fp16", "fp32", 4), (4, 1000, "bf16", "bf16", 1),
    (700, 129, "fp32", "bf16", 3), (300, 4096, "bf16", "bf16", 0)])
def test_glu(env, act, rows, d, src, xt, extra):
    torch, spax, dev = env
    g = _gen(torch, d + rows)
    y = _randn(torch, g, (rows, 2 * d + extra), _dtype(torch, src), 3.0)
    gate, up = y[:, :d], y[:, d:2 * d]
    if d > 8:
        gate[0, :8] = torch.tensor([0.0, -0.0, 80.0, -80.0, 300.0, -300.0, 6e4, -6e4], device=dev)
    x = torch.full((rows, d + extra), 7.0, dtype=_dtype(torch, xt), device=dev)[:, :d]
    spax.spax_glu(spax.make_glu(gate, up, x, act=act))
    torch.cuda.synchronize()
    ref = olayer.glu(_f64(gate), _f64(up), act)
    tol = (STEP[xt] + (2.0 ** -15 if act == "gelu" else 2.0 ** -20)) * np.abs(ref) + TINY[xt] + 1e-30
    big = 65504.0 + 16 if xt == "fp16" else np.inf
    keep = np.abs(ref) < big
    _check(_f64(x)[keep], ref[keep], tol[keep], "x")
    assert np.isinf(_f64(x)[~keep]).all()
    if extra:
        assert bool((x.as_strided((rows, d + extra), (d + extra, 1))[:, d:] == 7.0).all())


def test_glu_in_place(env):
    torch, spax, dev = env
    g = _gen(torch, 2)
    y = _randn(torch, g, (9, 200), torch.bfloat16)
    want = torch.empty(9, 100, dtype=torch.bfloat16, device=dev)
    spax.spax_glu(spax.make_glu(y[:, :100], y[:, 100:], want))
    for half in (0, 1):
        z = y.clone()
        spax.spax_glu(spax.make_glu(z[:, :100], z[:, 100:], z[:, 100 * half:100 * half + 100]))
        torch.cuda.synchronize()
        other = slice(100, 200) if half == 0 else slice(0, 100)
        assert torch.equal(z[:, 100 * half:100 * half + 100], want)
        assert torch.equal(z[:, other], y[:, other])


# ------------------------------------------------------------------ streams, graphs

def test_calls_take_the_current_stream(env):
    """Work queued on a side stream before the call is seen by it, through the current stream
    and through an explicit one."""
    torch, spax, dev = env
    side = torch.cuda.Stream()
    y = torch.zeros(64, 20000, device=dev)
    x = torch.zeros(64, 10000, dtype=torch.float16, device=dev)
    a = spax.make_glu(y[:, :10000], y[:, 10000:], x)
    big = torch.randn(4096, 4096, device=dev)
    torch.cuda.synchronize()
    for explicit in (False, True):
        y.zero_()
        x.zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            for _ in range(20):
                big @ big
            y.fill_(1.0)
            if not explicit:
                spax.spax_glu(a)
        if explicit:
            spax.spax_glu(a, stream=side)
        side.synchronize()
        assert bool((x == torch.tensor(1 / (1 + np.exp(-1.0))).half().to(dev)).all())


def test_graphs_that_share_a_workspace(env):
    """Append, attention, norm and glu captured into two graphs over one workspace, replayed in
    turn with eager calls between; each replay reads the lengths and inputs of its moment."""
    torch, spax, dev = env
    hq, hk, dim, page = 8, 2, 64, 16
    sets = []
    for seed in (1, 2):
        lens = [2000 + seed, 40 * seed]
        q, kc, vc, table, ln, sc = _attention_inputs(env, [v + 64 for v in lens], hq, hk, dim, page,
                                                     "fp16", "fp16", "heads", seed)
        kc.nan_to_num_(0.0)
        vc.nan_to_num_(0.0, posinf=0.0)
        ln -= 64
        g = _gen(torch, seed)
        k = _randn(torch, g, (2, hk, dim), torch.float32)
        positions = ln - 1
        inv = torch.rand(dim // 2, generator=g, device=dev)
        q32 = _randn(torch, g, (2, hq, dim), torch.float32)
        cache = spax.make_kv_cache(kc, vc, table)
        out = torch.empty_like(q)
        x = torch.empty(2, hq * dim, dtype=torch.float16, device=dev)
        z = torch.empty(2, hq * dim // 2, dtype=torch.float16, device=dev)
        ops = (spax.make_kv_append(cache, q32, k, k, positions, q, inv_freq=inv),
               spax.make_attention(cache, q, ln, out),
               spax.make_residual_norm(None, out.flatten(1), None, x),
               spax.make_glu(x[:, :hq * dim // 2], x[:, hq * dim // 2:], z))
        sets.append((ops, ln, positions, q32, (q, kc, vc, out, x, z)))
    need = max(spax.spax_attention_workspace_bytes(s[0][1]) for s in sets)
    assert need > 0
    ws = torch.empty(need, dtype=torch.uint8, device=dev)

    def run(ops):
        spax.spax_kv_append(ops[0])
        spax.spax_paged_attention(ops[1], ws)
        spax.spax_residual_norm(ops[2])
        spax.spax_glu(ops[3])

    graphs = []
    for ops, *_ in sets:
        run(ops)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            run(ops)
        graphs.append(graph)
    for turn in range(4):
        for (ops, ln, positions, q32, outs), graph in zip(sets, graphs):
            ln += 1
            positions += 1
            q32 *= -0.9
            graph.replay()
            torch.cuda.synchronize()
            got = [t.clone() for t in outs]
            for t in (outs[0], *outs[3:]):
                t.fill_(float("nan"))
            run(ops)
            torch.cuda.synchronize()
            for t, w in zip(outs, got):
                assert torch.equal(t, w), turn
