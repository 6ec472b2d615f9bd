"""Inputs for tests of the attention of a chunk that set single keys and values, and its formula in
float64 for whole sequences at once."""

import numpy as np

# (new, before) of each sequence, heads, kv, dim, room: keys that the page table has room for (0: the
# sequences' own)
KINDS = {
    "small": ([(40, 600), (7, 0)], 2, 1, 64, 0),                 # tiles of 32 rows
    "small-pieces": ([(3, 3000), (9, 700)], 2, 1, 128, 20000),
    "large": ([(130, 700), (101, 37)], 2, 1, 128, 0),            # of 128
    "large-pieces": ([(140, 2500)], 2, 1, 64, 20000),
    "wide": ([(100, 300)] * 8, 32, 32, 64, 2100),                # of 256
    "wide-pieces": ([(100, 300)] * 7 + [(120, 2500)], 32, 32, 128, 20000),
    "dim-96": ([(150, 400)], 6, 2, 96, 0),
    "dim-192": ([(70, 300), (33, 900)], 4, 2, 192, 20000),
    "dim-256": ([(70, 300)], 4, 2, 256, 0),
}


def build(torch, dev, kind, qt, ct, seed, page=16):
    """q, k and v [pages, kv, page, dim] in the sequences' order, table, starts, lens; and
    where(seq, position): page and row."""
    sizes, hq, hk, dim, room = KINDS[kind]
    g = torch.Generator(device="cuda").manual_seed(seed)
    lens = [a + b for a, b in sizes]
    used = [(n + page - 1) // page for n in lens]
    first = np.concatenate([[0], np.cumsum(used)])
    width = max(max(used), room // page)
    table = torch.full((len(sizes), width), -1, dtype=torch.int32)
    for s, u in enumerate(used):
        table[s, :u] = torch.arange(first[s], first[s] + u)
    shape = (int(first[-1]), hk, page, dim)
    kc, vc = (torch.randn(shape, generator=g, device=dev) for _ in range(2))
    starts = np.concatenate([[0], np.cumsum([a for a, _ in sizes])])
    q = torch.randn((int(starts[-1]), hq, dim), generator=g, device=dev).to(qt)
    return (q, kc.to(ct), vc.to(ct), table.to(dev),
            torch.tensor(starts, dtype=torch.int32, device=dev),
            torch.tensor(lens, dtype=torch.int32, device=dev),
            lambda s, p: (int(first[s]) + p // page, p % page))


def run(spax, torch, q, kc, vc, table, starts, lens, scale=None, window=0):
    out = torch.full_like(q, float("nan"))
    lse = torch.full(q.shape[:2], float("nan"), device=q.device)
    a = spax.make_chunk_attention(spax.make_kv_cache(kc, vc, table), q, starts, lens, out, lse=lse,
                                  scale=scale, window=window)
    need = spax.spax_chunk_attention_workspace_bytes(a)
    ws = torch.empty(need, dtype=torch.uint8, device=q.device) if need else None
    spax.spax_chunk_attention(a, ws)
    torch.cuda.synchronize()
    return out, lse


def reference(q, kc, vc, table, starts, lens, scale):
    """The rows of the sequences (float64 arrays, no window, every page there), out, lse and the
    sum of softmax |v|."""
    group = q.shape[1] // kc.shape[1]
    out, mass = np.zeros(q.shape), np.zeros(q.shape)
    lse = np.full(q.shape[:2], -np.inf)
    rows = [np.zeros(0, dtype=int)]
    for s, n in enumerate(int(x) for x in lens):
        new = int(starts[s + 1]) - int(starts[s])
        if new < 1:
            continue
        at = np.arange(int(starts[s]), int(starts[s + 1]))
        rows.append(at)
        pages = table[s, :(n + kc.shape[2] - 1) // kc.shape[2]]
        k, v = (c[pages].transpose(1, 0, 2, 3).reshape(c.shape[1], -1, c.shape[3])[:, :n]
                for c in (kc, vc))
        seen = np.arange(n)[None] <= (n - new + np.arange(new))[:, None]
        for h in range(q.shape[1]):
            score = np.where(seen, scale * (q[at, h] @ k[h // group].T), -np.inf)
            top = score.max(axis=1, keepdims=True)
            w = np.exp(score - np.where(np.isfinite(top), top, 0.0))
            total = w.sum(axis=1, keepdims=True)
            w = w / np.where(total > 0, total, 1.0)
            out[at, h], mass[at, h] = w @ v[h // group], w @ np.abs(v[h // group])
            with np.errstate(divide="ignore"):
                lse[at, h] = (top + np.log(total))[:, 0]
    return np.concatenate(rows), out, lse, mass
