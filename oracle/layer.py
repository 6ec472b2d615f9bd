"""The operators between the projections in float64, row by row, from their formulas.

Test infrastructure only; shares no code with the package.  Caches are arrays [n_pages, n_kv_heads,
page_size, head_dim] of the values they stand for (scales already applied, or apply = None).
"""

from __future__ import annotations

import numpy as np


def rotate(x, p, inv_freq, interleaved):
    """One head's vector at position p."""
    y = np.array(x, dtype=np.float64)
    n = len(inv_freq)
    for i in range(n):
        a = float(p) * float(inv_freq[i])
        u, w = (2 * i, 2 * i + 1) if interleaved else (i, n + i)
        c, s = np.cos(a), np.sin(a)
        y[u], y[w] = x[u] * c - x[w] * s, x[u] * s + x[w] * c
    return y


def kv_append(q, k, v, positions, seq, table, k_cache, v_cache, inv_freq, interleaved):
    """q_out and the caches after the append (caches are changed in place).  Values are unrounded;
    a caller that stores with a scale divides first."""
    n_pages, _, page_size, _ = k_cache.shape
    q_out = np.zeros(q.shape, dtype=np.float64)
    for t, p in enumerate(positions):
        if p < 0:
            continue
        for h in range(q.shape[1]):
            q_out[t, h] = rotate(q[t, h], p, inv_freq, interleaved)
        s = seq[t]
        if not 0 <= s < table.shape[0] or p // page_size >= table.shape[1]:
            continue
        page = table[s, p // page_size]
        if not 0 <= page < n_pages:
            continue
        for h in range(k.shape[1]):
            k_cache[page, h, p % page_size] = rotate(k[t, h], p, inv_freq, interleaved)
            v_cache[page, h, p % page_size] = v[t, h]
    return q_out


def attention(q, k_cache, v_cache, table, lens, scale, window=0, max_len=None):
    """out, lse and, for error bounds, sum softmax |v| and the largest sum |q_i k_i| |scale|."""
    n_seqs, n_heads, dim = q.shape
    n_pages, n_kv, page_size, _ = k_cache.shape
    group = n_heads // n_kv
    limit = table.shape[1] * page_size
    limit = limit if max_len is None else min(limit, max_len)
    out = np.zeros(q.shape)
    mass = np.zeros(q.shape)
    lse = np.full((n_seqs, n_heads), -np.inf)
    reach = np.zeros((n_seqs, n_heads))
    for s in range(n_seqs):
        n = min(max(int(lens[s]), 0), limit)
        pos = np.arange(max(0, n - window) if window else 0, n)
        page = table[s][pos // page_size]
        pos, page = pos[(page >= 0) & (page < n_pages)], page[(page >= 0) & (page < n_pages)]
        if not len(pos):
            continue
        for h in range(n_heads):
            kk = k_cache[page, h // group, pos % page_size]
            vv = v_cache[page, h // group, pos % page_size]
            score = scale * (kk @ q[s, h])
            top = score.max()
            if top == -np.inf:
                continue
            w = np.exp(score - top)
            out[s, h] = w @ vv / w.sum()
            mass[s, h] = w @ np.abs(vv) / w.sum()
            lse[s, h] = top + np.log(w.sum())
            reach[s, h] = abs(scale) * (np.abs(kk) @ np.abs(q[s, h])).max()
    return out, lse, mass, reach


def norm(x, kind, weight, bias, eps):
    x = np.asarray(x, dtype=np.float64)
    if kind == "layer":
        x = x - x.mean(axis=-1, keepdims=True)
    y = x / np.sqrt((x * x).mean(axis=-1, keepdims=True) + eps)
    if weight is not None:
        y = y * weight
    return y if bias is None else y + bias


def residual_norm(residual, block, kind, pre_w, pre_b, post_w, post_b, gate, scale, eps):
    """h and x."""
    h = 0.0 if residual is None else np.asarray(residual, dtype=np.float64)
    if block is not None:
        t = np.asarray(block, dtype=np.float64)
        if post_w is not None:
            t = norm(t, kind, post_w, post_b, eps)
        if gate is not None:
            t = t * gate
        h = h + scale * t
    return h, norm(h, kind, pre_w, pre_b, eps)


def glu(gate, up, act):
    gate = np.asarray(gate, dtype=np.float64)
    with np.errstate(over="ignore"):
        if act == "silu":
            y = gate / (1.0 + np.exp(-gate))
        else:
            # (1 + tanh u) / 2 = 1 / (1 + exp(-2 u)); the left side loses its digits near tanh = -1
            u = np.sqrt(2.0 / np.pi) * (gate + 0.044715 * gate ** 3)
            y = gate / (1.0 + np.exp(-2.0 * u))
    return y * up
