"""The operators of many tokens at once in float64, from their formulas.

Test infrastructure only; shares no code with the package.
"""

from __future__ import annotations

import numpy as np

from .layer import attention, glu, norm


def head_norm(x, kind, weight, bias, eps):
    """x [tokens, heads, dim]; weight and bias [dim], [heads, dim] or None (no norm)."""
    return np.asarray(x, dtype=np.float64) if weight is None else norm(x, kind, weight, bias, eps)


def chunk_attention(q, k_cache, v_cache, table, starts, lens, scale, window=0, max_len=None):
    """Each new token as a sequence of its own that ends with it: out, lse, mass, reach as
    oracle.layer.attention's for the rows of the sequences, and which rows those are."""
    limit = table.shape[1] * k_cache.shape[2]
    limit = limit if max_len is None else min(limit, max_len)
    rows, seqs, ends = [], [], []
    for s in range(len(lens)):
        new = int(starts[s + 1]) - int(starts[s])
        n = min(max(int(lens[s]), 0), limit)
        for i in range(new):
            rows.append(int(starts[s]) + i)
            seqs.append(s)
            ends.append(max(0, n - new + i + 1))
    rows = np.array(rows, dtype=np.int64)
    out, lse, mass, reach = attention(q[rows], k_cache, v_cache, table[np.array(seqs, dtype=int)],
                                      np.array(ends), scale, window)
    return rows, out, lse, mass, reach


def packed_gemm(x, w, bias, form, act, residual, scale):
    """y for w [d_in, d_out_total], and for error bounds: the sums of |x w| that reach each column
    of t, and t."""
    x, w = np.asarray(x, dtype=np.float64), np.asarray(w, dtype=np.float64)
    t, mass = x @ w, np.abs(x) @ np.abs(w)
    if bias is not None:
        t = t + bias
    if form == "gated":
        half = t.shape[1] // 2
        u = glu(t[:, :half], t[:, half:], act)
    elif form == "act":
        u = glu(t, np.ones_like(t), act)
    else:
        u = t
    y = scale * u
    return (y if residual is None else y + residual), t, mass
