"""Attention of a chunk with starts that do not ascend, or lie outside the rows: each counts as no
smaller than those before it, so a sequence has the rows between two running maxima, its last row
its last token; nothing else is written.  Tolerances as in test_gpu_prompt_ops."""

import numpy as np
import pytest

from tests import chunk_cases as cases
from tests.test_gpu_layer_ops import (STEP, TINY, _attention_inputs, _check, _dtype, _f64, _gen,  # noqa: F401
                                      _randn, env)

pytestmark = pytest.mark.gpu

STARTS = {
    "twice": (1000, [0, 500, 0, 500, 1000]),
    "thrice": (1000, [0, 400, 0, 400, 0, 400, 1000]),
    "part of it twice": (700, [0, 300, 150, 450, 400, 700]),
    "down only": (100, [100, 60, 20, 0]),
    "outside": (300, [-50, 40, 1 << 30, -7, 200, 300]),
    "from the end": (600, [300, 600, 0, 300]),
    "many": (500, [(i * 37) % 200 if i % 2 else i * 3 for i in range(160)] + [500]),
}


@pytest.mark.parametrize("name", list(STARTS))
@pytest.mark.parametrize("heads,kv,dim,kind", [(1, 1, 64, "fp16"), (4, 2, 128, "bf16"), (8, 2, 64, "fp16")])
@pytest.mark.parametrize("room", [0, 16384])
def test_starts_of_any_order(env, name, heads, kv, dim, kind, room):  # noqa: F811
    torch, spax, dev = env
    n, raw = STARTS[name]
    starts = np.maximum.accumulate(np.clip(raw, 0, n))
    new = np.diff(starts)
    lens = [int(a) + (i * 13) % 50 for i, a in enumerate(new)]
    _, kc, vc, table, ln, scales = _attention_inputs(env, lens, heads, kv, dim, 16, kind, kind, "heads", 5)
    if room:
        wide = torch.full((len(lens), room // 16), -1, dtype=torch.int32, device=dev)
        wide[:, :table.shape[1]] = table
        table = wide
    q = _randn(torch, _gen(torch, 6), (n, heads, dim), _dtype(torch, kind))
    out, lse = cases.run(spax, torch, q, kc, vc, table,
                         torch.tensor(raw, dtype=torch.int32, device=dev), ln)
    k, v = (np.nan_to_num(_f64(t), nan=0.0, posinf=0.0) for t in (kc, vc))   # unused rows
    rows, *ref = cases.reference(_f64(q), k, v, table.cpu().numpy(), starts, ln.cpu().numpy(),
                                 dim ** -0.5)
    ref, ref_lse, mass = (x[rows] for x in ref)
    score = (dim + 4) * 2.0 ** -24 * 4 * dim ** 0.5 * 4     # |q_i k_i| summed: below 4 dim here
    tol = STEP[kind] * np.abs(ref) + TINY[kind] + mass * (
        2 * score + 2048 * 2.0 ** -24 + 2.0 ** -16 + STEP[kind])
    _check(_f64(out)[rows], ref, tol, "out")
    _check(_f64(lse)[rows], ref_lse, score + 2048 * 2.0 ** -24 + 2.0 ** -21 * (1 + np.abs(ref_lse)),
           "lse")
    rest = np.setdiff1d(np.arange(n), rows)
    assert np.isnan(_f64(out)[rest]).all() and np.isnan(_f64(lse)[rest]).all()
