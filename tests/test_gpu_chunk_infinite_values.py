"""Attention of a chunk: a value that is not finite decides its dim for every row that sees its key,
however small the key's weight and wherever the key lies; other dims and rows keep their bits."""

import numpy as np
import pytest

from tests import chunk_cases as cases
from tests.test_gpu_layer_ops import _dtype, _f64, env  # noqa: F811,F401

pytestmark = pytest.mark.gpu

INF, NAN = float("inf"), float("nan")


@pytest.mark.parametrize("kind", list(cases.KINDS))
@pytest.mark.parametrize("qt", ["fp16", "bf16"])
@pytest.mark.parametrize("gap,window", [(0, 0), (10, 250), (30, 0), (30, 250), (110, 0), (110, 250)])
def test_weights_of_any_size(env, kind, qt, gap, window):  # noqa: F811
    """Keys at three places, scores `gap` nats below the rest: inf, -inf, both, NaN, each in a dim of
    its own."""
    torch, spax, dev = env
    q, kc, vc, table, starts, lens, where = cases.build(torch, dev, kind, _dtype(torch, qt),
                                                        _dtype(torch, qt), 43)
    q[:, :, 0] = 1.0
    kc[..., 0] = 0.0
    q[:, :, 1:] *= 0.125
    args = q, kc, vc, table, starts, lens
    sizes = cases.KINDS[kind][0]
    puts = []                                # sequence, position, dim, value
    for s, (new, before) in enumerate(sizes):
        n = new + before
        for i, p in enumerate(sorted({n // 7, n // 2, max(0, n - new // 2 - 1)})):
            page, row = where(s, p)
            kc[page, :, row, 0] = -float(gap)
            puts += [(s, p, 3 + i, INF), (s, p, 10 + i, -INF), (s, p, 20, [INF, -INF, INF][i]),
                     (s, p, 30 + i, NAN)]
    before_, lse = cases.run(spax, torch, *args, scale=1.0, window=window)
    for s, p, d, x in puts:
        page, row = where(s, p)
        vc[page, :, row, d] = x
    after, lse2 = cases.run(spax, torch, *args, scale=1.0, window=window)
    want = _f64(before_)
    for s, (new, before) in enumerate(sizes):
        for i in range(new):
            at = before + i                  # the row's own position
            row, met = int(starts[s]) + i, {}
            for t, p, d, x in puts:
                if t == s and p <= at and not (window and p <= at - window):
                    met.setdefault(d, []).append(x)
            for d, xs in met.items():
                with np.errstate(invalid="ignore"):
                    want[row, :, d] = np.sum(xs)
    assert np.array_equal(_f64(after), want, equal_nan=True)
    assert torch.equal(lse, lse2)


@pytest.mark.parametrize("far", [False, True])
def test_infinities_of_another_sequence(env, far):  # noqa: F811
    """They stay in it, whatever tile its rows share a workgroup with."""
    torch, spax, dev = env
    q, kc, vc, table, starts, lens, where = cases.build(
        torch, dev, "small-pieces" if far else "small", torch.float16, torch.float16, 47)
    args = q, kc, vc, table, starts, lens
    plain, _ = cases.run(spax, torch, *args)
    page, row = where(1, 3)
    vc[page, :, row] = INF
    got, _ = cases.run(spax, torch, *args)
    first = int(starts[1])
    assert torch.equal(got[:first], plain[:first])
    sizes = cases.KINDS["small-pieces" if far else "small"][0]
    seen = [i for i in range(sizes[1][0]) if sizes[1][1] + i >= 3]
    assert bool((got[first:][seen] == INF).all())


def test_values_whose_sum_is_not_finite(env):  # noqa: F811
    """Finite values whose weighted sum passes 32 bits are no infinities: NaN of a score still wins."""
    torch, spax, dev = env
    q, kc, vc, table, starts, lens, where = cases.build(torch, dev, "large", torch.bfloat16,
                                                        torch.bfloat16, 48)
    page, row = where(0, 5)
    kc[page, :, row] = NAN
    page, row = where(0, 300)
    vc[page, :, row, 7] = INF
    got, _ = cases.run(spax, torch, q, kc, vc, table, starts, lens)
    new = cases.KINDS["large"][0][0][0]
    assert bool(torch.isnan(got[:new]).all()) and bool(torch.isfinite(got[new:]).all())
