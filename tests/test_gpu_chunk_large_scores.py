"""Attention of a chunk where scores are large and close to each other: probabilities go by their
differences, whatever their size.

The scores here are exact in 32 bits (sums of integers, or of quarters, below 2^24 of their last
places), so a weight is off by what its exponent's arithmetic costs, (the differences, below 2^5 in
base 2) 2^-23, its rounding, half a step, and the sums' 2048 2^-24; 2^-16 covers the first and
the exponential.  lse = score + ln n is off by four roundings of the score.
"""

import numpy as np
import pytest

from tests import chunk_cases as cases
from tests.test_gpu_layer_ops import STEP, TINY, _check, _dtype, _f64, env  # noqa: F401

pytestmark = pytest.mark.gpu

TYPES = [("fp16", "fp16"), ("bf16", "bf16"), ("fp16", "e4m3")]


def _compare(env, kind, qt, ct, fill, scale):  # noqa: F811
    torch, spax, dev = env
    q, kc, vc, table, starts, lens, _ = cases.build(torch, dev, kind, _dtype(torch, qt),
                                                    _dtype(torch, ct), 41)
    fill(q, kc)
    out, lse = cases.run(spax, torch, q, kc, vc, table, starts, lens, scale)
    rows, *ref = cases.reference(_f64(q), _f64(kc), _f64(vc), table.cpu().numpy(),
                                 starts.cpu().numpy(), lens.cpu().numpy(), scale)
    ref, ref_lse, mass = (x[rows] for x in ref)
    tol = STEP[qt] * np.abs(ref) + TINY[qt] + mass * (2048 * 2.0 ** -24 + 2.0 ** -16 + STEP[qt])
    _check(_f64(out)[rows], ref, tol, "out")
    _check(_f64(lse)[rows], ref_lse, 2048 * 2.0 ** -24 + 2.0 ** -21 * (1 + np.abs(ref_lse)), "lse")


@pytest.mark.parametrize("kind", list(cases.KINDS))
@pytest.mark.parametrize("qt,ct", TYPES)
@pytest.mark.parametrize("x", [256.0, 2048.0, -2048.0, 49152.0])
def test_equal_scores(env, kind, qt, ct, x):  # noqa: F811
    """All scores x k dim scale: the mean of the values."""
    def fill(q, kc):
        q.fill_(x)
        kc.fill_(min(abs(x), 256.0))
    _compare(env, kind, qt, ct, fill, 0.125)


CLOSE = [
    # q0, dims, q1, scale
    (8.0, 1, 1.0, 1.0),                  # 3584 and up to two more
    (8192.0, 1, 1.0, 1.0),               # 3.7e6
    (-8192.0, 1, 1.0, 1.0),
    (32768.0, 1, 4.0, 1.0),              # 1.5e7, up to eight more
    (-65280.0, 32, 1024.0, 2.0 ** -8),   # 9.4e8 / 2^8, up to eight more
]
ORDERS = [(o, k) for o in ("rising", "falling", "mixed") for k in cases.KINDS
          if o == "rising" or k in ("small-pieces", "large-pieces")]


@pytest.mark.parametrize("order,kind", ORDERS, ids=["-".join(x) for x in ORDERS])
@pytest.mark.parametrize("qt,ct", TYPES)
@pytest.mark.parametrize("q0,dims,q1,scale", CLOSE, ids=[str(c[0]) for c in CLOSE])
def test_close_scores(env, order, kind, qt, ct, q0, dims, q1, scale):  # noqa: F811
    """448 q0 in each of `dims` dims, and q1 times a quarter's multiple below two."""
    torch, spax, dev = env

    def fill(q, kc):
        q.zero_()
        kc.zero_()
        q[:, :, :dims] = q0
        q[:, :, -1] = q1
        kc[..., :dims] = 448.0
        pages, hk, page, _ = kc.shape
        n = pages * page
        at = torch.arange(n, device=dev)
        step = {"rising": at * 8 // n, "falling": 7 - at * 8 // n, "mixed": at * 5 % 8}[order]
        kc[..., -1] = (0.25 * step).view(pages, 1, page).to(kc.dtype)
    _compare(env, kind, qt, ct, fill, scale)
