"""An e4m3 cache holds the value nearest to x / scale: ties of the exact quotient go to the even
value, and a scale whose reciprocal is rounded, or is past the range, changes nothing."""

import numpy as np
import pytest

from tests import test_gpu_layer_ops as ops

pytestmark = pytest.mark.gpu
env = ops.env


def _stored(env, x, scale, src):
    """What the cache holds of rows x [n, heads, 64] with a scale per head."""
    torch, spax, dev = env
    n, hk, dim = x.shape
    kc, vc = (torch.zeros(n, hk, 4, dim, device=dev).to(torch.float8_e4m3fn) for _ in range(2))
    table = torch.arange(n, dtype=torch.int32, device=dev)[:, None].contiguous()
    x = torch.from_numpy(x).to(dev).to(ops._dtype(torch, src))
    s = torch.from_numpy(scale).to(dev)
    spax.spax_kv_append(spax.make_kv_append(
        spax.make_kv_cache(kc, vc, table, s, s), None, x, x,
        torch.zeros(n, dtype=torch.int32, device=dev), None))
    torch.cuda.synchronize()
    got = ops._f64(kc)[:, :, 0]
    assert np.array_equal(got, ops._f64(vc)[:, :, 0], equal_nan=True)
    return got, ops._f64(x)


def _grid():
    import torch
    v = torch.arange(0, 127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    return np.unique(v)


def _nearest(x):
    """The e4m3 value nearest to x (float64), ties to the even one, clamped."""
    grid = _grid()
    a = np.minimum(np.abs(x), 448.0)
    hi = np.clip(np.searchsorted(grid, a), 1, len(grid) - 1)
    lo = hi - 1
    up = (a - grid[lo] > grid[hi] - a) | ((a - grid[lo] == grid[hi] - a) & (hi % 2 == 0))
    y = np.where(up, grid[hi], grid[lo])
    return np.where(np.isnan(x), np.nan, np.copysign(y, x))


def test_the_reference_rounds_as_the_type_does():
    import torch
    x = np.concatenate([_grid(), (_grid()[1:] + _grid()[:-1]) / 2, np.linspace(-448, 448, 9973)])
    want = torch.from_numpy(x).float().to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(_nearest(x.astype(np.float32).astype(np.float64)), want)


@pytest.mark.parametrize("part", range(4))
def test_ties(env, part):
    """x = m * scale exactly, m halfway between two e4m3 values."""
    mid = (_grid()[1:] + _grid()[:-1]) / 2
    scale = (np.arange(1, 1024, 2)[part::4] / 512.0).astype(np.float32)  # odd: few reciprocals are exact
    x = np.zeros((2, len(scale), 64))
    for i in range(2):
        m = mid[64 * i:64 * i + 64]
        x[i, :, :len(m)] = m[None] * scale[:, None].astype(np.float64)
        x[i, ::2] *= -1
    assert np.array_equal(x, x.astype(np.float32))
    got, back = _stored(env, x.astype(np.float32), scale, "fp32")
    want = _nearest(back / scale[None, :, None].astype(np.float64))
    assert np.array_equal(got, want), np.argwhere(got != want)[:5]


@pytest.mark.parametrize("src", ["fp32", "bf16"])
def test_scales_of_every_size(env, src):
    """From the smallest subnormal to near the largest value; zeros stay zeros."""
    rng = np.random.default_rng(3)
    e = np.arange(-149, 127, 2)
    scale = np.ldexp(1.0 + np.where(e > -127, rng.random(len(e)), 0), e).astype(np.float32)
    x = np.clip(rng.standard_normal((3, len(e), 64)) * 100 * scale[None, :, None].astype(np.float64),
                -3e38, 3e38).astype(np.float32)
    x[0, :, :4] = [0.0, -0.0, np.inf, -np.inf]
    x[1, :, 0] = np.nan
    got, back = _stored(env, x, scale, src)
    with np.errstate(over="ignore"):
        # the quotient in 32 bits, as a division gives it, then the nearest value
        want = _nearest((back / scale[None, :, None].astype(np.float64)).astype(np.float32).astype(np.float64))
    bad = ~((got == want) | (np.isnan(got) & np.isnan(want)))
    assert not bad.any(), [(scale[i[1]], back[tuple(i)], got[tuple(i)], want[tuple(i)])
                           for i in np.argwhere(bad)[:5]]
    assert np.isnan(got[1, :, 0]).all() and (got[0, :, :2] == 0).all()
