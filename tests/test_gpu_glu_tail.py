"""The activation's tail: far below zero act(g) is tiny but not zero, and times a large `up` it counts."""

import numpy as np
import pytest

from oracle import layer as olayer
from tests import test_gpu_layer_ops as ops

pytestmark = pytest.mark.gpu
env = ops.env


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("xt", ["fp32", "bf16"])
@pytest.mark.parametrize("d", [1024, 5])
def test_far_below_zero(env, act, xt, d):
    """act(g) times 2^100 down to where act(g) is 2^-200.

    The argument u of the exponential is off by 2^-22 |u|, |u| < 140, and the exponential by 2^-22: 2^-14
    of the value."""
    torch, spax, dev = env
    lo, hi = (-135.0, -80.0) if act == "silu" else (-11.7, -10.2)
    gate = torch.linspace(lo, hi, 3 * d, device=dev).view(3, d)
    up = torch.full_like(gate, 2.0 ** 100)
    x = torch.full((3, d), float("nan"), dtype=ops._dtype(torch, xt), device=dev)
    spax.spax_glu(spax.make_glu(gate, up, x, act=act))
    torch.cuda.synchronize()
    ref = olayer.glu(ops._f64(gate), ops._f64(up), act)
    assert (np.abs(ref) > 2.0 ** -100).all()
    ops._check(ops._f64(x), ref, (ops.STEP[xt] + 2.0 ** -14) * np.abs(ref), "x")


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_large_values(env, act):
    """Near the ends of the range: the gate itself, or zero, and products that overflow."""
    torch, spax, dev = env
    big = 3e38
    gate = torch.tensor([[big, -big, 20.0, -20.0, 0.0, -0.0, 1e20, -1e20, 0.5]], device=dev)
    up = torch.tensor([[0.5, 0.5, big, big, big, big, 1e18, 1e18, big]], device=dev)
    x = torch.full_like(gate, float("nan"))
    spax.spax_glu(spax.make_glu(gate, up, x, act=act))
    torch.cuda.synchronize()
    ref = olayer.glu(ops._f64(gate), ops._f64(up), act)
    got = ops._f64(x)
    over = np.abs(ref) > np.finfo(np.float32).max
    assert np.isinf(got[over]).all() and (np.sign(got[over]) == np.sign(ref[over])).all()
    ops._check(got[~over], ref[~over], 2.0 ** -15 * np.abs(ref[~over]) + ops.TINY["fp32"], "x")
    assert np.array_equal(np.signbit(got), np.signbit(ref))
