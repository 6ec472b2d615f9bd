"""Attention of one new token where scores are large and equal: the mean of the values, and lse =
score + ln n.  Scores are exact in 32 bits; the tolerances are those of test_gpu_layer_ops without
the scores' own error, and lse is off by four roundings of the score."""

import numpy as np
import pytest

from tests import test_gpu_layer_ops as ops

pytestmark = pytest.mark.gpu
env = ops.env


@pytest.mark.parametrize("qt,ct", [("fp16", "fp16"), ("bf16", "bf16"), ("fp16", "e4m3")])
@pytest.mark.parametrize("dim,x", [(128, x) for x in (256.0, 2048.0, -2048.0, 8192.0, 49152.0)] + [
    (d, -49152.0) for d in (64, 96, 128, 192, 256)])
@pytest.mark.parametrize("lens", [[40, 3, 0, 7], [509], [9000, 33]])
def test_equal_scores(env, lens, x, dim, qt, ct):
    torch, spax, dev = env
    q, kc, vc, table, ln, _ = ops._attention_inputs(env, lens, 4, 2, dim, 16, qt, ct, "heads", 3)
    q.fill_(x)
    kc.fill_(min(abs(x), 256.0))
    out = torch.full_like(q, float("nan"))
    lse = torch.full(q.shape[:2], float("nan"), device=dev)
    a = spax.make_attention(spax.make_kv_cache(kc, vc, table), q, ln, out, scale=0.125, lse=lse)
    need = spax.spax_attention_workspace_bytes(a)
    spax.spax_paged_attention(a, torch.empty(need, dtype=torch.uint8, device=dev) if need else None)
    torch.cuda.synchronize()
    ref, ref_lse, mass, _ = ops._attention_ref(q, kc, vc, table, ln, [None, None], scale=0.125)
    tol = ops.STEP[qt] * np.abs(ref) + ops.TINY[qt] + mass * ((512 + 4000) * 2.0 ** -24 + 2.0 ** -16)
    ops._check(ops._f64(out), ref, tol, "out")
    fine = np.where(np.isfinite(ref_lse), np.abs(ref_lse), 0.0)
    ops._check(ops._f64(lse), ref_lse, 5000 * 2.0 ** -24 + 2.0 ** -21 * (1 + fine), "lse")
