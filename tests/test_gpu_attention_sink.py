"""One key far above the others with a small value, as attention sinks are: the result is then the
long tail's, whose probabilities are small beside the largest.

Tolerance, per value: half a step of the result; mass = sum softmax |v| times what the fp32
arithmetic before it costs (a score off by (dim + 4) 2^-24 reach moves a weight and the total; chains
of at most 512 additions in a wave and one per piece, of at most 256 shares; a weight that enters
the product as two 16-bit values, 2^-17 of it); and where those values are fp16, the spacing of the
smallest ones: a weight is off by at most 2^-25 of a scale whose largest weight is 2^15 or more, 2^-40 of
the largest weight for each key.
"""

import numpy as np
import pytest

from tests import test_gpu_layer_ops as ops

pytestmark = pytest.mark.gpu
env = ops.env
SHARES = 256


def _sink(env, n, dim, qt, ct, gap, at, hq=4, hk=2, page=16):
    """Keys whose score is 0, but for one of `gap` nats, whose value is 0."""
    torch, spax, dev = env
    g = ops._gen(torch, n + dim)
    pages = (n + page - 1) // page
    kc = torch.zeros(pages, hk, page, dim, device=dev)
    vc = 1 + 0.5 * torch.rand(kc.shape, generator=g, device=dev)
    kc[at // page, :, at % page, 0] = gap
    vc[at // page, :, at % page] = 0
    q = torch.zeros(1, hq, dim, device=dev)
    q[:, :, 0] = 1
    table = torch.randperm(pages, generator=g, device=dev).int()[None]
    inverse = torch.argsort(table[0].long())
    kc, vc = (t[inverse].to(ops._dtype(torch, ct)) for t in (kc, vc))
    return (q.to(ops._dtype(torch, qt)), kc, vc, table,
            torch.tensor([n], dtype=torch.int32, device=dev))


@pytest.mark.parametrize("qt,ct", [("fp16", "fp16"), ("fp16", "e4m3"), ("bf16", "bf16")])
@pytest.mark.parametrize("gap", [9, 13, 18])
@pytest.mark.parametrize("n,dim,at", [
    (100, 64, 0), (100, 128, 99),                 # one wave, beside others
    (509, 128, 0), (509, 96, 300),                # one workgroup
    (4096, 128, 0), (32768, 64, 32767), (32768, 128, 0), (20000, 192, 7), (65536, 256, 31000)])
def test_a_tail_under_one_key(env, n, dim, at, gap, qt, ct):
    torch, spax, dev = env
    q, kc, vc, table, ln = _sink(env, n, dim, qt, ct, gap, at)
    if n == 100:                                  # several of them, so that each takes one wave
        table, ln = table.repeat(3, 1).contiguous(), ln.repeat(3)
        q = q.repeat(3, 1, 1).contiguous()
    out = torch.full_like(q, float("nan"))
    lse = torch.full(q.shape[:2], float("nan"), device=dev)
    a = spax.make_attention(spax.make_kv_cache(kc, vc, table), q, ln, out, scale=1.0, lse=lse)
    need = spax.spax_attention_workspace_bytes(a)
    spax.spax_paged_attention(a, torch.empty(need, dtype=torch.uint8, device=dev) if need else None)
    torch.cuda.synchronize()
    ref, ref_lse, mass, reach = ops._attention_ref(q, kc, vc, table, ln, [None, None], scale=1.0)
    tol = ops._attention_tol(ref, mass, reach, dim, qt, SHARES)
    if qt == "fp16":
        tol = tol + n * 2.0 ** -40 * 1.5
    ops._check(ops._f64(out), ref, tol, "out")
    ops._check(ops._f64(lse), ref_lse, (dim + 4) * 2.0 ** -24 * reach + (512 + SHARES) * 2.0 ** -24
               + 2.0 ** -22 * np.abs(ref_lse), "lse")


@pytest.mark.parametrize("case", ops.ATTENTION, ids=[f"{i}" for i in range(len(ops.ATTENTION))])
def test_within_what_the_shares_allow(env, case):
    """The ordinary cases, with the pieces of a plan's 256 shares in the tolerance."""
    torch, spax, dev = env
    lens, hq, hk, dim, page, qt, ct, window, order, max_len = case
    q, kc, vc, table, ln, scales = ops._attention_inputs(env, lens, hq, hk, dim, page, qt, ct, order,
                                                         sum(lens) + dim)
    out = torch.full_like(q, float("nan"))
    a = spax.make_attention(spax.make_kv_cache(kc, vc, table, *scales), q, ln, out, max_len=max_len,
                            window=window)
    need = spax.spax_attention_workspace_bytes(a)
    spax.spax_paged_attention(a, torch.empty(need, dtype=torch.uint8, device=dev) if need else None)
    torch.cuda.synchronize()
    ref, _, mass, reach = ops._attention_ref(q, kc, vc, table, ln, scales, scale=dim ** -0.5,
                                             window=window, max_len=max_len)
    tol = ops._attention_tol(ref, mass, reach, dim, qt, SHARES)
    ops._check(ops._f64(out), ref, tol, "out")
