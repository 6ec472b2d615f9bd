"""The operators between the projections where calls or buffers meet: two calls at once, keys and
values in one allocation, one row written twice, many wide rows, windows over 8-bit caches."""

import pytest

from tests import test_gpu_layer_ops as ops

pytestmark = pytest.mark.gpu
env = ops.env


def test_two_attentions_at_once(env):
    """Each on its own stream with its own workspace gives what it gives alone, bit for bit."""
    torch, spax, dev = env
    calls = []
    for seed, lens in ((1, [9000, 40]), (2, [300, 0, 7001])):
        q, kc, vc, table, ln, _ = ops._attention_inputs(env, lens, 8, 2, 128, 16, "fp16", "fp16",
                                                        "heads", seed)
        out = torch.empty_like(q)
        a = spax.make_attention(spax.make_kv_cache(kc, vc, table), q, ln, out)
        need = spax.spax_attention_workspace_bytes(a)
        assert need > 0
        ws = torch.empty(need, dtype=torch.uint8, device=dev)
        spax.spax_paged_attention(a, ws)
        torch.cuda.synchronize()
        calls.append((a, ws, out, out.clone(), torch.cuda.Stream()))
        out.fill_(float("nan"))
    torch.cuda.synchronize()
    for _ in range(10):
        for a, ws, _, _, stream in calls:
            spax.spax_paged_attention(a, ws, stream=stream)
    torch.cuda.synchronize()
    for _, _, out, want, _ in calls:
        assert torch.equal(out, want)


@pytest.mark.parametrize("kind", ["fp16", "e4m3"])
@pytest.mark.parametrize("together", ["pages", "rows"])
def test_keys_and_values_in_one_allocation(env, kind, together):
    """Interleaved page by page or row by row: what is written and read is what two allocations
    hold, and nothing else of the allocation changes."""
    torch, spax, dev = env
    hq, hk, dim, page, pages, n = 8, 2, 64, 16, 12, 3
    t = ops._dtype(torch, kind)
    g = ops._gen(torch, 5)
    apart = [ops._randn(torch, g, (pages, hk, page, dim), t) for _ in range(2)]
    spare = 2 * hk
    if together == "pages":
        whole = torch.zeros(pages, 3, hk, page, dim, device=dev).to(t)  # the third is nobody's
        one = [whole[:, 0], whole[:, 1]]
        rest = whole[:, 2]
    else:
        whole = torch.zeros(pages, page, spare + 1, dim, device=dev).to(t)
        one = [whole[:, :, :hk].transpose(1, 2), whole[:, :, hk:spare].transpose(1, 2)]
        rest = whole[:, :, spare]
    for x, y in zip(one, apart):
        x.copy_(y)
    table = torch.randperm(pages, generator=g, device=dev).int()[:n * 4].view(n, 4)
    lens = torch.tensor([1, 64, 33], dtype=torch.int32, device=dev)
    positions = lens - 1
    inv = torch.rand(dim // 2, generator=g, device=dev)
    q = ops._randn(torch, g, (n, hq, dim), torch.float32)
    k, v = (ops._randn(torch, g, (n, hk, dim), torch.float32) for _ in range(2))
    got = []
    for kc, vc in (apart, one):
        cache = spax.make_kv_cache(kc, vc, table)
        turned = torch.empty(n, hq, dim, dtype=torch.float16, device=dev)
        out = torch.empty_like(turned)
        spax.spax_kv_append(spax.make_kv_append(cache, q, k, v, positions, turned, inv_freq=inv))
        a = spax.make_attention(cache, turned, lens, out)
        need = spax.spax_attention_workspace_bytes(a)
        spax.spax_paged_attention(a, torch.empty(need, dtype=torch.uint8, device=dev) if need else None)
        got.append(out)
    torch.cuda.synchronize()
    assert torch.equal(*got) and bool(torch.isfinite(got[0]).all())
    for x, y in zip(one, apart):
        assert torch.equal(x.contiguous().view(torch.uint8), y.view(torch.uint8))
    assert not bool(rest.contiguous().view(torch.uint8).any())


def test_two_tokens_of_one_row(env):
    """Every value of the row is one of the two tokens', and the rows beside it are left alone."""
    torch, spax, dev = env
    hk, dim = 2, 128
    kc, vc = (torch.full((2, hk, 16, dim), 9.0, dtype=torch.float16, device=dev) for _ in range(2))
    table = torch.tensor([[1, 0]], dtype=torch.int32, device=dev)
    k = torch.empty(4, hk, dim, dtype=torch.float16, device=dev)
    for i in range(4):
        k[i] = i
    seq = torch.zeros(4, dtype=torch.int32, device=dev)
    positions = torch.tensor([5, 5, 20, 5], dtype=torch.int32, device=dev)
    spax.spax_kv_append(spax.make_kv_append(spax.make_kv_cache(kc, vc, table), None, k, k, positions,
                                            None, seq=seq))
    torch.cuda.synchronize()
    for c in (kc, vc):
        row = c[1, :, 5]
        assert bool(((row == 0) | (row == 1) | (row == 3)).all())
        assert bool((c[0, :, 4] == 2).all())
        c[1, :, 5] = 9.0
        c[0, :, 4] = 9.0
        assert bool((c == 9.0).all())


# More rows than the chip has compute units: four items a thread past 8192 values, where fewer
# rows take two.
@pytest.mark.parametrize("layout", ["plain", "odd"])
@pytest.mark.parametrize("case", [
    (256, 8200, "layer", "fp16", "fp32", "fp16", True, "row", 1.0),
    (257, 8200, "layer", "fp16", "fp32", "fp16", True, "row", 1.0),
    (257, 8193, "rms", "bf16", "bf16", "bf16", False, "channel", 0.5),
    (300, 12891, "layer", "bf16", "fp16", "fp32", True, "channel", 2.0),
    (258, 16384, "rms", "fp32", "fp32", "fp16", True, None, 1.0),
])
def test_many_wide_rows(env, case, layout):
    ops.test_norm(env, case, layout)


def test_many_wide_rows_in_place(env):
    torch, spax, dev = env
    g = ops._gen(torch, 8)
    rows, d = 300, 8203
    r, b = (ops._randn(torch, g, (rows, d), torch.float16) for _ in range(2))
    w, p = (1 + 0.1 * torch.randn(d, generator=g, device=dev) for _ in range(2))
    h, x = torch.empty_like(r), torch.empty_like(b)
    spax.spax_residual_norm(spax.make_residual_norm(r, b, h, x, pre_weight=w, post_weight=p))
    spax.spax_residual_norm(spax.make_residual_norm(r, b, r, b, pre_weight=w, post_weight=p))
    torch.cuda.synchronize()
    assert torch.equal(r, h) and torch.equal(b, x) and bool(torch.isfinite(x).all())


@pytest.mark.parametrize("n,longest,hq,hk,dim,window,ct", [
    (40, 3000, 8, 2, 128, 700, "e4m3"), (66, 400, 4, 4, 64, 33, "e4m3"),
    (5, 9000, 16, 1, 96, 4097, "e4m3"),
])
def test_windows_over_an_eight_bit_cache(env, n, longest, hq, hk, dim, window, ct):
    ops.test_attention_many_sequences(env, n, longest, hq, hk, dim, window, ct)


# Widths around the eight values of a thread: the last item of a row then begins inside its
# neighbour's, or the row is shorter than an item.
@pytest.mark.parametrize("layout", ["plain", "odd"])
@pytest.mark.parametrize("d", [2, 6, 8, 9, 15, 17, 511, 513, 8191, 8193, 16383])
@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_widths_around_a_thread(env, d, kind, layout):
    t = ("fp32", "fp16", "bf16")
    ops.test_norm(env, (5, d, kind, t[d % 3], t[(d + 1) % 3], t[(d + 2) % 3], True, "row", 1.0),
                  layout)


@pytest.mark.parametrize("d", [1, 5, 9, 15, 513, 4103, 8201, 16391, 32761])
def test_odd_widths_in_place(env, d):
    torch, spax, dev = env
    g = ops._gen(torch, d)
    for dtype in (torch.float32, torch.bfloat16):
        r, b, e = (ops._randn(torch, g, (7, d), dtype) for _ in range(3))
        w = 1 + 0.1 * torch.randn(d, generator=g, device=dev)
        h, x = torch.empty_like(r), torch.empty_like(b)
        spax.spax_residual_norm(spax.make_residual_norm(r, b, h, x, pre_weight=w, post_weight=w,
                                                        gate=e))
        spax.spax_residual_norm(spax.make_residual_norm(r, b, r, b, pre_weight=w, post_weight=w,
                                                        gate=e))
        torch.cuda.synchronize()
        assert torch.equal(r, h) and torch.equal(b, x) and bool(torch.isfinite(x).all())
