"""The operators of many tokens as they are used: a prompt through a decoder layer, the step after it,
whole layers with normed heads, captured graphs, two calls at once."""

import numpy as np
import pytest

import synth
from oracle import pack as opack
from tests.test_gpu_layer_ops import _attention_inputs, _dtype, _f64, _gen, _randn, env  # noqa: F401
from tests.test_gpu_layers import Stack

pytestmark = pytest.mark.gpu
EPS = 1e-5


def _ws(torch, n):
    return torch.empty(n, dtype=torch.uint8, device="cuda") if n else None


class PromptLayer:
    """One layer of width d, hq heads of dim over hk key heads, inner width f, fp16 or int4 blobs; its
    tokens come in chunks through the operators of many tokens, or one by one through
    spax_decode_layers with every column of the tier FULL."""

    def __init__(self, env, d, hq, hk, dim, f, fmt, most, seed):  # noqa: F811
        torch, spax, dev = env
        self.torch, self.spax, self.dev = torch, spax, dev
        g = _gen(torch, seed)
        self.d, self.hq, self.hk, self.dim, self.f = d, hq, hk, dim, f
        self.shapes = dict(qkv=(d, [hq * dim, hk * dim, hk * dim]), o=(hq * dim, [d]),
                           gate_up=(d, [f, f]), down=(f, [d]))
        self.blobs = {}
        for k, (name, (a, outs)) in enumerate(self.shapes.items()):
            L = spax.spax_layout_init(a, outs, fmt, 128, 64 if fmt == 0 else 128)
            Ws = [torch.from_numpy(synth.weights(seed, a, r, k, m)).to(dev) for m, r in enumerate(outs)]
            packed = torch.empty(int(L.total_bytes), dtype=torch.uint8, device=dev)
            spax.spax_pack_columns(L, Ws, packed)
            self.blobs[name] = (L, packed)
        pages = most // 16 + 3
        self.kc, self.vc = (_randn(torch, g, (pages, hk, 16, dim), torch.float16) for _ in range(2))
        self.table = torch.randperm(pages, generator=g, device=dev).int()[None, :most // 16 + 1].contiguous()
        self.cache = spax.make_kv_cache(self.kc, self.vc, self.table)
        self.inv = (1e4 ** (-torch.arange(0, dim, 2, device=dev).double() / dim)).float()

        def weight(n):
            return 1 + 0.1 * torch.randn(n, generator=g, device=dev)
        self.norm = spax.make_head_norm(weight(dim), weight(dim), eps=EPS)
        self.w1, self.w2, self.w3 = weight(d), weight(d), weight(d)

    def new(self, *shape, dtype=None):
        return self.torch.empty(*shape, dtype=dtype or self.torch.float16, device=self.dev)

    def prompt(self, tokens, before):
        """h and the next layer's x of a chunk of tokens (rows of the stream before the layer), and
        everything that was called, in order."""
        torch, spax = self.torch, self.spax
        n, d, hq, hk, dim = tokens.shape[0], self.d, self.hq, self.hk, self.dim
        h, x0, x1, x2 = self.new(n, d, dtype=torch.float32), *(self.new(n, d) for _ in range(3))
        y = self.new(n, (hq + 2 * hk) * dim, dtype=torch.float32)
        q, k, v = (t.unflatten(1, (-1, dim)) for t in y.split([hq * dim, hk * dim, hk * dim], 1))
        turned, att, act = self.new(n, hq, dim), self.new(n, hq, dim), self.new(n, self.f)
        positions = torch.arange(before, before + n, dtype=torch.int32, device=self.dev)
        seq = torch.zeros(n, dtype=torch.int32, device=self.dev)
        starts = torch.tensor([0, n], dtype=torch.int32, device=self.dev)
        lens = torch.tensor([before + n], dtype=torch.int32, device=self.dev)
        append = spax.make_kv_append(self.cache, q, k, v, positions, turned, seq=seq,
                                     inv_freq=self.inv)
        attention = spax.make_chunk_attention(self.cache, turned, starts, lens, att)
        gemms = dict(
            qkv=spax.make_packed_gemm(*self.blobs["qkv"], x0, y),
            o=spax.make_packed_gemm(*self.blobs["o"], att.flatten(1), h, residual=h),
            gate_up=spax.make_packed_gemm(*self.blobs["gate_up"], x1, act, act="silu", gated=True),
            down=spax.make_packed_gemm(*self.blobs["down"], act, h, residual=h))
        ws = {name: _ws(torch, spax.spax_packed_gemm_workspace_bytes(a)) for name, a in gemms.items()}
        attention_ws = _ws(torch, spax.spax_chunk_attention_workspace_bytes(attention))
        first = spax.make_residual_norm(tokens, None, h, x0, pre_weight=self.w1, eps=EPS)
        second = spax.make_residual_norm(h, None, None, x1, pre_weight=self.w2, eps=EPS)
        third = spax.make_residual_norm(h, None, None, x2, pre_weight=self.w3, eps=EPS)

        def gemm(name):
            return lambda: spax.spax_packed_gemm(gemms[name], ws[name])
        calls = [lambda: spax.spax_residual_norm(first), gemm("qkv"),
                 lambda: spax.spax_kv_append_normed(append, self.norm),
                 lambda: spax.spax_chunk_attention(attention, attention_ws), gemm("o"),
                 lambda: spax.spax_residual_norm(second), gemm("gate_up"), gemm("down"),
                 lambda: spax.spax_residual_norm(third)]
        return h, x2, calls

    def decode(self, token, before):
        """h and x of one token through spax_decode_layers."""
        torch, spax, dev = self.torch, self.spax, self.dev
        d, hq, hk, dim, f = self.d, self.hq, self.hk, self.dim, self.f
        h, x0, x1, x2 = self.new(1, d, dtype=torch.float32), *(self.new(1, d) for _ in range(3))
        turned, att, act = self.new(1, hq, dim), self.new(1, hq, dim), self.new(1, f)
        xs = dict(qkv=x0, o=att, gate_up=x1, down=act)
        phases, ys, keep = {}, {}, []
        for name, (a, outs) in self.shapes.items():
            lists = [self.new(a, dtype=torch.uint8)] + [self.new(a, dtype=torch.int32) for _ in range(2)]
            lists.append(self.new(3, dtype=torch.int32))
            ys[name] = self.new(sum(outs), dtype=torch.float32)
            phases[name] = spax.make_phase(*self.blobs[name], xs[name], spax.topk_params(a, 0), *lists,
                                           ys[name])
            keep.append(lists)
        y = ys["qkv"][None]
        q, k, v = (t.unflatten(1, (-1, dim)) for t in y.split([hq * dim, hk * dim, hk * dim], 1))
        position = torch.tensor([before], dtype=torch.int32, device=dev)
        lens = torch.tensor([before + 1], dtype=torch.int32, device=dev)
        gu = ys["gate_up"][None]
        layer = spax.make_layer(
            phases["qkv"], spax.make_kv_append(self.cache, q, k, v, position, turned, inv_freq=self.inv),
            spax.make_attention(self.cache, turned, lens, att), phases["o"],
            spax.make_residual_norm(h, ys["o"][None], h, x1, pre_weight=self.w2, eps=EPS),
            phases["gate_up"], spax.make_glu(gu[:, :f], gu[:, f:], act), phases["down"],
            spax.make_residual_norm(h, ys["down"][None], h, x2, pre_weight=self.w3, eps=EPS),
            head_norm=self.norm)
        spax.spax_residual_norm(spax.make_residual_norm(token, None, h, x0, pre_weight=self.w1, eps=EPS))
        spax.spax_decode_layers([layer], _ws(torch, spax.spax_layers_workspace_bytes([layer])))
        torch.cuda.synchronize()
        return h, x2


SIZES = [(512, 8, 2, 64, 1408, 0), (256, 4, 4, 128, 256, 0), (512, 4, 1, 128, 768, 1)]


@pytest.mark.parametrize("size", SIZES, ids=str)
def test_a_prompt_in_chunks_and_the_step_after_it(env, size):  # noqa: F811
    """The last token of a prompt taken whole, at the end of chunks, and by a decode step after a
    prompt one shorter: the same stream.  The paths round the same values to fp16 (queries, cache,
    attention, gate, norms), each to half a step of 2^-11 after sums in other orders, weights of the
    attention by another 2^-12 and int4 weights by 2^-11: under ten relative errors of 2^-11, which
    a product of random weights carries on about as they are (its rows' norms are equal), so 2^-7 of
    what the layer adds to the stream, in the 2-norm."""
    torch, spax, dev = env
    layer = PromptLayer(env, *size, 700, 31)
    n = 577
    tokens = torch.randn(n, size[0], generator=_gen(torch, 3), device=dev)
    h, x, calls = layer.prompt(tokens, 0)
    for c in calls:
        c()
    torch.cuda.synchronize()
    keys = layer.kc.clone()
    whole_h, whole_x = _f64(h), _f64(x)
    assert np.isfinite(whole_h).all()
    added = whole_h - _f64(tokens)

    def near(got, rows):
        off = np.linalg.norm(_f64(got) - whole_h[rows]) / np.linalg.norm(added[rows])
        assert off <= 2.0 ** -7, off

    at = 0
    for chunk in (130, 1, 64, 5, n - 200):
        part_h, part_x, calls = layer.prompt(tokens[at:at + chunk].contiguous(), at)
        for c in calls:
            c()
        torch.cuda.synchronize()
        near(part_h, slice(at, at + chunk))
        at += chunk
    assert at == n
    # another way through the products may round a key the other way, by a step of its value
    same = (layer.kc == keys).float().mean()
    assert float(same) > 0.99 and torch.allclose(layer.kc.float(), keys.float(), rtol=2.0 ** -8, atol=2.0 ** -8)
    step_h, step_x = layer.decode(tokens[-1:].contiguous(), n - 1)
    near(step_h, slice(n - 1, n))
    off = np.linalg.norm(_f64(step_x) - whole_x[-1:]) / np.linalg.norm(whole_x[-1:])
    assert off <= 2.0 ** -7, off


def test_a_prompt_captured(env):  # noqa: F811
    """A chunk's way through the layer as a graph: replays after changed inputs, between eager work, are
    the eager calls' results bit for bit."""
    torch, spax, dev = env
    layer = PromptLayer(env, 512, 8, 2, 64, 1408, 0, 1500, 5)
    tokens = torch.randn(40, 512, generator=_gen(torch, 3), device=dev)
    h, x, calls = layer.prompt(tokens, 1300)        # the attention is cut into pieces
    graph = torch.cuda.CUDAGraph()
    for c in calls:
        c()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        for c in calls:
            c()
    for i in range(4):
        tokens.mul_(-0.5).add_(0.1 * i)
        for c in calls:
            c()
        torch.cuda.synchronize()
        want = h.clone(), x.clone(), layer.kc.clone()
        h.fill_(float("nan"))
        x.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip((h, x, layer.kc), want))
        torch.randn(1000, device=dev).sum().item()


def test_two_calls_at_once(env):  # noqa: F811
    """Attentions and products on streams of their own with workspaces of their own: each what it is
    alone, bit for bit."""
    torch, spax, dev = env
    calls = []
    for seed, (new, before) in ((1, (7, 9000)), (2, (40, 5000))):
        q1, kc, vc, table, ln, _ = _attention_inputs(env, [new + before], 8, 2, 128, 16, "fp16",
                                                     "fp16", "heads", seed)
        q = _randn(torch, _gen(torch, seed), (new, 8, 128), torch.float16)
        out = torch.empty_like(q)
        a = spax.make_chunk_attention(spax.make_kv_cache(kc, vc, table), q,
                                      torch.tensor([0, new], dtype=torch.int32, device=dev), ln, out)
        ws = _ws(torch, spax.spax_chunk_attention_workspace_bytes(a))
        assert ws is not None
        calls.append((lambda stream, a=a, ws=ws: spax.spax_chunk_attention(a, ws, stream=stream), out))
    for seed, rows in ((3, 5), (4, 60)):
        L = spax.spax_layout_init(2048, [512], spax.FMT_FP16, 128, 64)
        packed = torch.empty(int(L.total_bytes), dtype=torch.uint8, device=dev)
        spax.spax_pack_columns(L, [_randn(torch, _gen(torch, seed), (2048, 512), torch.float16, 0.02)],
                               packed)
        x, y = _randn(torch, _gen(torch, seed), (rows, 2048), torch.float16), torch.empty(rows, 512, device=dev)
        a = spax.make_packed_gemm(L, packed, x, y)
        ws = _ws(torch, spax.spax_packed_gemm_workspace_bytes(a))
        assert ws is not None
        calls.append((lambda stream, a=a, ws=ws: spax.spax_packed_gemm(a, ws, stream=stream), y))
    torch.cuda.synchronize()
    want = []
    for call, out in calls:
        call(None)
        torch.cuda.synchronize()
        want.append(out.clone())
        assert bool(torch.isfinite(out).all())
        out.fill_(float("nan"))
    streams = [torch.cuda.Stream() for _ in calls]
    torch.cuda.synchronize()
    for _ in range(10):
        for (call, _), stream in zip(calls, streams):
            call(stream)
    torch.cuda.synchronize()
    for (_, out), w in zip(calls, want):
        assert torch.equal(out, w)


def test_layers_with_normed_heads(env):  # noqa: F811
    """spax_decode_layers with norms in some of its layers: its parts one by one, bit for bit."""
    torch, spax, dev = env
    s = Stack(env, 3, 512, 8, 2, 64, 1408, 0, 75, 77)
    g = _gen(torch, 1)
    norms = [spax.make_head_norm(1 + 0.2 * torch.randn(8, 64, generator=g, device=dev),
                                 1 + 0.2 * torch.randn(64, generator=g, device=dev), eps=1e-6), None,
             spax.make_head_norm(None, 1 + 0.2 * torch.randn(64, generator=g, device=dev),
                                 k_bias=torch.randn(64, generator=g, device=dev), kind="layer")]
    layers = [spax.make_layer(*[n["phases"][p] if p in n["phases"] else n["parts"][p] for p in (
        "qkv", "append", "attention", "o", "attn_norm", "gate_up", "glu", "down", "mlp_norm")],
        head_norm=m) for n, m in zip(s.info, norms)]
    arr = spax.layer_array(layers)
    flags = spax.STEP_DETERMINISTIC
    plain = spax.spax_kv_append
    by_append = {id(n["parts"]["append"]): m for n, m in zip(s.info, norms)}

    def append(a):
        m = by_append[id(a)]
        return plain(a) if m is None else spax.spax_kv_append_normed(a, m)
    spax.spax_kv_append = append
    try:
        s.step_by_parts(flags)
    finally:
        spax.spax_kv_append = plain
    torch.cuda.synchronize()
    want = s.state()
    s.h.fill_(float("nan"))
    spax.spax_residual_norm(s.first)
    spax.spax_decode_layers(arr, s.ws, flags=flags)
    torch.cuda.synchronize()
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(s.state(), want))
    # without the norms it is another result
    spax.spax_residual_norm(s.first)
    spax.spax_decode_layers(s.arr, s.ws, flags=flags)
    torch.cuda.synchronize()
    assert not torch.equal(s.h, want[0])
