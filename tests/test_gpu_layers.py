"""Whole decoder layers: spax_decode_layers against its parts called one by one (bit for bit, in
the deterministic form) and each part against the float64 oracle on the inputs it was given."""

import numpy as np
import pytest

import synth
from oracle import layer as olayer
from oracle import pack as opack
from oracle import tiers as otiers
from tests.parity_util import check_y_oracle
from tests.test_gpu_layer_ops import _attention_tol, _check, _f64

pytestmark = pytest.mark.gpu
EPS = 1e-5


@pytest.fixture(scope="module")
def env():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import activation_sparse_tiered_amd as spax
    return torch, spax, torch.device("cuda:0")


class Stack:
    """Layers of width d, hq heads of dim over hk key heads, inner width f, one token at a time."""

    def __init__(self, env, n_layers, d, hq, hk, dim, f, fmt, ctx, seed, shared=False, page=16):
        torch, spax, dev = env
        self.torch, self.spax = torch, spax
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.hq, self.hk, self.dim, self.f, self.ctx, self.page = hq, hk, dim, f, ctx, page
        width = (ctx + 63) // page + 1
        self.position = torch.tensor([ctx - 1], dtype=torch.int32, device=dev)
        self.lens = torch.tensor([ctx], dtype=torch.int32, device=dev)
        self.inv = (1e4 ** (-torch.arange(0, dim, 2, device=dev).double() / dim)).float()
        self.h = torch.empty(1, d, device=dev)          # the residual stream, fp32
        self.x0 = torch.empty(1, d, dtype=torch.float16, device=dev)
        self.token = torch.randn(1, d, generator=g, device=dev)
        self.layers, self.info, bufs = [], [], None
        x_in = self.x0
        first_w = 1 + 0.1 * torch.randn(d, generator=g, device=dev)
        self.first = spax.make_residual_norm(self.token, None, self.h, self.x0, pre_weight=first_w,
                                             eps=EPS)
        for i in range(n_layers):
            shapes = [("qkv", d, [hq * dim, hk * dim, hk * dim]), ("o", hq * dim, [d]),
                      ("gate_up", d, [f, f]), ("down", f, [d])]
            if bufs is None or not shared:
                bufs = dict(
                    y={n: torch.empty(sum(o), device=dev) for n, _, o in shapes},
                    m={n: [torch.empty(a, dtype=torch.uint8, device=dev)]
                       + [torch.empty(a, dtype=torch.int32, device=dev) for _ in range(2)]
                       + [torch.empty(3, dtype=torch.int32, device=dev)] for n, a, _ in shapes},
                    q=torch.empty(1, hq, dim, dtype=torch.float16, device=dev),
                    att=torch.empty(1, hq, dim, dtype=torch.float16, device=dev),
                    x1=torch.empty(1, d, dtype=torch.float16, device=dev),
                    act=torch.empty(1, f, dtype=torch.float16, device=dev),
                    x2=torch.empty(1, d, dtype=torch.float16, device=dev))
            b = bufs
            x2 = b["x2"] if i + 1 < n_layers or not shared else torch.empty_like(b["x2"])
            xs = {"qkv": x_in, "o": b["att"], "gate_up": b["x1"], "down": b["act"]}
            phases, blobs = {}, {}
            for k, (name, a, outs) in enumerate(shapes):
                L = spax.spax_layout_init(a, outs, fmt, 128, 64 if fmt == 0 else 128)
                Ws = [synth.weights(seed + i, a, r, k, m) for m, r in enumerate(outs)]
                packed = torch.empty(int(L.total_bytes), dtype=torch.uint8, device=dev)
                spax.spax_pack_columns(L, [torch.from_numpy(w).to(dev) for w in Ws], packed)
                nf, na = otiers.counts_from_fractions(a, 0.4, 0.4)
                phases[name] = spax.make_phase(L, packed, xs[name], spax.topk_params(nf, na),
                                               *b["m"][name], b["y"][name])
                blobs[name] = (opack.Layout(a, outs, fmt, 128, 64 if fmt == 0 else 128), Ws, nf, na)
            ids = torch.randperm(width + 3, generator=g, device=dev)[:width].int()[None].contiguous()
            kc = torch.randn(width + 3, hk, page, dim, generator=g, device=dev).half()
            vc = torch.randn(width + 3, hk, page, dim, generator=g, device=dev).half()
            cache = spax.make_kv_cache(kc, vc, ids)
            y = b["y"]["qkv"][None]
            q, k, v = (t.unflatten(1, (-1, dim)) for t in y.split([hq * dim, hk * dim, hk * dim], 1))
            w1, w2, p1 = (1 + 0.1 * torch.randn(d, generator=g, device=dev) for _ in range(3))
            gate = 1 + 0.1 * torch.randn(d, generator=g, device=dev)
            gu = b["y"]["gate_up"][None]
            parts = dict(
                append=spax.make_kv_append(cache, q, k, v, self.position, b["q"],
                                           inv_freq=self.inv),
                attention=spax.make_attention(cache, b["q"], self.lens, b["att"]),
                attn_norm=spax.make_residual_norm(self.h, b["y"]["o"][None], self.h, b["x1"],
                                                  pre_weight=w1, post_weight=p1, gate=gate,
                                                  scale=0.5, eps=EPS),
                glu=spax.make_glu(gu[:, :f], gu[:, f:], b["act"]),
                mlp_norm=spax.make_residual_norm(self.h, b["y"]["down"][None], self.h, x2,
                                                 pre_weight=w2, eps=EPS))
            self.layers.append(spax.make_layer(
                phases["qkv"], parts["append"], parts["attention"], phases["o"],
                parts["attn_norm"], phases["gate_up"], parts["glu"], phases["down"],
                parts["mlp_norm"]))
            self.info.append(dict(phases=phases, parts=parts, blobs=blobs, bufs=b, xs=xs, kc=kc,
                                  vc=vc, ids=ids, x2=x2, w=(w1, w2, p1, gate)))
            x_in = x2
        self.arr = spax.layer_array(self.layers)
        self.ws = torch.zeros(spax.spax_layers_workspace_bytes(self.arr), dtype=torch.uint8,
                              device=dev)

    def step(self, flags=0):
        self.spax.spax_residual_norm(self.first)
        self.spax.spax_decode_layers(self.arr, self.ws, flags=flags)

    def step_by_parts(self, flags, see=None):
        """The same calls one by one; see(layer, part) after each."""
        spax = self.spax
        spax.spax_residual_norm(self.first)
        for i, n in enumerate(self.info):
            p = n["parts"]

            def phase(name):
                spax.spax_decode_step_projections([n["phases"][name]], self.ws, flags=flags)

            for name, call in (
                    ("qkv", phase), ("append", lambda _: spax.spax_kv_append(p["append"])),
                    ("attention", lambda _: spax.spax_paged_attention(p["attention"], self.ws)),
                    ("o", phase), ("attn_norm", lambda _: spax.spax_residual_norm(p["attn_norm"])),
                    ("gate_up", phase), ("glu", lambda _: spax.spax_glu(p["glu"])),
                    ("down", phase), ("mlp_norm", lambda _: spax.spax_residual_norm(p["mlp_norm"]))):
                before = self.h.clone()
                call(name)
                if see:
                    see(i, name, before)

    def state(self):
        out = [self.h.clone()]
        for n in self.info:
            b = n["bufs"]
            out += [t.clone() for t in (*b["y"].values(), b["q"], b["att"], b["x1"], b["act"],
                                        n["x2"], n["kc"], n["vc"])]
        return out

    def advance(self):
        self.position += 1
        self.lens += 1
        self.token.mul_(-0.7)


SIZES = [  # d, heads, key heads, dim, inner, fmt, context
    (512, 8, 2, 64, 1408, 0, 75), (256, 4, 4, 128, 256, 0, 1), (512, 4, 1, 128, 768, 1, 3000)]


@pytest.mark.parametrize("size", SIZES, ids=str)
def test_parts_against_the_oracle(env, size):
    """Each part of a two-layer step, on what the parts before it left."""
    torch, spax, dev = env
    d, hq, hk, dim, f, fmt, ctx = size
    s = Stack(env, 2, d, hq, hk, dim, f, fmt, ctx, 50)

    def see(i, name, h_before):
        torch.cuda.synchronize()
        n = s.info[i]
        b, half = n["bufs"], 2.0 ** -11
        w1, w2, p1, gate = (_f64(t) for t in n["w"])
        if name in n["phases"]:
            O, Ws, nf, na = n["blobs"][name]
            x16 = n["xs"][name].flatten().cpu().numpy()
            _, wf, wa, wc = otiers.build_tiers(x16, otiers.MODE_TOPK, n_full=nf, n_approx=na)
            assert list(b["m"][name][3].cpu().numpy()) == list(wc)
            check_y_oracle(b["y"][name].cpu().numpy(), O, Ws, x16, wf, wa, f"layer {i} {name}")
        elif name == "append":
            q, k, v = np.split(_f64(b["y"]["qkv"]), [hq * dim, (hq + hk) * dim])
            p = ctx - 1
            ref = np.stack([olayer.rotate(r, p, _f64(s.inv), False) for r in q.reshape(hq, dim)])
            _check(_f64(b["q"])[0], ref, half * np.abs(ref) + 2.0 ** -19 * np.abs(q).max() + 2.0 ** -25,
                   "q")
            page = int(n["ids"][0, p // s.page])
            ref = np.stack([olayer.rotate(r, p, _f64(s.inv), False) for r in k.reshape(hk, dim)])
            _check(_f64(n["kc"])[page, :, p % s.page], ref,
                   half * np.abs(ref) + 2.0 ** -19 * np.abs(k).max() + 2.0 ** -25, "k")
            ref = v.reshape(hk, dim)
            _check(_f64(n["vc"])[page, :, p % s.page], ref, half * np.abs(ref) + 2.0 ** -25, "v")
        elif name == "attention":
            ref, _, mass, reach = olayer.attention(_f64(b["q"]), _f64(n["kc"]), _f64(n["vc"]),
                                                   n["ids"].cpu().numpy(), [ctx], dim ** -0.5)
            _check(_f64(b["att"]), ref, _attention_tol(ref, mass, reach, dim, "fp16", 4000), "att")
        elif name == "glu":
            y = _f64(b["y"]["gate_up"])
            ref = olayer.glu(y[:f], y[f:], "silu")
            _check(_f64(b["act"])[0], ref, (half + 2.0 ** -20) * np.abs(ref) + 2.0 ** -25, "act")
        else:
            first = name == "attn_norm"
            y = _f64(b["y"]["o" if first else "down"])[None]
            rh, rx = olayer.residual_norm(_f64(h_before), y, "rms", w1 if first else w2, None,
                                          p1 if first else None, None, gate if first else None,
                                          0.5 if first else 1.0, EPS)
            eh = 2.0 ** -17 * np.abs(rh - _f64(h_before)) + 2.0 ** -22 * (np.abs(rh) + np.abs(_f64(h_before)))
            _check(_f64(s.h), rh, eh, "h")
            x = b["x1"] if first else n["x2"]
            ex = 2 * eh.max() / np.sqrt((rh ** 2).mean()) * 2 + 2.0 ** -17 * np.abs(rx)
            _check(_f64(x), rx, half * np.abs(rx) + ex + 2.0 ** -25, "x")

    s.step_by_parts(spax.STEP_DEFAULT, see)
    torch.cuda.synchronize()


@pytest.mark.parametrize("size", SIZES, ids=str)
@pytest.mark.parametrize("shared", [False, True], ids=["own", "shared"])
@pytest.mark.parametrize("form", [0, 1])
def test_layers_equal_their_parts(env, size, shared, form):
    """Three tokens through the whole call and through its parts: the same bits (deterministic
    sums), with buffers of their own and with every layer on the same ones."""
    torch, spax, dev = env
    d, hq, hk, dim, f, fmt, ctx = size
    flags = spax.STEP_DETERMINISTIC | (spax.STEP_SEPARATE if form else 0)
    a = Stack(env, 3, d, hq, hk, dim, f, fmt, ctx, 60, shared)
    b = Stack(env, 3, d, hq, hk, dim, f, fmt, ctx, 60, shared)
    for token in range(3):
        a.step(flags)
        b.step_by_parts(flags)
        torch.cuda.synchronize()
        for x, y in zip(a.state(), b.state()):
            assert torch.equal(x, y), token
        a.advance()
        b.advance()


def test_layers_in_a_graph(env):
    """The step captured once and replayed token by token, against the eager call."""
    torch, spax, dev = env
    d, hq, hk, dim, f, fmt, ctx = 512, 8, 2, 64, 1408, 0, 2000
    flags = spax.STEP_DETERMINISTIC
    a = Stack(env, 2, d, hq, hk, dim, f, fmt, ctx, 70, True)
    b = Stack(env, 2, d, hq, hk, dim, f, fmt, ctx, 70, True)
    a.step(flags)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a.step(flags)
    for token in range(4):
        graph.replay()
        torch.cuda.synchronize()
        b.step(flags)
        torch.cuda.synchronize()
        for x, y in zip(a.state(), b.state()):
            assert torch.equal(x, y), token
        a.advance()
        b.advance()


def test_layers_default_form(env):
    """The default form (atomic sums) agrees with the deterministic one to fp32 reordering where
    the masks agree, which the first layer's first phase guarantees for its own y."""
    torch, spax, dev = env
    d, hq, hk, dim, f, fmt, ctx = SIZES[0]
    a = Stack(env, 2, d, hq, hk, dim, f, fmt, ctx, 80, True)
    a.step(spax.STEP_DETERMINISTIC)
    torch.cuda.synchronize()
    want = [n["kc"].clone() for n in a.info]
    for flags in (0, spax.STEP_SEPARATE):
        a.step(flags)
        torch.cuda.synchronize()
        diff = (a.info[0]["kc"].float() - want[0].float()).abs().max().item()
        assert diff <= 2.0 ** -9 * want[0].abs().max().item()
        assert bool(torch.isfinite(a.h).all()) and bool(torch.isfinite(a.info[-1]["x2"]).all())
