"""The default form of spax_decode_layers, whose launches clear the next projection's sums while the
operators in between run: every buffer of the whole call against the float64 oracle on the inputs
that the call left, with everything the call writes filled with large values before it."""

import numpy as np
import pytest

from oracle import layer as olayer
from oracle import tiers as otiers
from tests import test_gpu_layers as layers
from tests.parity_util import check_y_oracle
from tests.test_gpu_layer_ops import _attention_tol, _check, _f64

pytestmark = pytest.mark.gpu
env = layers.env
EPS, HALF = layers.EPS, 2.0 ** -11


def _fill(s):
    """Every value that the step writes (the cache's rows of this token aside)."""
    s.h.fill_(3e4)
    for n in s.info:
        b = n["bufs"]
        for t in b["y"].values():
            t.fill_(3e4)
        for t in (b["q"], b["att"], b["x1"], b["act"], n["x2"]):
            t.fill_(3e4)
        for tier, full, approx, counts in b["m"].values():
            tier.fill_(9)
            for t in (full, approx, counts):
                t.fill_(1 << 20)


def _check_step(s, size, gone=()):
    """What the step left, part by part; the parts in gone have lost their inputs or outputs since."""
    d, hq, hk, dim, f, fmt, ctx = size
    h = _f64(s.token)
    eh = 0.0
    for i, n in enumerate(s.info):
        b = n["bufs"]
        w1, w2, p1, gate = (_f64(t) for t in n["w"])
        for name in ("qkv", "o", "gate_up", "down"):
            O, Ws, nf, na = n["blobs"][name]
            x16 = n["xs"][name].flatten().cpu().numpy()
            tiers, wf, wa, wc = otiers.build_tiers(x16, otiers.MODE_TOPK, n_full=nf, n_approx=na)
            got = [t.cpu().numpy() for t in b["m"][name]]
            what = f"layer {i} {name}"
            assert np.array_equal(got[0], tiers) and list(got[3]) == list(wc), what
            assert np.array_equal(got[1][:len(wf)], wf) and np.array_equal(got[2][:len(wa)], wa), what
            check_y_oracle(b["y"][name].cpu().numpy(), O, Ws, x16, wf, wa, what)
        q, k, v = np.split(_f64(b["y"]["qkv"]), [hq * dim, (hq + hk) * dim])
        p = ctx - 1
        page, row = int(n["ids"][0, p // s.page]), p % s.page

        def turned(x, heads):
            return np.stack([olayer.rotate(r, p, _f64(s.inv), False) for r in x.reshape(heads, dim)])

        if "q" not in gone:
            ref = turned(q, hq)
            _check(_f64(b["q"])[0], ref, HALF * np.abs(ref) + 2.0 ** -19 * np.abs(q).max() + 2.0 ** -25,
                   f"layer {i} q")
            ref, _, mass, reach = olayer.attention(_f64(b["q"]), _f64(n["kc"]), _f64(n["vc"]),
                                                   n["ids"].cpu().numpy(), [ctx], dim ** -0.5)
            _check(_f64(b["att"]), ref, _attention_tol(ref, mass, reach, dim, "fp16", 256),
                   f"layer {i} att")
        ref = turned(k, hk)
        _check(_f64(n["kc"])[page, :, row], ref,
               HALF * np.abs(ref) + 2.0 ** -19 * np.abs(k).max() + 2.0 ** -25, f"layer {i} k")
        ref = v.reshape(hk, dim)
        _check(_f64(n["vc"])[page, :, row], ref, HALF * np.abs(ref) + 2.0 ** -25, f"layer {i} v")
        y = _f64(b["y"]["gate_up"])
        ref = olayer.glu(y[:f], y[f:], "silu")
        _check(_f64(b["act"])[0], ref, (HALF + 2.0 ** -20) * np.abs(ref) + 2.0 ** -25, f"layer {i} act")
        # the stream is updated in place twice a layer: carried along from the token, with its error
        for name, w, post, g, scale, x in (("o", w1, p1, gate, 0.5, b["x1"]),
                                           ("down", w2, None, None, 1.0, n["x2"])):
            new, rx = olayer.residual_norm(h, _f64(b["y"][name])[None], "rms", w, None, post, None, g,
                                           scale, EPS)
            eh = eh + (2.0 ** -17 * np.abs(new - h) + 2.0 ** -22 * (np.abs(new) + np.abs(h))).max()
            ex = np.abs(w) * 2 * eh / np.sqrt((new ** 2).mean()) + 2.0 ** -17 * np.abs(rx)
            _check(_f64(x), rx, HALF * np.abs(rx) + ex + 2.0 ** -25, f"layer {i} x after {name}")
            h = new
    _check(_f64(s.h), h, eh, "h")


@pytest.mark.parametrize("separate", [False, True], ids=["default", "separate"])
@pytest.mark.parametrize("size", layers.SIZES, ids=str)
def test_every_buffer_of_the_whole_call(env, size, separate):
    torch, spax, dev = env
    s = layers.Stack(env, 2, *size, 90)
    for token in range(2):
        _fill(s)
        s.step(spax.STEP_SEPARATE if separate else spax.STEP_DEFAULT)
        torch.cuda.synchronize()
        _check_step(s, size[:6] + (size[6] + token,))
        s.advance()


def _share(torch, s, what):
    """o's y on memory that the operators after qkv use and o no longer needs."""
    for n in s.info:
        b = n["bufs"]
        room = torch.empty(b["y"]["o"].numel(), device="cuda")
        b["y"]["o"] = room
        n["phases"]["o"].y = n["parts"]["attn_norm"].block = room.data_ptr()
        if what == "q":
            b["q"] = room.view(torch.float16)[:b["q"].numel()].view(b["q"].shape)
            n["parts"]["append"].q_out = n["parts"]["attention"].q = room.data_ptr()
        else:
            n["parts"]["attention"].lse = room.data_ptr()
        n["room"] = room


@pytest.mark.parametrize("what", ["q", "lse"])
@pytest.mark.parametrize("size", layers.SIZES, ids=str)
def test_sums_on_memory_that_the_operators_before_them_use(env, size, what):
    """They may only be cleared once those are done."""
    torch, spax, dev = env
    s = layers.Stack(env, 2, *size, 91)
    _share(torch, s, what)
    for token in range(2):
        _fill(s)
        s.step()
        torch.cuda.synchronize()
        _check_step(s, size[:6] + (size[6] + token,), gone=("q",) if what == "q" else ())
        s.advance()
    # the attention through the shared memory, against the same stack with memory of its own
    t = layers.Stack(env, 2, *size, 91)
    t.position.copy_(s.position)
    t.lens.copy_(s.lens)
    t.token.copy_(s.token)
    for n, m in zip(s.info, t.info):
        m["kc"].copy_(n["kc"])
        m["vc"].copy_(n["vc"])
    for x in (s, t):
        x.step(spax.STEP_DETERMINISTIC)
    torch.cuda.synchronize()
    for n, m in zip(s.info, t.info):
        assert torch.equal(n["bufs"]["att"], m["bufs"]["att"])
    assert torch.equal(s.h, t.h)
