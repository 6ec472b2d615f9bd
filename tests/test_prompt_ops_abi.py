"""Host-side checks of the operators of many tokens: struct sizes, what their calls refuse before
anything is enqueued, and what the tensor descriptions refuse (no GPU work)."""

import ctypes as C

import numpy as np
import pytest
import torch

import activation_sparse_tiered_amd as spax
from activation_sparse_tiered_amd import _lib
from oracle import prompt as oprompt
from tests.test_layer_ops_abi import (A, FAKE, MB, N, P, S, U, W, _append, _cache, _layer,
                                      needs_no_gpu)


def test_struct_sizes_match_c():
    want = {spax.HeadNorm: 56, spax.ChunkAttentionArgs: 104, spax.PackedGemmArgs: 96}
    for s, n in want.items():
        assert C.sizeof(s) == n, s


# ------------------------------------------------------------------ append with normed heads

def _head_norm(**kw):
    m = spax.HeadNorm()
    m.q_weight, m.k_weight, m.eps = FAKE + 210 * MB, FAKE + 211 * MB, 1e-6
    for name, v in kw.items():
        setattr(m, name, v)
    return m


HEAD_NORM_BAD = [
    (dict(q_weight=0, k_weight=0), N), (dict(kind=2), U), (dict(kind=-1), U),
    (dict(q_weight=FAKE + 210 * MB + 2), A), (dict(k_bias=FAKE + 212 * MB + 1), A),
    (dict(eps=-1.0), P), (dict(eps=float("nan")), P), (dict(eps=float("inf")), P),
    (dict(q_weight=0, q_bias=FAKE + 212 * MB), P), (dict(k_weight=0, k_bias=FAKE + 212 * MB), P),
    (dict(q_stride=127), P), (dict(k_stride=-128), P), (dict(k_stride=1 << 50), P),
    (dict(q_weight=FAKE + 203 * MB), P),                     # on q_out
    (dict(k_bias=FAKE + 64), P),                             # on the cache
    (dict(k_weight=FAKE + 64 * MB), P),
]


@needs_no_gpu
@pytest.mark.parametrize("kw,status", HEAD_NORM_BAD)
def test_head_norm_refusals(kw, status):
    call = _lib.lib.spax_kv_append_normed
    assert call(_append(), _head_norm(**kw), 0) == status, _lib.lib.spax_last_error()


@needs_no_gpu
def test_normed_append_refusals():
    call = _lib.lib.spax_kv_append_normed
    assert call(_append(), None, 0) == N and call(None, _head_norm(), 0) == N
    assert call(_append(rot_dim=63), _head_norm(), 0) == S       # the append's own
    assert call(_append(n_heads=0, q=0, q_out=0), _head_norm(), 0) == P   # q_weight without q
    assert call(_append(n_tokens=0), _head_norm(), 0) == _lib.SPAX_OK
    assert call(_append(n_tokens=0), _head_norm(kind=5), 0) == U


@needs_no_gpu
def test_layers_with_normed_heads_refusals():
    good, _ = _layer(0)
    arr = (spax.DecoderLayer * 1)(good)
    call = _lib.lib.spax_decode_layers_normed
    norms = (C.POINTER(spax.HeadNorm) * 1)(C.pointer(_head_norm(kind=3)))
    assert call(arr, None, 1, 0, 0, 0, 0) == N
    assert call(arr, norms, 1, 0, 0, 0, 0) == U
    assert _lib.lib.spax_last_error().startswith(b"layer 0, append")
    # a weight where the append writes
    norms = (C.POINTER(spax.HeadNorm) * 1)(C.pointer(_head_norm(k_weight=good.append.contents.q_out)))
    assert call(arr, norms, 1, 0, 0, 0, 0) == P
    # none for this layer: as without
    none = (C.POINTER(spax.HeadNorm) * 1)()
    assert call(arr, none, 1, 4, 0, 0, 0) == W
    assert _lib.lib.spax_decode_layers(arr, 1, 4, 0, 0, 0) == W


def _cpu_append(hq=4, hk=2, dim=64, n=3):
    kc = torch.zeros(4, hk, 16, dim, dtype=torch.float16)
    cache = spax.make_kv_cache(kc, kc.clone(), torch.zeros(n, 2, dtype=torch.int32))
    row = torch.zeros(n, (hq + 2 * hk) * dim)
    q, k, v = (t.unflatten(1, (-1, dim)) for t in row.split([hq * dim, hk * dim, hk * dim], 1))
    return spax.make_kv_append(cache, q, k, v, torch.zeros(n, dtype=torch.int32),
                               torch.zeros(n, hq, dim, dtype=torch.float16))


def test_head_norm_descriptions():
    f = torch.ones
    m = spax.make_head_norm(f(64), f(2, 64), q_bias=f(64), kind="layer", eps=1e-5)
    assert (m.q_stride, m.k_stride, m.kind) == (0, 64, spax.NORM_LAYER) and not m.k_bias
    assert spax.make_head_norm(f(1, 64), None).q_stride == 0
    for bad, error in (((f(64).half(), None), TypeError), ((None, None), ValueError),
                       ((f(2, 2, 64), None), ValueError), ((f(64, 64).t()[:4], None), ValueError)):
        with pytest.raises(error):
            spax.make_head_norm(*bad)
    with pytest.raises(ValueError):
        spax.make_head_norm(None, f(64), q_bias=f(64))
    with pytest.raises(ValueError):
        spax.make_head_norm(f(64), f(64), q_bias=f(2, 64))
    with pytest.raises(ValueError):     # a bias whose rows lie otherwise than the weight's
        spax.make_head_norm(f(4, 64), None, q_bias=f(4, 128)[:, :64])
    a = _cpu_append()
    for wrong in (spax.make_head_norm(f(128), None), spax.make_head_norm(f(3, 64), None),
                  spax.make_head_norm(None, f(4, 64))):
        with pytest.raises(ValueError, match="shape"):
            spax.spax_kv_append_normed(a, wrong)
    with pytest.raises(ValueError, match="not on a GPU"):
        spax.spax_kv_append_normed(a, spax.make_head_norm(f(4, 64), f(2, 64)))


# ------------------------------------------------------------------ attention of a chunk

def _chunk(cache=None, **kw):
    a = spax.ChunkAttentionArgs()
    a.cache = C.pointer(cache if cache is not None else _cache())
    a.q, a.out, a.lens = FAKE + 200 * MB, FAKE + 201 * MB, FAKE + 202 * MB
    a.starts = FAKE + 203 * MB
    a.q_token_stride = a.out_token_stride = 8 * 128
    a.q_head_stride = a.out_head_stride = 128
    a.type, a.n_heads, a.n_tokens, a.max_len, a.scale = spax.TYPE_F16, 8, 10, 64, 0.1
    for name, v in kw.items():
        setattr(a, name, v)
    return a


CHUNK_BAD = [
    (dict(q=0), N), (dict(out=0), N), (dict(lens=0), N), (dict(starts=0), N),
    (dict(type=spax.TYPE_F32), U), (dict(type=spax.TYPE_BF16), U), (dict(n_heads=7), S),
    (dict(n_heads=0), S), (dict(n_heads=1 << 17), S), (dict(n_tokens=-1), S),
    (dict(n_tokens=(1 << 27) + 1), S), (dict(max_len=0), S), (dict(max_len=65), S),
    (dict(window=-1), S), (dict(scale=float("nan")), P), (dict(scale=float("inf")), P),
    (dict(q=FAKE + 200 * MB + 8), A), (dict(out_head_stride=132), A), (dict(lens=FAKE + 1), A),
    (dict(starts=FAKE + 203 * MB + 2), A), (dict(lse=FAKE + 2), A),
    (dict(out=FAKE + 200 * MB), P), (dict(out=FAKE + 64), P), (dict(lse=FAKE + 201 * MB), P),
    (dict(out_head_stride=64), P), (dict(out_token_stride=512), P),
    (dict(lse=FAKE + 203 * MB), P), (dict(q_token_stride=-8), P),
]


@needs_no_gpu
@pytest.mark.parametrize("kw,status", CHUNK_BAD)
def test_chunk_refusals(kw, status):
    a = _chunk(**kw)
    assert _lib.lib.spax_chunk_attention(a, 0, 0, 0) == status, _lib.lib.spax_last_error()
    assert spax.spax_chunk_attention_workspace_bytes(a) == 0


@needs_no_gpu
def test_chunk_refuses_what_its_cache_does():
    call = _lib.lib.spax_chunk_attention
    assert call(None, 0, 0, 0) == N
    assert call(_chunk(_cache(head_dim=80)), 0, 0, 0) == S
    assert call(_chunk(_cache(k=0)), 0, 0, 0) == N
    assert call(_chunk(_cache(k_row_stride=132)), 0, 0, 0) == A


@needs_no_gpu
def test_chunk_of_nothing():
    call = _lib.lib.spax_chunk_attention
    assert call(_chunk(n_tokens=0), 0, 0, 0) == _lib.SPAX_OK
    assert call(_chunk(n_tokens=0, q=0, out=0, lens=0, starts=0), 0, 0, 0) == _lib.SPAX_OK
    assert spax.spax_chunk_attention_workspace_bytes(_chunk(n_tokens=0)) == 0


@needs_no_gpu
def test_chunk_workspace():
    long = _cache(max_pages=4096, table_stride=4096)
    a = _chunk(long, max_len=65536)
    need = spax.spax_chunk_attention_workspace_bytes(a)
    assert need >= 2 * 10 * 8 * (128 + 2) * 4 and need % 256 == 0
    call = _lib.lib.spax_chunk_attention
    assert call(a, 0, need, 0) == N
    assert call(a, FAKE + 300 * MB + 128, need, 0) == A
    assert call(a, FAKE + 300 * MB, need - 1, 0) == W
    assert call(a, FAKE + 200 * MB, need, 0) == P   # on q
    # short sequences, a short window and many tokens need none
    assert spax.spax_chunk_attention_workspace_bytes(_chunk(long, max_len=700)) == 0
    assert spax.spax_chunk_attention_workspace_bytes(_chunk(long, max_len=65536, window=10)) == 0
    big = dict(q_token_stride=1024, n_tokens=1 << 18, out=FAKE + 2000 * MB, lens=FAKE + 3000 * MB,
               starts=FAKE + 3001 * MB)
    assert spax.spax_chunk_attention_workspace_bytes(_chunk(long, max_len=65536, **big)) == 0
    # more sequences than tokens: no more tiles than tokens
    assert spax.spax_chunk_attention_workspace_bytes(
        _chunk(_cache(n_seqs=1 << 20, max_pages=4096, table_stride=4096), max_len=700)) == 0


def test_chunk_descriptions():
    kc = torch.zeros(4, 2, 16, 64, dtype=torch.float16)
    cache = spax.make_kv_cache(kc, kc.clone(), torch.zeros(3, 2, dtype=torch.int32))
    i32 = lambda n: torch.zeros(n, dtype=torch.int32)  # noqa: E731
    q, out = (torch.zeros(9, 4, 64, dtype=torch.float16) for _ in range(2))
    a = spax.make_chunk_attention(cache, q, i32(4), i32(3), out)
    assert (a.n_tokens, a.n_heads, a.max_len, a.window) == (9, 4, 32, 0) and not a.lse
    assert a.scale == 0.125
    bad = [(q, i32(3), i32(3), out, {}, ValueError), (q, i32(4), i32(4), out, {}, ValueError),
           (q, i32(4).long(), i32(3), out, {}, TypeError), (q, i32(4), i32(3), out[:8], {}, ValueError),
           (q, i32(4), i32(3), out.bfloat16(), {}, TypeError),
           (q[..., :32], i32(4), i32(3), out, {}, ValueError),
           (q, i32(4), i32(3), out, dict(lse=torch.zeros(9, 3)), ValueError),
           (q, i32(4), i32(3), out, dict(max_len=1 << 40), ValueError)]
    for x, s, n, o, kw, error in bad:
        with pytest.raises(error):
            spax.make_chunk_attention(cache, x, s, n, o, **kw)
    with pytest.raises(ValueError, match="not on a GPU"):
        spax.spax_chunk_attention(a)


# ------------------------------------------------------------------ product with a packed blob

def _gemm(d_in=512, d_out=(256, 256), fmt=0, **kw):
    L = spax.spax_layout_init(d_in, list(d_out), fmt, 128, 64)
    a = spax.PackedGemmArgs()
    a.layout = C.pointer(L)
    a._layout = L
    a.packed, a.x, a.y = FAKE, FAKE + 100 * MB, FAKE + 101 * MB
    a.x_stride, a.y_stride, a.residual_stride = d_in, sum(d_out), sum(d_out)
    a.n_rows, a.y_type, a.residual_type, a.scale = 5, spax.TYPE_F16, spax.TYPE_F32, 1.0
    for name, v in kw.items():
        setattr(a, name, v)
    return a


R = FAKE + 102 * MB
GEMM_BAD = [
    (dict(packed=0), N), (dict(x=0), N), (dict(y=0), N), (dict(form=3), U), (dict(form=-1), U),
    (dict(form=1, act=2), U), (dict(y_type=spax.TYPE_E4M3), U),
    (dict(residual=R, residual_type=spax.TYPE_E4M3), U), (dict(n_rows=-1), S),
    (dict(n_rows=1 << 20), S), (dict(scale=float("nan")), P), (dict(scale=float("-inf")), P),
    (dict(packed=FAKE + 128), A), (dict(x=FAKE + 100 * MB + 8), A), (dict(x_stride=513), A),
    (dict(x_stride=516), A), (dict(y=FAKE + 101 * MB + 1), A), (dict(bias=FAKE + 103 * MB + 2), A),
    (dict(residual=R + 2), A), (dict(x_stride=504), P), (dict(y_stride=511), P),
    (dict(residual=R, residual_stride=511), P), (dict(y_stride=1 << 50), P),
    (dict(y=FAKE + 64), P), (dict(y=FAKE + 100 * MB), P), (dict(bias=FAKE + 101 * MB), P),
    (dict(residual=FAKE + 101 * MB), P),                                     # y's bytes, other type
    (dict(residual=FAKE + 101 * MB, residual_type=spax.TYPE_F16, residual_stride=1024), P),
    (dict(residual=FAKE + 101 * MB + 4, residual_type=spax.TYPE_F16), P),
]


@needs_no_gpu
@pytest.mark.parametrize("kw,status", GEMM_BAD)
def test_gemm_refusals(kw, status):
    a = _gemm(**kw)
    assert _lib.lib.spax_packed_gemm(a, 0, 0, 0) == status, _lib.lib.spax_last_error()
    assert spax.spax_packed_gemm_workspace_bytes(a) == 0


@needs_no_gpu
def test_gemm_refuses_layouts():
    call = _lib.lib.spax_packed_gemm
    assert call(None, 0, 0, 0) == N
    a = _gemm()
    a.layout = C.POINTER(spax.Layout)()
    assert call(a, 0, 0, 0) == N
    a = _gemm()
    a.layout = C.pointer(spax.Layout())
    assert call(a, 0, 0, 0) == S
    for outs in ((256,), (256, 128), (128, 128, 128)):
        assert call(_gemm(d_out=outs, form=2), 0, 0, 0) == S
    assert call(_gemm(n_rows=0, packed=0, x=0, y=0), 0, 0, 0) == _lib.SPAX_OK
    # one row: its strides are not read
    assert call(_gemm(n_rows=1, x_stride=3, y_stride=0, y=FAKE + 64), 0, 0, 0) == P


@needs_no_gpu
def test_gemm_workspace():
    a = _gemm(d_in=4096, d_out=(4096,))
    need = spax.spax_packed_gemm_workspace_bytes(a)
    assert need >= 2 * 5 * 4096 * 4 and need % 256 == 0
    call = _lib.lib.spax_packed_gemm
    assert call(a, 0, need, 0) == N
    assert call(a, FAKE + 300 * MB + 128, need, 0) == A
    assert call(a, FAKE + 300 * MB, need - 1, 0) == W
    assert call(a, FAKE, need, 0) == P   # on the blob
    # a short product, and one of many rows, are not split
    assert spax.spax_packed_gemm_workspace_bytes(_gemm(d_in=64)) == 0
    many = _gemm(d_in=4096, d_out=(4096,), n_rows=8192, x=FAKE + 200 * MB, y=FAKE + 400 * MB)
    assert spax.spax_packed_gemm_workspace_bytes(many) == 0


def test_gemm_descriptions():
    L = spax.spax_layout_init(100, [64, 64], spax.FMT_FP16, 128, 64)
    packed = torch.zeros(int(L.total_bytes), dtype=torch.uint8)
    x = torch.zeros(3, 104, dtype=torch.float16)[:, :100]
    y = torch.zeros(3, 128)
    a = spax.make_packed_gemm(L, packed, x, y, bias=torch.zeros(128), residual=y)
    assert (a.n_rows, a.form, a.y_type, a.x_stride) == (3, spax.GEMM_PLAIN, spax.TYPE_F32, 104)
    assert spax.make_packed_gemm(L, packed, x, y, act="gelu").form == spax.GEMM_ACT
    assert spax.make_packed_gemm(L, packed, x, y[:, :64], act="silu", gated=True).form == spax.GEMM_GATED
    bad = [(dict(x=x.float()), TypeError), (dict(x=x[:, :99]), ValueError), (dict(y=y[:2]), ValueError),
           (dict(y=y[:, :64]), ValueError), (dict(act="silu", gated=True), ValueError),
           (dict(y=y[:, :64], gated=True), ValueError), (dict(bias=torch.zeros(64)), ValueError),
           (dict(bias=torch.zeros(128).half()), TypeError), (dict(residual=y[:, :64]), ValueError),
           (dict(packed=packed[:-1]), ValueError), (dict(y=y.to(torch.float8_e4m3fn)), None)]
    for kw, error in bad:
        args = dict(packed=packed, x=x, y=y, **{})
        args.update(kw)
        if error is None:
            spax.make_packed_gemm(L, **args)     # the call refuses it
            continue
        with pytest.raises(error):
            spax.make_packed_gemm(L, **args)
    with pytest.raises(ValueError, match="not on a GPU"):
        spax.spax_packed_gemm(a)


# ------------------------------------------------------------------ the oracle's own pins

def test_oracle_chunk_by_hand():
    """Two tokens after one cached key: the first sees two keys, the second three."""
    k = np.zeros((1, 1, 4, 2))
    v = np.zeros((1, 1, 4, 2))
    k[0, 0, :3, 0] = [0.0, np.log(3.0), np.log(4.0)]
    v[0, 0, :3, 0] = [8.0, 0.0, 16.0]
    q = np.zeros((2, 1, 2))
    q[:, 0, 0] = 1.0
    rows, out, lse, _, _ = oprompt.chunk_attention(q, k, v, np.zeros((1, 1), int), [0, 2], [3], 1.0)
    assert list(rows) == [0, 1]
    assert np.allclose(out[:, 0, 0], [8 / 4, (8 + 64) / 8]) and np.allclose(lse[:, 0], np.log([4, 8]))
    _, out, _, _, _ = oprompt.chunk_attention(q, k, v, np.zeros((1, 1), int), [0, 2], [3], 1.0, window=1)
    assert np.allclose(out[:, 0, 0], [0, 16])


def test_oracle_gemm_by_hand():
    x, w = np.array([[1.0, 2.0]]), np.array([[1.0, -1.0], [0.5, 3.0]])
    y, t, mass = oprompt.packed_gemm(x, w, np.array([1.0, 0.0]), "gated", "silu", np.array([[7.0]]), 2.0)
    assert np.allclose(t, [[3.0, 5.0]]) and np.allclose(mass, [[2.0, 7.0]])
    assert np.allclose(y, 7 + 2 * 3 / (1 + np.exp(-3.0)) * 5)
