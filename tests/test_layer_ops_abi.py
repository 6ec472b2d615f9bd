"""Host-side checks of the operators between the projections: struct sizes, what their calls
refuse before anything is enqueued, and what the tensor descriptions refuse (no GPU work)."""

import ctypes as C

import numpy as np
import pytest
import torch

import activation_sparse_tiered_amd as spax
from activation_sparse_tiered_amd import _lib
from oracle import layer as olayer

MB = 1 << 20
FAKE = 0x10000000
needs_no_gpu = pytest.mark.skipif(torch.cuda.device_count() != 0, reason="host-only validation")


def test_struct_sizes_match_c():
    want = {spax.KvCache: 128, spax.KvAppendArgs: 152, spax.AttentionArgs: 96,
            spax.ResidualNormArgs: 152, spax.GluArgs: 72, spax.DecoderLayer: 72}
    for s, n in want.items():
        assert C.sizeof(s) == n, s


def _cache(**kw):
    c = spax.KvCache()
    c.k, c.v, c.page_table = FAKE, FAKE + 64 * MB, FAKE + 128 * MB
    c.type, c.n_pages, c.page_size, c.n_kv_heads, c.head_dim = spax.TYPE_F16, 8, 16, 2, 128
    c.k_row_stride = c.v_row_stride = 128
    c.k_head_stride = c.v_head_stride = 16 * 128
    c.k_page_stride = c.v_page_stride = 2 * 16 * 128
    c.n_seqs, c.max_pages, c.table_stride = 3, 4, 4
    for name, v in kw.items():
        setattr(c, name, v)
    return c


def _append(cache=None, **kw):
    a = spax.KvAppendArgs()
    a.cache = C.pointer(cache if cache is not None else _cache())
    a.q, a.k, a.v = FAKE + 200 * MB, FAKE + 201 * MB, FAKE + 202 * MB
    a.q_out, a.positions, a.inv_freq = FAKE + 203 * MB, FAKE + 204 * MB, FAKE + 205 * MB
    a.q_token_stride = a.out_token_stride = 8 * 128
    a.k_token_stride = a.v_token_stride = 2 * 128
    a.q_head_stride = a.k_head_stride = a.v_head_stride = a.out_head_stride = 128
    a.src_type, a.out_type, a.n_tokens, a.n_heads, a.rot_dim = spax.TYPE_F16, spax.TYPE_F16, 3, 8, 128
    for name, v in kw.items():
        setattr(a, name, v)
    return a


def _attention(cache=None, **kw):
    a = spax.AttentionArgs()
    a.cache = C.pointer(cache if cache is not None else _cache())
    a.q, a.out, a.lens = FAKE + 200 * MB, FAKE + 201 * MB, FAKE + 202 * MB
    a.q_seq_stride = a.out_seq_stride = 8 * 128
    a.q_head_stride = a.out_head_stride = 128
    a.type, a.n_heads, a.max_len, a.scale = spax.TYPE_F16, 8, 64, 0.1
    for name, v in kw.items():
        setattr(a, name, v)
    return a


def _norm(**kw):
    a = spax.ResidualNormArgs()
    a.residual, a.block, a.residual_out, a.x = (FAKE + i * MB for i in range(4))
    a.residual_stride = a.block_stride = a.residual_out_stride = a.x_stride = 100
    a.x_type, a.n_rows, a.d, a.scale, a.eps = spax.TYPE_F16, 3, 100, 1.0, 1e-5
    for name, v in kw.items():
        setattr(a, name, v)
    return a


def _glu(**kw):
    a = spax.GluArgs()
    a.gate, a.up, a.x = (FAKE + i * MB for i in range(3))
    a.gate_stride = a.up_stride = a.x_stride = 100
    a.x_type, a.n_rows, a.d = spax.TYPE_F16, 3, 100
    for name, v in kw.items():
        setattr(a, name, v)
    return a


N, S, P, A = _lib.SPAX_ERR_NULL, _lib.SPAX_ERR_SHAPE, _lib.SPAX_ERR_PARAM, _lib.SPAX_ERR_ALIGN
U, W = _lib.SPAX_ERR_UNSUPPORTED, _lib.SPAX_ERR_WORKSPACE

CACHE_BAD = [
    (dict(k=0), N), (dict(v=0), N), (dict(page_table=0), N),
    (dict(type=spax.TYPE_F32), U), (dict(type=7), U), (dict(k_scale=FAKE), U),
    (dict(head_dim=80), S), (dict(head_dim=0), S), (dict(page_size=24), S), (dict(page_size=2), S),
    (dict(page_size=1 << 17), S), (dict(n_pages=0), S), (dict(n_kv_heads=0), S),
    (dict(n_seqs=0), S), (dict(max_pages=0), S), (dict(max_pages=1 << 28, table_stride=1 << 28), S),
    (dict(table_stride=3), S), (dict(k_row_stride=64), P), (dict(v_head_stride=128), P),
    (dict(k_page_stride=-4096), P), (dict(k_row_stride=132), A), (dict(k=FAKE + 8), A),
    (dict(page_table=FAKE + 128 * MB + 2), A), (dict(k_page_stride=1 << 50), P),
]


@needs_no_gpu
@pytest.mark.parametrize("kw,status", CACHE_BAD)
def test_cache_refusals(kw, status):
    for make, call in ((_append, lambda a: _lib.lib.spax_kv_append(a, 0)),
                       (_attention, lambda a: _lib.lib.spax_paged_attention(a, 0, 0, 0))):
        assert call(make(_cache(**kw))) == status, _lib.lib.spax_last_error()


APPEND_BAD = [
    (dict(k=0), N), (dict(v=0), N), (dict(positions=0), N), (dict(q=0), N), (dict(q_out=0), N),
    (dict(n_heads=0), N), (dict(inv_freq=0), N), (dict(src_type=spax.TYPE_E4M3), U),
    (dict(out_type=spax.TYPE_F32), U), (dict(out_type=spax.TYPE_BF16), U), (dict(n_tokens=-1), S),
    (dict(n_tokens=1 << 24, seq=FAKE + 206 * MB), S), (dict(n_heads=1 << 16), S),
    (dict(n_tokens=4), S), (dict(rot_dim=130), S), (dict(rot_dim=63), S), (dict(rot_dim=-2), S),
    (dict(q=FAKE + 200 * MB + 1), A), (dict(positions=FAKE + 2), A),
    (dict(out_token_stride=512), P), (dict(q_token_stride=-8), P), (dict(k_head_stride=-1), P),
    (dict(q_out=FAKE + 202 * MB), P),                       # on v
    (dict(q_out=FAKE), P),                                  # on the cache
    (dict(q_out=FAKE + 200 * MB + 2), P),                   # half on q
    (dict(q_out=FAKE + 200 * MB, src_type=spax.TYPE_F32), P),   # q in place, other type
    (dict(q_out=FAKE + 200 * MB, q_token_stride=2048), P),      # q in place, other stride
    (dict(k=FAKE + 64 * MB), P),                            # k read from the cache
]


@needs_no_gpu
@pytest.mark.parametrize("kw,status", APPEND_BAD)
def test_append_refusals(kw, status):
    assert _lib.lib.spax_kv_append(_append(**kw), 0) == status, _lib.lib.spax_last_error()


@needs_no_gpu
def test_append_of_nothing():
    assert _lib.lib.spax_kv_append(_append(n_tokens=0), 0) == _lib.SPAX_OK
    assert _lib.lib.spax_kv_append(_append(n_tokens=0, q=0, k=0, v=0, q_out=0, positions=0),
                                   0) == _lib.SPAX_OK
    assert _lib.lib.spax_kv_append(None, 0) == N
    # k and v in one allocation may be interleaved, not the same
    assert _lib.lib.spax_kv_append(_append(_cache(v=FAKE)), 0) == P


ATTENTION_BAD = [
    (dict(q=0), N), (dict(out=0), N), (dict(lens=0), N), (dict(type=spax.TYPE_F32), U),
    (dict(type=spax.TYPE_BF16), U), (dict(n_heads=7), S), (dict(n_heads=0), S),
    (dict(max_len=0), S), (dict(max_len=65), S), (dict(window=-1), S),
    (dict(scale=float("nan")), P), (dict(scale=float("inf")), P), (dict(q=FAKE + 200 * MB + 8), A),
    (dict(out_head_stride=132), A), (dict(lens=FAKE + 1), A), (dict(lse=FAKE + 2), A),
    (dict(out=FAKE + 200 * MB), P), (dict(out=FAKE + 64), P), (dict(lse=FAKE + 201 * MB), P),
    (dict(out_head_stride=64), P),
]


@needs_no_gpu
@pytest.mark.parametrize("kw,status", ATTENTION_BAD)
def test_attention_refusals(kw, status):
    a = _attention(**kw)
    assert _lib.lib.spax_paged_attention(a, 0, 0, 0) == status, _lib.lib.spax_last_error()
    assert spax.spax_attention_workspace_bytes(a) == 0


@needs_no_gpu
def test_attention_of_too_much():
    huge = dict(n_pages=1, page_size=65536, max_pages=16385, table_stride=16385, k_page_stride=1 << 30,
                k_head_stride=1 << 25, v_page_stride=1 << 30, v_head_stride=1 << 25)
    call = _lib.lib.spax_paged_attention
    assert call(_attention(_cache(**huge), max_len=(1 << 30) + 1), 0, 0, 0) == S
    assert call(_attention(_cache(n_seqs=1 << 20, **huge), max_len=1 << 30), 0, 0, 0) == S
    # one that long sequence is fine, and asks for its workspace
    assert call(_attention(_cache(n_seqs=1, **huge), max_len=1 << 30), 0, 0, 0) == N


@needs_no_gpu
def test_attention_workspace():
    c = _cache(max_pages=4096, table_stride=4096)
    a = _attention(c, max_len=65536)
    need = spax.spax_attention_workspace_bytes(a)
    assert need >= 3 * 8 * (128 + 2) * 4 and need % 256 == 0
    call = _lib.lib.spax_paged_attention
    assert call(a, 0, need, 0) == N
    assert call(a, FAKE + 300 * MB + 128, need, 0) == A
    assert call(a, FAKE + 300 * MB, need - 1, 0) == W
    assert call(a, FAKE + 200 * MB, need, 0) == P   # on q
    # a window bounds what is shared out, whatever the length
    assert spax.spax_attention_workspace_bytes(_attention(c, max_len=65536, window=10)) == 0
    # the sizes never change with anything but the description
    assert spax.spax_attention_workspace_bytes(a) == need


NORM_BAD = [
    (dict(residual=0, block=0), N), (dict(residual_out=0, x=0), N),
    (dict(residual_type=spax.TYPE_E4M3), U), (dict(x_type=9), U), (dict(block_type=3), U),
    (dict(kind=2), U), (dict(n_rows=1 << 30), S), (dict(n_rows=-1), S), (dict(d=0), S), (dict(d=32769), S),
    (dict(scale=float("nan")), P), (dict(eps=-1.0), P), (dict(eps=float("inf")), P),
    (dict(pre_bias=FAKE + 9 * MB), P), (dict(post_bias=FAKE + 9 * MB), P),
    (dict(block=0, gate=FAKE + 9 * MB), P), (dict(block_stride=99), P),
    (dict(gate=FAKE + 9 * MB, gate_stride=50), P), (dict(x=FAKE + 3 * MB + 1), A),
    (dict(block=FAKE + MB + 2), A), (dict(x=FAKE), P), (dict(x=FAKE + 2 * MB), P),
    (dict(residual_out=FAKE + 400), P), (dict(residual_out=FAKE, residual_out_stride=200), P),
    (dict(x=FAKE + MB), P),                                  # on block, other type
    (dict(residual_out=FAKE + MB), P),
]


@needs_no_gpu
@pytest.mark.parametrize("kw,status", NORM_BAD)
def test_norm_refusals(kw, status):
    assert _lib.lib.spax_residual_norm(_norm(**kw), 0) == status, _lib.lib.spax_last_error()


GLU_BAD = [
    (dict(gate=0), N), (dict(up=0), N), (dict(x=0), N), (dict(src_type=spax.TYPE_E4M3), U),
    (dict(x_type=3), U), (dict(act=2), U), (dict(n_rows=-1), S), (dict(d=0), S),
    (dict(d=2048 << 15, n_rows=1 << 17, gate_stride=1 << 26), S), (dict(up_stride=99), P),
    (dict(gate=FAKE + 2), A), (dict(x=FAKE + 2 * MB + 1), A), (dict(x=FAKE), P),
    (dict(x=FAKE + 40, x_type=0), P), (dict(x=FAKE, x_type=0, x_stride=200), P),
]


@needs_no_gpu
@pytest.mark.parametrize("kw,status", GLU_BAD)
def test_glu_refusals(kw, status):
    assert _lib.lib.spax_glu(_glu(**kw), 0) == status, _lib.lib.spax_last_error()


@needs_no_gpu
def test_an_output_in_place_of_one_input_is_refused_where_another_shares_its_address():
    """Only the input that the output stands in for, value by value, may share its bytes: another
    with the same first address and other strides or types is read by other threads meanwhile."""
    q, x, r, h = FAKE + 200 * MB, FAKE + 3 * MB, FAKE + MB, FAKE
    bad = [
        # q rotated in place, and the keys read from the same rows
        _lib.lib.spax_kv_append(_append(q_out=q, k=q), 0),
        _lib.lib.spax_kv_append(_append(q_out=q, v=q), 0),
        # x over block, whose first row gates every row
        _lib.lib.spax_residual_norm(_norm(block=x, x=x, block_type=spax.TYPE_F16,
                                          x_type=spax.TYPE_F16, gate=x, gate_stride=0,
                                          gate_type=spax.TYPE_F16), 0),
        # the stream over itself, whose first row gates every row, or whose rows are the block's
        _lib.lib.spax_residual_norm(_norm(residual=h, residual_out=h, gate=h, gate_stride=0,
                                          gate_type=spax.TYPE_F32), 0),
        _lib.lib.spax_residual_norm(_norm(residual=h, residual_out=h, block=h, block_stride=200,
                                          block_type=spax.TYPE_F32), 0),
        # x over gate, and up the same address with rows twice as far apart
        _lib.lib.spax_glu(_glu(gate=r, up=r, x=r, x_type=0, gate_stride=100, x_stride=100,
                               up_stride=200), 0),
    ]
    assert bad == [P] * len(bad)


@needs_no_gpu
def test_norm_and_glu_of_nothing():
    assert _lib.lib.spax_residual_norm(_norm(n_rows=0), 0) == _lib.SPAX_OK
    assert _lib.lib.spax_glu(_glu(n_rows=0), 0) == _lib.SPAX_OK
    assert _lib.lib.spax_residual_norm(None, 0) == N
    assert _lib.lib.spax_glu(None, 0) == N
    assert _lib.lib.spax_paged_attention(None, 0, 0, 0) == N


# ------------------------------------------------------------------ whole layers

def _phase(d_in, d_out, at, x, y):
    L = spax.spax_layout_init(d_in, d_out, 0, 128, 64)
    return spax.make_phase(L, at, x, spax.topk_params(8, 8), at + 8 * MB, at + 9 * MB, at + 10 * MB,
                           at + 11 * MB, y)


def _layer(i=0, x=FAKE, skip=(), **kw):
    """A wired layer of fake buffers: width 512, 4 heads of 64 over 2 key heads, inner width 256.
    kw: {part: {field: value}}."""
    B = FAKE + (i + 1) * 512 * MB

    def buf(n):
        return B + 16 * MB * n
    y = [buf(n) for n in range(4)]
    c = _cache(k=buf(4), v=buf(5), page_table=buf(6), head_dim=64, n_seqs=1)
    p = dict(
        qkv=_phase(512, [256, 128, 128], buf(10), x, y[0]),
        append=_append(c, q=y[0], k=y[0] + 1024, v=y[0] + 1536, q_out=buf(14), positions=buf(15),
                       inv_freq=buf(16), src_type=0, n_tokens=1, n_heads=4, rot_dim=64,
                       q_head_stride=64, k_head_stride=64, v_head_stride=64, out_head_stride=64,
                       q_token_stride=512, k_token_stride=512, v_token_stride=512,
                       out_token_stride=256),
        attention=_attention(c, q=buf(14), out=buf(17), lens=buf(18), n_heads=4,
                             q_head_stride=64, out_head_stride=64, q_seq_stride=256,
                             out_seq_stride=256),
        o=_phase(256, [512], buf(11), buf(17), y[1]),
        attn_norm=_norm(residual=buf(19), block=y[1], residual_out=buf(19), x=buf(20), n_rows=1,
                        d=512),
        gate_up=_phase(512, [256, 256], buf(12), buf(20), y[2]),
        glu=_glu(gate=y[2], up=y[2] + 1024, x=buf(21), n_rows=1, d=256),
        down=_phase(256, [512], buf(13), buf(21), y[3]),
        mlp_norm=_norm(residual=buf(19), block=y[3], residual_out=buf(19), x=buf(22), n_rows=1,
                       d=512))
    for part, fields in kw.items():
        for name, v in fields.items():
            setattr(p[part], name, v)
    L = spax.DecoderLayer()
    for name, part in p.items():
        if name not in skip:
            setattr(L, name, C.pointer(part))
    L._keep = (p, c)
    return L, buf


def _run_layers(layers, ws=0, ws_bytes=0, flags=0):
    arr = (spax.DecoderLayer * len(layers))(*layers)
    return _lib.lib.spax_decode_layers(arr, len(layers), flags, ws, ws_bytes, 0)


LAYER_BAD = [
    (dict(append=dict(n_tokens=0)), S), (dict(attn_norm=dict(n_rows=0)), S),
    (dict(mlp_norm=dict(n_rows=0)), S), (dict(append=dict(q=FAKE)), P),
    (dict(append=dict(v=FAKE)), P), (dict(append=dict(q=0, q_out=0, n_heads=0)), P),
    (dict(append=dict(src_type=spax.TYPE_F16)), P), (dict(attention=dict(q=FAKE)), P),
    (dict(attention=dict(out=FAKE)), P), (dict(attention=dict(n_heads=2)), P),
    (dict(attn_norm=dict(block=FAKE)), P), (dict(attn_norm=dict(d=256)), P),
    (dict(attn_norm=dict(x=0)), P), (dict(attn_norm=dict(x_type=spax.TYPE_BF16)), P),
    (dict(glu=dict(gate=FAKE)), P), (dict(glu=dict(x=FAKE)), P), (dict(glu=dict(d=128)), P),
    (dict(mlp_norm=dict(block=FAKE)), P), (dict(o=dict(x=FAKE)), P),
    (dict(down=dict(x=FAKE)), P), (dict(gate_up=dict(x=FAKE)), P),
    (dict(attn_norm=dict(eps=-1.0)), P), (dict(glu=dict(act=5)), U),
    (dict(qkv=dict(packed=0)), N),
    (dict(down=dict(counts=0)), N),
]


@needs_no_gpu
@pytest.mark.parametrize("kw,status", LAYER_BAD)
def test_layer_refusals(kw, status):
    good, _ = _layer(0)
    bad, _ = _layer(1, x=_layer(0)[1](22), **kw)
    assert _run_layers([good, bad]) == status, _lib.lib.spax_last_error()
    assert _lib.lib.spax_last_error().startswith(b"layer 1")
    assert _run_layers([bad]) == status


@needs_no_gpu
def test_layer_refusals_of_the_whole():
    good, buf = _layer(0)
    for part in ("qkv", "append", "attention", "o", "attn_norm", "gate_up", "glu", "down",
                 "mlp_norm"):
        assert _run_layers([_layer(0, skip=(part,))[0]]) == N
    assert _lib.lib.spax_decode_layers(None, 1, 0, 0, 0, 0) == N
    assert _lib.lib.spax_decode_layers(good, 0, 0, 0, 0, 0) == S
    assert _run_layers([good], flags=2) == U and _run_layers([good], flags=8) == U
    # the next layer reads something else than what this one leaves
    assert _run_layers([good, _layer(1, x=FAKE)[0]]) == P
    # the deterministic form needs its workspace, apart from the layers' buffers
    need = spax.spax_layers_workspace_bytes((spax.DecoderLayer * 1)(good))
    assert need > 0
    assert _run_layers([good], flags=4) == W
    assert _run_layers([good], buf(30), need - 1 - need // 2, flags=4) == W
    assert _run_layers([good], buf(21), need, flags=4) == P
    assert spax.spax_layers_workspace_bytes((spax.DecoderLayer * 1)(_layer(0, skip=("o",))[0])) == 0


@needs_no_gpu
@pytest.mark.parametrize("kw", [
    dict(page_size=8), dict(n_pages=4), dict(type=spax.TYPE_E4M3), dict(v_page_stride=8192),
    dict(k_row_stride=64, k_head_stride=1024, k_page_stride=8192)])
def test_layer_refuses_an_attention_that_reads_the_cache_otherwise_than_it_is_written(kw):
    layer, _ = _layer(0)
    other = spax.KvCache.from_buffer_copy(layer._keep[1])
    for name, v in kw.items():
        setattr(other, name, v)
    layer._keep[0]["attention"].cache = C.pointer(other)
    # the attention of that description is a call of its own right
    if kw.get("type") != spax.TYPE_E4M3:
        layer._keep[0]["attention"].max_len = 8
    assert _run_layers([layer]) == P, _lib.lib.spax_last_error()
    assert b"attention is not wired" in _lib.lib.spax_last_error()


# ------------------------------------------------------------------ tensor descriptions

def _tensors(dtype=torch.float16):
    k = torch.zeros(8, 2, 16, 64, dtype=dtype)
    return k, k.clone(), torch.zeros(3, 4, dtype=torch.int32)


def test_descriptions_take_their_strides_from_the_tensors():
    k, v, table = _tensors()
    rows = k.transpose(1, 2).contiguous().transpose(1, 2)
    c = spax.make_kv_cache(rows, v, table)
    assert (c.k_page_stride, c.k_head_stride, c.k_row_stride) == (2 * 16 * 64, 64, 2 * 64)
    assert (c.v_page_stride, c.v_head_stride, c.v_row_stride) == (2 * 16 * 64, 16 * 64, 64)
    y = torch.zeros(3, (6 + 2 + 2) * 64)
    a = spax.make_kv_append(c, y[:, :384].view(3, 6, 64), y[:, 384:512].view(3, 2, 64),
                            y[:, 512:].view(3, 2, 64), torch.zeros(3, dtype=torch.int32),
                            torch.zeros(3, 6, 64, dtype=torch.float16),
                            inv_freq=torch.ones(16))
    assert a.q_token_stride == a.v_token_stride == 640 and a.k - a.q == 4 * 384
    assert a.rot_dim == 32 and a.n_heads == 6 and a.n_tokens == 3


def test_descriptions_refuse():
    k, v, table = _tensors()
    with pytest.raises(ValueError):
        spax.make_kv_cache(k, v[:4], table)
    with pytest.raises(TypeError):
        spax.make_kv_cache(k, v.bfloat16(), table)
    with pytest.raises(TypeError):
        spax.make_kv_cache(k, v, table.long())
    with pytest.raises(ValueError):
        spax.make_kv_cache(k.transpose(2, 3), v.transpose(2, 3), table)
    with pytest.raises(TypeError):
        spax.make_kv_cache(k.double(), v.double(), table)
    with pytest.raises(ValueError):
        spax.make_kv_cache(k, v, table, k_scale=torch.ones(3))
    c = spax.make_kv_cache(k, v, table)
    q = torch.zeros(3, 4, 64, dtype=torch.float16)
    lens = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError):
        spax.make_attention(c, q[:2], lens, q[:2].clone())
    with pytest.raises(TypeError):
        spax.make_attention(c, q, lens, q.float())
    with pytest.raises(TypeError):
        spax.make_attention(c, q, lens.long(), q.clone())
    with pytest.raises(ValueError):
        spax.make_kv_append(c, q, q[:, :3], q[:, :3], lens, q.clone())
    with pytest.raises(TypeError):
        spax.make_kv_append(c, q.float(), q[:, :2], q[:, :2], lens, q.clone())
    with pytest.raises(ValueError):
        spax.make_kv_append(c, None, q[:, :2], q[:, :2], lens, q.clone())
    x = torch.zeros(3, 10)
    with pytest.raises(ValueError):
        spax.make_residual_norm(x, x[:2], x, None)
    with pytest.raises(TypeError):
        spax.make_residual_norm(x, None, x.half(), None)
    with pytest.raises(ValueError):
        spax.make_residual_norm(x, x, None, x.half(), gate=torch.zeros(2, 10))
    with pytest.raises(ValueError):
        spax.make_glu(x, x[:, :5], x)
    with pytest.raises(TypeError):
        spax.make_glu(x, x.half(), x)
    # a call needs its tensors on a GPU
    for call in (lambda: spax.spax_glu(spax.make_glu(x, x.clone(), x.half())),
                 lambda: spax.spax_residual_norm(spax.make_residual_norm(x, None, None, x.half())),
                 lambda: spax.spax_paged_attention(spax.make_attention(c, q, lens, q.clone()))):
        with pytest.raises(ValueError, match="GPU"):
            call()


def test_descriptions_keep_their_tensors():
    import gc
    import weakref
    k, v, table = _tensors()
    q, out = torch.zeros(3, 4, 64, dtype=torch.float16), torch.zeros(3, 4, 64, dtype=torch.float16)
    lens = torch.zeros(3, dtype=torch.int32)
    refs = [weakref.ref(t) for t in (k, v, table, q, out, lens)]
    a = spax.make_attention(spax.make_kv_cache(k, v, table), q, lens, out)
    del k, v, table, q, out, lens
    gc.collect()
    assert all(r() is not None for r in refs)
    del a
    gc.collect()
    assert all(r() is None for r in refs)


# ------------------------------------------------------------------ the oracle itself

def test_oracle_rotation_turns_by_the_angle():
    x = np.array([1.0, 0.0, 0.0, 2.0, 7.0])
    f = [np.pi / 2, np.pi]
    assert np.allclose(olayer.rotate(x, 1, f, True), [0, 1, 0, -2, 7])   # 90 and 180 degrees
    assert np.allclose(olayer.rotate(x, 1, f, False), [0, 0, 1, -2, 7])
    assert np.allclose(olayer.rotate(x, 4, f, True), x)


def test_oracle_attention_by_hand():
    k = np.zeros((2, 1, 4, 2))
    v = np.zeros((2, 1, 4, 2))
    k[1, 0, 0], k[1, 0, 1], k[0, 0, 0] = [np.log(2), 0], [0, 5], [np.log(3), 0]
    v[1, 0, 0], v[1, 0, 1], v[0, 0, 0] = [6, 0], [0, 6], [6, 6]
    q = np.array([[[1.0, 0.0]]])
    out, lse, mass, reach = olayer.attention(q, k, v, np.array([[1, 0]]), [2], 1.0)
    assert np.allclose(out, [[[4, 2]]]) and np.allclose(lse, np.log(3)) and reach[0, 0] == np.log(2)
    # keys 2 and 3 are zeros: weights 2, 1, 1, 1, 3
    out, lse, _, _ = olayer.attention(q, k, v, np.array([[1, 0]]), [5], 1.0)
    assert np.allclose(out, [[[30 / 8, 24 / 8]]]) and np.allclose(lse, np.log(8))
    out, lse, _, _ = olayer.attention(q, k, v, np.array([[1, 0]]), [5], 1.0, window=1)
    assert np.allclose(out, [[[6, 6]]])
    out, lse, _, _ = olayer.attention(q, k, v, np.array([[1, -1]]), [5], 1.0, window=1)
    assert np.all(out == 0) and lse[0, 0] == -np.inf
    out, _, _, _ = olayer.attention(q, k, v, np.array([[1, 0]]), [9], 1.0, max_len=1)
    assert np.allclose(out, [[[6, 0]]])


def test_oracle_norm_and_glu_by_hand():
    h, x = olayer.residual_norm([[1.0, 1.0]], [[3.0, -4.0]], "rms", [1.0, 2.0], None,
                                [1.0, 1.0], None, [2.0, 1.0], 0.5, 0.0)
    # 3 / sqrt(12.5), -4 / sqrt(12.5), gated by 2 and 1, halved
    assert np.allclose(h, [[1 + 3 / 12.5 ** 0.5, 1 - 2 / 12.5 ** 0.5]])
    assert np.allclose(x, h / np.sqrt((h ** 2).mean()) * [1, 2])
    assert np.allclose(olayer.norm([1.0, 3.0], "layer", [1, 1], [5, 5], 0.0), [4, 6])
    assert np.allclose(olayer.glu([0.0, np.log(3)], [1.0, 4.0], "silu"), [0, 3 * np.log(3)])
    assert np.allclose(olayer.glu([100.0, -100.0], [2.0, 2.0], "gelu"), [200, 0])
    g = np.linspace(-3, 3, 41)
    u = np.sqrt(2 / np.pi) * (g + 0.044715 * g ** 3)
    assert np.allclose(olayer.glu(g, np.ones(41), "gelu"), 0.5 * g * (1 + np.tanh(u)))
