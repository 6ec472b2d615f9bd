"""Python binding of libspax: three-tier activation-sparse decoding GEMV on MI355X (gfx950).

Thin argument marshalling over the C ABI in ``include/spax.h``: every step of the path
(packing, tier masks, tiered GEMV, decode step, and the cache append, attention, norms and gated
activation between the projections) runs in the HIP kernels of libspax.so.
torch is used only for device memory (tensors are passed by ``data_ptr()``) and streams
(``torch.cuda.current_stream()`` by default).  The names match the C entry points.
"""

from __future__ import annotations

import ctypes as C

STEP_DEFAULT, STEP_SEPARATE, STEP_BATCHED, STEP_DETERMINISTIC = 0, 1, 2, 4

from ._lib import (ACT_GELU_TANH, ACT_SILU, NORM_LAYER, NORM_RMS, TYPE_BF16,  # noqa: F401
                   TYPE_E4M3, TYPE_F16, TYPE_F32, AttentionArgs, DecoderLayer, GluArgs,
                   KvAppendArgs, KvCache, ResidualNormArgs)
from ._lib import (FMT_FP16, FMT_INT4, MAX_DIN, MAX_MATS, MODE_THRESHOLD, MODE_TOPK,  # noqa: F401
                   MODE_TOPK_GUIDED, TIER_APPROX, TIER_FULL, TIER_SKIP, BLOCK_ERROR_FN,
                   SPAX_ERR_WORKSPACE, Layout, MoveStats, Phase, SpaxError, Step, StorageStats,
                   TierParams, check, lib, LIB_PATH)

__all__ = [
    "spax_layout_init", "spax_pack_columns", "spax_pack_columns_placed", "spax_placement_order",
    "spax_build_tiers", "spax_gemv_workspace_bytes",
    "spax_tiered_gemv", "spax_step_workspace_bytes", "spax_decode_step_projections",
    "spax_decode_step_projections_noalloc",
    "spax_key_threshold", "spax_counts_from_fractions", "spax_guided_bounds", "spax_version",
    "spax_column_ranges", "spax_pinned_workspace_bytes", "spax_tiered_gemv_pinned", "MoveStats",
    "spax_read_probe", "spax_storage_ledger", "StorageStats", "spax_block_sparsity",
    "spax_greedy_allocation", "spax_allocation_at",
    "topk_params", "threshold_params", "guided_params", "make_phase", "Layout", "TierParams",
    "Phase", "Step", "SpaxError", "LIB_PATH",
    "spax_kv_append", "spax_attention_workspace_bytes", "spax_paged_attention",
    "spax_residual_norm", "spax_glu", "spax_layers_workspace_bytes", "spax_decode_layers",
    "make_kv_cache", "make_kv_append", "make_attention", "make_residual_norm", "make_glu",
    "make_layer", "layer_array", "KvCache", "KvAppendArgs", "AttentionArgs", "ResidualNormArgs",
    "GluArgs", "DecoderLayer",
]


def _ptr(t) -> int:
    if t is None:
        return 0
    if isinstance(t, int):
        return t
    return int(t.data_ptr())


def _stream(stream) -> int:
    if stream is None:
        import torch
        return int(torch.cuda.current_stream().cuda_stream)
    if isinstance(stream, int):
        return stream
    return int(stream.cuda_stream)


# ------------------------------------------------------------------ layout / pack

def spax_layout_init(d_in: int, d_out, base_fmt: int = FMT_FP16, base_group: int = 128,
                     approx_group: int = 128) -> Layout:
    d_out = [int(v) for v in d_out]
    L = Layout()
    L.n_mats = len(d_out)
    L.d_in = int(d_in)
    for m, v in enumerate(d_out[:MAX_MATS]):
        L.d_out[m] = v
    L.base_fmt = int(base_fmt)
    L.base_group = int(base_group)
    L.approx_group = int(approx_group)
    if len(d_out) > MAX_MATS:
        L.n_mats = len(d_out)   # rejected by the library
    check(lib.spax_layout_init(C.byref(L)), "spax_layout_init")
    return L


def spax_pack_columns(layout: Layout, Ws, packed, stream=None) -> None:
    arr = (C.c_void_p * max(1, len(Ws)))(*[_ptr(w) for w in Ws])
    check(lib.spax_pack_columns(C.byref(layout), arr, _ptr(packed), _stream(stream)),
          "spax_pack_columns")


def spax_pack_columns_placed(layout: Layout, Ws, perm, packed, stream=None) -> None:
    """Pack with record p holding column perm[p] (perm: device int32 tensor of d_in)."""
    arr = (C.c_void_p * max(1, len(Ws)))(*[_ptr(w) for w in Ws])
    check(lib.spax_pack_columns_placed(C.byref(layout), arr, _ptr(perm), _ptr(packed),
                                       _stream(stream)), "spax_pack_columns_placed")


def spax_placement_order(layout: Layout, tiers):
    """Placement from calibration masks: ``tiers`` (n_tokens, d_in) uint8 on the host; returns
    the int32 order (position p holds channel order[p])."""
    import numpy as np
    t = np.ascontiguousarray(np.asarray(tiers, dtype=np.uint8))
    if t.ndim == 1:
        t = t[None, :]
    order = np.zeros(int(layout.d_in), dtype=np.int32)
    check(lib.spax_placement_order(C.byref(layout), t.ctypes.data if t.size else None,
                                   int(t.shape[0]), order.ctypes.data), "spax_placement_order")
    return order


# ------------------------------------------------------------------ tier masks

def topk_params(n_full: int, n_approx: int) -> TierParams:
    p = TierParams()
    p.mode, p.n_full, p.n_approx = MODE_TOPK, int(n_full), int(n_approx)
    p.approx_den = 1
    return p


def threshold_params(tau_skip: float, tau_full: float) -> TierParams:
    p = TierParams()
    p.mode, p.tau_skip, p.tau_full = MODE_THRESHOLD, float(tau_skip), float(tau_full)
    p.approx_den = 1
    return p


def guided_params(tau: float, n_skip_lo: int, n_skip_hi: int, approx_num: int,
                  approx_den: int) -> TierParams:
    p = TierParams()
    p.mode, p.tau = MODE_TOPK_GUIDED, float(tau)
    p.n_skip_lo, p.n_skip_hi = int(n_skip_lo), int(n_skip_hi)
    p.approx_num, p.approx_den = int(approx_num), int(approx_den)
    return p


def spax_build_tiers(x, d_in: int, params: TierParams, tier, full_idx, approx_idx, counts,
                     stream=None) -> None:
    check(lib.spax_build_tiers(_ptr(x), int(d_in), C.byref(params), _ptr(tier), _ptr(full_idx),
                               _ptr(approx_idx), _ptr(counts), _stream(stream)),
          "spax_build_tiers")


# ------------------------------------------------------------------ GEMV

def spax_gemv_workspace_bytes(layout: Layout) -> int:
    return int(lib.spax_gemv_workspace_bytes(C.byref(layout)))


def _nbytes(t) -> int:
    return 0 if t is None else t.numel() * t.element_size()


def spax_tiered_gemv(layout: Layout, packed, x, full_idx, approx_idx, counts, y, ws=None,
                     ws_bytes: int | None = None, stream=None) -> None:
    if ws_bytes is None:
        ws_bytes = _nbytes(ws)
    check(lib.spax_tiered_gemv(C.byref(layout), _ptr(packed), _ptr(x), _ptr(full_idx),
                               _ptr(approx_idx), _ptr(counts), _ptr(y), _ptr(ws), int(ws_bytes),
                               _stream(stream)),
          "spax_tiered_gemv")


# ------------------------------------------------------------------ pinned-host path

def spax_column_ranges(idx, gap: int = 0):
    """Ascending channel indices -> [(first, count), ...] after merging gaps of <= gap."""
    import numpy as np
    a = np.ascontiguousarray(np.asarray(idx, dtype=np.int32))
    n = int(a.size)
    first = np.zeros(max(n, 1), dtype=np.int32)
    count = np.zeros(max(n, 1), dtype=np.int32)
    nr = C.c_int32()
    check(lib.spax_column_ranges(a.ctypes.data if n else None, n, int(gap), first.ctypes.data,
                                 count.ctypes.data, C.byref(nr)), "spax_column_ranges")
    return [(int(first[i]), int(count[i])) for i in range(nr.value)]


def spax_storage_ledger(layout: Layout, full_idx, approx_idx, gap: int = 0,
                        block_bytes: int = 4096) -> StorageStats:
    """Bytes selected against bytes physically read at a storage granularity (host lists)."""
    import numpy as np
    f = np.ascontiguousarray(np.asarray(full_idx, dtype=np.int32))
    a = np.ascontiguousarray(np.asarray(approx_idx, dtype=np.int32))
    out = StorageStats()
    check(lib.spax_storage_ledger(C.byref(layout), f.ctypes.data if f.size else None,
                                  int(f.size), a.ctypes.data if a.size else None, int(a.size),
                                  int(gap), int(block_bytes), C.byref(out)),
          "spax_storage_ledger")
    return out


def spax_pinned_workspace_bytes(layout: Layout) -> int:
    return int(lib.spax_pinned_workspace_bytes(C.byref(layout)))


PINNED_MEMCPY, PINNED_GATHER, PINNED_HOSTGATHER = 0, 1, 2


def spax_tiered_gemv_pinned(layout: Layout, packed_host, x, full_idx, approx_idx, counts, y,
                            gap: int, ws, ws_bytes: int | None = None, stream=None,
                            transfer: int = PINNED_MEMCPY, stats: bool = True):
    """The blob in pinned host memory (e.g. a torch tensor with pin_memory=True); returns the
    byte account of the call (MoveStats), or None with stats=False (the gather transfer then
    does not wait for the device)."""
    if ws_bytes is None:
        ws_bytes = _nbytes(ws)
    st = MoveStats() if stats else None
    check(lib.spax_tiered_gemv_pinned(C.byref(layout), _ptr(packed_host), _ptr(x), _ptr(full_idx),
                                      _ptr(approx_idx), _ptr(counts), _ptr(y), int(gap),
                                      int(transfer), _ptr(ws), int(ws_bytes),
                                      C.byref(st) if st is not None else None, _stream(stream)),
          "spax_tiered_gemv_pinned")
    return st


# ------------------------------------------------------------------ decode step

def make_phase(layout: Layout, packed, x, params: TierParams, tier, full_idx, approx_idx,
               counts, y) -> Phase:
    ph = Phase()
    ph.layout = C.pointer(layout)
    ph.packed, ph.x = _ptr(packed), _ptr(x)
    ph.params = params
    ph.tier, ph.full_idx, ph.approx_idx = _ptr(tier), _ptr(full_idx), _ptr(approx_idx)
    ph.counts, ph.y = _ptr(counts), _ptr(y)
    # The struct holds raw addresses: keep the layout and every buffer alive with it, so that
    # a caller dropping its own reference cannot free (and the allocator reuse) a buffer the
    # phase still points to.
    ph._keep = (layout, packed, x, tier, full_idx, approx_idx, counts, y)
    return ph


def phase_array(phases):
    arr = (Phase * len(phases))(*phases)
    arr._keep = [getattr(p, "_keep", None) for p in phases]  # the elements are copies
    return arr


def spax_step_workspace_bytes(phases) -> int:
    arr = phases if isinstance(phases, C.Array) else phase_array(phases)
    return int(lib.spax_step_workspace_bytes(arr, len(arr)))


def _step(phases, ws, ws_bytes, flags, events):
    arr = phases if isinstance(phases, C.Array) else phase_array(phases)
    if ws_bytes is None:
        ws_bytes = _nbytes(ws)
    st = Step()
    st.n_phases = len(arr)
    st.flags = int(flags)
    st.phases = C.cast(arr, C.POINTER(Phase))
    st.ws = _ptr(ws)
    st.ws_bytes = int(ws_bytes)
    if events is not None:
        if len(events) != 2 * len(arr):
            raise ValueError("need 2 * n_phases events")
        ev = (C.c_void_p * len(events))(*[int(e.cuda_event) for e in events])
        st.events = C.cast(ev, C.POINTER(C.c_void_p))
        st._keep = (arr, ev)
    else:
        st._keep = (arr,)
    return st


def spax_decode_step_projections(phases, ws, ws_bytes: int | None = None, flags: int = 0,
                                 stream=None, events=None) -> None:
    """``events``: optional list of 2 * n_phases torch.cuda.Event(enable_timing=True);
    events[2i] -> events[2i+1] then brackets phase i's GEMV launch on the stream."""
    st = _step(phases, ws, ws_bytes, flags, events)
    check(lib.spax_decode_step_projections(C.byref(st), _stream(stream)),
          "spax_decode_step_projections")


def spax_decode_step_projections_noalloc(phases, flags: int = 0, stream=None,
                                         events=None) -> None:
    """The same step with no workspace: the batched form keeps its descriptor tables in the
    library's static device scratch (calls on one GPU must not overlap)."""
    st = _step(phases, None, 0, flags, events)
    check(lib.spax_decode_step_projections_noalloc(C.byref(st), _stream(stream)),
          "spax_decode_step_projections_noalloc")


# ------------------------------------------------------------------ between the projections
#
# A make_* function describes one call in terms of tensors (shapes, strides, types and the device
# are checked here, the rest by the library); the struct it returns keeps its tensors alive and
# is handed to the call as often as their contents change.  The call runs on the tensors' own
# device, on that device's current stream unless one is given.

def _type_of(t) -> int:
    name = str(t.dtype)
    types = {"torch.float32": TYPE_F32, "torch.float16": TYPE_F16, "torch.bfloat16": TYPE_BF16,
             "torch.float8_e4m3fn": TYPE_E4M3}
    if name not in types:
        raise TypeError(f"no operator takes {name}")
    return types[name]


def _rows(t, name, dims):
    """Checks a tensor of `dims` axes whose last axis is contiguous."""
    if t.dim() != dims:
        raise ValueError(f"{name} has {t.dim()} axes, not {dims}")
    if t.shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name}: the last axis is not contiguous")
    return t


def _flat(t, name, n, dtype):
    if t is None:
        return None
    if str(t.dtype) != dtype:
        raise TypeError(f"{name} is {t.dtype}, not {dtype}")
    if t.numel() != n or not t.is_contiguous():
        raise ValueError(f"{name} is not a contiguous tensor of {n} values")
    return t


def _int32(n, name) -> int:
    """n for a 32-bit field, which would cut it off without a word."""
    n = int(n)
    if not -2 ** 31 <= n < 2 ** 31:
        raise ValueError(f"{name} {n} does not fit 32 bits")
    return n


def _same_shape(t, name, shape):
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, not {tuple(shape)}")


def _keep(struct, *tensors, parts=()):
    """Ties the tensors (and the structs in parts) to the struct; all are on one device."""
    devices = {t.device for t in tensors if t is not None}
    devices |= {p._device for p in parts}
    if len(devices) > 1:
        raise ValueError(f"tensors on different devices: {sorted(map(str, devices))}")
    struct._keep = (tensors, parts)
    return _on(struct, next(iter(devices)))


def _on(struct, device):
    struct._device = device
    struct._index = device.index if device.type == "cuda" else None
    return struct


def _workspace(ws, desc):
    """A workspace tensor is in one piece on the device of the tensors described."""
    device = getattr(ws, "device", None)
    if device is None:      # an address, or none needed
        return
    if not ws.is_contiguous():
        raise ValueError("the workspace is not contiguous")
    if device != desc._device and ws.numel():
        raise ValueError(f"the workspace is on {device}, the tensors are on {desc._device}")


def _fast(name, slow):
    """torch's own C function for `slow`, where this torch has it (a microsecond a call less)."""
    import torch
    return getattr(torch._C, name, slow)


def _public_stream(index):
    import torch
    return torch.cuda.current_stream(index).cuda_stream


def _public_device():
    import torch
    return torch.cuda.current_device()


_current_stream = _fast("_cuda_getCurrentRawStream", _public_stream)
_current_device = _fast("_cuda_getDevice", _public_device)


def _call(fn, where, desc, stream, *args):
    """Runs fn(*args, stream) with the device of desc's tensors current."""
    index = desc._index
    if index is None:
        raise ValueError(f"{where}: the tensors are on {desc._device}, not on a GPU")
    if index == _current_device():
        status = fn(*args, _current_stream(index) if stream is None else _stream(stream))
    else:
        import torch
        with torch.cuda.device(index):
            status = fn(*args, _stream(stream))
    if status:
        check(status, where)


def make_kv_cache(k, v, page_table, k_scale=None, v_scale=None) -> KvCache:
    """A paged cache: k and v [n_pages, n_kv_heads, page_size, head_dim] (a view of any order,
    e.g. of [n_pages, page_size, n_kv_heads, head_dim] with its middle axes swapped), page_table
    int32 [n_seqs, max_pages]; scales fp32 [n_kv_heads] for float8_e4m3fn."""
    _rows(k, "k", 4)
    _rows(v, "v", 4)
    _same_shape(v, "v", k.shape)
    if v.dtype != k.dtype:
        raise TypeError(f"v is {v.dtype}, k is {k.dtype}")
    _rows(page_table, "page_table", 2)
    if str(page_table.dtype) != "torch.int32":
        raise TypeError(f"page_table is {page_table.dtype}, not torch.int32")
    c = KvCache()
    c.type = _type_of(k)
    for name, n in zip(("n_pages", "n_kv_heads", "page_size", "head_dim"), k.shape):
        setattr(c, name, _int32(n, name))
    c.k, c.v, c.page_table = k.data_ptr(), v.data_ptr(), page_table.data_ptr()
    c.k_scale = _ptr(_flat(k_scale, "k_scale", k.shape[1], "torch.float32"))
    c.v_scale = _ptr(_flat(v_scale, "v_scale", k.shape[1], "torch.float32"))
    c.k_page_stride, c.k_head_stride, c.k_row_stride = k.stride()[:3]
    c.v_page_stride, c.v_head_stride, c.v_row_stride = v.stride()[:3]
    c.n_seqs = _int32(page_table.shape[0], "n_seqs")
    c.max_pages = _int32(page_table.shape[1], "max_pages")
    c.table_stride = page_table.stride(0)
    return _keep(c, k, v, page_table, k_scale, v_scale)


def make_kv_append(cache: KvCache, q, k, v, positions, q_out, seq=None, inv_freq=None,
                   interleaved: bool = False) -> KvAppendArgs:
    """q [n_tokens, n_heads, head_dim], k and v [n_tokens, n_kv_heads, head_dim] of one type (views
    of a fused row, for instance), q_out like q in the cache's type (float16 or bfloat16 for
    an e4m3 cache); q and q_out may both be None.  positions int32 [n_tokens], seq likewise
    (None: token t belongs to sequence t), inv_freq fp32 [rot_dim / 2] (None: no rotation)."""
    _rows(k, "k", 3)
    _rows(v, "v", 3)
    n = _int32(k.shape[0], "n_tokens")
    shape = (n, cache.n_kv_heads, cache.head_dim)
    _same_shape(k, "k", shape)
    _same_shape(v, "v", shape)
    a = KvAppendArgs()
    a.cache = C.pointer(cache)
    a.src_type = _type_of(k)
    a.n_tokens = n
    if (q is None) != (q_out is None):
        raise ValueError("q and q_out come together")
    if q is not None:
        _rows(q, "q", 3)
        _same_shape(q, "q", (n, q.shape[1], cache.head_dim))
        _rows(q_out, "q_out", 3)
        _same_shape(q_out, "q_out", q.shape)
        a.q, a.q_out, a.n_heads = q.data_ptr(), q_out.data_ptr(), _int32(q.shape[1], "n_heads")
        a.q_token_stride, a.q_head_stride = q.stride()[:2]
        a.out_token_stride, a.out_head_stride = q_out.stride()[:2]
        a.out_type = _type_of(q_out)
    else:
        a.out_type = TYPE_F16 if cache.type == TYPE_E4M3 else cache.type
    for t, name in ((q, "q"), (v, "v")):
        if t is not None and t.dtype != k.dtype:
            raise TypeError(f"{name} is {t.dtype}, k is {k.dtype}")
    a.k, a.v = k.data_ptr(), v.data_ptr()
    a.k_token_stride, a.k_head_stride = k.stride()[:2]
    a.v_token_stride, a.v_head_stride = v.stride()[:2]
    a.positions = _ptr(_flat(positions, "positions", n, "torch.int32"))
    a.seq = _ptr(_flat(seq, "seq", n, "torch.int32"))
    if inv_freq is not None:
        a.inv_freq = _ptr(_flat(inv_freq, "inv_freq", inv_freq.numel(), "torch.float32"))
        a.rot_dim = _int32(2 * inv_freq.numel(), "rot_dim")
    a.interleaved = int(bool(interleaved))
    return _keep(a, q, k, v, positions, q_out, seq, inv_freq, parts=(cache,))


def spax_kv_append(args: KvAppendArgs, stream=None) -> None:
    _call(lib.spax_kv_append, "spax_kv_append", args, stream, args)


def make_attention(cache: KvCache, q, lens, out, max_len: int | None = None,
                   scale: float | None = None, window: int = 0, lse=None) -> AttentionArgs:
    """q and out [n_seqs, n_heads, head_dim], lens int32 [n_seqs] (keys of each sequence, the new
    token's own among them), lse fp32 [n_seqs, n_heads] or None.  max_len: bound on lens
    (default: what the page table holds); scale: default 1 / sqrt(head_dim)."""
    _rows(q, "q", 3)
    _rows(out, "out", 3)
    _same_shape(q, "q", (cache.n_seqs, q.shape[1], cache.head_dim))
    _same_shape(out, "out", q.shape)
    if q.dtype != out.dtype:
        raise TypeError(f"out is {out.dtype}, q is {q.dtype}")
    a = AttentionArgs()
    a.cache = C.pointer(cache)
    a.q, a.out, a.type = q.data_ptr(), out.data_ptr(), _type_of(q)
    a.n_heads = _int32(q.shape[1], "n_heads")
    a.q_seq_stride, a.q_head_stride = q.stride()[:2]
    a.out_seq_stride, a.out_head_stride = out.stride()[:2]
    a.lens = _ptr(_flat(lens, "lens", cache.n_seqs, "torch.int32"))
    a.lse = _ptr(_flat(lse, "lse", cache.n_seqs * a.n_heads, "torch.float32"))
    a.max_len = _int32(cache.max_pages * cache.page_size if max_len is None else max_len, "max_len")
    a.scale = float(cache.head_dim ** -0.5 if scale is None else scale)
    a.window = _int32(window, "window")
    return _keep(a, q, lens, out, lse, parts=(cache,))


def spax_attention_workspace_bytes(args: AttentionArgs) -> int:
    return int(lib.spax_attention_workspace_bytes(C.byref(args)))


def spax_paged_attention(args: AttentionArgs, ws=None, ws_bytes: int | None = None,
                         stream=None) -> None:
    _workspace(ws, args)
    if ws_bytes is None:
        ws_bytes = _nbytes(ws)
    _call(lib.spax_paged_attention, "spax_paged_attention", args, stream, args, _ptr(ws),
          ws_bytes)


_NORMS = {"rms": NORM_RMS, "layer": NORM_LAYER}
_ACTS = {"silu": ACT_SILU, "gelu": ACT_GELU_TANH}


def make_residual_norm(residual, block, residual_out, x, kind: str = "rms", pre_weight=None,
                       pre_bias=None, post_weight=None, post_bias=None, gate=None,
                       scale: float = 1.0, eps: float = 1e-5) -> ResidualNormArgs:
    """residual, block, residual_out, x [n_rows, d] (any may be None, see the library), gate [d],
    [1, d] or [n_rows, d]; weights and biases fp32 [d].  kind: 'rms' or 'layer'."""
    a = ResidualNormArgs()
    a.kind = _NORMS.get(kind, kind)
    shape = None
    for t, name in ((residual, "residual"), (block, "block"), (residual_out, "residual_out"),
                    (x, "x")):
        if t is None:
            continue
        _rows(t, name, 2)
        if shape is None:
            shape = tuple(t.shape)
        _same_shape(t, name, shape)
        setattr(a, name, t.data_ptr())
        setattr(a, name + "_stride", t.stride(0))
    if shape is None:
        raise ValueError("no rows given")
    a.n_rows, a.d = _int32(shape[0], "n_rows"), _int32(shape[1], "d")
    if residual is not None and residual_out is not None and residual.dtype != residual_out.dtype:
        raise TypeError(f"residual_out is {residual_out.dtype}, residual is {residual.dtype}")
    stream_type = residual if residual is not None else residual_out
    a.residual_type = TYPE_F32 if stream_type is None else _type_of(stream_type)
    a.block_type = TYPE_F32 if block is None else _type_of(block)
    a.x_type = TYPE_F32 if x is None else _type_of(x)
    if gate is not None:
        if gate.dim() == 1:
            gate = gate.view(1, -1) if gate.is_contiguous() else gate[None]
        _rows(gate, "gate", 2)
        if tuple(gate.shape) not in ((1, shape[1]), shape):
            raise ValueError(f"gate has shape {tuple(gate.shape)}")
        a.gate, a.gate_type = gate.data_ptr(), _type_of(gate)
        a.gate_stride = 0 if gate.shape[0] == 1 else gate.stride(0)
    for t, name in ((pre_weight, "pre_weight"), (pre_bias, "pre_bias"),
                    (post_weight, "post_weight"), (post_bias, "post_bias")):
        setattr(a, name, _ptr(_flat(t, name, shape[1], "torch.float32")))
    a.scale, a.eps = float(scale), float(eps)
    return _keep(a, residual, block, residual_out, x, gate, pre_weight, pre_bias, post_weight,
                 post_bias)


def spax_residual_norm(args: ResidualNormArgs, stream=None) -> None:
    _call(lib.spax_residual_norm, "spax_residual_norm", args, stream, args)


def make_glu(gate, up, x, act: str = "silu") -> GluArgs:
    """gate, up and x [n_rows, d] (gate and up of one type).  act: 'silu' or 'gelu' (tanh form)."""
    a = GluArgs()
    for t, name in ((gate, "gate"), (up, "up"), (x, "x")):
        _rows(t, name, 2)
        _same_shape(t, name, gate.shape)
        setattr(a, name, t.data_ptr())
        setattr(a, name + "_stride", t.stride(0))
    if gate.dtype != up.dtype:
        raise TypeError(f"up is {up.dtype}, gate is {gate.dtype}")
    a.src_type, a.x_type, a.act = _type_of(gate), _type_of(x), _ACTS.get(act, act)
    a.n_rows, a.d = _int32(gate.shape[0], "n_rows"), _int32(gate.shape[1], "d")
    return _keep(a, gate, up, x)


def spax_glu(args: GluArgs, stream=None) -> None:
    _call(lib.spax_glu, "spax_glu", args, stream, args)


def make_layer(qkv: Phase, append: KvAppendArgs, attention: AttentionArgs, o: Phase,
               attn_norm: ResidualNormArgs, gate_up: Phase, glu: GluArgs, down: Phase,
               mlp_norm: ResidualNormArgs) -> DecoderLayer:
    """One decoder layer of spax_decode_layers, in the order in which its parts run."""
    parts = dict(qkv=qkv, append=append, attention=attention, o=o, attn_norm=attn_norm,
                 gate_up=gate_up, glu=glu, down=down, mlp_norm=mlp_norm)
    L = DecoderLayer()
    for name, p in parts.items():
        setattr(L, name, C.pointer(p))
    L._keep = parts
    devices = {p._device for p in (append, attention, attn_norm, glu, mlp_norm)}
    for p in (qkv, o, gate_up, down):
        devices |= {t.device for t in getattr(p, "_keep", ()) if hasattr(t, "device")}
    if len(devices) > 1:
        raise ValueError(f"parts on different devices: {sorted(map(str, devices))}")
    return _on(L, next(iter(devices)))


def layer_array(layers):
    arr = (DecoderLayer * len(layers))(*layers)
    arr._keep = [L._keep for L in layers]
    devices = {L._device for L in layers}
    if len(devices) != 1:
        raise ValueError(f"{len(layers)} layers on {len(devices)} devices")
    return _on(arr, next(iter(devices)))


def spax_layers_workspace_bytes(layers) -> int:
    arr = layers if isinstance(layers, C.Array) else layer_array(layers)
    return int(lib.spax_layers_workspace_bytes(arr, len(arr)))


def spax_decode_layers(layers, ws, ws_bytes: int | None = None, flags: int = 0,
                       stream=None) -> None:
    """A whole batch-one decode step through decoder layers: their projections with the operators
    between them.  layers: make_layer structs, or their layer_array."""
    arr = layers if isinstance(layers, C.Array) else layer_array(layers)
    _workspace(ws, arr)
    if ws_bytes is None:
        ws_bytes = _nbytes(ws)
    _call(lib.spax_decode_layers, "spax_decode_layers", arr, stream, arr, len(arr),
          int(flags), _ptr(ws), int(ws_bytes))


# ------------------------------------------------------------------ diagnostics

def spax_read_probe(buf, out, nbytes: int | None = None, offset: int = 0, stream=None) -> int:
    """Reads ``nbytes`` bytes of the device tensor ``buf`` from byte ``offset`` (default: all
    of it); every wave stores the XOR of the 32-bit words it read in its own word of the
    device tensor ``out`` (int32/uint32).  Returns how many leading words of ``out`` were
    written: their XOR is the XOR of all words read."""
    total = buf.numel() * buf.element_size()
    if nbytes is None:
        nbytes = total - offset
    if offset < 0 or nbytes < 0 or offset + nbytes > total:
        raise ValueError("read range outside the buffer")
    n = C.c_int32()
    words = out.numel() * out.element_size() // 4
    check(lib.spax_read_probe(C.c_void_p(_ptr(buf) + int(offset)), int(nbytes), _ptr(out),
                              int(min(words, 2**31 - 1)), C.byref(n), _stream(stream)),
          "spax_read_probe")
    return int(n.value)


# ------------------------------------------------------------------ sparsity budgets (host)

def spax_block_sparsity(sens, s: float, lam: float, s_min: float = 0.05, s_max: float = 0.95):
    """Per-block sparsity targets from block sensitivities (float64 array)."""
    import numpy as np
    a = np.ascontiguousarray(np.asarray(sens, dtype=np.float64))
    out = np.zeros(max(1, a.size), dtype=np.float64)
    check(lib.spax_block_sparsity(a.ctypes.data if a.size else None, int(a.size), float(s),
                                  float(lam), float(s_min), float(s_max), out.ctypes.data),
          "spax_block_sparsity")
    return out[:a.size]


def spax_greedy_allocation(params, alpha: float, P_max: float, block_error):
    """The greedy walk's rows as a float64 array [n_rows, 1 + n_mats] (P, then p per matrix).
    ``block_error(p)``: error of a trial allocation (a float64 array) -> float."""
    import numpy as np
    f = np.ascontiguousarray(np.asarray(params, dtype=np.float64))
    n = int(f.size)

    def _cb(p, n_mats, user):
        return float(block_error(np.ctypeslib.as_array(p, shape=(n_mats,)).copy()))

    cb = BLOCK_ERROR_FN(_cb)
    cap = 64
    while True:
        rows = np.zeros((cap, 1 + n), dtype=np.float64)
        nr = C.c_int32()
        st = lib.spax_greedy_allocation(f.ctypes.data if n else None, n, float(alpha),
                                        float(P_max), cb, None, rows.ctypes.data, cap,
                                        C.byref(nr))
        if st == SPAX_ERR_WORKSPACE and nr.value > cap:
            cap = nr.value
            continue
        check(st, "spax_greedy_allocation")
        return rows[:nr.value].copy()


def spax_allocation_at(rows, target: float):
    import numpy as np
    r = np.ascontiguousarray(np.asarray(rows, dtype=np.float64))
    n_mats = r.shape[1] - 1
    p = np.zeros(max(1, n_mats), dtype=np.float64)
    check(lib.spax_allocation_at(r.ctypes.data, int(r.shape[0]), int(n_mats), float(target),
                                 p.ctypes.data), "spax_allocation_at")
    return p[:n_mats]


# ------------------------------------------------------------------ host helpers

def spax_key_threshold(tau: float) -> int:
    return int(lib.spax_key_threshold(float(tau)))


def spax_counts_from_fractions(d: int, p_full: float, p_approx: float):
    a, b = C.c_int32(), C.c_int32()
    check(lib.spax_counts_from_fractions(int(d), float(p_full), float(p_approx), C.byref(a),
                                         C.byref(b)), "spax_counts_from_fractions")
    return int(a.value), int(b.value)


def spax_guided_bounds(d: int, s: float, delta: float):
    a, b = C.c_int32(), C.c_int32()
    check(lib.spax_guided_bounds(int(d), float(s), float(delta), C.byref(a), C.byref(b)),
          "spax_guided_bounds")
    return int(a.value), int(b.value)


def spax_version() -> str:
    return lib.spax_version().decode()
