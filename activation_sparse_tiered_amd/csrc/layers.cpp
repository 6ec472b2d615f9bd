// spax_decode_layers: a batch-one decode step through whole decoder layers.
#include <cstdio>
#include <vector>

#include "layer_ops.h"

using namespace spax;

namespace {

constexpr int kPhases = 4;
const char* const kPhaseName[kPhases] = {"qkv", "o", "gate_up", "down"};

const spax_phase* phase_of(const spax_decoder_layer& L, int k) {
  const spax_phase* p[kPhases] = {L.qkv, L.o, L.gate_up, L.down};
  return p[k];
}

void phase_name(int i, char* out, size_t n) {
  snprintf(out, n, "layer %d, %s", i / kPhases, kPhaseName[i % kPhases]);
}

bool inside(const void* p, size_t n, const void* base, size_t size) {
  const uintptr_t a = (uintptr_t)p, b = (uintptr_t)base;
  return a >= b && a + n <= b + size;
}

int part_fail(int st, int layer, const char* part) {
  char msg[400];
  snprintf(msg, sizeof(msg), "%s", spax_last_error());
  return fail(st, "layer %d, %s: %s", layer, part, msg);
}

// Two descriptions find the same values of one sequence.
bool same_cache(const spax_kv_cache& x, const spax_kv_cache& y) {
  return x.k == y.k && x.v == y.v && x.page_table == y.page_table && x.k_scale == y.k_scale &&
         x.v_scale == y.v_scale && x.type == y.type && x.n_pages == y.n_pages &&
         x.page_size == y.page_size && x.n_kv_heads == y.n_kv_heads &&
         x.head_dim == y.head_dim && x.k_page_stride == y.k_page_stride &&
         x.k_head_stride == y.k_head_stride && x.k_row_stride == y.k_row_stride &&
         x.v_page_stride == y.v_page_stride && x.v_head_stride == y.v_head_stride &&
         x.v_row_stride == y.v_row_stride;
}

// The operators after each phase, with the buffers they touch.
struct Parts {
  Spans append, attention, attn_norm, glu, mlp_norm;
};

int check_parts(const spax_decoder_layer& L, int i, Parts* b) {
  if (!L.qkv || !L.append || !L.attention || !L.o || !L.attn_norm || !L.gate_up || !L.glu ||
      !L.down || !L.mlp_norm)
    return fail(SPAX_ERR_NULL, "layer %d: a part is NULL", i);
  int st;
  if ((st = check_kv_append(L.append, &b->append))) return part_fail(st, i, "append");
  if ((st = check_attention(L.attention, &b->attention))) return part_fail(st, i, "attention");
  if ((st = check_residual_norm(L.attn_norm, &b->attn_norm))) return part_fail(st, i, "attn_norm");
  if ((st = check_glu(L.glu, &b->glu))) return part_fail(st, i, "glu");
  if ((st = check_residual_norm(L.mlp_norm, &b->mlp_norm))) return part_fail(st, i, "mlp_norm");
  for (int k = 0; k < kPhases; ++k)
    if (!phase_of(L, k)->layout)
      return part_fail(fail(SPAX_ERR_NULL, "layout is NULL"), i, kPhaseName[k]);
  const auto wired = [&](bool ok, const char* part, const char* to) {
    return ok ? SPAX_OK : fail(SPAX_ERR_PARAM, "layer %d: %s is not wired to %s", i, part, to);
  };
  const auto y_bytes = [](const spax_phase* p) { return 4 * (size_t)p->layout->d_out_total; };
  const spax_kv_append_args& ap = *L.append;
  const spax_attention_args& at = *L.attention;
  if (ap.n_tokens != 1 || at.cache->n_seqs != 1 || L.attn_norm->n_rows != 1 ||
      L.glu->n_rows != 1 || L.mlp_norm->n_rows != 1)
    return fail(SPAX_ERR_SHAPE, "layer %d: a batch-one step passes one row through every part", i);
  const int dim = at.cache->head_dim;
  bool ok = ap.src_type == SPAX_F32 && ap.q;
  for (int s = 0; ok && s < b->append.n; ++s) {
    const Span& x = b->append.s[s];
    if (x.p == ap.q || x.p == ap.k || x.p == ap.v)
      ok = inside(x.p, x.bytes, L.qkv->y, y_bytes(L.qkv));
  }
  if ((st = wired(ok, "append", "qkv's y"))) return st;
  ok = at.q == ap.q_out && at.type == ap.out_type && at.n_heads == ap.n_heads &&
       (at.n_heads == 1 || at.q_head_stride == ap.out_head_stride) &&
       same_cache(*at.cache, *ap.cache);
  if ((st = wired(ok, "attention", "append's q_out and cache"))) return st;
  ok = (const void*)L.o->x == at.out && at.type == SPAX_F16 &&
       (at.n_heads == 1 || at.out_head_stride == dim) &&
       L.o->layout->d_in == at.n_heads * dim;
  if ((st = wired(ok, "o", "the attention's out"))) return st;
  const auto norm_ok = [&](const spax_residual_norm_args* n, const spax_phase* from) {
    return n->block == from->y && n->block_type == SPAX_F32 && n->x && n->x_type == SPAX_F16 &&
           n->d == from->layout->d_out_total;
  };
  if ((st = wired(norm_ok(L.attn_norm, L.o), "attn_norm", "o's y"))) return st;
  ok = (const void*)L.gate_up->x == L.attn_norm->x && L.gate_up->layout->d_in == L.attn_norm->d;
  if ((st = wired(ok, "gate_up", "attn_norm's x"))) return st;
  ok = L.glu->src_type == SPAX_F32 &&
       inside(L.glu->gate, 4 * (size_t)L.glu->d, L.gate_up->y, y_bytes(L.gate_up)) &&
       inside(L.glu->up, 4 * (size_t)L.glu->d, L.gate_up->y, y_bytes(L.gate_up));
  if ((st = wired(ok, "glu", "gate_up's y"))) return st;
  ok = (const void*)L.down->x == L.glu->x && L.glu->x_type == SPAX_F16 &&
       L.down->layout->d_in == L.glu->d;
  if ((st = wired(ok, "down", "glu's x"))) return st;
  return wired(norm_ok(L.mlp_norm, L.down), "mlp_norm", "down's y");
}

struct LayerHooks final : StepHooks {
  const spax_decoder_layer* layers = nullptr;
  std::vector<Parts> parts;
  void* ws = nullptr;
  int after(int i, hipStream_t s) override {
    const spax_decoder_layer& L = layers[i / kPhases];
    int st = SPAX_OK;
    switch (i % kPhases) {
      case 0:
        st = launch_kv_append(L.append, s);
        return st ? st : launch_attention(L.attention, ws, s);
      case 1: return launch_residual_norm(L.attn_norm, s);
      case 2: return launch_glu(L.glu, s);
      default: return launch_residual_norm(L.mlp_norm, s);
    }
  }
  bool touches_after(int i, const void* p, size_t n) const override {
    const Parts& b = parts[i / kPhases];
    const Spans* use[2] = {nullptr, nullptr};
    switch (i % kPhases) {
      case 0: use[0] = &b.append; use[1] = &b.attention; break;
      case 1: use[0] = &b.attn_norm; break;
      case 2: use[0] = &b.glu; break;
      default: use[0] = &b.mlp_norm; break;
    }
    for (const Spans* u : use)
      for (int k = 0; u && k < u->n; ++k)
        if (overlaps(u->s[k].p, u->s[k].bytes, p, n)) return true;
    return false;
  }
};

std::vector<spax_phase> phases_of(const spax_decoder_layer* layers, int32_t n) {
  std::vector<spax_phase> v;
  v.reserve((size_t)n * kPhases);
  for (int i = 0; i < n; ++i)
    for (int k = 0; k < kPhases; ++k) v.push_back(*phase_of(layers[i], k));
  return v;
}

int decode_layers(const spax_decoder_layer* layers, int32_t n, int32_t flags, void* ws,
                  size_t ws_bytes, hipStream_t stream) {
  if (!layers) return fail(SPAX_ERR_NULL, "layers is NULL");
  if (n < 1 || n > 65536) return fail(SPAX_ERR_SHAPE, "n_layers %d outside 1..65536", n);
  if (flags & SPAX_STEP_BATCHED)
    return fail(SPAX_ERR_UNSUPPORTED, "SPAX_STEP_BATCHED needs independent phases");
  LayerHooks hooks;
  hooks.layers = layers;
  hooks.ws = ws;
  hooks.parts.resize((size_t)n);
  size_t need = 0;
  int st;
  for (int i = 0; i < n; ++i) {
    if ((st = check_parts(layers[i], i, &hooks.parts[i]))) return st;
    if (i + 1 < n && layers[i + 1].qkv &&
        ((const void*)layers[i + 1].qkv->x != layers[i].mlp_norm->x ||
         (layers[i + 1].qkv->layout &&
          layers[i + 1].qkv->layout->d_in != layers[i].mlp_norm->d)))
      return fail(SPAX_ERR_PARAM, "layer %d: qkv is not wired to the previous mlp_norm's x",
                  i + 1);
    const size_t w = attention_plan(layers[i].attention).ws_bytes;
    need = w > need ? w : need;
  }
  const std::vector<spax_phase> phases = phases_of(layers, n);
  spax_step step{};
  step.n_phases = n * kPhases;
  step.flags = flags;
  step.phases = phases.data();
  step.ws = ws;
  step.ws_bytes = ws_bytes;
  if ((st = validate_step(&step, false, phase_name))) return st;
  if (flags & SPAX_STEP_DETERMINISTIC) {
    const size_t det = deterministic_workspace_bytes(phases.data(), step.n_phases);
    need = det > need ? det : need;
  }
  if (need) {
    if (!ws) return fail(SPAX_ERR_NULL, "workspace is NULL");
    if (!aligned(ws, 256)) return fail(SPAX_ERR_ALIGN, "ws must be 256-byte aligned");
    if (ws_bytes < need)
      return fail(SPAX_ERR_WORKSPACE, "workspace %zu bytes < required %zu", ws_bytes, need);
    for (int i = 0; i < step.n_phases; ++i)
      if (phase_touches(phases[i], ws, need) || hooks.touches_after(i, ws, need))
        return fail(SPAX_ERR_PARAM, "the workspace overlaps a buffer of layer %d", i / kPhases);
  }
  return launch_decode_step(&step, stream, false, &hooks);
}

}  // namespace

extern "C" {

size_t spax_layers_workspace_bytes(const spax_decoder_layer* layers, int32_t n_layers) {
  if (!layers || n_layers < 1 || n_layers > 65536) return 0;
  size_t need = 0;
  const int st = no_throw([&] {
    Parts b;
    for (int i = 0; i < n_layers; ++i) {
      const int e = check_parts(layers[i], i, &b);
      if (e) return e;
      const size_t w = attention_plan(layers[i].attention).ws_bytes;
      need = w > need ? w : need;
    }
    const std::vector<spax_phase> phases = phases_of(layers, n_layers);
    const size_t w = spax_step_workspace_bytes(phases.data(), (int32_t)phases.size());
    if (w == 0) return (int)SPAX_ERR_SHAPE;
    need = w > need ? w : need;
    return (int)SPAX_OK;
  });
  if (st) {
    clear_error();
    return 0;
  }
  return need;
}

int spax_decode_layers(const spax_decoder_layer* layers, int32_t n_layers, int32_t flags,
                       void* ws, size_t ws_bytes, hipStream_t stream) {
  clear_error();
  return no_throw([&] { return decode_layers(layers, n_layers, flags, ws, ws_bytes, stream); });
}

}  // extern "C"
