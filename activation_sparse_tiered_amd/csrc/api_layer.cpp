// Entry points of the operators between the projections: argument validation, then launches.
// Every check runs before anything is enqueued; on error no output is touched.
#include <cmath>
#include <cstring>
#include <utility>

#include "layer_ops.h"

using namespace spax;

namespace spax {
namespace {

bool is_float_type(int t) { return t == SPAX_F32 || t == SPAX_F16 || t == SPAX_BF16; }

// n0 rows (step s0) of n1 pieces (step s1) of d values.
void add_rows(Spans* b, const void* p, int64_t n0, int64_t s0, int64_t n1, int64_t s1, int64_t d,
              int type, bool out, const char* name) {
  if (n0 < 1 || n1 < 1) return;
  const size_t eb = (size_t)elem::bytes_of(type);
  const int64_t row = (n1 - 1) * s1 + d;
  b->add(p, (size_t)((n0 - 1) * s0 + row) * eb, out, name, n0 > 1 ? (size_t)row * eb : 0,
         n0 > 1 ? (size_t)s0 * eb : 0);
}

// Strides of n0 x n1 x ... rows of d values do not make rows overlap: sorted by stride, each
// axis steps past everything the axes below it cover.
bool strides_ok(const int64_t* n, const int64_t* s, int axes, int64_t d) {
  int order[4] = {0, 1, 2, 3};
  for (int i = 0; i < axes; ++i)
    for (int k = i + 1; k < axes; ++k)
      if (s[order[k]] < s[order[i]]) std::swap(order[i], order[k]);
  int64_t extent = d;
  for (int i = 0; i < axes; ++i) {
    const int x = order[i];
    if (n[x] <= 1) continue;
    if (s[x] < extent) return false;
    extent = (n[x] - 1) * s[x] + extent;
  }
  return true;
}
// A stride of n rows that keeps every offset far inside 64 bits.
bool stride_range(int64_t n, int64_t s) {
  constexpr int64_t kMaxExtent = (int64_t)1 << 46;
  return s >= 0 && s <= kMaxExtent && (n <= 1 || s <= kMaxExtent / (n - 1));
}

int check_rows2(const char* name, int64_t n0, int64_t s0, int64_t n1, int64_t s1, int64_t d,
                bool out) {
  if (n0 < 1 || n1 < 1) return SPAX_OK;
  const int64_t n[2] = {n0, n1}, s[2] = {s0, s1};
  if (!stride_range(n0, s0) || !stride_range(n1, s1))
    return fail(SPAX_ERR_PARAM, "%s: strides (%lld, %lld) out of range", name, (long long)s0,
                (long long)s1);
  // inputs may repeat a row (a stride of 0 along an axis), outputs may not
  if (out && !strides_ok(n, s, 2, d))
    return fail(SPAX_ERR_PARAM, "%s: strides (%lld, %lld) make its rows overlap", name,
                (long long)s0, (long long)s1);
  return SPAX_OK;
}

bool is(const Span& x, const char* name) { return strcmp(x.name, name) == 0; }

// No output shares a byte with another buffer, save pairs that allowed(output, other) excuses.
// It goes by their names: another input may start at the same address with other strides.
template <class F>
int check_overlaps(const Spans& b, F&& allowed) {
  for (int i = 0; i < b.n; ++i)
    for (int k = 0; k < b.n; ++k) {
      if (i == k || !b.s[i].out || (b.s[k].out && k < i)) continue;
      if (shares(b.s[i], b.s[k]) && !allowed(b.s[i], b.s[k]))
        return fail(SPAX_ERR_PARAM, "%s overlaps %s", b.s[i].name, b.s[k].name);
    }
  return SPAX_OK;
}

int check_cache(const spax_kv_cache* c) {
  if (!c) return fail(SPAX_ERR_NULL, "cache is NULL");
  if (!c->k || !c->v || !c->page_table)
    return fail(SPAX_ERR_NULL, "cache: k, v and page_table are required");
  if (c->type != SPAX_F16 && c->type != SPAX_BF16 && c->type != SPAX_E4M3)
    return fail(SPAX_ERR_UNSUPPORTED, "cache: type %d", c->type);
  if (c->type != SPAX_E4M3 && (c->k_scale || c->v_scale))
    return fail(SPAX_ERR_UNSUPPORTED, "cache: scales belong to an E4M3 cache");
  const int d = c->head_dim;
  if (d != 64 && d != 96 && d != 128 && d != 192 && d != 256)
    return fail(SPAX_ERR_SHAPE, "cache: head_dim %d is not 64, 96, 128, 192 or 256", d);
  if (c->page_size < 4 || c->page_size > 65536 || (c->page_size & (c->page_size - 1)))
    return fail(SPAX_ERR_SHAPE, "cache: page_size %d is not a power of two in 4..65536",
                c->page_size);
  if (c->n_pages < 1 || c->n_kv_heads < 1 || c->n_seqs < 1 || c->max_pages < 1)
    return fail(SPAX_ERR_SHAPE, "cache: n_pages %d, n_kv_heads %d, n_seqs %d and max_pages %d "
                "must be >= 1", c->n_pages, c->n_kv_heads, c->n_seqs, c->max_pages);
  if ((int64_t)c->max_pages * c->page_size > INT32_MAX)
    return fail(SPAX_ERR_SHAPE, "cache: max_pages * page_size exceeds 2^31 - 1");
  if (c->table_stride < c->max_pages && c->n_seqs > 1)
    return fail(SPAX_ERR_SHAPE, "cache: table_stride %lld < max_pages %d",
                (long long)c->table_stride, c->max_pages);
  if (!stride_range(c->n_seqs, c->table_stride))
    return fail(SPAX_ERR_PARAM, "cache: table_stride out of range");
  const int64_t unit = 16 / elem::bytes_of(c->type);
  const int64_t n[3] = {c->n_pages, c->n_kv_heads, c->page_size};
  const int64_t sk[3] = {c->k_page_stride, c->k_head_stride, c->k_row_stride};
  const int64_t sv[3] = {c->v_page_stride, c->v_head_stride, c->v_row_stride};
  for (int i = 0; i < 3; ++i) {
    if (!stride_range(n[i], sk[i]) || !stride_range(n[i], sv[i]))
      return fail(SPAX_ERR_PARAM, "cache: a stride is out of range");
    if (sk[i] % unit || sv[i] % unit)
      return fail(SPAX_ERR_ALIGN, "cache: strides must be multiples of 16 bytes");
  }
  if (!strides_ok(n, sk, 3, d) || !strides_ok(n, sv, 3, d))
    return fail(SPAX_ERR_PARAM, "cache: strides make its rows overlap");
  if (!aligned(c->k, 16) || !aligned(c->v, 16))
    return fail(SPAX_ERR_ALIGN, "cache: k and v must be 16-byte aligned");
  if (!aligned(c->page_table, 4) || !aligned(c->k_scale, 4) || !aligned(c->v_scale, 4))
    return fail(SPAX_ERR_ALIGN, "cache: page_table and scales must be 4-byte aligned");
  return SPAX_OK;
}

// Keys or values: p's pages from the first to the last byte of each.
Span pages_of(const spax_kv_cache* c, const void* p, int64_t page, int64_t head, int64_t row,
              bool out, const char* name) {
  const size_t eb = (size_t)elem::bytes_of(c->type);
  const int64_t n = (c->n_kv_heads - 1) * head + (c->page_size - 1) * row + c->head_dim;
  const bool many = c->n_pages > 1;
  return Span{p, (size_t)((c->n_pages - 1) * page + n) * eb, out, name,
              many ? (size_t)n * eb : 0, many ? (size_t)page * eb : 0};
}

// The cache's buffers (out: it is written).
void add_cache(const spax_kv_cache* c, bool out, Spans* b) {
  b->s[b->n++] = pages_of(c, c->k, c->k_page_stride, c->k_head_stride, c->k_row_stride, out,
                          "cache k");
  b->s[b->n++] = pages_of(c, c->v, c->v_page_stride, c->v_head_stride, c->v_row_stride, out,
                          "cache v");
  b->add(c->page_table, 4 * (size_t)((int64_t)(c->n_seqs - 1) * c->table_stride + c->max_pages),
         false, "page_table");
  b->add(c->k_scale, 4 * (size_t)c->n_kv_heads, false, "k_scale");
  b->add(c->v_scale, 4 * (size_t)c->n_kv_heads, false, "v_scale");
}

// Whether k and v, interleaved in one allocation so that their pages' spans meet, still have no
// row in common: with equal strides, the distance from one to the other is then the stride of one
// more axis, of length two.
bool rows_apart(const spax_kv_cache& c) {
  if (c.k_page_stride != c.v_page_stride || c.k_head_stride != c.v_head_stride ||
      c.k_row_stride != c.v_row_stride)
    return false;
  const uintptr_t k = (uintptr_t)c.k, v = (uintptr_t)c.v;
  const int64_t n[4] = {c.n_pages, c.n_kv_heads, c.page_size, 2};
  const int64_t s[4] = {c.k_page_stride, c.k_head_stride, c.k_row_stride,
                        (int64_t)((v > k ? v - k : k - v) / (size_t)elem::bytes_of(c.type))};
  return strides_ok(n, s, 4, c.head_dim);
}

int check_head_norm(const spax_head_norm& m, const spax_kv_append_args& a, int64_t d) {
  if (!m.q_weight && !m.k_weight && !m.q_bias && !m.k_bias)
    return fail(SPAX_ERR_NULL, "norm: q_weight or k_weight is required");
  if (m.kind != SPAX_NORM_RMS && m.kind != SPAX_NORM_LAYER)
    return fail(SPAX_ERR_UNSUPPORTED, "norm: kind %d", m.kind);
  if (!aligned(m.q_weight, 4) || !aligned(m.q_bias, 4) || !aligned(m.k_weight, 4) ||
      !aligned(m.k_bias, 4))
    return fail(SPAX_ERR_ALIGN, "norm: weights and biases must be 4-byte aligned");
  if (!std::isfinite(m.eps) || m.eps < 0.0f)
    return fail(SPAX_ERR_PARAM, "norm: eps must be finite and >= 0");
  if ((m.q_bias && !m.q_weight) || (m.k_bias && !m.k_weight))
    return fail(SPAX_ERR_PARAM, "norm: a bias needs its weight");
  if (m.q_weight && a.n_heads == 0)
    return fail(SPAX_ERR_PARAM, "norm: q_weight needs q");
  if ((m.q_weight && ((m.q_stride != 0 && m.q_stride < d) || !stride_range(a.n_heads, m.q_stride))) ||
      (m.k_weight &&
       ((m.k_stride != 0 && m.k_stride < d) || !stride_range(a.cache->n_kv_heads, m.k_stride))))
    return fail(SPAX_ERR_PARAM, "norm: a stride is neither 0 nor from %lld up, or out of range",
                (long long)d);
  return SPAX_OK;
}

// A workspace that an operator needs: there, aligned, large enough, apart from its buffers.
int check_workspace(const Spans& b, const void* ws, size_t ws_bytes, size_t need) {
  if (!need) return SPAX_OK;
  if (!ws) return fail(SPAX_ERR_NULL, "workspace is NULL");
  if (!aligned(ws, 256)) return fail(SPAX_ERR_ALIGN, "ws must be 256-byte aligned");
  if (ws_bytes < need)
    return fail(SPAX_ERR_WORKSPACE, "workspace %zu bytes < required %zu", ws_bytes, need);
  for (int i = 0; i < b.n; ++i)
    if (overlaps(ws, need, b.s[i].p, b.s[i].bytes))
      return fail(SPAX_ERR_PARAM, "the workspace overlaps %s", b.s[i].name);
  return SPAX_OK;
}

}  // namespace

bool shares(const Span& x, const Span& y) {
  if (!overlaps(x.p, x.bytes, y.p, y.bytes)) return false;
  if (!x.row || !y.row || x.step != y.step || x.row > x.step || y.row > x.step) return true;
  // where y's rows start within x's
  const size_t step = x.step;
  const uintptr_t px = (uintptr_t)x.p, py = (uintptr_t)y.p;
  const size_t at = py >= px ? (py - px) % step : (step - (px - py) % step) % step;
  return at < x.row || at + y.row > step;
}

int check_kv_append(const spax_kv_append_args* a, const spax_head_norm* m, Spans* spans) {
  if (!a) return fail(SPAX_ERR_NULL, "args is NULL");
  int st = check_cache(a->cache);
  if (st) return st;
  const spax_kv_cache& c = *a->cache;
  const bool some = a->n_tokens != 0;
  if (some && (!a->k || !a->v || !a->positions))
    return fail(SPAX_ERR_NULL, "k, v and positions are required");
  if (some &&
      ((a->n_heads > 0) != (a->q != nullptr) || (a->n_heads > 0) != (a->q_out != nullptr)))
    return fail(SPAX_ERR_NULL, "q and q_out are required with n_heads > 0, and NULL without");
  if (!is_float_type(a->src_type))
    return fail(SPAX_ERR_UNSUPPORTED, "src_type %d", a->src_type);
  if (a->out_type != SPAX_F16 && a->out_type != SPAX_BF16)
    return fail(SPAX_ERR_UNSUPPORTED, "out_type %d", a->out_type);
  if (c.type != a->out_type && c.type != SPAX_E4M3)
    return fail(SPAX_ERR_UNSUPPORTED, "out_type %d with a cache of type %d", a->out_type, c.type);
  if (a->n_tokens < 0 || a->n_heads < 0)
    return fail(SPAX_ERR_SHAPE, "n_tokens %d and n_heads %d must be >= 0", a->n_tokens,
                a->n_heads);
  if (!a->seq && a->n_tokens > c.n_seqs)
    return fail(SPAX_ERR_SHAPE, "%d tokens of %d sequences need seq", a->n_tokens, c.n_seqs);
  if (a->rot_dim < 0 || a->rot_dim > c.head_dim || a->rot_dim % 2)
    return fail(SPAX_ERR_SHAPE, "rot_dim %d is not an even number in 0..%d", a->rot_dim,
                c.head_dim);
  if (a->rot_dim > 0 && !a->inv_freq) return fail(SPAX_ERR_NULL, "inv_freq is required");
  const int64_t heads = (int64_t)a->n_heads + 2 * (int64_t)c.n_kv_heads;
  if (heads > 65535 || a->n_tokens >= 1 << 24)  // a grid holds 2^32 threads
    return fail(SPAX_ERR_SHAPE, "%lld heads or %d tokens are too many", (long long)heads,
                a->n_tokens);
  const size_t sb = (size_t)elem::bytes_of(a->src_type);
  if (!aligned(a->q, sb) || !aligned(a->k, sb) || !aligned(a->v, sb) || !aligned(a->q_out, 2) ||
      !aligned(a->positions, 4) || !aligned(a->seq, 4) || !aligned(a->inv_freq, 4))
    return fail(SPAX_ERR_ALIGN, "a pointer is not aligned to its element");
  const int64_t n = a->n_tokens, d = c.head_dim;
  if (m && (st = check_head_norm(*m, *a, d))) return st;
  if ((st = check_rows2("q", n, a->q_token_stride, a->n_heads, a->q_head_stride, d, false)) ||
      (st = check_rows2("k", n, a->k_token_stride, c.n_kv_heads, a->k_head_stride, d, false)) ||
      (st = check_rows2("v", n, a->v_token_stride, c.n_kv_heads, a->v_head_stride, d, false)) ||
      (st = check_rows2("q_out", n, a->out_token_stride, a->n_heads, a->out_head_stride, d,
                        true)))
    return st;
  Spans b;
  if (n > 0) {
    add_rows(&b, a->q, n, a->q_token_stride, a->n_heads, a->q_head_stride, d, a->src_type, false,
             "q");
    add_rows(&b, a->k, n, a->k_token_stride, c.n_kv_heads, a->k_head_stride, d, a->src_type,
             false, "k");
    add_rows(&b, a->v, n, a->v_token_stride, c.n_kv_heads, a->v_head_stride, d, a->src_type,
             false, "v");
    add_rows(&b, a->q_out, n, a->out_token_stride, a->n_heads, a->out_head_stride, d, a->out_type,
             true, "q_out");
    b.add(a->positions, 4 * (size_t)n, false, "positions");
    b.add(a->seq, 4 * (size_t)n, false, "seq");
    b.add(a->inv_freq, 2 * (size_t)a->rot_dim, false, "inv_freq");
    add_cache(&c, true, &b);
    if (m) {
      const int64_t nq = m->q_stride ? a->n_heads : 1, nk = m->k_stride ? c.n_kv_heads : 1;
      add_rows(&b, m->q_weight, nq, m->q_stride, 1, 0, d, SPAX_F32, false, "q_weight");
      add_rows(&b, m->q_bias, nq, m->q_stride, 1, 0, d, SPAX_F32, false, "q_bias");
      add_rows(&b, m->k_weight, nk, m->k_stride, 1, 0, d, SPAX_F32, false, "k_weight");
      add_rows(&b, m->k_bias, nk, m->k_stride, 1, 0, d, SPAX_F32, false, "k_bias");
    }
  }
  // q may be rotated in place: a thread reads its values of a head, and a head's threads have all
  // read theirs where it is normed, before any is written
  const bool in_place = a->q == a->q_out && a->src_type == a->out_type &&
                        a->q_token_stride == a->out_token_stride &&
                        a->q_head_stride == a->out_head_stride;
  st = check_overlaps(b, [&](const Span& x, const Span& y) {
    if (is(x, "q_out") && is(y, "q")) return in_place;
    return is(x, "cache k") && is(y, "cache v") && rows_apart(c);
  });
  if (st) return st;
  if (spans) *spans = b;
  return SPAX_OK;
}

int check_attention(const spax_attention_args* a, Spans* spans) {
  if (!a) return fail(SPAX_ERR_NULL, "args is NULL");
  int st = check_cache(a->cache);
  if (st) return st;
  const spax_kv_cache& c = *a->cache;
  if (!a->q || !a->out || !a->lens) return fail(SPAX_ERR_NULL, "q, out and lens are required");
  if (a->type != SPAX_F16 && a->type != SPAX_BF16)
    return fail(SPAX_ERR_UNSUPPORTED, "type %d", a->type);
  if (c.type != a->type && c.type != SPAX_E4M3)
    return fail(SPAX_ERR_UNSUPPORTED, "type %d with a cache of type %d", a->type, c.type);
  if (a->n_heads < 1 || a->n_heads % c.n_kv_heads)
    return fail(SPAX_ERR_SHAPE, "n_heads %d is not a multiple of n_kv_heads %d", a->n_heads,
                c.n_kv_heads);
  if (a->max_len < 1 || a->max_len > (int64_t)c.max_pages * c.page_size)
    return fail(SPAX_ERR_SHAPE, "max_len %d outside 1..%lld", a->max_len,
                (long long)c.max_pages * c.page_size);
  if (a->window < 0) return fail(SPAX_ERR_SHAPE, "window %d < 0", a->window);
  if (!std::isfinite(a->scale)) return fail(SPAX_ERR_PARAM, "scale is not finite");
  if (!aligned(a->q, 16) || !aligned(a->out, 16) || a->q_seq_stride % 8 || a->q_head_stride % 8 ||
      a->out_seq_stride % 8 || a->out_head_stride % 8)
    return fail(SPAX_ERR_ALIGN, "q and out must be 16-byte aligned, their strides multiples of 8");
  if (!aligned(a->lens, 4) || !aligned(a->lse, 4))
    return fail(SPAX_ERR_ALIGN, "lens and lse must be 4-byte aligned");
  const int64_t n = c.n_seqs, d = c.head_dim;
  if ((st = check_rows2("q", n, a->q_seq_stride, a->n_heads, a->q_head_stride, d, false)) ||
      (st = check_rows2("out", n, a->out_seq_stride, a->n_heads, a->out_head_stride, d, true)))
    return st;
  if (a->n_heads > 65535 || a->max_len > (1 << 30) || attention_plan(a).units > (1 << 30))
    return fail(SPAX_ERR_SHAPE, "%d heads, or %d sequences of %d keys, are too many", a->n_heads,
                c.n_seqs, a->max_len);
  Spans b;
  add_rows(&b, a->q, n, a->q_seq_stride, a->n_heads, a->q_head_stride, d, a->type, false, "q");
  add_rows(&b, a->out, n, a->out_seq_stride, a->n_heads, a->out_head_stride, d, a->type, true,
           "out");
  b.add(a->lse, 4 * (size_t)n * (size_t)a->n_heads, true, "lse");
  b.add(a->lens, 4 * (size_t)n, false, "lens");
  add_cache(&c, false, &b);
  if ((st = check_overlaps(b, [](const Span&, const Span&) { return false; }))) return st;
  if (spans) *spans = b;
  return SPAX_OK;
}

int check_residual_norm(const spax_residual_norm_args* a, Spans* spans) {
  if (!a) return fail(SPAX_ERR_NULL, "args is NULL");
  const bool some = a->n_rows != 0;
  if (some && !a->residual && !a->block)
    return fail(SPAX_ERR_NULL, "residual or block is required");
  if (some && !a->residual_out && !a->x)
    return fail(SPAX_ERR_NULL, "residual_out or x is required");
  if (!is_float_type(a->residual_type) || !is_float_type(a->x_type) ||
      (a->block && !is_float_type(a->block_type)) || (a->gate && !is_float_type(a->gate_type)))
    return fail(SPAX_ERR_UNSUPPORTED, "types %d, %d, %d, %d", a->residual_type, a->block_type,
                a->gate_type, a->x_type);
  if (a->kind != SPAX_NORM_RMS && a->kind != SPAX_NORM_LAYER)
    return fail(SPAX_ERR_UNSUPPORTED, "kind %d", a->kind);
  if (a->n_rows < 0) return fail(SPAX_ERR_SHAPE, "n_rows %d < 0", a->n_rows);
  if (a->d < 1 || a->d > SPAX_MAX_DIN)
    return fail(SPAX_ERR_SHAPE, "d %d outside 1..%d", a->d, SPAX_MAX_DIN);
  if ((int64_t)a->n_rows * ((a->d + 7) / 8 + 63) >= (int64_t)1 << 32)  // a grid holds 2^32 threads
    return fail(SPAX_ERR_SHAPE, "%d rows of %d are too many", a->n_rows, a->d);
  if (!std::isfinite(a->scale) || !std::isfinite(a->eps) || a->eps < 0.0f)
    return fail(SPAX_ERR_PARAM, "scale and eps must be finite and eps >= 0");
  if ((a->post_bias && !a->post_weight) || (a->pre_bias && !a->pre_weight))
    return fail(SPAX_ERR_PARAM, "a bias needs its weight");
  if (some && !a->block && (a->gate || a->post_weight))
    return fail(SPAX_ERR_PARAM, "gate and post_weight need block");
  const size_t rb = (size_t)elem::bytes_of(a->residual_type);
  if (!aligned(a->residual, rb) || !aligned(a->residual_out, rb) ||
      !aligned(a->block, a->block ? (size_t)elem::bytes_of(a->block_type) : 1) ||
      !aligned(a->gate, a->gate ? (size_t)elem::bytes_of(a->gate_type) : 1) ||
      !aligned(a->x, (size_t)elem::bytes_of(a->x_type)) || !aligned(a->post_weight, 4) ||
      !aligned(a->post_bias, 4) || !aligned(a->pre_weight, 4) || !aligned(a->pre_bias, 4))
    return fail(SPAX_ERR_ALIGN, "a pointer is not aligned to its element");
  const int64_t n = a->n_rows, d = a->d;
  const struct {
    const void* p;
    int64_t stride;
    const char* name;
    bool broadcast;
  } rows[] = {{a->residual, a->residual_stride, "residual", false},
              {a->block, a->block_stride, "block", false},
              {a->residual_out, a->residual_out_stride, "residual_out", false},
              {a->x, a->x_stride, "x", false},
              {a->gate, a->gate_stride, "gate", true}};
  for (const auto& r : rows)
    if (r.p && n > 1 && (!stride_range(n, r.stride) || (r.stride < d && !(r.broadcast && !r.stride))))
      return fail(SPAX_ERR_PARAM, "%s: stride %lld is below d %d or out of range", r.name,
                  (long long)r.stride, a->d);
  Spans b;
  if (n > 0) {
    add_rows(&b, a->residual, n, a->residual_stride, 1, 0, d, a->residual_type, false,
             "residual");
    add_rows(&b, a->block, n, a->block_stride, 1, 0, d, a->block_type, false, "block");
    add_rows(&b, a->gate, n, a->gate_stride, 1, 0, d, a->gate_type, false, "gate");
    add_rows(&b, a->residual_out, n, a->residual_out_stride, 1, 0, d, a->residual_type, true,
             "residual_out");
    add_rows(&b, a->x, n, a->x_stride, 1, 0, d, a->x_type, true, "x");
    b.add(a->post_weight, 4 * (size_t)d, false, "post_weight");
    b.add(a->post_bias, 4 * (size_t)d, false, "post_bias");
    b.add(a->pre_weight, 4 * (size_t)d, false, "pre_weight");
    b.add(a->pre_bias, 4 * (size_t)d, false, "pre_bias");
  }
  // the stream updated in place, x in place of block (value for value: a row is read whole
  // before it is written)
  const bool stream = a->residual && a->residual == a->residual_out &&
                      (n == 1 || a->residual_stride == a->residual_out_stride);
  const bool over = a->block && a->block == a->x && a->block_type == a->x_type &&
                    (n == 1 || a->block_stride == a->x_stride);
  const int st = check_overlaps(b, [&](const Span& x, const Span& y) {
    return (stream && is(x, "residual_out") && is(y, "residual")) ||
           (over && is(x, "x") && is(y, "block"));
  });
  if (st) return st;
  if (spans) *spans = b;
  return SPAX_OK;
}

int check_glu(const spax_glu_args* a, Spans* spans) {
  if (!a) return fail(SPAX_ERR_NULL, "args is NULL");
  if (a->n_rows != 0 && (!a->gate || !a->up || !a->x))
    return fail(SPAX_ERR_NULL, "gate, up and x are required");
  if (!is_float_type(a->src_type) || !is_float_type(a->x_type))
    return fail(SPAX_ERR_UNSUPPORTED, "types %d, %d", a->src_type, a->x_type);
  if (a->act != SPAX_ACT_SILU && a->act != SPAX_ACT_GELU_TANH)
    return fail(SPAX_ERR_UNSUPPORTED, "act %d", a->act);
  if (a->n_rows < 0 || a->d < 1 || a->d > (1 << 30))
    return fail(SPAX_ERR_SHAPE, "n_rows %d must be >= 0 and d %d in 1..2^30", a->n_rows, a->d);
  if ((int64_t)a->n_rows * (((int64_t)a->d + 2047) / 2048) >= 1 << 24)  // workgroups of 256
    return fail(SPAX_ERR_SHAPE, "%d rows of %d are too many", a->n_rows, a->d);
  const size_t sb = (size_t)elem::bytes_of(a->src_type);
  if (!aligned(a->gate, sb) || !aligned(a->up, sb) ||
      !aligned(a->x, (size_t)elem::bytes_of(a->x_type)))
    return fail(SPAX_ERR_ALIGN, "a pointer is not aligned to its element");
  const int64_t n = a->n_rows, d = a->d;
  if (n > 1 && (a->gate_stride < d || a->up_stride < d || a->x_stride < d ||
                !stride_range(n, a->gate_stride) || !stride_range(n, a->up_stride) ||
                !stride_range(n, a->x_stride)))
    return fail(SPAX_ERR_PARAM, "a stride is below d or out of range");
  Spans b;
  if (n > 0) {
    add_rows(&b, a->gate, n, a->gate_stride, 1, 0, d, a->src_type, false, "gate");
    add_rows(&b, a->up, n, a->up_stride, 1, 0, d, a->src_type, false, "up");
    add_rows(&b, a->x, n, a->x_stride, 1, 0, d, a->x_type, true, "x");
  }
  // x in place of gate or up: a thread reads its own values of both before it writes
  const bool same = a->src_type == a->x_type;
  const bool on_gate = same && a->x == a->gate && (n == 1 || a->x_stride == a->gate_stride);
  const bool on_up = same && a->x == a->up && (n == 1 || a->x_stride == a->up_stride);
  const int st = check_overlaps(b, [&](const Span&, const Span& y) {
    return is(y, "gate") ? on_gate : on_up;
  });
  if (st) return st;
  if (spans) *spans = b;
  return SPAX_OK;
}

int check_chunk_attention(const spax_chunk_attention_args* a, Spans* spans) {
  if (!a) return fail(SPAX_ERR_NULL, "args is NULL");
  int st = check_cache(a->cache);
  if (st) return st;
  const spax_kv_cache& c = *a->cache;
  if (a->n_tokens != 0 && (!a->q || !a->out || !a->starts || !a->lens))
    return fail(SPAX_ERR_NULL, "q, out, starts and lens are required");
  if (a->type != SPAX_F16 && a->type != SPAX_BF16)
    return fail(SPAX_ERR_UNSUPPORTED, "type %d", a->type);
  if (c.type != a->type && c.type != SPAX_E4M3)
    return fail(SPAX_ERR_UNSUPPORTED, "type %d with a cache of type %d", a->type, c.type);
  if (a->n_heads < 1 || a->n_heads > 65535 || a->n_heads % c.n_kv_heads)
    return fail(SPAX_ERR_SHAPE, "n_heads %d is not a multiple of n_kv_heads %d in 1..65535",
                a->n_heads, c.n_kv_heads);
  if (a->n_tokens < 0 || (int64_t)a->n_tokens * a->n_heads > (1 << 30))
    return fail(SPAX_ERR_SHAPE, "n_tokens %d of %d heads outside 0..2^30 rows", a->n_tokens,
                a->n_heads);
  if (a->max_len < 1 || a->max_len > (int64_t)c.max_pages * c.page_size || a->max_len > (1 << 30))
    return fail(SPAX_ERR_SHAPE, "max_len %d outside 1..%lld", a->max_len,
                (long long)c.max_pages * c.page_size);
  if (a->window < 0) return fail(SPAX_ERR_SHAPE, "window %d < 0", a->window);
  if (!std::isfinite(a->scale)) return fail(SPAX_ERR_PARAM, "scale is not finite");
  if (!aligned(a->q, 16) || !aligned(a->out, 16) || a->q_token_stride % 8 ||
      a->q_head_stride % 8 || a->out_token_stride % 8 || a->out_head_stride % 8)
    return fail(SPAX_ERR_ALIGN, "q and out must be 16-byte aligned, their strides multiples of 8");
  if (!aligned(a->lens, 4) || !aligned(a->starts, 4) || !aligned(a->lse, 4))
    return fail(SPAX_ERR_ALIGN, "starts, lens and lse must be 4-byte aligned");
  const int64_t n = a->n_tokens, d = c.head_dim;
  if ((st = check_rows2("q", n, a->q_token_stride, a->n_heads, a->q_head_stride, d, false)) ||
      (st = check_rows2("out", n, a->out_token_stride, a->n_heads, a->out_head_stride, d, true)))
    return st;
  if (chunk_plan(a).blocks >= 1 << 23)  // a grid holds 2^32 threads
    return fail(SPAX_ERR_SHAPE, "%d tokens of %d sequences are too many", a->n_tokens, c.n_seqs);
  Spans b;
  if (n > 0) {
    add_rows(&b, a->q, n, a->q_token_stride, a->n_heads, a->q_head_stride, d, a->type, false, "q");
    add_rows(&b, a->out, n, a->out_token_stride, a->n_heads, a->out_head_stride, d, a->type, true,
             "out");
    b.add(a->lse, 4 * (size_t)n * (size_t)a->n_heads, true, "lse");
    b.add(a->starts, 4 * ((size_t)c.n_seqs + 1), false, "starts");
    b.add(a->lens, 4 * (size_t)c.n_seqs, false, "lens");
    add_cache(&c, false, &b);
  }
  if ((st = check_overlaps(b, [](const Span&, const Span&) { return false; }))) return st;
  if (spans) *spans = b;
  return SPAX_OK;
}

int check_packed_gemm(const spax_packed_gemm_args* a, Spans* spans) {
  if (!a || !a->layout) return fail(SPAX_ERR_NULL, "args or layout is NULL");
  const spax_layout& L = *a->layout;
  if (!layout_ok(&L)) return fail(SPAX_ERR_SHAPE, "layout is not initialised");
  if (a->n_rows != 0 && (!a->packed || !a->x || !a->y))
    return fail(SPAX_ERR_NULL, "packed, x and y are required");
  if (a->form < SPAX_GEMM_PLAIN || a->form > SPAX_GEMM_GATED)
    return fail(SPAX_ERR_UNSUPPORTED, "form %d", a->form);
  if (a->form != SPAX_GEMM_PLAIN && a->act != SPAX_ACT_SILU && a->act != SPAX_ACT_GELU_TANH)
    return fail(SPAX_ERR_UNSUPPORTED, "act %d", a->act);
  if (!is_float_type(a->y_type) || (a->residual && !is_float_type(a->residual_type)))
    return fail(SPAX_ERR_UNSUPPORTED, "types %d, %d", a->residual_type, a->y_type);
  const bool gated = a->form == SPAX_GEMM_GATED;
  if (gated && (L.n_mats != 2 || L.d_out[0] != L.d_out[1]))
    return fail(SPAX_ERR_SHAPE, "GATED needs two matrices of equal d_out");
  if (a->n_rows < 0 || a->n_rows >= 1 << 20)
    return fail(SPAX_ERR_SHAPE, "n_rows %d outside 0..2^20 - 1", a->n_rows);
  if (!std::isfinite(a->scale)) return fail(SPAX_ERR_PARAM, "scale is not finite");
  if (!aligned(a->packed, 256)) return fail(SPAX_ERR_ALIGN, "packed must be 256-byte aligned");
  if (!aligned(a->x, 16) || (a->n_rows > 1 && a->x_stride % 8))
    return fail(SPAX_ERR_ALIGN, "x must be 16-byte aligned, its stride a multiple of 8");
  if (!aligned(a->bias, 4) || !aligned(a->y, (size_t)elem::bytes_of(a->y_type)) ||
      !aligned(a->residual, a->residual ? (size_t)elem::bytes_of(a->residual_type) : 1))
    return fail(SPAX_ERR_ALIGN, "a pointer is not aligned to its element");
  const int64_t n = a->n_rows, d = gated ? L.d_out[0] : L.d_out_total;
  if (n > 1 && (a->x_stride < L.d_in || a->y_stride < d || !stride_range(n, a->x_stride) ||
                !stride_range(n, a->y_stride) ||
                (a->residual && (a->residual_stride < d || !stride_range(n, a->residual_stride)))))
    return fail(SPAX_ERR_PARAM, "a stride is below its row or out of range");
  if (gemm_plan(a).blocks >= 1 << 22)  // a grid holds 2^32 threads
    return fail(SPAX_ERR_SHAPE, "%d rows of %lld columns are too many", a->n_rows,
                (long long)L.d_out_total);
  Spans b;
  if (n > 0) {
    b.add(a->packed, (size_t)L.total_bytes, false, "packed");
    add_rows(&b, a->x, n, a->x_stride, 1, 0, L.d_in, SPAX_F16, false, "x");
    b.add(a->bias, 4 * (size_t)L.d_out_total, false, "bias");
    if (a->residual)
      add_rows(&b, a->residual, n, a->residual_stride, 1, 0, d, a->residual_type, false,
               "residual");
    add_rows(&b, a->y, n, a->y_stride, 1, 0, d, a->y_type, true, "y");
  }
  // the stream updated in place: a thread reads its own values before it writes them
  const bool stream = a->residual == a->y && a->residual_type == a->y_type &&
                      (n == 1 || a->residual_stride == a->y_stride);
  const int st =
      check_overlaps(b, [&](const Span&, const Span& y) { return stream && is(y, "residual"); });
  if (st) return st;
  if (spans) *spans = b;
  return SPAX_OK;
}

}  // namespace spax

extern "C" {

int spax_kv_append(const spax_kv_append_args* a, hipStream_t stream) {
  clear_error();
  const int st = check_kv_append(a, nullptr, nullptr);
  return st ? st : launch_kv_append(a, nullptr, stream);
}

int spax_kv_append_normed(const spax_kv_append_args* a, const spax_head_norm* norm,
                          hipStream_t stream) {
  clear_error();
  if (!norm) return fail(SPAX_ERR_NULL, "norm is NULL");
  const int st = check_kv_append(a, norm, nullptr);
  return st ? st : launch_kv_append(a, norm, stream);
}

size_t spax_attention_workspace_bytes(const spax_attention_args* a) {
  if (check_attention(a, nullptr)) {
    clear_error();
    return 0;
  }
  return attention_plan(a).ws_bytes;
}

int spax_paged_attention(const spax_attention_args* a, void* ws, size_t ws_bytes,
                         hipStream_t stream) {
  clear_error();
  Spans b;
  const int st = check_attention(a, &b);
  if (st) return st;
  const int bad = check_workspace(b, ws, ws_bytes, attention_plan(a).ws_bytes);
  return bad ? bad : launch_attention(a, ws, stream);
}

int spax_residual_norm(const spax_residual_norm_args* a, hipStream_t stream) {
  clear_error();
  const int st = check_residual_norm(a, nullptr);
  return st ? st : launch_residual_norm(a, stream);
}

int spax_glu(const spax_glu_args* a, hipStream_t stream) {
  clear_error();
  const int st = check_glu(a, nullptr);
  return st ? st : launch_glu(a, stream);
}

size_t spax_chunk_attention_workspace_bytes(const spax_chunk_attention_args* a) {
  if (check_chunk_attention(a, nullptr)) {
    clear_error();
    return 0;
  }
  return chunk_plan(a).ws_bytes;
}

int spax_chunk_attention(const spax_chunk_attention_args* a, void* ws, size_t ws_bytes,
                         hipStream_t stream) {
  clear_error();
  Spans b;
  int st = check_chunk_attention(a, &b);
  if (st) return st;
  st = check_workspace(b, ws, ws_bytes, chunk_plan(a).ws_bytes);
  return st ? st : launch_chunk_attention(a, ws, stream);
}

size_t spax_packed_gemm_workspace_bytes(const spax_packed_gemm_args* a) {
  if (check_packed_gemm(a, nullptr)) {
    clear_error();
    return 0;
  }
  return gemm_plan(a).ws_bytes;
}

int spax_packed_gemm(const spax_packed_gemm_args* a, void* ws, size_t ws_bytes,
                     hipStream_t stream) {
  clear_error();
  Spans b;
  int st = check_packed_gemm(a, &b);
  if (st) return st;
  st = check_workspace(b, ws, ws_bytes, gemm_plan(a).ws_bytes);
  return st ? st : launch_packed_gemm(a, ws, stream);
}

}  // extern "C"
