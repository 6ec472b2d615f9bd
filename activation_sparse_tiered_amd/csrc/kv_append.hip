// spax_kv_append: keys and values of new tokens into the paged cache, rotated on the way.
//
// For a pair (x, y) of a head at position p with frequency f:
//   a = p f,   (x, y) -> (x cos a - y sin a, x sin a + y cos a).
// p f reaches 1e6 radians, where a 32-bit angle is off by 0.06, so the turns p f / 2 pi and their
// fraction are 64-bit; the fraction, in [-1/2, 1/2], is then exact enough in 32 bits (2^-25 of a
// turn) for sine and cosine.
//
// Bound: bytes (each value is read once and written once) for prompts, launch latency for one
// token.  A thread keeps one place in the head (four pairs, or eight copied values) and walks
// over heads, so a token's sines are computed once per workgroup and live in registers.
#include "layer_ops.h"

namespace spax {
namespace {

using namespace elem;

constexpr int kAppendThreads = 256;

struct AppendArgs {
  const void *q, *k, *v;
  void* q_out;
  void *kc, *vc;
  const int32_t *positions, *seq, *table;
  const float *inv_freq, *k_scale, *v_scale;
  int64_t qt, qh, kt, kh, vt, vh, ot, oh;
  int64_t kc_page, kc_head, kc_row, vc_page, vc_head, vc_row, table_stride;
  int32_t n_heads, n_kv, dim, rot, interleaved, n_seqs, n_pages, max_pages, page_shift;
  int32_t heads_at_once, heads_per_block;
};

// Where token t's rows go: the row of key head 0, or -1.
struct Place {
  int64_t k, v;
  bool cached;
};
__device__ inline Place place_of(const AppendArgs& a, int t, int p) {
  Place w{0, 0, false};
  const int s = a.seq ? a.seq[t] : t;
  const int pg = p >> a.page_shift;
  if (p < 0 || (uint32_t)s >= (uint32_t)a.n_seqs || pg >= a.max_pages) return w;
  const int page = a.table[(int64_t)s * a.table_stride + pg];
  if ((uint32_t)page >= (uint32_t)a.n_pages) return w;
  const int row = p & ((1 << a.page_shift) - 1);
  w.k = (int64_t)page * a.kc_page + (int64_t)row * a.kc_row;
  w.v = (int64_t)page * a.vc_page + (int64_t)row * a.vc_row;
  w.cached = true;
  return w;
}

__device__ inline void sine(int p, float inv_freq, float* sn, float* cs) {
  constexpr double kTurn = 0.15915494309189533577;  // 1 / (2 pi)
  const double turns = (double)p * (double)inv_freq * kTurn;
  sincospif(2.0f * (float)(turns - rint(turns)), sn, cs);
}

// SRC: type of q, k, v; LOW: of q_out (and a 16-bit cache); C: of the cache.  VEC: eight values
// per thread and head (rot a multiple of 8, rows aligned to four elements); otherwise one pair
// or one copied value.
template <class SRC, class LOW, class C, bool VEC>
__global__ __launch_bounds__(kAppendThreads) void kv_append_kernel(AppendArgs a) {
  constexpr int N = VEC ? 4 : 1;  // pairs per item
  const int t = blockIdx.x;
  const int pairs = a.rot / 2;
  // items of a head: pairs / N rotated ones, then the copied values
  const int turned = pairs / N;
  const int items = turned + (a.dim - a.rot) / (VEC ? 8 : 1);
  const int slot = threadIdx.x / items;
  const int j = threadIdx.x - slot * items;
  if (slot >= a.heads_at_once) return;
  const int p = a.positions[t];
  const Place to = place_of(a, t, p);
  const bool turns = j < turned;
  // element offsets of the item's first and second values
  int e0, e1;
  if (turns) {
    e0 = a.interleaved ? 2 * N * j : N * j;
    e1 = a.interleaved ? e0 + N : pairs + N * j;
  } else {
    e0 = a.rot + (j - turned) * (VEC ? 8 : 1);
    e1 = e0 + N;
  }
  const bool single = !VEC && !turns;  // one value, no second
  float sn[N], cs[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    sn[i] = 0.0f;
    cs[i] = 1.0f;
    if (turns && p >= 0) sine(p, a.inv_freq[N * j + i], &sn[i], &cs[i]);
  }
  const int n_heads = a.n_heads, n_kv = a.n_kv;
  const int h0 = blockIdx.y * a.heads_per_block;
  const int total = n_heads + 2 * n_kv;
  const int h1 = h0 + a.heads_per_block < total ? h0 + a.heads_per_block : total;
  for (int h = h0 + slot; h < h1; h += a.heads_at_once) {
    const bool is_q = h < n_heads, is_v = h >= n_heads + n_kv;
    const int hh = is_q ? h : is_v ? h - n_heads - n_kv : h - n_heads;
    if (!is_q && !to.cached) continue;
    const SRC* src = is_q   ? (const SRC*)a.q + t * a.qt + hh * a.qh
                     : is_v ? (const SRC*)a.v + t * a.vt + hh * a.vh
                            : (const SRC*)a.k + t * a.kt + hh * a.kh;
    float x[N], y[N];
    if constexpr (VEC) {
      load4(src + e0, x);
      load4(src + e1, y);
    } else {
      x[0] = (float)src[e0];
      y[0] = single ? 0.0f : (float)src[e1];
    }
    if (turns && !is_v) {
      float u[N], w[N];
#pragma unroll
      for (int i = 0; i < N; ++i) {
        // neighbours: the loaded values alternate between first and second of a pair
        float px, py;
        if (VEC && a.interleaved) {
          px = i < 2 ? x[2 * i % N] : y[(2 * i) % N];
          py = i < 2 ? x[(2 * i + 1) % N] : y[(2 * i + 1) % N];
        } else {
          px = x[i];
          py = y[i];
        }
        u[i] = px * cs[i] - py * sn[i];
        w[i] = px * sn[i] + py * cs[i];
      }
      if (VEC && a.interleaved) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const float f = i % 2 ? w[i / 2] : u[i / 2];
          const float g = i % 2 ? w[(N + i) / 2 % N] : u[(N + i) / 2 % N];
          x[i] = f;
          y[i] = g;
        }
      } else {
#pragma unroll
        for (int i = 0; i < N; ++i) {
          x[i] = u[i];
          y[i] = w[i];
        }
      }
    }
    if (is_q) {
      LOW* dst = (LOW*)a.q_out + t * a.ot + hh * a.oh;
      if (p < 0) {
#pragma unroll
        for (int i = 0; i < N; ++i) x[i] = y[i] = 0.0f;
      }
      if constexpr (VEC) {
        store4(dst + e0, x);
        store4(dst + e1, y);
      } else {
        store1(dst + e0, x[0]);
        if (!single) store1(dst + e1, y[0]);
      }
    } else {
      C* dst = is_v ? (C*)a.vc + to.v + hh * a.vc_head : (C*)a.kc + to.k + hh * a.kc_head;
      if constexpr (sizeof(C) == 1) {
        const float* scale = is_v ? a.v_scale : a.k_scale;
        if (scale) {
          const float f = scale[hh];
#pragma unroll
          for (int i = 0; i < N; ++i) {
            x[i] = x[i] / f;
            y[i] = y[i] / f;
          }
        }
      }
      if constexpr (VEC) {
        store4(dst + e0, x);
        store4(dst + e1, y);
      } else {
        store1(dst + e0, x[0]);
        if (!single) store1(dst + e1, y[0]);
      }
    }
  }
}

template <class SRC, class LOW, class C>
int launch(const AppendArgs& a, dim3 grid, bool vec, hipStream_t s) {
  if (vec)
    hipLaunchKernelGGL((kv_append_kernel<SRC, LOW, C, true>), grid, dim3(kAppendThreads), 0, s, a);
  else
    hipLaunchKernelGGL((kv_append_kernel<SRC, LOW, C, false>), grid, dim3(kAppendThreads), 0, s,
                       a);
  SPAX_HIP_CHECK(hipGetLastError());
  return SPAX_OK;
}

template <class SRC>
int launch_src(const AppendArgs& a, int out_type, bool narrow, dim3 grid, bool vec,
               hipStream_t s) {
  if (out_type == SPAX_F16)
    return narrow ? launch<SRC, f16, e4m3>(a, grid, vec, s) : launch<SRC, f16, f16>(a, grid, vec, s);
  return narrow ? launch<SRC, bf16, e4m3>(a, grid, vec, s)
                : launch<SRC, bf16, bf16>(a, grid, vec, s);
}

}  // namespace

int launch_kv_append(const spax_kv_append_args* p, hipStream_t s) {
  if (p->n_tokens == 0) return SPAX_OK;
  const spax_kv_cache& c = *p->cache;
  AppendArgs a{};
  a.q = p->q; a.k = p->k; a.v = p->v; a.q_out = p->q_out; a.kc = c.k; a.vc = c.v;
  a.positions = p->positions; a.seq = p->seq; a.table = c.page_table;
  a.inv_freq = p->inv_freq; a.k_scale = c.k_scale; a.v_scale = c.v_scale;
  a.qt = p->q_token_stride; a.qh = p->q_head_stride;
  a.kt = p->k_token_stride; a.kh = p->k_head_stride;
  a.vt = p->v_token_stride; a.vh = p->v_head_stride;
  a.ot = p->out_token_stride; a.oh = p->out_head_stride;
  a.kc_page = c.k_page_stride; a.kc_head = c.k_head_stride; a.kc_row = c.k_row_stride;
  a.vc_page = c.v_page_stride; a.vc_head = c.v_head_stride; a.vc_row = c.v_row_stride;
  a.table_stride = c.table_stride;
  a.n_heads = p->n_heads; a.n_kv = c.n_kv_heads; a.dim = c.head_dim; a.rot = p->rot_dim;
  a.interleaved = p->interleaved != 0;
  a.n_seqs = c.n_seqs; a.n_pages = c.n_pages; a.max_pages = c.max_pages;
  a.page_shift = __builtin_ctz((unsigned)c.page_size);
  // Four values at a time where every row starts on four elements (the cache's always do).
  const size_t eb = 4 * (size_t)bytes_of(p->src_type);
  bool vec = p->rot_dim % 8 == 0 && aligned(p->k, eb) && aligned(p->v, eb) &&
             (a.kt | a.kh | a.vt | a.vh) % 4 == 0;
  if (p->n_heads)
    vec = vec && aligned(p->q, eb) && aligned(p->q_out, 8) && (a.qt | a.qh | a.ot | a.oh) % 4 == 0;
  const int items = vec ? a.dim / 8 : p->rot_dim / 2 + a.dim - p->rot_dim;
  a.heads_at_once = kAppendThreads / items;
  // One round of heads per workgroup while that keeps few of them: latency is then one load and
  // one store deep.  With many tokens a workgroup walks over all heads of its token.
  const int total = a.n_heads + 2 * a.n_kv;
  a.heads_per_block = p->n_tokens < 512 ? a.heads_at_once : total;
  const dim3 grid((unsigned)p->n_tokens,
                  (unsigned)((total + a.heads_per_block - 1) / a.heads_per_block));
  const bool narrow = c.type == SPAX_E4M3;
  switch (p->src_type) {
    case SPAX_F32: return launch_src<float>(a, p->out_type, narrow, grid, vec, s);
    case SPAX_F16: return launch_src<f16>(a, p->out_type, narrow, grid, vec, s);
    default: return launch_src<bf16>(a, p->out_type, narrow, grid, vec, s);
  }
}

}  // namespace spax
