// spax_kv_append, spax_kv_append_normed: keys and values of new tokens into the paged cache, rotated
// on the way, their heads and the queries' normed before that where asked.
//
// For a pair (x, y) of a head at position p with frequency f:
//   a = p f,   (x, y) -> (x cos a - y sin a, x sin a + y cos a).
// p f reaches 1e6 radians, where a 32-bit angle is off by 0.06, so the turns p f / 2 pi and their
// fraction are 64-bit; the fraction, in [-1/2, 1/2], is then exact enough in 32 bits (2^-25 of a
// turn) for sine and cosine.
//
// Bound: bytes (each value is read once and written once) for prompts, launch latency for one
// token.  A thread keeps one place in the head (up to eight pairs, or 16 copied values) and walks
// over heads; a token's sines are computed once per workgroup, a pair per thread.
//
// Measured: 4099 tokens of 32 + 8 + 8 heads of 128, fp16 to e4m3, 92 MB: 19.6 us, 4.7 TB/s (a large
// copy reaches 5.1); one token: 2.8 us on the device, a load of the position and one of the page
// before the stores can go.
//
// A normed head (x w / sqrt(mean x^2 + eps), or of x less its mean) is summed over its threads by moves
// between registers, in 32 bits, before it turns: the same bytes, 25.1 us for the same prompts,
// 3.7 TB/s; what it adds is the chain from a head's values through their sum to its stores.
#include "layer_ops.h"
#include "mask_core.h"

namespace spax {
namespace {

using namespace elem;

constexpr int kAppendThreads = 256;
constexpr int kMaxPairs = 128;  // head_dim at most 256

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
  // the normed form
  const float *q_w, *q_b, *k_w, *k_b;
  int64_t q_ws, k_ws;  // from head to head
  float eps;
  int32_t layer, lanes;  // lanes: threads set aside for a head, a power of two
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

// Rotates N pairs: (x[i], y[i]), or, where the loaded values alternate between first and second,
// (x[0], x[1]), (x[2], x[3]), .. (y[0], y[1]), ..
template <int N>
__device__ inline void turn(float x[N], float y[N], const float sn[N], const float cs[N],
                            bool alternate) {
  float u[N], w[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const float even = i < N / 2 ? x[2 * i % N] : y[2 * i % N];
    const float odd = i < N / 2 ? x[(2 * i + 1) % N] : y[(2 * i + 1) % N];
    const float px = alternate ? even : x[i], py = alternate ? odd : y[i];
    u[i] = px * cs[i] - py * sn[i];
    w[i] = px * sn[i] + py * cs[i];
  }
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int k = (N + i) / 2 % N;
    x[i] = !alternate ? u[i] : i % 2 ? w[i / 2] : u[i / 2];
    y[i] = !alternate ? w[i] : i % 2 ? w[k] : u[k];
  }
}

template <int N, class T>
__device__ inline void put(T* p, const float* v) {
  if constexpr (N == 1)
    store1(p, v[0]);
  else
    store_n<N>(p, v);
}

// x / scale, rounded to nearest, then clamped.  With r = 1 / s and p = x r the remainder x - p s is exact
// and p + (x - p s) r is the quotient; the rounded reciprocal alone puts ties of e4m3 on the wrong
// side.  p decides what is clamped, so an infinity never gets as far as its remainder.
template <int N>
__device__ inline void divide_e4m3(float v[N], float scale) {
  // scales near the ends of the range, whose reciprocal leaves it, come back with their values
  const float size = fabsf(scale);
  if (!(size >= 0x1p-64f && size <= 0x1p64f)) {
    const float t = size < 1.0f ? 0x1p64f : 0x1p-64f;
    scale *= t;
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] *= t;
  }
  const float r = 1.0f / scale;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const float p = v[i] * r;
    float x = fmaf(fmaf(-p, scale, v[i]), r, p);
    x = p > kE4m3Max ? kE4m3Max : x;
    v[i] = p < -kE4m3Max ? -kE4m3Max : x;
  }
}

template <int CTRL>
__device__ inline float add_moved(float v) {
  return v + __uint_as_float(__builtin_amdgcn_update_dpp(0, __float_as_uint(v), CTRL, 0xF, 0xF, false));
}

// The sum of v over the `lanes` threads (a power of two, aligned) that hold a head: within 16 lanes by
// moves between registers.  More than a wave's meet in `waves`; every thread of the workgroup calls
// it as often.
__device__ inline float sum_of_head(float v, int lanes, float* waves) {
  if (lanes > 1) v = add_moved<0xB1>(v);   // lane ^ 1
  if (lanes > 2) v = add_moved<0x4E>(v);   // lane ^ 2
  if (lanes > 4) v = add_moved<0x141>(v);  // the other four of eight
  if (lanes > 8) v = add_moved<0x140>(v);  // the other eight of sixteen
  if (lanes > 16) v += __shfl_xor(v, 16);
  if (lanes > 32) v += __shfl_xor(v, 32);
  if (lanes > 64) {
    const int wave = threadIdx.x >> 6, first = wave & ~(lanes / 64 - 1);
    __syncthreads();  // the last sums have been read
    if ((threadIdx.x & 63) == 0) waves[wave] = v;
    __syncthreads();
    v = 0.0f;
    for (int y = 0; y < lanes / 64; ++y) v += waves[first + y];
  }
  return v;
}

// N 32-bit values from any 4-byte aligned address.
template <int N>
__device__ inline void load_f32(const float* p, float v[N]) {
  typedef float FN __attribute__((ext_vector_type(N), aligned(4)));
  const FN x = *reinterpret_cast<const FN*>(p);
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = x[i];
}

// A head's norm and its weights, held from head to head as long as they are the same.
template <int N>
struct HeadNorm {
  float w[2 * N];
  int have = -1;  // 0: the queries' shared weights, 1: the keys'
  // x and y: this thread's values of a head, zeros where it has none (`on` false, or y with `single`).
  __device__ inline void apply(const AppendArgs& a, float x[N], float y[N], int h, bool on,
                               bool single, int e0, int e1, float* waves) {
    const int which = h < a.n_heads ? 0 : 1;
    const float* weight = which ? a.k_w : a.q_w;
    const float* bias = which ? a.k_b : a.q_b;
    const int64_t stride = which ? a.k_ws : a.q_ws;
    const int64_t at = (which ? h - a.n_heads : h) * stride;
    const bool normed = on && weight && h < a.n_heads + a.n_kv;
    if (normed && have != which) {
      load_f32<N>(weight + at + e0, w);
      if (!single) load_f32<N>(weight + at + e1, w + N);
      have = stride ? -1 : which;
    }
    const float share = 1.0f / (float)a.dim;
    float mean = 0.0f;
    if (a.layer) {
      float s = 0.0f;
#pragma unroll
      for (int i = 0; i < N; ++i) s += x[i] + y[i];
      mean = sum_of_head(s, a.lanes, waves) * share;
    }
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float u = x[i] - mean, v = single ? 0.0f : y[i] - mean;
      s += u * u + v * v;
    }
    s = sum_of_head(on ? s : 0.0f, a.lanes, waves);
    if (!normed) return;
    const float r = rsqrtf(s * share + a.eps);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      x[i] = (x[i] - mean) * r * w[i];
      y[i] = single ? 0.0f : (y[i] - mean) * r * w[N + i];
    }
    if (!bias) return;
    float b[N];
    load_f32<N>(bias + at + e0, b);
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] += b[i];
    if (single) return;
    load_f32<N>(bias + at + e1, b);
#pragma unroll
    for (int i = 0; i < N; ++i) y[i] += b[i];
  }
};
template <>
struct HeadNorm<0> {};

// SRC: type of q, k, v; LOW: of q_out (and a 16-bit cache); C: of the cache.  A thread's item is N
// pairs of a head, or as many values that are copied: 2 N of them, one for N = 1.  NORM: a head's
// threads lie in a.lanes neighbouring ones, some of them without an item, and all go through
// every round, since the sums of a norm pass through all of them.
template <class SRC, class LOW, class C, int N, bool NORM>
__global__ __launch_bounds__(kAppendThreads) void kv_append_kernel(AppendArgs a) {
  constexpr int kCopied = N > 1 ? 2 * N : 1;
  const int t = blockIdx.x;
  const int pairs = a.rot / 2;
  // items of a head: pairs / N rotated ones, then the copied values
  const int turned = pairs / N;
  const int items = turned + (a.dim - a.rot) / kCopied;
  const int slot = threadIdx.x / (NORM ? a.lanes : items);
  const int j = threadIdx.x - slot * (NORM ? a.lanes : items);
  const int p = a.positions[t];
  const bool turns = j < turned;
  // element offsets of the item's first and second values
  int e0, e1;
  if (turns) {
    e0 = a.interleaved ? 2 * N * j : N * j;
    e1 = a.interleaved ? e0 + N : pairs + N * j;
  } else {
    e0 = a.rot + (j - turned) * kCopied;
    e1 = e0 + N;
  }
  const bool single = N == 1 && !turns;  // one value, no second
  // The token's sines, one thread per pair; the barrier orders LDS only, so the first heads'
  // values, loaded before it, stay in flight.
  __shared__ float sines[2][kMaxPairs];
  const auto find_sines = [&] {
    if ((int)threadIdx.x < pairs)
      sine(p < 0 ? 0 : p, a.inv_freq[threadIdx.x], &sines[0][threadIdx.x],
           &sines[1][threadIdx.x]);
    mask::lds_barrier();
  };
  const int n_heads = a.n_heads, n_kv = a.n_kv;
  const int h0 = blockIdx.y * a.heads_per_block;
  const int total = n_heads + 2 * n_kv;
  const int h1 = h0 + a.heads_per_block < total ? h0 + a.heads_per_block : total;
  typedef SRC SN __attribute__((ext_vector_type(N)));
  SN rx, ry;  // as loaded
  const auto load = [&](int h) {
    if (h >= h1) return;
    const SRC* src = h < n_heads         ? (const SRC*)a.q + t * a.qt + h * a.qh
                     : h < n_heads + n_kv ? (const SRC*)a.k + t * a.kt + (h - n_heads) * a.kh
                                          : (const SRC*)a.v + t * a.vt + (h - n_heads - n_kv) * a.vh;
    rx = load_any<SN>(src + e0);
    if (!single) ry = load_any<SN>(src + e1);
  };
  // threads past the last slot, or past a head's last item: none
  const int mine = slot < a.heads_at_once && (!NORM || j < items) ? h0 + slot : h1;
  load(mine);
  HeadNorm<NORM ? N : 0> norm;
  const Place to = place_of(a, t, p);
  find_sines();
  float sn[N], cs[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    sn[i] = turns ? sines[0][N * j + i] : 0.0f;
    cs[i] = turns ? sines[1][N * j + i] : 1.0f;
  }
  __shared__ float waves[NORM ? kAppendThreads / 64 : 1];
  int base = h0;
  for (int h = mine; (NORM ? base : h) < h1; h += a.heads_at_once, base += a.heads_at_once) {
    const bool on = !NORM || h < h1;
    const bool is_q = h < n_heads, is_v = h >= n_heads + n_kv;
    float x[N], y[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      x[i] = on ? (float)rx[i] : 0.0f;
      y[i] = single || !on ? 0.0f : (float)ry[i];
    }
    load(h + a.heads_at_once);  // ahead of this head's stores
    if constexpr (NORM) {
      norm.apply(a, x, y, h, on, single, e0, e1, waves);
      if (!on) continue;
    }
    if (turns && !is_v) turn<N>(x, y, sn, cs, N > 1 && a.interleaved);
    if (is_q) {
      LOW* dst = (LOW*)a.q_out + t * a.ot + h * a.oh;
      if (p < 0) {
#pragma unroll
        for (int i = 0; i < N; ++i) x[i] = y[i] = 0.0f;
      }
      put<N>(dst + e0, x);
      if (!single) put<N>(dst + e1, y);
    } else if (to.cached) {
      const int hh = is_v ? h - n_heads - n_kv : h - n_heads;
      C* dst = is_v ? (C*)a.vc + to.v + hh * a.vc_head : (C*)a.kc + to.k + hh * a.kc_head;
      if constexpr (sizeof(C) == 1) {
        const float* scale = is_v ? a.v_scale : a.k_scale;
        if (scale) {
          const float by = scale[hh];
          divide_e4m3<N>(x, by);
          divide_e4m3<N>(y, by);
        } else {
#pragma unroll
          for (int i = 0; i < N; ++i) {
            x[i] = clamp_e4m3(x[i]);
            y[i] = clamp_e4m3(y[i]);
          }
        }
      }
      put<N>(dst + e0, x);
      if (!single) put<N>(dst + e1, y);
    }
  }
}

template <class SRC, class LOW, class C, bool NORM>
int launch(const AppendArgs& a, dim3 grid, int pairs, hipStream_t s) {
  const dim3 blk(kAppendThreads);
  if constexpr (NORM) {
    if (pairs == 4)
      hipLaunchKernelGGL((kv_append_kernel<SRC, LOW, C, 4, true>), grid, blk, 0, s, a);
    else
      hipLaunchKernelGGL((kv_append_kernel<SRC, LOW, C, 1, true>), grid, blk, 0, s, a);
  } else if (pairs == 8) {
    hipLaunchKernelGGL((kv_append_kernel<SRC, LOW, C, 8, false>), grid, blk, 0, s, a);
  } else if (pairs == 4) {
    hipLaunchKernelGGL((kv_append_kernel<SRC, LOW, C, 4, false>), grid, blk, 0, s, a);
  } else {
    hipLaunchKernelGGL((kv_append_kernel<SRC, LOW, C, 1, false>), grid, blk, 0, s, a);
  }
  SPAX_HIP_CHECK(hipGetLastError());
  return SPAX_OK;
}

template <class SRC, bool NORM>
int launch_src(const AppendArgs& a, int out_type, bool narrow, dim3 grid, int pairs,
               hipStream_t s) {
  if (out_type == SPAX_F16)
    return narrow ? launch<SRC, f16, e4m3, NORM>(a, grid, pairs, s)
                  : launch<SRC, f16, f16, NORM>(a, grid, pairs, s);
  return narrow ? launch<SRC, bf16, e4m3, NORM>(a, grid, pairs, s)
                : launch<SRC, bf16, bf16, NORM>(a, grid, pairs, s);
}

template <bool NORM>
int launch_norm(const AppendArgs& a, int src_type, int out_type, bool narrow, dim3 grid, int pairs,
                hipStream_t s) {
  switch (src_type) {
    case SPAX_F32: return launch_src<float, NORM>(a, out_type, narrow, grid, pairs, s);
    case SPAX_F16: return launch_src<f16, NORM>(a, out_type, narrow, grid, pairs, s);
    default: return launch_src<bf16, NORM>(a, out_type, narrow, grid, pairs, s);
  }
}

}  // namespace

int launch_kv_append(const spax_kv_append_args* p, const spax_head_norm* n, hipStream_t s) {
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
  // 16 bytes of a 16-bit head at a time where the rotated part divides into such pieces (the
  // prompts of 4099 tokens: 20.0 us with pieces of eight pairs, 20.6 of four, where 40 values are
  // rotated, and 59 of one, where 20 are).  Normed, pieces of four: their weights take half the registers
  // (24.0 us, 26.1 of eight, then).
  const int pairs = !n && p->rot_dim % 16 == 0 ? 8 : p->rot_dim % 8 == 0 ? 4 : 1;
  const int items = pairs > 1 ? a.dim / (2 * pairs) : p->rot_dim / 2 + a.dim - p->rot_dim;
  int lanes = items;
  if (n) {
    for (lanes = 1; lanes < items;) lanes <<= 1;
    a.q_w = n->q_weight; a.q_b = n->q_bias; a.q_ws = n->q_stride;
    a.k_w = n->k_weight; a.k_b = n->k_bias; a.k_ws = n->k_stride;
    a.eps = n->eps; a.layer = n->kind == SPAX_NORM_LAYER; a.lanes = lanes;
  }
  a.heads_at_once = kAppendThreads / lanes;
  // One round of heads per workgroup while there are few tokens: latency is then one load and one
  // store deep.  With many a workgroup walks over all heads of its token.  128 tokens: 4.65 us by
  // rounds, 4.9 walking; 511: equal; 1000: 8.4 and 7.5; 4099: 22.9 and 20.0.
  const int total = a.n_heads + 2 * a.n_kv;
  a.heads_per_block = p->n_tokens < 512 ? a.heads_at_once : total;
  const dim3 grid((unsigned)p->n_tokens,
                  (unsigned)((total + a.heads_per_block - 1) / a.heads_per_block));
  const bool narrow = c.type == SPAX_E4M3;
  return n ? launch_norm<true>(a, p->src_type, p->out_type, narrow, grid, pairs, s)
           : launch_norm<false>(a, p->src_type, p->out_type, narrow, grid, pairs, s);
}

}  // namespace spax
