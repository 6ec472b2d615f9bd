// spax_paged_attention: one new query token per sequence over a paged cache.
//
// Per (sequence, key head) with keys k_j, values v_j and the group's queries q_h, in one pass:
//   s_hj = scale q_h.k_j,  m = running max of s,  p = exp(s - m),
//   l <- l exp(m_old - m) + sum p,   o <- o exp(m_old - m) + sum p v,   out = o / l.
// Pieces of a sequence (m, l, o) join by the same rule.
//
// Bound: the cache's bytes, each read once.  A wave takes 32 keys at a time and keeps everything
// in registers:
//   * S^T = K Q^T by 16x16x32 matrix instructions, keys as rows and the group's query heads as
//     columns (16 columns are computed whatever the group; the matrix units have the room).  A
//     lane reads 16 bytes of its own key's row per step of 32 dims.
//   * S^T's layout (lane: one head, keys 4g..4g+3 of each half) is already that of the second
//     product's P operand if that product counts the tile's keys in the order {4g+i, 16+4g+i},
//     so probabilities never cross lanes.
//   * O^T = V^T P^T: a lane reads whole pieces of the rows of its 8 keys (16 lanes cover a row),
//     and swaps 2x2 blocks of 16-bit values with byte permutes to get 8 keys of one dim.
//   * p is split into two 16-bit values, p = hi + lo, each multiplied: rounding p to 16 bits
//     would cost as much error again as rounding the result.
#include "layer_ops.h"

namespace spax {
namespace {

using namespace elem;

constexpr int kTile = 32;        // keys per wave and step
constexpr int kAttnWaves = 4;
constexpr int kAttnThreads = 64 * kAttnWaves;
constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;

struct AttnArgs {
  const void *q, *k, *v;
  void* out;
  float *lse, *part_o, *part_ml;
  const int32_t *lens, *table;
  const float *k_scale, *v_scale;
  int64_t qs, qh, os, oh;
  int64_t k_page, k_head, k_row, v_page, v_head, v_row, table_stride;
  int32_t n_heads, n_kv, group, head_tiles, n_seqs, n_pages, page_shift;
  int32_t max_len, window, chunk_tiles, max_chunks;
  float scale;
};

template <class T>
struct Mma;
template <>
struct Mma<f16> {
  typedef f16 v8 __attribute__((ext_vector_type(8)));
  static __device__ inline f32x4 mul(u32x4 a, u32x4 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8, a),
                                                  __builtin_bit_cast(v8, b), c, 0, 0, 0);
  }
  // two e4m3 values (the low or high half of w) as 16-bit ones, exactly
  template <bool HI>
  static __device__ inline uint32_t widen(uint32_t w) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, HI));
  }
  typedef f16x2 v2;
};
template <>
struct Mma<bf16> {
  typedef bf16 v8 __attribute__((ext_vector_type(8)));
  static __device__ inline f32x4 mul(u32x4 a, u32x4 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8, a),
                                                   __builtin_bit_cast(v8, b), c, 0, 0, 0);
  }
  template <bool HI>
  static __device__ inline uint32_t widen(uint32_t w) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, HI));
  }
  typedef bf16x2 v2;
};

// N dwords at p (aligned to their own size, at most 16 bytes; 3 dwords never occur).
template <int N>
__device__ inline void load_words(const void* p, uint32_t* w) {
  if constexpr (N == 4) {
    const u32x4 x = *reinterpret_cast<const u32x4*>(p);
    w[0] = x.x; w[1] = x.y; w[2] = x.z; w[3] = x.w;
  } else if constexpr (N == 2) {
    const u32x2 x = *reinterpret_cast<const u32x2*>(p);
    w[0] = x.x; w[1] = x.y;
  } else {
    w[0] = *reinterpret_cast<const uint32_t*>(p);
  }
}

// Values of a lane's piece of a V row: 16 lanes cover a block of 16 * n dims.  A head of D dims
// is one or two such blocks, each lane's piece a power of two.
template <int D>
struct VDims {
  static constexpr int n0 = D == 64 || D == 96 ? 4 : 8;
  static constexpr int n1 = D / 16 - n0;
  static constexpr int n = D / 16;
};

template <class T, bool NARROW, int D>
struct Wave {
  static constexpr int KC = D / 32;          // steps of 32 dims
  static constexpr int VN = D / 16;          // a lane's dims of a V row
  static constexpr int EB = NARROW ? 1 : 2;  // bytes per cached value

  u32x4 q[KC];
  f32x4 o[VN];
  float m, l;  // of head lane % 16: the running max (scaled to log2), this lane's part of the sum

  // The K rows of 16 keys as the first operand, widened if need be.
  static __device__ inline void load_k(const uint8_t* row, int g, u32x4 k[KC]) {
    if constexpr (!NARROW) {
#pragma unroll
      for (int c = 0; c < KC; ++c) k[c] = *reinterpret_cast<const u32x4*>(row + 64 * c + 16 * g);
    } else {
#pragma unroll
      for (int c = 0; c < KC; ++c) {
        const u32x2 w = *reinterpret_cast<const u32x2*>(row + 32 * c + 8 * g);
        k[c].x = w.x;
        k[c].y = w.y;
      }
    }
  }
  static __device__ inline u32x4 widen_k(u32x4 k) {
    if constexpr (NARROW) {
      u32x4 r;
      r.x = Mma<T>::template widen<false>(k.x);
      r.y = Mma<T>::template widen<true>(k.x);
      r.z = Mma<T>::template widen<false>(k.y);
      r.w = Mma<T>::template widen<true>(k.y);
      return r;
    } else {
      return k;
    }
  }
  // A lane's piece of one V row: VN values, packed as stored.
  static constexpr int VW = (VN * EB + 3) / 4 < 1 ? 1 : (VN * EB + 3) / 4;
  static __device__ inline void load_v(const uint8_t* row, int r, uint32_t* w) {
    constexpr int n0 = VDims<D>::n0, n1 = VDims<D>::n1;
    load_words<n0 * EB / 4>(row + n0 * EB * r, w);
    if constexpr (n1 * EB >= 4)
      load_words<n1 * EB / 4>(row + 16 * n0 * EB + n1 * EB * r, w + n0 * EB / 4);
    else if constexpr (n1 * EB == 2)
      w[n0 * EB / 4] = *reinterpret_cast<const uint16_t*>(row + 16 * n0 * EB + n1 * EB * r);
  }
};

template <class T, bool NARROW, int D>
__global__ __launch_bounds__(kAttnThreads) void attention_kernel(AttnArgs a) {
  using W = Wave<T, NARROW, D>;
  constexpr int KC = W::KC, VN = W::VN, VW = W::VW, EB = W::EB;
  extern __shared__ float lds[];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int g = lane >> 4, r = lane & 15;

  // work item: chunk fastest, so that the pieces of one sequence start together
  int id = blockIdx.x;
  const int chunk = id % a.max_chunks;
  id /= a.max_chunks;
  const int ht = id % a.head_tiles;
  id /= a.head_tiles;
  const int kvh = id % a.n_kv;
  const int seq = id / a.n_kv;

  int hi = a.lens[seq];
  hi = hi < 0 ? 0 : hi > a.max_len ? a.max_len : hi;
  const int lo = a.window > 0 && hi > a.window ? hi - a.window : 0;
  const int first = lo / kTile, end = (hi + kTile - 1) / kTile;
  const int chunks = (end - first + a.chunk_tiles - 1) / a.chunk_tiles;
  if (chunk >= chunks && chunk > 0) return;
  const int t0 = first + chunk * a.chunk_tiles;
  const int t1 = t0 + a.chunk_tiles < end ? t0 + a.chunk_tiles : end;
  const int heads = a.group - 16 * ht < 16 ? a.group - 16 * ht : 16;  // of this workgroup
  const int head0 = kvh * a.group + 16 * ht;

  W w;
#pragma unroll
  for (int c = 0; c < KC; ++c) w.q[c] = u32x4{0u, 0u, 0u, 0u};
  if (r < heads) {
    const uint8_t* qrow = (const uint8_t*)a.q + 2 * (seq * a.qs + (head0 + r) * a.qh);
#pragma unroll
    for (int c = 0; c < KC; ++c) w.q[c] = *reinterpret_cast<const u32x4*>(qrow + 64 * c + 16 * g);
  }
#pragma unroll
  for (int t = 0; t < VN; ++t) w.o[t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  w.m = -INFINITY;
  w.l = 0.0f;

  float to_log2 = a.scale * kLog2e;
  if constexpr (NARROW)
    if (a.k_scale) to_log2 *= a.k_scale[kvh];

  const int32_t* table = a.table + seq * a.table_stride;
  const uint8_t* kbase = (const uint8_t*)a.k + (int64_t)EB * kvh * a.k_head;
  const uint8_t* vbase = (const uint8_t*)a.v + (int64_t)EB * kvh * a.v_head;
  const int row_mask = (1 << a.page_shift) - 1;

  for (int tile = t0 + wave; tile < t1; tile += kAttnWaves) {
    const int kb = tile * kTile;
    // lane l looks up the page of key l % 32 (a key outside [lo, hi) that of the nearest inside)
    int at = kb + (lane & 31);
    at = at < lo ? lo : at >= hi ? hi - 1 : at;
    const int entry = table[at >> a.page_shift];
    const int page_ok = (uint32_t)entry < (uint32_t)a.n_pages;
    const int page = page_ok ? entry : -1;
    const bool whole = kb >= lo && kb + kTile <= hi && __all(page_ok);

    u32x4 k[2][KC];
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int pg = __shfl(page, 16 * half + r);
      const int64_t row = (int64_t)(pg < 0 ? 0 : pg) * a.k_page +
                          (int64_t)((kb + 16 * half + r) & row_mask) * a.k_row;
      W::load_k(kbase + EB * row, g, k[half]);
    }
    uint32_t v[8][VW];
    int vpage[2];
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      vpage[half] = __shfl(page, 16 * half + 4 * g);
      const int64_t row = (int64_t)(vpage[half] < 0 ? 0 : vpage[half]) * a.v_page +
                          (int64_t)((kb + 16 * half + 4 * g) & row_mask) * a.v_row;
#pragma unroll
      for (int i = 0; i < 4; ++i) W::load_v(vbase + EB * (row + i * a.v_row), r, v[4 * half + i]);
    }

    f32x4 s[2];
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      s[half] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int c = 0; c < KC; ++c) s[half] = Mma<T>::mul(W::widen_k(k[half][c]), w.q[c], s[half]);
    }
    float p[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) p[i] = s[i / 4][i % 4] * to_log2;
    if (!whole) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int key = kb + 16 * (i / 4) + 4 * g + i % 4;
        if (!(key >= lo && key < hi && vpage[i / 4] >= 0)) {
          p[i] = -INFINITY;
#pragma unroll
          for (int x = 0; x < VW; ++x) v[i][x] = 0u;
        }
      }
    }
    float top = fmaxf(fmaxf(fmaxf(p[0], p[1]), fmaxf(p[2], p[3])),
                      fmaxf(fmaxf(p[4], p[5]), fmaxf(p[6], p[7])));
    top = fmaxf(top, __shfl_xor(top, 16));
    top = fmaxf(top, __shfl_xor(top, 32));
    if (__any(top > w.m)) {
      const float m = fmaxf(w.m, top);
      const float f = m == w.m ? 1.0f : __builtin_amdgcn_exp2f(w.m - m);
      w.m = m;
      w.l *= f;
#pragma unroll
      for (int t = 0; t < VN; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) w.o[t][i] *= f;
    }
    const float base = w.m == -INFINITY ? 0.0f : w.m;
    u32x4 hi2, lo2;
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      const float p0 = __builtin_amdgcn_exp2f(p[i] - base);
      const float p1 = __builtin_amdgcn_exp2f(p[i + 1] - base);
      w.l += p0 + p1;
      typename Mma<T>::v2 h;
      h.x = (T)p0;
      h.y = (T)p1;
      typename Mma<T>::v2 rest;
      rest.x = (T)(p0 - (float)h.x);
      rest.y = (T)(p1 - (float)h.y);
      hi2[i / 2] = __builtin_bit_cast(uint32_t, h);
      lo2[i / 2] = __builtin_bit_cast(uint32_t, rest);
    }
    // 8 keys of each dim, pair by pair: byte permutes of two rows' words
#pragma unroll
    for (int t2 = 0; t2 < VN / 2; ++t2) {
      uint32_t x[8];  // dims 2 t2 and 2 t2 + 1 of the 8 keys, 16-bit
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if constexpr (NARROW)
          x[i] = t2 % 2 ? Mma<T>::template widen<true>(v[i][t2 / 2])
                        : Mma<T>::template widen<false>(v[i][t2 / 2]);
        else
          x[i] = v[i][t2];
      }
      u32x4 even, odd;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        even[i] = __builtin_amdgcn_perm(x[2 * i + 1], x[2 * i], 0x05040100u);
        odd[i] = __builtin_amdgcn_perm(x[2 * i + 1], x[2 * i], 0x07060302u);
      }
      w.o[2 * t2] = Mma<T>::mul(even, hi2, w.o[2 * t2]);
      w.o[2 * t2 + 1] = Mma<T>::mul(odd, hi2, w.o[2 * t2 + 1]);
      w.o[2 * t2] = Mma<T>::mul(even, lo2, w.o[2 * t2]);
      w.o[2 * t2 + 1] = Mma<T>::mul(odd, lo2, w.o[2 * t2 + 1]);
    }
  }

  // Join the waves: each puts m, l and o of the group's heads into LDS, dims a block at a time.
  w.l += __shfl_xor(w.l, 16);
  w.l += __shfl_xor(w.l, 32);
  constexpr int n0 = VDims<D>::n0, n1 = VDims<D>::n1;
  constexpr int kPad = 4;
  constexpr int stride = 16 * n0 + kPad;  // n1 <= n0
  float* ml = lds;                         // [wave][16][2]
  float* ob = lds + kAttnWaves * 32;       // [wave][heads][stride]
  if (g == 0) {
    ml[(wave * 16 + r) * 2] = w.m;
    ml[(wave * 16 + r) * 2 + 1] = w.l;
  }
  const bool last = chunks <= 1;
  float v_mul = 1.0f;
  if constexpr (NARROW)
    if (a.v_scale) v_mul = a.v_scale[kvh];
#pragma unroll
  for (int block = 0; block < (n1 ? 2 : 1); ++block) {
    const int n = block ? n1 : n0;
    const int t_base = block ? n0 : 0;
    if (block) __syncthreads();
    if (r < heads) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int t = 0; t < (n1 > n0 ? n1 : n0); ++t)
          if (t < n) ob[(wave * heads + r) * stride + (4 * g + i) * n + t] = w.o[t_base + t][i];
    }
    __syncthreads();
    const int dims = 16 * n;
    for (int e = threadIdx.x; e < heads * (dims / 4); e += kAttnThreads) {
      const int h = e / (dims / 4), d = 4 * (e % (dims / 4));
      float m = -INFINITY;
#pragma unroll
      for (int x = 0; x < kAttnWaves; ++x) m = fmaxf(m, ml[(x * 16 + h) * 2]);
      const float base = m == -INFINITY ? 0.0f : m;
      float l = 0.0f;
      float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int x = 0; x < kAttnWaves; ++x) {
        const float f = __builtin_amdgcn_exp2f(ml[(x * 16 + h) * 2] - base);
        l += f * ml[(x * 16 + h) * 2 + 1];
        const f32x4 o4 = *reinterpret_cast<const f32x4*>(&ob[(x * heads + h) * stride + d]);
#pragma unroll
        for (int i = 0; i < 4; ++i) sum[i] += f * o4[i];
      }
      const int64_t row = (int64_t)seq * a.n_heads + head0 + h;
      const int dim = (block ? 16 * n0 : 0) + d;
      if (last) {
        const float inv = v_mul / l;
#pragma unroll
        for (int i = 0; i < 4; ++i) sum[i] = l == 0.0f ? 0.0f : sum[i] * inv;
        store4((T*)a.out + seq * a.os + (head0 + h) * a.oh + dim, sum);
        if (a.lse && dim == 0) a.lse[row] = l == 0.0f ? -INFINITY : (m + log2f(l)) * kLn2;
      } else {
        const int64_t part = row * a.max_chunks + chunk;
        *reinterpret_cast<f32x4*>(a.part_o + part * D + dim) =
            f32x4{sum[0], sum[1], sum[2], sum[3]};
        if (dim == 0) {
          a.part_ml[2 * part] = m;
          a.part_ml[2 * part + 1] = l;
        }
      }
    }
  }
}

// Joins the pieces of one (sequence, head) that was shared out: one workgroup each.
template <class T, int D>
__global__ __launch_bounds__(256) void attention_join_kernel(AttnArgs a) {
  constexpr int kLanes = D / 4;            // threads per piece
  constexpr int kAtOnce = 256 / kLanes;    // pieces in flight
  __shared__ float lds_o[kAtOnce][D];
  __shared__ float lds_l[kAtOnce];
  const int head = blockIdx.x % a.n_heads, seq = blockIdx.x / a.n_heads;
  int hi = a.lens[seq];
  hi = hi < 0 ? 0 : hi > a.max_len ? a.max_len : hi;
  const int lo = a.window > 0 && hi > a.window ? hi - a.window : 0;
  const int first = lo / kTile, end = (hi + kTile - 1) / kTile;
  const int chunks = (end - first + a.chunk_tiles - 1) / a.chunk_tiles;
  if (chunks <= 1) return;
  const int64_t row = (int64_t)seq * a.n_heads + head;
  const float* ml = a.part_ml + 2 * row * a.max_chunks;
  const float* po = a.part_o + row * a.max_chunks * D;
  float m = -INFINITY;
  for (int c = 0; c < chunks; ++c) m = fmaxf(m, ml[2 * c]);
  const float base = m == -INFINITY ? 0.0f : m;
  const int part = threadIdx.x / kLanes, d = 4 * (threadIdx.x % kLanes);
  float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  float l = 0.0f;
  if (part < kAtOnce) {
    for (int c = part; c < chunks; c += kAtOnce) {
      const float f = __builtin_amdgcn_exp2f(ml[2 * c] - base);
      l += f * ml[2 * c + 1];
      const f32x4 o = *reinterpret_cast<const f32x4*>(po + (int64_t)c * D + d);
#pragma unroll
      for (int i = 0; i < 4; ++i) sum[i] += f * o[i];
    }
    *reinterpret_cast<f32x4*>(&lds_o[part][d]) = f32x4{sum[0], sum[1], sum[2], sum[3]};
    if (d == 0) lds_l[part] = l;
  }
  __syncthreads();
  if (threadIdx.x >= kLanes) return;
  l = 0.0f;
  float out[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int x = 0; x < kAtOnce; ++x) {
    l += lds_l[x];
#pragma unroll
    for (int i = 0; i < 4; ++i) out[i] += lds_o[x][d + i];
  }
  float v_mul = 1.0f;
  if (a.v_scale) v_mul = a.v_scale[head / a.group];
  const float inv = v_mul / l;
#pragma unroll
  for (int i = 0; i < 4; ++i) out[i] = l == 0.0f ? 0.0f : out[i] * inv;
  store4((T*)a.out + seq * a.os + head * a.oh + d, out);
  if (a.lse && d == 0)
    a.lse[row] = l == 0.0f ? -INFINITY : (m + log2f(l)) * kLn2;
}

template <class T, bool NARROW, int D>
int launch(const AttnArgs& a, const AttentionPlan& plan, hipStream_t s) {
  const int heads = a.group < 16 ? a.group : 16;
  const size_t lds =
      sizeof(float) * kAttnWaves * (32 + (size_t)heads * (16 * VDims<D>::n0 + 4));
  const dim3 grid((unsigned)((int64_t)a.n_seqs * a.n_kv * a.head_tiles * a.max_chunks));
  hipLaunchKernelGGL((attention_kernel<T, NARROW, D>), grid, dim3(kAttnThreads), lds, s, a);
  SPAX_HIP_CHECK(hipGetLastError());
  if (a.max_chunks > 1) {
    hipLaunchKernelGGL((attention_join_kernel<T, D>), dim3((unsigned)(a.n_seqs * a.n_heads)),
                       dim3(256), 0, s, a);
    SPAX_HIP_CHECK(hipGetLastError());
  }
  return SPAX_OK;
}

template <class T, bool NARROW>
int launch_dim(const AttnArgs& a, const AttentionPlan& plan, int dim, hipStream_t s) {
  switch (dim) {
    case 64: return launch<T, NARROW, 64>(a, plan, s);
    case 96: return launch<T, NARROW, 96>(a, plan, s);
    case 128: return launch<T, NARROW, 128>(a, plan, s);
    case 192: return launch<T, NARROW, 192>(a, plan, s);
    default: return launch<T, NARROW, 256>(a, plan, s);
  }
}

}  // namespace

AttentionPlan attention_plan(const spax_attention_args* a) {
  const spax_kv_cache& c = *a->cache;
  AttentionPlan p{};
  const int group = a->n_heads / c.n_kv_heads;
  p.head_tiles = (group + 15) / 16;
  int64_t tiles = ((int64_t)a->max_len + kTile - 1) / kTile;
  if (a->window > 0) {
    const int64_t w = ((int64_t)a->window + kTile - 1) / kTile + 1;  // a window starts anywhere
    if (w < tiles) tiles = w;
  }
  const int64_t rows = (int64_t)c.n_seqs * c.n_kv_heads * p.head_tiles;
  int64_t chunk = (rows * tiles + 1023) / 1024;
  chunk = (chunk + kAttnWaves - 1) / kAttnWaves * kAttnWaves;
  if (chunk > 32) chunk = 32;
  p.chunk_tiles = (int32_t)chunk;
  p.max_chunks = (int32_t)((tiles + chunk - 1) / chunk);
  if (p.max_chunks > 1)
    p.ws_bytes = aligned_size((size_t)c.n_seqs * a->n_heads * p.max_chunks *
                              ((size_t)c.head_dim + 2) * sizeof(float));
  return p;
}

int launch_attention(const spax_attention_args* p, void* ws, hipStream_t s) {
  const spax_kv_cache& c = *p->cache;
  const AttentionPlan plan = attention_plan(p);
  AttnArgs a{};
  a.q = p->q; a.k = c.k; a.v = c.v; a.out = p->out; a.lse = p->lse;
  a.lens = p->lens; a.table = c.page_table; a.k_scale = c.k_scale; a.v_scale = c.v_scale;
  a.qs = p->q_seq_stride; a.qh = p->q_head_stride;
  a.os = p->out_seq_stride; a.oh = p->out_head_stride;
  a.k_page = c.k_page_stride; a.k_head = c.k_head_stride; a.k_row = c.k_row_stride;
  a.v_page = c.v_page_stride; a.v_head = c.v_head_stride; a.v_row = c.v_row_stride;
  a.table_stride = c.table_stride;
  a.n_heads = p->n_heads; a.n_kv = c.n_kv_heads; a.group = p->n_heads / c.n_kv_heads;
  a.head_tiles = plan.head_tiles; a.n_seqs = c.n_seqs; a.n_pages = c.n_pages;
  a.page_shift = __builtin_ctz((unsigned)c.page_size);
  a.max_len = p->max_len; a.window = p->window; a.scale = p->scale;
  a.chunk_tiles = plan.chunk_tiles; a.max_chunks = plan.max_chunks;
  a.part_o = (float*)ws;
  a.part_ml = (float*)ws + (size_t)c.n_seqs * p->n_heads * plan.max_chunks * c.head_dim;
  if (c.type == SPAX_E4M3)
    return p->type == SPAX_F16 ? launch_dim<f16, true>(a, plan, c.head_dim, s)
                               : launch_dim<bf16, true>(a, plan, c.head_dim, s);
  return p->type == SPAX_F16 ? launch_dim<f16, false>(a, plan, c.head_dim, s)
                             : launch_dim<bf16, false>(a, plan, c.head_dim, s);
}

}  // namespace spax
