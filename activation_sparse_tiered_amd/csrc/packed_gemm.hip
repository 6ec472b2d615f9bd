// spax_packed_gemm: rows of many tokens times the original columns of a packed blob.
//
//   t[m][n] = sum_k x[m][k] W[k][n] + bias[n];  u = t, act(t) or act(t_0) t_1;  y = r + scale u.
//
// The blob holds W by input channel: record k has all n side by side, while a matrix instruction
// wants eight k of one n in a lane.  So a lane reads eight n of each of its eight k and turns the
// block within its registers: operand j of the eight is value j of every k, and row i of
// operand j stands for column 8 i + j.
#include "act.h"
#include "layer_ops.h"

namespace spax {
namespace {

using namespace elem;

typedef f16 f16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

struct GemmArgs {
  const uint8_t* w;
  const f16* x;
  const float* bias;
  const void* residual;
  void* y;
  float* parts;
  int64_t w_stride, xs, rs, ys;
  int32_t rows, k, n, width;  // width: columns of y
  int32_t form, gelu, residual_type, y_type;
  int32_t row_tiles, col_tiles, splits, steps;  // steps per split
  float scale;
};

constexpr int kCols = 256;  // of a workgroup: two blocks of 128
constexpr int kStep = 16;   // k of one matrix instruction

// The two blocks of 128 columns of tile c: neighbours, or the same columns of both matrices.
__device__ inline int first_col(const GemmArgs& a, int c, int half) {
  return a.form == SPAX_GEMM_GATED ? half * a.width + 128 * c : kCols * c + 128 * half;
}
// Whether column `at` of a block is one.
__device__ inline bool has_col(const GemmArgs& a, int c, int half, int at) {
  return first_col(a, c, a.form == SPAX_GEMM_GATED ? 0 : half) + at < a.width;
}

template <int N>
__device__ inline void load_row(const void* p, int type, int64_t at, float v[N]) {
  if (type == SPAX_F32) {
    typedef float TN __attribute__((ext_vector_type(N)));
    const TN x = load_any<TN>((const float*)p + at);
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = x[i];
  } else if (type == SPAX_F16) {
    typedef f16 TN __attribute__((ext_vector_type(N)));
    const TN x = load_any<TN>((const f16*)p + at);
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = (float)x[i];
  } else {
    typedef bf16 TN __attribute__((ext_vector_type(N)));
    const TN x = load_any<TN>((const bf16*)p + at);
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = (float)x[i];
  }
}

// Four columns from `col` of row m: t0, and t1 with GATED, without bias.
__device__ inline void finish(const GemmArgs& a, int m, int col, f32x4 t0, f32x4 t1) {
  float u[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float t = t0[i];
    if (a.bias) t += a.bias[col + i];
    if (a.form == SPAX_GEMM_GATED) {
      const float up = a.bias ? t1[i] + a.bias[a.width + col + i] : t1[i];
      t = act_mul(t, up, a.gelu);
    } else if (a.form == SPAX_GEMM_ACT) {
      t = act_mul(t, 1.0f, a.gelu);
    }
    u[i] = a.scale * t;
  }
  if (a.residual) {
    float r[4];
    load_row<4>(a.residual, a.residual_type, m * a.rs + col, r);
#pragma unroll
    for (int i = 0; i < 4; ++i) u[i] += r[i];
  }
  const int64_t at = m * a.ys + col;
  if (a.y_type == SPAX_F32)
    store_n<4>((float*)a.y + at, u);
  else if (a.y_type == SPAX_F16)
    store_n<4>((f16*)a.y + at, u);
  else
    store_n<4>((bf16*)a.y + at, u);
}

// Two int4 values of one column (k and k + 1) as fp16, from words whose low and high halves hold them
// at bit 4 i: 0x6400 | q is 1024 + q, and the multiply-add rounds s q + z once.
__device__ inline uint32_t widen2(uint32_t u, int i, f16x2 s, f16x2 z) {
  const uint32_t q = ((u >> (4 * i)) & 0x000f000fu) | 0x64006400u;
  const f16x2 v = __builtin_bit_cast(f16x2, q) - f16x2{(f16)1024.0f, (f16)1024.0f};
  return __builtin_bit_cast(uint32_t, __builtin_elementwise_fma(v, s, z));
}

// TM tiles of 32 rows, 256 columns; the workgroup's waves take every kWaves-th step of its k.
template <bool INT4, int TM>
struct Few {
  static constexpr int kWaves = TM == 1 ? 8 : 4;
  static constexpr int kThreads = 64 * kWaves;
  static constexpr int kRound = 128 / kWaves;  // rows joined at once
  static constexpr int kPitch = kCols + 4;     // floats between rows in LDS
  static constexpr int kLds = kWaves * kRound * kPitch * 4;
  struct Step {
    u32x4 x[TM];
    u32x4 w[INT4 ? 1 : 8];
    uint32_t q[INT4 ? 8 : 1], sz[INT4 ? 8 : 1];
  };
};

template <bool INT4, int TM>
__global__ __launch_bounds__((Few<INT4, TM>::kThreads)) void gemm_few_kernel(GemmArgs a) {
  using F = Few<INT4, TM>;
  extern __shared__ float lds[];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int h = lane >> 5, r = lane & 31;
  // Workgroups go to the 8 XCDs in turn; those that read the same columns get the same one.
  const int per_xcd = gridDim.x >> 3;
  const int item = (blockIdx.x & 7) * per_xcd + (blockIdx.x >> 3);
  const int m_tile = item % a.row_tiles, rest = item / a.row_tiles;
  const int split = rest % a.splits, c_tile = rest / a.splits;
  if (c_tile >= a.col_tiles) return;

  const int half = r >> 4, at = 8 * (r & 15);
  const int col = has_col(a, c_tile, half, at) ? first_col(a, c_tile, half) + at : 0;
  // Addresses are a uniform part and 32 bits of the lane's own (8 records are below 2^28 bytes).
  const uint32_t w_at = 8u * h * (uint32_t)a.w_stride + (INT4 ? (uint32_t)col / 2 : 2u * col);
  const uint32_t sz_at = 8u * h * (uint32_t)a.w_stride + (uint32_t)a.n / 2 + (uint32_t)col / 128 * 4;
  const int m0 = 32 * TM * m_tile;
  int64_t x_at[TM];
#pragma unroll
  for (int t = 0; t < TM; ++t) {
    const int m = m0 + 32 * t + r;
    x_at[t] = (int64_t)(m < a.rows ? m : a.rows - 1) * a.xs + 8 * h;
  }
  const auto load = [&](typename F::Step& z, int step) {
    const int k0 = kStep * step;
    if (k0 + kStep <= a.k) {
      const f16* x = a.x + k0;
      const uint8_t* rec = a.w + (int64_t)k0 * a.w_stride;
#pragma unroll
      for (int t = 0; t < TM; ++t) z.x[t] = *reinterpret_cast<const u32x4*>(x + x_at[t]);
#pragma unroll
      for (int e = 0; e < 8; ++e, rec += a.w_stride) {
        if constexpr (INT4) {
          z.q[e] = *reinterpret_cast<const uint32_t*>(rec + w_at);
          z.sz[e] = *reinterpret_cast<const uint32_t*>(rec + sz_at);
        } else {
          z.w[e] = *reinterpret_cast<const u32x4*>(rec + w_at);
        }
      }
    } else {  // the last k: past them x counts as zeros, and the last record stands in
      const int valid = a.k - k0 - 8 * h;  // of the lane's eight
#pragma unroll
      for (int t = 0; t < TM; ++t) {
        u32x4 v = {0u, 0u, 0u, 0u};
        if (valid > 0) v = *reinterpret_cast<const u32x4*>(a.x + k0 + x_at[t]);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          v[i] &= 2 * i + 1 < valid ? ~0u : 2 * i < valid ? 0xffffu : 0u;
        z.x[t] = v;
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const uint8_t* rec = a.w + (int64_t)(e < valid ? k0 + 8 * h + e : a.k - 1) * a.w_stride;
        if constexpr (INT4) {
          z.q[e] = *reinterpret_cast<const uint32_t*>(rec + col / 2);
          z.sz[e] = *reinterpret_cast<const uint32_t*>(rec + a.n / 2 + col / 128 * 4);
        } else {
          z.w[e] = *reinterpret_cast<const u32x4*>(rec + 2 * (int64_t)col);
        }
      }
    }
  };
  f32x16 acc[8][TM];
#pragma unroll
  for (int j = 0; j < 8; ++j)
#pragma unroll
    for (int t = 0; t < TM; ++t)
#pragma unroll
      for (int i = 0; i < 16; ++i) acc[j][t][i] = 0.0f;
  const auto use = [&](const typename F::Step& z) {
    uint32_t lo[4], hi[4];  // int4: columns 0..3 and 4..7 of k and k + 1
    f16x2 s[4], zero[4];
    if constexpr (INT4) {
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        lo[p] = __builtin_amdgcn_perm(z.q[2 * p + 1], z.q[2 * p], 0x05040100u);
        hi[p] = __builtin_amdgcn_perm(z.q[2 * p + 1], z.q[2 * p], 0x07060302u);
        s[p] = __builtin_bit_cast(
            f16x2, __builtin_amdgcn_perm(z.sz[2 * p + 1], z.sz[2 * p], 0x05040100u));
        zero[p] = __builtin_bit_cast(
            f16x2, __builtin_amdgcn_perm(z.sz[2 * p + 1], z.sz[2 * p], 0x07060302u));
      }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      u32x4 f;
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        if constexpr (INT4)
          f[p] = widen2(j < 4 ? lo[p] : hi[p], j & 3, s[p], zero[p]);
        else
          f[p] = __builtin_amdgcn_perm(z.w[2 * p + 1][j / 2], z.w[2 * p][j / 2],
                                       j & 1 ? 0x07060302u : 0x05040100u);
      }
#pragma unroll
      for (int t = 0; t < TM; ++t)
        acc[j][t] = __builtin_amdgcn_mfma_f32_32x32x16_f16(
            __builtin_bit_cast(f16x8, f), __builtin_bit_cast(f16x8, z.x[t]), acc[j][t], 0, 0, 0);
    }
  };
  const int steps = (a.k + kStep - 1) / kStep;
  const int stop = (split + 1) * a.steps < steps ? (split + 1) * a.steps : steps;
  int s = split * a.steps + wave;
  typename F::Step z;
  if (s < stop) load(z, s);
  for (; s < stop; s += F::kWaves) {
    typename F::Step next = z;
    if (s + F::kWaves < stop) load(next, s + F::kWaves);
    use(z);
    z = next;
  }

  // Join the waves, some rows at a time.  A lane has row r of each tile, and of register i of every
  // operand columns 8 (8 (i / 4) + 4 h + i % 4) ..
#pragma unroll
  for (int t = 0; t < TM; ++t) {
#pragma unroll
    for (int from = 0; from < 32; from += F::kRound) {
      if (t || from) __syncthreads();
      if (r >= from && r < from + F::kRound) {
        float* to = lds + (wave * F::kRound + r - from) * F::kPitch;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          f32x4 v0, v1;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            v0[j] = acc[j][t][i];
            v1[j] = acc[j + 4][t][i];
          }
          float* p = to + 8 * (8 * (i / 4) + 4 * h + i % 4);
          *reinterpret_cast<f32x4*>(p) = v0;
          *reinterpret_cast<f32x4*>(p + 4) = v1;
        }
      }
      __syncthreads();
      const bool gated = a.form == SPAX_GEMM_GATED && a.splits == 1;
      for (int e = threadIdx.x; e < F::kRound * (gated ? 32 : 64); e += F::kThreads) {
        const int row = gated ? e / 32 : e / 64, c = 4 * (gated ? e % 32 : e % 64);
        const int m = m0 + 32 * t + from + row;
        if (m >= a.rows || !has_col(a, c_tile, c >> 7, c & 127)) continue;
        f32x4 sum0 = {0.0f, 0.0f, 0.0f, 0.0f}, sum1 = sum0;
        for (int w = 0; w < F::kWaves; ++w) {
          const float* p = lds + (w * F::kRound + row) * F::kPitch + c;
          sum0 += *reinterpret_cast<const f32x4*>(p);
          if (gated) sum1 += *reinterpret_cast<const f32x4*>(p + 128);
        }
        const int col = first_col(a, c_tile, c >> 7) + (c & 127);
        if (a.splits == 1)
          finish(a, m, col, sum0, sum1);
        else
          *reinterpret_cast<f32x4*>(a.parts + ((int64_t)split * a.rows + m) * a.n + col) = sum0;
      }
    }
  }
}

constexpr int kJoinThreads = 256;

// Adds the splits' sums, in order, four columns a thread.
__global__ __launch_bounds__(kJoinThreads) void gemm_join_kernel(GemmArgs a) {
  const int per_row = a.width / 4;
  const int64_t e = (int64_t)blockIdx.x * kJoinThreads + threadIdx.x;
  const int m = (int)(e / per_row), col = 4 * (int)(e % per_row);
  if (m >= a.rows) return;
  f32x4 t0 = {0.0f, 0.0f, 0.0f, 0.0f}, t1 = t0;
  for (int s = 0; s < a.splits; ++s) {
    const float* p = a.parts + ((int64_t)s * a.rows + m) * a.n + col;
    t0 += *reinterpret_cast<const f32x4*>(p);
    if (a.form == SPAX_GEMM_GATED) t1 += *reinterpret_cast<const f32x4*>(p + a.width);
  }
  finish(a, m, col, t0, t1);
}

template <bool INT4, int TM>
int launch_few(const GemmArgs& a, unsigned blocks, hipStream_t s) {
  using F = Few<INT4, TM>;
  hipLaunchKernelGGL((gemm_few_kernel<INT4, TM>), dim3(blocks), dim3(F::kThreads), F::kLds, s, a);
  SPAX_HIP_CHECK(hipGetLastError());
  return SPAX_OK;
}

}  // namespace

GemmPlan gemm_plan(const spax_packed_gemm_args* a) {
  const spax_layout& L = *a->layout;
  GemmPlan p{};
  const bool gated = a->form == SPAX_GEMM_GATED;
  const int tile = a->n_rows <= 32 ? 32 : 64;
  p.row_tiles = (a->n_rows + tile - 1) / tile;
  p.col_tiles = (int32_t)(gated ? (L.d_out[0] + 127) / 128 : (L.d_out_total + kCols - 1) / kCols);
  const int64_t items = (int64_t)p.row_tiles * p.col_tiles;
  const int steps = (L.d_in + kStep - 1) / kStep, waves = tile == 32 ? 8 : 4;
  int64_t splits = items ? 256 / items : 1;
  const int64_t most = steps / (2 * waves);
  splits = splits > most ? most : splits;
  p.splits = (int32_t)(splits < 1 ? 1 : splits);
  p.blocks = (items * p.splits + 7) / 8 * 8;
  if (p.splits > 1)
    p.ws_bytes = aligned_size((size_t)p.splits * a->n_rows * L.d_out_total * sizeof(float));
  return p;
}

int launch_packed_gemm(const spax_packed_gemm_args* p, void* ws, hipStream_t s) {
  if (p->n_rows == 0) return SPAX_OK;
  const spax_layout& L = *p->layout;
  const GemmPlan plan = gemm_plan(p);
  GemmArgs a{};
  a.w = (const uint8_t*)p->packed; a.x = (const f16*)p->x; a.bias = p->bias;
  a.residual = p->residual; a.y = p->y; a.parts = (float*)ws;
  a.w_stride = L.stride_F; a.xs = p->x_stride; a.rs = p->residual_stride; a.ys = p->y_stride;
  a.rows = p->n_rows; a.k = L.d_in; a.n = (int32_t)L.d_out_total;
  a.width = p->form == SPAX_GEMM_GATED ? L.d_out[0] : a.n;
  a.form = p->form; a.gelu = p->act == SPAX_ACT_GELU_TANH;
  a.residual_type = p->residual_type; a.y_type = p->y_type; a.scale = p->scale;
  a.row_tiles = plan.row_tiles; a.col_tiles = plan.col_tiles; a.splits = plan.splits;
  const int steps = (a.k + kStep - 1) / kStep;
  a.steps = (steps + a.splits - 1) / a.splits;
  const bool int4 = L.base_fmt == SPAX_FMT_INT4, one = p->n_rows <= 32;
  const unsigned blocks = (unsigned)plan.blocks;
  const int st = int4 ? (one ? launch_few<true, 1>(a, blocks, s) : launch_few<true, 2>(a, blocks, s))
                      : (one ? launch_few<false, 1>(a, blocks, s) : launch_few<false, 2>(a, blocks, s));
  if (st || a.splits == 1) return st;
  const int64_t items = (int64_t)a.rows * (a.width / 4);
  hipLaunchKernelGGL(gemm_join_kernel, dim3((unsigned)((items + kJoinThreads - 1) / kJoinThreads)),
                     dim3(kJoinThreads), 0, s, a);
  SPAX_HIP_CHECK(hipGetLastError());
  return SPAX_OK;
}

}  // namespace spax
