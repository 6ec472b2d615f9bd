// spax_packed_gemm: rows of many tokens times the original columns of a packed blob.
//
//   t[m][n] = sum_k x[m][k] W[k][n] + bias[n];  u = t, act(t) or act(t_0) t_1;  y = r + scale u.
//
// The blob holds W by input channel: record k has all n side by side, while a matrix instruction
// wants eight k of one n in a lane.  Tiles of 32 rows (gemm_few_kernel) turn them in registers: a lane
// reads eight n of each of its eight k, operand j of the eight is value j of every k, and row i of
// operand j stands for column 8 i + j.  Larger ones (gemm_many_kernel) stage x and W in LDS for eight
// waves and read W by transposing reads.  A workgroup has 256 columns, with GATED 128 of each matrix, so
// the gate is applied where the sums are.  Where tiles are few, k is cut into pieces whose sums
// (fp32) a second launch adds in order: results depend on the sizes alone.
//
// int4 weights become w_hat rounded to fp16 (one multiply-add of 16 bits per pair): half of a step of
// 2^-11 of each weight, which is what an fp16 base loses when it is packed; sums are in fp32.
//
// What bounds it (us of calls back to back, the weights in memory).  Many rows: 4096 x 4096 x 22016
// fp16 766, 964 TFLOP/s (a large library product reaches 1400), int4 809, 913: matrix
// instructions are under way in 0.52 of the SIMDs' cycles, the rest are LDS reads (6 KB for every eight
// of them) and the step's barrier; a wave with 128 x 128 sums would read a third less and needs all
// of its SIMD's registers.  Few rows: 5 x 4096 x 12288 fp16 23.7, of which the first launch takes 20
// (100 MB at 5 TB/s) and the join 4; 61 x 11008 x 4096 int4 21.0, of which 17 and 4: vector
// instructions, most of them to widen the codes once for every 32 rows, fill half of the cycles.
#include "act.h"
#include "layer_ops.h"
#include "mask_core.h"
#include "staging.h"

namespace spax {
namespace {

using namespace elem;
using namespace staging;

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
// at bit 4 i: 0x6400 | q is 1024 + q, with q one place higher 1024 + 16 q, and the multiply-add rounds
// s q + z once.  The constants are hidden in registers, where an and and an or become one
// instruction.
struct Widen {
  uint32_t low, high, magic;
  __device__ inline Widen() : low(0x000f000fu), high(0x00f000f0u), magic(0x64006400u) {
    asm("" : "+v"(low));
    asm("" : "+v"(high));
    asm("" : "+s"(magic));
  }
  __device__ inline uint32_t two(uint32_t u, int i, f16x2 s, f16x2 z) const {
    const uint32_t w = i < 2 ? u : u >> 8;
    f16x2 v = __builtin_bit_cast(f16x2, (w & (i % 2 ? high : low)) | magic);
    if (i % 2)
      v = __builtin_elementwise_fma(v, f16x2{(f16)0.0625f, (f16)0.0625f}, f16x2{(f16)-64.0f, (f16)-64.0f});
    else
      v -= f16x2{(f16)1024.0f, (f16)1024.0f};
    return __builtin_bit_cast(uint32_t, __builtin_elementwise_fma(v, s, z));
  }
};

// Lane L's value, of each 16 lanes.
template <int L>
__device__ inline f16x2 from_lane(uint32_t v) {
  return __builtin_bit_cast(f16x2, __builtin_amdgcn_update_dpp(0u, v, 0x150 + L, 0xf, 0xf, true));
}

// 32 rows, 256 columns; the workgroup's waves take every kWaves-th step of its k.
template <bool INT4>
struct Few {
  static constexpr int kWaves = 8;
  static constexpr int kAhead = INT4 ? 3 : 2;  // steps in flight
  static constexpr int kThreads = 64 * kWaves;
  static constexpr int kRound = 128 / kWaves;  // rows joined at once
  static constexpr int kPitch = kCols + 4;     // floats between rows in LDS
  static constexpr int kLds = kWaves * kRound * kPitch * 4;
  struct Step {
    u32x4 x;
    u32x4 w[INT4 ? 1 : 8];
    uint32_t q[INT4 ? 8 : 1], sz;  // sz: of record lane % 8 of the lane's eight
  };
};

template <bool INT4>
__global__ __launch_bounds__(Few<INT4>::kThreads) void gemm_few_kernel(GemmArgs a) {
  using F = Few<INT4>;
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
  const uint32_t sz_at = (8u * h + (lane & 7)) * (uint32_t)a.w_stride + (uint32_t)a.n / 2 +
                         (uint32_t)col / 128 * 4;
  const int m0 = 32 * m_tile;
  const int64_t x_at = (int64_t)(m0 + r < a.rows ? m0 + r : a.rows - 1) * a.xs + 8 * h;
  const auto load = [&](typename F::Step& z, int step) {
    const int k0 = kStep * step;
    if (k0 + kStep <= a.k) {
      const f16* x = a.x + k0;
      const uint8_t* rec = a.w + (int64_t)k0 * a.w_stride;
      z.x = *reinterpret_cast<const u32x4*>(x + x_at);
      if constexpr (INT4) z.sz = *reinterpret_cast<const uint32_t*>(rec + sz_at);
#pragma unroll
      for (int e = 0; e < 8; ++e, rec += a.w_stride) {
        if constexpr (INT4) {
          z.q[e] = *reinterpret_cast<const uint32_t*>(rec + w_at);
        } else {
          z.w[e] = *reinterpret_cast<const u32x4*>(rec + w_at);
        }
      }
    } else {  // the last k: past them x and the weights count as zeros (0 * inf is NaN)
      const int valid = a.k - k0 - 8 * h;  // of the lane's eight
      u32x4 v = {0u, 0u, 0u, 0u};
      if (valid > 0) v = *reinterpret_cast<const u32x4*>(a.x + k0 + x_at);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        v[i] &= 2 * i + 1 < valid ? ~0u : 2 * i < valid ? 0xffffu : 0u;
      z.x = v;
      const auto record = [&](int e) {
        return a.w + (int64_t)(e < valid ? k0 + 8 * h + e : a.k - 1) * a.w_stride;
      };
      if constexpr (INT4)
        z.sz = (lane & 7) < valid
                   ? *reinterpret_cast<const uint32_t*>(record(lane & 7) + a.n / 2 + col / 128 * 4)
                   : 0u;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const uint8_t* rec = record(e);
        if constexpr (INT4) {
          z.q[e] = *reinterpret_cast<const uint32_t*>(rec + col / 2);
        } else {
          z.w[e] = *reinterpret_cast<const u32x4*>(rec + 2 * (int64_t)col);
          if (e >= valid) z.w[e] = u32x4{0u, 0u, 0u, 0u};
        }
      }
    }
  };
  const Widen widen;
  f32x16 acc[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) acc[j] = f32x16{};
  const auto use = [&](const typename F::Step& z) {
    uint32_t lo[4], hi[4];  // int4: columns 0..3 and 4..7 of k and k + 1
    f16x2 s[4], zero[4];
    if constexpr (INT4) {
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        lo[p] = __builtin_amdgcn_perm(z.q[2 * p + 1], z.q[2 * p], 0x05040100u);
        hi[p] = __builtin_amdgcn_perm(z.q[2 * p + 1], z.q[2 * p], 0x07060302u);
      }
      // scales and zeros of two records, from their lanes
      const uint32_t up = __builtin_amdgcn_update_dpp(0u, z.sz, 0x101, 0xf, 0xf, true);  // lane + 1's
      const uint32_t ss = __builtin_amdgcn_perm(up, z.sz, 0x05040100u);
      const uint32_t zz = __builtin_amdgcn_perm(up, z.sz, 0x07060302u);
      s[0] = from_lane<0>(ss); s[1] = from_lane<2>(ss); s[2] = from_lane<4>(ss); s[3] = from_lane<6>(ss);
      zero[0] = from_lane<0>(zz); zero[1] = from_lane<2>(zz);
      zero[2] = from_lane<4>(zz); zero[3] = from_lane<6>(zz);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      u32x4 f;
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        if constexpr (INT4)
          f[p] = widen.two(j < 4 ? lo[p] : hi[p], j & 3, s[p], zero[p]);
        else
          f[p] = __builtin_amdgcn_perm(z.w[2 * p + 1][j / 2], z.w[2 * p][j / 2],
                                       j & 1 ? 0x07060302u : 0x05040100u);
      }
      acc[j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(
          __builtin_bit_cast(f16x8, f), __builtin_bit_cast(f16x8, z.x), acc[j], 0, 0, 0);
    }
  };
  const int steps = (a.k + kStep - 1) / kStep;
  const int stop = (split + 1) * a.steps < steps ? (split + 1) * a.steps : steps;
  int s = split * a.steps + wave;
  typename F::Step z[F::kAhead];
#pragma unroll
  for (int y = 0; y < F::kAhead; ++y)
    if (s + y * F::kWaves < stop) load(z[y], s + y * F::kWaves);
  for (; s < stop; s += F::kAhead * F::kWaves) {
#pragma unroll
    for (int y = 0; y < F::kAhead; ++y) {
      if (s + y * F::kWaves < stop) use(z[y]);
      if (s + (y + F::kAhead) * F::kWaves < stop) load(z[y], s + (y + F::kAhead) * F::kWaves);
    }
  }

  // Join the waves, half of the rows at a time.  A lane has row r, and of register i of every operand
  // columns 8 (8 (i / 4) + 4 h + i % 4) ..
#pragma unroll
  for (int from = 0; from < 32; from += F::kRound) {
    if (from) __syncthreads();
    if (r >= from && r < from + F::kRound) {
      float* to = lds + (wave * F::kRound + r - from) * F::kPitch;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        f32x4 v0, v1;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          v0[j] = acc[j][i];
          v1[j] = acc[j + 4][i];
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
      const int m = m0 + from + row;
      if (m >= a.rows || !has_col(a, c_tile, c >> 7, c & 127)) continue;
      f32x4 sum0 = {0.0f, 0.0f, 0.0f, 0.0f}, sum1 = sum0;
#pragma unroll
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

// Eight int4 values of one k, packed as stored, as fp16 in order.
__device__ inline u32x4 widen8(const Widen& widen, uint32_t w, f16x2 s, f16x2 z) {
  uint32_t r[4];  // columns i and i + 4
#pragma unroll
  for (int i = 0; i < 4; ++i) r[i] = widen.two(w, i, s, z);
  return u32x4{__builtin_amdgcn_perm(r[1], r[0], 0x05040100u),
               __builtin_amdgcn_perm(r[3], r[2], 0x05040100u),
               __builtin_amdgcn_perm(r[1], r[0], 0x07060302u),
               __builtin_amdgcn_perm(r[3], r[2], 0x07060302u)};
}

// Many rows: 64 TT of them by 256 columns, 64 k a step, staged in LDS for eight waves: two of 32 TT rows
// by four of 32 columns in each block of 128.
template <bool INT4, int TT>
struct Many {
  static constexpr int kThreads = 512, kRows = 64 * TT, kDepth = 64;
  static constexpr int kX = kRows * kDepth * 2, kW = kDepth * kCols * 2;
  static constexpr int kStage = kX + kW;
  static constexpr int kPitch = kCols + 4;            // floats between rows in the last exchange
  static constexpr int kExchange = 32 * TT * kPitch * 4;  // half of the rows at a time
  static constexpr int kLds = 2 * kStage > kExchange ? 2 * kStage : kExchange;
  // Where 16-byte piece c of a row of x (eight pieces) and of W (32) lies: 16 rows of a piece of x,
  // and four rows of four neighbouring pieces of W, are on different banks.
  static __device__ inline int x_place(int row, int c) { return c ^ ((row >> 1) & 7); }
  static __device__ inline int w_place(int row, int c) { return c ^ ((row & 3) << 2); }
};

template <bool INT4, int TT>
__global__ __launch_bounds__((Many<INT4, TT>::kThreads), 2) void gemm_many_kernel(GemmArgs a) {
  using M = Many<INT4, TT>;
  extern __shared__ __attribute__((aligned(256))) uint8_t stages[];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int h = lane >> 5, r = lane & 31;
  const int per_xcd = gridDim.x >> 3;
  const int item = (blockIdx.x & 7) * per_xcd + (blockIdx.x >> 3);
  const int m_tile = item % a.row_tiles, rest = item / a.row_tiles;
  const int split = rest % a.splits, c_tile = rest / a.splits;
  if (c_tile >= a.col_tiles) return;
  const int m0 = M::kRows * m_tile;

  const int steps = (a.k + M::kDepth - 1) / M::kDepth;
  const int first = split * a.steps;
  const int stop = first + a.steps < steps ? first + a.steps : steps;

  // A thread's pieces of a step: of x by rows, of W by k.
  constexpr int kXLoads = M::kX / 16 / M::kThreads, kWLoads = INT4 ? 1 : M::kW / 16 / M::kThreads;
  const f16* x_from[kXLoads];
#pragma unroll
  for (int i = 0; i < kXLoads; ++i) {
    const int e = (wave * kXLoads + i) * 64 + lane, row = e / 8, at = e % 8;
    const int m = m0 + row < a.rows ? m0 + row : a.rows - 1;
    x_from[i] = a.x + m * a.xs + 8 * M::x_place(row, at);
  }
  int w_row[kWLoads];
  const uint8_t* w_from[kWLoads];
  const uint8_t* sz_from = nullptr;
#pragma unroll
  for (int i = 0; i < kWLoads; ++i) {
    const int e = (wave * kWLoads + i) * 64 + lane;
    w_row[i] = INT4 ? e / 8 : e / 32;
    const int c = INT4 ? 32 * (e % 8) : 8 * M::w_place(w_row[i], e % 32);
    const int col = has_col(a, c_tile, c >> 7, c & 127) ? first_col(a, c_tile, c >> 7) + (c & 127) : 0;
    w_from[i] = a.w + (INT4 ? col / 2 : 2 * (int64_t)col);
    if constexpr (INT4) sz_from = a.w + a.n / 2 + col / 128 * 4;
  }
  const Widen widen;
  u32x4 codes = {};
  uint32_t sz = 0;
  const auto load = [&](int step) {
    uint8_t* stage = stages + (step & 1) * M::kStage;
    const int k0 = step * M::kDepth;
    if (k0 + M::kDepth <= a.k) {
#pragma unroll
      for (int i = 0; i < kXLoads; ++i)
        load_lds(x_from[i] + k0, stage + (wave * kXLoads + i) * 1024);
    } else {  // past the last k, zeros
#pragma unroll
      for (int i = 0; i < kXLoads; ++i) {
        const int e = (wave * kXLoads + i) * 64 + lane;
        const int valid = a.k - k0 - 8 * M::x_place(e / 8, e % 8);
        u32x4 v = {0u, 0u, 0u, 0u};
        if (valid > 0) v = *reinterpret_cast<const u32x4*>(x_from[i] + k0);
#pragma unroll
        for (int y = 0; y < 4; ++y)
          v[y] &= 2 * y + 1 < valid ? ~0u : 2 * y < valid ? 0xffffu : 0u;
        *reinterpret_cast<u32x4*>(stage + 16 * e) = v;
      }
    }
#pragma unroll
    for (int i = 0; i < kWLoads; ++i) {
      // past the last record: that one again, until clear_tail or lay_out
      const int k = k0 + w_row[i] < a.k ? k0 + w_row[i] : a.k - 1;
      const int64_t at = (int64_t)k * a.w_stride;
      if constexpr (INT4) {
        codes = *reinterpret_cast<const u32x4*>(w_from[i] + at);
        sz = *reinterpret_cast<const uint32_t*>(sz_from + at);
      } else {
        load_lds(w_from[i] + at, stage + M::kX + (wave * kWLoads + i) * 1024);
      }
    }
  };
  // The last step's weights past the last record are zeros (0 * inf is NaN): each thread clears what it
  // had loaded there, once that has come.
  const auto clear_tail = [&](int step) {
    if (INT4 || (step + 1) * M::kDepth <= a.k) return;
#pragma unroll
    for (int i = 0; i < kWLoads; ++i)
      if (step * M::kDepth + w_row[i] >= a.k)
        *reinterpret_cast<u32x4*>(stages + (step & 1) * M::kStage + M::kX +
                                  16 * ((wave * kWLoads + i) * 64 + lane)) = u32x4{0u, 0u, 0u, 0u};
  };
  const auto lay_out = [&](int step) {
    if constexpr (INT4) {
      const int e = wave * 64 + lane, row = e / 8;
      uint8_t* to = stages + (step & 1) * M::kStage + M::kX + row * (2 * kCols);
      // past the last record, scale and zero 0 (here and not in load, which would wait for them:
      // 4096 x 4096 x 22016 809 us, 896 there)
      const uint32_t words = step * M::kDepth + w_row[0] < a.k ? sz : 0u;
      const uint32_t s = __builtin_amdgcn_perm(words, words, 0x05040504u);
      const uint32_t z = __builtin_amdgcn_perm(words, words, 0x07060706u);
#pragma unroll
      for (int y = 0; y < 4; ++y)
        *reinterpret_cast<u32x4*>(to + 16 * M::w_place(row, 4 * (e % 8) + y)) =
            widen8(widen, codes[y], __builtin_bit_cast(f16x2, s), __builtin_bit_cast(f16x2, z));
    }
  };

  const int wm = wave >> 2, wn = wave & 3;
  f32x16 acc[2][TT];
#pragma unroll
  for (int f = 0; f < 2; ++f)
#pragma unroll
    for (int t = 0; t < TT; ++t) acc[f][t] = f32x16{};
  // The operands of 16 k, and the products with them.
  u32x4 x[2][TT], w[2][2];
  const auto read = [&](int step, int c) {
    const uint8_t* xs = stages + (step & 1) * M::kStage;
    const uint8_t* ws = xs + M::kX;
#pragma unroll
    for (int f = 0; f < 2; ++f) {
      const int i = lane & 15, g = lane >> 4;
      const int row = 16 * c + 8 * (g >> 1) + (i >> 2);
      const int piece = 16 * f + 4 * wn + 2 * (g & 1) + ((i & 3) >> 1);
      const uint8_t* p = ws + row * (2 * kCols) + 16 * M::w_place(row, piece) + 8 * (i & 1);
      const u32x2 lo = read_turned(p), hi = read_turned(p + 4 * 2 * kCols);
      w[c & 1][f] = u32x4{lo.x, lo.y, hi.x, hi.y};
    }
#pragma unroll
    for (int t = 0; t < TT; ++t) {
      const int row = 32 * (wm * TT + t) + r;
      x[c & 1][t] = *reinterpret_cast<const u32x4*>(xs + row * (2 * M::kDepth) +
                                                    16 * M::x_place(row, 2 * c + h));
    }
  };
  const auto multiply = [&](int c) {
#pragma unroll
    for (int t = 0; t < TT; ++t)
#pragma unroll
      for (int f = 0; f < 2; ++f)
        acc[f][t] = __builtin_amdgcn_mfma_f32_32x32x16_f16(
            __builtin_bit_cast(f16x8, w[c & 1][f]), __builtin_bit_cast(f16x8, x[c & 1][t]),
            acc[f][t], 0, 0, 0);
  };
  constexpr int kChunks = M::kDepth / 16;
  load(first);
  lay_out(first);
  if constexpr (INT4) {
    // The waves meet before the last products of a step, when it has been read and the next one is laid
    // out, so that these run while the next step's first operands come (4096 x 22016 842 us, 894
    // when they meet between steps, then; fp16, which lays nothing out, 787 and 784).  After the last step
    // they lay out and read once more what nothing uses.
    wait_loads();
    mask::lds_barrier();
    read(first, 0);
    if (first + 1 < stop) load(first + 1);
    for (int step = first; step < stop; ++step) {
#pragma unroll
      for (int c = 0; c < kChunks; ++c) {
        if (c + 1 < kChunks) {
          read(step, c + 1);
        } else {
          lay_out(step + 1);
          wait_loads();
          mask::lds_barrier();
          read(step + 1, 0);
          if (step + 2 < stop) load(step + 2);
        }
        __builtin_amdgcn_sched_barrier(0);
        multiply(c);
      }
    }
  } else {
    for (int step = first; step < stop; ++step) {
      wait_loads();
      clear_tail(step);
      mask::lds_barrier();  // this stage is laid out, the other one has been read
      if (step + 1 < stop) load(step + 1);
      read(step, 0);
#pragma unroll
      for (int c = 0; c < kChunks; ++c) {
        if (c + 1 < kChunks) read(step, c + 1);
        __builtin_amdgcn_sched_barrier(0);
        multiply(c);
      }
    }
  }

  // The sums go to their rows through LDS, half of the rows at a time.
  float* out = reinterpret_cast<float*>(stages);
#pragma unroll
  for (int round = 0; round < 2; ++round) {
    mask::lds_barrier();
    if (wm == round) {
#pragma unroll
      for (int f = 0; f < 2; ++f)
#pragma unroll
        for (int t = 0; t < TT; ++t)
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            f32x4 v;
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = acc[f][t][4 * g + i];
            *reinterpret_cast<f32x4*>(out + (32 * t + r) * M::kPitch + 128 * f + 32 * wn + 8 * g +
                                      4 * h) = v;
          }
    }
    mask::lds_barrier();
    const bool gated = a.form == SPAX_GEMM_GATED && a.splits == 1;
    for (int e = threadIdx.x; e < 32 * TT * (gated ? 32 : 64); e += M::kThreads) {
      const int row = gated ? e / 32 : e / 64, c = 4 * (gated ? e % 32 : e % 64);
      const int m = m0 + 32 * TT * round + row;
      if (m >= a.rows || !has_col(a, c_tile, c >> 7, c & 127)) continue;
      const float* p = out + row * M::kPitch + c;
      const f32x4 t0 = *reinterpret_cast<const f32x4*>(p);
      const f32x4 t1 = gated ? *reinterpret_cast<const f32x4*>(p + 128) : t0;
      const int col = first_col(a, c_tile, c >> 7) + (c & 127);
      if (a.splits == 1)
        finish(a, m, col, t0, t1);
      else
        *reinterpret_cast<f32x4*>(a.parts + ((int64_t)split * a.rows + m) * a.n + col) = t0;
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
  const bool gated = a.form == SPAX_GEMM_GATED;
  const float* p = a.parts + (int64_t)m * a.n + col;
  const int64_t step = (int64_t)a.rows * a.n;
  f32x4 t0 = {0.0f, 0.0f, 0.0f, 0.0f}, t1 = t0;
  constexpr int kLoads = 8;  // in flight
  for (int s = 0; s < a.splits; s += kLoads) {
    f32x4 x[kLoads], y[kLoads];
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      x[i] = y[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
      if (s + i >= a.splits) continue;
      x[i] = *reinterpret_cast<const f32x4*>(p + (s + i) * step);
      if (gated) y[i] = *reinterpret_cast<const f32x4*>(p + (s + i) * step + a.width);
    }
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      t0 += x[i];
      t1 += y[i];
    }
  }
  finish(a, m, col, t0, t1);
}

template <bool INT4>
int launch_few(const GemmArgs& a, unsigned blocks, hipStream_t s) {
  using F = Few<INT4>;
  hipLaunchKernelGGL(gemm_few_kernel<INT4>, dim3(blocks), dim3(F::kThreads), F::kLds, s, a);
  SPAX_HIP_CHECK(hipGetLastError());
  return SPAX_OK;
}

template <bool INT4, int TT>
int launch_many(const GemmArgs& a, unsigned blocks, hipStream_t s) {
  using M = Many<INT4, TT>;
  hipLaunchKernelGGL((gemm_many_kernel<INT4, TT>), dim3(blocks), dim3(M::kThreads), M::kLds, s, a);
  SPAX_HIP_CHECK(hipGetLastError());
  return SPAX_OK;
}

}  // namespace

// The tile and the splits of k by what they are expected to take, in us, with one workgroup on each of 256
// compute units: rounds of workgroups, their steps, and where k is split the sums' way through
// memory and a second launch.  The times of a step are fitted to 70 products of each base, each with
// as many blobs in turn as keep the weights out of the caches: what they choose took 0.8% (fp16) and
// 0.3% (int4) longer on average than the best tile of all four.  Some of them, us, tiles of 32, 64, 128 and
// 256 rows:
//   4096 x 22016 fp16, 5 rows     39.2   49.8   51.8   61.0
//   4096 x 22016 fp16, 64 rows    61.1   54.1   56.1   63.8
//   4096 x 22016 fp16, 128 rows   97.2   82.5   60.5   68.8
//   4096 x 22016 fp16, 512 rows  241.7  167.4  171.1  127.1
//   4096 x 22016 int4, 5 rows     29.4   47.1   49.5   62.6
//   4096 x 22016 int4, 128 rows   80.2   82.2   61.8   70.7
GemmPlan gemm_plan(const spax_packed_gemm_args* a) {
  const spax_layout& L = *a->layout;
  // a tile's rows, k of a step of the workgroup, its time, fewest steps of a split
  struct Kind {
    int32_t rows, depth;
    float step;
    int32_t least;
  };
  static const Kind kinds[2][4] = {
      {{32, 128, 2.20f, 2}, {64, 64, 1.21f, 4}, {128, 64, 1.50f, 4}, {256, 64, 2.03f, 4}},
      {{32, 128, 1.15f, 2}, {64, 64, 1.13f, 4}, {128, 64, 1.25f, 4}, {256, 64, 1.45f, 4}}};
  const bool gated = a->form == SPAX_GEMM_GATED;
  GemmPlan best{};
  if (a->n_rows < 1) return best;
  float least = 0.0f;
  for (const Kind& kind : kinds[L.base_fmt == SPAX_FMT_INT4]) {
    GemmPlan p{};
    p.tile = kind.rows;
    p.row_tiles = (a->n_rows + p.tile - 1) / p.tile;
    p.col_tiles = (int32_t)(gated ? (L.d_out[0] + 127) / 128 : (L.d_out_total + kCols - 1) / kCols);
    const int64_t items = (int64_t)p.row_tiles * p.col_tiles;
    const int32_t steps = (L.d_in + kind.depth - 1) / kind.depth;
    const float join = 8.0f * a->n_rows * (float)L.d_out_total / 4e6f;  // a split's sums there and back
    for (int32_t splits = 1; splits <= 32 && (splits == 1 || items * (splits - 1) < 256); ++splits) {
      const int32_t each = (steps + splits - 1) / splits;
      if (splits > 1 && each < kind.least) break;
      const float rounds = (float)((items * splits + 255) / 256);
      const float us = rounds * (4.0f + each * kind.step) + (splits > 1 ? 5.0f + splits * join : 0.0f);
      if (best.tile && us >= least) continue;
      least = us;
      p.splits = (steps + each - 1) / each;
      p.steps = each * (kind.depth / (p.tile == 32 ? kStep : kind.depth));
      p.blocks = (items * p.splits + 7) / 8 * 8;
      best = p;
    }
  }
  if (best.splits > 1)
    best.ws_bytes = aligned_size((size_t)best.splits * a->n_rows * L.d_out_total * sizeof(float));
  return best;
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
  a.steps = plan.steps;
  const bool int4 = L.base_fmt == SPAX_FMT_INT4;
  const unsigned blocks = (unsigned)plan.blocks;
  int st = SPAX_OK;
  switch (plan.tile) {
    case 32: st = int4 ? launch_few<true>(a, blocks, s) : launch_few<false>(a, blocks, s); break;
    case 64: st = int4 ? launch_many<true, 1>(a, blocks, s) : launch_many<false, 1>(a, blocks, s); break;
    case 128: st = int4 ? launch_many<true, 2>(a, blocks, s) : launch_many<false, 2>(a, blocks, s); break;
    default: st = int4 ? launch_many<true, 4>(a, blocks, s) : launch_many<false, 4>(a, blocks, s); break;
  }
  if (st || a.splits == 1) return st;
  const int64_t items = (int64_t)a.rows * (a.width / 4);
  hipLaunchKernelGGL(gemm_join_kernel, dim3((unsigned)((items + kJoinThreads - 1) / kJoinThreads)),
                     dim3(kJoinThreads), 0, s, a);
  SPAX_HIP_CHECK(hipGetLastError());
  return SPAX_OK;
}

}  // namespace spax
