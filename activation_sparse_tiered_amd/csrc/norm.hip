// spax_residual_norm: a block's output joins the residual stream and the next input leaves it.
//
//   t = norm(block) * gate,   h = residual + scale t,   x = norm(h)
//   norm(v) = (v - c) w / sqrt(mean (v - c)^2 + eps) + b,   c = 0 (RMS) or mean v (layer)
//
// Bound: bytes for many rows, the latency of two reductions for one.  A workgroup holds a whole
// row in registers, so every value is read once and written once; the centred sum of squares
// is a second pass over registers, with none of the cancellation of mean v^2 - mean^2.  One row
// per workgroup: walking over several rows with the weights in registers was slower (17.7 to 23 us
// against 15.8 for 2048 rows).
//
// Measured: 2048 x 4096 bf16, norms before and after and a gate: 14.6 us, 67 MB, 4.6 TB/s (a large
// copy reaches 5.1).  333 x 5003, layer norms, rows that start anywhere: 9.1 us, four sums one after
// another (256 rows 6.3 us: the rest is units that have two rows).  1 x 4096: 2.4 us on the device.
#include "layer_ops.h"
#include "mask_core.h"

namespace spax {
namespace {

using namespace elem;

struct NormArgs {
  const void *residual, *block, *gate;
  void *residual_out, *x;
  const float *post_w, *post_b, *pre_w, *pre_b;
  int64_t r_stride, b_stride, ro_stride, x_stride, g_stride;
  int32_t r_type, b_type, g_type, x_type, layer, d;
  float scale, eps, inv_d;
};

// Eight values as loaded, before conversion, so that several rows' loads are in flight at once.
struct Raw {
  u32x4 a, b;
};

// Thread's item j: eight values from element `at`, of which those before `lo` are not its own.
// Rows need not start on eight elements: the hardware reads 16 bytes from any address (of an
// element here).  The last item of a row whose width is not a multiple of eight is the row's last
// eight values, the first ones its neighbour's: those count as 0 in sums and are not stored, so it
// does not matter if the neighbour has overwritten them.  (With its own values read one by one,
// 333 x 5003 took 11.0 us.)  Items past the row own nothing (lo 8).  A row of fewer than eight
// values (TINY) is one item that starts at 0 and ends at d.
struct Item {
  int at, lo;
};
template <bool TINY>
__device__ inline Item item_of(int d, int j) {
  const int e = (j * (int)blockDim.x + (int)threadIdx.x) * 8;
  if (TINY) return Item{0, e ? 8 : 0};
  const int at = e + 8 <= d ? e : d - 8;
  return Item{at, e >= d ? 8 : e - at};
}

template <bool TINY>
__device__ inline void load_raw(const void* row, int type, int d, const Item& it, Raw& w) {
  if (it.lo == 8) return;
  if constexpr (TINY) {
#pragma unroll
    for (int i = 0; i < 7; ++i) {
      const int k = i < d ? i : d - 1;
      const uint32_t u =
          type == SPAX_F32 ? ((const uint32_t*)row)[k] : (uint32_t)((const uint16_t*)row)[k];
      if (type == SPAX_F32) {
        if (i < 4) w.a[i % 4] = u; else w.b[i % 4] = u;
      } else {
        w.a[i / 2] = i % 2 ? w.a[i / 2] | u << 16 : u;
      }
    }
  } else if (type == SPAX_F32) {
    w.a = load_any<u32x4>((const float*)row + it.at);
    w.b = load_any<u32x4>((const float*)row + it.at + 4);
  } else {
    w.a = load_any<u32x4>((const uint16_t*)row + it.at);
  }
}

__device__ inline float from_bits(uint32_t u, int type) {
  if (type == SPAX_F32) return __builtin_bit_cast(float, u);
  if (type == SPAX_F16) return (float)__builtin_bit_cast(f16, (uint16_t)u);
  return __builtin_bit_cast(float, u << 16);
}

// An item's values as loaded by load_raw, those that are not its own included.
__device__ inline void unpack(const Raw& w, int type, float v[8]) {
  if (type == SPAX_F32) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[i] = from_bits(w.a[i], SPAX_F32);
      v[4 + i] = from_bits(w.b[i], SPAX_F32);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (type == SPAX_F16) {
        v[2 * i] = from_bits(w.a[i] & 0xffffu, SPAX_F16);
        v[2 * i + 1] = from_bits(w.a[i] >> 16, SPAX_F16);
      } else {
        v[2 * i] = from_bits(w.a[i], SPAX_BF16);
        v[2 * i + 1] = __builtin_bit_cast(float, (uint32_t)w.a[i] & 0xffff0000u);
      }
    }
  }
}

// Zeros in place of values that are not the item's.
template <bool TINY>
__device__ inline void keep_own(float v[8], int d, const Item& it) {
  if constexpr (TINY) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = it.lo == 0 && i < d ? v[i] : 0.0f;
  } else if (it.lo) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i >= it.lo ? v[i] : 0.0f;
  }
}

template <class T, bool TINY>
__device__ inline void store8(T* row, int d, const Item& it, const float v[8]) {
  if (!TINY && it.lo == 0) {
    typedef T T8 __attribute__((ext_vector_type(8)));
    T8 x;
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = (T)v[i];
    store_any(row + it.at, x);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i >= it.lo && (!TINY || i < d)) row[it.at + i] = (T)v[i];
  }
}

template <bool TINY>
__device__ inline void store_row(void* p, int type, int64_t at, int d, const Item& it,
                                 const float v[8]) {
  if (type == SPAX_F32) store8<float, TINY>((float*)p + at, d, it, v);
  else if (type == SPAX_F16) store8<f16, TINY>((f16*)p + at, d, it, v);
  else store8<bf16, TINY>((bf16*)p + at, d, it, v);
}

__device__ inline const void* row_at(const void* p, int type, int64_t at) {
  return (const uint8_t*)p + at * (type == SPAX_F32 ? 4 : 2);
}

// Sum over the lanes of a wave, in every lane (row shifts, then row broadcasts, as for a scan).
__device__ inline float wave_sum(float v) {
#define SPAX_STEP(ctrl, rows)                                                                  \
  v += __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v),    \
                                                             ctrl, rows, 0xF, false))
  SPAX_STEP(0x111, 0xF);
  SPAX_STEP(0x112, 0xF);
  SPAX_STEP(0x114, 0xF);
  SPAX_STEP(0x118, 0xF);
  SPAX_STEP(0x142, 0xA);
  SPAX_STEP(0x143, 0xC);
#undef SPAX_STEP
  return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), 63));
}

// Sum over the workgroup, the same bits in every thread.  slot: 16 floats of LDS that no wave may
// still be reading.  The barrier orders LDS only, so loads stay in flight.
__device__ inline float sum_all(float v, float* slot) {
  v = wave_sum(v);
  const int waves = blockDim.x >> 6, lane = threadIdx.x & 63;
  if (lane == 0) slot[threadIdx.x >> 6] = v;
  mask::lds_barrier();
  // every row of 16 lanes adds up the waves' sums
  v = (lane & 15) < waves ? slot[lane & 15] : 0.0f;
#define SPAX_TURN(by)                                                                          \
  v += __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v),    \
                                                             0x120 + by, 0xF, 0xF, false))
  SPAX_TURN(8);
  SPAX_TURN(4);
  SPAX_TURN(2);
  SPAX_TURN(1);
#undef SPAX_TURN
  return __builtin_bit_cast(float, __builtin_amdgcn_readfirstlane(__builtin_bit_cast(int, v)));
}

// v <- norm(v) without weight; values that are not the items' own become 0.
template <int NV, bool TINY>
__device__ inline void normalise(float (*v)[8], const NormArgs& a, const Item* it, float* slot) {
#pragma unroll
  for (int j = 0; j < NV; ++j) keep_own<TINY>(v[j], a.d, it[j]);
  if (a.layer) {
    float s = 0.0f;
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int i = 0; i < 8; ++i) s += v[j][i];
    const float mean = sum_all(s, slot) * a.inv_d;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[j][i] -= mean;
      keep_own<TINY>(v[j], a.d, it[j]);
    }
  }
  float s = 0.0f;
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int i = 0; i < 8; ++i) s += v[j][i] * v[j][i];
  const float f = 1.0f / sqrtf(sum_all(s, slot + 16) * a.inv_d + a.eps);
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int i = 0; i < 8; ++i) v[j][i] *= f;
}

// v <- v * weight + bias; w and b hold them (EARLY) or are loaded here, an item at a time.
template <int NV, bool EARLY, bool TINY>
__device__ inline void weigh(float (*v)[8], const NormArgs& a, const Item* it, const float* weight,
                             const float* bias, Raw* w, Raw* b) {
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int k = EARLY ? j : 0;
    if (!EARLY && weight) load_raw<TINY>(weight, SPAX_F32, a.d, it[j], w[k]);
    if (!EARLY && bias) load_raw<TINY>(bias, SPAX_F32, a.d, it[j], b[k]);
    float x[8];
    if (weight) {
      unpack(w[k], SPAX_F32, x);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[j][i] *= x[i];
    }
    if (bias) {
      unpack(b[k], SPAX_F32, x);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[j][i] += x[i];
    }
  }
}

template <bool TINY>
__device__ inline void load_block(const NormArgs& a, int64_t row, const Item& it, Raw& b) {
  if (a.block)
    load_raw<TINY>(row_at(a.block, a.b_type, row * a.b_stride), a.b_type, a.d, it, b);
}
template <bool TINY>
__device__ inline void load_stream(const NormArgs& a, int64_t row, const Item& it, Raw& r, Raw& g) {
  if (a.residual)
    load_raw<TINY>(row_at(a.residual, a.r_type, row * a.r_stride), a.r_type, a.d, it, r);
  if (a.gate) load_raw<TINY>(row_at(a.gate, a.g_type, row * a.g_stride), a.g_type, a.d, it, g);
}

// One row per workgroup, NV items per thread.  Up to two items everything a row needs is loaded at
// once; wider rows (128 registers for each of 1024 threads) load residual, gate and weights when
// they are used.
template <int NV, bool TINY>
__global__ __launch_bounds__(1024) void residual_norm_kernel(NormArgs a) {
  constexpr bool EARLY = NV <= 2;
  __shared__ float slots[64];  // (post, pre) x (mean, square) x 16 waves
  Raw rb[NV], rr[NV], rg[NV], w[NV], b[NV];
  Item it[NV];
  const int64_t row = blockIdx.x;
#pragma unroll
  for (int j = 0; j < NV; ++j) it[j] = item_of<TINY>(a.d, j);
  const auto load_weights = [&](const float* weight, const float* bias) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if (weight) load_raw<TINY>(weight, SPAX_F32, a.d, it[j], w[j]);
      if (bias) load_raw<TINY>(bias, SPAX_F32, a.d, it[j], b[j]);
    }
  };
#pragma unroll
  for (int j = 0; j < NV; ++j) load_block<TINY>(a, row, it[j], rb[j]);
  if (EARLY) {
#pragma unroll
    for (int j = 0; j < NV; ++j) load_stream<TINY>(a, row, it[j], rr[j], rg[j]);
    load_weights(a.post_w, a.post_b);
  }
  float v[NV][8];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[j][i] = 0.0f;
    if (a.block) unpack(rb[j], a.b_type, v[j]);
  }
  if (a.post_w && a.block) {
    normalise<NV, TINY>(v, a, it, slots);
    weigh<NV, EARLY, TINY>(v, a, it, a.post_w, a.post_b, w, b);
  }
  if (EARLY) load_weights(a.pre_w, a.pre_b);
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    if (!EARLY) load_stream<TINY>(a, row, it[j], rr[0], rg[0]);
    float x[8];
    if (a.gate) {
      unpack(rg[EARLY ? j : 0], a.g_type, x);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[j][i] *= x[i];
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = 0.0f;
    if (a.residual) unpack(rr[EARLY ? j : 0], a.r_type, x);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[j][i] = x[i] + a.scale * v[j][i];
    if (a.residual_out)
      store_row<TINY>(a.residual_out, a.r_type, row * a.ro_stride, a.d, it[j], v[j]);
  }
  if (!a.x) return;
  normalise<NV, TINY>(v, a, it, slots + 32);
  weigh<NV, EARLY, TINY>(v, a, it, a.pre_w, a.pre_b, w, b);
#pragma unroll
  for (int j = 0; j < NV; ++j)
    store_row<TINY>(a.x, a.x_type, row * a.x_stride, a.d, it[j], v[j]);
}

}  // namespace

int launch_residual_norm(const spax_residual_norm_args* p, hipStream_t s) {
  if (p->n_rows == 0) return SPAX_OK;
  NormArgs a{};
  a.residual = p->residual; a.block = p->block; a.gate = p->gate;
  a.residual_out = p->residual_out; a.x = p->x;
  a.post_w = p->post_weight; a.post_b = p->post_bias;
  a.pre_w = p->pre_weight; a.pre_b = p->pre_bias;
  a.r_stride = p->residual_stride; a.b_stride = p->block_stride;
  a.ro_stride = p->residual_out_stride; a.x_stride = p->x_stride; a.g_stride = p->gate_stride;
  a.r_type = p->residual_type; a.b_type = p->block_type; a.g_type = p->gate_type;
  a.x_type = p->x_type; a.layer = p->kind == SPAX_NORM_LAYER; a.d = p->d;
  a.scale = p->scale; a.eps = p->eps; a.inv_d = 1.0f / (float)p->d;
  // Items of a thread: one while 1024 threads hold the row (333 x 5003: 9.2 us, 12.1 with two);
  // then two while a compute unit has one row (1 x 12891: 6.2 us, 7.7 with four), else four,
  // whose fewer threads let a unit hold more rows (256 x 16384: 12.7 with two, 13.5 with four;
  // 257 x 12891: 16.5 and 13.3; 2048 x 16384: 106 and 94).
  const int items = (p->d + 7) / 8;
  const int nv = items <= 1024 ? 1 : items <= 2048 && p->n_rows <= 256 ? 2 : 4;
  const unsigned threads = (unsigned)(((items + nv - 1) / nv + 63) / 64 * 64);
  const dim3 grid((unsigned)p->n_rows), block(threads);
  if (p->d < 8)
    hipLaunchKernelGGL((residual_norm_kernel<1, true>), grid, block, 0, s, a);
  else if (nv == 1)
    hipLaunchKernelGGL((residual_norm_kernel<1, false>), grid, block, 0, s, a);
  else if (nv == 2)
    hipLaunchKernelGGL((residual_norm_kernel<2, false>), grid, block, 0, s, a);
  else
    hipLaunchKernelGGL((residual_norm_kernel<4, false>), grid, block, 0, s, a);
  SPAX_HIP_CHECK(hipGetLastError());
  return SPAX_OK;
}

}  // namespace spax
