// spax_residual_norm: a block's output joins the residual stream and the next input leaves it.
//
//   t = norm(block) * gate,   h = residual + scale t,   x = norm(h)
//   norm(v) = (v - c) w / sqrt(mean (v - c)^2 + eps) + b,   c = 0 (RMS) or mean v (layer)
//
// Bound: bytes for many rows, the latency of two reductions for one.  A workgroup holds a whole
// row in registers, so every value is read once and written once; the centred sum of squares
// is a second pass over registers, with none of the cancellation of mean v^2 - mean^2.
#include "layer_ops.h"

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

// Thread's item j: VEC: elements [e, e + 8), e = (j * threads + tid) * 8; otherwise element
// (j * 8 + i) * threads + tid for i < 8.
template <bool VEC>
__device__ inline void load_raw(const void* row, int type, int d, int j, Raw& w) {
  w.a = w.b = u32x4{0u, 0u, 0u, 0u};
  const int nt = blockDim.x;
  if constexpr (VEC) {
    const int e = (j * nt + threadIdx.x) * 8;
    if (e + 8 <= d) {
      if (type == SPAX_F32) {
        w.a = *reinterpret_cast<const u32x4*>((const float*)row + e);
        w.b = *reinterpret_cast<const u32x4*>((const float*)row + e + 4);
      } else {
        w.a = *reinterpret_cast<const u32x4*>((const uint16_t*)row + e);
      }
    } else if (e < d) {
      for (int i = 0; i < d - e; ++i) {
        if (type == SPAX_F32) {
          const uint32_t u = ((const uint32_t*)row)[e + i];
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            if (i == x) w.a[x] = u;
            if (i == x + 4) w.b[x] = u;
          }
        } else {
          const uint32_t u = (uint32_t)((const uint16_t*)row)[e + i] << (16 * (i & 1));
#pragma unroll
          for (int x = 0; x < 4; ++x)
            if (i / 2 == x) w.a[x] |= u;
        }
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int e = (j * 8 + i) * nt + (int)threadIdx.x;
      if (e < d) {
        if (type == SPAX_F32) {
          const uint32_t u = ((const uint32_t*)row)[e];
          if (i < 4) w.a[i % 4] = u; else w.b[i % 4] = u;
        } else {
          w.a[i / 2] |= (uint32_t)((const uint16_t*)row)[e] << (16 * (i & 1));
        }
      }
    }
  }
}

__device__ inline void unpack(const Raw& w, int type, float v[8]) {
  if (type == SPAX_F32) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[i] = __builtin_bit_cast(float, (uint32_t)w.a[i]);
      v[4 + i] = __builtin_bit_cast(float, (uint32_t)w.b[i]);
    }
  } else if (type == SPAX_F16) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const f16x2 h = __builtin_bit_cast(f16x2, (uint32_t)w.a[i]);
      v[2 * i] = (float)h.x;
      v[2 * i + 1] = (float)h.y;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __builtin_bit_cast(float, (uint32_t)w.a[i] << 16);
      v[2 * i + 1] = __builtin_bit_cast(float, (uint32_t)w.a[i] & 0xffff0000u);
    }
  }
}

template <class T, bool VEC>
__device__ inline void store8(T* row, int d, int j, const float v[8]) {
  const int nt = blockDim.x;
  if constexpr (VEC) {
    const int e = (j * nt + threadIdx.x) * 8;
    if (e + 8 <= d) {
      typedef T T8 __attribute__((ext_vector_type(8)));
      T8 x;
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = (T)v[i];
      *reinterpret_cast<T8*>(row + e) = x;
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (e + i < d) row[e + i] = (T)v[i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int e = (j * 8 + i) * nt + (int)threadIdx.x;
      if (e < d) row[e] = (T)v[i];
    }
  }
}

template <bool VEC>
__device__ inline void store_row(void* p, int type, int64_t at, int d, int j, const float v[8]) {
  if (type == SPAX_F32) store8<float, VEC>((float*)p + at, d, j, v);
  else if (type == SPAX_F16) store8<f16, VEC>((f16*)p + at, d, j, v);
  else store8<bf16, VEC>((bf16*)p + at, d, j, v);
}

__device__ inline const void* row_at(const void* p, int type, int64_t at) {
  return (const uint8_t*)p + at * (type == SPAX_F32 ? 4 : 2);
}

// Sum over the workgroup, the same bits in every thread.  slot: LDS of one float per wave, not
// in use by an earlier sum of this row.
__device__ inline float sum_all(float v, float* slot) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
  const int waves = blockDim.x >> 6;
  if ((threadIdx.x & 63) == 0) slot[threadIdx.x >> 6] = v;
  __syncthreads();
  float s = 0.0f;
  for (int w = 0; w < waves; ++w) s += slot[w];
  return s;
}

// v <- norm(v) without weight; elements past d are 0 and stay out of the sums.
template <int NV, bool VEC>
__device__ inline void normalise(float (*v)[8], const NormArgs& a, float* slot) {
  const int nt = blockDim.x;
  if (a.layer) {
    float s = 0.0f;
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int i = 0; i < 8; ++i) s += v[j][i];
    const float mean = sum_all(s, slot) * a.inv_d;
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int e = VEC ? (j * nt + (int)threadIdx.x) * 8 + i : (j * 8 + i) * nt + (int)threadIdx.x;
        v[j][i] = e < a.d ? v[j][i] - mean : 0.0f;
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

template <int NV, bool VEC>
__device__ inline void weigh(float (*v)[8], const Raw* w, const Raw* b, bool has_w, bool has_b) {
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    if (has_w) {
      float x[8];
      unpack(w[j], SPAX_F32, x);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[j][i] *= x[i];
    }
    if (has_b) {
      float x[8];
      unpack(b[j], SPAX_F32, x);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[j][i] += x[i];
    }
  }
}

template <int NV, bool VEC>
__global__ void residual_norm_kernel(NormArgs a) {
  __shared__ float slots[64];  // 16 waves x (post, pre) x (mean, square)
  const int64_t row = blockIdx.x;
  Raw rb[NV], rr[NV], rg[NV], rw[NV], rc[NV];
  float v[NV][8];
  const void* pb = a.block ? row_at(a.block, a.b_type, row * a.b_stride) : nullptr;
  const void* pr = a.residual ? row_at(a.residual, a.r_type, row * a.r_stride) : nullptr;
  const void* pg = a.gate ? row_at(a.gate, a.g_type, row * a.g_stride) : nullptr;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    if (pb) load_raw<VEC>(pb, a.b_type, a.d, j, rb[j]);
    if (pr) load_raw<VEC>(pr, a.r_type, a.d, j, rr[j]);
    if (pg) load_raw<VEC>(pg, a.g_type, a.d, j, rg[j]);
    if (a.post_w) load_raw<VEC>(a.post_w, SPAX_F32, a.d, j, rw[j]);
    if (a.post_b) load_raw<VEC>(a.post_b, SPAX_F32, a.d, j, rc[j]);
  }
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    if (pb) {
      unpack(rb[j], a.b_type, v[j]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[j][i] = 0.0f;
    }
  }
  if (a.post_w && pb) {
    normalise<NV, VEC>(v, a, slots);
    weigh<NV, VEC>(v, rw, rc, true, a.post_b != nullptr);
  }
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    if (a.pre_w) load_raw<VEC>(a.pre_w, SPAX_F32, a.d, j, rw[j]);
    if (a.pre_b) load_raw<VEC>(a.pre_b, SPAX_F32, a.d, j, rc[j]);
  }
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    if (pg) {
      float x[8];
      unpack(rg[j], a.g_type, x);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[j][i] *= x[i];
    }
    float x[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
    if (pr) unpack(rr[j], a.r_type, x);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[j][i] = x[i] + a.scale * v[j][i];
    if (a.residual_out)
      store_row<VEC>(a.residual_out, a.r_type, row * a.ro_stride, a.d, j, v[j]);
  }
  if (!a.x) return;
  normalise<NV, VEC>(v, a, slots + 32);
  weigh<NV, VEC>(v, rw, rc, a.pre_w != nullptr, a.pre_b != nullptr);
#pragma unroll
  for (int j = 0; j < NV; ++j) store_row<VEC>(a.x, a.x_type, row * a.x_stride, a.d, j, v[j]);
}

template <int NV>
int launch(const NormArgs& a, bool vec, unsigned rows, unsigned threads, hipStream_t s) {
  if (vec)
    hipLaunchKernelGGL((residual_norm_kernel<NV, true>), dim3(rows), dim3(threads), 0, s, a);
  else
    hipLaunchKernelGGL((residual_norm_kernel<NV, false>), dim3(rows), dim3(threads), 0, s, a);
  SPAX_HIP_CHECK(hipGetLastError());
  return SPAX_OK;
}

// A row can be read eight values at a time if every row of the buffer starts on eight.
bool wide(const void* p, int type, int64_t stride) {
  return !p || (aligned(p, 8 * (size_t)bytes_of(type) > 16 ? 16 : 8 * (size_t)bytes_of(type)) &&
                stride % 8 == 0);
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
  const bool vec = wide(a.residual, a.r_type, a.r_stride) && wide(a.block, a.b_type, a.b_stride) &&
                   wide(a.gate, a.g_type, a.g_stride) &&
                   wide(a.residual_out, a.r_type, a.ro_stride) &&
                   wide(a.x, a.x_type, a.x_stride) && wide(a.post_w, SPAX_F32, 0) &&
                   wide(a.post_b, SPAX_F32, 0) && wide(a.pre_w, SPAX_F32, 0) &&
                   wide(a.pre_b, SPAX_F32, 0);
  const int items = (p->d + 7) / 8;
  const int nv = items <= 1024 ? 1 : items <= 2048 ? 2 : 4;
  const unsigned threads = (unsigned)(((items + nv - 1) / nv + 63) / 64 * 64);
  switch (nv) {
    case 1: return launch<1>(a, vec, (unsigned)p->n_rows, threads, s);
    case 2: return launch<2>(a, vec, (unsigned)p->n_rows, threads, s);
    default: return launch<4>(a, vec, (unsigned)p->n_rows, threads, s);
  }
}

}  // namespace spax
