// Element types of the operators between the projections: loads, stores and conversions.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "spax.h"

namespace spax {
namespace elem {

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef _Float16 f16;
typedef __bf16 bf16;
typedef f16 f16x2 __attribute__((ext_vector_type(2)));
typedef bf16 bf16x2 __attribute__((ext_vector_type(2)));

inline __host__ __device__ int bytes_of(int type) {
  return type == SPAX_F32 ? 4 : type == SPAX_E4M3 ? 1 : 2;
}

// A vector at any address that is aligned to two bytes (global memory takes such accesses whole).
template <class V>
__device__ inline V load_any(const void* p) {
  typedef V U __attribute__((aligned(2)));
  return *reinterpret_cast<const U*>(p);
}
template <class V>
__device__ inline void store_any(void* p, V v) {
  typedef V U __attribute__((aligned(2)));
  *reinterpret_cast<U*>(p) = v;
}

// N values from p (aligned to an element).
template <int N, class T>
__device__ inline void store_n(T* p, const float* v) {
  typedef T TN __attribute__((ext_vector_type(N)));
  TN x;
#pragma unroll
  for (int i = 0; i < N; ++i) x[i] = (T)v[i];
  store_any(p, x);
}

// E4M3 values, kept as bytes.  Stored values are clamped to +-448 before (the conversion alone would
// turn a value past the range into NaN); NaN passes.
struct e4m3 {
  uint8_t bits;
};
constexpr float kE4m3Max = 448.0f;
__device__ inline float clamp_e4m3(float v) {
  v = v > kE4m3Max ? kE4m3Max : v;
  return v < -kE4m3Max ? -kE4m3Max : v;
}
__device__ inline uint32_t pack_e4m3(const float v[4]) {
  int w = __builtin_amdgcn_cvt_pk_fp8_f32(v[0], v[1], 0, false);
  w = __builtin_amdgcn_cvt_pk_fp8_f32(v[2], v[3], w, true);
  return (uint32_t)w;
}
// N a multiple of four, p aligned to four bytes.
template <int N>
__device__ inline void store_n(e4m3* p, const float* v) {
  typedef uint32_t W __attribute__((ext_vector_type(N / 4), aligned(4)));
  W w;
#pragma unroll
  for (int i = 0; i < N / 4; ++i) w[i] = pack_e4m3(v + 4 * i);
  *reinterpret_cast<W*>(p) = w;
}
template <class T>
__device__ inline void store1(T* p, float v) {
  *p = (T)v;
}
__device__ inline void store1(e4m3* p, float v) {
  p->bits = (uint8_t)__builtin_amdgcn_cvt_pk_fp8_f32(v, 0.0f, 0, false);
}

}  // namespace elem
}  // namespace spax
