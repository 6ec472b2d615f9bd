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

template <class T>
__device__ inline float to_float(T v) {
  return (float)v;
}

// Four values at p, which is aligned to four elements.
template <class T>
__device__ inline void load4(const T* p, float v[4]) {
  typedef T T4 __attribute__((ext_vector_type(4)));
  const T4 x = *reinterpret_cast<const T4*>(p);
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = (float)x[i];
}

template <class T>
__device__ inline void store4(T* p, const float v[4]) {
  typedef T T4 __attribute__((ext_vector_type(4)));
  T4 x;
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = (T)v[i];
  *reinterpret_cast<T4*>(p) = x;
}

// E4M3 values, kept as bytes: clamped to +-448 first (the conversion alone would turn a value
// past the range into NaN); NaN passes.
struct e4m3 {
  uint8_t bits;
};
__device__ inline float clamp_e4m3(float v) {
  v = v > 448.0f ? 448.0f : v;
  return v < -448.0f ? -448.0f : v;
}
__device__ inline void store4(e4m3* p, const float v[4]) {
  int w = __builtin_amdgcn_cvt_pk_fp8_f32(clamp_e4m3(v[0]), clamp_e4m3(v[1]), 0, false);
  w = __builtin_amdgcn_cvt_pk_fp8_f32(clamp_e4m3(v[2]), clamp_e4m3(v[3]), w, true);
  *reinterpret_cast<int*>(p) = w;
}
template <class T>
__device__ inline void store1(T* p, float v) {
  *p = (T)v;
}
__device__ inline void store1(e4m3* p, float v) {
  p->bits = (uint8_t)__builtin_amdgcn_cvt_pk_fp8_f32(clamp_e4m3(v), 0.0f, 0, false);
}

}  // namespace elem
}  // namespace spax
