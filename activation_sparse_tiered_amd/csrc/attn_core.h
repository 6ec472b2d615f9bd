// What the attentions share: matrix instructions by element type, and the sums' logarithm.
#pragma once

#include "elem.h"

namespace spax {
namespace attn {

using namespace elem;

typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;

// kLift: the exponentials are taken of s - m + kLift (base 2), so the largest is 2^kLift, the most
// that fp16 holds with room for its rounding and 2^-13 of the base's.  It cancels in o / l, and lse takes it off again.
template <class T>
struct Mma;
template <>
struct Mma<f16> {
  static constexpr float kLift = 15.0f, kUnlift = 0x1p-15f;
  typedef f16 v8 __attribute__((ext_vector_type(8)));
  static __device__ inline f32x4 mul(u32x4 a, u32x4 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8, a),
                                                  __builtin_bit_cast(v8, b), c, 0, 0, 0);
  }
  static __device__ inline f32x16 mul32(u32x4 a, u32x4 b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(v8, a),
                                                  __builtin_bit_cast(v8, b), c, 0, 0, 0);
  }
  static constexpr uint32_t kExpStep = 0x04000400u;  // carries a full exponent into the sign bit
  // two e4m3 values (the low or high half of w) as 16-bit ones, exactly
  template <bool HI>
  static __device__ inline uint32_t widen(uint32_t w) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, HI));
  }
  typedef f16x2 v2;
};
template <>
struct Mma<bf16> {
  static constexpr float kLift = 0.0f, kUnlift = 1.0f;
  typedef bf16 v8 __attribute__((ext_vector_type(8)));
  static __device__ inline f32x4 mul(u32x4 a, u32x4 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8, a),
                                                   __builtin_bit_cast(v8, b), c, 0, 0, 0);
  }
  static __device__ inline f32x16 mul32(u32x4 a, u32x4 b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(v8, a),
                                                   __builtin_bit_cast(v8, b), c, 0, 0, 0);
  }
  static constexpr uint32_t kExpStep = 0x00800080u;
  template <bool HI>
  static __device__ inline uint32_t widen(uint32_t w) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, HI));
  }
  typedef bf16x2 v2;
};

// ln of the sum of exponentials whose largest exponent is m (base 2) and whose lifted sum is l.
template <class T>
__device__ inline float lse_of(float m, float l) {
  return l == 0.0f ? -INFINITY : (m + log2f(l * Mma<T>::kUnlift)) * kLn2;
}

}  // namespace attn
}  // namespace spax
