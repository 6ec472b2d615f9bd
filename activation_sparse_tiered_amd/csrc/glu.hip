// spax_glu: x = act(gate) * up, act(g) = g / (1 + exp(-g)) or the tanh form of gelu.
//
// The tanh form is the same with another argument: (1 + tanh u) / 2 = 1 / (1 + exp(-2u)), so
// act(g) = g / (1 + exp(-2u)), u = sqrt(2/pi) (g + 0.044715 g^3): no cancellation near tanh = -1.
// Bound: bytes (three rows move, nothing is reused) or, for one row, launch latency.
#include "layer_ops.h"

namespace spax {
namespace {

using namespace elem;

constexpr int kGluThreads = 256;

struct GluArgs {
  const void *gate, *up;
  void* x;
  int64_t gs, us, xs;
  int32_t d, gelu, blocks_per_row;
};

__device__ inline float act(float g, bool gelu) {
  float u = g;
  if (gelu) {
    constexpr float kTwoRootTwoOverPi = 1.59576912160573071176f;
    u = kTwoRootTwoOverPi * (g + 0.044715f * g * g * g);
  }
  // exp(-u) overflows to inf below u = -88: g / inf = -0, the limit
  return g / (1.0f + expf(-u));
}

template <class SRC, class X, bool VEC>
__global__ __launch_bounds__(kGluThreads) void glu_kernel(GluArgs a) {
  const int64_t row = blockIdx.x / (unsigned)a.blocks_per_row;
  const int part = blockIdx.x % (unsigned)a.blocks_per_row;
  const SRC* gate = (const SRC*)a.gate + row * a.gs;
  const SRC* up = (const SRC*)a.up + row * a.us;
  X* x = (X*)a.x + row * a.xs;
  const int e = (part * kGluThreads + (int)threadIdx.x) * 8;
  if constexpr (VEC) {
    if (e + 8 <= a.d) {
      float g[8], u[8];
      load4(gate + e, g);
      load4(gate + e + 4, g + 4);
      load4(up + e, u);
      load4(up + e + 4, u + 4);
#pragma unroll
      for (int i = 0; i < 8; ++i) g[i] = act(g[i], a.gelu) * u[i];
      store4(x + e, g);
      store4(x + e + 4, g + 4);
      return;
    }
    for (int i = e; i < a.d && i < e + 8; ++i)
      x[i] = (X)(act((float)gate[i], a.gelu) * (float)up[i]);
  } else {
    const int b = part * kGluThreads * 8 + (int)threadIdx.x;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int k = b + i * kGluThreads;
      if (k < a.d) x[k] = (X)(act((float)gate[k], a.gelu) * (float)up[k]);
    }
  }
}

template <class SRC, class X>
int launch(const GluArgs& a, unsigned grid, bool vec, hipStream_t s) {
  if (vec)
    hipLaunchKernelGGL((glu_kernel<SRC, X, true>), dim3(grid), dim3(kGluThreads), 0, s, a);
  else
    hipLaunchKernelGGL((glu_kernel<SRC, X, false>), dim3(grid), dim3(kGluThreads), 0, s, a);
  SPAX_HIP_CHECK(hipGetLastError());
  return SPAX_OK;
}

template <class SRC>
int launch_src(const GluArgs& a, int x_type, unsigned grid, bool vec, hipStream_t s) {
  switch (x_type) {
    case SPAX_F32: return launch<SRC, float>(a, grid, vec, s);
    case SPAX_F16: return launch<SRC, f16>(a, grid, vec, s);
    default: return launch<SRC, bf16>(a, grid, vec, s);
  }
}

}  // namespace

int launch_glu(const spax_glu_args* p, hipStream_t s) {
  if (p->n_rows == 0) return SPAX_OK;
  GluArgs a{};
  a.gate = p->gate; a.up = p->up; a.x = p->x;
  a.gs = p->gate_stride; a.us = p->up_stride; a.xs = p->x_stride;
  a.d = p->d; a.gelu = p->act == SPAX_ACT_GELU_TANH;
  a.blocks_per_row = (int32_t)(((int64_t)p->d + 8 * kGluThreads - 1) / (8 * kGluThreads));
  const size_t eb = 4 * (size_t)bytes_of(p->src_type), xb = 4 * (size_t)bytes_of(p->x_type);
  const bool vec = aligned(p->gate, eb) && aligned(p->up, eb) && aligned(p->x, xb) &&
                   (a.gs | a.us | a.xs) % 4 == 0;
  const unsigned grid = (unsigned)((int64_t)p->n_rows * a.blocks_per_row);
  switch (p->src_type) {
    case SPAX_F32: return launch_src<float>(a, p->x_type, grid, vec, s);
    case SPAX_F16: return launch_src<f16>(a, p->x_type, grid, vec, s);
    default: return launch_src<bf16>(a, p->x_type, grid, vec, s);
  }
}

}  // namespace spax
