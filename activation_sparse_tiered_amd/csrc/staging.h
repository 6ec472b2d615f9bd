// Tiles staged in LDS for matrix instructions: loads from memory straight to LDS, and reads that turn
// what lies there by rows.
#pragma once

#include "elem.h"

namespace spax {
namespace staging {

using namespace elem;

// 16 bytes a lane from memory to LDS, lane after lane from `to` (uniform) on.  By hand, since the
// compiler lets every later LDS access wait for such a load; wait_loads() does before a barrier.
__device__ inline void load_lds(const void* from, const void* to) {
  const uint32_t at = __builtin_amdgcn_readfirstlane(
      (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) uint8_t*)to);
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off"
               :
               : "s"(at), "v"(from)
               : "memory", "m0");
}
__device__ inline void wait_loads() { asm volatile("s_waitcnt vmcnt(0)" : : : "memory"); }

// Four rows of one column per lane: rows from p's on of 16 columns for every 16 lanes.
__device__ inline u32x2 read_turned(const uint8_t* p) {
  typedef short v4 __attribute__((ext_vector_type(4)));
  typedef __attribute__((address_space(3))) v4 lds_v4;
  return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4*)p));
}

}  // namespace staging
}  // namespace spax
