// Loads from global memory straight into LDS.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace muon {

typedef int32_t fi32x4 __attribute__((ext_vector_type(4)));

// Buffer resource over [p, p + 2 GiB), p the same in every lane.
__device__ __forceinline__ fi32x4 f_buffer(uint64_t p) {
  fi32x4 r;
  r[0] = __builtin_amdgcn_readfirstlane((int32_t)(uint32_t)p);
  r[1] = __builtin_amdgcn_readfirstlane((int32_t)(uint32_t)(p >> 32));
  r[2] = (int32_t)0x80000000u;
  r[3] = 0x00020000;
  return r;
}
constexpr uint32_t kFfnNowhere = 0x80000000u;  // outside every such buffer: reads as zero

// One 16-byte buffer→LDS load per lane: lane l writes lds_base + 16·l.
__device__ __forceinline__ void f_dma16(uint32_t lds_base, uint32_t off, fi32x4 rsrc) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
               :
               : "s"(lds_base), "v"(off), "s"(rsrc)
               : "memory", "m0");
}

}  // namespace muon
