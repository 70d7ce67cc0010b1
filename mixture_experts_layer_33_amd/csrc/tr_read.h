// Copies and transposing LDS reads of products whose reduction index is their operands' row
// (the backward's dgrad and weight gradients, the scored router's dW_r).
#pragma once

#include "common.h"

namespace moe {

// Global -> LDS copy of 16 bytes per lane from a per-lane address (the wave's 64
// lanes fill 1 KB of LDS at m0 + lane * 16), and a wait for this wave's copies.
__device__ __forceinline__ void dma16_at(const void* addr, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %1\n\tglobal_load_lds_dwordx4 %0, off"
               ::"v"(addr), "s"(lds) : "memory", "m0");
}
template <int N>
__device__ __forceinline__ void bwait_vm() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}
__device__ __forceinline__ int wsw(int r, int c) { return c ^ ((r & 3) << 2); }
typedef short v4i16_t __attribute__((ext_vector_type(4)));
__device__ __forceinline__ v4i16_t ds_tr16(const uint8_t* lds_ptr) {
  typedef __attribute__((address_space(3))) v4i16_t lds_v4;
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16(
      (lds_v4*)((__attribute__((address_space(3))) uint8_t*)lds_ptr));
}

}  // namespace moe
