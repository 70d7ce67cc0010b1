// MXFP4 weights (E2M1 codes, two a byte, the even column in the low half; one E8M0 byte per 32 columns in the
// MX scale layout [cols / 128][rows][4]) as operands of the bf16 MFMA: the loads and the widening that the
// weight-stream kernels share.
//
// A wavefront takes 16 weight rows x 256 columns (a "pair" of 128-column groups) per step: two 16-byte loads a lane,
// in which eight lanes cover the 128 contiguous bytes of one row (a request for half a 128-byte line moves the
// whole of it).  The first load holds rows 0-7, the second rows 8-15; lane l has row l & 7, 16-byte chunk l >> 3,
// and a chunk is one scale block of 32 columns.  The MFMA wants row l & 15 in every lane: lanes 8 apart trade halves
// (a DPP move of eight lanes within a row of 16), after which a lane holds chunks 2g and 2g + 1 of its row (g = l >> 4).
// Which columns a lane group holds is free as long as the tokens' operand agrees, so x is read in that
// order: columns 64 g .. 64 g + 63 of the pair.
//
// The codes widen to bf16 by gfx950's v_cvt_scalef32_pk_bf16_fp4 (two codes and the block's scale in one instruction at the
// full VALU rate; checked for every byte, byte place and scale from 2^-127 up: code value x 2^(byte - 127), NaN for byte
// 255).  E2M1 x 2^X is exact in bf16, products and sums are the bf16 MFMA's in fp32.
#pragma once

#include "common.h"

namespace moe {

typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));

constexpr uint32_t RSRC_WORD3 = 0x00027000;   // raw buffer, 32-bit data
constexpr uint32_t OUTSIDE = 0xfffffff0u;      // an offset past every buffer: the load returns zeros
constexpr int NT_LOAD = 2;                     // cache policy of a buffer load: non-temporal

__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_of(const void* base, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc((void*)base, 0, (int)bytes, (int)RSRC_WORD3);
}

struct W4Pair {
  u32x4 a, b;      // rows 0-7, rows 8-15
  uint32_t s;      // the four scale bytes of row l & 15, columns 128 (g / 2) .. of the pair
};

// Four dwords of codes of one row and block -> acc += W x over the block's 32 columns of each lane group.
__device__ __forceinline__ bf16x8 widen4(uint32_t codes, float scale) {
  const bf16x2_t p0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 0);
  const bf16x2_t p1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 1);
  const bf16x2_t p2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 2);
  const bf16x2_t p3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 3);
  return bf16x8{p0[0], p0[1], p1[0], p1[1], p2[0], p2[1], p3[0], p3[1]};
}

// The pair's halves traded between lanes 8 apart: p, q hold chunks 2g, 2g + 1 of row l & 15; sp, sq their scales.
struct W4Rows {
  u32x4 p, q;
  float sp, sq;
};
__device__ __forceinline__ W4Rows rows_of(const W4Pair& w) {
  W4Rows r;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    // row_ror:8 hands lane i the value of lane i ^ 8 of its row of 16; only the banks named are written
    r.p[i] = (uint32_t)__builtin_amdgcn_update_dpp((int)w.a[i], (int)w.b[i], 0x128, 0xf, 0xc, false);
    r.q[i] = (uint32_t)__builtin_amdgcn_update_dpp((int)w.b[i], (int)w.a[i], 0x128, 0xf, 0x3, false);
  }
  const uint32_t s = w.s >> (threadIdx.x & 16);   // bytes 2 (g & 1), 2 (g & 1) + 1
  r.sp = __uint_as_float((s & 0xffu) << 23);
  r.sq = __uint_as_float((s & 0xff00u) << 15);
  return r;
}

// acc0, acc1 += W x over the pair's 256 columns; x[i]: columns 64 g + 8 i .. + 7 of token l & 15.
__device__ __forceinline__ void mul_pair(const W4Rows& r, const bf16x8 (&x)[8], f32x4& acc0, f32x4& acc1) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    acc0 = __builtin_amdgcn_mfma_f32_16x16x32_bf16(widen4(r.p[i], r.sp), x[i], acc0, 0, 0, 0);
    acc1 = __builtin_amdgcn_mfma_f32_16x16x32_bf16(widen4(r.q[i], r.sq), x[4 + i], acc1, 0, 0, 0);
  }
}

// A barrier that publishes LDS only: loads into registers stay in flight (a full barrier may wait for them).
__device__ __forceinline__ void lds_barrier() {
  asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

}  // namespace moe
