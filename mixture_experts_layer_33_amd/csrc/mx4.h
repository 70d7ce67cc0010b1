// MXFP4 weights (E2M1 codes, two a byte, the even column in the low half; one E8M0 byte per 32 columns in the
// MX scale layout [cols / 128][rows][4]) as operands of the bf16 MFMA: the loads and the widening that the
// weight-stream kernels share.
//
// A wavefront takes 16 weight rows x 256 columns (a "pair" of 128-column groups) per step, in two 16-byte loads a lane of
// eight rows each: eight lanes cover the 128 contiguous bytes of one row (a request for half a 128-byte line moves
// the whole of it).  Lane l holds row l & 7, 16-byte chunk l >> 3, and a chunk is one scale block of 32 columns.
//
// The 16x16x32 MFMA reads lane l as row l & 15 of its first operand, columns of lane group g = l >> 4.  So rows 0-7 of the
// operand are the eight weight rows with chunk 2g, and rows 8-15 the same weight rows with chunk 2g + 1.  The second
// operand's columns are split alike: column c < 8 is token c's chunk 2g, column c + 8 its chunk 2g + 1.  Of the 16 x 16
// results those with row < 8 and column < 8 or with both >= 8 are sums of the product, in two halves to be added; the
// others mix a chunk with another's token and are dropped.  No lane moves a value to another, a token takes half the registers
// that an operand of 16 tokens would, and up to eight tokens the MFMAs are as many as without the split.
//
// The codes widen to bf16 by gfx950's v_cvt_scalef32_pk_bf16_fp4 (two codes and the block's scale in one instruction at the
// full VALU rate; checked for every byte, byte place and scale from 2^-127 up: code value x 2^(byte - 127), infinite from
// 2^128 on, NaN for byte 255).  E2M1 x 2^X is exact in bf16, whose subnormal values the bf16 MFMA takes as they are; products
// and sums are the MFMA's in fp32.
#pragma once

#include <type_traits>

#include "common.h"

namespace moe {

typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));

// Compute units of an MI355X.  The product's plan is made for these and not for the current device's: its workspace is a function of
// the sizes alone.
constexpr int CUS = 256;

constexpr uint32_t RSRC_WORD3 = 0x00027000;   // raw buffer, 32-bit data
constexpr uint32_t OUTSIDE = 0x80000000u;      // an offset past every buffer (they are below 2 GiB): the load returns zeros
constexpr int NT_LOAD = 2;                     // cache policy of a buffer load: non-temporal

// (offset: per lane; `at`: of the wavefront, at most the buffer's size: beyond it nothing counts as outside)
__device__ __forceinline__ u32x4 load_b128(__amdgpu_buffer_rsrc_t r, uint32_t offset, uint32_t at) {
  return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, (int)offset, (int)at, 0));
}
__device__ __forceinline__ u32x4 load_b128_nt(__amdgpu_buffer_rsrc_t r, uint32_t offset, uint32_t at) {
  return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, (int)offset, (int)at, NT_LOAD));
}
__device__ __forceinline__ uint32_t load_b32(__amdgpu_buffer_rsrc_t r, uint32_t offset, uint32_t at) {
  return __builtin_amdgcn_raw_buffer_load_b32(r, (int)offset, (int)at, 0);
}
// One of two addresses that are the same in the whole wavefront.  Both are scalar registers by then: a choice between kernel
// arguments may otherwise become a load from a chosen place of the argument block, address and buffer per lane.
__device__ __forceinline__ const uint8_t* either(bool first, const uint8_t* a, const uint8_t* b) {
  uint64_t u = (uint64_t)a, v = (uint64_t)b;
  asm("" : "+s"(u), "+s"(v));
  return (const uint8_t*)(first ? u : v);
}
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_of(const void* base, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc((void*)base, 0, (int)bytes, (int)RSRC_WORD3);
}

struct W4Pair {
  u32x4 a, b;          // two times eight rows
  uint32_t sa, sb;     // the four scale bytes of the row's 128 columns in which the chunk lies
};

// Eight codes of one row and block as bf16.
__device__ __forceinline__ bf16x8 widen4(uint32_t codes, float scale) {
  const bf16x2_t p0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 0);
  const bf16x2_t p1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 1);
  const bf16x2_t p2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 2);
  const bf16x2_t p3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 3);
  return bf16x8{p0[0], p0[1], p1[0], p1[1], p2[0], p2[1], p3[0], p3[1]};
}

// The scale of this lane's chunk, from the word that holds it, as the conversion takes it.
__device__ __forceinline__ float chunk_scale(uint32_t word) {
  const int c = (threadIdx.x >> 3) & 3;
  return __uint_as_float(__builtin_amdgcn_ubfe(word, 8 * c, 8) << 23);
}

__device__ __forceinline__ f32x4 mfma16(bf16x8 a, bf16x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

// This lane's results (rows 4 (g & 1) .. + 3 of the eight, token l & 7) are one of the two halves; else they are dropped.
__device__ __forceinline__ bool holds_half() { return ((threadIdx.x >> 5) & 1) == ((threadIdx.x >> 3) & 1); }

// f(0), ..., f(N - 1) with constant arguments.
template <int N, int I = 0, typename F>
__device__ __forceinline__ void unrolled(F f) {
  if constexpr (I < N) {
    f(std::integral_constant<int, I>{});
    unrolled<N, I + 1>(f);
  }
}

// Global -> LDS copy of 16 bytes a lane, to `lds` + 16 lane, that the compiler does not wait for (as gemm_body.h's).  The compiler
// does not look into the asm: five wait states between a vector instruction that writes the address's scalar
// registers and the copy that reads them, and one behind m0, are written out.
__device__ __forceinline__ void copy16(const void* base, uint32_t offset, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 4\n\tglobal_load_lds_dwordx4 %0, %1"
               ::"v"(offset), "s"(base), "s"(lds) : "memory", "m0");
}

// Waits for all copies (and loads) of this wavefront.
__device__ __forceinline__ void wait_all() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }

// Eight rows of x of one pair as second operands.  A lane's part is 64 contiguous bytes of a row: read straight into registers
// each of the four 16-byte loads touches 64 pieces of 64 bytes, so the block (4 KB) goes through LDS in
// four copies of whole 128-byte lines: copy i has chunks 2i and 2i + 1 of each row, 16-byte pieces exchanged among themselves
// so that 16 lanes read from all banks.
constexpr int XBLOCK = 4096;
// `base`: the first row at the pair's first column, `left` >= 128 columns from there on (a multiple of 128), `lds`: the block.
__device__ __forceinline__ void x_copy(const bf16_t* base, int last_row, uint32_t K, int left, uint32_t lds) {
  const int lane = threadIdx.x & 63, r = lane >> 3, piece = (lane & 7) ^ ((r >> 1) & 3);
  const uint32_t at = (uint32_t)min(r, last_row) * K * 2 + piece * 16;
#pragma unroll
  for (int i = 0; i < 4; ++i) copy16(base, at + (left > 128 || i < 2 ? i : i - 2) * 128, __builtin_amdgcn_readfirstlane(lds + i * 1024));
}
// `in`: the pair has this lane's chunk.
__device__ __forceinline__ void x_read(const uint8_t* block, bool in, bf16x8 (&x)[4]) {
  const int lane = threadIdx.x & 63, g = lane >> 4, col = lane & 15, r = col & 7;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const u32x4 v = *(const u32x4*)(block + g * 1024 + r * 128 + ((((col >> 3) * 4 + j) ^ ((r >> 1) & 3)) << 4));
    x[j] = __builtin_bit_cast(bf16x8, in ? v : u32x4{0, 0, 0, 0});
  }
}

// A barrier that publishes LDS only: loads into registers stay in flight (a full barrier may wait for them).
__device__ __forceinline__ void lds_barrier() {
  asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

}  // namespace moe
