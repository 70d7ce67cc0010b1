// FP8 with one scale per block of 128: the quantiser, the dense product and the experts'
// grouped products.
//
//   C[m,n] = sum_b a_scale[b][m] w_scale[n/128][b] sum_{i in block b} a[m,i] w[n,i]
//
// A block's 128 products are summed by the matrix cores without a scale; the block's two scales
// then multiply that partial sum on its way into the fp32 accumulator.  The weight rows are the
// MFMA's first operand, so that a lane's results all belong to one token row: its row scale
// is one register, the weight scale is uniform over a wavefront, and one product of the two
// serves every result of the block.
//
// Rounding inside the 8-bit MFMA (probed on gfx950 with single products): the products of eight
// consecutive bytes of a lane are added on a grid of 2^-13 of the largest one's binade, what lies
// below is cut off; these sums of eight are added in fp32.  On normal data that is 1.4e-5 of
// the result, far below a bf16 output's own half step (2e-3), which is why the full fp8 rate is taken
// there.  What asks for more has its codes widened to bf16 (every E4M3 value is a bf16 value) and multiplied by
// the bf16 MFMA, whose sums are fp32 (error against fp64 about 1e-7 of the output's norm), at half the rate: an fp32
// output, and the gate and up products of few rows, which wait for the weights in any case.
//
// The gate and up products of many rows keep the full rate.  Their 1.4e-5 moves values of h over a rounding border of H's 8
// bits, which is what an error of the experts' output beside its own rounding comes from: 2.0e-3 of its norm against fp64, 1.7e-3
// with fp32 sums (16,384 rows on 4 experts, d 7168, f 2048), for 705 us against 1,025 (2,048 tokens over 256 experts: 1.92 ms
// against 2.23).
#include <algorithm>
#include <cmath>

#include "common.h"
#include "fp8.h"
#include "fp8_tile.h"
#include "kernels.h"

namespace moe {

// ----------------------------------------------------------------------------- quantiser
// One block of 128 columns of a row sits in 16 consecutive lanes (8 bf16 each).
__global__ __launch_bounds__(256) void quantize_fp8_rows_kernel(const bf16_t* __restrict__ src, int64_t rows,
                                                                int64_t cols, uint8_t* __restrict__ codes,
                                                                float* __restrict__ scales) {
  const int64_t vpr = cols / 8, nvec = rows * vpr, stride = (int64_t)gridDim.x * 256;
  for (int64_t v0 = (int64_t)blockIdx.x * 256; v0 < nvec; v0 += stride) {
    const int64_t v = v0 + threadIdx.x;
    const bool ok = v < nvec;   // whole blocks of 16 lanes: nvec is a multiple of 16
    const u32x4 w = ok ? ((const u32x4*)src)[v] : u32x4{0, 0, 0, 0};
    float f[8];
#pragma unroll
    for (int q = 0; q < 4; ++q) { f[2 * q] = lo_bf(w[q]); f[2 * q + 1] = hi_bf(w[q]); }
    const float s = fp8_scale(block_amax<16>(f));
    const u32x2 c = fp8_encode8(f, s);
    if (ok) {
      ((u32x2*)codes)[v] = c;
      if ((v & 15) == 0) scales[((v % vpr) / 16) * rows + v / vpr] = s;
    }
  }
}

// One workgroup per 128 x 128 block: thread q holds rows
// q / 16 + 16 i, i < 8, columns 8 (q % 16) .. + 7.
__global__ __launch_bounds__(256) void quantize_fp8_blocks_kernel(const bf16_t* __restrict__ src, int64_t rows,
                                                                  int64_t cols, uint8_t* __restrict__ codes,
                                                                  float* __restrict__ scales) {
  __shared__ float red[4];
  const int64_t nb = cols / 128, rb = blockIdx.x / nb, cb = blockIdx.x % nb;
  const int tid = threadIdx.x;
  const int64_t r0 = rb * 128 + tid / 16, c0 = cb * 128 + (tid & 15) * 8;
  u32x4 w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i)
    w[i] = r0 + 16 * i < rows ? *(const u32x4*)(src + (r0 + 16 * i) * cols + c0) : u32x4{0, 0, 0, 0};
  float a = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int q = 0; q < 4; ++q) a = amax2(amax2(a, lo_bf(w[i][q])), hi_bf(w[i][q]));
  a = lanes_amax<64>(a);
  if ((tid & 63) == 0) red[tid >> 6] = a;
  __syncthreads();
  const float s = fp8_scale(amax2(amax2(red[0], red[1]), amax2(red[2], red[3])));
  if (tid == 0) scales[rb * nb + cb] = s;
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (r0 + 16 * i < rows) {
      const float f[8] = {lo_bf(w[i][0]), hi_bf(w[i][0]), lo_bf(w[i][1]), hi_bf(w[i][1]),
                          lo_bf(w[i][2]), hi_bf(w[i][2]), lo_bf(w[i][3]), hi_bf(w[i][3])};
      *(u32x2*)(codes + (r0 + 16 * i) * cols + c0) = fp8_encode8(f, s);
    }
}

hipError_t launch_quantize_fp8(const void* src, int64_t rows, int64_t cols, int row_block,
                               uint8_t* codes, float* scales, hipStream_t st) {
  if (row_block == 1) {
    const int64_t wgs = (rows * (cols / 8) + 255) / 256;
    quantize_fp8_rows_kernel<<<(unsigned)std::min<int64_t>(wgs, 65536), 256, 0, st>>>(
        (const bf16_t*)src, rows, cols, codes, scales);
  } else {
    quantize_fp8_blocks_kernel<<<(unsigned)(((rows + 127) / 128) * (cols / 128)), 256, 0, st>>>(
        (const bf16_t*)src, rows, cols, codes, scales);
  }
  return hipGetLastError();
}

// ----------------------------------------------------------------------------- products
// Wait until at most n stages of L copies are outstanding.
template <int L, int MOST>
__device__ __forceinline__ void wait_stages(int n) {
  if constexpr (MOST == 0) wait_vm<0>();
  else if (n >= MOST) wait_vm<MOST * L>();
  else wait_stages<L, MOST - 1>(n);
}

// Few token rows: a weight stream.  16 token rows x 32 W weight rows, W wavefronts, each with 32 weight rows
// (SWIGLU: 16 gate and the matching 16 up rows, W = 4: 64 columns a workgroup, half a block of H, so that twice
// the workgroups fill the chip; h leaves in fp32 for quantise_h_kernel: 46 -> 37 us for the gate and up
// products of one token, 8 of 64 experts, d 7168, f 2048).  The work is one pass over the weights, so what counts is bytes in flight: S stages
// of whole 128-byte lines are copied global -> LDS, S - 1 of them ahead.  The same stream read straight
// into registers in the MFMA's layout asks for each line in halves by 16 rows and ran at 3.7 TB/s where
// this one runs at 5 to 6 (one token, 8 of 64 experts, d 7168, f 2048).
//
// Per stage a wavefront issues four 1 KB copies of weights and EX small ones: the token rows' two
// kilobytes, the row scales and the block scales, dealt to the wavefronts in turn and padded with
// repeats so that all issue the same number (the stage waits count them).
template <int W, int S>
struct ThinStage {
  static constexpr int EX = (5 + W - 1) / W, L = 4 + EX;
  static constexpr int B = 0, A = W * 4096, SC = A + 2048;       // SC: row scales, S0's, S1's, padding
  static constexpr int SIZE = SC + 4 * 256;
};

template <int KIND, int W, int S>
__global__ __launch_bounds__(64 * W) void fp8_thin_kernel(Fp8Args p) {
  using SL = ThinStage<W, S>;
  constexpr bool SWIGLU = KIND >= FP8_SWIGLU;
  // fp32 sums for the gate and up products (one token's experts, 8 of 64, d 7168, f 2048: 60.3 us a call against 59.2, 8 experts x
  // 8 rows, d 2048, f 768, weights in the caches: 17.8 against 16.2; the output's error 1.66e-3, that of its rounding,
  // against 1.9e-3 to 2.3e-3)
  constexpr bool WIDE = KIND == FP8_F32 || SWIGLU;
  constexpr int L = SL::L, COLS = SWIGLU ? 16 * W : 32 * W;
  static_assert(!SWIGLU || W == 4, "half a block of H");
  extern __shared__ __attribute__((aligned(1024))) uint8_t lds[];
  const uint32_t lds0 = (uint32_t)(uintptr_t)lds;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), lr = lane & 15, lg = lane >> 4;
  const int nct = (p.N + COLS - 1) / COLS, nblk = (p.N + 127) / 128;
  const int z = blockIdx.x % p.Z, item = blockIdx.x / p.Z, mt = item / nct, ct = item % nct;
  int e = 0, row0 = 16 * mt, rows = 16;
  int32_t seg = 0;
  if (p.offset) {
    const SegmentTiles st = segment_tiles<16>(p.offset, p.E);
    if (mt >= st.total) return;
    int first;
    find_segment<16>(st, mt, e, first, seg, rows);
    auto uni = [](int v) { return __builtin_amdgcn_readfirstlane(v); };
    e = uni(e); row0 = uni(16 * (mt - first)); seg = uni(seg); rows = uni(min(16, rows - row0));
  } else {
    rows = (int)min((int64_t)16, p.a_rows - row0);
  }
  const uint32_t K = (uint32_t)p.K;
  const int KA = p.K / 128, kb = (int)((int64_t)KA * z / p.Z), KT = (int)((int64_t)KA * (z + 1) / p.Z) - kb;
  const int n0 = COLS * ct;
  auto slot_of = [&](int m) { return ring_slot(p.head, seg, row0 + m, p.C); };

  // weights: copy i is kilobyte W i + wave of the tile, rows 8 (W i + wave) .. + 7
  const uint8_t* b_base[4];
  uint32_t b_off[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = 8 * (W * i + wave) + lane / 8, c = (swz<128>(r, lane % 8) - r * 128) >> 4;
    const bool up = SWIGLU && i >= 2;
    b_base[i] = (up ? p.W1 : p.W0) + (int64_t)e * p.N * K;
    b_off[i] = (uint32_t)min(n0 + (up ? r - 16 * W : r), p.N - 1) * K + c * 16;
  }
  // small copy x of a stage (wavefront x % W): 0, 1 token rows, 2 row scales, 3 S0's, 4 S1's block scale, then repeats
  auto small = [&](int x, int kt, uint32_t st) __attribute__((always_inline)) {
    if (x < 2) {
      const int r = 8 * x + lane / 8, c = (swz<128>(r, lane % 8) - r * 128) >> 4;
      dma16(p.A + (size_t)kt * 128, (uint32_t)slot_of(min(r, rows - 1)) * K + c * 16,
            __builtin_amdgcn_readfirstlane(st + SL::A + x * 1024));
    } else if (x == 2) {
      dma4((const uint8_t*)(p.As + (size_t)kt * p.a_rows), (uint32_t)slot_of(min(lr, rows - 1)) * 4,
           __builtin_amdgcn_readfirstlane(st + SL::SC));
    } else {
      const float* s = SWIGLU && x == 4 ? p.S1 : p.S0;
      // the block of this lane's column: lane l < W of the plain product holds wavefront l's
      const int blk = SWIGLU ? n0 / 128 : min((n0 + 32 * (lane % W)) / 128, nblk - 1);
      dma4((const uint8_t*)(s + (int64_t)e * nblk * KA + kt), (uint32_t)blk * KA * 4,
           __builtin_amdgcn_readfirstlane(st + SL::SC + (x == 3 ? 256 : x == 4 ? 512 : 768)));
    }
  };
  auto issue = [&](int i_) __attribute__((always_inline)) {   // step i_: block kb + i_
    const uint32_t st = lds0 + (uint32_t)(i_ % S) * SL::SIZE;
    const int kt = kb + i_;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      dma16nt(b_base[i] + (size_t)kt * 128, b_off[i], __builtin_amdgcn_readfirstlane(st + SL::B + (W * i + wave) * 1024));
#pragma unroll
    for (int x = 0; x < SL::EX; ++x) small(W * x + wave, kt, st);
  };
  f32x4 acc[2] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
  const uint32_t l0 = (uint32_t)(lr * 128 + ((lg ^ ((lr >> 1) & 7)) << 4));   // as in fp8_tile.h
  const int f0 = SWIGLU ? wave : 2 * wave, f1 = SWIGLU ? wave + W : f0 + 1;   // weight fragments
  auto multiply = [&](int kt) __attribute__((always_inline)) {
    const uint8_t* st = lds + (kt % S) * SL::SIZE;
    auto frag = [&](uint32_t at) { return fp8_join(*(const u32x4*)(st + at + l0), *(const u32x4*)(st + at + (l0 ^ 64))); };
    const i32x8 a = frag(SL::A), w0 = frag(SL::B + f0 * 2048), w1 = frag(SL::B + f1 * 2048);
    const float* sc = (const float*)(st + SL::SC);
    const float sa = sc[lr], t0 = sa * sc[64 + (SWIGLU ? 0 : wave)], t1 = SWIGLU ? sa * sc[128] : t0;
    f32x4 q0, q1;
    if constexpr (WIDE) {
      const Wide16 aw = fp8_widen(a);
      q0 = fp8_wide16(fp8_widen(w0), aw);
      q1 = fp8_wide16(fp8_widen(w1), aw);
    } else {
      q0 = fp8_mfma16(w0, a);
      q1 = fp8_mfma16(w1, a);
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      acc[0][r] = fmaf(q0[r], t0, acc[0][r]);
      acc[1][r] = fmaf(q1[r], t1, acc[1][r]);
    }
  };
  for (int s = 0; s < S - 1 && s < KT; ++s) issue(s);
  int kt = 0;
  for (; kt < KT - (S - 1); ++kt) {
    wait_vm<(S - 2) * L>();
    __syncthreads();
    issue(kt + S - 1);
    multiply(kt);
  }
  for (; kt < KT; ++kt) {
    wait_stages<L, S - 2>(KT - 1 - kt);
    __syncthreads();
    multiply(kt);
  }
  // acc[c][r]: token row lr, weight row 16 f_c + 4 lg + r
  const int64_t slot = slot_of(min(lr, rows - 1));
  if constexpr (SWIGLU) {
    if (lr >= rows) return;
    const int col = n0 + 16 * wave + 4 * lg;
    *(f32x4*)(p.h32 + ((int64_t)seg + row0 + lr) * p.N + col) =
        f32x4{silu(acc[0][0]) * acc[1][0], silu(acc[0][1]) * acc[1][1], silu(acc[0][2]) * acc[1][2], silu(acc[0][3]) * acc[1][3]};
    if constexpr (KIND == FP8_SWIGLU_SAVE) {
      *(u32x2*)(p.saved_au + slot * 2 * p.N + col) = u32x2{pack_bf2(acc[0][0], acc[0][1]), pack_bf2(acc[0][2], acc[0][3])};
      *(u32x2*)(p.saved_au + (slot * 2 + 1) * p.N + col) = u32x2{pack_bf2(acc[1][0], acc[1][1]), pack_bf2(acc[1][2], acc[1][3])};
    }
  } else {
    if (lr >= rows) return;
    constexpr bool FLOATS = KIND != FP8_BF16;
    constexpr int EB = FLOATS ? 4 : 2;
    const bool whole = (p.N & 3) == 0 && ((uintptr_t)p.out & (4 * EB - 1)) == 0;
    const int64_t row = (z * p.C + slot) * p.N;
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int col = n0 + 16 * (f0 + c) + 4 * lg;
      const f32x4 v = acc[c];
      if (whole) {
        if (col >= p.N) continue;
        if constexpr (FLOATS) *(f32x4*)((float*)p.out + row + col) = v;
        else *(u32x2*)((bf16_t*)p.out + row + col) = u32x2{pack_bf2(v[0], v[1]), pack_bf2(v[2], v[3])};
      } else {
#pragma unroll
        for (int r = 0; r < 4; ++r)
          if (col + r < p.N) {
            if constexpr (FLOATS) ((float*)p.out)[row + col + r] = v[r];
            else ((bf16_t*)p.out)[row + col + r] = f2bf(v[r]);
          }
      }
    }
  }
}

// h [n, f] fp32, in segment order, to H's codes and scales at the rows' slots: a block of 128 columns sits in 16 lanes.
__global__ __launch_bounds__(256) void quantise_h_kernel(const float* __restrict__ h, int64_t n, int f, int64_t head,
                                                         int64_t C, uint8_t* __restrict__ codes,
                                                         float* __restrict__ scales) {
  const int64_t v = (int64_t)blockIdx.x * 256 + threadIdx.x, r = v / (f / 8);
  if (r >= n) return;   // whole blocks: f / 8 is a multiple of 16
  const int c = (int)(v % (f / 8));
  const f32x4 a = *(const f32x4*)(h + r * f + c * 8), b = *(const f32x4*)(h + r * f + c * 8 + 4);
  const float x[8] = {a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
  const float s = fp8_scale(block_amax<16>(x));
  const int64_t slot = ring_slot(head, 0, r, C);
  *(u32x2*)(codes + slot * f + c * 8) = u32x2{h_encode4(x[0], x[1], x[2], x[3], s), h_encode4(x[4], x[5], x[6], x[7], s)};
  if ((c & 15) == 0) scales[(int64_t)(c / 16) * C + slot] = s;
}

template <int KIND, int W, int S>
static hipError_t run_fp8_thin(const Fp8Args& a, int64_t tiles, hipStream_t st) {
  constexpr int cols = KIND >= FP8_SWIGLU ? 16 * W : 32 * W, lds = S * ThinStage<W, S>::SIZE;
  static_assert(lds <= 160 * 1024, "LDS");
  auto kern = fp8_thin_kernel<KIND, W, S>;
  hipError_t err = hipFuncSetAttribute((const void*)kern, hipFuncAttributeMaxDynamicSharedMemorySize, lds);
  if (err != hipSuccess) return err;
  kern<<<(unsigned)(tiles * ((a.N + cols - 1) / cols) * a.Z), 64 * W, lds, st>>>(a);
  return hipGetLastError();
}
// Wavefronts of a plain thin workgroup: the fewest columns that still run at once (two workgroups of two
// wavefronts share a CU's LDS, one of four or eight fills it).
static int thin_waves(int64_t tiles, int64_t N) {
  return tiles * ((N + 63) / 64) <= 512 ? 2 : tiles * ((N + 127) / 128) <= 256 ? 4 : 8;
}
template <int KIND>
static hipError_t run_fp8_thin_plain(const Fp8Args& a, int64_t tiles, int W, hipStream_t st) {
  if (W == 8) return run_fp8_thin<KIND, 8, 4>(a, tiles, st);
  if (W == 4) return run_fp8_thin<KIND, 4, 7>(a, tiles, st);
  return run_fp8_thin<KIND, 2, 7>(a, tiles, st);
}

// How a dense product runs: fm = 0 the thin kernel (16 token rows a tile, W wavefronts), else tiles of 64 fm rows;
// Z: K splits.  The least estimated time of all: rounds of 256 workgroups times the blocks of one,
// where a block of a tile of 64 / 128 / 192 / 256 rows took 0.95, 0.98, 1.07 and 1.25 us (M 2,045, N 4,168,
// K 7,168: low tiles are bound by their weight copies, not by the matrix cores; the fp32 output's
// bf16 MFMAs 1.1 and 2.0 us at 64 and 128 rows), and a block of a thin workgroup its share of a
// copy's latency (0.67, 0.33, 0.29 us with 8, 4, 2 wavefronts), or the weights at 6 TB/s.  A split fills
// idle CUs, but its planes are written and read once more, and the second launch costs 6 us.
struct DensePlan {
  int fm, W, Z;
};
static DensePlan dense_plan(int64_t M, int64_t N, int64_t K, bool f32, bool split) {
  const double us[4] = {0.95, f32 ? 2.0 : 0.98, 1.07, 1.25};
  const int64_t KT = K / 128;
  DensePlan best{};
  double least = 1e300;
  auto offer = [&](DensePlan p, int64_t wgs, double block, double floor_us) {
    const int64_t most = split ? std::min<int64_t>({256 / wgs, KT / 4, 16}) : 1;
    for (p.Z = 1; p.Z == 1 || p.Z <= most; p.Z *= 2) {
      const double rounds = (double)((wgs * p.Z + 255) / 256), blocks = (double)((KT + p.Z - 1) / p.Z);
      const double t = std::max(rounds * (blocks * block + 3.0), floor_us) +
                       (p.Z > 1 ? 6.0 + (double)p.Z * M * N * 8 / 4e6 : 0.0);
      if (t < least) { least = t; best = p; }
    }
  };
  for (int fm = 1; fm <= (f32 ? 2 : 4); ++fm) {
    if (f32 && fm == 1) offer({fm, 0, 1}, (M + 63) / 64 * ((N + 255) / 256), 1.1, 0.0);
    else offer({fm, 0, 1}, (M + 64 * fm - 1) / (64 * fm) * ((N + 255) / 256), us[fm - 1], 0.0);
  }
  if (M <= 256) {
    const int64_t tiles = (M + 15) / 16;
    const int W = thin_waves(tiles, N);
    const int64_t wgs = tiles * ((N + 32 * W - 1) / (32 * W));
    offer({0, W, 1}, W == 2 ? (wgs + 1) / 2 : wgs, W == 8 ? 0.67 : W == 4 ? 0.33 : 0.29, (double)tiles * N * K / 6e6);
  }
  return best;
}

int tile_add_height(int64_t M, int64_t N, int64_t K) { return std::max(1, dense_plan(M, N, K, false, false).fm); }

size_t matmul_fp8_workspace_bytes(int64_t M, int64_t N, int64_t K) {
  size_t b = 0;
  for (bool f32 : {false, true}) {
    const DensePlan d = dense_plan(M, N, K, f32, true);
    if (d.Z > 1) b = std::max(b, (size_t)d.Z * M * N * 4);
  }
  return b;
}

// out[i] = the sum of the Z planes in order, rounded once.
template <bool F32>
__global__ __launch_bounds__(256) void plane_join_kernel(const float* __restrict__ part, int Z, int64_t n, void* out) {
  const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
  if (i >= n) return;
  const int live = (int)min((int64_t)4, n - i);
  float s[4] = {0.f, 0.f, 0.f, 0.f};
  if (live == 4 && (n & 3) == 0) {   // every plane starts on 16 bytes
    f32x4 v = *(const f32x4*)(part + i);
    for (int z = 1; z < Z; ++z) v += *(const f32x4*)(part + z * n + i);
#pragma unroll
    for (int r = 0; r < 4; ++r) s[r] = v[r];
  } else {
    for (int r = 0; r < live; ++r)
      for (int z = 0; z < Z; ++z) s[r] += part[z * n + i + r];
  }
  const int EB = F32 ? 4 : 2;
  if (live == 4 && ((uintptr_t)out & (4 * EB - 1)) == 0) {
    if constexpr (F32) *(f32x4*)((float*)out + i) = f32x4{s[0], s[1], s[2], s[3]};
    else *(u32x2*)((bf16_t*)out + i) = u32x2{pack_bf2(s[0], s[1]), pack_bf2(s[2], s[3])};
  } else {
    for (int r = 0; r < live; ++r) {
      if constexpr (F32) ((float*)out)[i + r] = s[r];
      else ((bf16_t*)out)[i + r] = f2bf(s[r]);
    }
  }
}

template <int KIND>
static hipError_t run_dense(const Fp8Args& p, const DensePlan& d, hipStream_t st) {
  const int64_t M = p.a_rows, mt = d.fm ? (M + 64 * d.fm - 1) / (64 * d.fm) : (M + 15) / 16;
  if (d.fm == 0) return run_fp8_thin_plain<KIND>(p, mt, d.W, st);
  if (d.fm == 1) return run_fp8_tile<1, KIND, 3, false>(p, mt, st);
  if constexpr (KIND != FP8_F32) {
    if (d.fm == 3) return run_fp8_tile<3, KIND, 2, false>(p, mt, st);
    if (d.fm == 4) return run_fp8_tile<4, KIND, 2, false>(p, mt, st);
  }
  return run_fp8_tile<2, KIND, 3, false>(p, mt, st);
}

hipError_t launch_matmul_fp8(const uint8_t* a, const float* a_scale, const uint8_t* w,
                             const float* w_scale, int64_t M, int64_t N, int64_t K, bool f32_out,
                             void* out, void* ws, hipStream_t st) {
  const DensePlan d = dense_plan(M, N, K, f32_out, true);
  Fp8Args p{};
  p.A = a;
  p.As = a_scale;
  p.W0 = w;
  p.S0 = w_scale;
  p.a_rows = M;
  p.C = M;
  p.K = (int)K;
  p.N = (int)N;
  p.Z = d.Z;
  p.group = FP8_GROUP;
  p.out = d.Z > 1 ? ws : out;
  hipError_t err = f32_out ? run_dense<FP8_F32>(p, d, st) : d.Z > 1 ? run_dense<FP8_PART>(p, d, st) : run_dense<FP8_BF16>(p, d, st);
  if (err != hipSuccess || d.Z == 1) return err;
  const unsigned g = (unsigned)((M * N + 1023) / 1024);
  if (f32_out) plane_join_kernel<true><<<g, 256, 0, st>>>((const float*)ws, d.Z, M * N, out);
  else plane_join_kernel<false><<<g, 256, 0, st>>>((const float*)ws, d.Z, M * N, out);
  return hipGetLastError();
}

// How the experts' products run.  The host knows the mean rows of an expert, not their spread.
//   * `few`: fewer than THIN_FEW workgroups of 128 columns over all 16-row tiles: the thin kernel (4 experts x
//     16 rows, d 7168, f 2048: 47 us against 65 with a list of tiles of 64 rows; 64 experts x 8 rows: 309 us
//     either way, and a batch that falls on one expert would read its weights once per 16 rows).
//   * else tiles of 64 fm rows, the least estimated time of both products: rounds of 256 workgroups times the
//     blocks of one (dense_plan's times), or the weights at the rate that height streams them at
//     (5.3, 5.1, 4.6, 4.5 TB/s: the lower tiles keep three stages).
//     Measured at 64 experts, d 4096, f 2048, us for fm = 1 | 2 | 3 | 4: 32 rows 310 | 313 | 363 | 371, 64 rows 344 |
//     325 | 370 | 377, 128 rows 470 | 404 | 390 | 394, 200 rows 621 | 477 | 562 | 434, 300 rows 872 | 667 | 652 | 713.
constexpr int64_t THIN_FEW = 200;

static int ffn_tile(int64_t n, int d, int E, int f) {
  const double us[4] = {0.95, 0.98, 1.07, 1.25}, tbs[4] = {5.3, 5.1, 4.6, 4.5};
  const double r = (double)n / E, typical = r + 0.5 * std::sqrt(r);
  int best = 1;
  double least = 1e300;
  for (int fm = 1; fm <= 4; ++fm) {
    const double tiles = E * std::ceil(typical / (64 * fm));
    auto rounds = [&](double cols) { return std::ceil(tiles * cols / 256); };
    const double busy = (rounds(f / 128) * (d / 128) + rounds((d + 255) / 256) * (f / 128)) * us[fm - 1];
    const double t = std::max(busy, 3.0 * E * d * f / tbs[fm - 1] * 1e-6);
    if (t < least) { least = t; best = fm; }
  }
  return best;
}

struct FfnFp8Layout {
  size_t tiles, h, hs, h32, total;
  int fm;
  int64_t mt;   // bound on the row tiles: every tile holds a row
  bool few, list;
};
static FfnFp8Layout ffn_fp8_layout(int64_t n, int64_t C, int d, int E, int f) {
  auto al = [](size_t b) { return (b + 255) & ~(size_t)255; };
  FfnFp8Layout L;
  L.few = std::min<int64_t>(max_tiles_for(n, E, 16), n) * (f / 128) < THIN_FEW;
  L.fm = L.few ? 0 : ffn_tile(n, d, E, f);
  L.mt = std::min<int64_t>(max_tiles_for(n, E, L.few ? 16 : 64 * L.fm), n);
  // many workgroups: their row tiles come from a list (2,048 tokens over 256 experts, 17 thousand: 1,948 -> 1,926 us)
  L.list = !L.few && L.mt * (f / 128 + (d + 255) / 256) > 4096;
  size_t o = 0;
  L.tiles = o; o += L.list ? al((size_t)(2 * L.mt + 64) * 4) : 0;
  L.h = o; o += al((size_t)C * f);
  L.hs = o; o += al((size_t)C * (f / 128) * 4);
  L.h32 = o; o += L.few ? al((size_t)n * f * 4) : 0;
  L.total = o;
  return L;
}
size_t ffn_fp8_workspace_bytes(int64_t n, int64_t C, int d, int E, int f) {
  return ffn_fp8_layout(n, C, d, E, f).total;
}

hipError_t launch_ffn_fp8(const void* ring_x, const float* ring_x_scale, const int32_t* expert_offset,
                          int64_t head, int64_t C, int64_t n, int d, int E, int f,
                          const void* w_gate, const void* w_up, const void* w_down,
                          const float* sg, const float* su, const float* sd, void* ring_y,
                          void* saved_au, void* ws, hipEvent_t* events, hipStream_t st) {
  const FfnFp8Layout L = ffn_fp8_layout(n, C, d, E, f);
  uint8_t* w = (uint8_t*)ws;
  auto mark = [&](int i) { return events ? hipEventRecord(events[i], st) : hipSuccess; };
  const int fm = L.fm;
  const int64_t mt = L.mt;
  int32_t* ntiles = (int32_t*)(w + L.tiles);
  hipError_t err = L.list ? launch_build_tiles(expert_offset, E, 64 * fm, ntiles + 64, ntiles, st) : hipSuccess;
  if (err != hipSuccess || (err = mark(0)) != hipSuccess) return err;
  const bool once = n <= 64 * fm * (int64_t)E;   // about one row tile per expert: each weight is read once
  Fp8Args p{};
  p.A = (const uint8_t*)ring_x;
  p.As = ring_x_scale;
  p.W0 = (const uint8_t*)w_gate;
  p.W1 = (const uint8_t*)w_up;
  p.S0 = sg;
  p.S1 = su;
  p.a_rows = C;
  p.K = d;
  p.N = f;
  p.offset = expert_offset;
  p.tiles = L.list ? ntiles + 64 : nullptr;
  p.ntiles = ntiles;
  p.head = head;
  p.C = C;
  p.out = w + L.h;
  p.out_scale = (float*)(w + L.hs);
  p.saved_au = (bf16_t*)saved_au;
  p.E = E;
  p.Z = 1;
  p.h32 = (float*)(w + L.h32);
  p.group = FP8_GROUP;
#define RUN(FM, KIND, S, G)                                              \
  err = once ? run_fp8_tile<FM, KIND, S, true>(G, mt, st) : run_fp8_tile<FM, KIND, S, false>(G, mt, st);
  if (fm == 0) {
    err = saved_au ? run_fp8_thin<FP8_SWIGLU_SAVE, 4, 7>(p, mt, st) : run_fp8_thin<FP8_SWIGLU, 4, 7>(p, mt, st);
    if (err != hipSuccess) return err;
    quantise_h_kernel<<<(unsigned)((n * (f / 8) + 255) / 256), 256, 0, st>>>(p.h32, n, f, head, C, w + L.h, p.out_scale);
    err = hipGetLastError();
  } else if (fm == 1) {
    if (saved_au) RUN(1, FP8_SWIGLU_SAVE, 3, p) else RUN(1, FP8_SWIGLU, 3, p)
  } else if (fm == 2) {
    if (saved_au) RUN(2, FP8_SWIGLU_SAVE, 3, p) else RUN(2, FP8_SWIGLU, 3, p)
  } else if (fm == 3) {
    if (saved_au) RUN(3, FP8_SWIGLU_SAVE, 2, p) else RUN(3, FP8_SWIGLU, 2, p)
  } else {
    if (saved_au) RUN(4, FP8_SWIGLU_SAVE, 2, p) else RUN(4, FP8_SWIGLU, 2, p)
  }
  if (err != hipSuccess || (err = mark(1)) != hipSuccess) return err;
  Fp8Args q = p;
  q.A = w + L.h;
  q.As = p.out_scale;
  q.W0 = (const uint8_t*)w_down;
  q.W1 = nullptr;
  q.S0 = sd;
  q.S1 = nullptr;
  q.K = f;
  q.N = d;
  q.out = ring_y;
  q.out_scale = nullptr;
  q.saved_au = nullptr;
  if (fm == 0) {
    err = run_fp8_thin_plain<FP8_BF16>(q, mt, thin_waves(mt, d), st);
  } else if (fm == 1) RUN(1, FP8_BF16, 3, q)
  else if (fm == 2) RUN(2, FP8_BF16, 3, q)
  else if (fm == 3) RUN(3, FP8_BF16, 2, q)
  else RUN(4, FP8_BF16, 2, q)
#undef RUN
  if (err != hipSuccess) return err;
  return mark(2);
}

}  // namespace moe
