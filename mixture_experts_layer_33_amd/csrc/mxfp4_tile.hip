// out[m][n] = sum_k x[m][k] W[n][k] for more than a few rows of x (bf16) and MXFP4 weights: tiles of the bf16 MFMA.
//
// A workgroup has a tile of BM x BN outputs, K staged in steps of 64 columns through an S-stage LDS ring: BM x 128 bytes of x and
// BN x 32 bytes of codes, with each W row's word of scale bytes.  The codes stay four bits in LDS and are widened on the way
// into the MFMA (mx4.h's conversion, two values an instruction): for a wavefront of 128 x 64 outputs that is one conversion to
// 64 clocks of MFMA, on the vector unit that the MFMAs leave idle, and a sixteenth of the LDS traffic is W's.
//
// The 32x32x16 MFMA reads lane l as row l & 31, columns 8 (l >> 5) .. + 7 of its operands; any order of the K columns is right
// that both share.  Lane half h takes scale block h of a step's two, four MFMAs j with the block's columns 8j .. 8j + 7:
// a lane's codes of a step are one 16-byte read, under one scale.  W's rows are the first operand, so that a lane
// holds four neighbouring outputs of one row of x.
//
// 2045 x 7168 x 4096 takes 102 us, 1.18 PFLOP/s, in 224 tiles of 256 x 256 (bound by the MFMAs, busy 52 % of all clocks, and by 32 tiles
// too few for the chip; a call after a pause, at a higher clock, 95); the library's product of bf16 weights, four times the bytes,
// takes 95.  61 x 4168 x 7168: 15 us (library 28), of which the sums of three splits are 2: a tile's copies land 1 us after they are
// asked for, two steps ahead, and bring quarter lines of the codes.
#include <algorithm>

#include "kernels.h"
#include "mx4.h"

namespace moe {

struct TileArgs {
  const bf16_t* x;
  const uint8_t* w;
  const uint8_t* s;
  int64_t M;
  int N, K;
  void* out;          // [M][N], or with more than one split of K the partial sums [splits][M][N] (fp32)
  int splits;
  int64_t plane;      // elements from one split's sums to the next's
};

__device__ __forceinline__ void copy4(const void* base, uint32_t offset, uint32_t lds) {   // as copy16, 4 bytes a lane
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 4\n\tglobal_load_lds_dword %0, %1"
               ::"v"(offset), "s"(base), "s"(lds) : "memory", "m0");
}
template <int N>
__device__ __forceinline__ void wait_copies() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

// G groups of WM x WN wavefronts have a part of K each, with a ring of its own, and join their sums in LDS.
template <int BM, int BN, int WM, int WN, int S, int G>
struct Tile4 {
  static constexpr int NW = WM * WN, WTM = BM / WM, WTN = BN / WN, FM = WTM / 32, FN = WTN / 32;
  static constexpr int PA = BM / 8, PB = BN / 32, PS = BN / 64;   // a stage's copies: x, codes, scales
  static constexpr int L = (PA + PB + PS + NW - 1) / NW;          // of one wavefront (past the last piece: that once more)
  static constexpr int A = 0, B = BM * 128, SC = B + BN * 32, STAGE = SC + BN * 4;
  static constexpr int RING = S * STAGE, RS = BN * 4 + 16;
  static constexpr int EPI = G == 1 ? NW * 32 * (WTN * 4 + 16) : G * BM * RS, LDS = G * RING > EPI ? G * RING : EPI;
};

typedef u32x4 __attribute__((aligned(2))) u32x4_any;
typedef u32x2 __attribute__((aligned(2))) u32x2_any;
typedef f32x4 __attribute__((aligned(4))) f32x4_any;

template <int BM, int BN, int WM, int WN, int S, int G, bool F32OUT>
__global__ __launch_bounds__(64 * WM * WN * G) void mx4_tile_kernel(TileArgs p) {
  using T = Tile4<BM, BN, WM, WN, S, G>;
  constexpr int NW = T::NW, FM = T::FM, FN = T::FN;
  extern __shared__ __attribute__((aligned(1024))) uint8_t lds[];
  const int tid = threadIdx.x, lane = tid & 63, all_waves = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int group = all_waves / NW, wave = all_waves % NW;
  const int lr = lane & 31, half = lane >> 5, wm = wave / WN, wn = wave % WN;
  // XCD b % 8 takes one run of the tiles, in groups of four rows of tiles: tiles that run together share x and W in its L2
  const int mt = (int)((p.M + BM - 1) / BM), nt = (p.N + BN - 1) / BN, all = mt * nt * p.splits, per = (all + 7) / 8;
  const int t = (int)(blockIdx.x & 7) * per + (int)(blockIdx.x >> 3);
  if (t >= all) return;
  const int z = t / (mt * nt), tz = t - z * (mt * nt), grp = tz / (4 * nt), gs = min(4, mt - 4 * grp), tg = tz - grp * 4 * nt;
  const int nb = tg / gs, mb = grp * 4 + tg - nb * gs;
  const int64_t m0 = (int64_t)mb * BM;
  const int n0 = nb * BN, rows = (int)min((int64_t)BM, p.M - m0), cols = min(BN, p.N - n0);
  const int KA = p.K / 128, parts = p.splits * G, part = z * G + group;
  const int k0 = (int)((int64_t)KA * part / parts) * 2, steps = (int)((int64_t)KA * (part + 1) / parts) * 2 - k0;
  const int rounds = (KA + parts - 1) / parts * 2;      // the most steps of a part
  uint8_t* const ring = lds + group * T::RING;
  const uint32_t rowb = (uint32_t)p.K / 2, lds0 = (uint32_t)(uintptr_t)ring;
  const uint8_t* xb = (const uint8_t*)(p.x + m0 * p.K) + (size_t)k0 * 128;
  const uint8_t* wb = p.w + (size_t)n0 * rowb + (size_t)k0 * 32;
  const uint8_t* sb = p.s + ((size_t)(k0 / 2) * p.N + n0) * 4;
  // 16-byte chunks of a row are swapped among themselves so that 16 lanes that read one chunk of 16 rows hit all banks
  uint32_t off[T::L];
#pragma unroll
  for (int c = 0; c < T::L; ++c) {
    const int q = min(NW * c + wave, T::PA + T::PB + T::PS - 1);
    if (q < T::PA) {
      const int r = q * 8 + (lane >> 3), k = (lane & 7) ^ ((r >> 1) & 7);
      off[c] = (uint32_t)min(r, rows - 1) * (uint32_t)p.K * 2 + k * 16;
    } else if (q < T::PA + T::PB) {
      const int r = (q - T::PA) * 32 + (lane >> 1), k = (lane & 1) ^ ((r >> 3) & 1);
      off[c] = (uint32_t)min(r, cols - 1) * rowb + k * 16;
    } else {
      off[c] = (uint32_t)min((q - T::PA - T::PB) * 64 + lane, cols - 1) * 4;
    }
  }
  auto copy = [&](int i, int c) __attribute__((always_inline)) {   // copy c of step i
    const uint32_t st = lds0 + (uint32_t)(i % S) * T::STAGE;
    const int q = min(NW * c + wave, T::PA + T::PB + T::PS - 1);
    if (q < T::PA) copy16(xb + (size_t)i * 128, off[c], __builtin_amdgcn_readfirstlane(st + T::A + q * 1024));
    else if (q < T::PA + T::PB) copy16(wb + (size_t)i * 32, off[c], __builtin_amdgcn_readfirstlane(st + T::B + (q - T::PA) * 1024));
    else copy4(sb + (size_t)(i / 2) * p.N * 4, off[c], __builtin_amdgcn_readfirstlane(st + T::SC + (q - T::PA - T::PB) * 256));
  };
  f32x16 acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;
  bf16x8 af[2][FM];
  u32x4 codes[FN];
  float scale[FN];
  bf16x8 wf[2][FN];
  auto read_a = [&](const uint8_t* st, int j, int i, int set) __attribute__((always_inline)) {
    const int r = wm * T::WTM + i * 32 + lr;
    af[set][i] = __builtin_bit_cast(bf16x8, *(const u32x4*)(st + T::A + r * 128 + (((4 * half + j) ^ ((r >> 1) & 7)) << 4)));
  };
#pragma unroll
  for (int i = 0; i < S - 1; ++i)
    if (i < steps)
#pragma unroll
      for (int c = 0; c < T::L; ++c) copy(i, c);
  for (int i = 0; i < rounds; ++i) {
    if (steps - 1 - i >= S - 2) wait_copies<(S - 2) * T::L>();   // step i's have landed
    else wait_copies<0>();
    lds_barrier();     // for all wavefronts; and the stage before is read
    if (i >= steps) continue;
    const uint8_t* st = ring + (i % S) * T::STAGE;
#pragma unroll
    for (int n = 0; n < FN; ++n) {
      const int r = wn * T::WTN + n * 32 + lr;
      codes[n] = *(const u32x4*)(st + T::B + r * 32 + ((half ^ ((r >> 3) & 1)) << 4));
      scale[n] = __uint_as_float(__builtin_amdgcn_ubfe(*(const uint32_t*)(st + T::SC + r * 4), 16 * ((k0 + i) & 1) + 8 * half, 8) << 23);
    }
#pragma unroll
    for (int q = 0; q < FM; ++q) read_a(st, 0, q, 0);
#pragma unroll
    for (int n = 0; n < FN; ++n) wf[0][n] = widen4(codes[n][0], scale[n]);
    const int ahead = i + S - 1 < steps ? i + S - 1 : -1;
    // the reads and conversions of MFMAs j + 1, and the copies, stand between the MFMAs j: the compiler would put all first
#pragma unroll
    for (int j = 0; j < 4; ++j) {
#pragma unroll
      for (int m = 0; m < FM * FN; ++m) {
        const int q = m / FN, n = m % FN;
        acc[q][n] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(wf[j & 1][n], af[j & 1][q], acc[q][n], 0, 0, 0);
        if (j < 3) {
          if (m < FM) read_a(st, j + 1, m, (j + 1) & 1);
          if (m >= FM * FN - FN) {
            const uint32_t word = codes[m - (FM * FN - FN)][j < 3 ? j + 1 : 0];
            wf[(j + 1) & 1][m - (FM * FN - FN)] = widen4(word, scale[m - (FM * FN - FN)]);
          }
        }
#pragma unroll
        for (int c = 0; c < T::L; ++c)
          if (c * 4 * FM * FN / T::L == j * FM * FN + m && ahead >= 0) copy(ahead, c);
        __builtin_amdgcn_sched_barrier(0);
      }
#pragma unroll
      for (int q = FM * FN; q < FM; ++q)
        if (j < 3) read_a(st, j + 1, q, (j + 1) & 1);
    }
  }
  if constexpr (G > 1) {
    __syncthreads();
#pragma unroll
    for (int q = 0; q < FM; ++q)
#pragma unroll
      for (int n = 0; n < FN; ++n)
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          const f32x16& a = acc[q][n];
          *(f32x4*)(lds + (group * BM + wm * T::WTM + q * 32 + lr) * T::RS + (wn * T::WTN + n * 32 + 8 * v + 4 * half) * 4) =
              f32x4{a[4 * v], a[4 * v + 1], a[4 * v + 2], a[4 * v + 3]};
        }
    __syncthreads();
    for (int k = tid; k < BM * BN / 4; k += 64 * NW * G) {
      const int row = k / (BN / 4), col = k % (BN / 4) * 4;
      if (row >= rows || col >= cols) continue;
      f32x4 sum = *(const f32x4*)(lds + row * T::RS + col * 4);
#pragma unroll
      for (int g = 1; g < G; ++g) sum += *(const f32x4*)(lds + (g * BM + row) * T::RS + col * 4);
      const int64_t at = (m0 + row) * p.N + n0 + col;
      if constexpr (F32OUT) {
        float* o = (float*)p.out + z * p.plane + at;
        if (col + 4 <= cols) *(f32x4_any*)o = sum;
        else
          for (int b = 0; b < cols - col; ++b) o[b] = sum[b];
      } else {
        bf16_t* o = (bf16_t*)p.out + at;
        if (col + 4 <= cols)
          *(u32x2_any*)o = u32x2{(uint32_t)f2bf(sum[0]) | (uint32_t)f2bf(sum[1]) << 16, (uint32_t)f2bf(sum[2]) | (uint32_t)f2bf(sum[3]) << 16};
        else
          for (int b = 0; b < cols - col; ++b) o[b] = f2bf(sum[b]);
      }
    }
    return;
  }
  // 32 rows of x at a time through this wavefront's part of LDS, so that a store covers whole pieces of a row
  constexpr int EB = F32OUT ? 4 : 2, RS = T::WTN * EB + 16, CPR = T::WTN * EB / 16;
  __syncthreads();
  uint8_t* own = lds + wave * 32 * (T::WTN * 4 + 16);
  uint8_t* out = (uint8_t*)p.out + (F32OUT ? (int64_t)z * p.plane * 4 : 0);
  const int nw0 = wn * T::WTN;
#pragma unroll
  for (int q = 0; q < FM; ++q) {
#pragma unroll
    for (int n = 0; n < FN; ++n)
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        uint8_t* to = own + lr * RS + (n * 32 + 8 * v + 4 * half) * EB;
        const f32x16& a = acc[q][n];
        if constexpr (F32OUT) *(f32x4*)to = f32x4{a[4 * v], a[4 * v + 1], a[4 * v + 2], a[4 * v + 3]};
        else *(u32x2*)to = u32x2{(uint32_t)f2bf(a[4 * v]) | (uint32_t)f2bf(a[4 * v + 1]) << 16,
                                 (uint32_t)f2bf(a[4 * v + 2]) | (uint32_t)f2bf(a[4 * v + 3]) << 16};
      }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    for (int k = lane; k < 32 * CPR; k += 64) {
      const int r = k / CPR, c = k % CPR, row = wm * T::WTM + q * 32 + r, col = nw0 + c * (16 / EB);
      if (row >= rows || col >= cols) continue;
      const u32x4 v = *(const u32x4*)(own + r * RS + c * 16);
      uint8_t* o = out + ((m0 + row) * p.N + n0 + col) * EB;
      if (col + 16 / EB <= cols) *(u32x4_any*)o = v;
      else
        for (int b = 0; b < cols - col; ++b) {
          if constexpr (F32OUT) ((uint32_t*)o)[b] = v[b];
          else ((uint16_t*)o)[b] = (uint16_t)(v[b >> 1] >> (16 * (b & 1)));
        }
    }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  }
}

// The splits' sums, in their order.
template <bool F32OUT>
__global__ __launch_bounds__(256) void mx4_join_kernel(const float* planes, int64_t plane, int splits, int64_t n, void* out) {
  const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
  if (i >= n) return;
  f32x4 sum = *(const f32x4*)(planes + i);         // (a plane is padded to whole fours)
#pragma unroll 8
  for (int z = 1; z < splits; ++z) sum += *(const f32x4*)(planes + z * plane + i);
  for (int c = 0; c < 4; ++c)
    if (i + c < n) {
      if (F32OUT) ((float*)out)[i + c] = sum[c];
      else ((bf16_t*)out)[i + c] = f2bf(sum[c]);
    }
}

// The tile shape and the splits of K.  A round of CUS workgroups takes K / splits times its shape's nanoseconds a column
// (measured with about 256 tiles), and splits add a launch and the traffic of their sums; the least is taken.  Measured, us:
// 61 x 4168 x 7168 64 x 64 in 3 splits 14.9, in one 23.7, in 4 21.5, 32 x 64 in 3 16.6; 32 x 4096 x 7168 32 x 64 in 4 splits 11.5,
// 64 x 64 in 4 13.2; 128 x 4096 x 4096 32 x 64 10.9, 64 x 64 14.5; 256 x 4096 x 4096 64 x 64 15.8, 64 x 128 20.9; 512 x 4096 x 4096
// 64 x 128 23.4, 64 x 64 30.1, 128 x 128 29.6; 1024 x 4096 x 4096 128 x 128 36.3, 64 x 128 42.0, 128 x 256 51;
// 1024 x 7168 x 2048 128 x 256 32.9, 128 x 128 36.5, 256 x 256 45.5; 2045 x 7168 x 4096 256 x 256 102, 128 x 256 108.
struct TilePlan {
  int kind, splits;
  int64_t tiles;
};
static TilePlan tile_plan(int64_t M, int64_t N, int64_t K) {
  constexpr struct { int bm, bn, groups; double ns; } shapes[] = {{32, 64, 4, 2.1},   {64, 64, 4, 3.5},    {64, 128, 2, 5.0},
                                                                   {128, 128, 2, 7.6}, {128, 256, 1, 12.8}, {256, 256, 1, 23.5}};
  TilePlan best{0, 1, 0};
  double least = 0;
  for (int k = 0; k < 6; ++k) {
    const int64_t tiles = (M + shapes[k].bm - 1) / shapes[k].bm * ((N + shapes[k].bn - 1) / shapes[k].bn);
    for (int s = 1; s <= 16 && (s == 1 || K >= 128 * (int64_t)s * shapes[k].groups); ++s) {
      const double join = s == 1 ? 0 : 2600 + (double)M * N * s * 8 / 2400;      // ns
      const double t = (double)((tiles * s + CUS - 1) / CUS) * K / s * shapes[k].ns + join;
      if (best.tiles == 0 || t < least) {
        best = {k, s, tiles};
        least = t;
      }
    }
  }
  return best;
}
size_t mx4_tile_workspace_bytes(int64_t M, int64_t N, int64_t K) {
  const TilePlan t = tile_plan(M, N, K);
  return t.splits == 1 ? 0 : (size_t)t.splits * ((M * N + 3) / 4 * 4) * sizeof(float);
}

template <int BM, int BN, int WM, int WN, int S, int G>
static hipError_t run_tiles(const TileArgs& a, bool f32, int64_t tiles, hipStream_t st) {
  using T = Tile4<BM, BN, WM, WN, S, G>;
  auto kern = f32 ? mx4_tile_kernel<BM, BN, WM, WN, S, G, true> : mx4_tile_kernel<BM, BN, WM, WN, S, G, false>;
  const hipError_t err = hipFuncSetAttribute((const void*)kern, hipFuncAttributeMaxDynamicSharedMemorySize, T::LDS);
  if (err != hipSuccess) return err;
  kern<<<(unsigned)((tiles * a.splits + 7) / 8 * 8), 64 * T::NW * G, T::LDS, st>>>(a);
  return hipGetLastError();
}

hipError_t launch_mx4_tiles(const void* x, const uint8_t* w, const uint8_t* w_scale, int64_t M, int64_t N, int64_t K, bool f32_out,
                            void* out, void* ws, hipStream_t st) {
  const TilePlan t = tile_plan(M, N, K);
  const int64_t plane = (M * N + 3) / 4 * 4;
  const bool join = t.splits > 1;
  const TileArgs a{(const bf16_t*)x, w, w_scale, M, (int)N, (int)K, join ? ws : out, t.splits, plane};
  const bool f32 = join || f32_out;
  hipError_t err;
  switch (t.kind) {
    case 0: err = run_tiles<32, 64, 1, 2, 3, 4>(a, f32, t.tiles, st); break;
    case 1: err = run_tiles<64, 64, 2, 2, 3, 4>(a, f32, t.tiles, st); break;
    case 2: err = run_tiles<64, 128, 2, 2, 3, 2>(a, f32, t.tiles, st); break;
    case 3: err = run_tiles<128, 128, 2, 2, 3, 2>(a, f32, t.tiles, st); break;
    case 4: err = run_tiles<128, 256, 2, 4, 3, 1>(a, f32, t.tiles, st); break;
    default: err = run_tiles<256, 256, 2, 4, 3, 1>(a, f32, t.tiles, st);
  }
  if (err != hipSuccess || !join) return err;
  const unsigned grid = (unsigned)((M * N + 1023) / 1024);
  if (f32_out) mx4_join_kernel<true><<<grid, 256, 0, st>>>((const float*)ws, plane, t.splits, M * N, out);
  else mx4_join_kernel<false><<<grid, 256, 0, st>>>((const float*)ws, plane, t.splits, M * N, out);
  return hipGetLastError();
}

}  // namespace moe
