// MXFP4 weights: their quantisation, and the product of bf16 rows with them.
#include <algorithm>
#include <type_traits>

#include "kernels.h"
#include "mx4.h"

namespace moe {

// ------------------------------------------------------------------ quantisation
// Four lanes hold one block of 32 (8 bf16 each).  X = floor(log2 amax) - 2 (2 = exponent of the largest E2M1 value 6 =
// 1.5 2^2), clamped to -127 below; code = RNE_E2M1(v / 2^X), values above 6 saturating.  gfx950's
// v_cvt_scalef32_pk_fp4_bf16 divides, rounds and saturates two values at once.  A block with an infinity or a NaN: byte 255.
// What bounds it is HBM (2 bytes read and 17/32 written a value): 524,288 x 7168 1.95 ms (4.9 TB/s; a copy moves 4.8), 16,384 x 8192
// 76 us (4.5), 4,168 x 7168 20.5 us (3.7); one row 3.3 us, a launch.
__device__ __forceinline__ bf16x2_t pair_of(uint32_t v) { return __builtin_bit_cast(bf16x2_t, v); }

__global__ __launch_bounds__(256) void quantize_mxfp4_kernel(const bf16_t* __restrict__ src, int64_t nvec, int64_t rows,
                                                             int64_t vpr, uint32_t* __restrict__ codes,
                                                             uint8_t* __restrict__ scales) {
  const int64_t stride = (int64_t)gridDim.x * blockDim.x;
  const int64_t rounds = (nvec + stride - 1) / stride;
  for (int64_t it = 0; it < rounds; ++it) {
    const int64_t v = it * stride + (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    const bool ok = v < nvec;
    const u32x4 w = ok ? ((const u32x4*)src)[v] : u32x4{0, 0, 0, 0};
    float am = 0.f;
    bool odd = false;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      am = fmaxf(am, fmaxf(fabsf(lo_bf(w[q])), fabsf(hi_bf(w[q]))));
      odd = odd || (w[q] & 0x7f80u) == 0x7f80u || (w[q] & 0x7f800000u) == 0x7f800000u;
    }
    am = group_max<4>(odd ? INFINITY : am);
    const int ef = (int)(__float_as_uint(am) >> 23);
    const bool lost = ef == 255;
    const int X = ef == 0 ? -127 : max(ef - 127 - 2, -127);
    const float step = __uint_as_float((uint32_t)(X + 127) << 23);   // the conversion reads its exponent alone (0: 2^-127)
    uint32_t c = 0;
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, pair_of(w[0]), step, 0);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, pair_of(w[1]), step, 1);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, pair_of(w[2]), step, 2);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, pair_of(w[3]), step, 3);
    if (ok) {
      codes[v] = lost ? 0u : c;
      if ((v & 3) == 0) {   // block cb of row r: vpr = cols / 8 vectors per row
        const int64_t r = v / vpr, cb = (v - r * vpr) / 4;
        scales[((cb / 4) * rows + r) * 4 + (cb & 3)] = lost ? (uint8_t)255 : (uint8_t)(X + 127);
      }
    }
  }
}

hipError_t launch_quantize_mxfp4(const void* src, int64_t rows, int64_t cols, uint8_t* codes, uint8_t* scales,
                                 hipStream_t st) {
  const int64_t nvec = rows * cols / 8;
  if (nvec == 0) return hipSuccess;
  const int64_t blocks = std::min<int64_t>((nvec + 255) / 256, 65536);
  quantize_mxfp4_kernel<<<(unsigned)blocks, 256, 0, st>>>((const bf16_t*)src, nvec, rows, cols / 8, (uint32_t*)codes, scales);
  return hipGetLastError();
}

// ------------------------------------------------------------------ product, few rows
// out[m][n] = sum_k x[m][k] W[n][k] for few rows of x (few_rows): a weight stream (mx4.h).  A unit is 16 weight rows; a
// workgroup's NW wavefronts split its columns (wavefront w takes pairs w, w + NW, ...: together they read whole rows),
// keep their part of x in registers over all units of the workgroup (rows longer than NW PPW pairs, of up to eight tokens: read
// again for every chunk of them), and join their sums through LDS in a fixed order.  D chunks of codes are in flight, without a branch
// between their requests: what lies past the end has addresses outside its buffer.
// What bounds it is latency, of the launch, the first codes and x.  (Times here and in mxfp4_tile.hip: a call's, the median of replays
// of a graph of calls on different weights.)  1 x 7168 x 2048 5.4 us (1.5 TB/s), 8 x 4096 x 7168 8.0 (2.0 TB/s; with x read straight into
// the operand's layout the kernel took 9.9 where it takes 7.2), 12 x 16384 x 8192 20 (3.6 TB/s).
struct Mx4Args {
  const bf16_t* x;
  const uint8_t* w;
  const uint8_t* s;
  int64_t M;
  int N, K;
  void* out;
};

template <int PPW, int TS, int D, bool F32OUT>   // PPW: pairs a wavefront holds; TS: sets of eight rows of x
__global__ __launch_bounds__(512) void mx4_vec_kernel(Mx4Args p, int units) {
  __shared__ __attribute__((aligned(16))) float part[2][8][TS * 256];   // [half][first, second eight rows][row of x][row of W]
  constexpr int BLOCKS = PPW * TS < 4 ? PPW * TS : 4;     // of x on their way at a time
  __shared__ __attribute__((aligned(1024))) uint8_t stage[8][BLOCKS][XBLOCK];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), NW = blockDim.x >> 6;
  const int g = lane >> 4, col = lane & 15, chunk = lane >> 3, row = lane & 7, P = (p.K + 255) / 256;
  const int M = (int)p.M;
  const int chunks = TS == 1 ? (P + NW * PPW - 1) / (NW * PPW) : 1;
  const uint32_t rowb = (uint32_t)p.K / 2, srows = (uint32_t)p.N * 4;
  const __amdgpu_buffer_rsrc_t wr = buffer_of(p.w, (uint32_t)p.N * rowb), sr = buffer_of(p.s, (uint32_t)(p.K / 128) * srows);
  bf16x8 x[PPW][TS][4];
  auto first_column = [&](int c, int i) __attribute__((always_inline)) { return ((c * PPW + i) * NW + wave) * 256; };
  auto copy_x = [&](int c, int b0) __attribute__((always_inline)) {     // blocks b0 .. b0 + BLOCKS - 1: (pair, set)
#pragma unroll
    for (int b = 0; b < BLOCKS; ++b) {
      if (b0 + b >= PPW * TS) break;
      const int k = first_column(c, (b0 + b) / TS), s = (b0 + b) % TS, at = k < p.K ? k : 0, r0 = min(8 * s, M - 1);
      x_copy(p.x + (int64_t)r0 * p.K + at, M - 1 - r0, (uint32_t)p.K, p.K - at, (uint32_t)(uintptr_t)stage[wave][b]);
    }
  };
  auto read_x = [&](int c, int b0) __attribute__((always_inline)) {
#pragma unroll
    for (int b = 0; b < BLOCKS; ++b)
      if (b0 + b < PPW * TS)
        x_read(stage[wave][b], first_column(c, (b0 + b) / TS) + 64 * g + 32 * (col >> 3) < p.K,
               x[(b0 + b) / TS][(b0 + b) % TS]);
  };
  auto rest_of_x = [&](int c) __attribute__((always_inline)) {          // the first blocks are copied
    read_x(c, 0);
#pragma unroll
    for (int b0 = BLOCKS; b0 < PPW * TS; b0 += BLOCKS) {
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");                // the blocks before are read
      copy_x(c, b0);
      wait_all();
      read_x(c, b0);
    }
  };
  const int u0 = (int)((int64_t)units * blockIdx.x / gridDim.x), u1 = (int)((int64_t)units * (blockIdx.x + 1) / gridDim.x);
  const int steps = (u1 - u0) * chunks;
  W4Pair w[D][PPW];
  int n = -1, unit = u0, c = -1;            // the step whose loads come next
  uint32_t oa = OUTSIDE, ob = OUTSIDE, sa = 0, sb = 0;
  auto next = [&]() __attribute__((always_inline)) {
    ++n;
    if (++c == chunks) {
      c = 0;
      ++unit;
    }
    const int ra = unit * 16 + row, rb = ra + 8;
    oa = n < steps && ra < p.N ? ra * rowb + chunk * 16 : OUTSIDE;
    ob = n < steps && rb < p.N ? rb * rowb + chunk * 16 : OUTSIDE;
    sa = min(ra, p.N - 1) * 4;
    sb = min(rb, p.N - 1) * 4;
  };
  auto load = [&](W4Pair& q, int i) __attribute__((always_inline)) {
    const uint32_t pair = (c * PPW + i) * NW + wave;
    const bool in = pair * 128 + chunk * 16 < rowb;
    const uint32_t kb = in ? pair * 2 + (chunk >> 2) : 0;
    q.a = load_b128_nt(wr, in ? oa + pair * 128 : OUTSIDE, 0);
    q.b = load_b128_nt(wr, in ? ob + pair * 128 : OUTSIDE, 0);
    q.sa = load_b32(sr, kb * srows + sa, 0);
    q.sb = load_b32(sr, kb * srows + sb, 0);
  };
  f32x4 aa[TS], ab[TS];
  auto step = [&](int m, auto set) __attribute__((always_inline)) {
    constexpr int S = decltype(set)::value;
    const int mu = m / chunks, mc = m % chunks;
    if (chunks > 1) {
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
      copy_x(mc, 0);
      wait_all();
      rest_of_x(mc);
    }
    if (mc == 0) {
#pragma unroll
      for (int s = 0; s < TS; ++s) aa[s] = ab[s] = f32x4{0.f, 0.f, 0.f, 0.f};
    }
    next();
#pragma unroll
    for (int i = 0; i < PPW; ++i) {
      const float fa = chunk_scale(w[S][i].sa), fb = chunk_scale(w[S][i].sb);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const bf16x8 a = widen4(w[S][i].a[j], fa), b = widen4(w[S][i].b[j], fb);
#pragma unroll
        for (int s = 0; s < TS; ++s) {
          aa[s] = mfma16(a, x[i][s][j], aa[s]);
          ab[s] = mfma16(b, x[i][s][j], ab[s]);
        }
      }
      load(w[S][i], i);
      __builtin_amdgcn_sched_barrier(0);
    }
    if (mc != chunks - 1 || m >= steps) return;
    if (holds_half()) {
#pragma unroll
      for (int s = 0; s < TS; ++s) {
        float* to = part[mu & 1][wave] + s * 256 + (col >> 3) * 128 + (col & 7) * 8 + 4 * (g & 1);
        *(f32x4*)to = aa[s];
        *(f32x4*)(to + 64) = ab[s];
      }
    }
    lds_barrier();
    for (int q = tid; q < 16 * M; q += blockDim.x) {
      const int r = q & 15, t = q >> 4, o = (u0 + mu) * 16 + r;
      if (o >= p.N) continue;
      const int at = (t >> 3) * 256 + (r >> 3) * 64 + (t & 7) * 8 + (r & 7);
      float sum = 0.f;
      for (int v = 0; v < NW; ++v) sum += part[mu & 1][v][at] + part[mu & 1][v][at + 128];
      if (F32OUT) ((float*)p.out)[(int64_t)t * p.N + o] = sum;
      else ((bf16_t*)p.out)[(int64_t)t * p.N + o] = f2bf(sum);
    }
  };
  copy_x(0, 0);
#pragma unroll
  for (int s = 0; s < D; ++s) {
    next();
#pragma unroll
    for (int i = 0; i < PPW; ++i) load(w[s][i], i);
  }
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(4 * D * PPW) : "memory");    // the copies: only the loads are behind them
  if (chunks == 1) rest_of_x(0);
  for (int m = 0; m < steps; m += D) unrolled<D>([&](auto s) __attribute__((always_inline)) { step(m + decltype(s)::value, s); });
}

// Up to 8 rows the product is a stream of W, and up to 16 while all of x stays in registers; more are tiles (mxfp4_tile.hip).
// Stream | tiles, us: 8 x 4096 x 12288 13.5 | 15.1, 8 x 8192 x 28672 39.8 | 43.5; 16 x 512 x 1024 3.6 | 5.2, 12 x 2048 x 4096 5.9 | 8.7,
// 16 x 7168 x 8192 14.2 | 16.7, 9 x 4096 x 8192 10.6 | 11.7; longer rows, read again for every unit: 16 x 512 x 9216 14.5 | 9.7,
// 12 x 7168 x 9216 24.6 | 18.2, 16 x 4096 x 12288 17.1 | 15.3, 16 x 1024 x 28672 27.3 | 12.8.
static bool few_rows(int64_t M, int64_t K) { return M <= 8 || (M <= 16 && K <= 8192); }
size_t matmul_mxfp4_workspace_bytes(int64_t M, int64_t N, int64_t K) {
  return few_rows(M, K) ? 0 : mx4_tile_workspace_bytes(M, N, K);
}

template <int PPW>
static void run_vec(const Mx4Args& a, bool f32_out, dim3 grid, int units, int nw, hipStream_t st) {
  // One unit in flight: a workgroup has one to four at these sizes, and a second one's requests (or those past the end) delay the
  // first one's codes.  One | two, us: 1 x 7168 x 2048 (448 units on 256 workgroups) 5.3 | 5.4, 1 x 4096 x 7168 7.8 | 9.7, 8 x 4096 x
  // 7168 7.8 | 9.9, 12 x 16384 x 8192 20 | 25.6; two would win where many units are short: 1 x 16384 x 2048 7.8 | 7.1.
  constexpr int D = 1;
  if (a.M > 8) {
    if (f32_out) mx4_vec_kernel<PPW, 2, D, true><<<grid, 64 * nw, 0, st>>>(a, units);
    else mx4_vec_kernel<PPW, 2, D, false><<<grid, 64 * nw, 0, st>>>(a, units);
  } else {
    if (f32_out) mx4_vec_kernel<PPW, 1, D, true><<<grid, 64 * nw, 0, st>>>(a, units);
    else mx4_vec_kernel<PPW, 1, D, false><<<grid, 64 * nw, 0, st>>>(a, units);
  }
}

hipError_t launch_matmul_mxfp4(const void* x, const uint8_t* w, const uint8_t* w_scale, int64_t M, int64_t N, int64_t K,
                               bool f32_out, void* out, void* ws, hipStream_t st) {
  if (!few_rows(M, K)) return launch_mx4_tiles(x, w, w_scale, M, N, K, f32_out, out, ws, st);
  const Mx4Args a{(const bf16_t*)x, w, w_scale, M, (int)N, (int)K, out};
  const int units = (int)((N + 15) / 16), P = (int)((K + 255) / 256), nw = std::min(8, P);
  const int ppw = std::min(4, (P + nw - 1) / nw);
  const dim3 grid((unsigned)std::min(units, CUS));
  switch (ppw) {
    case 1: run_vec<1>(a, f32_out, grid, units, nw, st); break;
    case 2: run_vec<2>(a, f32_out, grid, units, nw, st); break;
    case 3: run_vec<3>(a, f32_out, grid, units, nw, st); break;
    default: run_vec<4>(a, f32_out, grid, units, nw, st);
  }
  return hipGetLastError();
}

}  // namespace moe
