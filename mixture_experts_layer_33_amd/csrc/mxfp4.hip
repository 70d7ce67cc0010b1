// MXFP4 weights: their quantisation, and the product of bf16 rows with them.
#include <algorithm>

#include "kernels.h"
#include "mx4.h"

namespace moe {

// ------------------------------------------------------------------ quantisation
// Four lanes hold one block of 32 (8 bf16 each).  X = floor(log2 amax) - 2 (2 = exponent of the largest E2M1 value 6 =
// 1.5 2^2), clamped to -127 below; code = RNE_E2M1(v / 2^X), values above 6 saturating.  gfx950's
// v_cvt_scalef32_pk_fp4_bf16 divides, rounds and saturates two values at once.  A block with an infinity or a NaN: byte 255.
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
// out[m][n] = sum_k x[m][k] W[n][k] for up to 16 rows of x: a weight stream.  A unit is 16 weight rows; a workgroup's
// wavefronts split its columns (wavefront w takes pairs w, w + NW, ...: together they read whole rows), keep
// their part of x in registers over all units of the workgroup, and join their 16 x 16 sums through LDS in a
// fixed order.  The next unit's codes are requested before a unit is multiplied.
struct Mx4Args {
  const bf16_t* x;
  const uint8_t* w;
  const uint8_t* s;
  int64_t M;
  int N, K;
  void* out;
};

template <int PPW, bool F32OUT>   // PPW: pairs a wavefront holds (x: 32 registers each)
__global__ __launch_bounds__(512) void mx4_vec_kernel(Mx4Args p, int units) {
  __shared__ __attribute__((aligned(16))) float part[2][8][256];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), NW = blockDim.x >> 6;
  const int g = lane >> 4, col = lane & 15, P = (p.K + 255) / 256;
  const int64_t m0 = (int64_t)blockIdx.y * 16;
  const int M = (int)min(p.M - m0, (int64_t)16);
  const int chunks = (P + NW * PPW - 1) / (NW * PPW);
  const uint32_t rowb = (uint32_t)p.K / 2;
  const __amdgpu_buffer_rsrc_t wr = buffer_of(p.w, (uint32_t)p.N * rowb);
  const bf16_t* xrow = p.x + (m0 + min(col, M - 1)) * p.K + 64 * g;
  bf16x8 x[PPW][8];
  auto load_x = [&](int chunk) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < PPW; ++i) {
      const int k = ((chunk * PPW + i) * NW + wave) * 256;
      const bool in = k + 64 * g < p.K;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const u32x4 v = *(const u32x4*)(xrow + (in ? k + 8 * j : -64 * g));
        x[i][j] = __builtin_bit_cast(bf16x8, in ? v : u32x4{0, 0, 0, 0});
      }
    }
  };
  const int u0 = (int)((int64_t)units * blockIdx.x / gridDim.x), u1 = (int)((int64_t)units * (blockIdx.x + 1) / gridDim.x);
  const int steps = (u1 - u0) * chunks;
  W4Pair w[2][PPW];
  auto load = [&](int step, auto set) __attribute__((always_inline)) {
    constexpr int S = decltype(set)::value;
    const int n0 = (u0 + step / chunks) * 16, chunk = step % chunks;
    const int ra = n0 + (lane & 7), rb = ra + 8, rs = min(n0 + col, p.N - 1);
#pragma unroll
    for (int i = 0; i < PPW; ++i) {
      const int pair = (chunk * PPW + i) * NW + wave;
      const uint32_t at = (uint32_t)pair * 128 + (lane >> 3) * 16;
      const bool in = at < rowb;
      w[S][i].a = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(
                                                wr, in && ra < p.N ? (uint32_t)ra * rowb + at : OUTSIDE, 0, NT_LOAD));
      w[S][i].b = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(
                                                wr, in && rb < p.N ? (uint32_t)rb * rowb + at : OUTSIDE, 0, NT_LOAD));
      const int kb = min(pair * 2 + (g >> 1), p.K / 128 - 1);
      w[S][i].s = *(const uint32_t*)(p.s + ((int64_t)kb * p.N + rs) * 4);
    }
  };
  f32x4 acc0{}, acc1{};
  auto consume = [&](int step, auto set) __attribute__((always_inline)) {
    constexpr int S = decltype(set)::value;
    const int unit = step / chunks, chunk = step % chunks;
    if (chunks > 1) load_x(chunk);
    if (chunk == 0) acc0 = acc1 = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < PPW; ++i) mul_pair(rows_of(w[S][i]), x[i], acc0, acc1);
    if (chunk != chunks - 1) return;
    float(*to)[256] = part[unit & 1];
    *(f32x4*)&to[wave][col * 16 + 4 * g] = acc0 + acc1;   // rows 4 g .. 4 g + 3 of token col
    lds_barrier();
    const int n0 = (u0 + unit) * 16;
    for (int q = tid; q < 16 * M; q += blockDim.x) {
      float sum = to[0][q];
      for (int v = 1; v < NW; ++v) sum += to[v][q];
      const int n = n0 + (q & 15);
      if (n < p.N) {
        const int64_t o = (m0 + (q >> 4)) * p.N + n;
        if (F32OUT) ((float*)p.out)[o] = sum;
        else ((bf16_t*)p.out)[o] = f2bf(sum);
      }
    }
  };
  using A = std::integral_constant<int, 0>;
  using B = std::integral_constant<int, 1>;
  if (steps > 0) load(0, A{});
  if (chunks == 1) load_x(0);
  for (int s = 0; s < steps; s += 2) {
    if (s + 1 < steps) load(s + 1, B{});
    consume(s, A{});
    if (s + 1 >= steps) break;
    if (s + 2 < steps) load(s + 2, A{});
    consume(s + 1, B{});
  }
}

size_t matmul_mxfp4_workspace_bytes(int64_t, int64_t, int64_t) { return 0; }

template <int PPW>
static void run_vec(const Mx4Args& a, bool f32_out, dim3 grid, int units, int nw, hipStream_t st) {
  if (f32_out) mx4_vec_kernel<PPW, true><<<grid, 64 * nw, 0, st>>>(a, units);
  else mx4_vec_kernel<PPW, false><<<grid, 64 * nw, 0, st>>>(a, units);
}

hipError_t launch_matmul_mxfp4(const void* x, const uint8_t* w, const uint8_t* w_scale, int64_t M, int64_t N, int64_t K,
                               bool f32_out, void* out, void*, hipStream_t st) {
  const Mx4Args a{(const bf16_t*)x, w, w_scale, M, (int)N, (int)K, out};
  const int units = (int)((N + 15) / 16), P = (int)((K + 255) / 256), nw = std::min(8, P);
  const int ppw = std::min(4, (P + nw - 1) / nw);
  for (int64_t m = 0; m < M; m += 16 * 65535) {   // grid.y
    Mx4Args b = a;
    b.x += m * K;
    b.out = (uint8_t*)out + m * N * (f32_out ? 4 : 2);
    b.M = std::min<int64_t>(M - m, 16 * 65535);
    const dim3 grid((unsigned)std::min(units, 256), (unsigned)((b.M + 15) / 16));
    switch (ppw) {
      case 1: run_vec<1>(b, f32_out, grid, units, nw, st); break;
      case 2: run_vec<2>(b, f32_out, grid, units, nw, st); break;
      case 3: run_vec<3>(b, f32_out, grid, units, nw, st); break;
      default: run_vec<4>(b, f32_out, grid, units, nw, st); break;
    }
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
  }
  return hipSuccess;
}

}  // namespace moe
