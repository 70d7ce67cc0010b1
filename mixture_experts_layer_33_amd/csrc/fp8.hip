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
// the result, far below a bf16 output's own half step (2e-3) and H's 8 bits, which is why
// the full fp8 rate is taken there.  An fp32 output asks for more: its codes are widened to
// bf16 (every E4M3 value is a bf16 value) and multiplied by the bf16 MFMA, whose sums are fp32
// (error against fp64 5e-7), at half the rate.
#include <algorithm>
#ifdef PROBE
#include <cstdlib>
#endif

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
// 16 token rows per tile; 8 wavefronts of 16 weight rows (SWIGLU: 16 gate and 16 up rows), so a
// workgroup covers one block of 128 output columns and a SWIGLU tile holds whole H blocks.
// Result i of lane l: output column n0 + 16 wave + 4 (l / 16) + i of token row l % 16.
template <bool SWIGLU, bool F32>
__global__ __launch_bounds__(512) void fp8_rows16_kernel(Fp8Args p) {
  __shared__ float hmax[8][16];
  const int nct = (p.N + 127) / 128;
  const int mt = blockIdx.x / nct, ct = blockIdx.x % nct;
  int e = 0, row0 = 16 * mt, rows;
  int64_t seg = 0;
  if (p.offset) {
    if (mt >= *p.ntiles) return;
    e = p.tiles[2 * mt];
    row0 = p.tiles[2 * mt + 1];
    seg = p.offset[e];
    rows = min(16, p.offset[e + 1] - (int)seg - row0);
  } else {
    rows = (int)min((int64_t)16, p.a_rows - row0);
  }
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, m = lane & 15, g = lane >> 4;
  const int KB = p.K / 128;
  const int64_t slot = ring_slot(p.head, seg, row0 + min(m, rows - 1), p.C);
  const uint8_t* a = p.A + slot * p.K + g * 32;
  const float* as = p.As + slot;
  const int64_t wrow = (int64_t)e * p.N + min(128 * ct + 16 * wave + m, p.N - 1);
  const uint8_t* w0 = p.W0 + wrow * p.K + g * 32;
  const uint8_t* w1 = SWIGLU ? p.W1 + wrow * p.K + g * 32 : nullptr;
  const float* s0 = p.S0 + ((int64_t)e * nct + ct) * KB;
  const float* s1 = SWIGLU ? p.S1 + ((int64_t)e * nct + ct) * KB : nullptr;
  f32x4 c0 = {0.f, 0.f, 0.f, 0.f}, c1 = c0;
#pragma unroll 4
  for (int b = 0; b < KB; ++b) {
    const i32x8 av = fp8_frag(a + (int64_t)b * 128);
    const float sa = as[b * p.a_rows];
    const i32x8 wv = fp8_frag(w0 + (int64_t)b * 128);
    const f32x4 q0 = F32 ? fp8_wide16(fp8_widen(wv), fp8_widen(av)) : fp8_mfma16(wv, av);
    const float t0 = sa * s0[b];
#pragma unroll
    for (int i = 0; i < 4; ++i) c0[i] = fmaf(q0[i], t0, c0[i]);
    if constexpr (SWIGLU) {
      const f32x4 q1 = fp8_mfma16(fp8_frag(w1 + (int64_t)b * 128), av);
      const float t1 = sa * s1[b];
#pragma unroll
      for (int i = 0; i < 4; ++i) c1[i] = fmaf(q1[i], t1, c1[i]);
    }
  }
  const int col = 128 * ct + 16 * wave + 4 * g;
  if constexpr (SWIGLU) {
    float h[4], am = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      h[i] = silu(c0[i]) * c1[i];
      am = amax2(am, h[i]);
    }
    am = amax2(am, __shfl_xor(am, 16, 64));
    am = amax2(am, __shfl_xor(am, 32, 64));
    if (g == 0) hmax[wave][m] = am;
    __syncthreads();
    am = 0.f;
#pragma unroll
    for (int w = 0; w < 8; ++w) am = amax2(am, hmax[w][m]);
    const float s = fp8_scale(am);
    if (m < rows) {
      *(uint32_t*)((uint8_t*)p.out + slot * p.N + col) = fp8_encode4(h[0], h[1], h[2], h[3], s);
      if (wave == 0 && g == 0) p.out_scale[(int64_t)ct * p.C + slot] = s;
      if (p.saved_au) {
        *(u32x2*)(p.saved_au + slot * 2 * p.N + col) = u32x2{pack_bf2(c0[0], c0[1]), pack_bf2(c0[2], c0[3])};
        *(u32x2*)(p.saved_au + (slot * 2 + 1) * p.N + col) = u32x2{pack_bf2(c1[0], c1[1]), pack_bf2(c1[2], c1[3])};
      }
    }
  } else if (m < rows) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (col + i < p.N) {
        if constexpr (F32) ((float*)p.out)[slot * p.N + col + i] = c0[i];
        else ((bf16_t*)p.out)[slot * p.N + col + i] = f2bf(c0[i]);
      }
  }
}

// ----------------------------------------------------------------------------- launchers
// Row tiles that take a column tile one after another (fp8_tile.h).
constexpr int FP8_GROUP = 4;

// Tile height (in 64 rows) of a product of M rows with `nct` column tiles of 256: the one with the least
// time, rounds of 256 workgroups times a stage's time.  Stages of 64 / 128 / 192 / 256 rows took
// 0.95, 0.98, 1.07 and 1.25 us (M 2,045, N 4,168, K 7,168): low tiles are bound by their
// weight copies, not by the matrix cores.
static int tile_height(int64_t M, int64_t nct) {
  const double us[4] = {0.95, 0.98, 1.07, 1.25};
  int best = 1;
  double least = 1e300;
  for (int fm = 1; fm <= 4; ++fm) {
    const double t = (double)(((M + 64 * fm - 1) / (64 * fm) * nct + 255) / 256) * us[fm - 1];
    if (t < least) { least = t; best = fm; }
  }
  return best;
}

hipError_t launch_tile_add(Fp8Args& a, hipStream_t st) {
  a.group = FP8_GROUP;
  const int fm = tile_height(a.a_rows, (a.N + 255) / 256);
  const int64_t mt = (a.a_rows + 64 * fm - 1) / (64 * fm);
  if (fm == 1) return run_fp8_tile<1, TILE_ADD, 3, 2>(a, mt, st);
  if (fm == 2) return run_fp8_tile<2, TILE_ADD, 3, 2>(a, mt, st);
  if (fm == 3) return run_fp8_tile<3, TILE_ADD, 2, 2>(a, mt, st);
  return run_fp8_tile<4, TILE_ADD, 2, 2>(a, mt, st);
}

size_t matmul_fp8_workspace_bytes(int64_t M, int64_t N, int64_t K) {
  (void)M; (void)N; (void)K;
  return 0;
}

hipError_t launch_matmul_fp8(const uint8_t* a, const float* a_scale, const uint8_t* w,
                             const float* w_scale, int64_t M, int64_t N, int64_t K, bool f32_out,
                             void* out, void* ws, hipStream_t st) {
  (void)ws;
  Fp8Args p{};
  p.A = a;
  p.As = a_scale;
  p.W0 = w;
  p.S0 = w_scale;
  p.a_rows = M;
  p.C = M;
  p.K = (int)K;
  p.N = (int)N;
  p.out = out;
#ifdef PROBE
  const int fm = getenv("FM") ? atoi(getenv("FM")) : 0;
#else
  const int fm = M <= 16 ? 0 : f32_out ? (M <= 64 ? 1 : 2) : tile_height(M, (N + 255) / 256);
#endif
  const int64_t mt = fm ? (M + 64 * fm - 1) / (64 * fm) : 0;
  p.group = FP8_GROUP;
  if (f32_out && fm == 1) return run_fp8_tile<1, FP8_F32, 3, 2>(p, mt, st);
  if (f32_out && fm) return run_fp8_tile<2, FP8_F32, 3, 2>(p, mt, st);
  if (fm == 1) return run_fp8_tile<1, FP8_BF16, 3, 2>(p, mt, st);
  if (fm == 2) return run_fp8_tile<2, FP8_BF16, 3, 2>(p, mt, st);
  if (fm == 3) return run_fp8_tile<3, FP8_BF16, 2, 2>(p, mt, st);
  if (fm == 4) return run_fp8_tile<4, FP8_BF16, 2, 2>(p, mt, st);
  const unsigned grid = (unsigned)(((M + 15) / 16) * ((N + 127) / 128));
  if (f32_out) fp8_rows16_kernel<false, true><<<grid, 512, 0, st>>>(p);
  else fp8_rows16_kernel<false, false><<<grid, 512, 0, st>>>(p);
  return hipGetLastError();
}

struct FfnFp8Layout {
  size_t tiles, h, hs, total;
};
static FfnFp8Layout ffn_fp8_layout(int64_t n, int64_t C, int E, int f) {
  auto al = [](size_t b) { return (b + 255) & ~(size_t)255; };
  FfnFp8Layout L;
  size_t o = 0;
  L.tiles = o; o += al((size_t)(2 * max_tiles_for(n, E, 16) + 64) * 4);
  L.h = o; o += al((size_t)C * f);
  L.hs = o; o += al((size_t)C * (f / 128) * 4);
  L.total = o;
  return L;
}
size_t ffn_fp8_workspace_bytes(int64_t n, int64_t C, int E, int f) { return ffn_fp8_layout(n, C, E, f).total; }

hipError_t launch_ffn_fp8(const void* ring_x, const float* ring_x_scale, const int32_t* expert_offset,
                          int64_t head, int64_t C, int64_t n, int d, int E, int f,
                          const void* w_gate, const void* w_up, const void* w_down,
                          const float* sg, const float* su, const float* sd, void* ring_y,
                          void* saved_au, void* ws, hipEvent_t* events, hipStream_t st) {
  const FfnFp8Layout L = ffn_fp8_layout(n, C, E, f);
  uint8_t* w = (uint8_t*)ws;
  int32_t* ntiles = (int32_t*)(w + L.tiles);
  int32_t* tiles = ntiles + 64;
  auto mark = [&](int i) { return events ? hipEventRecord(events[i], st) : hipSuccess; };
#ifdef PROBE
  const int fm = getenv("FM") ? atoi(getenv("FM")) : 0;
#else
  const int fm = n <= 16 * (int64_t)E ? 0 : n < 256 * (int64_t)E ? 2 : 4;
#endif
  const int BM = fm ? 64 * fm : 16;
  hipError_t err = launch_build_tiles(expert_offset, E, BM, tiles, ntiles, st);
  if (err != hipSuccess || (err = mark(0)) != hipSuccess) return err;
  const int mt = max_tiles_for(n, E, BM);
  const bool once = n <= BM * (int64_t)E;   // about one row tile per expert: each weight is read once
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
  p.tiles = tiles;
  p.ntiles = ntiles;
  p.head = head;
  p.C = C;
  p.out = w + L.h;
  p.out_scale = (float*)(w + L.hs);
  p.saved_au = (bf16_t*)saved_au;
#define RUN(FM, KIND, S, G)                                              \
  err = once ? run_fp8_tile<FM, KIND, S, 3>(G, mt, st) : run_fp8_tile<FM, KIND, S, 2>(G, mt, st);
  p.group = FP8_GROUP;
  if (fm == 0) {
    fp8_rows16_kernel<true, false><<<(unsigned)((int64_t)mt * (f / 128)), 512, 0, st>>>(p);
    err = hipGetLastError();
  } else if (fm == 1) {
    if (saved_au) RUN(1, FP8_SWIGLU_SAVE, 3, p) else RUN(1, FP8_SWIGLU, 3, p)
  } else if (fm == 2) {
    if (saved_au) RUN(2, FP8_SWIGLU_SAVE, 3, p) else RUN(2, FP8_SWIGLU, 3, p)
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
    fp8_rows16_kernel<false, false><<<(unsigned)((int64_t)mt * (d / 128)), 512, 0, st>>>(q);
    err = hipGetLastError();
  } else if (fm == 1) RUN(1, FP8_BF16, 3, q)
  else if (fm == 2) RUN(2, FP8_BF16, 3, q)
  else RUN(4, FP8_BF16, 2, q)
#undef RUN
  if (err != hipSuccess) return err;
  return mark(2);
}

}  // namespace moe
