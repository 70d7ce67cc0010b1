// Residual add and root-mean-square norm in front of the layer, and its gradient.
//
//   h = round(x + r);  rstd = (mean_i h_i^2 + eps)^-1/2;  y = h rstd w      (fp32 after h)
//   dx = dh + rstd (q - xh mean_i(q_i xh_i)),  xh = h rstd,  q = w dy;   dw = sum_t dy xh
//
// Both are one pass over the rows: a row sits in the registers of the lanes that own it
// between its sum and its outputs.  h is rounded before the norm, so that the gradient, which
// reads the stored h, is that of the very function the forward computed.
#include <algorithm>

#include "common.h"
#include "fp8.h"
#include "kernels.h"

namespace moe {

// Eight consecutive elements of an act row: as they are in memory, and as fp32.
template <bool F32>
struct Raw8 {
  u32x4 w[F32 ? 2 : 1];
};
template <bool F32>
__device__ __forceinline__ Raw8<F32> load_raw(const void* p, int64_t i) {
  Raw8<F32> r;
  if constexpr (F32) {
    r.w[0] = *(const u32x4*)((const float*)p + i);
    r.w[1] = *(const u32x4*)((const float*)p + i + 4);
  } else {
    r.w[0] = *(const u32x4*)((const bf16_t*)p + i);
  }
  return r;
}
template <bool F32>
__device__ __forceinline__ void widen8(const Raw8<F32>& r, float (&v)[8]) {
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    if constexpr (F32) {
      v[q] = __uint_as_float(r.w[0][q]);
      v[4 + q] = __uint_as_float(r.w[1][q]);
    } else {
      v[2 * q] = lo_bf(r.w[0][q]);
      v[2 * q + 1] = hi_bf(r.w[0][q]);
    }
  }
}
template <bool F32>
__device__ __forceinline__ void load8(const void* p, int64_t i, float (&v)[8]) {
  widen8<F32>(load_raw<F32>(p, i), v);
}

// Rows are written past the caches' retention (8,192 x 7168 with 8-bit rows: 111 -> 107 us).
template <bool F32>
__device__ __forceinline__ void store8(void* p, int64_t i, const float (&v)[8]) {
  if constexpr (F32) {
    __builtin_nontemporal_store(f32x4{v[0], v[1], v[2], v[3]}, (f32x4*)((float*)p + i));
    __builtin_nontemporal_store(f32x4{v[4], v[5], v[6], v[7]}, (f32x4*)((float*)p + i + 4));
  } else {
    __builtin_nontemporal_store(
        u32x4{pack_bf2(v[0], v[1]), pack_bf2(v[2], v[3]), pack_bf2(v[4], v[5]), pack_bf2(v[6], v[7])},
        (u32x4*)((bf16_t*)p + i));
  }
}

// Sum over the LANES threads that share a row (64: one wavefront; else the workgroup), in a
// fixed order.  `red` holds one float per wavefront.
template <int LANES>
__device__ __forceinline__ float row_sum(float v, float* red) {
  v = wave_sum(v);
  if constexpr (LANES > 64) {
    const int w = threadIdx.x >> 6;
    __syncthreads();   // the previous row's reads of red are over
    if ((threadIdx.x & 63) == 0) red[w] = v;
    __syncthreads();
    v = 0.f;
#pragma unroll
    for (int i = 0; i < LANES / 64; ++i) v += red[i];
  }
  return v;
}

struct NormArgs {
  const void* x;
  const void* r;
  const float* w;
  float eps;
  void* h;
  void* y;
  uint8_t* y8;
  void* y8_scale;
  float* rstd;
  int64_t T;
  int d;
};

// h of vector v of row t (x + r rounded to the act type, widened again).
template <bool F32>
__device__ __forceinline__ void norm_h(const NormArgs& p, int64_t at, float (&h)[8]) {
  load8<F32>(p.x, at, h);
  if (p.r) {
    float r[8];
    load8<F32>(p.r, at, r);
#pragma unroll
    for (int q = 0; q < 8; ++q) h[q] += r[q];
    if constexpr (!F32) {
#pragma unroll
      for (int q = 0; q < 8; ++q) h[q] = bf2f(f2bf(h[q]));
    }
  }
}

// The outputs of one vector.  Lanes whose vector is past the row's end (ok false) join the
// block maxima (their 16 lanes are past it together) and store nothing.
template <bool F32, int Q>
__device__ __forceinline__ void norm_out(const NormArgs& p, int64_t t, int v, bool ok, float rstd,
                                         const float (&h)[8]) {
  const int64_t at = t * p.d + v * 8;
  float y[8];
  if (ok) {
    if (p.h) store8<F32>(p.h, at, h);
    const f32x4 w0 = *(const f32x4*)(p.w + v * 8), w1 = *(const f32x4*)(p.w + v * 8 + 4);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      y[q] = h[q] * rstd * w0[q];
      y[4 + q] = h[4 + q] * rstd * w1[q];
    }
    if (p.y) store8<F32>(p.y, at, y);
  } else {
#pragma unroll
    for (int q = 0; q < 8; ++q) y[q] = 0.f;
  }
  if constexpr (Q == 1) {
    const float amax = block_amax<16>(y);
    const float s = fp8_scale(amax);
    const u32x2 c = fp8_encode8(y, s);
    if (ok) {
      *(u32x2*)(p.y8 + at) = c;
      if ((v & 15) == 0) ((float*)p.y8_scale)[(int64_t)(v / 16) * p.T + t] = s;
    }
  } else if constexpr (Q == 2) {
    const float amax = block_amax<4>(y);
    const bool bad = !(amax < INFINITY);
    const int X = mx_block_exp(amax);
    const uint32_t lo = e4m3_encode4(y[0], y[1], y[2], y[3], X);
    const uint32_t hi = e4m3_encode4(y[4], y[5], y[6], y[7], X);
    if (ok) {
      *(u32x2*)(p.y8 + at) = u32x2{lo, hi};
      if ((v & 3) == 0)
        ((uint8_t*)p.y8_scale)[((int64_t)(v / 16) * p.T + t) * 4 + ((v / 4) & 3)] =
            bad ? (uint8_t)255 : (uint8_t)(X + 127);
    }
  }
}

// Bound by memory: x, r, h, y and the codes each cross once (8,192 x 7168 bf16 with 8-bit rows: 107 us, 5.0 TB/s;
// a large copy reaches 4.8).  For a few rows by latency: two reads and the sum (6 us for 8).
//
// LANES threads per row, 256 threads per workgroup, NV vectors of 8 per thread in registers;
// NV = 0: a row too wide for that is read twice (every element by the thread that
// writes it, so h may be x or r there too).
template <bool F32, int Q, int LANES, int NV>
__global__ __launch_bounds__(256) void add_rmsnorm_kernel(NormArgs p) {
  __shared__ float red[4];
  const int64_t t = (int64_t)blockIdx.x * (256 / LANES) + threadIdx.x / LANES;
  if (t >= p.T) return;   // whole wavefronts (LANES = 64) or nobody (one row per workgroup)
  const int lane = threadIdx.x % LANES, nv = p.d / 8;
  float ss = 0.f;
  if constexpr (NV > 0) {
    float h[NV][8];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = lane + LANES * i;
      if (v < nv) norm_h<F32>(p, t * p.d + v * 8, h[i]);
      else {
#pragma unroll
        for (int q = 0; q < 8; ++q) h[i][q] = 0.f;
      }
    }
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int q = 0; q < 8; ++q) ss = fmaf(h[i][q], h[i][q], ss);
    const float rstd = 1.0f / sqrtf(row_sum<LANES>(ss, red) / (float)p.d + p.eps);
    if (lane == 0 && p.rstd) p.rstd[t] = rstd;
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (LANES * i < nv) norm_out<F32, Q>(p, t, lane + LANES * i, lane + LANES * i < nv, rstd, h[i]);
  } else {
    float h[8];
    for (int v = lane; v < nv; v += LANES) {
      norm_h<F32>(p, t * p.d + v * 8, h);
#pragma unroll
      for (int q = 0; q < 8; ++q) ss = fmaf(h[q], h[q], ss);
    }
    const float rstd = 1.0f / sqrtf(row_sum<LANES>(ss, red) / (float)p.d + p.eps);
    if (lane == 0 && p.rstd) p.rstd[t] = rstd;
    for (int v0 = 0; v0 < nv; v0 += LANES) {
      const int v = v0 + lane;
      if (v < nv) norm_h<F32>(p, t * p.d + v * 8, h);
      norm_out<F32, Q>(p, t, v, v < nv, rstd, h);
    }
  }
}

hipError_t launch_add_rmsnorm(bool f32, int q, const void* x, const void* residual, const float* w,
                              float eps, int64_t T, int d, void* h, void* y, uint8_t* y8,
                              void* y8_scale, float* rstd, hipStream_t st) {
  const NormArgs p{x, residual, w, eps, h, y, y8, y8_scale, rstd, T, d};
  const int nv = d / 8;
#define RUN(L, NV)                                                                              \
  {                                                                                             \
    const unsigned g = (unsigned)((T + 256 / L - 1) / (256 / L));                               \
    if (f32) add_rmsnorm_kernel<true, 0, L, NV><<<g, 256, 0, st>>>(p);                          \
    else if (q == 1) add_rmsnorm_kernel<false, 1, L, NV><<<g, 256, 0, st>>>(p);                 \
    else if (q == 2) add_rmsnorm_kernel<false, 2, L, NV><<<g, 256, 0, st>>>(p);                 \
    else add_rmsnorm_kernel<false, 0, L, NV><<<g, 256, 0, st>>>(p);                             \
  }
  if (nv <= 64) RUN(64, 1)
  else if (nv <= 256) RUN(256, 1)
  else if (nv <= 512) RUN(256, 2)
  else if (nv <= 1024) RUN(256, 4)
  else RUN(256, 0)
#undef RUN
  return hipGetLastError();
}

// ----------------------------------------------------------------------------- gradient
// A workgroup takes rows b, b + G, ... and keeps its columns' share of dw in registers; the
// G partial rows are then added in order.  Bound by memory: 8,192 x 4096 bf16 with dh takes 38 us (7.0 TB/s; 55
// without the next row's reads under way during a row's sum, 41 with stores that stay in the caches) and
// 5 us for the partial rows.
constexpr int NB_G = 512;

int norm_bwd_groups(int64_t T) { return (int)std::min<int64_t>(T, NB_G); }
size_t norm_bwd_workspace_bytes(int64_t T, int d) { return (size_t)norm_bwd_groups(T) * d * 4; }

__device__ __forceinline__ void store_part(float* at, const float (&v)[8]) {
  *(f32x4*)at = f32x4{v[0], v[1], v[2], v[3]};
  *(f32x4*)(at + 4) = f32x4{v[4], v[5], v[6], v[7]};
}

struct NormBwdArgs {
  const void* dy;
  const void* dh;
  const void* h;
  const float* w;
  const float* rstd;
  void* dx;
  float* part;   // [G, d], or NULL: no dw
  int64_t T;
  int d, G;
};

template <bool F32>
__device__ __forceinline__ void norm_bwd_out(const NormBwdArgs& p, int64_t at, const Raw8<F32>& dh, const float (&q)[8],
                                             const float (&xh)[8], float m, float rstd) {
  float o[8];
  widen8<F32>(dh, o);
#pragma unroll
  for (int i = 0; i < 8; ++i) o[i] = p.dh ? o[i] : 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) o[i] += rstd * (q[i] - xh[i] * m);
  store8<F32>(p.dx, at, o);
}

template <bool F32, int NV>
__global__ __launch_bounds__(256, 2) void rmsnorm_bwd_kernel(NormBwdArgs p) {
  __shared__ float red[4];
  const int tid = threadIdx.x, nv = p.d / 8;
  constexpr int KV = NV > 0 ? NV : 1;
  float dw[KV][8] = {}, w[KV][8];
  if constexpr (NV > 0) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = tid + 256 * i;
      if (v < nv) load8<true>(p.w, v * 8, w[i]);
    }
    // The next row is requested before this row's sum is joined, and dh before it is needed.  Loads are
    // unconditional (past the row's or the batch's end the last place again): a branch would make them wait.
    Raw8<F32> dy[NV], hh[NV], dh[NV];
    float rstd = p.rstd[blockIdx.x];
    const void* add = p.dh ? p.dh : p.dy;
    auto at = [&](int64_t t, int i) { return t * p.d + min(tid + 256 * i, nv - 1) * 8; };
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      dy[i] = load_raw<F32>(p.dy, at(blockIdx.x, i));
      hh[i] = load_raw<F32>(p.h, at(blockIdx.x, i));
    }
    for (int64_t t = blockIdx.x; t < p.T; t += p.G) {
      float q[NV][8], xh[NV][8], c = 0.f;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        dh[i] = load_raw<F32>(add, at(t, i));
        widen8<F32>(dy[i], q[i]);
        widen8<F32>(hh[i], xh[i]);
        if (tid + 256 * i < nv) {
#pragma unroll
          for (int u = 0; u < 8; ++u) {
            xh[i][u] *= rstd;
            dw[i][u] = fmaf(q[i][u], xh[i][u], dw[i][u]);
            q[i][u] *= w[i][u];
            c = fmaf(q[i][u], xh[i][u], c);
          }
        }
      }
      const int64_t next = min(t + p.G, p.T - 1);
      const float rstd_next = p.rstd[next];
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        dy[i] = load_raw<F32>(p.dy, at(next, i));
        hh[i] = load_raw<F32>(p.h, at(next, i));
      }
      const float m = row_sum<256>(c, red) / (float)p.d;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int v = tid + 256 * i;
        if (v < nv) norm_bwd_out<F32>(p, t * p.d + v * 8, dh[i], q[i], xh[i], m, rstd);
      }
      rstd = rstd_next;
    }
    if (p.part)
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int v = tid + 256 * i;
        if (v < nv) store_part(p.part + (int64_t)blockIdx.x * p.d + v * 8, dw[i]);
      }
  } else {
    // wide rows: read twice; the workgroup's own row of partials is kept in memory
    for (int64_t t = blockIdx.x; t < p.T; t += p.G) {
      const float rstd = p.rstd[t];
      float c = 0.f, q[8], xh[8];
      auto term = [&](int v) {
        load8<F32>(p.dy, t * p.d + v * 8, q);
        load8<F32>(p.h, t * p.d + v * 8, xh);
        load8<true>(p.w, v * 8, w[0]);
#pragma unroll
        for (int u = 0; u < 8; ++u) { xh[u] *= rstd; dw[0][u] = q[u] * xh[u]; q[u] *= w[0][u]; }
      };
      for (int v = tid; v < nv; v += 256) {
        term(v);
#pragma unroll
        for (int u = 0; u < 8; ++u) c = fmaf(q[u], xh[u], c);
        if (p.part) {
          float o[8];
          const int64_t at = (int64_t)blockIdx.x * p.d + v * 8;
          if (t != blockIdx.x) {
            load8<true>(p.part, at, o);
#pragma unroll
            for (int u = 0; u < 8; ++u) o[u] += dw[0][u];
          } else {
#pragma unroll
            for (int u = 0; u < 8; ++u) o[u] = dw[0][u];
          }
          store_part(p.part + at, o);
        }
      }
      const float m = row_sum<256>(c, red) / (float)p.d;
      for (int v = tid; v < nv; v += 256) {
        term(v);
        const int64_t at = t * p.d + v * 8;
        norm_bwd_out<F32>(p, at, load_raw<F32>(p.dh ? p.dh : p.dy, at), q, xh, m, rstd);
      }
    }
  }
}

// out[c] = sum over g of part[g, c]: 32 threads share a column, each adds rows g = its number
// mod 32 ascending, then the 32 sums in order.  Bound by the latency of a thread's loads: one thread per
// column took 131 us of the 187 us gradient at 8,192 x 4096, eight 4.9.
constexpr int CS = 32;
__global__ __launch_bounds__(32 * CS) void column_sum_kernel(const float* __restrict__ part, int G, int64_t d,
                                                             float* __restrict__ out) {
  __shared__ float red[CS][33];
  const int cl = threadIdx.x & 31, r = threadIdx.x >> 5;
  const int64_t c = (int64_t)blockIdx.x * 32 + cl;
  float s = 0.f;
  if (c < d) {
#pragma unroll 16
    for (int g = r; g < G; g += CS) s += part[(int64_t)g * d + c];
  }
  red[r][cl] = s;
  __syncthreads();
  if (r == 0 && c < d) {
    s = red[0][cl];
#pragma unroll
    for (int i = 1; i < CS; ++i) s += red[i][cl];
    out[c] = s;
  }
}

static hipError_t launch_column_sum(const float* part, int G, int64_t d, float* out, hipStream_t st) {
  column_sum_kernel<<<(unsigned)((d + 31) / 32), 32 * CS, 0, st>>>(part, G, d, out);
  return hipGetLastError();
}

hipError_t launch_rmsnorm_bwd(bool f32, const void* dy, const void* dh, const void* h, const float* w,
                              const float* rstd, int64_t T, int d, void* dx, float* dw, float* part,
                              hipStream_t st) {
  const int G = norm_bwd_groups(T), nv = d / 8;
  const NormBwdArgs p{dy, dh, h, w, rstd, dx, dw ? part : nullptr, T, d, G};
#define RUN(NV)                                                              \
  {                                                                          \
    if (f32) rmsnorm_bwd_kernel<true, NV><<<(unsigned)G, 256, 0, st>>>(p);   \
    else rmsnorm_bwd_kernel<false, NV><<<(unsigned)G, 256, 0, st>>>(p);      \
  }
  if (nv <= 256) RUN(1)
  else if (nv <= 512) RUN(2)
  else if (nv <= 1024) RUN(4)
  else RUN(0)
#undef RUN
  hipError_t err = hipGetLastError();
  if (err != hipSuccess || !dw) return err;
  return launch_column_sum(part, G, d, dw, st);
}

}  // namespace moe
