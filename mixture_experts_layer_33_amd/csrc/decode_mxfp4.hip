// The whole layer for a few tokens with MXFP4 weights: scored routing, then gate/up with SwiGLU over the experts that
// the tokens chose (and the shared one), then down and the gate-weighted sum.
//
//   h_tj = g_tj silu(W_gate[e] x_t) * (W_up[e] x_t)   (e: the j-th expert of token t; the shared expert's gate is 1)
//   y_t  = sum_j W_down[e_tj] h_tj + W_s_down h_ts
//
// Every used expert's weights are read once, whatever the number of tokens that chose it: the tokens are the 16
// columns of the MFMA's second operand.  h is formed in fp32 and kept as two bf16 parts, hi = bf16(h) and
// lo = bf16(h - hi) (2^-17 of h is left out; y's own rounding is 2^-9).  Up to eight tokens the two parts are
// columns t and t + 8 of one product, above that two products.
#include <algorithm>

#include "kernels.h"
#include "mx4.h"

namespace moe {

constexpr int D4_TMAX = 16;     // tokens
constexpr int D4_KMAX = 16;     // top-k
constexpr int D4_PAIRS = D4_TMAX * D4_KMAX;
constexpr int D4_ROWS = 32;     // most output rows of a workgroup of the down product

struct D4Args {
  const bf16_t* x;
  const uint8_t *w_gate, *w_up, *w_down, *s_gate, *s_up, *s_down;        // codes and scale bytes of the expert stacks
  const uint8_t *ws_gate, *ws_up, *ws_down, *ss_gate, *ss_up, *ss_down;   // the shared expert's
  int T, d, E, k, f, fs;
  const int32_t* topk_idx;
  const float* topk_gate;
  bf16_t* h;       // [2][T k][f] (hi, lo), then the shared expert's [2][T][fs]
  bf16_t* y;
};

// The experts that the tokens chose, ascending, and which token has which of them as its how-manieth.
struct D4List {
  uint32_t bits[32];                      // E <= 1024
  int32_t expert[D4_PAIRS];
  uint8_t slot[D4_PAIRS][D4_TMAX];        // [place in the list][token]: j + 1, 0: not chosen
  int32_t U;
};

__device__ __forceinline__ void d4_list(const D4Args& p, D4List& L) {
  const int tid = threadIdx.x, n = p.T * p.k;
  if (tid < 32) L.bits[tid] = 0u;
  for (int i = tid; i < D4_PAIRS * D4_TMAX / 4; i += blockDim.x) ((uint32_t*)L.slot)[i] = 0u;
  __syncthreads();
  for (int q = tid; q < n; q += blockDim.x) {
    const int e = p.topk_idx[q];
    atomicOr(&L.bits[e >> 5], 1u << (e & 31));
  }
  __syncthreads();
  for (int q = tid; q < n; q += blockDim.x) {
    const int e = p.topk_idx[q];
    int at = __popc(L.bits[e >> 5] & ((1u << (e & 31)) - 1u));
    for (int w = 0; w < (e >> 5); ++w) at += __popc(L.bits[w]);
    L.expert[at] = e;
    L.slot[at][q / p.k] = (uint8_t)(q % p.k + 1);
  }
  if (tid == 0) {
    int u = 0;
    for (int w = 0; w < 32; ++w) u += __popc(L.bits[w]);
    L.U = u;
  }
  __syncthreads();
}

// ------------------------------------------------------------------ gate and up
// A unit is eight columns of f of one expert: an MFMA tile of their eight W_gate rows over their eight W_up rows.  The
// workgroup's wavefronts split d and keep their part of the tokens in registers over all units.
template <int PPW>
__global__ __launch_bounds__(512) void d4_up_kernel(D4Args p) {
  __shared__ D4List L;
  __shared__ __attribute__((aligned(16))) float part[2][8][256];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), NW = blockDim.x >> 6;
  const int g = lane >> 4, col = lane & 15;
  const uint32_t rowb = (uint32_t)p.d / 2;
  bf16x8 x[PPW][8];
#pragma unroll
  for (int i = 0; i < PPW; ++i) {
    const int k = (i * NW + wave) * 256;
    const bool in = k + 64 * g < p.d;
    const bf16_t* xr = p.x + (int64_t)min(col, p.T - 1) * p.d + (in ? k + 64 * g : 0);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const u32x4 v = *(const u32x4*)(xr + 8 * j);
      x[i][j] = __builtin_bit_cast(bf16x8, in ? v : u32x4{0, 0, 0, 0});
    }
  }
  d4_list(p, L);
  // this workgroup's units: a share of the shared expert's, then of the routed ones
  const int U = L.U, per = p.f / 8, su = p.fs / 8, ru = U * per, G = gridDim.x, b = blockIdx.x;
  const int s0 = (int)((int64_t)su * b / G), s1 = (int)((int64_t)su * (b + 1) / G);
  const int r0 = (int)((int64_t)ru * b / G), r1 = (int)((int64_t)ru * (b + 1) / G);
  const int ns = s1 - s0, steps = ns + r1 - r0;
  W4Pair w[2][PPW];
  auto load = [&](int step, auto set) __attribute__((always_inline)) {
    constexpr int S = decltype(set)::value;
    const bool shared = step < ns;
    const int unit = shared ? s0 + step : r0 + step - ns;
    const int at = shared ? 0 : unit / per, i0 = (shared ? unit : unit % per) * 8;
    const int e = __builtin_amdgcn_readfirstlane(shared ? 0 : L.expert[at]), F = shared ? p.fs : p.f;
    const uint32_t bytes = (uint32_t)F * rowb;
    const __amdgpu_buffer_rsrc_t gr = buffer_of((shared ? p.ws_gate : p.w_gate) + (int64_t)e * bytes, bytes);
    const __amdgpu_buffer_rsrc_t ur = buffer_of((shared ? p.ws_up : p.w_up) + (int64_t)e * bytes, bytes);
    const int64_t rows = shared ? p.fs : (int64_t)p.E * p.f;
    const uint8_t* sc = col < 8 ? (shared ? p.ss_gate : p.s_gate) : (shared ? p.ss_up : p.s_up);
    const uint8_t* sr = sc + ((int64_t)e * F + i0 + (col & 7)) * 4;
#pragma unroll
    for (int i = 0; i < PPW; ++i) {
      const int pair = i * NW + wave;
      const uint32_t off = (uint32_t)pair * 128 + (lane >> 3) * 16;
      const uint32_t o = off < rowb ? (uint32_t)(i0 + (lane & 7)) * rowb + off : OUTSIDE;
      w[S][i].a = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(gr, o, 0, NT_LOAD));
      w[S][i].b = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(ur, o, 0, NT_LOAD));
      const int kb = min(pair * 2 + (g >> 1), p.d / 128 - 1);
      w[S][i].s = *(const uint32_t*)(sr + kb * rows * 4);
    }
  };
  auto consume = [&](int step, auto set) __attribute__((always_inline)) {
    constexpr int S = decltype(set)::value;
    f32x4 acc0{}, acc1{};
#pragma unroll
    for (int i = 0; i < PPW; ++i) mul_pair(rows_of(w[S][i]), x[i], acc0, acc1);
    float(*to)[256] = part[S];
    *(f32x4*)&to[wave][col * 16 + 4 * g] = acc0 + acc1;
    lds_barrier();
    for (int o8 = tid; o8 < 8 * p.T; o8 += blockDim.x) {
      const bool shared = step < ns;
      const int unit = shared ? s0 + step : r0 + step - ns;
      const int at = shared ? 0 : unit / per, i = (shared ? unit : unit % per) * 8 + (o8 & 7), t = o8 >> 3;
      const int j = shared ? 1 : (int)L.slot[at][t];
      if (j > 0) {
        const int q = t * 16 + (o8 & 7);
        float a = to[0][q], u = to[0][q + 8];
        for (int v = 1; v < NW; ++v) {
          a += to[v][q];
          u += to[v][q + 8];
        }
        float h = silu(a) * u;
        const int64_t n = (int64_t)p.T * p.k * p.f;
        if (!shared) h *= p.topk_gate[t * p.k + j - 1];
        const bf16_t hi = f2bf(h), lo = f2bf(fabsf(h) < 3.39e38f ? h - bf2f(hi) : 0.f);   // an infinite hi has no rest
        bf16_t* o = shared ? p.h + 2 * n + (int64_t)t * p.fs + i : p.h + (int64_t)(t * p.k + j - 1) * p.f + i;
        o[0] = hi;
        o[shared ? (int64_t)p.T * p.fs : n] = lo;
      }
    }
  };
  using A = std::integral_constant<int, 0>;
  using B = std::integral_constant<int, 1>;
  if (steps > 0) load(0, A{});
  for (int s = 0; s < steps; s += 2) {
    if (s + 1 < steps) load(s + 1, B{});
    consume(s, A{});
    if (s + 1 >= steps) break;
    if (s + 2 < steps) load(s + 2, A{});
    consume(s + 1, B{});
  }
}

// ------------------------------------------------------------------ down
// A workgroup owns RW <= 16 NT output rows.  The columns of all used experts (then the shared one's) are one long sum, cut into
// pairs of 256 that the wavefronts take in turn; a token that did not choose an expert reads zeros.
template <int NT, bool MANY>   // MANY: more than eight tokens
__global__ __launch_bounds__(512) void d4_down_kernel(D4Args p, int RW) {
  __shared__ D4List L;
  __shared__ __attribute__((aligned(16))) float part[NT][8][256];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), NW = blockDim.x >> 6;
  const int g = lane >> 4, col = lane & 15, t = MANY ? col : col & 7;
  d4_list(p, L);
  const int U = L.U, per = (p.f + 255) / 256, pers = (p.fs + 255) / 256, steps = U * per + pers;
  const int64_t n = (int64_t)p.T * p.k * p.f, ns = (int64_t)p.T * p.fs;
  const __amdgpu_buffer_rsrc_t hr = buffer_of(p.h, (uint32_t)(4 * (n + ns)));
  constexpr int PL = MANY ? 2 : 1;   // parts of h a lane holds
  struct Step {
    W4Pair w[NT];
    u32x4 h[PL][8];
  };
  for (int o0 = blockIdx.x * RW; o0 < p.d; o0 += gridDim.x * RW) {
    const int rows = min(RW, p.d - o0);
    auto load = [&](int step, Step& s) __attribute__((always_inline)) {
      const bool shared = step >= U * per;
      const int at = shared ? 0 : step / per, pair = shared ? step - U * per : step % per;
      const int e = __builtin_amdgcn_readfirstlane(shared ? 0 : L.expert[at]), F = shared ? p.fs : p.f;
      const uint32_t rowb = (uint32_t)F / 2, bytes = (uint32_t)p.d * rowb;
      const __amdgpu_buffer_rsrc_t wr = buffer_of((shared ? p.ws_down : p.w_down) + (int64_t)e * bytes, bytes);
      const uint32_t off = (uint32_t)pair * 128 + (lane >> 3) * 16;
      const int kb = min(pair * 2 + (g >> 1), F / 128 - 1);
      const uint8_t* sr = (shared ? p.ss_down : p.s_down) + ((int64_t)kb * (shared ? p.d : (int64_t)p.E * p.d) + (int64_t)e * p.d) * 4;
#pragma unroll
      for (int r = 0; r < NT; ++r) {
        const int ra = 16 * r + (lane & 7), rb = ra + 8;
        s.w[r].a = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(
                                                 wr, ra < rows && off < rowb ? (uint32_t)(o0 + ra) * rowb + off : OUTSIDE, 0, NT_LOAD));
        s.w[r].b = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(
                                                 wr, rb < rows && off < rowb ? (uint32_t)(o0 + rb) * rowb + off : OUTSIDE, 0, NT_LOAD));
        s.w[r].s = *(const uint32_t*)(sr + (int64_t)min(o0 + 16 * r + col, p.d - 1) * 4);
      }
      const int j = t >= p.T ? 0 : shared ? 1 : (int)L.slot[at][t], k0 = pair * 256 + 64 * g;
      const int64_t row = shared ? 2 * n + (int64_t)t * p.fs : (int64_t)(t * p.k + j - 1) * p.f;
#pragma unroll
      for (int q = 0; q < PL; ++q) {
        const int64_t plane = (MANY ? q : col >> 3) * (shared ? ns : n);
        const uint32_t o = j > 0 && k0 < F ? (uint32_t)(2 * (plane + row + k0)) : OUTSIDE;
#pragma unroll
        for (int i = 0; i < 8; ++i)
          s.h[q][i] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(hr, o == OUTSIDE ? o : o + 16 * i, 0, 0));
      }
    };
    f32x4 acc[NT][2];
#pragma unroll
    for (int r = 0; r < NT; ++r) acc[r][0] = acc[r][1] = f32x4{0.f, 0.f, 0.f, 0.f};
    auto consume = [&](const Step& s) __attribute__((always_inline)) {
#pragma unroll
      for (int r = 0; r < NT; ++r) {
        const W4Rows w = rows_of(s.w[r]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const bf16x8 wp = widen4(w.p[i], w.sp), wq = widen4(w.q[i], w.sq);
#pragma unroll
          for (int q = 0; q < PL; ++q) {
            acc[r][0] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wp, __builtin_bit_cast(bf16x8, s.h[q][i]), acc[r][0], 0, 0, 0);
            acc[r][1] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wq, __builtin_bit_cast(bf16x8, s.h[q][4 + i]), acc[r][1], 0, 0, 0);
          }
        }
      }
    };
    Step sa, sb;
    if (wave < steps) load(wave, sa);
    for (int s = wave; s < steps; s += 2 * NW) {
      if (s + NW < steps) load(s + NW, sb);
      consume(sa);
      if (s + NW >= steps) break;
      if (s + 2 * NW < steps) load(s + 2 * NW, sa);
      consume(sb);
    }
#pragma unroll
    for (int r = 0; r < NT; ++r) *(f32x4*)&part[r][wave][col * 16 + 4 * g] = acc[r][0] + acc[r][1];
    __syncthreads();
    for (int q = tid; q < 16 * NT * p.T; q += blockDim.x) {
      const int r = q % (16 * NT), tok = q / (16 * NT);
      if (r < rows) {
        const float(*from)[256] = part[r / 16];
        const int at = tok * 16 + r % 16;
        float sum = 0.f;
        for (int v = 0; v < NW; ++v) sum += MANY ? from[v][at] : from[v][at] + from[v][at + 128];
        p.y[(int64_t)tok * p.d + o0 + r] = f2bf(sum);
      }
    }
    __syncthreads();
  }
}

// Workspace: the router's logit planes | expert counts [E] | h [2][T k f] | [2][T fs].
static size_t d4_route_bytes(int T, int E, int d) {
  const size_t b = std::max(route_workspace_bytes(T, E, d), route_scored_workspace_bytes(T, E, d));
  return (b + 255) & ~(size_t)255;
}
size_t decode_mxfp4_workspace_bytes(int T, int d, int E, int k, int f, int fs) {
  return d4_route_bytes(T, E, d) + 4096 + 4 * ((size_t)T * k * f + (size_t)T * fs);
}

hipError_t launch_decode_mxfp4(const void* x, const float* w_r, const float* b_r, const float* balance, const ScoreRule& rule,
                               const Mx4Weights& w, const Mx4Weights& shared, int T, int d, int E, int k, int f, int fs, void* y,
                               int32_t* topk_idx, float* topk_gate, void* ws, hipStream_t st) {
  int dev = 0, ncu = 0;
  hipError_t err = hipGetDevice(&dev);
  if (err != hipSuccess) return err;
  if ((err = hipDeviceGetAttribute(&ncu, hipDeviceAttributeMultiprocessorCount, dev)) != hipSuccess) return err;
  uint8_t* base = (uint8_t*)ws;
  int32_t* count = (int32_t*)(base + d4_route_bytes(T, E, d));
  err = launch_route_scored(x, false, w_r, b_r, balance, rule, T, d, E, k, (float*)base, topk_idx, topk_gate, count, nullptr, st);
  if (err != hipSuccess) return err;
  const D4Args a{(const bf16_t*)x, w.gate, w.up, w.down, w.s_gate, w.s_up, w.s_down, shared.gate, shared.up, shared.down,
                 shared.s_gate, shared.s_up, shared.s_down, T, d, E, k, f, fs, topk_idx, topk_gate,
                 (bf16_t*)(base + d4_route_bytes(T, E, d) + 4096), (bf16_t*)y};
  const int P = (d + 255) / 256, nw = std::min(8, P), ppw = (P + nw - 1) / nw;
  switch (ppw) {
    case 1: d4_up_kernel<1><<<ncu, 64 * nw, 0, st>>>(a); break;
    case 2: d4_up_kernel<2><<<ncu, 64 * nw, 0, st>>>(a); break;
    case 3: d4_up_kernel<3><<<ncu, 64 * nw, 0, st>>>(a); break;
    case 4: d4_up_kernel<4><<<ncu, 64 * nw, 0, st>>>(a); break;
    default: return hipErrorInvalidValue;
  }
  if ((err = hipGetLastError()) != hipSuccess) return err;
  const int RW = std::min(D4_ROWS, std::max(8, (d + ncu - 1) / ncu)), g2 = (d + RW - 1) / RW;
  if (RW <= 16) {
    if (T > 8) d4_down_kernel<1, true><<<g2, 512, 0, st>>>(a, RW);
    else d4_down_kernel<1, false><<<g2, 512, 0, st>>>(a, RW);
  } else {
    if (T > 8) d4_down_kernel<2, true><<<g2, 512, 0, st>>>(a, RW);
    else d4_down_kernel<2, false><<<g2, 512, 0, st>>>(a, RW);
  }
  return hipGetLastError();
}

}  // namespace moe
