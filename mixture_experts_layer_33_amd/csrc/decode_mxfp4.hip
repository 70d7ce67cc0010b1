// The whole layer for a few tokens with MXFP4 weights: scored routing, then gate/up with SwiGLU over the experts that
// the tokens chose (and the shared one), then down and the gate-weighted sum.
//
//   h_tj = g_tj silu(W_gate[e] x_t) * (W_up[e] x_t)   (e: the j-th expert of token t; the shared expert's gate is 1)
//   y_t  = sum_j W_down[e_tj] h_tj + W_s_down h_ts
//
// Every used expert's weights are read once, whatever the number of tokens that chose it (mx4.h: up to eight tokens are
// columns of one product).  h is formed in fp32 and kept as two bf16 parts, hi = bf16(h) and lo = bf16(h - hi)
// (at most 2^-16 of h is left out; y's own rounding is 2^-8).
//
// Three launches: the logits (d in eight splits), gate and up, down.  Every workgroup of gate and up joins the logits and makes the
// choice for itself, 2 to 5 us in which it would wait for one that makes it (moe_route_scored's kernels, three launches, took
// 20 to 26 in this place); the first one leaves the down product's entries for the next launch while its weights come.
// What bounds it is the weight stream, each line of which is read once (fetched bytes: 1.03 times gate and up's, 1.07
// to 1.10 times down's).  One token of 8 + 1 of 256 experts, 7168 x 2048, medians of a kernel trace: logits 4.9 us, gate and up 34.8 (140 MB:
// the first codes are asked for after 6 us, then 5.2 TB/s), down 18.6 (70 MB).  Eight tokens, the least and the median of 31 calls:
// 7.5 and 9.6, 164 and 182 (5.6 and 5.1 TB/s), 79 and 96 (5.8 and 4.8 TB/s).
#include <algorithm>
#include <type_traits>

#include "decode_runs.h"
#include "fp8_tile.h"
#include "kernels.h"
#include "mx4.h"
#include "score_body.h"

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
  const float *w_r, *b_r, *balance;
  ScoreRule rule;
  int run;         // group_run of the experts' groups, for the lanes' experts in the choice
  float* planes;   // [D4_KS][T][E] partial logits
  struct D4Entries* entries;   // of the down product
  int32_t* topk_idx;
  float* topk_gate;
  bf16_t* h;       // [2][T k][f] (hi, lo), then the shared expert's [2][T][fs]
  bf16_t* y;
};

// What the tokens chose: the experts, ascending (gate and up read each one's weights once for all tokens).
struct D4List {
  int32_t id[D4_PAIRS];                   // [token, j]
  uint32_t bits[32];                      // E <= 1024
  int32_t below[32];                      // bits in the words before
  int32_t expert[D4_PAIRS];
  float gate[D4_PAIRS];                   // [token, j]
  __attribute__((aligned(16))) uint8_t slot[D4_PAIRS][D4_TMAX];   // [place in the list][token]: j + 1, 0: not chosen
  int32_t U;
};
// ... and, for the down product, entries of an expert (the shared one, E, last) with up to four of its tokens, the columns of
// one product: an expert of more tokens has several.  Up to four tokens in all a column is a token's own (-1: not chosen).
constexpr int D4_COLS = 4;
constexpr int D4_ENTRIES = D4_PAIRS + D4_TMAX / D4_COLS;
struct __attribute__((aligned(16))) D4Entries {
  int32_t n, routed;
  int16_t before[D4_PAIRS];               // entries of the experts before
  int16_t expert[D4_ENTRIES];
  int16_t row[D4_ENTRIES][D4_COLS];       // rows of h (t k + j; in the shared expert's part: t), -1: none
};

__device__ __forceinline__ void d4_clear(D4List& L) {   // before the barrier before d4_list
  for (int i = threadIdx.x; i < D4_PAIRS * D4_TMAX / 4; i += blockDim.x) ((uint32_t*)L.slot)[i] = 0u;
  if (threadIdx.x < 32) L.bits[threadIdx.x] = 0u;
}
__device__ __forceinline__ void d4_list(const D4Args& p, D4List& L) {   // L.id is known
  const int tid = threadIdx.x, n = p.T * p.k;
  if (p.T == 1) {       // one token's choice is ascending and distinct: it is the list (gate and up 35.9 -> 35.2 us)
    if (tid < n) {
      L.expert[tid] = L.id[tid];
      L.slot[tid][0] = (uint8_t)(tid + 1);
    }
    if (tid == 0) L.U = n;
    __syncthreads();
    return;
  }
  for (int q = tid; q < n; q += blockDim.x) atomicOr(&L.bits[L.id[q] >> 5], 1u << (L.id[q] & 31));
  __syncthreads();
  if (tid < 64) {
    const int own = tid < 32 ? __popc(L.bits[tid & 31]) : 0, incl = lanes_scan(own);
    if (tid < 32) L.below[tid] = incl - own;
    if (tid == 31) L.U = incl;
  }
  __syncthreads();
  for (int q = tid; q < n; q += blockDim.x) {
    const int e = L.id[q], at = L.below[e >> 5] + __popc(L.bits[e >> 5] & ((1u << (e & 31)) - 1u));
    L.expert[at] = e;
    L.slot[at][q / p.k] = (uint8_t)(q % p.k + 1);
  }
  __syncthreads();
}

__device__ __forceinline__ void d4_entries(const D4Args& p, const D4List& L, D4Entries& N) {
  // chosen by which tokens: the slots that are not 0 in a place's 16 bytes
  auto chosen = [&](int u) {
    const u32x4 s = *(const u32x4*)L.slot[u];
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) m |= ((s[i / 4] >> (8 * (i % 4))) & 0xffu) ? 1u << i : 0u;
    return m;
  };
  if (threadIdx.x < 64) {   // entries of the experts before each one: a scan, 64 experts at a time
    int sum = 0;
    for (int u0 = 0; u0 < L.U; u0 += 64) {
      const int u = u0 + (int)threadIdx.x;
      const int own = u < L.U ? (__popc(chosen(u)) + D4_COLS - 1) / D4_COLS : 0, incl = lanes_scan(own);
      if (u < L.U) N.before[u] = (int16_t)(sum + incl - own);
      sum += __builtin_amdgcn_readlane(incl, 63);
    }
    if (threadIdx.x == 0) N.routed = sum;
  }
  lds_barrier();
  for (int u = threadIdx.x; u <= L.U; u += blockDim.x) {
    const bool shared = u == L.U;
    const int at = shared ? N.routed : N.before[u];
    uint32_t m = !shared ? chosen(u) : p.fs > 0 ? (1u << p.T) - 1u : 0u;
    const int parts = (__popc(m) + D4_COLS - 1) / D4_COLS;
    for (int r = 0; r < parts; ++r) {
      N.expert[at + r] = (int16_t)(shared ? p.E : L.expert[u]);
      for (int i = 0; i < D4_COLS; ++i) {
        int t = __ffs(m) - 1;             // -1: none left
        if (p.T > D4_COLS) m &= m - 1;
        else t = (m >> i) & 1u ? i : -1;
        N.row[at + r][i] = (int16_t)(t < 0 || shared ? t : t * p.k + L.slot[u][t] - 1);
      }
    }
    if (shared) N.n = at + parts;
  }
  lds_barrier();
}

// ------------------------------------------------------------------ gate and up
// A unit is eight columns of f of one expert: their eight W_gate rows and eight W_up rows.  The workgroup's NW wavefronts
// split d (wavefront w has pairs w, w + NW, ...), keep their part of the tokens in registers over all units, and join
// their sums through LDS in a fixed order, a group of units at a time.  D units are in flight: a pair's registers are
// requested again, for the unit D further on, as soon as the pair is multiplied.  No branch stands between (a load that a branch
// may skip makes every later wait a wait for all): past the last unit, and where d ends inside a pair, the addresses
// lie outside their buffers, which costs no memory access, and x is zero.
template <int TS>
struct D4Part {                          // [half][gate, up][token][column]
  static constexpr int GROUP = 4 / TS, SIZE = TS * 256;
  float v[2 * GROUP][8][SIZE];
};
// `lds`: the tokens' blocks first, then the sums.
template <int PPW, int TS>
constexpr int D4_UP_LDS = (PPW * TS < 4 ? PPW * TS : 4) * 8 * XBLOCK > (int)sizeof(D4Part<TS>) ? (PPW * TS < 4 ? PPW * TS : 4) * 8 * XBLOCK
                                                                                              : (int)sizeof(D4Part<TS>);
template <int PPW, int TS, int D>        // TS: sets of eight tokens
__device__ __forceinline__ void d4_up(const D4Args& p, D4List& L, D4Entries& N, uint8_t* stage) {
  D4Part<TS>& part = *(D4Part<TS>*)stage;
  constexpr int GROUP = D4Part<TS>::GROUP;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), NW = blockDim.x >> 6;
  const int g = lane >> 4, col = lane & 15, chunk = lane >> 3, row = lane & 7, P = (p.d + 255) / 256;
  const uint32_t rowb = (uint32_t)p.d / 2;
  bf16x8 x[PPW][TS][4];
  constexpr int BLOCKS = PPW * TS < 4 ? PPW * TS : 4;     // of x on their way at a time (the first ones while the list is made)
#pragma unroll
  for (int b0 = 0; b0 < PPW * TS; b0 += BLOCKS) {
#pragma unroll
    for (int b = 0; b < BLOCKS; ++b) {
      if (b0 + b >= PPW * TS) break;
      const int k = ((b0 + b) / TS * NW + wave) * 256, at = k < p.d ? k : 0, r0 = min((b0 + b) % TS * 8, p.T - 1);
      x_copy(p.x + (int64_t)r0 * p.d + at, p.T - 1 - r0, (uint32_t)p.d, p.d - at,
             (uint32_t)(uintptr_t)(stage + (wave * BLOCKS + b) * XBLOCK));
    }
    if (b0 == 0) d4_list(p, L);
    wait_all();
#pragma unroll
    for (int b = 0; b < BLOCKS; ++b)
      if (b0 + b < PPW * TS)
        x_read(stage + (wave * BLOCKS + b) * XBLOCK, ((b0 + b) / TS * NW + wave) * 256 + 64 * g + 32 * (col >> 3) < p.d,
               x[(b0 + b) / TS][(b0 + b) % TS]);
    lds_barrier();      // read: the next blocks, or the sums, may come
  }
  // this workgroup's units: a share of the shared expert's, then of the routed ones
  const int U = L.U, per = p.f / 8, su = p.fs / 8, ru = U * per, G = gridDim.x, b = blockIdx.x;
  const int s0 = (int)((int64_t)su * b / G), s1 = (int)((int64_t)su * (b + 1) / G);
  const int r0 = (int)((int64_t)ru * b / G), r1 = (int)((int64_t)ru * (b + 1) / G);
  const int ns = s1 - s0, steps = ns + r1 - r0;
  // the place of the unit whose loads come next
  int n = -1, at = 0, i0 = 0;
  __amdgpu_buffer_rsrc_t gr, ur, gs, us;
  uint32_t from = 0, srows = 0, off = OUTSIDE, last_off = OUTSIDE;
  const int last = (PPW - 1) * NW + wave;   // its last pair, which d may cut in half or leave out
  const bool cut = last * 128 + chunk * 16 >= (int)rowb;
  auto next = [&]() __attribute__((always_inline)) {
    ++n;
    const bool shared = n < ns, live = n < steps;
    if (shared || n == ns) {
      i0 = (shared ? s0 + n : r0 % per) * 8;
      at = shared ? 0 : r0 / per;
    } else {
      i0 += 8;
      if (i0 == p.f) {
        i0 = 0;
        ++at;
      }
    }
    const int e = __builtin_amdgcn_readfirstlane(shared ? 0 : L.expert[min(at, U - 1)]), F = shared ? p.fs : p.f;
    const uint32_t size = (uint32_t)F * rowb;
    gr = buffer_of(either(shared, p.ws_gate, p.w_gate) + (int64_t)e * size, size);
    ur = buffer_of(either(shared, p.ws_up, p.w_up) + (int64_t)e * size, size);
    from = live ? i0 * rowb : 0;
    off = live ? row * rowb + chunk * 16 : OUTSIDE;
    last_off = cut ? OUTSIDE : off;
    srows = (uint32_t)(shared ? p.fs : p.E * p.f) * 4;
    const uint32_t sfrom = (uint32_t)(e * F + (live ? i0 : 0)) * 4, sbytes = (uint32_t)(p.d / 128) * srows - sfrom;
    gs = buffer_of(either(shared, p.ss_gate, p.s_gate) + sfrom, sbytes);
    us = buffer_of(either(shared, p.ss_up, p.s_up) + sfrom, sbytes);
  };
  W4Pair w[D][PPW];
  auto load = [&](W4Pair& q, int i) __attribute__((always_inline)) {
    const uint32_t pair = i * NW + wave, so = min(pair, (uint32_t)P - 1) * 2 * srows;
    const uint32_t sl = (i == PPW - 1 && cut ? 0 : (chunk >> 2) * srows) + row * 4;
    q.a = load_b128_nt(gr, i == PPW - 1 ? last_off : off, from + pair * 128);
    q.b = load_b128_nt(ur, i == PPW - 1 ? last_off : off, from + pair * 128);
    q.sa = load_b32(gs, sl, so);
    q.sb = load_b32(us, sl, so);
  };
  // unit m of the workgroup, whose codes are in the set; the set takes the unit D further on
  auto step = [&](int m, auto set) __attribute__((always_inline)) {
    constexpr int S = decltype(set)::value;
    f32x4 ag[TS] = {}, au[TS] = {};
    next();
#pragma unroll
    for (int i = 0; i < PPW; ++i) {
      const float fa = chunk_scale(w[S][i].sa), fb = chunk_scale(w[S][i].sb);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const bf16x8 a = widen4(w[S][i].a[j], fa), u = widen4(w[S][i].b[j], fb);
#pragma unroll
        for (int s = 0; s < TS; ++s) {
          ag[s] = mfma16(a, x[i][s][j], ag[s]);
          au[s] = mfma16(u, x[i][s][j], au[s]);
        }
      }
      load(w[S][i], i);
      __builtin_amdgcn_sched_barrier(0);
    }
    if (holds_half()) {
#pragma unroll
      for (int s = 0; s < TS; ++s) {
        float* to = part.v[m % (2 * GROUP)][wave] + s * 256 + (col >> 3) * 128 + (col & 7) * 8 + 4 * (g & 1);
        *(f32x4*)to = ag[s];
        *(f32x4*)(to + 64) = au[s];
      }
    }
  };
  // h of units m0 .. m0 + count - 1
  auto flush = [&](int m0, int count) __attribute__((always_inline)) {
    lds_barrier();
    const int turn = wave + m0 / GROUP % NW, first = (turn >= NW ? turn - NW : turn) * 64 + lane;
    for (int q = first; q < 8 * GROUP * p.T; q += blockDim.x) {
      const int m = q / 8 % GROUP, t = q / (8 * GROUP);
      if (m >= count) continue;
      const bool shared = m0 + m < ns;
      const int unit = shared ? s0 + m0 + m : r0 + m0 + m - ns;
      const int place = shared ? 0 : unit / per, i = (shared ? unit : unit % per) * 8 + q % 8;
      const int j = shared ? 1 : (int)L.slot[place][t];
      if (j == 0) continue;
      const float(*sums)[D4Part<TS>::SIZE] = part.v[(m0 + m) % (2 * GROUP)];
      const int c = (t >> 3) * 256 + (t & 7) * 8 + q % 8;
      float a = 0.f, u = 0.f;
      for (int v = 0; v < NW; ++v) {
        a += sums[v][c] + sums[v][c + 128];
        u += sums[v][c + 64] + sums[v][c + 192];
      }
      float h = silu(a) * u;
      if (!shared) h *= L.gate[t * p.k + j - 1];
      const bf16_t hi = f2bf(h), lo = f2bf(fabsf(h) < 3.39e38f ? h - bf2f(hi) : 0.f);   // an infinite hi has no rest
      const int64_t all = (int64_t)p.T * p.k * p.f;
      bf16_t* o = shared ? p.h + 2 * all + (int64_t)t * p.fs + i : p.h + (int64_t)(t * p.k + j - 1) * p.f + i;
      o[0] = hi;
      o[shared ? (int64_t)p.T * p.fs : all] = lo;
    }
  };
#pragma unroll
  for (int s = 0; s < D; ++s) {
    next();
#pragma unroll
    for (int i = 0; i < PPW; ++i) load(w[s][i], i);
  }
  if (b == 0) {       // while the first weights come: the entries, for every workgroup of the down product
    d4_entries(p, L, N);
    for (int i = tid; i < (int)(sizeof(D4Entries) / 16); i += blockDim.x) ((u32x4*)p.entries)[i] = ((const u32x4*)&N)[i];
  }
  for (int m = 0; m < steps; m += D) {
    unrolled<D>([&](auto s) __attribute__((always_inline)) {
      constexpr int S = decltype(s)::value;
      step(m + S, s);
      const int done = m + S + 1;
      if (done <= steps && (done % GROUP == 0 || done == steps)) {
        const int m0 = (done - 1) / GROUP * GROUP;
        flush(m0, done - m0);
      }
    });
  }
}

// ------------------------------------------------------------------ router
// Partial logits of W_r (fp32) and the tokens: K split z of two expert rows by a wavefront, in plain fp32.
// What bounds it is latency: a workgroup requests its rows of W_r at once, then brings the tokens' part into LDS.
constexpr int D4_KS = 8, D4_SLICE = 1024 + 64;   // d <= 8192 in 8 splits of whole 64
__global__ __launch_bounds__(256) void d4_logits_kernel(D4Args p) {
  __shared__ __attribute__((aligned(16))) bf16_t xs[D4_TMAX * D4_SLICE];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int z = blockIdx.x % D4_KS, e0 = ((int)(blockIdx.x / D4_KS) * 4 + wave) * 2, KA = p.d / 64;
  const int i0 = KA * z / D4_KS * 64, n = KA * (z + 1) / D4_KS * 64 - i0;
  constexpr int IT = (D4_SLICE + 255) / 256;
  f32x4 w[2][IT];
#pragma unroll
  for (int r = 0; r < 2; ++r)
#pragma unroll
    for (int q = 0; q < IT; ++q) {
      const int i = q * 256 + lane * 4;
      w[r][q] = i < n ? __builtin_nontemporal_load((const f32x4*)(p.w_r + (int64_t)min(e0 + r, p.E - 1) * p.d + i0 + i)) : f32x4{0.f, 0.f, 0.f, 0.f};
    }
  for (int v = tid; v < p.T * (n / 8); v += 256) {
    const int t = v / (n / 8), i = v % (n / 8) * 8;
    *(u32x4*)(xs + t * D4_SLICE + i) = *(const u32x4*)(p.x + (int64_t)t * p.d + i0 + i);
  }
  __syncthreads();
  float mine = 0.f;      // lane 16 r + t: expert e0 + r, token t
  for (int t0 = 0; t0 < p.T; t0 += 4) {
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int t = min(t0 + u, p.T - 1);
      float a[2] = {0.f, 0.f};
#pragma unroll
      for (int q = 0; q < IT; ++q) {
        if (q * 256 >= n) break;
        const int i = min(q * 256 + lane * 4, max(n - 4, 0));   // past the slice w is zero
        const u32x2 v = n > 0 ? *(const u32x2*)(xs + t * D4_SLICE + i) : u32x2{0, 0};
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          if (q * 256 + lane * 4 >= n) continue;   // not 0 times a token's infinity
          a[r] = fmaf(w[r][q][0], lo_bf(v[0]), a[r]);
          a[r] = fmaf(w[r][q][1], hi_bf(v[0]), a[r]);
          a[r] = fmaf(w[r][q][2], lo_bf(v[1]), a[r]);
          a[r] = fmaf(w[r][q][3], hi_bf(v[1]), a[r]);
        }
      }
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const float sum = lanes_sum<1>(a[r]);
        if (lane == 16 * r + t) mine = sum;
      }
    }
  }
  const int e = e0 + (lane >> 4), t = lane & 15;
  if (lane < 32 && t < p.T && e < p.E) p.planes[((int64_t)z * p.T + t) * p.E + e] = mine;
}

// One token's choice by this wavefront into the list (and, by workgroup 0, to the caller).
template <int VPL, int Z>
__device__ __forceinline__ void d4_choose(const D4Args& p, D4List& L, float* row, int t, const float (&v)[Z][VPL],
                                          const float (&bias)[VPL], const float (&bal)[VPL]) {
  const int lane = threadIdx.x & 63, e0 = lane * VPL;
  float l[VPL];
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    l[i] = v[0][i];
#pragma unroll
    for (int z = 1; z < Z; ++z) l[i] += v[z][i];
    if (p.b_r) l[i] += bias[i];
    if (e0 + i >= p.E) l[i] = -INFINITY;
    row[e0 + i] = l[i];
  }
  int choice, rank;
  float gate;
  select_row<VPL>(p.rule, p.balance != nullptr, p.E, p.k, p.run, l, bal, row, choice, rank, gate);
  if (lane < p.k) {
    L.id[t * p.k + rank] = choice;
    L.gate[t * p.k + rank] = gate;
    if (blockIdx.x == 0) {
      p.topk_idx[t * p.k + rank] = choice;
      p.topk_gate[t * p.k + rank] = gate;
    }
  }
}
template <int VPL, int Z>
__device__ __forceinline__ void d4_planes(const D4Args& p, int t, int z0, float (&v)[Z][VPL], float (&bias)[VPL], float (&bal)[VPL]) {
  auto read = [&](auto vec) __attribute__((always_inline)) {
    constexpr bool VEC = decltype(vec)::value;
#pragma unroll
    for (int z = 0; z < Z; ++z) lane_row<VEC>(p.planes + ((int64_t)(z0 + z) * p.T + t) * p.E, p.E, v[z]);
    lane_row<VEC>(p.b_r ? p.b_r : p.planes, p.E, bias);
    lane_row<VEC>(p.balance ? p.balance : p.planes, p.E, bal);
  };
  if (p.E % 4 == 0) read(std::true_type{});
  else read(std::false_type{});
}

// VPL: experts a lane looks at in the choice.
template <int PPW, int TS, int D, int VPL>
__global__ __launch_bounds__(512) void d4_up_kernel(D4Args p) {
  __shared__ D4List L;
  __shared__ D4Entries N;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[D4_UP_LDS<PPW, TS>];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), NW = blockDim.x >> 6;
  float* row = (float*)lds + wave * 64 * VPL;      // the choice's, before anything else
  constexpr int Z = VPL == 4 ? D4_KS : 4;          // planes in flight: of 8 experts a lane eight spill (the choice among 16 spills 86 registers with any number)
  float v[Z][VPL], bias[VPL], bal[VPL];
  d4_planes<VPL, Z>(p, min(wave, p.T - 1), 0, v, bias, bal);
  d4_clear(L);
  for (int t = wave; t < p.T; t += NW) {
    if (t > wave) d4_planes<VPL, Z>(p, t, 0, v, bias, bal);
    float l[1][VPL];
#pragma unroll
    for (int z0 = 0; z0 < D4_KS; z0 += Z) {
      if (z0 > 0) d4_planes<VPL, Z>(p, t, z0, v, bias, bal);
#pragma unroll
      for (int i = 0; i < VPL; ++i)
#pragma unroll
        for (int z = 0; z < Z; ++z) l[0][i] = z0 + z == 0 ? v[0][i] : l[0][i] + v[z][i];
      __builtin_amdgcn_sched_barrier(0);
    }
    d4_choose<VPL, 1>(p, L, row, t, l, bias, bal);
  }
  __syncthreads();
  d4_up<PPW, TS, D>(p, L, N, lds);
}

// ------------------------------------------------------------------ down
// A workgroup owns `rows` <= 16 NT output rows from o0 on.  The columns of all entries are cut into runs of up to `run` pairs,
// which the wavefronts take in turn, D pairs in flight.  A run of four starts at another of its pairs from workgroup to
// workgroup: all of the chip would read the same 128 bytes of every 1024 at a time.
//
// A pair's h (up to four tokens, hi and lo of 256 columns: 1 KB a token) comes by global -> LDS copies of one
// instruction a token; read straight into the MFMA's layout it took eight 16-byte loads a lane, nearly all of them of
// columns without a token, at 16 clocks each (decode of 8 tokens, this kernel: 103 us, 82 with no h at all).  Columns
// c and c + 4 of a chunk are hi and lo of token c: one MFMA for both.  The copies are issued before the pair's weights,
// so a wait that leaves no more than the weights of D pairs outstanding is past them.
//
// At the end, and with more than four tokens when the entry changes, the sums of the columns are added to the
// wavefront's sums of all tokens in LDS, [NW][half][16][16 NT].
template <int NT, int D>
struct D4Down {
  u32x4 h[8][D][D4_COLS][64];            // [wavefront][in flight][column][hi, lo: 32 pieces of eight columns each]
  float y[8][2][D4_TMAX][16 * NT];
};
template <int NT, int D>
__device__ __forceinline__ void d4_down(const D4Args& p, const D4Entries& N, D4Down<NT, D>& m, int o0, int rows) {
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), NW = blockDim.x >> 6;
  const int g = lane >> 4, col = lane & 15, chunk = lane >> 3, row = lane & 7;
  for (int i = tid; i < NW * 2 * D4_TMAX * 16 * NT; i += blockDim.x) (&m.y[0][0][0][0])[i] = 0.f;
  const D4Runs runs = d4_runs(__builtin_amdgcn_readfirstlane(N.routed), __builtin_amdgcn_readfirstlane(N.n), (p.f + 255) / 256,
                              (p.fs + 255) / 256, p.T > D4_COLS ? 4 : 1);
  const int all = runs.all;
  const int64_t nh = (int64_t)p.T * p.k * p.f, nsh = (int64_t)p.T * p.fs;
  auto advance = [&](D4Place& at) __attribute__((always_inline)) { return d4_advance(runs, NW, at); };
  const int turned = blockIdx.x & 3;
  int F = 0;
  D4Place next{wave, 0, 0, 0, 0};    // whose loads come next
  d4_set(runs, next);
  __amdgpu_buffer_rsrc_t wr, sr;
  const bf16_t* hbase = nullptr;
  int hrow[D4_COLS];
  uint32_t plane = 0, rowb = 0, srows = 0, lane_off[2 * NT];
  auto enter = [&]() __attribute__((always_inline)) {   // next.entry
    const int at = next.entry, ex = __builtin_amdgcn_readfirstlane((int)N.expert[at]);
    const bool shared = ex == p.E;
    const int e = shared ? 0 : ex;
    F = shared ? p.fs : p.f;
    rowb = (uint32_t)F / 2;
    const uint32_t bytes = (uint32_t)p.d * rowb;
    wr = buffer_of(either(shared, p.ws_down, p.w_down) + (int64_t)e * bytes, bytes);
    srows = (uint32_t)(shared ? p.d : p.E * p.d) * 4;
    const uint32_t sfrom = (uint32_t)(e * p.d + o0) * 4;
    sr = buffer_of(either(shared, p.ss_down, p.s_down) + sfrom, (uint32_t)(F / 128) * srows - sfrom);
#pragma unroll
    for (int r = 0; r < 2 * NT; ++r) lane_off[r] = 8 * r + row < rows ? (uint32_t)(o0 + 8 * r + row) * rowb + chunk * 16 : OUTSIDE;
    const uint2 rw = *(const uint2*)N.row[at];
#pragma unroll
    for (int c = 0; c < D4_COLS; ++c)
      hrow[c] = (int)(int16_t)(__builtin_amdgcn_readfirstlane((int)(c < 2 ? rw.x : rw.y)) >> (16 * (c & 1)));
    hbase = p.h + (shared ? 2 * nh : 0);
    plane = (uint32_t)(2 * (shared ? nsh : nh));
  };
  enter();
  struct Step {
    W4Pair w[NT];
  };
  auto load = [&](Step& s, int slot) __attribute__((always_inline)) {
    const bool live = next.n < all;
    const int pair = live ? next.from + (next.length == 4 ? (next.i + turned) & 3 : next.i) : 0;
    if (live) {
      // 16 bytes a lane: lanes 0-31 hi, 32-63 lo; where F ends inside the pair its first half again (the codes are zeros there)
      const uint32_t at = ((uint32_t)lane & 31) * 8 + pair * 256 < (uint32_t)F ? (lane & 31) * 16 : (lane & 15) * 16;
      const uint32_t off = (lane < 32 ? 0 : plane) + at;
#pragma unroll
      for (int c = 0; c < D4_COLS; ++c) {
        u32x4* to = m.h[wave][slot][c];
        if (hrow[c] >= 0)
          copy16(hbase + (int64_t)hrow[c] * F + pair * 256, off, __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)to));
        else if (p.T <= D4_COLS && c < p.T)
          to[lane] = u32x4{0, 0, 0, 0};
      }
    }
    const uint32_t so = pair * 128, ss = pair * 2 * srows;
    const uint32_t sl = (pair * 2 + (chunk >> 2) < F / 128 ? (chunk >> 2) * srows : 0) + row * 4;
    const bool in = live && so + chunk * 16 < rowb;
#pragma unroll
    for (int r = 0; r < NT; ++r) {
      s.w[r].a = load_b128_nt(wr, in ? lane_off[2 * r] + so : OUTSIDE, 0);
      s.w[r].b = load_b128_nt(wr, in ? lane_off[2 * r + 1] + so : OUTSIDE, 0);
      s.w[r].sa = load_b32(sr, 8 * (2 * r) + row < rows ? sl + 64 * r : 0, ss);
      s.w[r].sb = load_b32(sr, 8 * (2 * r + 1) + row < rows ? sl + 64 * r + 32 : 0, ss);
    }
    __builtin_amdgcn_sched_barrier(0);
    if (advance(next) && next.n < all) enter();
  };
  f32x4 acc[2 * NT];
#pragma unroll
  for (int r = 0; r < 2 * NT; ++r) acc[r] = f32x4{0.f, 0.f, 0.f, 0.f};
  D4Place now{wave, 0, 0, 0, 0};     // which is multiplied next
  d4_set(runs, now);
  auto flush = [&](int entry) __attribute__((always_inline)) {
    const int ex = (int)N.expert[entry], hr = N.row[entry][col & 3];
    const int t = p.T <= D4_COLS ? ((col & 3) < p.T ? col & 3 : -1) : ex == p.E ? hr : hr >= 0 ? hr / p.k : -1;
    const bool mine = holds_half() && (col & 4) == 0 && t >= 0;
    float* to = m.y[wave][col >> 3][max(t, 0)] + 4 * (g & 1);
#pragma unroll
    for (int r = 0; r < 2 * NT; ++r) {
      f32x4 v = acc[r];
#pragma unroll
      for (int i = 0; i < 4; ++i)   // hi's sum and lo's, four lanes on
        v[i] += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v[i]), 0x104, 0xf, 0xf, true));
      if (mine) *(f32x4*)(to + 8 * r) = *(f32x4*)(to + 8 * r) + v;
      acc[r] = f32x4{0.f, 0.f, 0.f, 0.f};
    }
  };
  auto consume = [&](Step& s, int slot) __attribute__((always_inline)) {
    wait_vm<4 * NT * D>();
    __builtin_amdgcn_sched_barrier(0);
    const u32x4* from = m.h[wave][slot][col & 3] + ((col >> 2) & 1) * 32 + 8 * g + 4 * (col >> 3);
    bf16x8 h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = __builtin_bit_cast(bf16x8, from[i]);
#pragma unroll
    for (int r = 0; r < NT; ++r) {
      const float fa = chunk_scale(s.w[r].sa), fb = chunk_scale(s.w[r].sb);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        acc[2 * r] = mfma16(widen4(s.w[r].a[i], fa), h[i], acc[2 * r]);
        acc[2 * r + 1] = mfma16(widen4(s.w[r].b[i], fb), h[i], acc[2 * r + 1]);
      }
    }
    __builtin_amdgcn_sched_barrier(0);
    if (now.n >= all) return;
    const int was = now.entry;
    if (advance(now) && (p.T > D4_COLS || now.n >= all)) flush(was);
  };
  __syncthreads();   // the zeros
  {
    Step s[D];
#pragma unroll
    for (int i = 0; i < D; ++i) load(s[i], i);
    while (now.n < all) {
#pragma unroll
      for (int i = 0; i < D; ++i) {
        consume(s[i], i);
        load(s[i], i);
      }
    }
  }
  wait_vm<0>();      // no copy outlives the array
  __syncthreads();
  for (int q = tid; q < 16 * NT * p.T; q += blockDim.x) {
    const int r = q % (16 * NT), t = q / (16 * NT);
    if (r >= rows) continue;
    float sum = 0.f;
    for (int v = 0; v < NW; ++v) sum += m.y[v][0][t][r] + m.y[v][1][t][r];
    p.y[(int64_t)t * p.d + o0 + r] = f2bf(sum);
  }
}

template <int NT, int D>
__global__ __launch_bounds__(512) void d4_down_kernel(D4Args p, int RW) {
  __shared__ D4Entries N;
  extern __shared__ __attribute__((aligned(1024))) uint8_t lds[];
  for (int i = threadIdx.x; i < (int)(sizeof(D4Entries) / 16); i += blockDim.x) ((u32x4*)&N)[i] = ((const u32x4*)p.entries)[i];
  __syncthreads();
  for (int o0 = blockIdx.x * RW; o0 < p.d; o0 += gridDim.x * RW) {
    d4_down<NT, D>(p, N, *(D4Down<NT, D>*)lds, o0, min(RW, p.d - o0));
    __syncthreads();
  }
}

template <int NT, int D>
static hipError_t run_down(const D4Args& a, int RW, int grid, hipStream_t st) {
  auto kern = d4_down_kernel<NT, D>;
  const size_t lds = sizeof(D4Down<NT, D>);
  const hipError_t err = hipFuncSetAttribute((const void*)kern, hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
  if (err != hipSuccess) return err;
  kern<<<grid, 512, lds, st>>>(a, RW);
  return hipGetLastError();
}

// Workspace: partial logits [D4_KS][T][E] | entries | h [2][T k][f] | [2][T fs].
static size_t d4_planes_bytes(int T, int E) { return ((size_t)D4_KS * T * E * sizeof(float) + 255) & ~(size_t)255; }
constexpr size_t D4_ENTRY_BYTES = (sizeof(D4Entries) + 255) & ~(size_t)255;
size_t decode_mxfp4_workspace_bytes(int T, int E, int k, int f, int fs) {
  return d4_planes_bytes(T, E) + D4_ENTRY_BYTES + 4 * ((size_t)T * k * f + (size_t)T * fs);
}

template <int PPW, int TS>
static hipError_t run_up(const D4Args& a, int grid, int nw, hipStream_t st) {
  // Units in flight.  Two are the fewest that keep the stream going, and more delay the first unit's codes (its requests queue
  // behind theirs) or spill (16 tokens, d 7168).  With 1 | 2 | 3 | 4, the whole call, us: 8 tokens, d 2048, f 1408, 64 experts
  // 77.5 | 70.2 | 70.8 | 71.8; 1 token, d 4096, f 1024, 512 experts 37.0 | 37.9 | 38.5 | 40.4, 16 tokens 224 | 202 | 207 | 210;
  // 1 token, d 7168, f 2048, 256 experts 60.1 | 61.4 | 62.6 | 65.1, 16 tokens 449 | 454 | 971 | 1267.
  constexpr int D = 2;
  if (a.E > 512) d4_up_kernel<PPW, TS, D, 16><<<grid, 64 * nw, 0, st>>>(a);
  else if (a.E > 256) d4_up_kernel<PPW, TS, D, 8><<<grid, 64 * nw, 0, st>>>(a);
  else d4_up_kernel<PPW, TS, D, 4><<<grid, 64 * nw, 0, st>>>(a);
  return hipGetLastError();
}

hipError_t launch_decode_mxfp4(const void* x, const float* w_r, const float* b_r, const float* balance, const ScoreRule& rule,
                               const Mx4Weights& w, const Mx4Weights& shared, int T, int d, int E, int k, int f, int fs, void* y,
                               int32_t* topk_idx, float* topk_gate, void* ws, hipStream_t st) {
  int dev = 0, ncu = 0;
  hipError_t err = hipGetDevice(&dev);
  if (err != hipSuccess) return err;
  if ((err = hipDeviceGetAttribute(&ncu, hipDeviceAttributeMultiprocessorCount, dev)) != hipSuccess) return err;
  uint8_t* base = (uint8_t*)ws;
  const D4Args a{(const bf16_t*)x, w.gate, w.up, w.down, w.s_gate, w.s_up, w.s_down, shared.gate, shared.up, shared.down,
                 shared.s_gate, shared.s_up, shared.s_down, T, d, E, k, f, fs, w_r, b_r, balance, rule,
                 group_run(E / rule.groups, E <= 256 ? 4 : E <= 512 ? 8 : 16), (float*)base, (D4Entries*)(base + d4_planes_bytes(T, E)),
                 topk_idx, topk_gate, (bf16_t*)(base + d4_planes_bytes(T, E) + D4_ENTRY_BYTES), (bf16_t*)y};
  d4_logits_kernel<<<(E + 7) / 8 * D4_KS, 256, 0, st>>>(a);
  if ((err = hipGetLastError()) != hipSuccess) return err;
  const int P = (d + 255) / 256, nw = std::min(8, P), ppw = (P + nw - 1) / nw;
  switch (ppw) {
    case 1: err = T > 8 ? run_up<1, 2>(a, ncu, nw, st) : run_up<1, 1>(a, ncu, nw, st); break;
    case 2: err = T > 8 ? run_up<2, 2>(a, ncu, nw, st) : run_up<2, 1>(a, ncu, nw, st); break;
    case 3: err = T > 8 ? run_up<3, 2>(a, ncu, nw, st) : run_up<3, 1>(a, ncu, nw, st); break;
    default: err = T > 8 ? run_up<4, 2>(a, ncu, nw, st) : run_up<4, 1>(a, ncu, nw, st);
  }
  if (err != hipSuccess) return err;
  const int RW = std::min(D4_ROWS, std::max(8, (d + ncu - 1) / ncu)), g2 = (d + RW - 1) / RW;
  return RW <= 16 ? run_down<1, 4>(a, RW, g2, st) : run_down<2, 3>(a, RW, g2, st);
}

}  // namespace moe
