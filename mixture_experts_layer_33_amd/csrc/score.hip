// Scored routing: softmax or sigmoid scores, a balance bias that decides the choice only,
// groups of experts, top-k, optionally renormalised gates; and the gradient of the gates.
//
//   l = x W_r^T (+ b);  s = softmax(l) | sigmoid(l);  c = s (+ balance);
//   group score = sum of its group_top largest c; the top_groups best groups are kept;
//   S = k largest c in them (ties to the lower id);  g = scale s_S (/ sum_S s)
//
// The logits come in partial planes, a K split each, by kernels for few, some and many tokens (here and in route.hip);
// the selection adds them, one wavefront per token.
#include <algorithm>

#include "common.h"
#include "fp8_tile.h"
#include "kernels.h"
#include "route_body.h"
#include "tr_read.h"

namespace moe {

// fp32 as an unsigned integer of the same order; a NaN below every number, nothing is 0
// (0 marks what may not be chosen).  -0 counts as +0.
__device__ __forceinline__ uint32_t order_key(float v) {
  const uint32_t u = __float_as_uint(v + 0.0f);
  return v != v ? 1u : (u & 0x80000000u) ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float key_value(uint32_t key) {
  return __uint_as_float((key & 0x80000000u) ? key & 0x7fffffffu : ~key);
}

template <int G>
__device__ __forceinline__ uint32_t group_max_u(uint32_t u) {
  auto mx = [](uint32_t a, uint32_t b) { return a > b ? a : b; };
  u = mx(u, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)u, 0xB1, 0xf, 0xf, false));
  if constexpr (G >= 4) u = mx(u, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)u, 0x4E, 0xf, 0xf, false));
  if constexpr (G >= 8) u = mx(u, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)u, 0x141, 0xf, 0xf, false));
  if constexpr (G >= 16) u = mx(u, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)u, 0x140, 0xf, 0xf, false));
  if constexpr (G >= 32) {
    const auto s = __builtin_amdgcn_permlane16_swap(u, u, false, false);
    u = mx(s[0], s[1]);
  }
  if constexpr (G >= 64) {
    const auto s = __builtin_amdgcn_permlane32_swap(u, u, false, false);
    u = mx(s[0], s[1]);
  }
  return u;
}

// Sum over the wavefront in VALU cross-lane moves (as group_max), the same bits in every lane.
template <int FROM>
__device__ __forceinline__ float lanes_sum(float v) {   // over lanes that differ in bits FROM .. 32
  auto dpp = [](float u, auto ctl) __attribute__((always_inline)) {
    return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(u), decltype(ctl)::value, 0xf, 0xf, false));
  };
  if constexpr (FROM <= 1) v += dpp(v, std::integral_constant<int, 0xB1>{});    // quad_perm [1,0,3,2]
  if constexpr (FROM <= 2) v += dpp(v, std::integral_constant<int, 0x4E>{});    // [2,3,0,1]
  if constexpr (FROM <= 4) v += dpp(v, std::integral_constant<int, 0x141>{});   // row_half_mirror
  v += dpp(v, std::integral_constant<int, 0x128>{});                            // row_ror:8
  const auto a = __builtin_amdgcn_permlane16_swap(__float_as_int(v), __float_as_int(v), false, false);
  v = __int_as_float(a[0]) + __int_as_float(a[1]);
  const auto b = __builtin_amdgcn_permlane32_swap(__float_as_int(v), __float_as_int(v), false, false);
  return __int_as_float(b[0]) + __int_as_float(b[1]);
}

// The value of the lane `O` apart (O = 4: some lane of the other quad, 8 lanes holding one value per quad).
template <int O>
__device__ __forceinline__ uint32_t partner(uint32_t u) {
  if constexpr (O == 1) return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)u, 0xB1, 0xf, 0xf, false);
  else if constexpr (O == 2) return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)u, 0x4E, 0xf, 0xf, false);
  else if constexpr (O == 4) return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)u, 0x141, 0xf, 0xf, false);
  else if constexpr (O == 8) return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)u, 0x128, 0xf, 0xf, false);
  else if constexpr (O == 16) {
    const auto s = __builtin_amdgcn_permlane16_swap(u, u, false, false);
    return s[0] == u ? s[1] : s[0];
  } else {
    const auto s = __builtin_amdgcn_permlane32_swap(u, u, false, false);
    return s[0] == u ? s[1] : s[0];
  }
}

// A lane's keys, largest first, equal ones by their place (an odd-even merge network).
template <int N>
__device__ __forceinline__ void sort_keys(uint32_t (&key)[N], int (&at)[N]) {
#pragma unroll
  for (int p = 1; p < N; p *= 2)
#pragma unroll
    for (int k = p; k >= 1; k /= 2)
#pragma unroll
      for (int j = k % p; j + k < N; j += 2 * k)
#pragma unroll
        for (int i = 0; i < k; ++i) {
          const int a = i + j, b = i + j + k;
          if (b >= N || a / (2 * p) != b / (2 * p)) continue;
          const bool swap = key[b] > key[a] || (key[b] == key[a] && at[b] < at[a]);
          const uint32_t ka = key[a];
          const int ia = at[a];
          key[a] = swap ? key[b] : ka;
          at[a] = swap ? at[b] : ia;
          key[b] = swap ? ka : key[b];
          at[b] = swap ? ia : at[b];
        }
}

struct SelectArgs {
  const float* planes;   // KS partial planes of the logits [KS, T, E]
  int KS;
  const float* b_r;
  const float* balance;
  int64_t T;
  int E, k;
  ScoreRule rule;
  int32_t* topk_idx;
  float* topk_gate;
  int32_t* count;        // [E]; with several workgroups the first clears it for score_count_kernel
  float* logits;
};

typedef float __attribute__((ext_vector_type(4), aligned(4))) f32x4_any;   // 16 bytes at a float's alignment

// Row `at` of a [., E] array, this lane's experts lane VPL .. + VPL - 1 (past E: some other's), in 16-byte pieces
// (VEC: E a multiple of 4).  Without a branch: a branch around a load makes the next one wait for it.
template <bool VEC, int VPL>
__device__ __forceinline__ void lane_row(const float* __restrict__ at, int E, float (&v)[VPL]) {
  const int e0 = (threadIdx.x & 63) * VPL;
  if constexpr (VEC && VPL % 4 == 0) {
#pragma unroll
    for (int c = 0; c < VPL / 4; ++c) {
      const f32x4 w = *(const f32x4_any*)(at + min(e0 + 4 * c, E - 4));
#pragma unroll
      for (int q = 0; q < 4; ++q) v[4 * c + q] = w[q];
    }
  } else {
#pragma unroll
    for (int i = 0; i < VPL; ++i) v[i] = at[min(e0 + i, E - 1)];
  }
}

// One wavefront per token; lane l owns the consecutive experts l VPL .. l VPL + VPL - 1, so that the lowest lane
// of a tie holds the lowest id, and a group of experts is a run of lanes where its size allows it
// (`run` lanes, a power of two; 0: the general form).  What bounds it is the latency of one token's
// chain (loads, then k rounds of a 64-lane maximum): all planes' loads are issued first, a lane sorts
// its own keys once, and a round is a maximum of the lanes' first keys in VALU moves, one ballot and
// one lane read (8 of 256 experts in 8 groups, 2,048 tokens: 8 us; 30 with strided ownership, plane
// after plane, and two butterflies a round).  Past four keys a lane the sort costs more than looking
// through them each round (512 experts, 8,192 tokens: 26 us sorted, 18 not).
template <int VPL, int PB>   // PB: planes in flight after the first
__global__ __launch_bounds__(256) void score_select_kernel(SelectArgs p, int run) {
  __shared__ int chosen[4 * 32];
  __shared__ __attribute__((aligned(16))) float rows[4][64 * VPL];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t t = (int64_t)blockIdx.x * 4 + wave;
  const int E = p.E, k = p.k, e0 = lane * VPL;
  const bool alone = gridDim.x == 1;   // one workgroup counts its own choices
  if (!alone && blockIdx.x == 0)
    for (int e = threadIdx.x; e < E; e += 256) p.count[e] = 0;
  if (t < p.T) {
    float l[VPL], s[VPL], bias[VPL], bal[VPL];
    uint32_t key[VPL];
    auto read = [&](auto vec) __attribute__((always_inline)) {
      constexpr bool VEC = decltype(vec)::value;
      lane_row<VEC>(p.b_r ? p.b_r : p.planes, E, bias);
      lane_row<VEC>(p.balance ? p.balance : p.planes, E, bal);
      lane_row<VEC>(p.planes + t * E, E, l);
      for (int z0 = 1; z0 < p.KS; z0 += PB) {
        float v[PB][VPL];
#pragma unroll
        for (int z = 0; z < PB; ++z)   // past the last plane: the last again, not added
          lane_row<VEC>(p.planes + ((int64_t)min(z0 + z, p.KS - 1) * p.T + t) * E, E, v[z]);
#pragma unroll
        for (int z = 0; z < PB; ++z)
#pragma unroll
          for (int i = 0; i < VPL; ++i) l[i] += z0 + z < p.KS ? v[z][i] : 0.f;
      }
    };
    if (E % 4 == 0) read(std::true_type{});
    else read(std::false_type{});
    if (p.b_r) {
#pragma unroll
      for (int i = 0; i < VPL; ++i) l[i] += bias[i];
    }
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      if (e0 + i >= E) l[i] = -INFINITY;
      else if (p.logits) p.logits[t * E + e0 + i] = l[i];
    }
#pragma unroll
    for (int i = 0; i < VPL; ++i) rows[wave][e0 + i] = l[i];
    const bool grouped = p.rule.top_groups < p.rule.groups, by_score = grouped || p.balance;
    float m = -INFINITY, sum = 0.f;   // softmax over all experts, where something asks for it
    auto sigmoid = [](float v) { return 1.0f / (1.0f + expf(-v)); };
    auto term = [&](float v) { return v == -INFINITY ? 0.f : expf(v - m); };   // also where every logit is -inf
    if (!p.rule.sigmoid && (by_score || !p.rule.renormalise)) {
#pragma unroll
      for (int i = 0; i < VPL; ++i) m = fmaxf(m, l[i]);
      m = group_max<64>(m);
#pragma unroll
      for (int i = 0; i < VPL; ++i) sum += s[i] = term(l[i]);
      sum = lanes_sum<1>(sum);
    }
    const bool none = sum == 0.f;
    if (by_score) {
#pragma unroll
      for (int i = 0; i < VPL; ++i) s[i] = p.rule.sigmoid ? sigmoid(l[i]) : none ? 0.f : s[i] / sum;
    }
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      key[i] = e0 + i < E ? order_key(p.balance ? s[i] + bal[i] : grouped ? s[i] : l[i]) : 0u;
    if (grouped) {
      auto score_key = [&](uint32_t top, uint32_t second) {
        float v = top > 1u ? key_value(top) : -INFINITY;
        if (p.rule.group_top == 2) v += second > 1u ? key_value(second) : -INFINITY;
        return order_key(v);
      };
      auto drop = [&](int i, bool kept) {
        if (e0 + i < E) {
          if (!kept) key[i] = 0u;
          else if (!p.balance) key[i] = order_key(l[i]);
        }
      };
      if (run) {
        // the two largest keys of a run of lanes, merged pairwise
        uint32_t a = 0, b = 0;
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
          b = max(b, min(a, key[i]));
          a = max(a, key[i]);
        }
        auto merge = [&](auto o) __attribute__((always_inline)) {
          if (run <= decltype(o)::value) return;
          const uint32_t c = partner<decltype(o)::value>(a), d = partner<decltype(o)::value>(b);
          b = max(min(a, c), max(b, d));
          a = max(a, c);
        };
        merge(std::integral_constant<int, 1>{});
        merge(std::integral_constant<int, 2>{});
        merge(std::integral_constant<int, 4>{});
        merge(std::integral_constant<int, 8>{});
        merge(std::integral_constant<int, 16>{});
        merge(std::integral_constant<int, 32>{});
        const uint32_t mine = score_key(a, b);
        const int g = lane / run;
        int before = 0;
        for (int o = 0; o < p.rule.groups; ++o) {
          const uint32_t other = (uint32_t)__builtin_amdgcn_readlane((int)mine, o * run);
          before += (other > mine || (other == mine && o < g)) ? 1 : 0;
        }
#pragma unroll
        for (int i = 0; i < VPL; ++i) drop(i, before < p.rule.top_groups);
      } else {
        const int per = E / p.rule.groups;
        uint32_t mine = 0;   // lane g: the key of group g's score
        for (int g = 0; g < p.rule.groups; ++g) {
          uint32_t a = 0, b = 0;
#pragma unroll
          for (int i = 0; i < VPL; ++i)
            if (e0 + i >= g * per && e0 + i < (g + 1) * per) {
              b = max(b, min(a, key[i]));
              a = max(a, key[i]);
            }
          const uint32_t top = group_max_u<64>(a);
          const unsigned long long holders = __ballot(a == top);
          const uint32_t second = __popcll(holders) > 1 ? top : group_max_u<64>(a == top ? b : a);
          const uint32_t score = score_key(top, second);
          if (lane == g) mine = score;
        }
        int before = 0;
        for (int g = 0; g < p.rule.groups; ++g) {
          const uint32_t o = (uint32_t)__builtin_amdgcn_readlane((int)mine, g);
          before += (o > mine || (o == mine && g < lane)) ? 1 : 0;
        }
        const unsigned long long keep = __ballot(lane < p.rule.groups && before < p.rule.top_groups);
#pragma unroll
        for (int i = 0; i < VPL; ++i) drop(i, e0 + i < E && ((keep >> ((e0 + i) / per)) & 1ull));
      }
    }
    int at[VPL], choice = 0;
#pragma unroll
    for (int i = 0; i < VPL; ++i) at[i] = i;
    constexpr bool SORTED = VPL <= 4;   // else a lane looks through its keys in every round
    if constexpr (SORTED) sort_keys<VPL>(key, at);
    for (int r = 0; r < k; ++r) {
      uint32_t first = key[0];
      int place = at[0];
      if constexpr (!SORTED) {
#pragma unroll
        for (int i = 1; i < VPL; ++i)
          if (key[i] > first) { first = key[i]; place = i; }
      }
      const int owner = __builtin_ctzll(__ballot(first == group_max_u<64>(first)));
      place = __builtin_amdgcn_readlane(place, owner);
      if (lane == r) choice = owner * VPL + place;
      const bool pop = lane == owner;
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        if constexpr (SORTED) {
          key[i] = !pop ? key[i] : i + 1 < VPL ? key[min(i + 1, VPL - 1)] : 0u;
          at[i] = pop ? at[min(i + 1, VPL - 1)] : at[i];
        } else {
          key[i] = pop && i == place ? 0u : key[i];
        }
      }
    }
    __builtin_amdgcn_wave_barrier();
    const float my_l = lane < k ? rows[wave][choice] : -INFINITY;
    float g = p.rule.sigmoid ? sigmoid(my_l) : none ? 0.f : term(my_l) / sum;
    if (p.rule.renormalise) {
      if (!p.rule.sigmoid) {   // over S alone: exact also where every s of S is tiny
        m = group_max<64>(my_l);
        g = term(my_l);
      }
      const float sum = lanes_sum<1>(lane < k ? g : 0.f);
      g = sum == 0.f ? 0.f : g / sum;
    }
    int rank = 0;
    for (int i = 0; i < k; ++i) rank += (__builtin_amdgcn_readlane(choice, i) < choice) ? 1 : 0;
    if (lane < k) {
      p.topk_idx[t * k + rank] = choice;
      p.topk_gate[t * k + rank] = p.rule.scale * g;
      chosen[wave * 32 + lane] = choice;
    }
  }
  if (!alone) return;
  __syncthreads();
  const int T = (int)p.T;
  for (int e = threadIdx.x; e < E; e += 256) {
    int n = 0;
    for (int w = 0; w < T; ++w)
      for (int j = 0; j < k; ++j) n += chosen[w * 32 + j] == e ? 1 : 0;
    p.count[e] = n;
  }
}

// count[e] += the copies of e among 8,192 ids per workgroup: an LDS histogram, then one integer addition per
// workgroup and expert (the same counts in any order).  One addition per copy would put a hot
// expert's thousands on one address.
__global__ __launch_bounds__(1024) void score_count_kernel(const int32_t* __restrict__ idx, int64_t n, int E,
                                                           int32_t* __restrict__ count) {
  extern __shared__ int32_t hist[];
  for (int e = threadIdx.x; e < E; e += 1024) hist[e] = 0;
  __syncthreads();
  const int64_t c0 = (int64_t)blockIdx.x * 8192 + threadIdx.x;
  int32_t v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = c0 + 1024 * i < n ? idx[c0 + 1024 * i] : -1;
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (v[i] >= 0) atomicAdd(&hist[v[i]], 1);
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += 1024)
    if (hist[e]) atomicAdd(&count[e], hist[e]);
}

// Logits of a few tokens (T <= SMALL_T, bf16): a weight stream.  One wavefront per expert row and K split (the
// splits of the MFMA router, whose tiles of 128 tokens would be empty here and its workgroups few: one
// token, 256 experts, d 7168: 24 -> 4 us), W_r in fp32 and x widened: plain fp32 sums.
constexpr int SMALL_T = 8, SCORE_KS = 32;
template <int NT>
__global__ __launch_bounds__(256) void router_small_kernel(const bf16_t* __restrict__ x, const float* __restrict__ w_r,
                                                           float* __restrict__ planes, int T, int d, int E, int KS) {
  const int lane = threadIdx.x & 63, item = blockIdx.x * 4 + (threadIdx.x >> 6);
  if (item >= E * KS) return;
  const int e = item / KS, z = item % KS, KA = d / 64;
  const int i0 = (int)((int64_t)KA * z / KS) * 64, i1 = (int)((int64_t)KA * (z + 1) / KS) * 64;
  float acc[NT] = {};
#pragma unroll 4
  for (uint32_t i = i0 + lane * 4; i < (uint32_t)i1; i += 256) {
    const f32x4 w = __builtin_nontemporal_load((const f32x4*)(w_r + (int64_t)e * d + i));
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const u32x2 v = *(const u32x2*)(x + (int64_t)min(t, T - 1) * d + i);
      acc[t] = fmaf(w[0], lo_bf(v[0]), acc[t]);
      acc[t] = fmaf(w[1], hi_bf(v[0]), acc[t]);
      acc[t] = fmaf(w[2], lo_bf(v[1]), acc[t]);
      acc[t] = fmaf(w[3], hi_bf(v[1]), acc[t]);
    }
  }
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const float sum = lanes_sum<1>(acc[t]);
    if (lane == 0 && t < T) planes[((int64_t)z * T + t) * E + e] = sum;
  }
}

// Logits of many tokens over 128 or more experts: partial planes of x W_r^T by 128 x 128 tiles, eight wavefronts of 64
// tokens x 32 experts, K in slices of 64 through two LDS buffers, W_r split into its three bf16 parts in
// registers (route_body.h).  The 32 x 32 wavefront tiles of the plain router read 4 KB of LDS for three MFMAs, this one
// 5 KB for six, and the next slice's parts are made and stored among a slice's MFMAs (its loads were issued
// two slices ahead).  hi's products have their own sum; mid's and lo's share one, 2^-8 of it.  Split z runs on XCD z
// (8 splits), so that each byte of x and W_r enters one L2 only.  The whole call, against the plain router's logits: 8,192
// tokens, d 7168, 512 experts 220 -> 194 us, 2,048 tokens, 256 experts 40 -> 37; a slice takes 1.5 us, its MFMAs 0.7.
// Rows of 128 bytes are swizzled by r / 2 (a 128-bit read is served in groups like rows 0-3, 12-15, 20-27, whose 16 places
// are then distinct; by r they meet in pairs).
__device__ __forceinline__ int lswz(int r, int c) { return r * RM_K + ((c ^ ((r >> 1) & 7)) << 4); }
constexpr int LG_T = 128, LG_BUF = 4 * LG_T * RM_K, LG_LDS = 2 * LG_BUF;
__global__ __launch_bounds__(512) void score_logits_kernel(const bf16_t* __restrict__ x, const float* __restrict__ w_r,
                                                           float* __restrict__ planes, int64_t T, int d, int E, int KS) {
  extern __shared__ __attribute__((aligned(1024))) uint8_t lds[];
  const int ne = (E + LG_T - 1) / LG_T, z = (int)(blockIdx.x % KS);
  int tile = (int)(blockIdx.x / KS);
  if (KS == 1) {   // XCD b % 8 takes a run of tiles, so that a token tile's expert tiles meet in one L2
    const int n = (int)gridDim.x, b = tile & 7, j = tile >> 3;
    tile = b * (n / 8) + min(b, n % 8) + j;
  }
  const int e0 = tile % ne * LG_T;
  const int64_t t0 = (int64_t)(tile / ne) * LG_T;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int wm = wave >> 2, wn = wave & 3, lr = lane & 31, lg = lane >> 5;
  const int KA = d / 64, kb = (int)((int64_t)KA * z / KS), KT = (int)((int64_t)KA * (z + 1) / KS) - kb;
  const bf16_t* xs[2];
  const float* ws[2];
  int at[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {   // piece q: row q / 8, elements 8 (q % 8) .. + 7 of a slice
    const int q = tid + 512 * i, r = q / 8, c = q % 8;
    xs[i] = x + min(t0 + r, T - 1) * d + (int64_t)kb * 64 + c * 8;
    ws[i] = w_r + (int64_t)min(e0 + r, E - 1) * d + (int64_t)kb * 64 + c * 8;
    at[i] = lswz(r, c);
  }
  u32x4 rx[2][2];
  f32x4 rw[2][2][2];
  auto load = [&](int kt, auto set) __attribute__((always_inline)) {
    constexpr int P = decltype(set)::value;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      rx[P][i] = *(const u32x4*)(xs[i] + kt * 64);
      rw[P][i][0] = *(const f32x4*)(ws[i] + kt * 64);
      rw[P][i][1] = *(const f32x4*)(ws[i] + kt * 64 + 4);
    }
  };
  auto store = [&](int i, auto set) __attribute__((always_inline)) {   // piece i of the set's slice to its buffer
    constexpr int P = decltype(set)::value;
    uint8_t* to = lds + P * LG_BUF + at[i];
    u32x4 h, m, l;
    router_split8(rw[P][i], h, m, l);
    *(u32x4*)to = rx[P][i];
    *(u32x4*)(to + LG_T * RM_K) = h;
    *(u32x4*)(to + 2 * LG_T * RM_K) = m;
    *(u32x4*)(to + 3 * LG_T * RM_K) = l;
  };
  f32x16 acc[2][2];   // [token half][hi | mid, lo]
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int p = 0; p < 2; ++p)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][p][r] = 0.f;
  // Slice kt (buffer P); slice kt + 1 is in the other set, kt + 2 goes into this one.
  auto step = [&](int kt, auto set, auto more, auto next) __attribute__((always_inline)) {
    constexpr int P = decltype(set)::value;
    using Other = std::integral_constant<int, 1 - P>;
    if constexpr (decltype(more)::value) load(kt + 2, set);
    // Scheduling barriers: the loads stay here, the stores, which wait for the loads before, come late in the slice.
    // (Reading a quarter's fragments before the MFMAs of the quarter before measured no better.)
    __builtin_amdgcn_sched_barrier(0);
    const uint8_t* b = lds + P * LG_BUF;
#pragma unroll
    for (int kk = 0; kk < 4; ++kk) {
      const int c = kk * 2 + lg;
      auto frag = [&](int row) __attribute__((always_inline)) {
        return __builtin_bit_cast(bf16x8, *(const u32x4*)(b + lswz(row, c)));
      };
      const bf16x8 a0 = frag(wm * 64 + lr), a1 = frag(wm * 64 + 32 + lr);
#pragma unroll
      for (int p = 0; p < 3; ++p) {
        const bf16x8 w = frag((p + 1) * LG_T + wn * 32 + lr);
        acc[0][p > 0] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a0, w, acc[0][p > 0], 0, 0, 0);
        acc[1][p > 0] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a1, w, acc[1][p > 0], 0, 0, 0);
      }
      if constexpr (decltype(next)::value) {
        if (kk == 2) store(0, Other{});
        if (kk == 3) store(1, Other{});
      }
      if (kk > 0) __builtin_amdgcn_sched_barrier(0);
    }
    __syncthreads();
  };
  using A = std::integral_constant<int, 0>;
  using B = std::integral_constant<int, 1>;
  using Yes = std::true_type;
  using No = std::false_type;
  load(0, A{});
  if (KT > 1) load(1, B{});
  store(0, A{});
  store(1, A{});
  __syncthreads();
  int kt = 0;
  for (; kt + 3 < KT; kt += 2) {
    step(kt, A{}, Yes{}, Yes{});
    step(kt + 1, B{}, Yes{}, Yes{});
  }
  if (KT - kt == 3) {
    step(kt, A{}, Yes{}, Yes{});
    step(kt + 1, B{}, No{}, Yes{});
    step(kt + 2, A{}, No{}, No{});
  } else if (KT - kt == 2) {
    step(kt, A{}, No{}, Yes{});
    step(kt + 1, B{}, No{}, No{});
  } else {
    step(kt, A{}, No{}, No{});
  }
  const int e = e0 + wn * 32 + lr;
  if (e >= E) return;
  float* out = planes + (int64_t)z * T * E;
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      const int64_t t = t0 + wm * 64 + 32 * i + 8 * (r / 4) + 4 * lg + (r % 4);
      if (t < T) out[t * E + e] = acc[i][0][r] + acc[i][1][r];
    }
}

// K splits of 64 x 64 logit tiles where the 128 x 128 tiles (or the plain router's fewer splits) would leave
// half of the CUs idle, at least four slices of 64 each; 0: the plain router's choice.  (256 experts, d 7168, the
// whole call: 9 tokens 33 -> 16 us, 400 tokens 35 -> 24; 128 experts, d 4096, 200 tokens 23 -> 15.)
static int fine_splits(int64_t T, int E, int d) {
  if (T <= SMALL_T) return 0;
  const int64_t big = ((T + 127) / 128) * ((E + 127) / 128), tiles = ((T + 63) / 64) * ((E + 63) / 64);
  if ((router_big(E) ? big : (tiles + 1) / 2) * router_ksplit(T, E, d) >= 128) return 0;
  return (int)std::max<int64_t>(1, std::min<int64_t>({SCORE_KS, 512 / tiles, d / 256}));
}
size_t route_scored_workspace_bytes(int64_t T, int E, int d) {
  return ((size_t)fine_splits(T, E, d) * T * E * sizeof(float) + 255) & ~(size_t)255;
}

hipError_t launch_route_scored(const void* x, bool x_f32, const float* w_r, const float* b_r,
                               const float* balance, const ScoreRule& rule, int64_t T, int d, int E,
                               int k, float* planes, int32_t* topk_idx, float* topk_gate,
                               int32_t* count, float* logits, hipStream_t st) {
  int ks = 1;
  hipError_t err = hipSuccess;
  if (!x_f32 && T <= SMALL_T) {
    ks = router_ksplit(T, E, d);
    const unsigned g = (unsigned)((E * ks + 3) / 4);
    if (T == 1) router_small_kernel<1><<<g, 256, 0, st>>>((const bf16_t*)x, w_r, planes, (int)T, d, E, ks);
    else if (T <= 4) router_small_kernel<4><<<g, 256, 0, st>>>((const bf16_t*)x, w_r, planes, (int)T, d, E, ks);
    else router_small_kernel<8><<<g, 256, 0, st>>>((const bf16_t*)x, w_r, planes, (int)T, d, E, ks);
    err = hipGetLastError();
  } else if (const int fine = x_f32 ? 0 : fine_splits(T, E, d)) {
    ks = fine;
    err = launch_router_logits_64(x, w_r, T, d, E, ks, planes, st);
  } else if (!x_f32 && router_big(E)) {
    ks = router_ksplit(T, E, d);
    if ((err = hipFuncSetAttribute((const void*)score_logits_kernel, hipFuncAttributeMaxDynamicSharedMemorySize, LG_LDS)) !=
        hipSuccess)
      return err;
    const int64_t tiles = ((T + LG_T - 1) / LG_T) * ((E + LG_T - 1) / LG_T);
    score_logits_kernel<<<(unsigned)(tiles * ks), 512, LG_LDS, st>>>((const bf16_t*)x, w_r, planes, T, d, E, ks);
    err = hipGetLastError();
  } else {
    err = launch_router_logits(x, x_f32, w_r, T, d, E, planes, &ks, st);
  }
  if (err != hipSuccess) return err;
  const SelectArgs p{planes, ks, b_r, balance, T, E, k, rule, topk_idx, topk_gate, count, logits};
  const unsigned g = (unsigned)((T + 3) / 4);
  const int vpl = (E + 63) / 64, per = E / rule.groups;
#define SELECT(V)                                                                             \
  {                                                                                           \
    const int q = per % V == 0 ? per / V : 0;                                                 \
    const int run = q > 0 && (q & (q - 1)) == 0 ? q : 0;                                      \
    if (ks <= 2) score_select_kernel<V, 1><<<g, 256, 0, st>>>(p, run);                        \
    else if (ks <= 8 || V >= 8) score_select_kernel<V, V <= 8 ? 7 : 4><<<g, 256, 0, st>>>(p, run); \
    else score_select_kernel<V, V <= 4 ? 16 : V <= 8 ? 7 : 4><<<g, 256, 0, st>>>(p, run);                  \
  }
  if (vpl <= 1) SELECT(1)
  else if (vpl <= 2) SELECT(2)
  else if (vpl <= 4) SELECT(4)
  else if (vpl <= 8) SELECT(8)
  else SELECT(16)
#undef SELECT
  if (g > 1)
    score_count_kernel<<<(unsigned)((T * k + 8191) / 8192), 1024, E * sizeof(int32_t), st>>>(topk_idx, T * k, E, count);
  return hipGetLastError();
}

// ----------------------------------------------------------------------------- gradient
// dl [T, E] of the gates, one wavefront per token and DL_TW tokens in turn.  1 - s of a sigmoid is
// taken as 1 / (1 + exp(l)), which keeps its digits where s is next to 1.
//
// For bf16 tokens dl leaves as three bf16 parts, hi = bf16(dl), mid = bf16(dl - hi) and lo = bf16(dl - hi - mid),
// which hold all 24 bits of it, as rows [hi | mid] of 2 Ep values (Ep: E rounded up to 64, the
// padding 0) and [lo] of Ep.  With W_r's columns as [hi | mid], hi hi + hi mid + mid hi is dl W_r
// to 2^-15 of its terms (mid x mid and the third parts are left out: dx is rounded to bf16, half a
// step 2^-8); the three parts against the exact bf16 x are dl^T x to fp32, in which dW_r leaves.
constexpr int DL_TW = 2;

struct DlArgs {
  const float* dgate;
  const float* dlogits;
  const float* logits;
  const int32_t* topk_idx;
  int64_t T, Tp;        // Tp: rows written, those from T on zero
  int E, Ep, k;
  ScoreRule rule;
  float* dl;            // fp32 tokens: [T, E]
  bf16_t* planes;       // bf16 tokens: [Tp, 2 Ep]
  bf16_t* low;          // bf16 tokens: [Tp, Ep]
  uint32_t* zero;       // bf16 tokens: 256 words set to 0
  const float* w_r;     // bf16 tokens: W_r [E, d] to be turned by the workgroups from G on
  bf16_t* wt;           // [d, 2 Ep]
  int d, G;
  float* db_part;       // [workgroups, E] sums over a workgroup's tokens, or NULL
};

// W_r [E, d] fp32 -> [d, 2 Ep] bf16, rows [hi | mid] of W_r's columns: 64 x 64 of them, turned through LDS,
// read and written in 16-byte pieces.
__device__ __forceinline__ void score_turn(const DlArgs& p, int at, float (*tile)[65]) {
  const int c0 = at % (p.d / 64) * 64, e0 = at / (p.d / 64) * 64;   // d is a multiple of 64
  const int tid = threadIdx.x;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int e = tid / 16 + 16 * i, c = tid % 16 * 4;
    const f32x4 w = e0 + e < p.E ? *(const f32x4*)(p.w_r + (int64_t)(e0 + e) * p.d + c0 + c) : f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int q = 0; q < 4; ++q) tile[e][c + q] = w[q];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int c = tid / 8 + 32 * i, e = tid % 8 * 8;
    u32x4 hi, mid;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const float u = tile[e + 2 * q][c], v = tile[e + 2 * q + 1][c];
      hi[q] = pack_bf2(u, v);
      mid[q] = pack_bf2(u - lo_bf(hi[q]), v - hi_bf(hi[q]));
    }
    bf16_t* row = p.wt + (int64_t)(c0 + c) * 2 * p.Ep + e0 + e;
    *(u32x4*)row = hi;
    *(u32x4*)(row + p.Ep) = mid;
  }
}

// dl of token t by one wavefront: lane l holds experts l, l + 64, ... (zeros where ok is false).
template <int VPL>
__device__ __forceinline__ void token_dl(const DlArgs& p, int64_t t, bool ok, float (&dl)[VPL]) {
  const int lane = threadIdx.x & 63, E = p.E, k = p.k;
  float l[VPL];
  float dg = 0.f, lj = -INFINITY;
  int ej = -1;
  if (ok && lane < k) {
    const int e = p.topk_idx[t * k + lane];
    if (e >= 0 && e < E) {
      ej = e;
      dg = p.rule.scale * p.dgate[t * k + lane];
      lj = p.logits[t * E + e];
    }
  }
  const bool dense = !p.rule.renormalise && !p.rule.sigmoid;   // every logit moves every softmax score
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const int e = lane + 64 * i;
    l[i] = dense && ok && e < E ? p.logits[t * E + e] : -INFINITY;
    dl[i] = ok && e < E && p.dlogits ? p.dlogits[t * E + e] : 0.f;
  }
  float v = 0.f;   // lane j: dl of the j-th chosen expert (the softmax's own part)
  if (p.rule.renormalise) {
    float g;
    if (p.rule.sigmoid) g = 1.0f / (1.0f + expf(-lj));
    else {
      const float m = group_max<64>(lj);
      g = lj == -INFINITY ? 0.f : expf(lj - m);
    }
    g = ej >= 0 ? g : 0.f;
    const float sum = lanes_sum<1>(g);
    g = sum == 0.f ? 0.f : g / sum;
    v = g * (dg - lanes_sum<1>(g * dg));
    if (p.rule.sigmoid) v *= 1.0f / (1.0f + expf(lj));
  } else if (p.rule.sigmoid) {
    v = dg * (1.0f / (1.0f + expf(-lj))) * (1.0f / (1.0f + expf(lj)));
  } else {
    float m = -INFINITY, sum = 0.f;
#pragma unroll
    for (int i = 0; i < VPL; ++i) m = fmaxf(m, l[i]);
    m = group_max<64>(m);
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      l[i] = l[i] == -INFINITY ? 0.f : expf(l[i] - m);
      sum += l[i];
    }
    sum = lanes_sum<1>(sum);
    const float inv = sum == 0.f ? 0.f : 1.0f / sum;
    v = ej >= 0 && lj != -INFINITY ? expf(lj - m) * inv * dg : 0.f;
    const float all = lanes_sum<1>(v);
#pragma unroll
    for (int i = 0; i < VPL; ++i) dl[i] -= l[i] * inv * all;
  }
  if (ej < 0 || lj == -INFINITY) v = 0.f;
  for (int j = 0; j < k; ++j) {
    const int e = __builtin_amdgcn_readlane(ej, j);
    const float add = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), j));
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      if (lane + 64 * i == e) dl[i] += add;
  }
}

template <int VPL, bool F32>
__global__ __launch_bounds__(256) void score_dl_kernel(DlArgs p) {
  __shared__ float dbs[4][64 * VPL];
  __shared__ float tile[F32 ? 1 : 64][65];
  if constexpr (!F32)
    if ((int)blockIdx.x >= p.G) return score_turn(p, (int)blockIdx.x - p.G, tile);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int E = p.E;
  if (!F32 && blockIdx.x == 0) p.zero[threadIdx.x] = 0u;
  float db[VPL] = {};
  for (int w = 0; w < DL_TW; ++w) {
    const int64_t t = ((int64_t)blockIdx.x * 4 + wave) * DL_TW + w;
    if (t >= p.Tp) break;
    const bool ok = t < p.T;
    float dl[VPL];
    token_dl<VPL>(p, t, ok, dl);
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const int e = lane + 64 * i;
      db[i] += dl[i];
      if constexpr (F32) {
        if (e < E) p.dl[t * E + e] = dl[i];
      } else if (e < p.Ep) {
        const bf16_t hi = f2bf(dl[i]), mid = f2bf(dl[i] - bf2f(hi));
        bf16_t* row = p.planes + t * 2 * p.Ep + e;
        row[0] = hi;
        row[p.Ep] = mid;
        p.low[t * p.Ep + e] = f2bf(dl[i] - bf2f(hi) - bf2f(mid));
      }
    }
  }
  if (!p.db_part) return;
#pragma unroll
  for (int i = 0; i < VPL; ++i) dbs[wave][lane + 64 * i] = db[i];
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += 256)
    p.db_part[(int64_t)blockIdx.x * E + e] = (dbs[0][e] + dbs[1][e]) + (dbs[2][e] + dbs[3][e]);
}

// The whole gradient of a few bf16 tokens (T <= NT) in one launch, in fp32: one pass over W_r (dx) and dW_r. A
// workgroup owns 32 columns, a thread four of them and every 64th expert; each workgroup makes
// dl for itself (T rows of logits from the L2), which costs less than another launch.  dx is
// joined over the lanes, then over the wavefronts in order.  (One token, d 4096, 512 experts: 34 us with the four
// launches below, 9 here, of which 8 in the kernel; 16 tokens, 64 experts: 20 -> 9.)
template <int VPL, int NT>
__global__ __launch_bounds__(512) void score_bwd_few_kernel(DlArgs p, const bf16_t* __restrict__ x, const bf16_t* dx_in,
                                                            bf16_t* dx, float* __restrict__ dw, float* __restrict__ db) {
  constexpr int PITCH = NT + 4;            // floats per expert of dl
  __shared__ __attribute__((aligned(16))) float red[8][NT][32];
  extern __shared__ __attribute__((aligned(16))) float dls[];   // [E][PITCH]
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int T = (int)p.T, E = p.E, c0 = blockIdx.x * 32 + (tid & 7) * 4;
  for (int t = wave; t < NT; t += 8) {
    float dl[VPL];
    token_dl<VPL>(p, t, t < T, dl);
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      if (lane + 64 * i < E) dls[(lane + 64 * i) * PITCH + t] = dl[i];
  }
  float xf[NT][4], acc[NT][4];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const u32x2 v = *(const u32x2*)(x + (int64_t)min(t, T - 1) * p.d + c0);   // rows past T meet zeros of dl
    xf[t][0] = lo_bf(v[0]); xf[t][1] = hi_bf(v[0]); xf[t][2] = lo_bf(v[1]); xf[t][3] = hi_bf(v[1]);
#pragma unroll
    for (int q = 0; q < 4; ++q) acc[t][q] = 0.f;
  }
  __syncthreads();
  if (db && blockIdx.x == 0)
    for (int e = tid; e < E; e += 512) {
      float s = 0.f;
      for (int t = 0; t < T; ++t) s += dls[e * PITCH + t];
      db[e] = s;
    }
#pragma unroll 2
  for (int e = tid >> 3; e < E; e += 64) {
    const f32x4 w = __builtin_nontemporal_load((const f32x4*)(p.w_r + (int64_t)e * p.d + c0));
    f32x4 o = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const float s = dls[e * PITCH + t];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        o[q] = fmaf(s, xf[t][q], o[q]);
        acc[t][q] = fmaf(s, w[q], acc[t][q]);
      }
    }
    *(f32x4*)(dw + (int64_t)e * p.d + c0) = o;
  }
#pragma unroll
  for (int t = 0; t < NT; ++t) {
#pragma unroll
    for (int q = 0; q < 4; ++q) acc[t][q] = lanes_sum<8>(acc[t][q]);
    if (lane < 8) *(f32x4*)&red[wave][t][lane * 4] = f32x4{acc[t][0], acc[t][1], acc[t][2], acc[t][3]};
  }
  __syncthreads();
  for (int i = tid; i < T * 32; i += 512) {
    const int t = i / 32, c = i % 32;
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < 8; ++w) s += red[w][t][c];
    const int64_t at = (int64_t)t * p.d + blockIdx.x * 32 + c;
    dx[at] = f2bf((dx_in ? bf2f(dx_in[at]) : 0.f) + s);
  }
}

// Partial planes of dW_r [E, d] = dl^T x for bf16 tokens.  Both operands are row-major with the
// reduction index (the token) as the row, so a stage holds 32 token rows as they are, of x once and of the
// three parts of dl, and the MFMA fragments are read with the transposing LDS reads of the weight
// gradients (backward.hip).  256 experts x 256 columns per workgroup, eight wavefronts of 64 x 128: a
// fragment of x meets all three parts (with a stage per part instead, x staged and read three times:
// 122 us where this takes 100, 8,192 tokens, d 4,096, 512 experts).  The tokens are split over Z
// workgroups, each with a plane of its own; split z runs on XCD z (Z = 8), so that a token row of
// x crosses into one L2 only.
struct DwArgs {
  const bf16_t* planes;   // [Tp, 2 Ep]: hi | mid
  const bf16_t* low;      // [Tp, Ep]
  const bf16_t* x;        // [T, d]
  const bf16_t* zero;     // 1 KB of zeros: rows past T of x
  int64_t T, Tp;
  int E, Ep, d, Z;
  float* part;            // [Z, E, d]
};
constexpr int DW_M = 256, DW_N = 256, DW_K = 32, DW_S = 2, DW_ROW = 512;   // bytes of a staged row
constexpr int DW_TILE = DW_K * DW_ROW, DW_STAGE = 4 * DW_TILE, DW_LDS = DW_S * DW_STAGE;

__device__ __forceinline__ void score_dw_body(const DwArgs& p, const int block) {
  extern __shared__ __attribute__((aligned(1024))) uint8_t lds[];
  const uint32_t lds0 = (uint32_t)(uintptr_t)lds;
  const int z = block % p.Z, tile = block / p.Z;
  const int mt = (p.E + DW_M - 1) / DW_M;
  const int m0 = (tile % mt) * DW_M, n0 = (tile / mt) * DW_N;
  const int64_t steps = p.Tp / DW_K, s0 = steps * z / p.Z;
  const int KT = (int)(steps * (z + 1) / p.Z - s0);
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave >> 1, wn = wave & 1, lr = lane & 31, lg = lane >> 5;
  // copies: kilobyte 8 c + wave of a tile (x, hi, mid, lo) is its rows 2 (8 c + wave) and + 1
  const int crow = lane / 32;
  int acol[2], bcol[2];
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    const int r = 2 * (8 * c + wave) + crow, lc = wsw(r, lane % 32);
    acol[c] = min(m0 + lc * 8, p.Ep - 8);
    bcol[c] = min(n0 + lc * 8, p.d - 8);
  }
  auto issue = [&](int i) __attribute__((always_inline)) {
    const uint32_t st = lds0 + (uint32_t)(i % DW_S) * DW_STAGE;
    const int64_t r0 = (s0 + i) * DW_K;
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int64_t t = r0 + 2 * (8 * c + wave) + crow;
      const uint32_t to = __builtin_amdgcn_readfirstlane(st + (8 * c + wave) * 1024);
      const bf16_t* row = p.planes + t * 2 * p.Ep + acol[c];
      dma16_at(t < p.T ? p.x + t * p.d + bcol[c] : p.zero + (lane & 31) * 8, to);
      dma16_at(row, to + DW_TILE);
      dma16_at(row + p.Ep, to + 2 * DW_TILE);
      dma16_at(p.low + t * p.Ep + acol[c], to + 3 * DW_TILE);
    }
  };
  f32x16 acc[4][2];
#pragma unroll
  for (int j = 0; j < 4; ++j)
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[j][i][r] = 0.f;
  int foff[6];   // offsets in a stage: 2 fragments of dl's first part, 4 of x
  {
    const int g = lane >> 4, gi = lane & 15, qq = gi >> 2, ss = gi & 3;
    const int r0 = 8 * (g >> 1) + qq;
#pragma unroll
    for (int q = 0; q < 6; ++q) {
      const int col = (q < 2 ? wm * 64 + q * 32 : wn * 128 + (q - 2) * 32) + 16 * (g & 1) + 4 * ss;
      foff[q] = (q < 2 ? DW_TILE : 0) + r0 * DW_ROW + wsw(r0, col >> 3) * 16 + (col & 7) * 2;
    }
  }
  auto frag = [&](const uint8_t* sb, int at) __attribute__((always_inline)) -> bf16x8 {
    const v4i16_t lo = ds_tr16(sb + at), hi = ds_tr16(sb + at + 4 * DW_ROW);
    return __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
  };
  const bool live = m0 + wm * 64 < p.E && n0 + wn * 128 < p.d;   // else none of this wavefront's results exists
  if (KT > 0) issue(0);
  for (int kt = 0; kt < KT; ++kt) {
    bwait_vm<0>();
    __syncthreads();
    if (kt + 1 < KT) issue(kt + 1);
    if (!live) continue;
    const uint8_t* sb = lds + (kt % DW_S) * DW_STAGE;
#pragma unroll
    for (int kk = 0; kk < DW_K / 16; ++kk) {
      const int o = kk * 16 * DW_ROW;
      bf16x8 fa[3][2], fb[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) fb[j] = frag(sb, foff[2 + j] + o);
#pragma unroll
      for (int q = 0; q < 3; ++q)
#pragma unroll
        for (int i = 0; i < 2; ++i) fa[q][i] = frag(sb, foff[i] + q * DW_TILE + o);
#pragma unroll
      for (int q = 0; q < 3; ++q)
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int i = 0; i < 2; ++i) acc[j][i] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fb[j], fa[q][i], acc[j][i], 0, 0, 0);
    }
  }
  // acc[j][i][r]: expert m0 + 64 wm + 32 i + lr, column n0 + 128 wn + 32 j + 8 (r / 4) + 4 lg + r % 4.  Each half i is
  // staged in a wavefront's own 16 KB (32 rows of 32 16-byte chunks, XOR-swizzled by the row) and
  // written as whole rows of 512 bytes.
  __syncthreads();
  uint8_t* wl = lds + wave * 16384;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int h = 0; h < 4; ++h)
        *(f32x4*)(wl + lr * 512 + (((8 * j + 2 * h + lg) ^ lr) << 4)) =
            f32x4{acc[j][i][4 * h], acc[j][i][4 * h + 1], acc[j][i][4 * h + 2], acc[j][i][4 * h + 3]};
    __builtin_amdgcn_wave_barrier();
#pragma unroll 4
    for (int q = 0; q < 16; ++q) {
      const int r = 2 * q + (lane >> 5), c = lane & 31;
      const f32x4 v = *(const f32x4*)(wl + r * 512 + ((c ^ r) << 4));
      const int e = m0 + wm * 64 + 32 * i + r, n = n0 + wn * 128 + 4 * c;
      if (e < p.E && n < p.d) *(f32x4*)(p.part + ((int64_t)z * p.E + e) * p.d + n) = v;
    }
    __builtin_amdgcn_wave_barrier();
  }
}

// dW_r's workgroups (below nw; up to nb, a multiple of 8 that keeps the rest's XCDs, they are none) and dx's tiles in one
// launch: neither needs the other, and for few tokens neither fills the chip (the whole gradient, us before and after:
// 64 tokens, d 2048, 256 experts 29 -> 19; 2,000 tokens, d 1024, 256 experts 47 -> 37; 8,192 tokens, d 4096, 512
// experts 183 for the two either way).
template <int FM, int S>
__global__ __launch_bounds__(512) void score_products_kernel(Fp8Args a, DwArgs q, int nw, int nb) {
  const int b = (int)blockIdx.x;
  if (b >= nb) fp8_tile_body<FM, TILE_ADD, S, false>(a, b - nb);
  else if (b < nw) score_dw_body(q, b);
}

template <int FM, int S>
static hipError_t run_products(const Fp8Args& a, const DwArgs& q, int nw, hipStream_t st) {
  constexpr int tile = fp8_tile_lds<FM, TILE_ADD, S>(), lds = tile > DW_LDS ? tile : DW_LDS;
  static_assert(lds <= 160 * 1024, "LDS");
  auto kern = score_products_kernel<FM, S>;
  hipError_t err = hipFuncSetAttribute((const void*)kern, hipFuncAttributeMaxDynamicSharedMemorySize, lds);
  if (err != hipSuccess) return err;
  const int nb = (nw + 7) / 8 * 8;
  const int64_t tiles = (a.a_rows + 64 * FM - 1) / (64 * FM) * ((a.N + 255) / 256);
  kern<<<(unsigned)(nb + (tiles + 7) / 8 * 8), 512, lds, st>>>(a, q, nw, nb);
  return hipGetLastError();
}

// fp32 tokens: dx [T, d] = dx_in + dl [T, E] W_r [E, d], and partial planes of dW_r [E, d] = dl^T x, on the
// vector units.  64 x 64 tiles, 256 threads of 4 x 4, the reduction in steps of 16 through LDS, each step's
// sum added to the running one (two levels).
constexpr int GB = 64, GK = 16;

__global__ __launch_bounds__(256) void score_dx_kernel(const float* __restrict__ dl,
                                                       const float* __restrict__ w_r, const float* dx_in,
                                                       int64_t T, int E, int d, float* dx) {
  __shared__ float as[GK][GB + 4], bs[GK][GB + 4];
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  const int64_t t0 = (int64_t)blockIdx.y * GB;
  const int c0 = blockIdx.x * GB;
  float acc[4][4] = {};
  for (int e0 = 0; e0 < E; e0 += GK) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int r = tid >> 2, ke = e0 + (tid & 3) * 4 + q;
      as[(tid & 3) * 4 + q][r] = t0 + r < T && ke < E ? dl[(t0 + r) * E + ke] : 0.f;
      const int kr = tid >> 4, c = (tid & 15) * 4 + q;
      bs[kr][c] = e0 + kr < E && c0 + c < d ? w_r[(int64_t)(e0 + kr) * d + c0 + c] : 0.f;
    }
    __syncthreads();
    float part[4][4] = {};
#pragma unroll
    for (int kk = 0; kk < GK; ++kk)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) part[i][j] = fmaf(as[kk][ty * 4 + i], bs[kk][tx * 4 + j], part[i][j]);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i][j] += part[i][j];
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t t = t0 + ty * 4 + i;
      const int c = c0 + tx * 4 + j;
      if (t < T && c < d) {
        const int64_t at = t * d + c;
        dx[at] = (dx_in ? dx_in[at] : 0.f) + acc[i][j];
      }
    }
}

__global__ __launch_bounds__(256) void score_dw_kernel(const float* __restrict__ dl, const float* __restrict__ x,
                                                       int64_t T, int E, int d, float* __restrict__ part) {
  __shared__ float as[GK][GB + 4], bs[GK][GB + 4];
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  const int e0 = blockIdx.y * GB, c0 = blockIdx.x * GB;
  const int64_t steps = (T + GK - 1) / GK;
  const int64_t s0 = steps * blockIdx.z / gridDim.z, s1 = steps * (blockIdx.z + 1) / gridDim.z;
  float acc[4][4] = {};
  for (int64_t s = s0; s < s1; ++s) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int kr = tid >> 4, c = (tid & 15) * 4 + q;
      const int64_t t = s * GK + kr;
      as[kr][c] = t < T && e0 + c < E ? dl[t * E + e0 + c] : 0.f;
      float v = 0.f;
      if (t < T && c0 + c < d) v = x[t * d + c0 + c];
      bs[kr][c] = v;
    }
    __syncthreads();
    float part_[4][4] = {};
#pragma unroll
    for (int kk = 0; kk < GK; ++kk)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) part_[i][j] = fmaf(as[kk][ty * 4 + i], bs[kk][tx * 4 + j], part_[i][j]);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i][j] += part_[i][j];
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int e = e0 + ty * 4 + i, c = c0 + tx * 4 + j;
      if (e < E && c < d) part[((int64_t)blockIdx.z * E + e) * d + c] = acc[i][j];
    }
}

// The last sums: dw[i] = sum over z of part[z, i], z ascending (workgroups below `planes`), and
// db[e] = sum over g of db_part[g, e], eight interleaved sums per expert (the rest).
__global__ __launch_bounds__(256) void score_sum_kernel(const float* __restrict__ part, int Z, int64_t n, float* __restrict__ dw,
                                                        int planes, const float* __restrict__ db_part, int G, int E,
                                                        float* __restrict__ db) {
  __shared__ float red[8][32];
  if ((int)blockIdx.x < planes) {
    const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
    if (i >= n) return;
    f32x4 s = *(const f32x4*)(part + i);
#pragma unroll 8
    for (int z = 1; z < Z; ++z) s += *(const f32x4*)(part + z * n + i);
    *(f32x4*)(dw + i) = s;
    return;
  }
  const int cl = threadIdx.x & 31, r = threadIdx.x >> 5, e = ((int)blockIdx.x - planes) * 32 + cl;
  float s = 0.f;
  if (e < E) {
#pragma unroll 8
    for (int g = r; g < G; g += 8) s += db_part[(int64_t)g * E + e];
  }
  red[r][cl] = s;
  __syncthreads();
  if (r == 0 && e < E) {
    s = red[0][cl];
#pragma unroll
    for (int i = 1; i < 8; ++i) s += red[i][cl];
    db[e] = s;
  }
}

// fp32: about four workgroups a CU.  bf16: the least estimated time of one round of steps of 32 tokens, 1.3 us each,
// and of the planes, written and read once.
static int dw_splits(bool f32, int64_t T, int E, int d) {
  const int m = f32 ? GB : DW_M, n = f32 ? GB : DW_N;
  const int64_t tiles = (int64_t)((E + m - 1) / m) * ((d + n - 1) / n);
  if (f32) return (int)std::max<int64_t>(1, std::min<int64_t>({8, 1024 / tiles, T / 128}));
  const int64_t steps = (T + DW_K - 1) / DW_K;
  int best = 1;
  double least = 1e300;
  for (int Z = 1; Z == 1 || (Z <= 64 && Z * tiles <= 256 && Z * 4 <= steps); Z *= 2) {
    const double t = (double)((steps + Z - 1) / Z) * 1.3 + (Z > 1 ? 2.0 + (double)Z * E * d * 8 / 4.5e6 : 0.0);
    if (t < least) { least = t; best = Z; }
  }
  return best;
}

// One launch, without a workspace (score_bwd_few_kernel).
static bool bwd_few(bool f32, int64_t T) { return !f32 && T <= 16; }

struct ScoreBwdLayout {
  size_t dl, low, wt, zero, dw, db, total;
  int64_t Tp;
  int Ep, Z, G;
};
static ScoreBwdLayout score_bwd_layout(bool f32, int64_t T, int E, int d) {
  auto al = [](size_t b) { return (b + 255) & ~(size_t)255; };
  ScoreBwdLayout L{};
  L.Ep = (E + 63) / 64 * 64;
  L.Tp = f32 ? T : (T + DW_K - 1) / DW_K * DW_K;
  L.Z = dw_splits(f32, T, E, d);
  L.G = (int)((L.Tp + 4 * DL_TW - 1) / (4 * DL_TW));
  size_t o = 0;
  if (bwd_few(f32, T)) {   // keeps nothing: the least a call asks for
    L.total = 256;
    return L;
  }
  L.dl = o; o += al(f32 ? (size_t)T * E * 4 : (size_t)L.Tp * 2 * L.Ep * 2);
  L.low = o; o += f32 ? 0 : al((size_t)L.Tp * L.Ep * 2);
  L.wt = o; o += f32 ? 0 : al((size_t)d * 2 * L.Ep * 2);
  L.zero = o; o += 1024;
  L.dw = o; o += L.Z > 1 ? al((size_t)L.Z * E * d * 4) : 0;   // one split writes dW_r itself
  L.db = o; o += al((size_t)L.G * E * 4);
  L.total = o;
  return L;
}
size_t route_scored_bwd_workspace_bytes(bool f32, int64_t T, int E, int d) {
  return T == 0 ? 0 : score_bwd_layout(f32, T, E, d).total;
}

hipError_t launch_route_scored_bwd(bool f32, const ScoreRule& rule, const float* dgate,
                                   const float* dlogits, const void* x, const float* w_r,
                                   const float* logits, const int32_t* topk_idx, const void* dx_in,
                                   int64_t T, int d, int E, int k, void* dx, float* dw, float* db,
                                   void* ws, hipStream_t st) {
  const ScoreBwdLayout L = score_bwd_layout(f32, T, E, d);
  uint8_t* w = (uint8_t*)ws;
  float* part = L.Z > 1 ? (float*)(w + L.dw) : dw;
  float* dbp = (float*)(w + L.db);
  const DlArgs p{dgate, dlogits, logits, topk_idx, T, L.Tp, E, L.Ep, k, rule, (float*)(w + L.dl),
                 (bf16_t*)(w + L.dl), (bf16_t*)(w + L.low), (uint32_t*)(w + L.zero),
                 w_r, (bf16_t*)(w + L.wt), d, L.G, db ? dbp : nullptr};
  const int vpl = (E + 63) / 64;
  if (bwd_few(f32, T)) {
#define FEW(V, N)                                                                                                \
  {                                                                                                             \
    hipError_t e_ = hipFuncSetAttribute((const void*)score_bwd_few_kernel<V, N>,                                 \
                                        hipFuncAttributeMaxDynamicSharedMemorySize, 64 * V * (N + 4) * 4);       \
    if (e_ != hipSuccess) return e_;                                                                             \
    score_bwd_few_kernel<V, N><<<(unsigned)(d / 32), 512, E * (N + 4) * 4, st>>>(                               \
        p, (const bf16_t*)x, (const bf16_t*)dx_in, (bf16_t*)dx, dw, db);                                         \
  }
#define FEW_V(V) if (T <= 4) FEW(V, 4) else FEW(V, 16)
    if (vpl <= 1) FEW_V(1)
    else if (vpl <= 2) FEW_V(2)
    else if (vpl <= 4) FEW_V(4)
    else if (vpl <= 8) FEW_V(8)
    else FEW_V(16)
#undef FEW_V
#undef FEW
    return hipGetLastError();
  }
#define DL(V)                                                                   \
  {                                                                             \
    if (f32) score_dl_kernel<V, true><<<(unsigned)L.G, 256, 0, st>>>(p);        \
    else score_dl_kernel<V, false><<<(unsigned)(L.G + d / 64 * (L.Ep / 64)), 256, 0, st>>>(p); \
  }
  if (vpl <= 1) DL(1)
  else if (vpl <= 2) DL(2)
  else if (vpl <= 4) DL(4)
  else if (vpl <= 8) DL(8)
  else DL(16)
#undef DL
  hipError_t err = hipGetLastError();
  if (err != hipSuccess) return err;
  if (f32) {
    score_dx_kernel<<<dim3((d + GB - 1) / GB, (unsigned)((T + GB - 1) / GB)), 256, 0, st>>>(
        p.dl, w_r, (const float*)dx_in, T, E, d, (float*)dx);
    score_dw_kernel<<<dim3((d + GB - 1) / GB, (E + GB - 1) / GB, L.Z), 256, 0, st>>>(p.dl, (const float*)x, T, E,
                                                                                    d, part);
  } else {
    const DwArgs q{p.planes, p.low, (const bf16_t*)x, (const bf16_t*)p.zero, T, L.Tp, E, L.Ep, d, L.Z, part};
    int nw = (int)((int64_t)((E + DW_M - 1) / DW_M) * ((d + DW_N - 1) / DW_N) * L.Z);
    // dx: at most 2^18 rows a launch (32-bit offsets inside the operands), dW_r beside the first
    for (int64_t t0 = 0; t0 < T; t0 += (int64_t)1 << 18, nw = 0) {
      Fp8Args a{};
      a.A = (const uint8_t*)(p.planes + t0 * 2 * L.Ep);
      a.W0 = (const uint8_t*)p.wt;
      a.a_rows = std::min<int64_t>(T - t0, (int64_t)1 << 18);
      a.C = a.a_rows;
      a.K = 4 * L.Ep;
      a.N = d;
      a.Z = 1;
      a.group = FP8_GROUP;
      a.out = (bf16_t*)dx + t0 * d;
      a.add = dx_in ? (const bf16_t*)dx_in + t0 * d : nullptr;
      const int fm = tile_add_height(a.a_rows, d, 6 * L.Ep);
      err = fm == 1   ? run_products<1, 3>(a, q, nw, st)
            : fm == 2 ? run_products<2, 3>(a, q, nw, st)
            : fm == 3 ? run_products<3, 2>(a, q, nw, st)
                      : run_products<4, 2>(a, q, nw, st);
      if (err != hipSuccess) return err;
    }
  }
  if ((err = hipGetLastError()) != hipSuccess) return err;
  const int64_t n = (int64_t)E * d;   // d is a multiple of 8
  const int planes = L.Z > 1 ? (int)((n / 4 + 255) / 256) : 0, sums = db ? (E + 31) / 32 : 0;
  if (planes + sums)
    score_sum_kernel<<<(unsigned)(planes + sums), 256, 0, st>>>(part, L.Z, n, dw, planes, dbp, L.G, E, db);
  return hipGetLastError();
}

}  // namespace moe
