// The choice of one token by one wavefront: scores, groups, top-k and gates from its logits (the scored router's selection
// kernel and the few-token layer with 4-bit weights).
#pragma once

#include <type_traits>

#include "common.h"
#include "kernels.h"

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

// A group of `per` experts as a run of lanes of VPL experts each: its length, a power of two, or 0 (none).
__host__ __device__ __forceinline__ int group_run(int per, int VPL) {
  const int q = per % VPL == 0 ? per / VPL : 0;
  return (q & (q - 1)) == 0 ? q : 0;
}

// l: the token's logits, lane l's experts l VPL .. + VPL - 1, -inf past E, also in `row` [64 VPL] in LDS; bal: the balance
// bias likewise.  On return lane r < k holds the r-th choice, its rank by expert id and its gate.
template <int VPL>
__device__ __forceinline__ void select_row(const ScoreRule& rule, bool balanced, int E, int k, int run, const float (&l)[VPL],
                                           const float (&bal)[VPL], const float* row, int& choice, int& rank, float& gate) {
  const int lane = threadIdx.x & 63, e0 = lane * VPL;
  float s[VPL];
  uint32_t key[VPL];
  const bool grouped = rule.top_groups < rule.groups, by_score = grouped || balanced;
  float m = -INFINITY, sum = 0.f;   // softmax over all experts, where something asks for it
  auto sigmoid = [](float v) { return 1.0f / (1.0f + expf(-v)); };
  auto term = [&](float v) { return v == -INFINITY ? 0.f : expf(v - m); };   // also where every logit is -inf
  if (!rule.sigmoid && (by_score || !rule.renormalise)) {
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
    for (int i = 0; i < VPL; ++i) s[i] = rule.sigmoid ? sigmoid(l[i]) : none ? 0.f : s[i] / sum;
  }
#pragma unroll
  for (int i = 0; i < VPL; ++i)
    key[i] = e0 + i < E ? order_key(balanced ? s[i] + bal[i] : grouped ? s[i] : l[i]) : 0u;
  if (grouped) {
    auto score_key = [&](uint32_t top, uint32_t second) {
      float v = top > 1u ? key_value(top) : -INFINITY;
      if (rule.group_top == 2) v += second > 1u ? key_value(second) : -INFINITY;
      return order_key(v);
    };
    auto drop = [&](int i, bool kept) {
      if (e0 + i < E) {
        if (!kept) key[i] = 0u;
        else if (!balanced) key[i] = order_key(l[i]);
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
      for (int o = 0; o < rule.groups; ++o) {
        const uint32_t other = (uint32_t)__builtin_amdgcn_readlane((int)mine, o * run);
        before += (other > mine || (other == mine && o < g)) ? 1 : 0;
      }
#pragma unroll
      for (int i = 0; i < VPL; ++i) drop(i, before < rule.top_groups);
    } else {
      const int per = E / rule.groups;
      uint32_t mine = 0;   // lane g: the key of group g's score
      for (int g = 0; g < rule.groups; ++g) {
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
      for (int g = 0; g < rule.groups; ++g) {
        const uint32_t o = (uint32_t)__builtin_amdgcn_readlane((int)mine, g);
        before += (o > mine || (o == mine && g < lane)) ? 1 : 0;
      }
      const unsigned long long keep = __ballot(lane < rule.groups && before < rule.top_groups);
#pragma unroll
      for (int i = 0; i < VPL; ++i) drop(i, e0 + i < E && ((keep >> ((e0 + i) / per)) & 1ull));
    }
  }
  int at[VPL];
  choice = 0;
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
  const float my_l = lane < k ? row[choice] : -INFINITY;
  gate = rule.sigmoid ? sigmoid(my_l) : none ? 0.f : term(my_l) / sum;
  if (rule.renormalise) {
    if (!rule.sigmoid) {   // over S alone: exact also where every s of S is tiny
      m = group_max<64>(my_l);
      gate = term(my_l);
    }
    const float sum = lanes_sum<1>(lane < k ? gate : 0.f);
    gate = sum == 0.f ? 0.f : gate / sum;
  }
  rank = 0;
  for (int i = 0; i < k; ++i) rank += (__builtin_amdgcn_readlane(choice, i) < choice) ? 1 : 0;
  gate *= rule.scale;
}

}  // namespace moe
