// Scored routing: softmax or sigmoid scores, a balance bias that decides the choice only,
// groups of experts, top-k, optionally renormalised gates; and the gradient of the gates.
//
//   l = x W_r^T (+ b);  s = softmax(l) | sigmoid(l);  c = s (+ balance);
//   group score = sum of its group_top largest c; the top_groups best groups are kept;
//   S = k largest c in them (ties to the lower id);  g = scale s_S (/ sum_S s)
//
// The logits come from the router's MFMA kernels (route.hip); here one wavefront owns a token.
#include <algorithm>

#include "common.h"
#include "kernels.h"
#include "route_body.h"

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
  int32_t* count;        // [E], zeroed before
  float* logits;
};

// One wavefront per token; lane l owns experts l + 64 i.
template <int VPL>
__global__ __launch_bounds__(256) void score_select_kernel(SelectArgs p) {
  const int lane = threadIdx.x & 63;
  const int64_t t = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (t >= p.T) return;
  const int E = p.E, k = p.k;
  float l[VPL], s[VPL];
  uint32_t key[VPL];
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const int e = lane + 64 * i;
    if (e < E) {
      float v = p.planes[t * E + e];
      for (int z = 1; z < p.KS; ++z) v += p.planes[((int64_t)z * p.T + t) * E + e];
      l[i] = v + (p.b_r ? p.b_r[e] : 0.f);
      if (p.logits) p.logits[t * E + e] = l[i];
    } else {
      l[i] = -INFINITY;
    }
  }
  if (p.rule.sigmoid) {
#pragma unroll
    for (int i = 0; i < VPL; ++i) s[i] = 1.0f / (1.0f + expf(-l[i]));
  } else {
    float m = -INFINITY, sum = 0.f;
#pragma unroll
    for (int i = 0; i < VPL; ++i) m = fmaxf(m, l[i]);
    m = group_max<64>(m);
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      s[i] = l[i] == -INFINITY ? 0.f : expf(l[i] - m);   // also where every logit is -inf
      sum += s[i];
    }
    sum = wave_sum(sum);
    const bool none = sum == 0.f;
#pragma unroll
    for (int i = 0; i < VPL; ++i) s[i] = none ? 0.f : s[i] / sum;
  }
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const int e = lane + 64 * i;
    key[i] = e < E ? order_key(p.balance ? s[i] + p.balance[e] : p.rule.groups > 1 && p.rule.top_groups < p.rule.groups ? s[i] : l[i]) : 0u;
  }
  if (p.rule.top_groups < p.rule.groups) {
    const int per = E / p.rule.groups;
    uint32_t mine = 0;   // lane g: the key of group g's score
    for (int g = 0; g < p.rule.groups; ++g) {
      uint32_t best = 0;
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        const int e = lane + 64 * i;
        if (e >= g * per && e < (g + 1) * per && key[i] > best) best = key[i];
      }
      const uint32_t top = group_max_u<64>(best);
      float score = top > 1u ? key_value(top) : -INFINITY;
      if (p.rule.group_top == 2) {
        // the second largest: the largest below `top`, or `top` again if two experts hold it
        int holders = 0;
        uint32_t next = 0;
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
          const int e = lane + 64 * i;
          if (e >= g * per && e < (g + 1) * per) {
            if (key[i] == top) ++holders;
            else if (key[i] > next) next = key[i];
          }
        }
        const unsigned long long once = __ballot(holders > 0), twice = __ballot(holders > 1);
        const uint32_t second = (__popcll(once) > 1 || twice) ? top : group_max_u<64>(next);
        score += second > 1u ? key_value(second) : -INFINITY;
      }
      if (lane == g) mine = order_key(score);
    }
    int before = 0;
    for (int g = 0; g < p.rule.groups; ++g) {
      const uint32_t o = (uint32_t)__builtin_amdgcn_readlane((int)mine, g);
      before += (o > mine || (o == mine && g < lane)) ? 1 : 0;
    }
    const unsigned long long keep = __ballot(lane < p.rule.groups && before < p.rule.top_groups);
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const int e = lane + 64 * i;
      if (e < E) {
        if (!((keep >> (e / per)) & 1ull)) key[i] = 0u;
        else if (!p.balance) key[i] = order_key(l[i]);
      }
    }
  }
  int choice = 0;
  float my_s = 0.f, my_l = -INFINITY;
  for (int r = 0; r < k; ++r) {
    uint32_t bk = 0;
    int bi = 0x7fffffff;
    float bs = 0.f, bl = 0.f;
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      if (key[i] > bk) { bk = key[i]; bi = lane + 64 * i; bs = s[i]; bl = l[i]; }
    const uint32_t mk = group_max_u<64>(bk);
    const int e = group_min_i<64>(bk == mk ? bi : 0x7fffffff);
    const float se = __int_as_float(__builtin_amdgcn_ds_bpermute((e & 63) * 4, __float_as_int(bs)));
    const float le = __int_as_float(__builtin_amdgcn_ds_bpermute((e & 63) * 4, __float_as_int(bl)));
    if (lane == r) { choice = e; my_s = se; my_l = le; }
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      if (lane + 64 * i == e) key[i] = 0u;
  }
  float g = my_s;
  if (p.rule.renormalise) {
    if (!p.rule.sigmoid) {   // over S alone: exact also where every s of S is tiny
      const float m = group_max<64>(lane < k ? my_l : -INFINITY);
      g = lane < k && my_l != -INFINITY ? expf(my_l - m) : 0.f;
    }
    const float sum = wave_sum(lane < k ? g : 0.f);
    g = sum == 0.f ? 0.f : g / sum;
  }
  int rank = 0;
  for (int i = 0; i < k; ++i) rank += (__builtin_amdgcn_readlane(choice, i) < choice) ? 1 : 0;
  if (lane < k) {
    p.topk_idx[t * k + rank] = choice;
    p.topk_gate[t * k + rank] = p.rule.scale * g;
    atomicAdd(&p.count[choice], 1);   // integers: the same counts in any order
  }
}

__global__ __launch_bounds__(1024) void zero_count_kernel(int32_t* __restrict__ count, int E) {
  for (int e = threadIdx.x; e < E; e += 1024) count[e] = 0;
}

hipError_t launch_route_scored(const void* x, bool x_f32, const float* w_r, const float* b_r,
                               const float* balance, const ScoreRule& rule, int64_t T, int d, int E,
                               int k, float* planes, int32_t* topk_idx, float* topk_gate,
                               int32_t* count, float* logits, hipStream_t st) {
  int ks = 1;
  zero_count_kernel<<<1, 1024, 0, st>>>(count, E);
  hipError_t err = launch_router_logits(x, x_f32, w_r, T, d, E, planes, &ks, st);
  if (err != hipSuccess) return err;
  const SelectArgs p{planes, ks, b_r, balance, T, E, k, rule, topk_idx, topk_gate, count, logits};
  const unsigned g = (unsigned)((T + 3) / 4);
  const int vpl = (E + 63) / 64;
  if (vpl <= 1) score_select_kernel<1><<<g, 256, 0, st>>>(p);
  else if (vpl <= 2) score_select_kernel<2><<<g, 256, 0, st>>>(p);
  else if (vpl <= 4) score_select_kernel<4><<<g, 256, 0, st>>>(p);
  else if (vpl <= 8) score_select_kernel<8><<<g, 256, 0, st>>>(p);
  else score_select_kernel<16><<<g, 256, 0, st>>>(p);
  return hipGetLastError();
}

// ----------------------------------------------------------------------------- gradient
// dl [T, E] of the gates, one wavefront per token.  1 - s of a sigmoid is taken as
// 1 / (1 + exp(l)), which keeps its digits where s is next to 1.
struct DlArgs {
  const float* dgate;
  const float* dlogits;
  const float* logits;
  const int32_t* topk_idx;
  int64_t T;
  int E, k;
  ScoreRule rule;
  float* dl;
};

template <int VPL>
__global__ __launch_bounds__(256) void score_dl_kernel(DlArgs p) {
  const int lane = threadIdx.x & 63;
  const int64_t t = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (t >= p.T) return;
  const int E = p.E, k = p.k;
  float l[VPL], dl[VPL];
  float dg = 0.f, lj = -INFINITY;
  int ej = -1;
  if (lane < k) {
    const int e = p.topk_idx[t * k + lane];
    if (e >= 0 && e < E) {
      ej = e;
      dg = p.rule.scale * p.dgate[t * k + lane];
      lj = p.logits[t * E + e];
    }
  }
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const int e = lane + 64 * i;
    l[i] = e < E ? p.logits[t * E + e] : -INFINITY;
    dl[i] = 0.f;
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
    const float sum = wave_sum(g);
    g = sum == 0.f ? 0.f : g / sum;
    v = g * (dg - wave_sum(g * dg));
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
    sum = wave_sum(sum);
    const float inv = sum == 0.f ? 0.f : 1.0f / sum;
    v = ej >= 0 && lj != -INFINITY ? expf(lj - m) * inv * dg : 0.f;
    const float all = wave_sum(v);
#pragma unroll
    for (int i = 0; i < VPL; ++i) dl[i] = -l[i] * inv * all;
  }
  if (ej < 0 || lj == -INFINITY) v = 0.f;
  for (int j = 0; j < k; ++j) {
    const int e = __builtin_amdgcn_readlane(ej, j);
    const float add = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), j));
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      if (lane + 64 * i == e) dl[i] += add;
  }
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const int e = lane + 64 * i;
    if (e < E) p.dl[t * E + e] = dl[i] + (p.dlogits ? p.dlogits[t * E + e] : 0.f);
  }
}

// dx [T, d] = dx_in + dl [T, E] W_r [E, d], and partial planes of dW_r [E, d] = dl^T x.
// 64 x 64 tiles, 256 threads of 4 x 4, the reduction in steps of 16 through LDS, each step's
// sum added to the running one (two levels).
constexpr int GB = 64, GK = 16;

template <bool F32>
__global__ __launch_bounds__(256) void score_dx_kernel(const float* __restrict__ dl,
                                                       const float* __restrict__ w_r, const void* dx_in,
                                                       int64_t T, int E, int d, void* dx) {
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
        if constexpr (F32) ((float*)dx)[at] = (dx_in ? ((const float*)dx_in)[at] : 0.f) + acc[i][j];
        else ((bf16_t*)dx)[at] = f2bf((dx_in ? bf2f(((const bf16_t*)dx_in)[at]) : 0.f) + acc[i][j]);
      }
    }
}

template <bool F32>
__global__ __launch_bounds__(256) void score_dw_kernel(const float* __restrict__ dl, const void* __restrict__ x,
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
      if (t < T && c0 + c < d) v = F32 ? ((const float*)x)[t * d + c0 + c] : bf2f(((const bf16_t*)x)[t * d + c0 + c]);
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

// out[i] = sum over z of part[z, i], z ascending.
__global__ __launch_bounds__(256) void plane_sum_kernel(const float* __restrict__ part, int Z, int64_t n,
                                                        float* __restrict__ out) {
  const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
  if (i >= n) return;
  f32x4 s = *(const f32x4*)(part + i);
  for (int z = 1; z < Z; ++z) s += *(const f32x4*)(part + z * n + i);
  *(f32x4*)(out + i) = s;
}

// db partials: workgroup b adds rows b, b + G, ... of dl.
constexpr int DB_G = 64;
__global__ __launch_bounds__(256) void score_db_kernel(const float* __restrict__ dl, int64_t T, int E,
                                                       float* __restrict__ part) {
  for (int e = threadIdx.x; e < E; e += 256) {
    float s = 0.f;
    for (int64_t t = blockIdx.x; t < T; t += gridDim.x) s += dl[t * E + e];
    part[(int64_t)blockIdx.x * E + e] = s;
  }
}

static int dw_splits(int64_t T, int E, int d) {
  const int64_t tiles = (int64_t)((E + GB - 1) / GB) * ((d + GB - 1) / GB);
  return (int)std::max<int64_t>(1, std::min<int64_t>({8, 1024 / tiles, T / 128}));
}

struct ScoreBwdLayout {
  size_t dl, dw, db, total;
};
static ScoreBwdLayout score_bwd_layout(int64_t T, int E, int d) {
  auto al = [](size_t b) { return (b + 255) & ~(size_t)255; };
  ScoreBwdLayout L;
  size_t o = 0;
  L.dl = o; o += al((size_t)T * E * 4);
  L.dw = o; o += al((size_t)dw_splits(T, E, d) * E * d * 4);
  L.db = o; o += al((size_t)DB_G * E * 4);
  L.total = o;
  return L;
}
size_t route_scored_bwd_workspace_bytes(int64_t T, int E, int d) {
  return T == 0 ? 0 : score_bwd_layout(T, E, d).total;
}

hipError_t launch_route_scored_bwd(bool f32, const ScoreRule& rule, const float* dgate,
                                   const float* dlogits, const void* x, const float* w_r,
                                   const float* logits, const int32_t* topk_idx, const void* dx_in,
                                   int64_t T, int d, int E, int k, void* dx, float* dw, float* db,
                                   void* ws, hipStream_t st) {
  const ScoreBwdLayout L = score_bwd_layout(T, E, d);
  float* dl = (float*)((uint8_t*)ws + L.dl);
  float* part = (float*)((uint8_t*)ws + L.dw);
  float* dbp = (float*)((uint8_t*)ws + L.db);
  const DlArgs p{dgate, dlogits, logits, topk_idx, T, E, k, rule, dl};
  const unsigned g = (unsigned)((T + 3) / 4);
  const int vpl = (E + 63) / 64;
  if (vpl <= 1) score_dl_kernel<1><<<g, 256, 0, st>>>(p);
  else if (vpl <= 2) score_dl_kernel<2><<<g, 256, 0, st>>>(p);
  else if (vpl <= 4) score_dl_kernel<4><<<g, 256, 0, st>>>(p);
  else if (vpl <= 8) score_dl_kernel<8><<<g, 256, 0, st>>>(p);
  else score_dl_kernel<16><<<g, 256, 0, st>>>(p);
  const dim3 gx((d + GB - 1) / GB, (unsigned)((T + GB - 1) / GB));
  const int Z = dw_splits(T, E, d);
  const dim3 gw((d + GB - 1) / GB, (E + GB - 1) / GB, Z);
  if (f32) {
    score_dx_kernel<true><<<gx, 256, 0, st>>>(dl, w_r, dx_in, T, E, d, dx);
    score_dw_kernel<true><<<gw, 256, 0, st>>>(dl, x, T, E, d, part);
  } else {
    score_dx_kernel<false><<<gx, 256, 0, st>>>(dl, w_r, dx_in, T, E, d, dx);
    score_dw_kernel<false><<<gw, 256, 0, st>>>(dl, x, T, E, d, part);
  }
  const int64_t n = (int64_t)E * d;
  plane_sum_kernel<<<(unsigned)((n / 4 + 255) / 256), 256, 0, st>>>(part, Z, n, dw);
  if (db) {
    const int G = (int)std::min<int64_t>(T, DB_G);
    score_db_kernel<<<G, 256, 0, st>>>(dl, T, E, dbp);
    hipError_t err = launch_column_sum(dbp, G, E, db, st);
    if (err != hipSuccess) return err;
  }
  return hipGetLastError();
}

}  // namespace moe
