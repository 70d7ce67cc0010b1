// The FP8 product's tile for many rows: BM = 64 FM token rows x 256 weight rows, eight wavefronts in
// 4 x 2, K in blocks of 128 through a ring of S LDS stages filled by global -> LDS copies.
//
// One 16x16x128 MFMA is exactly one block of 128: its result is the block's partial sum of 16
// weight rows x 16 token rows, and enters the accumulators with four multiply-adds per lane while
// the next MFMAs run (the matrix pipe is busy 32 clocks per MFMA, the four multiply-adds take
// 16).  A wavefront holds token fragments wm, wm + 4, ... of 16 rows (so that the rows of a
// partly filled tile are spread over all wavefronts) and 128 weight rows, all of one scale block:
// 64 gate and the matching 64 up rows (SWIGLU), or 128 rows of W.
#pragma once

#include <type_traits>

#include "fp8.h"
#include "gemm_body.h"

namespace moe {

struct Fp8Args {
  const uint8_t* A;        // token rows [C, K] codes
  const float* As;         // [K/128][a_rows]
  const uint8_t* W0;       // [E, N, K]
  const uint8_t* W1;       // SWIGLU: the up weights
  const float* S0;         // [E][ceil(N/128)][K/128]
  const float* S1;
  int64_t a_rows;
  int K, N;
  const int32_t* offset;   // ring segments; NULL: one product of all a_rows rows
  const int32_t* tiles;    // the row tiles' list, or NULL: found from the offsets
  const int32_t* ntiles;
  int64_t head, C;
  void* out;               // SWIGLU: H codes [C, N]; else bf16 or fp32 [C, N]
  float* out_scale;        // SWIGLU: [N/128][C]
  bf16_t* saved_au;        // SWIGLU: [C, 2N] or NULL
  const bf16_t* add;       // TILE_ADD: [C, N] or NULL (may be out)
  int Z;                   // K splits of a dense product (1 elsewhere)
  int E;                   // experts
  float* h32;              // the thin kernel's h in fp32 [n, N], segment order
  int group;               // row tiles that take the same column tile one after another
};

constexpr int FP8_GROUP = 4;   // row tiles that take a column tile one after another

// The row tiles of all experts' segments, BM rows each, in expert order, found by every wavefront for itself from
// the offsets (lane l counts the tiles of experts l V .. l V + V - 1): a launch that writes a list of them costs 5 us
// (16 experts x 64 rows, d 1024, f 512: 23 -> 20 us), this scan 0.3 us more in each workgroup than reading the list.
struct SegmentTiles {
  const int32_t* offset;
  int32_t o[5];               // V <= 4: the offsets around this lane's experts
  int V, n, incl, total;      // this lane's tiles, those up to it, all
};
// Inclusive sum over the lanes, in VALU moves: within rows of 16, then their last lanes into the rows behind.
__device__ __forceinline__ int lanes_scan(int v) {
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xf, 0xf, false);   // row_shr:1, 2, 4, 8
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xf, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xf, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xf, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xa, 0xf, false);   // row_bcast:15 into rows 1 and 3
  v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xc, 0xf, false);   // row_bcast:31 into rows 2 and 3
  return v;
}
template <int BM>
__device__ __forceinline__ SegmentTiles segment_tiles(const int32_t* offset, int E) {
  SegmentTiles s{offset, {}, (E + 63) / 64, 0, 0, 0};
  const int e0 = (threadIdx.x & 63) * s.V;
#pragma unroll
  for (int i = 0; i < 5; ++i) s.o[i] = offset[min(e0 + i, E)];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (i < s.V) s.n += (s.o[i + 1] - s.o[i] + BM - 1) / BM;
  int32_t lo = s.o[4];
  for (int i = 5; i <= s.V; ++i) {
    const int32_t hi = offset[min(e0 + i, E)];
    s.n += (hi - lo + BM - 1) / BM;
    lo = hi;
  }
  s.incl = lanes_scan(s.n);
  s.total = __builtin_amdgcn_readlane(s.incl, 63);
  return s;
}
// The expert e of tile mt < total, its first tile, its segment's start and its rows.
template <int BM>
__device__ __forceinline__ void find_segment(const SegmentTiles& s, int mt, int& e, int& first, int32_t& seg, int& rows) {
  const int owner = __builtin_ctzll(__ballot(s.incl > mt));
  first = __builtin_amdgcn_readlane(s.incl, owner) - __builtin_amdgcn_readlane(s.n, owner);
  e = owner * s.V;
  bool found = false;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (!found && i < s.V) {
      seg = __builtin_amdgcn_readlane(s.o[i], owner);
      rows = __builtin_amdgcn_readlane(s.o[i + 1], owner) - seg;
      const int t = (rows + BM - 1) / BM;
      found = mt < first + t;
      if (!found) { first += t; ++e; }
    }
  while (!found) {   // V > 4; ends: the owner's experts hold tile mt
    seg = s.offset[e];
    rows = s.offset[e + 1] - seg;
    const int t = (rows + BM - 1) / BM;
    found = mt < first + t;
    if (!found) { first += t; ++e; }
  }
}

// Lane l's 32 bytes of a row's block.  (Which of the block's 128 positions a lane's byte is does
// not matter as long as both operands agree.)
__device__ __forceinline__ i32x8 fp8_join(u32x4 a, u32x4 b) {
  return i32x8{(int)a[0], (int)a[1], (int)a[2], (int)a[3], (int)b[0], (int)b[1], (int)b[2], (int)b[3]};
}
__device__ __forceinline__ f32x4 fp8_mfma16(i32x8 w, i32x8 a) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, a, f32x4{0.f, 0.f, 0.f, 0.f}, 0, 0, 0, 0, 0, 0);
}
// The same sum on the bf16 MFMA: the 32 codes of a lane in four steps of 8.
struct Wide16 {
  bf16x8 v[4];
};
__device__ __forceinline__ bf16x8 fp8_widen8(int lo, int hi) {
  union {
    __bf16 __attribute__((ext_vector_type(2))) p[4];
    bf16x8 v;
  } o;
  o.p[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, false);
  o.p[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, true);
  o.p[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, false);
  o.p[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, true);
  return o.v;
}
__device__ __forceinline__ Wide16 fp8_widen(i32x8 w) {
  return Wide16{{fp8_widen8(w[0], w[1]), fp8_widen8(w[2], w[3]), fp8_widen8(w[4], w[5]), fp8_widen8(w[6], w[7])}};
}
__device__ __forceinline__ f32x4 fp8_wide16(const Wide16& w, const Wide16& a) {
  f32x4 c = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int q = 0; q < 4; ++q) c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w.v[q], a.v[q], c, 0, 0, 0);
  return c;
}

// FP8_PART: K split over Z workgroups, each with an fp32 plane of its own [Z, C, N] (FP8_F32 with Z > 1 likewise).
// TILE_ADD: two bf16 parts [hi | mid] of each operand's rows (K: bytes of such a row, a stage holds 64 elements),
// without scales: out = round(add + hi hi^T + hi mid^T + mid hi^T).
enum { FP8_BF16 = 0, FP8_F32 = 1, FP8_PART = 2, TILE_ADD = 3, FP8_SWIGLU = 4, FP8_SWIGLU_SAVE = 5 };

template <int FM, int KIND>
struct Fp8Stage {
  static constexpr int BM = 64 * FM, BN = 256;
  static constexpr int A = 0, B = BM * 128, SC = B + BN * 128;   // SC: BM row scales, 2 block scales, padding
  static constexpr int SIZE = SC + (KIND == TILE_ADD ? 0 : 8 * 256);
  static constexpr int L = FM + 4 + (KIND == TILE_ADD ? 0 : 1);  // copies per wavefront and stage
};

// NT: the weights are read past the caches' retention (each is read about once).
template <int FM, int KIND, int S, bool NT>
__device__ __forceinline__ void fp8_tile_body(const Fp8Args& p, const int block) {
  using SL = Fp8Stage<FM, KIND>;
  constexpr int BM = SL::BM, BN = SL::BN, L = SL::L;
  constexpr bool SWIGLU = KIND >= FP8_SWIGLU, WIDE = KIND == FP8_F32, ADD = KIND == TILE_ADD;
  static_assert(FM >= 1 && FM <= 4 && S >= 2 && S <= 4, "tile");
  extern __shared__ __attribute__((aligned(1024))) uint8_t lds[];
  const uint32_t lds0 = (uint32_t)(uintptr_t)lds;
  constexpr int CB = SWIGLU ? 1 : 2;             // output blocks of 128 columns per tile
  const int nblk = (p.N + 127) / 128, nct = (nblk + CB - 1) / CB;
  SegmentTiles st{};
  if (p.offset && !p.tiles) st = segment_tiles<BM>(p.offset, p.E);
  const int nmt = p.tiles ? *p.ntiles : p.offset ? st.total : (int)((p.a_rows + BM - 1) / BM);
  // Tile order: XCD x (workgroup b runs on XCD b % 8) takes one run of the logical tiles.  An expert's
  // row tiles form groups of `group`; inside a group the column tile is the slower index, so that
  // tiles running together on an XCD share both their token rows and their weight rows in its L2
  // (groups of 4 against 1, 4 experts x 4,096 rows: 749 -> 737 us; starting tiles at different K blocks, as
  // the bf16 GEMMs do, then loses: 752 us).
  const int V = nmt * nct, per = (V * p.Z + 7) / 8, li = block >> 3;
  const int TZ = (block & 7) * per + li;
  if (li >= per || TZ >= V * p.Z) return;
  const int z = TZ / V, T = TZ - z * V;          // the K split, the tile
  int e = 0, t0 = 0, R = nmt, mt = T / nct;      // expert, its first row tile, its row tiles
  int32_t seg = 0;
  int64_t all = p.a_rows;                        // its rows
  if (p.tiles) {
    e = p.tiles[2 * mt];
    t0 = mt - p.tiles[2 * mt + 1] / BM;
    seg = p.offset[e];
    all = p.offset[e + 1] - seg;
    R = (int)((all + BM - 1) / BM);
  } else if (p.offset) {
    int n;
    find_segment<BM>(st, mt, e, t0, seg, n);
    auto uni = [](int v) { return __builtin_amdgcn_readfirstlane(v); };
    e = uni(e); t0 = uni(t0); seg = uni(seg); all = uni(n);
    R = (int)((all + BM - 1) / BM);
  }
  const int local = T - t0 * nct, grp = local / (p.group * nct), rem = local - grp * p.group * nct;
  const int rg = min(p.group, R - grp * p.group), ct = rem / rg;
  const int rt = grp * p.group + rem % rg;       // the row tile inside its expert
  mt = t0 + rt;
  const int row0 = rt * BM, rows = (int)min((int64_t)BM, all - row0);
  const int n0 = ct * CB * 128;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave >> 1, wn = wave & 1, lr = lane & 15, lg = lane >> 4;
  const uint32_t K = (uint32_t)p.K;
  const int part = p.K / 256;                    // ADD: blocks of one part of a row
  const int KA = ADD ? 3 * part : p.K / 128, kb = (int)((int64_t)KA * z / p.Z), KT = (int)((int64_t)KA * (z + 1) / p.Z) - kb;

  // copies: 16-byte chunk j of a tile is slot j % 8 of row j / 8 and holds the chunk of that row whose
  // swizzled place it is (swz of gemm_body.h)
  uint32_t a_off[FM], b_off[4], s_off;
  const uint8_t* b_base[4];
  const uint8_t* s_base;
  int64_t s_step;
#pragma unroll
  for (int i = 0; i < FM; ++i) {
    const int j = (8 * i + wave) * 64 + lane, r = j / 8;
    const int c = (swz<128>(r, j % 8) - r * 128) >> 4;
    a_off[i] = (uint32_t)ring_slot(p.head, seg, row0 + min(r, rows - 1), p.C) * K + c * 16;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int j = (8 * i + wave) * 64 + lane, r = j / 8;
    const int c = (swz<128>(r, j % 8) - r * 128) >> 4;
    const bool up = SWIGLU && i >= 2;            // rows 128 .. 255
    b_base[i] = (up ? p.W1 : p.W0) + (int64_t)e * p.N * K;
    b_off[i] = (uint32_t)min(n0 + (up ? r - 128 : r), p.N - 1) * K + c * 16;
  }
  if constexpr (ADD) {
    s_base = nullptr;
    s_off = 0;
    s_step = 0;
  } else if (wave < FM) {                        // 64 row scales
    const int r = 64 * wave + lane;
    s_base = (const uint8_t*)p.As;
    s_off = (uint32_t)ring_slot(p.head, seg, row0 + min(r, rows - 1), p.C) * 4;
    s_step = p.a_rows * 4;
  } else if constexpr (SWIGLU) {                 // a block scale in every lane: wavefront FM gate, FM + 1 up
    s_base = (const uint8_t*)(((wave - FM) & 1 ? p.S1 : p.S0) + ((int64_t)e * nblk + ct) * KA);
    s_off = 0;
    s_step = 4;
  } else {                                       // the tile's two block scales in turn
    s_base = (const uint8_t*)(p.S0 + (int64_t)e * nblk * KA);
    s_off = (uint32_t)min(2 * ct + (lane & 1), nblk - 1) * KA * 4;
    s_step = 4;
  }
  auto issue_one = [&](int i_, int c) __attribute__((always_inline)) {   // step i_: block kb + i_
    const uint32_t st = lds0 + (uint32_t)(i_ % S) * SL::SIZE;
    const int kt = kb + i_;
    if (c < FM) {
      const int ka = ADD && kt >= part ? kt - part : kt;
      dma16(p.A + (size_t)ka * 128, a_off[c], __builtin_amdgcn_readfirstlane(st + SL::A + (8 * c + wave) * 1024));
    } else if (c < FM + 4) {
      const int i = c - FM;
      const uint32_t to = __builtin_amdgcn_readfirstlane(st + SL::B + (8 * i + wave) * 1024);
      const int kw = ADD && kt >= 2 * part ? kt - 2 * part : kt;
      if (NT) dma16nt(b_base[i] + (size_t)kw * 128, b_off[i], to);
      else dma16(b_base[i] + (size_t)kw * 128, b_off[i], to);
    } else {
      dma4(s_base + (size_t)kt * s_step, s_off, __builtin_amdgcn_readfirstlane(st + SL::SC + wave * 256));
    }
  };
  auto wait_stage = [&](int later) __attribute__((always_inline)) {
    if (later <= 0) wait_vm<0>();
    else if (later == 1) wait_vm<L>();
    else wait_vm<2 * L>();
  };

  f32x4 acc[FM][8];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

  // A lane takes the 16-byte chunks lg and lg + 4 of row 16 q + lr, which sit at r * 128 + (chunk ^ (r >> 1 & 7)) * 16,
  // and r >> 1 & 7 is lr >> 1: one per-lane offset and a multiple of 2048.  A 128-bit read is served in
  // groups like lanes 0-3, 12-15, 20-27: with chunks that differ by 1 between lg = 0 and 1 (2 and 3) their
  // 16 places are distinct; with chunks 2 lg, 2 lg + 1 the bank-conflict counter read 47 % of the
  // LDS cycles (2,045 x 4,168 x 7,168: 80 -> 76 us).
  const uint32_t l0 = (uint32_t)(lr * 128 + ((lg ^ ((lr >> 1) & 7)) << 4));
  auto bfrag = [&](int j) { return SWIGLU ? (j < 4 ? 4 * wn + j : 8 + 4 * wn + j - 4) : 8 * wn + j; };

  // One block of 128: NL live token fragments, and with COPY the copies of stage kt + S - 1 spread
  // over the MFMAs (with two stages they are issued at once instead, so that they have the
  // whole step to land: 4 experts x 4,096 rows 762 -> 743 us).  The multiply-adds of an MFMA's result follow LAG MFMAs later, past the matrix
  // pipe's latency.  Both are compile-time choices: a branch inside the step would let the
  // compiler sink every multiply-add to the step's end, with all partial sums live.
  constexpr int LAG = 3;
  auto step = [&](int kt, auto nl, auto copy) __attribute__((always_inline)) {
    constexpr int NL = decltype(nl)::value;
    constexpr bool COPY = decltype(copy)::value;
    constexpr int NM = 8 * NL;                   // MFMAs per block
    if constexpr (NL == 0) {
      if constexpr (COPY) {
#pragma unroll
        for (int c = 0; c < L; ++c) issue_one(kt + S - 1, c);
      }
    } else {
      // Four per-lane addresses per stage (both chunks of the token and of the weight fragments); everything
      // else is a constant offset.  They pass through an empty asm so that the compiler does not
      // keep one address per fragment and stage live across the loop, which spills.
      const uint32_t st = (uint32_t)(kt % S) * SL::SIZE;
      uint32_t pa = st + SL::A + wm * 2048 + l0, pb = st + SL::B + wn * (SWIGLU ? 8192 : 16384) + l0;
      uint32_t pa1 = st + SL::A + wm * 2048 + (l0 ^ 64), pb1 = st + SL::B + wn * (SWIGLU ? 8192 : 16384) + (l0 ^ 64);
      uint32_t ps = st + SL::SC + (16 * wm + lr) * 4;
      asm volatile("" : "+v"(pa), "+v"(pb), "+v"(pa1), "+v"(pb1), "+v"(ps));
      auto atile = [&](int i) __attribute__((always_inline)) {
        return fp8_join(*(const u32x4*)(lds + pa + i * 8192), *(const u32x4*)(lds + pa1 + i * 8192));
      };
      auto btile = [&](int j) __attribute__((always_inline)) {   // fragment bfrag(j)
        const int q = SWIGLU && j >= 4 ? j + 4 : j;
        return fp8_join(*(const u32x4*)(lds + pb + q * 2048), *(const u32x4*)(lds + pb1 + q * 2048));
      };
      if constexpr (ADD) {
        i32x8 af[NL], bq[2];
        bq[0] = btile(0);
#pragma unroll
        for (int i = 0; i < NL; ++i) af[i] = atile(i);
        auto half = [](const i32x8& v, int h) __attribute__((always_inline)) {
          return __builtin_bit_cast(bf16x8, h ? __builtin_shufflevector(v, v, 4, 5, 6, 7) : __builtin_shufflevector(v, v, 0, 1, 2, 3));
        };
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          if (j + 1 < 8) bq[(j + 1) & 1] = btile(j + 1);
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < NL; ++i) {
              const int m = (j * 2 + h) * NL + i;
              acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(half(bq[j & 1], h), half(af[i], h), acc[i][j], 0, 0, 0);
              if constexpr (COPY) {
#pragma unroll
                for (int c = 0; c < L; ++c)
                  if ((S == 2 ? (c < 2 * NM ? c : 2 * NM - 1) : c * 2 * NM / L) == m) issue_one(kt + S - 1, c);
              }
              __builtin_amdgcn_sched_barrier(0);
            }
        }
        return;
      }
      const float* sc = (const float*)(lds + st + SL::SC);
      i32x8 af[NL], bq[2];
      float t[NL][2];
      bq[0] = btile(0);
#pragma unroll
      for (int i = 0; i < NL; ++i) af[i] = atile(i);
      const float sw0 = SWIGLU ? sc[64 * FM] : sc[64 * FM + wn], sw1 = SWIGLU ? sc[64 * FM + 64] : sw0;
#pragma unroll
      for (int i = 0; i < NL; ++i) {
        const float sa = *(const float*)(lds + ps + i * 256);
        t[i][0] = sa * sw0;
        t[i][1] = SWIGLU ? sa * sw1 : t[i][0];
      }
      f32x4 part[LAG + 1];
      auto add = [&](int m) __attribute__((always_inline)) {
        const int j = m / NL, i = m % NL;
        const float s = t[i][j >> 2];
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[i][j][r] = fmaf(part[m % (LAG + 1)][r], s, acc[i][j][r]);
      };
      Wide16 aw[WIDE ? NL : 1];
      if constexpr (WIDE) {
#pragma unroll
        for (int i = 0; i < NL; ++i) aw[i] = fp8_widen(af[i]);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (j + 1 < 8) bq[(j + 1) & 1] = btile(j + 1);
        Wide16 bw;
        if constexpr (WIDE) bw = fp8_widen(bq[j & 1]);
#pragma unroll
        for (int i = 0; i < NL; ++i) {
          const int m = j * NL + i;
          if constexpr (WIDE) part[m % (LAG + 1)] = fp8_wide16(bw, aw[i]);
          else part[m % (LAG + 1)] = fp8_mfma16(bq[j & 1], af[i]);
          if constexpr (COPY) {
#pragma unroll
            for (int c = 0; c < L; ++c)
              if ((S == 2 ? (c < NM ? c : NM - 1) : c * NM / L) == m) issue_one(kt + S - 1, c);
          }
          if (m >= LAG) add(m - LAG);
          __builtin_amdgcn_sched_barrier(0);
        }
      }
#pragma unroll
      for (int m = NM - LAG; m < NM; ++m) add(m);
    }
  };
  auto kloop = [&](auto nl) __attribute__((always_inline)) {
    const int copied = max(KT - (S - 1), 0);
    for (int kt = 0; kt < copied; ++kt) {
      wait_vm<(S - 2) * L>();
      __syncthreads();
      step(kt, nl, std::true_type{});
    }
    for (int kt = copied; kt < KT; ++kt) {
      wait_stage(KT - 1 - kt);
      __syncthreads();
      step(kt, nl, std::false_type{});
    }
  };
  for (int s = 0; s < S - 1 && s < KT; ++s)
#pragma unroll
    for (int c = 0; c < L; ++c) issue_one(s, c);
  // live token fragments of this wavefront: rows 16 (wm + 4 i) below `rows`
  const int nlive = rows > 16 * wm ? min(FM, (rows - 16 * wm + 63) / 64) : 0;
  if (nlive >= FM) kloop(std::integral_constant<int, FM>{});
  else if (FM > 3 && nlive == 3) kloop(std::integral_constant<int, (FM > 3 ? 3 : 0)>{});
  else if (FM > 2 && nlive == 2) kloop(std::integral_constant<int, (FM > 2 ? 2 : 0)>{});
  else if (FM > 1 && nlive == 1) kloop(std::integral_constant<int, (FM > 1 ? 1 : 0)>{});
  else kloop(std::integral_constant<int, 0>{});
  __syncthreads();

  // ---------------------------------------------------------------- epilogue
  // acc[i][j][r]: token row 16 (wm + 4 i) + lr, weight row 16 bfrag(j) + 4 lg + r of the tile.  Output planes
  // are staged row-major in the idle stage ring (rows padded by 16 bytes) and written as 16-byte pieces.
  auto slot_of = [&](int m) { return ring_slot(p.head, seg, row0 + m, p.C); };
  auto flush = [&](uint8_t* dst, int64_t pitch, int col0b, int rowb, int rs) __attribute__((always_inline)) {
    __syncthreads();
    const int cpr = (rs - 16) / 16;
    for (int q = tid; q < BM * cpr; q += 512) {
      const int m = q / cpr, cb = (q % cpr) * 16;
      if (m < rows && col0b + cb < rowb)
        __builtin_nontemporal_store(*(const u32x4*)(lds + m * rs + cb), (u32x4*)(dst + slot_of(m) * pitch + col0b + cb));
    }
    __syncthreads();
  };
  if constexpr (SWIGLU) {
    if constexpr (KIND == FP8_SWIGLU_SAVE) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const f32x4 v = acc[i][4 * h + j];
            *(u32x2*)(lds + (16 * (wm + 4 * i) + lr) * 272 + (64 * wn + 16 * j + 4 * lg) * 2) =
                u32x2{pack_bf2(v[0], v[1]), pack_bf2(v[2], v[3])};
          }
        flush((uint8_t*)p.saved_au + (int64_t)h * p.N * 2, (int64_t)p.N * 4, n0 * 2, p.N * 2, 272);
      }
    }
    // h = silu(a) u in place of a; the row's maximum over 128 columns: 16 values here, four lanes (lg), two
    // wavefronts (wn, through LDS)
    float* hmax = (float*)lds;                   // [2][BM]
    float am[FM];
#pragma unroll
    for (int i = 0; i < FM; ++i) {
      am[i] = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          acc[i][j][r] = silu(acc[i][j][r]) * acc[i][4 + j][r];
          am[i] = amax2(am[i], acc[i][j][r]);
        }
      am[i] = amax2(am[i], __shfl_xor(am[i], 16, 64));
      am[i] = amax2(am[i], __shfl_xor(am[i], 32, 64));
      if (lg == 0) hmax[wn * BM + 16 * (wm + 4 * i) + lr] = am[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < FM; ++i) am[i] = amax2(am[i], hmax[(wn ^ 1) * BM + 16 * (wm + 4 * i) + lr]);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < FM; ++i) {
      const int m = 16 * (wm + 4 * i) + lr;
      const float s = fp8_scale(am[i]);
      if (wn == 0 && lg == 0 && m < rows) p.out_scale[(int64_t)ct * p.C + slot_of(m)] = s;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        *(uint32_t*)(lds + m * 144 + 64 * wn + 16 * j + 4 * lg) =
            h_encode4(acc[i][j][0], acc[i][j][1], acc[i][j][2], acc[i][j][3], s);
    }
    flush((uint8_t*)p.out, p.N, n0, p.N, 144);
  } else if constexpr (ADD) {
    // fp32 halves of 128 columns through LDS (rows of 512 + 16 bytes), so that the addend is read and the
    // sum written in whole 16-byte pieces; a half's addend is requested before its sums are staged
    constexpr int PC = BM * 16 / 512;            // pieces per thread and half
    u32x4 w[2][PC];
    auto place = [&](int h, int q, int& m, int& col) __attribute__((always_inline)) {
      m = (tid + 512 * q) / 16;
      col = n0 + 128 * h + (tid % 16) * 8;
      return m < rows && col < p.N;
    };
    auto request = [&](int h) __attribute__((always_inline)) {
#pragma unroll
      for (int q = 0; q < PC; ++q) {
        int m, col;
        w[h][q] = u32x4{0, 0, 0, 0};
        if (place(h, q, m, col) && p.add) w[h][q] = *(const u32x4*)(p.add + slot_of(m) * p.N + col);
      }
    };
    request(0);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (wn == h) {
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
          for (int j = 0; j < 8; ++j) *(f32x4*)(lds + (16 * (wm + 4 * i) + lr) * 528 + (16 * j + 4 * lg) * 4) = acc[i][j];
      }
      if (h == 0) request(1);
      __syncthreads();
#pragma unroll
      for (int q = 0; q < PC; ++q) {
        int m, col;
        if (!place(h, q, m, col)) continue;
        const f32x4 a = *(const f32x4*)(lds + m * 528 + (tid % 16) * 32), b = *(const f32x4*)(lds + m * 528 + (tid % 16) * 32 + 16);
        const u32x4 v = w[h][q];
        __builtin_nontemporal_store(
            u32x4{pack_bf2(lo_bf(v[0]) + a[0], hi_bf(v[0]) + a[1]), pack_bf2(lo_bf(v[1]) + a[2], hi_bf(v[1]) + a[3]),
                  pack_bf2(lo_bf(v[2]) + b[0], hi_bf(v[2]) + b[1]), pack_bf2(lo_bf(v[3]) + b[2], hi_bf(v[3]) + b[3])},
            (u32x4*)((bf16_t*)p.out + slot_of(m) * p.N + col));
      }
      __syncthreads();
    }
  } else if constexpr (KIND == FP8_F32 || KIND == FP8_PART) {
    const bool whole = (p.N & 3) == 0 && ((uintptr_t)p.out & 15) == 0;
#pragma unroll
    for (int i = 0; i < FM; ++i) {
      const int m = 16 * (wm + 4 * i) + lr;
      if (m >= rows) continue;
      float* row = (float*)p.out + (z * p.C + slot_of(m)) * p.N;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int col = n0 + 16 * bfrag(j) + 4 * lg;
        if (whole) {
          if (col < p.N) *(f32x4*)(row + col) = acc[i][j];
        } else {
#pragma unroll
          for (int r = 0; r < 4; ++r)
            if (col + r < p.N) row[col + r] = acc[i][j][r];
        }
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const f32x4 v = acc[i][j];
        *(u32x2*)(lds + (16 * (wm + 4 * i) + lr) * 528 + (16 * bfrag(j) + 4 * lg) * 2) =
            u32x2{pack_bf2(v[0], v[1]), pack_bf2(v[2], v[3])};
      }
    if ((p.N & 7) == 0 && ((uintptr_t)p.out & 15) == 0) {
      flush((uint8_t*)p.out, (int64_t)p.N * 2, n0 * 2, p.N * 2, 528);
    } else {                                     // rows that 16-byte pieces do not fit
      __syncthreads();
      for (int q = tid; q < BM * 256; q += 512) {
        const int m = q / 256, c = q % 256;
        if (m < rows && n0 + c < p.N)
          ((bf16_t*)p.out)[slot_of(m) * p.N + n0 + c] = *(const bf16_t*)(lds + m * 528 + 2 * c);
      }
    }
  }
}

template <int FM, int KIND, int S, bool NT>
__global__ __launch_bounds__(512) void fp8_tile_kernel(Fp8Args p) {
  fp8_tile_body<FM, KIND, S, NT>(p, (int)blockIdx.x);
}

template <int FM, int KIND, int S>
constexpr int fp8_tile_lds() {
  constexpr int BM = 64 * FM;
  constexpr int epi = KIND == FP8_BF16 || KIND == TILE_ADD ? BM * 528 : KIND == FP8_SWIGLU_SAVE ? BM * 272 : KIND == FP8_SWIGLU ? BM * 144 : 0;
  constexpr int ring = S * Fp8Stage<FM, KIND>::SIZE;
  return ring > epi ? ring : epi;
}

template <int FM, int KIND, int S, bool NT>
inline hipError_t run_fp8_tile(const Fp8Args& a, int64_t max_tiles, hipStream_t st) {
  const int nblk = (a.N + 127) / 128, nct = KIND >= FP8_SWIGLU ? nblk : (nblk + 1) / 2;
  constexpr int lds = fp8_tile_lds<FM, KIND, S>();
  static_assert(lds <= 160 * 1024, "LDS");
  auto kern = fp8_tile_kernel<FM, KIND, S, NT>;
  hipError_t err = hipFuncSetAttribute((const void*)kern, hipFuncAttributeMaxDynamicSharedMemorySize, lds);
  if (err != hipSuccess) return err;
  const int64_t grid = 8 * ((max_tiles * nct * a.Z + 7) / 8);
  kern<<<(unsigned)grid, 512, lds, st>>>(a);
  return hipGetLastError();
}

}  // namespace moe
