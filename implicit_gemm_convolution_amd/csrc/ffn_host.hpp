// ffn_host.hpp -- host side of the feed-forward products: the launch plan
// (tile, split, workspace bytes) and the launch on the caller's stream.
// launch_product<BF, MODE> and launch_back<BF> are instantiated in
// ffn_launch.hip and i8_launch.hip, once per type and operand layout, so that they compile in parallel; ffn.hip
// and i8.hip plan and call them.
#pragma once

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstddef>
#include <cstdint>

#include "../../include/igc.h"
#include "ffn_kernels.hpp"

namespace igc_host {
// Defined in igc.hip: the thread's error detail, the current device's check
// and its compute units.
int fail(int status, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
int check_device(int* dev_out);
int device_cus(int dev);
}  // namespace igc_host

namespace igc_ffn_host {

using igc_host::fail;

inline long long ceil_div(long long a, long long b) { return (a + b - 1) / b; }

// The kernels of a product, by output tile (the gated block's tiles hold two
// products: half as many output columns).
// P_TILE_*: aligned operands, straight into LDS (P_TILE_32: 64 x 32); P_ANY_*: any operand,
// through registers; P_SKINNY_*: few rows, any operand, 16 or 32 weight rows
// per workgroup; P_BYTES: 8 bits, any operand, through registers.
enum Variant { P_TILE_256, P_TILE_128, P_TILE_64, P_TILE_32, P_ANY_128, P_ANY_64, P_SKINNY_16, P_SKINNY_32, P_BYTES };

struct Plan {
  int variant = P_ANY_64;
  int tiles_m = 0, tiles_n = 0;
  long long whole = 0;    // tiles [0, whole) have a workgroup each,
  int splits = 1;         // the others this many that share the reduction
  size_t part_bytes = 0;  // their partial tiles
  float us = 0;           // estimate
};

inline void plan_tile(int mode, int variant, int& bm, int& bn) {
  switch (variant) {
    case P_TILE_256: bm = 256; bn = mode == igc_ffn::M_GLU ? 128 : 256; return;
    case P_TILE_128:
    case P_ANY_128: bm = 128; bn = mode == igc_ffn::M_GLU ? 64 : 128; return;
    case P_TILE_32: bm = 64; bn = 32; return;
    default: bm = 64; bn = 64; return;
  }
}

// What every row of an operand starts at a multiple of, of 2, 4 and (as below)
// 16 bytes.
inline bool dma_operand(const void* p, long long ld, long long length);
inline int row_align(const void* p, long long ld, long long length) {
  return dma_operand(p, ld, length) ? 16 : (reinterpret_cast<uintptr_t>(p) & 3u) || (ld & 1) ? 2 : 4;
}

// Operands of the direct-to-LDS loaders: 16-byte aligned rows, lengths in
// whole 16-byte chunks (at least one), and a tile's worth of rows within a descriptor (256
// rows below 2^30 bytes).
inline bool dma_operand(const void* p, long long ld, long long length) {
  return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && ld % 8 == 0 && length > 0 && length % 8 == 0 && ld <= (1 << 21) - 8;
}

// What a launch of the aligned tiles takes, in us, fitted to timings on MI355X
// (bf16; 52 outputs of 16 x 4096 to 8192 x 8192 in the four layouts, reductions
// of 300 to 30000, one to sixteen splits; profiles/ has them).  Over 197 of
// those products, 2001 timings, the plan with the smallest estimate takes 1.2%
// longer than the fastest one in the mean and 18% at most (gated block 0.8%
// and 10%).  Tiles chosen by how many fill the card,
// split only below one per compute unit: 5%, and twice as long at
// 640 x 2432 x 27392.
//   k0, k1, k2  a K tile of 64 in an empty card; with one workgroup on every
//               compute unit (where there is one place: on half of them); with
//               every place taken
//   out         the prologue and the outputs of a workgroup
//   join        the second launch of a split reduction: itself, for each MB
//               of partial tiles, for each split
struct TileCost {
  float launch, k0, k1, k2, out, join, join_mb, join_split;
};
inline const TileCost& tile_cost(int mode, int variant) {
  static constexpr TileCost one[4] = {{2.1f, 0.77f, 1.02f, 1.35f, 11.8f, 0.0f, 0.17f, 0.0f},
                                      {2.4f, 0.35f, 0.51f, 0.91f, 2.3f, 2.1f, 0.15f, 0.32f},
                                      {2.8f, 0.18f, 0.23f, 0.37f, 1.0f, 1.4f, 0.31f, 0.40f},
                                      {2.8f, 0.11f, 0.14f, 0.18f, 1.0f, 1.4f, 0.31f, 0.40f}};
  static constexpr TileCost two[4] = {{2.6f, 0.96f, 1.07f, 1.40f, 10.2f, 0.0f, 0.20f, 0.0f},
                                      {3.8f, 0.33f, 0.53f, 0.94f, 1.5f, 2.4f, 0.11f, 0.43f},
                                      {3.0f, 0.19f, 0.24f, 0.30f, 2.3f, 1.2f, 0.64f, 0.0f},
                                      {3.0f, 0.13f, 0.19f, 0.47f, 1.0f, 1.2f, 0.64f, 0.0f}};
  return (mode == igc_ffn::M_GLU ? two : one)[variant];
}
// workgroups of a tile that share a compute unit (160 KB of LDS)
inline int tile_places(int mode, int variant) {
  const bool glu = mode == igc_ffn::M_GLU;
  return variant == P_TILE_256 || (variant == P_TILE_64 && glu) || (variant == P_TILE_32 && !glu) ? 1 : 2;
}
// `count` workgroups of n K tiles each
inline float rounds_us(const TileCost& c, int places, float n, long long count, int cus) {
  const long long cap = (long long)places * cus;
  auto round = [&](long long w) {
    const float f = 2.0f * (float)w / (float)cap;
    float k = c.k0 + (c.k1 - c.k0) * f;
    // (two to a compute unit: the first pair is half the way there)
    if (f > 1.0f) k = c.k1 + (c.k2 - c.k1) * (places == 1 ? f - 1.0f : 0.5f * f);
    return n * k + c.out * (f > 1.0f ? (float)places : 1.0f);
  };
  return (float)(count / cap) * round(cap) + (count % cap ? round(count % cap) : 0.0f);
}
inline float join_us(const TileCost& c, const Plan& pl) {
  return pl.splits > 1 ? c.join + c.join_mb * (float)pl.part_bytes * 1e-6f + c.join_split * (float)pl.splits : 0.0f;
}

inline long long workgroups(const Plan& pl) {
  return pl.whole + ((long long)pl.tiles_m * pl.tiles_n - pl.whole) * pl.splits;
}
inline Plan tile_plan(int mode, int variant, long long M, long long N, long long whole = 0, int splits = 1) {
  Plan pl;
  int bm, bn;
  plan_tile(mode, variant, bm, bn);
  pl.variant = variant;
  pl.tiles_m = (int)ceil_div(M, bm);
  pl.tiles_n = (int)ceil_div(N, bn);
  pl.whole = whole;
  pl.splits = splits;
  if (splits > 1) pl.part_bytes = (size_t)((long long)pl.tiles_m * pl.tiles_n - whole) * splits * bm * bn * (mode == igc_ffn::M_GLU ? 8 : 4);
  return pl;
}
inline long long k_tiles(long long R) { return std::max(1LL, ceil_div(R, 64)); }

// The best plan on one of the aligned tiles.  Where the last round of
// workgroups does not fill the card, its tiles may be split: into at most 16
// parts of at least four K tiles, and into no more workgroups than run at once.
inline Plan best_split(int mode, int variant, long long M, long long N, long long R, int cus, bool may_split) {
  const TileCost& c = tile_cost(mode, variant);
  const int places = tile_places(mode, variant);
  const long long cap = (long long)places * cus;
  const float nk = (float)k_tiles(R);
  Plan best = tile_plan(mode, variant, M, N);
  const long long tiles = (long long)best.tiles_m * best.tiles_n, whole = tiles / cap * cap;
  best.us = c.launch + rounds_us(c, places, nk, tiles, cus);
  for (int s = 2; may_split && s <= 16 && (float)s <= nk / 4 && (tiles - whole) * s <= cap; ++s) {
    Plan pl = tile_plan(mode, variant, M, N, whole, s);
    pl.us = c.launch + rounds_us(c, places, nk, whole, cus) + rounds_us(c, places, nk / (float)s, (tiles - whole) * s, cus) + join_us(c, pl);
    if (pl.us + (best.splits == 1 ? 1.0f : 0.0f) < best.us) best = pl;  // (to gain 1 us at least)
  }
  return best;
}

// The plan on one of the tiles for any operands, whose K loop waits for its
// loads: so many us for a K tile, or for each K tile of each workgroup where
// there are many.  (bf16, 128 x 128 | 64 x 64, rows of odd length:
// 136 x 4000 x 2001 42 | 27 us, 2000 x 2000 x 2001 46 | 50,
// 6900 x 2600 x 2201 156 | 203.)  A second launch and the partial tiles'
// traffic cost about 20 K tiles' time.
inline Plan any_plan(int mode, int variant, long long M, long long N, long long R, int cus, bool may_split) {
  Plan pl = tile_plan(mode, variant, M, N);
  const long long count = (long long)pl.tiles_m * pl.tiles_n, nk = k_tiles(R);
  const bool large = variant == P_ANY_128, glu = mode == igc_ffn::M_GLU;
  const float alone = large ? (glu ? 1.25f : 1.2f) : (glu ? 1.0f : 0.75f);
  const float each = large ? (glu ? 3.2e-3f : 3.6e-3f) : (glu ? 2.2e-3f : 1.45e-3f);
  if (may_split && count > 0) {
    const long long s = std::min(nk / 8, (long long)cus / count);
    if (s > 1 && nk - nk / s > 24) pl = tile_plan(mode, variant, M, N, 0, (int)s);
  }
  pl.us = 3.0f + (float)nk / (float)pl.splits * std::max(alone, each * (float)(count * pl.splits)) + (pl.splits > 1 ? 4.0f : 0.0f);
  return pl;
}

// The plan on one of the kernels for few rows (at most 64): every wave loads
// its part of the reduction in batches, so the time goes with the reduction's
// length and, more weakly, with the rows that share it; rows at odd multiples
// of 2 bytes take two loads for one.  bf16, us, 16 | 32 weight rows | 64-row
// tiles: 1x4096x4096 8.5 | 11.4 | 11.0, 16x11008x4096 28 | 30 | 18,
// 32x512x512 4.3 | 6.2 | 5.3, 32x16384x1024 16 | 11 | 8; the gated block at
// 1x11008x4096 - | 37 | 40, 16x11008x4096 - | 46 | 41, 16x2048x1024 - | 5.7 |
// 7.8.  Odd rows, and the tiles for any rows: 1x4096x4097 11 | 19 | 22,
// 32x2048x1025 6.7 | 8.0 | 11, 16x2048x8193 26 | 35 | 22.
inline Plan skinny_plan(int mode, int variant, long long M, long long N, long long R, int align, int cus) {
  Plan pl;
  const bool two = variant == P_SKINNY_32, glu = mode == igc_ffn::M_GLU, odd = align < 4;
  pl.variant = variant;
  pl.tiles_m = 1;
  pl.tiles_n = (int)ceil_div(N, two && !glu ? 32 : 16);
  const float per_k = ((two ? 1.8f : 0.9f) + 0.05f * (float)M) * (!odd ? 1.0f : glu ? 1.75f : 1.5f);  // us per 1024 of the reduction
  const float rounds = (float)pl.tiles_n / (float)cus;
  const float fill = odd ? 1.45f * rounds : rounds * (!two ? 1.3f : glu ? 1.45f : 1.5f) - (two ? 0.0f : 0.15f);
  const float each = two ? 0.0f : 0.5f;  // joining sixteen waves' sums instead of eight
  const float run = (per_k * (float)R / 1024.0f + each) * std::max(1.0f, fill) - each;
  const float weights = (float)N * (float)R * (glu ? 4.0f : 2.0f) / (odd ? 3.0e6f : 5.2e6f);
  pl.us = 3.6f + std::max(run, weights + 0.05f * run);
  return pl;
}

// A pure function of the problem and the device, so that the size queries and
// the calls agree.  align: the bytes (2, 4 or 16) that every row of the
// operands starts at a multiple of; may_split: the call has (or the query
// assumes) a workspace.
inline Plan make_plan(int mode, long long M, long long N, long long R, int align, int cus, bool may_split) {
  Plan pl;
  auto take = [&](const Plan& q) {
    if (pl.tiles_m == 0 || q.us < pl.us) pl = q;
  };
  if ((mode == igc_ffn::M_FWD || mode == igc_ffn::M_GLU) && M <= 64) {
    if (mode == igc_ffn::M_FWD) take(skinny_plan(mode, P_SKINNY_16, M, N, R, align, cus));
    take(skinny_plan(mode, P_SKINNY_32, M, N, R, align, cus));
  }
  if (align == 16) {
    // (streaming the operands, no faster than 5 TB/s)
    const float least = 4.5f + ((float)M + (float)N * (mode == igc_ffn::M_GLU ? 2.0f : 1.0f)) * (float)R * 2.0f / 5e6f;
    for (int v = P_TILE_256; v <= (mode == igc_ffn::M_DW ? P_TILE_64 : P_TILE_32); ++v) {
      Plan q = best_split(mode, v, M, N, R, cus, may_split);
      if (M <= 64) q.us = std::max(q.us, least + 0.05f * q.us);  // (the faster tile still comes first)
      take(q);
    }
    return pl;
  }
  for (int v = P_ANY_128; v <= P_ANY_64; ++v) take(any_plan(mode, v, M, N, R, cus, may_split));
  return pl;
}

// (8 bits: a is an I8Args)
template <bool BF, int MODE>
int launch_product(const igc_ffn::GemmArgs& a, const Plan& pl, hipStream_t stream);

#define IGC_FFN_KINDS(X)         \
  X(0, false, igc_ffn::M_FWD)    \
  X(1, true, igc_ffn::M_FWD)     \
  X(2, false, igc_ffn::M_GLU)    \
  X(3, true, igc_ffn::M_GLU)     \
  X(4, false, igc_ffn::M_DX)     \
  X(5, true, igc_ffn::M_DX)      \
  X(6, false, igc_ffn::M_DW)     \
  X(7, true, igc_ffn::M_DW)

// Products in 8 bits: the type of their outputs, the layout.
#define IGC_I8_KINDS(X)          \
  X(0, false, igc_ffn::M_I8)     \
  X(1, true, igc_ffn::M_I8)      \
  X(2, false, igc_ffn::M_I8_GLU) \
  X(3, true, igc_ffn::M_I8_GLU)

// Both backward products, planned on one tile size, and the column sums
// (s.which_n 0: none).
template <bool BF>
int launch_back(const igc_ffn::GemmArgs& x, const Plan& px, const igc_ffn::GemmArgs& w, const Plan& pw, const igc_ffn::ColsumArgs& s,
                hipStream_t stream);
extern template int launch_back<false>(const igc_ffn::GemmArgs&, const Plan&, const igc_ffn::GemmArgs&, const Plan&,
                                       const igc_ffn::ColsumArgs&, hipStream_t);
extern template int launch_back<true>(const igc_ffn::GemmArgs&, const Plan&, const igc_ffn::GemmArgs&, const Plan&,
                                      const igc_ffn::ColsumArgs&, hipStream_t);

#define IGC_FFN_EXTERN(n, BF, MODE) \
  extern template int launch_product<BF, MODE>(const igc_ffn::GemmArgs&, const Plan&, hipStream_t);
IGC_FFN_KINDS(IGC_FFN_EXTERN)
IGC_I8_KINDS(IGC_FFN_EXTERN)
#undef IGC_FFN_EXTERN

// workgroups of the column sums
inline long long colsum_groups(const igc_ffn::ColsumArgs& s) { return s.which_n * ceil_div(s.N, 64); }

inline int launch_status() {
  const hipError_t e = hipGetLastError();
  return e == hipSuccess ? IGC_OK : fail(IGC_EHIP, "kernel launch failed: %s", hipGetErrorString(e));
}

}  // namespace igc_ffn_host
