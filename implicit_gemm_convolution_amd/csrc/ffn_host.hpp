// ffn_host.hpp -- host side of the feed-forward products: the launch plan
// (tile, split, workspace bytes) and the launch on the caller's stream.
// launch_product<BF, MODE> and launch_back<BF> are instantiated in
// ffn_launch.hip, once per type and operand layout, so that they compile in parallel; ffn.hip plans and
// calls it.
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
// P_TILE_*: aligned operands, straight into LDS; P_ANY_*: any operand,
// through registers; P_SKINNY_*: few rows, any operand, 16 or 32 weight rows
// per workgroup.
enum Variant { P_TILE_256, P_TILE_128, P_TILE_64, P_ANY_128, P_ANY_64, P_SKINNY_16, P_SKINNY_32 };

struct Plan {
  int variant = P_ANY_64;
  int tiles_m = 0, tiles_n = 0;
  int splits = 1;
  size_t part_bytes = 0;  // partial tiles of a split reduction
};

inline void plan_tile(int mode, int variant, int& bm, int& bn) {
  switch (variant) {
    case P_TILE_256: bm = 256; bn = mode == igc_ffn::M_GLU ? 128 : 256; return;
    case P_TILE_128:
    case P_ANY_128: bm = 128; bn = mode == igc_ffn::M_GLU ? 64 : 128; return;
    default: bm = 64; bn = 64; return;
  }
}

// Operands of the direct-to-LDS loaders: 16-byte aligned rows, lengths in
// whole 16-byte chunks (at least one), and a tile's worth of rows within a descriptor (256
// rows below 2^30 bytes).
inline bool dma_operand(const void* p, long long ld, long long length) {
  return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && ld % 8 == 0 && length > 0 && length % 8 == 0 && ld <= (1 << 21) - 8;
}

// A pure function of the problem and the device, so that the size queries and
// the calls agree.  may_split: the call has (or the query assumes) a
// workspace.  Times below: bf16 on MI355X, N = K = 4096 unless said.
inline Plan make_plan(int mode, long long M, long long N, long long R, bool aligned, int cus, bool may_split) {
  Plan pl;
  int bm, bn;
  // Few rows: streaming the weights into registers beats 64-row tiles up to
  // 16 rows (12 rows 10.0 us against 11.9) and, on short reductions, up to 32
  // (24x2048x1024 5.1 against 6.3; 32 rows 14.0 against 12.3).  Rows of any
  // alignment have no better kernel up to 64.
  if ((mode == igc_ffn::M_FWD || mode == igc_ffn::M_GLU) && (M <= 16 || (M <= 32 && R <= 1024) || (M <= 64 && !aligned))) {
    // 32 weight rows share the loads of X; 16 where there would be too few workgroups
    pl.variant = mode == igc_ffn::M_GLU || N >= 32LL * cus ? P_SKINNY_32 : P_SKINNY_16;
    pl.tiles_m = 1;
    pl.tiles_n = (int)ceil_div(N, pl.variant == P_SKINNY_32 && mode == igc_ffn::M_FWD ? 32 : 16);
    return pl;
  }
  // The largest tile that fills the card: 256 x 256 from three quarters of
  // the compute units (M = 4096: 102 us against 118 on 128 x 128 tiles; at
  // half of them, M = 2048, 93 against 66), 128 x 128 likewise (M = 1024
  // 37 us against 53 on 64 x 64; M = 512 29.4 against 28.4).
  auto tiles = [&](int variant) {
    plan_tile(mode, variant, bm, bn);
    return ceil_div(M, bm) * ceil_div(N, bn);
  };
  if (aligned && 4 * tiles(P_TILE_256) >= 3 * cus)
    pl.variant = P_TILE_256;
  else if (4 * tiles(P_TILE_128) >= 3 * cus)
    pl.variant = aligned ? P_TILE_128 : P_ANY_128;
  else
    pl.variant = aligned ? P_TILE_64 : P_ANY_64;
  plan_tile(mode, pl.variant, bm, bn);
  pl.tiles_m = (int)ceil_div(M, bm);
  pl.tiles_n = (int)ceil_div(N, bn);
  const long long count = (long long)pl.tiles_m * pl.tiles_n;
  const long long nk = std::max(1LL, ceil_div(R, 64));
  // Splitting the reduction costs a second launch and the partial tiles'
  // traffic, about 20 K tiles' time: 64 tiles of 64 K tiles (M = 64) in four
  // splits 12.5 us against 15.4, 128 tiles (M = 128) in two 13.8 against
  // 16.0, but 64 tiles of 32 K tiles in two 11.8 against 9.7.
  if (may_split && count > 0) {
    const long long s = std::min(nk / 8, (long long)cus / count);
    if (s > 1 && nk - nk / s > 24) {
      pl.splits = (int)s;
      pl.part_bytes = (size_t)count * pl.splits * bm * bn * (mode == igc_ffn::M_GLU ? 8 : 4);
    }
  }
  return pl;
}

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
#undef IGC_FFN_EXTERN

// workgroups of the column sums
inline long long colsum_groups(const igc_ffn::ColsumArgs& s) { return s.which_n * ceil_div(s.N, 64); }

inline int launch_status() {
  const hipError_t e = hipGetLastError();
  return e == hipSuccess ? IGC_OK : fail(IGC_EHIP, "kernel launch failed: %s", hipGetErrorString(e));
}

}  // namespace igc_ffn_host
