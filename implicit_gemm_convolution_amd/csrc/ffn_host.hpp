// ffn_host.hpp -- host side of the feed-forward products: the launch plan
// (tile, split, workspace bytes) and the launch on the caller's stream.
// launch_product<BF, MODE> is instantiated in ffn_launch.hip, once per type
// and operand layout, so that they compile in parallel; ffn.hip plans and
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
constexpr int kSkinnyRows = 64;

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
// workspace.
inline Plan make_plan(int mode, long long M, long long N, long long R, bool aligned, int cus, bool may_split) {
  Plan pl;
  if ((mode == igc_ffn::M_FWD || mode == igc_ffn::M_GLU) && M <= kSkinnyRows) {
    // 32 weight rows share the loads of X; 16 where there would be too few workgroups
    pl.variant = mode == igc_ffn::M_GLU || N >= 32LL * cus ? P_SKINNY_32 : P_SKINNY_16;
    pl.tiles_m = 1;
    pl.tiles_n = (int)ceil_div(N, pl.variant == P_SKINNY_32 && mode == igc_ffn::M_FWD ? 32 : 16);
    return pl;
  }
  int bm, bn;
  plan_tile(mode, P_TILE_256, bm, bn);
  if (aligned && ceil_div(M, bm) * ceil_div(N, bn) >= cus * 3 / 4) {
    pl.variant = P_TILE_256;
  } else {
    plan_tile(mode, P_TILE_128, bm, bn);
    const bool large = ceil_div(M, bm) * ceil_div(N, bn) >= cus;
    pl.variant = aligned ? (large ? P_TILE_128 : P_TILE_64) : (large ? P_ANY_128 : P_ANY_64);
  }
  plan_tile(mode, pl.variant, bm, bn);
  pl.tiles_m = (int)ceil_div(M, bm);
  pl.tiles_n = (int)ceil_div(N, bn);
  const long long tiles = (long long)pl.tiles_m * pl.tiles_n;
  const long long nk = std::max(1LL, ceil_div(R, 64));
  if (may_split && tiles > 0 && tiles < cus) {
    pl.splits = (int)std::max(1LL, std::min(nk / 4, (long long)cus / tiles));
    if (pl.splits > 1) pl.part_bytes = (size_t)tiles * pl.splits * bm * bn * (mode == igc_ffn::M_GLU ? 8 : 4);
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

#define IGC_FFN_EXTERN(n, BF, MODE) \
  extern template int launch_product<BF, MODE>(const igc_ffn::GemmArgs&, const Plan&, hipStream_t);
IGC_FFN_KINDS(IGC_FFN_EXTERN)
#undef IGC_FFN_EXTERN

inline int launch_status() {
  const hipError_t e = hipGetLastError();
  return e == hipSuccess ? IGC_OK : fail(IGC_EHIP, "kernel launch failed: %s", hipGetErrorString(e));
}

}  // namespace igc_ffn_host
