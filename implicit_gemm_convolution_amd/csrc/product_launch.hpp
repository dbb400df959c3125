// product_launch.hpp -- launch_product of ffn_host.hpp: a planned product's
// kernels on the caller's stream.  Instantiated once per type and operand layout
// (ffn_launch.hip, i8_launch.hip).
#pragma once

#include "ffn_host.hpp"

namespace igc_ffn_host {

template <bool BF, int MODE, int MB, int NB, int NW>
void launch_skinny(const igc_ffn::Args<MODE>& a, const Plan& pl, hipStream_t stream) {
  const dim3 g((unsigned)pl.tiles_n), t(64 * NW);
  if constexpr (igc_ffn::is_i8(MODE)) {
    if (a.odd_rows)
      hipLaunchKernelGGL((igc_ffn::i8_skinny_kernel<BF, MODE, MB, NB, NW, true>), g, t, 0, stream, a);
    else
      hipLaunchKernelGGL((igc_ffn::i8_skinny_kernel<BF, MODE, MB, NB, NW, false>), g, t, 0, stream, a);
  } else {
    if (a.odd_rows)
      hipLaunchKernelGGL((igc_ffn::gemm_skinny_kernel<BF, MODE, MB, NB, NW, true>), g, t, 0, stream, a);
    else
      hipLaunchKernelGGL((igc_ffn::gemm_skinny_kernel<BF, MODE, MB, NB, NW, false>), g, t, 0, stream, a);
  }
}
template <bool BF, int MODE, int MB>
void launch_skinny(const igc_ffn::Args<MODE>& a, const Plan& pl, hipStream_t stream) {
  if (pl.variant == P_SKINNY_32)
    launch_skinny<BF, MODE, MB, 2, 8>(a, pl, stream);
  else if constexpr (igc_ffn::is_fwd(MODE))
    launch_skinny<BF, MODE, MB, 1, 16>(a, pl, stream);
}

inline dim3 join_grid(const Plan& pl, int bm) {
  return dim3((unsigned)(((long long)pl.tiles_m * pl.tiles_n - pl.whole) * igc_ffn::join_waves(bm)));
}

template <bool BF, int MODE, int BM, int BN, int DEPTH>
void launch_tile(const igc_ffn::Args<MODE>& a, const Plan& pl, dim3 g, hipStream_t stream) {
  if constexpr (igc_ffn::is_i8(MODE)) {
    hipLaunchKernelGGL((igc_ffn::i8_tile_kernel<BF, MODE, BM, BN, DEPTH>), g, dim3(256), 0, stream, a);
    if (pl.splits > 1) hipLaunchKernelGGL((igc_ffn::i8_join_kernel<BF, MODE, BM, BN>), join_grid(pl, BM), dim3(64), 0, stream, a);
  } else {
    hipLaunchKernelGGL((igc_ffn::gemm_tile_kernel<BF, MODE, BM, BN, DEPTH>), g, dim3(256), 0, stream, a);
    if (pl.splits > 1) hipLaunchKernelGGL((igc_ffn::gemm_join_kernel<BF, MODE, BM, BN>), join_grid(pl, BM), dim3(64), 0, stream, a);
  }
}

template <bool BF, int MODE, int BM, int BN>
void launch_any(const igc_ffn::GemmArgs& a, const Plan& pl, dim3 g, hipStream_t stream) {
  hipLaunchKernelGGL((igc_ffn::gemm_any_kernel<BF, MODE, BM, BN>), g, dim3(256), 0, stream, a);
  if (pl.splits > 1) hipLaunchKernelGGL((igc_ffn::gemm_join_kernel<BF, MODE, BM, BN>), join_grid(pl, BM), dim3(64), 0, stream, a);
}

template <bool BF, int MODE>
int launch_product(const igc_ffn::GemmArgs& args, const Plan& pl, hipStream_t stream) {
  const long long grid = workgroups(pl);
  if (grid == 0) return IGC_OK;
  if (grid > 0x7fffffffLL) return fail(IGC_EUNSUPPORTED, "too many tiles (%lld)", grid);
  const auto& a = static_cast<const igc_ffn::Args<MODE>&>(args);
  constexpr int BN64 = igc_ffn::is_glu(MODE) ? 128 : 64;
  if constexpr (igc_ffn::is_fwd(MODE) || igc_ffn::is_glu(MODE)) {
    if (pl.variant == P_SKINNY_16 || pl.variant == P_SKINNY_32) {
      if (a.M <= 16)
        launch_skinny<BF, MODE, 1>(a, pl, stream);
      else if (a.M <= 32)
        launch_skinny<BF, MODE, 2>(a, pl, stream);
      else
        launch_skinny<BF, MODE, 4>(a, pl, stream);
      return launch_status();
    }
  }
  const dim3 g((unsigned)grid);
  switch (pl.variant) {
    case P_TILE_256: launch_tile<BF, MODE, 256, 256, 2>(a, pl, g, stream); return launch_status();
    case P_TILE_128: launch_tile<BF, MODE, 128, 128, 2>(a, pl, g, stream); return launch_status();
    case P_TILE_64: launch_tile<BF, MODE, 64, BN64, 4>(a, pl, g, stream); return launch_status();
    case P_TILE_32:
      if constexpr (igc_ffn::is_glu(MODE))
        launch_tile<BF, MODE, 64, 64, 4>(a, pl, g, stream);
      else if constexpr (MODE != igc_ffn::M_DW)
        launch_tile<BF, MODE, 64, 32, 6>(a, pl, g, stream);
      return launch_status();
    default: break;
  }
  if constexpr (igc_ffn::is_i8(MODE)) {
    if (pl.variant == P_BYTES) {
      hipLaunchKernelGGL((igc_ffn::i8_any_kernel<BF, MODE, 4>), g, dim3(256), 0, stream, a);
      return launch_status();
    }
  } else {
    if (pl.variant == P_ANY_128) {
      launch_any<BF, MODE, 128, 128>(a, pl, g, stream);
      return launch_status();
    }
    if (pl.variant == P_ANY_64) {
      launch_any<BF, MODE, 64, BN64>(a, pl, g, stream);
      return launch_status();
    }
  }
  return fail(IGC_EUNSUPPORTED, "internal: no kernel for variant %d", pl.variant);
}

}  // namespace igc_ffn_host
