// ffn_launch.hip -- the kernels of the feed-forward products: launch_product
// of ffn_host.hpp for the pairs of IGC_FFN_KINDS, and launch_back for both
// types.  The build compiles this file once for each with -DIGC_FFN_UNIT=<n>.
#include "ffn_host.hpp"

namespace igc_ffn_host {

template <bool BF, int MODE, int MB, bool ODD>
void launch_skinny(const igc_ffn::GemmArgs& a, const Plan& pl, hipStream_t stream) {
  if (pl.variant == P_SKINNY_32)
    hipLaunchKernelGGL((igc_ffn::gemm_skinny_kernel<BF, MODE, MB, 2, 8, ODD>), dim3((unsigned)pl.tiles_n), dim3(512), 0, stream, a);
  else if constexpr (MODE == igc_ffn::M_FWD)
    hipLaunchKernelGGL((igc_ffn::gemm_skinny_kernel<BF, MODE, MB, 1, 16, ODD>), dim3((unsigned)pl.tiles_n), dim3(1024), 0, stream, a);
}
template <bool BF, int MODE, int MB>
void launch_skinny(const igc_ffn::GemmArgs& a, const Plan& pl, hipStream_t stream) {
  if (a.odd_rows)
    launch_skinny<BF, MODE, MB, true>(a, pl, stream);
  else
    launch_skinny<BF, MODE, MB, false>(a, pl, stream);
}

inline dim3 join_grid(const Plan& pl, int bm) {
  return dim3((unsigned)(((long long)pl.tiles_m * pl.tiles_n - pl.whole) * igc_ffn::join_waves(bm)));
}

template <bool BF, int MODE>
int launch_product(const igc_ffn::GemmArgs& a, const Plan& pl, hipStream_t stream) {
  const long long grid = workgroups(pl);
  if (grid == 0) return IGC_OK;
  if (grid > 0x7fffffffLL) return fail(IGC_EUNSUPPORTED, "too many tiles (%lld)", grid);
  constexpr int BN64 = MODE == igc_ffn::M_GLU ? 128 : 64;
  if constexpr (MODE == igc_ffn::M_FWD || MODE == igc_ffn::M_GLU) {
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
  const dim3 g((unsigned)grid), t(256);
  const dim3 tj(64);
#define IGC_FFN_TILE(kernel, BM, BN, ...)                                                                       \
  do {                                                                                                          \
    hipLaunchKernelGGL((igc_ffn::kernel<BF, MODE, BM, BN, ##__VA_ARGS__>), g, t, 0, stream, a);                  \
    if (pl.splits > 1)                                                                                          \
      hipLaunchKernelGGL((igc_ffn::gemm_join_kernel<BF, MODE, BM, BN>), join_grid(pl, BM), tj, 0, stream, a);    \
  } while (0)
  switch (pl.variant) {
    case P_TILE_256: IGC_FFN_TILE(gemm_tile_kernel, 256, 256, 2); break;
    case P_TILE_128: IGC_FFN_TILE(gemm_tile_kernel, 128, 128, 2); break;
    case P_TILE_64: IGC_FFN_TILE(gemm_tile_kernel, 64, BN64, 4); break;
    case P_TILE_32:
      if constexpr (MODE == igc_ffn::M_GLU)
        IGC_FFN_TILE(gemm_tile_kernel, 64, 64, 4);
      else if constexpr (MODE != igc_ffn::M_DW)
        IGC_FFN_TILE(gemm_tile_kernel, 64, 32, 6);
      break;
    case P_ANY_128: IGC_FFN_TILE(gemm_any_kernel, 128, 128); break;
    case P_ANY_64: IGC_FFN_TILE(gemm_any_kernel, 64, BN64); break;
    default: return fail(IGC_EUNSUPPORTED, "internal: no kernel for variant %d", pl.variant);
  }
#undef IGC_FFN_TILE
  return launch_status();
}

template <bool BF>
int launch_back(const igc_ffn::GemmArgs& x, const Plan& px, const igc_ffn::GemmArgs& w, const Plan& pw, const igc_ffn::ColsumArgs& s,
                hipStream_t stream) {
  const long long nx = workgroups(px), nw = workgroups(pw);
  // K tiles of the longest workgroup of each
  const long long kx = k_tiles(x.R) / (px.whole ? 1 : px.splits), kw = k_tiles(w.R) / (pw.whole ? 1 : pw.splits);
  const bool x_first = kx >= kw;
  const long long first = x_first ? nx : nw, second = x_first ? nw : nx;
  const long long grid = ceil_div(first, 8) * 8 + second + colsum_groups(s);
  if (grid > 0x7fffffffLL) return fail(IGC_EUNSUPPORTED, "too many tiles (%lld)", grid);
  const dim3 g((unsigned)grid), t(256), tj(64);
#define IGC_FFN_BACK(BM, BN, DEPTH)                                                                                            \
  do {                                                                                                                         \
    hipLaunchKernelGGL((igc_ffn::gemm_back_kernel<BF, BM, BN, DEPTH>), g, t, 0, stream, x, w, s, (int)x_first, (int)first, (int)second); \
    if (px.splits > 1)                                                                                                         \
      hipLaunchKernelGGL((igc_ffn::gemm_join_kernel<BF, igc_ffn::M_DX, BM, BN>), join_grid(px, BM), tj, 0, stream, x);         \
    if (pw.splits > 1)                                                                                                         \
      hipLaunchKernelGGL((igc_ffn::gemm_join_kernel<BF, igc_ffn::M_DW, BM, BN>), join_grid(pw, BM), tj, 0, stream, w);         \
  } while (0)
  switch (px.variant) {
    case P_TILE_256: IGC_FFN_BACK(256, 256, 2); break;
    case P_TILE_128: IGC_FFN_BACK(128, 128, 2); break;
    case P_TILE_64: IGC_FFN_BACK(64, 64, 4); break;
    default: return fail(IGC_EUNSUPPORTED, "internal: no joint kernel for variant %d", px.variant);
  }
#undef IGC_FFN_BACK
  return launch_status();
}
#define IGC_FFN_DEFINE_BACK(BF)                                                                                       \
  template int launch_back<BF>(const igc_ffn::GemmArgs&, const Plan&, const igc_ffn::GemmArgs&, const Plan&,          \
                               const igc_ffn::ColsumArgs&, hipStream_t);

#define IGC_FFN_DEFINE(BF, MODE) template int launch_product<BF, MODE>(const igc_ffn::GemmArgs&, const Plan&, hipStream_t);
#if IGC_FFN_UNIT == 0
IGC_FFN_DEFINE(false, igc_ffn::M_FWD)
#elif IGC_FFN_UNIT == 1
IGC_FFN_DEFINE(true, igc_ffn::M_FWD)
#elif IGC_FFN_UNIT == 2
IGC_FFN_DEFINE(false, igc_ffn::M_GLU)
#elif IGC_FFN_UNIT == 3
IGC_FFN_DEFINE(true, igc_ffn::M_GLU)
#elif IGC_FFN_UNIT == 4
IGC_FFN_DEFINE(false, igc_ffn::M_DX)
#elif IGC_FFN_UNIT == 5
IGC_FFN_DEFINE(true, igc_ffn::M_DX)
#elif IGC_FFN_UNIT == 6
IGC_FFN_DEFINE(false, igc_ffn::M_DW)
#elif IGC_FFN_UNIT == 7
IGC_FFN_DEFINE(true, igc_ffn::M_DW)
#elif IGC_FFN_UNIT == 8
IGC_FFN_DEFINE_BACK(false)
#elif IGC_FFN_UNIT == 9
IGC_FFN_DEFINE_BACK(true)
#else
#error "IGC_FFN_UNIT: 0 .. 9"
#endif

}  // namespace igc_ffn_host
