// op_host.hpp -- what the C entries of the feed-forward operators and of the
// operators around them share: argument checks, workspace checks, and the
// arguments of a product.
#pragma once

#include <hip/hip_runtime.h>

#include <cstring>

#include "ffn_host.hpp"

namespace igc_ffn_host {

// ---------------------------------------------------------------- validation
struct Checker {
  int status = IGC_OK;
  bool ok() const { return status == IGC_OK; }
  void fail_if(bool bad, const char* what) {
    if (ok() && bad) status = fail(IGC_EINVAL, "%s", what);
  }
  // a matrix of rows x cols: NULL only where allowed, its leading dimension
  // at least a row, its address a multiple of the element size
  void matrix(const char* name, const void* p, int ld, long long rows, long long cols, int bytes, bool optional) {
    if (!ok() || (optional && !p)) return;
    if (rows > 0 && cols > 0 && !p) status = fail(IGC_EINVAL, "%s is NULL", name);
    else if (ld < cols) status = fail(IGC_EINVAL, "leading dimension %d of %s < its row length %lld", ld, name, cols);
    else if (reinterpret_cast<uintptr_t>(p) % bytes) status = fail(IGC_EINVAL, "%s is not %d-byte aligned", name, bytes);
  }
  void vector(const char* name, const void* p) {
    if (ok() && reinterpret_cast<uintptr_t>(p) % 4) status = fail(IGC_EINVAL, "%s is not 4-byte aligned", name);
  }
  void problem(int M, int N, int K, int type, int act) {
    fail_if(M < 0 || N < 0 || K < 0, "negative size");
    fail_if(type != IGC_F16 && type != IGC_BF16, "type must be IGC_F16 or IGC_BF16");
    fail_if(act < IGC_ACT_NONE || act > IGC_ACT_SIGMOID, "unknown activation");
    extent("M", M, MOST);
    extent("N", N, MOST);
    extent("K", K, MOST);
  }
  // The kernels index rows, columns and the reduction in 32 bits and step past
  // the end by a tile, a batch of K tiles or (the element-wise rows) four
  // workgroups per compute unit: all less than 4096.
  static constexpr int MOST = 0x7fffffff - 4095;
  void extent(const char* name, int n, int most) {
    if (ok() && n > most) status = fail(IGC_EUNSUPPORTED, "%s = %d > %d", name, n, most);
  }
};

inline int check_ws(const void* ws, size_t have, size_t need, bool required) {
  if (!need || (!ws && !required)) return IGC_OK;
  if (!ws) return fail(IGC_EINVAL, "this call needs a workspace of %zu bytes", need);
  if (have < need) return fail(IGC_EINVAL, "workspace of %zu bytes < the %zu bytes this call needs", have, need);
  if (reinterpret_cast<uintptr_t>(ws) & 255u) return fail(IGC_EINVAL, "workspace not 256-byte aligned");
  return IGC_OK;
}

inline size_t round256(size_t n) { return (n + 255) & ~size_t(255); }

// ---------------------------------------------------------------- products
inline igc_ffn::GemmArgs product(long long M, long long N, long long R, const void* A, long long lda, const void* B, long long ldb, void* Y,
                 long long ldy) {
  igc_ffn::GemmArgs a;
  std::memset(&a, 0, sizeof(a));
  a.M = (int)M;
  a.N = (int)N;
  a.R = (int)R;
  a.A = static_cast<const uint8_t*>(A);
  a.lda = lda;
  a.B = static_cast<const uint8_t*>(B);
  a.ldb = ldb;
  a.r_split = a.b_rows = a.R;
  a.m_split = a.m_rows = a.M;
  a.Y = static_cast<uint8_t*>(Y);
  a.ldy = ldy;
  return a;
}

// part: where the partial tiles of a split reduction go.
inline void apply_plan(igc_ffn::GemmArgs& a, const Plan& pl, uint8_t* part) {
  auto lines = [](const void* p, long long ld, int bytes) {  // (an output that is left out has no say)
    return !p || ((reinterpret_cast<uintptr_t>(p) & 127u) == 0 && ld * bytes % 128 == 0);
  };
  a.stream = lines(a.Y, a.ldy, a.y_f32 ? 4 : 2) && lines(a.Z, a.ldz, 2) && lines(a.U, a.ldu, 2) && lines(a.Y2, a.ldy2, 2);
  a.tiles_m = pl.tiles_m;
  a.tiles_n = pl.tiles_n;
  a.whole = (int)pl.whole;
  a.splits = pl.splits;
  a.part = reinterpret_cast<float*>(part);
}

}  // namespace igc_ffn_host
