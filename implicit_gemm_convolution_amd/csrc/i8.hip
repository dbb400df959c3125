// i8.hip -- the C ABI of the products in 8 bits with a scale for each row and
// each column (declared in igc.h): argument checks, plans, workspace layout and
// launches.  The kernels are those of ffn_kernels.hpp in the modes M_I8 and
// M_I8_GLU, instantiated in i8_launch.hip.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstring>

#include "../../include/igc.h"
#include "op_host.hpp"

namespace igc_i8_host {

using namespace igc_ffn_host;
using igc_ffn::I8Args;
using igc_host::check_device;
using igc_host::device_cus;

// 128 * 128 * K has to fit in int32.
constexpr int K_MOST = 131071;

// What every row of an operand starts at a multiple of: 16 (and its length is
// whole chunks of 16: the direct-to-LDS loaders take it as it is), 4, or 1 byte.
int row_align(const void* p, long long ld, long long length) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p);
  if (length % 2 == 0 && ld % 2 == 0 && dma_operand(p, ld / 2, length / 2)) return 16;
  return (a & 3u) || (ld & 3) ? 1 : 4;
}

// Operands that are copied into rows of whole chunks.
struct Pads {
  igc_ffn::PadArgs args;
  size_t bytes = 0;     // workspace
  long long moved = 0;  // bytes read and written
  size_t at[igc_ffn::PAD_MOST] = {};
  bool possible = true;
  Pads() { std::memset(&args, 0, sizeof(args)); }
  static long long padded(long long cols) { return std::max(16LL, ceil_div(cols, 16) * 16); }
  int add(const void* p, long long ld, long long rows, long long cols) {
    const int i = args.count++;
    const long long chunks = rows * (padded(cols) / 16);
    possible = possible && chunks <= 0x7fffffffLL;
    args.src[i] = static_cast<const uint8_t*>(p);
    args.ld[i] = ld;
    args.cols[i] = (int)cols;
    args.chunks[i] = (uint32_t)chunks;
    args.first[i + 1] = args.first[i] + (int)ceil_div(chunks, 1024);
    at[i] = bytes;
    bytes += round256((size_t)rows * padded(cols));
    moved += 2 * rows * cols;
    return i;
  }
  const uint8_t* place(int i, uint8_t* ws) {
    args.dst[i] = ws + at[i];
    return args.dst[i];
  }
  float us() const { return 4.0f + (float)moved / 5.7e6f; }
};

// The plan of the kernel that takes rows of any alignment as they lie: a chain
// of K tiles of 128, or so much for each of its workgroups where they fill the
// card, and their outputs.  us, as they lie | copied first or few rows streamed:
// 131 x 5003 x 2049 11.0 | 18.0, 64 x 5003 x 2049 10.7 | 13.2, 300 x 16001 x 2049
// 33.9 | 35.6, 1000 x 16001 x 2049 94.7 | 52.9, 8 x 1001 x 2049 9.8 | 6.2; the gated block
// 131 x 5003 x 2049 16.4 | 21.6, 600 x 5003 x 2049 55.6 | 32.8.
Plan bytes_plan(bool glu, long long M, long long N, long long K, int cus) {
  Plan pl = tile_plan(glu ? igc_ffn::M_GLU : igc_ffn::M_FWD, P_TILE_64, M, N);
  pl.variant = P_BYTES;
  const float count = (float)pl.tiles_m * (float)pl.tiles_n * 256.0f / (float)cus, tiles = (float)ceil_div(K, 128);
  pl.us = glu ? 6.0f + tiles * std::max(0.52f, 2.7e-3f * count) + 0.014f * count : 4.5f + tiles * std::max(0.35f, 1.3e-3f * count) + 0.005f * count;
  return pl;
}

template <int MODE>
int product_i8(I8Args& a, int type, void* ws, size_t ws_bytes, size_t* query, hipStream_t stream) {
  if (a.M == 0 || a.N == 0) {
    if (query) *query = 0;
    return IGC_OK;
  }
  int dev;
  if (int s = check_device(&dev)) return s;
  const int cus = device_cus(dev);
  constexpr bool GLU = igc_ffn::is_glu(MODE);
  constexpr int AS = GLU ? igc_ffn::M_GLU : igc_ffn::M_FWD;  // the 16-bit product whose rows have as many bytes
  const int a_al = row_align(a.A, a.lda, a.R), b_al = row_align(a.B, a.ldb, a.R), b2_al = GLU ? row_align(a.B2, a.ldb2, a.R) : 16;
  const int align = std::min(a_al, std::min(b_al, b2_al));
  const long long units = ceil_div(a.R, 2), whole = Pads::padded(a.R);
  Pads pads;
  Plan pl;
  int ia = -1, ib = -1, ib2 = -1;
  // (Plans of aligned operands go by the times of 16-bit products whose rows have as
  // many bytes: over 175 shapes 1.3% slower than the best plan in the mean, but with M <= 24 and
  // N = 11008 by 14 to 38%, weights partly in the memory-side cache.)
  if (align == 16) {
    pl = make_plan(AS, a.M, a.N, units, 16, cus, true);
  } else {
    // Rows of another alignment or length: taken from where they lie, or copied
    // into rows of whole chunks first.
    if (a_al != 16) ia = pads.add(a.A, a.lda, a.M, a.R);
    if (b_al != 16) ib = pads.add(a.B, a.ldb, a.N, a.R);
    if (b2_al != 16) ib2 = pads.add(a.B2, a.ldb2, a.N, a.R);
    pl = make_plan(AS, a.M, a.N, whole / 2, 16, cus, true);
    pl.us = pads.possible ? pl.us + pads.us() : 1e30f;
    bool copy = true;
    auto take = [&](const Plan& q) {
      if (q.us >= pl.us) return;
      pl = q;
      copy = false;
    };
    if (a.M <= 64) {
      const int skinny_align = align < 4 ? 2 : 4;
      take(skinny_plan(AS, P_SKINNY_32, a.M, a.N, units, skinny_align, cus));
      if (!GLU) take(skinny_plan(AS, P_SKINNY_16, a.M, a.N, units, skinny_align, cus));
    }
    take(bytes_plan(GLU, a.M, a.N, a.R, cus));
    if (!copy) {
      pads = Pads();
      ia = ib = ib2 = -1;
      a.odd_rows = align < 4;
    }
  }
  const size_t need = pads.bytes + pl.part_bytes;
  if (query) {
    *query = need;
    return IGC_OK;
  }
  if (int s = check_ws(ws, ws_bytes, need, true)) return s;
  uint8_t* const to = static_cast<uint8_t*>(ws);
  if (pads.args.count > 0) {
    if (ia >= 0) a.A = pads.place(ia, to), a.lda = whole;
    if (ib >= 0) a.B = pads.place(ib, to), a.ldb = whole;
    if (ib2 >= 0) a.B2 = pads.place(ib2, to), a.ldb2 = whole;
    a.R = a.r_split = a.b_rows = (int)whole;
    hipLaunchKernelGGL((igc_ffn::pad_bytes_kernel<0>), dim3((unsigned)pads.args.first[pads.args.count]), dim3(256), 0, stream, pads.args);
    if (int s = launch_status()) return s;
  }
  apply_plan(a, pl, to + pads.bytes);
  return type == IGC_F16 ? launch_product<false, MODE>(a, pl, stream) : launch_product<true, MODE>(a, pl, stream);
}

void check_problem(Checker& c, int M, int N, int K, int act) {
  c.problem(M, N, K, IGC_BF16, act);
  if (c.ok() && K > K_MOST) c.status = fail(IGC_EOVERFLOW, "K = %d > %d: the int32 sums could overflow", K, K_MOST);
}
void check_scale(Checker& c, const char* what, const void* p, bool needed) {
  if (c.ok() && needed && !p) c.status = fail(IGC_EINVAL, "%s is NULL", what);
  c.vector(what, p);
}

int linear_i8_impl(const igc_linear_i8* d, size_t* query, hipStream_t stream) {
  Checker c;
  c.fail_if(!d, "descriptor is NULL");
  if (!c.ok()) return c.status;
  check_problem(c, d->M, d->N, d->K, d->act);
  c.fail_if(d->y_type != IGC_F16 && d->y_type != IGC_BF16 && d->y_type != IGC_F32, "unknown y_type");
  const int yb = d->y_type == IGC_F32 ? 4 : 2;
  const bool some = d->M > 0 && d->N > 0;
  c.matrix("X", d->X, d->ldx, some ? d->M : 0, d->K, 1, false);
  c.matrix("W", d->W, d->ldw, some ? d->N : 0, d->K, 1, false);
  check_scale(c, "x_scale", d->x_scale, some);
  check_scale(c, "w_scale", d->w_scale, some);
  c.matrix("Y", d->Y, d->ldy, d->M, d->N, yb, false);
  c.matrix("R", d->R, d->ldr, d->M, d->N, yb, true);
  c.vector("bias", d->bias);
  if (!c.ok()) return c.status;
  I8Args a{product(d->M, d->N, d->K, d->X, d->ldx, d->W, d->ldw, d->Y, d->ldy), d->x_scale, d->w_scale, nullptr};
  a.act = d->act;
  a.bias = d->bias;
  a.res = static_cast<const uint8_t*>(d->R);
  a.ldr = d->ldr;
  a.y_f32 = d->y_type == IGC_F32;
  return product_i8<igc_ffn::M_I8>(a, d->y_type, d->workspace, d->ws_bytes, query, stream);
}

int glu_i8_impl(const igc_glu_i8* d, size_t* query, hipStream_t stream) {
  Checker c;
  c.fail_if(!d, "descriptor is NULL");
  if (!c.ok()) return c.status;
  check_problem(c, d->M, d->N, d->K, d->act);
  c.fail_if(d->type != IGC_F16 && d->type != IGC_BF16, "type must be IGC_F16 or IGC_BF16");
  const bool some = d->M > 0 && d->N > 0;
  c.matrix("X", d->X, d->ldx, some ? d->M : 0, d->K, 1, false);
  c.matrix("Wg", d->Wg, d->ldwg, some ? d->N : 0, d->K, 1, false);
  c.matrix("Wu", d->Wu, d->ldwu, some ? d->N : 0, d->K, 1, false);
  check_scale(c, "x_scale", d->x_scale, some);
  check_scale(c, "wg_scale", d->wg_scale, some);
  check_scale(c, "wu_scale", d->wu_scale, some);
  c.matrix("H", d->H, d->ldh, d->M, d->N, 2, false);
  c.vector("bias_g", d->bias_g);
  c.vector("bias_u", d->bias_u);
  if (!c.ok()) return c.status;
  I8Args a{product(d->M, d->N, d->K, d->X, d->ldx, d->Wg, d->ldwg, d->H, d->ldh), d->x_scale, d->wg_scale, d->wu_scale};
  a.B2 = reinterpret_cast<const uint8_t*>(d->Wu);
  a.ldb2 = d->ldwu;
  a.act = d->act;
  a.bias = d->bias_g;
  a.bias2 = d->bias_u;
  return product_i8<igc_ffn::M_I8_GLU>(a, d->type, d->workspace, d->ws_bytes, query, stream);
}

}  // namespace igc_i8_host

extern "C" {

int linear_i8(const igc_linear_i8* d, void* stream) { return igc_i8_host::linear_i8_impl(d, nullptr, static_cast<hipStream_t>(stream)); }
int linear_i8_workspace_size(const igc_linear_i8* d, size_t* bytes) {
  if (!bytes) return igc_host::fail(IGC_EINVAL, "bytes is NULL");
  return igc_i8_host::linear_i8_impl(d, bytes, nullptr);
}
int glu_i8(const igc_glu_i8* d, void* stream) { return igc_i8_host::glu_i8_impl(d, nullptr, static_cast<hipStream_t>(stream)); }
int glu_i8_workspace_size(const igc_glu_i8* d, size_t* bytes) {
  if (!bytes) return igc_host::fail(IGC_EINVAL, "bytes is NULL");
  return igc_i8_host::glu_i8_impl(d, bytes, nullptr);
}

}  // extern "C"
