// rows.hip -- the C ABI of the row operators (declared in igc.h): layer norm in
// both directions, rows in 8 bits, dropout.  Argument checks, workspace layout
// and the launches of each call; the arithmetic is in row_kernels.hpp and
// dropout.hpp.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstring>

#include "../../include/igc.h"
#include "dropout.hpp"
#include "op_host.hpp"
#include "row_kernels.hpp"

namespace igc_rows_host {

using igc_ffn_host::ceil_div;
using igc_ffn_host::check_ws;
using igc_ffn_host::Checker;
using igc_ffn_host::launch_status;
using igc_ffn_host::round256;
using igc_host::check_device;
using igc_host::device_cus;
using igc_host::fail;
using igc_rows::DropArgs;
using igc_rows::NormBackArgs;
using igc_rows::RowArgs;

int elem(int type) { return type == IGC_F32 ? 4 : 2; }

// Sizes and types of a norm: `type` 16 bits wide, x_type the same or fp32.
void check_rows(Checker& c, int M, int N, int type) {
  c.fail_if(M < 0 || N < 0, "negative size");
  c.fail_if(type != IGC_F16 && type != IGC_BF16, "type must be IGC_F16 or IGC_BF16");
  c.extent("M", M, Checker::MOST);
  c.extent("N", N, Checker::MOST);
}

// ---------------------------------------------------------------- rows
// Threads to a row: as many as it has chunks, up to 1024 with two chunks each
// (so more rows at once in a compute unit's registers than with more chunks a
// thread: 8192 x 4096 bf16 32.6 us with 512 threads, 36.0 with 256 and two chunks;
// 8192 x 1024 10.4, and 14.6 by a wave with two).  Longer rows are read again in
// every pass (2048 x 20000 bf16 39 to 41 us: 4.1 TB/s; 2048 x 65536 168: 3.2).
template <bool NORM, int XT, int OT>
void launch_rows(const RowArgs& a, int cus, hipStream_t stream) {
  // Rows that are read again are two to a compute unit, but one where two are more
  // than its share of an L2 (128 KB) and one is not (us, two and one, when it was chosen: 2048 x 20000
  // bf16 35.5 and 40.5, 1024 x 32768 32.1 and 35.0, 1024 x 40000 42.4 and 37.9, 512 x 65536
  // 38.8 and 34.2, 256 x 262144 81.5 and 81.3; of 300 x 65536, less than two each, 23.9
  // and 27.8; to 8 bits without a norm, read twice, 2048 x 65536 99 and 118).
  const long long row_bytes = (long long)a.N * igc_rows::Raw<XT>::EB;
  const bool one = NORM && a.N > 16384 && row_bytes > 64 * 1024 && row_bytes <= 128 * 1024 && a.M >= 2LL * cus;
  auto groups = [&](int threads, int rows) { return dim3((unsigned)std::min(ceil_div(a.M, rows), (one ? 1024LL : 2048LL) / threads * cus)); };
#define IGC_ROWS(threads, rows, ...) \
  hipLaunchKernelGGL((igc_rows::__VA_ARGS__), groups(threads, rows), dim3(threads), 0, stream, a)
  if constexpr (NORM && XT == igc_ffn::T_F32) {
    // Many rows of fp32 are bound by instructions, and what a row takes of them in
    // every thread is shared by two chunks (us, one chunk and two: fp32 to bf16 of 8192
    // x 4096 40.0 and 36.9, of 4096 x 4096 17.3 and 16.5, of 2100 x 4096 10.0 and 11.5, of 4000 x
    // 8192 36.0 and 36.4; bf16 to 8 bits of 4096 x 4096 16.7 and 17.6, of 8192 x 8192 60 and 64).
    if (a.N > 2048 && a.N <= 4096 && a.M >= 16LL * cus) {
      IGC_ROWS(256, 1, row_kernel<NORM, XT, OT, 256, 2>);
      return;
    }
  }
  if (a.N <= 128) IGC_ROWS(256, 16, row_kernel<NORM, XT, OT, 16, 1>);
  else if (a.N <= 256) IGC_ROWS(256, 8, row_kernel<NORM, XT, OT, 32, 1>);
  else if (a.N <= 512) IGC_ROWS(256, 4, row_kernel<NORM, XT, OT, 64, 1>);
  else if (a.N <= 1024) IGC_ROWS(256, 2, row_kernel<NORM, XT, OT, 128, 1>);
  else if (a.N <= 2048) IGC_ROWS(256, 1, row_kernel<NORM, XT, OT, 256, 1>);
  else if (a.N <= 4096) IGC_ROWS(512, 1, row_kernel<NORM, XT, OT, 512, 1>);
  else if (a.N <= 8192) IGC_ROWS(1024, 1, row_kernel<NORM, XT, OT, 1024, 1>);
  else if (a.N <= 16384) IGC_ROWS(1024, 1, row_kernel<NORM, XT, OT, 1024, 2>);
  else IGC_ROWS(1024, 1, long_row_kernel<NORM, XT, OT, 1024>);
#undef IGC_ROWS
}

int layer_norm_forward_impl(const igc_layer_norm_forward* d, hipStream_t stream) {
  Checker c;
  c.fail_if(!d, "descriptor is NULL");
  if (!c.ok()) return c.status;
  check_rows(c, d->M, d->N, d->type);
  c.fail_if(d->x_type != d->type && d->x_type != IGC_F32, "x_type must be `type` or IGC_F32");
  c.fail_if(!(d->eps >= 0.0f) || std::isinf(d->eps), "eps must be a finite number, not negative");
  c.fail_if(!d->Y && !d->Q && !d->mean && !d->rstd && d->M > 0 && d->N > 0, "no output requested");  // (matrices of nothing may be NULL)
  c.matrix("X", d->X, d->ldx, d->M, d->N, elem(d->x_type), false);
  c.matrix("Y", d->Y, d->ldy, d->M, d->N, 2, true);
  c.matrix("Q", d->Q, d->ldq, d->M, d->N, 1, true);
  c.fail_if(d->Q && !d->scale, "Q needs scale");
  c.vector("gamma", d->gamma);
  c.vector("beta", d->beta);
  c.vector("mean", d->mean);
  c.vector("rstd", d->rstd);
  c.vector("scale", d->scale);
  if (!c.ok() || d->M == 0) return c.status;
  int dev;
  if (int s = check_device(&dev)) return s;
  RowArgs a;
  std::memset(&a, 0, sizeof(a));
  a.M = d->M;
  a.N = d->N;
  a.X = static_cast<const uint8_t*>(d->X);
  a.ldx = d->ldx;
  a.n = igc_rows::Divisor::by(d->N);
  a.eps = d->eps;
  a.gamma = d->gamma;
  a.beta = d->beta;
  a.Y = static_cast<uint8_t*>(d->Y);
  a.ldy = d->ldy;
  a.mean = d->mean;
  a.rstd = d->rstd;
  a.Q = d->Q;
  a.ldq = d->ldq;
  a.scale = d->Q || d->N == 0 ? d->scale : nullptr;
  using namespace igc_ffn;
  const int cus = device_cus(dev);
  const bool wide = d->x_type == IGC_F32;
  if (d->type == IGC_BF16)
    wide ? launch_rows<true, T_F32, T_BF16>(a, cus, stream) : launch_rows<true, T_BF16, T_BF16>(a, cus, stream);
  else
    wide ? launch_rows<true, T_F32, T_F16>(a, cus, stream) : launch_rows<true, T_F16, T_F16>(a, cus, stream);
  return launch_status();
}

int quantize_rows_impl(const igc_quantize_rows* d, hipStream_t stream) {
  Checker c;
  c.fail_if(!d, "descriptor is NULL");
  if (!c.ok()) return c.status;
  check_rows(c, d->M, d->N, d->type);
  c.matrix("X", d->X, d->ldx, d->M, d->N, 2, false);
  c.matrix("Q", d->Q, d->ldq, d->M, d->N, 1, false);
  c.fail_if(d->M > 0 && !d->scale, "scale is NULL");
  c.vector("scale", d->scale);
  if (!c.ok() || d->M == 0) return c.status;
  int dev;
  if (int s = check_device(&dev)) return s;
  RowArgs a;
  std::memset(&a, 0, sizeof(a));
  a.M = d->M;
  a.N = d->N;
  a.X = static_cast<const uint8_t*>(d->X);
  a.ldx = d->ldx;
  a.Q = d->Q;
  a.ldq = d->ldq;
  a.scale = d->scale;
  using namespace igc_ffn;
  if (d->type == IGC_BF16)
    launch_rows<false, T_BF16, T_BF16>(a, device_cus(dev), stream);
  else
    launch_rows<false, T_F16, T_F16>(a, device_cus(dev), stream);
  return launch_status();
}

// ---------------------------------------------------------------- backward
// How a backward pass splits its rows: registers hold rows of up to 8192
// elements, a chunk a thread; longer ones go by columns, after a launch for
// their means (2048 x 16384 bf16 76 us; two chunks a thread, which do not fit
// the registers of 1024 threads, 105).
struct BackPlan {
  bool in_registers;
  int rows, groups, blocks;  // rows at a time (a block, by columns); workgroups
};
// Rows that a thread adds one after the other: more of them get more blocks, so that
// no sum takes so many fp32 additions that their roundings show (2^17 rows to a
// thread, of 0.1: off by two in a thousand).
constexpr long long MOST_ROWS = 4096;
BackPlan plan_back(long long M, int N, int cus) {
  BackPlan b;
  b.in_registers = N <= 8192;
  if (b.in_registers) {
    int threads = 16;  // to a row
    while (threads * 8 < N) threads *= 2;
    b.rows = 1024 / threads;
    b.groups = 1;
    b.blocks = (int)std::min(ceil_div(M, b.rows), std::max((long long)cus, ceil_div(M, b.rows * MOST_ROWS)));
  } else {
    // enough workgroups to fill the card, and few enough that their sums stay small beside the rows
    b.groups = (int)ceil_div(N, 512);
    b.rows = (int)std::min(std::max(16LL, ceil_div(M, std::max(1LL, 4LL * cus / b.groups))), 4 * MOST_ROWS);
    b.rows = (int)std::max<long long>(b.rows, ceil_div(M, std::max(1LL, 0x7fffffLL / b.groups)));
    b.blocks = (int)ceil_div(M, b.rows);
  }
  return b;
}

template <int XT, int OT>
int launch_back(const NormBackArgs& a, const BackPlan& pl, int cus, hipStream_t stream) {
  if (pl.in_registers) {
    const dim3 g((unsigned)a.blocks);
#define IGC_BACK(T) hipLaunchKernelGGL((igc_rows::norm_back_rows_kernel<XT, OT, T>), g, dim3(1024), 0, stream, a)
    if (a.N <= 128) IGC_BACK(16);
    else if (a.N <= 256) IGC_BACK(32);
    else if (a.N <= 512) IGC_BACK(64);
    else if (a.N <= 1024) IGC_BACK(128);
    else if (a.N <= 2048) IGC_BACK(256);
    else if (a.N <= 4096) IGC_BACK(512);
    else IGC_BACK(1024);
#undef IGC_BACK
    return launch_status();
  }
  if (a.dX) {
    // (three workgroups of 512 threads a compute unit; of 1024 threads with these registers one fits: 8192 x 12288 bf16 94 us, so 69)
    hipLaunchKernelGGL((igc_rows::norm_back_stats_kernel<XT, OT, 512>), dim3((unsigned)std::min<long long>(a.M, 3LL * cus)), dim3(512), 0,
                       stream, a);
    if (int s = launch_status()) return s;
  }
  hipLaunchKernelGGL((igc_rows::norm_back_kernel<XT, OT>), dim3((unsigned)((long long)a.groups * a.blocks)), dim3(256), 0, stream, a);
  return launch_status();
}

int layer_norm_backward_impl(const igc_layer_norm_backward* d, size_t* query, hipStream_t stream) {
  Checker c;
  c.fail_if(!d, "descriptor is NULL");
  if (!c.ok()) return c.status;
  check_rows(c, d->M, d->N, d->type);
  c.fail_if(d->x_type != d->type && d->x_type != IGC_F32, "x_type must be `type` or IGC_F32");
  c.fail_if(!d->dX && !d->dgamma && !d->dbeta && d->M > 0 && d->N > 0, "no output requested");
  c.matrix("dY", d->dY, d->lddy, d->M, d->N, 2, false);
  c.matrix("X", d->X, d->ldx, d->M, d->N, elem(d->x_type), false);
  c.fail_if(d->M > 0 && d->N > 0 && (!d->mean || !d->rstd), "mean or rstd is NULL");
  c.matrix("R", d->R, d->ldr, d->M, d->N, elem(d->x_type), true);
  c.matrix("dX", d->dX, d->lddx, d->M, d->N, elem(d->x_type), true);
  c.vector("mean", d->mean);
  c.vector("rstd", d->rstd);
  c.vector("gamma", d->gamma);
  c.vector("dgamma", d->dgamma);
  c.vector("dbeta", d->dbeta);
  if (!c.ok()) return c.status;
  if (d->N == 0) {
    if (query) *query = 0;
    return IGC_OK;
  }
  int dev;
  if (int s = check_device(&dev)) return s;
  const int cus = device_cus(dev);
  const bool sums = d->dgamma || d->dbeta;
  const int width = (int)ceil_div(d->N, 64) * 64;
  const BackPlan pl = plan_back(d->M, d->N, cus);
  const size_t stat_bytes = d->dX && !pl.in_registers ? round256((size_t)d->M * sizeof(float2)) : 0;
  const size_t need = stat_bytes + (sums ? round256((size_t)pl.blocks * 2 * width * sizeof(float)) : 0);
  if (query) {
    *query = need;
    return IGC_OK;
  }
  if ((long long)pl.groups * pl.blocks > 0x7fffffLL)
    return fail(IGC_EUNSUPPORTED, "too many workgroups (%lld)", (long long)pl.groups * pl.blocks);
  if (int s = check_ws(d->workspace, d->ws_bytes, need, true)) return s;
  NormBackArgs a;
  std::memset(&a, 0, sizeof(a));
  a.M = d->M;
  a.N = d->N;
  a.dY = static_cast<const uint8_t*>(d->dY);
  a.lddy = d->lddy;
  a.X = static_cast<const uint8_t*>(d->X);
  a.ldx = d->ldx;
  a.R = static_cast<const uint8_t*>(d->R);
  a.ldr = d->ldr;
  a.mean = d->mean;
  a.rstd = d->rstd;
  a.gamma = d->gamma;
  a.inv_n = 1.0f / (float)d->N;
  a.dX = static_cast<uint8_t*>(d->dX);
  a.lddx = d->lddx;
  a.stats = static_cast<float2*>(d->workspace);
  a.sums = sums ? reinterpret_cast<float*>(static_cast<uint8_t*>(d->workspace) + stat_bytes) : nullptr;
  a.width = width;
  a.rows = pl.rows;
  a.groups = pl.groups;
  a.blocks = pl.blocks;
  if (d->M > 0) {
    using namespace igc_ffn;
    const bool wide = d->x_type == IGC_F32;
    int s;
    if (d->type == IGC_BF16)
      s = wide ? launch_back<T_F32, T_BF16>(a, pl, cus, stream) : launch_back<T_BF16, T_BF16>(a, pl, cus, stream);
    else
      s = wide ? launch_back<T_F32, T_F16>(a, pl, cus, stream) : launch_back<T_F16, T_F16>(a, pl, cus, stream);
    if (s) return s;
  }
  if (!sums) return IGC_OK;
  const igc_ffn::ColsumArgs cs{a.sums, pl.blocks, 2, width, d->N, d->dgamma, d->dbeta};
  hipLaunchKernelGGL((igc_ffn::colsum_kernel<0>), dim3((unsigned)igc_ffn_host::colsum_groups(cs)), dim3(256), 0, stream, cs);
  return launch_status();
}

// ---------------------------------------------------------------- dropout
int dropout_impl(const igc_dropout* d, hipStream_t stream) {
  Checker c;
  c.fail_if(!d, "descriptor is NULL");
  if (!c.ok()) return c.status;
  c.fail_if(d->M < 0 || d->N < 0, "negative size");
  auto known = [](int t) { return t == IGC_F16 || t == IGC_BF16 || t == IGC_F32; };
  c.fail_if(!known(d->type) || !known(d->y_type), "unknown type");
  c.fail_if(d->type != d->y_type && d->type != IGC_F32 && d->y_type != IGC_F32, "y_type must be `type`, or one of them IGC_F32");
  c.extent("M", d->M, Checker::MOST);
  c.extent("N", d->N, Checker::MOST);
  c.fail_if(!(d->p >= 0.0 && d->p <= 1.0), "p must be in [0, 1]");
  c.matrix("X", d->X, d->ldx, d->M, d->N, elem(d->type), false);
  c.matrix("R", d->R, d->ldr, d->M, d->N, elem(d->y_type), true);
  c.matrix("Y", d->Y, d->ldy, d->M, d->N, elem(d->y_type), false);
  c.fail_if(reinterpret_cast<uintptr_t>(d->step) % 8 != 0, "step is not 8-byte aligned");
  if (!c.ok() || d->M == 0 || d->N == 0) return c.status;
  int dev;
  if (int s = check_device(&dev)) return s;
  const uint64_t border = (uint64_t)std::nearbyint(d->p * 0x1p32);
  DropArgs a;
  std::memset(&a, 0, sizeof(a));
  a.M = d->M;
  a.N = d->N;
  a.X = static_cast<const uint8_t*>(d->X);
  a.ldx = d->ldx;
  a.R = static_cast<const uint8_t*>(d->R);
  a.ldr = d->ldr;
  a.Y = static_cast<uint8_t*>(d->Y);
  a.ldy = d->ldy;
  a.per = (int)ceil_div(d->N, 8);
  a.drops = border != 0;
  a.last = (uint32_t)(border - 1);
  a.scale = border >> 32 ? 0.0f : (float)(0x1p32 / (double)((1ULL << 32) - border));
  a.seed0 = (uint32_t)d->seed;
  a.seed1 = (uint32_t)(d->seed >> 32);
  a.offset = d->offset;
  a.step = d->step;
  const long long chunks = a.M * a.per;
  const long long groups = std::min(ceil_div(chunks, 256), 32LL * device_cus(dev));
  a.step_row = groups * 256 / a.per;
  a.step_chunk = (int)(groups * 256 % a.per);
  const dim3 g((unsigned)groups), t(256);
#define IGC_DROP(xt, yt) hipLaunchKernelGGL((igc_rows::dropout_kernel<igc_ffn::xt, igc_ffn::yt>), g, t, 0, stream, a)
  const int x = d->type, y = d->y_type;
  if (x == IGC_F32 && y == IGC_F32) IGC_DROP(T_F32, T_F32);
  else if (x == IGC_F32 && y == IGC_BF16) IGC_DROP(T_F32, T_BF16);
  else if (x == IGC_F32) IGC_DROP(T_F32, T_F16);
  else if (x == IGC_BF16 && y == IGC_F32) IGC_DROP(T_BF16, T_F32);
  else if (x == IGC_BF16) IGC_DROP(T_BF16, T_BF16);
  else if (y == IGC_F32) IGC_DROP(T_F16, T_F32);
  else IGC_DROP(T_F16, T_F16);
#undef IGC_DROP
  return launch_status();
}

}  // namespace igc_rows_host

extern "C" {

using namespace igc_rows_host;

int layer_norm_forward(const igc_layer_norm_forward* d, void* stream) {
  return layer_norm_forward_impl(d, static_cast<hipStream_t>(stream));
}
int layer_norm_backward(const igc_layer_norm_backward* d, void* stream) {
  return layer_norm_backward_impl(d, nullptr, static_cast<hipStream_t>(stream));
}
int layer_norm_backward_workspace_size(const igc_layer_norm_backward* d, size_t* bytes) {
  if (!bytes) return fail(IGC_EINVAL, "bytes is NULL");
  return layer_norm_backward_impl(d, bytes, nullptr);
}
int quantize_rows(const igc_quantize_rows* d, void* stream) { return quantize_rows_impl(d, static_cast<hipStream_t>(stream)); }
int dropout(const igc_dropout* d, void* stream) { return dropout_impl(d, static_cast<hipStream_t>(stream)); }

}  // extern "C"
