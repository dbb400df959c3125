// ffn.hip -- the C ABI of the feed-forward operators and of gradient clipping
// (declared in igc.h): argument validation, workspace layout and the sequence
// of launches of each call.  All arithmetic happens in the kernels of
// ffn_kernels.hpp and grad_clip.hpp; the library allocates no device memory.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstring>

#include "../../include/igc.h"
#include "ffn_host.hpp"
#include "grad_clip.hpp"

namespace igc_ffn_host {

using igc_ffn::GemmArgs;
using igc_host::check_device;
using igc_host::device_cus;

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

int check_ws(const void* ws, size_t have, size_t need, bool required) {
  if (!need || (!ws && !required)) return IGC_OK;
  if (!ws) return fail(IGC_EINVAL, "this call needs a workspace of %zu bytes", need);
  if (have < need) return fail(IGC_EINVAL, "workspace of %zu bytes < the %zu bytes this call needs", have, need);
  if (reinterpret_cast<uintptr_t>(ws) & 255u) return fail(IGC_EINVAL, "workspace not 256-byte aligned");
  return IGC_OK;
}

size_t round256(size_t n) { return (n + 255) & ~size_t(255); }

// ---------------------------------------------------------------- products
GemmArgs product(long long M, long long N, long long R, const void* A, long long lda, const void* B, long long ldb, void* Y,
                 long long ldy) {
  GemmArgs a;
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
void apply_plan(GemmArgs& a, const Plan& pl, uint8_t* part) {
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

template <int MODE>
int run_product(GemmArgs& a, const Plan& pl, int type, uint8_t* part, hipStream_t stream) {
  apply_plan(a, pl, part);
  return type == IGC_BF16 ? launch_product<true, MODE>(a, pl, stream) : launch_product<false, MODE>(a, pl, stream);
}

// Operands that are copied into padded rows of the workspace, in the order in
// which they are added.
struct Pads {
  igc_ffn::PadArgs args;
  size_t bytes = 0;       // workspace
  long long moved = 0;    // bytes read and written
  size_t at[igc_ffn::PAD_MOST] = {};
  bool possible = true;
  Pads() { std::memset(&args, 0, sizeof(args)); }
  static long long padded(long long cols) { return ceil_div(cols, 8) * 8; }
  int add(const void* p, long long ld, long long rows, long long cols) {
    const int i = args.count++;
    const long long chunks = rows * (padded(cols) / 8);
    possible = possible && rows > 0 && cols >= 8 && chunks <= 0x7fffffffLL && padded(cols) <= (1 << 21) - 8;
    args.src[i] = static_cast<const uint8_t*>(p);
    args.ld[i] = ld * 2;
    args.cols[i] = (int)cols;
    args.chunks[i] = (uint32_t)chunks;
    args.first[i + 1] = args.first[i] + (int)ceil_div(chunks, 1024);
    at[i] = bytes;
    bytes += round256((size_t)rows * padded(cols) * 2);
    moved += 4 * rows * cols;
    return i;
  }
  int groups() const { return args.first[args.count]; }
  const uint8_t* place(int i, uint8_t* ws) {
    args.dst[i] = ws + at[i];
    return args.dst[i];
  }
};

// What the copy takes in a launch of its own: 5 to 6 TB/s (130 + 4096 rows of
// 4093 11.8 us).
inline float pad_us(const Pads& p) { return 4.0f + (float)p.moved / 5.7e6f; }

// ---------------------------------------------------------------- forward
template <int MODE>
int forward(GemmArgs& a, int type, void* ws, size_t ws_bytes, size_t* query, hipStream_t stream) {
  if (a.M == 0 || a.N == 0) {
    if (query) *query = 0;
    return IGC_OK;
  }
  int dev;
  if (int s = check_device(&dev)) return s;
  const int cus = device_cus(dev);
  const bool may = query || ws;
  const int a_al = row_align(a.A, a.lda, a.R), b_al = row_align(a.B, a.ldb, a.R);
  const int b2_al = MODE == igc_ffn::M_GLU ? row_align(a.B2, a.ldb2, a.R) : 16;
  const bool a_ok = a_al == 16, b_ok = b_al == 16, b2_ok = b2_al == 16;
  const int align = std::min(a_al, std::min(b_al, b2_al));
  a.odd_rows = align < 4;
  Plan pl = make_plan(MODE, a.M, a.N, a.R, align, cus, may);
  Pads pads;
  // Operands of another alignment are copied into padded rows where the copy
  // costs less than the faster kernel gains (bf16, us, without and with:
  // 200 x 1000 x 257 7.4 and 9.5, 727 x 1344 x 6130 65 and 39, the gated block
  // at 304 x 7200 x 5402 125 and 148, at 6900 x 2600 x 2201 260 and 170).
  if (may && !(a_ok && b_ok && b2_ok)) {
    const int ia = a_ok ? -1 : pads.add(a.A, a.lda, a.M, a.R), ib = b_ok ? -1 : pads.add(a.B, a.ldb, a.N, a.R);
    const int ib2 = b2_ok ? -1 : pads.add(a.B2, a.ldb2, a.N, a.R);
    const Plan aligned = make_plan(MODE, a.M, a.N, Pads::padded(a.R), 16, cus, may);
    if (pads.possible && pad_us(pads) + aligned.us < pl.us) {
      pl = aligned;
      uint8_t* const to = static_cast<uint8_t*>(ws);
      if (ia >= 0) a.A = pads.place(ia, to), a.lda = Pads::padded(a.R);
      if (ib >= 0) a.B = pads.place(ib, to), a.ldb = Pads::padded(a.R);
      if (ib2 >= 0) a.B2 = pads.place(ib2, to), a.ldb2 = Pads::padded(a.R);
      a.R = a.r_split = a.b_rows = (int)Pads::padded(a.R);
      a.odd_rows = 0;
    } else {
      pads = Pads();
    }
  }
  const size_t need = pads.bytes + pl.part_bytes;
  if (query) {
    *query = need;
    return IGC_OK;
  }
  if (int s = check_ws(ws, ws_bytes, need, false)) return s;
  if (pads.groups() > 0) {
    hipLaunchKernelGGL((igc_ffn::pad_kernel<0>), dim3((unsigned)pads.groups()), dim3(256), 0, stream, pads.args);
    if (int s = launch_status()) return s;
  }
  return run_product<MODE>(a, pl, type, static_cast<uint8_t*>(ws) + pads.bytes, stream);
}

int linear_forward_impl(const igc_linear_forward* d, size_t* query, hipStream_t stream) {
  Checker c;
  c.fail_if(!d, "descriptor is NULL");
  if (!c.ok()) return c.status;
  c.problem(d->M, d->N, d->K, d->type, d->act);
  c.fail_if(d->y_type != d->type && d->y_type != IGC_F32, "y_type must be the operands' type or IGC_F32");
  const int yb = d->y_type == IGC_F32 ? 4 : 2;
  const bool some = d->M > 0 && d->N > 0;
  c.matrix("X", d->X, d->ldx, some ? d->M : 0, d->K, 2, false);
  c.matrix("W", d->W, d->ldw, some ? d->N : 0, d->K, 2, false);
  c.matrix("Y", d->Y, d->ldy, d->M, d->N, yb, false);
  c.matrix("R", d->R, d->ldr, d->M, d->N, yb, true);
  c.matrix("Z", d->Z, d->ldz, d->M, d->N, 2, true);
  c.vector("bias", d->bias);
  if (!c.ok()) return c.status;
  GemmArgs a = product(d->M, d->N, d->K, d->X, d->ldx, d->W, d->ldw, d->Y, d->ldy);
  a.act = d->act;
  a.bias = d->bias;
  a.res = static_cast<const uint8_t*>(d->R);
  a.ldr = d->ldr;
  a.y_f32 = d->y_type == IGC_F32;
  a.Z = static_cast<uint8_t*>(d->Z);
  a.ldz = d->ldz;
  return forward<igc_ffn::M_FWD>(a, d->type, d->workspace, d->ws_bytes, query, stream);
}

int glu_forward_impl(const igc_glu_forward* d, size_t* query, hipStream_t stream) {
  Checker c;
  c.fail_if(!d, "descriptor is NULL");
  if (!c.ok()) return c.status;
  c.problem(d->M, d->N, d->K, d->type, d->act);
  const bool some = d->M > 0 && d->N > 0;
  c.matrix("X", d->X, d->ldx, some ? d->M : 0, d->K, 2, false);
  c.matrix("Wg", d->Wg, d->ldwg, some ? d->N : 0, d->K, 2, false);
  c.matrix("Wu", d->Wu, d->ldwu, some ? d->N : 0, d->K, 2, false);
  c.matrix("H", d->H, d->ldh, d->M, d->N, 2, false);
  c.matrix("G", d->G, d->ldg, d->M, d->N, 2, true);
  c.matrix("U", d->U, d->ldu, d->M, d->N, 2, true);
  c.vector("bias_g", d->bias_g);
  c.vector("bias_u", d->bias_u);
  if (!c.ok()) return c.status;
  GemmArgs a = product(d->M, d->N, d->K, d->X, d->ldx, d->Wg, d->ldwg, d->H, d->ldh);
  a.B2 = static_cast<const uint8_t*>(d->Wu);
  a.ldb2 = d->ldwu;
  a.act = d->act;
  a.bias = d->bias_g;
  a.bias2 = d->bias_u;
  a.Z = static_cast<uint8_t*>(d->G);
  a.ldz = d->ldg;
  a.U = static_cast<uint8_t*>(d->U);
  a.ldu = d->ldu;
  return forward<igc_ffn::M_GLU>(a, d->type, d->workspace, d->ws_bytes, query, stream);
}

// ---------------------------------------------------------------- backward
// What both backward passes do: the element-wise part (D, or dG and dU, into
// the workspace, and the column sums), then the two products.
struct Backward {
  int M, N, K, type, act;
  bool glu;
  const void *dY, *Z, *U, *X, *W, *W2;
  int lddy, ldz, ldu, ldx, ldw, ldw2;
  void *dX, *dW, *dW2;
  int lddx, lddw, lddw2;
  float *db, *db2;
  void* ws;
  size_t ws_bytes;
};

// Rows per workgroup of the element-wise kernel: enough workgroups to fill
// the card, with at least 8 rows each so that the partial column sums stay
// small beside D.
int act_rows(int M, int width, int cus) {
  const long long cols = ceil_div(width, 512);
  const long long want = std::max(1LL, 4LL * cus / cols);
  return (int)std::max(8LL, ceil_div(M, want));
}

template <bool BF>
void launch_act_back(const igc_ffn::ActBackArgs& e, bool glu, const igc_ffn::PadArgs& pads, dim3 grid, hipStream_t stream) {
  if (glu)
    hipLaunchKernelGGL((igc_ffn::act_back_kernel<BF, true>), grid, dim3(256), 0, stream, e, pads);
  else
    hipLaunchKernelGGL((igc_ffn::act_back_kernel<BF, false>), grid, dim3(256), 0, stream, e, pads);
}

// Both products in one launch, or each in its own: whichever is estimated
// to be faster.  True for one launch (on one tile).
bool plan_back(Plan& px, Plan& pw, long long M, long long K, long long red, bool sums, int cus) {
  float best = px.us + pw.us + (sums ? 3.0f : 0.0f);
  bool joint = false;
  for (int v = P_TILE_256; v <= P_TILE_64; ++v) {
    const TileCost& c = tile_cost(igc_ffn::M_DX, v);
    const int places = tile_places(igc_ffn::M_DX, v);
    const Plan sx = best_split(igc_ffn::M_DX, v, M, K, red, cus, true), sw = best_split(igc_ffn::M_DW, v, red, K, M, cus, true);
    for (int i = 0; i < 4; ++i) {
      if (((i & 1) && sx.splits == 1) || ((i & 2) && sw.splits == 1)) continue;
      const Plan x = i & 1 ? sx : tile_plan(igc_ffn::M_DX, v, M, K), w = i & 2 ? sw : tile_plan(igc_ffn::M_DW, v, red, K);
      // (the second product starts at a multiple of 8 workgroups; a whole
      // round must not run over by those that keep it there)
      const long long cx = ceil_div(workgroups(x), 8) * 8, cw = ceil_div(workgroups(w), 8) * 8;
      // K tiles in all and of the longest workgroup
      const float kx = (float)k_tiles(red) * (float)x.tiles_m * (float)x.tiles_n, kw = (float)k_tiles(M) * (float)w.tiles_m * (float)w.tiles_n;
      const float nx = (float)k_tiles(red) / (float)(x.whole ? 1 : x.splits), nw = (float)k_tiles(M) / (float)(w.whole ? 1 : w.splits);
      // (the longer ones come first: more than run at once take what the
      // average does, or as long as the longest)
      const float most = std::max(nx, nw), mean = (kx + kw) / (float)(cx + cw);
      const bool several = cx + cw > (long long)places * cus;
      const float run = rounds_us(c, places, several ? mean : most, cx + cw, cus);
      const float us = c.launch + std::max(run, most * c.k1 + c.out) + join_us(c, x) + join_us(c, w);
      if (us < best) {
        best = us;
        joint = true;
        px = x;
        pw = w;
      }
    }
  }
  return joint;
}

int backward(const Backward& b, size_t* query, hipStream_t stream) {
  const bool sums = b.db || b.db2;
  const int np = b.glu ? 2 : 1;
  const int width = (int)ceil_div(b.N, 64) * 64;
  int dev;
  if (int s = check_device(&dev)) return s;
  const int cus = device_cus(dev);

  const bool want_x = b.dX && b.M > 0 && b.K > 0, want_w = (b.dW || b.dW2) && b.N > 0 && b.K > 0;
  const bool act = b.glu || b.act != IGC_ACT_NONE;
  // What the direct loads take as it is.  D made here is padded with zeros
  // to `width` columns.  (The two weights of the gated block take turns
  // under one set of lane offsets, so they need one leading dimension.)
  const bool d_fits = (long long)np * width <= (1 << 21) - 8;
  bool make_d = act && (want_x || want_w);
  bool d_ok = make_d ? d_fits : dma_operand(b.dY, b.lddy, b.N);
  bool w_ok = dma_operand(b.W, b.ldw, b.K) && (!b.glu || (dma_operand(b.W2, b.ldw2, b.K) && b.ldw == b.ldw2));
  bool x_ok = dma_operand(b.X, b.ldx, b.K);
  auto red = [&]() { return make_d ? np * width : b.N; };  // columns of D

  // Operands of another alignment are copied into padded rows, by the launch
  // that makes D if there is one.  (Down the rows, loads of any alignment wait
  // longest: dW of 72 x 601 x 400 9.2 us without and 9.0 with the copy,
  // 600 x 1001 x 1000 25.6 and 12.7, 727 x 1345 x 6130 285 and 38.)
  Pads pads;
  int iw = -1, iw2 = -1, ix = -1;
  const bool fix_x = want_x && !(d_ok && w_ok), fix_w = want_w && !(d_ok && x_ok);
  if ((fix_x || fix_w) && b.M > 0 && b.N > 0 && d_fits) {
    if (want_x && !w_ok) {
      iw = pads.add(b.W, b.ldw, b.N, b.K);
      if (b.glu) iw2 = pads.add(b.W2, b.ldw2, b.N, b.K);
    }
    if (want_w && !x_ok) ix = pads.add(b.X, b.ldx, b.M, b.K);
    if (pads.possible) {
      make_d = make_d || !d_ok;
      d_ok = w_ok = x_ok = true;
    } else {
      pads = Pads();
      iw = iw2 = ix = -1;
    }
  }
  Plan px = make_plan(igc_ffn::M_DX, b.M, b.K, red(), d_ok && w_ok ? 16 : 2, cus, true);
  Plan pw = make_plan(igc_ffn::M_DW, red(), b.K, b.M, d_ok && x_ok ? 16 : 2, cus, true);
  const bool joint = want_x && want_w && d_ok && w_ok && x_ok && plan_back(px, pw, b.M, b.K, red(), sums, cus);

  // workspace: D, column sums, D's largest elements and scale, padded operands, partial tiles
  const int rows = act_rows(b.M, std::max(width, 1), cus);
  const int blocks = (int)ceil_div(b.M, rows);
  const size_t d_bytes = make_d ? round256((size_t)b.M * np * width * 2) : 0;
  const size_t s_bytes = sums ? round256((size_t)blocks * np * width * 4) : 0;
  const size_t x_part = want_x ? round256(px.part_bytes) : 0, w_part = want_w ? round256(pw.part_bytes) : 0;
  const size_t part = joint ? x_part + w_part : std::max(x_part, w_part);
  const bool element = (make_d || sums) && b.M > 0 && b.N > 0;
  // (relu's D is dY or 0: fp16 holds it as it is)
  const bool scaled = b.type == IGC_F16 && (b.glu || (act && b.act != IGC_ACT_RELU)) && make_d && element;
  const long long act_blocks = ceil_div(width, 512) * blocks;
  const size_t m_bytes = scaled ? round256((act_blocks + 1) * sizeof(float)) : 0;
  const size_t need = d_bytes + s_bytes + m_bytes + pads.bytes + part;
  if (query) {
    *query = need;
    return IGC_OK;
  }
  if (int s = check_ws(b.ws, b.ws_bytes, need, true)) return s;
  uint8_t* const ws = static_cast<uint8_t*>(b.ws);
  uint8_t* const D = make_d ? ws : nullptr;
  float* const part_sums = sums ? reinterpret_cast<float*>(ws + d_bytes) : nullptr;
  float* const most = scaled ? reinterpret_cast<float*>(ws + d_bytes + s_bytes) : nullptr;
  uint8_t* const padded = ws + d_bytes + s_bytes + m_bytes;
  uint8_t* const parts = padded + pads.bytes;

  const void *W = b.W, *W2 = b.W2, *X = b.X;
  long long ldw = b.ldw, ldw2 = b.ldw2, ldx = b.ldx;
  if (iw >= 0) W = pads.place(iw, padded), ldw = Pads::padded(b.K);
  if (iw2 >= 0) W2 = pads.place(iw2, padded), ldw2 = Pads::padded(b.K);
  if (ix >= 0) X = pads.place(ix, padded), ldx = Pads::padded(b.K);
  if (element) {
    igc_ffn::ActBackArgs e;
    std::memset(&e, 0, sizeof(e));
    e.M = b.M;
    e.N = b.N;
    e.dY = static_cast<const uint8_t*>(b.dY);
    e.lddy = b.lddy;
    if (act) {
      e.Z = static_cast<const uint8_t*>(b.Z);
      e.ldz = b.ldz;
    }
    e.U = static_cast<const uint8_t*>(b.U);
    e.ldu = b.ldu;
    e.act = b.act;
    e.D = D;
    e.ldd = (long long)np * width;
    e.width = width;
    e.sums = part_sums;
    e.rows = rows;
    e.groups = (int)ceil_div(width, 512);
    e.blocks = blocks;
    const long long grid = act_blocks + pads.groups();
    if (grid > 0x7fffffffLL) return fail(IGC_EUNSUPPORTED, "too many workgroups (%lld)", grid);
    if (scaled) {
      e.most = most;
      e.undo = most + act_blocks;
    }
    if (b.type == IGC_BF16)
      launch_act_back<true>(e, b.glu, pads.args, dim3((unsigned)grid), stream);
    else
      launch_act_back<false>(e, b.glu, pads.args, dim3((unsigned)grid), stream);
    if (int s = launch_status()) return s;
    if (scaled) {
      const dim3 again((unsigned)std::min(act_blocks, 2LL * cus));
      if (b.glu)
        hipLaunchKernelGGL((igc_ffn::act_again_kernel<true>), again, dim3(256), 0, stream, e);
      else
        hipLaunchKernelGGL((igc_ffn::act_again_kernel<false>), again, dim3(256), 0, stream, e);
      if (int s = launch_status()) return s;
    }
  } else if (pads.groups() > 0) {
    hipLaunchKernelGGL((igc_ffn::pad_kernel<0>), dim3((unsigned)pads.groups()), dim3(256), 0, stream, pads.args);
    if (int s = launch_status()) return s;
  }
  const igc_ffn::ColsumArgs cs{part_sums, blocks, sums && b.N > 0 ? np : 0, width, b.N, b.db, b.db2};
  if (cs.which_n && !joint) {
    hipLaunchKernelGGL((igc_ffn::colsum_kernel<0>), dim3((unsigned)colsum_groups(cs)), dim3(256), 0, stream, cs);
    if (int s = launch_status()) return s;
  }
  const void* const A = make_d ? D : b.dY;
  const long long lda = make_d ? (long long)np * width : b.lddy;
  GemmArgs ax = product(b.M, b.K, red(), A, lda, W, ldw, b.dX, b.lddx);
  ax.b_rows = b.N;
  ax.undo = scaled ? most + act_blocks : nullptr;
  GemmArgs aw = product(red(), b.K, b.M, A, lda, X, ldx, b.dW, b.lddw);
  aw.m_rows = b.N;
  aw.undo = ax.undo;
  if (b.glu) {
    ax.B2 = static_cast<const uint8_t*>(W2);
    ax.ldb2 = ldw2;
    ax.r_split = width;
    aw.Y2 = static_cast<uint8_t*>(b.dW2);
    aw.ldy2 = b.lddw2;
    aw.m_split = width;
  }
  if (joint) {
    apply_plan(ax, px, parts);
    apply_plan(aw, pw, parts + x_part);
    return b.type == IGC_BF16 ? launch_back<true>(ax, px, aw, pw, cs, stream) : launch_back<false>(ax, px, aw, pw, cs, stream);
  }
  if (want_x)
    if (int s = run_product<igc_ffn::M_DX>(ax, px, b.type, parts, stream)) return s;
  if (want_w)
    if (int s = run_product<igc_ffn::M_DW>(aw, pw, b.type, parts, stream)) return s;
  return IGC_OK;
}

int linear_backward_impl(const igc_linear_backward* d, size_t* query, hipStream_t stream) {
  Checker c;
  c.fail_if(!d, "descriptor is NULL");
  if (!c.ok()) return c.status;
  c.problem(d->M, d->N, d->K, d->type, d->act);
  c.fail_if(!d->dX && !d->dW && !d->dbias, "no output requested");
  c.matrix("dY", d->dY, d->lddy, d->M, d->N, 2, false);
  if (d->act != IGC_ACT_NONE) c.matrix("Z", d->Z, d->ldz, d->M, d->N, 2, false);
  if (d->dX) c.matrix("W", d->W, d->ldw, d->M > 0 ? d->N : 0, d->K, 2, false);
  if (d->dW) c.matrix("X", d->X, d->ldx, d->N > 0 ? d->M : 0, d->K, 2, false);
  c.matrix("dX", d->dX, d->lddx, d->M, d->K, 2, true);
  c.matrix("dW", d->dW, d->lddw, d->N, d->K, 2, true);
  c.vector("dbias", d->dbias);
  if (!c.ok()) return c.status;
  Backward b{d->M,  d->N,   d->K,  d->type, d->act, false,  d->dY,   d->Z,    nullptr,  d->X,     d->W,    nullptr,      d->lddy,    d->ldz,
             0,     d->ldx, d->ldw, 0,      d->dX,  d->dW,  nullptr, d->lddx, d->lddw, 0,        d->dbias, nullptr, d->workspace, d->ws_bytes};
  return backward(b, query, stream);
}

int glu_backward_impl(const igc_glu_backward* d, size_t* query, hipStream_t stream) {
  Checker c;
  c.fail_if(!d, "descriptor is NULL");
  if (!c.ok()) return c.status;
  c.problem(d->M, d->N, d->K, d->type, d->act);
  c.extent("N", d->N, Checker::MOST / 2);  // (dG and dU lie side by side)
  c.fail_if(!d->dX && !d->dWg && !d->dWu && !d->dbias_g && !d->dbias_u, "no output requested");
  c.matrix("dH", d->dH, d->lddh, d->M, d->N, 2, false);
  c.matrix("G", d->G, d->ldg, d->M, d->N, 2, false);
  c.matrix("U", d->U, d->ldu, d->M, d->N, 2, false);
  if (d->dX) {
    c.matrix("Wg", d->Wg, d->ldwg, d->M > 0 ? d->N : 0, d->K, 2, false);
    c.matrix("Wu", d->Wu, d->ldwu, d->M > 0 ? d->N : 0, d->K, 2, false);
  }
  if (d->dWg || d->dWu) c.matrix("X", d->X, d->ldx, d->N > 0 ? d->M : 0, d->K, 2, false);
  c.matrix("dX", d->dX, d->lddx, d->M, d->K, 2, true);
  c.matrix("dWg", d->dWg, d->lddwg, d->N, d->K, 2, true);
  c.matrix("dWu", d->dWu, d->lddwu, d->N, d->K, 2, true);
  c.vector("dbias_g", d->dbias_g);
  c.vector("dbias_u", d->dbias_u);
  if (!c.ok()) return c.status;
  Backward b{d->M,    d->N,   d->K,    d->type,  d->act, true,   d->dH,  d->G,    d->U,     d->X,       d->Wg,      d->Wu,        d->lddh,     d->ldg,
             d->ldu,  d->ldx, d->ldwg, d->ldwu,  d->dX,  d->dWg, d->dWu, d->lddx, d->lddwg, d->lddwu,   d->dbias_g, d->dbias_u,   d->workspace, d->ws_bytes};
  return backward(b, query, stream);
}

// ---------------------------------------------------------------- clipping
int grad_clip_impl(const igc_grad_clip* d, size_t* query, hipStream_t stream) {
  Checker c;
  c.fail_if(!d, "descriptor is NULL");
  if (!c.ok()) return c.status;
  c.fail_if(d->count < 0, "negative count");
  c.fail_if(d->max_norm < 0, "negative max_norm");
  c.fail_if(!d->norm, "norm is NULL");
  c.vector("norm", d->norm);
  c.fail_if(d->count > 0 && (!d->grads || !d->sizes || !d->types), "grads, sizes or types is NULL");
  for (int i = 0; c.ok() && i < d->count; ++i) {
    c.fail_if(d->sizes[i] < 0, "negative tensor size");
    c.fail_if(d->types[i] != IGC_F16 && d->types[i] != IGC_BF16 && d->types[i] != IGC_F32, "unknown tensor type");
    c.fail_if(d->sizes[i] > (1LL << 43), "tensor too large");
    if (!c.ok() || d->sizes[i] == 0) continue;
    const uintptr_t mask = d->types[i] == IGC_F32 ? 3 : 1;
    const void* const out = d->outs ? d->outs[i] : d->grads[i];
    c.fail_if(!d->grads[i] || !out, "a tensor is NULL");
    c.fail_if(((reinterpret_cast<uintptr_t>(d->grads[i]) | reinterpret_cast<uintptr_t>(out)) & mask) != 0, "a tensor is misaligned");
  }
  if (!c.ok()) return c.status;

  // tensors per launch, and each launch's slots for its partial sums
  using namespace igc_ffn;
  const int launches = std::max(1, (int)ceil_div(d->count, CLIP_TENSORS));
  auto fill = [&](int l, ClipTable& t) -> int {  // returns the launch's workgroups
    t.count = std::min(CLIP_TENSORS, d->count - l * CLIP_TENSORS);
    long long chunks = 0;
    for (int i = 0; i < t.count; ++i) {
      const int g = l * CLIP_TENSORS + i;
      t.in[i] = static_cast<const uint8_t*>(d->grads[g]);
      t.out[i] = d->outs ? static_cast<uint8_t*>(d->outs[g]) : static_cast<uint8_t*>(const_cast<void*>(d->grads[g]));
      t.size[i] = d->sizes[g];
      t.type[i] = (uint8_t)d->types[g];
      t.first[i] = (int)std::min(chunks, 0x7fffffffLL);
      chunks += ceil_div(d->sizes[g], CLIP_CHUNK);
    }
    if (chunks > 0x7fffffffLL - CLIP_GRID) return -1;
    t.first[t.count] = (int)chunks;
    return (int)std::min<long long>(chunks, CLIP_GRID);
  };
  const size_t need = (size_t)launches * CLIP_GRID * sizeof(double);
  if (query) {
    *query = need;
    return IGC_OK;
  }
  int dev;
  if (int s = check_device(&dev)) return s;
  if (int s = check_ws(d->workspace, d->ws_bytes, need, true)) return s;
  ClipTable t;
  std::memset(&t, 0, sizeof(t));
  t.part = static_cast<double*>(d->workspace);
  t.max_norm = d->max_norm;
  int slots = 0;
  for (int l = 0; l < launches; ++l)
    if (fill(l, t) < 0) return fail(IGC_EUNSUPPORTED, "too many elements");
  for (int l = 0; l < launches; ++l) {
    const int grid = fill(l, t);
    t.partials = slots;
    if (grid > 0) hipLaunchKernelGGL((clip_norm_kernel<0>), dim3(grid), dim3(256), 0, stream, t);
    slots += grid;
  }
  t.partials = slots;
  for (int l = 0; l < launches; ++l) {
    const int grid = fill(l, t);
    t.norm = l == 0 ? d->norm : nullptr;
    if (grid > 0 || l == 0) hipLaunchKernelGGL((clip_scale_kernel<0>), dim3(std::max(grid, 1)), dim3(256), 0, stream, t);
  }
  return launch_status();
}

// No C++ exception leaves the C entries: nothing below throws (no
// allocation, no container).
}  // namespace igc_ffn_host

extern "C" {

using namespace igc_ffn_host;

#define IGC_FFN_ENTRY(name)                                                                          \
  int name(const igc_##name* d, void* stream) {                                                      \
    return name##_impl(d, nullptr, static_cast<hipStream_t>(stream));                                \
  }                                                                                                  \
  int name##_workspace_size(const igc_##name* d, size_t* bytes) {                                    \
    if (!bytes) return fail(IGC_EINVAL, "bytes is NULL");                                            \
    return name##_impl(d, bytes, nullptr);                                                           \
  }

IGC_FFN_ENTRY(linear_forward)
IGC_FFN_ENTRY(linear_backward)
IGC_FFN_ENTRY(glu_forward)
IGC_FFN_ENTRY(glu_backward)
IGC_FFN_ENTRY(grad_clip)

}  // extern "C"
