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
  a.tiles_m = pl.tiles_m;
  a.tiles_n = pl.tiles_n;
  a.splits = pl.splits;
  a.part = reinterpret_cast<float*>(part);
}

template <int MODE>
int run_product(GemmArgs& a, const Plan& pl, int type, uint8_t* part, hipStream_t stream) {
  apply_plan(a, pl, part);
  return type == IGC_BF16 ? launch_product<true, MODE>(a, pl, stream) : launch_product<false, MODE>(a, pl, stream);
}

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
  const bool aligned = dma_operand(a.A, a.lda, a.R) && dma_operand(a.B, a.ldb, a.R) &&
                       (MODE != igc_ffn::M_GLU || dma_operand(a.B2, a.ldb2, a.R));
  const Plan pl = make_plan(MODE, a.M, a.N, a.R, aligned, cus, query || ws);
  const size_t need = pl.part_bytes;
  if (query) {
    *query = need;
    return IGC_OK;
  }
  if (int s = check_ws(ws, ws_bytes, need, false)) return s;
  return run_product<MODE>(a, pl, type, static_cast<uint8_t*>(ws), stream);
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
void launch_act_back(const igc_ffn::ActBackArgs& e, bool glu, dim3 grid, hipStream_t stream) {
  if (glu)
    hipLaunchKernelGGL((igc_ffn::act_back_kernel<BF, true>), grid, dim3(256), 0, stream, e);
  else
    hipLaunchKernelGGL((igc_ffn::act_back_kernel<BF, false>), grid, dim3(256), 0, stream, e);
}

int backward(const Backward& b, size_t* query, hipStream_t stream) {
  const bool products = b.dX || b.dW || b.dW2;
  const bool sums = b.db || b.db2;
  const bool make_d = products && (b.glu || b.act != IGC_ACT_NONE);
  const int np = b.glu ? 2 : 1;
  const int width = (int)std::min<long long>(ceil_div(b.N, 64) * 64, 0x7fffffc0);
  if (b.glu && width > (1 << 30)) return fail(IGC_EUNSUPPORTED, "N too large");
  int dev;
  if (int s = check_device(&dev)) return s;
  const int cus = device_cus(dev);

  // workspace: D, column sums, partial tiles
  const int rows = act_rows(b.M, std::max(width, 1), cus);
  const int blocks = (int)ceil_div(b.M, rows);
  const size_t d_bytes = make_d ? round256((size_t)b.M * np * width * 2) : 0;
  const size_t s_bytes = sums ? round256((size_t)blocks * np * width * 4) : 0;
  // D made here is padded with zeros to `width` columns
  const int red = make_d ? np * width : b.N;
  // (the two weights of the gated block take turns under one set of lane
  // offsets, so the direct loads need one leading dimension for both)
  const bool d_ok = make_d ? (long long)np * width <= (1 << 21) - 8 : dma_operand(b.dY, b.lddy, b.N);
  const bool x_ok = d_ok && dma_operand(b.W, b.ldw, b.K) && (!b.glu || (dma_operand(b.W2, b.ldw2, b.K) && b.ldw == b.ldw2));
  const Plan px = make_plan(igc_ffn::M_DX, b.M, b.K, red, x_ok, cus, true);
  const Plan pw = make_plan(igc_ffn::M_DW, red, b.K, b.M, d_ok && dma_operand(b.X, b.ldx, b.K), cus, true);
  // one launch for both where they want the same tile
  const bool want_x = b.dX && b.M > 0 && b.K > 0, want_w = (b.dW || b.dW2) && b.N > 0 && b.K > 0;
  const bool joint = want_x && want_w && px.variant == pw.variant && px.variant <= P_TILE_64;
  const size_t x_part = want_x ? round256(px.part_bytes) : 0, w_part = want_w ? round256(pw.part_bytes) : 0;
  const size_t part = joint ? x_part + w_part : std::max(x_part, w_part);
  const size_t need = d_bytes + s_bytes + part;
  if (query) {
    *query = need;
    return IGC_OK;
  }
  if (int s = check_ws(b.ws, b.ws_bytes, need, true)) return s;
  uint8_t* const ws = static_cast<uint8_t*>(b.ws);
  uint8_t* const D = make_d ? ws : nullptr;
  float* const part_sums = sums ? reinterpret_cast<float*>(ws + d_bytes) : nullptr;
  uint8_t* const parts = ws + d_bytes + s_bytes;

  if ((make_d || sums) && b.M > 0 && b.N > 0) {
    igc_ffn::ActBackArgs e;
    std::memset(&e, 0, sizeof(e));
    e.M = b.M;
    e.N = b.N;
    e.dY = static_cast<const uint8_t*>(b.dY);
    e.lddy = b.lddy;
    if (b.glu || b.act != IGC_ACT_NONE) {
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
    const dim3 grid((unsigned)ceil_div(width, 512), (unsigned)blocks);
    if (b.type == IGC_BF16)
      launch_act_back<true>(e, b.glu, grid, stream);
    else
      launch_act_back<false>(e, b.glu, grid, stream);
    if (int s = launch_status()) return s;
  }
  const igc_ffn::ColsumArgs cs{part_sums, blocks, sums && b.N > 0 ? np : 0, width, b.N, b.db, b.db2};
  if (cs.which_n && !joint) {
    hipLaunchKernelGGL((igc_ffn::colsum_kernel<0>), dim3((unsigned)colsum_groups(cs)), dim3(256), 0, stream, cs);
    if (int s = launch_status()) return s;
  }
  const void* const A = make_d ? D : b.dY;
  const long long lda = make_d ? (long long)np * width : b.lddy;
  GemmArgs ax = product(b.M, b.K, red, A, lda, b.W, b.ldw, b.dX, b.lddx);
  ax.b_rows = b.N;
  GemmArgs aw = product(red, b.K, b.M, A, lda, b.X, b.ldx, b.dW, b.lddw);
  aw.m_rows = b.N;
  if (b.glu) {
    ax.B2 = static_cast<const uint8_t*>(b.W2);
    ax.ldb2 = b.ldw2;
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
