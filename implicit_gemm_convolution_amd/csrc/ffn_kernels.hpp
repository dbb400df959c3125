// ffn_kernels.hpp -- the feed-forward operators on gfx950: 16-bit (fp16 or
// bf16) matrix products with fused epilogues, the element-wise part of their
// backward passes, and gradient clipping.
//
//   linear   Z = X W^T + b;  Y = act(Z) + R
//   glu      G = X Wg^T + bg;  U = X Wu^T + bu;  H = act(G) * U
//   back     D = dY act'(Z);  dX = D W;  dW = D^T X;  db = sum over rows of D
//            dG = dH U act'(G), dU = dH act(G);  dX = dG Wg + dU Wu; ...
//   clip     norm = sqrt(sum g^2);  out = g min(1, max_norm / (norm + 1e-6))
//
// Every product accumulates in fp32 on the 16x16x32 matrix instructions, and
// bias, activation and residual are applied to the fp32 sums: one rounding,
// at the store.  db sums fp32 values.  The backward products take D rounded to
// the operands' type, which is what the matrix cores multiply; in fp32 D would
// take them two products for one.  Each term is then off by up to half a step
// of that type relative to itself, independently of the others, so relative to
// its size a sum is off by about as much as its own final rounding, whatever
// its length: the error of dX and dW is that of unrounded D times the square
// root of 2 (bf16 2.3e-3 for 1.7e-3).  bf16 has the range of fp32.  In fp16 D
// could leave the range although every input and every gradient is inside it,
// so D is scaled by a power of two, which the epilogue takes back: both exact.
// act_back_kernel has the scales.
#pragma once

#include "igc_kernels.hpp"

namespace igc_ffn {

using igc::CHUNK_BYTES;
using igc::Rsrc;
using igc::f32x4;
using igc::lds_barrier;
using igc::lds_read16;
using igc::lds_write16;
using igc::make_rsrc;
using igc::static_for;
using igc::swz;
using igc::wait_vmcnt_lgkm0;
using igc::wave_id;

// ---------------------------------------------------------------------------
// Element types.
// ---------------------------------------------------------------------------
enum Type : int { T_F16 = 0, T_BF16 = 1, T_F32 = 2 };
enum Act : int { ACT_NONE = 0, ACT_RELU = 1, ACT_GELU = 2, ACT_GELU_TANH = 3, ACT_SILU = 4, ACT_SIGMOID = 5 };

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

template <bool BF>
__device__ __forceinline__ void unpack2(uint32_t v, float& a, float& b) {
  if constexpr (BF) {
    a = __builtin_bit_cast(float, v << 16);
    b = __builtin_bit_cast(float, v & 0xffff0000u);
  } else {
    const f16x2 h = __builtin_bit_cast(f16x2, v);
    a = (float)h[0];
    b = (float)h[1];
  }
}
template <bool BF>
__device__ __forceinline__ uint32_t pack2(float a, float b) {  // round to nearest even
  if constexpr (BF) {
    bf16x2 h;
    h[0] = (__bf16)a;
    h[1] = (__bf16)b;
    return __builtin_bit_cast(uint32_t, h);
  } else {
    f16x2 h;
    h[0] = (_Float16)a;
    h[1] = (_Float16)b;
    return __builtin_bit_cast(uint32_t, h);
  }
}
template <bool BF>
__device__ __forceinline__ void unpack8(const uint4& v, float (&f)[8]) {
  unpack2<BF>(v.x, f[0], f[1]);
  unpack2<BF>(v.y, f[2], f[3]);
  unpack2<BF>(v.z, f[4], f[5]);
  unpack2<BF>(v.w, f[6], f[7]);
}
template <bool BF>
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  return make_uint4(pack2<BF>(f[0], f[1]), pack2<BF>(f[2], f[3]), pack2<BF>(f[4], f[5]), pack2<BF>(f[6], f[7]));
}

// Eight 16-bit elements from any 2-byte aligned address; elements past
// `valid` read as zero and are not touched.  (The GPU takes 16-byte loads at
// any address.)
__device__ __forceinline__ uint4 load8(const uint8_t* p, int valid) {
  uint4 v = make_uint4(0, 0, 0, 0);
  if (valid >= 8) {
    __builtin_memcpy(&v, p, 16);
  } else if (valid > 0) {
    const uint16_t* const q = reinterpret_cast<const uint16_t*>(p);
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (e < valid) w[e / 2] |= (uint32_t)q[e] << (16 * (e & 1));
    v = make_uint4(w[0], w[1], w[2], w[3]);
  }
  return v;
}
__device__ __forceinline__ void store8(uint8_t* p, const uint4& v, int valid) {
  if (valid >= 8) {
    __builtin_memcpy(p, &v, 16);
  } else {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint16_t* const q = reinterpret_cast<uint16_t*>(p);
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (e < valid) q[e] = (uint16_t)(w[e / 2] >> (16 * (e & 1)));
  }
}

// Eight 16-bit elements from any 2-byte aligned address by loads of aligned
// words, which the GPU takes several times as fast as a 16-byte load across
// them.  Reads no word that holds none of the eight.
__device__ __forceinline__ uint4 load8_words(const uint8_t* p) {
  const uint32_t odd = (uint32_t)(uintptr_t)p & 2;
  const uint8_t* const q = p - odd;
  uint4 v;
  uint32_t last;
  __builtin_memcpy(&v, __builtin_assume_aligned(q, 4), 16);
  __builtin_memcpy(&last, __builtin_assume_aligned(q + 12 + 2 * odd, 4), 4);  // (an even address: v.w again)
  const uint32_t bits = odd * 8;
  return make_uint4(__builtin_amdgcn_alignbit(v.y, v.x, bits), __builtin_amdgcn_alignbit(v.z, v.y, bits),
                    __builtin_amdgcn_alignbit(v.w, v.z, bits), __builtin_amdgcn_alignbit(last, v.w, bits));
}

// V (4 or 8) 16-bit or fp32 elements as fp32 values, from and to any address;
// those past `valid` are left alone.
template <bool BF, int V>
__device__ __forceinline__ void load_n(const uint8_t* p, int valid, float (&f)[V]) {
  if constexpr (V == 8) {
    unpack8<BF>(load8(p, valid), f);
  } else {
    uint32_t w[2] = {0, 0};
    if (valid >= 4) {
      __builtin_memcpy(w, p, 8);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (e < valid) w[e / 2] |= (uint32_t)reinterpret_cast<const uint16_t*>(p)[e] << (16 * (e & 1));
    }
    unpack2<BF>(w[0], f[0], f[1]);
    unpack2<BF>(w[1], f[2], f[3]);
  }
}
template <bool BF, int V>
__device__ __forceinline__ void store_n(uint8_t* p, int valid, const float (&f)[V]) {
  if constexpr (V == 8) {
    store8(p, pack8<BF>(f), valid);
  } else {
    const uint32_t w[2] = {pack2<BF>(f[0], f[1]), pack2<BF>(f[2], f[3])};
    if (valid >= 4) {
      __builtin_memcpy(p, w, 8);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (e < valid) reinterpret_cast<uint16_t*>(p)[e] = (uint16_t)(w[e / 2] >> (16 * (e & 1)));
    }
  }
}
template <int V>
__device__ __forceinline__ void load_f32(const float* p, int valid, float (&f)[V]) {
  if (valid >= V) {
    __builtin_memcpy(f, p, 4 * V);
  } else {
#pragma unroll
    for (int e = 0; e < V; ++e) f[e] = e < valid ? p[e] : 0.0f;
  }
}
template <int V>
__device__ __forceinline__ void store_f32(float* p, int valid, const float (&f)[V]) {
  if (valid >= V) {
    __builtin_memcpy(p, f, 4 * V);
  } else {
#pragma unroll
    for (int e = 0; e < V; ++e)
      if (e < valid) p[e] = f[e];
  }
}

// ---------------------------------------------------------------------------
// Activations, in fp32.
// ---------------------------------------------------------------------------
// (exp2's argument is rounded: relative error about |x| 2^-24)
__device__ __forceinline__ float exp_f(float x) { return __builtin_amdgcn_exp2f(x * 1.44269504088896341f); }
// 1 / (1 + exp(-z)); exp overflowing to infinity gives 0
__device__ __forceinline__ float sigmoid_f(float z) { return __builtin_amdgcn_rcpf(1.0f + exp_f(-z)); }
// The normal distribution function of z and e = exp(-z^2 / 2):
// erfc(x) = exp(-x^2) t P(t), t = 1 / (1 + x/2), x = |z| / sqrt 2: the
// substitution of the published fits of erfc (Numerical Recipes has one by
// Chebyshev polynomials), with P a least-squares fit of exp(x^2) erfc(x) / t
// made for this file (relative error 4e-8, about 4e-7 evaluated in fp32).  The
// exponent is rounded twice, so the tail's relative error grows with it: at
// most (20 + 1.2 z^2) 2^-24, which is 3e-6 at z = -5 and 1.3e-5 at z = -13,
// far below half a step of a 16-bit output.
__device__ __forceinline__ float normal_cdf(float z, float& e) {
  const float x = __builtin_fabsf(z) * 0.70710678118654752f;
  const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(0.5f, x, 1.0f));
  e = exp_f(-0.5f * z * z);
  float q = -0.05781668414637441f;
  q = __builtin_fmaf(q, t, 0.27839578762714456f);
  q = __builtin_fmaf(q, t, -0.47423681396851763f);
  q = __builtin_fmaf(q, t, 0.26300854998394246f);
  q = __builtin_fmaf(q, t, -0.01606377351405429f);
  q = __builtin_fmaf(q, t, 0.1981216336858939f);
  q = __builtin_fmaf(q, t, 0.2442873611701233f);
  q = __builtin_fmaf(q, t, 0.2822075600438619f);
  q = __builtin_fmaf(q, t, 0.28209634074354567f);
  const float tail = 0.5f * e * t * q;  // erfc(x) / 2
  return z > 0.0f ? 1.0f - tail : tail;
}
constexpr float kGeluC = 0.79788456080286536f;  // sqrt(2 / pi)
constexpr float kGeluA = 0.044715f;

// f(z) and, with SLOPE, f'(z).  (gelu_tanh: (1 + tanh a) / 2 = sigmoid(2a).)
template <int ACT, bool SLOPE>
__device__ __forceinline__ void act_one(float z, float& f, float& d) {
  if constexpr (ACT == ACT_NONE) {
    f = z;
    if constexpr (SLOPE) d = 1.0f;
  } else if constexpr (ACT == ACT_RELU) {
    f = z < 0.0f ? 0.0f : z;  // (NaN stays NaN)
    if constexpr (SLOPE) d = z > 0.0f ? 1.0f : 0.0f;
  } else if constexpr (ACT == ACT_GELU) {
    float e;
    const float c = normal_cdf(z, e);
    f = z * c;
    if constexpr (SLOPE) d = __builtin_fmaf(z * 0.39894228040143268f, e, c);
  } else if constexpr (ACT == ACT_GELU_TANH) {
    // (the sigmoid's exponent -2a log2(e), its constants folded)
    const float z2 = z * z;
    const float w = __builtin_fmaf(z2, -2.0f * kGeluC * kGeluA * 1.44269504088896341f, -2.0f * kGeluC * 1.44269504088896341f);
    const float s = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(z * w));
    f = z * s;
    // (s is 0 or 1 long before z2 could overflow: 0 times infinity)
    if constexpr (SLOPE) d = s + f * (1.0f - s) * (2.0f * kGeluC) * __builtin_fmaf(3.0f * kGeluA, __builtin_fminf(z2, 1e30f), 1.0f);
  } else {
    const float s = sigmoid_f(z);
    if constexpr (ACT == ACT_SILU) {
      f = z * s;
      if constexpr (SLOPE) d = __builtin_fmaf(f, 1.0f - s, s);
    } else {
      f = s;
      if constexpr (SLOPE) d = s * (1.0f - s);
    }
  }
}
template <int ACT, bool SLOPE, int N>
__device__ __forceinline__ void act_all(const float (&z)[N], float (&f)[N], float (&d)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) act_one<ACT, SLOPE>(z[i], f[i], d[i]);
}
// the activation is a wave-uniform value: one scalar branch per N elements
template <bool SLOPE, int N>
__device__ __forceinline__ void act_n(int act, const float (&z)[N], float (&f)[N], float (&d)[N]) {
  switch (act) {
    case ACT_RELU: return act_all<ACT_RELU, SLOPE>(z, f, d);
    case ACT_GELU: return act_all<ACT_GELU, SLOPE>(z, f, d);
    case ACT_GELU_TANH: return act_all<ACT_GELU_TANH, SLOPE>(z, f, d);
    case ACT_SILU: return act_all<ACT_SILU, SLOPE>(z, f, d);
    case ACT_SIGMOID: return act_all<ACT_SIGMOID, SLOPE>(z, f, d);
    default: return act_all<ACT_NONE, SLOPE>(z, f, d);
  }
}

// ---------------------------------------------------------------------------
// The matrix products.
// ---------------------------------------------------------------------------
// How the operands lie in memory.  ROW: the reduction runs along a row (one
// row per output row or column).  COL: the reduction runs down the rows.
//   FWD   out[m][n] = sum_k X[m][k] W[n][k]             A ROW, B ROW
//   GLU   the same with two B operands, side by side    A ROW, B ROW
//   DX    out[m][k] = sum_n D[m][n] W[n][k]             A ROW, B COL
//   DW    out[n][k] = sum_m D[m][n] X[m][k]             A COL, B COL
enum Mode : int { M_FWD = 0, M_GLU = 1, M_DX = 2, M_DW = 3 };

struct GemmArgs {
  int M, N, R;  // output rows, output columns (of each product), reduction
  const uint8_t *A, *B, *B2;
  long long lda, ldb, ldb2;  // elements
  // DX over two weights: reduction rows [0, b_rows) come from B and
  // [r_split, r_split + b_rows) from B2; r_split is a multiple of 64, and A
  // holds zeros between.  Without: r_split = b_rows = R.
  int r_split, b_rows;
  // epilogue
  int act;
  const float *bias, *bias2;
  const uint8_t* res;  // R, of Y's type
  long long ldr;
  uint8_t* Y;
  long long ldy;
  int y_f32;
  uint8_t *Z, *U;  // kept sums, of the operands' type
  long long ldz, ldu;
  // DW of two weights: output rows [0, m_rows) go to Y and
  // [m_split, m_split + m_rows) to Y2.  Without: m_split = m_rows = M.
  uint8_t* Y2;
  long long ldy2;
  int m_split, m_rows;
  int stream;  // the rows of every output are whole 128-byte lines: written past the caches
  const float* undo;  // (DX and DW of fp16) what takes D's scale back, or NULL
  // work split
  int tiles_m, tiles_n;
  int whole;    // tiles [0, whole) have a workgroup each
  int splits;   // workgroups that share the reduction of each tile after those
  int odd_rows; // (few rows) rows start at odd multiples of 2 bytes
  float* part;  // their partial tiles
};

template <bool BF>
__device__ __forceinline__ void mfma16(f32x4& c, const uint4& a, const uint4& b) {
  if constexpr (BF)
    c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  else
    c = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}

// An operand's K tile in LDS: W rows (or columns) x 64 reduction elements.
//  ROW: W rows of 128 bytes, chunk c of row r in slot c ^ ((r >> 1) & 7).
//  COL: 64 reduction rows of W elements.  Fragments are read with the
//  transposing LDS load: 16 lanes take a 4 x 16 block (4 reduction rows of
//  32 bytes) and each lane gets one column.  A half wave reads reduction rows
//  {0..3, 8..11} of one 32-byte granule: the granule index is XOR-ed with
//  those row bits, so the 8 pieces cover all 64 banks.
template <int W, bool COL>
struct LdsTile {
  static constexpr int BYTES = W * 128;
  static constexpr int ROWB = W * 2;  // COL: bytes per reduction row
  __device__ static __forceinline__ int gran(int kr) {  // COL: the granule XOR of reduction row kr
    if constexpr (W >= 128) return (kr & 3) | (((kr >> 3) & 1) << 2);
    if constexpr (W == 32) return (kr >> 3) & 1;
    return ((kr >> 1) & 1) | (((kr >> 3) & 1) << 1);
  }
  // byte offset of 16-byte chunk c of (ROW) row r / (COL) reduction row r
  __device__ static __forceinline__ int chunk_off(int r, int c) {
    if constexpr (!COL) return swz(r, c);
    return r * ROWB + (((c >> 1) ^ gran(r)) << 5) + (c & 1) * 16;
  }
  // fragment of rows (columns) blk0 .. blk0+15, k-step ks: lane l holds row
  // l % 16, reduction elements 32 ks + 8 (l / 16) .. +7
  __device__ static __forceinline__ uint4 frag(const uint8_t* st, int blk0, int ks) {
    const int lane = threadIdx.x & 63;
    if constexpr (!COL) {
      return lds_read16(st, swz(blk0 + (lane & 15), ks * 4 + (lane >> 4)));
    } else {
      const int i = lane & 15, g = lane >> 4;
      const int kr = 8 * g + (i >> 2);  // (bit 2 and the bits from 5 up do not enter gran())
      const int off = kr * ROWB + (((blk0 >> 4) ^ gran(kr)) << 5) + (i & 3) * 8;
      typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
      const uint8_t* const p = st + off + ks * 32 * ROWB;
      const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(p));
      const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(p + 4 * ROWB));
      const uint2 l2 = __builtin_bit_cast(uint2, lo), h2 = __builtin_bit_cast(uint2, hi);
      return make_uint4(l2.x, l2.y, h2.x, h2.y);
    }
  }
};

// Loading an operand's K tiles through registers, from rows of any
// alignment, stride and length.
template <int W, bool COL, bool TWO>
struct RegOperand {
  typedef LdsTile<W, COL> Tile;
  static constexpr int NC = W * 8 / 256;  // 16-byte chunks per thread
  const uint8_t *p, *p2;
  long long ld, ld2;  // bytes
  int o0, extent, R, r_split, r_rows;
  __device__ __forceinline__ void init(const uint8_t* ptr, long long l, const uint8_t* ptr2, long long l2, int o, int ext,
                                       int red, int split, int rows) {
    p = ptr;
    p2 = ptr2;
    ld = l * 2;
    ld2 = l2 * 2;
    o0 = o;
    extent = ext;
    R = red;
    r_split = split;
    r_rows = rows;
  }
  __device__ __forceinline__ void load(int kt, uint4 (&v)[NC]) const {
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      const int idx = threadIdx.x + 256 * j;
      if constexpr (!COL) {
        const int c = idx & 7, k = kt * 64 + c * 8;
        int row = idx >> 3;
        const bool second = TWO && row >= W / 2;
        if (second) row -= W / 2;
        const int o = o0 + row;
        const uint8_t* const q = (second ? p2 : p) + (long long)o * (second ? ld2 : ld) + (long long)k * 2;
        v[j] = load8(q, o < extent ? R - k : 0);
      } else {
        const int c = idx % (W / 8);
        int r = kt * 64 + idx / (W / 8);
        const int o = o0 + c * 8;
        const bool in = r < R;  // (without a second operand r_split is R: rows past it are no rows of p2)
        const bool second = TWO && r >= r_split;
        if (second) r -= r_split;
        const uint8_t* const q = (second ? p2 : p) + (long long)r * (second ? ld2 : ld) + (long long)o * 2;
        v[j] = load8(q, in && r < r_rows ? extent - o : 0);
      }
    }
  }
  __device__ __forceinline__ void store(uint8_t* st, const uint4 (&v)[NC]) const {
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      const int idx = threadIdx.x + 256 * j;
      lds_write16(st, COL ? Tile::chunk_off(idx / (W / 8), idx % (W / 8)) : Tile::chunk_off(idx >> 3, idx & 7), v[j]);
    }
  }
};

// Loading an operand's K tiles straight into LDS (no registers): 16-byte
// aligned rows whose length is a multiple of 8.  A wave instruction fills
// 1 KB of the tile; instruction i of wave w fills the KB 4 i + w.  Each lane
// fetches the chunk that belongs in its slot, so the swizzle costs nothing.
// Out of range reads as zeros: rows (columns) past the operand and reduction
// elements past R.
//  ROW: each load is one of the lane's fixed offsets plus a scalar offset
//  along the row; the lanes past R are moved out of range when the last K
//  tile comes up.
//  COL: the descriptor moves down the rows, with the rows that are left as
//  its size.  Columns go up to the next multiple of 8 (what a padded copy
//  holds as zeros; other operands have no more columns than that).
template <int W, bool COL, bool TWO>
struct DmaOperand {
  typedef LdsTile<W, COL> Tile;
  static constexpr int NQ = Tile::BYTES / 4096;  // instructions per wave and tile
  static constexpr uint32_t OUT = 0x80000000u;   // past every descriptor (they end below 2^30)
  uint32_t voff[NQ];
  Rsrc rs, rs2;
  uint32_t wofs;
  uint32_t soff;  // ROW: this tile's scalar offset
  int R, kend, nk;
  // COL
  const uint8_t *p, *p2;
  long long ldb;  // bytes
  int o0, extent, r_split, r_rows;

  __device__ __forceinline__ void init(const uint8_t* ptr, long long l, const uint8_t* ptr2, long long l2, int o, int ext,
                                       int red, int split, int rows, int k_end) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    wofs = (uint32_t)wave_id() * 1024u;
    R = red;
    kend = k_end;
    nk = max(1, (R + 63) / 64);
    if constexpr (!COL) {
      // (the two products of the gated block: half of the rows from each)
      constexpr int WR = TWO ? W / 2 : W;
      const int nrows = min(ext - o, WR);
      rs = make_rsrc(ptr + (long long)o * l * 2, (uint32_t)((long long)(nrows - 1) * l * 2 + R * 2));
      if constexpr (TWO) rs2 = make_rsrc(ptr2 + (long long)o * l2 * 2, (uint32_t)((long long)(nrows - 1) * l2 * 2 + R * 2));
      const uint32_t chunk = (uint32_t)((lane & 7) ^ ((4 * (wave & 1) + (lane >> 4)) & 7));
#pragma unroll
      for (int i = 0; i < NQ; ++i) {
        const bool second = TWO && i >= NQ / 2;
        const int row = (i * 4 + wave) * 8 + (lane >> 3) - (second ? WR : 0);
        voff[i] = (uint32_t)(row * (int)(second ? l2 : l) * 2) + chunk * 16;
      }
    } else {
      p = ptr;
      p2 = ptr2;
      ldb = l * 2;
      o0 = o;
      extent = (ext + 7) & ~7;
      r_split = split;
      r_rows = rows;
#pragma unroll
      for (int i = 0; i < NQ; ++i) {
        const int kr = (i * 4 + wave) * (512 / W) + lane / (W / 8), s = lane % (W / 8);
        const int c = (((s >> 1) ^ Tile::gran(kr)) << 1) | (s & 1);
        voff[i] = o + c * 8 < ext ? (uint32_t)(kr * (int)ldb) + (uint32_t)c * 16 : OUT;
      }
    }
  }
  // before the loads of tile kt
  __device__ __forceinline__ void prepare(int kt) {
    if constexpr (!COL) {
      soff = kt < kend ? (uint32_t)kt * 128u : 0x40000000u;
      if (kt == nk - 1 && (R & 63)) {
        const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
        const int chunk = (lane & 7) ^ ((4 * (wave & 1) + (lane >> 4)) & 7);
        const bool in = kt * 64 + chunk * 8 < R;
#pragma unroll
        for (int i = 0; i < NQ; ++i) voff[i] = in ? voff[i] : OUT;
      }
    } else {
      int r = kt * 64;
      const bool second = TWO && r >= r_split;
      if (second) r -= r_split;
      const int rows = kt < kend ? min(max(r_rows - r, 0), 64) : 0;
      const uint8_t* const q = (second ? p2 : p) + (long long)r * ldb + (long long)o0 * 2;
      rs = make_rsrc(q, rows > 0 ? (uint32_t)((rows - 1) * (int)ldb + min(W, extent - o0) * 2) : 0u);
    }
  }
  template <int NOPS = igc::NOPS_LOOP>
  __device__ __forceinline__ void part(uint8_t* st, int i) const {
    uint8_t* const dst = st + i * 4096 + wofs;
    if constexpr (COL)
      igc::dma16<NOPS>(rs, dst, voff[i]);
    else
      igc::dma16s<NOPS>(TWO && i >= NQ / 2 ? rs2 : rs, dst, voff[i], soff);
  }
};

// Tile of workgroup t of p.tiles_m x p.tiles_n.  The dispatcher hands
// workgroups to the 8 XCDs round-robin: each XCD gets a contiguous run of
// tiles, laid out in groups of 8 tile rows, so the workgroups that share an
// L2 share operand panels (256 x 4096 x 4096 on 64 x 64 tiles 22.6 -> 16.9 us,
// 4096^3 on 256 x 256 109 -> 102 us).
__device__ __forceinline__ void tile_of(const GemmArgs& p, int b, int& tm, int& tn) {
  const int n = p.tiles_m * p.tiles_n, x = b & 7;
  const int t = x * (n >> 3) + min(x, n & 7) + (b >> 3);
  const int per = 8 * p.tiles_n, group = t / per, first = group * 8;
  const int in = t - group * per, rows = min(8, p.tiles_m - first);
  tn = in / rows;
  tm = first + in - tn * rows;
}

// U rows of V consecutive sums (`f`, and `u` of the second product) leave for
// the outputs.  FULL: every lane has V columns.  STREAM: whole lines, written
// past the caches (8192 x 16384 x 4096 with kept sums 811 -> 803 us, 5728 x 5120 x
// 1088 74 -> 71; parts of lines must meet in the caches: 1000 x 32003 in fp32 81
// -> 100 us streamed).
template <bool BF, int MODE, int V, int U, bool FULL, bool STREAM>
struct Epilogue {
  const GemmArgs& p;
  int col;       // this lane's first column
  int left;      // columns from there to the end
  float b1[V], b2[V];
  bool has_bias;
  float undo;
  __device__ __forceinline__ Epilogue(const GemmArgs& args, int c) : p(args), col(c), left(args.N - c) {
    if constexpr (!BF && (MODE == M_DX || MODE == M_DW)) undo = p.undo ? *p.undo : 1.0f;
    has_bias = (MODE == M_FWD && p.bias) || (MODE == M_GLU && (p.bias || p.bias2));
    if constexpr (MODE == M_FWD || MODE == M_GLU) {
#pragma unroll
      for (int e = 0; e < V; ++e) {
        b1[e] = p.bias && e < have() ? p.bias[col + e] : 0.0f;
        b2[e] = MODE == M_GLU && p.bias2 && e < have() ? p.bias2[col + e] : 0.0f;
      }
    }
  }
  __device__ __forceinline__ int have() const { return FULL ? V : left; }
  // row q of the U rows
  template <class T>
  __device__ __forceinline__ void write(uint8_t* base, long long ld, int row, const float (&f)[U * V], int q) const {
    float v[V];
#pragma unroll
    for (int e = 0; e < V; ++e) v[e] = f[q * V + e];
    uint8_t* const to = base + ((long long)row * ld + col) * sizeof(T);
    typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
    if constexpr (STREAM && sizeof(T) == 4) {
#pragma unroll
      for (int e = 0; e < V; e += 4) {
        u32x4 w;
        __builtin_memcpy(&w, v + e, 16);
        __builtin_nontemporal_store(w, reinterpret_cast<u32x4*>(to + e * 4));
      }
    } else if constexpr (STREAM) {
      static_assert(V == 8, "16-byte stores");
      const uint4 w = pack8<BF>(v);
      __builtin_nontemporal_store(u32x4{w.x, w.y, w.z, w.w}, reinterpret_cast<u32x4*>(to));
    } else if constexpr (sizeof(T) == 4) {
      store_f32(reinterpret_cast<float*>(to), have(), v);
    } else {
      store_n<BF, V>(to, have(), v);
    }
  }
  // rows row0, row0 + step, ...
  __device__ __forceinline__ void operator()(int row0, int step, float (&f)[U * V], float (&u)[U * V]) const {
    if (!FULL && left <= 0) return;
    if constexpr (MODE == M_DX || MODE == M_DW) {
      if constexpr (!BF) {
#pragma unroll
        for (int e = 0; e < U * V; ++e) f[e] *= undo;
      }
#pragma unroll
      for (int q = 0; q < U; ++q) {
        const int row = row0 + q * step;
        if (row >= p.M) continue;
        if constexpr (MODE == M_DX) {
          write<uint16_t>(p.Y, p.ldy, row, f, q);
        } else {
          const bool second = row >= p.m_split;
          const int r = second ? row - p.m_split : row;
          uint8_t* const y = second ? p.Y2 : p.Y;  // (either may be left out)
          if (y && r < p.m_rows) write<uint16_t>(y, second ? p.ldy2 : p.ldy, r, f, q);
        }
      }
    } else {
      float res[U * V], y[U * V], unused[U * V];
      if (MODE == M_FWD && p.res) {
#pragma unroll
        for (int q = 0; q < U; ++q) {
          const int row = row0 + q * step;
          const int n = row < p.M ? have() : 0;
          float r[V];
          if (p.y_f32)
            load_f32(reinterpret_cast<const float*>(p.res) + (long long)row * p.ldr + col, n, r);
          else
            load_n<BF, V>(p.res + ((long long)row * p.ldr + col) * 2, n, r);
#pragma unroll
          for (int e = 0; e < V; ++e) res[q * V + e] = r[e];
        }
      }
      if (has_bias) {
#pragma unroll
        for (int e = 0; e < U * V; ++e) f[e] += b1[e % V];
        if constexpr (MODE == M_GLU) {
#pragma unroll
          for (int e = 0; e < U * V; ++e) u[e] += b2[e % V];
        }
      }
      if (p.Z) {
#pragma unroll
        for (int q = 0; q < U; ++q)
          if (row0 + q * step < p.M) write<uint16_t>(p.Z, p.ldz, row0 + q * step, f, q);
      }
      act_n<false>(p.act, f, y, unused);
      if constexpr (MODE == M_GLU) {
#pragma unroll
        for (int q = 0; q < U; ++q)
          if (p.U && row0 + q * step < p.M) write<uint16_t>(p.U, p.ldu, row0 + q * step, u, q);
#pragma unroll
        for (int e = 0; e < U * V; ++e) y[e] *= u[e];
      } else if (p.res) {
#pragma unroll
        for (int e = 0; e < U * V; ++e) y[e] += res[e];
      }
#pragma unroll
      for (int q = 0; q < U; ++q) {
        const int row = row0 + q * step;
        if (row >= p.M) continue;
        if (MODE == M_FWD && p.y_f32)
          write<float>(p.Y, p.ldy, row, y, q);
        else
          write<uint16_t>(p.Y, p.ldy, row, y, q);
      }
    }
  }
};

// A reduction split between workgroups (of every tile, or of those that are
// left when the others have filled the card a whole number of times): each leaves its accumulators in lane
// order, and a second launch adds them in split order and runs the epilogue.
// (Joined in the same launch by the last workgroup to arrive, every arrival
// writes its XCD's L2 back and every join drops it: 256 x 4096 x 4096 on
// 64 x 64 tiles in two splits took 51 us so, against 23 unsplit.)
template <int NQ>
__device__ __forceinline__ f32x4* partial(const GemmArgs& p, int tile, int split, int thread) {
  return reinterpret_cast<f32x4*>(p.part) + ((long long)(tile - p.whole) * p.splits + split) * NQ * 256 + thread;
}
// Workgroup b's tile and split.  (One split after the other, so that the
// workgroups of an XCD keep neighbouring tiles of one split.)
__device__ __forceinline__ void split_of(const GemmArgs& p, int b, int& tile, int& split) {
  tile = b;
  split = 0;
  if (b >= p.whole && p.splits > 1) {
    const int rest = p.tiles_m * p.tiles_n - p.whole;
    split = (b - p.whole) / rest;
    tile = b - split * rest;
  }
}

// The accumulators of a wave (FM x FN blocks, each transposed by the matrix
// instruction: lane l holds row l % 16, columns 4 (l / 16) .. +3) leave
// through the wave's own REGION bytes of LDS, as many block rows at a time as
// fit, so that every lane gets 8 consecutive columns of a row and a store
// instruction covers whole 128-byte lines.  No barrier: a wave's LDS accesses
// are in order.  The arithmetic sits in a real loop over the staged rows
// (unrolled over the accumulators, its six activations overflow the
// instruction cache).
template <bool BF, int MODE, int FM, int FN, int REGION>
__device__ __forceinline__ void write_out(const GemmArgs& p, const f32x4 (&acc)[FM][FN], uint8_t* lds, int row0, int col0) {
  constexpr bool GLU = MODE == M_GLU;
  constexpr int TN = FN * 16, OUT = GLU ? TN / 2 : TN;  // staged columns, output columns
  constexpr int LPR = OUT / 8, RPP = 64 / LPR;          // lanes per row, rows per pass
  constexpr int FIT = REGION / (16 * TN * 4), GR = FIT >= FM ? FM : FM / 2;  // block rows staged at a time
  static_assert(FIT >= GR && FM % GR == 0, "staging");
  constexpr int XM = TN / 4 < 16 ? TN / 4 - 1 : 15;
  const int lane = threadIdx.x & 63;
  const int wr = lane & 15, rr = lane / LPR, rc = lane % LPR;
  auto quad = [&](int r, int q) { return r * (TN * 4) + ((q ^ (r & XM)) << 4); };  // 4 columns of a staged row
  constexpr int U = GR * 16 / RPP > 1 ? 2 : 1;  // rows per lane and turn, so that their latencies overlap
  auto turns = [&](const auto& out, int row) {
    for (int r = rr; r < GR * 16; r += RPP * U) {
      float f[U * 8], u[U * 8];
#pragma unroll
      for (int q = 0; q < U; ++q) {
        const int at = r + q * RPP, c = rc * 2;
        uint4 v = lds_read16(lds, quad(at, c));
        __builtin_memcpy(f + q * 8, &v, 16);
        v = lds_read16(lds, quad(at, c + 1));
        __builtin_memcpy(f + q * 8 + 4, &v, 16);
        if constexpr (GLU) {
          v = lds_read16(lds, quad(at, OUT / 4 + c));
          __builtin_memcpy(u + q * 8, &v, 16);
          v = lds_read16(lds, quad(at, OUT / 4 + c + 1));
          __builtin_memcpy(u + q * 8 + 4, &v, 16);
        }
      }
      out(row + r, RPP, f, u);
    }
  };
  auto rows = [&](const auto& out) {
    static_for<FM / GR>([&](auto g) {
      constexpr int G0 = decltype(g)::value * GR;
      asm volatile("" ::: "memory");
      static_for<GR>([&](auto i) {
        constexpr int I = decltype(i)::value;
#pragma unroll
        for (int j = 0; j < FN; ++j)
          lds_write16(lds, quad(I * 16 + wr, j * 4 + (lane >> 4)), __builtin_bit_cast(uint4, acc[G0 + I][j]));
      });
      asm volatile("" ::: "memory");
      turns(out, row0 + G0 * 16);
    });
  };
  if (col0 + OUT > p.N)
    rows(Epilogue<BF, MODE, 8, U, false, false>(p, col0 + rc * 8));
  else if (p.stream)
    rows(Epilogue<BF, MODE, 8, U, true, true>(p, col0 + rc * 8));
  else
    rows(Epilogue<BF, MODE, 8, U, true, false>(p, col0 + rc * 8));
}

// The simple product: K tiles go through registers into two LDS stages.
// Takes every alignment and stride.
template <bool BF, int MODE, int BM, int BN>
__global__ void __launch_bounds__(256, 2) gemm_any_kernel(const GemmArgs p) {
  constexpr bool GLU = MODE == M_GLU, ACOL = MODE == M_DW, BCOL = MODE == M_DX || MODE == M_DW;
  constexpr int TM = BM / 2, TN = BN / 2, FM = TM / 16, FN = TN / 16;
  typedef LdsTile<BM, ACOL> TA;
  typedef LdsTile<BN, BCOL> TB;
  __shared__ __attribute__((aligned(16))) uint8_t smem[2 * (TA::BYTES + TB::BYTES)];
  const int wave = wave_id(), wm = wave >> 1, wn = wave & 1;
  int tile, split, tm, tn;
  split_of(p, blockIdx.x, tile, split);
  tile_of(p, tile, tm, tn);
  constexpr int ON = GLU ? BN / 2 : BN;  // output columns of a tile
  const int m0 = tm * BM, n0 = tn * ON;
  const int nk = max(1, (p.R + 63) / 64);
  const int k0 = (int)((long long)nk * split / p.splits), k1 = (int)((long long)nk * (split + 1) / p.splits);
  RegOperand<BM, ACOL, false> la;
  RegOperand<BN, BCOL, GLU || MODE == M_DX> lb;
  la.init(p.A, p.lda, nullptr, 0, m0, p.M, p.R, p.R, p.R);
  lb.init(p.B, p.ldb, p.B2, p.ldb2, n0, p.N, p.R, p.r_split, p.b_rows);
  f32x4 acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  auto blk_b = [&](int j) {
    if constexpr (GLU) return j < FN / 2 ? wn * (TN / 2) + j * 16 : BN / 2 + wn * (TN / 2) + (j - FN / 2) * 16;
    return wn * TN + j * 16;
  };
  uint4 va[RegOperand<BM, ACOL, false>::NC], vb[RegOperand<BN, BCOL, true>::NC];
  la.load(k0, va);
  lb.load(k0, vb);
  uint8_t* const sa = smem;
  uint8_t* const sb = smem + 2 * TA::BYTES;
  la.store(sa, va);
  lb.store(sb, vb);
  __syncthreads();
  for (int kt = k0; kt < k1; ++kt) {
    const int cur = (kt - k0) & 1;
    if (kt + 1 < k1) {
      la.load(kt + 1, va);
      lb.load(kt + 1, vb);
    }
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
      uint4 fa[FM], fb[FN];
#pragma unroll
      for (int i = 0; i < FM; ++i) fa[i] = TA::frag(sa + cur * TA::BYTES, wm * TM + i * 16, ks);
#pragma unroll
      for (int j = 0; j < FN; ++j) fb[j] = TB::frag(sb + cur * TB::BYTES, blk_b(j), ks);
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j) mfma16<BF>(acc[i][j], fb[j], fa[i]);
    }
    if (kt + 1 < k1) {
      la.store(sa + (cur ^ 1) * TA::BYTES, va);
      lb.store(sb + (cur ^ 1) * TB::BYTES, vb);
    }
    __syncthreads();
  }
  if (p.splits > 1) {
    f32x4* const out = partial<FM * FN>(p, tile, split, threadIdx.x);
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j) out[(i * FN + j) * 256] = acc[i][j];
    return;
  }
  write_out<BF, MODE, FM, FN, sizeof(smem) / 4>(p, acc, smem + wave * (sizeof(smem) / 4), m0 + wm * TM, n0 + wn * (ON / 2));
}

// The forward products of few rows (M <= 16 MB): bound by streaming the
// weights once.  A workgroup takes NB blocks of 16 weight rows (the gated
// block: half of them from each weight) and its waves split the reduction;
// every lane loads its matrix-instruction operands straight into registers,
// UN steps of 32 elements at once, so that a compute unit keeps over 100 KB
// of weights in flight, which is what it takes to reach the memory's rate.
// The waves' sums are added through LDS in wave order.  Any alignment.
// ODD: rows may start at odd multiples of 2 bytes.
template <bool BF, int MODE, int MB, int NB, int NW, bool ODD>
__global__ void __launch_bounds__(64 * NW) gemm_skinny_kernel(const GemmArgs p) {
  constexpr bool GLU = MODE == M_GLU;
  constexpr int PB = GLU ? NB / 2 : NB;  // column blocks
  constexpr int UN = MB == 1 ? 8 : 4;
  __shared__ f32x4 red[NW][NB * MB][64];
  const int lane = threadIdx.x & 63, wave = wave_id();
  const int r = lane & 15, g = lane >> 4;
  const int n0 = blockIdx.x * (PB * 16);
  // rows past the end repeat the last one; their sums are not stored
  const uint8_t *w[NB], *x[MB];
#pragma unroll
  for (int j = 0; j < NB; ++j) {
    const bool second = GLU && j >= PB;
    const long long n = min(n0 + (second ? j - PB : j) * 16 + r, p.N - 1);
    w[j] = (second ? p.B2 + n * p.ldb2 * 2 : p.B + n * p.ldb * 2) + g * 16;
  }
#pragma unroll
  for (int i = 0; i < MB; ++i) x[i] = p.A + (long long)min(i * 16 + r, p.M - 1) * p.lda * 2 + g * 16;
  f32x4 acc[NB][MB];
#pragma unroll
  for (int j = 0; j < NB; ++j)
#pragma unroll
    for (int i = 0; i < MB; ++i) acc[j][i] = f32x4{0.f, 0.f, 0.f, 0.f};

  const int steps = p.R / 32 + (p.R % 32 >= 8);  // (what is left of a chunk of 8 follows below)
  const int s1 = (int)((long long)steps * (wave + 1) / NW);
  int s = (int)((long long)steps * wave / NW);
  uint4 fw[UN][NB], fx[UN][MB];
  auto multiply = [&](int u) {
#pragma unroll
    for (int j = 0; j < NB; ++j)
#pragma unroll
      for (int i = 0; i < MB; ++i) mfma16<BF>(acc[j][i], fw[u][j], fx[u][i]);
  };
  auto chunk = [](const uint8_t* q) {
    if constexpr (ODD) return load8_words(q);
    uint4 v;
    __builtin_memcpy(&v, q, 16);
    return v;
  };
  for (; s + UN <= s1 && (s + UN) * 32 <= p.R; s += UN) {
#pragma unroll
    for (int u = 0; u < UN; ++u) {
#pragma unroll
      for (int j = 0; j < NB; ++j) fw[u][j] = chunk(w[j] + (long long)(s + u) * 64);
#pragma unroll
      for (int i = 0; i < MB; ++i) fx[u][i] = chunk(x[i] + (long long)(s + u) * 64);
    }
#pragma unroll
    for (int u = 0; u < UN; ++u) multiply(u);
  }
  if (s < s1) {  // the last batch: the steps that are left, the lanes whose chunk is whole
#pragma unroll
    for (int u = 0; u < UN; ++u) {
      const bool in = s + u < s1 && (s + u) * 32 + g * 8 + 8 <= p.R;
#pragma unroll
      for (int j = 0; j < NB; ++j) fw[u][j] = in ? chunk(w[j] + (long long)(s + u) * 64) : make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int i = 0; i < MB; ++i) fx[u][i] = in ? chunk(x[i] + (long long)(s + u) * 64) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int u = 0; u < UN; ++u) multiply(u);
  }
  if ((p.R & 7) && wave == NW - 1) {  // the elements past the last whole chunk
    const int k = p.R & ~7, left = g == 0 ? p.R & 7 : 0;
#pragma unroll
    for (int j = 0; j < NB; ++j) fw[0][j] = load8(w[j] - g * 16 + (long long)k * 2, left);
#pragma unroll
    for (int i = 0; i < MB; ++i) fx[0][i] = load8(x[i] - g * 16 + (long long)k * 2, left);
    multiply(0);
  }
#pragma unroll
  for (int j = 0; j < NB; ++j)
#pragma unroll
    for (int i = 0; i < MB; ++i) red[wave][j * MB + i][lane] = acc[j][i];
  __syncthreads();
  // lane l of a block holds row l % 16, columns 4 (l / 16) .. +3
  for (int t = threadIdx.x; t < PB * MB * 64; t += 64 * NW) {
    const int b = t >> 6, l = t & 63;
    f32x4 f4 = red[0][b][l], u4 = GLU ? red[0][PB * MB + b][l] : f4;
#pragma unroll
    for (int q = 1; q < NW; ++q) {
      f4 += red[q][b][l];
      if constexpr (GLU) u4 += red[q][PB * MB + b][l];
    }
    float f[4] = {f4[0], f4[1], f4[2], f4[3]}, u[4] = {u4[0], u4[1], u4[2], u4[3]};
    const Epilogue<BF, MODE, 4, 1, false, false> out(p, n0 + (b / MB) * 16 + 4 * (l >> 4));
    out((b % MB) * 16 + (l & 15), 0, f, u);
  }
}

// The product on aligned operands: both go from memory straight into LDS,
// DEPTH K tiles ahead, and the K loop is software-pipelined over the stages.
// A K tile of 64 is two k-steps of FM chunks; a chunk is the FN matrix
// instructions of one block row, with at most one load and its share of the
// next k-step's fragment reads between them, fenced so that program order is
// issue order.  During the first k-step of tile kt the loads of A tile
// kt + DEPTH go out; then the wave waits until tile kt + 1 has landed (only
// later tiles' loads may still fly) and a barrier frees tile kt's stages;
// during the second k-step the loads of B tile kt + DEPTH go out and tile
// kt + 1's first fragments are read.
// Four waves, 2 x 2.  256 x 256 at depth 2 (A in three stages, B in two, all
// 160 KB of LDS): a wave holds 128 x 128 sums (all 256 accumulation
// registers), the least LDS traffic per matrix instruction; bound by the
// matrix cores at the clock that the power limit leaves them (2200 cycles per
// K tile, of which they take 2048).  128 x 128 at depth 2, two workgroups per
// compute unit.  64 x 64 at depth 4 (80 KB: two workgroups), where a compute
// unit's loads in flight are the bound: 64 x 4096 x 4096 unsplit 26.7 us at
// depth 2, 15.4 at 4, 15.5 at 6.  64 x 32 at depth 6 spreads the loads of small
// outputs over twice as many compute units: 24 x 8192 x 2048 9.0 -> 8.0 us,
// 500 x 1024 x 1024 of the gated block 8.0 -> 6.6.
constexpr int tile_lds(int bm, int bn, int depth) { return 128 * ((depth + 1) * bm + (depth == 2 ? 2 : depth + 1) * bn); }
constexpr int tile_waves(int bm, int bn, int depth) { return 160 * 1024 / tile_lds(bm, bn, depth) > 1 ? 2 : 1; }  // per SIMD
template <bool BF, int MODE, int BM, int BN, int DEPTH>
__device__ __forceinline__ void tile_product(const GemmArgs& p, const int block, uint8_t* const smem) {
  constexpr bool GLU = MODE == M_GLU, ACOL = MODE == M_DW, BCOL = MODE == M_DX || MODE == M_DW;
  constexpr int TM = BM / 2, TN = BN / 2, FM = TM / 16, FN = TN / 16;
  typedef LdsTile<BM, ACOL> TA;
  typedef LdsTile<BN, BCOL> TB;
  typedef DmaOperand<BM, ACOL, false> LoadA;
  typedef DmaOperand<BN, BCOL, GLU || MODE == M_DX> LoadB;
  constexpr int RA = DEPTH + 1, RB = DEPTH == 2 ? 2 : DEPTH + 1, UNR = RA == RB ? RA : RA * RB;
  constexpr int LDS = RA * TA::BYTES + RB * TB::BYTES;
  static_assert(LDS == tile_lds(BM, BN, DEPTH), "stages");
  auto stA = [&](auto u) -> uint8_t* { return smem + (decltype(u)::value % RA) * TA::BYTES; };
  auto stB = [&](auto u) -> uint8_t* { return smem + RA * TA::BYTES + (decltype(u)::value % RB) * TB::BYTES; };
  const int wave = wave_id(), wm = wave >> 1, wn = wave & 1;
  int tile, split, tm, tn;
  split_of(p, block, tile, split);
  const bool shared = p.splits > 1 && tile >= p.whole;
  tile_of(p, tile, tm, tn);
  constexpr int ON = GLU ? BN / 2 : BN;
  const int m0 = tm * BM, n0 = tn * ON;
  const int nk = max(1, (p.R + 63) / 64);
  int k0 = 0, k1 = nk;
  if (shared) {
    k0 = (int)((long long)nk * split / p.splits);
    k1 = (int)((long long)nk * (split + 1) / p.splits);
  }
  LoadA la;
  LoadB lb;
  la.init(p.A, p.lda, nullptr, 0, m0, p.M, p.R, p.R, p.R, k1);
  lb.init(p.B, p.ldb, p.B2, p.ldb2, n0, p.N, p.R, p.r_split, p.b_rows, k1);

  f32x4 acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  auto blk_b = [&](int j) {
    if constexpr (GLU) return j < FN / 2 ? wn * (TN / 2) + j * 16 : BN / 2 + wn * (TN / 2) + (j - FN / 2) * 16;
    return wn * TN + j * 16;
  };
  uint4 fa[2][FM], fb[2][FN];

  // one block row c of a k-step
  auto chunk = [&](int c, const uint4(&a)[FM], const uint4(&b)[FN], const uint8_t* An, const uint8_t* Bn, int ksn,
                   uint4(&an)[FM], uint4(&bn)[FN], auto issue) {
    __builtin_amdgcn_sched_barrier(0);
    mfma16<BF>(acc[c][0], b[0], a[c]);
    __builtin_amdgcn_sched_barrier(0);
    issue();
    __builtin_amdgcn_sched_barrier(0);
    // the next k-step's fragments: B first (its first chunk needs all of them)
    int nrd = 0;
#pragma unroll
    for (int r = 0; r < FN + FM; ++r)
      if (r * FM / (FN + FM) == c) {
        if (r < FN) {
          bn[r] = TB::frag(Bn, blk_b(r), ksn);
          nrd += BCOL ? 2 : 1;
        } else {
          an[r - FN] = TA::frag(An, wm * TM + (r - FN) * 16, ksn);
          nrd += ACOL ? 2 : 1;
        }
      }
#pragma unroll
    for (int j = 1; j < FN; ++j) mfma16<BF>(acc[c][j], b[j], a[c]);
#pragma unroll
    for (int q = 1; q < FN; ++q) {
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);  // MFMA
      if (q <= nrd) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);  // LDS read
    }
  };

  static_for<DEPTH>([&](auto d) {
    constexpr int D = decltype(d)::value;
    la.prepare(k0 + D);
    lb.prepare(k0 + D);
#pragma unroll
    for (int i = 0; i < LoadA::NQ; ++i) la.template part<igc::NOPS_SAFE>(stA(d), i);
#pragma unroll
    for (int i = 0; i < LoadB::NQ; ++i) lb.template part<igc::NOPS_SAFE>(stB(d), i);
  });
  wait_vmcnt_lgkm0<(DEPTH - 1) * (LoadA::NQ + LoadB::NQ)>();
  lds_barrier();
#pragma unroll
  for (int i = 0; i < FM; ++i) fa[0][i] = TA::frag(smem, wm * TM + i * 16, 0);
#pragma unroll
  for (int j = 0; j < FN; ++j) fb[0][j] = TB::frag(smem + RA * TA::BYTES, blk_b(j), 0);

  auto ktile = [&](int kt, auto U) {
    constexpr int u = decltype(U)::value;
    const uint8_t *As = stA(U), *Bs = stB(U);
    uint8_t* const An = stA(std::integral_constant<int, u + DEPTH>());
    uint8_t* const Bn = stB(std::integral_constant<int, u + DEPTH>());
    const uint8_t* const A1 = stA(std::integral_constant<int, u + 1>());
    const uint8_t* const B1 = stB(std::integral_constant<int, u + 1>());
    la.prepare(kt + DEPTH);
    lb.prepare(kt + DEPTH);
#pragma unroll
    for (int c = 0; c < FM; ++c)
      chunk(c, fa[0], fb[0], As, Bs, 1, fa[1], fb[1], [&]() {
#pragma unroll
        for (int i = 0; i < LoadA::NQ; ++i)
          if (i * FM / LoadA::NQ == c) la.part(An, i);
      });
    __builtin_amdgcn_sched_barrier(0);
    wait_vmcnt_lgkm0<(DEPTH - 2) * (LoadA::NQ + LoadB::NQ) + LoadA::NQ>();
    lds_barrier();
#pragma unroll
    for (int c = 0; c < FM; ++c)
      chunk(c, fa[1], fb[1], A1, B1, 0, fa[0], fb[0], [&]() {
#pragma unroll
        for (int i = 0; i < LoadB::NQ; ++i)
          if (i * FM / LoadB::NQ == c) lb.part(Bn, i);
      });
  };
  for (int kt = k0; kt < k1; kt += UNR) {
    ktile(kt, std::integral_constant<int, 0>());
    static_for<UNR - 1>([&](auto J) {
      constexpr int j = decltype(J)::value + 1;
      if (kt + j < k1) ktile(kt + j, std::integral_constant<int, j>());
    });
  }
  // loads past the last tile may still be writing LDS
  wait_vmcnt_lgkm0<0>();
  lds_barrier();
  if (shared) {
    f32x4* const out = partial<FM * FN>(p, tile, split, threadIdx.x);
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j) out[(i * FN + j) * 256] = acc[i][j];
    return;
  }
  write_out<BF, MODE, FM, FN, LDS / 4>(p, acc, smem + wave * (LDS / 4), m0 + wm * TM, n0 + wn * (ON / 2));
}

template <bool BF, int MODE, int BM, int BN, int DEPTH>
__global__ void __launch_bounds__(256, tile_waves(BM, BN, DEPTH)) gemm_tile_kernel(const GemmArgs p) {
  __shared__ __attribute__((aligned(16))) uint8_t smem[tile_lds(BM, BN, DEPTH)];
  tile_product<BF, MODE, BM, BN, DEPTH>(p, blockIdx.x, smem);
}

// Column sums of D over its row blocks: out[n] = sum over blocks of
// sums[block][which][n], in a fixed order.  A workgroup takes 64 columns, each
// of its waves every fourth block.
struct ColsumArgs {
  const float* sums;
  int blocks, which_n, width, N;
  float *out0, *out1;
};
__device__ __forceinline__ void colsum(const ColsumArgs& p, int group, float* lds) {
  const int per = (p.N + 63) / 64, which = group / per;
  const int n = (group - which * per) * 64 + (threadIdx.x & 63), wave = wave_id();
  float* const out = which ? p.out1 : p.out0;
  float s = 0.0f;
  if (out && n < p.N) {
    const float* const in = p.sums + (long long)which * p.width + n;
    const long long step = (long long)p.which_n * p.width;
#pragma unroll 8
    for (int b = wave; b < p.blocks; b += 4) s += in[b * step];
  }
  lds[threadIdx.x] = s;
  __syncthreads();
  if (wave == 0 && out && n < p.N) out[n] = (s + lds[64 + threadIdx.x]) + (lds[128 + threadIdx.x] + lds[192 + threadIdx.x]);
}
template <int NONE = 0>
__global__ void __launch_bounds__(256) colsum_kernel(const ColsumArgs p) {
  __shared__ float lds[256];
  colsum(p, blockIdx.x, lds);
}

// Both backward products on one tile size, and the column sums, in one
// launch: the product with the longer workgroups first (x_first: dX), then, at
// a multiple of 8 so that its tiles keep their XCDs, the other, then the sums.
// What one leaves of the last round of compute units the next fills.
template <bool BF, int BM, int BN, int DEPTH>
__global__ void __launch_bounds__(256, tile_waves(BM, BN, DEPTH))
    gemm_back_kernel(const GemmArgs px, const GemmArgs pw, const ColsumArgs ps, int x_first, int first, int second) {
  __shared__ __attribute__((aligned(16))) uint8_t smem[tile_lds(BM, BN, DEPTH)];
  const int pad = (first + 7) & ~7, b = blockIdx.x;
  if (b >= pad + second) {
    colsum(ps, b - pad - second, reinterpret_cast<float*>(smem));
  } else if ((b < pad) == (x_first != 0)) {
    if (b < first || b >= pad) tile_product<BF, M_DX, BM, BN, DEPTH>(px, b < pad ? b : b - pad, smem);
  } else {
    if (b < first || b >= pad) tile_product<BF, M_DW, BM, BN, DEPTH>(pw, b < pad ? b : b - pad, smem);
  }
}

// The second launch of a split reduction: one wave for each block row of each
// wave of a tile (one wave for all its block rows keeps too little in flight:
// 16 tiles of 256 x 256 in two splits 30 us).
constexpr int join_waves(int bm) { return 4 * (bm / 2 / 16); }  // per tile
template <bool BF, int MODE, int BM, int BN>
__global__ void __launch_bounds__(64) gemm_join_kernel(const GemmArgs p) {
  constexpr int TM = BM / 2, TN = BN / 2, FM = TM / 16, FN = TN / 16;
  constexpr int ON = MODE == M_GLU ? BN / 2 : BN;
  __shared__ __attribute__((aligned(16))) uint8_t smem[16 * TN * 4];
  const int tile = p.whole + blockIdx.x / (4 * FM), rest = blockIdx.x % (4 * FM);
  const int wave = rest / FM, i = rest % FM, wm = wave >> 1, wn = wave & 1;
  int tm, tn;
  tile_of(p, tile, tm, tn);
  f32x4 acc[1][FN];
#pragma unroll
  for (int j = 0; j < FN; ++j) acc[0][j] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
  for (int s = 0; s < p.splits; ++s) {
    const f32x4* const in = partial<FM * FN>(p, tile, s, wave * 64 + threadIdx.x) + (long long)i * FN * 256;
#pragma unroll
    for (int j = 0; j < FN; ++j) acc[0][j] += in[j * 256];
  }
  write_out<BF, MODE, 1, FN, sizeof(smem)>(p, acc, smem, tm * BM + wm * TM + i * 16, tn * ON + wn * (ON / 2));
}

// ---------------------------------------------------------------------------
// The element-wise part of the backward passes.
// ---------------------------------------------------------------------------
struct ActBackArgs {
  int M, N;
  const uint8_t *dY, *Z, *U;
  long long lddy, ldz, ldu;  // elements
  int act;
  uint8_t* D;      // out (NULL: only the column sums): D, or dG and dU side by side, each `width` columns
  long long ldd;   // elements
  int width;       // N rounded up to a multiple of 64; columns past N are written as zeros
  float* sums;     // out (NULL: none): column sums of each row block, [row blocks][1 or 2][width]
  int rows;        // rows per block
  int groups, blocks;  // workgroups across the columns and down the rows
  // fp16 (NULL: D is not scaled): the largest finite |D| of each block, and
  // what takes D's scale back
  float *most, *undo;
};

// Rows of any alignment and at least 8 elements, copied into rows of whole
// 16-byte chunks (zeros past the end) so that the product can load them
// straight into LDS.  One thread takes four chunks; a row's last chunk is
// loaded as the row's last 8 elements and shifted, so that no lane branches
// between the loads.  Bound by memory.
constexpr int PAD_MOST = 3;  // operands per launch
struct PadArgs {
  int count;
  const uint8_t* src[PAD_MOST];
  long long ld[PAD_MOST];   // bytes
  int cols[PAD_MOST];
  uint32_t chunks[PAD_MOST];  // rows x chunks per row
  uint8_t* dst[PAD_MOST];
  int first[PAD_MOST + 1];  // first workgroup of each operand; [count]: all of them
};
__device__ __forceinline__ void pad_rows(const PadArgs& p, int block) {
  int op = 0;
  while (op + 1 < p.count && block >= p.first[op + 1]) ++op;
  const uint8_t* const src = p.src[op];
  const long long ld = p.ld[op];
  const int cols = p.cols[op];
  const uint32_t per = (uint32_t)(cols + 7) / 8, end = p.chunks[op];
  const uint32_t i0 = (uint32_t)(block - p.first[op]) * 1024 + threadIdx.x;
  unsigned __int128 v[4];
  int back[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t i = min(i0 + 256 * j, end - 1), row = i / per, c = (i - row * per) * 8;
    back[j] = max((int)c + 8 - cols, 0);
    __builtin_memcpy(&v[j], src + row * ld + (long long)((int)c - back[j]) * 2, 16);
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    v[j] >>= 16 * back[j];
    if (i0 + 256 * j < end) __builtin_memcpy(p.dst[op] + (long long)(i0 + 256 * j) * 16, &v[j], 16);
  }
}
template <int NONE = 0>
__global__ void __launch_bounds__(256) pad_kernel(const PadArgs p) {
  pad_rows(p, blockIdx.x);
}

// Block b of the element-wise work: 512 columns (8 per lane) x `rows` rows; the
// four waves take rows in turn, UR at a time so that their loads fly together.
// Calls f(row, column, d, du) with D (dG and dU) in fp32, zeros past N.
template <bool BF, bool GLU, class F>
__device__ __forceinline__ void act_rows(const ActBackArgs& p, int b, F&& f) {
  constexpr int UR = GLU ? 2 : 4;
  const int lane = threadIdx.x & 63, wave = wave_id();
  const int by = b / p.groups, bx = b - by * p.groups;
  const int c = bx * 512 + lane * 8;
  const int left = p.N - c;
  const int r0 = by * p.rows, r1 = min(p.M, r0 + p.rows);
  if (c >= p.width) return;
  for (int rb = r0 + wave; rb < r1; rb += 4 * UR) {
    uint4 vy[UR], vz[UR], vu[UR];
#pragma unroll
    for (int q = 0; q < UR; ++q) {
      const long long r = rb + 4 * q;
      const int have = r < r1 ? left : 0;
      vy[q] = load8(p.dY + (r * p.lddy + c) * 2, have);
      vz[q] = p.Z ? load8(p.Z + (r * p.ldz + c) * 2, have) : make_uint4(0, 0, 0, 0);
      if constexpr (GLU) vu[q] = load8(p.U + (r * p.ldu + c) * 2, have);
    }
#pragma unroll
    for (int q = 0; q < UR; ++q) {
      const long long r = rb + 4 * q;
      if (r >= r1) break;
      float dy[8], z[8], fz[8], d[8], du[8];
      unpack8<BF>(vy[q], dy);
      unpack8<BF>(vz[q], z);
      if constexpr (GLU) {
        float u[8];
        unpack8<BF>(vu[q], u);
        act_n<true>(p.act, z, fz, d);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          du[e] = dy[e] * fz[e];
          d[e] = dy[e] * u[e] * d[e];
          if (e >= left) du[e] = d[e] = 0.0f;
        }
      } else {
        if (p.Z) {
          act_n<true>(p.act, z, fz, d);
#pragma unroll
          for (int e = 0; e < 8; ++e) dy[e] *= d[e];
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) d[e] = e >= left ? 0.0f : dy[e];
      }
      f(r, c, d, du);
    }
  }
}

// The scale of D in fp16.  2^10 to begin with: every |D| below 32 fits, an
// element from 2^-24 up keeps all its bits, and a smaller one is off by at most
// 2^-35, which is 2^-10 of the smallest step of the gradients themselves.
// Where the largest |D| is not in [2^-18, 2^5), act_again_kernel makes D anew
// at the scale that takes the largest to [2^14, 2^15): elements down to 2^-28
// of it keep all their bits.  (A search for the largest before D is made, in
// every call: 777 x 1001 x 1128 with silu 17.0 -> 22.1 us, 4096 x 8192 x 4096
// 437 -> 478; this way 19.7 and 446.)
constexpr float ACT_SCALE = 1024.0f, ACT_LEAST = 0x1p-18f, ACT_MOST = 0x1p5f;
__device__ __forceinline__ void most_of(float& m, float v) {  // (neither infinities nor NaN)
  const float a = __builtin_fabsf(v);
  if (a <= 3.402823466e38f) m = __builtin_fmaxf(m, a);
}
__device__ __forceinline__ float group_max(float m, float* sm) {  // in every thread of the workgroup
#pragma unroll
  for (int o = 32; o; o >>= 1) m = __builtin_fmaxf(m, __shfl_xor(m, o));
  if ((threadIdx.x & 63) == 0) sm[wave_id()] = m;
  __syncthreads();
  return __builtin_fmaxf(__builtin_fmaxf(sm[0], sm[1]), __builtin_fmaxf(sm[2], sm[3]));
}
template <bool GLU>
__global__ void __launch_bounds__(256) act_again_kernel(const ActBackArgs p) {
  __shared__ float sm[4];
  const int all = p.groups * p.blocks;
  float m = 0.0f;
  for (int i = threadIdx.x; i < all; i += 256) m = __builtin_fmaxf(m, p.most[i]);
  m = group_max(m, sm);
  if (m == 0.0f || (m >= ACT_LEAST && m < ACT_MOST)) return;
  // (2^100 at most: where the largest is less than 2^-86, no product of D is left in fp16)
  const int n = min(14 - ((int)(__builtin_bit_cast(uint32_t, m) >> 23) - 127), 100);
  const float scale = __builtin_bit_cast(float, (uint32_t)(127 + n) << 23);
  if (blockIdx.x == 0 && threadIdx.x == 0) *p.undo = __builtin_bit_cast(float, (uint32_t)(127 - n) << 23);
  for (int b = blockIdx.x; b < all; b += gridDim.x)
    act_rows<false, GLU>(p, b, [&](long long r, int c, float (&d)[8], float (&du)[8]) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        d[e] *= scale;
        if constexpr (GLU) du[e] *= scale;
      }
      store8(p.D + (r * p.ldd + c) * 2, pack8<false>(d), 8);
      if constexpr (GLU) store8(p.D + (r * p.ldd + p.width + c) * 2, pack8<false>(du), 8);
    });
}

// D and its column sums: every block a workgroup.  Streams its inputs once:
// bound by memory (bf16, 4096 x 8192 with gelu: 201 MB in 42 us; the gated
// block at 4096 x 10944: 448 MB in 78 us).  Workgroups past its own pad the
// operands of the products that follow.
template <bool BF, bool GLU>
__global__ void __launch_bounds__(256) act_back_kernel(const ActBackArgs p, const PadArgs pad) {
  __shared__ float part[GLU ? 2 : 1][4][512];
  const int lane = threadIdx.x & 63, wave = wave_id();
  const int act_blocks = p.groups * p.blocks;
  if ((int)blockIdx.x >= act_blocks) return pad_rows(pad, blockIdx.x - act_blocks);
  const float scale = !BF && p.undo ? ACT_SCALE : 1.0f;
  float m = 0.0f;
  float s1[8], s2[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) s1[e] = s2[e] = 0.0f;
  act_rows<BF, GLU>(p, blockIdx.x, [&](long long r, int c, float (&d)[8], float (&du)[8]) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      s1[e] += d[e];
      if constexpr (GLU) s2[e] += du[e];
      if constexpr (!BF) {
        most_of(m, d[e]);
        d[e] *= scale;
        if constexpr (GLU) {
          most_of(m, du[e]);
          du[e] *= scale;
        }
      }
    }
    if (p.D) {
      store8(p.D + (r * p.ldd + c) * 2, pack8<BF>(d), 8);
      if constexpr (GLU) store8(p.D + (r * p.ldd + p.width + c) * 2, pack8<BF>(du), 8);
    }
  });
  if constexpr (!BF) {
    __shared__ float sm[4];
    if (p.undo) {
      m = group_max(m, sm);
      if (threadIdx.x == 0) p.most[blockIdx.x] = m;
      if (threadIdx.x == 0 && blockIdx.x == 0) *p.undo = 1.0f / ACT_SCALE;
    }
  }
  if (!p.sums) return;
  const int by = blockIdx.x / p.groups, bx = blockIdx.x - by * p.groups;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    part[0][wave][lane * 8 + e] = s1[e];
    if constexpr (GLU) part[1][wave][lane * 8 + e] = s2[e];
  }
  __syncthreads();
  constexpr int NP = GLU ? 2 : 1;
  for (int i = threadIdx.x; i < NP * 512; i += 256) {
    const int which = i / 512, cc = i % 512, col = bx * 512 + cc;
    if (col < p.width)
      p.sums[((long long)by * NP + which) * p.width + col] =
          (part[which][0][cc] + part[which][1][cc]) + (part[which][2][cc] + part[which][3][cc]);
  }
}

}  // namespace igc_ffn
