// row_kernels.hpp -- the operators that work on rows around the feed-forward
// products, on gfx950:
//
//   norm      mean = sum x / N;  rstd = (sum (x - mean)^2 / N + eps)^-1/2
//             y = (x - mean) rstd gamma + beta
//   back      xh = (x - mean) rstd;  g = dy gamma
//             dx = rstd (g - mean(g) - xh mean(g xh)) + r
//             dgamma = sum over rows of dy xh;  dbeta = sum over rows of dy
//   quantize  s = max|x| / 127;  q = round(127 x / max|x|), ties to even
//
// All of them are bound by memory.  Statistics and sums are held in fp32 and
// added in an order that the sizes alone set.
#pragma once

#include "ffn_kernels.hpp"

namespace igc_rows {

using igc::wave_id;
using igc_ffn::T_BF16;
using igc_ffn::T_F16;
using igc_ffn::T_F32;
using igc_ffn::load8;
using igc_ffn::load_f32;
using igc_ffn::pack8;
using igc_ffn::store8;
using igc_ffn::store_f32;
using igc_ffn::unpack8;

// Eight elements of type T (igc_ffn::Type) as they lie in memory.
template <int T>
struct Raw {
  static constexpr int EB = 2;
  uint4 v;
  __device__ __forceinline__ void load(const uint8_t* p, int valid) { v = load8(p, valid); }  // (zeros past `valid`)
  __device__ __forceinline__ void get(float (&f)[8]) const { unpack8<T == T_BF16>(v, f); }
  __device__ __forceinline__ void set(const float (&f)[8]) { v = pack8<T == T_BF16>(f); }
  __device__ __forceinline__ void store(uint8_t* p, int valid) const { store8(p, v, valid); }
};
template <>
struct Raw<T_F32> {
  static constexpr int EB = 4;
  float v[8];
  __device__ __forceinline__ void load(const uint8_t* p, int valid) { load_f32<8>(reinterpret_cast<const float*>(p), valid, v); }
  __device__ __forceinline__ void get(float (&f)[8]) const {
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = v[e];
  }
  __device__ __forceinline__ void set(const float (&f)[8]) {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = f[e];
  }
  __device__ __forceinline__ void store(uint8_t* p, int valid) const { store_f32<8>(reinterpret_cast<float*>(p), valid, v); }
};

// A value of every thread of a row's T threads, combined in every one of
// them: lanes of a wave first, then the waves through LDS.  Calls in a row take
// slots in turn (two are enough: who writes a slot again has passed the
// barrier of the other one, which everyone reaches after reading this one).
template <int T, class V, class F>
__device__ __forceinline__ V row_combine(V v, V* slot, F&& f) {
#pragma unroll
  for (int o = 32; o; o >>= 1) v = f(v, __shfl_xor(v, o));
  if constexpr (T > 64) {
    if ((threadIdx.x & 63) == 0) slot[threadIdx.x >> 6] = v;
    __syncthreads();
    v = slot[0];
#pragma unroll
    for (int i = 1; i < T / 64; ++i) v = f(v, slot[i]);
  }
  return v;
}
template <int T>
__device__ __forceinline__ float row_sum(float v, float* slot) {
  return row_combine<T>(v, slot, [](float a, float b) { return a + b; });
}
template <int T>
__device__ __forceinline__ uint32_t row_max(uint32_t v, uint32_t* slot) {
  return row_combine<T>(v, slot, [](uint32_t a, uint32_t b) { return a > b ? a : b; });
}

// ---------------------------------------------------------------------------
// Rows in 8 bits.
// ---------------------------------------------------------------------------
// q = round(127 x / m) with ties to even, exact for x and m (the largest |x|)
// of a 16-bit type: with significands a and c below 2^11 the quotient is a tie
// or at least 1 / 254 a > 2^-19 of its own size off every tie.  127 x is exact, the
// reciprocal and the product are off by 2^-23 together, and rounding to 20
// significant bits moves the result by 2^-20 at most: it takes quotients that
// are ties back to them (a tie has 8 significant bits) and the others across
// none.  Seven operations an element, where a division takes about as many
// again.  `by` is 127 times a power of two and `inv` the reciprocal of m times
// the same power, which keeps both products of any m within fp32.
struct Quantizer {
  float by, inv, scale;
  // m: the bits of the largest |x|, which order as the values do, infinities and NaN on top.
  // Rows that hold one of those get NaN as their scale and zeros, which carries the NaN into what is made of them.
  __device__ __forceinline__ explicit Quantizer(uint32_t m) {
    const float top = __builtin_bit_cast(float, m);
    const bool finite = m < 0x7f800000u, some = m != 0;
    const float k = top >= 0x1p100f ? 0x1p-64f : top < 0x1p-64f ? 0x1p64f : 1.0f;
    by = finite && some ? 127.0f * k : 0.0f;
    inv = finite && some ? 1.0f / (top * k) : 0.0f;
    scale = finite ? top / 127.0f : __builtin_nanf("");
  }
  __device__ __forceinline__ int operator()(float x) const {
    const float t = (x * by) * inv;
    const uint32_t u = (__builtin_bit_cast(uint32_t, t) + 8u) & ~15u;
    return (int)__builtin_rintf(__builtin_bit_cast(float, u));
  }
  __device__ __forceinline__ void store(int8_t* p, int valid, const float (&f)[8]) const {
    uint32_t w[2] = {0, 0};
#pragma unroll
    for (int e = 0; e < 8; ++e) w[e / 4] |= ((uint32_t)(*this)(f[e]) & 255u) << (8 * (e & 3));
    if (inv == 0.0f) w[0] = w[1] = 0;  // (infinities and NaN times zero)
    if (valid >= 8) {
      __builtin_memcpy(p, w, 8);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (e < valid) p[e] = (int8_t)(w[e / 4] >> (8 * (e & 3)));
    }
  }
};
__device__ __forceinline__ uint32_t abs_bits(float x) { return __builtin_bit_cast(uint32_t, x) & 0x7fffffffu; }
__device__ __forceinline__ uint32_t max_bits(uint32_t m, const float (&f)[8], int valid) {
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (e < valid) m = max(m, abs_bits(f[e]));
  return m;
}

// ---------------------------------------------------------------------------
// Forward: the norm, and rows in 8 bits.
// ---------------------------------------------------------------------------
struct RowArgs {
  long long M;
  int N;
  const uint8_t* X;
  long long ldx;  // elements, as all of them
  float inv_n, eps;
  const float *gamma, *beta;  // or NULL: 1, 0
  uint8_t* Y;                 // or NULL
  long long ldy;
  float *mean, *rstd;  // or NULL
  int8_t* Q;
  long long ldq;
  float* scale;  // or NULL: no rows in 8 bits
};

// A row by T threads: 64 take rows of a wave each, more share a workgroup's
// row.  C: the row stays in registers, C chunks of 8 elements a thread; 0: it is
// read again in every pass.  NORM: the norm of the rows (Y, Q or both);
// otherwise Q alone.  X of type XT, Y and what is put into 8 bits of type OT.
template <bool NORM, int XT, int OT, int T, int C>
__global__ void __launch_bounds__(T < 256 ? 256 : T) row_kernel(const RowArgs p) {
  constexpr int RG = T < 256 ? 256 / T : 1;  // rows of a workgroup
  constexpr int W = T / 64;
  __shared__ float sums[2][W];
  __shared__ uint32_t tops[2][W];
  const int t = threadIdx.x % T;
  int turn = 0;
  for (long long row = (long long)blockIdx.x * RG + threadIdx.x / T; row < p.M; row += (long long)gridDim.x * RG, turn ^= 1) {
    const uint8_t* const x = p.X + row * p.ldx * Raw<XT>::EB;
    Raw<XT> keep[C ? C : 1];
    // f(chunk of 8, its first column, how many of its columns are in the row)
    auto chunks = [&](bool first, auto&& f) {
      if constexpr (C > 0) {
#pragma unroll
        for (int j = 0; j < C; ++j) {
          const int c = (j * T + t) * 8;
          if (first && c < p.N) keep[j].load(x + (long long)c * Raw<XT>::EB, p.N - c);
        }
#pragma unroll
        for (int j = 0; j < C; ++j) {
          const int c = (j * T + t) * 8;
          if (c < p.N) {
            float v[8];
            keep[j].get(v);
            f(v, c, min(p.N - c, 8));
          }
        }
      } else {
        for (int c = t * 8; c < p.N; c += T * 8) {
          float v[8];
          keep[0].load(x + (long long)c * Raw<XT>::EB, p.N - c);
          keep[0].get(v);
          f(v, c, min(p.N - c, 8));
        }
      }
    };
    float mean = 0.0f, rstd = 1.0f;
    if constexpr (NORM) {
      float s = 0.0f;
      chunks(true, [&](const float(&v)[8], int, int n) {
#pragma unroll
        for (int e = 0; e < 8; ++e) s += v[e];  // (zeros past the row)
      });
      mean = row_sum<T>(s, sums[0]) * p.inv_n;
      s = 0.0f;
      chunks(false, [&](const float(&v)[8], int, int n) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float d = e < n ? v[e] - mean : 0.0f;
          s = __builtin_fmaf(d, d, s);
        }
      });
      rstd = 1.0f / __builtin_sqrtf(row_sum<T>(s, sums[1]) * p.inv_n + p.eps);
      if (t == 0 && p.mean) p.mean[row] = mean;
      if (t == 0 && p.rstd) p.rstd[row] = rstd;
    }
    auto normed = [&](float(&v)[8], int c, int n) {
      if constexpr (NORM) {
        float g[8], b[8];
        if (p.gamma) load_f32<8>(p.gamma + c, n, g);
        if (p.beta) load_f32<8>(p.beta + c, n, b);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          v[e] = (v[e] - mean) * rstd;
          if (p.gamma) v[e] *= g[e];
          if (p.beta) v[e] += b[e];
        }
      }
    };
    uint32_t top = 0;
    if (!NORM || p.Y || p.scale) {
      chunks(!NORM, [&](float(&v)[8], int c, int n) {
        normed(v, c, n);
        Raw<OT> out;
        out.set(v);
        if (p.Y) out.store(p.Y + (row * p.ldy + c) * Raw<OT>::EB, n);
        if (p.scale) {
          out.get(v);
          top = max_bits(top, v, n);
        }
      });
    }
    if (p.scale) {
      const Quantizer q(row_max<T>(top, tops[turn]));
      if (t == 0) p.scale[row] = q.scale;
      chunks(false, [&](float(&v)[8], int c, int n) {
        normed(v, c, n);
        Raw<OT> out;
        out.set(v);
        out.get(v);
        q.store(p.Q + row * p.ldq + c, n, v);
      });
    }
  }
}

// ---------------------------------------------------------------------------
// Backward.
// ---------------------------------------------------------------------------
struct NormBackArgs {
  long long M;
  int N;
  const uint8_t *dY, *X, *R;  // R: or NULL
  long long lddy, ldx, ldr;
  const float *mean, *rstd, *gamma;  // gamma: or NULL
  float inv_n;
  uint8_t* dX;  // or NULL
  long long lddx;
  float2* stats;  // mean(g) and mean(g xh) of each row
  float* sums;    // or NULL: dgamma and dbeta of each row block, [blocks][2][width]
  int width;      // N rounded up to a multiple of 64
  int rows, groups, blocks;  // rows of a block; workgroups across the columns and down the rows
};

// mean(g) and mean(g xh) of every row.
template <int XT, int OT, int T>
__global__ void __launch_bounds__(T < 256 ? 256 : T) norm_back_stats_kernel(const NormBackArgs p) {
  constexpr int RG = T < 256 ? 256 / T : 1, W = T / 64;
  __shared__ float sums[2][W];
  const int t = threadIdx.x % T;
  for (long long row = (long long)blockIdx.x * RG + threadIdx.x / T; row < p.M; row += (long long)gridDim.x * RG) {
    const float mean = p.mean[row], rstd = p.rstd[row];
    float s = 0.0f, sx = 0.0f;
    for (int c = t * 8; c < p.N; c += T * 8) {
      const int n = min(p.N - c, 8);
      Raw<OT> dy;
      Raw<XT> x;
      dy.load(p.dY + (row * p.lddy + c) * Raw<OT>::EB, n);
      x.load(p.X + (row * p.ldx + c) * Raw<XT>::EB, n);
      float d[8], v[8], g[8];
      dy.get(d);
      x.get(v);
      if (p.gamma) load_f32<8>(p.gamma + c, n, g);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float ge = e < n ? (p.gamma ? d[e] * g[e] : d[e]) : 0.0f;
        s += ge;
        if (e < n) sx = __builtin_fmaf(ge, (v[e] - mean) * rstd, sx);
      }
    }
    s = row_sum<T>(s, sums[0]);
    sx = row_sum<T>(sx, sums[1]);
    if (t == 0) p.stats[row] = make_float2(s * p.inv_n, sx * p.inv_n);
  }
}

// dX, and the sums down the rows of a block: 512 columns (8 a lane) by p.rows
// rows, which the four waves take in turn.
template <int XT, int OT>
__global__ void __launch_bounds__(256) norm_back_kernel(const NormBackArgs p) {
  __shared__ float part[2][4][512];
  const int lane = threadIdx.x & 63, wave = wave_id();
  const int by = blockIdx.x / p.groups, bx = blockIdx.x - by * p.groups;
  const int c = bx * 512 + lane * 8, n = min(p.N - c, 8);
  float sg[8], sb[8], gamma[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) sg[e] = sb[e] = 0.0f;
  if (n > 0) {
#pragma unroll
    for (int e = 0; e < 8; ++e) gamma[e] = 1.0f;
    if (p.gamma) load_f32<8>(p.gamma + c, n, gamma);
    const long long r0 = (long long)by * p.rows, r1 = min(p.M, r0 + p.rows);
    for (long long row = r0 + wave; row < r1; row += 4) {
      const float mean = p.mean[row], rstd = p.rstd[row];
      Raw<OT> dy;
      Raw<XT> x, r;
      dy.load(p.dY + (row * p.lddy + c) * Raw<OT>::EB, n);
      x.load(p.X + (row * p.ldx + c) * Raw<XT>::EB, n);
      float d[8], v[8], a[8];
      dy.get(d);
      x.get(v);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        v[e] = (v[e] - mean) * rstd;
        sg[e] = __builtin_fmaf(d[e], v[e], sg[e]);
        sb[e] += d[e];
      }
      if (p.dX) {
        const float2 m = p.stats[row];
        if (p.R) {
          r.load(p.R + (row * p.ldr + c) * Raw<XT>::EB, n);
          r.get(a);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          v[e] = rstd * (__builtin_fmaf(-v[e], m.y, d[e] * gamma[e]) - m.x);
          if (p.R) v[e] += a[e];
        }
        x.set(v);
        x.store(p.dX + (row * p.lddx + c) * Raw<XT>::EB, n);
      }
    }
  }
  if (!p.sums) return;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    part[0][wave][lane * 8 + e] = sg[e];
    part[1][wave][lane * 8 + e] = sb[e];
  }
  __syncthreads();
  for (int i = threadIdx.x; i < 2 * 512; i += 256) {
    const int which = i / 512, cc = i % 512, col = bx * 512 + cc;
    if (col < p.N)
      p.sums[((long long)by * 2 + which) * p.width + col] =
          (part[which][0][cc] + part[which][1][cc]) + (part[which][2][cc] + part[which][3][cc]);
  }
}

}  // namespace igc_rows
