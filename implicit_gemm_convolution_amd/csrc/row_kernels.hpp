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

// Eight elements of type T (igc_ffn::Type) as they lie in memory: those of a row
// of n elements from column c, zeros past the row.  The chunk at a row's end is
// loaded as the row's last eight elements (element by element, its loads would
// wait for one another) and shifted into place by settle(), where it is used: at
// the load the shift would wait for the data, and the workgroup's other waves for
// that one at the next barrier (backward of 8192 x 4095 bf16 73 us, so 54; rows in 8
// bits of 8192 x 4097 25, so 22).
// Whole chunks are written past the caches, wherever they lie.  In the caches and
// past them, us, each in the form that its kernel had when this was tried: norm of
// 8192 x 4096 bf16 32.7 and 26.7 (22 now), of 1000 x 4096 9.1 and 7.8 (5.6 now), of 8192 x
// 4095 35 and 26.6, of 2048 x 20001 63 and 52; rows in 8 bits of 8192 x 4097 33 and 25
// (22 now); the backward pass of 8192 x 4095 75 and 73 (54 now); dropout of 8192 x 8191
// from -3 to +3%.
typedef uint32_t u32x4 __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2), aligned(1)));
typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
template <int T>
struct Raw {
  static constexpr int EB = 2;
  uint4 v;
  __device__ __forceinline__ void load(const uint8_t* row, int c, int n) {
    if (n >= 8)
      v = load8(row + (long long)min(c, n - 8) * 2, 8);
    else
      v = load8(row, n);
  }
  __device__ __forceinline__ void settle(int c, int n) {
    if (n - c >= 8 || c == 0) return;
    unsigned __int128 w;
    __builtin_memcpy(&w, &v, 16);
    w >>= 16 * (c + 8 - n);
    __builtin_memcpy(&v, &w, 16);
  }
  __device__ __forceinline__ void get(float (&f)[8]) const { unpack8<T == T_BF16>(v, f); }
  __device__ __forceinline__ void set(const float (&f)[8]) { v = pack8<T == T_BF16>(f); }
  __device__ __forceinline__ void clear_from(int n) {  // zeros from element n (1 to 7) on
    unsigned __int128 w;
    __builtin_memcpy(&w, &v, 16);
    w = w << 16 * (8 - n) >> 16 * (8 - n);
    __builtin_memcpy(&v, &w, 16);
  }
  // The bits of the largest |value|: they order as the values do, infinities
  // and NaN on top.
  __device__ __forceinline__ uint32_t top() const {
    auto abs = [](uint32_t w) { return __builtin_bit_cast(u16x2, w & 0x7fff7fffu); };
    const u16x2 m = __builtin_elementwise_max(__builtin_elementwise_max(abs(v.x), abs(v.y)), __builtin_elementwise_max(abs(v.z), abs(v.w)));
    return max((uint32_t)m[0], (uint32_t)m[1]);
  }
  __device__ __forceinline__ void store(uint8_t* row, int c, int n) const {
    uint8_t* const p = row + (long long)c * 2;
    if (n - c >= 8)
      __builtin_nontemporal_store(u32x4{v.x, v.y, v.z, v.w}, reinterpret_cast<u32x4*>(p));
    else
      store8(p, v, n - c);
  }
};
template <>
struct Raw<T_F32> {
  static constexpr int EB = 4;
  float v[8];
  __device__ __forceinline__ void load(const uint8_t* row, int c, int n) {
    const float* const p = reinterpret_cast<const float*>(row);
    if (n >= 8)
      load_f32<8>(p + min(c, n - 8), 8, v);
    else
      load_f32<8>(p, n, v);
  }
  __device__ __forceinline__ void settle(int c, int n) {
    if (n - c >= 8 || c == 0) return;
    const int over = c + 8 - n;
#pragma unroll
    for (int s = 4; s; s >>= 1)
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = !(over & s) ? v[e] : e + s < 8 ? v[(e + s) & 7] : 0.0f;
  }
  __device__ __forceinline__ void get(float (&f)[8]) const {
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = v[e];
  }
  __device__ __forceinline__ void set(const float (&f)[8]) {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = f[e];
  }
  __device__ __forceinline__ void store(uint8_t* row, int c, int n) const {
    float* const p = reinterpret_cast<float*>(row) + c;
    if (n - c >= 8) {
      u32x4 w[2];
      __builtin_memcpy(w, v, 32);
      __builtin_nontemporal_store(w[0], reinterpret_cast<u32x4*>(p));
      __builtin_nontemporal_store(w[1], reinterpret_cast<u32x4*>(p) + 1);
    } else {
      store_f32<8>(p, n - c, v);
    }
  }
};
// Of a vector of n fp32 values.
__device__ __forceinline__ void load_vector(const float* p, int c, int n, float (&f)[8]) {
  Raw<T_F32> r;
  r.load(reinterpret_cast<const uint8_t*>(p), c, n);
  r.settle(c, n);
  r.get(f);
}

// ---------------------------------------------------------------------------
// Sums and maxima over the threads of a row.
// ---------------------------------------------------------------------------
// The lanes of a group of T (2 to 64) combined in every one of them:
// within rows of 16 lanes by cross-lane operands of the vector unit, the four
// rows of a wave through scalar registers (the way through LDS, a shuffle a step,
// takes twelve trips of over 60 cycles each).  The order is fixed, and the same
// in every lane.
template <int T, class V, class F>
__device__ __forceinline__ V wave_combine(V v, F&& f) {
  static_assert(sizeof(V) == 4, "one register");
  auto other = [](V x, auto ctrl) {
    return __builtin_bit_cast(V, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, x), decltype(ctrl)::value, 0xf, 0xf, true));
  };
  v = f(v, other(v, std::integral_constant<int, 0xB1>()));                          // quad_perm [1, 0, 3, 2]
  if constexpr (T >= 4) v = f(v, other(v, std::integral_constant<int, 0x4E>()));    // quad_perm [2, 3, 0, 1]
  if constexpr (T >= 8) v = f(v, other(v, std::integral_constant<int, 0x141>()));   // the other half of 8
  if constexpr (T >= 16) v = f(v, other(v, std::integral_constant<int, 0x140>()));  // the other half of 16
  if constexpr (T <= 16) return v;
  auto lane = [&](int l) { return __builtin_bit_cast(V, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), l)); };
  const V low = f(lane(0), lane(16)), high = f(lane(32), lane(48));
  if constexpr (T == 32) return (threadIdx.x & 32) ? high : low;
  return f(low, high);
}

// N values of every thread of a row's T threads, combined in every one of
// them: the lanes of a wave, then the waves through LDS, a lane for each, with
// one barrier (of the whole workgroup).  slot: W entries of the row.  Calls take
// slots in turn, two at least: who writes a slot again has passed the barrier of
// the other one, which everyone reaches after reading this one.
template <int T, int N, class V, class F>
__device__ __forceinline__ void row_combine(V (&v)[N], V (*slot)[N], F&& f) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = wave_combine<(T < 64 ? T : 64)>(v[i], f);
  if constexpr (T > 64) {
    const int t = threadIdx.x % T;
    if ((t & 63) == 0) {
#pragma unroll
      for (int i = 0; i < N; ++i) slot[t >> 6][i] = v[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = wave_combine<T / 64>(slot[t % (T / 64)][i], f);
  }
}
template <int T>
__device__ __forceinline__ float row_sum(float v, float (*slot)[1]) {
  float a[1] = {v};
  row_combine<T, 1>(a, slot, [](float x, float y) { return x + y; });
  return a[0];
}
template <int T>
__device__ __forceinline__ uint32_t row_max(uint32_t v, uint32_t (*slot)[1]) {
  uint32_t a[1] = {v};
  row_combine<T, 1>(a, slot, [](uint32_t x, uint32_t y) { return x > y ? x : y; });
  return a[0];
}

// ---------------------------------------------------------------------------
// Rows in 8 bits.
// ---------------------------------------------------------------------------
// q = round(127 x / m) with ties to even, exact for x and m (the largest |x|)
// of a 16-bit type: with significands a and c below 2^11 the quotient is a tie
// or at least 1 / 254 a > 2^-19 of its own size off every tie.  127 x is exact, the
// reciprocal (an ulp) and the product (half of one) are off by 1.5 2^-23
// together, and rounding to 20 significant bits moves the result by 2^-20 at
// most: it takes quotients that are ties back to them (a tie has 8 significant
// bits) and the others across none.  Adding 1.5 2^23 then rounds to a whole
// number, ties to even, and leaves it in the lowest byte.  Five operations an
// element, and three for four to pack them (8192 x 4096 bf16 17.0 us, 5.9 TB/s;
// 21.9 with a conversion and shifts).  `by` is 127 times a power of two and `inv`
// the reciprocal of m times the same power, which keeps both products of any m
// within fp32.
struct Quantizer {
  float by, inv;
  // m: the bits of the largest |x| of a row of type T.  Rows with an infinity or NaN
  // get NaN as their scale and zeros, which carries the NaN into what is made of them.
  template <int T>
  __device__ __forceinline__ static Quantizer of(uint32_t m) {
    const float top = value<T>(m);
    const bool finite = m < limit<T>(), some = m != 0;
    const float k = top >= 0x1p100f ? 0x1p-64f : top < 0x1p-64f ? 0x1p64f : 1.0f;
    Quantizer q;
    q.by = 127.0f * k;
    q.inv = finite && some ? __builtin_amdgcn_rcpf(top * k) : 0.0f;
    return q;
  }
  template <int T>
  __device__ __forceinline__ static float scale(uint32_t m) {
    return m < limit<T>() ? value<T>(m) / 127.0f : __builtin_nanf("");
  }
  template <int T>
  __device__ __forceinline__ static float value(uint32_t m) {
    return T == T_BF16 ? __builtin_bit_cast(float, m << 16) : (float)__builtin_bit_cast(_Float16, (uint16_t)m);
  }
  template <int T>
  __device__ __forceinline__ static constexpr uint32_t limit() {
    return T == T_BF16 ? 0x7f80u : 0x7c00u;
  }
  __device__ __forceinline__ uint32_t operator()(float x) const {  // in the lowest byte
    const float t = (x * by) * inv;
    const uint32_t u = (__builtin_bit_cast(uint32_t, t) + 8u) & ~15u;
    return __builtin_bit_cast(uint32_t, __builtin_bit_cast(float, u) + 12582912.0f);
  }
  __device__ __forceinline__ void store(int8_t* p, int valid, const float (&f)[8]) const {
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t a = __builtin_amdgcn_perm((*this)(f[i * 4 + 1]), (*this)(f[i * 4]), 0x0c0c0400u);
      const uint32_t b = __builtin_amdgcn_perm((*this)(f[i * 4 + 3]), (*this)(f[i * 4 + 2]), 0x0c0c0400u);
      w[i] = inv == 0.0f ? 0u : a | b << 16;  // (infinities and NaN times zero)
    }
    if (valid >= 8) {
      __builtin_nontemporal_store(u32x2{w[0], w[1]}, reinterpret_cast<u32x2*>(p));
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (e < valid) p[e] = (int8_t)(w[e / 4] >> (8 * (e & 3)));
    }
  }
};

// ---------------------------------------------------------------------------
// Forward: the norm, and rows in 8 bits.
// ---------------------------------------------------------------------------
// Division by a whole number: with 1 / n in two parts the quotient is the nearest
// number.  (By the first part alone it may be the one next to an exact quotient: a
// row of 41 times 60000 has 59999.996 as its mean then, which eps = 1e-5 turns into
// values of 0.7.)
struct Divisor {
  float inv, rest;
  __host__ __device__ static Divisor by(int n) {
    const float f = (float)n, inv = n > 0 ? 1.0f / f : 0.0f;
    return Divisor{inv, n > 0 ? __builtin_fmaf(-inv, f, 1.0f) * inv : 0.0f};
  }
  __device__ __forceinline__ float of(float s) const { return __builtin_fmaf(s, inv, s * rest); }
};

struct RowArgs {
  long long M;
  int N;
  const uint8_t* X;
  long long ldx;  // elements, as all of them
  Divisor n;
  float eps;
  const float *gamma, *beta;  // or NULL: 1, 0
  uint8_t* Y;                 // or NULL
  long long ldy;
  float *mean, *rstd;  // or NULL
  int8_t* Q;
  long long ldq;
  float* scale;  // or NULL: no rows in 8 bits
};

// 1 / sqrt(v), off by 2^-23 of its size at most (the square root and the division
// in full, 27 instructions in every thread for 2, where v may be too small for
// the instruction).
__device__ __forceinline__ float rsqrt_of(float v) {
  return v < 0x1p-100f ? 1.0f / __builtin_sqrtf(v) : __builtin_amdgcn_rsqf(v);
}

// What does not change from row to row: the number of elements that this thread's
// wave holds, and how many the wave holds whose part this lane takes.
struct WaveShare {
  Divisor own{};
  float lane = 0.0f;
  template <int T, int C>
  __device__ __forceinline__ static WaveShare of(int t, int n) {
    WaveShare r;
    auto held = [&](int w) {
      int k = 0;
#pragma unroll
      for (int j = 0; j < C; ++j) k += min(max(n - (j * T + w * 64) * 8, 0), 512);
      return k;
    };
    if constexpr (T > 64) {
      r.own = Divisor::by(__builtin_amdgcn_readfirstlane(held(t >> 6)));
      r.lane = (float)held(t % (T / 64));
    }
    return r;
  }
};
// Mean and variance of a row in its threads' registers, with one barrier: every
// wave takes the mean of its own elements and their squared distances from it,
// and the waves' parts join as M2 = sum of M2_w + n_w (mean_w - mean)^2: no
// difference of large squares anywhere.  Rows of one 16-bit value have it as their
// mean: sums of 11 bits over up to 8192 elements are exact, and of longer rows the
// means' distances from the first one are summed.  (With a barrier for the mean and
// one for the distances from it 8192 x 4096 bf16 took 26.7 us, so 24.2, and 22.3 with
// what came after.)
template <int T, int C>
__device__ __forceinline__ void row_stats(float (&v)[C][8], int t, int n, const Divisor& by, const WaveShare& w, float2* parts, float& mean,
                                          float& var) {
  constexpr int WT = T < 64 ? T : 64, W = T / 64;
  auto add = [](float a, float b) { return a + b; };
  float s = 0.0f;
#pragma unroll
  for (int j = 0; j < C; ++j)
#pragma unroll
    for (int e = 0; e < 8; ++e) s += v[j][e];  // (zeros past the row)
  s = wave_combine<WT>(s, add);
  const float m = T <= 64 ? by.of(s) : w.own.of(s);
  float d2 = 0.0f;
#pragma unroll
  for (int j = 0; j < C; ++j) {
    const int c = (j * T + t) * 8;
    const float mc = c < n ? m : 0.0f;  // (chunks past the row are zeros, and their distances)
    if ((n & 7) && c < n && c + 8 > n) {  // the row's last chunk: no distance from the mean past the row
#pragma unroll
      for (int e = 1; e < 8; ++e) v[j][e] = c + e < n ? v[j][e] : m;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float d = v[j][e] - mc;
      d2 = __builtin_fmaf(d, d, d2);
    }
  }
  d2 = wave_combine<WT>(d2, add);
  if constexpr (T <= 64) {
    mean = m;
    var = d2 * by.inv;
  } else {
    if ((t & 63) == 0) parts[t >> 6] = make_float2(m, d2);
    __syncthreads();
    const float2 a = parts[t % W];  // (a lane for each wave's part)
    if constexpr (C > 1) {
      const float first = parts[0].x;
      mean = first + wave_combine<W>((a.x - first) * w.lane, add) * by.inv;
    } else {
      mean = by.of(wave_combine<W>(a.x * w.lane, add));
    }
    // (a wave past the row has no mean: 0 of its squares may be 0 times infinity.  Rows by two waves, or by two chunks a thread, leave none.)
    const float d = W > 2 && C == 1 && w.lane == 0.0f ? 0.0f : a.x - mean;
    var = wave_combine<W>(__builtin_fmaf(d * d, w.lane, a.y), add) * by.inv;
  }
}

// A row by T threads, in registers: C chunks of 8 elements a thread, 256 / T
// rows of a workgroup at a time where T is less.  NORM: the norm of the rows (Y,
// Q or both); otherwise Q alone.  X of type XT, Y and what is put into 8 bits of
// type OT.  A workgroup walks over rows: gamma and beta stay in registers, and
// the next row is on its way while this one is summed.
template <int T>
constexpr int row_threads = T < 256 ? 256 : T;
template <bool NORM, int XT, int OT, int T, int C>
__global__ void __launch_bounds__(row_threads<T>, C > 1 ? 4 : T == 128 || (XT == T_F32 && T < 1024) ? 7 : 8) row_kernel(const RowArgs p) {
  constexpr int RG = row_threads<T> / T;  // rows of a workgroup
  constexpr int W = T < 64 ? 1 : T / 64;
  __shared__ float2 parts[2][RG][W];
  __shared__ uint32_t tops[2][RG][W][1];
  const int t = threadIdx.x % T, rg = threadIdx.x / T;
  auto col = [&](int j) { return (j * T + t) * 8; };
  const WaveShare share = WaveShare::of<T, C>(t, p.N);
  float gamma[C][8], beta[C][8];
  Raw<XT> next[C];
  auto load = [&](long long row) {
#pragma unroll
    for (int j = 0; j < C; ++j)
      if (col(j) < p.N) next[j].load(p.X + row * p.ldx * Raw<XT>::EB, col(j), p.N);
  };
  const long long step = (long long)gridDim.x * RG;
  long long first = (long long)blockIdx.x * RG;
  if (first + rg < p.M) load(first + rg);
  if constexpr (NORM) {
#pragma unroll
    for (int j = 0; j < C; ++j) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        gamma[j][e] = 1.0f;
        beta[j][e] = 0.0f;
      }
      if (p.gamma && col(j) < p.N) load_vector(p.gamma, col(j), p.N, gamma[j]);
      if (p.beta && col(j) < p.N) load_vector(p.beta, col(j), p.N, beta[j]);
    }
  }
  for (int turn = 0; first < p.M; first += step, turn ^= 1) {  // (as often for every row of the workgroup: the barriers)
    const long long row = first + rg;
    const bool in = row < p.M;
    Raw<OT> out[C];
    if constexpr (NORM) {
      float v[C][8];
#pragma unroll
      for (int j = 0; j < C; ++j)
        if (in && col(j) < p.N) {
          next[j].settle(col(j), p.N);
          next[j].get(v[j]);
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) v[j][e] = 0.0f;
        }
      if (row + step < p.M) load(row + step);
      float mean, var;
      row_stats<T, C>(v, t, p.N, p.n, share, parts[turn][rg], mean, var);
      const float rstd = rsqrt_of(var + p.eps);
      if (in && t == 0 && p.mean) p.mean[row] = mean;
      if (in && t == 0 && p.rstd) p.rstd[row] = rstd;
#pragma unroll
      for (int j = 0; j < C; ++j) {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[j][e] = __builtin_fmaf((v[j][e] - mean) * rstd, gamma[j][e], beta[j][e]);
        out[j].set(v[j]);
        if (p.Y && in && col(j) < p.N) out[j].store(p.Y + row * p.ldy * Raw<OT>::EB, col(j), p.N);
        if ((p.N & 7) && col(j) < p.N && p.N - col(j) < 8) out[j].clear_from(p.N - col(j));
      }
    } else {
#pragma unroll
      for (int j = 0; j < C; ++j) {
        out[j] = next[j];
        if (col(j) < p.N) out[j].settle(col(j), p.N);
      }
      if (row + step < p.M) load(row + step);
    }
    if (p.scale) {
      uint32_t top = 0;
#pragma unroll
      for (int j = 0; j < C; ++j)
        if (in && col(j) < p.N) top = max(top, out[j].top());
      top = row_max<T>(top, tops[turn][rg]);
      const Quantizer q = Quantizer::of<OT>(top);
      if (in && t == 0) p.scale[row] = Quantizer::scale<OT>(top);
#pragma unroll
      for (int j = 0; j < C; ++j)
        if (in && col(j) < p.N) {
          float v[8];
          out[j].get(v);
          q.store(p.Q + row * p.ldq + col(j), p.N - col(j), v);
        }
    }
  }
}

// Elements that a thread adds one after the other in fp32: of longer rows these
// sums are added in fp64 (2^18 additions of 40.1 in fp32 alone would be off by one
// in a thousand, each of them rounded the same way).
constexpr uint32_t SEGMENT = 512;

// Rows that registers do not hold: read again in every pass.
template <bool NORM, int XT, int OT, int T>
__global__ void __launch_bounds__(T, 8) long_row_kernel(const RowArgs p) {
  constexpr int W = T / 64;
  __shared__ float sums[W][1], squares[W][2];
  __shared__ uint32_t tops[2][W][1];
  int turn = 0;
  for (long long row = blockIdx.x; row < p.M; row += gridDim.x, turn ^= 1) {
    const uint8_t* const x = p.X + row * p.ldx * Raw<XT>::EB;
    // f(chunk of 8, its first column, how many of its columns are in the row) for this
    // thread's chunks from column u to column `end`; the next one's column
    auto chunks = [&](uint32_t u, uint32_t end, auto&& f) {
      for (; u < end; u += T * 8) {  // (steps past 2^31 at most once)
        const int c = (int)u;
        float v[8];
        Raw<XT> raw;
        raw.load(x, c, p.N);
        raw.settle(c, p.N);
        raw.get(v);
        f(v, c, min(p.N - c, 8));
      }
      return u;
    };
    // K sums over the row: f as above adds to sums[K].
    auto sum = [&](auto& sums, auto&& f) {
      constexpr int K = sizeof(sums) / sizeof(float);
      double total[K] = {};
      for (uint32_t u = threadIdx.x * 8; u < (uint32_t)p.N;) {
#pragma unroll
        for (int i = 0; i < K; ++i) sums[i] = 0.0f;
        u = chunks(u, (uint32_t)min((long long)p.N, (long long)u + SEGMENT * T), f);
#pragma unroll
        for (int i = 0; i < K; ++i) total[i] += (double)sums[i];
      }
#pragma unroll
      for (int i = 0; i < K; ++i) sums[i] = (float)total[i];
    };
    auto all = [&](auto&& f) { chunks(threadIdx.x * 8, (uint32_t)p.N, f); };
    float mean = 0.0f, rstd = 1.0f;
    if constexpr (NORM) {
      float s[1];
      sum(s, [&](const float(&v)[8], int, int) {
#pragma unroll
        for (int e = 0; e < 8; ++e) s[0] += v[e];  // (zeros past the row)
      });
      mean = p.n.of(row_sum<T>(s[0], sums));
      // The mean is off by the rounding of so many additions: by the mean of the
      // distances from it, which is added to it and whose square goes out of theirs.
      float m[2];
      sum(m, [&](float(&v)[8], int, int n) {
        if (n < 8) {  // (nothing past the row)
#pragma unroll
          for (int e = 1; e < 8; ++e) v[e] = e < n ? v[e] : mean;
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float d = v[e] - mean;
          m[0] += d;
          m[1] = __builtin_fmaf(d, d, m[1]);
        }
      });
      row_combine<T, 2>(m, squares, [](float f, float g) { return f + g; });
      const float off = m[0] * p.n.inv, around = m[1] * p.n.inv, least = around - off * off;
      mean += off;
      const float var = around < __builtin_inff() ? (least < 0.0f ? 0.0f : least) : around;
      rstd = rsqrt_of(var + p.eps);
      if (threadIdx.x == 0 && p.mean) p.mean[row] = mean;
      if (threadIdx.x == 0 && p.rstd) p.rstd[row] = rstd;
    }
    auto normed = [&](float(&v)[8], int c, int n) {  // rounded to OT
      if constexpr (NORM) {
        float g[8], b[8];
        if (p.gamma) load_vector(p.gamma, c, p.N, g);
        if (p.beta) load_vector(p.beta, c, p.N, b);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          v[e] = __builtin_fmaf((v[e] - mean) * rstd, p.gamma ? g[e] : 1.0f, p.beta ? b[e] : 0.0f);
          // (both passes round this fp32 value: an instruction that rounds the sum straight to fp16 may be chosen in one alone)
          asm("" : "+v"(v[e]));
        }
      }
      Raw<OT> out;
      out.set(v);
      out.get(v);
      return out;
    };
    uint32_t top = 0;
    if (!NORM || p.Y || p.scale) {
      all([&](float(&v)[8], int c, int n) {
        Raw<OT> out = normed(v, c, n);
        if (p.Y) out.store(p.Y + row * p.ldy * Raw<OT>::EB, c, p.N);
        if (n < 8) out.clear_from(n);
        top = max(top, out.top());
      });
    }
    if (p.scale) {
      top = row_max<T>(top, tops[turn]);
      const Quantizer q = Quantizer::of<OT>(top);
      if (threadIdx.x == 0) p.scale[row] = Quantizer::scale<OT>(top);
      all([&](float(&v)[8], int c, int n) {
        normed(v, c, n);
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

// Rows in registers: T threads a row, a chunk of 8 elements a thread, 1024 / T
// rows at a time, one reduction of two sums a row, and the sums down the rows
// in the registers of the threads that hold their columns.  Each input is read
// once.  The next row is on its way while this one is summed.  (8192 x 4096 bf16
// with a residual 49 us, 5.4 TB/s, and 4.5 for the second launch; two launches that read
// dY and X twice 75.)
template <int XT, int OT, int T>
__global__ void __launch_bounds__(1024) norm_back_rows_kernel(const NormBackArgs p) {
  constexpr int RG = 1024 / T, W = T < 64 ? 1 : T / 64, COLS = T * 8;
  __shared__ float slots[2][RG][W][2];
  __shared__ float part[RG > 1 ? RG * COLS : 1];
  const int t = threadIdx.x % T, rg = threadIdx.x / T;
  const int c = t * 8;
  const bool have = c < p.N;
  float gamma[8], sg[8], sb[8];
  Raw<OT> dy;
  Raw<XT> x, r;
  float next_mean = 0.0f, next_rstd = 0.0f;
  auto load = [&](long long row) {
    next_mean = p.mean[row];
    next_rstd = p.rstd[row];
    if (have) {
      dy.load(p.dY + row * p.lddy * Raw<OT>::EB, c, p.N);
      x.load(p.X + row * p.ldx * Raw<XT>::EB, c, p.N);
      if (p.R) r.load(p.R + row * p.ldr * Raw<XT>::EB, c, p.N);
    }
  };
  const long long step = (long long)gridDim.x * RG;
  long long first = (long long)blockIdx.x * RG;
  if (first + rg < p.M) load(first + rg);
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    gamma[e] = 1.0f;
    sg[e] = sb[e] = 0.0f;
  }
  if (p.gamma && have) load_vector(p.gamma, c, p.N, gamma);
  for (int turn = 0; first < p.M; first += step, turn ^= 1) {  // (as often for every row of the workgroup: the barrier)
    const long long row = first + rg;
    const bool in = row < p.M;
    const float mean = in ? next_mean : 0.0f, rstd = in ? next_rstd : 0.0f;
    float d[8], v[8], a[8];
    if (in && have) {
      dy.settle(c, p.N);
      dy.get(d);
      x.settle(c, p.N);
      x.get(v);
      if (p.R) {
        r.settle(c, p.N);
        r.get(a);
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) d[e] = v[e] = a[e] = 0.0f;
    }
    if (row + step < p.M) load(row + step);
    float m[2] = {0.0f, 0.0f};
    const float from = have ? mean : 0.0f;  // (what lies past the row is 0, and 0 from there)
    if ((p.N & 7) && have && c + 8 > p.N) {
#pragma unroll
      for (int e = 1; e < 8; ++e) v[e] = c + e < p.N ? v[e] : from;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      v[e] = (v[e] - from) * rstd;
      sg[e] = __builtin_fmaf(d[e], v[e], sg[e]);
      sb[e] += d[e];
      d[e] *= gamma[e];
      m[0] += d[e];
      m[1] = __builtin_fmaf(d[e], v[e], m[1]);
    }
    if (!p.dX) continue;
    row_combine<T, 2>(m, slots[turn][rg], [](float f, float g) { return f + g; });
    m[0] *= p.inv_n;
    m[1] *= p.inv_n;
    if (in && have) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        v[e] = rstd * (__builtin_fmaf(-v[e], m[1], d[e]) - m[0]);
        if (p.R) v[e] += a[e];
      }
      Raw<XT> out;
      out.set(v);
      out.store(p.dX + row * p.lddx * Raw<XT>::EB, c, p.N);
    }
  }
  if (!p.sums) return;
  float* const to = p.sums + (long long)blockIdx.x * 2 * p.width;
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    const auto& s = which ? sb : sg;
    if constexpr (RG == 1) {
      if (have) store_f32<8>(to + which * p.width + c, p.N - c, s);
    } else {
      __syncthreads();
      __builtin_memcpy(part + rg * COLS + c, s, 32);
      __syncthreads();
      for (int i = threadIdx.x; i < COLS && i < p.N; i += 1024) {
        float f = part[i];
#pragma unroll
        for (int g = 1; g < RG; ++g) f += part[g * COLS + i];
        to[which * p.width + i] = f;
      }
    }
  }
}

// Rows that registers do not hold: two launches, which read dY and X twice.

// mean(g) and mean(g xh) of every row, of more than 8 T elements each.  A
// thread's next chunk, of this row or of the next one, is on its way while this one
// is summed (8192 x 12288 bf16 75 us without, 69 with it).
template <int XT, int OT, int T>
__global__ void __launch_bounds__(T) norm_back_stats_kernel(const NormBackArgs p) {
  constexpr int W = T / 64;
  __shared__ float sums[2][W][2];
  const int t = threadIdx.x;
  Raw<OT> dy;
  Raw<XT> x;
  Raw<T_F32> gamma;
  float next_mean, next_rstd;
  auto load = [&](long long row, int c) {
    next_mean = p.mean[row];
    next_rstd = p.rstd[row];
    dy.load(p.dY + row * p.lddy * Raw<OT>::EB, c, p.N);
    x.load(p.X + row * p.ldx * Raw<XT>::EB, c, p.N);
    if (p.gamma) gamma.load(reinterpret_cast<const uint8_t*>(p.gamma), c, p.N);
  };
  if (blockIdx.x < p.M) load(blockIdx.x, t * 8);
  int turn = 0;
  for (long long row = blockIdx.x; row < p.M; row += gridDim.x, turn ^= 1) {
    float m[2] = {0.0f, 0.0f};
    double total[2] = {0.0, 0.0};
    for (uint32_t u = t * 8, turns = 0; u < (uint32_t)p.N; u += T * 8, ++turns) {
      const int c = (int)u, n = p.N - c;
      if (turns == SEGMENT / 8) {
        turns = 0;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          total[i] += (double)m[i];
          m[i] = 0.0f;
        }
      }
      const float mean = next_mean, rstd = next_rstd;
      float d[8], v[8], g[8];
      dy.settle(c, p.N);
      dy.get(d);
      x.settle(c, p.N);
      x.get(v);
      if (p.gamma) {
        gamma.settle(c, p.N);
        gamma.get(g);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) g[e] = 1.0f;
      }
      if (u + T * 8 < (uint32_t)p.N)
        load(row, c + T * 8);
      else if (row + gridDim.x < p.M)
        load(row + gridDim.x, t * 8);
      if (n < 8) {  // (zeros past the row, and 0 from there)
#pragma unroll
        for (int e = 1; e < 8; ++e) v[e] = e < n ? v[e] : mean;
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        d[e] *= g[e];
        m[0] += d[e];
        m[1] = __builtin_fmaf(d[e], (v[e] - mean) * rstd, m[1]);
      }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) m[i] = (float)(total[i] + (double)m[i]);
    row_combine<T, 2>(m, sums[turn], [](float f, float g) { return f + g; });
    if (t == 0) p.stats[row] = make_float2(m[0] * p.inv_n, m[1] * p.inv_n);
  }
}

// dX, and the sums down the rows of a block: 512 columns (8 a lane) by p.rows
// rows, which the four waves take in turn, each with its next row on the way.
template <int XT, int OT>
__global__ void __launch_bounds__(256) norm_back_kernel(const NormBackArgs p) {
  __shared__ float part[2][4][512];
  const int lane = threadIdx.x & 63, wave = wave_id();
  const int by = blockIdx.x / p.groups, bx = blockIdx.x - by * p.groups;
  const int c = bx * 512 + lane * 8;
  float sg[8], sb[8], gamma[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) sg[e] = sb[e] = 0.0f;
  if (c < p.N) {
    Raw<OT> dy;
    Raw<XT> x, r;
    float next_mean, next_rstd;
    float2 next_m = make_float2(0.0f, 0.0f);
    auto load = [&](long long row) {
      next_mean = p.mean[row];
      next_rstd = p.rstd[row];
      if (p.dX) next_m = p.stats[row];
      dy.load(p.dY + row * p.lddy * Raw<OT>::EB, c, p.N);
      x.load(p.X + row * p.ldx * Raw<XT>::EB, c, p.N);
      if (p.dX && p.R) r.load(p.R + row * p.ldr * Raw<XT>::EB, c, p.N);
    };
    const long long r0 = (long long)by * p.rows, r1 = min(p.M, r0 + p.rows);
    if (r0 + wave < r1) load(r0 + wave);
#pragma unroll
    for (int e = 0; e < 8; ++e) gamma[e] = 1.0f;
    if (p.gamma) load_vector(p.gamma, c, p.N, gamma);
    for (long long row = r0 + wave; row < r1; row += 4) {
      const float mean = next_mean, rstd = next_rstd;
      const float2 m = next_m;
      float d[8], v[8], a[8];
      dy.settle(c, p.N);
      dy.get(d);
      x.settle(c, p.N);
      x.get(v);
      if (p.dX && p.R) {
        r.settle(c, p.N);
        r.get(a);
      }
      if (row + 4 < r1) load(row + 4);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        v[e] = (v[e] - mean) * rstd;
        sg[e] = __builtin_fmaf(d[e], v[e], sg[e]);
        sb[e] += d[e];
      }
      if (p.dX) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          v[e] = rstd * (__builtin_fmaf(-v[e], m.y, d[e] * gamma[e]) - m.x);
          if (p.R) v[e] += a[e];
        }
        Raw<XT> out;
        out.set(v);
        out.store(p.dX + row * p.lddx * Raw<XT>::EB, c, p.N);
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
