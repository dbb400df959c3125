// dropout.hpp -- dropout from a counter-based generator, its mask never stored:
//   y = (word < T ? 0 : x 2^32 / (2^32 - T)) + r,  T = p 2^32 to the nearest
// The words are those of Philox4x32-10 (J. Salmon, M. Moraes, R. Dror, D. Shaw,
// "Parallel random numbers: as easy as 1, 2, 3", 2011): a function of a key (the
// seed) and a counter (column / 4, row, offset), so the backward pass makes the
// same mask anew from the same numbers.
#pragma once

#include "row_kernels.hpp"

namespace igc_rows {

// Ten rounds of two 32 x 32 bit products each: four words.
__device__ __forceinline__ void philox(uint32_t c0, uint32_t c1, uint32_t c2, uint32_t c3, uint32_t k0, uint32_t k1, uint32_t* out) {
#pragma unroll
  for (int i = 0; i < 10; ++i) {
    const uint64_t a = (uint64_t)0xD2511F53u * c0, b = (uint64_t)0xCD9E8D57u * c2;
    const uint32_t n0 = (uint32_t)(b >> 32) ^ c1 ^ k0, n2 = (uint32_t)(a >> 32) ^ c3 ^ k1;
    c0 = n0;
    c1 = (uint32_t)b;
    c2 = n2;
    c3 = (uint32_t)a;
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  out[0] = c0;
  out[1] = c1;
  out[2] = c2;
  out[3] = c3;
}

struct DropArgs {
  long long M;
  int N;
  const uint8_t *X, *R;  // R: or NULL
  uint8_t* Y;
  long long ldx, ldr, ldy;
  int per;             // chunks of 8 elements in a row
  long long step_row;  // from one chunk of a thread to its next: rows,
  int step_chunk;      // and chunks
  int drops;           // T > 0
  uint32_t last;       // T - 1: the largest word that drops its element
  float scale;
  uint32_t seed0, seed1;
  uint64_t offset;
  const uint64_t* step;  // added to offset, or NULL
};

// Eight elements a thread and turn, two calls of the generator.  X of type XT,
// R and Y of type YT.
template <int XT, int YT>
__global__ void __launch_bounds__(256) dropout_kernel(const DropArgs p) {
  const uint64_t at = p.offset + (p.step ? *p.step : 0);
  const uint32_t first = blockIdx.x * 256 + threadIdx.x;
  long long row = first / (uint32_t)p.per;
  int chunk = (int)(first - (uint32_t)row * (uint32_t)p.per);
  while (row < p.M) {
    const int c = chunk * 8;
    Raw<XT> x;
    Raw<YT> r;
    x.load(p.X + row * p.ldx * Raw<XT>::EB, c, p.N);
    if (p.R) r.load(p.R + row * p.ldr * Raw<YT>::EB, c, p.N);
    float f[8];
    x.settle(c, p.N);
    x.get(f);
    if (p.drops) {
      uint32_t w[8];
      philox(chunk * 2, (uint32_t)row, (uint32_t)at, (uint32_t)(at >> 32), p.seed0, p.seed1, w);
      philox(chunk * 2 + 1, (uint32_t)row, (uint32_t)at, (uint32_t)(at >> 32), p.seed0, p.seed1, w + 4);
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = w[e] > p.last ? f[e] * p.scale : 0.0f;
    }
    if (p.R) {
      float a[8];
      r.settle(c, p.N);
      r.get(a);
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] += a[e];
    }
    r.set(f);
    r.store(p.Y + row * p.ldy * Raw<YT>::EB, c, p.N);
    row += p.step_row;
    chunk += p.step_chunk;
    if (chunk >= p.per) {
      chunk -= p.per;
      ++row;
    }
  }
}

}  // namespace igc_rows
