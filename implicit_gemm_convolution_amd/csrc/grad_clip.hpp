// grad_clip.hpp -- the global norm of many gradients, and clipping:
//   norm = sqrt(sum g^2);  out = g min(1, max_norm / (norm + 1e-6))
//
// Two passes over the gradients, which is what the formula needs where they
// do not fit on the chip: the first leaves one 64-bit partial sum per
// workgroup, the second adds those (every workgroup for itself, in one fixed
// order) and scales.  Both are bound by memory.  The squares are summed in 64
// bits: 10^8 values would lose digits in 32, and squares of bf16 values
// overflow there.
#pragma once

#include "ffn_kernels.hpp"

namespace igc_ffn {

constexpr int CLIP_TENSORS = 64;   // tensors per launch (the table travels in the kernel's arguments)
constexpr int CLIP_CHUNK = 8192;   // elements per workgroup step
constexpr int CLIP_GRID = 1024;    // workgroups per launch at most

struct ClipTable {
  const uint8_t* in[CLIP_TENSORS];
  uint8_t* out[CLIP_TENSORS];
  long long size[CLIP_TENSORS];      // elements
  int first[CLIP_TENSORS + 1];       // first chunk of each tensor; [count] = all chunks
  uint8_t type[CLIP_TENSORS];
  int count;
  int partials;     // norm pass: this launch's first slot; scale pass: slots in use
  double* part;
  float max_norm;
  float* norm;      // scale pass: written by the launch that has it
};

__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int o = 32; o; o >>= 1) v += __shfl_xor(v, o);
  return v;
}

// Lane i of every wave holds tensor i of the table, so that all of it is on its
// way at once (looked up entry by entry, each dependent read of the arguments
// waits for host memory).
struct ClipEntry {
  uint64_t in, out;
  long long size;
  int first, type;
  __device__ __forceinline__ explicit ClipEntry(const ClipTable& p) {
    static_assert(CLIP_TENSORS == 64, "a tensor for each lane");
    const int i = threadIdx.x & 63, t = min(i, max(p.count - 1, 0));
    in = reinterpret_cast<uint64_t>(p.in[t]);
    out = reinterpret_cast<uint64_t>(p.out[t]);
    size = p.size[t];
    type = p.type[t];
    first = i < p.count ? p.first[t] : 0x7fffffff;
  }
};
__device__ __forceinline__ uint64_t of_lane(uint64_t v, int lane) {
  const uint32_t lo = __builtin_amdgcn_readlane((uint32_t)v, lane), hi = __builtin_amdgcn_readlane((uint32_t)(v >> 32), lane);
  return (uint64_t)hi << 32 | lo;
}

// Runs f(in, out, type, first element, elements) for every chunk of this
// workgroup.  REVERSE: from the last chunk to the first, so that the second
// pass begins with what the first one read last and the memory-side cache
// (256 MB) still holds.
template <bool REVERSE, class F>
__device__ __forceinline__ void clip_chunks(const ClipTable& p, const ClipEntry& e, F&& f) {
  const int chunks = p.first[p.count];
  for (int b = blockIdx.x; b < chunks; b += gridDim.x) {
    const int c = REVERSE ? chunks - 1 - b : b;
    // the last tensor whose first chunk is <= c (empty tensors have none)
    const int t = 63 - __builtin_clzll(__builtin_amdgcn_ballot_w64(e.first <= c));
    const long long e0 = (long long)(c - (int)__builtin_amdgcn_readlane(e.first, t)) * CLIP_CHUNK;
    f(reinterpret_cast<const uint8_t*>(of_lane(e.in, t)), reinterpret_cast<uint8_t*>(of_lane(e.out, t)),
      (int)__builtin_amdgcn_readlane(e.type, t), e0, (int)min((long long)CLIP_CHUNK, (long long)of_lane(e.size, t) - e0));
  }
}

template <int T>
__device__ __forceinline__ double chunk_squares(const uint8_t* in, int n) {
  constexpr int EB = T == T_F32 ? 4 : 2, V = 16 / EB;
  double s = 0.0;
#pragma unroll 4
  for (int e = threadIdx.x * V; e < n; e += 256 * V) {
    float f[8] = {};
    if constexpr (T == T_F32) {
      if (n - e >= 4)
        __builtin_memcpy(f, in + (long long)e * 4, 16);
      else
        for (int q = 0; q < 4; ++q)
          if (e + q < n) f[q] = reinterpret_cast<const float*>(in)[e + q];
    } else {
      unpack8<T == T_BF16>(load8(in + (long long)e * 2, n - e), f);
    }
#pragma unroll
    for (int q = 0; q < V; ++q) s += (double)f[q] * (double)f[q];
  }
  return s;
}

// 16 bytes past the caches, at any address of the element type's alignment.
__device__ __forceinline__ void stream16(uint8_t* p, const uint4& v) {
  typedef uint32_t u32x4 __attribute__((ext_vector_type(4), aligned(2)));
  __builtin_nontemporal_store(u32x4{v.x, v.y, v.z, v.w}, reinterpret_cast<u32x4*>(p));
}

template <int T>
__device__ __forceinline__ void chunk_scale(const uint8_t* in, uint8_t* out, int n, float scale) {
  constexpr int EB = T == T_F32 ? 4 : 2, V = 16 / EB;
#pragma unroll 4
  for (int e = threadIdx.x * V; e < n; e += 256 * V) {
    if constexpr (T == T_F32) {
      if (n - e >= 4) {
        float f[4];
        __builtin_memcpy(f, in + (long long)e * 4, 16);
#pragma unroll
        for (int q = 0; q < 4; ++q) f[q] *= scale;
        uint4 w;
        __builtin_memcpy(&w, f, 16);
        stream16(out + (long long)e * 4, w);
      } else {
        for (int q = 0; q < 4; ++q)
          if (e + q < n) reinterpret_cast<float*>(out)[e + q] = reinterpret_cast<const float*>(in)[e + q] * scale;
      }
    } else {
      float f[8];
      unpack8<T == T_BF16>(load8(in + (long long)e * 2, n - e), f);
#pragma unroll
      for (int q = 0; q < 8; ++q) f[q] *= scale;
      if (n - e >= 8)
        stream16(out + (long long)e * 2, pack8<T == T_BF16>(f));
      else
        store8(out + (long long)e * 2, pack8<T == T_BF16>(f), n - e);
    }
  }
}

template <int NONE = 0>
__global__ void __launch_bounds__(256) clip_norm_kernel(const ClipTable p) {
  __shared__ double sm[4];
  double s = 0.0;
  clip_chunks<false>(p, ClipEntry(p), [&](const uint8_t* in, uint8_t*, int type, long long e0, int n) {
    if (type == T_F32)
      s += chunk_squares<T_F32>(in + e0 * 4, n);
    else if (type == T_BF16)
      s += chunk_squares<T_BF16>(in + e0 * 2, n);
    else
      s += chunk_squares<T_F16>(in + e0 * 2, n);
  });
  s = wave_sum(s);
  if ((threadIdx.x & 63) == 0) sm[wave_id()] = s;
  __syncthreads();
  if (threadIdx.x == 0) p.part[p.partials + blockIdx.x] = (sm[0] + sm[1]) + (sm[2] + sm[3]);
}

template <int NONE = 0>
__global__ void __launch_bounds__(256) clip_scale_kernel(const ClipTable p) {
  __shared__ double sm[4];
  const ClipEntry entry(p);
  double s = 0.0;
  for (int i = threadIdx.x; i < p.partials; i += 256) s += p.part[i];
  s = wave_sum(s);
  if ((threadIdx.x & 63) == 0) sm[wave_id()] = s;
  __syncthreads();
  const double norm = __builtin_sqrt((sm[0] + sm[1]) + (sm[2] + sm[3]));
  if (p.norm && blockIdx.x == 0 && threadIdx.x == 0) *p.norm = (float)norm;
  const double ratio = (double)p.max_norm / (norm + 1e-6);
  const float scale = ratio > 1.0 ? 1.0f : (float)ratio;  // (NaN stays NaN)
  clip_chunks<true>(p, entry, [&](const uint8_t* in, uint8_t* out, int type, long long e0, int n) {
    if (type == T_F32)
      chunk_scale<T_F32>(in + e0 * 4, out + e0 * 4, n, scale);
    else if (type == T_BF16)
      chunk_scale<T_BF16>(in + e0 * 2, out + e0 * 2, n, scale);
    else
      chunk_scale<T_F16>(in + e0 * 2, out + e0 * 2, n, scale);
  });
}

}  // namespace igc_ffn
