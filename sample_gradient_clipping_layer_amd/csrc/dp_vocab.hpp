// Rows of a vocabulary streamed by a workgroup (internal to libdpclip). Shared
// by the kernels over logits.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "dp_common.hpp"

namespace dpk {

constexpr float kLog2e = 1.4426950408889634f;

// 2^x by the hardware's instruction: within one step, results below 2^-126
// flushed to 0 (they are terms of sums of order 1, or probabilities).
__device__ __forceinline__ float exp2_hw(float x) { return __builtin_amdgcn_exp2f(x); }

template <int NT>
__device__ __forceinline__ float block_max(float v, float* red) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) v = fmaxf(v, __shfl_xor(v, off, kWave));
  __syncthreads();
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  v = red[0];
#pragma unroll
  for (int w = 1; w < NT / 64; ++w) v = fmaxf(v, red[w]);
  return v;
}
template <int NT>
__device__ __forceinline__ float block_add(float v, float* red) {
  v = wave_sum(v);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  v = red[0];
#pragma unroll
  for (int w = 1; w < NT / 64; ++w) v += red[w];
  return v;
}

template <int P>
__device__ __forceinline__ void unpack16(u32x4 raw, float* v) {
  if constexpr (P == 8) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      v[2 * e] = __uint_as_float(raw[e] << 16);
      v[2 * e + 1] = __uint_as_float(raw[e] & 0xFFFF0000u);
    }
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = __uint_as_float(raw[e]);
  }
}

// Elements [v0, v1) of a row as single elements up to the first 16-byte
// boundary, 16-byte vectors, and single elements after the last: rows of odd
// V start anywhere.
template <typename T>
struct Span {
  int64_t head, vecs, tail0;  // [v0, head) single, head + P*i vectors, [tail0, v1) single
  __device__ __forceinline__ Span(const T* row, int64_t v0, int64_t v1) {
    constexpr int P = elem_traits<T>::per16;
    const int64_t mis = (int64_t)((reinterpret_cast<uintptr_t>(row + v0) & 15) / sizeof(T));
    head = v0 + (mis ? P - mis : 0);
    if (head > v1) head = v1;
    vecs = (v1 - head) / P;
    tail0 = head + vecs * P;
  }
};

}  // namespace dpk
