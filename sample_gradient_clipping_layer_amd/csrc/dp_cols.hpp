// Rows read by whole vectors whatever their width (internal to libdpclip):
// shared by the kernels of the table of words and of the balance loss.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "dp_common.hpp"
#include "dp_lm.hpp"

namespace dpk {

// What is read in place of a row that is not there, so that loads of several rows need no branches between them.
static __device__ const uint32_t kZeros[16] = {};

// The P columns that a lane holds of a row of d: those from `c` on, or, where fewer are left, the row's last P (the
// first `skip` of them are its neighbour's too). So every access is one whole vector, aligned or not: a row's end read
// element by element has to be put together before the next row's loads are issued (8 rows of 333 fp32: 11 us instead
// of 3). TINY: rows of fewer than P columns, element by element.
template <typename T, int P, bool TINY>
struct Cols {
  static constexpr int columns = P, bytes = P * (int)sizeof(T);
  typedef uint32_t Raw __attribute__((ext_vector_type(bytes / 4)));
  int at, skip, d;
  bool on;
  __device__ __forceinline__ Cols(int c, int64_t width) : d((int)width) {
    on = c < d;
    at = TINY || c + P <= d ? c : d - P;
    skip = c - at;
  }
  // row n of X, zeros for n < 0 and in lanes past the row
  __device__ __forceinline__ Raw fetch(const void* X, int64_t n) const {
    const T* row = static_cast<const T*>(X) + (n < 0 ? 0 : n) * d;
    Raw raw;
    if (TINY) {
#pragma unroll
      for (int w = 0; w < bytes / 4; ++w) raw[w] = 0u;
#pragma unroll
      for (int e = 0; e < P - 1; ++e)
        if (at + e < d && n >= 0) {
          const uint32_t bits = raw_bits(row[at + e]);
          if constexpr (sizeof(T) == 2) raw[e >> 1] |= bits << (16 * (e & 1));
          else raw[e] = bits;
        }
    } else {
      __builtin_memcpy(&raw, on && n >= 0 ? row + at : reinterpret_cast<const T*>(kZeros), bytes);
    }
    return raw;
  }
  static __device__ __forceinline__ float value(Raw raw, int e) {
    if constexpr (sizeof(T) == 2) return __uint_as_float(e & 1 ? raw[e >> 1] & 0xFFFF0000u : raw[e >> 1] << 16);
    else return __uint_as_float(raw[e]);
  }
  static __device__ __forceinline__ void add(float* acc, Raw raw, float f) {
#pragma unroll
    for (int e = 0; e < P; ++e) acc[e] = __builtin_fmaf(f, value(raw, e), acc[e]);
  }
  // row n of X from fp32; columns that two lanes hold are stored by both, with the same value
  __device__ __forceinline__ void put(void* X, int64_t n, const float* v) const {
    T* row = static_cast<T*>(X) + n * d;
    Raw raw;
#pragma unroll
    for (int w = 0; w < bytes / 4; ++w) {
      if constexpr (sizeof(T) == 2) raw[w] = pack_bf16(v[2 * w], v[2 * w + 1]);
      else raw[w] = __float_as_uint(v[w]);
    }
    if (TINY) {
#pragma unroll
      for (int e = 0; e < P - 1; ++e)
        if (at + e < d) __builtin_memcpy(row + at + e, reinterpret_cast<const char*>(&raw) + e * sizeof(T), sizeof(T));
    } else if (on) {
      __builtin_memcpy(row + at, &raw, bytes);
    }
  }
  // row n of fp32 sums, zeros for n < 0
  __device__ __forceinline__ void fetch_sums(const float* X, int64_t n, float* v) const {
    const float* row = X + (n < 0 ? 0 : n) * d;
    if (TINY) {
#pragma unroll
      for (int e = 0; e < P; ++e) v[e] = e < P - 1 && at + e < d && n >= 0 ? row[at + e] : 0.f;
    } else {
      __builtin_memcpy(v, on && n >= 0 ? row + at : reinterpret_cast<const float*>(kZeros), 4 * P);
    }
  }
  // past the caches; rows at 16-byte boundaries of a multiple of P columns
  __device__ __forceinline__ void stream_sums(float* row, const float* acc) const {
#pragma unroll
    for (int q = 0; q < P / 4; ++q) {
      const f32x4 v{acc[4 * q], acc[4 * q + 1], acc[4 * q + 2], acc[4 * q + 3]};
      if (on) __builtin_nontemporal_store(v, reinterpret_cast<f32x4*>(row + at + 4 * q));
    }
  }
  // a row's columns that two lanes hold are stored by both, with the same value
  __device__ __forceinline__ void put_sums(float* row, const float* acc) const {
    if (TINY) {
#pragma unroll
      for (int e = 0; e < P - 1; ++e)
        if (at + e < d) row[at + e] = acc[e];
    } else if (on) {
      __builtin_memcpy(row + at, acc, 4 * P);
    }
  }
};

}  // namespace dpk
