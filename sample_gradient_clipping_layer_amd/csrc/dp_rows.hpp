// Rows held in registers (internal to libdpclip): the columns that a lane of
// one or several waves holds, and the reductions over a row. Shared by
// the norms' kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "dp_common.hpp"
#include "dp_lm.hpp"

namespace dpk {

// fp32 value -> storage, rounded to nearest even (NaN kept).
__device__ __forceinline__ void put(float& d, float v) { d = v; }
__device__ __forceinline__ void put(bf16s& d, float v) { d.u = f32_to_bf16(v); }

// The columns a lane holds: E elements as vectors of 16 bytes, the row's LPR
// lanes side by side. Rows may start at any element (odd widths, views): the
// hardware takes unaligned 16-byte accesses, and the row's last vector is
// taken element by element when it is not whole (WHOLE: it always is).
// Single-element accesses for such rows: 19.6 us a call instead of 11.6 for a
// backward pass of 1001 rows of 1001 fp32.
template <typename T, bool WHOLE, int E, int LPR>
struct RowMap {
  static constexpr int P = elem_traits<T>::per16;
  static constexpr int N = E / P;
  static __device__ __forceinline__ int col(int j, int lane) { return (j * LPR + lane) * P; }  // d <= 32768

  using Raw = u32x4[N];

  // elements past d read as 0
  static __device__ __forceinline__ void fetch(const T* __restrict__ row, int d, int lane, Raw& raw) {
#pragma unroll
    for (int j = 0; j < N; ++j) {
      raw[j] = u32x4{0u, 0u, 0u, 0u};
      const int c = col(j, lane);
      if (WHOLE ? c < d : c + P <= d) {
        __builtin_memcpy(&raw[j], row + c, 16);
      } else if (!WHOLE && c < d) {
#pragma unroll
        for (int e = 0; e < P - 1; ++e)
          if (c + e < d) {
            const uint32_t bits = raw_bits(row[c + e]);
            if constexpr (P == 8) raw[j][e >> 1] |= bits << (16 * (e & 1));
            else raw[j][e] = bits;
          }
      }
    }
  }
  static __device__ __forceinline__ void unpack(const Raw& raw, float* v) {
#pragma unroll
    for (int j = 0; j < N; ++j) {
      if constexpr (P == 8) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          v[j * 8 + 2 * e] = __uint_as_float(raw[j][e] << 16);
          v[j * 8 + 2 * e + 1] = __uint_as_float(raw[j][e] & 0xFFFF0000u);
        }
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) v[j * 4 + e] = __uint_as_float(raw[j][e]);
      }
    }
  }

  static __device__ __forceinline__ void store(T* __restrict__ row, int d, int lane, const float* v) {
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const int c = col(j, lane);
      if (WHOLE ? c < d : c + P <= d) {
        u32x4 raw;
        if constexpr (P == 8) {
#pragma unroll
          for (int e = 0; e < 4; ++e) raw[e] = pack_bf16(v[j * 8 + 2 * e], v[j * 8 + 2 * e + 1]);
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) raw[e] = __float_as_uint(v[j * 4 + e]);
        }
        __builtin_memcpy(row + c, &raw, 16);
      } else if (!WHOLE && c < d) {
#pragma unroll
        for (int e = 0; e < P - 1; ++e)
          if (c + e < d) put(row[c + e], v[j * P + e]);
      }
    }
  }

  static __device__ __forceinline__ void store_f32(float* __restrict__ row, int d, int lane, const float* v) {
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const int c = col(j, lane);
      if (WHOLE ? c < d : c + P <= d) {
        __builtin_memcpy(row + c, v + j * P, 4 * P);
      } else if (!WHOLE && c < d) {
#pragma unroll
        for (int e = 0; e < P - 1; ++e)
          if (c + e < d) row[c + e] = v[j * P + e];
      }
    }
  }

  // the gain, fp32 or bf16
  template <typename GT>
  static __device__ __forceinline__ void load_gain_as(const GT* __restrict__ gain, int d, int lane, float* v) {
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const int c = col(j, lane);
      if (WHOLE ? c < d : c + P <= d) {
        GT raw[P];
        __builtin_memcpy(raw, gain + c, sizeof(raw));
#pragma unroll
        for (int e = 0; e < P; ++e) v[j * P + e] = to_f32(raw[e]);
      } else {
#pragma unroll
        for (int e = 0; e < P; ++e) v[j * P + e] = !WHOLE && c + e < d ? to_f32(gain[c + e]) : 0.f;
      }
    }
  }
  static __device__ __forceinline__ void load_gain(const void* gain, int gain_bf16, int d, int lane, float* v) {
    if (gain_bf16) load_gain_as(static_cast<const bf16s*>(gain), d, lane, v);
    else load_gain_as(static_cast<const float*>(gain), d, lane, v);
  }
};

// Sums of NV values over the lanes of a row, the same bits in every lane.
// WPR > 1: through LDS, `red` holding NV floats per wave of the block, twice
// (alternating calls use alternating halves, so one barrier a call suffices).
template <int WPR, int NV>
__device__ __forceinline__ void row_sums(float (&v)[NV], float* red, int wave, int& phase) {
#pragma unroll
  for (int i = 0; i < NV; ++i) v[i] = wave_sum(v[i]);
  if constexpr (WPR > 1) {
    float* r = red + phase * 16 * NV;
    if ((threadIdx.x & 63) == 0) {
#pragma unroll
      for (int i = 0; i < NV; ++i) r[NV * wave + i] = v[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NV; ++i) v[i] = 0.f;
#pragma unroll
    for (int w = 0; w < WPR; ++w)
#pragma unroll
      for (int i = 0; i < NV; ++i) v[i] += r[NV * w + i];
    phase ^= 1;
  }
}

// Threads of a workgroup whose rows take WPR waves each.
template <int WPR>
constexpr int row_threads() {
  return WPR > 4 ? 64 * WPR : 256;
}

// One instantiation per (elements per lane, waves per row) the width needs; up to 8192 columns.
template <typename F>
hipError_t row_dispatch_to_8192(int64_t d, F f) {
  if (d <= 512) return f(std::integral_constant<int, 8>{}, std::integral_constant<int, 1>{});
  if (d <= 1024) return f(std::integral_constant<int, 16>{}, std::integral_constant<int, 1>{});
  if (d <= 1536) return f(std::integral_constant<int, 24>{}, std::integral_constant<int, 1>{});
  if (d <= 2048) return f(std::integral_constant<int, 32>{}, std::integral_constant<int, 1>{});
  if (d <= 4096) return f(std::integral_constant<int, 16>{}, std::integral_constant<int, 4>{});
  return f(std::integral_constant<int, 32>{}, std::integral_constant<int, 4>{});
}
template <typename F>
hipError_t row_dispatch(int64_t d, F f) {
  if (d <= 8192) return row_dispatch_to_8192(d, f);
  if (d <= 16384) return f(std::integral_constant<int, 16>{}, std::integral_constant<int, 16>{});
  return f(std::integral_constant<int, 32>{}, std::integral_constant<int, 16>{});
}
inline int row_groups(int64_t d) { return d <= 2048 ? 4 : 1; }  // rows that a workgroup takes side by side

}  // namespace dpk
