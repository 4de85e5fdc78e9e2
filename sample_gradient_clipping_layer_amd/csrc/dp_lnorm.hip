// Layer norm with the residual's addition, and its backward pass with the
// gain's and the bias's gradient of every sample.
//
//   forward:   s = x + r,  u = (s - mean(s)) / sqrt(var(s) + eps),  y = u * gain + bias
//   backward:  h = dy * gain,  ds = dsum + rstd * (h - mean(h) - u * mean(h * u)),
//              gain_rows[b] = sum_t dy[b][t] * u[b][t],  bias_rows[b] = sum_t dy[b][t]
//
// Bound by HBM: 32 x 1024 rows of 1280 bf16 with a residual take 58 us forward
// (336 MB, 5.8 TB/s), 72 + 5 back with both gradients (the rows of 252 MB read
// and 84 written at 4.8 TB/s, then the workgroups' sums). A row is held in the
// registers of one, four, eight or sixteen waves, so one pass over memory
// serves both its statistics and its outputs. The variance is that of the
// centred row, whose own mean (the rounding of the first one) is taken off
// again: rows far from zero lose nothing to a difference of large sums.
// That mean and the mean square are quotients, not products with 1/d alone: in
// a row of one value every column is off by the same few steps of it, sums and
// quotients of those are exact, and the deviation is 0 whatever the value's
// size. (Products left parts of a step: at 1601 columns rows of one large value
// had other outputs than the bias.)
// A lane keeps the columns it holds over all its rows, so the per-sample
// gradients are register sums; the waves of a workgroup add theirs through LDS
// in wave order, and when a sample is spread over several workgroups their
// partial sums go through the workspace and a second kernel adds them in
// order. Nothing is atomic.
#include "dp_common.hpp"
#include "dp_lm.hpp"
#include "dp_rows.hpp"

namespace dpk {

namespace {

// A product rounded on its own: a mean that some columns took with its rounding and others, fused into their
// subtraction, without it would differ from column to column.
__device__ __forceinline__ float mul_rounded(float a, float b) {
#pragma clang fp contract(off)
  return a * b;
}

__device__ __forceinline__ float sub_rounded(float a, float b) {
#pragma clang fp contract(off)
  return a - b;
}

// The same value in every lane, in a scalar register (in vector registers the width and its reciprocal cost rows of 768
// fp32 a sixth wave per SIMD: 79.5 us instead of 76.7 for 32768 of them).
__device__ __forceinline__ float scalar(float v) {
  return __uint_as_float((uint32_t)__builtin_amdgcn_readfirstlane((int)__float_as_uint(v)));
}

// x / d from d's reciprocal, the product's rounding made good: exact where the quotient has 24 bits.
__device__ __forceinline__ float quotient(float x, float d, float inv_d) {
  const float q = mul_rounded(x, inv_d);
  return __builtin_fmaf(__builtin_fmaf(-q, d, x), inv_d, q);
}

// The P values of a vector of a row. `again`: unpacked anew, so that the compiler does not keep them in fp32 from the
// last time (bf16: half the registers).
template <int P>
__device__ __forceinline__ void unpack_vec(u32x4& raw, float* v, bool again) {
  if constexpr (P == 8) {
    if (again) {
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        uint32_t x = raw[w];
        asm volatile("" : "+v"(x));
        raw[w] = x;
      }
    }
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

// Vector j of a row's lane from fp32, as RowMap::store does it.
template <typename T, typename M, bool WHOLE>
__device__ __forceinline__ void store_vec(T* __restrict__ row, int d, int lane, int j, const float* v) {
  const int c = M::col(j, lane);
  if (WHOLE ? c < d : c + M::P <= d) {
    u32x4 raw;
    if constexpr (M::P == 8) {
#pragma unroll
      for (int e = 0; e < 4; ++e) raw[e] = pack_bf16(v[2 * e], v[2 * e + 1]);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) raw[e] = __float_as_uint(v[e]);
    }
    __builtin_memcpy(row + c, &raw, 16);
  } else if (!WHOLE && c < d) {
#pragma unroll
    for (int e = 0; e < M::P - 1; ++e)
      if (c + e < d) put(row[c + e], v[e]);
  }
}

// v - mean over the row's columns, 0 past its end; the sums of squares and of the values are added to q and r.
template <typename M, bool WHOLE, int E>
__device__ __forceinline__ void centre(float* v, float mean, int d, int lane, float& q, float& r) {
#pragma unroll
  for (int j = 0; j < M::N; ++j) {
    const int c = M::col(j, lane);
#pragma unroll
    for (int e = 0; e < M::P; ++e) {
      const float o = (WHOLE ? c : c + e) < d ? v[j * M::P + e] - mean : 0.f;
      v[j * M::P + e] = o;
      q = __builtin_fmaf(o, o, q);
      r += o;
    }
  }
}

}  // namespace

template <typename T, bool WHOLE, int E, int WPR>
__global__ __launch_bounds__(row_threads<WPR>()) void k_layer_norm(LayerNormArgs a) {
  constexpr int NW = row_threads<WPR>() / 64, GROUPS = NW / WPR, LPR = 64 * WPR;
  using M = RowMap<T, WHOLE, E, LPR>;
  __shared__ float red1[32], red2[64];
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));  // scalar: so are a row's addresses
  const int group = WPR == 1 ? wave : 0;
  const int lane = WPR == 1 ? (threadIdx.x & 63) : threadIdx.x;
  int phase1 = 0, phase2 = 0;
  float g[E], b[E];
  M::load_gain(a.gain, a.gain_bf16, (int)a.d, lane, g);
  if (a.bias) {
    M::load_gain(a.bias, a.gain_bf16, (int)a.d, lane, b);
  } else {
#pragma unroll
    for (int e = 0; e < E; ++e) b[e] = 0.f;
  }
  const float width = scalar((float)a.d), inv_d = scalar(1.0f / (float)a.d);
  // WPR > 1: one group, so every wave of the block takes the same rows
  for (int64_t row = (int64_t)blockIdx.x * GROUPS + group; row < a.rows; row += (int64_t)gridDim.x * GROUPS) {
    typename M::Raw rx, rr;
    M::fetch(static_cast<const T*>(a.x) + row * a.d, (int)a.d, lane, rx);
    if (a.residual) M::fetch(static_cast<const T*>(a.residual) + row * a.d, (int)a.d, lane, rr);
    float v[E];
    M::unpack(rx, v);
    if (a.residual) {
      float r[E];
      M::unpack(rr, r);
#pragma unroll
      for (int e = 0; e < E; ++e) v[e] += r[e];
    }
    float sum[1] = {0.f};
#pragma unroll
    for (int e = 0; e < E; ++e) sum[0] += v[e];
    if (a.sum_out) M::store(static_cast<T*>(a.sum_out) + row * a.d, (int)a.d, lane, v);
    row_sums<WPR, 1>(sum, red1, wave, phase1);
    float qr[2] = {0.f, 0.f};
    centre<M, WHOLE, E>(v, mul_rounded(sum[0], inv_d), (int)a.d, lane, qr[0], qr[1]);
    row_sums<WPR, 2>(qr, red2, wave, phase2);
    const float rest = quotient(qr[1], width, inv_d);  // what the rounded mean left
    const float var = fmaxf(__builtin_fmaf(-rest, rest, quotient(qr[0], width, inv_d)), 0.f);
    const float rstd = 1.0f / sqrtf(var + a.eps);
    // y from the sum before its rounding to the storage type
#pragma unroll
    for (int e = 0; e < E; ++e) v[e] = __builtin_fmaf((v[e] - rest) * rstd, g[e], b[e]);
    M::store(static_cast<T*>(a.out) + row * a.d, (int)a.d, lane, v);
  }
}

// Waves per SIMD that the backward pass asks for.
template <typename T, int E, int WPR>
constexpr int backward_waves() {
  return WPR >= 8 ? WPR / 4 : E * sizeof(T) <= 32 ? 4 : E * sizeof(T) <= 48 ? 3 : 2;
}

// Work items: (sample, chunk of its rows); with `own_groups` every group of
// a block takes a sample of its own (chunks == 1).
template <typename T, bool WHOLE, int E, int WPR>
__global__ __launch_bounds__(row_threads<WPR>(),
                             (backward_waves<T, E, WPR>())) void k_layer_norm_backward(LayerNormBackArgs a) {
  constexpr int NW = row_threads<WPR>() / 64, GROUPS = NW / WPR, LPR = 64 * WPR;
  using M = RowMap<T, WHOLE, E, LPR>;
  __shared__ float red1[64], red2[96];
  __shared__ float part[GROUPS > 1 ? (GROUPS - 1) * E * 64 : 1];
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));  // scalar: so are a row's addresses
  const int group = WPR == 1 ? wave : 0;
  const int lane = WPR == 1 ? (threadIdx.x & 63) : threadIdx.x;
  int phase1 = 0, phase2 = 0;
  // Registers for rows in flight are what is short, with the two sums of every column: the gain is held in LDS (read
  // again from L2 by 1024-thread blocks), a row as it was loaded, unpacked a vector at a time in each of its three
  // passes. (32 x 1024 tokens of 1600 bf16: 140 us with the row and the gain in fp32 over the reductions, 97 so. The
  // next row loaded meanwhile takes the registers that a further wave would: 107.)
  constexpr bool HELD = WPR < 16;
  constexpr int P = M::P, N = M::N;
  __shared__ __attribute__((aligned(16))) float held[HELD ? E * LPR : 4];
  if constexpr (HELD) {
    if (group == 0) {
      float g[E];
      M::load_gain(a.gain, a.gain_bf16, (int)a.d, lane, g);
#pragma unroll
      for (int q = 0; q < E / 4; ++q)
        *reinterpret_cast<f32x4*>(held + (q * LPR + lane) * 4) = f32x4{g[4 * q], g[4 * q + 1], g[4 * q + 2], g[4 * q + 3]};
    }
    __syncthreads();
  }
  auto gain = [&](int j, float* g) {
    if constexpr (HELD) {
      int at = lane;
      asm volatile("" : "+v"(at));  // read where it is used, not kept in registers over the rows
#pragma unroll
      for (int q = 0; q < P / 4; ++q) {
        const f32x4 v = *reinterpret_cast<const f32x4*>(held + ((j * (P / 4) + q) * LPR + at) * 4);
#pragma unroll
        for (int e = 0; e < 4; ++e) g[4 * q + e] = v[e];
      }
    } else {
      const int c = M::col(j, lane);
#pragma unroll
      for (int e = 0; e < P; ++e) {
        const int at = c + e < a.d ? c + e : 0;
        g[e] = a.gain_bf16 ? to_f32(static_cast<const bf16s*>(a.gain)[at]) : static_cast<const float*>(a.gain)[at];
      }
    }
  };
  const int d = (int)a.d;
  const float width = scalar((float)a.d), inv_d = scalar(1.0f / (float)a.d);
  const int64_t per_block = a.own_groups ? GROUPS : 1;
  const int64_t items = a.B * a.chunks;
  for (int64_t item0 = (int64_t)blockIdx.x * per_block; item0 < items; item0 += (int64_t)gridDim.x * per_block) {
    const int64_t item = item0 + (a.own_groups ? group : 0);
    const int64_t b = item / a.chunks, ch = item - b * a.chunks;
    const int64_t t0 = ch * a.chunk_rows;
    int64_t t1 = t0 + a.chunk_rows < a.T ? t0 + a.chunk_rows : a.T;
    if (item >= items) t1 = t0;  // a group past the last sample (WPR == 1: no barrier is skipped below)
    float acc_g[E], acc_b[E];
#pragma unroll
    for (int e = 0; e < E; ++e) acc_g[e] = acc_b[e] = 0.f;
    typename M::Raw rs, rh, ro;
    auto fetch = [&](int64_t t) {
      const int64_t off = (b * a.T + t) * a.d;
      M::fetch(static_cast<const T*>(a.s) + off, d, lane, rs);
      M::fetch(static_cast<const T*>(a.dy) + off, d, lane, rh);
      if (a.dsum) M::fetch(static_cast<const T*>(a.dsum) + off, d, lane, ro);
    };
    const int64_t step = a.own_groups ? 1 : GROUPS, first = t0 + (a.own_groups ? 0 : group);
    for (int64_t t = first; t < t1; t += step) {
      fetch(t);
      float sums[2] = {0.f, 0.f};
#pragma unroll
      for (int j = 0; j < N; ++j) {
        float s[P], h[P], g[P];
        gain(j, g);
        unpack_vec<P>(rs[j], s, false);
        unpack_vec<P>(rh[j], h, false);
#pragma unroll
        for (int e = 0; e < P; ++e) {
          sums[0] += s[e];
          sums[1] = __builtin_fmaf(h[e], g[e], sums[1]);
        }
      }
      row_sums<WPR, 2>(sums, red1, wave, phase1);
      const float mean = mul_rounded(sums[0], inv_d), mean_h = sums[1] * inv_d;
      float qrh[3] = {0.f, 0.f, 0.f};
#pragma unroll
      for (int j = 0; j < N; ++j) {
        float s[P], h[P], g[P];
        gain(j, g);
        unpack_vec<P>(rs[j], s, true);
        unpack_vec<P>(rh[j], h, true);
        const int c = M::col(j, lane);
#pragma unroll
        for (int e = 0; e < P; ++e) {
          const float o = (WHOLE ? c : c + e) < d ? sub_rounded(s[e], mean) : 0.f;
          qrh[0] = __builtin_fmaf(o, o, qrh[0]);
          qrh[1] += o;
          qrh[2] = __builtin_fmaf(h[e] * g[e], o, qrh[2]);
        }
      }
      row_sums<WPR, 3>(qrh, red2, wave, phase2);
      const float rest = quotient(qrh[1], width, inv_d);  // what the rounded mean left
      const float var = fmaxf(__builtin_fmaf(-rest, rest, quotient(qrh[0], width, inv_d)), 0.f);
      const float rstd = 1.0f / sqrtf(var + a.eps);
      // mean(h u) * rstd, for u = (s - rest) * rstd
      const float along = __builtin_fmaf(-rest, mean_h, qrh[2] * inv_d) * rstd * rstd;
      T* out = static_cast<T*>(a.dx) + (b * a.T + t) * a.d;
#pragma unroll
      for (int j = 0; j < N; ++j) {
        float s[P], h[P];
        unpack_vec<P>(rs[j], s, true);
        unpack_vec<P>(rh[j], h, true);
#pragma unroll
        for (int e = 0; e < P; ++e) {
          s[e] = sub_rounded(s[e], mean) - rest;  // past the row's end dy is 0
          acc_g[j * P + e] = __builtin_fmaf(h[e], s[e] * rstd, acc_g[j * P + e]);
          acc_b[j * P + e] += h[e];
        }
        if (a.dx) {
          float o[P], g[P];
          gain(j, g);
          if (a.dsum) {
            unpack_vec<P>(ro[j], o, false);
          } else {
#pragma unroll
            for (int e = 0; e < P; ++e) o[e] = 0.f;
          }
#pragma unroll
          for (int e = 0; e < P; ++e)
            o[e] = __builtin_fmaf(rstd, __builtin_fmaf(h[e], g[e], -mean_h) - s[e] * along, o[e]);
          store_vec<T, M, WHOLE>(out, d, lane, j, o);
        }
      }
    }
    if (!a.gain_rows && !a.bias_rows) continue;
    // one after the other through the same LDS; with a chunk's partial sums the gain's come first
    auto give = [&](float* acc, float* rows, int64_t which) {
      bool writes = item < items;
      if constexpr (GROUPS > 1) {
        if (!a.own_groups) {
          if (group > 0) {
#pragma unroll
            for (int e = 0; e < E; ++e) part[((group - 1) * E + e) * 64 + lane] = acc[e];
          }
          __syncthreads();
          if (group == 0) {
#pragma unroll 1
            for (int k = 0; k < GROUPS - 1; ++k)
#pragma unroll
              for (int e = 0; e < E; ++e) acc[e] += part[(k * E + e) * 64 + lane];
          }
          __syncthreads();
          writes = writes && group == 0;
        }
      }
      float* row = a.chunks == 1 ? rows + item * a.d : a.partial + (which * items + item) * a.d;
      if (writes) M::store_f32(row, (int)a.d, lane, acc);
    };
    if (a.gain_rows) give(acc_g, a.gain_rows, 0);
    if (a.bias_rows) give(acc_b, a.bias_rows, 1);
  }
}

// rows[b][c] = the sum of the sample's chunk partials in chunk order.
__global__ __launch_bounds__(256) void k_layer_norm_finish(LayerNormBackArgs a) {
  const int64_t n = a.B * a.d, first = a.gain_rows ? 0 : n, last = a.bias_rows ? 2 * n : n;
  for (int64_t i = first + (int64_t)blockIdx.x * 256 + threadIdx.x; i < last; i += (int64_t)gridDim.x * 256) {
    const int64_t at = i < n ? i : i - n;
    const int64_t b = at / a.d, c = at - b * a.d;
    const float* p = a.partial + ((i < n ? 0 : a.B) + b) * a.chunks * a.d + c;
    float s = 0.f;
#pragma unroll 4
    for (int64_t k = 0; k < a.chunks; ++k) s += p[k * a.d];
    (i < n ? a.gain_rows : a.bias_rows)[at] = s;
  }
}

namespace {

// The backward pass holds five rows' worth of values. Rows of 8193 to 16384 columns take eight waves of up to 256
// registers a lane; with sixteen waves of 128 the kernel spills, which wider rows put up with.
template <typename F>
hipError_t row_dispatch_backward(int64_t d, F f) {
  if (d <= 8192) return row_dispatch_to_8192(d, f);
  if (d <= 16384) return f(std::integral_constant<int, 32>{}, std::integral_constant<int, 8>{});
  return f(std::integral_constant<int, 32>{}, std::integral_constant<int, 16>{});
}

constexpr int64_t kLnBlocks = 256 * 8;  // blocks that fill the 256 CUs; more rows than that are looped over

// Workgroups of the backward pass that the 256 CUs hold at once.
template <typename T>
int64_t backward_resident(int64_t d) {
  int64_t n = 0;
  (void)row_dispatch_backward(d, [&](auto e, auto w) {
    constexpr int E = decltype(e)::value, WPR = decltype(w)::value;
    n = (int64_t)256 * backward_waves<T, E, WPR>() * 256 / row_threads<WPR>();
    return hipSuccess;
  });
  return n;
}

template <typename T, bool WHOLE>
hipError_t launch_fwd(hipStream_t st, const LayerNormArgs& a) {
  return row_dispatch(a.d, [&](auto e, auto w) {
    constexpr int E = decltype(e)::value, WPR = decltype(w)::value;
    const int64_t groups = row_groups(a.d);
    const int64_t blocks = std::min<int64_t>((a.rows + groups - 1) / groups, kLnBlocks);
    k_layer_norm<T, WHOLE, E, WPR><<<dim3((unsigned)blocks), row_threads<WPR>(), 0, st>>>(a);
    return hipGetLastError();
  });
}

template <typename T, bool WHOLE>
hipError_t launch_bwd(hipStream_t st, const LayerNormBackArgs& a) {
  return row_dispatch_backward(a.d, [&](auto e, auto w) {
    constexpr int E = decltype(e)::value, WPR = decltype(w)::value;
    const int64_t per = a.own_groups ? row_groups(a.d) : 1;
    const int64_t blocks = std::min<int64_t>((a.B * a.chunks + per - 1) / per, kLnBlocks);
    k_layer_norm_backward<T, WHOLE, E, WPR><<<dim3((unsigned)blocks), row_threads<WPR>(), 0, st>>>(a);
    return hipGetLastError();
  });
}

}  // namespace

// How a sample's rows are spread over workgroups: as far as all of them are held at once (32 samples of 1024 tokens of
// 1280 bf16: 768 are held; 83 us by 1024 workgroups), each of at least four rows (one per wave).
int64_t layer_norm_chunks(int dtype, int64_t B, int64_t T, int64_t d) {
  const int64_t held = dtype == 1 ? backward_resident<bf16s>(d) : backward_resident<float>(d);
  return std::max<int64_t>(1, std::min(held / B, (T + 3) / 4));
}

hipError_t launch_layer_norm(hipStream_t st, int dtype, const LayerNormArgs& a) {
  const bool whole = a.d % (dtype == 1 ? 8 : 4) == 0;
  if (dtype == 1) return whole ? launch_fwd<bf16s, true>(st, a) : launch_fwd<bf16s, false>(st, a);
  return whole ? launch_fwd<float, true>(st, a) : launch_fwd<float, false>(st, a);
}

hipError_t launch_layer_norm_backward(hipStream_t st, int dtype, LayerNormBackArgs a) {
  const bool rows = a.gain_rows || a.bias_rows;
  a.chunks = rows ? layer_norm_chunks(dtype, a.B, a.T, a.d) : layer_norm_chunks(dtype, 1, a.B * a.T, a.d);
  if (!rows) {  // no per-sample sums: the rows are one run
    a.T = a.B * a.T;
    a.B = 1;
  }
  a.chunk_rows = (a.T + a.chunks - 1) / a.chunks;
  // samples of few rows: a wave each, no sum across waves
  a.own_groups = a.chunks == 1 && a.d <= 2048 && (a.T < 8 || a.B >= 4096);
  const bool whole = a.d % (dtype == 1 ? 8 : 4) == 0;
  hipError_t e;
  if (dtype == 1)
    e = whole ? launch_bwd<bf16s, true>(st, a) : launch_bwd<bf16s, false>(st, a);
  else
    e = whole ? launch_bwd<float, true>(st, a) : launch_bwd<float, false>(st, a);
  if (e != hipSuccess || !rows || a.chunks == 1) return e;
  const int64_t blocks = std::min<int64_t>((2 * a.B * a.d + 255) / 256, kLnBlocks);
  k_layer_norm_finish<<<dim3((unsigned)blocks), 256, 0, st>>>(a);
  return hipGetLastError();
}

}  // namespace dpk
