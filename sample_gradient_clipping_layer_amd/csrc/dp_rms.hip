// Root-mean-square norm with the residual's addition, and its backward pass
// with the gain's gradient of every sample.
//
//   forward:   s = x + r,  u = s / sqrt(mean(s^2) + eps),  y = u * gain
//   backward:  h = dy * gain,  ds = dsum + rstd * (h - u * mean(h * u)),
//              gain_rows[b] = sum_t dy[b][t] * u[b][t]
//
// Both are bound by HBM: each element is read once and written once, about
// 10 fp32 operations in between (32768 x 1280 bf16: forward 60 us, 5.6 TB/s;
// backward 67 us, 5.0 TB/s, and 5 us for the join of the gains' partial sums;
// a large copy reaches 5.1 TB/s). A row is held in the registers of one, four
// or sixteen waves (8 to 32 elements per lane), so that one pass over memory
// serves the row's reductions and its outputs. Rows of up to 2048 elements
// take one wave, whose reductions are lane shuffles without a barrier.
//
// The backward recomputes the row's 1/rms (the row is in registers anyway)
// and forms both row sums, sum(s^2) and sum(h * s), in one reduction:
// mean(h * u) = rstd * sum(h * s) / d. A lane keeps the columns it holds over
// all its rows, so the gain's per-sample gradient is a register sum; the
// waves of a workgroup add theirs through LDS in wave order, and when a
// sample is spread over several workgroups their partial sums go through the
// workspace and a second kernel adds them in order. Nothing is atomic.
#include "dp_common.hpp"
#include "dp_lm.hpp"
#include "dp_rows.hpp"

namespace dpk {

namespace {

// Sums of two values over the LPR lanes of a row, the same bits in every
// lane. WPR > 1: through LDS, `red` holding 2 floats per wave of the block,
// twice (alternating rows use alternating halves, so one barrier a row
// suffices).
template <int WPR>
__device__ __forceinline__ void row_sum2(float& a, float& b, float* red, int wave, int& phase) {
  a = wave_sum(a);
  b = wave_sum(b);
  if constexpr (WPR > 1) {
    float* r = red + phase * 32;
    if ((threadIdx.x & 63) == 0) {
      r[2 * wave] = a;
      r[2 * wave + 1] = b;
    }
    __syncthreads();
    a = 0.f;
    b = 0.f;
#pragma unroll
    for (int w = 0; w < WPR; ++w) {
      a += r[2 * w];
      b += r[2 * w + 1];
    }
    phase ^= 1;
  }
}

}  // namespace

template <typename T, bool WHOLE, int E, int WPR>
__global__ __launch_bounds__(row_threads<WPR>()) void k_rms_norm(RmsArgs a) {
  constexpr int NW = row_threads<WPR>() / 64, GROUPS = NW / WPR, LPR = 64 * WPR;
  using M = RowMap<T, WHOLE, E, LPR>;
  __shared__ float red[64];
  const int wave = threadIdx.x >> 6;
  const int group = WPR == 1 ? wave : 0;
  const int lane = WPR == 1 ? (threadIdx.x & 63) : threadIdx.x;
  int phase = 0;
  float g[E];
  M::load_gain(a.gain, a.gain_bf16, (int)a.d, lane, g);
  const float inv_d = 1.0f / (float)a.d;
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
    float ss = 0.f, unused = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) ss = __builtin_fmaf(v[e], v[e], ss);
    if (a.sum_out) M::store(static_cast<T*>(a.sum_out) + row * a.d, (int)a.d, lane, v);
    row_sum2<WPR>(ss, unused, red, wave, phase);
    const float rstd = 1.0f / sqrtf(__builtin_fmaf(ss, inv_d, a.eps));
    // y from the sum before its rounding to the storage type
#pragma unroll
    for (int e = 0; e < E; ++e) v[e] = v[e] * rstd * g[e];
    M::store(static_cast<T*>(a.out) + row * a.d, (int)a.d, lane, v);
  }
}

// Work items: (sample, chunk of its rows); with `own_groups` every group of
// a block takes a sample of its own (chunks == 1).
template <typename T, bool WHOLE, int E, int WPR>
__global__ __launch_bounds__(row_threads<WPR>()) void k_rms_norm_backward(RmsBackArgs a) {
  constexpr int NW = row_threads<WPR>() / 64, GROUPS = NW / WPR, LPR = 64 * WPR;
  using M = RowMap<T, WHOLE, E, LPR>;
  __shared__ float red[64];
  __shared__ float part[GROUPS > 1 ? (GROUPS - 1) * E * 64 : 1];
  const int wave = threadIdx.x >> 6;
  const int group = WPR == 1 ? wave : 0;
  const int lane = WPR == 1 ? (threadIdx.x & 63) : threadIdx.x;
  int phase = 0;
  float g[E];
  // 1024-thread blocks have 128 registers a lane: the gain is read again for every row there (from L2)
  if constexpr (WPR < 16) M::load_gain(a.gain, a.gain_bf16, (int)a.d, lane, g);
  const float inv_d = 1.0f / (float)a.d;
  const int64_t per_block = a.own_groups ? GROUPS : 1;
  const int64_t items = a.B * a.chunks;
  for (int64_t item0 = (int64_t)blockIdx.x * per_block; item0 < items; item0 += (int64_t)gridDim.x * per_block) {
    const int64_t item = item0 + (a.own_groups ? group : 0);
    const int64_t b = item / a.chunks, ch = item - b * a.chunks;
    const int64_t t0 = ch * a.chunk_rows;
    int64_t t1 = t0 + a.chunk_rows < a.T ? t0 + a.chunk_rows : a.T;
    if (item >= items) t1 = t0;  // a group past the last sample (WPR == 1: no barrier is skipped below)
    float acc[E];
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = 0.f;
    for (int64_t t = t0 + (a.own_groups ? 0 : group); t < t1; t += (a.own_groups ? 1 : GROUPS)) {
      const int64_t off = (b * a.T + t) * a.d;
      typename M::Raw rs, rh, ro;
      M::fetch(static_cast<const T*>(a.s) + off, (int)a.d, lane, rs);
      M::fetch(static_cast<const T*>(a.dy) + off, (int)a.d, lane, rh);
      if (WPR < 16 && a.dsum) M::fetch(static_cast<const T*>(a.dsum) + off, (int)a.d, lane, ro);
      if constexpr (WPR == 16) M::load_gain(a.gain, a.gain_bf16, (int)a.d, lane, g);
      float s[E], h[E];
      M::unpack(rs, s);
      M::unpack(rh, h);
      float ss = 0.f, hs = 0.f;
#pragma unroll
      for (int e = 0; e < E; ++e) {
        ss = __builtin_fmaf(s[e], s[e], ss);
        hs = __builtin_fmaf(h[e] * g[e], s[e], hs);
      }
      row_sum2<WPR>(ss, hs, red, wave, phase);
      const float rstd = 1.0f / sqrtf(__builtin_fmaf(ss, inv_d, a.eps));
      if (a.dx) {
        const float along = hs * inv_d * rstd * rstd;  // mean(h u) * rstd, for u = s * rstd
        float o[E];
        if (a.dsum) {
          if (WPR == 16) M::fetch(static_cast<const T*>(a.dsum) + off, (int)a.d, lane, ro);
          M::unpack(ro, o);
        } else {
#pragma unroll
          for (int e = 0; e < E; ++e) o[e] = 0.f;
        }
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = __builtin_fmaf(rstd, h[e] * g[e] - s[e] * along, o[e]);
        M::store(static_cast<T*>(a.dx) + off, (int)a.d, lane, o);
      }
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] = __builtin_fmaf(h[e], s[e] * rstd, acc[e]);
    }
    if (!a.gain_rows) continue;
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
    if (writes) {
      float* dst = (a.chunks == 1 ? a.gain_rows : a.partial) + item * a.d;
      M::store_f32(dst, (int)a.d, lane, acc);
    }
  }
}

// gain_rows[b][c] = the sum of the sample's chunk partials in chunk order.
__global__ __launch_bounds__(256) void k_rms_gain_finish(const float* __restrict__ partial, int64_t B, int64_t chunks,
                                                         int64_t d, float* __restrict__ gain_rows) {
  const int64_t n = B * d;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
    const int64_t b = i / d, c = i - b * d;
    const float* p = partial + b * chunks * d + c;
    float s = 0.f;
#pragma unroll 4
    for (int64_t k = 0; k < chunks; ++k) s += p[k * d];
    gain_rows[i] = s;
  }
}

namespace {

constexpr int64_t kRmsBlocks = 256 * 8;  // blocks that fill the 256 CUs; more rows than that are looped over

template <typename T, bool WHOLE>
hipError_t launch_fwd(hipStream_t st, const RmsArgs& a) {
  return row_dispatch(a.d, [&](auto e, auto w) {
    constexpr int E = decltype(e)::value, WPR = decltype(w)::value;
    const int64_t groups = row_groups(a.d);
    const int64_t blocks = std::min<int64_t>((a.rows + groups - 1) / groups, kRmsBlocks);
    k_rms_norm<T, WHOLE, E, WPR><<<dim3((unsigned)blocks), row_threads<WPR>(), 0, st>>>(a);
    return hipGetLastError();
  });
}

template <typename T, bool WHOLE>
hipError_t launch_bwd(hipStream_t st, const RmsBackArgs& a) {
  return row_dispatch(a.d, [&](auto e, auto w) {
    constexpr int E = decltype(e)::value, WPR = decltype(w)::value;
    const int64_t per = a.own_groups ? row_groups(a.d) : 1;
    const int64_t blocks = std::min<int64_t>((a.B * a.chunks + per - 1) / per, kRmsBlocks);
    k_rms_norm_backward<T, WHOLE, E, WPR><<<dim3((unsigned)blocks), row_threads<WPR>(), 0, st>>>(a);
    return hipGetLastError();
  });
}

}  // namespace

// How a sample's rows are spread over workgroups: as many chunks as it takes
// for about four workgroups per CU, each of at least four rows (one per wave).
int64_t rms_chunks(int64_t B, int64_t T) {
  const int64_t want = (1024 + B - 1) / B;
  const int64_t most = (T + 3) / 4;
  return std::max<int64_t>(1, std::min(want, most));
}

hipError_t launch_rms_norm(hipStream_t st, int dtype, const RmsArgs& a) {
  const bool whole = a.d % (dtype == 1 ? 8 : 4) == 0;
  if (dtype == 1) return whole ? launch_fwd<bf16s, true>(st, a) : launch_fwd<bf16s, false>(st, a);
  return whole ? launch_fwd<float, true>(st, a) : launch_fwd<float, false>(st, a);
}

hipError_t launch_rms_norm_backward(hipStream_t st, int dtype, RmsBackArgs a) {
  a.chunks = a.gain_rows ? rms_chunks(a.B, a.T) : rms_chunks(1, a.B * a.T);
  if (!a.gain_rows) {  // no per-sample sums: the rows are one run
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
  if (e != hipSuccess || !a.gain_rows || a.chunks == 1) return e;
  const int64_t blocks = std::min<int64_t>((a.B * a.d + 255) / 256, kRmsBlocks);
  k_rms_gain_finish<<<dim3((unsigned)blocks), 256, 0, st>>>(a.partial, a.B, a.chunks, a.d, a.gain_rows);
  return hipGetLastError();
}

}  // namespace dpk
