// A router's balance loss per sample with its rows per expert, and the
// gradient of the router's logits.
//
// With p_t = softmax(z_t) over the E experts, a place of a token used when its
// expert lies in [0, E), a token used when one of its places is, n the sample's
// used tokens and counts_e its used places that name e:
//   f_e = counts_e / sum_e' counts_e'      P_e = sum_{t used} p_te / n
//   loss = E sum_e f_e P_e
//   dz_te = p_te (a_e - sum_e' p_te' a_e'),  a_e = dloss E f_e / n   (0 for a token that is not used)
// A sample without a used token has loss 0 and gradient 0. The gradient does
// not change with a share that all experts have more, so a_e is formed from
// counts_e - min counts: whole numbers, and an even routing gives exactly 0.
//
// Bound by launches and latency at a router's usual sizes (some MB of logits),
// by HBM above. A token's logits are held by 1 to 64 lanes, 8 or 16 of them
// each, as 16-byte vectors; a lane keeps its experts over all its tokens, so
// the sums of probabilities are register sums, added across lanes and waves in
// a fixed order; counts are whole numbers, added by atomics in LDS. Samples of
// many tokens are spread over workgroups whose sums a second launch adds in
// order.
#include "dp_common.hpp"
#include "dp_lm.hpp"
#include "dp_rows.hpp"
#include "dp_vocab.hpp"

namespace dpk {

namespace {

constexpr int kBalanceThreads = 256;

// One token's probabilities from its L lanes' logits (columns past E: 0). A row of -inf alone gives NaN, as a row
// with a NaN does.
template <typename M, int L, int N>
__device__ __forceinline__ void softmax_of(const typename M::Raw& raw, int E, int sub, float* v) {
  M::unpack(raw, v);
  float m = -INFINITY;
#pragma unroll
  for (int k = 0; k < N; ++k) {
    if (M::col(k / M::P, sub) + k % M::P >= E) v[k] = -INFINITY;
    m = fmaxf(m, v[k]);
  }
#pragma unroll
  for (int off = L / 2; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor(m, off, kWave));
  float s = 0.f;
#pragma unroll
  for (int k = 0; k < N; ++k) {
    v[k] = M::col(k / M::P, sub) + k % M::P < E ? exp2_hw((v[k] - m) * kLog2e) : 0.f;
    s += v[k];
  }
#pragma unroll
  for (int off = L / 2; off > 0; off >>= 1) s += __shfl_xor(s, off, kWave);
  const float inv = 1.0f / s;
#pragma unroll
  for (int k = 0; k < N; ++k) v[k] *= inv;
}

__device__ __forceinline__ float loss_of(float fp, uint64_t places, uint64_t tokens, int64_t E) {
  return places && tokens ? (float)E * (fp / (float)places) / (float)tokens : 0.f;
}

// Sum over the workgroup, the same in every thread. Contains barriers.
__device__ __forceinline__ uint64_t block_count(uint64_t v, uint64_t* red) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) v += __shfl_xor(v, off, kWave);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  return red[0] + red[1] + red[2] + red[3];
}

}  // namespace

// Work item: (sample, chunk of its tokens), by one workgroup. One chunk: the sample's loss and counts at once.
template <typename T, bool WHOLE, int L, int N>
__global__ __launch_bounds__(kBalanceThreads) void k_balance_sums(BalanceArgs a) {
  using M = RowMap<T, WHOLE, N, L>;
  constexpr int TOKENS = kBalanceThreads / L, WAVES = kBalanceThreads / 64;
  __shared__ float sums[WAVES][L * N];
  __shared__ uint32_t counts[L * N];
  __shared__ uint32_t used_tokens;
  __shared__ float red[WAVES];
  __shared__ uint64_t redc[WAVES];
  const int E = (int)a.E, top = (int)a.top;
  const int slot = threadIdx.x / L, sub = threadIdx.x % L, wave = threadIdx.x >> 6;
  for (int64_t item = blockIdx.x; item < a.B * a.chunks; item += gridDim.x) {
    const int64_t b = item / a.chunks, ch = item - b * a.chunks;
    const int64_t t0 = ch * a.chunk_rows, t1 = t0 + a.chunk_rows < a.T ? t0 + a.chunk_rows : a.T;
    for (int k = threadIdx.x; k < L * N; k += kBalanceThreads) counts[k] = 0;
    if (threadIdx.x == 0) used_tokens = 0;
    __syncthreads();
    float acc[N];
#pragma unroll
    for (int k = 0; k < N; ++k) acc[k] = 0.f;
    for (int64_t t = t0 + slot; t < t1; t += TOKENS) {
      const int64_t n = b * a.T + t;
      typename M::Raw raw;
      M::fetch(static_cast<const T*>(a.logits) + n * a.E, E, sub, raw);
      bool used = false;
      for (int k = 0; k < top; ++k) {
        const int64_t e = a.ids[n * top + k];
        if (e < 0 || e >= a.E) continue;
        used = true;
        if (k % L == sub) atomicAdd(&counts[e], 1u);
      }
      if (used && sub == 0) atomicAdd(&used_tokens, 1u);
      float p[N];
      softmax_of<M, L, N>(raw, E, sub, p);  // a token's lanes go through it together
#pragma unroll
      for (int k = 0; k < N; ++k) acc[k] += used ? p[k] : 0.f;
    }
    // over the wave's tokens (the lanes that hold the same experts), then over the waves
#pragma unroll
    for (int off = L; off < 64; off <<= 1)
#pragma unroll
      for (int k = 0; k < N; ++k) acc[k] += __shfl_xor(acc[k], off, kWave);
    if ((threadIdx.x & 63) < L) {
#pragma unroll
      for (int k = 0; k < N; ++k) sums[wave][M::col(k / M::P, sub) + k % M::P] = acc[k];
    }
    __syncthreads();
    float fp = 0.f;
    uint64_t places = 0;
    for (int e = threadIdx.x; e < E; e += kBalanceThreads) {
      const float s = ((sums[0][e] + sums[1][e]) + sums[2][e]) + sums[3][e];
      const uint32_t c = counts[e];
      if (a.chunks == 1) {
        a.counts[b * a.E + e] = c;
        fp = __builtin_fmaf((float)c, s, fp);
        places += c;
      } else {
        a.part_sums[item * a.E + e] = s;
        a.part_counts[item * (a.E + 1) + e] = c;
      }
    }
    if (a.chunks == 1) {
      places = block_count(places, redc);
      fp = block_sum<kBalanceThreads>(fp, red);
      if (threadIdx.x == 0) {
        a.loss[b] = loss_of(fp, places, used_tokens, a.E);
        a.tokens[b] = used_tokens;
      }
    } else if (threadIdx.x == 0) {
      a.part_counts[item * (a.E + 1) + a.E] = used_tokens;
    }
    __syncthreads();
  }
}

// A sample's chunks, added in order.
__global__ __launch_bounds__(kBalanceThreads) void k_balance_finish(BalanceArgs a) {
  __shared__ float red[kBalanceThreads / 64];
  __shared__ uint64_t redc[kBalanceThreads / 64];
  const int E = (int)a.E;
  for (int64_t b = blockIdx.x; b < a.B; b += gridDim.x) {
    float fp = 0.f;
    uint64_t places = 0, tokens = 0;
    for (int e = threadIdx.x; e < E; e += kBalanceThreads) {
      float s = 0.f;
      uint64_t c = 0;
#pragma unroll 8
      for (int64_t ch = 0; ch < a.chunks; ++ch) {
        s += a.part_sums[(b * a.chunks + ch) * a.E + e];
        c += a.part_counts[(b * a.chunks + ch) * (a.E + 1) + e];
      }
      a.counts[b * a.E + e] = (int64_t)c;
      fp = __builtin_fmaf((float)c, s, fp);
      places += c;
    }
    for (int64_t ch = threadIdx.x; ch < a.chunks; ch += kBalanceThreads)
      tokens += a.part_counts[(b * a.chunks + ch) * (a.E + 1) + a.E];
    places = block_count(places, redc);
    tokens = block_count(tokens, redc);
    fp = block_sum<kBalanceThreads>(fp, red);
    if (threadIdx.x == 0) {
      a.loss[b] = loss_of(fp, places, tokens, a.E);
      a.tokens[b] = (int64_t)tokens;
    }
    __syncthreads();
  }
}

// Work item: (sample, chunk of its tokens), by one workgroup.
template <typename T, bool WHOLE, int L, int N>
__global__ __launch_bounds__(kBalanceThreads) void k_balance_backward(BalanceArgs a) {
  using M = RowMap<T, WHOLE, N, L>;
  constexpr int TOKENS = kBalanceThreads / L;
  const int E = (int)a.E, top = (int)a.top;
  const int slot = threadIdx.x / L, sub = threadIdx.x % L;
  for (int64_t item = blockIdx.x; item < a.B * a.chunks; item += gridDim.x) {
    const int64_t b = item / a.chunks, ch = item - b * a.chunks;
    const int64_t t0 = ch * a.chunk_rows, t1 = t0 + a.chunk_rows < a.T ? t0 + a.chunk_rows : a.T;
    // ---- what the loss passes to the probabilities of this lane's experts
    int64_t c[N], least = INT64_MAX, places = 0;
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const int e = M::col(k / M::P, sub) + k % M::P;
      c[k] = e < E ? a.counts[b * a.E + e] : -1;
      if (e < E) {
        places += c[k];
        least = c[k] < least ? c[k] : least;
      }
    }
#pragma unroll
    for (int off = L / 2; off > 0; off >>= 1) {
      const int64_t o = __shfl_xor(least, off, kWave);
      least = o < least ? o : least;
      places += __shfl_xor(places, off, kWave);
    }
    const int64_t tokens = a.tokens[b];
    const float dl = a.dloss ? a.dloss[b] : 1.0f;
    const float f = places > 0 && tokens > 0 ? dl * (float)E / ((float)places * (float)tokens) : 0.f;
    float w[N];
#pragma unroll
    for (int k = 0; k < N; ++k) w[k] = c[k] < 0 ? 0.f : (float)(c[k] - least) * f;
    for (int64_t t = t0 + slot; t < t1; t += TOKENS) {
      const int64_t n = b * a.T + t;
      typename M::Raw raw;
      M::fetch(static_cast<const T*>(a.logits) + n * a.E, E, sub, raw);
      bool used = false;
      for (int k = 0; k < top; ++k) {
        const int64_t e = a.ids[n * top + k];
        used = used || (e >= 0 && e < a.E);
      }
      used = used && f != 0.f;
      float p[N];
      softmax_of<M, L, N>(raw, E, sub, p);
      float inner = 0.f;
#pragma unroll
      for (int k = 0; k < N; ++k) inner = __builtin_fmaf(p[k], w[k], inner);
#pragma unroll
      for (int off = L / 2; off > 0; off >>= 1) inner += __shfl_xor(inner, off, kWave);
#pragma unroll
      for (int k = 0; k < N; ++k) p[k] = used ? p[k] * (w[k] - inner) : 0.f;
      M::store(static_cast<T*>(a.grad) + n * a.E, E, sub, p);
    }
  }
}

namespace {

unsigned grid_of(int64_t n) { return (unsigned)std::min<int64_t>(n, 1 << 20); }

// Lanes for a token, 8 experts each (16 above 512).
template <typename F>
hipError_t balance_dispatch(int64_t E, F f) {
  if (E <= 8) return f(std::integral_constant<int, 1>{}, std::integral_constant<int, 8>{});
  if (E <= 16) return f(std::integral_constant<int, 2>{}, std::integral_constant<int, 8>{});
  if (E <= 32) return f(std::integral_constant<int, 4>{}, std::integral_constant<int, 8>{});
  if (E <= 64) return f(std::integral_constant<int, 8>{}, std::integral_constant<int, 8>{});
  if (E <= 128) return f(std::integral_constant<int, 16>{}, std::integral_constant<int, 8>{});
  if (E <= 256) return f(std::integral_constant<int, 32>{}, std::integral_constant<int, 8>{});
  if (E <= 512) return f(std::integral_constant<int, 64>{}, std::integral_constant<int, 8>{});
  return f(std::integral_constant<int, 64>{}, std::integral_constant<int, 16>{});
}

// How a sample's tokens are spread over workgroups: about two workgroups per CU, each of at least 32 tokens.
int64_t balance_chunks(int64_t B, int64_t T) {
  const int64_t want = (512 + B - 1) / B, most = (T + 31) / 32;
  return std::max<int64_t>(1, std::min(want, most));
}

template <typename T, bool WHOLE>
hipError_t launch_sums(hipStream_t st, const BalanceArgs& a) {
  return balance_dispatch(a.E, [&](auto l, auto n) {
    k_balance_sums<T, WHOLE, decltype(l)::value, decltype(n)::value>
        <<<grid_of(a.B * a.chunks), kBalanceThreads, 0, st>>>(a);
    return hipGetLastError();
  });
}

template <typename T, bool WHOLE>
hipError_t launch_back(hipStream_t st, const BalanceArgs& a) {
  return balance_dispatch(a.E, [&](auto l, auto n) {
    k_balance_backward<T, WHOLE, decltype(l)::value, decltype(n)::value>
        <<<grid_of(a.B * a.chunks), kBalanceThreads, 0, st>>>(a);
    return hipGetLastError();
  });
}

}  // namespace

size_t balance_ws_bytes(int64_t B, int64_t T, int64_t E) {
  const int64_t chunks = balance_chunks(B, T);
  return chunks > 1 ? ((size_t)(B * chunks) * (size_t)(2 * E + 1) * 4 + 255) / 256 * 256 : 0;
}

hipError_t launch_balance_loss(hipStream_t st, int dtype, BalanceArgs a, void* ws) {
  a.chunks = balance_chunks(a.B, a.T);
  a.chunk_rows = (a.T + a.chunks - 1) / a.chunks;
  a.part_sums = static_cast<float*>(ws);
  a.part_counts = reinterpret_cast<uint32_t*>(a.part_sums + a.B * a.chunks * a.E);
  const bool whole = a.E % (dtype == 1 ? 8 : 4) == 0;
  hipError_t e;
  if (dtype == 1) e = whole ? launch_sums<bf16s, true>(st, a) : launch_sums<bf16s, false>(st, a);
  else e = whole ? launch_sums<float, true>(st, a) : launch_sums<float, false>(st, a);
  if (e != hipSuccess || a.chunks == 1) return e;
  k_balance_finish<<<grid_of(a.B), kBalanceThreads, 0, st>>>(a);
  return hipGetLastError();
}

hipError_t launch_balance_backward(hipStream_t st, int dtype, BalanceArgs a) {
  a.chunks = balance_chunks(a.B, a.T);
  a.chunk_rows = (a.T + a.chunks - 1) / a.chunks;
  const bool whole = a.E % (dtype == 1 ? 8 : 4) == 0;
  if (dtype == 1) return whole ? launch_back<bf16s, true>(st, a) : launch_back<bf16s, false>(st, a);
  return whole ? launch_back<float, true>(st, a) : launch_back<float, false>(st, a);
}

}  // namespace dpk
