// A router's balance loss per sample with its rows per expert, and the
// gradient of the router's logits.
//
// With p_t = softmax(z_t) over the E experts, a place of a token used when its
// expert lies in [0, E), a token used when one of its places is, n the sample's
// used tokens and counts_e its used places that name e:
//   f_e = counts_e / sum_e' counts_e'      P_e = sum_{t used} p_te / n
//   loss = E sum_e f_e P_e
//   dz_te = p_te (a_e - sum_e' p_te' a_e'),  a_e = dloss E f_e / n   (0 for a token that is not used)
// A sample without a used token has loss 0 and gradient 0, and a used token
// whose logits are all -inf has p = 0 and gradient 0. The gradient does
// not change with a share that all experts have more, so a_e is formed from
// counts_e - min counts: whole numbers, and an even routing gives exactly 0.
//
// Bound by launches and latency at a router's usual sizes (some MB of logits),
// by HBM above. A token's logits are held by 1 to 64 lanes, 8 or 16 of them
// each; a lane keeps its experts over all its tokens, so the sums of
// probabilities are register sums, added across lanes and waves in a fixed
// order; counts are whole numbers, added by atomics in LDS. Two tokens are in
// flight per lane. A sample that gives a workgroup's 1024 threads up to two
// tokens is one workgroup's, so that the loss is one launch; larger ones are
// spread over workgroups whose sums a second launch adds in order (32 samples of
// 1024 tokens, 64 experts: 6 + 4 us, 14 by one workgroup a sample; 9 x 611 tokens
// of 130 experts back: 8 us).
#include "dp_cols.hpp"
#include "dp_common.hpp"
#include "dp_lm.hpp"
#include "dp_vocab.hpp"

namespace dpk {

namespace {

// One token's probabilities from its L lanes' logits: p of every column that this lane holds (its neighbour's among
// them, which do not count in the sums). A row of -inf alone has no distribution, and every p is 0; one with a NaN or
// +inf gives NaN.
template <typename C, int P, int L>
__device__ __forceinline__ void softmax_of(const C& cols, const typename C::Raw& raw, float* v) {
  float m = -INFINITY;
#pragma unroll
  for (int e = 0; e < P; ++e) {
    v[e] = cols.on && cols.at + e < cols.d ? C::value(raw, e) : -INFINITY;
    m = fmaxf(m, v[e]);
  }
#pragma unroll
  for (int off = L / 2; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor(m, off, kWave));
  m = m == -INFINITY ? 0.f : m;  // no difference of infinities: the terms of such a row are 0
  float s = 0.f;
#pragma unroll
  for (int e = 0; e < P; ++e) {
    v[e] = exp2_hw((v[e] - m) * kLog2e);
    s += e < cols.skip || cols.at + e >= cols.d ? 0.f : v[e];
  }
#pragma unroll
  for (int off = L / 2; off > 0; off >>= 1) s += __shfl_xor(s, off, kWave);
  const float inv = s == 0.f ? 0.f : 1.0f / s;  // with a largest logit s is 1 at least
#pragma unroll
  for (int e = 0; e < P; ++e) v[e] *= inv;
}

__device__ __forceinline__ float loss_of(float fp, uint64_t places, uint64_t tokens, int64_t E) {
  return places && tokens ? (float)E * (fp / (float)places) / (float)tokens : 0.f;
}

// Sum over the workgroup, the same in every thread. Contains barriers.
template <int NT>
__device__ __forceinline__ uint64_t block_count(uint64_t v, uint64_t* red) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) v += __shfl_xor(v, off, kWave);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  v = 0;
#pragma unroll
  for (int w = 0; w < NT / 64; ++w) v += red[w];
  return v;
}

// Whether one of token n's places names an expert, of the L lanes that hold the token; they share out the places. A
// place that does is counted (counts != null).
template <int L>
__device__ __forceinline__ bool token_used(const BalanceArgs& a, int64_t n, int sub, uint32_t* counts) {
  bool mine = false;
  for (int k = sub; k < (int)a.top; k += L) {
    const int64_t e = a.ids[n * a.top + k];
    if (e < 0 || e >= a.E) continue;
    mine = true;
    if (counts) atomicAdd(&counts[e], 1u);
  }
  if constexpr (L == 1) return mine;
  const uint64_t lanes = L == 64 ? ~0ull : ((1ull << L) - 1) << (threadIdx.x & 63 & ~(L - 1));
  return (__ballot(mine) & lanes) != 0;
}

}  // namespace

// Work item: (sample, chunk of its tokens), by one workgroup. One chunk: the sample's loss and counts at once.
template <typename T, bool TINY, int L, int P, int NT>
__global__ __launch_bounds__(NT) void k_balance_sums(BalanceArgs a) {
  using C = Cols<T, P, TINY>;
  constexpr int TOKENS = NT / L, WAVES = NT / 64;
  __shared__ float sums[WAVES][L * P];
  __shared__ uint32_t counts[L * P];
  __shared__ uint32_t used_tokens;
  __shared__ float red[WAVES];
  __shared__ uint64_t redc[WAVES];
  const int E = (int)a.E;
  const int slot = threadIdx.x / L, sub = threadIdx.x % L, wave = threadIdx.x >> 6;
  const C cols(sub * P, a.E);
  for (int64_t item = blockIdx.x; item < a.B * a.chunks; item += gridDim.x) {
    const int64_t b = item / a.chunks, ch = item - b * a.chunks;
    const int64_t t0 = ch * a.chunk_rows, t1 = t0 + a.chunk_rows < a.T ? t0 + a.chunk_rows : a.T;
    for (int k = threadIdx.x; k < L * P; k += NT) counts[k] = 0;
    if (threadIdx.x == 0) used_tokens = 0;
    __syncthreads();
    float acc[P];
#pragma unroll
    for (int e = 0; e < P; ++e) acc[e] = 0.f;
    uint32_t tokens = 0;
    for (int64_t t = t0 + slot; t < t1; t += 2 * TOKENS) {  // a token's lanes go through it together
      typename C::Raw raw[2];
      bool used[2];
#pragma unroll
      for (int u = 0; u < 2; ++u) raw[u] = cols.fetch(a.logits, t + u * TOKENS < t1 ? b * a.T + t + u * TOKENS : -1);
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        used[u] = t + u * TOKENS < t1 && token_used<L>(a, b * a.T + t + u * TOKENS, sub, counts);
        tokens += used[u] && sub == 0;
      }
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        float p[P];
        softmax_of<C, P, L>(cols, raw[u], p);
#pragma unroll
        for (int e = 0; e < P; ++e) acc[e] += used[u] ? p[e] : 0.f;
      }
    }
    if (tokens) atomicAdd(&used_tokens, tokens);
    // over the wave's tokens (the lanes that hold the same experts), then over the waves
#pragma unroll
    for (int off = L; off < 64; off <<= 1)
#pragma unroll
      for (int e = 0; e < P; ++e) acc[e] += __shfl_xor(acc[e], off, kWave);
    if ((threadIdx.x & 63) < L) {
#pragma unroll
      for (int e = 0; e < P; ++e)
        if (e >= cols.skip && cols.at + e < E) sums[wave][cols.at + e] = acc[e];
    }
    __syncthreads();
    float fp = 0.f;
    uint64_t places = 0;
    for (int e = threadIdx.x; e < E; e += NT) {
      float s = 0.f;
#pragma unroll
      for (int w = 0; w < WAVES; ++w) s += sums[w][e];
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
      places = block_count<NT>(places, redc);
      fp = block_sum<NT>(fp, red);
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

// A sample's chunks, added in order, by one workgroup: its waves take parts of the chunks, the first wave the rest.
__global__ __launch_bounds__(512) void k_balance_finish(BalanceArgs a) {
  constexpr int WAVES = 8;
  __shared__ float part[2][WAVES][64];
  __shared__ uint32_t partc[2][WAVES][64];
  const int E = (int)a.E, wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  for (int64_t b = blockIdx.x; b < a.B; b += gridDim.x) {
    float fp = 0.f;
    uint64_t places = 0, tokens = 0;
    if (wave == 0)
      for (int64_t ch = lane; ch < a.chunks; ch += 64) tokens += a.part_counts[(b * a.chunks + ch) * (a.E + 1) + a.E];
    int half = 0;
    for (int e0 = 0; e0 < E; e0 += 64, half ^= 1) {  // the halves take turns: one barrier a round
      const int e = e0 + lane;
      float s = 0.f;
      uint32_t c = 0;
      if (e < E) {
#pragma unroll 4
        for (int64_t ch = wave; ch < a.chunks; ch += WAVES) {
          s += a.part_sums[(b * a.chunks + ch) * a.E + e];
          c += a.part_counts[(b * a.chunks + ch) * (a.E + 1) + e];
        }
      }
      part[half][wave][lane] = s;
      partc[half][wave][lane] = c;
      __syncthreads();
      if (wave == 0 && e < E) {
#pragma unroll
        for (int w = 1; w < WAVES; ++w) {
          s += part[half][w][lane];
          c += partc[half][w][lane];
        }
        a.counts[b * a.E + e] = c;
        fp = __builtin_fmaf((float)c, s, fp);
        places += c;
      }
    }
    if (wave == 0) {
      fp = wave_sum(fp);
#pragma unroll
      for (int off = 32; off > 0; off >>= 1) {
        places += __shfl_xor(places, off, kWave);
        tokens += __shfl_xor(tokens, off, kWave);
      }
      if (lane == 0) {
        a.loss[b] = loss_of(fp, places, tokens, a.E);
        a.tokens[b] = (int64_t)tokens;
      }
    }
    __syncthreads();
  }
}

// Work item: (sample, chunk of its tokens), by one workgroup.
template <typename T, bool TINY, int L, int P>
__global__ __launch_bounds__(256) void k_balance_backward(BalanceArgs a) {
  using C = Cols<T, P, TINY>;
  constexpr int TOKENS = 256 / L;
  const int slot = threadIdx.x / L, sub = threadIdx.x % L;
  const C cols(sub * P, a.E);
  for (int64_t item = blockIdx.x; item < a.B * a.chunks; item += gridDim.x) {
    const int64_t b = item / a.chunks, ch = item - b * a.chunks;
    const int64_t t0 = ch * a.chunk_rows, t1 = t0 + a.chunk_rows < a.T ? t0 + a.chunk_rows : a.T;
    // ---- what the loss passes to the probabilities of this lane's experts
    int64_t c[P], least = INT64_MAX, places = 0;
#pragma unroll
    for (int e = 0; e < P; ++e) {
      const bool in = cols.on && cols.at + e < cols.d;
      c[e] = in ? a.counts[b * a.E + cols.at + e] : 0;
      if (in) least = c[e] < least ? c[e] : least;
      if (in && e >= cols.skip) places += c[e];
    }
#pragma unroll
    for (int off = L / 2; off > 0; off >>= 1) {
      const int64_t o = __shfl_xor(least, off, kWave);
      least = o < least ? o : least;
      places += __shfl_xor(places, off, kWave);
    }
    const int64_t tokens = a.tokens[b];
    const float dl = a.dloss ? a.dloss[b] : 1.0f;
    const float f = places > 0 && tokens > 0 ? dl * (float)a.E / ((float)places * (float)tokens) : 0.f;
    float w[P];
#pragma unroll
    for (int e = 0; e < P; ++e) w[e] = cols.on && cols.at + e < cols.d ? (float)(c[e] - least) * f : 0.f;
    for (int64_t t = t0 + slot; t < t1; t += 2 * TOKENS) {
      typename C::Raw raw[2];
      bool used[2];
#pragma unroll
      for (int u = 0; u < 2; ++u) raw[u] = cols.fetch(a.logits, t + u * TOKENS < t1 ? b * a.T + t + u * TOKENS : -1);
#pragma unroll
      for (int u = 0; u < 2; ++u)
        used[u] = t + u * TOKENS < t1 && token_used<L>(a, b * a.T + t + u * TOKENS, sub, nullptr) && f != 0.f;
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        float p[P], inner = 0.f;
        softmax_of<C, P, L>(cols, raw[u], p);
#pragma unroll
        for (int e = 0; e < P; ++e) inner = __builtin_fmaf(p[e], e < cols.skip ? 0.f : w[e], inner);
#pragma unroll
        for (int off = L / 2; off > 0; off >>= 1) inner += __shfl_xor(inner, off, kWave);
#pragma unroll
        for (int e = 0; e < P; ++e) p[e] = used[u] ? p[e] * (w[e] - inner) : 0.f;
        if (t + u * TOKENS < t1) cols.put(a.grad, b * a.T + t + u * TOKENS, p);
      }
    }
  }
}

namespace {

unsigned grid_of(int64_t n) { return (unsigned)std::min<int64_t>(n, 1 << 20); }

// f(lanes for a token, experts of a lane, whether rows are narrower than that): 8 experts a lane, 16 above 512.
template <typename F>
hipError_t balance_dispatch(int64_t E, F f) {
  constexpr std::integral_constant<int, 8> eight{};
  if (E < 8) return f(std::integral_constant<int, 1>{}, eight, std::true_type{});
  if (E == 8) return f(std::integral_constant<int, 1>{}, eight, std::false_type{});
  if (E <= 16) return f(std::integral_constant<int, 2>{}, eight, std::false_type{});
  if (E <= 32) return f(std::integral_constant<int, 4>{}, eight, std::false_type{});
  if (E <= 64) return f(std::integral_constant<int, 8>{}, eight, std::false_type{});
  if (E <= 128) return f(std::integral_constant<int, 16>{}, eight, std::false_type{});
  if (E <= 256) return f(std::integral_constant<int, 32>{}, eight, std::false_type{});
  if (E <= 512) return f(std::integral_constant<int, 64>{}, eight, std::false_type{});
  return f(std::integral_constant<int, 64>{}, std::integral_constant<int, 16>{}, std::false_type{});
}

// How a sample's tokens are spread over workgroups. The sums: not at all up to
// 2048 lanes' tokens (two for each thread of a workgroup), or where there are
// samples for every CU; else about two workgroups per CU, each of at least 32 tokens.
int64_t spread(int64_t B, int64_t T, int64_t least) {
  const int64_t want = (512 + B - 1) / B, most = (T + least - 1) / least;
  return std::max<int64_t>(1, std::min(want, most));
}
int64_t balance_chunks(int64_t B, int64_t T, int64_t E) {
  const int64_t lanes = T * ((E + 7) / 8);
  return lanes <= 2048 || (B >= 256 && lanes <= 65536) ? 1 : spread(B, T, 32);
}

template <typename T>
hipError_t launch_sums(hipStream_t st, const BalanceArgs& a) {
  return balance_dispatch(a.E, [&](auto l, auto p, auto tiny) {
    constexpr int L = decltype(l)::value, P = decltype(p)::value;
    constexpr bool TINY = decltype(tiny)::value;
    // a sample to a workgroup: as many threads as its tokens' lanes need
    if (a.chunks == 1 && a.T * L > 256) k_balance_sums<T, TINY, L, P, 1024><<<grid_of(a.B), 1024, 0, st>>>(a);
    else k_balance_sums<T, TINY, L, P, 256><<<grid_of(a.B * a.chunks), 256, 0, st>>>(a);
    return hipGetLastError();
  });
}

template <typename T>
hipError_t launch_back(hipStream_t st, const BalanceArgs& a) {
  return balance_dispatch(a.E, [&](auto l, auto p, auto tiny) {
    k_balance_backward<T, decltype(tiny)::value, decltype(l)::value, decltype(p)::value>
        <<<grid_of(a.B * a.chunks), 256, 0, st>>>(a);
    return hipGetLastError();
  });
}

}  // namespace

size_t balance_ws_bytes(int64_t B, int64_t T, int64_t E) {
  const int64_t chunks = balance_chunks(B, T, E);
  return chunks > 1 ? ((size_t)(B * chunks) * (size_t)(2 * E + 1) * 4 + 255) / 256 * 256 : 0;
}

hipError_t launch_balance_loss(hipStream_t st, int dtype, BalanceArgs a, void* ws) {
  a.chunks = balance_chunks(a.B, a.T, a.E);
  a.chunk_rows = (a.T + a.chunks - 1) / a.chunks;
  a.part_sums = static_cast<float*>(ws);
  a.part_counts = reinterpret_cast<uint32_t*>(a.part_sums + a.B * a.chunks * a.E);
  const hipError_t e = dtype == 1 ? launch_sums<bf16s>(st, a) : launch_sums<float>(st, a);
  if (e != hipSuccess || a.chunks == 1) return e;
  k_balance_finish<<<grid_of(a.B), 512, 0, st>>>(a);
  return hipGetLastError();
}

hipError_t launch_balance_backward(hipStream_t st, int dtype, BalanceArgs a) {
  // about four workgroups per CU, each of at least two rounds of its tokens
  const int64_t lanes = a.E <= 512 ? (a.E + 7) / 8 : 64;
  a.chunks = std::max<int64_t>(1, std::min<int64_t>((1024 + a.B - 1) / a.B, a.T * lanes / 512));
  a.chunk_rows = (a.T + a.chunks - 1) / a.chunks;
  return dtype == 1 ? launch_back<bf16s>(st, a) : launch_back<float>(st, a);
}

}  // namespace dpk
