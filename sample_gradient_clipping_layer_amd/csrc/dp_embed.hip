// A table of words: the lookup of scaled rows, the order of tokens by word,
// and the clipping of the table's gradient.
//
//   lookup:  out[n] = scale * W[ids[n]]  (0 for an id outside [0, V): a dropped token)
//   order:   word 2^32 + token of every token, ascending, dropped ones (word V) last; the places of word w are
//            [starts[w], starts[w + 1])
//   norm:    sqnorm[b] = scale^2 * sum_w || sum_{t: ids[b][t] = w} G[b][t] ||^2
//   sum:     out[w] = (scale * sum_{n of w} c[sample of n] * G[n] + (sigma C) z_w) / denom, every word of the table
//
// A per-sample gradient of the table has at most T rows that are not 0, so
// nothing of its size [B][V][d] is ever formed: in the order, the tokens of
// one (word, sample) are a run of neighbouring places, and the tokens of one
// word a run of those. The norm and the sum read G once each.
//
// The lookup is bound by HBM: 32768 tokens of 1280 bf16 take 26 us, 6.4 TB/s of
// rows read and written (rows met again come from the caches). The clipping
// pass of 32 x 1024 such tokens over 50257 words takes 122 us in its ten
// launches: the order 26 (four launches), the norm 34 (three), the factors 2,
// the sum 60 (two; 257 MB of it are the table, written at 5 TB/s). (Whole calls
// in a loop. A kernel trace, which adds about a microsecond to every launch,
// sums up to some 134.) What is not the table's is latency: chains of a place, its
// row, its run's end. Noise adds 70 us of fp32 work (as much as the noise kernel
// takes for as many elements).
//
// A run may be long (a frequent word, a batch padded with one word). Sums over
// long runs take the sums of tiles: a first launch adds up every tile of 16
// neighbouring places (and of 16 such tiles, and so on) that lies within one
// run, and what reads a run takes whole tiles from there. (The same batch with
// one word in the last quarter of every sequence: 133 us, the norm 45 of them;
// one sequence of 32768 such tokens: 186 and 100, as a wave goes to a run's end
// 64 places a step.) Sums are formed in fp32 in an order that the sizes and the
// ids alone decide; nothing is atomic but the counts of the sort, which are
// whole numbers. A place holds its word beside its token, so that finding a
// run's ends takes no second load.
//
// The sort is by digits of the word, least significant first, each digit in a
// launch of its own: a workgroup ranks the tokens of its tile by digit (within
// a wave by ballots, in order), and finds where its share of every digit goes
// from the counts that all workgroups left. Up to 4096 tokens are sorted by one
// workgroup, and others beside it count the starts. Places and starts are
// checked where they are read: whatever they hold, accesses stay inside the
// tensors.
#include "dp_cols.hpp"
#include "dp_common.hpp"
#include "dp_lm.hpp"
#include "dp_noise.hpp"
#include "dp_rows.hpp"

namespace dpk {

// ---- lookup

// One thread per 16 bytes of out, tokens side by side; four in flight per thread.
template <typename T, typename WT, bool WHOLE>
__global__ __launch_bounds__(256) void k_embedding(EmbedArgs a, int vpr, FastDiv by_vpr, int tokens) {
  constexpr int P = elem_traits<T>::per16, U = 4;
  const int d = (int)a.d;
  for (int64_t n0 = (int64_t)blockIdx.x * tokens; n0 < a.N; n0 += (int64_t)gridDim.x * tokens) {
    const int here = (int)(a.N - n0 < tokens ? a.N - n0 : tokens);
    const uint32_t work = (uint32_t)here * (uint32_t)vpr;
    for (uint32_t i0 = threadIdx.x; i0 < work; i0 += U * 256) {
      int64_t id[U], n[U];
      int c[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const uint32_t i = i0 + u * 256 < work ? i0 + u * 256 : i0;
        const uint32_t t = fast_div(i, by_vpr);
        n[u] = n0 + t;
        c[u] = (int)(i - t * (uint32_t)vpr) * P;
        id[u] = a.ids[n[u]];
      }
      float v[U][P];
#pragma unroll
      for (int u = 0; u < U; ++u) {
#pragma unroll
        for (int e = 0; e < P; ++e) v[u][e] = 0.f;
        if (id[u] < 0 || id[u] >= a.V) continue;
        const WT* w = static_cast<const WT*>(a.weight) + id[u] * a.d + c[u];
        if (WHOLE || c[u] + P <= d) {
          WT raw[P];
          __builtin_memcpy(raw, w, sizeof(raw));
#pragma unroll
          for (int e = 0; e < P; ++e) v[u][e] = to_f32(raw[e]) * a.scale;
        } else {
#pragma unroll
          for (int e = 0; e < P - 1; ++e)
            if (c[u] + e < d) v[u][e] = to_f32(w[e]) * a.scale;
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (i0 + u * 256 >= work) break;
        T* o = static_cast<T*>(a.out) + n[u] * a.d + c[u];
        if (WHOLE || c[u] + P <= d) {
          u32x4 raw;
          if constexpr (P == 8) {
#pragma unroll
            for (int e = 0; e < 4; ++e) raw[e] = pack_bf16(v[u][2 * e], v[u][2 * e + 1]);
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) raw[e] = __float_as_uint(v[u][e]);
          }
          __builtin_memcpy(o, &raw, 16);
        } else {
#pragma unroll
          for (int e = 0; e < P - 1; ++e)
            if (c[u] + e < d) put(o[e], v[u][e]);
        }
      }
    }
  }
}

// ---- order

namespace {

constexpr int kSortThreads = 1024, kSortWaves = kSortThreads / 64;
constexpr int kSortMaxDigits = 512;
constexpr int kSortSmall = 4096;  // tokens that one workgroup sorts in one launch
constexpr int kSortDirect = 64;  // workgroups whose counts each workgroup adds up by itself

// How the sort of N ids over V words goes: digits per pass, ids per workgroup.
struct SortPlan {
  int passes, bits;
  int rounds, log_tile;  // ids per thread and, as a power of two, per workgroup
  int64_t blocks;
  __host__ __device__ int digits() const { return 1 << bits; }
  __host__ __device__ int64_t tile() const { return (int64_t)1 << log_tile; }
};

SortPlan sort_plan(int64_t N, int64_t V) {
  int bits = 1;
  while (((int64_t)1 << bits) <= V) ++bits;  // keys 0 .. V (V: dropped)
  SortPlan p;
  p.passes = (bits + 8) / 9;
  p.bits = (bits + p.passes - 1) / p.passes;
  // a token a thread; more from 128 workgroups on, up to 16
  p.rounds = 1;
  p.log_tile = 10;
  while (p.rounds < 16 && (N + p.tile() - 1) / p.tile() > 128) {
    p.rounds *= 2;
    ++p.log_tile;
  }
  p.blocks = (N + p.tile() - 1) / p.tile();
  return p;
}

__device__ __forceinline__ uint32_t key_of(int64_t id, int64_t V) {
  return id < 0 || id >= V ? (uint32_t)V : (uint32_t)id;
}

__device__ __forceinline__ int64_t place_of(uint32_t word, uint32_t tok) {
  return (int64_t)(((uint64_t)word << 32) | tok);
}

// The lanes of `among` whose value's bits [0, bits) are this lane's.
__device__ __forceinline__ uint64_t same_bits(uint64_t among, uint32_t value, int bits) {
  for (int q = 0; q < bits; ++q) {
    const uint64_t has = __ballot((value >> q) & 1);
    among &= ((value >> q) & 1) ? has : ~has;
  }
  return among;
}

}  // namespace

// The first digit's counts of every workgroup's tile; clears the counts of the later passes.
__global__ __launch_bounds__(kSortThreads) void k_order_count(const int64_t* __restrict__ ids, int64_t N, int64_t V,
                                                              SortPlan p, uint32_t* __restrict__ counts) {
  __shared__ uint32_t bins[kSortMaxDigits];
  const int D = p.digits();
  const int64_t b = blockIdx.x;
  const int64_t later = (int64_t)(p.passes - 1) * p.blocks * D;
  for (int64_t i = b * kSortThreads + threadIdx.x; i < later; i += p.blocks * kSortThreads) counts[p.blocks * D + i] = 0;
  for (int k = threadIdx.x; k < D; k += kSortThreads) bins[k] = 0;
  __syncthreads();
  const int64_t i0 = b * p.tile();
  for (int r = 0; r < p.rounds; ++r) {
    const int64_t i = i0 + r * kSortThreads + threadIdx.x;
    if (i < N) atomicAdd(&bins[key_of(ids[i], V) & (D - 1)], 1u);
  }
  __syncthreads();
  for (int k = threadIdx.x; k < D; k += kSortThreads) counts[b * D + k] = bins[k];
}

// Exclusive sums down the workgroups, per digit, in place, and each digit's total behind them (many workgroups).
__global__ __launch_bounds__(64) void k_order_scan(SortPlan p, uint32_t* __restrict__ counts,
                                                   uint32_t* __restrict__ totals) {
  const int D = p.digits();
  const int k = blockIdx.x * 64 + threadIdx.x;
  if (k >= D) return;
  uint32_t sum = 0;
#pragma unroll 8
  for (int64_t b = 0; b < p.blocks; ++b) {
    const uint32_t c = counts[b * D + k];
    counts[b * D + k] = sum;
    sum += c;
  }
  totals[k] = sum;
}

// One digit's pass: the tokens of a workgroup's tile to their places by that
// digit, in order. ids_in: the first pass reads the ids themselves; else keys
// and tokens of the pass before. The next digit is counted on the way, where
// the tokens go (one add for the tokens of one word in a wave: a frequent
// word's go to one count, and adds to one address wait for each other, 10 us
// at 32768 tokens). totals: the counts are sums already (k_order_scan).
__global__ __launch_bounds__(kSortThreads) void k_order_scatter(const int64_t* __restrict__ ids_in,
                                                                const uint32_t* __restrict__ keys_in,
                                                                const uint32_t* __restrict__ toks_in, int64_t N,
                                                                int64_t V, SortPlan p, int pass,
                                                                const uint32_t* __restrict__ counts,
                                                                const uint32_t* __restrict__ totals,
                                                                uint32_t* __restrict__ next_counts,
                                                                uint32_t* __restrict__ keys_out,
                                                                uint32_t* __restrict__ toks_out,
                                                                int64_t* __restrict__ order) {
  __shared__ uint32_t seen[kSortWaves][kSortMaxDigits];  // of a wave so far; then where its tokens of a digit go
  __shared__ uint32_t base[kSortMaxDigits], all[kSortMaxDigits];
  __shared__ uint32_t scan[kSortWaves];
  const int D = p.digits(), shift = pass * p.bits;
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int64_t b = blockIdx.x;
  const int64_t w0 = b * p.tile() + (int64_t)wave * 64 * p.rounds;  // this wave's ids, `rounds` times 64 of them
  auto key_at = [&](int64_t i) { return i >= N ? 0u : ids_in ? key_of(ids_in[i], V) : keys_in[i]; };
  const uint32_t first_key = key_at(w0 + lane);  // on its way while the counts are added up
  for (int k = threadIdx.x; k < kSortWaves * D; k += kSortThreads) seen[k / D][k % D] = 0;
  for (int k = threadIdx.x; k < D; k += kSortThreads) base[k] = all[k] = 0;
  __syncthreads();
  // ---- the counts of the digit in earlier workgroups and in all, several threads to a digit
  if (totals) {
    for (int k = threadIdx.x; k < D; k += kSortThreads) {
      base[k] = counts[b * D + k];
      all[k] = totals[k];
    }
  } else {
    const int parts = kSortThreads / D, k = threadIdx.x & (D - 1), part = threadIdx.x / D;
    uint32_t before = 0, total = 0;
#pragma unroll 8
    for (int64_t j = part; j < p.blocks; j += parts) {
      const uint32_t c = counts[j * D + k];
      total += c;
      before += j < b ? c : 0u;
    }
    if (total) atomicAdd(&all[k], total);
    if (before) atomicAdd(&base[k], before);
  }
  __syncthreads();
  // ---- exclusive sum over the digits
  uint32_t mine = (int)threadIdx.x < D ? all[threadIdx.x] : 0, run = mine;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const uint32_t o = __shfl_up(run, off, kWave);
    if (lane >= off) run += o;
  }
  if (lane == 63) scan[wave] = run;
  // ---- ranks within the wave, in order: the lanes before this one with its digit, and those of earlier rounds
  const uint64_t below = lane == 0 ? 0 : (~0ull >> (64 - lane));
  for (int r = 0; r < p.rounds; ++r) {
    const int64_t i = w0 + r * 64 + lane;
    const uint32_t digit = ((r == 0 ? first_key : key_at(i)) >> shift) & (D - 1);
    const uint64_t same = same_bits(__ballot(i < N), digit, p.bits);
    if (i < N && (same & below) == 0) seen[wave][digit] += (uint32_t)__popcll(same);
  }
  __syncthreads();
  // ---- where each wave's tokens of a digit start
  if ((int)threadIdx.x < D) {
    uint32_t s = base[threadIdx.x] + run - mine;
    for (int w = 0; w < wave; ++w) s += scan[w];
#pragma unroll
    for (int w = 0; w < kSortWaves; ++w) {
      const uint32_t c = seen[w][threadIdx.x];
      seen[w][threadIdx.x] = s;
      s += c;
    }
  }
  __syncthreads();
  for (int r = 0; r < p.rounds; ++r) {
    const int64_t i = w0 + r * 64 + lane;
    const bool in = i < N;
    const uint32_t key = r == 0 ? first_key : key_at(i), tok = in && toks_in ? toks_in[i] : (uint32_t)i;
    const uint32_t digit = (key >> shift) & (D - 1);
    const uint64_t same = same_bits(__ballot(in), digit, p.bits);
    uint32_t to = 0;
    if (in) to = seen[wave][digit] + (uint32_t)__popcll(same & below);
    __builtin_amdgcn_wave_barrier();  // every lane has read its digit's place before one moves it on
    if (in && (same & below) == 0) seen[wave][digit] = to + (uint32_t)__popcll(same);
    __builtin_amdgcn_wave_barrier();
    if (in) {
      keys_out[to] = key;
      if (order) order[to] = place_of(key, tok);
      else toks_out[to] = tok;
    }
    if (next_counts) {
      const uint32_t next = (key >> (shift + p.bits)) & (D - 1);
      // neighbours by this digit share their tile but where one ends
      const uint32_t tile = to >> p.log_tile;
      uint64_t twins = same_bits(same, next, p.bits);
      const uint32_t first_tile = __shfl(tile, in ? __builtin_ctzll(twins) : lane, kWave);
      twins &= __ballot(tile == first_tile);
      if (in && (tile != first_tile || (twins & below) == 0))
        atomicAdd(&next_counts[(int64_t)tile * D + next], tile != first_tile ? 1u : (uint32_t)__popcll(twins));
    }
  }
}

namespace {

struct StartsLds {
  uint32_t count[kSortThreads], waves[kSortWaves], less[kSortWaves];
};

// The starts of the 1024 words from w0 on, by a workgroup of 1024 threads: how many ids are smaller than w0, and how many
// are each of the words. All ids are read.
__device__ __forceinline__ void starts_of_ids(const int64_t* __restrict__ ids, int N, int64_t V, int64_t w0,
                                              int64_t* __restrict__ starts, StartsLds& l) {
  constexpr int U = 4;
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  l.count[threadIdx.x] = 0;
  __syncthreads();
  uint32_t less = 0;
  for (int i0 = threadIdx.x; i0 < N; i0 += U * kSortThreads) {
    uint32_t key[U];
#pragma unroll
    for (int u = 0; u < U; ++u) key[u] = i0 + u * kSortThreads < N ? key_of(ids[i0 + u * kSortThreads], V) : ~0u;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      less += key[u] < (uint32_t)w0;
      const uint32_t at = key[u] - (uint32_t)w0;  // past the 1024 for a smaller key too
      if (at < (uint32_t)kSortThreads) {
        // one add for the lanes with the first one's word: a frequent one's would wait for each other
        const uint32_t first = (uint32_t)__builtin_amdgcn_readfirstlane((int)at);
        const uint64_t same = __ballot(at == first);
        if (at != first) atomicAdd(&l.count[at], 1u);
        else if (lane == __builtin_ctzll(same)) atomicAdd(&l.count[at], (uint32_t)__popcll(same));
      }
    }
  }
  __syncthreads();
  const uint32_t mine = l.count[threadIdx.x];
  uint32_t run = mine;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const uint32_t o = __shfl_up(run, off, kWave);
    if (lane >= off) run += o;
  }
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) less += __shfl_xor(less, off, kWave);
  if (lane == 63) {
    l.waves[wave] = run;
    l.less[wave] = less;
  }
  __syncthreads();
  uint32_t s = run - mine;
#pragma unroll
  for (int w = 0; w < kSortWaves; ++w) s += l.less[w] + (w < wave ? l.waves[w] : 0u);
  if (w0 + threadIdx.x <= V) starts[w0 + threadIdx.x] = s;
}

}  // namespace

// All digits of up to 4096 tokens by one workgroup, the tokens in LDS between the passes; workgroups behind it: the
// starts (or, without, the keys in order are left for them in keys_out, null otherwise).
__global__ __launch_bounds__(kSortThreads) void k_order_small(const int64_t* __restrict__ ids, int N, int64_t V,
                                                              SortPlan p, uint32_t* __restrict__ keys_out,
                                                              int64_t* __restrict__ order,
                                                              int64_t* __restrict__ starts) {
  __shared__ StartsLds lds;
  if (blockIdx.x > 0) {
    starts_of_ids(ids, N, V, (int64_t)(blockIdx.x - 1) * kSortThreads, starts, lds);
    return;
  }
  __shared__ uint32_t keys[2][kSortSmall];
  __shared__ uint16_t toks[2][kSortSmall];
  __shared__ uint32_t seen[kSortWaves][kSortMaxDigits];
  __shared__ uint32_t scan[kSortWaves];
  const int D = p.digits();
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int rounds = (N + kSortThreads - 1) / kSortThreads, w0 = wave * 64 * rounds;
  const uint64_t below = lane == 0 ? 0 : (~0ull >> (64 - lane));
  for (int i = threadIdx.x; i < N; i += kSortThreads) {
    keys[0][i] = key_of(ids[i], V);
    toks[0][i] = (uint16_t)i;
  }
  for (int pass = 0; pass < p.passes; ++pass) {
    const uint32_t* key = keys[pass & 1];
    const uint16_t* tok = toks[pass & 1];
    const int shift = pass * p.bits;
    for (int k = threadIdx.x; k < kSortWaves * D; k += kSortThreads) seen[k / D][k % D] = 0;
    __syncthreads();
    for (int r = 0; r < rounds; ++r) {
      const int i = w0 + r * 64 + lane;
      const uint32_t digit = ((i < N ? key[i] : 0u) >> shift) & (D - 1);
      const uint64_t same = same_bits(__ballot(i < N), digit, p.bits);
      if (i < N && (same & below) == 0) seen[wave][digit] += (uint32_t)__popcll(same);
    }
    __syncthreads();
    uint32_t mine = 0;
    if ((int)threadIdx.x < D) {
#pragma unroll
      for (int w = 0; w < kSortWaves; ++w) mine += seen[w][threadIdx.x];
    }
    uint32_t run = mine;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
      const uint32_t o = __shfl_up(run, off, kWave);
      if (lane >= off) run += o;
    }
    if (lane == 63) scan[wave] = run;
    __syncthreads();
    if ((int)threadIdx.x < D) {
      uint32_t s = run - mine;
      for (int w = 0; w < wave; ++w) s += scan[w];
#pragma unroll
      for (int w = 0; w < kSortWaves; ++w) {
        const uint32_t c = seen[w][threadIdx.x];
        seen[w][threadIdx.x] = s;
        s += c;
      }
    }
    __syncthreads();
    const bool last = pass + 1 == p.passes;
    for (int r = 0; r < rounds; ++r) {
      const int i = w0 + r * 64 + lane;
      const bool in = i < N;
      const uint32_t k = in ? key[i] : 0u, digit = (k >> shift) & (D - 1);
      const uint64_t same = same_bits(__ballot(in), digit, p.bits);
      uint32_t to = 0;
      if (in) to = seen[wave][digit] + (uint32_t)__popcll(same & below);
      __builtin_amdgcn_wave_barrier();  // every lane has read its digit's place before one moves it on
      if (in && (same & below) == 0) seen[wave][digit] = to + (uint32_t)__popcll(same);
      __builtin_amdgcn_wave_barrier();
      if (in) {
        if (last) {
          if (keys_out) keys_out[to] = k;
          order[to] = place_of(k, tok[i]);
        } else {
          keys[(pass + 1) & 1][to] = k;
          toks[(pass + 1) & 1][to] = tok[i];
        }
      }
    }
    __syncthreads();
  }
}

// starts[w] = how many keys are smaller than w. A workgroup's 256 words lie
// close together in the keys: each of its waves finds where the first one's
// and the last one's are, 64 keys a step, and a word is then looked up in the
// few between them, held in LDS where they fit.
__global__ __launch_bounds__(256) void k_order_starts(const uint32_t* __restrict__ keys, int64_t N, int64_t V,
                                                      int64_t* __restrict__ starts) {
  constexpr int kHeld = 2048;
  __shared__ uint32_t held[kHeld];
  const int lane = threadIdx.x & 63;
  for (int64_t w0 = (int64_t)blockIdx.x * 256; w0 <= V; w0 += (int64_t)gridDim.x * 256) {
    const int64_t last = w0 + 255 < V ? w0 + 255 : V;
    // [s[q], e[q]]: where the first place with a key of w0 (q = 0) or `last` (q = 1) or more lies
    int64_t s[2] = {0, 0}, e[2] = {N, N};
    while (s[0] < e[0] || s[1] < e[1]) {
      int64_t step[2], at[2];
      uint32_t key[2];
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        step[q] = (e[q] - s[q] + 63) / 64;
        at[q] = s[q] + (lane + 1) * step[q] - 1;
        key[q] = at[q] < e[q] ? keys[at[q]] : ~0u;
      }
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const uint64_t less = __ballot(at[q] < e[q] && key[q] < (uint32_t)(q ? last : w0));
        s[q] += __popcll(less) * step[q];  // the pivots ascend: the first so many are smaller
        if (step[q]) e[q] = s[q] + step[q] - 1 < e[q] ? s[q] + step[q] - 1 : e[q];
      }
    }
    const int64_t lo = s[0], hi = s[1];
    const bool fits = hi - lo <= kHeld;
    __syncthreads();
    if (fits)
      for (int64_t i = threadIdx.x; i < hi - lo; i += 256) held[i] = keys[lo + i];
    __syncthreads();
    const int64_t w = w0 + threadIdx.x;
    if (w > last) continue;
    int64_t from = lo, to = hi;
    while (from < to) {
      const int64_t mid = (from + to) >> 1;
      if ((fits ? held[mid - lo] : keys[mid]) < (uint32_t)w) from = mid + 1;
      else to = mid;
    }
    starts[w] = from;
  }
}

// ---- sums over runs of places

namespace {

constexpr int kTile = kEmbedTile;

// This wave's number in its workgroup, in a scalar register: what follows from it is the wave's, not a lane's.
__device__ __forceinline__ int wave_id() { return __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6)); }

__device__ __forceinline__ uint32_t sample_of(const EmbedGradArgs& a, int tok) { return fast_div((uint32_t)tok, a.by_t); }

// A place's token, -1 if it holds none, and what its run shares: the word, and for the norm the sample too; -1 for a
// dropped token.
struct Place {
  int tok;
  int64_t run;
};
template <bool NORM>
__device__ __forceinline__ Place place_at(const EmbedGradArgs& a, int64_t i) {
  const int64_t o = a.order[i], word = o >> 32, tok = o & 0xFFFFFFFF;
  Place p{-1, -1};
  if (tok < a.N) {
    p.tok = (int)tok;
    if (word >= 0 && word < a.V) p.run = NORM ? word * a.B + sample_of(a, p.tok) : word;
  }
  return p;
}

__device__ __forceinline__ int lane_int(int v, int lane) { return __builtin_amdgcn_readlane(v, lane); }
__device__ __forceinline__ float lane_float(float v, int lane) {
  return __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(v), lane));
}

__device__ __forceinline__ int64_t lane_int64(int64_t v, int lane) {
  return (int64_t)(((uint64_t)(uint32_t)lane_int((int)(v >> 32), lane) << 32) | (uint32_t)lane_int((int)v, lane));
}

// Place i if it lies below e: its token (-1 for none), its sample's factor (1 in the norm) and its run.
struct Places {
  int tok;
  float f;
  int64_t run;
};
template <bool NORM>
__device__ __forceinline__ Places places_at(const EmbedGradArgs& a, int64_t i, int64_t e) {
  Places p{-1, 0.f, -1};
  if (i < e) {
    const Place q = place_at<NORM>(a, i);
    p.tok = q.tok;
    p.run = q.run;
    if (p.tok >= 0) p.f = NORM ? 1.0f : a.c[sample_of(a, p.tok)];
  }
  return p;
}

// acc += the rows of lanes [r0, r0 + U) of p; lanes past the last place hold none.
template <int U, typename C>
__device__ __forceinline__ void add_places(const EmbedGradArgs& a, const C& cols, float* acc, const Places& p, int r0) {
  typename C::Raw raw[U];
#pragma unroll
  for (int u = 0; u < U; ++u) raw[u] = cols.fetch(a.G, lane_int(p.tok, r0 + u));
#pragma unroll
  for (int u = 0; u < U; ++u) C::add(acc, raw[u], lane_float(p.f, r0 + u));
}

// Rows in flight of a long run. The norm has eight rows of its own in flight already: with 16 it takes 36 us for 32768
// tokens of Zipf's law, 34 with 8.
template <bool NORM>
constexpr int kAhead = NORM ? 8 : 16;

// acc += the rows of places [s, e) (the sum: times their samples' factors), by a wave. Places of one run.
template <bool NORM, typename C>
__device__ __forceinline__ void add_rows(const EmbedGradArgs& a, const C& cols, float* acc, int64_t s, int64_t e) {
  for (; s < e; s += 64) {
    const Places p = places_at<NORM>(a, s + (threadIdx.x & 63), e);
    const int m = (int)(e - s < 64 ? e - s : 64);
#pragma unroll 1
    for (int r = 0; r < m; r += kAhead<NORM>) add_places<kAhead<NORM>>(a, cols, acc, p, r);
  }
}

// acc += rows [lo, hi) of sums, eight in flight.
template <typename C>
__device__ __forceinline__ void add_sums(const C& cols, float* acc, const float* sums, int64_t lo, int64_t hi) {
  constexpr int U = 8, N = C::columns;
#pragma unroll 1
  for (int64_t i = lo; i < hi; i += U) {
    float v[U][N];
#pragma unroll
    for (int u = 0; u < U; ++u) cols.fetch_sums(sums, i + u < hi ? i + u : -1, v[u]);
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int e = 0; e < N; ++e) acc[e] += v[u][e];
  }
}

// The same with whole tiles taken from their sums: the ends by places (both
// together, in the lanes of one load), then by tiles of 16, of 256 and so on, up
// to the highest level there is.
template <bool NORM, typename C>
__device__ __forceinline__ void add_run(const EmbedGradArgs& a, const C& cols, float* acc, int64_t s, int64_t e) {
  const int64_t up = (s + kTile - 1) / kTile * kTile, down = e / kTile * kTile;
  if (a.levels == 0 || up >= down) {
    add_rows<NORM>(a, cols, acc, s, e);
    return;
  }
  const int lane = threadIdx.x & 63;
  const Places p = places_at<NORM>(a, lane < kTile ? s + lane : down + lane - kTile,
                                   lane < kTile ? up : lane < 2 * kTile ? e : 0);
#pragma unroll 1
  for (int r = 0; r < 2 * kTile; r += kAhead<NORM>) add_places<kAhead<NORM>>(a, cols, acc, p, r);
  int64_t lo = up / kTile, hi = down / kTile;
  for (int l = 0; lo < hi; ++l) {
    const float* sums = a.sums + a.level_at[l] * a.d;
    // the tiles of the next level inside [lo, hi): [in_lo, in_hi) of this one
    int64_t in_lo = (lo + kTile - 1) / kTile * kTile, in_hi = hi / kTile * kTile;
    if (l + 1 == a.levels || in_lo >= in_hi) in_lo = in_hi = hi;
    add_sums(cols, acc, sums, lo, in_lo);
    add_sums(cols, acc, sums, in_hi, hi);
    if (in_lo >= in_hi) break;
    lo = in_lo / kTile;
    hi = in_hi / kTile;
  }
}

}  // namespace

// Sums of the tiles of level l (of `span` = 16^(l+1) places) that lie within
// one run and, where `both`, of those of level l + 1 above them: a workgroup
// for 16 tiles and 64 x 16 bytes' worth of columns, a wave for each tile.
template <typename T, bool TINY, bool NORM>
__global__ __launch_bounds__(1024) void k_embed_tiles(EmbedGradArgs a, int l, int64_t span, int64_t tiles, int col_waves,
                                                      int both) {
  constexpr int P = elem_traits<T>::per16;
  using C = Cols<T, P, TINY>;
  __shared__ float part[kTile][64 * P];
  __shared__ int64_t ends[2];  // the runs of the first and the last place of the 16 tiles
  const int wave = wave_id(), lane = threadIdx.x & 63;
  const int64_t items = (tiles + kTile - 1) / kTile * col_waves;
  for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
    const int64_t group = item / col_waves, tile = group * kTile + wave;
    const C cols(((int)(item - group * col_waves) * 64 + lane) * P, a.d);
    int64_t first = -1, last = -2;
    Places p{-1, 0.f, -1};
    if (tile < tiles) {
      const int64_t i0 = tile * span;
      int64_t r = -1;
      if (l == 0) {  // every place: its row is read if they are one run
        p = places_at<NORM>(a, i0 + lane, i0 + kTile);
        r = p.run;
        last = lane_int64(r, kTile - 1);
      } else {
        if (lane < 2) r = place_at<NORM>(a, lane == 0 ? i0 : i0 + span - 1).run;
        last = lane_int64(r, 1);
      }
      first = lane_int64(r, 0);
    }
    if (lane == 0 && wave == 0) ends[0] = first;
    if (lane == 0 && wave == kTile - 1) ends[1] = last;
    float acc[P];
#pragma unroll
    for (int e = 0; e < P; ++e) acc[e] = 0.f;
    if (first >= 0 && first == last) {
      if (l == 0) {
        add_places<kTile>(a, cols, acc, p, 0);
      } else {
        add_sums(cols, acc, a.sums + a.level_at[l - 1] * a.d, tile * kTile, tile * kTile + kTile);
      }
      cols.put_sums(a.sums + (a.level_at[l] + tile) * a.d, acc);
    }
    if (!both) continue;
    __syncthreads();
    const bool whole = ends[0] >= 0 && ends[0] == ends[1];
    if (whole) {  // the same in every wave
#pragma unroll
      for (int e = 0; e < P; ++e) part[wave][e * 64 + lane] = acc[e];
    }
    __syncthreads();
    if (whole && wave == 0) {
#pragma unroll
      for (int e = 0; e < P; ++e) acc[e] = 0.f;
#pragma unroll 4
      for (int w = 0; w < kTile; ++w)
#pragma unroll
        for (int e = 0; e < P; ++e) acc[e] += part[w][e * 64 + lane];
      cols.put_sums(a.sums + (a.level_at[l + 1] + group) * a.d, acc);
    }
    __syncthreads();  // part and ends are written again
  }
}

// Squared norms of the runs that start in a wave's 8 places, over its part of
// the columns, each written at the token of the run's last of these places, 0
// at the other tokens. The rows of all 8 places are read together; what
// follows of the last run behind them is added from its tiles. All that a
// wave decides by is in scalar registers: with branches by lanes the compiler
// waits for each row before the next (36 us for 32 x 1024 tokens of 1280 bf16,
// 24 so: 84 MB at 3.5 TB/s).
template <typename T, bool TINY>
__global__ __launch_bounds__(256, 4) void k_embed_norm(EmbedGradArgs a, int col_groups) {
  constexpr int R = kEmbedNormPlaces, P = elem_traits<T>::per16;
  using C = Cols<T, P, TINY>;
  const int lane = threadIdx.x & 63;
  const int64_t items = (a.N + R - 1) / R * col_groups;
  for (int64_t item = (int64_t)blockIdx.x * 4 + wave_id(); item < items; item += (int64_t)gridDim.x * 4) {
    const int64_t w = item / col_groups;
    const int cg = (int)(item - w * col_groups);
    const int64_t i0 = w * R;
    const int m = (int)(a.N - i0 < R ? a.N - i0 : R);  // this wave's places
    // lane k + 1 holds place i0 + k; lane 0 the one before, further lanes those behind
    const int64_t i = i0 - 1 + lane;
    Place here{-1, -1};
    if (i >= 0 && i < a.N) here = place_at<true>(a, i);
    const int n = here.tok;
    const int64_t run = here.run;
    const int64_t prev = __shfl_up(run, 1, kWave);
    const uint64_t heads = __ballot(lane > 0 && run >= 0 && run != prev);
    const uint64_t goes_on = __ballot(lane > 0 && run >= 0 && run == prev);  // same run as the place before
    // the places of runs that start here, and the last place of each of them
    uint32_t mine = 0, lasts = 0;
#pragma unroll
    for (int k = 0; k < R; ++k) {
      const bool on = k > 0 && ((goes_on >> (k + 1)) & 1) && ((mine >> (k - 1)) & 1);
      const bool in = k < m && (((heads >> (k + 1)) & 1) || on);
      mine |= (uint32_t)in << k;
      const bool more = k + 1 < R && k + 1 < m && ((goes_on >> (k + 2)) & 1);
      lasts |= (uint32_t)(in && !more) << k;
    }
    // the last run's places behind these
    int64_t end = i0 + m;
    if (((mine >> (m - 1)) & 1) && ((goes_on >> (m + 1)) & 1)) {
      const uint64_t rest = ~(goes_on >> (m + 1));
      end += __builtin_ctzll(rest);  // bits past the lanes are ones: at most to lane 63
      if (end == i0 + 63) {          // on past the last lane
        const int64_t same = lane_int64(run, m);
        while (end < a.N) {
          const int64_t j = end + lane;
          const uint64_t stops = __ballot(j >= a.N || place_at<true>(a, j < a.N ? j : a.N - 1).run != same);
          if (stops) {
            end += __builtin_ctzll(stops);
            break;
          }
          end += 64;
        }
      }
    }
    const bool tail = end > i0 + m;
    if (tail) lasts &= ~(1u << (m - 1));  // that run ends behind these places
    float sq[R], sq_tail = 0.f;
#pragma unroll
    for (int k = 0; k < R; ++k) sq[k] = 0.f;
    if (mine) {
      for (int c0 = cg * 64 * P; c0 < (int)a.d; c0 += col_groups * 64 * P) {
        const C cols(c0 + lane * P, a.d);
        typename C::Raw raw[R];
#pragma unroll
        for (int k = 0; k < R; ++k) raw[k] = cols.fetch(a.G, (mine >> k) & 1 ? lane_int(n, k + 1) : -1);
        float acc[P];
#pragma unroll
        for (int e = 0; e < P; ++e) acc[e] = 0.f;
#pragma unroll
        for (int k = 0; k < R; ++k) {
          C::add(acc, raw[k], 1.0f);
          if ((lasts >> k) & 1) {
#pragma unroll
            for (int e = 0; e < P; ++e) {
              const float v = e < cols.skip ? 0.f : acc[e];
              sq[k] = __builtin_fmaf(v, v, sq[k]);
              acc[e] = 0.f;
            }
          }
        }
        if (tail) {
          add_run<true>(a, cols, acc, i0 + m, end);
#pragma unroll
          for (int e = 0; e < P; ++e) {
            const float v = e < cols.skip ? 0.f : acc[e];
            sq_tail = __builtin_fmaf(v, v, sq_tail);
          }
        }
      }
    }
    sq_tail = wave_sum(sq_tail);
    float out = 0.f;
#pragma unroll
    for (int k = 0; k < R; ++k) {
      const float s = (lasts >> k) & 1 ? wave_sum(sq[k]) : 0.f;
      if (lane == k + 1) out = s;
    }
    if (tail && lane == m) out = sq_tail;
    if (lane >= 1 && lane <= m && n >= 0) a.token_sq[cg * a.N + n] = out;
  }
}

// sqnorm[b] (+)= scale^2 * the sum of its tokens' values.
__global__ __launch_bounds__(256) void k_embed_norm_finish(EmbedGradArgs a, int col_groups) {
  __shared__ float red[4];
  for (int64_t b = blockIdx.x; b < a.B; b += gridDim.x) {
    float s = 0.f;
    for (int g = 0; g < col_groups; ++g)
#pragma unroll 4
      for (int64_t t = threadIdx.x; t < a.T; t += 256) s += a.token_sq[g * a.N + b * a.T + t];
    s = block_sum<256>(s, red);
    if (threadIdx.x == 0) {
      s = s * a.scale * a.scale;  // one by one: the scale's square may be out of range where the norm is not
      a.sqnorm[b] = a.accumulate ? a.sqnorm[b] + s : s;
    }
    __syncthreads();
  }
}

// The clipped, noised mean of 4 neighbouring words (whose noise shares its
// blocks) and 256 columns, by a wave: four columns a lane, so that 16 sums
// leave room for 16 rows in flight beside 16 to 20 waves a CU (with eight
// columns 152 registers, and 85 us instead of 62 for 32768 tokens of 1280 bf16
// before further steps). Past the caches where it can: the table is larger than
// they are (72 us through them, 55 so). Rows in flight: four up to eight places,
// else sixteen (55 us by four alone, 50 so).
template <typename T, bool TINY>
__global__ __launch_bounds__(256, sizeof(T) == 2 ? 5 : 4) void k_embed_sum(EmbedGradArgs a, NoiseArgs na,
                                                                           float* __restrict__ out, int col_waves) {
  constexpr int P = 4;
  using C = Cols<T, P, TINY>;
  const int lane = threadIdx.x & 63;
  const bool stream = !TINY && a.d % 4 == 0 && (reinterpret_cast<uintptr_t>(out) & 15) == 0;
  const int64_t groups = (a.V + 3) / 4, items = groups * col_waves;
  for (int64_t item = (int64_t)blockIdx.x * 4 + wave_id(); item < items; item += (int64_t)gridDim.x * 4) {
    const int64_t g = item / col_waves;
    const C cols(((int)(item - g * col_waves) * 64 + lane) * P, a.d);
    int64_t st = 0;
    if (lane < 5) {  // words past the table have no places
      st = a.starts[4 * g + lane <= a.V ? 4 * g + lane : a.V];
      st = st < 0 ? 0 : st > a.N ? a.N : st;
    }
    float acc[4][P];
#pragma unroll
    for (int k = 0; k < 4; ++k)
#pragma unroll
      for (int e = 0; e < P; ++e) acc[k][e] = 0.f;
    int64_t at[5];  // where the words' places start
#pragma unroll
    for (int k = 0; k < 5; ++k) at[k] = lane_int64(st, k);
    bool few = at[0] <= at[1] && at[1] <= at[2] && at[2] <= at[3] && at[3] <= at[4] && at[4] - at[0] <= 64;
    if (few) {  // the rows of all four words, read together
      const int m = (int)(at[4] - at[0]);
      Places p{-1, 0.f, -1};
      if (m > 0) p = places_at<false>(a, at[0] + lane, at[4]);
      const int e1 = (int)(at[1] - at[0]), e2 = (int)(at[2] - at[0]), e3 = (int)(at[3] - at[0]);
      auto add = [&](auto ahead) {
        constexpr int U = decltype(ahead)::value;
#pragma unroll 1
        for (int r = 0; r < m; r += U) {  // lanes past m hold no place
          typename C::Raw raw[U];
#pragma unroll
          for (int u = 0; u < U; ++u) raw[u] = cols.fetch(a.G, lane_int(p.tok, r + u));
#pragma unroll
          for (int u = 0; u < U; ++u) {
            const float f = lane_float(p.f, r + u);
            if (r + u < e1) C::add(acc[0], raw[u], f);
            else if (r + u < e2) C::add(acc[1], raw[u], f);
            else if (r + u < e3) C::add(acc[2], raw[u], f);
            else C::add(acc[3], raw[u], f);
          }
        }
      };
      if (m <= 8) add(std::integral_constant<int, 4>{});
      else add(std::integral_constant<int, 16>{});
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (4 * g + k < a.V && at[k] < at[k + 1]) add_run<false>(a, cols, acc[k], at[k], at[k + 1]);
    }
#pragma unroll
    for (int k = 0; k < 4; ++k)
#pragma unroll
      for (int e = 0; e < P; ++e) acc[k][e] *= a.scale;
    if (na.sc != 0.0f) {
#pragma unroll
      for (int e = 0; e < P; ++e) {
        const f32x4 z = normals4((uint32_t)g * (uint32_t)a.d + (uint32_t)(cols.at + e), 2 * na.layer, na.step, 0, na.k0, na.k1);
#pragma unroll
        for (int k = 0; k < 4; ++k) acc[k][e] = noised_mean_spec(acc[k][e], na.sc, z[k], na.inv_denom);
      }
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k)
#pragma unroll
        for (int e = 0; e < P; ++e) acc[k][e] *= na.inv_denom;
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (4 * g + k >= a.V) break;
      if (stream) cols.stream_sums(out + (4 * g + k) * a.d, acc[k]);
      else cols.put_sums(out + (4 * g + k) * a.d, acc[k]);
    }
  }
}

namespace {

constexpr int64_t kEmbedBlocks = 1 << 20;
unsigned grid_of(int64_t blocks) { return (unsigned)std::max<int64_t>(1, std::min(blocks, kEmbedBlocks)); }

template <typename T>
int col_waves_of(int64_t d) {
  constexpr int per = 64 * elem_traits<T>::per16;
  return (int)((d + per - 1) / per);
}

// The tiles' sums, level by level.
template <typename T, bool TINY, bool NORM>
hipError_t launch_tiles(hipStream_t st, const EmbedGradArgs& a) {
  const int cw = col_waves_of<T>(a.d);
  int64_t span = kTile;
  for (int l = 0; l < a.levels; l += 2, span *= kTile * kTile) {
    const int64_t tiles = a.N / span;
    k_embed_tiles<T, TINY, NORM><<<grid_of((tiles + kTile - 1) / kTile * cw), 1024, 0, st>>>(a, l, span, tiles, cw,
                                                                                              l + 1 < a.levels);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

// Parts of the columns that waves of k_embed_norm share out: as many as give about 8192 waves (the norm of 32768 tokens of
// 1600 bf16 36 us, 42 by one wave for all columns; of 2048 tokens of 1280 16 and 23).
int64_t norm_col_groups(int64_t N, int col_waves) {
  const int64_t waves = (N + kEmbedNormPlaces - 1) / kEmbedNormPlaces;
  return std::max<int64_t>(1, std::min<int64_t>(col_waves, 8192 / waves));
}

template <typename T, bool TINY>
hipError_t launch_norm(hipStream_t st, const EmbedGradArgs& a) {
  hipError_t e = launch_tiles<T, TINY, true>(st, a);
  if (e != hipSuccess) return e;
  const int64_t groups = norm_col_groups(a.N, col_waves_of<T>(a.d));
  const int64_t waves = (a.N + kEmbedNormPlaces - 1) / kEmbedNormPlaces * groups;
  k_embed_norm<T, TINY><<<grid_of((waves + 3) / 4), 256, 0, st>>>(a, (int)groups);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  k_embed_norm_finish<<<grid_of(a.B), 256, 0, st>>>(a, (int)groups);
  return hipGetLastError();
}

template <typename T, bool TINY>
hipError_t launch_sum(hipStream_t st, const EmbedGradArgs& a, const NoiseArgs& na, float* out) {
  const hipError_t e = launch_tiles<T, TINY, false>(st, a);
  if (e != hipSuccess) return e;
  const int cw = (int)((a.d + 255) / 256);
  const unsigned grid = grid_of(((a.V + 3) / 4 * cw + 3) / 4);
  if (TINY && a.d < 4) k_embed_sum<T, true><<<grid, 256, 0, st>>>(a, na, out, cw);  // four columns a lane
  else k_embed_sum<T, false><<<grid, 256, 0, st>>>(a, na, out, cw);
  return hipGetLastError();
}

// Levels of tiles for runs of up to `longest` places: none up to 64, else as many as leave a run at most 128
// tiles of the highest.
int levels_for(int64_t N, int64_t longest) {
  int levels = 0;
  int64_t n = N;
  while (levels < kEmbedMaxLevels && longest > (levels ? 128 : 64) && n >= kTile) {
    ++levels;
    longest /= kTile;
    n /= kTile;
  }
  return levels;
}

void set_levels(EmbedGradArgs& a, int64_t longest) {
  a.levels = levels_for(a.N, longest);
  int64_t rows = 0, n = a.N;
  for (int l = 0; l < a.levels; ++l) {
    n /= kTile;
    a.level_at[l] = rows;
    rows += n;
  }
}

int64_t level_rows(int64_t N, int levels) {
  int64_t rows = 0;
  for (int l = 0; l < levels; ++l) {
    N /= kTile;
    rows += N;
  }
  return rows;
}

// Floats of the tokens' squared norms, a list for each part of the columns.
int64_t token_floats(int dtype, int64_t N, int64_t d) {
  const int cw = dtype == 1 ? col_waves_of<bf16s>(d) : col_waves_of<float>(d);
  return (N * norm_col_groups(N, cw) + 63) / 64 * 64;
}

}  // namespace

hipError_t launch_embedding(hipStream_t st, int dtype, int weight_dtype, const EmbedArgs& a) {
  const int P = dtype == 1 ? 8 : 4;
  const int vpr = (int)((a.d + P - 1) / P);
  const int tokens = std::max(1, 1024 / vpr);  // four vectors a thread, or one token
  const FastDiv by = make_fastdiv((uint32_t)vpr);
  const bool whole = a.d % P == 0;
  auto run = [&](auto t, auto w, auto wh) {
    k_embedding<decltype(t), decltype(w), decltype(wh)::value>
        <<<grid_of((a.N + tokens - 1) / tokens), 256, 0, st>>>(a, vpr, by, tokens);
    return hipGetLastError();
  };
  auto pick = [&](auto t, auto w) { return whole ? run(t, w, std::true_type{}) : run(t, w, std::false_type{}); };
  if (dtype == 1) return weight_dtype == 1 ? pick(bf16s{}, bf16s{}) : pick(bf16s{}, float{});
  return weight_dtype == 1 ? pick(float{}, bf16s{}) : pick(float{}, float{});
}

// Workspace: the counts of every pass, the digits' totals, two lists of keys and of tokens.
size_t embed_order_ws_bytes(int64_t N, int64_t V) {
  const SortPlan p = sort_plan(N, V);
  const int64_t words = (p.passes * p.blocks + 1) * p.digits() + 4 * ((N + 3) / 4 * 4);
  return ((size_t)words * 4 + 255) / 256 * 256;
}

hipError_t launch_embed_order(hipStream_t st, const int64_t* ids, int64_t N, int64_t V, void* ws, int64_t* order,
                              int64_t* starts) {
  const SortPlan p = sort_plan(N, V);
  const int64_t D = p.digits(), list = (N + 3) / 4 * 4;
  uint32_t* counts = static_cast<uint32_t*>(ws);
  uint32_t* totals = counts + p.passes * p.blocks * D;
  uint32_t* lists = totals + D;  // keys, tokens, keys, tokens
  const bool summed = p.blocks > kSortDirect;
  auto find_starts = [&](const uint32_t* keys) {
    k_order_starts<<<grid_of((V + 256) / 256), 256, 0, st>>>(keys, N, V, starts);
    return hipGetLastError();
  };
  if (N <= kSortSmall) {
    // The starts from the ids beside the sort: every workgroup of 1024 words reads all ids, worth it for few of both
    // (1001 tokens, 5003 words: 7.1 us, 10.7 in two launches; 32768 tokens beside the first of theirs: 30 and 26).
    const bool beside = V < (1 << 19);
    const unsigned more = beside ? (unsigned)((V + kSortThreads) / kSortThreads) : 0;
    k_order_small<<<1 + more, kSortThreads, 0, st>>>(ids, (int)N, V, p, beside ? nullptr : lists, order, starts);
    const hipError_t e = hipGetLastError();
    return e == hipSuccess && !beside ? find_starts(lists) : e;
  }
  k_order_count<<<(unsigned)p.blocks, kSortThreads, 0, st>>>(ids, N, V, p, counts);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  for (int pass = 0; pass < p.passes; ++pass) {
    uint32_t* c = counts + pass * p.blocks * D;
    if (summed) {
      k_order_scan<<<(unsigned)((D + 63) / 64), 64, 0, st>>>(p, c, totals);
      e = hipGetLastError();
      if (e != hipSuccess) return e;
    }
    uint32_t* in = lists + ((pass + 1) & 1) * 2 * list;
    uint32_t* out = lists + (pass & 1) * 2 * list;
    const bool last = pass + 1 == p.passes;
    k_order_scatter<<<(unsigned)p.blocks, kSortThreads, 0, st>>>(
        pass == 0 ? ids : nullptr, pass == 0 ? nullptr : in, pass == 0 ? nullptr : in + list, N, V, p, pass, c,
        summed ? totals : nullptr, last ? nullptr : c + p.blocks * D, out, out + list, last ? order : nullptr);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
    if (last) e = find_starts(out);
  }
  return e;
}

// The tokens' squared norms, then the tiles' sums; the norm's runs are within a sample, the sum's are not.
size_t embed_ws_bytes(int dtype, int64_t B, int64_t T, int64_t d) {
  const int64_t N = B * T;
  const size_t norm = (size_t)token_floats(dtype, N, d) * 4 + (size_t)level_rows(N, levels_for(N, T)) * (size_t)d * 4;
  const size_t sum = (size_t)level_rows(N, levels_for(N, N)) * (size_t)d * 4;
  return (std::max(norm, sum) + 255) / 256 * 256;
}

hipError_t launch_embed_norm(hipStream_t st, int dtype, EmbedGradArgs a, void* ws) {
  set_levels(a, a.T);
  a.token_sq = static_cast<float*>(ws);
  a.sums = a.token_sq + token_floats(dtype, a.N, a.d);
  if (dtype == 1) return a.d < 8 ? launch_norm<bf16s, true>(st, a) : launch_norm<bf16s, false>(st, a);
  return a.d < 4 ? launch_norm<float, true>(st, a) : launch_norm<float, false>(st, a);
}

hipError_t launch_embed_sum(hipStream_t st, int dtype, EmbedGradArgs a, void* ws, const NoiseArgs& na, float* out) {
  set_levels(a, a.N);
  a.sums = static_cast<float*>(ws);
  if (dtype == 1) return a.d < 8 ? launch_sum<bf16s, true>(st, a, na, out) : launch_sum<bf16s, false>(st, a, na, out);
  return a.d < 4 ? launch_sum<float, true>(st, a, na, out) : launch_sum<float, false>(st, a, na, out);
}

}  // namespace dpk
