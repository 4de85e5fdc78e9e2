// Log probabilities of given tokens, with the entropy of the distribution and
// its top alternatives, and the gradient of the first two.
//
// With x_j = (z_j - m) / tau, m the largest logit, s = sum_j exp(x_j):
//   logp = x_y - log s           (0 for a target outside [0, V))
//   H = log s - sum_j exp(x_j) x_j / s     (every term of the sum has one sign)
//   top: the K largest logits, equal ones by ascending word, as log probabilities
//   dz_j = (dlogp (1[j = y] - p_j) - dH p_j (log p_j + H)) / tau
//
// Both directions are bound by HBM: the logits are read once (and the gradient
// written once). A token's words are streamed by one workgroup with a running
// maximum, sum and weighted sum per thread, joined at the end. For 4096 tokens
// of 50257 bf16: 76 us (5.4 TB/s), with 64 top words 106; the gradient 160 us
// (5.1 TB/s, the rate of a copy).
//
// The top words come out of the same pass, which leaves the largest logit of
// every 16-byte vector of the row (from 2048 vectors on, of every 8
// neighbouring ones, a cache line; of 4 bytes in short rows). With those dealt to 256 groups, the K-th
// largest of the groups' is a floor that at least K words reach, and in a row
// without a pattern hardly more (K = 64: 74 on average). One wave finds it by
// bisection of its bits, counting with ballots; the vectors or lines that reach
// it are read once more, by all threads, the words that reach it are collected,
// and put in order by counting the larger ones. Where too many reach the floor
// (rows of few different values, words of a mask's value) or fewer than K (rows
// with NaN, masks that leave almost nothing) the K-th largest is found from
// counts of the leading digits instead, in further passes over the row.
//
// A row whose logits are all -inf has no distribution: logp and the top words'
// are -inf, H is 0 and the gradient 0. A row with a NaN or +inf gives NaN.
#include "dp_common.hpp"
#include "dp_lm.hpp"
#include "dp_vocab.hpp"

#include <float.h>

namespace dpk {

namespace {

constexpr float kLn2 = 0.6931471805599453f;
// A distance from the maximum, in powers of two, beyond which 2^t is 0: it stands for larger ones (and infinite ones) in
// the products 2^t t.
constexpr float kFar = 256.0f;

// s = sum of 2^t and u = sum of 2^t t over the values seen, t = z k - base of the largest of them, m; k = log2(e) / tau.
// The initial maximum is finite, so that no difference of infinities arises.
struct Stat {
  float m, s, u;
};
__device__ __forceinline__ Stat stat_empty() { return Stat{-FLT_MAX, 0.f, 0.f}; }

// FAST: t = z k - fl(m k), a fused multiply-add; that the base is off m k is made good in the logarithm of the sum.
// It holds while |m k| < 2^20, where the base is off by 1/16 at most (kept above -2^20: values down to the type's
// lowest before a larger one is seen are 0 then). Else t = (z - m) k, two operations, for any m.
constexpr float kFastBase = 0x1p20f;
template <bool FAST>
__device__ __forceinline__ float base_of(float m, float k) {
  return FAST ? fmaxf(m * k, -kFastBase) : m;
}
template <bool FAST>
__device__ __forceinline__ float below(float z, float base, float k) {
  return FAST ? __builtin_fmaf(z, k, -base) : (z - base) * k;
}

// r as seen from the maximum m >= r.m
template <bool FAST, bool ENT>
__device__ __forceinline__ void stat_move(Stat& r, float m, float k) {
  const float x = FAST ? base_of<FAST>(r.m, k) - base_of<FAST>(m, k) : (r.m - m) * k, f = exp2_hw(x);
  if constexpr (ENT) r.u = f * __builtin_fmaf(fmaxf(x, -kFar), r.s, r.u);
  r.s *= f;
  r.m = m;
}
template <bool FAST, bool ENT>
__device__ __forceinline__ Stat stat_join(Stat a, Stat b, float k) {
  const float m = fmaxf(a.m, b.m);
  stat_move<FAST, ENT>(a, m, k);
  stat_move<FAST, ENT>(b, m, k);
  return Stat{m, a.s + b.s, a.u + b.u};
}
// top: the largest of the P values
template <bool FAST, bool ENT, int P>
__device__ __forceinline__ void stat_add(Stat& r, const float* z, float top, float k) {
  stat_move<FAST, ENT>(r, fmaxf(r.m, top), k);
  const float base = base_of<FAST>(r.m, k);
#pragma unroll
  for (int e = 0; e < P; ++e) {
    const float t = below<FAST>(z[e], base, k), p = exp2_hw(t);
    r.s += p;
    if constexpr (ENT) r.u = __builtin_fmaf(p, fmaxf(t, -kFar), r.u);
  }
}
template <int P>
__device__ __forceinline__ float largest(const float* z) {
  float m = z[0];
#pragma unroll
  for (int e = 1; e < P; ++e) m = fmaxf(m, z[e]);
  return m;
}
// The largest of eight neighbouring lanes' values, in each of them. All eight take part.
__device__ __forceinline__ float largest_of_8(float v) {
  const auto other = [](float x, auto ctrl) {
    const int i = (int)__float_as_uint(x);
    return __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(i, i, decltype(ctrl)::value, 0xf, 0xf, false));
  };
  v = fmaxf(v, other(v, std::integral_constant<int, 0xB1>{}));   // the neighbour
  v = fmaxf(v, other(v, std::integral_constant<int, 0x4E>{}));   // two lanes on
  return fmaxf(v, other(v, std::integral_constant<int, 0x141>{}));  // the mirrored lane of the eight
}

// one(word, value) and many(word, P values) over a thread's part of a row: single elements to the first 16-byte
// boundary, 16-byte vectors, single elements at the end.
template <typename T, int NT, typename F1, typename FP>
__device__ __forceinline__ void thread_words(const T* z, int64_t V, F1 one, FP many) {
  constexpr int P = elem_traits<T>::per16;
  const Span<T> sn(z, 0, V);
  const int64_t j = threadIdx.x;
  if (j < sn.head) one(j, to_f32(z[j]));
  const u32x4* vz = reinterpret_cast<const u32x4*>(z + sn.head);
  for (int64_t i = threadIdx.x; i < sn.vecs; i += NT) {
    float v[P];
    unpack16<P>(vz[i], v);
    many(sn.head + i * P, v);
  }
  const int64_t jt = sn.tail0 + threadIdx.x;
  if (jt < V) one(jt, to_f32(z[jt]));
}

// A wave's first lane's, in every lane. (The lanes of a butterfly of fused multiply-adds do not all end with the same
// bits.)
__device__ __forceinline__ float first_lane(float v) {
  return __uint_as_float((uint32_t)__builtin_amdgcn_readfirstlane((int)__float_as_uint(v)));
}

// Joined over the block; the same value in every thread. Contains barriers.
template <bool FAST, bool ENT, int NT>
__device__ __forceinline__ Stat block_stat(Stat r, float k, float* red) {
  auto join = [&](Stat& t, int off) {
    Stat o{__shfl_xor(t.m, off, kWave), __shfl_xor(t.s, off, kWave), 0.f};
    if constexpr (ENT) o.u = __shfl_xor(t.u, off, kWave);
    t = stat_join<FAST, ENT>(t, o, k);
  };
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) join(r, off);
  if constexpr (NT > 64) {
    constexpr int NW = NT / 64;
    __syncthreads();
    if ((threadIdx.x & 63) == 0) {
      red[3 * (threadIdx.x >> 6)] = r.m;
      red[3 * (threadIdx.x >> 6) + 1] = r.s;
      red[3 * (threadIdx.x >> 6) + 2] = r.u;
    }
    __syncthreads();
    const int w = threadIdx.x & (NW - 1);  // each wave joins them all, over its lanes
    r = Stat{red[3 * w], red[3 * w + 1], red[3 * w + 2]};
#pragma unroll
    for (int off = NW / 2; off > 0; off >>= 1) join(r, off);
  }
  return Stat{first_lane(r.m), first_lane(r.s), first_lane(r.u)};
}

// A logit and its word as one number: larger logits first, among equal ones (0 and -0 are) the lower word; NaN above
// all.
__device__ __forceinline__ uint32_t key_of(float z) {
  const uint32_t b = __float_as_uint(z + 0.0f);
  return z != z ? 0xFFFFFFFFu : b ^ ((b >> 31) ? 0xFFFFFFFFu : 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t key) {
  return __uint_as_float((key >> 31) ? key ^ 0x80000000u : ~key);
}
__device__ __forceinline__ uint64_t place_of(float z, int64_t word) {
  return ((uint64_t)key_of(z) << 32) | (uint32_t)~(uint32_t)word;
}

constexpr int kGroups = 256;

// LDS of the selection: the largest logit of every part of the row (a vector, or 8) or the collected words, the groups'
// largest keys or digit counts, the parts that reach the floor.
template <int NT>
struct TopLds {
  static constexpr int parts = NT <= 128 ? 1024 : 2048, cap = NT <= 128 ? 512 : 1024;
  union {  // the words are collected once the parts have been looked through
    __attribute__((aligned(16))) float part[parts];
    __attribute__((aligned(16))) uint64_t found[cap];
  };
  union {
    __attribute__((aligned(16))) uint32_t best[kGroups];
    uint32_t bins[256];
  };
  uint16_t reach[cap];
  uint32_t floor, reaches, count, digit, above, at;
};

template <>
struct TopLds<0> {  // no top words
  static constexpr int parts = 1;
  float part[1];
};

// The words whose place is at least `least`.
template <typename T, int NT>
__device__ __forceinline__ void collect(const T* z, int64_t V, uint64_t least, TopLds<NT>& l) {
  constexpr int P = elem_traits<T>::per16;
  auto one = [&](int64_t j, float v) {
    const uint64_t p = place_of(v, j);
    if (p >= least) {
      const uint32_t at = atomicAdd(&l.count, 1u);
      if (at < (uint32_t)TopLds<NT>::cap) l.found[at] = p;
    }
  };
  thread_words<T, NT>(z, V, one, [&](int64_t j, const float* v) {
#pragma unroll
    for (int e = 0; e < P; ++e) one(j + e, v[e]);
  });
}

// A place that K words of the row reach, and at most `cap`: digits of 8 bits from the top, each from the counts of
// the words that share the digits so far.
template <typename T, int NT>
__device__ uint64_t least_place(const T* z, int64_t V, int64_t K, TopLds<NT>& l) {
  constexpr int P = elem_traits<T>::per16;
  uint64_t prefix = 0;
  uint32_t want = (uint32_t)K, above = 0;
  for (int shift = 56; ; shift -= 8) {
    if (shift < 32 && shift >= 8 && V <= ((int64_t)1 << shift)) {  // a digit of 255 in every word
      prefix = (prefix << 8) | 255;
      continue;
    }
    for (int k = threadIdx.x; k < 256; k += NT) l.bins[k] = 0;
    __syncthreads();
    auto one = [&](int64_t j, float v) {
      const uint64_t p = place_of(v, j);
      if (shift < 56 && (p >> (shift + 8)) != prefix) return;
      const uint32_t digit = (uint32_t)(p >> shift) & 255u;
      // rows of one value: one add for the wave
      const uint32_t first = (uint32_t)__builtin_amdgcn_readfirstlane((int)digit);
      const uint64_t same = __ballot(digit == first), here = __ballot(true);
      if (same == here) {
        if ((here & ((1ull << (threadIdx.x & 63)) - 1)) == 0) atomicAdd(&l.bins[digit], (uint32_t)__popcll(here));
      } else {
        atomicAdd(&l.bins[digit], 1u);
      }
    };
    thread_words<T, NT>(z, V, one, [&](int64_t j, const float* v) {
#pragma unroll
      for (int e = 0; e < P; ++e) one(j + e, v[e]);
    });
    __syncthreads();
    if (threadIdx.x < 64) {  // four digits a lane, from 255 down
      uint32_t c[4], sum = 0;
#pragma unroll
      for (int u = 0; u < 4; ++u) sum += c[u] = l.bins[255 - 4 * threadIdx.x - u];
      uint32_t run = sum;
#pragma unroll
      for (int off = 1; off < 64; off <<= 1) {
        const uint32_t o = __shfl_up(run, off, kWave);
        if ((int)threadIdx.x >= off) run += o;
      }
      uint32_t before = run - sum;
      if (before < want && run >= want) {
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          if (before < want && before + c[u] >= want) {
            l.digit = 255 - 4 * threadIdx.x - u;
            l.above = before;
            l.at = c[u];
          }
          before += c[u];
        }
      }
    }
    __syncthreads();
    prefix = (prefix << 8) | l.digit;
    above += l.above;
    want -= l.above;
    const uint32_t at = l.at;
    __syncthreads();  // read before the next digit's
    if (shift == 0 || above + at <= (uint32_t)TopLds<NT>::cap) return prefix << shift;
  }
}

// The K-th largest of the groups' largest keys, its low bits 0 (the 16 that bf16 does not have, or 12), by one wave,
// four groups a lane.
template <typename T, int NT>
__device__ __forceinline__ uint32_t find_floor(int K, const TopLds<NT>& l) {
  constexpr int last = elem_traits<T>::per16 == 8 ? 16 : 12;
  const u32x4 best = *reinterpret_cast<const u32x4*>(l.best + 4 * threadIdx.x);
  uint32_t floor = 0;
  for (int bit = 31; bit >= last; --bit) {
    const uint32_t t = floor | (1u << bit);
    int n = 0;
#pragma unroll
    for (int u = 0; u < 4; ++u) n += __popcll(__ballot(best[u] >= t));
    if (n >= K) floor = t;
    if (n == K) break;
  }
  return floor;
}

// The row's K top words into top_ids and top_logp, from the parts' largest logits in l.part. A part is a vector; by8: 8
// of them; SMALL: 4 bytes, one word or two.
// r: the largest logit, the sum (0: no distribution, NaN: NaN or +inf in the row) and log of the sum.
template <typename T, int NT, bool SMALL>
__device__ __forceinline__ void top_words(const LogprobArgs& a, int64_t row, const T* z, bool by8, Stat r, TopLds<NT>& l) {
  constexpr int P = elem_traits<T>::per16;
  const int K = (int)a.K;
  const Span<T> sn(z, 0, a.V);
  const int64_t parts64 = SMALL ? 4 * sn.vecs : by8 ? (sn.vecs + 7) / 8 : sn.vecs;
  const int parts = (int)(parts64 < TopLds<NT>::parts ? parts64 : TopLds<NT>::parts);
  __syncthreads();  // l.part is whole
  for (int g = threadIdx.x; g < kGroups; g += NT) {
    float m = -FLT_MAX;
    for (int p = g; p < parts; p += kGroups) m = fmaxf(m, l.part[p]);
    l.best[g] = key_of(m);
  }
  if (threadIdx.x == 0) l.count = l.reaches = 0;
  __syncthreads();
  if (threadIdx.x < 64) {
    const uint32_t f = find_floor<T, NT>(K, l);
    if (threadIdx.x == 0) l.floor = f;
  }
  __syncthreads();
  const uint32_t floor = l.floor;
  for (int p = threadIdx.x; p < parts; p += NT)
    if (key_of(l.part[p]) >= floor) {
      const uint32_t at = atomicAdd(&l.reaches, 1u);
      if (at < (uint32_t)TopLds<NT>::cap) l.reach[at] = (uint16_t)p;
    }
  __syncthreads();
  const uint32_t reaches = l.reaches;
  if (r.s == r.s && reaches <= (uint32_t)TopLds<NT>::cap) {  // no NaN, no +inf
    auto one = [&](int64_t j, float v) {
      if (key_of(v) >= floor) {
        const uint32_t at = atomicAdd(&l.count, 1u);
        if (at < (uint32_t)TopLds<NT>::cap) l.found[at] = place_of(v, j);
      }
    };
    const int64_t j = threadIdx.x, jt = sn.tail0 + threadIdx.x;
    if (j < sn.head) one(j, to_f32(z[j]));
    if (jt < a.V) one(jt, to_f32(z[jt]));
    const u32x4* vz = reinterpret_cast<const u32x4*>(z + sn.head);
    if constexpr (SMALL) {
      for (uint32_t i = threadIdx.x; i < reaches; i += NT) {
        const int p = l.reach[i];
        const uint32_t raw = reinterpret_cast<const uint32_t*>(vz)[p];
        if constexpr (P == 8) {
          one(sn.head + 2 * p, __uint_as_float(raw << 16));
          one(sn.head + 2 * p + 1, __uint_as_float(raw & 0xFFFF0000u));
        } else {
          one(sn.head + p, __uint_as_float(raw));
        }
      }
    }
    // a part number stands for all that share it: parts, 2 * parts ... on (rows of very many words)
    const int shift = by8 ? 3 : 0;
    const uint32_t work = reaches << shift;
    constexpr int U = 2;
    for (int64_t first = SMALL ? sn.vecs : 0; first < sn.vecs; first += (int64_t)TopLds<NT>::parts << shift) {
      for (uint32_t i0 = threadIdx.x; i0 < work; i0 += U * NT) {
        u32x4 raw[U];
        int64_t at[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const uint32_t i = i0 + u * NT;
          at[u] = i < work ? first + ((int64_t)l.reach[i >> shift] << shift) + (i & ((1u << shift) - 1)) : sn.vecs;
          raw[u] = u32x4{0u, 0u, 0u, 0u};
          if (at[u] < sn.vecs) raw[u] = vz[at[u]];
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
          if (at[u] >= sn.vecs) continue;
          float v[P];
          unpack16<P>(raw[u], v);
          if (key_of(largest<P>(v)) < floor) continue;
#pragma unroll
          for (int e = 0; e < P; ++e) one(sn.head + at[u] * P + e, v[e]);
        }
      }
    }
  }
  __syncthreads();
  uint32_t n = l.count;
  if (n < (uint32_t)K || n > (uint32_t)TopLds<NT>::cap) {  // uniform
    __syncthreads();  // count is read before it is cleared
    const uint64_t least = least_place<T, NT>(z, a.V, K, l);
    if (threadIdx.x == 0) l.count = 0;
    __syncthreads();
    collect<T, NT>(z, a.V, least, l);
    __syncthreads();
    n = l.count < (uint32_t)TopLds<NT>::cap ? l.count : (uint32_t)TopLds<NT>::cap;
  }
  const float inv_tau = 1.0f / a.tau, log_s = r.u;
  for (uint32_t i = threadIdx.x; i < n; i += NT) {
    const uint64_t p = l.found[i];
    uint32_t rank = 0;
#pragma unroll 4
    for (uint32_t j = 0; j + 1 < n; j += 2) {  // two words a read
      const ulonglong2 o = *reinterpret_cast<const ulonglong2*>(l.found + j);
      rank += (o.x > p) + (o.y > p);
    }
    if (n & 1) rank += l.found[n - 1] > p;
    if (rank < (uint32_t)K) {
      const float v = key_value((uint32_t)(p >> 32));
      a.top_ids[row * K + rank] = (int64_t)(uint32_t)~(uint32_t)p;
      a.top_logp[row * K + rank] = r.s == 0.0f ? -INFINITY : __builtin_fmaf(v - r.m, inv_tau, -log_s);
    }
  }
  __syncthreads();  // found and the parts are written again by the next row
}

}  // namespace

// One workgroup per token. TOP: 0 without top words, 1 with, 2 with parts of 4 bytes. (Six waves per SIMD with top words:
// with eight the compiler spills, 4096 tokens of 50257 bf16 and 64 top words take 121 us instead of 109.)
template <typename T, int NT, bool ENT, int TOP>
__global__ __launch_bounds__(NT, TOP ? 6 : 8) void k_token_logprob(LogprobArgs a) {
  constexpr int P = elem_traits<T>::per16;
  __shared__ float red[3 * NT / 64];
  __shared__ TopLds<TOP ? NT : 0> lds;
  const float k = kLog2e / a.tau;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const T* z = static_cast<const T*>(a.logits) + row * a.V;
    const int64_t y = a.targets[row];
    const bool given = y >= 0 && y < a.V;
    const float zy = given ? to_f32(z[y]) : 0.0f;
    Stat r = stat_empty();
    const Span<T> sn(z, 0, a.V);
    const u32x4* vz = reinterpret_cast<const u32x4*>(z + sn.head);
    const bool by8 = TOP == 1 && sn.vecs > TopLds<NT>::parts;  // a part of the row is 8 vectors
    // Round n holds vectors n * NT ..; a part number stands again for parts behind the last one. Both are the wave's.
    auto keep = [&](const float* v, float top, int n) {
      if constexpr (TOP == 2) {
        f32x4 m;
#pragma unroll
        for (int e = 0; e < 4; ++e) m[e] = P == 8 ? fmaxf(v[2 * e % P], v[(2 * e + 1) % P]) : v[e];
        *reinterpret_cast<f32x4*>(lds.part + 4 * (n * NT + threadIdx.x)) = m;
      } else if constexpr (TOP == 1) {
        if (by8) {
          const float m = largest_of_8(top);
          const int at = n * (NT / 8);
          float& part = lds.part[(at & (TopLds<NT>::parts - 1)) + (threadIdx.x >> 3)];
          if ((threadIdx.x & 7) == 0) part = at < TopLds<NT>::parts ? m : fmaxf(part, m);
        } else {
          lds.part[n * NT + threadIdx.x] = top;
        }
      }
    };
    constexpr int U = 4;  // vectors in flight
    const int full = (int)(sn.vecs / NT);  // rounds of all threads
    const int rest = (int)(sn.vecs - (int64_t)full * NT);
    int n = 0;
    for (; n + U <= full; n += U) {
      u32x4 raw[U];
#pragma unroll
      for (int u = 0; u < U; ++u) raw[u] = vz[(int64_t)(n + u) * NT + threadIdx.x];
#pragma unroll
      for (int u = 0; u < U; u += 2) {  // two vectors to a step of the maximum
        float v[2 * P];
        unpack16<P>(raw[u], v);
        unpack16<P>(raw[u + 1], v + P);
        const float top0 = largest<P>(v), top1 = largest<P>(v + P);
        keep(v, top0, n + u);
        keep(v + P, top1, n + u + 1);
        stat_add<true, ENT, 2 * P>(r, v, fmaxf(top0, top1), k);
      }
    }
    {
      // The last rounds, the last of them not of all threads: those have -inf there, which counts for nothing, and take
      // part in the eight lanes' largest.
      constexpr uint32_t kNothing = P == 8 ? 0xFF80FF80u : 0xFF800000u;
      u32x4 raw[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        raw[u] = u32x4{kNothing, kNothing, kNothing, kNothing};
        if (n + u < full || (n + u == full && (int)threadIdx.x < rest)) raw[u] = vz[(int64_t)(n + u) * NT + threadIdx.x];
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (n + u > full || (n + u == full && rest == 0)) break;  // the same in every thread
        float v[P];
        unpack16<P>(raw[u], v);
        const float top = largest<P>(v);
        keep(v, top, n + u);
        stat_add<true, ENT, P>(r, v, top, k);
      }
    }
    auto single = [&](int64_t j, int64_t end, auto fast) {
      if (j >= end) return;
      const float v = to_f32(z[j]);
      stat_add<decltype(fast)::value, ENT, 1>(r, &v, v, k);
    };
    single(threadIdx.x, sn.head, std::true_type{});
    single(sn.tail0 + threadIdx.x, a.V, std::true_type{});
    r = block_stat<true, ENT, NT>(r, k, red);
    float shift = __builtin_fmaf(r.m, k, -base_of<true>(r.m, k));  // m k less the base
    if (!(fabsf(r.m * k) < kFastBase)) {  // the same in every thread: a mask's value, +inf, a temperature near 0
      shift = 0.0f;
      r = stat_empty();
      thread_words<T, NT>(
          z, a.V, [&](int64_t, float v) { stat_add<false, ENT, 1>(r, &v, v, k); },
          [&](int64_t, const float* v) { stat_add<false, ENT, P>(r, v, largest<P>(v), k); });
      r = block_stat<false, ENT, NT>(r, k, red);
    }
    const bool none = r.s == 0.0f;  // every logit is -inf
    const float log_s = none ? 0.0f : __builtin_fmaf(-kLn2, shift, logf(r.s));
    if (threadIdx.x == 0) {
      a.logp[row] = !given ? 0.0f : none ? -INFINITY : (zy - r.m) / a.tau - log_s;
      a.stats[2 * row] = none ? -INFINITY : r.m;
      a.stats[2 * row + 1] = log_s;
      if (ENT) a.entropy[row] = none ? 0.0f : logf(r.s) - kLn2 * (r.u / r.s);
    }
    r.u = log_s;
    if constexpr (TOP) top_words<T, NT, TOP == 2>(a, row, z, by8, r, lds);
  }
}

// One workgroup per (token, split of its words).
template <typename T, int NT, bool ENT>
__global__ __launch_bounds__(NT) void k_token_logprob_backward(LogprobArgs a) {
  constexpr int P = elem_traits<T>::per16;
  const float inv_tau = 1.0f / a.tau;
  const int64_t items = a.rows * a.splits, len = (a.V + a.splits - 1) / a.splits;
  for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
    const int64_t row = item / a.splits, sp = item - row * a.splits;
    const int64_t v0 = sp * len, v1 = v0 + len < a.V ? v0 + len : a.V;
    if (v0 >= v1) continue;  // uniform
    const T* z = static_cast<const T*>(a.logits) + row * a.V;
    T* g = static_cast<T*>(a.grad) + row * a.V;
    const int64_t y = a.targets[row];
    const float dl = a.dlogp && y >= 0 && y < a.V ? a.dlogp[row] * inv_tau : 0.0f;
    const float dh = ENT ? a.dentropy[row] * inv_tau : 0.0f;
    const float m = a.stats[2 * row], log_s = a.stats[2 * row + 1];
    const float h = ENT ? a.entropy[row] : 0.0f;
    // nothing to pass on, or a row without a distribution: 0 whatever the logits hold
    const bool on = (dl != 0.0f || dh != 0.0f) && m != -INFINITY;
    auto grad_of = [&](float zz) {
      const float lp = __builtin_fmaf(zz - m, inv_tau, -log_s);
      const float p = exp2_hw(lp * kLog2e);
      // beyond exp(-200) p is 0: its logarithm may be -inf
      return ENT ? -p * __builtin_fmaf(dh, fmaxf(lp, -200.0f) + h, dl) : -p * dl;
    };
    const Span<T> sn(z, v0, v1);
    auto put1 = [&](int64_t j) {
      const float v = on ? grad_of(to_f32(z[j])) + (j == y ? dl : 0.0f) : 0.0f;
      if constexpr (P == 8) g[j].u = f32_to_bf16(v);
      else g[j] = v;
    };
    {
      const int64_t j = v0 + threadIdx.x, jt = sn.tail0 + threadIdx.x;
      if (j < sn.head) put1(j);
      if (jt < v1) put1(jt);
    }
    const u32x4* vz = reinterpret_cast<const u32x4*>(z + sn.head);
    // grad and logits share their misalignment (checked on the host), so these are aligned too
    u32x4* vg = reinterpret_cast<u32x4*>(g + sn.head);
    if (!on) {
      for (int64_t i = threadIdx.x; i < sn.vecs; i += NT) vg[i] = u32x4{0u, 0u, 0u, 0u};
      continue;
    }
    const int64_t yv = y >= sn.head && y < sn.tail0 ? (y - sn.head) / P : -1;  // the target's vector and place in it
    const int ye = (int)(y - sn.head - yv * P);
    auto vec = [&](u32x4 raw, int64_t i) {
      float v[P];
      unpack16<P>(raw, v);
#pragma unroll
      for (int e = 0; e < P; ++e) v[e] = grad_of(v[e]);
      if (i == yv) {
#pragma unroll
        for (int e = 0; e < P; ++e) v[e] += e == ye ? dl : 0.0f;
      }
      u32x4 o;
      if constexpr (P == 8) {
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] = pack_bf16(v[2 * e], v[2 * e + 1]);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] = __float_as_uint(v[e]);
      }
      return o;
    };
    // eight vectors in flight per thread, past the caches both ways
    constexpr int U = 8;
    int64_t i = threadIdx.x;
    for (; i + (U - 1) * NT < sn.vecs; i += U * NT) {
      u32x4 raw[U];
#pragma unroll
      for (int u = 0; u < U; ++u) raw[u] = __builtin_nontemporal_load(vz + i + u * NT);
#pragma unroll
      for (int u = 0; u < U; ++u) __builtin_nontemporal_store(vec(raw[u], i + u * NT), vg + i + u * NT);
    }
    for (; i < sn.vecs; i += NT) vg[i] = vec(vz[i], i);
  }
}

namespace {

unsigned grid_of(int64_t n) { return (unsigned)std::min<int64_t>(n, 1 << 20); }

template <typename T, int NT>
hipError_t launch_fwd(hipStream_t st, const LogprobArgs& a) {
  const unsigned blocks = grid_of(a.rows);
  auto run = [&](auto top) {
    constexpr int TOP = decltype(top)::value;
    if (a.entropy) k_token_logprob<T, NT, true, TOP><<<blocks, NT, 0, st>>>(a);
    else k_token_logprob<T, NT, false, TOP><<<blocks, NT, 0, st>>>(a);
    return hipGetLastError();
  };
  if (a.K == 0) return run(std::integral_constant<int, 0>{});
  // Rows of up to 128 vectors, with a top word in every fourth or more: the largest of whole vectors are so few that the
  // floor lets many others through, and ranking takes the square of them (20000 tokens of 600 bf16: 32 top words 31 us
  // against 34 with parts of a vector, 100 top words 50 against 90).
  constexpr int P = elem_traits<T>::per16;
  if constexpr (NT == 64)
    if (a.V <= 128 * P && 4 * P * a.K > a.V) return run(std::integral_constant<int, 2>{});
  return run(std::integral_constant<int, 1>{});
}

template <typename T, int NT>
hipError_t launch_bwd(hipStream_t st, const LogprobArgs& a) {
  const unsigned blocks = grid_of(a.rows * a.splits);
  if (a.dentropy) k_token_logprob_backward<T, NT, true><<<blocks, NT, 0, st>>>(a);
  else k_token_logprob_backward<T, NT, false><<<blocks, NT, 0, st>>>(a);
  return hipGetLastError();
}

// Threads for a token's words. Few tokens: as many as a workgroup may have, so
// that a row is few loads of each. Many tokens of a small vocabulary: a wave
// each, or two (20000 tokens of 8000 words, 20 top words: 93 us with two waves,
// 120 with four; 4096 of 16000: 35 and 39, but with 100 top words 57 and 46).
int logprob_threads(int64_t rows, int64_t V, int64_t K) {
  if (V <= 256 || (rows > 512 && V <= 4096)) return 64;
  if (rows > 512 && V <= 16384 && K <= 128) return 128;
  if (rows > 512 || V <= 2048) return 256;
  return rows > 256 || V <= 4096 ? 512 : 1024;
}

}  // namespace

hipError_t launch_token_logprob(hipStream_t st, int dtype, const LogprobArgs& a) {
  auto run = [&](auto nt) {
    constexpr int NT = decltype(nt)::value;
    return dtype == 1 ? launch_fwd<bf16s, NT>(st, a) : launch_fwd<float, NT>(st, a);
  };
  switch (logprob_threads(a.rows, a.V, a.K)) {
    case 64: return run(std::integral_constant<int, 64>{});
    case 128: return run(std::integral_constant<int, 128>{});
    case 256: return run(std::integral_constant<int, 256>{});
    case 512: return run(std::integral_constant<int, 512>{});
    default: return run(std::integral_constant<int, 1024>{});
  }
}

hipError_t launch_token_logprob_backward(hipStream_t st, int dtype, LogprobArgs a) {
  // Splits of a token's words: none from 512 tokens on; below, as many as give about 1024 workgroups, each of at
  // least 2048 words.
  a.splits = 1;
  if (a.rows < 512) {
    const int64_t want = (1024 + a.rows - 1) / a.rows, most = (a.V + 2047) / 2048;
    a.splits = std::max<int64_t>(1, std::min(want, most));
  }
  if (a.splits == 1 && a.V <= 4096)
    return dtype == 1 ? launch_bwd<bf16s, 64>(st, a) : launch_bwd<float, 64>(st, a);
  return dtype == 1 ? launch_bwd<bf16s, 256>(st, a) : launch_bwd<float, 256>(st, a);
}

}  // namespace dpk
