// Distillation loss from a teacher's top logits, per sample, and its gradient.
//
// For each token the teacher gives K places (word, logit); a place is used
// when its word lies in [0, V) and its logit is not -inf. With temperature tau,
//   q = softmax of the used places' teacher logits / tau   (the teacher, renormalised)
//   p = softmax(z / tau) over all V words                  (the student)
//   loss[b] = tau^2 * sum_t w[b][t] * sum_k q_k (log q_k - log p_{id_k})
//   dz[b][t][j] = dloss[b] * w[b][t] * tau * (p_j - sum_{k: id_k = j} q_k)
// A token without a used place, or with weight 0, has loss 0 and gradient 0
// whatever its logits hold.
//
// Both directions are bound by HBM (2048 x 32003 fp32 forward 44 us, 6.0 TB/s;
// 4096 x 50257 bf16 backward 165 us, 5.0 TB/s): the logits are read once (and
// the gradient written once); a token's V words are streamed with a running
// maximum and sum per thread, joined across the block at the end. The
// logarithm's argument is kept as (z - max) in raw logits, so that rows holding
// the type's lowest value neither overflow nor give NaN. Where tokens are few,
// each takes a workgroup of 1024 threads (a row of 50257 bf16 is then six
// loads of a thread, all in flight together, and the loss is one launch).
// Sums over a sample's tokens run in a fixed order in a kernel of their own;
// nothing is atomic.
#include "dp_common.hpp"
#include "dp_lm.hpp"

#include <float.h>

namespace dpk {

namespace {

constexpr int kDt = 256;  // threads per block
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kFarLse = 1024.0f;  // from here on the backward forms a row's statistics again

// 2^x by the hardware's instruction: within one step, results below 2^-126
// flushed to 0 (they are terms of sums of order 1, or probabilities).
__device__ __forceinline__ float exp2_hw(float x) { return __builtin_amdgcn_exp2f(x); }

// (m, s): s = sum of 2^((z - m) k) over the values seen, k = log2(e)/tau. The
// initial maximum is finite, so that no difference of infinities arises.
struct Run {
  float m, s;
};
__device__ __forceinline__ Run run_empty() { return Run{-FLT_MAX, 0.f}; }
__device__ __forceinline__ Run run_join(Run a, Run b, float k) {
  const float m = fmaxf(a.m, b.m);
  return Run{m, a.s * exp2_hw((a.m - m) * k) + b.s * exp2_hw((b.m - m) * k)};
}
__device__ __forceinline__ void run_one(Run& r, float z, float k) {
  const float m = fmaxf(r.m, z);
  r.s = r.s * exp2_hw((r.m - m) * k) + exp2_hw((z - m) * k);
  r.m = m;
}
// P values at once: one rescale for all of them.
template <int P>
__device__ __forceinline__ void run_many(Run& r, const float* z, float k) {
  float m = r.m;
#pragma unroll
  for (int e = 0; e < P; ++e) m = fmaxf(m, z[e]);
  float s = r.s * exp2_hw((r.m - m) * k);
#pragma unroll
  for (int e = 0; e < P; ++e) s += exp2_hw((z[e] - m) * k);
  r.m = m;
  r.s = s;
}

__device__ __forceinline__ Run wave_join(Run r, float k) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) {
    const Run o{__shfl_xor(r.m, off, kWave), __shfl_xor(r.s, off, kWave)};
    r = run_join(r, o, k);
  }
  return r;
}

// Joined over the block; the same value in every thread. Contains barriers.
template <int NT>
__device__ __forceinline__ Run block_join(Run r, float k, float* red) {
  r = wave_join(r, k);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) {
    red[2 * (threadIdx.x >> 6)] = r.m;
    red[2 * (threadIdx.x >> 6) + 1] = r.s;
  }
  __syncthreads();
  float m = red[0], s = 0.f;
#pragma unroll
  for (int w = 1; w < NT / 64; ++w) m = fmaxf(m, red[2 * w]);
#pragma unroll
  for (int w = 0; w < NT / 64; ++w) s += red[2 * w + 1] * exp2_hw((red[2 * w] - m) * k);
  return Run{m, s};
}
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

// Teacher logit i, fp32 or bf16.
__device__ __forceinline__ float teacher_at(const DistillArgs& a, int64_t i) {
  return a.teacher_bf16 ? to_f32(static_cast<const bf16s*>(a.teacher)[i]) : static_cast<const float*>(a.teacher)[i];
}

// The maximum over the used places. A NaN counts as the largest: a maximum that
// passed it over would leave a token whose teacher is all NaN without a place.
__device__ __forceinline__ float teacher_max(float m, float t) { return fmaxf(m, t == t ? t : INFINITY); }

// A token's weight and the place of its first K that this thread holds, read
// ahead of the student's statistics.
struct FirstPlace {
  float weight, teacher;
  int64_t id;
};
__device__ __forceinline__ FirstPlace first_place(const DistillArgs& a, int64_t row) {
  FirstPlace f{1.0f, 0.0f, -1};
  if (a.weight) f.weight = a.weight[row];
  if (threadIdx.x < a.K) {
    f.id = a.ids[row * a.K + threadIdx.x];
    f.teacher = teacher_at(a, row * a.K + threadIdx.x);
  }
  return f;
}

// The loss of one token from its student statistics, by the whole block.
template <typename T, int NT>
__device__ float token_loss(const DistillArgs& a, int64_t row, const FirstPlace& fp, Run r, float* red) {
  const float w = fp.weight;
  if (w == 0.0f) return 0.0f;  // uniform over the block
  const T* z = static_cast<const T*>(a.logits) + row * a.V;
  const int64_t* id = a.ids + row * a.K;
  const float inv_tau = 1.0f / a.tau;
  float tm = -INFINITY, z0 = 0.0f;
  if (fp.id >= 0 && fp.id < a.V) {
    tm = teacher_max(tm, fp.teacher);
    z0 = to_f32(z[fp.id]);
  }
  for (int64_t k = threadIdx.x + NT; k < a.K; k += NT)
    if (id[k] >= 0 && id[k] < a.V) tm = teacher_max(tm, teacher_at(a, row * a.K + k));
  tm = block_max<NT>(tm, red);
  if (tm == -INFINITY) return 0.0f;  // no used place
  float total = 0.f, s = 0.f;
  for (int64_t k = threadIdx.x; k < a.K; k += NT) {
    const bool ahead = k == threadIdx.x;
    const int64_t j = ahead ? fp.id : id[k];
    if (j < 0 || j >= a.V) continue;
    const float dt = ((ahead ? fp.teacher : teacher_at(a, row * a.K + k)) - tm) * inv_tau;
    const float e = exp2_hw(dt * kLog2e);
    if (e == 0.0f) continue;  // no mass there: its logits (infinite ones among them) do not count
    total += e;
    s += e * (dt - ((ahead ? z0 : to_f32(z[j])) - r.m) * inv_tau);
  }
  total = block_add<NT>(total, red);
  s = block_add<NT>(s, red);
  // sum_k q_k (log q_k - log p_k), with log q = dt - log total, log p = (z - m)/tau - log s_student
  const float kl = s / total - logf(total) + logf(r.s);
  return a.tau * a.tau * w * kl;
}

__device__ __forceinline__ float lse_of(Run r, float tau) { return r.m / tau + logf(r.s); }

// A thread's part of a row's words [v0, v1), the block's NT threads side by side.
template <typename T, int NT>
__device__ __forceinline__ Run run_span(const T* z, int64_t v0, int64_t v1, float k) {
  constexpr int P = elem_traits<T>::per16;
  Run r = run_empty();
  const Span<T> sn(z, v0, v1);
  const int64_t j = v0 + threadIdx.x;
  if (j < sn.head) run_one(r, to_f32(z[j]), k);
  const u32x4* vz = reinterpret_cast<const u32x4*>(z + sn.head);
  constexpr int U = 4;  // vectors in flight per thread
  int64_t i = threadIdx.x;
  for (; i + (U - 1) * NT < sn.vecs; i += U * NT) {
    u32x4 raw[U];
#pragma unroll
    for (int u = 0; u < U; ++u) raw[u] = vz[i + u * NT];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float v[P];
      unpack16<P>(raw[u], v);
      run_many<P>(r, v, k);
    }
  }
  if (i < sn.vecs) {  // up to U - 1 more, in flight together (the last of them read again where there are fewer)
    u32x4 raw[U - 1];
#pragma unroll
    for (int u = 0; u < U - 1; ++u) raw[u] = vz[i + u * NT < sn.vecs ? i + u * NT : i];
#pragma unroll
    for (int u = 0; u < U - 1; ++u) {
      if (i + u * NT >= sn.vecs) break;
      float v[P];
      unpack16<P>(raw[u], v);
      run_many<P>(r, v, k);
    }
  }
  const int64_t jt = sn.tail0 + threadIdx.x;
  if (jt < v1) run_one(r, to_f32(z[jt]), k);
  return r;
}

}  // namespace

// One block per token: its statistics, then its loss.
template <typename T, int NT>
__global__ __launch_bounds__(NT) void k_distill_loss(DistillArgs a) {
  __shared__ float red[2 * NT / 64];
  const float k = kLog2e / a.tau;
  for (int64_t row = blockIdx.x; row < a.B * a.T; row += gridDim.x) {
    const FirstPlace fp = first_place(a, row);
    const Run r = block_join<NT>(run_span<T, NT>(static_cast<const T*>(a.logits) + row * a.V, 0, a.V, k), k, red);
    const float loss = token_loss<T, NT>(a, row, fp, r, red);
    if (threadIdx.x == 0) {
      a.lse[row] = lse_of(r, a.tau);
      (a.T == 1 ? a.loss : a.row_loss)[row] = loss;
    }
  }
}

__global__ __launch_bounds__(kDt) void k_distill_sum(const float* __restrict__ row_loss, int64_t B, int64_t Tn,
                                                     float* __restrict__ loss) {
  __shared__ float red[kDt / 64];
  for (int64_t b = blockIdx.x; b < B; b += gridDim.x) {
    float s = 0.f;
    for (int64_t t = threadIdx.x; t < Tn; t += kDt) s += row_loss[b * Tn + t];
    s = block_add<kDt>(s, red);
    if (threadIdx.x == 0) loss[b] = s;
  }
}

// One block per (token, split): the split's p_j f first, then, after a
// barrier, the used words inside the split are overwritten with (p - q) f by
// the threads that hold them (q summed over the places naming the word, in
// place order). Their logits are read before the barrier, so grad may be the
// logits' own buffer.
template <typename T>
__global__ __launch_bounds__(kDt) void k_distill_backward(DistillArgs a) {
  constexpr int P = elem_traits<T>::per16;
  __shared__ float red[2 * kDt / 64];
  __shared__ __attribute__((aligned(16))) int32_t ids[kDistillMaxTop + 4];
  __shared__ __attribute__((aligned(16))) float qs[kDistillMaxTop + 4];
  const float inv_tau = 1.0f / a.tau;
  const int64_t items = a.B * a.T * a.splits;
  const int64_t len = (a.V + a.splits - 1) / a.splits;
  const int K = (int)a.K, K4 = (K + 3) / 4;
  for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
    const int64_t row = item / a.splits, sp = item - row * a.splits;
    const int64_t v0 = sp * len, v1 = v0 + len < a.V ? v0 + len : a.V;
    if (v0 >= v1) continue;  // uniform
    const T* z = static_cast<const T*>(a.logits) + row * a.V;
    T* g = static_cast<T*>(a.grad) + row * a.V;
    const int64_t* id = a.ids + row * a.K;
    float f = a.weight ? a.weight[row] : 1.0f;
    if (a.dloss) f *= a.dloss[row / a.T];
    f *= a.tau;
    // ---- the teacher's distribution: a place's word (-1: unused) and probability
    float tm = -INFINITY;
    if (f != 0.0f)
      for (int k = threadIdx.x; k < K; k += kDt)
        if (id[k] >= 0 && id[k] < a.V) tm = teacher_max(tm, teacher_at(a, row * a.K + k));
    tm = block_max<kDt>(tm, red);
    const bool any = f != 0.0f && tm != -INFINITY;
    float total = 0.f;
    if (any) {
      for (int k = threadIdx.x; k < 4 * K4; k += kDt) {
        int32_t w = -1;
        float e = 0.f;
        if (k < K && id[k] >= 0 && id[k] < a.V) {
          w = (int32_t)id[k];
          e = exp2_hw((teacher_at(a, row * a.K + k) - tm) * inv_tau * kLog2e);
        }
        ids[k] = w;
        qs[k] = e;
        total += e;
      }
    }
    total = block_add<kDt>(total, red);  // its barriers also publish ids and qs
    const float inv_total = any ? 1.0f / total : 0.0f;
    // log p_j = (z_j - m) / tau - shift. m = 0 and shift = lse, whose rounding costs p 2^-24 |lse|. Where that
    // would show (rows of a mask's value, down to the type's lowest, have no room for log V in lse) m and the
    // logarithm of the sum are formed again from the row.
    float shift = any ? a.lse[row] : 0.0f, m = 0.0f;
    if (!(fabsf(shift) < kFarLse)) {
      const Run r = block_join<kDt>(run_span<T, kDt>(z, 0, a.V, kLog2e * inv_tau), kLog2e * inv_tau, red);
      m = r.m;
      shift = logf(r.s);
    }
    // ---- the used words of this split: their logits, before anything is written
    constexpr int KPT = kDistillMaxTop / kDt;  // places per thread
    float pv[KPT];
#pragma unroll
    for (int u = 0; u < KPT; ++u) {
      const int k = threadIdx.x + u * kDt;
      pv[u] = 0.f;
      if (any && k < K && ids[k] >= v0 && ids[k] < v1) pv[u] = to_f32(z[ids[k]]);
    }
    __syncthreads();  // every logit of a used word is read
    // ---- p_j f over the split
    auto p_of = [&](float zz) {
      return any ? f * exp2_hw(__builtin_fmaf(zz - m, inv_tau, -shift) * kLog2e) : 0.0f;
    };
    const Span<T> sn(z, v0, v1);
    auto put1 = [&](int64_t j, float v) {
      if constexpr (P == 8)
        g[j].u = f32_to_bf16(v);
      else
        g[j] = v;
    };
    {
      const int64_t j = v0 + threadIdx.x;
      if (j < sn.head) put1(j, p_of(to_f32(z[j])));
      const int64_t jt = sn.tail0 + threadIdx.x;
      if (jt < v1) put1(jt, p_of(to_f32(z[jt])));
    }
    const u32x4* vz = reinterpret_cast<const u32x4*>(z + sn.head);
    // grad and logits share their misalignment (checked on the host), so these are aligned too
    u32x4* vg = reinterpret_cast<u32x4*>(g + sn.head);
    auto vec = [&](u32x4 raw) {
      float v[P];
      unpack16<P>(raw, v);
#pragma unroll
      for (int e = 0; e < P; ++e) v[e] = p_of(v[e]);
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
    if (any) {
      // eight vectors in flight per thread, past the caches both ways (4096 x 50257 bf16: 186 us with four,
      // 182 with eight, 170 without caching)
      constexpr int U = 8;
      int64_t i = threadIdx.x;
      for (; i + (U - 1) * kDt < sn.vecs; i += U * kDt) {
        u32x4 raw[U];
#pragma unroll
        for (int u = 0; u < U; ++u) raw[u] = __builtin_nontemporal_load(vz + i + u * kDt);
#pragma unroll
        for (int u = 0; u < U; ++u) __builtin_nontemporal_store(vec(raw[u]), vg + i + u * kDt);
      }
      for (; i < sn.vecs; i += kDt) vg[i] = vec(vz[i]);
    } else {
      for (int64_t i = threadIdx.x; i < sn.vecs; i += kDt) vg[i] = u32x4{0u, 0u, 0u, 0u};
    }
    __syncthreads();  // every p_j f of the split is written
    if (any) {
#pragma unroll
      for (int u = 0; u < KPT; ++u) {
        const int k = threadIdx.x + u * kDt;
        if (k >= K) break;
        const int32_t w = ids[k];
        if (w < v0 || w >= v1) continue;
        // q of the word, over every place that names it; the first such place writes it
        float q = 0.f;
        bool first = true;
        for (int i = 0; i < K4; ++i) {
          const int4 o = *reinterpret_cast<const int4*>(ids + 4 * i);
          const float4 e = *reinterpret_cast<const float4*>(qs + 4 * i);
          if (o.x == w) { q += e.x; first = first && 4 * i >= k; }
          if (o.y == w) { q += e.y; first = first && 4 * i + 1 >= k; }
          if (o.z == w) { q += e.z; first = first && 4 * i + 2 >= k; }
          if (o.w == w) { q += e.w; first = first && 4 * i + 3 >= k; }
        }
        if (first) put1(w, p_of(pv[u]) - f * (q * inv_total));
      }
    }
    __syncthreads();  // ids and qs are reused by the next item
  }
}

// Splits of a token's words in the backward pass: none from 512 tokens on (two blocks per CU stream
// HBM at its rate); below, as many as give about 1024 blocks, each of at
// least 2048 words (8 per thread).
static int64_t distill_splits(int64_t rows, int64_t V) {
  if (rows >= 512) return 1;
  const int64_t want = (1024 + rows - 1) / rows, most = (V + 2047) / 2048;
  return std::max<int64_t>(1, std::min(want, most));
}

hipError_t launch_distill_loss(hipStream_t st, int dtype, DistillArgs a) {
  const int64_t rows = a.B * a.T;
  const unsigned blocks = (unsigned)std::min<int64_t>(rows, 1 << 20);
  // Up to a token per CU 1024 threads for it, up to two 512 (a CU holds one workgroup of 1024: 300 tokens of
  // 50257 bf16 take 15.3 us with 1024 threads, 10.2 with 512). Rows split over several workgroups with a second
  // launch that joins them took longer: 4 tokens 12.0 us a call against 9.0, 300 tokens 14.1.
  auto run = [&](auto nt) {
    constexpr int NT = decltype(nt)::value;
    if (dtype == 1) k_distill_loss<bf16s, NT><<<blocks, NT, 0, st>>>(a);
    else k_distill_loss<float, NT><<<blocks, NT, 0, st>>>(a);
  };
  if (rows <= 256) run(std::integral_constant<int, 1024>{});
  else if (rows <= 512) run(std::integral_constant<int, 512>{});
  else run(std::integral_constant<int, kDt>{});
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || a.T == 1) return e;
  k_distill_sum<<<(unsigned)std::min<int64_t>(a.B, 1 << 20), kDt, 0, st>>>(a.row_loss, a.B, a.T, a.loss);
  return hipGetLastError();
}

hipError_t launch_distill_backward(hipStream_t st, int dtype, DistillArgs a) {
  const int64_t rows = a.B * a.T;
  // in place a row is one block's: it may be read a second time, before anything of it is overwritten
  a.splits = a.grad == a.logits ? 1 : distill_splits(rows, a.V);
  const unsigned blocks = (unsigned)std::min<int64_t>(rows * a.splits, 1 << 20);
  if (dtype == 1)
    k_distill_backward<bf16s><<<blocks, kDt, 0, st>>>(a);
  else
    k_distill_backward<float><<<blocks, kDt, 0, st>>>(a);
  return hipGetLastError();
}

}  // namespace dpk
