// Products grouped by expert, and the clipping pass of expert layers.
//
// Rows are sorted by expert and, within an expert, by sample; seg[e*B + b] ..
// seg[e*B + b + 1] are the rows of sample b in expert e (device memory: the
// sizes are known only there, and no call reads them back). Per expert
//   product      Y_r = W_e x_r,  dX_r = W_e^T dy_r          (W_e [p, d])
//   norm         n_b^2 = sum_e || sum_{r in (e,b)} a_r g_r^T ||_F^2
//                      = sum_e sum_{r,r' in (e,b)} (a_r . a_r') (g_r . g_r')
//   clipped sum  out_e = (sum_b c_b sum_{r in (e,b)} a_r g_r^T + sigma C z) / denom
// all on MFMA 32x32 blocks with fp32 accumulators.
//
// Ragged sizes without a host round trip: tile t of group g (an expert, or an
// (expert, sample) segment) of rows [off_g, end_g) takes slot
// off_g / TS + g + t. Slots are unique, since off_g / TS + g + ceil(rows / TS)
// <= end_g / TS + g + 1, and there are at most R / TS + groups of them, so the
// host sizes the grid from R alone and a workgroup finds its group from the
// offsets by a 64-way search, one load per round.
#include "dp_common.hpp"
#include "dp_lds.hpp"
#include "dp_lm.hpp"
#include "dp_noise.hpp"

namespace dpk {

namespace {

__device__ __forceinline__ int64_t clamp_row(int64_t v, int64_t R) { return v < 0 ? 0 : v > R ? R : v; }

// The group whose slots hold `slot`: the last g with off_g / TS + g <= slot.
// Every lane of the wave takes part and gets the same answer. Offsets are
// clamped to [0, R], so that wrong ones cannot lead outside the rows.
struct Group {
  int64_t g, row0, rows;  // group, first row and row count of the slot's tile run to the group's end
  int64_t tile;           // tile index within the group
};
template <int TS>
__device__ __forceinline__ bool find_group(const int64_t* __restrict__ seg, int64_t stride, int64_t n, int64_t R,
                                           int64_t slot, Group* out) {
  const int lane = threadIdx.x & 63;
  int64_t lo = 0, len = n;
  while (true) {
    const int64_t step = (len + 63) / 64;
    const int64_t g = lo + lane * step;
    bool le = false;
    if (lane * step < len) le = clamp_row(seg[g * stride], R) / TS + g <= slot;
    const int cnt = __popcll(__ballot(le));
    if (cnt == 0) return false;
    lo += (cnt - 1) * step;
    if (step == 1) break;
    const int64_t left = len - (cnt - 1) * step;
    len = left < step ? left : step;
  }
  const int64_t off = clamp_row(seg[lo * stride], R), end = clamp_row(seg[(lo + 1) * stride], R);
  const int64_t t = slot - (off / TS + lo);
  out->g = lo;
  out->tile = t;
  out->row0 = off + t * TS;
  out->rows = end - out->row0;
  return out->rows > 0;
}

__device__ __forceinline__ int64_t uniform64(int64_t v) {
  const uint32_t lo = (uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)(uint64_t)v);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)((uint64_t)v >> 32));
  return (int64_t)(((uint64_t)hi << 32) | lo);
}

// ---- operand tiles in LDS
//
// A chunk is 128 bytes of K per feature: 64 bf16 or 32 fp32. KCONT operands
// hold K along their rows: LDS rows are features, 128 bytes each. The others
// hold features along their rows: LDS rows are the chunk's K rows. Both are
// windows of a row-major matrix, stored in 16-byte pieces; piece q of LDS row
// r sits at position q ^ swz(r), which puts every fragment read on 64
// distinct banks.
template <typename T, bool KCONT, int NF>
struct Opnd {
  static constexpr int SZ = sizeof(T);
  static constexpr int P = elem_traits<T>::per16;
  static constexpr int KC = 128 / SZ;               // K per chunk
  static constexpr int ROWB = KCONT ? 128 : NF * SZ;  // LDS row bytes
  static constexpr int NROWS = KCONT ? NF : KC;
  static constexpr int BYTES = NF * 128;
  static constexpr int PIECES = ROWB / 16;
  static __device__ __forceinline__ int swz(int r) {
    if constexpr (KCONT) return (r >> 1) & 7;
    else if constexpr (SZ == 2) return 4 * (r & 3);
    else return 8 * ((r >> 2) & 1);
  }
  static_assert(KCONT || PIECES % 16 == 0, "the swizzle stays inside a row");
};

// A window's position: base of its first element, row length in bytes, valid
// rows and valid columns from there on.
template <typename T>
struct Win {
  const T* base;
  int64_t ldb;   // bytes from row to row
  int64_t rows;  // valid rows
  int64_t cols;  // valid columns (elements)
};

// 16 bytes per lane from a buffer straight into LDS; lanes whose offset lies
// at or past num_records write zeros.
__device__ __forceinline__ void dma16_buf(u32x4 srd, uint32_t voff, uint32_t lds_base) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tbuffer_load_dwordx4 %0, %1, 0 offen lds" ::"v"(voff), "s"(srd),
               "s"(lds_base)
               : "memory", "m0");
}

template <typename T>
__device__ __forceinline__ u32x4 make_srd(const T* base, uint32_t bytes) {
  const uint64_t a = reinterpret_cast<uint64_t>(base);
  u32x4 s;
  s[0] = (uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)a);
  s[1] = (uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)(a >> 32) & 0xFFFFu);
  s[2] = (uint32_t)__builtin_amdgcn_readfirstlane(bytes);
  s[3] = 0x00020000u;  // raw buffer, 32-bit data
  return s;
}

// Filling one operand's LDS image of a window with NW waves.
template <typename O, typename T, int NW>
struct Filler {
  static constexpr int LOADS = O::BYTES / (1024 * NW);
  static_assert(LOADS * 1024 * NW == O::BYTES, "whole 1 KB loads per wave");
  uint32_t voff[LOADS];
  int qp[LOADS];  // first column of the lane's piece within the window
  __device__ __forceinline__ void init(int64_t ldb, int wave, int lane) {
#pragma unroll
    for (int i = 0; i < LOADS; ++i) {
      const int byte = (wave + NW * i) * 1024 + 16 * lane;
      const int r = byte / O::ROWB, q = ((byte % O::ROWB) / 16) ^ O::swz(r);
      voff[i] = (uint32_t)(r * ldb + 16 * q);
      qp[i] = q * O::P;
    }
  }
  // asynchronous: the caller waits for LOADS more vector-memory operations
  __device__ __forceinline__ void dma(const Win<T>& w, uint32_t lds, int wave) const {
    const int64_t rows = w.rows < O::NROWS ? w.rows : O::NROWS;
    // the window's bytes: its last row ends at its last valid column
    const uint32_t bytes = rows > 0 && w.cols > 0 ? (uint32_t)((rows - 1) * w.ldb + w.cols * O::SZ) : 0u;
    const u32x4 srd = make_srd(w.base, bytes);
    const int cols = (int)(w.cols < (1 << 30) ? w.cols : (1 << 30));
#pragma unroll
    for (int i = 0; i < LOADS; ++i)
      dma16_buf(srd, qp[i] < cols ? voff[i] : 0x80000000u, lds + (wave + NW * i) * 1024);
  }
  // through registers, element by element where needed: any alignment
  __device__ __forceinline__ void regs(const Win<T>& w, unsigned char* lds, int wave, int lane) const {
#pragma unroll
    for (int i = 0; i < LOADS; ++i) {
      const int byte = (wave + NW * i) * 1024 + 16 * lane;
      const int r = byte / O::ROWB;
      uint32_t v[4] = {0u, 0u, 0u, 0u};
      if (r < w.rows) {
        const T* src = reinterpret_cast<const T*>(reinterpret_cast<const char*>(w.base) + (int64_t)r * w.ldb);
#pragma unroll
        for (int e = 0; e < O::P; ++e) {
          uint32_t bits = 0u;
          if (qp[i] + e < w.cols) bits = raw_bits(src[qp[i] + e]);
          if constexpr (O::P == 8) v[e >> 1] |= bits << (16 * (e & 1));
          else v[e] = bits;
        }
      }
      *reinterpret_cast<u32x4*>(lds + byte) = u32x4{v[0], v[1], v[2], v[3]};
    }
  }
};

// Reading MFMA fragments: a step is 32 bytes of K per feature (16 bf16: one
// MFMA; 8 fp32: four of K = 2). Lane l holds feature l % 32 of each 32-block;
// its 16 bytes are K piece 2*step + l/32.
template <typename T, int NF, int NB>
struct ReadK {  // KCONT
  using O = Opnd<T, true, NF>;
  int off[4];
  __device__ __forceinline__ void init(int w0, int lane) {
#pragma unroll
    for (int s = 0; s < 4; ++s)
      off[s] = (w0 + (lane & 31)) * 128 + 16 * ((2 * s + (lane >> 5)) ^ (((lane & 31) >> 1) & 7));
  }
  __device__ __forceinline__ u32x4 get(uint32_t sbase, int s, int blk) const {
    return *(lds_u32x4*)(uintptr_t)(sbase + off[s] + blk * 4096);
  }
};
template <typename T, int NF, int NB>
struct ReadF {  // features along the rows
  using O = Opnd<T, false, NF>;
  int off[NB];
  __device__ __forceinline__ void init(int w0, int lane) {
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      if constexpr (sizeof(T) == 2) {
        // transposing reads: within a 16-lane group the lane at row k0 + (l % 16) / 4 supplies four features
        const int s = lane & 15, lo = 2 * ((lane >> 4) & 1) + ((s & 3) >> 1);
        const int piece0 = (w0 + b * 32) / 8;
        off[b] = (8 * (lane >> 5) + (s >> 2)) * O::ROWB + 16 * ((piece0 ^ (4 * (s >> 2))) + lo) + 8 * (s & 1);
      } else {
        const int g = lane >> 5, f = w0 + b * 32 + (lane & 31);
        off[b] = 4 * g * O::ROWB + 4 * (f ^ (32 * g));
      }
    }
  }
  __device__ __forceinline__ u32x4 get(uint32_t sbase, int s, int blk) const {
    if constexpr (sizeof(T) == 2) {
      const uint32_t a = sbase + off[blk] + s * 16 * O::ROWB;
      const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(uintptr_t)a);
      const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(uintptr_t)(a + 4 * O::ROWB));
      u32x4 r;
      r[0] = (uint32_t)(uint16_t)lo[0] | ((uint32_t)(uint16_t)lo[1] << 16);
      r[1] = (uint32_t)(uint16_t)lo[2] | ((uint32_t)(uint16_t)lo[3] << 16);
      r[2] = (uint32_t)(uint16_t)hi[0] | ((uint32_t)(uint16_t)hi[1] << 16);
      r[3] = (uint32_t)(uint16_t)hi[2] | ((uint32_t)(uint16_t)hi[3] << 16);
      return r;
    } else {
      typedef __attribute__((address_space(3))) uint32_t lds_u32;
      const uint32_t a = sbase + off[blk] + s * 8 * O::ROWB;
      u32x4 r;
#pragma unroll
      for (int e = 0; e < 4; ++e) r[e] = *(lds_u32*)(uintptr_t)(a + e * O::ROWB);
      return r;
    }
  }
};
template <typename T, bool KCONT, int NF, int NB>
using ReadOf = std::conditional_t<KCONT, ReadK<T, NF, NB>, ReadF<T, NF, NB>>;

template <typename T>
__device__ __forceinline__ f32x16 mma_step(u32x4 a, u32x4 b, f32x16 c) {
  if constexpr (sizeof(T) == 2) {
    return mfma32_bf16(a, b, c);
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) c = mfma32_f32(__uint_as_float(a[e]), __uint_as_float(b[e]), c);
    return c;
  }
}

template <int NBM, int NBN>
__device__ __forceinline__ void zero_acc(f32x16 (&acc)[NBM][NBN]) {
#pragma unroll
  for (int i = 0; i < NBM; ++i)
#pragma unroll
    for (int j = 0; j < NBN; ++j)
#pragma unroll
      for (int k = 0; k < 16; ++k) acc[i][j][k] = 0.f;
}

// Workgroup id -> work item such that each of the 8 XCDs (id % 8) takes a
// contiguous range of the items, whose operand tiles then share its L2.
__device__ __forceinline__ int64_t xcd_item(int64_t bid, int64_t items) {
  const int64_t per = (items + 7) / 8;
  return (bid & 7) * per + (bid >> 3);
}
int64_t xcd_grid(int64_t items) { return (items + 7) / 8 * 8; }

// One chunk's MFMAs: acc[i][j] += (a block i) x (b block j).
template <typename T, int NBA, int NBB, typename RA, typename RB>
__device__ __forceinline__ void chunk_mma(uint32_t sa, uint32_t sb, const RA& ra, const RB& rb, int steps,
                                          f32x16 (&acc)[NBA][NBB]) {
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    if (s >= steps) break;
    u32x4 fa[NBA], fb[NBB];
#pragma unroll
    for (int i = 0; i < NBA; ++i) fa[i] = ra.get(sa, s, i);
#pragma unroll
    for (int j = 0; j < NBB; ++j) fb[j] = rb.get(sb, s, j);
#pragma unroll
    for (int i = 0; i < NBA; ++i)
#pragma unroll
      for (int j = 0; j < NBB; ++j) acc[i][j] = mma_step<T>(fa[i], fb[j], acc[i][j]);
  }
}

}  // namespace

// ---------------------------------------------------------------------------
// Products: Y [R, N] = X [R, K] * op(W_e), op(W) [K, N]; W_e is [N, K] (TRANS
// false: K along its rows) or [K, N] (TRANS true).
//
// The weight is the MFMA's first operand, so an accumulator lane holds four
// consecutive columns of one row of Y and stores them together.
struct MatmulArgs {
  const void *X, *W;
  void* Y;
  const int64_t* seg;
  int64_t B, E, R, K, N;
  int64_t slots;  // R / BM + E
  int64_t ntn;    // column tiles
};

constexpr int64_t kSlotGroup = 4;  // row tiles that neighbouring workgroups share a weight tile over

template <typename T, bool TRANS, int BM, int BN, int WGM, int WGN, int ST, bool DMA>
__global__ __launch_bounds__(64 * WGM * WGN) void k_grouped_matmul(MatmulArgs a) {
  constexpr int NW = WGM * WGN, WM = BM / WGM, WN = BN / WGN, NBM = WM / 32, NBN = WN / 32;
  using OX = Opnd<T, true, BM>;
  using OW = Opnd<T, !TRANS, BN>;
  constexpr int KC = OX::KC, STAGE = OX::BYTES + OW::BYTES;
  extern __shared__ __attribute__((aligned(1024))) unsigned char lds[];

  const int64_t items = a.slots * a.ntn;
  const int64_t w = xcd_item(blockIdx.x, items);
  if (w >= items) return;
  const int64_t sg = w / (kSlotGroup * a.ntn), rem = w - sg * kSlotGroup * a.ntn;
  const int64_t in_group = a.slots - sg * kSlotGroup < kSlotGroup ? a.slots - sg * kSlotGroup : kSlotGroup;
  const int64_t tn = rem / in_group, slot = sg * kSlotGroup + (rem - tn * in_group);
  Group gr;
  if (!find_group<BM>(a.seg, a.B, a.E, a.R, slot, &gr)) return;  // whole workgroup
  const int64_t row0 = uniform64(gr.row0), rows = uniform64(gr.rows), e = uniform64(gr.g);
  const int64_t n0 = tn * BN;

  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave % WGM, wn = wave / WGM;
  const T* X = static_cast<const T*>(a.X) + row0 * a.K;
  const T* W = static_cast<const T*>(a.W) + e * a.K * a.N + (TRANS ? n0 : n0 * a.K);
  const int64_t xb = a.K * (int64_t)sizeof(T), wb = (TRANS ? a.N : a.K) * (int64_t)sizeof(T);
  const int64_t mrows = rows < BM ? rows : BM;

  Filler<OX, T, NW> fx;
  Filler<OW, T, NW> fw;
  fx.init(xb, wave, lane);
  fw.init(wb, wave, lane);
  ReadOf<T, true, BM, NBM> rx;
  ReadOf<T, !TRANS, BN, NBN> rw;
  rx.init(wm * WM, lane);
  rw.init(wn * WN, lane);
  auto xwin = [&](int64_t k0) { return Win<T>{X + k0, xb, mrows, a.K - k0}; };
  auto wwin = [&](int64_t k0) {
    return TRANS ? Win<T>{W + k0 * a.N, wb, a.K - k0, a.N - n0} : Win<T>{W + k0, wb, a.N - n0, a.K - k0};
  };

  f32x16 acc[NBN][NBM];
  zero_acc(acc);
  const int nq = (int)((a.K + KC - 1) / KC);
  const uint32_t l0 = lds_addr(lds);
  auto issue = [&](int q) {
    const uint32_t sb = l0 + (uint32_t)(q % ST) * STAGE;
    fx.dma(xwin((int64_t)q * KC), sb, wave);
    fw.dma(wwin((int64_t)q * KC), sb + OX::BYTES, wave);
  };
  if constexpr (DMA) {
    constexpr int LPC = Filler<OX, T, NW>::LOADS + Filler<OW, T, NW>::LOADS;
#pragma unroll
    for (int q = 0; q < ST - 1; ++q)
      if (q < nq) issue(q);
    for (int q = 0; q < nq; ++q) {
      const int later = nq - 1 - q < ST - 2 ? nq - 1 - q : ST - 2;
      wait_chunks<LPC, ST - 2>(later);
      lds_barrier();  // chunk q landed for every wave; every wave is done with chunk q-1
      if (q + ST - 1 < nq) issue(q + ST - 1);
      const uint32_t sb = l0 + (uint32_t)(q % ST) * STAGE;
      chunk_mma<T, NBN, NBM>(sb + OX::BYTES, sb, rw, rx, 4, acc);
    }
  } else {
    for (int q = 0; q < nq; ++q) {
      __syncthreads();
      fx.regs(xwin((int64_t)q * KC), lds, wave, lane);
      fw.regs(wwin((int64_t)q * KC), lds + OX::BYTES, wave, lane);
      __syncthreads();
      chunk_mma<T, NBN, NBM>(l0 + OX::BYTES, l0, rw, rx, 4, acc);
    }
  }

  // ---- rows of Y: lane l holds row l % 32 of each row block, columns in fours
  T* Y = static_cast<T*>(a.Y);
  const bool vec = a.N % 4 == 0 && (reinterpret_cast<uintptr_t>(Y) & (4 * sizeof(T) - 1)) == 0;
#pragma unroll
  for (int i = 0; i < NBM; ++i) {
    const int64_t m = wm * WM + i * 32 + (lane & 31);
    if (m >= mrows) continue;
    T* yr = Y + (row0 + m) * a.N;
#pragma unroll
    for (int j = 0; j < NBN; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int64_t n = n0 + wn * WN + j * 32 + 8 * q + 4 * (lane >> 5);
        const f32x16& c = acc[j][i];
        if (vec) {
          if (n >= a.N) continue;
          if constexpr (sizeof(T) == 2)
            *reinterpret_cast<uint2*>(yr + n) = make_uint2(pack_bf16(c[4 * q], c[4 * q + 1]),
                                                           pack_bf16(c[4 * q + 2], c[4 * q + 3]));
          else
            *reinterpret_cast<float4*>(yr + n) = make_float4(c[4 * q], c[4 * q + 1], c[4 * q + 2], c[4 * q + 3]);
        } else {
#pragma unroll
          for (int r = 0; r < 4; ++r)
            if (n + r < a.N) {
              if constexpr (sizeof(T) == 2) yr[n + r].u = f32_to_bf16(c[4 * q + r]);
              else yr[n + r] = c[4 * q + r];
            }
        }
      }
  }
}

// ---------------------------------------------------------------------------
// Norms: one workgroup per (segment, row tile of TS rows); it takes the Gram
// tiles (t, u), u >= t, of its segment in turn: both Grams' 32x32 blocks in
// registers, their elementwise product summed, counted twice off the
// diagonal. The tile's value goes to partial[slot].
struct GNormArgs {
  const void *A, *G;
  const int64_t* seg;
  int64_t R, E, B, d, p;
  float* partial;  // [slots]
  int64_t slots;   // R / TS + E * B
};

template <typename T, int TS, int WG, bool DMA>
__global__ __launch_bounds__(64 * WG * WG) void k_grouped_norm(GNormArgs a) {
  constexpr int NW = WG * WG, WT = TS / WG, NB = WT / 32;
  using O = Opnd<T, true, TS>;
  constexpr int KC = O::KC, STAGE = 2 * O::BYTES, ST = 2;
  extern __shared__ __attribute__((aligned(1024))) unsigned char lds[];
  __shared__ float red[NW];

  const int64_t slot = xcd_item(blockIdx.x, a.slots);
  if (slot >= a.slots) return;
  Group gr;
  if (!find_group<TS>(a.seg, 1, a.E * a.B, a.R, slot, &gr)) return;  // an unused slot: nothing reads its partial
  const int64_t row0 = uniform64(gr.row0), rows = uniform64(gr.rows);
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave % WG, wn = wave / WG;
  const uint32_t l0 = lds_addr(lds);
  ReadK<T, TS, NB> rm, rn;
  rm.init(wm * WT, lane);
  rn.init(wn * WT, lane);

  const int64_t trows = rows < TS ? rows : TS;
  float total = 0.f;
  for (int64_t u = 0; u * TS < rows; ++u) {
    const int64_t urows = rows - u * TS < TS ? rows - u * TS : TS;
    const bool diag = u == 0;
    f32x16 ga[NB][NB], gg[NB][NB];
    zero_acc(ga);
    zero_acc(gg);
    auto gram = [&](const T* M, int64_t K, f32x16 (&acc)[NB][NB]) {
      const T* Mt = M + row0 * K;
      const T* Mu = M + (row0 + u * TS) * K;
      const int64_t kb = K * (int64_t)sizeof(T);
      Filler<O, T, NW> f;
      f.init(kb, wave, lane);
      const int nq = (int)((K + KC - 1) / KC);
      auto wt = [&](int q) { return Win<T>{Mt + (int64_t)q * KC, kb, trows, K - (int64_t)q * KC}; };
      auto wu = [&](int q) { return Win<T>{Mu + (int64_t)q * KC, kb, urows, K - (int64_t)q * KC}; };
      if constexpr (DMA) {
        auto issue = [&](int q) {
          const uint32_t sb = l0 + (uint32_t)(q % ST) * STAGE;
          f.dma(wt(q), sb, wave);
          if (!diag) f.dma(wu(q), sb + O::BYTES, wave);
        };
        lds_barrier();  // every wave is done with the stages of the previous Gram
        issue(0);
        for (int q = 0; q < nq; ++q) {
          wait_vmcnt<0>();
          lds_barrier();
          if (q + 1 < nq) issue(q + 1);
          const uint32_t sb = l0 + (uint32_t)(q % ST) * STAGE;
          chunk_mma<T, NB, NB>(sb, diag ? sb : sb + O::BYTES, rm, rn, 4, acc);
        }
      } else {
        for (int q = 0; q < nq; ++q) {
          __syncthreads();
          f.regs(wt(q), lds, wave, lane);
          if (!diag) f.regs(wu(q), lds + O::BYTES, wave, lane);
          __syncthreads();
          chunk_mma<T, NB, NB>(l0, diag ? l0 : l0 + O::BYTES, rm, rn, 4, acc);
        }
      }
    };
    gram(static_cast<const T*>(a.A), a.d, ga);
    gram(static_cast<const T*>(a.G), a.p, gg);
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < NB; ++i)
#pragma unroll
      for (int j = 0; j < NB; ++j)
#pragma unroll
        for (int k = 0; k < 16; ++k) s = __builtin_fmaf(ga[i][j][k], gg[i][j][k], s);
    total += diag ? s : 2.0f * s;
  }
  total = wave_sum(total);
  if (lane == 0) red[wave] = total;
  __syncthreads();
  if (threadIdx.x == 0) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < NW; ++i) s += red[i];
    a.partial[slot] = s;
  }
}

// sqnorm[b] (+)= the values of the sample's tiles, in tile order per
// segment, one lane per segment, the segments joined in a fixed order. One
// wave per sample.
template <int TS>
__global__ __launch_bounds__(64) void k_grouped_norm_finish(GNormArgs a, float* __restrict__ sqnorm, int accumulate) {
  for (int64_t b = blockIdx.x; b < a.B; b += gridDim.x) {
    float s = 0.f;
    for (int64_t e = threadIdx.x; e < a.E; e += 64) {
      const int64_t g = e * a.B + b;
      const int64_t off = clamp_row(a.seg[g], a.R), end = clamp_row(a.seg[g + 1], a.R);
      const int64_t base = off / TS + g;
      for (int64_t t = 0; off + t * TS < end; ++t) s += a.partial[base + t];
    }
    s = wave_sum(s);
    if (threadIdx.x == 0) sqnorm[b] = accumulate ? sqnorm[b] + s : s;
  }
}

// ---------------------------------------------------------------------------
// Clipped sums. A list of K pieces is formed first: piece t of segment g
// covers up to KC rows of one sample and carries its clip factor, at slot
// off_g / KC + g + t (rows = 0 where a slot is unused).
struct Piece {
  int32_t row0, rows;
  int32_t last;  // last piece of its segment
  float c;
};
struct GSumArgs {
  const void *A, *G;
  const int64_t* seg;
  const Piece* pieces;
  int64_t R, E, B, d, p;
  int64_t mt, nt, ks;
  float* ws;  // partials [ks][E*d][p]
};

template <int KC>
__global__ __launch_bounds__(256) void k_grouped_pieces(const int64_t* __restrict__ seg, int64_t R, int64_t E,
                                                        int64_t B, const float* __restrict__ c, int64_t slots,
                                                        Piece* __restrict__ out) {
  const int64_t slot = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (slot >= slots) return;
  // the last g with off_g / KC + g <= slot, by each thread on its own
  int64_t g = 0, hi = E * B;
  while (hi - g > 1) {
    const int64_t mid = (g + hi) / 2;
    if (clamp_row(seg[mid], R) / KC + mid <= slot) g = mid;
    else hi = mid;
  }
  const int64_t off = clamp_row(seg[g], R), end = clamp_row(seg[g + 1], R);
  const int64_t t = slot - (off / KC + g), row0 = off + t * KC;
  Piece pc{0, 0, 0, 0.f};
  if (t >= 0 && row0 < end) {
    pc.row0 = (int32_t)row0;
    pc.rows = (int32_t)(end - row0 < KC ? end - row0 : KC);
    pc.last = row0 + KC >= end;
    pc.c = c[g % B];
  }
  out[slot] = pc;
}

// One workgroup per (expert, tile of [d, p], split of the expert's pieces):
// every piece's product accumulates unscaled and is folded in as
// acc += c * tmp in fp32 at the end of its sample, so the clip factor is
// applied exactly.
template <typename T, int BM, int BN, int WGM, int WGN, int ST, bool DMA>
__global__ __launch_bounds__(64 * WGM * WGN) void k_grouped_sum(GSumArgs a) {
  constexpr int NW = WGM * WGN, WM = BM / WGM, WN = BN / WGN, NBM = WM / 32, NBN = WN / 32;
  using OA = Opnd<T, false, BM>;
  using OG = Opnd<T, false, BN>;
  constexpr int KC = OA::KC, STAGE = OA::BYTES + OG::BYTES;
  extern __shared__ __attribute__((aligned(1024))) unsigned char lds[];

  const int64_t tiles = a.mt * a.nt, items = a.E * tiles * a.ks;
  const int64_t w = xcd_item(blockIdx.x, items);
  if (w >= items) return;
  const int64_t sp = w / (a.E * tiles), r0 = w - sp * a.E * tiles;
  const int64_t e = r0 / tiles, t = r0 - e * tiles;
  const int64_t tm = t % a.mt, tn = t / a.mt;
  const int64_t m0 = tm * BM, n0 = tn * BN;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave % WGM, wn = wave / WGM;

  // this split's slots
  const int64_t g0 = e * a.B, g1 = (e + 1) * a.B;
  const int64_t o0 = uniform64(clamp_row(a.seg[g0], a.R)), o1 = uniform64(clamp_row(a.seg[g1], a.R));
  const int64_t s0 = o0 / KC + g0, s1 = o1 / KC + g1;
  const int64_t per = (s1 - s0 + a.ks - 1) / a.ks;
  const int64_t b0 = s0 + sp * per, b1 = b0 + per < s1 ? b0 + per : s1;

  const T* A = static_cast<const T*>(a.A) + m0;
  const T* G = static_cast<const T*>(a.G) + n0;
  const int64_t ab = a.d * (int64_t)sizeof(T), gb = a.p * (int64_t)sizeof(T);
  Filler<OA, T, NW> fa;
  Filler<OG, T, NW> fg;
  fa.init(ab, wave, lane);
  fg.init(gb, wave, lane);
  ReadF<T, BM, NBM> ra;
  ReadF<T, BN, NBN> rg;
  ra.init(wm * WM, lane);
  rg.init(wn * WN, lane);

  f32x16 acc[NBM][NBN], tmp[NBM][NBN];
  zero_acc(acc);
  zero_acc(tmp);
  const uint32_t l0 = lds_addr(lds);

  // The pieces in use, 64 slots at a time: lane i holds slot base + i. Two
  // walkers go over them, one for the loads and one for the products.
  struct Walk {
    int64_t base;
    uint64_t mask;
    Piece mine;
  };
  auto load64 = [&](Walk& wk) {
    wk.mine = Piece{0, 0, 0, 0.f};
    if (wk.base + lane < b1) wk.mine = a.pieces[wk.base + lane];
    wk.mask = __ballot(wk.mine.rows > 0);
  };
  auto next = [&](Walk& wk, Piece* pc) -> bool {
    while (wk.mask == 0) {
      wk.base += 64;
      if (wk.base >= b1) return false;
      load64(wk);
    }
    const int i = __ffsll((unsigned long long)wk.mask) - 1;
    wk.mask &= wk.mask - 1;
    pc->row0 = __builtin_amdgcn_readlane(wk.mine.row0, i);
    pc->rows = __builtin_amdgcn_readlane(wk.mine.rows, i);
    pc->last = __builtin_amdgcn_readlane(wk.mine.last, i);
    pc->c = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(wk.mine.c), i));
    return true;
  };
  auto awin = [&](const Piece& pc) { return Win<T>{A + pc.row0 * a.d, ab, pc.rows, a.d - m0}; };
  auto gwin = [&](const Piece& pc) { return Win<T>{G + pc.row0 * a.p, gb, pc.rows, a.p - n0}; };
  auto steps_of = [&](const Piece& pc) { return (pc.rows + KC / 4 - 1) / (KC / 4); };

  bool open = false;
  float cur = 0.f;
  auto fold = [&]() {
#pragma unroll
    for (int i = 0; i < NBM; ++i)
#pragma unroll
      for (int j = 0; j < NBN; ++j)
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          acc[i][j][k] = __builtin_fmaf(cur, tmp[i][j][k], acc[i][j][k]);
          tmp[i][j][k] = 0.f;
        }
    open = false;
  };
  if (b0 < b1) {
    Walk wl{b0, 0, {}};
    load64(wl);
    if constexpr (DMA) {
      static_assert(ST == 2, "one piece ahead");
      Piece cp, np;
      bool have = next(wl, &cp);
      int q = 0;
      if (have) {
        fa.dma(awin(cp), l0, wave);
        fg.dma(gwin(cp), l0 + OA::BYTES, wave);
      }
      while (have) {
        wait_vmcnt<0>();
        lds_barrier();
        const bool more = next(wl, &np);
        const uint32_t sb = l0 + (uint32_t)(q & 1) * STAGE, sn = l0 + (uint32_t)((q + 1) & 1) * STAGE;
        if (more) {
          fa.dma(awin(np), sn, wave);
          fg.dma(gwin(np), sn + OA::BYTES, wave);
        }
        chunk_mma<T, NBM, NBN>(sb, sb + OA::BYTES, ra, rg, steps_of(cp), tmp);
        cur = cp.c;
        open = true;
        if (cp.last) fold();
        cp = np;
        have = more;
        ++q;
      }
    } else {
      Piece cp;
      while (next(wl, &cp)) {
        __syncthreads();
        fa.regs(awin(cp), lds, wave, lane);
        fg.regs(gwin(cp), lds + OA::BYTES, wave, lane);
        __syncthreads();
        chunk_mma<T, NBM, NBN>(l0, l0 + OA::BYTES, ra, rg, steps_of(cp), tmp);
        cur = cp.c;
        open = true;
        if (cp.last) fold();
      }
    }
    if (open) fold();
  }

  float* out = a.ws + (sp * a.E + e) * a.d * a.p;
#pragma unroll
  for (int i = 0; i < NBM; ++i)
#pragma unroll
    for (int j = 0; j < NBN; ++j)
#pragma unroll
      for (int k = 0; k < 16; ++k) {
        const int64_t m = m0 + wm * WM + i * 32 + acc_row(k, lane), n = n0 + wn * WN + j * 32 + acc_col(lane);
        if (m < a.d && n < a.p) out[m * a.p + n] = acc[i][j][k];
      }
}

// ---------------------------------------------------------------------------
namespace {

bool dma_ok(int dtype, std::initializer_list<int64_t> widths) {
  for (int64_t v : widths)
    if (v % (dtype == 1 ? 8 : 4)) return false;
  return true;
}

template <typename F>
hipError_t dyn_lds(F* f, int bytes) {
  return hipFuncSetAttribute(reinterpret_cast<const void*>(f), hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
}

template <typename T, bool TRANS, int BM, int BN, int WGM, int WGN, int ST, bool DMA>
hipError_t run_matmul(hipStream_t st, MatmulArgs a) {
  auto* f = &k_grouped_matmul<T, TRANS, BM, BN, WGM, WGN, ST, DMA>;
  constexpr int LDS = (DMA ? ST : 1) * (BM + BN) * 128;
  a.slots = a.R / BM + a.E;
  a.ntn = (a.N + BN - 1) / BN;
  hipError_t e = dyn_lds(f, LDS);
  if (e != hipSuccess) return e;
  f<<<dim3((unsigned)xcd_grid(a.slots * a.ntn)), 64 * WGM * WGN, LDS, st>>>(a);
  return hipGetLastError();
}

template <typename T, bool TRANS>
hipError_t matmul_t(hipStream_t st, int dtype, const MatmulArgs& a) {
  const bool dma = dma_ok(dtype, {a.K, a.N});
  if (!dma) return run_matmul<T, TRANS, 128, 128, 2, 2, 2, false>(st, a);
  return run_matmul<T, TRANS, 128, 128, 2, 2, 2, true>(st, a);
}

int64_t norm_slots(const GroupedArgs& g, int ts) { return g.R / ts + g.E * g.B; }
int64_t piece_rows(int dtype) { return dtype == 1 ? 64 : 32; }
int64_t piece_slots(int dtype, const GroupedArgs& g) { return g.R / piece_rows(dtype) + g.E * g.B; }
size_t round256(size_t x) { return (x + 255) / 256 * 256; }

int64_t sum_splits(int dtype, const GroupedArgs& g) {
  const int64_t tiles = ((g.d + 127) / 128) * ((g.p + 127) / 128) * g.E;
  const int64_t want = (512 + tiles - 1) / tiles;
  const int64_t most = std::max<int64_t>(1, g.R / g.E / 256);
  return std::max<int64_t>(1, std::min(want, most));
}

template <typename T, int TS, int WG>
hipError_t run_norm(hipStream_t st, int dtype, GNormArgs a, float* sqnorm, int accumulate) {
  a.slots = a.R / TS + a.E * a.B;
  const bool dma = dma_ok(dtype, {a.d, a.p});
  const int lds = (dma ? 2 : 1) * 2 * TS * 128;
  hipError_t e;
  if (dma) {
    auto* f = &k_grouped_norm<T, TS, WG, true>;
    e = dyn_lds(f, lds);
    if (e != hipSuccess) return e;
    f<<<dim3((unsigned)xcd_grid(a.slots)), 64 * WG * WG, lds, st>>>(a);
  } else {
    auto* f = &k_grouped_norm<T, TS, WG, false>;
    e = dyn_lds(f, lds);
    if (e != hipSuccess) return e;
    f<<<dim3((unsigned)xcd_grid(a.slots)), 64 * WG * WG, lds, st>>>(a);
  }
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  k_grouped_norm_finish<TS><<<dim3((unsigned)std::min<int64_t>(a.B, 1 << 20)), 64, 0, st>>>(a, sqnorm, accumulate);
  return hipGetLastError();
}

template <typename T, bool DMA>
hipError_t run_sum(hipStream_t st, const GSumArgs& a) {
  auto* f = &k_grouped_sum<T, 128, 128, 2, 2, 2, DMA>;
  constexpr int LDS = (DMA ? 2 : 1) * 256 * 128;
  hipError_t e = dyn_lds(f, LDS);
  if (e != hipSuccess) return e;
  f<<<dim3((unsigned)xcd_grid(a.E * a.mt * a.nt * a.ks)), 256, LDS, st>>>(a);
  return hipGetLastError();
}

}  // namespace

size_t grouped_matmul_ws_bytes(int, const GroupedArgs&) { return 0; }

hipError_t launch_grouped_matmul(hipStream_t st, int dtype, const GroupedArgs& g, const void* X, const void* W,
                                 bool transpose, void*, void* Y) {
  MatmulArgs a{};
  a.X = X;
  a.W = W;
  a.Y = Y;
  a.seg = g.seg;
  a.B = g.B;
  a.E = g.E;
  a.R = g.R;
  a.K = transpose ? g.p : g.d;
  a.N = transpose ? g.d : g.p;
  if (dtype == 1) return transpose ? matmul_t<bf16s, true>(st, dtype, a) : matmul_t<bf16s, false>(st, dtype, a);
  return transpose ? matmul_t<float, true>(st, dtype, a) : matmul_t<float, false>(st, dtype, a);
}

size_t grouped_norm_ws_bytes(int, const GroupedArgs& g) { return round256((size_t)norm_slots(g, 128) * sizeof(float)); }

hipError_t launch_grouped_norm(hipStream_t st, int dtype, const GroupedArgs& g, const void* A, const void* G, void* ws,
                               float* sqnorm, int accumulate) {
  GNormArgs a{};
  a.A = A;
  a.G = G;
  a.seg = g.seg;
  a.R = g.R;
  a.E = g.E;
  a.B = g.B;
  a.d = g.d;
  a.p = g.p;
  a.partial = static_cast<float*>(ws);
  return dtype == 1 ? run_norm<bf16s, 128, 2>(st, dtype, a, sqnorm, accumulate)
                    : run_norm<float, 128, 2>(st, dtype, a, sqnorm, accumulate);
}

size_t grouped_sum_ws_bytes(int dtype, const GroupedArgs& g) {
  return round256((size_t)piece_slots(dtype, g) * sizeof(Piece)) +
         round256((size_t)sum_splits(dtype, g) * (size_t)g.E * (size_t)g.d * (size_t)g.p * sizeof(float));
}

hipError_t launch_grouped_sum(hipStream_t st, int dtype, const GroupedArgs& g, const void* A, const void* G,
                              const float* c, void* ws, const NoiseArgs& na, float* out) {
  const int64_t slots = piece_slots(dtype, g);
  Piece* pieces = static_cast<Piece*>(ws);
  const unsigned pb = (unsigned)((slots + 255) / 256);
  if (dtype == 1)
    k_grouped_pieces<64><<<pb, 256, 0, st>>>(g.seg, g.R, g.E, g.B, c, slots, pieces);
  else
    k_grouped_pieces<32><<<pb, 256, 0, st>>>(g.seg, g.R, g.E, g.B, c, slots, pieces);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  GSumArgs a{};
  a.A = A;
  a.G = G;
  a.seg = g.seg;
  a.pieces = pieces;
  a.R = g.R;
  a.E = g.E;
  a.B = g.B;
  a.d = g.d;
  a.p = g.p;
  a.mt = (g.d + 127) / 128;
  a.nt = (g.p + 127) / 128;
  a.ks = sum_splits(dtype, g);
  a.ws = reinterpret_cast<float*>(static_cast<char*>(ws) + round256((size_t)slots * sizeof(Piece)));
  const bool dma = dma_ok(dtype, {g.d, g.p});
  if (dtype == 1)
    e = dma ? run_sum<bf16s, true>(st, a) : run_sum<bf16s, false>(st, a);
  else
    e = dma ? run_sum<float, true>(st, a) : run_sum<float, false>(st, a);
  if (e != hipSuccess) return e;
  return launch_split_reduce(st, a.ks, a.ws, g.E * g.d, g.p, na, out);
}

bool grouped_fits(int dtype, const GroupedArgs& g) {
  constexpr int64_t kMax = ((int64_t)1 << 32) / 512;
  const int64_t cols = (std::max(g.d, g.p) + 127) / 128;
  if ((g.R / 32 + g.E) * cols + 8 >= kMax) return false;
  if (g.R / 32 + g.E * g.B + 8 >= kMax) return false;
  return g.E * ((g.d + 127) / 128) * ((g.p + 127) / 128) * sum_splits(dtype, g) + 8 < kMax;
}

}  // namespace dpk
