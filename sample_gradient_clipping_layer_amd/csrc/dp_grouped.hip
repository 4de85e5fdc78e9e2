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

#include <cmath>

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
  return t >= 0 && out->rows > 0;  // t < 0 only where the offsets do not ascend
}

__device__ __forceinline__ int64_t uniform64(int64_t v) {
  const uint32_t lo = (uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)(uint64_t)v);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)((uint64_t)v >> 32));
  return (int64_t)(((uint64_t)hi << 32) | lo);
}

// ---- operand tiles in LDS
//
// A chunk is KB bytes of K per feature (128: 64 bf16 or 32 fp32). KCONT
// operands hold K along their rows: LDS rows are features, KB bytes each. The
// others hold features along their rows: LDS rows are the chunk's K rows.
// Both are windows of a row-major matrix, stored in 16-byte pieces; piece q of
// LDS row r sits at position q ^ swz(r), which puts every fragment read on 64
// distinct banks.
template <typename T, bool KCONT, int NF, int KB = 128>
struct Opnd {
  static constexpr int SZ = sizeof(T);
  static constexpr int P = elem_traits<T>::per16;
  static constexpr bool FEAT = !KCONT;               // features along the rows
  static constexpr int KC = KB / SZ;                 // K per chunk
  static constexpr int ROWB = KCONT ? KB : NF * SZ;  // LDS row bytes
  static constexpr int NROWS = KCONT ? NF : KC;
  static constexpr int BYTES = NF * KB;
  static constexpr int PIECES = ROWB / 16;
  static_assert(KB == 64 || KB == 128, "chunk depth");
  static __device__ __forceinline__ int swz(int r) {
    if constexpr (KCONT) return KB == 128 ? (r >> 1) & 7 : (r >> 2) & 3;
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
  int64_t over = 0;  // rows that may be read past their end: all but the matrix's last one
};

// Between a wave's LDS writes and its reads of what other lanes wrote (and
// before the next writes over it): in order in hardware, kept so by the compiler.
__device__ __forceinline__ void lds_wave_fence() { asm volatile("" ::: "memory"); }

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef __attribute__((address_space(3))) u32x2 lds_u32x2;

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

// 16 bytes of elements [col, col + P) of a row of K, zero past K and where !ok;
// rows of odd widths start at any element. `over`: 16 bytes there may be read,
// and what lies past K does no harm.
template <typename T>
__device__ __forceinline__ u32x4 load_piece(const T* __restrict__ row, int64_t col, int64_t K, bool ok,
                                            bool over = false) {
  constexpr int P = elem_traits<T>::per16;
  u32x4 v = {0u, 0u, 0u, 0u};
  if (!ok || col >= K) return v;
  if (over || col + P <= K) {
    __builtin_memcpy(&v, row + col, 16);
    return v;
  }
  uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
  for (int e = 0; e < P - 1; ++e)
    if (col + e < K) {
      const uint32_t bits = raw_bits(row[col + e]);
      if constexpr (P == 8) w[e >> 1] |= bits << (16 * (e & 1));
      else w[e] = bits;
    }
  return u32x4{w[0], w[1], w[2], w[3]};
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
  // Through registers (any alignment): load, and after the LDS image's readers are done, store. Features past
  // the width only reach products that are not stored, so a row's last piece is read whole where the matrix goes
  // on (element by element, with a wait for each, it held up every chunk of a tile at the edge).
  __device__ __forceinline__ void load(const Win<T>& w, u32x4 (&v)[LOADS], int wave, int lane) const {
    // a piece that starts in a row ends in the next one at the latest when rows have 16 bytes
    const int64_t over = O::FEAT && w.ldb >= 16 ? w.over : 0;
#pragma unroll
    for (int i = 0; i < LOADS; ++i) {
      const int r = ((wave + NW * i) * 1024 + 16 * lane) / O::ROWB;
      v[i] = load_piece(reinterpret_cast<const T*>(reinterpret_cast<const char*>(w.base) + (int64_t)r * w.ldb),
                        qp[i], w.cols, r < w.rows, r < over);
    }
  }
  __device__ __forceinline__ void store(const u32x4 (&v)[LOADS], unsigned char* lds, int wave, int lane) const {
#pragma unroll
    for (int i = 0; i < LOADS; ++i)
      *reinterpret_cast<u32x4*>(lds + (wave + NW * i) * 1024 + 16 * lane) = v[i];
  }
};

// Reading MFMA fragments: a step is 32 bytes of K per feature (16 bf16: one
// MFMA; 8 fp32: four of K = 2). Lane l holds feature l % 32 of each 32-block;
// its 16 bytes are K piece 2*step + l/32.
template <typename T, int NF, int NB, int KB = 128>
struct ReadK {  // KCONT
  using O = Opnd<T, true, NF, KB>;
  int off[KB / 32];
  __device__ __forceinline__ void init(int w0, int lane) {
#pragma unroll
    for (int s = 0; s < KB / 32; ++s)
      off[s] = (w0 + (lane & 31)) * KB + 16 * ((2 * s + (lane >> 5)) ^ O::swz(lane & 31));
  }
  __device__ __forceinline__ u32x4 get(uint32_t sbase, int s, int blk) const {
    return *(lds_u32x4*)(uintptr_t)(sbase + off[s] + blk * 32 * KB);
  }
};
template <typename T, int NF, int NB, int KB = 128>
struct ReadF {  // features along the rows
  using O = Opnd<T, false, NF, KB>;
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
template <typename T, bool KCONT, int NF, int NB, int KB>
using ReadOf = std::conditional_t<KCONT, ReadK<T, NF, NB, KB>, ReadF<T, NF, NB, KB>>;

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
//
// k_grouped_matmul: 128 x 128 tiles, and 32 x 128 ones for few rows, which are
// bound by the experts' weights (8 rows over 8 experts of 1280 x 5120 bf16:
// 16 us, 4.3 TB/s of the weights in use).
struct MatmulArgs {
  const void *X, *W;
  void* Y;
  const int64_t* seg;
  int64_t B, E, R, K, N;
  int64_t slots;  // R / BM + E
  int64_t ntn;    // column tiles
  int64_t ks;     // K splits
  int64_t kper;   // K per split, whole chunks
  float* part;    // ks > 1: partial products [ks][R][N]
};

constexpr int64_t kSlotGroup = 4;  // row tiles that neighbouring workgroups share a weight tile over

template <typename T, bool TRANS, int BM, int BN, int WGM, int WGN, int KB, int ST, bool DMA, bool SPLIT>
__global__ __launch_bounds__(64 * WGM * WGN) void k_grouped_matmul(MatmulArgs a) {
  constexpr int NW = WGM * WGN, WM = BM / WGM, WN = BN / WGN, NBM = WM / 32, NBN = WN / 32, NS = KB / 32;
  using OX = Opnd<T, true, BM, KB>;
  using OW = Opnd<T, !TRANS, BN, KB>;
  constexpr int KC = OX::KC, STAGE = OX::BYTES + OW::BYTES;
  extern __shared__ __attribute__((aligned(1024))) unsigned char lds[];

  const int64_t items = a.slots * a.ntn;
  int64_t w = xcd_item(blockIdx.x, items * a.ks);
  if (w >= items * a.ks) return;
  const int64_t sp = SPLIT ? w / items : 0;
  if (SPLIT) w -= sp * items;
  const int64_t sg = w / (kSlotGroup * a.ntn), rem = w - sg * kSlotGroup * a.ntn;
  const int64_t in_group = a.slots - sg * kSlotGroup < kSlotGroup ? a.slots - sg * kSlotGroup : kSlotGroup;
  const int64_t tn = rem / in_group, slot = sg * kSlotGroup + (rem - tn * in_group);
  Group gr;
  if (!find_group<BM>(a.seg, a.B, a.E, a.R, slot, &gr)) return;  // whole workgroup
  const int64_t row0 = uniform64(gr.row0), rows = uniform64(gr.rows), e = uniform64(gr.g);
  const int64_t n0 = tn * BN;
  const int64_t kb0 = SPLIT ? sp * a.kper : 0;
  const int64_t klen = SPLIT ? (a.K - kb0 < a.kper ? a.K - kb0 : a.kper) : a.K;  // > 0: checked on the host

  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave % WGM, wn = wave / WGM;
  const T* X = static_cast<const T*>(a.X) + row0 * a.K + kb0;
  const T* W = static_cast<const T*>(a.W) + e * a.K * a.N + (TRANS ? kb0 * a.N + n0 : n0 * a.K + kb0);
  const int64_t xb = a.K * (int64_t)sizeof(T), wb = (TRANS ? a.N : a.K) * (int64_t)sizeof(T);
  const int64_t mrows = rows < BM ? rows : BM;

  Filler<OX, T, NW> fx;
  Filler<OW, T, NW> fw;
  fx.init(xb, wave, lane);
  fw.init(wb, wave, lane);
  ReadOf<T, true, BM, NBM, KB> rx;
  ReadOf<T, !TRANS, BN, NBN, KB> rw;
  rx.init(wm * WM, lane);
  rw.init(wn * WN, lane);
  auto xwin = [&](int64_t k0) { return Win<T>{X + k0, xb, mrows, klen - k0}; };
  auto wwin = [&](int64_t k0) {
    return TRANS ? Win<T>{W + k0 * a.N, wb, klen - k0, a.N - n0, (a.E - e) * a.K - 1 - kb0 - k0} : Win<T>{W + k0, wb, a.N - n0, klen - k0};
  };

  f32x16 acc[NBN][NBM];
  zero_acc(acc);
  const int nq = (int)((klen + KC - 1) / KC);
  const uint32_t l0 = lds_addr(lds);
  struct Frags {
    u32x4 w[NBN], x[NBM];
  };
  auto read = [&](uint32_t sb, int s, Frags& f) {
#pragma unroll
    for (int j = 0; j < NBN; ++j) f.w[j] = rw.get(sb + OX::BYTES, s, j);
#pragma unroll
    for (int i = 0; i < NBM; ++i) f.x[i] = rx.get(sb, s, i);
  };
  auto mma = [&](const Frags& f) {
#pragma unroll
    for (int j = 0; j < NBN; ++j)
#pragma unroll
      for (int i = 0; i < NBM; ++i) acc[j][i] = mma_step<T>(f.w[j], f.x[i], acc[j][i]);
  };
  if constexpr (DMA) {
    constexpr int LPC = Filler<OX, T, NW>::LOADS + Filler<OW, T, NW>::LOADS;
    auto issue = [&](int q) {
      const uint32_t sb = l0 + (uint32_t)(q % ST) * STAGE;
      fx.dma(xwin((int64_t)q * KC), sb, wave);
      fw.dma(wwin((int64_t)q * KC), sb + OX::BYTES, wave);
    };
    auto stage_of = [&](int q) { return l0 + (uint32_t)(q % ST) * STAGE; };
    // chunk q landed for every wave, and every wave is done with chunk q - 1, whose stage takes chunk q + ST - 1
    auto arrive = [&](int q) {
      const int later = nq - 1 - q < ST - 2 ? nq - 1 - q : ST - 2;
      wait_chunks<LPC, ST - 2>(later);
      lds_barrier();
      if (q + ST - 1 < nq) issue(q + ST - 1);
    };
#pragma unroll
    for (int q = 0; q < ST - 1; ++q)
      if (q < nq) issue(q);
    // step s + 1's fragments are read while step s is on the matrix cores, across chunks too
    Frags f[2];
    arrive(0);
    read(stage_of(0), 0, f[0]);
    for (int q = 0; q + 1 < nq; ++q) {
#pragma unroll
      for (int s = 0; s < NS; ++s) {
        if (s + 1 < NS) {
          read(stage_of(q), s + 1, f[(s + 1) & 1]);
        } else {
          arrive(q + 1);
          read(stage_of(q + 1), 0, f[0]);
        }
        mma(f[s & 1]);
      }
    }
#pragma unroll
    for (int s = 0; s < NS; ++s) {
      if (s + 1 < NS) read(stage_of(nq - 1), s + 1, f[(s + 1) & 1]);
      mma(f[s & 1]);
    }
  } else {
    u32x4 vx[Filler<OX, T, NW>::LOADS], vw[Filler<OW, T, NW>::LOADS];
    fx.load(xwin(0), vx, wave, lane);
    fw.load(wwin(0), vw, wave, lane);
    for (int q = 0; q < nq; ++q) {
      __syncthreads();
      fx.store(vx, lds, wave, lane);
      fw.store(vw, lds + OX::BYTES, wave, lane);
      __syncthreads();
      fx.load(xwin((int64_t)(q + 1) * KC), vx, wave, lane);  // past the last chunk: an empty window
      fw.load(wwin((int64_t)(q + 1) * KC), vw, wave, lane);
#pragma unroll
      for (int s = 0; s < NS; ++s) {
        Frags f;
        read(l0, s, f);
        mma(f);
      }
    }
  }

  // ---- rows of Y: lane l holds row l % 32 of each row block, columns in fours
  using D = std::conditional_t<SPLIT, float, T>;
  D* Y = SPLIT ? reinterpret_cast<D*>(a.part) + sp * a.R * a.N : static_cast<D*>(a.Y);
  const bool vec = a.N % 4 == 0;
#pragma unroll
  for (int i = 0; i < NBM; ++i) {
    const int64_t m = wm * WM + i * 32 + (lane & 31);
    if (m >= mrows) continue;
    D* yr = Y + (row0 + m) * a.N;
#pragma unroll
    for (int j = 0; j < NBN; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int64_t n = n0 + wn * WN + j * 32 + 8 * q + 4 * (lane >> 5);
        const f32x16& c = acc[j][i];
        if (vec) {
          if (n >= a.N) continue;
          if constexpr (sizeof(D) == 2)
            *reinterpret_cast<uint2*>(yr + n) = make_uint2(pack_bf16(c[4 * q], c[4 * q + 1]),
                                                           pack_bf16(c[4 * q + 2], c[4 * q + 3]));
          else
            *reinterpret_cast<float4*>(yr + n) = make_float4(c[4 * q], c[4 * q + 1], c[4 * q + 2], c[4 * q + 3]);
        } else {
#pragma unroll
          for (int r = 0; r < 4; ++r)
            if (n + r < a.N) {
              if constexpr (sizeof(D) == 2) yr[n + r].u = f32_to_bf16(c[4 * q + r]);
              else yr[n + r] = c[4 * q + r];
            }
        }
      }
  }
}

// The 256 x 256 tile of bf16 products, for up to 64 experts: one workgroup per
// CU (128 KB of stages) that goes over its tiles in turn, as one stream of
// chunks. The loads run ST - 1 chunks ahead of the products, into the next
// tile where this one ends, so that neither the search for a tile nor its
// first loads stand alone; only the writing of a tile's rows does, with the
// next tile's loads in flight.
//
// Lane e of each wave holds expert e's row range and tile count, so a tile's
// expert is found without memory, and the tiles are numbered without gaps.
//
// 32768 rows over 8 experts, 1280 -> 5120: 430 us, 1.0 PFLOP/s. The matrix
// cores are busy 0.61 of the cycles, and the clock falls to 1.6 GHz. The
// products and their loop alone take 264 us; the LDS reads, each added alone,
// 110 more, the loads 95, the stores 50. 8192 rows over 16 experts, 5120 -> 1280: 130 us,
// 0.83 PFLOP/s, 200 tiles on the 256 CUs.
//
// Each wave writes its 64 x 128 part of the tile through 4 KB of LDS of its
// own (no barrier): 32 x 64 values at a time, 8-byte units swizzled by the
// row, read back as 16-byte pieces and stored 128 contiguous bytes per row.
template <bool TRANS>
__global__ __launch_bounds__(512) void k_grouped_matmul_big(MatmulArgs a) {
  using T = bf16s;
  constexpr int BM = 256, BN = 256, WGM = 4, WGN = 2, NW = WGM * WGN, WM = BM / WGM, WN = BN / WGN;
  constexpr int NBM = WM / 32, NBN = WN / 32, KB = 64, ST = 4;
  using OX = Opnd<T, true, BM, KB>;
  using OW = Opnd<T, !TRANS, BN, KB>;
  using FX = Filler<OX, T, NW>;
  using FW = Filler<OW, T, NW>;
  constexpr int KC = OX::KC, STAGE = OX::BYTES + OW::BYTES, LPC = FX::LOADS + FW::LOADS;
  extern __shared__ __attribute__((aligned(1024))) unsigned char lds[];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave % WGM, wn = wave / WGM;

  // ---- the experts' rows and tiles
  int off = 0, end = 0;
  if (lane < a.E) {
    off = (int)clamp_row(a.seg[(int64_t)lane * a.B], a.R);
    end = (int)clamp_row(a.seg[(int64_t)(lane + 1) * a.B], a.R);
  }
  const int mine = end > off ? (end - off + BM - 1) / BM : 0;
  int incl = mine;  // tiles of experts 0 .. lane
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int v = __shfl_up(incl, d, kWave);
    if (lane >= d) incl += v;
  }
  const int64_t slots = __builtin_amdgcn_readlane(incl, 63);
  // this workgroup's items: its XCD's contiguous range, strided by the XCD's workgroups
  const int64_t items = slots * a.ntn, per = (items + 7) / 8, wgs = gridDim.x >> 3, xcd = blockIdx.x & 7;
  const int64_t w_end = (xcd + 1) * per < items ? (xcd + 1) * per : items;
  int64_t w = xcd * per + (blockIdx.x >> 3);
  if (w >= w_end) return;  // whole workgroup

  struct Tile {
    int64_t row0, mrows, e, n0;
  };
  auto tile_of = [&](int64_t item) {
    const int64_t sg = item / (kSlotGroup * a.ntn), rem = item - sg * kSlotGroup * a.ntn;
    const int64_t left = slots - sg * kSlotGroup, in_group = left < kSlotGroup ? left : kSlotGroup;
    const int64_t tn = rem / in_group;
    const int slot = (int)(sg * kSlotGroup + (rem - tn * in_group));
    const int e = __popcll(__ballot(incl <= slot));  // the experts whose tiles all come before this one
    const int t = slot - (__builtin_amdgcn_readlane(incl, e) - __builtin_amdgcn_readlane(mine, e));
    const int row0 = __builtin_amdgcn_readlane(off, e) + t * BM;
    const int rows = __builtin_amdgcn_readlane(end, e) - row0;
    return Tile{row0, rows < BM ? rows : BM, e, tn * BN};
  };

  const int64_t xb = a.K * (int64_t)sizeof(T), wb = (TRANS ? a.N : a.K) * (int64_t)sizeof(T);
  FX fx;
  FW fw;
  fx.init(xb, wave, lane);
  fw.init(wb, wave, lane);
  ReadOf<T, true, BM, NBM, KB> rx;
  ReadOf<T, !TRANS, BN, NBN, KB> rw;
  rx.init(wm * WM, lane);
  rw.init(wn * WN, lane);
  const int nq = (int)((a.K + KC - 1) / KC);
  const uint32_t l0 = lds_addr(lds), eb = l0 + ST * STAGE + wave * 4096;

  // ---- the loads' side: the next chunk to load and where it goes
  Tile lt;
  const T *lx, *lw;
  int lk = 0;                // K left to load of its tile; <= 0 past the last tile: the loads go on, of empty windows
  uint32_t ls = l0;          // stage
  uint32_t xrows_b, wrows_b; // X: bytes of the rows before the window's last; W: the same, or (TRANS) its row's bytes
  int wcols;                 // TRANS: columns of W from n0 on
  auto load_tile = [&]() {
    lt = tile_of(w);
    lx = static_cast<const T*>(a.X) + lt.row0 * a.K;
    lw = static_cast<const T*>(a.W) + lt.e * a.K * a.N + (TRANS ? lt.n0 : lt.n0 * a.K);
    lk = (int)a.K;
    xrows_b = (uint32_t)((lt.mrows - 1) * xb);
    const int64_t n = a.N - lt.n0;
    wrows_b = TRANS ? (uint32_t)(n * 2) : (uint32_t)(((n < BN ? n : BN) - 1) * wb);
    wcols = (int)n;
  };
  auto xload = [&](int P) {
    const u32x4 srd = make_srd(lx, lk > 0 ? xrows_b + 2u * (uint32_t)lk : 0u);
    dma16_buf(srd, fx.qp[P] < lk ? fx.voff[P] : 0x80000000u, ls + (wave + NW * P) * 1024);
  };
  auto wload = [&](int P) {
    const uint32_t krows = (uint32_t)(lk < KC ? lk : KC);
    const uint32_t bytes = TRANS ? (krows - 1) * (uint32_t)wb + wrows_b : wrows_b + 2u * (uint32_t)lk;
    const u32x4 srd = make_srd(lw, lk > 0 ? bytes : 0u);
    dma16_buf(srd, fw.qp[P] < (TRANS ? wcols : lk) ? fw.voff[P] : 0x80000000u, ls + OX::BYTES + (wave + NW * P) * 1024);
  };
  auto load_next = [&]() {  // after a chunk's X and W parts
    ls = ls == l0 + (ST - 1) * STAGE ? l0 : ls + STAGE;
    lx += KC;
    lw += TRANS ? KC * a.N : KC;
    lk -= KC;
    if (lk <= 0) {
      w += wgs;
      if (w < w_end) load_tile();
    }
  };
  load_tile();

  struct Frags {
    u32x4 w[NBN], x[NBM];
  };
  auto read1 = [&](uint32_t sb, int s, Frags& f, int k) {  // the k-th of a step's fragments, in the order of their use
    if (k == 0) f.w[0] = rw.get(sb + OX::BYTES, s, 0);
    else if (k <= NBM) f.x[k - 1] = rx.get(sb, s, k - 1);
    else f.w[k - NBM] = rw.get(sb + OX::BYTES, s, k - NBM);
  };
  f32x16 acc[NBN][NBM];
  // One step: the products of `f`, and between them the reads of the next step's fragments and this wave's
  // share of a later chunk's loads (its X or its W part). A burst of either would hold up the products.
  auto step = [&](const Frags& f, Frags& g, uint32_t sb, int s, auto wpart) {
#pragma unroll
    for (int k = 0; k < NBN * NBM; ++k) {
      const int j = k / NBM, i = k % NBM;
      acc[j][i] = mma_step<T>(f.w[j], f.x[i], acc[j][i]);
      if (k < NBN + NBM) read1(sb, s, g, k);
      if (k % 4 == 1) {
        if constexpr (decltype(wpart)::value) wload(k / 4);
        else xload(k / 4);
      }
    }
    if constexpr (decltype(wpart)::value) load_next();
  };
  static_assert(4 * FX::LOADS == NBM * NBN && 4 * FW::LOADS == NBM * NBN, "a load every four products");

#pragma unroll
  for (int q = 0; q < ST - 1; ++q) {
#pragma unroll
    for (int i = 0; i < FX::LOADS; ++i) xload(i);
#pragma unroll
    for (int i = 0; i < FW::LOADS; ++i) wload(i);
    load_next();
  }
#pragma unroll
  for (int i = 0; i < FX::LOADS; ++i) xload(i);
  // Wait for the stream's next chunk, for every wave; every wave is then done with the chunk before it. Behind
  // it in flight are ST - 2 whole chunks, at the first wait also the X part of one more, and after a tile's
  // end the stores of its rows.
  constexpr int kStores = NBM * (NBN / 2) * 4;
  wait_vmcnt<LPC*(ST - 2) + FX::LOADS>();
  lds_barrier();
  Frags f0, f1;
#pragma unroll
  for (int k = 0; k < NBN + NBM; ++k) read1(l0, 0, f0, k);
  uint32_t cs = l0;  // the chunk being multiplied
  bool stored = false;
  for (int64_t cw = xcd * per + (blockIdx.x >> 3); cw < w_end; cw += wgs) {
    zero_acc(acc);
    for (int q = 0; q < nq; ++q) {
      step(f0, f1, cs, 1, std::true_type{});
      if (stored) {
        wait_vmcnt<LPC*(ST - 2) + kStores>();
        stored = false;
      } else {
        wait_vmcnt<LPC*(ST - 2)>();
      }
      lds_barrier();
      cs = cs == l0 + (ST - 1) * STAGE ? l0 : cs + STAGE;
      step(f1, f0, cs, 0, std::false_type{});
    }
    // ---- this wave's rows: accumulator lane l holds row l % 32, columns 8q + 4(l / 32) .. + 3 of a 32-block
    const Tile ct = tile_of(cw);
    const uint32_t yb = (uint32_t)(ct.mrows * a.N * 2);
    const __amdgpu_buffer_rsrc_t ysrd =
        __builtin_amdgcn_make_buffer_rsrc(static_cast<T*>(a.Y) + ct.row0 * a.N, 0, yb, 0x00020000);
    const int r = lane & 31, fr = (r >> 1) & 15;
#pragma unroll
    for (int i = 0; i < NBM; ++i)
#pragma unroll
      for (int h = 0; h < NBN / 2; ++h) {
#pragma unroll
        for (int jj = 0; jj < 2; ++jj)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const f32x16& c = acc[2 * h + jj][i];
            const int unit = jj * 8 + 2 * q + (lane >> 5);
            u32x2 v;
            v[0] = pack_bf16(c[4 * q], c[4 * q + 1]);
            v[1] = pack_bf16(c[4 * q + 2], c[4 * q + 3]);
            *(lds_u32x2*)(uintptr_t)(eb + r * 128 + 8 * (unit ^ fr)) = v;
          }
        lds_wave_fence();
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          const int rr = 8 * t + (lane >> 3), pp = lane & 7, f2 = (rr >> 1) & 15;
          u32x4 v = *(lds_u32x4*)(uintptr_t)(eb + rr * 128 + 16 * (pp ^ (f2 >> 1)));
          if (f2 & 1) v = u32x4{v[2], v[3], v[0], v[1]};
          const int64_t m = wm * WM + i * 32 + rr, n = ct.n0 + wn * WN + h * 64 + 8 * pp;
          // always issued (the waits count the stores); rows and columns outside the tile are dropped
          const uint32_t vo = m < ct.mrows && n < a.N ? (uint32_t)((m * a.N + n) * 2) : 0x80000000u;
          __builtin_amdgcn_raw_buffer_store_b128(v, ysrd, vo, 0, 0);
        }
        lds_wave_fence();
      }
    stored = true;
  }
  wait_vmcnt<0>();  // the empty loads past the last tile: none may land after this workgroup's LDS is given away
}

// Y = the splits' partial products, added in order, for the rows that belong
// to an expert.
template <typename T>
__global__ __launch_bounds__(256) void k_grouped_join(MatmulArgs a) {
  const int64_t lo = clamp_row(a.seg[0], a.R), hi = clamp_row(a.seg[a.E * a.B], a.R);
  const int64_t n = a.R * a.N;
  for (int64_t i = lo * a.N + (int64_t)blockIdx.x * 256 + threadIdx.x; i < hi * a.N; i += (int64_t)gridDim.x * 256) {
    float s = 0.f;
#pragma unroll 4
    for (int64_t k = 0; k < a.ks; ++k) s += a.part[k * n + i];
    if constexpr (sizeof(T) == 2) static_cast<T*>(a.Y)[i].u = f32_to_bf16(s);
    else static_cast<T*>(a.Y)[i] = s;
  }
}

// ---------------------------------------------------------------------------
// Norms. Both Grams of a pair of row tiles in registers, their elementwise
// product summed, off-diagonal pairs counted twice.
struct GNormArgs {
  const void *A, *G;
  const int64_t* seg;
  int64_t R, E, B, d, p;
  float* partial;   // tiles: [slots * J]; packed: J values per row [R][J]
  int32_t* row_seg; // packed: a row's segment, -1 for none [R]
  int64_t slots;    // R / TS + E * B
  int64_t J;        // workgroups a row tile's pairs are dealt to
};

template <typename T>
constexpr int norm_tile() {
  return sizeof(T) == 2 ? 128 : 64;
}

// Segments of about 64 rows or more: row tiles of TS within a segment (128 for
// bf16, where memory bounds; 64 for fp32, where the products do).
// Workgroup (tile t, j) takes the pairs (t, u), u - t = j, j + J, ...: a long
// segment's pairs spread over J workgroups (one after another they were the
// launch's critical path: 276 -> 181 us at 256 segments of 128 rows on
// average, d + p = 6400; 151 us with the deeper stages of the diagonal, 2.8
// TB/s of rows: a workgroup's chunks one after another still bound it). A wave
// whose 64 x 64 part lies below the diagonal or past the segment only takes
// part in the loads.
template <typename T, bool DMA>
__global__ __launch_bounds__(256, DMA ? 2 : 1) void k_grouped_norm(GNormArgs a) {
  constexpr int TS = norm_tile<T>(), WG = 2, NW = 4, WT = TS / 2, NB = WT / 32;
  using O = Opnd<T, true, TS>;
  constexpr int KC = O::KC;
  extern __shared__ __attribute__((aligned(1024))) unsigned char lds[];
  __shared__ float red[NW];

  // XCD x takes every eighth run of four row tiles, whose pairs share rows in its L2
  const int64_t local = blockIdx.x >> 3, run = local / (4 * a.J), in_run = local - run * 4 * a.J;
  const int64_t slot = (run * 8 + (blockIdx.x & 7)) * 4 + in_run / a.J, j = in_run % a.J;
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
  for (int64_t u = j; u * TS < rows; u += a.J) {
    const int64_t urows = rows - u * TS < TS ? rows - u * TS : TS;
    const bool diag = u == 0;
    const bool active = !(diag && wm > wn) && wm * WT < trows && wn * WT < urows;
    f32x16 ga[NB][NB], gg[NB][NB];
    zero_acc(ga);
    zero_acc(gg);
    // Pairs of a tile with itself load one operand, and use the other's LDS for two more stages: three chunks in
    // flight instead of one.
    auto gram = [&](const T* M, int64_t K, f32x16 (&acc)[NB][NB], auto dg) {
      constexpr bool DIAG = decltype(dg)::value;
      constexpr int ST = DIAG ? 4 : 2, STAGE = (DIAG ? 1 : 2) * O::BYTES, UOFF = DIAG ? 0 : O::BYTES;
      using F = Filler<O, T, NW>;
      const T* Mt = M + row0 * K;
      const T* Mu = M + (row0 + u * TS) * K;
      const int64_t kb = K * (int64_t)sizeof(T);
      F f;
      f.init(kb, wave, lane);
      const int nq = (int)((K + KC - 1) / KC);
      auto wt = [&](int q) { return Win<T>{Mt + (int64_t)q * KC, kb, trows, K - (int64_t)q * KC}; };
      auto wu = [&](int q) { return Win<T>{Mu + (int64_t)q * KC, kb, urows, K - (int64_t)q * KC}; };
      if constexpr (DMA) {
        constexpr int LPC = F::LOADS * (DIAG ? 1 : 2);
        auto stage_of = [&](int q) { return l0 + (uint32_t)(q % ST) * STAGE; };
        auto issue = [&](int q) {
          f.dma(wt(q), stage_of(q), wave);
          if constexpr (!DIAG) f.dma(wu(q), stage_of(q) + UOFF, wave);
        };
        lds_barrier();  // every wave is done with the stages of the previous Gram
#pragma unroll
        for (int q = 0; q < ST - 1; ++q)
          if (q < nq) issue(q);
        for (int q = 0; q < nq; ++q) {
          wait_chunks<LPC, ST - 2>(nq - 1 - q < ST - 2 ? nq - 1 - q : ST - 2);
          lds_barrier();
          if (q + ST - 1 < nq) issue(q + ST - 1);
          if (active) chunk_mma<T, NB, NB>(stage_of(q), stage_of(q) + UOFF, rm, rn, 4, acc);
        }
      } else {
        u32x4 vt[F::LOADS], vu[F::LOADS];
        f.load(wt(0), vt, wave, lane);
        if constexpr (!DIAG) f.load(wu(0), vu, wave, lane);
        for (int q = 0; q < nq; ++q) {
          __syncthreads();
          f.store(vt, lds, wave, lane);
          if constexpr (!DIAG) f.store(vu, lds + UOFF, wave, lane);
          __syncthreads();
          f.load(wt(q + 1), vt, wave, lane);  // past the last chunk: an empty window
          if constexpr (!DIAG) f.load(wu(q + 1), vu, wave, lane);
          if (active) chunk_mma<T, NB, NB>(l0, l0 + UOFF, rm, rn, 4, acc);
        }
      }
    };
    if (diag) {
      gram(static_cast<const T*>(a.A), a.d, ga, std::true_type{});
      gram(static_cast<const T*>(a.G), a.p, gg, std::true_type{});
    } else {
      gram(static_cast<const T*>(a.A), a.d, ga, std::false_type{});
      gram(static_cast<const T*>(a.G), a.p, gg, std::false_type{});
    }
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < NB; ++i)
#pragma unroll
      for (int k = 0; k < NB; ++k)
#pragma unroll
        for (int e = 0; e < 16; ++e) s = __builtin_fmaf(ga[i][k][e], gg[i][k][e], s);
    if (active) total += diag && wm == wn ? s : 2.0f * s;
  }
  total = wave_sum(total);
  if (lane == 0) red[wave] = total;
  __syncthreads();
  if (threadIdx.x == 0) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < NW; ++i) s += red[i];
    a.partial[slot * a.J + j] = s;
  }
}

// Shorter segments: row tiles of 32 consecutive rows whatever their segments,
// both Grams of a tile with itself masked to pairs of one segment, and with
// the following tiles as far as the tile's last segment reaches. The rows go
// from memory straight into fragments (a Gram of a tile with itself takes one
// load per product), K dealt to the four waves and joined through LDS. Each
// row's share of its segment's value goes to partial[row]. 16384 rows in 1024
// segments of 16, d + p = 6400 bf16: 117 us a call, 1.8 TB/s; a wave's loads, in
// turns of four, bound it.
template <typename T>
__global__ __launch_bounds__(256) void k_grouped_norm_packed(GNormArgs a) {
  constexpr int P = elem_traits<T>::per16, U = 4;
  __shared__ float gram[2][4][32 * 33];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 31, g = lane >> 5;
  const int orow = threadIdx.x >> 3, ocol = (threadIdx.x & 7) * 4;  // this thread's four elements of the product
  const int64_t J = a.J;
  for (int64_t item = blockIdx.x; item < (a.R + 31) / 32 * J; item += gridDim.x) {
    const int64_t t = item / J, j = item - t * J;  // pairs (t, t + j), (t, t + j + J), ...
    const int64_t trow = t * 32 + r;
    const bool tok = trow < a.R && a.row_seg[trow] >= 0;
    const int oseg = t * 32 + orow < a.R ? a.row_seg[t * 32 + orow] : -1;
    const int last = a.row_seg[t * 32 + 31 < a.R ? t * 32 + 31 : a.R - 1];
    float value = 0.f;
    for (int64_t u = t + j;; u += J) {
      if (u > t && (u * 32 >= a.R || last < 0 || a.row_seg[u * 32] != last)) break;  // uniform
      const int64_t urow = u * 32 + r;
      const bool uok = urow < a.R && a.row_seg[urow] >= 0;
      f32x16 acc[2];
#pragma unroll
      for (int m = 0; m < 2; ++m) {
#pragma unroll
        for (int k = 0; k < 16; ++k) acc[m][k] = 0.f;
        const int64_t K = m ? a.p : a.d;
        const T* X = static_cast<const T*>(m ? a.G : a.A);
        const T* xt = X + (tok ? trow : 0) * K;
        const T* xu = X + (uok ? urow : 0) * K;
        const int64_t steps = (K + 2 * P - 1) / (2 * P);
        // the next U steps' pieces are loaded ahead of this U's products
        u32x4 nt[U], nu[U];
        auto load = [&](int64_t s) {
#pragma unroll
          for (int i = 0; i < U; ++i) nt[i] = load_piece(xt, (2 * (s + i) + g) * P, K, tok);
          if (u != t) {
#pragma unroll
            for (int i = 0; i < U; ++i) nu[i] = load_piece(xu, (2 * (s + i) + g) * P, K, uok);
          } else {
#pragma unroll
            for (int i = 0; i < U; ++i) nu[i] = nt[i];
          }
        };
        load(wave * U);
        for (int64_t s = wave * U; s < steps; s += 4 * U) {
          u32x4 ft[U], fu[U];
#pragma unroll
          for (int i = 0; i < U; ++i) {
            ft[i] = nt[i];
            fu[i] = nu[i];
          }
          if (s + 4 * U < steps) load(s + 4 * U);
#pragma unroll
          for (int i = 0; i < U; ++i)
            if (s + i < steps) acc[m] = mma_step<T>(ft[i], fu[i], acc[m]);
        }
      }
      __syncthreads();  // the previous pair's elements are read
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int k = 0; k < 16; ++k) gram[m][wave][acc_row(k, lane) * 33 + r] = acc[m][k];
      __syncthreads();
      float s = 0.f;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int64_t col = u * 32 + ocol + c;
        const int at = orow * 33 + ocol + c;
        const float x = (gram[0][0][at] + gram[0][1][at]) + (gram[0][2][at] + gram[0][3][at]);
        const float y = (gram[1][0][at] + gram[1][1][at]) + (gram[1][2][at] + gram[1][3][at]);
        if (col < a.R && oseg >= 0 && a.row_seg[col] == oseg) s = __builtin_fmaf(x, y, s);
      }
#pragma unroll
      for (int off = 4; off > 0; off >>= 1) s += __shfl_xor(s, off, kWave);
      value += u == t ? s : 2.0f * s;
    }
    if ((threadIdx.x & 7) == 0 && t * 32 + orow < a.R) a.partial[(t * 32 + orow) * J + j] = value;
  }
}

__global__ __launch_bounds__(256) void k_grouped_row_segments(const int64_t* __restrict__ seg, int64_t R, int64_t n,
                                                              int32_t* __restrict__ row_seg) {
  const int64_t row = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (row >= R) return;
  int64_t g = -1;
  if (row >= seg[0] && row < seg[n]) {
    int64_t hi = n;  // the last segment that starts at or before the row
    g = 0;
    while (hi - g > 1) {
      const int64_t mid = (g + hi) / 2;
      if (seg[mid] <= row) g = mid;
      else hi = mid;
    }
  }
  row_seg[row] = (int32_t)g;
}

// sqnorm[b] (+)= the values of the sample's tiles (or, packed, rows). One
// workgroup per sample: 16 groups of 16 lanes take the experts in turn, a
// lane every sixteenth value of a segment; the lanes' sums are joined in a
// fixed order. (One lane per segment, its values one after another: 14 us at
// 5 experts of 12 rows, 45 values each.)
template <bool PACKED, int TS>
__global__ __launch_bounds__(256) void k_grouped_norm_finish(GNormArgs a, float* __restrict__ sqnorm, int accumulate) {
  __shared__ float red[4];
  const int sub = threadIdx.x >> 4, l = threadIdx.x & 15;
  for (int64_t b = blockIdx.x; b < a.B; b += gridDim.x) {
    float s = 0.f;
    for (int64_t e = sub; e < a.E; e += 16) {
      const int64_t g = e * a.B + b;
      const int64_t off = clamp_row(a.seg[g], a.R), end = clamp_row(a.seg[g + 1], a.R);
      const int64_t first = (PACKED ? off : off / TS + g) * a.J;
      const int64_t n = end <= off ? 0 : (PACKED ? end - off : (end - off + TS - 1) / TS) * a.J;
#pragma unroll 4
      for (int64_t t = l; t < n; t += 16) s += a.partial[first + t];
    }
    s = wave_sum(s);
    __syncthreads();  // the previous sample's sums are read
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = s;
    __syncthreads();
    if (threadIdx.x == 0) {
      s = (red[0] + red[1]) + (red[2] + red[3]);
      sqnorm[b] = accumulate ? sqnorm[b] + s : s;
    }
  }
}

// ---------------------------------------------------------------------------
// Clipped sums: out_e = sum_r c_r a_r g_r^T over the rows r of expert e, c_r
// the clip factor of the row's sample. bf16 products leave no room for the
// factor in an operand (c g rounded to bf16 would cost 2^-9 of the sum), so it
// enters in one of three ways:
//   ratio  (bf16, samples with about 32 rows or more per expert) K runs over
//          pieces of up to 32 rows of one sample, the accumulators hold the
//          sum divided by the current factor and are rescaled where the
//          factor changes (one fp32 rounding per sample);
//   split  (bf16, shorter ranges) K runs over the expert's rows as they lie; a
//          chunk's A operand becomes c a = hi + mid + lo, three bf16 values
//          that hold the 24 bits of the fp32 product (two would leave an error
//          of 2^-17), and takes three products;
//   fold   (bf16, 128 x 128 tiles) pieces as for ratio, each sample's product
//          in a second accumulator set, added as acc += c tmp;
//   scale  (fp32) the A operand is multiplied by c in fp32.

// Piece t of segment g covers up to kPieceRows rows of one sample and carries
// its clip factor, at slot off_g / kPieceRows + g + t (rows = 0: unused slot).
constexpr int kPieceRows = 32;
struct Piece {
  int32_t row0, rows;
  float c;
  int32_t pad;
};
struct GSumArgs {
  const void *A, *G;
  const int64_t* seg;
  const Piece* pieces;  // ratio
  const float* crow;    // split, scale: factor of every row [R]
  int64_t R, E, B, d, p;
  int64_t mt, nt, ks;
  NoiseArgs na;
  float* out;    // ks == 1: the result [E*d][p], noise and mean applied
  float* part;   // else the splits' sums [ks][E*d][p]
  int fused;     // the epilogue writes out
  int32_t* queue;  // next item of each XCD's list, past the workgroups' first ones
};

// The tiles of all (expert, split) pairs, dealt evenly to the 8 XCDs. A pair's
// tiles form 8 runs of neighbours, which share operand rows in an XCD's L2:
// run j holds tiles [j tiles / 8, (j + 1) tiles / 8) and goes to XCD
// (j - pair) mod 8. Over 8 pairs an XCD takes every run once, so its items
// follow the tiles round from its own run on. (Run j always to XCD j: 182 us
// for the sums of 4 experts of 1280 x 1280, whose 25 tiles do not divide by 8.)
__host__ __device__ inline int deal_count(int64_t pairs, int64_t tiles, int xcd) {
  const int64_t blocks = pairs / 8, left = pairs - 8 * blocks, j1 = xcd + left;  // runs [xcd, j1) of the last block
  const int64_t t0 = xcd * tiles / 8, t1 = j1 <= 8 ? j1 * tiles / 8 : tiles + (j1 - 8) * tiles / 8;
  return (int)(blocks * tiles + t1 - t0);
}
__device__ __forceinline__ void dealt(int tiles, int xcd, int l, int* pair, int* tile) {
  const uint32_t n = (uint32_t)tiles, blk = (uint32_t)l / n;
  uint32_t t = (uint32_t)xcd * n / 8 + ((uint32_t)l - blk * n);
  if (t >= n) t -= n;
  const uint32_t run = (8 * t + 7 + n) / n - 1;
  *pair = (int)(8 * blk + ((run - (uint32_t)xcd) & 7));
  *tile = (int)t;
}

__global__ __launch_bounds__(256) void k_grouped_pieces(const int64_t* __restrict__ seg, int64_t R, int64_t E,
                                                        int64_t B, const float* __restrict__ c, int64_t slots,
                                                        Piece* __restrict__ out, int32_t* __restrict__ queue) {
  const int64_t slot = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (blockIdx.x == 0 && threadIdx.x < 8) queue[threadIdx.x] = 0;
  if (slot >= slots) return;
  // the last g with off_g / kPieceRows + g <= slot, by each thread on its own
  int64_t g = 0, hi = E * B;
  while (hi - g > 1) {
    const int64_t mid = (g + hi) / 2;
    if (clamp_row(seg[mid], R) / kPieceRows + mid <= slot) g = mid;
    else hi = mid;
  }
  const int64_t off = clamp_row(seg[g], R), end = clamp_row(seg[g + 1], R);
  const int64_t t = slot - (off / kPieceRows + g), row0 = off + t * kPieceRows;
  Piece pc{0, 0, 0.f, 0};
  if (t >= 0 && row0 < end) {
    pc.row0 = (int32_t)row0;
    pc.rows = (int32_t)(end - row0 < kPieceRows ? end - row0 : kPieceRows);
    pc.c = c[g % B];
  }
  out[slot] = pc;
}

// The clip factor of every row; 0 for rows outside the segments.
__global__ __launch_bounds__(256) void k_grouped_row_factors(const int64_t* __restrict__ seg, int64_t R, int64_t E,
                                                             int64_t B, const float* __restrict__ c,
                                                             float* __restrict__ crow, int32_t* __restrict__ queue) {
  const int64_t row = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (blockIdx.x == 0 && threadIdx.x < 8) queue[threadIdx.x] = 0;
  if (row >= R) return;
  float v = 0.f;
  if (row >= seg[0] && row < seg[E * B]) {
    int64_t g = 0, hi = E * B;  // the last segment that starts at or before the row
    while (hi - g > 1) {
      const int64_t mid = (g + hi) / 2;
      if (seg[mid] <= row) g = mid;
      else hi = mid;
    }
    v = c[g % B];
  }
  crow[row] = v;
}

// c a of eight (k, feature) elements as three bf16 terms; ck: the eight rows' factors.
__device__ __forceinline__ void split_scaled(u32x4 a, const f32x4 (&ck)[2], u32x4 (&t)[3]) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    float y0 = __uint_as_float(a[e] << 16) * ck[e >> 1][2 * (e & 1)];
    float y1 = __uint_as_float(a[e] & 0xFFFF0000u) * ck[e >> 1][2 * (e & 1) + 1];
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      const uint32_t h = pack_bf16(y0, y1);
      t[k][e] = h;
      y0 -= __uint_as_float(h << 16);  // exact
      y1 -= __uint_as_float(h & 0xFFFF0000u);
    }
  }
}

// 4 bytes per lane from a buffer straight into LDS
__device__ __forceinline__ void dma4_buf(u32x4 srd, uint32_t voff, uint32_t lds_base) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tbuffer_load_dword %0, %1, 0 offen lds" ::"v"(voff), "s"(srd),
               "s"(lds_base)
               : "memory", "m0");
}

// A wave's accumulators to the result: (S + sc z) * inv_denom, or S itself as
// a split's partial (sc = 0, inv_denom = 1 there). Half a 32x32 block at a time
// goes through 2 KB of the wave's own LDS (16 rows of 32 fp32), so that rows
// are stored 128 bytes at a time, and the four rows of a quad, which share a
// Philox block, are drawn by one lane (d is a multiple of 4 where noise is
// added here, so quads start at multiples of 4 of the flat row e*d + m).
struct Emit {
  float* dst;  // [d][p]
  int64_t d, p, e;
  bool vec;  // 16-byte stores
};
template <int NBM, int NBN>
__device__ __forceinline__ void emit_tile(const f32x16 (&acc)[NBM][NBN], const Emit& o, const NoiseArgs& na,
                                          uint32_t scratch, int64_t m0, int64_t n0, int lane) {
  typedef __attribute__((address_space(3))) float lds_f;
#pragma unroll
  for (int i = 0; i < NBM; ++i)
#pragma unroll
    for (int j = 0; j < NBN; ++j)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int q = 0; q < 2; ++q)
#pragma unroll
          for (int r = 0; r < 4; ++r)
            *(lds_f*)(uintptr_t)(scratch + 128 * (8 * q + 4 * (lane >> 5) + r) + 4 * (lane & 31)) =
                acc[i][j][8 * h + 4 * q + r];
        lds_wave_fence();
        const int64_t mb = m0 + 32 * i + 16 * h, nb = n0 + 32 * j;
        if (na.sc == 0.0f) {
          f32x4 v[2];
#pragma unroll
          for (int t = 0; t < 2; ++t)
            v[t] = __builtin_bit_cast(
                f32x4, *(lds_u32x4*)(uintptr_t)(scratch + 128 * (8 * t + (lane >> 3)) + 16 * (lane & 7)));
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            const int64_t m = mb + 8 * t + (lane >> 3), n = nb + 4 * (lane & 7);
#pragma unroll
            for (int k = 0; k < 4; ++k) v[t][k] = noised_mean_spec(v[t][k], 0.0f, 0.0f, na.inv_denom);
            if (m >= o.d || n >= o.p) continue;
            float* dst = o.dst + m * o.p + n;
            if (o.vec) {
              __builtin_nontemporal_store(v[t], reinterpret_cast<f32x4*>(dst));
            } else {
#pragma unroll
              for (int k = 0; k < 4; ++k)
                if (n + k < o.p) dst[k] = v[t][k];
            }
          }
        } else {
#pragma unroll 1
          for (int t = 0; t < 2; ++t) {
            const int quad = 2 * t + (lane >> 5);
            const int64_t m = mb + 4 * quad, n = nb + (lane & 31);
            if (m >= o.d || n >= o.p) continue;
            const f32x4 z = normals4((uint32_t)(((o.e * o.d + m) >> 2) * o.p + n), 2u * na.layer, na.step, 0u, na.k0,
                                     na.k1);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              const float S = *(lds_f*)(uintptr_t)(scratch + 128 * (4 * quad + r) + 4 * (lane & 31));
              if (m + r < o.d) o.dst[(m + r) * o.p + n] = noised_mean_spec(S, na.sc, z[r], na.inv_denom);
            }
          }
        }
        lds_wave_fence();
      }
}

__device__ __forceinline__ Emit emit_at(const GSumArgs& a, int64_t e, int64_t sp) {
  float* dst = a.fused ? a.out + e * a.d * a.p : a.part + (sp * a.E + e) * a.d * a.p;
  return Emit{dst, a.d, a.p, e, a.p % 4 == 0 && (reinterpret_cast<uintptr_t>(a.fused ? a.out : a.part) & 15) == 0};
}

// bf16, 256 x 256 tiles, one workgroup per CU over its (expert, split, tile)
// items in turn, as one stream of 32-row chunks (the structure of
// k_grouped_matmul_big; both operands are read with transposing LDS reads).
// XCD x takes its share of every expert's tiles, experts with more rows
// first, and its workgroups take the next item off the XCD's list as they
// come free: uneven experts even out, and the workgroups share operand tiles
// in their L2. (Which workgroup forms an item does not enter its result.)
//
// 32768 rows over 8 experts of 32 samples, 1280 x 5120: 550 to 615 us call
// after call, whatever the factors (650 to 710 as single calls in a trace), 0.7
// to 0.78 PFLOP/s; the matrix cores are busy a third of the cycles. The rest is the loads (110 us, also from L2), the
// rescale (90 us where every sample clips), the writing of the fp32 tiles
// (70 us), a piece's unused rows (an eighth here) and a last round of items
// that does not fill the GPU (splitting those over K gained nothing: the items
// in flight share what the loads and the power allow).
template <bool RATIO>
__global__ __launch_bounds__(512) void k_grouped_sum_big(GSumArgs a) {
  using T = bf16s;
  constexpr int BM = 256, BN = 256, WGM = 4, NW = 8, WM = 64, WN = 128, NBM = 2, NBN = 4, KB = 64, ST = 4;
  using OA = Opnd<T, false, BM, KB>;
  using OG = Opnd<T, false, BN, KB>;
  using FA = Filler<OA, T, NW>;
  using FG = Filler<OG, T, NW>;
  static_assert(OA::KC == kPieceRows, "a chunk holds a piece");
  constexpr int KC = 32, CB = RATIO ? 0 : NW * 128;  // split: the rows' factors, a copy per wave
  constexpr int STAGE = OA::BYTES + OG::BYTES + CB, LPC = FA::LOADS + FG::LOADS + (RATIO ? 0 : 1);
  extern __shared__ __attribute__((aligned(1024))) unsigned char lds[];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave % WGM, wn = wave / WGM;

  // ---- experts by rows, the largest first (up to 64 of them; more keep their order)
  int order = lane;
  if (a.E <= 64) {
    int mine = -1;
    if (lane < a.E) mine = (int)(clamp_row(a.seg[(int64_t)(lane + 1) * a.B], a.R) - clamp_row(a.seg[(int64_t)lane * a.B], a.R));
    int rank = 0;
    for (int j = 0; j < (int)a.E; ++j) {
      const int o = __builtin_amdgcn_readlane(mine, j);
      rank += o > mine || (o == mine && j < lane);
    }
    // lane r <- the expert of rank r
    for (int j = 0; j < (int)a.E; ++j)
      if (__builtin_amdgcn_readlane(rank, j) == lane) order = j;
  }

  // ---- items: this XCD's (expert by rank, split) and tile
  const int wgs = (int)(gridDim.x >> 3), xcd = (int)(blockIdx.x & 7), tiles = (int)(a.mt * a.nt);
  const int nlocal = deal_count(a.E * a.ks, tiles, xcd);
  if ((int)(blockIdx.x >> 3) >= nlocal) return;  // whole workgroup
  struct Item {
    int e, sp, m0, n0;
  };
  auto item_at = [&](int l) {
    int pair, tile;
    dealt(tiles, xcd, l, &pair, &tile);
    const int er = (int)((uint32_t)pair / (uint32_t)a.ks), tn = (int)((uint32_t)tile / (uint32_t)a.mt);
    Item it;
    it.sp = pair - er * (int)a.ks;
    it.e = a.E <= 64 ? __builtin_amdgcn_readlane(order, er) : er;
    it.m0 = (tile - tn * (int)a.mt) * BM;
    it.n0 = tn * BN;
    return it;
  };

  const uint32_t ab = (uint32_t)a.d * 2u, gb = (uint32_t)a.p * 2u;
  FA fa;
  FG fg;
  fa.init(ab, wave, lane);
  fg.init(gb, wave, lane);
  ReadF<T, BM, NBM, KB> ra;
  ReadF<T, BN, NBN, KB> rg;
  ra.init(wm * WM, lane);
  rg.init(wn * WN, lane);
  const uint32_t l0 = lds_addr(lds);

  // ---- the loads' side: buffers of its chunk (no bytes: an empty window, for chunks past the last item, experts
  // without rows, and samples with factor 0, whose rows add nothing), and where its item stands
  __shared__ int next_item[2];
  int litem = (int)(blockIdx.x >> 3), turn = 0;
  bool first = true;
  if (threadIdx.x == 0) next_item[0] = wgs + atomicAdd(a.queue + xcd, 1);
  __syncthreads();
  const char *abase = nullptr, *gbase = nullptr;  // the item's first columns
  uint32_t acols = 0, gcols = 0;                  // bytes of them to the row's end
  uint32_t va[FA::LOADS], vg[FG::LOADS];          // the lane's offsets; past num_records where its columns do not exist
#pragma unroll
  for (int i = 0; i < FA::LOADS; ++i) va[i] = 0x80000000u;
#pragma unroll
  for (int i = 0; i < FG::LOADS; ++i) vg[i] = 0x80000000u;
  u32x4 sa = make_srd(static_cast<const char*>(nullptr), 0u), sg = sa, sc = sa;
  bool lopen = false;       // the item has chunks left
  int lpos = 0, lend = 0;   // ratio: slot window and end; split: next row and end
  uint64_t lmask = 0;
  Piece lmine{0, 0, 0.f, 0};
  uint32_t ls = l0;
  struct Desc {
    float c;
    int id;  // 2 * item + (last chunk of its item); -1: past the last
  };
  auto load64 = [&]() {
    lmine = Piece{0, 0, 0.f, 0};
    if (lpos + lane < lend) lmine = a.pieces[lpos + lane];
    lmask = __ballot(lmine.rows > 0);
  };
  auto skip_unused = [&]() {
    while (lmask == 0 && lpos + 64 < lend) {
      lpos += 64;
      load64();
    }
  };
  auto window = [&](int row, int rows) {
    const uint32_t n = (uint32_t)rows;
    sa = make_srd(abase + (uint64_t)(uint32_t)row * ab, n ? (n - 1) * ab + acols : 0u);
    sg = make_srd(gbase + (uint64_t)(uint32_t)row * gb, n ? (n - 1) * gb + gcols : 0u);
    if constexpr (!RATIO) sc = make_srd(a.crow + row, 4u * n);
  };
  auto open_item = [&]() -> bool {
    // The item after this one is taken off the list now, by the first wave, and read by all when this one's
    // chunks have been fetched: at least one barrier later.
    if (first) {
      first = false;
    } else if (litem >= 0) {
      litem = __builtin_amdgcn_readfirstlane(next_item[turn]);
      turn ^= 1;
      if (threadIdx.x == 0) next_item[turn] = wgs + atomicAdd(a.queue + xcd, 1);
    }
    if (litem < 0 || litem >= nlocal) {
      litem = -1;
      return false;
    }
    const Item it = item_at(litem);
    abase = static_cast<const char*>(a.A) + 2 * it.m0;
    gbase = static_cast<const char*>(a.G) + 2 * it.n0;
    acols = ab - 2u * (uint32_t)it.m0;
    gcols = gb - 2u * (uint32_t)it.n0;
#pragma unroll
    for (int i = 0; i < FA::LOADS; ++i) va[i] = 2u * (uint32_t)fa.qp[i] < acols ? fa.voff[i] : 0x80000000u;
#pragma unroll
    for (int i = 0; i < FG::LOADS; ++i) vg[i] = 2u * (uint32_t)fg.qp[i] < gcols ? fg.voff[i] : 0x80000000u;
    const int g0 = it.e * (int)a.B, g1 = g0 + (int)a.B;
    const int o0 = __builtin_amdgcn_readfirstlane((int)clamp_row(a.seg[g0], a.R));
    const int o1 = __builtin_amdgcn_readfirstlane((int)clamp_row(a.seg[g1], a.R));
    // the split's share of the expert's slots, or of its rows in whole chunks
    const int s0 = RATIO ? o0 / KC + g0 : 0, s1 = RATIO ? o1 / KC + g1 : (o1 - o0 + KC - 1) / KC;
    const int share = (s1 - s0 + (int)a.ks - 1) / (int)a.ks;
    const int b0 = s0 + it.sp * share, b1 = b0 + share < s1 ? b0 + share : s1;
    lpos = RATIO ? b0 : o0 + b0 * KC;
    lend = RATIO ? b1 : (b1 < s1 ? o0 + b1 * KC : o1);
    lmask = 0;
    if constexpr (RATIO) {
      if (lpos < lend) {
        load64();
        skip_unused();
      }
    }
    return true;
  };
  auto fetch = [&]() -> Desc {  // the next chunk
    if (!lopen && !open_item()) {
      window(0, 0);
      return Desc{0.f, -1};
    }
    float c = 0.f;
    if constexpr (RATIO) {
      int row = 0, rows = 0;
      if (lmask != 0) {  // else: no rows in this item, one empty chunk
        const int i = __ffsll((unsigned long long)lmask) - 1;
        lmask &= lmask - 1;
        row = __builtin_amdgcn_readlane(lmine.row0, i);
        c = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(lmine.c), i));
        rows = c == 0.0f ? 0 : __builtin_amdgcn_readlane(lmine.rows, i);
        if (lmask == 0) skip_unused();
      }
      window(row, rows);
      lopen = lmask != 0;
    } else {
      const int left = lend - lpos;
      window(lpos, left <= 0 ? 0 : left < KC ? left : KC);
      lpos += KC;
      lopen = lpos < lend;
    }
    return Desc{c, 2 * litem + (lopen ? 0 : 1)};
  };
  auto aload = [&](int P) { dma16_buf(sa, va[P], ls + (wave + NW * P) * 1024); };
  auto gload = [&](int P) { dma16_buf(sg, vg[P], ls + OA::BYTES + (wave + NW * P) * 1024); };
  auto cload = [&]() {
    if constexpr (!RATIO)
      if (lane < KC) dma4_buf(sc, 4u * lane, ls + OA::BYTES + OG::BYTES + wave * 128);
  };
  auto next_stage = [&](uint32_t st) { return st == l0 + (ST - 1) * STAGE ? l0 : st + STAGE; };

  struct Frags {
    u32x4 a[NBM], g[NBN];
  };
  // the k-th of a step's fragments, in the order of their use
  auto read1 = [&](uint32_t sb, int s, Frags& f, int k) {
    if (k < NBM) f.a[k] = ra.get(sb, s, k);
    else f.g[k - NBM] = rg.get(sb + OA::BYTES, s, k - NBM);
  };
  f32x16 acc[NBM][NBN];
  // One step (16 rows): as in k_grouped_matmul_big, the next step's reads and a later chunk's loads between the
  // products. With split, sb/s of the fragments in hand give the rows' factors.
  // Ratio, at a sample's first step: each block is rescaled by r while its predecessor's product runs.
  auto step = [&](const Frags& f, uint32_t csb, int cstep, Frags& g, uint32_t sb, int s, auto gpart, bool rescale,
                  float r) {
    u32x4 t[NBM][3];
    if constexpr (!RATIO) {
      f32x4 ck[2];
      const uint32_t cb = csb + OA::BYTES + OG::BYTES + wave * 128 + 4 * (16 * cstep + 8 * (lane >> 5));
      ck[0] = __builtin_bit_cast(f32x4, *(lds_u32x4*)(uintptr_t)cb);
      ck[1] = __builtin_bit_cast(f32x4, *(lds_u32x4*)(uintptr_t)(cb + 16));
#pragma unroll
      for (int i = 0; i < NBM; ++i) split_scaled(f.a[i], ck, t[i]);
    }
#pragma unroll
    for (int k = 0; k < NBM * NBN; ++k) {
      const int j = k / NBM, i = k % NBM;
      if constexpr (RATIO) {
        if (decltype(gpart)::value && rescale) {
#pragma unroll
          for (int x = 0; x < 16; ++x) acc[i][j][x] *= r;
        }
        acc[i][j] = mfma32_bf16(f.a[i], f.g[j], acc[i][j]);
      } else {
#pragma unroll
        for (int u = 2; u >= 0; --u) acc[i][j] = mfma32_bf16(t[i][u], f.g[j], acc[i][j]);  // the small terms first
      }
      if (k < NBN + NBM) read1(sb, s, g, k);
      if (k % 4 == 1) {
        if constexpr (decltype(gpart)::value) gload(k / 4);
        else aload(k / 4);
      }
    }
    if constexpr (decltype(gpart)::value) {
      cload();
      ls = next_stage(ls);
    }
  };
  static_assert(4 * FA::LOADS == NBM * NBN && 4 * FG::LOADS == NBM * NBN, "a load every four products");

  // ---- the stream: descriptors of the chunk being multiplied and the ones in flight
  Desc q0 = fetch();
  auto issue_all = [&]() {
#pragma unroll
    for (int i = 0; i < FA::LOADS; ++i) aload(i);
#pragma unroll
    for (int i = 0; i < FG::LOADS; ++i) gload(i);
    cload();
    ls = next_stage(ls);
  };
  issue_all();
  lds_barrier();  // between fetches: see there
  Desc q1 = fetch();
  issue_all();
  lds_barrier();
  Desc q2 = fetch();
  issue_all();
  lds_barrier();
  Desc q3 = fetch();
#pragma unroll
  for (int i = 0; i < FA::LOADS; ++i) aload(i);
  static_assert(ST == 4, "three chunks ahead");
  wait_vmcnt<LPC*(ST - 2) + FA::LOADS>();
  lds_barrier();
  Frags f0, f1;
#pragma unroll
  for (int k = 0; k < NBN + NBM; ++k) read1(l0, 0, f0, k);
  uint32_t cs = l0;

  while (q0.id >= 0) {
    const Item it = item_at(q0.id >> 1);
    const Emit em = emit_at(a, it.e, it.sp);
    zero_acc(acc);
    float prev = 0.f, ref = 0.f;  // ratio: the factor acc is in units of, and that of the run's first sample
    bool flushed = false;
    // this lane's elements inside [0, d) x [0, p): element = f(element, its place in the result)
    auto for_elems = [&](auto f) {
      // an opaque copy of the row stride: the addresses are formed where they are used (rarely), not ahead of
      // the loop and held in registers through it
      int64_t ps = a.p;
      asm volatile("" : "+s"(ps));
      const int64_t lr = it.m0 + wm * WM + 4 * (lane >> 5), lc = it.n0 + wn * WN + (lane & 31);
      float* const base = em.dst + lr * ps + lc;
      const int64_t rem_r = a.d - lr, rem_c = a.p - lc;
#pragma unroll
      for (int i = 0; i < NBM; ++i)
#pragma unroll
        for (int j = 0; j < NBN; ++j)
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            const int ro = i * 32 + 8 * (k >> 2) + (k & 3), co = j * 32;
            if (ro < rem_r && co < rem_c) acc[i][j][k] = f(acc[i][j][k], base + ro * ps + co);
          }
    };
    while (true) {
      bool rescale = false;
      float r = 1.0f;
      if constexpr (RATIO) {
        if (q0.c != 0.0f && q0.c != prev) {
          if (prev != 0.0f) {
            const float mag = fabsf(q0.c), rmag = fabsf(ref);
            rescale = true;
            r = prev / q0.c;
            if (mag < rmag * 0x1p-32f || mag > rmag * 0x1p32f) {
              // factors this far apart would overflow the quotient: bank the sum so far in the result's place
              for_elems([&](float v, float* o) {
                *o = flushed ? *o + v * prev : v * prev;
                return 0.0f;
              });
              flushed = true;
              ref = q0.c;
              rescale = false;
            }
          } else {
            ref = q0.c;
          }
          prev = q0.c;
        }
      }
      step(f0, cs, 0, f1, cs, 1, std::true_type{}, rescale, r);
      const Desc q4 = fetch();
      wait_vmcnt<LPC*(ST - 2)>();
      lds_barrier();
      const uint32_t nx = next_stage(cs);
      step(f1, cs, 1, f0, nx, 0, std::false_type{}, false, 1.0f);
      cs = nx;
      const int end = q0.id & 1;
      q0 = q1;
      q1 = q2;
      q2 = q3;
      q3 = q4;
      if (end) break;
    }
    if constexpr (RATIO) {
      // back to units of 1, and the banked part (if any)
#pragma unroll
      for (int i = 0; i < NBM; ++i)
#pragma unroll
        for (int j = 0; j < NBN; ++j)
#pragma unroll
          for (int k = 0; k < 16; ++k) acc[i][j][k] *= prev;
      if (flushed) for_elems([&](float v, const float* o) { return v + *o; });
    }
    emit_tile<NBM, NBN>(acc, em, a.na, l0 + ST * STAGE + wave * 2048, it.m0 + wm * WM, it.n0 + wn * WN, lane);
  }
  wait_vmcnt<0>();  // the empty loads past the last item: none may land after this workgroup's LDS is given away
}

// Any widths and both types, 128 x 128 tiles, one workgroup per (expert, split,
// tile). FOLD: pieces of one sample; else the expert's rows as they lie (scale
// for fp32, split for bf16).
template <typename T, bool FOLD, bool DMA>
__global__ __launch_bounds__(256) void k_grouped_sum(GSumArgs a) {
  constexpr int BM = 128, BN = 128, WGM = 2, NW = 4, WM = 64, WN = 64, NBM = 2, NBN = 2, ST = 2;
  constexpr bool SPLIT = !FOLD && sizeof(T) == 2;
  constexpr int KB = FOLD ? 64 : 128;
  using OA = Opnd<T, false, BM, KB>;
  using OG = Opnd<T, false, BN, KB>;
  constexpr int KC = OA::KC, STAGE = OA::BYTES + OG::BYTES + (FOLD ? 0 : NW * 256);
  static_assert(!FOLD || (sizeof(T) == 2 && KC == kPieceRows), "fold: bf16 pieces");
  constexpr int NC = 32 / sizeof(T);  // rows per step
  extern __shared__ __attribute__((aligned(1024))) unsigned char lds[];
  const int xcd = (int)(blockIdx.x & 7), local = (int)(blockIdx.x >> 3), tiles = (int)(a.mt * a.nt);
  if (local >= deal_count(a.E * a.ks, tiles, xcd)) return;
  int es, t;
  dealt(tiles, xcd, local, &es, &t);
  const int64_t e = es / a.ks, sp = es - e * a.ks;
  const int64_t m0 = (t % a.mt) * BM, n0 = (t / a.mt) * BN;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave % WGM, wn = wave / WGM;

  // this split's share of the expert's slots (FOLD) or chunks
  const int64_t g0 = e * a.B, g1 = g0 + a.B;
  const int64_t o0 = uniform64(clamp_row(a.seg[g0], a.R)), o1 = uniform64(clamp_row(a.seg[g1], a.R));
  const int64_t s0 = FOLD ? o0 / KC + g0 : 0, s1 = FOLD ? o1 / KC + g1 : (o1 > o0 ? (o1 - o0 + KC - 1) / KC : 0);
  const int64_t share = (s1 - s0 + a.ks - 1) / a.ks;
  const int64_t c0 = s0 + sp * share, c1 = c0 + share < s1 ? c0 + share : s1;

  const int64_t ab = a.d * (int64_t)sizeof(T), gb = a.p * (int64_t)sizeof(T);
  Filler<OA, T, NW> fa;
  Filler<OG, T, NW> fg;
  fa.init(ab, wave, lane);
  fg.init(gb, wave, lane);
  ReadF<T, BM, NBM, KB> ra;
  ReadF<T, BN, NBN, KB> rg;
  ra.init(wm * WM, lane);
  rg.init(wn * WN, lane);
  const uint32_t l0 = lds_addr(lds);

  f32x16 acc[NBM][NBN];
  zero_acc(acc);
  const T* A = static_cast<const T*>(a.A) + m0;
  const T* G = static_cast<const T*>(a.G) + n0;
  auto awin = [&](int64_t row, int64_t rows) { return Win<T>{A + row * a.d, ab, rows, a.d - m0, a.R - 1 - row}; };
  auto gwin = [&](int64_t row, int64_t rows) { return Win<T>{G + row * a.p, gb, rows, a.p - n0, a.R - 1 - row}; };

  if constexpr (FOLD) {
    f32x16 tmp[NBM][NBN];
    zero_acc(tmp);
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
    };
    // the pieces in use, 64 slots at a time: lane i holds slot pos + i
    int64_t pos = c0;
    uint64_t mask = 0;
    Piece mine{0, 0, 0.f, 0};
    auto load64 = [&]() {
      mine = Piece{0, 0, 0.f, 0};
      if (pos + lane < c1) mine = a.pieces[pos + lane];
      mask = __ballot(mine.rows > 0 && mine.c != 0.0f);  // a factor of 0: its rows add nothing
    };
    auto next = [&](Piece* pc) -> bool {
      while (mask == 0) {
        pos += 64;
        if (pos >= c1) return false;
        load64();
      }
      const int i = __ffsll((unsigned long long)mask) - 1;
      mask &= mask - 1;
      pc->row0 = __builtin_amdgcn_readlane(mine.row0, i);
      pc->rows = __builtin_amdgcn_readlane(mine.rows, i);
      pc->c = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(mine.c), i));
      return true;
    };
    auto use = [&](const Piece& pc, uint32_t sb) {
      if (!(pc.c == cur)) {  // another factor (or NaN): what was gathered under the last one is folded in
        fold();
        cur = pc.c;
      }
      chunk_mma<T, NBM, NBN>(sb, sb + OA::BYTES, ra, rg, pc.rows > 16 ? 2 : 1, tmp);
    };
    if (c0 < c1) {
      load64();
      Piece cp, np{0, 0, 0.f, 0};
      bool have = next(&cp);
      if constexpr (DMA) {
        auto issue = [&](const Piece& pc, uint32_t sb) {
          fa.dma(awin(pc.row0, pc.rows), sb, wave);
          fg.dma(gwin(pc.row0, pc.rows), sb + OA::BYTES, wave);
        };
        uint32_t sb = l0, sn = l0 + STAGE;
        if (have) issue(cp, sb);
        while (have) {
          wait_vmcnt<0>();
          lds_barrier();
          const bool more = next(&np);
          if (more) issue(np, sn);
          use(cp, sb);
          cp = np;
          have = more;
          const uint32_t x = sb;
          sb = sn;
          sn = x;
        }
      } else {
        u32x4 va[Filler<OA, T, NW>::LOADS], vg[Filler<OG, T, NW>::LOADS];
        auto load = [&](const Piece& pc) {
          fa.load(awin(pc.row0, pc.rows), va, wave, lane);
          fg.load(gwin(pc.row0, pc.rows), vg, wave, lane);
        };
        if (have) load(cp);
        while (have) {
          __syncthreads();
          fa.store(va, lds, wave, lane);
          fg.store(vg, lds + OA::BYTES, wave, lane);
          __syncthreads();
          const bool more = next(&np);
          if (more) load(np);
          use(cp, l0);
          cp = np;
          have = more;
        }
      }
      fold();
    }
  } else {
    auto chunk = [&](uint32_t sb) {
      const uint32_t cb = sb + OA::BYTES + OG::BYTES + wave * 256;
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        u32x4 fragA[NBM], fragG[NBN];
#pragma unroll
        for (int i = 0; i < NBM; ++i) fragA[i] = ra.get(sb, s, i);
#pragma unroll
        for (int j = 0; j < NBN; ++j) fragG[j] = rg.get(sb + OA::BYTES, s, j);
        const uint32_t cl = cb + 4 * (NC * s + NC / 2 * (lane >> 5));
        f32x4 ck[2];
        ck[0] = __builtin_bit_cast(f32x4, *(lds_u32x4*)(uintptr_t)cl);
        if constexpr (SPLIT) {
          ck[1] = __builtin_bit_cast(f32x4, *(lds_u32x4*)(uintptr_t)(cl + 16));
#pragma unroll
          for (int i = 0; i < NBM; ++i) {
            u32x4 tr[3];
            split_scaled(fragA[i], ck, tr);
#pragma unroll
            for (int u = 2; u >= 0; --u)
#pragma unroll
              for (int j = 0; j < NBN; ++j) acc[i][j] = mfma32_bf16(tr[u], fragG[j], acc[i][j]);
          }
        } else {
#pragma unroll
          for (int i = 0; i < NBM; ++i)
#pragma unroll
            for (int e4 = 0; e4 < 4; ++e4) fragA[i][e4] = __float_as_uint(__uint_as_float(fragA[i][e4]) * ck[0][e4]);
#pragma unroll
          for (int i = 0; i < NBM; ++i)
#pragma unroll
            for (int j = 0; j < NBN; ++j) acc[i][j] = mma_step<T>(fragA[i], fragG[j], acc[i][j]);
        }
      }
    };
    auto crows = [&](int64_t q, uint32_t dst) {  // the chunk's factors (KC <= 64 of them), a copy per wave
      const int64_t row = o0 + q * KC, left = o1 - row < KC ? o1 - row : KC;
      dma4_buf(make_srd(a.crow + row, 4u * (uint32_t)left), 4u * lane, dst + wave * 256);
    };
    auto rows_of = [&](int64_t q) { return o1 - (o0 + q * KC); };
    if constexpr (DMA) {
      auto issue = [&](int64_t q) {
        const uint32_t sb = l0 + (uint32_t)((q - c0) % ST) * STAGE;
        fa.dma(awin(o0 + q * KC, rows_of(q)), sb, wave);
        fg.dma(gwin(o0 + q * KC, rows_of(q)), sb + OA::BYTES, wave);
        crows(q, sb + OA::BYTES + OG::BYTES);
      };
      if (c0 < c1) issue(c0);
      for (int64_t q = c0; q < c1; ++q) {
        wait_vmcnt<0>();
        lds_barrier();
        if (q + 1 < c1) issue(q + 1);
        chunk(l0 + (uint32_t)((q - c0) % ST) * STAGE);
      }
    } else {
      u32x4 va[Filler<OA, T, NW>::LOADS], vg[Filler<OG, T, NW>::LOADS];
      float vc = 0.f;  // lane l < KC: the factor of the chunk's row l
      auto load = [&](int64_t q) {
        fa.load(awin(o0 + q * KC, rows_of(q)), va, wave, lane);
        fg.load(gwin(o0 + q * KC, rows_of(q)), vg, wave, lane);
        vc = lane < KC && lane < rows_of(q) ? a.crow[o0 + q * KC + lane] : 0.f;
      };
      if (c0 < c1) load(c0);
      for (int64_t q = c0; q < c1; ++q) {
        __syncthreads();
        fa.store(va, lds, wave, lane);
        fg.store(vg, lds + OA::BYTES, wave, lane);
        *reinterpret_cast<float*>(lds + OA::BYTES + OG::BYTES + wave * 256 + 4 * lane) = vc;
        __syncthreads();
        if (q + 1 < c1) load(q + 1);
        chunk(l0);
      }
    }
  }
  __syncthreads();  // the stages are free: the epilogue's scratch lies over them
  emit_tile<NBM, NBN>(acc, emit_at(a, e, sp), a.na, l0 + wave * 2048, m0 + wm * WM, n0 + wn * WN, lane);
}

// The splits' sums added in order, noise and mean applied, for widths without
// 16-byte vectors: a thread takes one column of a row quad, lanes side by side
// (the layers' reduce gives a thread 4 x 4 elements, 16 loads of 4 bytes a
// split: 20 us against 11 at six splits of 1665 x 517).
__global__ __launch_bounds__(256) void k_grouped_reduce(GSumArgs a, NoiseArgs na) {
  const int64_t rows = a.E * a.d, n = (rows + 3) / 4 * a.p, stride = rows * a.p;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
    const int64_t q = i / a.p, at = 4 * q * a.p + (i - q * a.p);
    float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
    for (int64_t k = 0; k < a.ks; ++k)
#pragma unroll
      for (int r = 0; r < 4; ++r)
        if (4 * q + r < rows) s[r] += a.part[k * stride + at + r * a.p];
    f32x4 z = {0.f, 0.f, 0.f, 0.f};
    if (na.sc != 0.0f) z = normals4((uint32_t)i, 2u * na.layer, na.step, 0u, na.k0, na.k1);
#pragma unroll
    for (int r = 0; r < 4; ++r)
      if (4 * q + r < rows) a.out[at + r * a.p] = noised_mean_spec(s[r], na.sc, z[r], na.inv_denom);
  }
}

// ---------------------------------------------------------------------------
namespace {

bool dma_ok(int dtype, std::initializer_list<int64_t> widths) {
  for (int64_t v : widths)
    if (v % (dtype == 1 ? 8 : 4)) return false;
  return true;
}

// More than 64 KB of LDS per workgroup has to be asked for.
template <typename F>
hipError_t dyn_lds(F* f, int bytes) {
  if (bytes <= 64 * 1024) return hipSuccess;
  return hipFuncSetAttribute(reinterpret_cast<const void*>(f), hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
}

size_t round256(size_t x) { return (x + 255) / 256 * 256; }

// Tile and K splits of a product: the least of the measured times per chunk
// of 32 K and per item, in rounds of items over the CUs, plus the traffic of the
// splits' partial products and their joining launch. 256 x 256 tiles (bf16)
// read the fewest operand bytes per product; 128 x 128 tiles run two to a CU;
// tiles of 32 rows waste little on experts with few rows, and K can be split
// for them, so that single tokens' weights are read by the whole GPU. The wide
// tile takes up to 64 experts, one a lane (32768 rows of 1280 x 1280: 188 us over
// 64 experts, 193 us over 65 on 128 x 128 tiles). Widths without 16-byte vectors
// have the 128 x 128 tile alone (8192 rows over 8 experts, 1281 x 5119: 290 us,
// 117 at 1280 x 5120; 8 rows, 5119 x 517: 83 us, 15 at 5120 x 512).
struct MatmulPlan {
  int bm;
  int64_t ks, kper;
};
// A grid of 256-thread workgroups, rounded up to the XCDs, has fewer than 2^32 threads.
constexpr int64_t kMaxGrid = ((int64_t)1 << 24) - 8;
int64_t matmul_items(int64_t bm, int64_t R, int64_t E, int64_t N, int64_t ks) {
  return (R / bm + E) * ((N + 127) / 128) * ks;
}
MatmulPlan matmul_plan(int dtype, int64_t R, int64_t E, int64_t K, int64_t N) {
  const bool bf16 = dtype == 1, dma = dma_ok(dtype, {K, N});
  MatmulPlan best{128, 1, K};
  if (!dma) return best;
  const int64_t kc = bf16 ? 64 : 32;  // K per chunk of the smaller tiles
  const double k32 = std::ceil((double)K / 32);
  double best_us = 1e30;
  auto consider = [&](int bm, int bn, int64_t ks, int64_t kper, double chunk_us, double item_us, int per_cu) {
    if (bm == 32 && matmul_items(bm, R, E, N, ks) > kMaxGrid) return;
    const double tiles = ((double)R / bm + 0.5 * (double)std::min(E, R)) * (double)((N + bn - 1) / bn) * (double)ks;
    // workgroups that share a CU share its matrix cores
    const double share = tiles <= 256 ? 1.0 / per_cu : 1.0;
    const double us = std::ceil(tiles / (256.0 * per_cu)) * (k32 / (double)ks * chunk_us * share + item_us) +
                      (ks > 1 ? (double)ks * R * N * 8.0 / 4.5e6 + 5.0 : 0.0);
    if (us < best_us) {
      best_us = us;
      best = MatmulPlan{bm, ks, kper};
    }
  };
  if (bf16 && E <= 64 && K >= 128) consider(256, 256, 1, K, 1.0, 9.0, 1);
  consider(128, 128, 1, K, bf16 ? 0.66 : 4.8, 5.0, 2);
  const int64_t chunks = (K + kc - 1) / kc;
  for (int64_t want = 1; want <= 32 && want * 2 <= std::max<int64_t>(2, chunks); want *= 2) {
    const int64_t kper = (chunks + want - 1) / want * kc, ks = (K + kper - 1) / kper;
    consider(32, 128, ks, kper, bf16 ? 0.3 : 1.35, 5.0, 2);
  }
  return best;
}

template <typename T, bool TRANS, int BM, int BN, int WGM, int WGN, int KB, int ST, bool DMA, bool SPLIT>
hipError_t run_matmul(hipStream_t st, MatmulArgs a) {
  auto* f = &k_grouped_matmul<T, TRANS, BM, BN, WGM, WGN, KB, ST, DMA, SPLIT>;
  constexpr int LDS = (DMA ? ST : 1) * (BM + BN) * KB;
  a.slots = a.R / BM + a.E;
  a.ntn = (a.N + BN - 1) / BN;
  hipError_t e = dyn_lds(f, LDS);
  if (e != hipSuccess) return e;
  f<<<dim3((unsigned)xcd_grid(a.slots * a.ntn * a.ks)), 64 * WGM * WGN, LDS, st>>>(a);
  return hipGetLastError();
}

template <bool TRANS>
hipError_t run_matmul_big(hipStream_t st, MatmulArgs a) {
  auto* f = &k_grouped_matmul_big<TRANS>;
  constexpr int LDS = 4 * 512 * 64 + 8 * 4096;
  a.ntn = (a.N + 255) / 256;
  hipError_t e = dyn_lds(f, LDS);
  if (e != hipSuccess) return e;
  f<<<dim3((unsigned)std::min<int64_t>(256, xcd_grid((a.R / 256 + a.E) * a.ntn))), 512, LDS, st>>>(a);
  return hipGetLastError();
}

template <typename T, bool TRANS>
hipError_t matmul_t(hipStream_t st, int dtype, MatmulArgs a) {
  const MatmulPlan m = matmul_plan(dtype, a.R, a.E, a.K, a.N);
  a.ks = m.ks;
  a.kper = m.kper;
  if (!dma_ok(dtype, {a.K, a.N})) return run_matmul<T, TRANS, 128, 128, 2, 2, 128, 2, false, false>(st, a);
  if (m.bm == 32) {
    if (a.ks == 1) return run_matmul<T, TRANS, 32, 128, 1, 4, 128, 3, true, false>(st, a);
    hipError_t e = run_matmul<T, TRANS, 32, 128, 1, 4, 128, 3, true, true>(st, a);
    if (e != hipSuccess) return e;
    const int64_t blocks = std::min<int64_t>((a.R * a.N + 255) / 256, 4096);
    k_grouped_join<T><<<dim3((unsigned)blocks), 256, 0, st>>>(a);
    return hipGetLastError();
  }
  if constexpr (sizeof(T) == 2) {
    if (m.bm == 256) return run_matmul_big<TRANS>(st, a);
  }
  return run_matmul<T, TRANS, 128, 128, 2, 2, 128, 2, true, false>(st, a);
}

// The norm's kernel by the average rows per segment, and the workgroups per
// row tile (enough for segments three times as long as the average). The sizes
// of single segments are known on the device only: a routing that sends 16384
// rows to one of 1024 segments takes the packed tiles (1280 + 1280 bf16: 5.6 ms,
// 61 us dealt evenly; its pairs' products alone are 0.67 TFLOP).
struct NormPlan {
  bool packed;
  int64_t ts, J;
};
NormPlan norm_plan(int dtype, const GroupedArgs& g) {
  const int64_t avg = g.R / (g.E * g.B), ts = dtype == 1 ? norm_tile<bf16s>() : norm_tile<float>();
  // row tiles whose grid takes at least one workgroup each, else packed tiles, whose workgroups go over the items
  const int64_t most = kMaxGrid / ((g.R / ts + g.E * g.B + 31) / 32 * 32);
  if (avg < 64 || most < 1) return NormPlan{true, 32, 1 + (std::min<int64_t>(avg, 63) + 15) / 16};
  return NormPlan{false, ts, std::max<int64_t>(1, std::min({(int64_t)16, most, (3 * avg + ts - 1) / ts}))};
}
int64_t piece_slots(const GroupedArgs& g) { return g.R / kPieceRows + g.E * g.B; }

// The clipped sum's kernel, tile and K splits: 256 x 256 tiles (bf16, aligned
// widths) where the layer is wide enough to fill them.
struct SumPlan {
  bool big, pieces, dma, fused;
  int64_t mt, nt, ks;
};
constexpr int64_t kMaxSumItems = (int64_t)1 << 23;  // (expert, split, tile) items of a sum: an XCD's share is an int
// The items of the XCD with the most of them.
int64_t most_items(int64_t pairs, int64_t tiles) {
  int most = 0;
  for (int xcd = 0; xcd < 8; ++xcd) most = std::max(most, deal_count(pairs, tiles, xcd));
  return most;
}
SumPlan sum_plan(int dtype, const GroupedArgs& g) {
  SumPlan best{};
  double best_us = 1e30;
  const bool dma = dma_ok(dtype, {g.d, g.p}), pieces = dtype == 1 && g.R / (g.E * g.B) >= 16;
  const double out_us = (double)g.E * g.d * g.p * 8.0 / 4.5e6;  // a split's sums written and read once, 4.5 TB/s
  const int64_t chunks = std::max<int64_t>(1, g.R / g.E / 32);
  for (int big = 0; big < 2; ++big) {
    if (big && !(dtype == 1 && dma && g.d >= 192 && g.p >= 192)) continue;
    SumPlan s{};
    s.big = big;
    s.pieces = pieces;
    s.dma = dma;
    const int64_t t = big ? 256 : 128;
    s.mt = (g.d + t - 1) / t;
    s.nt = (g.p + t - 1) / t;
    // rounds of items over the CUs (one 256 x 256 tile or two 128 x 128 tiles at a time), each the time of its
    // 32-row chunks and a fixed part, as measured; then the traffic of the splits' sums and their reduce launch
    const double slots = big ? 256 : 512, item_us = big ? 20 : 6;
    const double chunk_us = big ? (pieces ? 1.1 : 1.7) : dtype == 1 ? (pieces ? 1.3 : 2.5) : dma ? 4.0 : 6.5;
    for (int64_t ks = 1; ks <= 64 && (ks == 1 || (ks * 2 <= chunks && g.E * ks * s.mt * s.nt < kMaxSumItems));
         ks = ks < 4 ? ks + 1 : ks * 3 / 2) {
      const double items = (double)(8 * most_items(g.E * ks, s.mt * s.nt));
      const double us = std::ceil(items / slots) * (std::ceil((double)chunks / ks) * chunk_us + item_us) +
                        (ks > 1 ? ks * out_us + 14.0 : 0.0);
      if (us < best_us) {
        best_us = us;
        s.ks = ks;
        best = s;
      }
    }
  }
  best.fused = best.ks == 1 && g.d % 4 == 0;
  return best;
}

template <typename T>
hipError_t run_norm(hipStream_t st, int dtype, GNormArgs a, const NormPlan& pl, float* sqnorm, int accumulate) {
  const unsigned fin = (unsigned)std::min<int64_t>(a.B, 1 << 20);
  a.J = pl.J;
  if (pl.packed) {
    k_grouped_row_segments<<<dim3((unsigned)((a.R + 255) / 256)), 256, 0, st>>>(a.seg, a.R, a.E * a.B, a.row_seg);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const int64_t items = (a.R + 31) / 32 * a.J;
    k_grouped_norm_packed<T><<<dim3((unsigned)std::min<int64_t>(items, 1 << 20)), 256, 0, st>>>(a);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
    k_grouped_norm_finish<true, 32><<<fin, 256, 0, st>>>(a, sqnorm, accumulate);
    return hipGetLastError();
  }
  constexpr int TS = norm_tile<T>();
  a.slots = a.R / TS + a.E * a.B;
  const bool dma = dma_ok(dtype, {a.d, a.p});
  const int lds = (dma ? 2 : 1) * 2 * TS * 128;
  const unsigned grid = (unsigned)((a.slots + 31) / 32 * 32 * a.J);
  hipError_t e;
  if (dma) {
    auto* f = &k_grouped_norm<T, true>;
    e = dyn_lds(f, lds);
    if (e != hipSuccess) return e;
    f<<<dim3(grid), 256, lds, st>>>(a);
  } else {
    auto* f = &k_grouped_norm<T, false>;
    e = dyn_lds(f, lds);
    if (e != hipSuccess) return e;
    f<<<dim3(grid), 256, lds, st>>>(a);
  }
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  k_grouped_norm_finish<false, TS><<<fin, 256, 0, st>>>(a, sqnorm, accumulate);
  return hipGetLastError();
}

template <typename F>
hipError_t run_sum(F* f, hipStream_t st, const GSumArgs& a, int64_t grid, int threads, int lds) {
  hipError_t e = dyn_lds(f, lds);
  if (e != hipSuccess) return e;
  f<<<dim3((unsigned)grid), threads, lds, st>>>(a);
  return hipGetLastError();
}

}  // namespace

size_t grouped_matmul_ws_bytes(int dtype, const GroupedArgs& g) {
  size_t need = 0;
  for (int tr = 0; tr < 2; ++tr) {
    const int64_t K = tr ? g.p : g.d, N = tr ? g.d : g.p;
    const MatmulPlan m = matmul_plan(dtype, g.R, g.E, K, N);
    if (m.ks > 1) need = std::max(need, round256((size_t)m.ks * (size_t)g.R * (size_t)N * sizeof(float)));
  }
  return need;
}

hipError_t launch_grouped_matmul(hipStream_t st, int dtype, const GroupedArgs& g, const void* X, const void* W,
                                 bool transpose, void* ws, void* Y) {
  MatmulArgs a{};
  a.X = X;
  a.W = W;
  a.Y = Y;
  a.part = static_cast<float*>(ws);
  a.seg = g.seg;
  a.B = g.B;
  a.E = g.E;
  a.R = g.R;
  a.K = transpose ? g.p : g.d;
  a.N = transpose ? g.d : g.p;
  if (dtype == 1) return transpose ? matmul_t<bf16s, true>(st, dtype, a) : matmul_t<bf16s, false>(st, dtype, a);
  return transpose ? matmul_t<float, true>(st, dtype, a) : matmul_t<float, false>(st, dtype, a);
}

size_t grouped_norm_ws_bytes(int dtype, const GroupedArgs& g) {
  const NormPlan pl = norm_plan(dtype, g);
  if (pl.packed) return round256((size_t)g.R * (size_t)pl.J * sizeof(float)) + round256((size_t)g.R * sizeof(int32_t));
  return round256((size_t)(g.R / pl.ts + g.E * g.B) * (size_t)pl.J * sizeof(float));
}

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
  const NormPlan pl = norm_plan(dtype, g);
  a.row_seg = reinterpret_cast<int32_t*>(static_cast<char*>(ws) +
                                         round256((size_t)g.R * (size_t)pl.J * sizeof(float)));
  return dtype == 1 ? run_norm<bf16s>(st, dtype, a, pl, sqnorm, accumulate)
                    : run_norm<float>(st, dtype, a, pl, sqnorm, accumulate);
}

// workspace: the XCDs' item queues, the piece list or the rows' factors, then the splits' sums
constexpr size_t kQueueBytes = 256;
size_t sum_list_bytes(const SumPlan& s, const GroupedArgs& g) {
  return kQueueBytes + round256(s.pieces ? (size_t)piece_slots(g) * sizeof(Piece) : (size_t)g.R * sizeof(float));
}
size_t grouped_sum_ws_bytes(int dtype, const GroupedArgs& g) {
  const SumPlan s = sum_plan(dtype, g);
  return sum_list_bytes(s, g) +
         (s.fused ? 0 : round256((size_t)s.ks * (size_t)g.E * (size_t)g.d * (size_t)g.p * sizeof(float)));
}

hipError_t launch_grouped_sum(hipStream_t st, int dtype, const GroupedArgs& g, const void* A, const void* G,
                              const float* c, void* ws, const NoiseArgs& na, float* out) {
  const SumPlan s = sum_plan(dtype, g);
  const bool fused = s.fused || (s.ks == 1 && na.sc == 0.0f);  // without noise the quads do not matter
  GSumArgs a{};
  a.queue = static_cast<int32_t*>(ws);
  void* list = static_cast<char*>(ws) + kQueueBytes;
  if (s.pieces) {
    Piece* pieces = static_cast<Piece*>(list);
    const int64_t slots = piece_slots(g);
    k_grouped_pieces<<<dim3((unsigned)((slots + 255) / 256)), 256, 0, st>>>(g.seg, g.R, g.E, g.B, c, slots, pieces,
                                                                            a.queue);
    a.pieces = pieces;
  } else {
    float* crow = static_cast<float*>(list);
    k_grouped_row_factors<<<dim3((unsigned)((g.R + 255) / 256)), 256, 0, st>>>(g.seg, g.R, g.E, g.B, c, crow, a.queue);
    a.crow = crow;
  }
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  a.A = A;
  a.G = G;
  a.seg = g.seg;
  a.R = g.R;
  a.E = g.E;
  a.B = g.B;
  a.d = g.d;
  a.p = g.p;
  a.mt = s.mt;
  a.nt = s.nt;
  a.ks = s.ks;
  a.na = fused ? na : make_noise_args(0.0f, 1.0f, 0, 0, 0);
  a.out = out;
  a.fused = fused;
  a.part = reinterpret_cast<float*>(static_cast<char*>(ws) + sum_list_bytes(s, g));
  if (s.big) {
    const int64_t grid = 8 * std::min<int64_t>(32, most_items(g.E * s.ks, s.mt * s.nt));
    e = s.pieces ? run_sum(&k_grouped_sum_big<true>, st, a, grid, 512, 4 * 32768 + 8 * 2048)
                 : run_sum(&k_grouped_sum_big<false>, st, a, grid, 512, 4 * (32768 + 1024) + 8 * 2048);
  } else {
    const int64_t grid = 8 * most_items(g.E * s.ks, s.mt * s.nt);
    const int st_n = s.dma ? 2 : 1;
    if (dtype == 1 && s.pieces)
      e = s.dma ? run_sum(&k_grouped_sum<bf16s, true, true>, st, a, grid, 256, st_n * 16384)
                : run_sum(&k_grouped_sum<bf16s, true, false>, st, a, grid, 256, st_n * 16384);
    else if (dtype == 1)
      e = s.dma ? run_sum(&k_grouped_sum<bf16s, false, true>, st, a, grid, 256, st_n * (32768 + 1024))
                : run_sum(&k_grouped_sum<bf16s, false, false>, st, a, grid, 256, st_n * (32768 + 1024));
    else
      e = s.dma ? run_sum(&k_grouped_sum<float, false, true>, st, a, grid, 256, st_n * (32768 + 1024))
                : run_sum(&k_grouped_sum<float, false, false>, st, a, grid, 256, st_n * (32768 + 1024));
  }
  if (e != hipSuccess || fused) return e;
  if (g.p % 4) {
    const int64_t n = (g.E * g.d + 3) / 4 * g.p;
    k_grouped_reduce<<<dim3((unsigned)std::min<int64_t>((n + 255) / 256, 1 << 16)), 256, 0, st>>>(a, na);
    return hipGetLastError();
  }
  return launch_split_reduce(st, a.ks, a.part, g.E * g.d, g.p, na, out);
}

bool grouped_fits(const GroupedArgs& g, GroupedCall call, int dtype) {
  if (call == GroupedCall::norm) return true;  // the plan takes any size
  if (call == GroupedCall::sum) return g.E * ((g.d + 127) / 128) * ((g.p + 127) / 128) < kMaxSumItems;
  const bool tr = call == GroupedCall::matmul_transposed;
  const int64_t N = tr ? g.d : g.p;
  const MatmulPlan m = matmul_plan(dtype, g.R, g.E, tr ? g.p : g.d, N);
  return m.bm == 256 || matmul_items(m.bm, g.R, g.E, N, m.ks) <= kMaxGrid;
}

}  // namespace dpk
