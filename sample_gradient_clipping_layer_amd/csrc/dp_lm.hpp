// Host-side launchers of the language-model operators (internal to
// libdpclip), and device helpers they share.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <initializer_list>
#include <type_traits>

#include "dp_common.hpp"
#include "dp_launch.hpp"

namespace dpk {

// fp32 -> bf16 bits, to nearest even. The compiler's conversion is the
// hardware's: NaN stays NaN.
__device__ __forceinline__ uint16_t f32_to_bf16(float v) { return __builtin_bit_cast(uint16_t, (__bf16)v); }
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  return (uint32_t)f32_to_bf16(lo) | ((uint32_t)f32_to_bf16(hi) << 16);
}

// ---- root-mean-square norm
constexpr int64_t kRmsMaxWidth = 32768;
struct RmsArgs {
  const void *x, *residual;  // residual may be null
  const void* gain;
  int gain_bf16;
  float eps;
  int64_t rows, d;
  void *out, *sum_out;  // sum_out may be null
};
struct RmsBackArgs {
  const void *dy, *s, *dsum;  // dsum may be null
  const void* gain;
  int gain_bf16;
  float eps;
  int64_t B, T, d;
  void* dx;          // may be null
  float* gain_rows;  // [B][d], may be null
  float* partial;    // [B][chunks][d] when chunks > 1
  // set by the launcher
  int64_t chunks, chunk_rows;
  int own_groups;
};
int64_t rms_chunks(int64_t B, int64_t T);
hipError_t launch_rms_norm(hipStream_t st, int dtype, const RmsArgs& a);
hipError_t launch_rms_norm_backward(hipStream_t st, int dtype, RmsBackArgs a);

// ---- layer norm
struct LayerNormArgs {
  const void *x, *residual;  // residual may be null
  const void *gain, *bias;   // one type; bias may be null
  int gain_bf16;
  float eps;
  int64_t rows, d;
  void *out, *sum_out;  // sum_out may be null
};
struct LayerNormBackArgs {
  const void *dy, *s, *dsum;  // dsum may be null
  const void* gain;
  int gain_bf16;
  float eps;
  int64_t B, T, d;
  void* dx;                        // may be null
  float *gain_rows, *bias_rows;    // [B][d], may be null
  float* partial;                  // [2][B][chunks][d] when chunks > 1
  // set by the launcher
  int64_t chunks, chunk_rows;
  int own_groups;
};
int64_t layer_norm_chunks(int dtype, int64_t B, int64_t T, int64_t d);
hipError_t launch_layer_norm(hipStream_t st, int dtype, const LayerNormArgs& a);
hipError_t launch_layer_norm_backward(hipStream_t st, int dtype, LayerNormBackArgs a);

// ---- table of words
constexpr int kEmbedTile = 16;         // places (or tiles) of a tile
constexpr int kEmbedMaxLevels = 8;
constexpr int kEmbedNormPlaces = 8;    // places whose runs a wave sums
struct EmbedArgs {
  const int64_t* ids;  // [N]
  const void* weight;  // [V][d]
  int64_t N, V, d;
  float scale;
  void* out;  // [N][d]
};
struct EmbedGradArgs {
  const void* G;         // [N][d]
  const int64_t* order;  // [N]
  const int64_t* starts; // [V + 1] (sum)
  const float* c;        // [B] (sum)
  int64_t N, B, T, V, d; // N = B T
  FastDiv by_t;
  float scale;
  float* sqnorm;  // [B] (norm)
  int accumulate;
  // set by the launcher
  float* token_sq;  // [parts of the columns][N] (norm)
  float* sums;      // tiles' sums, [rows of all levels][d]
  int levels;
  int64_t level_at[kEmbedMaxLevels];  // first row of a level in sums
};
size_t embed_order_ws_bytes(int64_t N, int64_t V);
size_t embed_ws_bytes(int dtype, int64_t B, int64_t T, int64_t d);
hipError_t launch_embedding(hipStream_t st, int dtype, int weight_dtype, const EmbedArgs& a);
hipError_t launch_embed_order(hipStream_t st, const int64_t* ids, int64_t N, int64_t V, void* ws, int64_t* order,
                              int64_t* starts);
hipError_t launch_embed_norm(hipStream_t st, int dtype, EmbedGradArgs a, void* ws);
hipError_t launch_embed_sum(hipStream_t st, int dtype, EmbedGradArgs a, void* ws, const NoiseArgs& na, float* out);

// ---- log probabilities of given tokens
constexpr int64_t kLogprobMaxTop = 256;
struct LogprobArgs {
  const void* logits;      // [rows][V]
  const int64_t* targets;  // [rows]
  float tau;
  int64_t rows, V, K;
  float *logp, *entropy;   // [rows]; entropy may be null
  float* stats;            // [rows][2]
  int64_t* top_ids;        // [rows][K], null when K == 0
  float* top_logp;
  // backward
  const float *dlogp, *dentropy;  // [rows], either may be null
  void* grad;              // [rows][V]
  int64_t splits;          // set by the launcher
};
hipError_t launch_token_logprob(hipStream_t st, int dtype, const LogprobArgs& a);
hipError_t launch_token_logprob_backward(hipStream_t st, int dtype, LogprobArgs a);

// ---- balance loss
constexpr int64_t kBalanceMaxExperts = 1024;
struct BalanceArgs {
  const void* logits;   // [B][T][E]
  const int64_t* ids;   // [B][T][top]
  int64_t B, T, E, top;
  float* loss;          // [B]
  int64_t *counts, *tokens;  // [B][E], [B]
  const float* dloss;   // [B] or null
  void* grad;           // [B][T][E]
  // set by the launcher
  int64_t chunks, chunk_rows;
  float* part_sums;     // [B][chunks][E] sums of probabilities (chunks > 1)
  uint32_t* part_counts;  // [B][chunks][E + 1] used places per expert, used tokens
};
size_t balance_ws_bytes(int64_t B, int64_t T, int64_t E);
hipError_t launch_balance_loss(hipStream_t st, int dtype, BalanceArgs a, void* ws);
hipError_t launch_balance_backward(hipStream_t st, int dtype, BalanceArgs a);

// ---- distillation loss
constexpr int64_t kDistillMaxTop = 2048;
struct DistillArgs {
  const void* logits;
  const int64_t* ids;
  const void* teacher;
  int teacher_bf16;
  const float* weight;  // [B][T] or null
  float tau;
  int64_t B, T, V, K;
  float* loss;        // [B]
  float* lse;         // [B][T]
  float* row_loss;    // workspace [B][T] (T > 1)
  const float* dloss; // [B] or null
  void* grad;         // backward: [B][T][V]
  int64_t splits;     // set by the launcher
};
hipError_t launch_distill_loss(hipStream_t st, int dtype, DistillArgs a);
hipError_t launch_distill_backward(hipStream_t st, int dtype, DistillArgs a);

// ---- products grouped by expert
struct GroupedArgs {
  const int64_t* seg;  // [E*B + 1]
  int64_t R, E, B, d, p;
};
hipError_t launch_grouped_matmul(hipStream_t st, int dtype, const GroupedArgs& g, const void* X, const void* W,
                                 bool transpose, void* ws, void* Y);
size_t grouped_matmul_ws_bytes(int dtype, const GroupedArgs& g);
hipError_t launch_grouped_norm(hipStream_t st, int dtype, const GroupedArgs& g, const void* A, const void* G, void* ws,
                               float* sqnorm, int accumulate);
size_t grouped_norm_ws_bytes(int dtype, const GroupedArgs& g);
hipError_t launch_grouped_sum(hipStream_t st, int dtype, const GroupedArgs& g, const void* A, const void* G,
                              const float* c, void* ws, const NoiseArgs& na, float* out);
size_t grouped_sum_ws_bytes(int dtype, const GroupedArgs& g);
enum class GroupedCall { matmul, matmul_transposed, norm, sum };
bool grouped_fits(const GroupedArgs& g, GroupedCall call, int dtype);  // a launch of the call takes these sizes

}  // namespace dpk
