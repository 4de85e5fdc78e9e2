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
