// extern "C" entry points of the language-model operators (declared in
// include/dpclip.h): root-mean-square norm, distillation loss, products
// grouped by expert. As in dp_abi.hip, every argument is validated before the
// first HIP call, and nothing is synchronised.
#include <math.h>
#include <stdint.h>

#include <algorithm>

#include "../../include/dpclip.h"
#include "dp_lm.hpp"

namespace {

constexpr int64_t kMaxDim = (int64_t)1 << 31;
constexpr int64_t kMaxElems = (int64_t)1 << 50;
constexpr int64_t kMaxRowWidth = (int64_t)1 << 20;  // grouped products: a 256-row window's bytes fit 31 bits
constexpr int64_t kMaxRows = (int64_t)1 << 30;      // rows, and rows rounded up to chunks, fit 31 bits
constexpr int64_t kMaxRanges = (int64_t)1 << 24;    // (expert, sample) ranges

bool aligned(const void* ptr, uintptr_t a) { return (reinterpret_cast<uintptr_t>(ptr) & (a - 1)) == 0; }
bool finite(float x) { return isfinite(x) != 0; }
bool dtype_ok(dp_dtype t) { return t == DP_F32 || t == DP_BF16; }
uintptr_t elem_bytes(dp_dtype t) { return t == DP_BF16 ? 2 : 4; }
size_t round256(size_t x) { return (x + 255) / 256 * 256; }

dp_status device_ready() {
  int n = 0;
  if (hipGetDeviceCount(&n) != hipSuccess || n < 1) return DP_ERR_NO_DEVICE;
  return DP_OK;
}
dp_status hip_status(hipError_t e) { return e == hipSuccess ? DP_OK : DP_ERR_HIP; }

dp_status check_workspace(const void* ws, size_t have, size_t need) {
  if (need == 0) return DP_OK;
  if (!ws) return DP_ERR_NULL;
  if (have < need) return DP_ERR_WORKSPACE;
  if (!aligned(ws, 16)) return DP_ERR_ALIGN;
  return DP_OK;
}

dp_status check_rms(int64_t B, int64_t T, int64_t d) {
  if (B < 1 || T < 1 || d < 1 || d > dpk::kRmsMaxWidth) return DP_ERR_SHAPE;
  if (B >= kMaxDim || T >= kMaxDim || B * T > kMaxElems / d) return DP_ERR_SHAPE;
  return DP_OK;
}

size_t rms_ws_bytes(int64_t B, int64_t T, int64_t d) {
  const int64_t chunks = dpk::rms_chunks(B, T);
  return chunks > 1 ? round256((size_t)B * (size_t)chunks * (size_t)d * sizeof(float)) : 0;
}

dp_status check_distill(int64_t B, int64_t T, int64_t V, int64_t K, float tau) {
  if (B < 1 || T < 1 || V < 1 || K < 1 || K > dpk::kDistillMaxTop) return DP_ERR_SHAPE;
  if (B >= kMaxDim || T >= kMaxDim || V >= kMaxDim || B * T > kMaxElems / V) return DP_ERR_SHAPE;
  if (!(tau >= 0x1p-63f && tau <= 0x1p63f)) return DP_ERR_VALUE;  // 1 / tau and tau^2 inside fp32's range
  return DP_OK;
}

size_t distill_ws_bytes(int64_t B, int64_t T) { return T > 1 ? round256((size_t)B * (size_t)T * sizeof(float)) : 0; }

dp_status check_grouped(dp_dtype dtype, const dpk::GroupedArgs& g, dpk::GroupedCall call) {
  if (g.R < 1 || g.E < 1 || g.B < 1 || g.d < 1 || g.p < 1) return DP_ERR_SHAPE;
  if (g.R > kMaxRows || g.E > kMaxRanges || g.B > kMaxRanges / g.E) return DP_ERR_SHAPE;
  if (g.d > kMaxRowWidth || g.p > kMaxRowWidth || g.E > kMaxElems / (g.d * g.p)) return DP_ERR_SHAPE;
  if (!dtype_ok(dtype)) return DP_ERR_DTYPE;
  // noise group index fits 32 bits
  if (call == dpk::GroupedCall::sum && (g.E * g.d + 3) / 4 >= ((int64_t)1 << 32) / g.p) return DP_ERR_SHAPE;
  if (!dpk::grouped_fits(g, call, dtype)) return DP_ERR_SHAPE;
  return DP_OK;
}

}  // namespace

extern "C" {

size_t dp_rms_norm_workspace_bytes(dp_dtype dtype, int64_t B, int64_t T, int64_t d) {
  if (!dtype_ok(dtype) || check_rms(B, T, d) != DP_OK) return 0;
  return rms_ws_bytes(B, T, d);
}

dp_status dp_rms_norm(void* stream, const void* x, const void* residual, const void* gain, dp_dtype dtype,
                      dp_dtype gain_dtype, int64_t rows, int64_t d, float eps, void* out, void* sum_out) {
  if (!x || !gain || !out) return DP_ERR_NULL;
  dp_status s = check_rms(1, rows, d);
  if (s != DP_OK) return s;
  if (!dtype_ok(dtype) || !dtype_ok(gain_dtype)) return DP_ERR_DTYPE;
  if (!finite(eps) || eps < 0.0f) return DP_ERR_VALUE;
  const uintptr_t eb = elem_bytes(dtype);
  if (!aligned(x, eb) || !aligned(residual, eb) || !aligned(out, eb) || !aligned(sum_out, eb) ||
      !aligned(gain, elem_bytes(gain_dtype)))
    return DP_ERR_ALIGN;
  s = device_ready();
  if (s != DP_OK) return s;
  const dpk::RmsArgs a{x, residual, gain, gain_dtype == DP_BF16, eps, rows, d, out, sum_out};
  return hip_status(dpk::launch_rms_norm(static_cast<hipStream_t>(stream), dtype, a));
}

dp_status dp_rms_norm_backward(void* stream, const void* dy, const void* s, const void* dsum, const void* gain,
                               dp_dtype dtype, dp_dtype gain_dtype, int64_t B, int64_t T, int64_t d, float eps,
                               void* workspace, size_t ws_bytes, void* dx, float* gain_rows) {
  if (!dy || !s || !gain || (!dx && !gain_rows)) return DP_ERR_NULL;
  dp_status st = check_rms(B, T, d);
  if (st != DP_OK) return st;
  if (!dtype_ok(dtype) || !dtype_ok(gain_dtype)) return DP_ERR_DTYPE;
  if (!finite(eps) || eps < 0.0f) return DP_ERR_VALUE;
  const uintptr_t eb = elem_bytes(dtype);
  if (!aligned(dy, eb) || !aligned(s, eb) || !aligned(dsum, eb) || !aligned(dx, eb) ||
      !aligned(gain, elem_bytes(gain_dtype)) || !aligned(gain_rows, 4))
    return DP_ERR_ALIGN;
  st = check_workspace(workspace, ws_bytes, gain_rows ? rms_ws_bytes(B, T, d) : 0);
  if (st != DP_OK) return st;
  st = device_ready();
  if (st != DP_OK) return st;
  dpk::RmsBackArgs a{};
  a.dy = dy;
  a.s = s;
  a.dsum = dsum;
  a.gain = gain;
  a.gain_bf16 = gain_dtype == DP_BF16;
  a.eps = eps;
  a.B = B;
  a.T = T;
  a.d = d;
  a.dx = dx;
  a.gain_rows = gain_rows;
  a.partial = static_cast<float*>(workspace);
  return hip_status(dpk::launch_rms_norm_backward(static_cast<hipStream_t>(stream), dtype, a));
}

size_t dp_distill_workspace_bytes(dp_dtype dtype, int64_t B, int64_t T, int64_t V, int64_t K) {
  if (!dtype_ok(dtype) || check_distill(B, T, V, K, 1.0f) != DP_OK) return 0;
  return distill_ws_bytes(B, T);
}

dp_status dp_distill_loss(void* stream, const void* logits, const int64_t* ids, const void* teacher, dp_dtype dtype,
                          dp_dtype teacher_dtype, int64_t B, int64_t T, int64_t V, int64_t K, float tau, const float* weight,
                          void* workspace, size_t ws_bytes, float* loss, float* lse) {
  if (!logits || !ids || !teacher || !loss || !lse) return DP_ERR_NULL;
  dp_status s = check_distill(B, T, V, K, tau);
  if (s != DP_OK) return s;
  if (!dtype_ok(dtype) || !dtype_ok(teacher_dtype)) return DP_ERR_DTYPE;
  if (!aligned(logits, 16) || !aligned(ids, 8) || !aligned(teacher, elem_bytes(teacher_dtype)) || !aligned(weight, 4) ||
      !aligned(loss, 4) || !aligned(lse, 4))
    return DP_ERR_ALIGN;
  s = check_workspace(workspace, ws_bytes, distill_ws_bytes(B, T));
  if (s != DP_OK) return s;
  s = device_ready();
  if (s != DP_OK) return s;
  dpk::DistillArgs a{};
  a.logits = logits;
  a.ids = ids;
  a.teacher = teacher;
  a.teacher_bf16 = teacher_dtype == DP_BF16;
  a.weight = weight;
  a.tau = tau;
  a.B = B;
  a.T = T;
  a.V = V;
  a.K = K;
  a.loss = loss;
  a.lse = lse;
  a.row_loss = static_cast<float*>(workspace);
  return hip_status(dpk::launch_distill_loss(static_cast<hipStream_t>(stream), dtype, a));
}

dp_status dp_distill_loss_backward(void* stream, const void* logits, const int64_t* ids, const void* teacher,
                                   dp_dtype dtype, dp_dtype teacher_dtype, int64_t B, int64_t T, int64_t V,
                                   int64_t K, float tau,
                                   const float* weight, const float* dloss, const float* lse, void* grad) {
  if (!logits || !ids || !teacher || !lse || !grad) return DP_ERR_NULL;
  dp_status s = check_distill(B, T, V, K, tau);
  if (s != DP_OK) return s;
  if (!dtype_ok(dtype) || !dtype_ok(teacher_dtype)) return DP_ERR_DTYPE;
  if (!aligned(logits, 16) || !aligned(grad, 16) || !aligned(ids, 8) || !aligned(teacher, elem_bytes(teacher_dtype)) ||
      !aligned(weight, 4) || !aligned(dloss, 4) || !aligned(lse, 4))
    return DP_ERR_ALIGN;
  s = device_ready();
  if (s != DP_OK) return s;
  dpk::DistillArgs a{};
  a.logits = logits;
  a.ids = ids;
  a.teacher = teacher;
  a.teacher_bf16 = teacher_dtype == DP_BF16;
  a.weight = weight;
  a.tau = tau;
  a.B = B;
  a.T = T;
  a.V = V;
  a.K = K;
  a.lse = const_cast<float*>(lse);
  a.dloss = dloss;
  a.grad = grad;
  return hip_status(dpk::launch_distill_backward(static_cast<hipStream_t>(stream), dtype, a));
}

size_t dp_grouped_workspace_bytes(dp_dtype dtype, int64_t R, int64_t E, int64_t B, int64_t d, int64_t p) {
  const dpk::GroupedArgs g{nullptr, R, E, B, d, p};
  using dpk::GroupedCall;
  auto takes = [&](GroupedCall call) { return check_grouped(dtype, g, call) == DP_OK; };
  size_t need = 0;
  if (takes(GroupedCall::matmul) || takes(GroupedCall::matmul_transposed))
    need = std::max(need, dpk::grouped_matmul_ws_bytes(dtype, g));
  if (takes(GroupedCall::norm)) need = std::max(need, dpk::grouped_norm_ws_bytes(dtype, g));
  if (takes(GroupedCall::sum)) need = std::max(need, dpk::grouped_sum_ws_bytes(dtype, g));
  return need;
}

dp_status dp_grouped_matmul(void* stream, const void* X, const void* W, dp_dtype dtype, const int64_t* segments,
                            int64_t R, int64_t E, int64_t B, int64_t d, int64_t p, int32_t transpose, void* workspace,
                            size_t ws_bytes, void* Y) {
  if (!X || !W || !segments || !Y) return DP_ERR_NULL;
  const dpk::GroupedArgs g{segments, R, E, B, d, p};
  dp_status s = check_grouped(dtype, g, transpose ? dpk::GroupedCall::matmul_transposed : dpk::GroupedCall::matmul);
  if (s != DP_OK) return s;
  if (!aligned(X, 16) || !aligned(W, 16) || !aligned(Y, 16) || !aligned(segments, 8)) return DP_ERR_ALIGN;
  s = check_workspace(workspace, ws_bytes, dpk::grouped_matmul_ws_bytes(dtype, g));
  if (s != DP_OK) return s;
  s = device_ready();
  if (s != DP_OK) return s;
  return hip_status(dpk::launch_grouped_matmul(static_cast<hipStream_t>(stream), dtype, g, X, W, transpose != 0,
                                               workspace, Y));
}

dp_status dp_grouped_norm(void* stream, const void* A, const void* G, dp_dtype dtype, const int64_t* segments,
                          int64_t R, int64_t E, int64_t B, int64_t d, int64_t p, void* workspace, size_t ws_bytes,
                          float* sqnorm, int32_t accumulate) {
  if (!A || !G || !segments || !sqnorm) return DP_ERR_NULL;
  const dpk::GroupedArgs g{segments, R, E, B, d, p};
  dp_status s = check_grouped(dtype, g, dpk::GroupedCall::norm);
  if (s != DP_OK) return s;
  if (!aligned(A, 16) || !aligned(G, 16) || !aligned(segments, 8) || !aligned(sqnorm, 4)) return DP_ERR_ALIGN;
  s = check_workspace(workspace, ws_bytes, dpk::grouped_norm_ws_bytes(dtype, g));
  if (s != DP_OK) return s;
  s = device_ready();
  if (s != DP_OK) return s;
  return hip_status(dpk::launch_grouped_norm(static_cast<hipStream_t>(stream), dtype, g, A, G, workspace, sqnorm,
                                             accumulate ? 1 : 0));
}

dp_status dp_grouped_clipped_sum_noise(void* stream, const void* A, const void* G, dp_dtype dtype,
                                       const int64_t* segments, int64_t R, int64_t E, int64_t B, int64_t d, int64_t p,
                                       const float* c, float C, float sigma, float denom, uint64_t seed,
                                       uint32_t layer_id, uint32_t step, void* workspace, size_t ws_bytes,
                                       float* out) {
  if (!A || !G || !segments || !c || !out) return DP_ERR_NULL;
  const dpk::GroupedArgs g{segments, R, E, B, d, p};
  dp_status s = check_grouped(dtype, g, dpk::GroupedCall::sum);
  if (s != DP_OK) return s;
  if (!aligned(A, 16) || !aligned(G, 16) || !aligned(segments, 8) || !aligned(c, 4) || !aligned(out, 4))
    return DP_ERR_ALIGN;
  if (!finite(C) || !(C > 0.0f) || !finite(sigma) || sigma < 0.0f || !finite(denom) || !(denom > 0.0f))
    return DP_ERR_VALUE;
  s = check_workspace(workspace, ws_bytes, dpk::grouped_sum_ws_bytes(dtype, g));
  if (s != DP_OK) return s;
  s = device_ready();
  if (s != DP_OK) return s;
  const dpk::NoiseArgs na = dpk::make_noise_args(sigma * C, denom, seed, layer_id, step);
  return hip_status(dpk::launch_grouped_sum(static_cast<hipStream_t>(stream), dtype, g, A, G, c, workspace, na, out));
}

}  // extern "C"
