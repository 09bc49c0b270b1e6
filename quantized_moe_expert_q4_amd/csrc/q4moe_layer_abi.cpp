// C ABI of the layer operators: argument validation and dispatch of the
// group-scaled linear, the router and the combination of expert outputs.
#include <stdint.h>

#include "q4moe.h"
#include "q4moe_error.h"
#include "q4moe_layer.h"

namespace {

using q4::report;

constexpr int64_t kMaxK = 65536;
constexpr int64_t kMaxRows = 65535;
constexpr int64_t kMaxRouteTokens = 1ll << 24;
constexpr uint64_t kMaxWeightBytes = (1ull << 31) - 16;
constexpr int64_t kMaxPairs = (1ll << 31) - 1;

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

int launched(hipError_t e) {
  if (e == hipSuccess) return report(Q4_OK, "");
  return report(Q4_ERR_HIP, hipGetErrorString(e));
}

int check_linear(bool f32, const void* w, const void* scales, const void* biases, int scale_type, int64_t group,
                 const void* x, int64_t M, int64_t N, int64_t K, const void* out) {
  if (M < 1) return report(Q4_ERR_INVALID_ARGUMENT, "linear requires input [M,K] with M >= 1");
  if (N <= 0) return report(Q4_ERR_INVALID_ARGUMENT, "output rows must be a positive integer");
  if (K <= 0 || K % 8 != 0) return report(Q4_ERR_INVALID_ARGUMENT, "linear needs K positive and divisible by 8");
  if (group != 32 && group != 64 && group != 128)
    return report(Q4_ERR_UNSUPPORTED, "the weights of a group must be 32, 64 or 128");
  if (scale_type != Q4_SCALE_BF16 && scale_type != Q4_SCALE_F32)
    return report(Q4_ERR_INVALID_ARGUMENT, "scale type must be Q4_SCALE_BF16 or Q4_SCALE_F32");
  if (M > kMaxRows) return report(Q4_ERR_UNSUPPORTED, "more than 65535 tokens per call is not supported");
  if (K > kMaxK) return report(Q4_ERR_UNSUPPORTED, "K above 65536 is not supported");
  if ((uint64_t)N > kMaxWeightBytes / (uint64_t)(K / 2))
    return report(Q4_ERR_UNSUPPORTED, "a matrix above 2^31 - 16 bytes is not supported");
  if (!w || !scales || !x || !out)
    return report(Q4_ERR_INVALID_ARGUMENT, "weights, scales, x and output must be non-null device pointers");
  if (!aligned(w, 16)) return report(Q4_ERR_ALIGNMENT, "weights must be 16-byte aligned");
  if (!aligned(x, 16)) return report(Q4_ERR_ALIGNMENT, "input x must be 16-byte aligned");
  const uintptr_t sa = scale_type == Q4_SCALE_F32 ? 4 : 2;
  if (!aligned(scales, sa) || (biases && !aligned(biases, sa)))
    return report(Q4_ERR_ALIGNMENT, "scales and biases must be aligned to their type");
  if (!aligned(out, f32 ? 4 : 2)) return report(Q4_ERR_ALIGNMENT, "output must be aligned to its type");
  return report(Q4_OK, "");
}

int run_linear(bool f32, const void* w, const void* scales, const void* biases, int scale_type, int64_t group,
               const void* x, int64_t M, int64_t N, int64_t K, void* out, q4_stream_t stream) {
  const int rc = check_linear(f32, w, scales, biases, scale_type, group, x, M, N, K, out);
  if (rc) return rc;
  q4::LinearParams p{};
  p.w = static_cast<const uint8_t*>(w);
  p.scales = scales;
  p.biases = biases;
  p.x = x;
  p.out = out;
  p.M = (int)M;
  p.N = (int)N;
  p.K = (int)K;
  p.group = (int)group;
  p.groups = (int)((K + group - 1) / group);
  p.scale_f32 = scale_type == Q4_SCALE_F32;
  p.xf32 = f32;
  return launched(q4::launch_linear(p, reinterpret_cast<hipStream_t>(stream)));
}

int check_route_sizes(int64_t M, int64_t E, int64_t K, int score) {
  if (M < 1) return report(Q4_ERR_INVALID_ARGUMENT, "router requires logits [M,E] with M >= 1");
  if (E < 1) return report(Q4_ERR_INVALID_ARGUMENT, "number of experts must be a positive integer");
  if (K < 1 || K > E) return report(Q4_ERR_INVALID_ARGUMENT, "top-k must lie between 1 and the number of experts");
  if (score != Q4_SCORE_SOFTMAX && score != Q4_SCORE_SIGMOID)
    return report(Q4_ERR_INVALID_ARGUMENT, "score must be Q4_SCORE_SOFTMAX or Q4_SCORE_SIGMOID");
  if (M > kMaxRouteTokens) return report(Q4_ERR_UNSUPPORTED, "more than 2^24 tokens per call is not supported");
  if (E > q4::kRouteMaxExperts) return report(Q4_ERR_UNSUPPORTED, "more than 1024 experts is not supported");
  if (K > q4::kRouteMaxTopK) return report(Q4_ERR_UNSUPPORTED, "top-k above 64 is not supported");
  return Q4_OK;
}

// `logit_align` is the size of a logit.
int check_route(uintptr_t logit_align, const void* logits, int64_t M, int64_t E, int64_t K, int score,
                const float* bias, const uint8_t* mask, const int32_t* ids, const float* weights,
                const int32_t* counts, const float* loss, const float* loss_grad, const void* ws, size_t ws_bytes) {
  (void)mask;
  const int rc = check_route_sizes(M, E, K, score);
  if (rc) return rc;
  if (!logits || !ids || !weights)
    return report(Q4_ERR_INVALID_ARGUMENT, "logits, ids and weights must be non-null device pointers");
  if (!aligned(logits, logit_align)) return report(Q4_ERR_ALIGNMENT, "logits must be aligned to their type");
  if (!aligned(ids, 4) || !aligned(weights, 4) || !aligned(bias, 4) || !aligned(counts, 4) || !aligned(loss, 4) ||
      !aligned(loss_grad, 4))
    return report(Q4_ERR_ALIGNMENT, "ids, weights, bias and statistics must be 4-byte aligned");
  if (counts || loss || loss_grad) {
    if (!ws) return report(Q4_ERR_WORKSPACE, "statistics need a workspace");
    if (!aligned(ws, 256)) return report(Q4_ERR_ALIGNMENT, "workspace must be 256-byte aligned");
    if (ws_bytes < q4_route_workspace_bytes(M, E))
      return report(Q4_ERR_WORKSPACE, "workspace is smaller than q4_route_workspace_bytes()");
  }
  return report(Q4_OK, "");
}

int run_route(bool f32, const void* logits, int64_t M, int64_t E, int64_t K, int score, int renormalize, float scale,
              const float* bias, const uint8_t* mask, int32_t* ids, float* weights, int32_t* counts, float* loss,
              float* loss_grad, void* ws, size_t ws_bytes, q4_stream_t stream) {
  const int rc = check_route(f32 ? 4 : 2, logits, M, E, K, score, bias, mask, ids, weights, counts, loss, loss_grad,
                             ws, ws_bytes);
  if (rc) return rc;
  q4::RouteParams p{};
  p.logits = logits;
  p.bias = bias;
  p.mask = mask;
  p.ids = ids;
  p.weights = weights;
  p.counts = counts;
  p.loss = loss;
  p.loss_grad = loss_grad;
  p.partials = (counts || loss || loss_grad) ? ws : nullptr;
  p.scale = scale;
  p.M = (int)M;
  p.E = (int)E;
  p.K = (int)K;
  p.sigmoid = score == Q4_SCORE_SIGMOID;
  p.renormalize = renormalize != 0;
  p.lf32 = f32;
  return launched(q4::launch_route(p, reinterpret_cast<hipStream_t>(stream)));
}

int check_route_backward(uintptr_t logit_align, const void* logits, int64_t M, int64_t E, int64_t K, int score,
                         const int32_t* ids, const float* d_weights, const float* d_loss, const float* loss_grad,
                         const void* d_logits) {
  const int rc = check_route_sizes(M, E, K, score);
  if (rc) return rc;
  if (!logits || !ids || !d_logits)
    return report(Q4_ERR_INVALID_ARGUMENT, "logits, ids and the logits' gradient must be non-null device pointers");
  if ((d_loss == nullptr) != (loss_grad == nullptr))
    return report(Q4_ERR_INVALID_ARGUMENT, "d_loss and loss_grad must be given together");
  if (!d_weights && !d_loss) return report(Q4_ERR_INVALID_ARGUMENT, "d_weights or d_loss must be given");
  if (!aligned(logits, logit_align) || !aligned(d_logits, logit_align))
    return report(Q4_ERR_ALIGNMENT, "logits and their gradient must be aligned to their type");
  if (!aligned(ids, 4) || !aligned(d_weights, 4) || !aligned(d_loss, 4) || !aligned(loss_grad, 4))
    return report(Q4_ERR_ALIGNMENT, "ids and gradients must be 4-byte aligned");
  return report(Q4_OK, "");
}

int run_route_backward(bool f32, const void* logits, int64_t M, int64_t E, int64_t K, int score, int renormalize,
                       float scale, const int32_t* ids, const float* d_weights, const float* d_loss,
                       const float* loss_grad, void* d_logits, q4_stream_t stream) {
  const int rc = check_route_backward(f32 ? 4 : 2, logits, M, E, K, score, ids, d_weights, d_loss, loss_grad, d_logits);
  if (rc) return rc;
  q4::RouteBackwardParams p{};
  p.logits = logits;
  p.ids = ids;
  p.d_weights = d_weights;
  p.d_loss = d_loss;
  p.loss_grad = loss_grad;
  p.d_logits = d_logits;
  p.scale = scale;
  p.M = (int)M;
  p.E = (int)E;
  p.K = (int)K;
  p.sigmoid = score == Q4_SCORE_SIGMOID;
  p.renormalize = renormalize != 0;
  p.lf32 = f32;
  return launched(q4::launch_route_backward(p, reinterpret_cast<hipStream_t>(stream)));
}

int check_combine_sizes(const int32_t* slot_ids, int64_t num_slots, int64_t M, int64_t K, int64_t H) {
  if (M < 1) return report(Q4_ERR_INVALID_ARGUMENT, "combine requires outputs [M,K,H] with M >= 1");
  if (K < 1) return report(Q4_ERR_INVALID_ARGUMENT, "top-k must be a positive integer");
  if (H <= 0 || H % 8 != 0) return report(Q4_ERR_INVALID_ARGUMENT, "combine needs H positive and divisible by 8");
  if (slot_ids && num_slots < 1) return report(Q4_ERR_INVALID_ARGUMENT, "number of slots must be a positive integer");
  if (H > kMaxK) return report(Q4_ERR_UNSUPPORTED, "hidden size above 65536 is not supported");
  if (M > kMaxPairs || K > kMaxPairs / M)
    return report(Q4_ERR_UNSUPPORTED, "more than 2^31 - 1 pairs per call is not supported");
  return Q4_OK;
}

q4::CombineParams combine_params(bool f32, const void* y, const float* weights, const int32_t* slot_ids,
                                 int64_t num_slots, int64_t M, int64_t K, int64_t H) {
  q4::CombineParams p{};
  p.y = y;
  p.weights = weights;
  p.ids = slot_ids;
  p.num_slots = num_slots > INT32_MAX ? INT32_MAX : (int)num_slots;
  p.M = (int)M;
  p.K = (int)K;
  p.H = (int)H;
  p.xf32 = f32;
  return p;
}

int check_combine(const void* y, const float* weights, const int32_t* slot_ids, int64_t num_slots, const void* base,
                  int64_t M, int64_t K, int64_t H, const void* out) {
  const int rc = check_combine_sizes(slot_ids, num_slots, M, K, H);
  if (rc) return rc;
  if (!y || !weights || !out)
    return report(Q4_ERR_INVALID_ARGUMENT, "expert outputs, weights and output must be non-null device pointers");
  if (!aligned(y, 16) || !aligned(base, 16) || !aligned(out, 16))
    return report(Q4_ERR_ALIGNMENT, "expert outputs, base and output must be 16-byte aligned");
  if (!aligned(weights, 4) || !aligned(slot_ids, 4))
    return report(Q4_ERR_ALIGNMENT, "weights and slot ids must be 4-byte aligned");
  return report(Q4_OK, "");
}

int run_combine(bool f32, const void* y, const float* weights, const int32_t* slot_ids, int64_t num_slots,
                const void* base, int64_t M, int64_t K, int64_t H, void* out, q4_stream_t stream) {
  const int rc = check_combine(y, weights, slot_ids, num_slots, base, M, K, H, out);
  if (rc) return rc;
  q4::CombineParams p = combine_params(f32, y, weights, slot_ids, num_slots, M, K, H);
  p.base = base;
  p.out = out;
  return launched(q4::launch_combine(p, reinterpret_cast<hipStream_t>(stream)));
}

int check_combine_backward(const void* d_out, const void* y, const float* weights, const int32_t* slot_ids,
                           int64_t num_slots, int64_t M, int64_t K, int64_t H, const void* d_y,
                           const float* d_weights) {
  const int rc = check_combine_sizes(slot_ids, num_slots, M, K, H);
  if (rc) return rc;
  if (!d_out || !weights)
    return report(Q4_ERR_INVALID_ARGUMENT, "the output's gradient and weights must be non-null device pointers");
  if (!d_y && !d_weights) return report(Q4_ERR_INVALID_ARGUMENT, "d_y or d_weights must be given");
  if (d_weights && !y) return report(Q4_ERR_INVALID_ARGUMENT, "d_weights needs the expert outputs");
  if (!aligned(d_out, 16) || !aligned(y, 16) || !aligned(d_y, 16))
    return report(Q4_ERR_ALIGNMENT, "expert outputs and row gradients must be 16-byte aligned");
  if (!aligned(weights, 4) || !aligned(slot_ids, 4) || !aligned(d_weights, 4))
    return report(Q4_ERR_ALIGNMENT, "weights, their gradient and slot ids must be 4-byte aligned");
  return report(Q4_OK, "");
}

int run_combine_backward(bool f32, const void* d_out, const void* y, const float* weights, const int32_t* slot_ids,
                         int64_t num_slots, int64_t M, int64_t K, int64_t H, void* d_y, float* d_weights,
                         q4_stream_t stream) {
  const int rc = check_combine_backward(d_out, y, weights, slot_ids, num_slots, M, K, H, d_y, d_weights);
  if (rc) return rc;
  q4::CombineParams p = combine_params(f32, y, weights, slot_ids, num_slots, M, K, H);
  p.d_out = d_out;
  p.d_y = d_y;
  p.d_weights = d_weights;
  return launched(q4::launch_combine_backward(p, reinterpret_cast<hipStream_t>(stream)));
}

}  // namespace

extern "C" {

int q4_linear(const void* weights, const void* scales, const void* biases, int scale_type, int64_t group,
              const void* x_bf16, int64_t M, int64_t N, int64_t K, void* out_bf16, q4_stream_t stream) {
  return run_linear(false, weights, scales, biases, scale_type, group, x_bf16, M, N, K, out_bf16, stream);
}

int q4_linear_f32(const void* weights, const void* scales, const void* biases, int scale_type, int64_t group,
                  const void* x_f32, int64_t M, int64_t N, int64_t K, void* out_f32, q4_stream_t stream) {
  return run_linear(true, weights, scales, biases, scale_type, group, x_f32, M, N, K, out_f32, stream);
}

int q4_validate_linear(const void* weights, const void* scales, const void* biases, int scale_type, int64_t group,
                       const void* x_bf16, int64_t M, int64_t N, int64_t K, const void* out_bf16) {
  return check_linear(false, weights, scales, biases, scale_type, group, x_bf16, M, N, K, out_bf16);
}

int q4_validate_linear_f32(const void* weights, const void* scales, const void* biases, int scale_type, int64_t group,
                           const void* x_f32, int64_t M, int64_t N, int64_t K, const void* out_f32) {
  return check_linear(true, weights, scales, biases, scale_type, group, x_f32, M, N, K, out_f32);
}

size_t q4_route_workspace_bytes(int64_t M, int64_t E) {
  if (M < 1 || E < 1 || M > kMaxRouteTokens || E > q4::kRouteMaxExperts) return 0;
  return q4::route_partial_bytes(M, E);
}

int q4_route(const void* logits_bf16, int64_t M, int64_t E, int64_t K, int score, int renormalize, float scale,
             const float* select_bias, const uint8_t* token_mask, int32_t* ids, float* weights, int32_t* counts,
             float* loss, float* loss_grad, void* workspace, size_t workspace_bytes, q4_stream_t stream) {
  return run_route(false, logits_bf16, M, E, K, score, renormalize, scale, select_bias, token_mask, ids, weights,
                   counts, loss, loss_grad, workspace, workspace_bytes, stream);
}

int q4_route_f32(const void* logits_f32, int64_t M, int64_t E, int64_t K, int score, int renormalize, float scale,
                 const float* select_bias, const uint8_t* token_mask, int32_t* ids, float* weights, int32_t* counts,
                 float* loss, float* loss_grad, void* workspace, size_t workspace_bytes, q4_stream_t stream) {
  return run_route(true, logits_f32, M, E, K, score, renormalize, scale, select_bias, token_mask, ids, weights, counts,
                   loss, loss_grad, workspace, workspace_bytes, stream);
}

int q4_route_backward(const void* logits_bf16, int64_t M, int64_t E, int64_t K, int score, int renormalize,
                      float scale, const int32_t* ids, const float* d_weights, const float* d_loss,
                      const float* loss_grad, void* d_logits_bf16, q4_stream_t stream) {
  return run_route_backward(false, logits_bf16, M, E, K, score, renormalize, scale, ids, d_weights, d_loss, loss_grad,
                            d_logits_bf16, stream);
}

int q4_route_backward_f32(const void* logits_f32, int64_t M, int64_t E, int64_t K, int score, int renormalize,
                          float scale, const int32_t* ids, const float* d_weights, const float* d_loss,
                          const float* loss_grad, void* d_logits_f32, q4_stream_t stream) {
  return run_route_backward(true, logits_f32, M, E, K, score, renormalize, scale, ids, d_weights, d_loss, loss_grad,
                            d_logits_f32, stream);
}

int q4_validate_route(const void* logits_bf16, int64_t M, int64_t E, int64_t K, int score, const float* select_bias,
                      const uint8_t* token_mask, const int32_t* ids, const float* weights, const int32_t* counts,
                      const float* loss, const float* loss_grad, const void* workspace, size_t workspace_bytes) {
  return check_route(2, logits_bf16, M, E, K, score, select_bias, token_mask, ids, weights, counts, loss, loss_grad,
                     workspace, workspace_bytes);
}

int q4_validate_route_f32(const void* logits_f32, int64_t M, int64_t E, int64_t K, int score, const float* select_bias,
                          const uint8_t* token_mask, const int32_t* ids, const float* weights, const int32_t* counts,
                          const float* loss, const float* loss_grad, const void* workspace, size_t workspace_bytes) {
  return check_route(4, logits_f32, M, E, K, score, select_bias, token_mask, ids, weights, counts, loss, loss_grad,
                     workspace, workspace_bytes);
}

int q4_validate_route_backward(const void* logits_bf16, int64_t M, int64_t E, int64_t K, int score, const int32_t* ids,
                               const float* d_weights, const float* d_loss, const float* loss_grad,
                               const void* d_logits_bf16) {
  return check_route_backward(2, logits_bf16, M, E, K, score, ids, d_weights, d_loss, loss_grad, d_logits_bf16);
}

int q4_validate_route_backward_f32(const void* logits_f32, int64_t M, int64_t E, int64_t K, int score,
                                   const int32_t* ids, const float* d_weights, const float* d_loss,
                                   const float* loss_grad, const void* d_logits_f32) {
  return check_route_backward(4, logits_f32, M, E, K, score, ids, d_weights, d_loss, loss_grad, d_logits_f32);
}

int q4_combine(const void* y_bf16, const float* weights, const int32_t* slot_ids, int64_t num_slots,
               const void* base_bf16, int64_t M, int64_t K, int64_t H, void* out_bf16, q4_stream_t stream) {
  return run_combine(false, y_bf16, weights, slot_ids, num_slots, base_bf16, M, K, H, out_bf16, stream);
}

int q4_combine_f32(const void* y_f32, const float* weights, const int32_t* slot_ids, int64_t num_slots,
                   const void* base_f32, int64_t M, int64_t K, int64_t H, void* out_f32, q4_stream_t stream) {
  return run_combine(true, y_f32, weights, slot_ids, num_slots, base_f32, M, K, H, out_f32, stream);
}

int q4_combine_backward(const void* d_out_bf16, const void* y_bf16, const float* weights, const int32_t* slot_ids,
                        int64_t num_slots, int64_t M, int64_t K, int64_t H, void* d_y_bf16, float* d_weights,
                        q4_stream_t stream) {
  return run_combine_backward(false, d_out_bf16, y_bf16, weights, slot_ids, num_slots, M, K, H, d_y_bf16, d_weights,
                              stream);
}

int q4_combine_backward_f32(const void* d_out_f32, const void* y_f32, const float* weights, const int32_t* slot_ids,
                            int64_t num_slots, int64_t M, int64_t K, int64_t H, void* d_y_f32, float* d_weights,
                            q4_stream_t stream) {
  return run_combine_backward(true, d_out_f32, y_f32, weights, slot_ids, num_slots, M, K, H, d_y_f32, d_weights,
                              stream);
}

int q4_validate_combine(const void* y, const float* weights, const int32_t* slot_ids, int64_t num_slots,
                        const void* base, int64_t M, int64_t K, int64_t H, const void* out) {
  return check_combine(y, weights, slot_ids, num_slots, base, M, K, H, out);
}

int q4_validate_combine_backward(const void* d_out, const void* y, const float* weights, const int32_t* slot_ids,
                                 int64_t num_slots, int64_t M, int64_t K, int64_t H, const void* d_y,
                                 const float* d_weights) {
  return check_combine_backward(d_out, y, weights, slot_ids, num_slots, M, K, H, d_y, d_weights);
}

}  // extern "C"
