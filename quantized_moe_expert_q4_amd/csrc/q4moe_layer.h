// Internal interface between the C ABI of the layer operators
// (q4moe_layer_abi.cpp) and their kernels: the grouped-scale linear, the
// router and the combination of expert outputs.
#pragma once
#include <hip/hip_runtime_api.h>
#include <stdint.h>

namespace q4 {

// out[m][n] = sum_k W[n][k] x[m][k], W from packed nibbles and a scale (and
// bias) for each `group` weights of a row.
struct LinearParams {
  const uint8_t* w;       // packed nibbles [N][K/2]
  const void* scales;     // [N][groups], F32 or bf16
  const void* biases;     // the same shape and type, or nullptr (zero point 8)
  const void* x;          // [M][K], bf16 or float
  void* out;              // [M][N], the type of x
  int M, N, K;
  int group, groups;      // 32, 64 or 128; groups = ceil(K / group)
  int scale_f32, xf32;
};

// Router: logits [M][E] to the K chosen ids and weights of each token and,
// with `partials`, the batch statistics.
struct RouteParams {
  const void* logits;         // [M][E], bf16 or float
  const float* bias;          // [E] added to the scores for the choice, or nullptr
  const uint8_t* mask;        // [M], 0 = no token there, or nullptr
  int32_t* ids;               // [M][K]
  float* weights;             // [M][K]
  int32_t* counts;            // [E] or nullptr
  float* loss;                // [1] or nullptr
  float* loss_grad;           // [E] or nullptr
  void* partials;             // workspace of the statistics, or nullptr
  float scale;
  int M, E, K;
  int sigmoid, renormalize, lf32;
};

struct RouteBackwardParams {
  const void* logits;         // [M][E]
  const int32_t* ids;         // [M][K]
  const float* d_weights;     // [M][K] or nullptr
  const float* d_loss;        // [1] or nullptr
  const float* loss_grad;     // [E] or nullptr
  void* d_logits;             // [M][E], the type of logits
  float scale;
  int M, E, K;
  int sigmoid, renormalize, lf32;
};

// Combination of a token's K expert outputs; backward when d_out is set.
struct CombineParams {
  const void* y;              // [M][K][H], bf16 or float
  const float* weights;       // [M][K]
  const int32_t* ids;         // [M][K] or nullptr (every pair counts)
  const void* base;           // [M][H] or nullptr
  void* out;                  // [M][H]
  const void* d_out;          // [M][H]
  void* d_y;                  // [M][K][H] or nullptr
  float* d_weights;           // [M][K] or nullptr
  int M, K, H, num_slots, xf32;
};

hipError_t launch_linear(const LinearParams& p, hipStream_t stream);

constexpr int kRouteMaxExperts = 1024;
constexpr int kRouteMaxTopK = 64;

// Bytes of the statistics' workspace for M tokens and E experts.
size_t route_partial_bytes(int64_t M, int64_t E);
hipError_t launch_route(const RouteParams& p, hipStream_t stream);
hipError_t launch_route_backward(const RouteBackwardParams& p, hipStream_t stream);

hipError_t launch_combine(const CombineParams& p, hipStream_t stream);
hipError_t launch_combine_backward(const CombineParams& p, hipStream_t stream);

}  // namespace q4
