// Linear with 4-bit weights and a scale (and bias) for each group of a row.
#include "q4moe_device.h"
#include "q4moe_layer.h"

namespace q4 {

namespace {

constexpr int kTokens = 4;  // tokens a wave carries past one row

__device__ __forceinline__ float scale_at(const void* s, int f32, size_t i) {
  return f32 ? static_cast<const float*>(s)[i] : bf16_val(static_cast<const uint16_t*>(s)[i]);
}

// One wave per (row, kTokens tokens): lanes stride the row's words, each
// word's eight products are summed in F32 and scaled by their group.
__global__ __launch_bounds__(256) void linear_kernel(LinearParams p) {
  const int lane = threadIdx.x & 63;
  for (int64_t n = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); n < p.N; n += (int64_t)gridDim.x * 4) {
  const int m0 = (int)blockIdx.y * kTokens;
  const uint32_t* row = reinterpret_cast<const uint32_t*>(p.w) + (size_t)n * (size_t)(p.K / 8);
  float acc[kTokens] = {};
  for (int i = lane; i < p.K / 8; i += 64) {
    const uint32_t w = row[i];
    const size_t g = (size_t)n * p.groups + (size_t)(i * 8 / p.group);
    const float s = scale_at(p.scales, p.scale_f32, g);
    const float b = p.biases ? scale_at(p.biases, p.scale_f32, g) : 0.0f;
    const float zero = p.biases ? 0.0f : 8.0f;
#pragma unroll
    for (int t = 0; t < kTokens; ++t) {
      if (m0 + t >= p.M) break;
      const size_t at = (size_t)(m0 + t) * p.K + (size_t)i * 8;
      float sum = 0.0f, xs = 0.0f;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float xv = p.xf32 ? static_cast<const float*>(p.x)[at + j]
                                : bf16_val(static_cast<const uint16_t*>(p.x)[at + j]);
        sum = fmaf((float)((w >> (4 * j)) & 15u) - zero, xv, sum);
        xs += xv;
      }
      acc[t] = fmaf(s, sum, acc[t]);
      if (p.biases) acc[t] = fmaf(b, xs, acc[t]);
    }
  }
#pragma unroll
  for (int t = 0; t < kTokens; ++t) {
    float v = acc[t];
    for (int d = 32; d; d >>= 1) v += __shfl_xor(v, d);
    if (lane == 0 && m0 + t < p.M) {
      const size_t at = (size_t)(m0 + t) * p.N + (size_t)n;
      if (p.xf32) static_cast<float*>(p.out)[at] = v;
      else static_cast<uint16_t*>(p.out)[at] = bf16_rne(v);
    }
  }
  }
}

}  // namespace

hipError_t launch_linear(const LinearParams& p, hipStream_t stream) {
  LinearParams q = p;
  void* args[] = {&q};
  const int rows = (p.N + 3) / 4;
  const int blocks = rows < (1 << 16) ? rows : (1 << 16);
  return hipLaunchKernel(reinterpret_cast<const void*>(&linear_kernel),
                         dim3((unsigned)blocks, (unsigned)((p.M + kTokens - 1) / kTokens)), dim3(256), args, 0,
                         stream);
}

}  // namespace q4
