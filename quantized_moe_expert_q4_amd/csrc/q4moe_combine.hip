// Weighted combination of a token's expert outputs, and its gradients.
//
//   out[t] = base[t] + sum_j w[t,j] y[t,j]
//   dy[t,j] = w[t,j] dout[t],   dw[t,j] = <dout[t], y[t,j]>
//
// Every row of y is read (and of dy written) once: both are bound by memory.
#include "q4moe_device.h"
#include "q4moe_layer.h"

namespace q4 {

namespace {

// Sixteen bytes of a row as F32 values: eight bf16 or four floats.
template <bool F32>
struct Piece {
  static constexpr int kValues = F32 ? 4 : 8;
  float v[kValues];
};

template <bool F32>
__device__ __forceinline__ Piece<F32> unpack(const v4u u) {
  Piece<F32> r;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (F32) {
      r.v[i] = __uint_as_float(u[i]);
    } else {
      r.v[2 * i] = __uint_as_float(u[i] << 16);
      r.v[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
    }
  }
  return r;
}

template <bool F32>
__device__ __forceinline__ v4u pack(const Piece<F32>& r) {
  v4u u;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (F32) u[i] = __float_as_uint(r.v[i]);
    else u[i] = (uint32_t)bf16_rne(r.v[2 * i]) | ((uint32_t)bf16_rne(r.v[2 * i + 1]) << 16);
  }
  return u;
}

// The pair's weight and whether it counts (its id names a slot).
__device__ __forceinline__ bool live(const CombineParams& p, size_t pair) {
  return !p.ids || (uint32_t)p.ids[pair] < (uint32_t)p.num_slots;
}

// One thread per 16 bytes of an output row.
template <bool F32>
__global__ __launch_bounds__(256) void combine_kernel(CombineParams p) {
  constexpr int V = Piece<F32>::kValues;
  const int pieces = p.H / V;
  const size_t n = (size_t)p.M * pieces;
  for (size_t at = (size_t)blockIdx.x * 256 + threadIdx.x; at < n; at += (size_t)gridDim.x * 256) {
  const size_t t = at / pieces;
  const size_t h = at % pieces;
  Piece<F32> acc{};
  if (p.base) acc = unpack<F32>(static_cast<const v4u*>(p.base)[at]);
  for (int j = 0; j < p.K; ++j) {
    const size_t pair = t * p.K + j;
    if (!live(p, pair)) continue;
    const float w = p.weights[pair];
    const Piece<F32> y = unpack<F32>(static_cast<const v4u*>(p.y)[pair * pieces + h]);
#pragma unroll
    for (int i = 0; i < V; ++i) acc.v[i] = fmaf(w, y.v[i], acc.v[i]);
  }
  static_cast<v4u*>(p.out)[at] = pack<F32>(acc);
  }
}

// One work-group per pair.
template <bool F32>
__global__ __launch_bounds__(256) void combine_backward_kernel(CombineParams p) {
  constexpr int V = Piece<F32>::kValues;
  __shared__ float part[4];
  const int pieces = p.H / V;
  for (size_t pair = blockIdx.x; pair < (size_t)p.M * p.K; pair += gridDim.x) {
  const size_t t = pair / p.K;
  const bool on = live(p, pair);
  const float w = on ? p.weights[pair] : 0.0f;
  float dot = 0.0f;
  for (int h = threadIdx.x; h < pieces; h += 256) {
    Piece<F32> d{};
    if (on) {
      d = unpack<F32>(static_cast<const v4u*>(p.d_out)[t * pieces + h]);
      if (p.d_weights) {
        const Piece<F32> y = unpack<F32>(static_cast<const v4u*>(p.y)[pair * pieces + h]);
#pragma unroll
        for (int i = 0; i < V; ++i) dot = fmaf(d.v[i], y.v[i], dot);
      }
#pragma unroll
      for (int i = 0; i < V; ++i) d.v[i] *= w;
    }
    if (p.d_y) static_cast<v4u*>(p.d_y)[pair * pieces + h] = pack<F32>(d);
  }
  if (!p.d_weights) continue;
  for (int s = 32; s; s >>= 1) dot += __shfl_xor(dot, s);
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = dot;
  __syncthreads();
  if (threadIdx.x == 0) p.d_weights[pair] = (part[0] + part[1]) + (part[2] + part[3]);
  __syncthreads();
  }
}

template <bool F32>
hipError_t launch(const CombineParams& p, bool backward, hipStream_t stream) {
  CombineParams q = p;
  void* args[] = {&q};
  const size_t work = (size_t)p.M * (p.H / Piece<F32>::kValues);
  size_t blocks = backward ? (size_t)p.M * p.K : (work + 255) / 256;
  if (blocks > (1u << 20)) blocks = 1u << 20;  // the kernels stride the rest
  const void* f = backward ? reinterpret_cast<const void*>(&combine_backward_kernel<F32>)
                           : reinterpret_cast<const void*>(&combine_kernel<F32>);
  return hipLaunchKernel(f, dim3((unsigned)blocks), dim3(256), args, 0, stream);
}

}  // namespace

hipError_t launch_combine(const CombineParams& p, hipStream_t stream) {
  return p.xf32 ? launch<true>(p, false, stream) : launch<false>(p, false, stream);
}

hipError_t launch_combine_backward(const CombineParams& p, hipStream_t stream) {
  return p.xf32 ? launch<true>(p, true, stream) : launch<false>(p, true, stream);
}

}  // namespace q4
