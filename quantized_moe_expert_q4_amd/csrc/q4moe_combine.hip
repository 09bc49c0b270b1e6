// Weighted combination of a token's expert outputs, and its gradients.
//
//   out[t] = base[t] + sum_j w[t,j] y[t,j]
//   dy[t,j] = w[t,j] dout[t],   dw[t,j] = <dout[t], y[t,j]>
//
// Every row of y is read (and of dy written) once: both are bound by memory.
// Measured: 4096 tokens x 8 rows of 7168 in bf16 onto a base 91 us (6.4 TB/s; a
// stream that is only read reaches 6.9), the gradients of 2048 x 8 rows of 6144
// 81 us (5.3 TB/s, half of it written; a large copy reaches 5.0).
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

// 16 bytes that no later call is likely to find in a cache (without the hint
// the two take 97 and 89 us).
__device__ __forceinline__ v4u load_once(const void* base, size_t i) {
  return __builtin_nontemporal_load(static_cast<const v4u*>(base) + i);
}
__device__ __forceinline__ void store_once(void* base, size_t i, v4u v) {
  __builtin_nontemporal_store(v, static_cast<v4u*>(base) + i);
}

constexpr int kBatch = 8;   // rows of y in flight

constexpr int kThreads = 128;   // of a work-group of the combination

// One thread per 16 bytes of an output row: the rows of y of kBatch places are
// loaded together (a place that is left out loads nothing), then added in order.
// With one place after the other it took 112 us.
template <bool F32>
__global__ __launch_bounds__(kThreads) void combine_kernel(CombineParams p) {
  constexpr int V = Piece<F32>::kValues;
  const uint32_t pieces = (uint32_t)(p.H / V);
  const uint32_t wide = (pieces + kThreads - 1) / kThreads;          // work-groups of a row
  const int lane = threadIdx.x & 63;
  for (size_t block = blockIdx.x; block < (size_t)p.M * wide; block += gridDim.x) {
    const size_t t = block / wide;
    const uint32_t h = (uint32_t)(block % wide) * kThreads + threadIdx.x;
    const size_t at = t * pieces + h;
    const bool in = h < pieces;
    Piece<F32> acc{};
    if (p.base && in) acc = unpack<F32>(load_once(p.base, at));
    for (int j0 = 0; j0 < p.K; j0 += kBatch) {
      // lane j looks at place j0 + j; the wave then has them in scalar registers
      const size_t first = t * p.K + j0;
      const bool mine = lane < kBatch && j0 + lane < p.K && live(p, first + lane);
      const float weight = mine ? p.weights[first + lane] : 0.0f;
      const uint64_t lives = __ballot(mine);
      v4u y[kBatch];
#pragma unroll
      for (int j = 0; j < kBatch; ++j)
        if ((lives >> j) & 1) y[j] = in ? load_once(p.y, (first + j) * pieces + h) : v4u{0, 0, 0, 0};
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        if (!((lives >> j) & 1)) continue;
        const float w = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(weight), j));
        const Piece<F32> r = unpack<F32>(y[j]);
#pragma unroll
        for (int i = 0; i < V; ++i) acc.v[i] = fmaf(w, r.v[i], acc.v[i]);
      }
    }
    if (in) store_once(p.out, at, pack<F32>(acc));
  }
}

// A wave per pair: its dot product needs no other wave.  d_out is read again by
// a token's other pairs and stays in the caches.
template <bool F32>
__global__ __launch_bounds__(256) void combine_backward_kernel(CombineParams p) {
  constexpr int V = Piece<F32>::kValues;
  const int pieces = p.H / V;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  for (size_t pair = (size_t)blockIdx.x * 4 + wave; pair < (size_t)p.M * p.K; pair += (size_t)gridDim.x * 4) {
    const size_t t = pair / p.K;
    const bool on = live(p, pair);
    const float w = on ? p.weights[pair] : 0.0f;
    float dot = 0.0f;
#pragma unroll 4
    for (int h = lane; h < pieces; h += 64) {
      Piece<F32> d{};
      if (on) {
        d = unpack<F32>(static_cast<const v4u*>(p.d_out)[t * pieces + h]);
        if (p.d_weights) {
          const Piece<F32> y = unpack<F32>(load_once(p.y, pair * pieces + h));
#pragma unroll
          for (int i = 0; i < V; ++i) dot = fmaf(d.v[i], y.v[i], dot);
        }
#pragma unroll
        for (int i = 0; i < V; ++i) d.v[i] *= w;
      }
      if (p.d_y) store_once(p.d_y, pair * pieces + h, pack<F32>(d));
    }
    if (!p.d_weights) continue;
    for (int s = 32; s; s >>= 1) dot += __shfl_xor(dot, s);
    if (lane == 0) p.d_weights[pair] = dot;
  }
}

template <bool F32>
hipError_t launch(const CombineParams& p, bool backward, hipStream_t stream) {
  CombineParams q = p;
  void* args[] = {&q};
  const size_t wide = (p.H / Piece<F32>::kValues + kThreads - 1) / kThreads;
  size_t blocks = backward ? ((size_t)p.M * p.K + 3) / 4 : (size_t)p.M * wide;
  if (blocks > (1u << 20)) blocks = 1u << 20;  // the kernels stride the rest
  const void* f = backward ? reinterpret_cast<const void*>(&combine_backward_kernel<F32>)
                           : reinterpret_cast<const void*>(&combine_kernel<F32>);
  return hipLaunchKernel(f, dim3((unsigned)blocks), dim3(backward ? 256 : kThreads), args, 0, stream);
}

}  // namespace

hipError_t launch_combine(const CombineParams& p, hipStream_t stream) {
  return p.xf32 ? launch<true>(p, false, stream) : launch<false>(p, false, stream);
}

hipError_t launch_combine_backward(const CombineParams& p, hipStream_t stream) {
  return p.xf32 ? launch<true>(p, true, stream) : launch<false>(p, true, stream);
}

}  // namespace q4
