// Router: scores, choice of the K best experts, weights, batch statistics of
// the balance loss, and the gradient of the logits.
//
// One wave per token.  Lane l holds experts v * 64 + l (v < VPT), so a row is
// read once into registers; softmax sums, the choice and the weights stay
// there.  Padding experts (e >= E) hold -inf.
#include "q4moe_device.h"
#include "q4moe_layer.h"

namespace q4 {

namespace {

constexpr int kWaves = 4;            // waves (tokens in flight) of a work-group
constexpr int kMaxBlocks = 256;      // work-groups of a call with statistics

__device__ __forceinline__ float load_logit(const void* l, int f32, size_t i) {
  return f32 ? static_cast<const float*>(l)[i] : bf16_val(static_cast<const uint16_t*>(l)[i]);
}

__device__ __forceinline__ float wave_sum(float v) {
  for (int d = 32; d; d >>= 1) v += __shfl_xor(v, d);
  return v;
}
__device__ __forceinline__ double wave_sum(double v) {
  for (int d = 32; d; d >>= 1) v += __shfl_xor(v, d);
  return v;
}
__device__ __forceinline__ float wave_max(float v) {
  for (int d = 32; d; d >>= 1) v = fmaxf(v, __shfl_xor(v, d));
  return v;
}

// Unsigned keys in the order of the values they stand for: 0 for -inf (never
// chosen), the highest for NaN, and -0 as +0.
__device__ __forceinline__ uint32_t order_key(float v) {
  if (v != v) return 0xFFFFFFFFu;
  if (v == -__builtin_inff()) return 0u;
  const uint32_t u = __float_as_uint(v + 0.0f);
  return u ^ ((u >> 31) ? 0xFFFFFFFFu : 0x80000000u);
}
__device__ __forceinline__ uint64_t order_key(double v) {
  if (v != v) return ~0ull;
  if (v == -__builtin_inf()) return 0ull;
  const uint64_t u = (uint64_t)__double_as_longlong(v + 0.0);
  return u ^ ((u >> 63) ? ~0ull : 0x8000000000000000ull);
}
__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xFFFFFFFFu));
}

__device__ __forceinline__ uint32_t wave_max_key(uint32_t k) { return wave_extreme<true>(k); }
__device__ __forceinline__ uint64_t wave_max_key(uint64_t k) {
  for (int d = 32; d; d >>= 1) {
    const uint64_t o = (uint64_t)__shfl_xor((unsigned long long)k, d);
    k = o > k ? o : k;
  }
  return k;
}

// The K experts of highest key, best first, ties to the lowest index: lane j
// returns the j-th (or -1).  Keys are used up.  `closest` (keys of 32 bits)
// receives the smallest distance between neighbours in that order, the first
// one left out among them.
template <int VPT, class Key>
__device__ __forceinline__ int choose(Key (&key)[VPT], int K, int lane, bool* close) {
  int mine = -1;
  float last = 0.0f;
  for (int j = 0; j < K + (close ? 1 : 0); ++j) {
    Key best = key[0];
#pragma unroll
    for (int v = 1; v < VPT; ++v) best = key[v] > best ? key[v] : best;
    best = wave_max_key(best);
    if (best == 0) break;
    if constexpr (sizeof(Key) == 4) {
      if (close) {
        const float now = key_value((uint32_t)best);
        // an F32 score is within 2^-21 of the exact one, a sum with the bias
        // within half a step more: neighbours further apart are in order
        if (j && !(last - now > 0x1p-20f * (1.0f + fabsf(last)))) *close = true;
        last = now;
      }
    }
    int at = 0;
    bool found = false;
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      const uint64_t who = __ballot(key[v] == best);
      if (!found && who) {
        found = true;
        const int l = __builtin_ctzll(who);
        at = v * 64 + l;
        if (lane == l) key[v] = 0;
      }
    }
    if (lane == j && j < K) mine = at;
  }
  return mine;
}

// Scores of a row in T (float or double): softmax, or sigmoids; `sum` is the
// sum of the scores (softmax: 1 up to rounding).
template <int VPT, class T>
__device__ __forceinline__ void scores(const float (&l)[VPT], int sigmoid, int E, int lane, T (&s)[VPT], T& sum) {
  T part = 0;
  if (sigmoid) {
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      s[v] = v * 64 + lane < E ? (T)1 / ((T)1 + exp(-(T)l[v])) : (T)0;
      part += s[v];
    }
    sum = wave_sum(part);
    return;
  }
  float m = l[0];
#pragma unroll
  for (int v = 1; v < VPT; ++v) m = fmaxf(m, l[v]);
  m = wave_max(m);
#pragma unroll
  for (int v = 0; v < VPT; ++v) {
    s[v] = v * 64 + lane < E ? exp((T)l[v] - (T)m) : (T)0;
    part += s[v];
  }
  const T all = wave_sum(part);
#pragma unroll
  for (int v = 0; v < VPT; ++v) s[v] /= all;
  sum = 1;
}

// The value of register array a at expert e (the same e in every lane).
template <int VPT>
__device__ __forceinline__ float pick(const float (&a)[VPT], int e) {
  float r = a[0];
#pragma unroll
  for (int v = 1; v < VPT; ++v) r = (e >> 6) == v ? a[v] : r;
  return __shfl(r, e & 63);
}

// Workspace of the statistics: per work-group the sums of the probabilities
// [E], then the counts [E] and the number of tokens, all 32-bit.
__host__ __device__ constexpr size_t partial_words(int E) { return 2 * (size_t)E + 1; }

template <int VPT>
__global__ __launch_bounds__(kWaves * 64) void route_kernel(RouteParams p) {
  __shared__ float s_sum[kWaves][VPT * 64];
  __shared__ int s_count[kWaves][VPT * 64];
  __shared__ int s_tokens[kWaves];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  float psum[VPT] = {};
  int count[VPT] = {};
  int tokens = 0;
  for (int t = (int)blockIdx.x * kWaves + wave; t < p.M; t += (int)gridDim.x * kWaves) {
    float l[VPT];
    bool any = false;
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      const int e = v * 64 + lane;
      l[v] = e < p.E ? load_logit(p.logits, p.lf32, (size_t)t * p.E + e) : -__builtin_inff();
      any = any || !(l[v] == -__builtin_inff());
    }
    const bool here = (!p.mask || p.mask[t] != 0) && __ballot(any) != 0;
    int mine = -1;
    float w = 0.0f;
    if (here) {
      float s[VPT], sum;
      scores<VPT, float>(l, p.sigmoid, p.E, lane, s, sum);
      bool close = false;
      uint32_t key[VPT];
#pragma unroll
      for (int v = 0; v < VPT; ++v) {
        const int e = v * 64 + lane;
        key[v] = order_key(l[v]);
        if (p.bias && key[v]) key[v] = order_key(s[v] + p.bias[e]);
      }
      mine = choose<VPT>(key, p.K, lane, p.bias ? &close : nullptr);
      if (close) {
        // neighbours that F32 cannot tell apart: the same choice in double
        double ds[VPT], dsum;
        uint64_t dkey[VPT];
        scores<VPT, double>(l, p.sigmoid, p.E, lane, ds, dsum);
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
          const int e = v * 64 + lane;
          dkey[v] = order_key((double)l[v]);
          if (dkey[v]) dkey[v] = order_key(ds[v] + (double)p.bias[e]);
        }
        mine = choose<VPT>(dkey, p.K, lane, nullptr);
      }
      for (int j = 0; j < p.K; ++j) {
        const int e = __shfl(mine, j);
        if (e < 0) break;
        const float se = pick<VPT>(s, e);
        if (lane == j) w = se;
#pragma unroll
        for (int v = 0; v < VPT; ++v) count[v] += v * 64 + lane == e;
      }
      if (p.renormalize) {
        const float total = wave_sum(w);
        w = total == 0.0f ? 0.0f : w / total;
      }
      if (mine >= 0) w *= p.scale;
      ++tokens;
      const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
      for (int v = 0; v < VPT; ++v) psum[v] += s[v] * inv;
    }
    if (lane < p.K) {
      p.ids[(size_t)t * p.K + lane] = mine;
      p.weights[(size_t)t * p.K + lane] = w;
    }
  }
  if (!p.partials) return;
#pragma unroll
  for (int v = 0; v < VPT; ++v) {
    s_sum[wave][v * 64 + lane] = psum[v];
    s_count[wave][v * 64 + lane] = count[v];
  }
  if (lane == 0) s_tokens[wave] = tokens;
  __syncthreads();
  float* out = static_cast<float*>(p.partials) + (size_t)blockIdx.x * partial_words(p.E);
  for (int e = threadIdx.x; e < p.E; e += kWaves * 64) {
    float a = 0.0f;
    int c = 0;
    for (int i = 0; i < kWaves; ++i) {
      a += s_sum[i][e];
      c += s_count[i][e];
    }
    out[e] = a;
    reinterpret_cast<int*>(out)[p.E + e] = c;
  }
  if (threadIdx.x == 0) {
    int n = 0;
    for (int i = 0; i < kWaves; ++i) n += s_tokens[i];
    reinterpret_cast<int*>(out)[2 * p.E] = n;
  }
}

// Joins the work-groups' statistics: one work-group, a thread per expert.
__global__ __launch_bounds__(1024) void route_stats_kernel(RouteParams p, int blocks) {
  __shared__ double s_part[16];
  const int e = threadIdx.x, lane = threadIdx.x & 63;
  const size_t words = partial_words(p.E);
  const float* sums = static_cast<const float*>(p.partials);
  const int* ints = static_cast<const int*>(p.partials);
  double sum = 0.0;
  int count = 0, tokens = 0;
  for (int b = 0; b < blocks; ++b) {
    if (e < p.E) {
      sum += (double)sums[b * words + e];
      count += ints[b * words + p.E + e];
    }
    tokens += ints[b * words + 2 * p.E];
  }
  const double grad = tokens ? (double)p.E * count / ((double)p.K * tokens * tokens) : 0.0;
  if (e < p.E) {
    if (p.counts) p.counts[e] = count;
    if (p.loss_grad) p.loss_grad[e] = (float)grad;
  }
  const double part = wave_sum(grad * sum);
  if (lane == 0) s_part[threadIdx.x >> 6] = part;
  __syncthreads();
  if (p.loss && threadIdx.x == 0) {
    double total = 0.0;
    for (int i = 0; i < 16; ++i) total += s_part[i];
    p.loss[0] = (float)total;
  }
}

template <int VPT>
__global__ __launch_bounds__(kWaves * 64) void route_backward_kernel(RouteBackwardParams p) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const float d_loss = p.d_loss ? p.d_loss[0] : 0.0f;
  for (int t = (int)blockIdx.x * kWaves + wave; t < p.M; t += (int)gridDim.x * kWaves) {
    const int id = lane < p.K ? p.ids[(size_t)t * p.K + lane] : -1;
    const bool here = __shfl(id, 0) >= 0;
    float d[VPT] = {};
    if (here) {
      float l[VPT], s[VPT], sum;
#pragma unroll
      for (int v = 0; v < VPT; ++v) {
        const int e = v * 64 + lane;
        l[v] = e < p.E ? load_logit(p.logits, p.lf32, (size_t)t * p.E + e) : -__builtin_inff();
      }
      scores<VPT, float>(l, p.sigmoid, p.E, lane, s, sum);
      const bool on = id >= 0 && id < p.E;
      float dw = on && p.d_weights ? p.scale * p.d_weights[(size_t)t * p.K + lane] : 0.0f;
      if (p.renormalize) {
        // w_j = s_j / S: ds_j = (dw_j - sum_i dw_i s_i / S) / S
        float mine = 0.0f;
        for (int j = 0; j < p.K; ++j) {
          const int e = __shfl(id, j);
          if (e < 0 || e >= p.E) continue;
          const float se = pick<VPT>(s, e);
          if (lane == j) mine = se;
        }
        const float total = wave_sum(mine);
        const float mean = wave_sum(dw * mine) / total;
        dw = on && total != 0.0f ? (dw - mean) / total : 0.0f;
      }
      float g[VPT] = {}, gl[VPT];
      for (int j = 0; j < p.K; ++j) {
        const int e = __shfl(id, j);
        const float x = __shfl(dw, j);
#pragma unroll
        for (int v = 0; v < VPT; ++v) g[v] += v * 64 + lane == e ? x : 0.0f;
      }
      float dot = 0.0f;
#pragma unroll
      for (int v = 0; v < VPT; ++v) {
        const int e = v * 64 + lane;
        gl[v] = p.d_loss && e < p.E ? d_loss * p.loss_grad[e] : 0.0f;
        dot += s[v] * (p.sigmoid ? gl[v] : g[v] + gl[v]);
      }
      dot = wave_sum(dot);
      // softmax: dl = s (g - <s, g>); sigmoid: the loss reaches s through s / sum, dl = ds s (1 - s)
      const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
      for (int v = 0; v < VPT; ++v) {
        // 1 - s = 1 / (1 + exp(l)), without cancellation
        if (p.sigmoid) d[v] = (g[v] + (gl[v] - dot * inv) * inv) * s[v] * (1.0f / (1.0f + expf(l[v])));
        else d[v] = s[v] * (g[v] + gl[v] - dot);
      }
    }
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      const int e = v * 64 + lane;
      if (e >= p.E) continue;
      const size_t at = (size_t)t * p.E + e;
      if (p.lf32) static_cast<float*>(p.d_logits)[at] = d[v];
      else static_cast<uint16_t*>(p.d_logits)[at] = bf16_rne(d[v]);
    }
  }
}

int stat_blocks(int M) {
  const int b = (M + kWaves - 1) / kWaves;
  return b < kMaxBlocks ? b : kMaxBlocks;
}

template <class P>
hipError_t run(const void* const (&kernels)[5], const P& p, int blocks, hipStream_t stream) {
  P q = p;
  void* args[] = {&q};
  int i = 0;
  while ((64 << i) < p.E) ++i;  // VPT 1, 2, 4, 8, 16
  return hipLaunchKernel(kernels[i], dim3((unsigned)blocks), dim3(kWaves * 64), args, 0, stream);
}

#define Q4_ROUTE_KERNELS(k)                                                                             \
  {reinterpret_cast<const void*>(&k<1>), reinterpret_cast<const void*>(&k<2>),                          \
   reinterpret_cast<const void*>(&k<4>), reinterpret_cast<const void*>(&k<8>), reinterpret_cast<const void*>(&k<16>)}

}  // namespace

size_t route_partial_bytes(int64_t M, int64_t E) {
  const size_t bytes = (size_t)stat_blocks((int)M) * partial_words((int)E) * 4;
  return (bytes + 255) / 256 * 256;
}

hipError_t launch_route(const RouteParams& p, hipStream_t stream) {
  static const void* const kernels[5] = Q4_ROUTE_KERNELS(route_kernel);
  const int all = (p.M + kWaves - 1) / kWaves;
  const int blocks = p.partials ? stat_blocks(p.M) : (all < 65536 ? all : 65536);
  hipError_t e = run(kernels, p, blocks, stream);
  if (e != hipSuccess || !p.partials) return e;
  RouteParams q = p;
  int nb = blocks;
  void* args[] = {&q, &nb};
  return hipLaunchKernel(reinterpret_cast<const void*>(&route_stats_kernel), dim3(1), dim3(1024), args, 0, stream);
}

hipError_t launch_route_backward(const RouteBackwardParams& p, hipStream_t stream) {
  static const void* const kernels[5] = Q4_ROUTE_KERNELS(route_backward_kernel);
  const int all = (p.M + kWaves - 1) / kWaves;
  return run(kernels, p, all < 65536 ? all : 65536, stream);
}

}  // namespace q4
