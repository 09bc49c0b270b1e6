// Router: scores, choice of the K best experts, weights, batch statistics of
// the balance loss, and the gradient of the logits.
//
// A group of L lanes holds one token: lane l has experts v * L + l (v < VPT),
// so a row is read once into registers and its softmax sums and choice stay
// there.  Padding experts (e >= E) hold -inf.
//
// L is 16 or 64.  The choice costs K dependent rounds of a maximum over the
// lanes; with 16 lanes a round has four steps inside one lane row instead of
// six and serves the wave's four tokens at once.
//
// These kernels are short enough that fetching their code counts: the loops
// over a lane's experts have no branches, and the rare choice in double
// precision is one loop over the tokens that need it, a whole wave for each
// (with both unrolled in place the router below took 25 us).
//
// Measured: 8192 tokens, 256 experts, sigmoid and bias, eight chosen, with the
// statistics 15 + 6.7 us, bound by the instructions of the nine rounds (4 MB of
// logits are 1 us of memory traffic); its gradient 8.8; one token 3.4.
#include "q4moe_device.h"
#include "q4moe_layer.h"

namespace q4 {

namespace {

constexpr int kWaves = 8;            // waves of a work-group
constexpr int kMaxBlocks = 256;      // work-groups of a call with statistics
constexpr int kStatThreads = 256;
constexpr int kStatExperts = 32;     // experts of a work-group that joins the statistics
constexpr int kRun = 32;             // tokens whose probabilities a lane adds up in F32

// Lane l's logits of the row at byte offset `row` (-inf where there is no
// expert).  The type is asked once, so that the loads are in flight together.
template <int L, int VPT>
__device__ __forceinline__ void load_row(__amdgpu_buffer_rsrc_t src, int f32, uint32_t row, int E, int l,
                                         float (&x)[VPT]) {
  uint32_t u[VPT];
  if (f32) {
#pragma unroll
    for (int v = 0; v < VPT; ++v)
      u[v] = __builtin_amdgcn_raw_buffer_load_b32(src, (int)(row + 4u * (uint32_t)l) + 4 * L * v, 0, 0);
  } else {
#pragma unroll
    for (int v = 0; v < VPT; ++v)
      u[v] = (uint32_t)__builtin_amdgcn_raw_buffer_load_b16(src, (int)(row + 2u * (uint32_t)l) + 2 * L * v, 0, 0) << 16;
  }
#pragma unroll
  for (int v = 0; v < VPT; ++v) x[v] = v * L + l < E ? __uint_as_float(u[v]) : -__builtin_inff();
}

// Lane l's values of a vector over the experts (0 where there are none, or no vector).
template <int L, int VPT>
__device__ __forceinline__ void load_experts(const float* a, int E, int l, float (&x)[VPT]) {
  const __amdgpu_buffer_rsrc_t src = make_rsrc(a, a ? 4u * (uint32_t)E : 0u);
#pragma unroll
  for (int v = 0; v < VPT; ++v)
    x[v] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(src, 4 * (v * L + l), 0, 0));
}

template <class T>
struct Halves {
  static constexpr int kCount = sizeof(T) / 4;
  int w[kCount];
};

// v of the lane C positions on in its row of 16 (row_ror).
template <int C, class T>
__device__ __forceinline__ T ror(T v) {
  auto h = __builtin_bit_cast(Halves<T>, v);
#pragma unroll
  for (int i = 0; i < Halves<T>::kCount; ++i) h.w[i] = __builtin_amdgcn_mov_dpp(h.w[i], 0x120 + C, 0xF, 0xF, true);
  return __builtin_bit_cast(T, h);
}

// The values of the even and the odd rows of 16 lanes (of the two halves of the wave), in every lane.
template <bool WIDE, class T, class F>
__device__ __forceinline__ T join_rows(T v, F f) {
  Halves<T> a = __builtin_bit_cast(Halves<T>, v), b = a;
#pragma unroll
  for (int i = 0; i < Halves<T>::kCount; ++i) {
    const auto r = WIDE ? __builtin_amdgcn_permlane32_swap(a.w[i], b.w[i], false, false)
                        : __builtin_amdgcn_permlane16_swap(a.w[i], b.w[i], false, false);
    a.w[i] = (int)r[0];
    b.w[i] = (int)r[1];
  }
  return f(__builtin_bit_cast(T, a), __builtin_bit_cast(T, b));
}

// f over the group's L lanes, the same bits in each of them (f commutes).  All 64 lanes take part.
template <int L, class T, class F>
__device__ __forceinline__ T group_join(T v, F f) {
  v = f(v, ror<8>(v));
  v = f(v, ror<4>(v));
  v = f(v, ror<2>(v));
  v = f(v, ror<1>(v));
  if constexpr (L == 64) {
    v = join_rows<false>(v, f);
    v = join_rows<true>(v, f);
  }
  return v;
}
template <int L, class T>
__device__ __forceinline__ T group_sum(T v) {
  return group_join<L>(v, [](T a, T b) { return a + b; });
}
template <int L, class T>
__device__ __forceinline__ T group_max(T v) {
  return group_join<L>(v, [](T a, T b) { return b > a ? b : a; });
}
template <int L>
__device__ __forceinline__ float group_fmax(float v) {
  return group_join<L>(v, [](float a, float b) { return fmaxf(a, b); });
}
template <int L>
__device__ __forceinline__ uint32_t group_min(uint32_t v) {
  return group_join<L>(v, [](uint32_t a, uint32_t b) { return b < a ? b : a; });
}

// Joins a lane's N values in a tree (N a power of two): log2(N) roundings for a sum.
template <int N, class T, class F>
__device__ __forceinline__ T tree(const T (&a)[N], F f) {
  T t[N];
#pragma unroll
  for (int v = 0; v < N; ++v) t[v] = a[v];
#pragma unroll
  for (int d = N / 2; d; d >>= 1)
#pragma unroll
    for (int v = 0; v < d; ++v) t[v] = f(t[v], t[v + d]);
  return t[0];
}

// Unsigned keys in the order of the values they stand for: 0 for -inf (never
// chosen), the highest for NaN, and -0 as +0.
__device__ __forceinline__ uint32_t order_key(float v) {
  const uint32_t u = __float_as_uint(v + 0.0f);
  uint32_t k = u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
  k = v == -__builtin_inff() ? 0u : k;
  return v != v ? 0xFFFFFFFFu : k;
}
__device__ __forceinline__ uint64_t order_key(double v) {
  const uint64_t u = (uint64_t)__double_as_longlong(v + 0.0);
  uint64_t k = u ^ ((uint64_t)((int64_t)u >> 63) | 0x8000000000000000ull);
  k = v == -__builtin_inf() ? 0ull : k;
  return v != v ? ~0ull : k;
}
__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xFFFFFFFFu));
}

// The K experts of highest key, best first, ties to the lowest index, then -1,
// into the group's out[0..K).  Keys are used up.  With `watch` (keys of 32
// bits) the result tells the groups where neighbours in that order, the first
// one left out among them, are too close to trust F32.
template <int L, int VPT, class Key>
__device__ __forceinline__ bool choose(Key (&key)[VPT], int K, int l, bool watch, int* out) {
  bool close = false;
  float last = 0.0f;
  for (int j = 0; j < K + (watch ? 1 : 0); ++j) {
    const Key best = group_max<L>(tree<VPT>(key, [](Key a, Key b) { return b > a ? b : a; }));
    if constexpr (sizeof(Key) == 4) {
      if (watch) {
        // two F32 scores differ by less than 32 roundings (2^-19) from what
        // they should, the sums with the bias by half a step each:
        // neighbours further apart are in order
        const float now = key_value(best);
        close = close || (j && best && !(last - now > 0x1p-19f + 0x1p-22f * fabsf(last)));
        last = now;
        if (j == K) break;
      }
    }
    uint32_t mine = 0x10000u;
#pragma unroll
    for (int v = VPT - 1; v >= 0; --v) mine = key[v] == best ? (uint32_t)(v * L) : mine;
    const uint32_t first = group_min<L>(mine + (uint32_t)l);
    const uint32_t mark = first - (uint32_t)l;
#pragma unroll
    for (int v = 0; v < VPT; ++v) key[v] = (uint32_t)(v * L) == mark ? (Key)0 : key[v];
    if (l == 0) out[j] = best ? (int)first : -1;
  }
  return close;
}

__device__ __forceinline__ float exp_of(float x) { return expf(x); }
__device__ __forceinline__ double exp_of(double x) { return exp(x); }
__device__ __forceinline__ float inverse(float x) { return __builtin_amdgcn_rcpf(x); }   // within 2^-23 relative
__device__ __forceinline__ double inverse(double x) { return 1.0 / x; }

// Scores of a row in T (float or double): softmax, or sigmoids; `sum` is the
// sum of the scores (softmax: 1 up to rounding).  A padding expert scores 0.
template <int L, int VPT, class T>
__device__ __forceinline__ void scores(const float (&x)[VPT], int sigmoid, T (&s)[VPT], T& sum) {
  const auto add = [](T a, T b) { return a + b; };
  if (sigmoid) {
#pragma unroll
    for (int v = 0; v < VPT; ++v) s[v] = inverse((T)1 + exp_of(-(T)x[v]));
    sum = group_sum<L>(tree<VPT>(s, add));
    return;
  }
  const T m = (T)group_fmax<L>(tree<VPT>(x, [](float a, float b) { return fmaxf(a, b); }));
#pragma unroll
  for (int v = 0; v < VPT; ++v) s[v] = exp_of((T)x[v] - m);
  const T inv = (T)1 / group_sum<L>(tree<VPT>(s, add));
#pragma unroll
  for (int v = 0; v < VPT; ++v) s[v] *= inv;
  sum = 1;
}

// The choice by score plus bias in double precision, for one token by a whole wave.
template <int VPT>
__device__ __forceinline__ void choose_exact(const RouteParams& p, __amdgpu_buffer_rsrc_t src, uint32_t row, int lane,
                                             int* out) {
  float x[VPT], bias[VPT];
  load_row<64, VPT>(src, p.lf32, row, p.E, lane, x);
  load_experts<64, VPT>(p.bias, p.E, lane, bias);
  double s[VPT], sum;
  scores<64, VPT, double>(x, p.sigmoid, s, sum);
  uint64_t key[VPT];
#pragma unroll
  for (int v = 0; v < VPT; ++v) {
    key[v] = order_key(s[v] + (double)bias[v]);
    key[v] = x[v] == -__builtin_inff() ? 0ull : key[v];
  }
  choose<64, VPT>(key, p.K, lane, false, out);
}

// Workspace of the statistics: a ticket, the parts of the loss (a double per
// joining work-group), then per work-group of the router its tokens [blocks],
// sums of the probabilities [blocks][E] and counts [blocks][E].
constexpr size_t kLossPartsAt = 256, kTokensAt = 512;
static_assert(kLossPartsAt + 8 * (kRouteMaxExperts / kStatExperts) <= kTokensAt, "loss parts fit the header");

struct Partials {
  uint32_t* ticket;
  double* loss_parts;
  int* tokens;
  float* sums;
  int* counts;
  __device__ Partials(void* ws, int blocks, int E) {
    uint8_t* at = static_cast<uint8_t*>(ws);
    ticket = reinterpret_cast<uint32_t*>(at);
    loss_parts = reinterpret_cast<double*>(at + kLossPartsAt);
    tokens = reinterpret_cast<int*>(at + kTokensAt);
    sums = reinterpret_cast<float*>(tokens + blocks);
    counts = reinterpret_cast<int*>(sums + (size_t)blocks * E);
  }
};

// STATS: with the batch statistics (p.partials).  They have kernels of their own
// for the registers of their sums: with them 257..512 experts take 141, which
// would leave the call without statistics one work-group a CU instead of two.
template <int L, int VPT, bool STATS>
__global__ __launch_bounds__(kWaves * 64) void route_kernel(RouteParams p) {
  constexpr int G = 64 / L;          // tokens of a wave
  constexpr int kRow = L * VPT + 16; // floats of a token's scores in LDS (the four tokens on different banks)
  __shared__ float s_score[kWaves][G][kRow];
  __shared__ int s_pick[kWaves][G][kRouteMaxTopK];
  __shared__ int s_count[STATS ? L * VPT : 1];
  __shared__ int s_tokens;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int l = lane % L, group = lane / L;
  int* const pick = s_pick[wave][group];
  float* const score = s_score[wave][group];
  const uint32_t pitch = (uint32_t)p.E * (p.lf32 ? 4u : 2u);
  // a lane's sums over its tokens: kRun of them in F32, the runs in double
  float psum[VPT] = {}, bias[VPT];
  double psums[VPT] = {};
  int in_run = 0;
  load_experts<L, VPT>(p.bias, p.E, l, bias);
  if constexpr (STATS) {
    for (int e = threadIdx.x; e < L * VPT; e += kWaves * 64) s_count[e] = 0;
    if (threadIdx.x == 0) s_tokens = 0;
    __syncthreads();
  }
  for (int t0 = ((int)blockIdx.x * kWaves + wave) * G; t0 < p.M; t0 += (int)gridDim.x * kWaves * G) {
    const int t = t0 + group;
    const int tokens = min(G, p.M - t0);
    const __amdgpu_buffer_rsrc_t src =
        make_rsrc(static_cast<const uint8_t*>(p.logits) + (size_t)t0 * pitch, (uint32_t)tokens * pitch);
    bool on = t < p.M;
    if (on && p.mask) on = p.mask[t] != 0;
    float x[VPT], s[VPT], sum;
    load_row<L, VPT>(src, p.lf32, (uint32_t)group * pitch, p.E, l, x);
    scores<L, VPT, float>(x, p.sigmoid, s, sum);
    uint32_t key[VPT];
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      score[v * L + l] = s[v];
      key[v] = order_key(p.bias ? s[v] + bias[v] : x[v]);
      key[v] = on && x[v] != -__builtin_inff() ? key[v] : 0u;
    }
    const bool close = choose<L, VPT>(key, p.K, l, p.bias != nullptr, pick);
    // neighbours that F32 cannot tell apart: the same choice in double
    const uint64_t doubt = __ballot(close);
    for (int g = 0; g < G && doubt; ++g)
      if ((doubt >> (g * L)) & 1) choose_exact<(L * VPT + 63) / 64>(p, src, (uint32_t)g * pitch, lane, s_pick[wave][g]);
    wave_sync();
    const bool here = pick[0] >= 0;
    float total = 1.0f;
    if (p.renormalize) {
      float part = 0.0f;
      for (int j = l; j < p.K; j += L) part += pick[j] >= 0 ? score[pick[j]] : 0.0f;
      total = group_sum<L>(part);
    }
    if (t < p.M) {
      for (int j = l; j < p.K; j += L) {
        const int e = pick[j];
        float w = 0.0f;
        if (e >= 0) {
          w = score[e];
          if (p.renormalize) w = total == 0.0f ? 0.0f : w / total;
          if constexpr (STATS) atomicAdd(&s_count[e], 1);
        }
        p.ids[(size_t)t * p.K + j] = e;
        p.weights[(size_t)t * p.K + j] = w * p.scale;
      }
    }
    if constexpr (STATS) {
      if (l == 0 && here) atomicAdd(&s_tokens, 1);
      const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
      for (int v = 0; v < VPT; ++v) psum[v] += here ? s[v] * inv : 0.0f;
      if (++in_run == kRun) {
        in_run = 0;
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
          psums[v] += (double)psum[v];
          psum[v] = 0.0f;
        }
      }
    }
    wave_sync();
  }
  if constexpr (!STATS) return;
#pragma unroll
  for (int v = 0; v < VPT; ++v) {
    psum[v] = (float)(psums[v] + (double)psum[v]);
    if constexpr (G > 1) {             // the wave's four tokens, in one order
      const auto add = [](float a, float b) { return a + b; };
      psum[v] = join_rows<false>(psum[v], add);
      psum[v] = join_rows<true>(psum[v], add);
    }
    if (group == 0) score[v * L + l] = psum[v];
  }
  __syncthreads();
  const Partials out(p.partials, (int)gridDim.x, p.E);
  for (int e = threadIdx.x; e < p.E; e += kWaves * 64) {
    float a = 0.0f;
#pragma unroll
    for (int i = 0; i < kWaves; ++i) a += s_score[i][0][e];
    out.sums[(size_t)blockIdx.x * p.E + e] = a;
    out.counts[(size_t)blockIdx.x * p.E + e] = s_count[e];
  }
  if (threadIdx.x == 0) {
    out.tokens[blockIdx.x] = s_tokens;
    if (blockIdx.x == 0) *out.ticket = 0u;
  }
}

// Joins the router's work-groups: 32 experts a work-group, eight slices of the
// partials side by side.  The last work-group to finish (by the ticket that
// the router's launch cleared) adds the parts of the loss, in order.
// (Latency only: 6.9 us for 256 partials of 256 experts; with 32 slices 8.3.)
__global__ __launch_bounds__(kStatThreads) void route_stats_kernel(RouteParams p, int blocks) {
  constexpr int kSlices = kStatThreads / kStatExperts;
  __shared__ double s_sum[kSlices][kStatExperts];
  __shared__ int s_count[kSlices][kStatExperts];
  __shared__ int s_tokens;
  const Partials in(p.partials, blocks, p.E);
  const int x = threadIdx.x % kStatExperts, y = threadIdx.x / kStatExperts;
  const int e = (int)blockIdx.x * kStatExperts + x;
  static_assert(kMaxBlocks <= kStatThreads, "a thread for each work-group's tokens");
  const int part = (int)threadIdx.x < blocks ? in.tokens[threadIdx.x] : 0;
  if (threadIdx.x == 0) s_tokens = 0;
  __syncthreads();
  if (part) atomicAdd(&s_tokens, part);
  double sum = 0.0;
  int count = 0;
  if (e < p.E) {
#pragma unroll 16
    for (int b = y; b < blocks; b += kSlices) {
      sum += (double)in.sums[(size_t)b * p.E + e];
      count += in.counts[(size_t)b * p.E + e];
    }
  }
  s_sum[y][x] = sum;
  s_count[y][x] = count;
  __syncthreads();
  if (threadIdx.x >= kStatExperts) return;
#pragma unroll
  for (int i = 1; i < kSlices; ++i) {
    sum += s_sum[i][x];
    count += s_count[i][x];
  }
  const double tokens = (double)s_tokens;
  const double grad = s_tokens ? (double)p.E * count / ((double)p.K * tokens * tokens) : 0.0;
  if (e < p.E) {
    if (p.counts) p.counts[e] = count;
    if (p.loss_grad) p.loss_grad[e] = (float)grad;
  }
  if (!p.loss) return;
  double loss = grad * sum;
  for (int d = kStatExperts / 2; d; d >>= 1) loss += __shfl_xor(loss, d);
  if (threadIdx.x != 0) return;
  __hip_atomic_store(&in.loss_parts[blockIdx.x], loss, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  if (__hip_atomic_fetch_add(in.ticket, 1u, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT) != gridDim.x - 1) return;
  double total = 0.0;
  for (unsigned b = 0; b < gridDim.x; ++b)
    total += __hip_atomic_load(&in.loss_parts[b], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  p.loss[0] = (float)total;
}

template <int L, int VPT>
__global__ __launch_bounds__(kWaves * 64) void route_backward_kernel(RouteBackwardParams p) {
  constexpr int G = 64 / L;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int l = lane % L, group = lane / L;
  const auto add = [](float a, float b) { return a + b; };
  const uint32_t size = p.lf32 ? 4u : 2u, pitch = (uint32_t)p.E * size;
  const float d_loss = p.d_loss ? p.d_loss[0] : 0.0f;
  float gl[VPT];
  load_experts<L, VPT>(p.loss_grad, p.E, l, gl);
#pragma unroll
  for (int v = 0; v < VPT; ++v) gl[v] *= d_loss;
  for (int t0 = ((int)blockIdx.x * kWaves + wave) * G; t0 < p.M; t0 += (int)gridDim.x * kWaves * G) {
    const int t = t0 + group;
    const int tokens = min(G, p.M - t0);
    const bool in = t < p.M;
    const __amdgpu_buffer_rsrc_t src =
        make_rsrc(static_cast<const uint8_t*>(p.logits) + (size_t)t0 * pitch, (uint32_t)tokens * pitch);
    const __amdgpu_buffer_rsrc_t dst =
        make_rsrc(static_cast<uint8_t*>(p.d_logits) + (size_t)t0 * pitch, (uint32_t)tokens * pitch);
    const uint32_t row = (uint32_t)group * pitch;
    // lane l holds the places l, l + L, ...; an id that names no expert is
    // dropped here: it could name a padding expert, whose score of 0 would
    // still carry an infinite or NaN gradient into the row's sums
    const auto named = [&](int e) { return (uint32_t)e < (uint32_t)p.E ? e : -1; };
    const size_t places = (size_t)t * p.K;
    int id = in && l < p.K ? p.ids[places + l] : -1;
    float dw = in && l < p.K && p.d_weights ? p.d_weights[places + l] : 0.0f;
    float x[VPT], s[VPT], sum;
    load_row<L, VPT>(src, p.lf32, row, p.E, l, x);
    const bool here = __shfl(id, 0, L) >= 0;
    id = named(id);
    scores<L, VPT, float>(x, p.sigmoid, s, sum);
    // g: the gradients that reach each expert, n: the places that chose it
    float g[VPT] = {};
    int n[VPT] = {};
    for (int j = 0; j < p.K; ++j) {
      if (j && j % L == 0) {
        id = in && j + l < p.K ? named(p.ids[places + j + l]) : -1;
        dw = in && j + l < p.K && p.d_weights ? p.d_weights[places + j + l] : 0.0f;
      }
      const int e = __shfl(id, j % L, L) - l;
      const float d = p.scale * __shfl(dw, j % L, L);
#pragma unroll
      for (int v = 0; v < VPT; ++v) {
        g[v] += v * L == e ? d : 0.0f;
        n[v] += v * L == e;
      }
    }
    if (p.renormalize) {
      // w_j = s_j / S: ds_j = (dw_j - sum_i dw_i s_i / S) / S
      float a[VPT], b[VPT];
#pragma unroll
      for (int v = 0; v < VPT; ++v) {
        a[v] = n[v] ? (float)n[v] * s[v] : 0.0f;
        b[v] = n[v] ? g[v] * s[v] : 0.0f;
      }
      const float total = group_sum<L>(tree<VPT>(a, add));
      const float inv = total != 0.0f ? 1.0f / total : 0.0f;
      const float mean = group_sum<L>(tree<VPT>(b, add)) * inv;
#pragma unroll
      for (int v = 0; v < VPT; ++v) g[v] = n[v] ? (g[v] - (float)n[v] * mean) * inv : 0.0f;
    }
    // softmax: dl = s (g - <s, g>); sigmoid: the loss reaches s through s / sum, dl = ds s (1 - s)
    float d[VPT];
    if (p.sigmoid) {
#pragma unroll
      for (int v = 0; v < VPT; ++v) d[v] = s[v] * gl[v];
      const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
      const float mean = group_sum<L>(tree<VPT>(d, add)) * inv;
      // 1 - s = 1 / (1 + exp(l)), without cancellation
#pragma unroll
      for (int v = 0; v < VPT; ++v)
        d[v] = (g[v] + (gl[v] - mean) * inv) * s[v] * inverse(1.0f + exp_of(x[v]));
    } else {
#pragma unroll
      for (int v = 0; v < VPT; ++v) d[v] = s[v] * (g[v] + gl[v]);
      const float mean = group_sum<L>(tree<VPT>(d, add));
#pragma unroll
      for (int v = 0; v < VPT; ++v) d[v] = s[v] * (g[v] + gl[v] - mean);
    }
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      const uint32_t at = in && v * L + l < p.E ? row + (uint32_t)(v * L + l) * size : kOffNone;
      const float r = here ? d[v] : 0.0f;
      if (p.lf32) __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(r), dst, (int)at, 0, 0);
      else __builtin_amdgcn_raw_buffer_store_b16(bf16_rne(r), dst, (int)at, 0, 0);
    }
  }
}

// Lanes of a token.  A wave with 16 experts a lane is long: with few tokens,
// where only its latency shows, 64 lanes a token finish sooner (router and
// gradient at 256 experts, 1000 tokens: 6.2 and 4.6 us against 10.1 and 7.3;
// 4000: 9.8 and 5.7 against 10.6 and 7.4), with many the four tokens of a wave
// do (64000: 59 us against 116, the gradient 55 against 46).  Up to 64 experts
// 16 lanes are as fast at 64 tokens (5.0 us against 4.8) and faster from 4000 on.
int lanes_of(int M, int E) { return E > 256 || (E > 64 && M <= 4096) ? 64 : 16; }

// Work-groups that give every token its group of lanes.
int token_blocks(int M, int E) {
  const int tokens = kWaves * (64 / lanes_of(M, E));
  return (M + tokens - 1) / tokens;
}

int stat_blocks(int M, int E) {
  const int b = token_blocks(M, E);
  return b < kMaxBlocks ? b : kMaxBlocks;
}

template <class P>
hipError_t run(const void* const (&kernels)[10], const P& p, int blocks, hipStream_t stream) {
  P q = p;
  void* args[] = {&q};
  const int L = lanes_of(p.M, p.E);
  int i = 0;
  while ((L << i) < p.E) ++i;
  if (L == 64) i += 5;
  return hipLaunchKernel(kernels[i], dim3((unsigned)blocks), dim3(kWaves * 64), args, 0, stream);
}

// A kernel's variants by lanes of a token and experts of a lane.
#define Q4_ROUTE_KERNELS(k) \
  {k(16, 1), k(16, 2), k(16, 4), k(16, 8), k(16, 16), k(64, 1), k(64, 2), k(64, 4), k(64, 8), k(64, 16)}
#define Q4_ROUTE_PLAIN(L, VPT) reinterpret_cast<const void*>(&route_kernel<L, VPT, false>)
#define Q4_ROUTE_STATS(L, VPT) reinterpret_cast<const void*>(&route_kernel<L, VPT, true>)
#define Q4_ROUTE_BACKWARD(L, VPT) reinterpret_cast<const void*>(&route_backward_kernel<L, VPT>)

}  // namespace

// For as many work-groups as any smaller batch has: those of 64 lanes a token,
// whatever lanes this one takes.
size_t route_partial_bytes(int64_t M, int64_t E) {
  const int64_t most = (M + kWaves - 1) / kWaves;
  const size_t bytes = kTokensAt + (size_t)(most < kMaxBlocks ? most : kMaxBlocks) * (2 * (size_t)E + 1) * 4;
  return (bytes + 255) / 256 * 256;
}

hipError_t launch_route(const RouteParams& p, hipStream_t stream) {
  static const void* const plain[10] = Q4_ROUTE_KERNELS(Q4_ROUTE_PLAIN);
  static const void* const stats[10] = Q4_ROUTE_KERNELS(Q4_ROUTE_STATS);
  const int all = token_blocks(p.M, p.E);
  if (!p.partials) return run(plain, p, all < 65536 ? all : 65536, stream);
  const int blocks = stat_blocks(p.M, p.E);
  const hipError_t e = run(stats, p, blocks, stream);
  if (e != hipSuccess) return e;
  RouteParams q = p;
  int nb = blocks;
  void* args[] = {&q, &nb};
  return hipLaunchKernel(reinterpret_cast<const void*>(&route_stats_kernel),
                         dim3((unsigned)((p.E + kStatExperts - 1) / kStatExperts)), dim3(kStatThreads), args, 0, stream);
}

hipError_t launch_route_backward(const RouteBackwardParams& p, hipStream_t stream) {
  static const void* const kernels[10] = Q4_ROUTE_KERNELS(Q4_ROUTE_BACKWARD);
  const int all = token_blocks(p.M, p.E);
  return run(kernels, p, all < 65536 ? all : 65536, stream);
}

}  // namespace q4
