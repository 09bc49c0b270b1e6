// Gradient of the input of the linear with 4-bit weights and group scales:
// d_x[m][k] = sum_n d_out[m][n] W[n][k].
//
// A work-group computes BM tokens by 128 columns k.  A step covers 128 bytes of
// the tokens' rows (64 values n in bf16, 32 in float); tokens and weights of the
// next step are fetched into registers while one is multiplied.  Weights run
// along k in memory and along n in the product, so a thread unpacks the words of
// neighbouring rows n at one place k and writes them side by side: a tile in LDS
// is [row][8 chunks of 16 bytes], tokens and columns alike, and a matrix operand
// is one 16-byte read.
#include "q4moe_device.h"
#include "q4moe_layer.h"
#include "q4moe_rows.h"

namespace q4 {

namespace {

typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef float v2f __attribute__((ext_vector_type(2)));
typedef uint32_t v2u __attribute__((ext_vector_type(2)));

constexpr int kThreads = 256;
constexpr int kCols = 128;           // columns k of a work-group
constexpr int kChunks = 8;           // 16-byte chunks of a tile's row
constexpr int kMaxSplits = 16;       // parts of n that work-groups share
constexpr int kFill = 512;           // work-groups that fill the device: no more parts than give so many

// Place of a row's chunk: the eight chunks change places from row to row and
// from eight rows to the next, so that neither the reads (16 rows of one chunk)
// nor the weights' writes (rows eight apart) meet in a bank.
__device__ __forceinline__ int place(int row, int chunk) { return row * kChunks + (chunk ^ ((row ^ (row >> 3)) & 7)); }

template <class T>
__device__ __forceinline__ v4f multiply(const v4u a, const v4u b, v4f c) {
  if constexpr (sizeof(T) == 2) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, a), __builtin_bit_cast(v8bf, b), c, 0, 0, 0);
  } else {
    const v4f x = __builtin_bit_cast(v4f, a), y = __builtin_bit_cast(v4f, b);
#pragma unroll
    for (int i = 0; i < 4; ++i) c = __builtin_amdgcn_mfma_f32_16x16x4f32(x[i], y[i], c, 0, 0, 0);
    return c;
  }
}

template <bool F32>
__device__ __forceinline__ float load_scale(const void* a, size_t i) {
  if constexpr (F32) return static_cast<const float*>(a)[i];
  else return bf16_val(static_cast<const uint16_t*>(a)[i]);
}

// T: the type of d_out as stored (uint16_t: bf16).  WM: waves along the tokens, 4 / WM along the columns.
template <class T, int BM, int WM, bool AFF, bool SF>
__global__ __launch_bounds__(kThreads) void linear_back_kernel(LinearBackParams p, int splits) {
  constexpr int kVec = 16 / sizeof(T), kStep = kChunks * kVec, kWords = kStep / 16;
  constexpr int MT = BM / WM / 16, KT = kCols / (4 / WM) / 16;     // 16 x 16 tiles of a wave
  constexpr int kRows = BM / 32 ? BM / 32 : 1;                     // token chunks of a thread
  __shared__ v4u s_d[2][BM * kChunks], s_w[2][kCols * kChunks];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave % WM, wk = wave / WM;
  const int k0 = (int)blockIdx.x * kCols, m0 = (int)blockIdx.y * BM;
  const int steps = (p.N + kStep - 1) / kStep;
  const int begin = (int)((int64_t)steps * blockIdx.z / splits), end = (int)((int64_t)steps * (blockIdx.z + 1) / splits);

  // a thread's place among the weights: words of rows nq * kWords .. at the eight columns kb
  const int kb = (tid >> 1) & 15, nq = (tid & 1) + 2 * (tid >> 5);
  const bool col_in = k0 + 8 * kb < p.K;
  const size_t pitch = (size_t)p.K / 8;                            // words of a row
  const uint32_t* const w_at = reinterpret_cast<const uint32_t*>(p.w) + (k0 / 8 + (col_in ? kb : 0));
  const int group = (k0 + (col_in ? 8 * kb : 0)) / p.group;

  const RowMatrix<T> d_out(p.d_out, p.M, p.N);

  struct Fetched {
    v4u d[kRows];
    uint32_t w[kWords];
    float s[kWords], b[kWords];
  };
  auto fetch = [&](int step, Fetched& f) {
    const int n0 = step * kStep;
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const int row = tid / kChunks + 32 * i, m = min(m0 + row, p.M - 1);      // rows past the last one repeat it
      if (BM >= 32 || row < BM)
        f.d[i] = d_out.chunk(m, n0 + (tid % kChunks) * kVec);
    }
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
      const int n = n0 + nq * kWords + i;
      const bool in = n < p.N;
      const size_t row = (size_t)(in ? n : p.N - 1);
      f.w[i] = w_at[row * pitch];
      f.s[i] = load_scale<SF>(p.scales, row * p.groups + group);
      f.b[i] = AFF ? load_scale<SF>(p.biases, row * p.groups + group) : -8.0f * f.s[i];
      f.s[i] = in ? f.s[i] : 0.0f;
      f.b[i] = in ? f.b[i] : 0.0f;
    }
  };
  auto stage = [&](int buf, const Fetched& f) {
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const int row = tid / kChunks + 32 * i;
      if (BM >= 32 || row < BM) s_d[buf][place(row, tid % kChunks)] = f.d[i];
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      // (q - 8) s, or q s + b, rounded once (to F32, and for bf16 once more: as a
      // bf16 matrix of these weights would hold them)
      float v[kWords];
#pragma unroll
      for (int i = 0; i < kWords; ++i)
        v[i] = __builtin_fmaf((float)((f.w[i] >> (4 * j)) & 15u), f.s[i], f.b[i]);
      v2u r;
      if constexpr (sizeof(T) == 2) {
        const v2f lo = {v[0], v[1]}, hi = {v[2 % kWords], v[3 % kWords]};
        r.x = __builtin_bit_cast(uint32_t, __builtin_convertvector(lo, v2bf));
        r.y = __builtin_bit_cast(uint32_t, __builtin_convertvector(hi, v2bf));
      } else {
        r.x = __float_as_uint(v[0]);
        r.y = __float_as_uint(v[1]);
      }
      const int row = 8 * kb + j;
      reinterpret_cast<v2u*>(&s_w[buf][place(row, nq >> 1)])[nq & 1] = r;
    }
  };

  v4f acc[KT][MT] = {};
  Fetched next;
  if (begin < end) fetch(begin, next);
  for (int step = begin; step < end; ++step) {
    const int buf = (step - begin) & 1;
    stage(buf, next);
    __syncthreads();
    if (step + 1 < end) fetch(step + 1, next);
#pragma unroll
    for (int h = 0; h < kChunks / 4; ++h) {
      v4u a[KT], b[MT];
      const int c = 4 * h + (lane >> 4);
#pragma unroll
      for (int t = 0; t < KT; ++t) a[t] = s_w[buf][place(wk * (16 * KT) + 16 * t + (lane & 15), c)];
#pragma unroll
      for (int t = 0; t < MT; ++t) b[t] = s_d[buf][place(wm * (16 * MT) + 16 * t + (lane & 15), c)];
#pragma unroll
      for (int t = 0; t < KT; ++t)
#pragma unroll
        for (int u = 0; u < MT; ++u) acc[t][u] = multiply<T>(a[t], b[u], acc[t][u]);
    }
    // one barrier a step: a wave writes buffer 1 - buf only after every wave has passed this
    // step's barrier, and so has read it in the step before
  }
#pragma unroll
  for (int u = 0; u < MT; ++u) {
    const int m = m0 + wm * (16 * MT) + 16 * u + (lane & 15);
#pragma unroll
    for (int t = 0; t < KT; ++t) {
      const int k = k0 + wk * (16 * KT) + 16 * t + 4 * (lane >> 4);
      if (m >= p.M || k >= p.K) continue;
      const v4f v = acc[t][u];
      if (splits > 1) {
        *reinterpret_cast<v4f*>(p.partials + ((size_t)blockIdx.z * p.M + m) * p.K + k) = v;
      } else if constexpr (sizeof(T) == 2) {
        const v2f lo = {v[0], v[1]}, hi = {v[2], v[3]};
        const v2u r = {__builtin_bit_cast(uint32_t, __builtin_convertvector(lo, v2bf)),
                       __builtin_bit_cast(uint32_t, __builtin_convertvector(hi, v2bf))};
        *reinterpret_cast<v2u*>(static_cast<uint16_t*>(p.d_x) + (size_t)m * p.K + k) = r;
      } else {
        *reinterpret_cast<v4f*>(static_cast<float*>(p.d_x) + (size_t)m * p.K + k) = v;
      }
    }
  }
}

// Adds up the parts of n, in order.
template <class T>
__global__ __launch_bounds__(kThreads) void linear_back_join_kernel(LinearBackParams p, int splits) {
  const size_t all = (size_t)p.M * p.K / 4;
  const size_t i = (size_t)blockIdx.x * kThreads + threadIdx.x;
  if (i >= all) return;
  const v4f* const at = reinterpret_cast<const v4f*>(p.partials) + i;
  v4f v = at[0];
  for (int z = 1; z < splits; ++z) v += at[(size_t)z * all];
  if constexpr (sizeof(T) == 2) {
    const v2f lo = {v[0], v[1]}, hi = {v[2], v[3]};
    const v2u r = {__builtin_bit_cast(uint32_t, __builtin_convertvector(lo, v2bf)),
                   __builtin_bit_cast(uint32_t, __builtin_convertvector(hi, v2bf))};
    reinterpret_cast<v2u*>(p.d_x)[i] = r;
  } else {
    reinterpret_cast<v4f*>(p.d_x)[i] = v;
  }
}

int tile_rows(int M) { return M <= 16 ? 16 : M <= 32 ? 32 : M <= 64 ? 64 : 128; }

template <class T, int BM, int WM>
const void* pick(const LinearBackParams& p) {
  if (p.biases)
    return p.scale_f32 ? reinterpret_cast<const void*>(&linear_back_kernel<T, BM, WM, true, true>)
                       : reinterpret_cast<const void*>(&linear_back_kernel<T, BM, WM, true, false>);
  return p.scale_f32 ? reinterpret_cast<const void*>(&linear_back_kernel<T, BM, WM, false, true>)
                     : reinterpret_cast<const void*>(&linear_back_kernel<T, BM, WM, false, false>);
}

template <class T>
hipError_t run(const LinearBackParams& p, hipStream_t stream) {
  const int bm = tile_rows(p.M);
  const void* kernel = bm == 16   ? pick<T, 16, 1>(p)
                       : bm == 32 ? pick<T, 32, 1>(p)
                       : bm == 64 ? pick<T, 64, 2>(p)
                                  : pick<T, 128, 2>(p);
  const int tiles_k = (p.K + kCols - 1) / kCols, tiles_m = (p.M + bm - 1) / bm;
  const int steps = (p.N * (int)sizeof(T) + 127) / 128;
  int splits = kFill / (tiles_k * tiles_m);
  splits = splits > kMaxSplits ? kMaxSplits : splits;
  splits = splits > steps ? steps : splits;
  splits = splits < 1 ? 1 : splits;
  LinearBackParams q = p;
  void* args[] = {&q, &splits};
  const hipError_t e = hipLaunchKernel(kernel, dim3((unsigned)tiles_k, (unsigned)tiles_m, (unsigned)splits),
                                       dim3(kThreads), args, 0, stream);
  if (e != hipSuccess || splits == 1) return e;
  const size_t all = (size_t)p.M * p.K / 4;
  return hipLaunchKernel(reinterpret_cast<const void*>(&linear_back_join_kernel<T>),
                         dim3((unsigned)((all + kThreads - 1) / kThreads)), dim3(kThreads), args, 0, stream);
}

}  // namespace

// Room for the parts of n: there are at most kMaxSplits, and more than one only
// while all work-groups together are no more than kFill.
size_t linear_back_partial_bytes(int64_t M, int64_t K) {
  const size_t parts = (size_t)M * (size_t)K * 4 * kMaxSplits, most = (size_t)kFill * 128 * kCols * 4;
  return ((parts < most ? parts : most) + 255) / 256 * 256;
}

hipError_t launch_linear_backward(const LinearBackParams& p, hipStream_t stream) {
  return p.xf32 ? run<float>(p, stream) : run<uint16_t>(p, stream);
}

}  // namespace q4
