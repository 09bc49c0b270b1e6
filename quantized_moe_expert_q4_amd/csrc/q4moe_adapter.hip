// Low-rank adapters of many requests: each row has an adapter (A [R][K],
// B [N][R]) of its own, or none.
//   forward   h = A x, out = base + s B h
//   backward  g = s B^T d, d_x = base + A^T g, d_A = sum_t g x^T, d_B = s sum_t d h^T
//
// A work-group takes 16 rows of one adapter, gathered from a window of 256 rows
// (group_rows), so that rows of one adapter need not stand together.  Two kernels
// serve both directions: "shrink" takes the long rows to R sums, "expand" takes
// R values to long rows; the adapter's matrix runs along the sum or across it
// (ACROSS).
#include "q4moe_adapter.h"

namespace q4 {

namespace {

constexpr int kThreads = 256;
constexpr int kWindow = 256;         // rows whose adapters a work-group looks at
constexpr int kTile = 16;            // rows of a work-group
constexpr int kSlice = 256;          // columns of an expanding work-group
constexpr int kMaxSplits = 16;       // parts of a long sum
constexpr int kFill = 512;           // work-groups that fill the device: no more parts than give so many

// A chunk's values as floats.
template <class T>
__device__ __forceinline__ void values(const v4u chunk, float (&v)[16 / sizeof(T)]) {
#pragma unroll
  for (int i = 0; i < (int)(16 / sizeof(T)); ++i) {
    if constexpr (sizeof(T) == 2) v[i] = __uint_as_float(i & 1 ? chunk[i / 2] & 0xFFFF0000u : chunk[i / 2] << 16);
    else v[i] = __uint_as_float(chunk[i]);
  }
}

// The rows of one work-group: `count` of them, all of `adapter` (-1: none).
struct Rows {
  int row[kTile];
  int adapter, count;
};

// Tile `index` of the window's rows: the rows of each adapter, in their order,
// in tiles of 16, adapters by their first row.  False where there is none.
__device__ __forceinline__ bool group_rows(const int32_t* ids, int M, int n, int window, int index, Rows& out) {
  __shared__ int s_id[kWindow], s_first[kWindow], s_total[kThreads / 64];
  const int t = threadIdx.x, row = window * kWindow + t, lane = t & 63, wave = t >> 6;
  const int rows = min(kWindow, M - window * kWindow);
  const int id = t < rows ? adapter_of(ids, row, n) : -2;
  s_id[t] = id;
  if (t == 0) out.count = 0;
  __syncthreads();
  int before = 0, same = 0, first = t;
  for (int j = 0; j < rows; ++j) {
    const bool eq = s_id[j] == id;
    same += eq;
    before += eq && j < t;
    first = eq && j < first ? j : first;
  }
  // tiles of the adapters whose first row comes earlier
  const int tiles = t < rows && before == 0 ? (same + kTile - 1) / kTile : 0;
  int sum = tiles;
  for (int d = 1; d < 64; d <<= 1) {
    const int other = __shfl_up(sum, d);
    sum += lane >= d ? other : 0;
  }
  if (lane == 63) s_total[wave] = sum;
  __syncthreads();
  int start = sum - tiles;
  for (int w = 0; w < wave; ++w) start += s_total[w];
  s_first[t] = start;
  __syncthreads();
  if (t < rows && s_first[first] + before / kTile == index) {
    out.row[before % kTile] = row;
    if (before % kTile == 0) {
      out.adapter = id;
      out.count = min(kTile, same - before);
    }
  }
  __syncthreads();
  return out.count > 0;
}

// Tiles that a window of M rows can have.
int window_tiles(int M, int n, bool ids) {
  const int rows = M < kWindow ? M : kWindow;
  const int kinds = !ids ? 1 : n + 1 < rows ? n + 1 : rows;
  return (rows + 15 * kinds) / 16;
}

struct ShrinkParams {
  const void* x;          // [M][C]
  const void* w;          // per adapter [R][C], ACROSS: [C][R]
  const int32_t* ids;
  float* partial;         // [splits][M][R]
  int M, C, R, n, splits;
};

// partial[split][row][r] = the split's part of sum_c w[r][c] x[row][c].
template <class T, int NR, bool ACROSS>
__global__ __launch_bounds__(kThreads) void shrink_kernel(ShrinkParams p) {
  constexpr int kVec = 16 / sizeof(T), kStep = 4 * kVec;
  __shared__ Rows s_rows;
  __shared__ float s_sum[4][NR][64][4];
  if (!group_rows(p.ids, p.M, p.n, (int)blockIdx.y, (int)blockIdx.x, s_rows)) return;
  const int adapter = s_rows.adapter, count = s_rows.count;
  const int lane = threadIdx.x & 63, l = lane & 15, g = lane >> 4, wave = threadIdx.x >> 6;
  v4f acc[NR] = {};
  if (adapter >= 0) {
    const T* const w = static_cast<const T*>(p.w) + (size_t)adapter * p.R * p.C;
    const RowMatrix<T> along(w, p.R, p.C);
    const RowMatrix<T> x(p.x, p.M, p.C);
    const int row = s_rows.row[min(l, count - 1)];
    const int steps = (p.C + kStep - 1) / kStep;
    const int begin = steps * (int)blockIdx.z / p.splits, end = steps * ((int)blockIdx.z + 1) / p.splits;
    for (int step = begin + wave; step < end; step += 4) {
      const int c = step * kStep + kVec * g;
      float xv[kVec];
      values<T>(x.chunk(row, c), xv);
#pragma unroll
      for (int j = 0; j < NR; ++j) {
        const int r = 16 * j + l;
        float wv[kVec] = {};
        if (r < p.R) {
          if constexpr (ACROSS) {
#pragma unroll
            for (int i = 0; i < kVec; ++i) wv[i] = c + i < p.C ? value<T>(w[(size_t)(c + i) * p.R + r]) : 0.0f;
          } else {
            values<T>(along.chunk(r, c), wv);
          }
        }
#pragma unroll
        for (int i = 0; i < kVec; ++i) acc[j] = __builtin_amdgcn_mfma_f32_16x16x4f32(wv[i], xv[i], acc[j], 0, 0, 0);
      }
    }
  }
#pragma unroll
  for (int j = 0; j < NR; ++j) *reinterpret_cast<v4f*>(s_sum[wave][j][lane]) = acc[j];
  __syncthreads();
  // lane 16 g + l of a tile: row l, r = 4 g ..
  for (int i = threadIdx.x; i < NR * 64; i += kThreads) {
    const int j = i >> 6, at = i & 63, row = at & 15, r = 16 * j + 4 * (at >> 4);
    v4f v = *reinterpret_cast<v4f*>(s_sum[0][j][at]);
    for (int k = 1; k < 4; ++k) v += *reinterpret_cast<v4f*>(s_sum[k][j][at]);
    if (row < count && r < p.R)
      *reinterpret_cast<v4f*>(p.partial + ((size_t)blockIdx.z * p.M + s_rows.row[row]) * p.R + r) = v;
  }
}

struct ExpandParams {
  const float* partial;   // [splits][M][R]
  const void* w;          // per adapter [O][R], ACROSS: [R][O]
  const int32_t* ids;
  const float* scales;    // per adapter, or nullptr (1)
  const void* base;       // [M][O] or nullptr
  void* out;              // [M][O]
  float* hidden;          // [M][R] or nullptr: the sum of the parts (ACROSS: scaled)
  int M, O, R, n, splits;
};

// out[row] = base[row] + scale * sum_r w[.][r] * (sum of the row's parts)[r].
template <class T, int NR, bool ACROSS>
__global__ __launch_bounds__(kThreads) void expand_kernel(ExpandParams p) {
  constexpr int kVec = 16 / sizeof(T), kStep = 4 * kVec, kPitch = 16 * NR + (NR * 16 < kStep ? kStep - 16 * NR : 0) + 1;
  __shared__ Rows s_rows;
  __shared__ float s_h[kTile][kPitch];
  if (!group_rows(p.ids, p.M, p.n, (int)blockIdx.z, (int)blockIdx.y, s_rows)) return;
  const int adapter = s_rows.adapter, count = s_rows.count;
  const float scale = adapter >= 0 && p.scales ? p.scales[adapter] : 1.0f;
  for (int i = threadIdx.x; i < kTile * kPitch; i += kThreads) {
    const int row = i / kPitch, r = i % kPitch;
    float h = 0.0f;
    if (row < count && r < p.R) {
      const size_t at = (size_t)s_rows.row[row] * p.R + r;
      for (int k = 0; k < p.splits; ++k) h += p.partial[(size_t)k * p.M * p.R + at];
      if (!ACROSS && p.hidden && blockIdx.x == 0) p.hidden[at] = h;
      h *= scale;
      if (ACROSS && p.hidden && blockIdx.x == 0) p.hidden[at] = h;
    }
    s_h[row][r] = h;
  }
  if (!p.out) return;
  __syncthreads();
  const int lane = threadIdx.x & 63, l = lane & 15, g = lane >> 4, wave = threadIdx.x >> 6;
  const T* const w = static_cast<const T*>(p.w) + (size_t)max(adapter, 0) * p.R * p.O;
  for (int tile = 0; tile < kSlice / 64; ++tile) {
    const int o0 = (int)blockIdx.x * kSlice + 64 * wave + 16 * tile;
    if (o0 >= p.O) break;
    v4f acc = {0.0f, 0.0f, 0.0f, 0.0f};
    if (adapter >= 0) {
      const int o = min(o0 + l, p.O - 1);
      for (int r0 = 0; r0 < p.R; r0 += kStep) {
        const int r = r0 + kVec * g;
        float wv[kVec] = {};
        if constexpr (ACROSS) {
#pragma unroll
          for (int i = 0; i < kVec; ++i) wv[i] = r + i < p.R ? value<T>(w[(size_t)(r + i) * p.O + o]) : 0.0f;
        } else {
          values<T>(RowMatrix<T>(w, p.O, p.R).chunk(o, r), wv);
        }
#pragma unroll
        for (int i = 0; i < kVec; ++i)
          acc = __builtin_amdgcn_mfma_f32_16x16x4f32(wv[i], s_h[l][min(r + i, kPitch - 1)], acc, 0, 0, 0);
      }
    }
    if (l < count) {
      const size_t at = (size_t)s_rows.row[l] * p.O;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int o = o0 + 4 * g + i;
        if (o >= p.O) break;
        const float b = p.base ? value<T>(static_cast<const T*>(p.base)[at + o]) : 0.0f;
        static_cast<T*>(p.out)[at + o] = rounded<T>(b + acc[i]);
      }
    }
  }
}

// Kernels by type, tiles of 16 ranks and direction.
#define Q4_ADAPTER_RANKS(k, T, ACROSS)                                                                       \
  {reinterpret_cast<const void*>(&k<T, 1, ACROSS>), reinterpret_cast<const void*>(&k<T, 2, ACROSS>),         \
   reinterpret_cast<const void*>(&k<T, 4, ACROSS>), reinterpret_cast<const void*>(&k<T, 8, ACROSS>),         \
   reinterpret_cast<const void*>(&k<T, 16, ACROSS>)}
#define Q4_ADAPTER_KERNELS(k)                                                                                \
  {{Q4_ADAPTER_RANKS(k, uint16_t, false), Q4_ADAPTER_RANKS(k, uint16_t, true)},                              \
   {Q4_ADAPTER_RANKS(k, float, false), Q4_ADAPTER_RANKS(k, float, true)}}

int rank_index(int R) { return R <= 16 ? 0 : R <= 32 ? 1 : R <= 64 ? 2 : R <= 128 ? 3 : 4; }

// Parts of a sum over C: as many as fill the device.
int sum_splits(int M, int C) {
  const int tiles = (M + kTile - 1) / kTile, steps = (C + 255) / 256;
  int s = kFill / tiles;
  s = s > kMaxSplits ? kMaxSplits : s;
  s = s > steps ? steps : s;
  return s < 1 ? 1 : s;
}

template <class P>
hipError_t launch(const void* kernel, P p, dim3 grid, hipStream_t stream) {
  void* args[] = {&p};
  return hipLaunchKernel(kernel, grid, dim3(kThreads), args, 0, stream);
}

hipError_t shrink(ShrinkParams p, bool f32, bool across, hipStream_t stream) {
  static const void* const kernels[2][2][5] = Q4_ADAPTER_KERNELS(shrink_kernel);
  const dim3 grid((unsigned)window_tiles(p.M, p.n, p.ids != nullptr), (unsigned)((p.M + kWindow - 1) / kWindow),
                  (unsigned)p.splits);
  return launch(kernels[f32][across][rank_index(p.R)], p, grid, stream);
}

hipError_t expand(ExpandParams p, bool f32, bool across, hipStream_t stream) {
  static const void* const kernels[2][2][5] = Q4_ADAPTER_KERNELS(expand_kernel);
  const dim3 grid((unsigned)((p.O + kSlice - 1) / kSlice), (unsigned)window_tiles(p.M, p.n, p.ids != nullptr),
                  (unsigned)((p.M + kWindow - 1) / kWindow));
  return launch(kernels[f32][across][rank_index(p.R)], p, grid, stream);
}

}  // namespace

// The parts of the hidden sums: M rows, or while there are several parts at
// most kFill tiles in all.
size_t hidden_bytes(int64_t M, int64_t R) {
  const int64_t several = M * kMaxSplits < kFill * kTile ? M * kMaxSplits : kFill * kTile;
  const size_t rows = (size_t)(M > several ? M : several);
  return (rows * (size_t)R * 4 + 255) / 256 * 256;
}

size_t adapter_workspace(int64_t M, int64_t N, int64_t K, int64_t R, int64_t n) {
  return hidden_bytes(M, R) + (size_t)M * R * 4 / 256 * 256 + 256 + adapter_grad_workspace(M, N, K, R, n);
}

hipError_t launch_adapter(const AdapterParams& p, hipStream_t stream) {
  const int splits = sum_splits(p.M, p.K);
  const hipError_t e = shrink({p.x, p.a, p.ids, p.partial, p.M, p.K, p.R, p.n, splits}, p.xf32, false, stream);
  if (e != hipSuccess) return e;
  return expand({p.partial, p.b, p.ids, p.scales, p.base, p.out, p.hidden, p.M, p.N, p.R, p.n, splits}, p.xf32, false,
                stream);
}

hipError_t launch_adapter_backward(const AdapterBackwardParams& p, hipStream_t stream) {
  const int splits = sum_splits(p.M, p.N);
  float* const g = p.partial + hidden_bytes(p.M, p.R) / 4;
  float* const rest = g + (size_t)p.M * p.R / 64 * 64 + 64;
  hipError_t e = hipSuccess;
  if (p.d_x || p.d_a) {
    e = shrink({p.d_out, p.b, p.ids, p.partial, p.M, p.N, p.R, p.n, splits}, p.xf32, true, stream);
    if (e == hipSuccess)
      e = expand({p.partial, p.a, p.ids, p.scales, p.base, p.d_x, g, p.M, p.K, p.R, p.n, splits}, p.xf32, true, stream);
  }
  if (e != hipSuccess || (!p.d_a && !p.d_b)) return e;
  AdapterGradParams q{};
  q.x = p.x;
  q.d_out = p.d_out;
  q.g = g;
  q.hidden = p.hidden;
  q.ids = p.ids;
  q.scales = p.scales;
  q.d_a = p.d_a;
  q.d_b = p.d_b;
  q.order = reinterpret_cast<int32_t*>(rest);
  q.offsets = q.order + ((size_t)p.M + 63) / 64 * 64;
  q.parts = reinterpret_cast<float*>(q.offsets + ((size_t)p.n + 64) / 64 * 64);
  q.M = p.M;
  q.N = p.N;
  q.K = p.K;
  q.R = p.R;
  q.n = p.n;
  q.xf32 = p.xf32;
  return launch_adapter_grad(q, stream);
}

}  // namespace q4
