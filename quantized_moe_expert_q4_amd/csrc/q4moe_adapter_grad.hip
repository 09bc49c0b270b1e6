// Gradients of the adapters' matrices,
//   d_a[r][k] = sum_t g[t][r] x[t][k],   d_b[n][r] = s sum_t d_out[t][n] hidden[t][r],
// over the rows t of each adapter.
//
// The rows are sorted by adapter first (order_rows, beside the call's first
// product where it has one) and cut into chunks of `rows`.  A work-group takes a slice
// of the long dimension and a chunk: its eight waves each take 32 rows at a time,
// read 16 bytes of each (whole runs of 256 bytes), turn them in registers into
// matrix operands along the rows, and multiply them with the short vectors, which
// enter as three bf16 parts, so that nothing of their 24 bits is lost.  An
// adapter whose rows end within one chunk is written at once, the others' parts
// are joined in order by a second launch, which also writes the zeros of the
// adapters without rows.
//
// Both gradients of 8192 rows of 4096 + 4096 columns, rank 16, in 26 us (134 MB,
// 5.2 TB/s) and 5 to join; 4096 rows of 7168 + 1536, rank 64, four adapters, in 42 + 5,
// where each value of a row goes into twelve matrix operations and the rows pass
// two waves.  The first is at the rate of a large copy (5.1 TB/s); the second reads
// 71 MB, 1.7 TB/s.
#include "q4moe_adapter.h"

namespace q4 {

namespace {

constexpr int kWaves = 8;
constexpr int kThreads = 64 * kWaves;
constexpr int kRanks = 32;           // ranks of a wave at most: more sums would not fit its registers
constexpr int kTogether = 4;         // tiles of sums that the waves join at a time
constexpr int kFill = 256;           // work-groups that the device runs at a time: no more chunks than give so many
constexpr int kLeastRows = 256;      // rows that a chunk has at least: 32 of each wave

// Columns of a work-group's slice.
template <class T>
constexpr int kColumns = 256 / (int)sizeof(T);

// The sorting alone, for a call that has no product of rows to do beside it.
__global__ __launch_bounds__(kThreads) void order_kernel(const int32_t* ids, int M, int n, int32_t* order,
                                                         int32_t* offsets) {
  order_rows(ids, M, n, (int)blockIdx.x, order, offsets);
}

// One of the two gradients: y's columns against h's ranks.
struct Grad {
  const void* y;          // [M][O]
  const float* h;         // [M][R]
  float* out;             // per adapter [O][R], or [R][O] for d_a
  float* parts;           // [2 chunks][O][R] or [R][O]: of the adapter that began before the chunk, of one that goes on
  const float* scales;    // or nullptr
  int O, slices, rows, chunks;
};

struct GradLaunch {
  Grad a, b;
  const int32_t* ids;
  const int32_t* order;
  const int32_t* offsets;
  int M, R, n;
  int shift;              // 1 << shift waves share the ranks, the others the rows
};

// The 32 rows from `at` on as a lane takes them: of bf16 the eight rows of its
// lane group (a matrix operation takes 32 rows), of float one of each four (it
// takes 4).
template <class T>
__device__ __forceinline__ int row_of(int lane_group, int i) {
  return sizeof(T) == 2 ? 8 * lane_group + i : 4 * i + lane_group;
}

// NR: tiles of 16 ranks of a wave.
template <class T, int NR, bool IS_A>
__device__ __forceinline__ void grad_slice(const GradLaunch& p, const Grad& q, int slice, int chunk,
                                           v4f (*s_sum)[kWaves][NR][64]) {
  constexpr int kVec = 16 / sizeof(T);           // columns of a lane, one in each of as many tiles of 16
  const int lane = threadIdx.x & 63, l = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int rank_waves = 1 << p.shift, rank0 = 16 * NR * (wave & (rank_waves - 1));
  const int step = 32 * (kWaves >> p.shift);     // rows of the work-group at a time
  const int o0 = slice * kColumns<T>, col = o0 + kVec * l;
  const int total = p.ids ? p.offsets[p.n] : p.M;
  const int chunk_begin = chunk * q.rows, chunk_end = min(total, chunk_begin + q.rows);
  const ColumnRuns<T> y(q.y, p.M, q.O);
  const bool ragged = o0 + kColumns<T> > q.O;    // the slice with the rows' ends
  int begin = chunk_begin;
  while (begin < chunk_end) {                    // the adapters of the chunk
    const int adapter = p.ids ? p.ids[p.order[begin]] : 0;
    const int whole_end = p.ids ? p.offsets[adapter + 1] : p.M, end = min(chunk_end, whole_end);
    const bool before = begin == chunk_begin && (p.ids ? p.offsets[adapter] : 0) < chunk_begin;
    const bool several = before || whole_end > end;
    v4f acc[kVec][NR] = {};
    // The next rows are fetched as soon as the registers of these are free: y
    // once it is turned, h rank tile by rank tile.  Loads are unconditional: past
    // the adapter's rows the last one is repeated, with h = 0; past the columns
    // and ranks other values come along, whose results are not stored.
    v4u rows[8];
    float h[NR][8];
    int t[8], next_t[8];             // the rows' numbers are known a step earlier
    auto fetch_numbers = [&](int at, int (&t)[8]) {
      if (!p.ids) {
#pragma unroll
        for (int i = 0; i < 8; ++i) t[i] = min(at + row_of<T>(g, i), end - 1);
      } else if (sizeof(T) == 2 && at + 32 <= end) {
        __builtin_memcpy(t, p.order + at + 8 * g, 32);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) t[i] = p.order[min(at + row_of<T>(g, i), end - 1)];
      }
    };
    auto fetch_rows = [&]() {
#pragma unroll
      for (int i = 0; i < 8; ++i) rows[i] = y.load(t[i], col);
      if (ragged) {
#pragma unroll
        for (int i = 0; i < 8; ++i) rows[i] = y.aligned(rows[i], t[i], col);
      }
    };
    auto fetch_ranks = [&](int at, int j) {
      const int r = min(rank0 + 16 * j + l, p.R - 1);
#pragma unroll
      for (int i = 0; i < 8; ++i) h[j][i] = q.h[(size_t)t[i] * p.R + r];
      if (at + 32 > end) {
#pragma unroll
        for (int i = 0; i < 8; ++i) h[j][i] = at + row_of<T>(g, i) < end ? h[j][i] : 0.0f;
      }
    };
    int at = rank0 < p.R ? begin + 32 * (wave >> p.shift) : end;
    if (at < end) {
      fetch_numbers(at, t);
      fetch_numbers(at + step, next_t);
      fetch_rows();
#pragma unroll
      for (int j = 0; j < NR; ++j) fetch_ranks(at, j);
    }
    while (at < end) {
      const int next = at + step;
      v4u column[8];
      if constexpr (sizeof(T) == 2) {
        turn(rows, column);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) column[i] = rows[i];
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) t[i] = next_t[i];
      if (next < end) {
        fetch_rows();
        fetch_numbers(next + step, next_t);
      }
#pragma unroll
      for (int j = 0; j < NR; ++j) {
        if constexpr (sizeof(T) == 2) {
          v4u part[3];
          split<3>(h[j], part);
          if (next < end) fetch_ranks(next, j);
#pragma unroll
          for (int d = 0; d < 3; ++d)
#pragma unroll
            for (int c = 0; c < kVec; ++c)
              acc[c][j] = IS_A ? multiply_bf16(column[c], part[d], acc[c][j]) : multiply_bf16(part[d], column[c], acc[c][j]);
        } else {
          float now[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) now[i] = h[j][i];
          if (next < end) fetch_ranks(next, j);
#pragma unroll
          for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int c = 0; c < kVec; ++c) {
              const float v = __uint_as_float(column[i][c]);
              acc[c][j] = IS_A ? __builtin_amdgcn_mfma_f32_16x16x4f32(v, now[i], acc[c][j], 0, 0, 0)
                               : __builtin_amdgcn_mfma_f32_16x16x4f32(now[i], v, acc[c][j], 0, 0, 0);
            }
        }
      }
      at = next;
    }
    // the waves' sums
    const float scale = q.scales ? q.scales[adapter] : 1.0f;
    float* const out = several ? q.parts + (size_t)(2 * chunk + (begin == chunk_begin ? 0 : 1)) * q.O * p.R
                               : q.out + (size_t)adapter * q.O * p.R;
#pragma unroll
    for (int c0 = 0; c0 < kVec; c0 += kTogether) {
      __syncthreads();
#pragma unroll
      for (int c = 0; c < kTogether; ++c)
#pragma unroll
        for (int j = 0; j < NR; ++j) s_sum[c][wave][j][lane] = acc[c0 + c][j];
      __syncthreads();
      for (int i = threadIdx.x; i < (kTogether * NR * 64) << p.shift; i += kThreads) {
        const int c = i / 64 % kTogether, tile = i / (64 * kTogether), j = tile % NR, first = tile / NR;
        const int from = i & 63, fl = from & 15, fg = from >> 4;
        v4f v = s_sum[c][first][j][from];
        for (int w = first + rank_waves; w < kWaves; w += rank_waves) v += s_sum[c][w][j][from];
        v *= scale;
        if constexpr (IS_A) {
          const int r = 16 * tile + fl;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int o = o0 + kVec * (4 * fg + e) + c0 + c;
            if (r < p.R && o < q.O) out[(size_t)r * q.O + o] = v[e];
          }
        } else {
          const int r = 16 * tile + 4 * fg, o = o0 + kVec * fl + c0 + c;
          if (r < p.R && o < q.O) *reinterpret_cast<v4f*>(out + (size_t)o * p.R + r) = v;
        }
      }
    }
    begin = end;
  }
}

template <class T, int NR>
__global__ __launch_bounds__(kThreads, 2) void grad_kernel(GradLaunch p) {
  __shared__ v4f s_sum[kTogether][kWaves][NR][64];
  int i = (int)blockIdx.x;
  if (i < p.a.slices * p.a.chunks) {
    grad_slice<T, NR, true>(p, p.a, i % p.a.slices, i / p.a.slices, s_sum);
  } else {
    i -= p.a.slices * p.a.chunks;
    grad_slice<T, NR, false>(p, p.b, i % p.b.slices, i / p.b.slices, s_sum);
  }
}

// The adapters that the chunks left: those of several chunks, and those without rows.
__global__ __launch_bounds__(256) void join_kernel(GradLaunch p, int blocks_a) {
  const bool is_a = (int)blockIdx.x < blocks_a;
  const Grad& q = is_a ? p.a : p.b;
  const size_t all = (size_t)q.O * p.R / 4;
  const size_t i = (size_t)((int)blockIdx.x - (is_a ? 0 : blocks_a)) * 256 + threadIdx.x;
  const int adapter = (int)blockIdx.y;
  const int begin = p.ids ? p.offsets[adapter] : adapter ? p.M : 0, end = p.ids ? p.offsets[adapter + 1] : p.M;
  const int first = begin / q.rows, last = (end - 1) / q.rows;
  if ((begin < end && first == last) || i >= all) return;
  v4f sum = {0.0f, 0.0f, 0.0f, 0.0f};
  if (begin < end) {
#pragma unroll 4
    for (int c = first; c <= last; ++c) {
      const int slot = 2 * c + (c == first && begin != c * q.rows ? 1 : 0);
      sum += reinterpret_cast<const v4f*>(q.parts)[(size_t)slot * all + i];
    }
  }
  reinterpret_cast<v4f*>(q.out)[(size_t)adapter * all + i] = sum;
}

// 8192 rows of 4096 + 4096 columns, rank 16, in 2, 4, 8 and 16 chunks (128 to
// 1024 work-groups): the backward call takes 110, 99, 107 and 117 us.
int chunk_count(int M, int slices) {
  const int most = (M + kLeastRows - 1) / kLeastRows, c = kFill / slices;
  return c < 1 ? 1 : c < most ? c : most;
}

Grad grad_of(const AdapterGradParams& p, const void* y, const float* h, float* out, const float* scales, int O, int slices,
             float* parts) {
  const int columns = p.xf32 ? kColumns<float> : kColumns<uint16_t>;
  Grad q{y, h, out, parts, scales, O, out ? (O + columns - 1) / columns : 0, 0, 0};
  const int chunks = chunk_count(p.M, slices);
  q.rows = ((p.M + chunks - 1) / chunks + 31) / 32 * 32;
  q.chunks = (p.M + q.rows - 1) / q.rows;
  return q;
}

// Bytes of a gradient's parts, two for each chunk where there are several: the
// chunks times O are at most the smaller of ceil(M / kLeastRows) * O and kFill *
// columns (an only chunk has no parts).
size_t part_bytes(int64_t M, int64_t O, int64_t R) {
  if (M <= kLeastRows) return 0;
  const int64_t by_rows = (M + kLeastRows - 1) / kLeastRows * O, by_fill = kFill * kColumns<uint16_t>;
  return (size_t)(by_rows < by_fill ? by_rows : by_fill) * (size_t)R * 8;
}

size_t up(size_t bytes) { return (bytes + 255) / 256 * 256; }

template <class T>
const void* pick(int R) {
  return R <= 16 ? reinterpret_cast<const void*>(&grad_kernel<T, 1>) : reinterpret_cast<const void*>(&grad_kernel<T, 2>);
}

}  // namespace

// In this order: sorted rows, where the adapters begin, the parts of d_b and of d_a.
size_t adapter_grad_workspace(int64_t M, int64_t N, int64_t K, int64_t R, int64_t n) {
  return up((size_t)M * 4) + up((size_t)(n + 1) * 4) + up(part_bytes(M, N, R)) + up(part_bytes(M, K, R));
}

hipError_t launch_adapter_grad(const AdapterGradParams& p, hipStream_t stream) {
  hipError_t e = hipSuccess;
  if (p.ids && !p.sorted) {
    const int32_t* ids = p.ids;
    int M = p.M, n = p.n;
    int32_t *order = p.order, *offsets = p.offsets;
    void* args[] = {&ids, &M, &n, &order, &offsets};
    e = hipLaunchKernel(reinterpret_cast<const void*>(&order_kernel), dim3((unsigned)n),
                        dim3(kThreads), args, 0, stream);
    if (e != hipSuccess) return e;
  }
  float* const parts_a = p.parts + up(part_bytes(p.M, p.N, p.R)) / 4;
  const int columns = p.xf32 ? kColumns<float> : kColumns<uint16_t>;
  const int slices = (p.d_a ? (p.K + columns - 1) / columns : 0) + (p.d_b ? (p.N + columns - 1) / columns : 0);
  GradLaunch q{grad_of(p, p.x, p.g, p.d_a, nullptr, p.K, slices, parts_a),
               grad_of(p, p.d_out, p.hidden, p.d_b, p.scales, p.N, slices, p.parts),
               p.ids, p.order, p.offsets, p.M, p.R, p.n, 0};
  while ((kRanks << q.shift) < p.R) ++q.shift;
  void* args[] = {&q};
  const unsigned blocks = (unsigned)(q.a.slices * q.a.chunks + q.b.slices * q.b.chunks);
  e = hipLaunchKernel(p.xf32 ? pick<float>(p.R) : pick<uint16_t>(p.R), dim3(blocks),
                      dim3(kThreads), args, 0, stream);
  if (e != hipSuccess) return e;
  const auto joins = [&](const Grad& g) {
    const bool left = g.out && (p.ids || p.n > 1 || g.chunks > 1);
    return left ? (int)(((size_t)g.O * p.R / 4 + 255) / 256) : 0;
  };
  int blocks_a = joins(q.a);
  const int all = blocks_a + joins(q.b);
  if (!all) return e;
  void* join_args[] = {&q, &blocks_a};
  e = hipLaunchKernel(reinterpret_cast<const void*>(&join_kernel), dim3((unsigned)all, (unsigned)p.n), dim3(256), join_args,
                      0, stream);
  return e;
}

}  // namespace q4
