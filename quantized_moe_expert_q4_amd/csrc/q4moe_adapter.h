// Shared by the kernels of the low-rank adapters (q4moe_adapter.hip: rows,
// q4moe_adapter_grad.hip: the gradients of the adapters' matrices).
#pragma once
#include "q4moe_device.h"
#include "q4moe_layer.h"
#include "q4moe_rows.h"

namespace q4 {

typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef uint32_t v2u __attribute__((ext_vector_type(2)));

// A float as bf16, which is held in a uint16_t.
__device__ __forceinline__ uint16_t rounded(float v) { return __builtin_bit_cast(uint16_t, (__bf16)v); }

__device__ __forceinline__ v4f multiply_bf16(const v4u a, const v4u b, v4f c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, a), __builtin_bit_cast(v8bf, b), c, 0, 0, 0);
}

// Eight rows of eight (four) 16-bit values as their columns.
template <class ROW, int COLUMNS>
__device__ __forceinline__ void turn(const ROW (&row)[8], v4u (&column)[COLUMNS]) {
  static_assert(sizeof(ROW) == 2 * COLUMNS, "a row holds the columns");
#pragma unroll
  for (int d = 0; d < COLUMNS / 2; ++d)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      column[2 * d][i] = perm(row[2 * i + 1][d], row[2 * i][d], 0x05040100u);
      column[2 * d + 1][i] = perm(row[2 * i + 1][d], row[2 * i][d], 0x07060302u);
    }
}

// Eight floats as PARTS bf16 numbers of eight bits each, highest first (24 bits: all of a float).
template <int PARTS>
__device__ __forceinline__ void split(const float (&v)[8], v4u (&part)[PARTS]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t a = __float_as_uint(v[2 * i]), b = __float_as_uint(v[2 * i + 1]);
#pragma unroll
    for (int d = 0; d < PARTS; ++d) {
      part[d][i] = perm(b, a, 0x07060302u);
      a = __float_as_uint(__uint_as_float(a) - __uint_as_float(a & 0xFFFF0000u));
      b = __float_as_uint(__uint_as_float(b) - __uint_as_float(b & 0xFFFF0000u));
    }
  }
}

// Row's adapter, -1 for an id that names none.
__device__ __forceinline__ int adapter_of(const int32_t* ids, int row, int n) {
  const int id = ids ? ids[row] : 0;
  return (uint32_t)id < (uint32_t)n ? id : -1;
}

// A work-group of eight waves sorts out an adapter's rows: where they begin among
// those sorted by adapter, and the rows.  Each wave takes a run of the rows; it is
// read twice, first to count.  No atomics: the same order on every run.
__device__ __forceinline__ void order_rows(const int32_t* ids, int M, int n, int adapter, int32_t* order,
                                           int32_t* offsets) {
  constexpr int kWaves = 8, kAhead = 8;
  __shared__ int s_below[kWaves], s_mine[kWaves];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int steps = (M + 63) / 64, begin = 64 * (steps * wave / kWaves), end = min(M, 64 * (steps * (wave + 1) / kWaves));
  const auto visit = [&](auto&& see) {
    for (int t0 = begin; t0 < end; t0 += 64 * kAhead) {
      int id[kAhead];
#pragma unroll
      for (int k = 0; k < kAhead; ++k) id[k] = ids[min(t0 + 64 * k + lane, M - 1)];
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const int t = t0 + 64 * k + lane;
        see(t, t < end ? id[k] : -1);
      }
    }
  };
  int below = 0, mine = 0;
  visit([&](int, int id) {
    below += __popcll(__ballot(id >= 0 && id < adapter));
    mine += __popcll(__ballot(id == adapter));
  });
  if (lane == 0) {
    s_below[wave] = below;
    s_mine[wave] = mine;
  }
  __syncthreads();
  int start = 0, at = 0, count = 0;
  for (int w = 0; w < kWaves; ++w) {
    start += s_below[w];
    at += w < wave ? s_mine[w] : 0;
    count += s_mine[w];
  }
  if (threadIdx.x == 0) {
    offsets[adapter] = start;
    if (adapter == n - 1) offsets[n] = start + count;
  }
  if (!mine) return;
  at += start;
  visit([&](int t, int id) {
    const uint64_t votes = __ballot(id == adapter);
    if (id == adapter) order[at + __popcll(votes & ((1ull << lane) - 1))] = t;
    at += __popcll(votes);
  });
}

// The gradients of the matrices.  `order` are the rows that have an adapter,
// by adapter and then in their own order, `offsets` [n + 1] where each adapter's
// begin; without ids neither is used.
struct AdapterGradParams {
  const void* x;          // [M][K]
  const void* d_out;      // [M][N]
  const float* g;         // [M][R]
  const float* hidden;    // [M][R]
  const int32_t* ids;
  const float* scales;
  float* d_a;             // or nullptr
  float* d_b;             // or nullptr
  int32_t* order;
  int32_t* offsets;
  float* parts;           // sums of adapters whose rows several work-groups share
  int M, N, K, R, n, xf32;
  bool sorted;            // order and offsets are there
};

size_t adapter_grad_workspace(int64_t M, int64_t N, int64_t K, int64_t R, int64_t n);
hipError_t launch_adapter_grad(const AdapterGradParams& p, hipStream_t stream);

}  // namespace q4
