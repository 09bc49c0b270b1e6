// Low-rank adapters of many requests: each row has an adapter (A [R][K],
// B [N][R]) of its own, or none.
//   forward   h = A x, out = base + s B h
//   backward  g = s B^T d, d_x = base + A^T g (and in q4moe_adapter_grad.hip
//             d_A = sum_t g x^T, d_B = s sum_t d h^T)
//
// A work-group takes 16 rows of one adapter, gathered from a window of 256 rows
// (group_rows), so that rows of one adapter need not stand together.  Both
// directions take long rows to R sums ("shrink") and those to long rows
// ("expand"); the adapter's matrix runs along the sum, or across it (ACROSS, the
// backward pass).  The R sums of the rows stay in LDS between the two; only
// where few rows would leave the device idle are there two launches, the first
// with several work-groups along the long sum.
//
// Matrix operations take the adapter as rows and the 16 tokens as columns.  bf16:
// the values between the products enter the second as two bf16 parts (16 bits).
#include "q4moe_adapter.h"

namespace q4 {

namespace {

constexpr int kWaves = 8;
constexpr int kThreads = 64 * kWaves;
constexpr int kWindow = 256;         // rows whose adapters a work-group looks at
constexpr int kTile = 16;            // rows of a work-group
constexpr int kMaxSplits = 16;       // parts of a long sum
constexpr int kFill = 512;           // work-groups that fill the device: no more parts than give so many

// The rows of one work-group: `count` of them, all of `adapter` (-1: none).
struct Rows {
  int row[kTile];
  int adapter, count;
};

// Tile `index` of the window's rows: the rows of each adapter, in their order,
// in tiles of 16, adapters by their first row.  False where there is none.
__device__ __forceinline__ bool group_rows(const int32_t* ids, int M, int n, int window, int index, Rows& out) {
  __shared__ int s_id[kWindow], s_first[kWindow], s_total[kWindow / 64];
  const int t = threadIdx.x, row = window * kWindow + t, lane = t & 63, wave = t >> 6;
  const int rows = min(kWindow, M - window * kWindow);
  const int id = t < rows ? adapter_of(ids, row, n) : -2;
  if (t < kWindow) s_id[t] = id;
  if (t == 0) out.count = 0;
  __syncthreads();
  int before = t, same = rows, first = 0;
  // most windows hold one adapter
  if (!__syncthreads_and(t >= rows || id == s_id[0])) {
    before = same = 0;
    first = t;
    if (t < rows)
      for (int j = 0; j < rows; ++j) {
        const bool eq = s_id[j] == id;
        same += eq;
        before += eq && j < t;
        first = eq && j < first ? j : first;
      }
  }
  // tiles of the adapters whose first row comes earlier
  const int tiles = t < rows && before == 0 ? (same + kTile - 1) / kTile : 0;
  int sum = tiles;
  for (int d = 1; d < 64; d <<= 1) {
    const int other = __shfl_up(sum, d);
    sum += lane >= d ? other : 0;
  }
  if (lane == 63 && t < kWindow) s_total[wave] = sum;
  __syncthreads();
  int start = sum - tiles;
  for (int w = 0; w < min(wave, kWindow / 64); ++w) start += s_total[w];
  if (t < kWindow) s_first[t] = start;
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

struct RowsParams {
  const void* x;          // [M][C]
  const void* shrink;     // per adapter [R][C], ACROSS: [C][R]
  const void* expand;     // per adapter [O][R], ACROSS: [R][O]
  const int32_t* ids;
  const float* scales;    // per adapter, or nullptr (1)
  const void* base;       // [M][O] or nullptr
  void* out;              // [M][O] or nullptr
  float* hidden;          // [M][R] or nullptr: the sums (ACROSS: scaled)
  float* partial;         // [splits][M][R]
  int M, C, O, R, n;
  int splits;             // parts of the long sum
  int slice;              // columns of a work-group's results
};

// What a launch does: all of it, or one of the two products.
enum Stage { kBoth, kShrink, kExpand };

constexpr int kRankBlock = 128;      // ranks that a pass over the long rows sums
constexpr int kTurnBytes = 8192;     // LDS of a wave where the adapter is turned

template <class T, int NR, bool ACROSS>
constexpr int kSumBytes = ACROSS && sizeof(T) == 2 ? kWaves * kTurnBytes : kWaves * NR * 1024;

// Bytes of a row of the values between the products: two bf16 parts, or floats,
// and 16 bytes so that rows start at different banks.
template <class T>
__device__ __forceinline__ int hidden_pitch(int R) {
  return sizeof(T) == 2 ? 2 * R + 16 : 4 * R + 16;
}
constexpr int kHiddenBytes = kTile * (4 * 256 + 32);

// acc[j]: of the wave's part of the sum, ranks rank0 + 16 j + 4 (lane / 16) .. of row lane % 16.
template <class T, int NR, bool ACROSS>
__device__ __forceinline__ void shrink_rows(const RowsParams& p, const T* w, int row, int rank0, int begin, int end,
                                            uint8_t* s_turn, v4f (&acc)[NR]) {
  const int lane = threadIdx.x & 63, l = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  if constexpr (!ACROSS && sizeof(T) == 2) {
    // steps of 64 elements: two operations; 128 bytes of a row are read together.
    // Past the row's end x is 0 (and what it meets there an element of the same
    // row of the adapter); ranks past R are dropped later.
    const T* const x = static_cast<const T*>(p.x) + (size_t)row * p.C;
    constexpr int kBatch = NR >= 4 ? 1 : NR == 2 ? 2 : 4;
    for (int s0 = begin + wave * kBatch; s0 < end; s0 += kWaves * kBatch) {
      v4u xv[kBatch][2], wv[kBatch][NR][2];
#pragma unroll
      for (int b = 0; b < kBatch; ++b)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int c = 64 * (s0 + b) + 16 * g + 8 * h, at = min(c, p.C - 8);
          xv[b][h] = *reinterpret_cast<const v4u*>(x + at);
          if (c >= p.C || s0 + b >= end) xv[b][h] = v4u{0, 0, 0, 0};
#pragma unroll
          for (int j = 0; j < NR; ++j)
            wv[b][j][h] = *reinterpret_cast<const v4u*>(w + (size_t)min(rank0 + 16 * j + l, p.R - 1) * p.C + at);
        }
#pragma unroll
      for (int b = 0; b < kBatch; ++b)
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int j = 0; j < NR; ++j) acc[j] = multiply_bf16(wv[b][j][h], xv[b][h], acc[j]);
    }
  } else if constexpr (sizeof(T) == 2) {
    // Chunks of kCount elements: a lane reads eight rows of eight ranks, turns
    // them, and leaves them in the wave's LDS as [rank][eight elements].
    constexpr int kCount = 256 / NR, kChunks = kCount / 8, kOctets = 2 * NR;
    v4u* const s_w = reinterpret_cast<v4u*>(s_turn + wave * kTurnBytes);
    const auto place = [](int r, int c) {
      constexpr int kMove = NR == 1 ? 2 : NR == 2 ? 1 : 0;
      if constexpr (NR <= 4) return r * kChunks + (c ^ ((r & 7) ^ (((r >> 3) & (kOctets - 1)) << kMove)));
      else return r * kChunks + (c ^ ((r >> 1) & 3));
    };
    const int octet = lane % kOctets, part = lane / kOctets;
    const int rank = min(rank0 + 8 * octet, p.R - 8);
    const RowMatrix<T> x(p.x, p.M, p.C);
    for (int s = begin + wave; s < end; s += kWaves) {
      const int c0 = s * kCount;
      v4u from[8], column[8], xv[kCount / 32];
#pragma unroll
      for (int i = 0; i < 8; ++i)
        from[i] = *reinterpret_cast<const v4u*>(w + (size_t)min(c0 + 8 * part + i, p.C - 1) * p.R + rank);
#pragma unroll
      for (int h = 0; h < kCount / 32; ++h) xv[h] = x.chunk(row, c0 + 32 * h + 8 * g);
      turn(from, column);
      wave_sync();
#pragma unroll
      for (int i = 0; i < 8; ++i) s_w[place(8 * octet + i, part)] = column[i];
      wave_sync();
#pragma unroll
      for (int h = 0; h < kCount / 32; ++h)
#pragma unroll
        for (int j = 0; j < NR; ++j) acc[j] = multiply_bf16(s_w[place(16 * j + l, 4 * h + g)], xv[h], acc[j]);
    }
  } else {
    const RowMatrix<T> x(p.x, p.M, p.C);
    for (int s = begin + wave; s < end; s += kWaves) {
      const int c = 16 * s + 4 * g;
      const v4u xv = x.chunk(row, c);
#pragma unroll
      for (int j = 0; j < NR; ++j) {
        const int r = min(rank0 + 16 * j + l, p.R - 1);
        v4u wv;
        if constexpr (ACROSS) {
#pragma unroll
          for (int i = 0; i < 4; ++i) wv[i] = __float_as_uint(w[(size_t)min(c + i, p.C - 1) * p.R + r]);
        } else {
          wv = *reinterpret_cast<const v4u*>(w + (size_t)r * p.C + min(c, p.C - 4));
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
          acc[j] = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(wv[i]), __uint_as_float(xv[i]), acc[j], 0, 0, 0);
      }
    }
  }
}

// Elements of a step of shrink_rows, a work-group's unit of the long sum.
template <class T, int NR, bool ACROSS>
constexpr int kStep = sizeof(T) == 4 ? 16 : ACROSS ? 256 / NR : 64;

// Keeps four values of the sums (ranks r ..) for the second product.
template <class T>
__device__ __forceinline__ void keep_hidden(uint8_t* s_hidden, int R, int row, int r, v4f v) {
  if constexpr (sizeof(T) == 2) {
    uint32_t part[2][2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t a = __float_as_uint(v[2 * i]), b = __float_as_uint(v[2 * i + 1]);
      const float ra = __uint_as_float(a) - __uint_as_float(a & 0xFFFF0000u);
      const float rb = __uint_as_float(b) - __uint_as_float(b & 0xFFFF0000u);
      part[0][i] = perm(b, a, 0x07060302u);
      part[1][i] = perm(__float_as_uint(rb), __float_as_uint(ra), 0x07060302u);
    }
#pragma unroll
    for (int d = 0; d < 2; ++d)
      __builtin_memcpy(s_hidden + (d * kTile + row) * hidden_pitch<T>(R) + 2 * r, part[d], 8);
  } else {
    __builtin_memcpy(s_hidden + row * hidden_pitch<T>(R) + 4 * r, &v, 16);
  }
}

// Eight consecutive results of a row onto base; O any: rows may start at any element.
__device__ __forceinline__ void put8(const RowsParams& p, const RowMatrix<uint16_t>& base, int row, int o, const float (&v)[8]) {
  v4u b = {0, 0, 0, 0};
  if (p.base) b = base.chunk(row, o);
  uint16_t r[8];
#pragma unroll
  for (int i = 0; i < 8; ++i)
    r[i] = rounded<uint16_t>(v[i] + __uint_as_float(i & 1 ? b[i / 2] & 0xFFFF0000u : b[i / 2] << 16));
  uint16_t* const out = static_cast<uint16_t*>(p.out) + (size_t)row * p.O + o;
  if (o + 8 <= p.O) {
    __builtin_memcpy(out, r, 16);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (o + i < p.O) out[i] = r[i];
  }
}
__device__ __forceinline__ void put4(const RowsParams& p, const RowMatrix<float>& base, int row, int o, const v4f v) {
  v4f r = v;
  if (p.base) r += __builtin_bit_cast(v4f, base.chunk(row, o));
  float* const out = static_cast<float*>(p.out) + (size_t)row * p.O + o;
  if (o + 4 <= p.O) {
    __builtin_memcpy(out, &r, 16);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (o + i < p.O) out[i] = r[i];
  }
}

// The work-group's columns [begin, end) of its rows' results.
template <class T, bool ACROSS>
__device__ __forceinline__ void expand_rows(const RowsParams& p, const T* w, bool live, const Rows& rows,
                                            const uint8_t* s_hidden, int begin, int end) {
  const int lane = threadIdx.x & 63, l = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int row = rows.row[min(l, rows.count - 1)];
  const bool mine = l < rows.count;
  const RowMatrix<T> base(p.base, p.M, p.O);
  const int pitch = hidden_pitch<T>(p.R);
  if constexpr (sizeof(T) == 2) {
    // Eight ranks are a chunk of the sum, of the high parts and then of the low
    // ones; past those h is 0 (and meets an element of the same row of the adapter).
    const int chunks = p.R / 8, steps = live ? (2 * chunks + 3) / 4 : 0;
    const auto part = [&](int s, int& chunk) {
      const int c = 4 * s + g;
      const bool low = c >= chunks;
      chunk = min(low ? c - chunks : c, chunks - 1);
      v4u h = *reinterpret_cast<const v4u*>(s_hidden + ((low ? kTile : 0) + l) * pitch + 16 * chunk);
      if (c >= 2 * chunks) h = v4u{0, 0, 0, 0};
      return h;
    };
    if constexpr (ACROSS) {
      // 128 columns: lane l reads eight of them, which eight tiles share; a lane's
      // results are the eight columns of octet g + 4 i.
      const int octet = (l >> 2) + 4 * (l & 3);
      for (int o0 = begin + 128 * wave; o0 < end; o0 += 128 * kWaves) {
        v4f acc[8] = {};
        for (int s = 0; s < steps; ++s) {
          int chunk;
          const v4u h = part(s, chunk);
          v4u from[8], column[8];
#pragma unroll
          for (int i = 0; i < 8; ++i)
            from[i] = *reinterpret_cast<const v4u*>(w + (size_t)(8 * chunk + i) * p.O + min(o0 + 8 * octet, p.O - 8));
          turn(from, column);
#pragma unroll
          for (int j = 0; j < 8; ++j) acc[j] = multiply_bf16(column[j], h, acc[j]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int o = o0 + 8 * (g + 4 * i);
          float v[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) v[j] = acc[j][i];
          if (mine && o < p.O) put8(p, base, row, o, v);
        }
      }
    } else {
      // 64 columns, in pairs of tiles whose results give a lane eight neighbours.
      for (int o0 = begin + 64 * wave; o0 < end; o0 += 64 * kWaves) {
        v4f acc[2][2] = {};
        for (int s = 0; s < steps; ++s) {
          int chunk;
          const v4u h = part(s, chunk);
          v4u wv[2][2];
#pragma unroll
          for (int q = 0; q < 2; ++q)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const int o = min(o0 + 32 * q + 8 * (l >> 2) + 4 * j + (l & 3), p.O - 1);
              wv[q][j] = *reinterpret_cast<const v4u*>(w + (size_t)o * p.R + 8 * chunk);
            }
#pragma unroll
          for (int q = 0; q < 2; ++q)
#pragma unroll
            for (int j = 0; j < 2; ++j) acc[q][j] = multiply_bf16(wv[q][j], h, acc[q][j]);
        }
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const int o = o0 + 32 * q + 8 * g;
          float v[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] = acc[q][i / 4][i % 4];
          if (mine && o < p.O) put8(p, base, row, o, v);
        }
      }
    }
  } else if constexpr (ACROSS) {
    // 64 columns: lane l reads four of them, which four tiles share.
    for (int o0 = begin + 64 * wave; o0 < end; o0 += 64 * kWaves) {
      v4f acc[4] = {};
      for (int r = g; live && r < p.R; r += 4) {
        const float h = *reinterpret_cast<const float*>(s_hidden + l * pitch + 4 * r);
        const v4f wv = *reinterpret_cast<const v4f*>(w + (size_t)r * p.O + min(o0 + 4 * l, p.O - 4));
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[j] = __builtin_amdgcn_mfma_f32_16x16x4f32(wv[j], h, acc[j], 0, 0, 0);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int o = o0 + 4 * (4 * g + i);
        if (mine && o < p.O) put4(p, base, row, o, v4f{acc[0][i], acc[1][i], acc[2][i], acc[3][i]});
      }
    }
  } else {
    for (int o0 = begin + 64 * wave; o0 < end; o0 += 64 * kWaves) {
      v4f acc[4] = {};
      for (int r0 = 0; live && r0 < p.R; r0 += 16) {
        const int r = r0 + 4 * g, at = min(r, p.R - 4);
        v4f h = *reinterpret_cast<const v4f*>(s_hidden + l * pitch + 4 * at);
        if (r >= p.R) h = v4f{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const v4f wv = *reinterpret_cast<const v4f*>(w + (size_t)min(o0 + 16 * j + l, p.O - 1) * p.R + at);
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[j] = __builtin_amdgcn_mfma_f32_16x16x4f32(wv[i], h[i], acc[j], 0, 0, 0);
        }
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int o = o0 + 16 * j + 4 * g;
        if (mine && o < p.O) put4(p, base, row, o, acc[j]);
      }
    }
  }
}

// grid: slices of the results or parts of the sum, tiles of a window, windows.
template <class T, int NR, bool ACROSS, int STAGE>
__global__ __launch_bounds__(kThreads) void rows_kernel(RowsParams p) {
  __shared__ Rows s_rows;
  __shared__ __align__(16) uint8_t s_sum[STAGE == kExpand ? 16 : kSumBytes<T, NR, ACROSS>];
  __shared__ __align__(16) uint8_t s_hidden[STAGE == kShrink ? 16 : kHiddenBytes];
  if (!group_rows(p.ids, p.M, p.n, (int)blockIdx.z, (int)blockIdx.y, s_rows)) return;
  const int adapter = s_rows.adapter, count = s_rows.count;
  const bool live = adapter >= 0;
  const size_t table = (size_t)max(adapter, 0) * p.R;
  const float scale = live && p.scales ? p.scales[adapter] : 1.0f;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const bool first = blockIdx.x == 0;
  // four sums of a row, complete
  const auto finish = [&](int row, int r, v4f v) {
    if (row >= count || r >= p.R) return;
    const v4f scaled = v * scale;
    if (p.hidden && first) *reinterpret_cast<v4f*>(p.hidden + (size_t)s_rows.row[row] * p.R + r) = ACROSS ? scaled : v;
    keep_hidden<T>(s_hidden, p.R, row, r, scaled);
  };
  if constexpr (STAGE != kExpand) {
    const int steps = (p.C + kStep<T, NR, ACROSS> - 1) / kStep<T, NR, ACROSS>;
    const int split = STAGE == kShrink ? (int)blockIdx.x : 0, splits = STAGE == kShrink ? p.splits : 1;
    const int begin = (int)((int64_t)steps * split / splits), end = (int)((int64_t)steps * (split + 1) / splits);
    v4f(*const sums)[NR][64] = reinterpret_cast<v4f(*)[NR][64]>(s_sum);
    for (int rank0 = 0; rank0 < p.R; rank0 += kRankBlock) {
      v4f acc[NR] = {};
      if (live)
        shrink_rows<T, NR, ACROSS>(p, static_cast<const T*>(p.shrink) + table * p.C, s_rows.row[min(lane & 15, count - 1)],
                                   rank0, begin, end, s_sum, acc);
      __syncthreads();
#pragma unroll
      for (int j = 0; j < NR; ++j) sums[wave][j][lane] = acc[j];
      __syncthreads();
      for (int i = threadIdx.x; i < NR * 64; i += kThreads) {
        const int j = i >> 6, from = i & 63, row = from & 15, r = rank0 + 16 * j + 4 * (from >> 4);
        v4f v = sums[0][j][from];
        for (int k = 1; k < kWaves; ++k) v += sums[k][j][from];
        if constexpr (STAGE == kBoth) {
          finish(row, r, v);
        } else if (row < count && r < p.R) {
          *reinterpret_cast<v4f*>(p.partial + ((size_t)split * p.M + s_rows.row[row]) * p.R + r) = v;
        }
      }
      __syncthreads();
    }
  } else {
    for (int i = threadIdx.x; i < kTile * p.R / 4; i += kThreads) {
      const int row = i / (p.R / 4), r = 4 * (i % (p.R / 4));
      if (row >= count) break;
      const float* const at = p.partial + (size_t)s_rows.row[row] * p.R + r;
      v4f v = *reinterpret_cast<const v4f*>(at);
      for (int k = 1; k < p.splits; ++k) v += *reinterpret_cast<const v4f*>(at + (size_t)k * p.M * p.R);
      finish(row, r, v);
    }
    __syncthreads();
  }
  if constexpr (STAGE != kShrink) {
    if (!p.out) return;
    const int begin = (int)blockIdx.x * p.slice, end = min(p.O, begin + p.slice);
    expand_rows<T, ACROSS>(p, static_cast<const T*>(p.expand) + table * p.O, live, s_rows, s_hidden, begin, end);
  }
}

// Kernels by type, tiles of 16 ranks in a pass, and direction.
template <class T, bool ACROSS, int STAGE>
const void* pick(int R) {
  if constexpr (STAGE != kExpand) {
    if (R > 64) return reinterpret_cast<const void*>(&rows_kernel<T, 8, ACROSS, STAGE>);
    if (R > 32) return reinterpret_cast<const void*>(&rows_kernel<T, 4, ACROSS, STAGE>);
    if (R > 16) return reinterpret_cast<const void*>(&rows_kernel<T, 2, ACROSS, STAGE>);
  }
  return reinterpret_cast<const void*>(&rows_kernel<T, 1, ACROSS, STAGE>);
}
template <int STAGE>
const void* pick(int R, bool f32, bool across) {
  if (f32) return across ? pick<float, true, STAGE>(R) : pick<float, false, STAGE>(R);
  return across ? pick<uint16_t, true, STAGE>(R) : pick<uint16_t, false, STAGE>(R);
}

template <int STAGE>
hipError_t launch(RowsParams p, int blocks, bool f32, bool across, hipStream_t stream) {
  void* args[] = {&p};
  const dim3 grid((unsigned)blocks, (unsigned)window_tiles(p.M, p.n, p.ids != nullptr),
                  (unsigned)((p.M + kWindow - 1) / kWindow));
  return hipLaunchKernel(pick<STAGE>(p.R, f32, across), grid, dim3(kThreads), args, 0, stream);
}

// Work-groups along the results: as many as fill the device, of 512 columns (one
// unit of each wave) at least.
int slices_for(int M, int O, int& slice) {
  const int tiles = (M + kTile - 1) / kTile, most = (O + 511) / 512;
  int s = (kFill / 2 + tiles - 1) / tiles;
  s = s > most ? most : s;
  slice = ((O + s - 1) / s + 511) / 512 * 512;
  return (O + slice - 1) / slice;
}

hipError_t launch_rows(RowsParams p, bool f32, bool across, hipStream_t stream) {
  const int tiles = (p.M + kTile - 1) / kTile, steps = (p.C + 511) / 512;
  int slices = slices_for(p.M, p.O, p.slice);
  if (!p.out) slices = 1;
  int splits = kFill / tiles;
  splits = splits > kMaxSplits ? kMaxSplits : splits;
  splits = splits > steps ? steps : splits;
  const size_t table = (size_t)p.R * p.C * (f32 ? 4 : 2);
  if (splits <= 1 || table <= (1u << 18)) {
    p.splits = 1;
    return launch<kBoth>(p, slices, f32, across, stream);
  }
  p.splits = splits;
  const hipError_t e = launch<kShrink>(p, splits, f32, across, stream);
  return e != hipSuccess ? e : launch<kExpand>(p, slices, f32, across, stream);
}

// The parts of the hidden sums: M rows, or while there are several parts at
// most kFill tiles in all.
size_t hidden_bytes(int64_t M, int64_t R) {
  const int64_t several = M * kMaxSplits < kFill * kTile ? M * kMaxSplits : kFill * kTile;
  const size_t rows = (size_t)(M > several ? M : several);
  return (rows * (size_t)R * 4 + 255) / 256 * 256;
}

}  // namespace

size_t adapter_workspace(int64_t M, int64_t N, int64_t K, int64_t R, int64_t n) {
  return hidden_bytes(M, R) + (size_t)M * R * 4 / 256 * 256 + 256 + adapter_grad_workspace(M, N, K, R, n);
}

hipError_t launch_adapter(const AdapterParams& p, hipStream_t stream) {
  return launch_rows({p.x, p.a, p.b, p.ids, p.scales, p.base, p.out, p.hidden, p.partial, p.M, p.K, p.N, p.R, p.n, 0, 0},
                     p.xf32, false, stream);
}

hipError_t launch_adapter_backward(const AdapterBackwardParams& p, hipStream_t stream) {
  float* const g = p.partial + hidden_bytes(p.M, p.R) / 4;
  float* const rest = g + (size_t)p.M * p.R / 64 * 64 + 64;
  if (p.d_x || p.d_a) {
    const hipError_t e = launch_rows({p.d_out, p.b, p.a, p.ids, p.scales, p.base, p.d_x, p.d_a ? g : nullptr, p.partial,
                                      p.M, p.N, p.K, p.R, p.n, 0, 0},
                                     p.xf32, true, stream);
    if (e != hipSuccess) return e;
  }
  if (!p.d_a && !p.d_b) return hipSuccess;
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
