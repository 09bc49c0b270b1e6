// Low-rank adapters of many requests: each row has an adapter (A [R][K],
// B [N][R]) of its own, or none.
//   forward   h = A x, out = base + s B h
//   backward  g = s B^T d, d_x = base + A^T g (and in q4moe_adapter_grad.hip
//             d_A = sum_t g x^T, d_B = s sum_t d h^T)
//
// A work-group takes 16 rows of one adapter (of large batches 64, which read the
// adapter a quarter as often), gathered from a window of 256 rows (group_rows),
// so that rows of one adapter need not stand together.  Both directions take long
// rows to R sums ("shrink") and those to long rows ("expand"); the adapter's matrix
// runs along the sum, or across it (ACROSS, the backward pass).  Small calls do
// both in one launch, with the R sums of the rows in LDS between them; where the
// long sum has to be shared by several work-groups to fill the device there are
// two, the second joining the parts.
//
// What bounds it.  Large batches: memory and the latency of their loads: 4096 rows
// of 7168 x 4096, rank 32, in kernels of 25 + 22 us (59 MB read; 34 MB read and 34
// written; 2.3 and 3.0 TB/s, a copy 5.1); across, 8192 rows of 4096 x 4096, rank
// 16, in 22 + 30 (3.1 and 4.4).  Results stored past the caches, whole lines each:
// the two expanding kernels took 26 and 37 before.  Small calls: latency, a call of
// one row takes 10 us and one of 64 rows of 24 adapters 16, where calls whose
// kernels do nothing take 7.5 (one launch) and 10.3 (two).
//
// Matrix operations take the adapter as rows and 16 tokens as columns.  bf16:
// the values between the products enter the second as two bf16 parts: 2^-16 at
// most, a 256th of the output's rounding, at two thirds of the operations that
// all 24 bits would take.
#include "q4moe_adapter.h"

namespace q4 {

namespace {

constexpr int kWaves = 8;
constexpr int kThreads = 64 * kWaves;
constexpr int kWindow = 256;         // rows whose adapters a work-group looks at
constexpr int kTile = 16;            // rows of a matrix operation
constexpr int kMaxSplits = 16;       // parts of a long sum
// Rows from which on a work-group takes 64 of an adapter instead of 16.  Forward,
// 7168 to 4096, eight adapters, rows of one together, bf16 rank 32: 19 us against
// 17 with 16 rows for 512 rows, 23 against 20 for 1024, 33 against 30 for 2048, 55
// against 62 for 4096; rank 16 18 against 31 for 512, 21 against 32 for 1024, 47
// against 56 for 4096; float rank 32 29 against 23, 37 against 34, 104 against 135.
// The backward call gains from 768 rows on (bf16, rank 32: 58 against 65; 63
// against 70 for 1024, 121 against 145 for 4096).
constexpr int kLargeBatch = 1024;
constexpr int kFill = 512;           // work-groups that fill the device: no more parts than give so many

// The rows of one work-group: `count` of them, all of `adapter` (-1: none);
// row(i) is the i-th.
struct Rows {
  const int* list;
  int adapter, count;
  __device__ __forceinline__ int row(int i) const { return list[i]; }
};

// Tile `index` of the window's rows: the rows of each adapter, in their order,
// in tiles of ROWS, adapters by their first row; count 0 where there is none.
// Every wave finds its own copy: four rows a lane, an adapter after the other by
// votes, without a barrier.
template <int ROWS>
__device__ __forceinline__ Rows group_rows(const int32_t* ids, int M, int n, int window, int index) {
  constexpr int kRuns = kWindow / 64;
  __shared__ int s_list[kWaves][ROWS];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  Rows out{s_list[wave], -1, 0};
  if (M <= 64) {
    // every row against every other: the adapters' first tiles by their first
    // rows, then their second ones, and so on (64 rows of 24 adapters: 0.4 us,
    // by the loop below 3)
    const int id = lane < M ? adapter_of(ids, lane, n) : -2;
    int before = 0, count = 0;
#pragma unroll
    for (int j = 0; j < 64; ++j) {
      const bool eq = __builtin_amdgcn_readlane(id, j) == id;
      count += eq;
      before += eq && j < lane;
    }
    uint64_t firsts = __ballot(lane < M && before == 0);
    int skip = 0;                                // rows of the adapter in earlier tiles
    while (firsts && index >= __popcll(firsts)) {
      index -= __popcll(firsts);
      skip += ROWS;
      firsts = __ballot(lane < M && before == 0 && count > skip);
    }
    if (!firsts) return out;
    const bool chosen = ((firsts >> lane) & 1) && __popcll(firsts & ((1ull << lane) - 1)) == index;
    const int first = __builtin_ctzll(__ballot(chosen));
    out.adapter = __builtin_amdgcn_readlane(id, first);
    out.count = min(ROWS, __builtin_amdgcn_readlane(count, first) - skip);
    if (id == out.adapter && (uint32_t)(before - skip) < ROWS) s_list[wave][before - skip] = lane;
    wave_sync();
    return out;
  }
  int id[kRuns];
  uint64_t left[kRuns], same[kRuns];
#pragma unroll
  for (int k = 0; k < kRuns; ++k) {
    const int row = window * kWindow + 64 * k + lane;
    id[k] = adapter_of(ids, min(row, M - 1), n);
    left[k] = __ballot(row < M);
  }
  bool found = false;
#pragma unroll
  for (int k = 0; k < kRuns; ++k) {              // the adapters whose first row is of run k
    while (!found && left[k]) {
      const int adapter = __builtin_amdgcn_readlane(id[k], __builtin_ctzll(left[k]));
      int count = 0;
#pragma unroll
      for (int m = 0; m < kRuns; ++m) {
        same[m] = m < k ? 0 : __ballot(id[m] == adapter) & left[m];
        count += __popcll(same[m]);
        left[m] &= ~same[m];
      }
      const int tiles = (count + ROWS - 1) / ROWS;
      found = index < tiles;
      if (found) {
        out.adapter = adapter;
        out.count = min(ROWS, count - ROWS * index);
      } else {
        index -= tiles;
      }
    }
  }
  if (!found) return out;
  int before = -ROWS * index;
#pragma unroll
  for (int k = 0; k < kRuns; ++k) {
    const int at = before + __popcll(same[k] & ((1ull << lane) - 1));
    if (((same[k] >> lane) & 1) && (uint32_t)at < ROWS) s_list[wave][at] = window * kWindow + 64 * k + lane;
    before += __popcll(same[k]);
  }
  wave_sync();
  return out;
}

// Tiles that a window of M rows can have.
int window_tiles(int M, int n, bool ids, int tile) {
  const int rows = M < kWindow ? M : kWindow;
  const int kinds = !ids ? 1 : n + 1 < rows ? n + 1 : rows;
  return (rows + (tile - 1) * kinds) / tile;
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
  int32_t* order;         // or nullptr: the work-groups past the windows sort the rows
  int32_t* offsets;
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
template <int NR, int TT>
constexpr int kHiddenBytes = TT * kTile * (4 * (NR < 8 ? 16 * NR : 256) + 32);

// acc[t][j]: of the wave's part of the sum, ranks rank0 + 16 j + 4 (lane / 16) ..
// of row 16 t + lane % 16; tiles of rows past `tiles` are left out.
template <class T, int NR, bool ACROSS, int TT>
__device__ __forceinline__ void shrink_rows(const RowsParams& p, const T* w, const int (&row)[TT], int tiles, int rank0,
                                            int begin, int end, uint8_t* s_turn, v4f (&acc)[TT][NR]) {
  const int lane = threadIdx.x & 63, l = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  if constexpr (!ACROSS && sizeof(T) == 2) {
    // Steps of 64 elements: two operations; 128 bytes of a row are read together.
    // Past the row's end x is 0 (and what it meets there an element of the same
    // row of the adapter); ranks past R are dropped later.
    const T* x[TT];
#pragma unroll
    for (int t = 0; t < TT; ++t) x[t] = static_cast<const T*>(p.x) + (size_t)row[t] * p.C;
    constexpr int kBatch = TT > 1 || NR >= 4 ? 1 : NR == 2 ? 2 : 4;
    for (int s0 = begin + wave * kBatch; s0 < end; s0 += kWaves * kBatch) {
      v4u xv[kBatch][2][TT], wv[kBatch][NR][2];
#pragma unroll
      for (int b = 0; b < kBatch; ++b)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int c = 64 * (s0 + b) + 32 * h + 8 * g, at = min(c, p.C - 8);
#pragma unroll
          for (int t = 0; t < TT; ++t) {
            xv[b][h][t] = *reinterpret_cast<const v4u*>(x[t] + at);
            if (c >= p.C || s0 + b >= end) xv[b][h][t] = v4u{0, 0, 0, 0};
          }
#pragma unroll
          for (int j = 0; j < NR; ++j)
            wv[b][j][h] = *reinterpret_cast<const v4u*>(w + (size_t)min(rank0 + 16 * j + l, p.R - 1) * p.C + at);
        }
#pragma unroll
      for (int b = 0; b < kBatch; ++b)
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int t = 0; t < TT; ++t)
            if (t < tiles) {
#pragma unroll
              for (int j = 0; j < NR; ++j) acc[t][j] = multiply_bf16(wv[b][j][h], xv[b][h][t], acc[t][j]);
            }
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
      const bool whole = c0 + kCount <= p.C;
      // as much on its way at once as 64 registers hold
      constexpr int kSteps = kCount / 32, kAhead = kSteps * TT > 16 ? 16 / TT : kSteps;
      v4u from[8], column[8], xv[kAhead][TT];
      const auto load_x = [&](int h0) {
        if (whole) {
#pragma unroll
          for (int h = 0; h < kAhead; ++h)
#pragma unroll
            for (int t = 0; t < TT; ++t)
              __builtin_memcpy(&xv[h][t], x.data + (size_t)row[t] * p.C + c0 + 32 * (h0 + h) + 8 * g, 16);
        } else {
#pragma unroll
          for (int h = 0; h < kAhead; ++h)
#pragma unroll
            for (int t = 0; t < TT; ++t) xv[h][t] = x.chunk(row[t], c0 + 32 * (h0 + h) + 8 * g);
        }
      };
#pragma unroll
      for (int i = 0; i < 8; ++i)
        from[i] = *reinterpret_cast<const v4u*>(w + (size_t)min(c0 + 8 * part + i, p.C - 1) * p.R + rank);
      load_x(0);
      turn(from, column);
      wave_sync();
#pragma unroll
      for (int i = 0; i < 8; ++i) s_w[place(8 * octet + i, part)] = column[i];
      wave_sync();
#pragma unroll 1
      for (int h0 = 0; h0 < kSteps; h0 += kAhead) {
        if (h0) load_x(h0);
#pragma unroll
        for (int h = 0; h < kAhead; ++h)
#pragma unroll
          for (int j = 0; j < NR; ++j) {
            const v4u wv = s_w[place(16 * j + l, 4 * (h0 + h) + g)];
#pragma unroll
            for (int t = 0; t < TT; ++t)
              if (t < tiles) acc[t][j] = multiply_bf16(wv, xv[h][t], acc[t][j]);
          }
      }
    }
  } else {
    const RowMatrix<T> x(p.x, p.M, p.C);
    for (int s = begin + wave; s < end; s += kWaves) {
      const int c = 16 * s + 4 * g;
      v4u xv[TT];
#pragma unroll
      for (int t = 0; t < TT; ++t) xv[t] = x.chunk(row[t], c);
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
        for (int t = 0; t < TT; ++t)
          if (t < tiles) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
              acc[t][j] = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(wv[i]), __uint_as_float(xv[t][i]), acc[t][j],
                                                               0, 0, 0);
          }
      }
    }
  }
}

// Elements of a step of shrink_rows, a work-group's unit of the long sum.
template <class T, int NR, bool ACROSS>
constexpr int kStep = sizeof(T) == 4 ? 16 : ACROSS ? 256 / NR : 64;

// A float as the bits of two bf16 numbers, both to the nearest: within 2^-17 of
// it.  Where that would round to infinity both are cut off: there (2^128 less
// 2^120 at least) the second's last place is 2^112, so within 2^-16.
__device__ __forceinline__ void two_parts(float v, uint32_t& high, uint32_t& low) {
  high = (uint32_t)rounded(v) << 16;
  const bool cut = (high & 0x7FFFFFFFu) == 0x7F800000u;
  if (cut) high = __float_as_uint(v) & 0xFFFF0000u;
  const float rest = v - __uint_as_float(high);
  low = cut ? __float_as_uint(rest) : (uint32_t)rounded(rest) << 16;
}

// Keeps four values of the sums (ranks r ..) for the second product.
template <class T, int TT>
__device__ __forceinline__ void keep_hidden(uint8_t* s_hidden, int R, int row, int r, v4f v) {
  if constexpr (sizeof(T) == 2) {
    uint32_t part[2][2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      uint32_t a[2], b[2];
      two_parts(v[2 * i], a[0], a[1]);
      two_parts(v[2 * i + 1], b[0], b[1]);
#pragma unroll
      for (int d = 0; d < 2; ++d) part[d][i] = perm(b[d], a[d], 0x07060302u);
    }
#pragma unroll
    for (int d = 0; d < 2; ++d)
      __builtin_memcpy(s_hidden + (d * TT * kTile + row) * hidden_pitch<T>(R) + 2 * r, part[d], 8);
  } else {
    __builtin_memcpy(s_hidden + row * hidden_pitch<T>(R) + 4 * r, &v, 16);
  }
}

// 16 bytes of a row of the results, which leave no trace in the caches (8192 rows
// of 4096 + 4096 columns: the backward call takes 87 us with the hint, 95 without);
// rows may start at any element.
typedef uint32_t v4u_any __attribute__((ext_vector_type(4), aligned(2)));
template <class T>
__device__ __forceinline__ void put(const RowsParams& p, int row, int o, const T (&r)[16 / sizeof(T)]) {
  constexpr int kVec = 16 / sizeof(T);
  if (row < 0) return;
  T* const out = static_cast<T*>(p.out) + (size_t)row * p.O + o;
  if (o + kVec <= p.O) {
    v4u_any v;
    __builtin_memcpy(&v, r, 16);
    __builtin_nontemporal_store(v, reinterpret_cast<v4u_any*>(out));
  } else {
#pragma unroll
    for (int i = 0; i < kVec; ++i)
      if (o + i < p.O) out[i] = r[i];
  }
}

constexpr int kUnit = 64;            // columns of a wave's unit of the results
constexpr int kCols = kUnit / 16;    // operations of a unit

// The results of 16 rows by a unit's columns go through the wave's LDS, so that
// a load of base and a store cover whole lines of a row: the
// operation leaves a row's results with four lanes (64-byte pieces, half as fast).
// Chunks are four floats; bf16 rows take two for a lane's eight columns.
template <class T>
struct Bounce {
  static constexpr int kVec = 16 / (int)sizeof(T);                 // columns of a lane's load
  static constexpr int kPieces = kUnit / kVec;                     // of a row
  static constexpr int kRows = 64 / kPieces, kPasses = kTile / kRows;
  static constexpr int kHalves = sizeof(T) == 2 ? 2 : 1;
  static constexpr int kBytes = kTile * kUnit * 4;
  v4f* lds;

  __device__ __forceinline__ v4f& at(int half, int row, int piece) const {
    return lds[(half * kTile + row) * kPieces + (piece ^ (row & (kPieces - 1)))];
  }
};

// The work-group's columns [begin, end) of its rows' results.  A wave takes units
// of columns: its part of the adapter (blocks of 32 ranks, STEPS of them at a
// time) stays in registers for all tiles of rows where it is KEPT there.
template <class T, int STEPS, bool KEPT, bool ACROSS, int TT>
__device__ __forceinline__ void expand_rows(const RowsParams& p, const T* w, bool live, const Rows& rows,
                                            const uint8_t* s_hidden, uint8_t* s_bounce, int begin, int end) {
  using B = Bounce<T>;
  constexpr int kRanks = 32;
  constexpr int kLoads = sizeof(T) == 2 ? 1 : 2;                   // 16 bytes of a column's (ACROSS: a rank's) 32 ranks
  const int lane = threadIdx.x & 63, l = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int tiles = (rows.count + kTile - 1) / kTile;
  const B bounce{reinterpret_cast<v4f*>(s_bounce + wave * B::kBytes)};
  const int pass_row = lane / B::kPieces, piece = lane % B::kPieces;
  const RowMatrix<T> base_rows(p.base, p.M, p.O);
  const int pitch = hidden_pitch<T>(p.R);
  const int blocks = live ? (p.R + kRanks * STEPS - 1) / (kRanks * STEPS) : 0;
  for (int o0 = begin + kUnit * wave; o0 < end; o0 += kUnit * kWaves) {
    const int o = o0 + B::kVec * piece;
    // the base of all tiles, so that much is on its way
    v4u base[TT][B::kPasses];
    const auto row_of = [&](int t, int k) {
      const int i = kTile * t + B::kRows * k + pass_row;
      return i < rows.count && o < p.O ? rows.row(i) : -1;
    };
#pragma unroll
    for (int t = 0; t < TT; ++t)
#pragma unroll
      for (int k = 0; k < B::kPasses; ++k) base[t][k] = v4u{0, 0, 0, 0};
    if (p.base && o0 + kUnit <= p.O) {
#pragma unroll
      for (int t = 0; t < TT; ++t)
#pragma unroll
        for (int k = 0; k < B::kPasses; ++k)
          if (t < tiles) __builtin_memcpy(&base[t][k], base_rows.data + (size_t)max(row_of(t, k), 0) * p.O + o, 16);
    } else if (p.base) {
#pragma unroll
      for (int t = 0; t < TT; ++t)
#pragma unroll
        for (int k = 0; k < B::kPasses; ++k)
          if (t < tiles) base[t][k] = base_rows.chunk(max(row_of(t, k), 0), o);
    }
    // bf16: lane group g holds ranks 8 g .. of a block; float: ranks 4 i + g of
    // it (ACROSS), or 16 i + 4 g .. (two loads).  Past R h is 0, and meets
    // elements of the same columns.
    v4u wv[STEPS][sizeof(T) == 2 ? kCols : ACROSS ? 8 : kCols * kLoads];     // ACROSS: of columns 4 l + j
    const auto load_w = [&](int block) {
#pragma unroll
      for (int s = 0; s < STEPS; ++s) {
        const int rank0 = kRanks * (STEPS * block + s);
        if constexpr (sizeof(T) == 2 && ACROSS) {
          // lane l reads four columns, which four operations share
          v2u from[8];
#pragma unroll
          for (int i = 0; i < 8; ++i)
            from[i] = *reinterpret_cast<const v2u*>(w + (size_t)min(rank0 + 8 * g + i, p.R - 1) * p.O +
                                                    min(o0 + 4 * l, p.O - 4));
          turn(from, wv[s]);
        } else if constexpr (ACROSS) {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            wv[s][i] = *reinterpret_cast<const v4u*>(w + (size_t)min(rank0 + 4 * i + g, p.R - 1) * p.O +
                                                     min(o0 + 4 * l, p.O - 4));
        } else {
#pragma unroll
          for (int j = 0; j < kCols; ++j) {
            // bf16: pairs of operations whose results give a lane eight neighbours
            const int at = min(o0 + (sizeof(T) == 2 ? 32 * (j / 2) + 8 * (l >> 2) + 4 * (j % 2) + (l & 3) : 16 * j + l),
                               p.O - 1);
#pragma unroll
            for (int i = 0; i < kLoads; ++i)
              wv[s][kLoads * j + i] = *reinterpret_cast<const v4u*>(
                  w + (size_t)at * p.R + min(rank0 + (sizeof(T) == 2 ? 8 * g : 16 * i + 4 * g), p.R - 16 / (int)sizeof(T)));
          }
        }
      }
    };
    // acc[j]: column(j, i) of row l of the tile
    const auto multiply = [&](int t, int block, v4f (&acc)[kCols]) {
      const uint8_t* const h_row = s_hidden + (kTile * t + l) * pitch;
#pragma unroll
      for (int s = 0; s < STEPS; ++s) {
        const int rank0 = kRanks * (STEPS * block + s);
        if (rank0 >= p.R) break;
        if constexpr (sizeof(T) == 2) {
          const int r = rank0 + 8 * g, at = min(r, p.R - 8);
#pragma unroll
          for (int d = 0; d < 2; ++d) {          // high and low parts
            v4u h = *reinterpret_cast<const v4u*>(h_row + d * (TT * kTile) * pitch + 2 * at);
            if (r >= p.R) h = v4u{0, 0, 0, 0};
#pragma unroll
            for (int j = 0; j < kCols; ++j) acc[j] = multiply_bf16(wv[s][j], h, acc[j]);
          }
        } else if constexpr (ACROSS) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int r = rank0 + 4 * i + g;
            float h = *reinterpret_cast<const float*>(h_row + 4 * min(r, p.R - 1));
            h = r < p.R ? h : 0.0f;
#pragma unroll
            for (int j = 0; j < kCols; ++j)
              acc[j] = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(wv[s][i][j]), h, acc[j], 0, 0, 0);
          }
        } else {
#pragma unroll
          for (int i = 0; i < kLoads; ++i) {
            const int r = rank0 + 16 * i + 4 * g;
            v4f h = *reinterpret_cast<const v4f*>(h_row + 4 * min(r, p.R - 4));
            if (r >= p.R) h = v4f{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int j = 0; j < kCols; ++j)
#pragma unroll
              for (int e = 0; e < 4; ++e)
                acc[j] = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(wv[s][kLoads * j + i][e]), h[e], acc[j], 0, 0, 0);
          }
        }
      }
    };
    if constexpr (KEPT) load_w(0);
#pragma unroll
    for (int t = 0; t < TT; ++t) {
      if (t >= tiles) continue;
      v4f acc[kCols] = {};
      if constexpr (KEPT) {
        if (live) multiply(t, 0, acc);
      } else {
        for (int block = 0; block < blocks; ++block) {
          load_w(block);
          multiply(t, block, acc);
        }
      }
      wave_sync();
      if constexpr (ACROSS) {
        // column(j, i) = 4 (4 g + i) + j
#pragma unroll
        for (int i = 0; i < 4; ++i)
          bounce.at(sizeof(T) == 2 ? i % 2 : 0, l, sizeof(T) == 2 ? 2 * g + i / 2 : 4 * g + i) =
              v4f{acc[0][i], acc[1][i], acc[2][i], acc[3][i]};
      } else {
        // column(j, i) = 32 (j / 2) + 8 g + 4 (j % 2) + i (bf16), 16 j + 4 g + i (float)
#pragma unroll
        for (int j = 0; j < kCols; ++j) {
          if constexpr (sizeof(T) == 2) bounce.at(j % 2, l, 4 * (j / 2) + g) = acc[j];
          else bounce.at(0, l, 4 * j + g) = acc[j];
        }
      }
      wave_sync();
#pragma unroll
      for (int k = 0; k < B::kPasses; ++k) {
        const int i = B::kRows * k + pass_row;
        const v4f v = bounce.at(0, i, piece);
        if constexpr (sizeof(T) == 2) {
          const v4f u = bounce.at(1, i, piece);
          const v4u b = base[t][k];
          uint16_t r[8];
#pragma unroll
          for (int e = 0; e < 8; ++e)
            r[e] = rounded((e < 4 ? v[e % 4] : u[e % 4]) +
                           __uint_as_float(e & 1 ? b[e / 2] & 0xFFFF0000u : b[e / 2] << 16));
          put<uint16_t>(p, row_of(t, k), o, r);
        } else {
          const v4f sum = v + __builtin_bit_cast(v4f, base[t][k]);
          float r[4];
          __builtin_memcpy(r, &sum, 16);
          put<float>(p, row_of(t, k), o, r);
        }
      }
    }
  }
}

// grid: slices of the results or parts of the sum, tiles of a window, windows.
// TT: tiles of 16 rows of a work-group.
template <class T, int NR, bool ACROSS, int STAGE, int TT>
__global__ __launch_bounds__(kThreads, TT == 1 && NR < 8 && !(ACROSS && sizeof(T) == 2) ? 4 : 2) void rows_kernel(RowsParams p) {
  // the waves' sums of the first product, then the results of the second
  constexpr int kSum = STAGE == kExpand ? 0 : kSumBytes<T, NR, ACROSS>;
  constexpr int kOut = STAGE == kShrink ? 0 : kWaves * Bounce<T>::kBytes;
  __shared__ __align__(16) uint8_t s_sum[kSum > kOut ? kSum : kOut];
  __shared__ __align__(16) uint8_t s_hidden[STAGE == kShrink ? 16 : kHiddenBytes<NR, TT>];
  if constexpr (STAGE != kExpand) {
    if ((int)blockIdx.z * kWindow >= p.M) {
      for (int i = (int)(blockIdx.x + blockIdx.y * gridDim.x); i < p.n; i += (int)(gridDim.x * gridDim.y)) {
        order_rows(p.ids, p.M, p.n, i, p.order, p.offsets);
        __syncthreads();
      }
      return;
    }
  }
  const Rows rows = group_rows<TT * kTile>(p.ids, p.M, p.n, (int)blockIdx.z, (int)blockIdx.y);
  const int adapter = rows.adapter, count = rows.count;
  if (!count) return;
  const bool live = adapter >= 0;
  const size_t table = (size_t)max(adapter, 0) * p.R;
  const float scale = live && p.scales ? p.scales[adapter] : 1.0f;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int tiles = (count + kTile - 1) / kTile;
  const bool first = blockIdx.x == 0;
  // four sums of a row, complete
  const auto finish = [&](int row, int r, v4f v) {
    if (row >= count || r >= p.R) return;
    const v4f scaled = v * scale;
    if (p.hidden && first) *reinterpret_cast<v4f*>(p.hidden + (size_t)rows.row(row) * p.R + r) = ACROSS ? scaled : v;
    keep_hidden<T, TT>(s_hidden, p.R, row, r, scaled);
  };
  if constexpr (STAGE != kExpand) {
    const int steps = (p.C + kStep<T, NR, ACROSS> - 1) / kStep<T, NR, ACROSS>;
    const int split = STAGE == kShrink ? (int)blockIdx.x : 0, splits = STAGE == kShrink ? p.splits : 1;
    const int begin = (int)((int64_t)steps * split / splits), end = (int)((int64_t)steps * (split + 1) / splits);
    v4f(*const sums)[NR][64] = reinterpret_cast<v4f(*)[NR][64]>(s_sum);
    int row[TT];
#pragma unroll
    for (int t = 0; t < TT; ++t) row[t] = rows.row(min(kTile * t + (lane & 15), count - 1));
    for (int rank0 = 0; rank0 < p.R; rank0 += kRankBlock) {
      v4f acc[TT][NR] = {};
      if (live)
        shrink_rows<T, NR, ACROSS, TT>(p, static_cast<const T*>(p.shrink) + table * p.C, row, tiles, rank0, begin, end, s_sum,
                                       acc);
#pragma unroll
      for (int t = 0; t < TT; ++t) {
        if (t >= tiles) break;
        __syncthreads();
#pragma unroll
        for (int j = 0; j < NR; ++j) sums[wave][j][lane] = acc[t][j];
        __syncthreads();
        for (int i = threadIdx.x; i < NR * 64; i += kThreads) {
          const int j = i >> 6, from = i & 63, at = kTile * t + (from & 15), r = rank0 + 16 * j + 4 * (from >> 4);
          v4f v = sums[0][j][from];
          for (int k = 1; k < kWaves; ++k) v += sums[k][j][from];
          if constexpr (STAGE == kBoth) {
            finish(at, r, v);
          } else if (at < count && r < p.R) {
            *reinterpret_cast<v4f*>(p.partial + ((size_t)split * p.M + rows.row(at)) * p.R + r) = v;
          }
        }
      }
      __syncthreads();
    }
  } else {
    for (int i = threadIdx.x; i < TT * kTile * p.R / 4; i += kThreads) {
      const int row = i / (p.R / 4), r = 4 * (i % (p.R / 4));
      if (row >= count) break;
      const float* const at = p.partial + (size_t)rows.row(row) * p.R + r;
      v4f v = *reinterpret_cast<const v4f*>(at);
      for (int k = 1; k < p.splits; ++k) v += *reinterpret_cast<const v4f*>(at + (size_t)k * p.M * p.R);
      finish(row, r, v);
    }
    __syncthreads();
  }
  if constexpr (STAGE != kShrink) {
    if (!p.out) return;
    const int begin = (int)blockIdx.x * p.slice, end = min(p.O, begin + p.slice);
    const T* const w = static_cast<const T*>(p.expand) + table * p.O;
    // two blocks of 32 ranks and 64 registers are kept at most
    constexpr int kSteps = TT > 1 && NR == 4 ? 2 : 1;
    expand_rows<T, kSteps, (TT > 1 && NR <= 4), ACROSS, TT>(p, w, live, rows, s_hidden, s_sum, begin, end);
  }
}

// Kernels by type, tiles of 16 ranks in a pass, and direction.
template <class T, bool ACROSS, int STAGE, int TT>
const void* pick(int R) {
  if (R > 64) return reinterpret_cast<const void*>(&rows_kernel<T, 8, ACROSS, STAGE, TT>);
  if (R > 32) return reinterpret_cast<const void*>(&rows_kernel<T, 4, ACROSS, STAGE, TT>);
  if (R > 16) return reinterpret_cast<const void*>(&rows_kernel<T, 2, ACROSS, STAGE, TT>);
  return reinterpret_cast<const void*>(&rows_kernel<T, 1, ACROSS, STAGE, TT>);
}
template <int STAGE, int TT>
hipError_t launch(RowsParams p, int blocks, bool f32, bool across, hipStream_t stream) {
  const void* const kernel = f32 ? across ? pick<float, true, STAGE, TT>(p.R) : pick<float, false, STAGE, TT>(p.R)
                                 : across ? pick<uint16_t, true, STAGE, TT>(p.R) : pick<uint16_t, false, STAGE, TT>(p.R);
  void* args[] = {&p};
  const dim3 grid((unsigned)blocks, (unsigned)window_tiles(p.M, p.n, p.ids != nullptr, TT * kTile),
                  (unsigned)((p.M + kWindow - 1) / kWindow + (STAGE != kExpand && p.order ? 1 : 0)));
  return hipLaunchKernel(kernel, grid, dim3(kThreads), args, 0, stream);
}

// Work-groups along the results: as many as make `fill` of them, of one unit of
// each wave at least.
int slices_for(const RowsParams& p, int tiles, int fill, int& slice) {
  constexpr int unit = kWaves * kUnit;
  const int most = p.out ? (p.O + unit - 1) / unit : 1;
  int s = (fill + tiles - 1) / tiles;
  s = s > most ? most : s;
  slice = ((p.O + s - 1) / s + unit - 1) / unit * unit;
  return p.out ? (p.O + slice - 1) / slice : 1;
}

// Parts of the long sum.
int splits_for(const RowsParams& p, int tiles, int fill) {
  const int steps = (p.C + 511) / 512;
  int s = fill / tiles;
  s = s > kMaxSplits ? kMaxSplits : s;
  s = s > steps ? steps : s;
  return s < 1 ? 1 : s;
}

hipError_t launch_rows(RowsParams p, bool f32, bool across, hipStream_t stream) {
  if (p.M >= kLargeBatch) {
    const int tiles = (p.M + 63) / 64;
    p.splits = splits_for(p, tiles, kFill);
    const hipError_t e = launch<kShrink, 4>(p, p.splits, f32, across, stream);
    if (e != hipSuccess) return e;
    const int slices = slices_for(p, tiles, 2 * kFill, p.slice);
    return launch<kExpand, 4>(p, slices, f32, across, stream);
  }
  const int tiles = (p.M + kTile - 1) / kTile;
  const int slices = slices_for(p, tiles, kFill / 2, p.slice);
  p.splits = splits_for(p, tiles, kFill);
  // One launch while a work-group reads an adapter's matrix sooner than a second
  // launch starts.  Forward to 4096 columns, three adapters, one launch against two:
  // 24 KB (bf16, rank 8, of 1544) 8.6 us against 11.3 for one row, 8.3 against 11.0
  // for 333; 128 KB (rank 16 of 4096) 10.1 against 12.3, 13.1 against 11.7; 224 KB
  // (rank 16 of 7168) 13.2 against 13.0, 17.8 against 14.3; 448 KB (rank 32) 19.2
  // against 14.5, 23.7 against 15.1.  The rule asks nothing about rows: 1000 of them
  // are better off with two launches from 128 KB on (22 against 16; 224 KB 32
  // against 18).
  const size_t table = (size_t)p.R * p.C * (f32 ? 4 : 2);
  if (p.splits == 1 || table <= (1u << 18)) return launch<kBoth, 1>(p, slices, f32, across, stream);
  const hipError_t e = launch<kShrink, 1>(p, p.splits, f32, across, stream);
  return e != hipSuccess ? e : launch<kExpand, 1>(p, slices, f32, across, stream);
}

// The parts of the hidden sums: M rows, or while there are several parts at
// most kFill tiles of 64 rows in all.
size_t hidden_bytes(int64_t M, int64_t R) {
  const int64_t several = M * kMaxSplits < kFill * 64 ? M * kMaxSplits : kFill * 64;
  const size_t rows = (size_t)(M > several ? M : several);
  return (rows * (size_t)R * 4 + 255) / 256 * 256;
}

}  // namespace

size_t adapter_workspace(int64_t M, int64_t N, int64_t K, int64_t R, int64_t n) {
  return hidden_bytes(M, R) + (size_t)M * R * 4 / 256 * 256 + 256 + adapter_grad_workspace(M, N, K, R, n);
}

hipError_t launch_adapter(const AdapterParams& p, hipStream_t stream) {
  return launch_rows({p.x, p.a, p.b, p.ids, p.scales, p.base, p.out, p.hidden, p.partial, p.M, p.K, p.N, p.R, p.n, 0, 0,
                      nullptr, nullptr},
                     p.xf32, false, stream);
}

hipError_t launch_adapter_backward(const AdapterBackwardParams& p, hipStream_t stream) {
  float* const g = p.partial + hidden_bytes(p.M, p.R) / 4;
  float* const rest = g + (size_t)p.M * p.R / 64 * 64 + 64;
  int32_t* const order = reinterpret_cast<int32_t*>(rest);
  int32_t* const offsets = order + ((size_t)p.M + 63) / 64 * 64;
  const bool grads = p.d_a || p.d_b, sorting = p.ids && grads;
  if (p.d_x || p.d_a) {
    const hipError_t e = launch_rows({p.d_out, p.b, p.a, p.ids, p.scales, p.base, p.d_x, p.d_a ? g : nullptr, p.partial,
                                      p.M, p.N, p.K, p.R, p.n, 0, 0, sorting ? order : nullptr, offsets},
                                     p.xf32, true, stream);
    if (e != hipSuccess) return e;
  }
  if (!grads) return hipSuccess;
  AdapterGradParams q{};
  q.x = p.x;
  q.d_out = p.d_out;
  q.g = g;
  q.hidden = p.hidden;
  q.ids = p.ids;
  q.scales = p.scales;
  q.d_a = p.d_a;
  q.d_b = p.d_b;
  q.order = order;
  q.offsets = offsets;
  q.sorted = p.d_x || p.d_a;
  q.parts = reinterpret_cast<float*>(offsets + ((size_t)p.n + 64) / 64 * 64);
  q.M = p.M;
  q.N = p.N;
  q.K = p.K;
  q.R = p.R;
  q.n = p.n;
  q.xf32 = p.xf32;
  return launch_adapter_grad(q, stream);
}

}  // namespace q4
