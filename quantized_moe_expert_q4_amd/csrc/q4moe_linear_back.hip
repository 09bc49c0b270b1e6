// Gradient of the input of the linear with 4-bit weights and group scales:
// d_x[m][k] = sum_n d_out[m][n] W[n][k].
//
// A work-group computes BM tokens by COLS columns k.  A step covers 128 bytes of
// the tokens' rows (64 values n in bf16, 32 in float).  Weights run along k in
// memory and along n in the product, so a thread unpacks the words of neighbouring
// rows n at one place k and writes them side by side: a tile in LDS is [row][8
// chunks of 16 bytes], tokens and columns alike, and a matrix operand is one
// 16-byte read.
//
// bf16, more than 128 tokens: 256 x 256, eight waves of 128 x 64, which fills the
// registers (128 of them sums).  Per step and CU the operations take 2048 cycles,
// the LDS as many (counters: each is busy for 37% of the kernel's time, the LDS for
// 37% of that with conflicts, see place()), unpacking 960 of each SIMD's vector
// unit; what counts is that they overlap.  4096 tokens through 14336 x 7168: 1420
// us with 128 x 128 and the loads' branches and conversions between the steps, 1212
// without those, 1064 with 256 x 256, 900 with the next step staged between a
// step's operations (936 TFLOP/s; a library product of bf16 matrices reaches 1191
// here, 1385 elsewhere).
// Its 448 tiles are 1.75 rounds of the 256 CUs, so an eighth of the time is idle.
// 64 tokens 42 us.  Float rows take F32 operations, 1024 tokens 1.87 ms (112
// TFLOP/s; a library product of F32 matrices reaches 152); 77 tokens through 6147 x
// 4104 take 70 us and 6 to join, a tile of 128 rows being filled to three fifths.
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

constexpr int kChunks = 8;           // 16-byte chunks of a tile's row
constexpr int kJoinThreads = 256;
constexpr int kCus = 256;
constexpr int kMaxSplits = 16;       // parts of n that work-groups share
constexpr int kFill = 512;           // work-groups that fill the device: no more parts than give so many

// Place of a row's chunk: the eight chunks change places from row to row and
// from eight rows to the next, so that the weights' writes (rows eight apart) do
// not meet in a bank.  The operands' reads do: they take one chunk of 16 rows KT
// or MT (four or eight, in the largest tile) apart, all odd or all even ones,
// which lie in one half of the banks, so that they meet at least twice there.
// (Tokens and columns are dealt out to the operations in that order so that a
// lane's results are neighbours.)
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

template <bool FIRST, class A, class B>
struct Pick {
  typedef A type;
};
template <class A, class B>
struct Pick<false, A, B> {
  typedef B type;
};

// T: the type of d_out as stored (uint16_t: bf16).  BM tokens by COLS columns, by
// WAVES waves, WM of them along the tokens.
template <class T, int BM, int COLS, int WAVES, int WM, bool AFF, bool SF>
__global__ __launch_bounds__(64 * WAVES, 2) void linear_back_kernel(LinearBackParams p, int splits) {
  constexpr int kThreads = 64 * WAVES, kCols = COLS;
  constexpr int kVec = 16 / sizeof(T), kStep = kChunks * kVec;
  constexpr int kWords = kStep * (COLS / 8) / kThreads;            // words of a thread: neighbouring rows n
  constexpr int kLanes = kVec / kWords;                            // threads that fill a chunk
  constexpr int MT = BM / WM / 16, KT = kCols / (WAVES / WM) / 16; // 16 x 16 tiles of a wave
  constexpr int kSpan = kThreads / kChunks;                        // token rows that the threads load at a time
  constexpr int kRows = BM / kSpan ? BM / kSpan : 1;               // token chunks of a thread
  static_assert(kWords == 1 || kWords == 2 || kWords == 4, "a thread's weights at a column are written at once");
  // two buffers, apart so that a store to one may pass a load from the other
  __shared__ v4u s_d0[BM * kChunks], s_d1[BM * kChunks], s_w0[kCols * kChunks], s_w1[kCols * kChunks];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave % WM, wk = wave / WM;
  const int k0 = (int)blockIdx.x * kCols, m0 = (int)blockIdx.y * BM;
  const int steps = (p.N + kStep - 1) / kStep;
  const int begin = (int)((int64_t)steps * blockIdx.z / splits), end = (int)((int64_t)steps * (blockIdx.z + 1) / splits);

  // a thread's place among the weights: words of rows nq * kWords .. at the eight
  // columns kb; loads past the matrix give 0
  const int kb = tid / kLanes % (kCols / 8), sub = tid % kLanes, chunk = tid / (kLanes * (kCols / 8));
  const int nq = sub + kLanes * chunk;
  const bool col_in = k0 + 8 * kb < p.K;
  const uint32_t w_pitch = (uint32_t)p.K / 2, s_pitch = (uint32_t)p.groups * (SF ? 4 : 2);
  const __amdgpu_buffer_rsrc_t w_src = make_rsrc(p.w, (uint32_t)p.N * w_pitch);
  const __amdgpu_buffer_rsrc_t s_src = make_rsrc(p.scales, (uint32_t)p.N * s_pitch);
  const __amdgpu_buffer_rsrc_t b_src = make_rsrc(p.biases, AFF ? (uint32_t)p.N * s_pitch : 0u);
  const uint32_t w_col = (uint32_t)(k0 / 2 + 4 * kb), s_col = (uint32_t)((k0 + 8 * kb) / p.group) * (SF ? 4 : 2);
  const auto load_scale = [](__amdgpu_buffer_rsrc_t src, uint32_t at) {
    if constexpr (SF) return __builtin_amdgcn_raw_buffer_load_b32(src, (int)at, 0, 0);
    else return (uint32_t)__builtin_amdgcn_raw_buffer_load_b16(src, (int)at, 0, 0);
  };
  const auto scale_value = [](uint32_t u) { return __uint_as_float(SF ? u : u << 16); };
  const RowMatrix<T> d_out(p.d_out, p.M, p.N);
  // Where a thread's token rows start, from the tile's first on (32 bits at 256
  // tokens, for the registers: the host keeps N below 2^22 there).  Rows past the
  // last one repeat it.
  using Offset = typename Pick<BM == 256, uint32_t, size_t>::type;
  const T* const d_tile = d_out.data + (size_t)m0 * p.N;
  const auto d_row = [&](int i) { return min(tid / kChunks + kSpan * i, p.M - 1 - m0); };
  Offset d_at[kRows];
#pragma unroll
  for (int i = 0; i < kRows; ++i) d_at[i] = (Offset)d_row(i) * (Offset)p.N + (Offset)((tid % kChunks) * kVec);

  // A step as loaded: nothing is done with a value before it is staged, so that
  // no load is waited for here.
  struct Fetched {
    v4u d[kRows];
    uint32_t w[kWords], s[kWords], b[kWords];
  };
  auto fetch_weights = [&](int n0, Fetched& f) {
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
      const uint32_t n = (uint32_t)(n0 + nq * kWords + i);
      const bool in = col_in && n < (uint32_t)p.N;
      const uint32_t w_off = in ? n * w_pitch + w_col : kOffNone, s_off = in ? n * s_pitch + s_col : kOffNone;
      f.w[i] = __builtin_amdgcn_raw_buffer_load_b32(w_src, (int)w_off, 0, 0);
      f.s[i] = load_scale(s_src, s_off);
      if constexpr (AFF) f.b[i] = load_scale(b_src, s_off);
    }
  };
  auto fetch = [&](int step, Fetched& f) {             // a step whose rows are all there
#pragma unroll
    for (int i = 0; i < kRows; ++i) __builtin_memcpy(&f.d[i], d_tile + step * kStep + d_at[i], 16);
    fetch_weights(step * kStep, f);
  };
  auto fetch_end = [&](int step, Fetched& f) {
#pragma unroll
    for (int i = 0; i < kRows; ++i) f.d[i] = d_out.chunk(m0 + d_row(i), step * kStep + (tid % kChunks) * kVec);
    fetch_weights(step * kStep, f);
  };
  auto stage = [&](int buf, const Fetched& f) {
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const int row = tid / kChunks + kSpan * i;
      if (BM >= kSpan || row < BM) (buf ? s_d1 : s_d0)[place(row, tid % kChunks)] = f.d[i];
    }
    uint32_t half[kWords][2];            // the even and the odd columns' nibbles, a byte each
    float scale[kWords], off[kWords];
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
      half[i][0] = f.w[i] & 0x0F0F0F0Fu;
      half[i][1] = (f.w[i] >> 4) & 0x0F0F0F0Fu;
      scale[i] = scale_value(f.s[i]);
      off[i] = AFF ? scale_value(f.b[i]) : -8.0f * scale[i];
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      // (q - 8) s, or q s + b, rounded once (to F32, and for bf16 once more: as a
      // bf16 matrix of these weights would hold them; two bf16 parts would take
      // twice the operations to bring the error against 64 bits from 2.1e-3 to the
      // 1.7e-3 of the output's own rounding)
      float v[kWords];
#pragma unroll
      for (int i = 0; i < kWords; ++i)
        v[i] = __builtin_fmaf((float)((half[i][j & 1] >> (8 * (j >> 1))) & 0xFFu), scale[i], off[i]);
      T r[kWords];
#pragma unroll
      for (int i = 0; i < kWords; ++i) {
        if constexpr (sizeof(T) == 2) r[i] = __builtin_bit_cast(uint16_t, (__bf16)v[i]);
        else r[i] = v[i];
      }
      const int row = 8 * kb + j;
      uint8_t* const to = reinterpret_cast<uint8_t*>(&(buf ? s_w1 : s_w0)[place(row, chunk)]) + sub * (kWords * sizeof(T));
      __builtin_memcpy(__builtin_assume_aligned(to, kWords * sizeof(T)), r, sizeof(r));
    }
  };

  v4f acc[KT][MT] = {};
  // Operation t of a wave takes the rows first + TILES l + t: their chunk's place
  // is that of t = 0 with bits of t turned over (see place), so that one register
  // holds all addresses.  It is hidden from the compiler, which would keep each.
  const auto operand = [&](const v4u* tile, uint32_t at, int t, int h) {
    return *reinterpret_cast<const v4u*>(reinterpret_cast<const uint8_t*>(tile) + (at ^ (16u * (uint32_t)(t ^ (4 * h)))) +
                                         16 * kChunks * t);
  };
  uint32_t w_read = 16u * (uint32_t)place(wk * (16 * KT) + KT * (lane & 15), lane >> 4);
  uint32_t d_read = 16u * (uint32_t)place(wm * (16 * MT) + MT * (lane & 15), lane >> 4);
  auto multiply_half = [&](int buf, int h) {
    asm("" : "+v"(w_read), "+v"(d_read));
    v4u a[KT], b[MT];
#pragma unroll
    for (int t = 0; t < KT; ++t) a[t] = operand(buf ? s_w1 : s_w0, w_read, t, h);
#pragma unroll
    for (int t = 0; t < MT; ++t) b[t] = operand(buf ? s_d1 : s_d0, d_read, t, h);
#pragma unroll
    for (int t = 0; t < KT; ++t)
#pragma unroll
      for (int u = 0; u < MT; ++u) acc[t][u] = multiply<T>(a[t], b[u], acc[t][u]);
  };
  // A step is staged in the middle of the one before it, while its operations
  // run, and the one after it fetched into the same registers.  One barrier a
  // step: past it every wave has read the buffer that is written next.
  const int whole = min(end, p.N / kStep);             // past it at most one step, the rows' end
  const auto fetch_any = [&](int step, Fetched& f) {
    if (step < whole) fetch(step, f);
    else if (step < end) fetch_end(step, f);
  };
  Fetched next;
  fetch_any(begin, next);
  stage(0, next);
  fetch_any(begin + 1, next);
  __syncthreads();
  for (int step = begin; step < end; step += 2) {
#pragma unroll
    for (int buf = 0; buf < 2; ++buf) {
      if (step + buf >= end) break;
      multiply_half(buf, 0);
      stage(1 - buf, next);
      if (step + buf + 2 < whole) fetch(step + buf + 2, next);
      else if (step + buf + 2 < end) fetch_end(step + buf + 2, next);
      multiply_half(buf, 1);
      __syncthreads();
    }
  }
  // acc[t][u][i]: column KT (4 (lane / 16) + i) + t of token MT (lane % 16) + u
#pragma unroll
  for (int u = 0; u < MT; ++u) {
    const int m = m0 + wm * (16 * MT) + MT * (lane & 15) + u;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int k = k0 + wk * (16 * KT) + KT * (4 * (lane >> 4) + i);
      float v[KT];
#pragma unroll
      for (int t = 0; t < KT; ++t) v[t] = acc[t][u][i];
      if (m >= p.M || k >= p.K) continue;
      const size_t at = (size_t)m * p.K + k;
      if (splits > 1) {
        float* const to = p.partials + (size_t)blockIdx.z * p.M * p.K + at;
        __builtin_memcpy(__builtin_assume_aligned(to, 4 * (KT < 4 ? KT : 4)), v, sizeof(v));
      } else {
        T r[KT];
#pragma unroll
        for (int t = 0; t < KT; ++t) {
          if constexpr (sizeof(T) == 2) r[t] = __builtin_bit_cast(uint16_t, (__bf16)v[t]);
          else r[t] = v[t];
        }
        constexpr int kBytes = KT * (int)sizeof(T);
        __builtin_memcpy(__builtin_assume_aligned(static_cast<T*>(p.d_x) + at, kBytes < 16 ? kBytes : 16), r, sizeof(r));
      }
    }
  }
}

// Adds up the parts of n, in order.
template <class T>
__global__ __launch_bounds__(kJoinThreads) void linear_back_join_kernel(LinearBackParams p, int splits) {
  const size_t all = (size_t)p.M * p.K / 4;
  const size_t i = (size_t)blockIdx.x * kJoinThreads + threadIdx.x;
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

template <class T, int BM, int COLS, int WAVES, int WM>
const void* pick(const LinearBackParams& p) {
  if (p.biases)
    return p.scale_f32 ? reinterpret_cast<const void*>(&linear_back_kernel<T, BM, COLS, WAVES, WM, true, true>)
                       : reinterpret_cast<const void*>(&linear_back_kernel<T, BM, COLS, WAVES, WM, true, false>);
  return p.scale_f32 ? reinterpret_cast<const void*>(&linear_back_kernel<T, BM, COLS, WAVES, WM, false, true>)
                     : reinterpret_cast<const void*>(&linear_back_kernel<T, BM, COLS, WAVES, WM, false, false>);
}

// Parts of n for `tiles` work-groups of `steps` steps each: as many as give the
// least time, a step of all CUs taking 2 us (measured: 4096 tokens through 14336 x
// 7168) and the parts' way to memory and back 4 bytes a ps.
int large_splits(const LinearBackParams& p, int tiles, int steps) {
  int best = 1;
  double least = 0.0;
  for (int s = 1; s <= kMaxSplits && (s == 1 || (s * tiles <= kFill && 4 * s <= steps)); ++s) {
    const int rounds = (s * tiles + kCus - 1) / kCus;
    const double parts = s > 1 ? 3.0 + (2 * s + 1) * (double)p.M * p.K * 4e-6 / 4.0 : 0.0;
    const double us = rounds * ((steps + s - 1) / s) * 2.0 + parts;
    if (s == 1 || us < least) {
      best = s;
      least = us;
    }
  }
  return best;
}

template <class T>
hipError_t run(const LinearBackParams& p, hipStream_t stream) {
  int bm = p.M <= 16 ? 16 : p.M <= 32 ? 32 : p.M <= 64 ? 64 : 128, cols = 128;
  const void* kernel = bm == 16   ? pick<T, 16, 128, 4, 1>(p)
                       : bm == 32 ? pick<T, 32, 128, 4, 1>(p)
                       : bm == 64 ? pick<T, 64, 128, 4, 2>(p)
                                  : pick<T, 128, 128, 4, 2>(p);
  if constexpr (sizeof(T) == 2) {
    if (p.M > 128 && p.N < (1 << 22)) {
      bm = cols = 256;
      kernel = pick<T, 256, 256, 8, 2>(p);
    }
  }
  const int tiles_k = (p.K + cols - 1) / cols, tiles_m = (p.M + bm - 1) / bm, tiles = tiles_k * tiles_m;
  const int steps = (int)(((int64_t)p.N * (int)sizeof(T) + 127) / 128);
  int splits;
  if (bm == 256) {
    splits = large_splits(p, tiles, steps);
  } else {
    splits = kFill / tiles;
    splits = splits > kMaxSplits ? kMaxSplits : splits;
    splits = splits > steps ? steps : splits;
    splits = splits < 1 ? 1 : splits;
  }
  LinearBackParams q = p;
  void* args[] = {&q, &splits};
  const hipError_t e = hipLaunchKernel(kernel, dim3((unsigned)tiles_k, (unsigned)tiles_m, (unsigned)splits),
                                       dim3(bm == 256 ? 512 : 256), args, 0, stream);
  if (e != hipSuccess || splits == 1) return e;
  const size_t all = (size_t)p.M * p.K / 4;
  return hipLaunchKernel(reinterpret_cast<const void*>(&linear_back_join_kernel<T>),
                         dim3((unsigned)((all + kJoinThreads - 1) / kJoinThreads)), dim3(kJoinThreads), args, 0, stream);
}

}  // namespace

// Room for the parts of n: there are at most kMaxSplits, and more than one only
// while all work-groups together are no more than kFill, of 256 x 256 at most.
size_t linear_back_partial_bytes(int64_t M, int64_t K) {
  const size_t parts = (size_t)M * (size_t)K * 4 * kMaxSplits, most = (size_t)kFill * 256 * 256 * 4;
  return ((parts < most ? parts : most) + 255) / 256 * 256;
}

hipError_t launch_linear_backward(const LinearBackParams& p, hipStream_t stream) {
  return p.xf32 ? run<float>(p, stream) : run<uint16_t>(p, stream);
}

}  // namespace q4
