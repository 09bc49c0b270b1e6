// Kernel of the linear with 4-bit weights and group scales (one instantiation
// file per group size includes this).
//
// A work-group of eight waves owns T tiles of 16 weight rows for each of its
// 8 / S row sets; the S waves of a set split K in units of 256 weights (128
// bytes of a row) and join their F32 sums through LDS at the end.  A
// matrix-core operation (16x16x32 bf16, F32 accumulation) takes 16 tokens as
// rows and 16 weight rows as columns, so one token costs what sixteen do, and
// the weights are unpacked once for up to 16 MT tokens.
//
// Staging.  Every wave needs the tokens as matrix operands, and a few bytes of
// each row's scales a unit: the work-group brings both to LDS in loads of whole
// lines (a wave's own scale reads moved a cache line each: the 131072-row head
// below took 67 us so; token reads with 16 lanes on 16 rows kept 64 tokens at
// 70 us).  Weights go straight to registers, a unit or two ahead.
//
// What bounds it (one call, bf16 unless said).  One token: the weight stream,
// 131072 x 4096 with biases in 50 us (5.7 TB/s; its vector instructions alone
// take about 39); 14336 x 7168 in 15.  One float token through the former in 80
// us: its exact unpacking takes the vector units more than twice the work.
// Many: 64 tokens of 14336 x 7168 in 41 to 43 us, where a step's vector
// instructions (3600 cycles a SIMD), LDS reads (2800) and matrix operations
// (1400) overlap little at two waves a SIMD; 16 tokens 19 us, 64 float tokens 65.
// More are taken 64 (float: 32) at a time and unpack the weights each time: 4096
// tokens take 2.1 ms, which the matrix operations alone would take 0.6 of.  Few
// rows: steps of about 3 us each, bound by latency.
//
// Unpacking.  Bits 3..6 of a bf16 in [16, 32) count in steps of one: a nibble
// q moved there under the bit pattern of 16 is the number 16 + q, exactly, two
// of them per shift and and-or.  The offset is taken off by one further matrix
// product per 32 weights, of the tokens with a constant -24 (symmetric: 16 + 8)
// or -16 (affine), shared by the row tiles; it starts the sums of every group:
//   sum (16 + q) x - 24 sum x = sum (q - 8) x
//   s sum q x + b sum x = s (sum (16 + q) x - 16 sum x) - (b / 16) (-16 sum x)
// Group sums are scaled in F32 into the running total, so products and the
// scale are exact up to F32 rounding.  Float activations enter as three bf16
// parts whose sum is the float (8 bits each), three products per weight, and
// meet the exact (q - 8) / 16 (20 operations for 8 weights instead of 8):
//   16 s sum (q - 8) / 16 x + (b + 8 s) sum x
//
// Every variant adds a token's products in the same order (K in eight segments,
// joined in one tree), so its result does not depend on the number of tokens.
#pragma once
#include "q4moe_device.h"
#include "q4moe_layer.h"

namespace q4 {

typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));

__device__ __forceinline__ v4f mfma_bf16(const v4u a, const v4u b, const v4f c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, a), __builtin_bit_cast(v8bf, b), c, 0, 0, 0);
}

// Exchanges lanes 32..63 of a with lanes 0..31 of b / odd 16-lane rows of a with even ones of b.
__device__ __forceinline__ void swap32(uint32_t& a, uint32_t& b) {
  const auto r = __builtin_amdgcn_permlane32_swap(a, b, false, false);
  a = r[0];
  b = r[1];
}
__device__ __forceinline__ void swap16(uint32_t& a, uint32_t& b) {
  const auto r = __builtin_amdgcn_permlane16_swap(a, b, false, false);
  a = r[0];
  b = r[1];
}

// One unit of a 16-row tile as loaded: lane 16 q + 8 h + r holds the 16 bytes
// (a piece, 32 weights) 4 h + q of the unit's eight, of rows r (a) and 8 + r
// (b), so that every load instruction covers whole lines.
struct UnitW {
  v4u a, b;
};

// The unit as eight matrix operands: word[o] of lane 16 q + n holds weights
// 32 o + 8 q .. + 8 of row n.  Lanes 8 apart trade rows for pieces, then a 4x4
// transpose over the lane rows trades pieces for words.
__device__ __forceinline__ void unit_words(const UnitW& w, bool high, uint32_t (&word)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t send = high ? w.a[i] : w.b[i];
    const uint32_t got = (uint32_t)__builtin_amdgcn_mov_dpp((int)send, 0x128, 0xF, 0xF, true);  // row_ror:8
    word[i] = high ? got : w.a[i];
    word[4 + i] = high ? w.b[i] : got;
  }
#pragma unroll
  for (int h = 0; h < 8; h += 4) {
    swap32(word[h], word[h + 2]);
    swap32(word[h + 1], word[h + 3]);
    swap16(word[h], word[h + 1]);
    swap16(word[h + 2], word[h + 3]);
  }
}

// Eight nibbles as the bf16 numbers 16 + q, in the order (0,4) (1,5) (2,6)
// (3,7).  `sixteen` (0x41804180) comes in a vector register: one and-or then
// takes the mask from a scalar one.
__device__ __forceinline__ v4u unpack_word(uint32_t w, uint32_t sixteen) {
  v4u r;
  r.x = ((w << 3) & 0x00780078u) | sixteen;
  r.y = ((w >> 1) & 0x00780078u) | sixteen;
  r.z = ((w >> 5) & 0x00780078u) | sixteen;
  r.w = ((w >> 9) & 0x00780078u) | sixteen;
  return r;
}

// The same as (q - 8) / 16, exactly: float activations, whose results keep all
// their digits, would lose three bits to the offset of 16 + q.  q ^ 8 is the
// two's complement of q - 8; the conversion takes the low four bits.
__device__ __forceinline__ v4u unpack_word_exact(uint32_t w) {
  w ^= 0x88888888u;
  v4u r;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float lo = __builtin_amdgcn_cvt_off_f32_i4((int)(w >> (4 * i)));
    const float hi = __builtin_amdgcn_cvt_off_f32_i4((int)(w >> (4 * i + 16)));
    r[i] = perm(__float_as_uint(hi), __float_as_uint(lo), 0x07060302u);
  }
  return r;
}

// Eight consecutive bf16 activations in that order.
__device__ __forceinline__ v4u order_x(const v4u v) {
  v4u r;
  r.x = perm(v.z, v.x, 0x05040100u);
  r.y = perm(v.z, v.x, 0x07060302u);
  r.z = perm(v.w, v.y, 0x05040100u);
  r.w = perm(v.w, v.y, 0x07060302u);
  return r;
}

// Eight consecutive floats as bf16 parts of 8 bits each (high, middle, low), in that order.
__device__ __forceinline__ void order_split_x(const v4u lo, const v4u hi, v4u (&part)[3]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t a = lo[i], b = hi[i];
#pragma unroll
    for (int d = 0; d < 3; ++d) {
      part[d][i] = perm(b, a, 0x07060302u);
      a = __float_as_uint(__uint_as_float(a) - __uint_as_float(a & 0xFFFF0000u));
      b = __float_as_uint(__uint_as_float(b) - __uint_as_float(b & 0xFFFF0000u));
    }
  }
}

// COUNT consecutive scales in LDS, as floats.
template <int COUNT, bool F32>
__device__ __forceinline__ void read_scales(const uint8_t* at, float (&f)[COUNT]) {
  uint32_t v[F32 ? COUNT : COUNT / 2];
  __builtin_memcpy(v, __builtin_assume_aligned(at, sizeof(v) < 16 ? sizeof(v) : 16), sizeof(v));
#pragma unroll
  for (int i = 0; i < COUNT; ++i)
    f[i] = __uint_as_float(F32 ? v[i] : i & 1 ? v[i / 2] & 0xFFFF0000u : v[i / 2] << 16);
}

constexpr int kLinearWaves = 8;

// Weights of a wave in flight, in units; a chunk has as many steps.
template <bool XF, int TK>
constexpr int kLinearRing = TK * (XF ? 3 : 1) <= 4 ? 2 : 1;

// Bytes in LDS of a unit's tokens.
template <bool XF, int TK>
constexpr int kLinearUnitX = 8 * (XF ? 3 : 1) * 64 * TK;

template <bool V>
struct Bool {
  static constexpr bool value = V;
};

// What a launch chose: its first work-group along the rows, S waves along K (1,
// 2, 4 or 8), the steps of S units (powers of two) whose tokens and whose scales
// are staged in LDS together, and the bytes there of the tokens, of their sums,
// of a row's scales and of all rows' scales.
struct LinearPlan {
  int block0;
  int S, shift, log_chunk, log_scales;
  int x_bytes, xs_bytes, pitch, scale_bytes;
};

// KPG: 32-weight blocks of a group (1, 2, 4).  TK: tokens of the work-group at
// most; up to four keep one sum a lane (matrix row 4 t + i holds token t).  T:
// row tiles of a wave.  kSplit: waves along K, as the launch chooses (0, up to
// four tokens) or fixed, so that a step's staged tokens, 64 KB (float: 96 KB) at
// most, are fetched into a fixed number of registers while the step before is
// at work.  The four waves a SIMD asked for up to 16 tokens (float: 4) leave 128
// registers; ten of the two-tile variants spill 12 to 80 bytes a lane over it (the
// rule in linear_tiles takes them where they gain all the same).
template <int KPG, bool AFF, bool SF, bool XF, int TK, int T, int kSplit>
__global__ __launch_bounds__(kLinearWaves * 64, TK <= (XF ? 4 : 16) ? 4 : 2) void linear_kernel(LinearParams p, LinearPlan plan) {
  constexpr int kParts = XF ? 3 : 1;
  constexpr int kGroups = 8 / KPG;                 // groups of a unit
  constexpr int MT = TK > 16 ? TK / 16 : 1;        // tiles of 16 tokens
  constexpr int TR = TK <= 4 ? 1 : 4;              // result registers in use
  constexpr int kRing = kLinearRing<XF, TK>;
  constexpr int kUnitX = kLinearUnitX<XF, TK>, kOperandX = 64 * TK;   // bytes in LDS of a unit's tokens and of one operand
  constexpr int kScaleBytes = SF ? 4 : 2;
  constexpr int kThreads = kLinearWaves * 64;
  // tokens, their sums, scales and biases; at the end [wave][T][MT][TR][64] sums
  extern __shared__ __align__(16) uint8_t s_mem[];
  uint8_t* const s_sums = s_mem + plan.x_bytes;
  uint8_t* const s_scales = s_sums + plan.xs_bytes;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int n = lane & 15, q = lane >> 4;
  const bool high = (lane & 8) != 0;
  const int S = kSplit ? kSplit : plan.S, shift = kSplit ? __builtin_ctz(kSplit) : plan.shift;
  const int log_chunk = kSplit ? 0 : plan.log_chunk, chunk = 1 << log_chunk;
  const int ks = wave & (S - 1), set = wave >> shift, sets = kLinearWaves >> shift;
  const int wg_row0 = (plan.block0 + (int)blockIdx.x) * sets * (16 * T), row0 = wg_row0 + set * (16 * T);
  const int m0 = (int)blockIdx.y * TK;
  const int tokens = min(TK, p.M - m0);
  const int units = (p.K + 255) / 256;
  const uint32_t pitch = (uint32_t)(p.K / 2);
  const int rows = max(0, min(16 * T, p.N - row0));
  const __amdgpu_buffer_rsrc_t wsrc =
      make_rsrc(p.w + (size_t)min(row0, p.N) * pitch, (uint32_t)max(0, p.N - row0) * pitch);
  constexpr uint32_t kXBytes = XF ? 4 : 2;
  const __amdgpu_buffer_rsrc_t xsrc = make_rsrc(static_cast<const uint8_t*>(p.x) + (size_t)m0 * p.K * kXBytes,
                                                (uint32_t)tokens * (uint32_t)p.K * kXBytes);
  // the 16 bytes that hold the matrix's end may reach past it: these are loaded again in dwords before their use
  const bool ragged = p.K % 32 != 0 && row0 + 16 * T >= p.N;
  uint32_t sixteen = 0x41804180u;
  asm("" : "+v"(sixteen));

  constexpr bool kSums = AFF || !XF;               // the tokens' sums over each group are needed
  const uint32_t cbits = XF ? 0x3F803F80u : AFF ? 0xC180C180u : 0xC1C0C1C0u;   // 1, -16 or -24
  const v4u offs = {cbits, cbits, cbits, cbits};

  // wave k's units are [first(k), first(k + 1))
  const auto first = [&](int k) { return (units * k) >> shift; };
  const int begin = first(ks), end = first(ks + 1);
  const int steps = (units + S - 1) >> shift;

  struct Ring {
    UnitW w[T];
  };
  const uint32_t wlane = (uint32_t)(lane & 7) * pitch + (uint32_t)(4 * (lane >> 3 & 1) + q) * 16u;
  // Always the same number of loads (past the last unit none of them touches
  // memory), so that the waits for one unit leave the next in flight.
  auto load_unit = [&](int u, Ring& r) {
    const uint32_t at0 = wlane + (uint32_t)u * 128u;
#pragma unroll
    for (int t = 0; t < T; ++t) {
      r.w[t].a = load16<true, kLoadNT>(wsrc, u < end ? at0 + (uint32_t)(16 * t) * pitch : kOffNone);
      r.w[t].b = load16<true, kLoadNT>(wsrc, u < end ? at0 + (uint32_t)(16 * t + 8) * pitch : kOffNone);
    }
  };

  // A chunk of steps: slot (step, wave) of every wave's unit (zeros past its
  // last).  The scales as [row][slot][group], read in whole runs, since a
  // wave's own reads of a few bytes of each row would move a cache line each.
  const int log_slots = log_chunk + shift, log_scale_slots = plan.log_scales + shift;
  auto unit_of = [&](int i0, int slot) {      // -1: none
    const int k = slot & (S - 1), u = first(k) + i0 + (slot >> shift);
    return u < first(k + 1) ? u : -1;
  };
  const uint32_t scale_bytes = (uint32_t)p.N * (uint32_t)p.groups * kScaleBytes;
  const __amdgpu_buffer_rsrc_t ssrc = make_rsrc(p.scales, scale_bytes);
  const __amdgpu_buffer_rsrc_t bsrc = make_rsrc(p.biases, AFF ? scale_bytes : 0u);
  auto stage_scales = [&](int i0, auto dword) {
    constexpr int kPer = decltype(dword)::value ? 4 / kScaleBytes : 1;   // scales of a load
    constexpr int kLoads = kGroups / kPer, kLog = __builtin_ctz(kLoads);
    constexpr int kBatch = 8;                                            // loads in flight
    auto load = [&](__amdgpu_buffer_rsrc_t src, uint32_t at) {
      if constexpr (kPer * kScaleBytes == 4) return __builtin_amdgcn_raw_buffer_load_b32(src, (int)at, 0, 0);
      else return (uint32_t)__builtin_amdgcn_raw_buffer_load_b16(src, (int)at, 0, 0);
    };
    auto store = [&](uint8_t* to, uint32_t v) {
      if constexpr (kPer * kScaleBytes == 4) *reinterpret_cast<uint32_t*>(to) = v;
      else *reinterpret_cast<uint16_t*>(to) = (uint16_t)v;
    };
    const int runs = (sets * 16 * T) << (log_scale_slots + kLog);
    for (int i1 = threadIdx.x; i1 < runs; i1 += kBatch * kThreads) {
      uint32_t s[kBatch], b[kBatch];
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const int i = i1 + k * kThreads;
        const int slot = (i >> kLog) & ((1 << log_scale_slots) - 1), row = i >> (log_scale_slots + kLog);
        const int u = unit_of(i0, slot), g = u * kGroups + (i & (kLoads - 1)) * kPer;
        const uint32_t e = (uint32_t)min(wg_row0 + row, p.N - 1) * (uint32_t)p.groups + (uint32_t)g;
        const uint32_t at = i < runs && u >= 0 && g < p.groups ? e * (uint32_t)kScaleBytes : kOffNone;
        s[k] = load(ssrc, at);
        if constexpr (AFF) b[k] = load(bsrc, at);
      }
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const int i = i1 + k * kThreads;
        const int slot = (i >> kLog) & ((1 << log_scale_slots) - 1), row = i >> (log_scale_slots + kLog);
        if (i >= runs) break;
        uint8_t* const to = s_scales + row * plan.pitch + (slot * kGroups + (i & (kLoads - 1)) * kPer) * kScaleBytes;
        store(to, s[k]);
        if constexpr (AFF) store(to + plan.scale_bytes, b[k]);
      }
    }
  };
  const bool pairs = SF || (((uint32_t)p.groups & 1) == 0 && (((uintptr_t)p.scales | (uintptr_t)p.biases) & 3) == 0);

  // Staged tokens, as [slot][operand][part][lane row][token] of 16 bytes; an item
  // is the eight values c of a token's unit: operand c / 4, lane row c % 4.  Its
  // place among 16 tokens is token ^ (c % 16): the lanes of a load, which take
  // neighbouring items so that it covers whole lines, then write to different
  // banks, and the lanes of an operand's read, 16 tokens of one lane row each,
  // still cover all of them.
  constexpr int kSwizzle = TK >= 16 ? 15 : TK >= 8 ? 7 : 0;
  struct Item {
    v4u x[XF ? 2 : 1];
  };
  auto place = [&](int slot, int c, int tok) {
    return s_mem + slot * kUnitX + (c >> 2) * (kParts * kOperandX) + (c & 3) * (TK * 16) + (tok ^ (c & kSwizzle)) * 16;
  };
  auto load_item = [&](uint32_t at, int tok, Item& f) {
    const int row = tok * p.K * (int)kXBytes;
    f.x[0] = __builtin_amdgcn_raw_buffer_load_b128(xsrc, (int)at, row, 0);
    if constexpr (XF) f.x[1] = __builtin_amdgcn_raw_buffer_load_b128(xsrc, (int)at + 16, row, 0);
  };
  auto store_item = [&](uint8_t* to, const Item& f) {
    v4u part[3];
    if constexpr (XF) order_split_x(f.x[0], f.x[1], part);
    else part[0] = order_x(f.x[0]);
#pragma unroll
    for (int d = 0; d < kParts; ++d) *reinterpret_cast<v4u*>(to + d * kOperandX) = part[d];
  };
  // A fixed split's step: half a wave takes a slot's 32 items of one token, wave
  // by wave down the tokens (the last one again past the end).
  constexpr int kHalves = kThreads / 32, kStride = kSplit ? kHalves / kSplit : 1;   // half-waves, tokens between a wave's items
  constexpr int kFetch = kSplit ? TK / kStride : TK;
  const int my_slot = (lane >> 5) + 2 * (wave & (S / 2 - 1)), my_tok = kSplit ? wave / (kSplit / 2) : 0;
  Item next[kFetch];
  auto item_at = [&](int i0, int slot, int c) {
    const int u = unit_of(i0, slot), k = 256 * u + 8 * c;
    return u >= 0 && k < p.K ? (uint32_t)k * kXBytes : kOffNone;
  };
  auto fetch_step = [&](int i0) {
    if constexpr (kSplit != 0) {
      const uint32_t at = item_at(i0, my_slot, lane & 31);
#pragma unroll
      for (int j = 0; j < kFetch; ++j) load_item(at, min(my_tok + j * kStride, tokens - 1), next[j]);
    } else {
      const uint32_t at = (int)threadIdx.x < 32 << log_slots ? item_at(i0, threadIdx.x >> 5, lane & 31) : kOffNone;
#pragma unroll
      for (int j = 0; j < kFetch; ++j) load_item(at, min(j, tokens - 1), next[j]);
    }
  };
  auto put_step = [&](int i0) {
    if constexpr (kSplit != 0) {
#pragma unroll
      for (int j = 0; j < kFetch; ++j) store_item(place(my_slot, lane & 31, my_tok + j * kStride), next[j]);
    } else {
      for (int i = threadIdx.x; i < 32 << log_slots; i += kThreads) {
        if (i >= kThreads) {
          const uint32_t at = item_at(i0, i >> 5, i & 31);
#pragma unroll
          for (int j = 0; j < kFetch; ++j) load_item(at, min(j, tokens - 1), next[j]);
        }
#pragma unroll
        for (int j = 0; j < kFetch; ++j) store_item(place(i >> 5, i & 31, j), next[j]);
      }
    }
  };
  // Rows past the last token repeat one or hold what LDS held: their sums are not used.
  const int mrow = (TR == 1 ? n >> 2 : n) & (TK < 16 ? TK - 1 : 15);
  uint32_t xlane[kSwizzle ? 4 : 1];          // by operand mod 4
#pragma unroll
  for (int o = 0; o < (kSwizzle ? 4 : 1); ++o) xlane[o] = (uint32_t)(q * TK + (mrow ^ ((4 * o + q) & kSwizzle))) * 16u;
  auto operand = [&](uint32_t xu, int o, int d, int mt) {   // xu: of the unit
    return *reinterpret_cast<const v4u*>(s_mem + xu + xlane[kSwizzle ? o & 3 : 0] + (o * kParts + d) * kOperandX + mt * 256);
  };
  // -24 (-16; 1 for floats) times the tokens' sums over each group, as
  // [slot][group][token]; a wave keeps to one group of the unit.
  auto stage_sums = [&]() {
    const int g = wave & (kGroups - 1);
    uint32_t at[KPG];
#pragma unroll
    for (int j = 0; j < KPG; ++j) {
      const int o = g * KPG + j;
      at[j] = (uint32_t)(o * (kParts * kOperandX) + (q * TK + (mrow ^ ((4 * o + q) & kSwizzle))) * 16);
    }
#pragma unroll 4
    for (int r = wave / kGroups; r < MT << log_slots; r += kLinearWaves / kGroups) {
      const int mt = r % MT, slot = r / MT;
      v4f sum = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int j = 0; j < KPG; ++j)
#pragma unroll
        for (int d = 0; d < kParts; ++d)
          sum = mfma_bf16(*reinterpret_cast<const v4u*>(s_mem + at[j] + slot * kUnitX + mt * 256 + d * kOperandX), offs, sum);
      float* const to = reinterpret_cast<float*>(s_sums) + (slot * kGroups + g) * TK;
      if constexpr (TR == 1) {
        if (n == 0 && q < TK) to[q] = sum[0];
      } else {
        if (n == 0 && 4 * q < TK) *reinterpret_cast<v4f*>(to + 16 * mt + 4 * q) = sum;
      }
    }
  };

  // Running sums of the wave's segment of K (an eighth of the units), and sums
  // of one, two and four segments that wait for their neighbours: every variant
  // joins the eight in this tree, whichever waves took them.
  constexpr int kLevels = kSplit ? 3 - __builtin_ctz(kSplit) : 3;
  typedef float Sums[T][MT][TR];
  Sums tot = {}, level[kLevels ? kLevels : 1];
  const int segments = 8 >> shift;
  int segment = 0;
  const auto segment_end = [&]() { return (units * ((ks << (3 - shift)) + segment + 1)) >> 3; };
  const auto each = [&](auto f) {
#pragma unroll
    for (int t = 0; t < T; ++t)
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int j = 0; j < TR; ++j) f(t, mt, j);
  };
  auto close_segment = [&]() {
    bool open = true;
#pragma unroll
    for (int l = 0; l < kLevels; ++l) {
      if (open && (segment >> l & 1)) {
        each([&](int t, int mt, int j) { tot[t][mt][j] = level[l][t][mt][j] + tot[t][mt][j]; });
      } else if (open && segment + 1 < segments) {
        each([&](int t, int mt, int j) {
          level[l][t][mt][j] = tot[t][mt][j];
          tot[t][mt][j] = 0.0f;
        });
        open = false;
      }
    }
    ++segment;
  };
  auto close_segments = [&](int u) {
    if constexpr (kLevels != 0) {
      while (segment < segments && u >= segment_end()) close_segment();
    }
  };

  if constexpr (kSplit != 0) fetch_step(0);
  Ring ring[kRing];
#pragma unroll
  for (int i = 0; i < kRing; ++i) {
    load_unit(begin + i, ring[i]);
    __builtin_amdgcn_sched_barrier(0);
  }

  // unit i of the wave; no path around it inside the loop, so that the waits
  // stay exact (a wave without a unit left in a step works on zeros)
  auto step = [&](int i, Ring& r) {
    const int u = begin + i;
    close_segments(u);
    if (ragged && u == units - 1) {
#pragma unroll
      for (int t = 0; t < T; ++t) {
        r.w[t].a = load16<false>(wsrc, wlane + (uint32_t)u * 128u + (uint32_t)(16 * t) * pitch);
        r.w[t].b = load16<false>(wsrc, wlane + (uint32_t)u * 128u + (uint32_t)(16 * t + 8) * pitch);
      }
      __builtin_amdgcn_s_waitcnt(kWaitVmem0);
    }
    const int slot = ((i & (chunk - 1)) << shift) + ks, scale_slot = ((i & ((1 << plan.log_scales) - 1)) << shift) + ks;
    const uint8_t* const su = s_scales + (set * 16 * T + n) * plan.pitch + scale_slot * (kGroups * kScaleBytes);
    const uint32_t xu = (uint32_t)(slot * kUnitX);
    uint32_t word[T][8];
    float s[T][kGroups], b[T][AFF ? kGroups : 1];
#pragma unroll
    for (int t = 0; t < T; ++t) {
      unit_words(r.w[t], high, word[t]);
      read_scales<kGroups, SF>(su + 16 * t * plan.pitch, s[t]);
      if constexpr (AFF) read_scales<kGroups, SF>(su + 16 * t * plan.pitch + plan.scale_bytes, b[t]);
    }
    load_unit(u + kRing, r);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
      v4f xsum[MT];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        const float* const at = reinterpret_cast<const float*>(s_sums) + (slot * kGroups + g) * TK;
        if constexpr (!kSums) {
          xsum[mt] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
        } else if constexpr (TR == 1) {
          const float v = at[q & (TK - 1)];
          xsum[mt] = v4f{v, v, v, v};
        } else {
          xsum[mt] = *reinterpret_cast<const v4f*>(at + 16 * mt + (TK == 8 ? 4 * (q & 1) : 4 * q));
        }
      }
      v4f acc[T][MT];
#pragma unroll
      for (int t = 0; t < T; ++t)
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) acc[t][mt] = XF ? v4f{0.0f, 0.0f, 0.0f, 0.0f} : xsum[mt];
#pragma unroll
      for (int j = 0; j < KPG; ++j) {
        v4u bw[T];
#pragma unroll
        for (int t = 0; t < T; ++t) bw[t] = XF ? unpack_word_exact(word[t][g * KPG + j]) : unpack_word(word[t][g * KPG + j], sixteen);
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int d = 0; d < kParts; ++d) {
            const v4u op = operand(xu, g * KPG + j, d, mt);
#pragma unroll
            for (int t = 0; t < T; ++t) acc[t][mt] = mfma_bf16(op, bw[t], acc[t][mt]);
          }
      }
      each([&](int t, int mt, int j) {
        tot[t][mt][j] = __builtin_fmaf(XF ? 16.0f * s[t][g] : s[t][g], acc[t][mt][j], tot[t][mt][j]);
        if constexpr (AFF) {
          const float b1 = XF ? __builtin_fmaf(8.0f, s[t][g], b[t][g]) : -0.0625f * b[t][g];
          tot[t][mt][j] = __builtin_fmaf(b1, xsum[mt][j], tot[t][mt][j]);
        }
      });
    }
  };
  auto stage = [&](int i) {
    if ((i & (chunk - 1)) != 0) return;
    if (i) __syncthreads();
    if constexpr (kSplit == 0) fetch_step(i);
    if ((i & ((1 << plan.log_scales) - 1)) == 0) {
      if (pairs) stage_scales(i, Bool<true>{});
      else stage_scales(i, Bool<false>{});
    }
    put_step(i);
    __syncthreads();
    if constexpr (kSums) {
      stage_sums();
      __syncthreads();
    }
    if constexpr (kSplit != 0) fetch_step(i + 1);
    __builtin_amdgcn_sched_barrier(0);
  };
  // two steps a round, so that each knows its place in the ring; the last of an odd number follows
  const int rounds = steps & ~(kRing - 1);
  int i = 0;
  for (; i < rounds; i += kRing) {
    stage(i);
    step(i, ring[0]);
    if constexpr (kRing == 2) step(i + 1, ring[1]);     // (a chunk has two steps or more)
  }
  if constexpr (kRing == 2) {
    if (i < steps) {
      stage(i);
      step(i, ring[0]);
    }
  }
  close_segments(units);

  auto store = [&](int t, int mt, int j, float v) {
    const int token = TR == 1 ? q : 16 * mt + 4 * q + j;
    const int row = 16 * t + n;
    if (token < tokens && row < rows) {
      const size_t at = (size_t)(m0 + token) * (size_t)p.N + (size_t)(row0 + row);
      if constexpr (XF) static_cast<float*>(p.out)[at] = v;
      else static_cast<uint16_t*>(p.out)[at] = bf16_rne(v);
    }
  };
  constexpr int kItems = T * MT * TR;
  if (S == 1) {
    each([&](int t, int mt, int j) { store(t, mt, j, tot[t][mt][j]); });
    return;
  }
  // the sums of a set's waves, joined in the tree
  float* const part = reinterpret_cast<float*>(s_mem);
  __syncthreads();
  each([&](int t, int mt, int j) { part[(wave * kItems + (t * MT + mt) * TR + j) * 64 + lane] = tot[t][mt][j]; });
  __syncthreads();
  for (int item = ks; item < kItems; item += S) {
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = j < S ? part[((set * S + j) * kItems + item) * 64 + lane] : 0.0f;
    store(item / (MT * TR), item / TR % MT, item % TR, ((v[0] + v[1]) + (v[2] + v[3])) + ((v[4] + v[5]) + (v[6] + v[7])));
  }
}

// Bytes of LDS that a launch stages where one step allows it: two work-groups a CU.
constexpr int kLinearStage = 72 * 1024;
// Most that it takes.
constexpr int kLinearLds = 144 * 1024;
// Work-groups along the rows of one launch: a grid takes fewer than 2^32 threads
// there, which five tokens or more (64 rows a work-group) of the most rows of
// eight weights reach.
constexpr int kLinearBlocks = 1 << 22;

template <int KPG, bool AFF, bool SF, bool XF, int TK, int T, int kSplit>
hipError_t linear_launch(const LinearParams& p, int split, hipStream_t stream) {
  constexpr int MT = TK > 16 ? TK / 16 : 1, kGroups = 8 / KPG, kScale = SF ? 4 : 2;
  const int units = (p.K + 255) / 256;
  LinearPlan plan{};
  int steps = 1, sets = 1;
  auto staged = [&](int S, int log_chunk, int log_scales) {   // bytes of LDS
    steps = (units + S - 1) / S;
    sets = kLinearWaves / S;
    plan.S = S;
    plan.shift = __builtin_ctz(S);
    plan.log_chunk = log_chunk;
    plan.log_scales = log_scales;
    plan.x_bytes = (S << log_chunk) * kLinearUnitX<XF, TK>;
    plan.xs_bytes = ((S << log_chunk) * kGroups * TK * 4 + 15) / 16 * 16;
    plan.pitch = ((S << log_scales) * kGroups * kScale + 15) / 16 * 16 + 16;   // 16 bytes off a multiple of the banks
    plan.scale_bytes = 16 * T * sets * plan.pitch;
    return plan.x_bytes + plan.xs_bytes + (AFF ? 2 : 1) * plan.scale_bytes;
  };
  int log_chunk = kLinearRing<XF, TK> - 1, log_scales = log_chunk, stage;
  if constexpr (kSplit != 0) {
    split = kSplit;
    const int at_most = staged(split, 0, 0) < kLinearStage ? kLinearStage : kLinearLds;
    while (staged(split, 0, log_scales + 1) <= at_most && (1 << log_scales) < steps) ++log_scales;
  } else {
    while (split > 1 && staged(split, log_chunk, log_chunk) > kLinearLds) split /= 2;
    while (staged(split, log_chunk + 1, log_chunk + 1) <= kLinearStage && (1 << log_chunk) < steps) ++log_chunk;
    log_scales = log_chunk;
  }
  stage = staged(split, log_chunk, log_scales);
  const int sums = split > 1 ? kLinearWaves * T * MT * (TK <= 4 ? 1 : 4) * 256 : 0;
  const size_t lds = (size_t)(stage > sums ? stage : sums);
  LinearParams q = p;
  void* args[] = {&q, &plan};
  const void* const f = reinterpret_cast<const void*>(&linear_kernel<KPG, AFF, SF, XF, TK, T, kSplit>);
  const int blocks = (p.N + 16 * T * sets - 1) / (16 * T * sets);
  for (; plan.block0 < blocks; plan.block0 += kLinearBlocks) {
    const int here = blocks - plan.block0 < kLinearBlocks ? blocks - plan.block0 : kLinearBlocks;
    const hipError_t e = hipLaunchKernel(f, dim3((unsigned)here, (unsigned)((p.M + TK - 1) / TK)), dim3(kLinearWaves * 64),
                                         args, lds, stream);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

// Row tiles of a wave and waves along K (figures: one call, bf16 tokens
// unless said, groups of 128 with biases).
template <int KPG, bool AFF, bool SF, bool XF, int TK>
hipError_t linear_tiles(const LinearParams& p, hipStream_t stream) {
  const int tiles = (p.N + 15) / 16;
  if constexpr (TK <= 4) {
    // as many waves along K as give the card 2048 waves or more: 14336 rows of
    // 7168 take 15 us with four, 17 with two, 21 with eight
    const int units = (p.K + 255) / 256;
    int split = 1;
    while (split < 8 && split * 2 <= units && split * tiles < 2048) split *= 2;
    return linear_launch<KPG, AFF, SF, XF, TK, 1, 0>(p, split, stream);
  } else if constexpr (TK == 64) {
    return linear_launch<KPG, AFF, SF, XF, TK, 1, 2>(p, 0, stream);
  } else {
    constexpr int S = XF && TK == 32 ? 2 : 4;
    if constexpr (!XF && TK <= 16) {
      // few rows: all waves along K, as long as every work-group has a CU of its
      // own (their tokens and sums take one each).  16 tokens, rows of 7168:
      // 4096 of them take 11.9 us against 12.6 with four waves, 4112 take 15.8
      // against 12.8; groups of 32 with biases 15.3 against 18.2 and 27.4
      // against 18.1.  (Eight tokens of 14336 alone would gain on, 18.3 against 19.5.)
      constexpr int kCus = 256;
      if (tiles <= kCus) return linear_launch<KPG, AFF, SF, XF, TK, 1, 8>(p, 0, stream);
    }
    // two tiles of a wave share the tokens' reads from LDS, once there are more
    // work-groups than the 256 CUs hold at a time (one each by their LDS or
    // registers, two of the smaller variants).  Rows of 4096, one tile against
    // two: 32 tokens 14.9 us against 18.3 with 8192 rows (256 work-groups), 23.6
    // against 16.4 with 10240, 44.1 against 30.9 with 32768; 16 tokens 25.4
    // against 23.7 and 8 tokens 22.7 against 19.6 with 32768 (groups of 64
    // without biases).  With up to 16 tokens, where four waves a SIMD leave 128
    // registers, the two tiles spill some of them, most with biases of small
    // groups: 16 tokens and groups of 32 never gain (24576 rows 24.4 against
    // 32.3, 131072 rows 112 against 119), groups of 64 from 65536 rows on (20.6
    // against 24.6 with 24576, 48.3 against 48.4, 96.9 against 89.8 with
    // 131072).  Eight float tokens have two work-groups a CU with one tile and
    // one with two: groups of 128 gain from 32768 rows on (24.1 against 26.0
    // with 24576, 30.7 against 27.0), smaller ones lose up to 35% below and gain
    // 5% at most at 131072.
    constexpr bool kFew = TK * (XF ? 2 : 1) <= 16;
    constexpr bool kTwo = !kFew || (XF ? KPG == 4 : !AFF || KPG > 1);
    if constexpr (kTwo) {
      constexpr int kAtOnce = !kFew ? 256 : XF ? 900 : AFF && KPG == 2 ? 2000 : 512;
      const int groups = (tiles * S + kLinearWaves - 1) / kLinearWaves * ((p.M + TK - 1) / TK);
      if (groups > kAtOnce) return linear_launch<KPG, AFF, SF, XF, TK, 2, S>(p, 0, stream);
    }
    return linear_launch<KPG, AFF, SF, XF, TK, 1, S>(p, 0, stream);
  }
}

// Tokens of a work-group: as many as the call has; with too few work-groups
// fewer, which spreads the tokens over more of them and unpacks the weights for
// each.  64 tokens of 4096, work-groups with 64, 32 and 16 of them (groups of
// 128 with biases): 24.6, 30.6 and 28.2 us with 9600 rows (150 work-groups in one
// pass), 24.6, 16.3 and 19.1 with 8192 (128), 24.2, 13.0 and 19.1 with 4096, 24.3,
// 12.4 and 10.2 with 1536 (96 work-groups in passes of 32 tokens); rows of 7168
// and groups of 32 change sides at the same numbers.  32 float tokens, 32 and 16
// at a time: 30.0 and 19.7 with 8192 rows (128).
template <int KPG, bool AFF, bool SF, bool XF>
hipError_t linear_select(const LinearParams& p, hipStream_t stream) {
  constexpr int kEnough = 150;
  const int tiles = (p.N + 15) / 16;
  const auto groups = [&](int tokens, int S) { return tiles * S / kLinearWaves * ((p.M + tokens - 1) / tokens); };
  if (p.M == 1) return linear_tiles<KPG, AFF, SF, XF, 1>(p, stream);
  if (p.M <= 4) return linear_tiles<KPG, AFF, SF, XF, 4>(p, stream);
  if (p.M <= 8) return linear_tiles<KPG, AFF, SF, XF, 8>(p, stream);
  if constexpr (!XF) {
    if (p.M > 32 && groups(64, 2) >= kEnough) return linear_tiles<KPG, AFF, SF, XF, 64>(p, stream);
  }
  if (p.M > 16 && groups(32, XF ? 2 : 4) >= kEnough) return linear_tiles<KPG, AFF, SF, XF, 32>(p, stream);
  return linear_tiles<KPG, AFF, SF, XF, 16>(p, stream);
}

template <int KPG, bool AFF, bool SF>
hipError_t linear_types(const LinearParams& p, hipStream_t stream) {
  return p.xf32 ? linear_select<KPG, AFF, SF, true>(p, stream) : linear_select<KPG, AFF, SF, false>(p, stream);
}

template <int KPG>
hipError_t linear_group(const LinearParams& p, hipStream_t stream) {
  if (p.biases) return p.scale_f32 ? linear_types<KPG, true, true>(p, stream) : linear_types<KPG, true, false>(p, stream);
  return p.scale_f32 ? linear_types<KPG, false, true>(p, stream) : linear_types<KPG, false, false>(p, stream);
}

hipError_t launch_linear32(const LinearParams& p, hipStream_t stream);
hipError_t launch_linear64(const LinearParams& p, hipStream_t stream);
hipError_t launch_linear128(const LinearParams& p, hipStream_t stream);

}  // namespace q4
