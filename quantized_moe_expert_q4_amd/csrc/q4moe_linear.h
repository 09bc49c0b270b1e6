// Kernel of the linear with 4-bit weights and group scales (one instantiation
// file per group size includes this).
//
// One work-group owns T tiles of 16 weight rows; its W waves split K in units
// of 256 weights (128 bytes of a row) and join their F32 sums through LDS at
// the end.  A matrix-core operation (16x16x32 bf16, F32 accumulation) takes 16
// tokens as rows and 16 weight rows as columns, so one token costs what
// sixteen do, and the weights are unpacked once for up to 16 MT tokens.
//
// Unpacking.  Bits 3..6 of a bf16 in [16, 32) count in steps of one: a nibble
// q moved there under the bit pattern of 16 is the number 16 + q, exactly, two
// of them per shift and and-or.  The offset is taken off by one further matrix
// product per 32 weights, of the tokens with a constant -24 (symmetric: 16 + 8)
// or -16 (affine), shared by the T tiles; it starts the sums of every group:
//   sum (16 + q) x - 24 sum x = sum (q - 8) x
//   s sum q x + b sum x = s (sum (16 + q) x - 16 sum x) - (b / 16) (-16 sum x)
// Group sums are scaled in F32 into the running total, so products and the
// scale are exact up to F32 rounding.  Float activations enter as three bf16
// parts whose sum is the float (8 bits each), three products per weight.
#pragma once
#include "q4moe_device.h"
#include "q4moe_layer.h"

namespace q4 {

typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef unsigned int v2u __attribute__((ext_vector_type(2)));

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

// One unit of a 16-row tile as loaded: lane L holds bytes 16 (L / 8) .. +16 of
// the unit's 128 bytes of rows L % 8 (a) and 8 + L % 8 (b), so that every load
// instruction covers whole lines.
struct UnitW {
  v4u a, b;
};

// The unit as eight matrix operands: word[kb] of lane 16 q + n holds weights
// 32 kb + 8 q .. + 8 of row n.  Lanes 8 apart trade rows for 16-byte pieces,
// then a 4x4 transpose over the lane rows trades pieces for words.
__device__ __forceinline__ void unit_words(const UnitW& w, bool high, uint32_t (&word)[8]) {
  uint32_t p[2][4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t send = high ? w.a[i] : w.b[i];
    const uint32_t got = (uint32_t)__builtin_amdgcn_mov_dpp((int)send, 0x128, 0xF, 0xF, true);  // row_ror:8
    p[0][i] = high ? got : w.a[i];
    p[1][i] = high ? w.b[i] : got;
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    swap32(p[h][0], p[h][2]);
    swap32(p[h][1], p[h][3]);
    swap16(p[h][0], p[h][1]);
    swap16(p[h][2], p[h][3]);
#pragma unroll
    for (int j = 0; j < 4; ++j) word[2 * j + h] = p[h][j];
  }
}

// Eight nibbles as the bf16 numbers 16 + q, in the order (0,4) (1,5) (2,6) (3,7).
__device__ __forceinline__ v4u unpack_word(uint32_t w) {
  v4u r;
  r.x = ((w << 3) & 0x00780078u) | 0x41804180u;
  r.y = ((w >> 1) & 0x00780078u) | 0x41804180u;
  r.z = ((w >> 5) & 0x00780078u) | 0x41804180u;
  r.w = ((w >> 9) & 0x00780078u) | 0x41804180u;
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

// CNT consecutive scales from element i of a row of `groups` (0 past its end).
template <int CNT>
__device__ __forceinline__ void load_scales(const void* base, int f32, size_t row, int i, int groups, float (&s)[CNT]) {
  const size_t at = row + (size_t)i;
  if (i + CNT <= groups) {
    if (f32) {
      __builtin_memcpy(s, static_cast<const float*>(base) + at, 4 * CNT);
    } else {
      uint16_t h[CNT];
      __builtin_memcpy(h, static_cast<const uint16_t*>(base) + at, 2 * CNT);
#pragma unroll
      for (int j = 0; j < CNT; ++j) s[j] = bf16_val(h[j]);
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < CNT; ++j) {
    s[j] = 0.0f;
    if (i + j < groups)
      s[j] = f32 ? static_cast<const float*>(base)[at + j] : bf16_val(static_cast<const uint16_t*>(base)[at + j]);
  }
}

// KPG: 32-weight blocks of a group (1, 2, 4).  MT: 16-token tiles.  TR: result
// registers in use; with TR = 1 (at most four tokens) matrix row 4 t + i holds
// token t, so each lane keeps one sum instead of four.
template <int KPG, bool AFF, bool XF, int MT, int TR, int T, int MAXW>
__global__ __launch_bounds__(MAXW * 64) void linear_kernel(LinearParams p) {
  constexpr int kParts = XF ? 3 : 1;
  constexpr int kGroups = 8 / KPG;                 // groups of a unit
  constexpr int kTokens = TR == 1 ? 4 : 16 * MT;   // tokens of the work-group
  extern __shared__ float s_part[];                // [wave][T][MT][TR][64]
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int waves = (int)(blockDim.x >> 6);
  const int n = lane & 15, q = lane >> 4;
  const bool high = (lane & 8) != 0;
  const int row0 = (int)blockIdx.x * (16 * T);
  const int m0 = (int)blockIdx.y * kTokens;
  const int tokens = min(kTokens, p.M - m0);
  const int units = (p.K + 255) / 256;
  const uint32_t pitch = (uint32_t)(p.K / 2);
  const int rows = min(16 * T, p.N - row0);
  const __amdgpu_buffer_rsrc_t wsrc = make_rsrc(p.w + (size_t)row0 * pitch, (uint32_t)(p.N - row0) * pitch);
  constexpr uint32_t kXBytes = XF ? 4 : 2;
  const __amdgpu_buffer_rsrc_t xsrc = make_rsrc(static_cast<const uint8_t*>(p.x) + (size_t)m0 * p.K * kXBytes,
                                                (uint32_t)tokens * (uint32_t)p.K * kXBytes);
  // the 16 bytes that hold a row's end may reach past the matrix: there (and only there) dwords are loaded one by one
  const bool ragged = p.K % 32 != 0 && row0 + 16 * T >= p.N;

  uint32_t xrow[MT];
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
    const int t = TR == 1 ? n >> 2 : 16 * mt + n;
    xrow[mt] = t < tokens ? (uint32_t)t * (uint32_t)p.K * kXBytes : kOffNone;
  }
  size_t srow[T];
#pragma unroll
  for (int t = 0; t < T; ++t) srow[t] = (size_t)min(row0 + 16 * t + n, p.N - 1) * (size_t)p.groups;

  float tot[T][MT][TR] = {};
  const uint32_t cbits = AFF ? 0xC180C180u : 0xC1C0C1C0u;   // -16 or -24
  const v4u offs = {cbits, cbits, cbits, cbits};

  auto load_w = [&](int u, UnitW (&w)[T]) {
#pragma unroll
    for (int t = 0; t < T; ++t) {
      const uint32_t at = (uint32_t)(16 * t + (lane & 7)) * pitch + (uint32_t)u * 128u + (uint32_t)(lane >> 3) * 16u;
      if (ragged && u == units - 1) {
        w[t].a = load16<false, kLoadNT>(wsrc, at);
        w[t].b = load16<false, kLoadNT>(wsrc, at + 8u * pitch);
      } else {
        w[t].a = load16<true, kLoadNT>(wsrc, at);
        w[t].b = load16<true, kLoadNT>(wsrc, at + 8u * pitch);
      }
    }
  };

  UnitW w[T];
  if (wave < units) load_w(wave, w);
  for (int u = wave; u < units; u += waves) {
    float s[T][kGroups], b[T][AFF ? kGroups : 1];
#pragma unroll
    for (int t = 0; t < T; ++t) {
      load_scales<kGroups>(p.scales, p.scale_f32, srow[t], u * kGroups, p.groups, s[t]);
      if constexpr (AFF) load_scales<kGroups>(p.biases, p.scale_f32, srow[t], u * kGroups, p.groups, b[t]);
    }
    v4u x[2][MT][4][XF ? 2 : 1];
    auto load_x = [&](int half) {
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int k = 256 * u + 128 * half + 32 * j + 8 * q;
          const uint32_t at = k < p.K ? xrow[mt] + (uint32_t)k * kXBytes : kOffNone;
          x[half][mt][j][0] = load16<true>(xsrc, at);
          if constexpr (XF) x[half][mt][j][1] = load16<true>(xsrc, at + 16u);
        }
    };
    load_x(0);
    uint32_t word[T][8];
#pragma unroll
    for (int t = 0; t < T; ++t) unit_words(w[t], high, word[t]);
    if (u + waves < units) load_w(u + waves, w);
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      if (half == 1) load_x(1);
#pragma unroll
      for (int g = 0; g < 4 / KPG; ++g) {
        v4u a[MT][KPG][kParts];
        v4f xsum[MT];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          xsum[mt] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
          for (int j = 0; j < KPG; ++j) {
            if constexpr (XF) order_split_x(x[half][mt][g * KPG + j][0], x[half][mt][g * KPG + j][1], a[mt][j]);
            else a[mt][j][0] = order_x(x[half][mt][g * KPG + j][0]);
#pragma unroll
            for (int d = 0; d < kParts; ++d) xsum[mt] = mfma_bf16(a[mt][j][d], offs, xsum[mt]);
          }
        }
#pragma unroll
        for (int t = 0; t < T; ++t) {
          v4f acc[MT];
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) acc[mt] = xsum[mt];
#pragma unroll
          for (int j = 0; j < KPG; ++j) {
            const v4u bw = unpack_word(word[t][4 * half + g * KPG + j]);
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
              for (int d = 0; d < kParts; ++d) acc[mt] = mfma_bf16(a[mt][j][d], bw, acc[mt]);
          }
          const int at = half * (4 / KPG) + g;
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int r = 0; r < TR; ++r) {
              tot[t][mt][r] = __builtin_fmaf(s[t][at], acc[mt][r], tot[t][mt][r]);
              if constexpr (AFF) tot[t][mt][r] = __builtin_fmaf(-0.0625f * b[t][at], xsum[mt][r], tot[t][mt][r]);
            }
        }
      }
    }
  }

  // the waves' sums, joined in order
  constexpr int kItems = T * MT * TR;
#pragma unroll
  for (int t = 0; t < T; ++t)
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int r = 0; r < TR; ++r) s_part[(wave * kItems + (t * MT + mt) * TR + r) * 64 + lane] = tot[t][mt][r];
  __syncthreads();
  for (int i = wave; i < kItems; i += waves) {
    const int t = i / (MT * TR), mt = i / TR % MT, r = i % TR;
    const int token = TR == 1 ? q : 16 * mt + 4 * q + r;
    const int row = 16 * t + n;
    float v = s_part[i * 64 + lane];
    for (int j = 1; j < waves; ++j) v += s_part[(j * kItems + i) * 64 + lane];
    if (token < tokens && row < rows) {
      const size_t at = (size_t)(m0 + token) * (size_t)p.N + (size_t)(row0 + row);
      if constexpr (XF) static_cast<float*>(p.out)[at] = v;
      else static_cast<uint16_t*>(p.out)[at] = bf16_rne(v);
    }
  }
}

// Rows of a matrix from which a work-group takes several tiles: below it there
// are too few work-groups to fill the card, and K is split over more waves.
constexpr int kLinearManyRows = 16384;

template <int KPG, bool AFF, bool XF, int MT, int TR, int T, int MAXW>
hipError_t linear_launch(const LinearParams& p, hipStream_t stream) {
  LinearParams q = p;
  void* args[] = {&q};
  const int units = (p.K + 255) / 256;
  const int waves = units < MAXW ? units : MAXW;
  constexpr int kTokens = TR == 1 ? 4 : 16 * MT;
  return hipLaunchKernel(reinterpret_cast<const void*>(&linear_kernel<KPG, AFF, XF, MT, TR, T, MAXW>),
                         dim3((unsigned)((p.N + 16 * T - 1) / (16 * T)), (unsigned)((p.M + kTokens - 1) / kTokens)),
                         dim3((unsigned)waves * 64), args, (size_t)waves * T * MT * TR * 256, stream);
}

template <int KPG, bool AFF, bool XF>
hipError_t linear_select(const LinearParams& p, hipStream_t stream) {
  if (p.N < kLinearManyRows) {
    if (p.M <= 4) return linear_launch<KPG, AFF, XF, 1, 1, 1, 8>(p, stream);
    if (p.M <= 16) return linear_launch<KPG, AFF, XF, 1, 4, 1, 8>(p, stream);
    if (p.M <= 32) return linear_launch<KPG, AFF, XF, 2, 4, 1, 8>(p, stream);
    return linear_launch<KPG, AFF, XF, 4, 4, 1, 8>(p, stream);
  }
  if (p.M <= 4) return linear_launch<KPG, AFF, XF, 1, 1, 4, 8>(p, stream);
  if (p.M <= 16) return linear_launch<KPG, AFF, XF, 1, 4, 4, 8>(p, stream);
  if (p.M <= 32) return linear_launch<KPG, AFF, XF, 2, 4, 2, 8>(p, stream);
  return linear_launch<KPG, AFF, XF, 4, 4, 2, 8>(p, stream);
}

template <int KPG>
hipError_t linear_group(const LinearParams& p, hipStream_t stream) {
  if (p.biases) return p.xf32 ? linear_select<KPG, true, true>(p, stream) : linear_select<KPG, true, false>(p, stream);
  return p.xf32 ? linear_select<KPG, false, true>(p, stream) : linear_select<KPG, false, false>(p, stream);
}

hipError_t launch_linear32(const LinearParams& p, hipStream_t stream);
hipError_t launch_linear64(const LinearParams& p, hipStream_t stream);
hipError_t launch_linear128(const LinearParams& p, hipStream_t stream);

}  // namespace q4
