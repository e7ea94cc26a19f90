// Pieces shared by the kernels of the 8-bit path: e4m3 codes (OCP: bias 7,
// largest 448, no infinities), the block-scaled products' MFMA, and the rule
// that turns the largest magnitude of a span into its scale.
#pragma once

#include "device_common.h"
#include "kernels.h"

namespace lowbit {

typedef int32_t i32x8_t __attribute__((ext_vector_type(8)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u32v4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u32v2_t __attribute__((ext_vector_type(2)));

constexpr int kF8Block = 128;          // K elements (and weight rows) that share a scale
constexpr float kE4m3Max = 448.0f;
constexpr float kI8Max = 127.0f;

// D = A . B over 128 K positions of e4m3 codes.  Lane l supplies row (A) or
// column (B) l % 16; D: lane l holds rows 4 (l / 16) + i of column l % 16.
// A lane's 32 bytes may hold any 32 K positions as long as A and B agree.
//
// EXACT == false: one fp8 MFMA (the builtin with zero scale operands is the
// unscaled instruction).  Its adder aligns each eight consecutive products to
// the largest of them and cuts off what lies below 2^-13 of that one (observed:
// beside a product of 2^16, 2^3 survives and 2^2 does not; from one eight to
// the next 24 bits survive), so a sum is off by at most 7 * 2^-13 of its
// magnitudes' sum A.  It is used for 16-bit outputs, at twice the rate.  Measured
// on normal activations, plain and with one in a hundred twenty times as large,
// K of 1024 to 14336: the cuts come to 2^-18.5 to 2^-22.4 of A (rms, falling with
// the root of K).  To bf16 that is nothing (rms error 1.0002 times that of the
// rounding alone, 1 to 2 % of the outputs not the nearest number).  In fp16 it
// shows: 1.2 % more rms error, 6 to 12 % of the outputs not the nearest, and
// outputs that cancel (|y| far below A) are off by many half steps of their own
// (one in a thousand by 38 at K = 4096 with outliers, the rms of A being 22
// times that of y).
// EXACT == true, for fp32 outputs: the codes as bf16 (exact) and four bf16
// MFMAs, whose sums keep 24 bits, at half the fp8 rate.
typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
template <bool EXACT> struct F8Fragment;
template <> struct F8Fragment<false> {
  i32x8_t v;
  __device__ __forceinline__ void set(u32v4_t lo, u32v4_t hi) {
    v = i32x8_t{(int)lo.x, (int)lo.y, (int)lo.z, (int)lo.w, (int)hi.x, (int)hi.y, (int)hi.z, (int)hi.w};
  }
};
template <> struct F8Fragment<true> {
  bf16x8_t v[4];
  __device__ __forceinline__ void set(u32v4_t lo, u32v4_t hi) {
    const uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const bf162_t a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[i], 1.0f, false);
      const bf162_t b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[i], 1.0f, true);
      v[i >> 1][4 * (i & 1) + 0] = a[0];
      v[i >> 1][4 * (i & 1) + 1] = a[1];
      v[i >> 1][4 * (i & 1) + 2] = b[0];
      v[i >> 1][4 * (i & 1) + 3] = b[1];
    }
  }
};
__device__ __forceinline__ f32x4_t mfma_f8(const F8Fragment<false>& a, const F8Fragment<false>& b) {
  const f32x4_t zero = {0.0f, 0.0f, 0.0f, 0.0f};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a.v, b.v, zero, 0, 0, 0, 0, 0, 0);
}
__device__ __forceinline__ f32x4_t mfma_f8(const F8Fragment<true>& a, const F8Fragment<true>& b) {
  f32x4_t d = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int i = 0; i < 4; ++i) d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.v[i], b.v[i], d, 0, 0, 0);
  return d;
}

// The scale of a span from the bits of its largest magnitude (as unsigned
// integers the magnitudes order as 0 < finite < infinity < NaN), and the
// factor its values are multiplied by before they are rounded to codes:
//   not finite: scale NaN, factor 0 (the codes are set to 0 by the caller)
//   below 2^-110: scale 0, factor 0 (its reciprocal would leave fp32)
//   else scale = amax / top, factor = top / amax, each correctly rounded.
// The factor in place of a division per value: one rounding more, 2^-24 of
// the value against the codes' half steps of 2^-4 (e4m3) and 2^-8 (int8).
struct SpanScale {
  float scale, factor;
  bool finite;
};
__device__ __forceinline__ SpanScale span_scale(uint32_t amax_bits, float top) {
  const float amax = __uint_as_float(amax_bits);
  SpanScale s;
  s.finite = amax_bits < 0x7f800000u;
  if (!s.finite) {
    s.scale = __builtin_nanf("");
    s.factor = 0.0f;
  } else if (amax < 0x1p-110f) {
    s.scale = 0.0f;
    s.factor = 0.0f;
  } else {
    s.scale = amax / top;
    s.factor = top / amax;
  }
  return s;
}

// Four values -> four e4m3 codes, nearest even, in the bytes of a word (the
// values are at most 448 (1 + 2^-23), which rounds to 448).
__device__ __forceinline__ uint32_t pack4_e4m3(float a, float b, float c, float d) {
  int w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  w = __builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true);
  return static_cast<uint32_t>(w);
}
// Four values of magnitude at most 127.5 - 2^-17 -> four int8 codes, nearest even.
__device__ __forceinline__ uint32_t pack4_i8(float a, float b, float c, float d) {
  auto code = [](float v) { return static_cast<uint32_t>(static_cast<int>(__builtin_rintf(v))) & 0xffu; };
  return code(a) | (code(b) << 8) | (code(c) << 16) | (code(d) << 24);
}

// Two fp32 values -> two values of a 16-bit type, nearest even, in one word.
template <int OUT>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  const f32x2 v = {lo, hi};
  if constexpr (OUT == ACT_F16) return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, half2_t));
  else return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf162_t));
}

// Eight consecutive values of a row (chunk c) as fp32, exact for every type.
template <int ACT>
__device__ __forceinline__ void load8(const void* row, int64_t c, float (&v)[8]) {
  const u32v4_t* src = static_cast<const u32v4_t*>(row);
  if constexpr (ACT == ACT_F32) {
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const u32v4_t w = src[2 * c + q];
      v[4 * q] = __uint_as_float(w.x);
      v[4 * q + 1] = __uint_as_float(w.y);
      v[4 * q + 2] = __uint_as_float(w.z);
      v[4 * q + 3] = __uint_as_float(w.w);
    }
  } else {
    const u32v4_t w = src[c];
    const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = act_bits_to_float<ACT>(ws[i] & 0xffffu);
      v[2 * i + 1] = act_bits_to_float<ACT>(ws[i] >> 16);
    }
  }
}

// Eight fp32 values rounded to the type (nearest even) and stored as chunk c;
// v becomes the rounded values.
template <int ACT>
__device__ __forceinline__ void store8(void* row, int64_t c, float (&v)[8]) {
  u32v4_t* dst = static_cast<u32v4_t*>(row);
  if constexpr (ACT == ACT_F32) {
#pragma unroll
    for (int q = 0; q < 2; ++q)
      dst[2 * c + q] = u32v4_t{__float_as_uint(v[4 * q]), __float_as_uint(v[4 * q + 1]),
                               __float_as_uint(v[4 * q + 2]), __float_as_uint(v[4 * q + 3])};
  } else {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      w[i] = pack2<ACT>(v[2 * i], v[2 * i + 1]);
      v[2 * i] = act_bits_to_float<ACT>(w[i] & 0xffffu);
      v[2 * i + 1] = act_bits_to_float<ACT>(w[i] >> 16);
    }
    dst[c] = u32v4_t{w[0], w[1], w[2], w[3]};
  }
}

}  // namespace lowbit
