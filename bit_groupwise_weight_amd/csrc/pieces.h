// Eight consecutive elements of a row at any element's address: rows of any
// width on any buffer.  (The vector accesses need no alignment beyond the
// element's: global memory takes 16-byte accesses at every address here.)
#pragma once

#include "f8_common.h"

namespace lowbit {

typedef u32v4_t u32v4_any_t __attribute__((aligned(2)));

template <int ACT> struct Piece { u32v4_t w[Act<ACT>::bytes / 2]; };

// The first `n` elements from p on, zeros behind them (n < 1: only zeros).
template <int ACT>
__device__ __forceinline__ void load_piece(const typename Act<ACT>::bits_t* p, int n, Piece<ACT>& v) {
  if (n >= 8) {
#pragma unroll
    for (int q = 0; q < Act<ACT>::bytes / 2; ++q) v.w[q] = reinterpret_cast<const u32v4_any_t*>(p)[q];
    return;
  }
  uint32_t e[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) e[i] = i < n ? p[i] : 0u;
  if constexpr (ACT == ACT_F32) {
    v.w[0] = u32v4_t{e[0], e[1], e[2], e[3]};
    v.w[1] = u32v4_t{e[4], e[5], e[6], e[7]};
  } else {
    v.w[0] = u32v4_t{e[0] | (e[1] << 16), e[2] | (e[3] << 16), e[4] | (e[5] << 16), e[6] | (e[7] << 16)};
  }
}

template <int ACT>
__device__ __forceinline__ void piece_to_float(const Piece<ACT>& v, float (&f)[8]) {
  if constexpr (ACT == ACT_F32) {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(v.w[i >> 2][i & 3]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = act_bits_to_float<ACT>(v.w[0][i] & 0xffffu);
      f[2 * i + 1] = act_bits_to_float<ACT>(v.w[0][i] >> 16);
    }
  }
}

// The first n of eight values, rounded to the type (nearest even), to p.
template <int ACT>
__device__ __forceinline__ void store_piece(typename Act<ACT>::bits_t* p, int n, const float (&f)[8]) {
  Piece<ACT> v;
  if constexpr (ACT == ACT_F32) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v.w[i >> 2][i & 3] = __float_as_uint(f[i]);
  } else {
    v.w[0] = u32v4_t{pack2<ACT>(f[0], f[1]), pack2<ACT>(f[2], f[3]), pack2<ACT>(f[4], f[5]), pack2<ACT>(f[6], f[7])};
  }
  if (n >= 8) {
#pragma unroll
    for (int q = 0; q < Act<ACT>::bytes / 2; ++q)
      __builtin_nontemporal_store(v.w[q], reinterpret_cast<u32v4_any_t*>(p) + q);
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (i < n) {
      if constexpr (ACT == ACT_F32) p[i] = v.w[i >> 2][i & 3];
      else p[i] = static_cast<uint16_t>(v.w[0][i >> 1] >> (16 * (i & 1)));
    }
  }
}

}  // namespace lowbit
