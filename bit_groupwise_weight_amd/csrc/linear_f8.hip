// Product of e4m3 codes with a scale for each block of 128 along K (and of 128
// weight rows), dense or grouped by expert:
//
//   y[t, n] = sum_b xs[t, b] ws[n / 128, b] P_b[t, n] (+ bias[n])
//   P_b     = sum over the 128 K positions of block b of xq * wq
//
// MFMAs over the block's 128 K positions give P_b of an output tile (fp32, from
// a zero accumulator); the two scales are multiplied once per column of the
// tile and applied by one fused multiply-add per output.  The weights are the MFMA's A
// operand, so that a lane holds four consecutive n of one output row: the row's
// scale is one value a lane, and the outputs leave in 8- or 16-byte pieces.
//
// Grouped: the rows offsets[e] .. offsets[e + 1] - 1 of y use weight e.  The
// launch has as many row tiles as any offsets can need; a block finds its
// expert and rows by a prefix sum over the experts' tile counts and leaves if
// there is none.  Offsets are clamped to 0 .. T, an index outside xq gives a
// NaN row, so that no value in either reads or writes out of range.
#include "f8_common.h"

namespace lowbit {

namespace {

// K positions of a step's 16-byte chunk of a row in LDS: chunk c of row r sits
// at position c ^ ((r >> 1) & 7) of the row's 128 bytes.  Two rows span the 64
// banks, so the 16 rows that a 16-byte read covers at one chunk start in 16
// different 4-bank groups.
__device__ __forceinline__ int swizzle(int r) { return (r >> 1) & 7; }

__device__ __forceinline__ void load_lds16(const uint8_t* src, uint8_t* dst) {
  __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)src,
                                   (__attribute__((address_space(3))) void*)dst, 16, 0, 0);
}

// The expert and rows of row tile `tile` of the launch (BM rows a tile).
struct RowTile {
  int64_t begin, end;     // rows of y
  int expert;             // -1: none
};
template <int BM>
__device__ __forceinline__ RowTile find_rows(const LinearF8Params& p, int64_t tile) {
  RowTile t;
  if (p.offsets == nullptr) {
    t.begin = tile * BM;
    t.end = min(t.begin + BM, p.T);
    t.expert = 0;
    return t;
  }
  t.begin = t.end = 0;
  t.expert = -1;
  const int lane = threadIdx.x & 63;
  int64_t before = 0;     // tiles of the experts already passed
  for (int e0 = 0; e0 < p.E; e0 += 64) {
    const int e = e0 + lane;
    int64_t lo = 0, hi = 0;
    if (e < p.E) {
      lo = min(max(static_cast<int64_t>(p.offsets[e]), int64_t{0}), p.T);
      hi = min(max(static_cast<int64_t>(p.offsets[e + 1]), lo), p.T);
    }
    const int own = static_cast<int>((hi - lo + BM - 1) / BM);
    int upto = own;       // inclusive prefix sum over the lanes
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int v = __shfl_up(upto, o);
      if (lane >= o) upto += v;
    }
    const int64_t first = before + upto - own;
    const uint64_t hit = __ballot(tile >= first && tile < first + own);
    if (hit != 0) {       // one lane at most: the ranges do not overlap
      const int src = __builtin_ctzll(hit);
      const int64_t at = __shfl(static_cast<int>(tile - first), src);
      const int64_t lo_s = __shfl(static_cast<int>(lo), src), hi_s = __shfl(static_cast<int>(hi), src);
      t.begin = lo_s + at * BM;
      t.end = min(t.begin + BM, hi_s);
      t.expert = e0 + src;
      return t;
    }
    before += __shfl(upto, 63);
  }
  return t;
}

// Four consecutive outputs of row m from column n on (n % 4 == 0).
template <int OUT>
__device__ __forceinline__ void store4(const LinearF8Params& p, int64_t m, int n, const float (&v)[4],
                                       bool wide) {
  const size_t at = static_cast<size_t>(m) * p.N + n;
  if (wide && n + 4 <= p.N) {
    if constexpr (OUT == ACT_F32) {
      *reinterpret_cast<f32x4_t*>(static_cast<float*>(p.y) + at) = f32x4_t{v[0], v[1], v[2], v[3]};
    } else {
      *reinterpret_cast<u32v2_t*>(static_cast<uint16_t*>(p.y) + at) =
          u32v2_t{float_to_act_bits<OUT>(v[0]) | (float_to_act_bits<OUT>(v[1]) << 16),
                  float_to_act_bits<OUT>(v[2]) | (float_to_act_bits<OUT>(v[3]) << 16)};
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (n + i < p.N) store_act<OUT>(p.y, at + i, v[i]);
  }
}

}  // namespace

// Block of WN x WM waves over BN columns (n) and BM rows (t) of y; K steps of
// 128 staged through two LDS buffers by direct loads one step ahead.
template <int BN, int BM, int WN, int WM, int OUT>
__global__ __launch_bounds__(64 * WN * WM) void linear_f8_tile_kernel(LinearF8Params p) {
  constexpr int NW = WN * WM;
  constexpr bool EXACT = OUT == ACT_F32;
  constexpr int NT = BN / WN / 16, MT = BM / WM / 16;   // 16-wide tiles of a wave
  constexpr int ROWS = BN + BM;
  constexpr int LOADS = ROWS / 8 / NW;                  // 1 KiB loads of a wave per step
  static_assert(ROWS % (8 * NW) == 0 && BN % 8 == 0, "whole loads");
  static_assert(BM <= 64 * NW && kF8Block % BN == 0, "one scale row a block of columns");
  __shared__ __attribute__((aligned(16))) uint8_t s_codes[2][ROWS * kF8Block];
  __shared__ float s_xs[2][BM];

  const int tid = threadIdx.x, lane = tid & 63;
  const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int tile_n = blockIdx.x % p.tiles_n;
  const RowTile rt = find_rows<BM>(p, blockIdx.x / p.tiles_n);
  if (rt.expert < 0) return;
  const int n0 = tile_n * BN;
  const uint8_t* wq = p.wq + static_cast<size_t>(rt.expert) * p.N * p.K;
  const float* ws = p.ws + (static_cast<size_t>(rt.expert) * p.nb + n0 / kF8Block) * p.kb;

  // source row of output row t (clamped to the tile); ok: inside xq
  auto source_row = [&](int64_t t, bool* ok) -> int64_t {
    t = min(t, rt.end - 1);
    if (p.rows == nullptr) {
      *ok = true;
      return t;
    }
    const int64_t r = p.rows[t];
    *ok = r >= 0 && r < p.M;
    return *ok ? r : 0;
  };

  // load i of this wave: rows 8 (wv LOADS + i) .. + 7 of the step's BN weight
  // rows and BM activation rows; lane l fills position l % 8 of row l / 8
  const uint8_t* src[LOADS];
  int chunk[LOADS];
#pragma unroll
  for (int i = 0; i < LOADS; ++i) {
    const int r = 8 * (wv * LOADS + i) + (lane >> 3);
    chunk[i] = (lane & 7) ^ swizzle(r);
    if (r < BN) {
      src[i] = wq + static_cast<size_t>(min(n0 + r, p.N - 1)) * p.K;
    } else {
      bool ok;
      src[i] = p.xq + static_cast<size_t>(source_row(rt.begin + (r - BN), &ok)) * p.K;
    }
  }
  const int tail = (p.K & (kF8Block - 1)) / 16;         // chunks of a last, partial step (0: none)
  auto load_step = [&](int b, int buf) {
    const int valid = (tail != 0 && b == p.kb - 1) ? tail : 8;
#pragma unroll
    for (int i = 0; i < LOADS; ++i) {
      // past the row's end: the step's first chunk again (masked out below)
      const int c = chunk[i] < valid ? chunk[i] : 0;
      load_lds16(src[i] + static_cast<size_t>(b) * kF8Block + 16 * c,
                 &s_codes[buf][(wv * LOADS + i) * 8 * kF8Block]);
    }
  };
  const float* xs_row = nullptr;
  bool xs_ok = true;
  if (tid < BM) xs_row = p.xs + source_row(rt.begin + tid, &xs_ok) * p.kb;
  auto load_scale = [&](int b) -> float {
    return tid >= BM ? 0.0f : xs_ok ? xs_row[b] : __builtin_nanf("");
  };

  const int wn = wv % WN, wm = wv / WN;
  const int c16 = lane & 15, g = lane >> 4;
  // 32 bytes of row r: chunks g and g + 4 (lane group g's K positions), those
  // from chunk `valid` on as zeros
  auto fragment = [&](int buf, int r, int valid) -> F8Fragment<EXACT> {
    const uint8_t* row = &s_codes[buf][r * kF8Block];
    u32v4_t lo = *reinterpret_cast<const u32v4_t*>(row + 16 * (g ^ swizzle(r)));
    u32v4_t hi = *reinterpret_cast<const u32v4_t*>(row + 16 * ((g + 4) ^ swizzle(r)));
    if (valid < 8) {
      if (g >= valid) lo = u32v4_t{0u, 0u, 0u, 0u};
      if (g + 4 >= valid) hi = u32v4_t{0u, 0u, 0u, 0u};
    }
    F8Fragment<EXACT> f;
    f.set(lo, hi);
    return f;
  };

  f32x4_t acc[NT][MT];
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int j = 0; j < MT; ++j) acc[i][j] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};

  load_step(0, 0);
  if (tid < BM) s_xs[0][tid] = load_scale(0);
  __syncthreads();
  for (int b = 0; b < p.kb; ++b) {
    const int buf = b & 1;
    float xs_next = 0.0f;
    if (b + 1 < p.kb) {
      load_step(b + 1, buf ^ 1);
      xs_next = load_scale(b + 1);
    }
    const float w_scale = ws[b];
    const int valid = (tail != 0 && b == p.kb - 1) ? tail : 8;
    F8Fragment<EXACT> xf[MT];
    float s[MT];
#pragma unroll
    for (int j = 0; j < MT; ++j) {
      const int r = (wm * MT + j) * 16 + c16;
      xf[j] = fragment(buf, BN + r, valid);
      s[j] = w_scale * s_xs[buf][r];
    }
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      const F8Fragment<EXACT> wf = fragment(buf, (wn * NT + i) * 16 + c16, 8);
#pragma unroll
      for (int j = 0; j < MT; ++j) {
        const f32x4_t P = mfma_f8(wf, xf[j]);
#pragma unroll
        for (int q = 0; q < 4; ++q) acc[i][j][q] = fmaf(s[j], P[q], acc[i][j][q]);
      }
    }
    if (b + 1 < p.kb && tid < BM) s_xs[buf ^ 1][tid] = xs_next;
    __syncthreads();                   // the next step has landed; this buffer's readers are done
  }

  const bool wide = p.N % 4 == 0 && reinterpret_cast<uintptr_t>(p.y) % (4 * Act<OUT>::bytes) == 0;
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    const int n = n0 + (wn * NT + i) * 16 + 4 * g;
    if (n >= p.N) continue;
    float bias[4] = {};
    if (p.bias) {
#pragma unroll
      for (int q = 0; q < 4; ++q)
        bias[q] = load_act<OUT>(p.bias, static_cast<size_t>(rt.expert) * p.N + min(n + q, p.N - 1));
    }
#pragma unroll
    for (int j = 0; j < MT; ++j) {
      const int64_t m = rt.begin + (wm * MT + j) * 16 + c16;
      if (m < rt.end) {
        float v[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) v[q] = acc[i][j][q] + bias[q];
        store4<OUT>(p, m, n, v, wide);
      }
    }
  }
}

template <int BN, int BM, int WN, int WM, int OUT>
hipError_t launch_tile(LinearF8Params p, hipStream_t s) {
  p.tiles_n = (p.N + BN - 1) / BN;
  // row tiles: with experts, each adds less than one tile to T / BM
  int64_t tiles_m = (p.T + BM - 1) / BM;
  if (p.offsets) tiles_m = p.T / BM + (p.T < p.E ? p.T : p.E);
  const int64_t blocks = tiles_m * p.tiles_n;
  if (blocks > 0x7fffffff / (64 * WN * WM)) return hipErrorInvalidConfiguration;
  linear_f8_tile_kernel<BN, BM, WN, WM, OUT>
      <<<dim3(static_cast<unsigned>(blocks)), dim3(64 * WN * WM), 0, s>>>(p);
  return hipGetLastError();
}

template <int OUT>
hipError_t launch_out(const LinearF8Params& p, hipStream_t s) {
  return launch_tile<64, 64, 2, 2, OUT>(p, s);
}

hipError_t launch_linear_f8(const LinearF8Params& p, int out, hipStream_t s) {
  switch (out) {
    case ACT_F32: return launch_out<ACT_F32>(p, s);
    case ACT_F16: return launch_out<ACT_F16>(p, s);
    default: return launch_out<ACT_BF16>(p, s);
  }
}

}  // namespace lowbit
