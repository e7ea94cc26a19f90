// Product of e4m3 codes with a scale for each block of 128 along K (and of 128
// weight rows), dense or grouped by expert:
//
//   y[t, n] = sum_b xs[t, b] ws[n / 128, b] P_b[t, n] (+ bias[n])
//   P_b     = sum over the 128 K positions of block b of xq * wq
//
// MFMAs over the block's 128 K positions give P_b of an output tile (fp32, from
// a zero accumulator); the two scales are multiplied once per column of the
// tile and applied by one fused multiply-add per output.  (Their product may
// leave fp32's normal range before the result does: below 2^-126 a term is off
// by up to 2^-150 |P_b| < 2^-125, past 2^128 it is infinite.  Applying them one
// after the other would move that border and cost a multiplication an output,
// which the 256 x 256 tiles have no room for beside their MFMAs.)  The weights are the MFMA's A
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

// Direct global -> LDS loads and their waits in inline assembly: the compiler
// drains every load before it reads LDS, the kernel waits only for the step
// that it reads next.  Lane l writes LDS at m0 + 16 l; there is no
// destination register.
__device__ __forceinline__ void dma16(const void* vaddr, uint32_t m0) {
  asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off"
               : : "v"(vaddr), "s"(m0) : "memory", "m0");
}
// At most N of this wave's loads still in flight and its LDS accesses done,
// then meet the block's other waves.
template <int N>
__device__ __forceinline__ void wait_loads_then_barrier() {
  static_assert(N >= 0 && N < 64, "vmcnt range (63: no wait for loads)");
  asm volatile("s_waitcnt vmcnt(%0)\n\ts_waitcnt lgkmcnt(0)\n\ts_barrier" : : "n"(N) : "memory");
}
template <typename T>
__device__ __forceinline__ uint32_t lds_address(T* p) {
  return static_cast<uint32_t>(reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) void*)p));
}

// Rows of expert e (clamped to 0 .. T; none past the last expert).
__device__ __forceinline__ void expert_rows(const LinearF8Params& p, int e, int64_t* lo, int64_t* hi) {
  *lo = *hi = 0;
  if (e < p.E) {
    *lo = min(max(static_cast<int64_t>(p.offsets[e]), int64_t{0}), p.T);
    *hi = min(max(static_cast<int64_t>(p.offsets[e + 1]), *lo), p.T);
  }
}

// Row tiles of BM rows that the call has in all (the same in every lane).
template <int BM>
__device__ __forceinline__ int64_t count_row_tiles(const LinearF8Params& p) {
  if (p.offsets == nullptr) return (p.T + BM - 1) / BM;
  int64_t n = 0;
  for (int e0 = 0; e0 < p.E; e0 += 64) {
    int64_t lo, hi;
    expert_rows(p, e0 + (threadIdx.x & 63), &lo, &hi);
    int own = static_cast<int>((hi - lo + BM - 1) / BM);
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) own += __shfl_xor(own, o);
    n += __builtin_amdgcn_readfirstlane(own);
  }
  return n;
}

// The expert and rows of row tile `tile` of the call.
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
    int64_t lo, hi;
    expert_rows(p, e0 + lane, &lo, &hi);
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
      const int at = __builtin_amdgcn_readlane(static_cast<int>(tile - first), src);
      const int lo_s = __builtin_amdgcn_readlane(static_cast<int>(lo), src);
      const int hi_s = __builtin_amdgcn_readlane(static_cast<int>(hi), src);
      t.begin = lo_s + static_cast<int64_t>(at) * BM;
      t.end = min(t.begin + BM, static_cast<int64_t>(hi_s));
      t.expert = e0 + src;
      return t;
    }
    before += __builtin_amdgcn_readlane(upto, 63);
  }
  return t;
}

// Tile of this block among tiles_m x tiles_n: blocks go to the 8 XCDs in turn,
// so each XCD takes a contiguous run of the tiles, and the runs go through
// patches GM row tiles high, so that the tiles an XCD has in flight share
// rows of both operands in its L2.
template <int GM>
__device__ __forceinline__ bool tile_of_block(int64_t tiles_m, int64_t tiles_n, int64_t* tm, int* tn) {
  const int64_t all = tiles_m * tiles_n, id = blockIdx.x;
  if (id >= all) return false;
  const int64_t q = all / 8, r = all % 8, xcd = id % 8;
  const int64_t at = xcd * q + min(xcd, r) + id / 8;
  const int64_t patch = at / (GM * tiles_n), rest = at - patch * (GM * tiles_n);
  const int64_t high = min(static_cast<int64_t>(GM), tiles_m - patch * GM);
  *tm = patch * GM + rest % high;
  *tn = static_cast<int>(rest / high);
  return true;
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

// A wave's outputs (NT x MT tiles, rows m0 .., columns n0 ..) rounded and
// turned through LDS, so that they leave as whole 16-byte pieces of y's rows
// from a short loop (unrolled stores of the accumulators with their edge cases
// are some 80 KB of code a wave runs once: 20 us of instruction fetches).
template <int OUT, int NT>
constexpr int kOutPitch = NT * 16 * Act<OUT>::bytes + 16;   // bytes of a row in LDS: 16 rows hit 16 bank groups
template <int OUT, int NT, int MT>
constexpr int kOutBytes = MT * 16 * kOutPitch<OUT, NT>;
template <int OUT, int NT, int MT>
__device__ __forceinline__ void store_outputs(const LinearF8Params& p, const f32x4_t (&acc)[NT][MT],
                                              uint8_t* lds, int expert, int64_t m0, int64_t m_end, int n0) {
  constexpr int E = Act<OUT>::bytes, PITCH = kOutPitch<OUT, NT>;
  const int lane = threadIdx.x & 63, c16 = lane & 15, g = lane >> 4;
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    float bias[4] = {};
    if (p.bias) {
#pragma unroll
      for (int q = 0; q < 4; ++q)
        bias[q] = load_act<OUT>(p.bias, static_cast<size_t>(expert) * p.N + min(n0 + 16 * i + 4 * g + q, p.N - 1));
    }
#pragma unroll
    for (int j = 0; j < MT; ++j) {
      uint8_t* at = lds + (16 * j + c16) * PITCH + (16 * i + 4 * g) * E;
      const f32x4_t v = acc[i][j];
      if constexpr (OUT == ACT_F32) {
        *reinterpret_cast<f32x4_t*>(at) = f32x4_t{v[0] + bias[0], v[1] + bias[1], v[2] + bias[2], v[3] + bias[3]};
      } else {
        *reinterpret_cast<u32v2_t*>(at) =
            u32v2_t{pack2<OUT>(v[0] + bias[0], v[1] + bias[1]), pack2<OUT>(v[2] + bias[2], v[3] + bias[3])};
      }
    }
  }
  constexpr int PIECE = 16 / E;        // outputs of 16 bytes
  constexpr int LANES = NT * 16 / PIECE;                // lanes of a row
  const bool wide = p.N % PIECE == 0 && reinterpret_cast<uintptr_t>(p.y) % 16 == 0;
  const int n = n0 + lane % LANES * PIECE;
#pragma unroll 1
  for (int r = lane / LANES; r < MT * 16; r += 64 / LANES) {
    const int64_t m = m0 + r;
    if (m >= m_end || n >= p.N) continue;
    const uint8_t* at = lds + r * PITCH + lane % LANES * 16;
    const u32v4_t v = *reinterpret_cast<const u32v4_t*>(at);
    typedef typename Act<OUT>::bits_t T;
    T* to = static_cast<T*>(p.y) + static_cast<size_t>(m) * p.N + n;
    if (wide) {
      *reinterpret_cast<u32v4_t*>(to) = v;
    } else {
#pragma unroll 1
      for (int k = 0; k < PIECE && n + k < p.N; ++k) to[k] = reinterpret_cast<const T*>(at)[k];
    }
  }
}

// What the activations past a row's end in its last, partial block are read
// from (the weights there read the block's first chunk: finite or NaN as the
// products they meet anyway), and a gathered row outside xq its scales.
__device__ __attribute__((aligned(16))) const uint32_t kZeroCodes[4] = {0u, 0u, 0u, 0u};
__device__ __attribute__((aligned(16))) const float kNanScales[4] = {
    __builtin_nanf(""), __builtin_nanf(""), __builtin_nanf(""), __builtin_nanf("")};

// Block of KG groups of WN x WM waves over BN columns (n) and BM rows (t) of y:
// each group takes a run of the block's K steps through a ring of its own, and
// their sums meet in LDS.  K steps of 128 go through a ring of S LDS stages, loaded S - 1 steps ahead; a step has
// one barrier, before which a wave waits for its own loads of that step; the
// loads of later steps go out behind the step's LDS reads.
// SPLIT: blockIdx.y takes a run of K blocks and writes fp32 partial sums.
// Two groups: the waves of two blocks a CU for tiles of which each CU has one,
// with no sums in memory to join (us, 64 x 32: 64 rows, 4096 x 4096 9.0 against
// 10.3 in K splits; 128 rows 9.5 against 11.3; 64 x 64: 200 rows 11.5 against 12.9
// of 64 x 32; four groups on rings of two stages 10.9 and 12.5; 128 x 128: 600
// rows 21.8 against 25.7, 1024 rows 24.4 against 27.2).
// Bound by the weights' bytes with few rows (8 rows, 14336 x 4096: 11.2 us, 5.2
// TB/s), in between by LDS: a step of 128 x 128 in waves of 64 x 32 reads 96 KiB
// and writes 32, 1024 cycles at 128 bytes each, for 512 cycles of MFMAs (64 x 64:
// 384 for 128; 64 x 32: 288 for 64).  Two blocks' steps take 1.29 us (0.57,
// 0.46), of which that is 0.85 (0.32, 0.24) at 2.4 GHz and more at the clock that
// the power leaves; the rest are the 1 KiB loads (some 50 cycles of the issuing
// wave each) and the barrier.  1024 rows, 4096 x 4096, 128 x 128: 24 us, 1.4
// PFLOP/s.  What follows moves no fewer bytes through LDS; measured and
// not kept: loads before the LDS reads (64 x 64, 512 rows, 4096 x 4096: 18.1
// against 17.4), loads between the MFMAs (20.1 against 18.6), a ring of four
// stages for 128 x 128, which leaves one block a CU (777 rows, 5000 x 4112: 46
// against 32.5; 1024 rows, 4096 x 4096, one block a CU anyway: 25 against 27), of
// two for 64 x 64 (64 rows, 14336 x 4096: 20 against 14), 128 x 64 tiles (512
// rows, 4096 x 4096: 16.8 against 17.3 of 64 x 64; 1024 rows: 31 against 27).
template <int BN, int BM, int WN, int WM, int S, int KG, bool SPLIT, int OUT>
__global__ __launch_bounds__(64 * WN * WM * KG) void linear_f8_tile_kernel(LinearF8Params p) {
  constexpr bool EXACT = OUT == ACT_F32;
  constexpr int NW = WN * WM;
  constexpr int NT = BN / WN / 16, MT = BM / WM / 16;   // 16-wide tiles of a wave
  constexpr int ROWS = BN + BM;
  constexpr int LOADS = ROWS / 8 / NW;                  // 1 KiB loads of a wave per step
  static_assert(ROWS % (8 * NW) == 0 && BN % 8 == 0, "whole loads");
  constexpr int XROWS = BM > 64 ? BM : 64;              // rows of scales: one load of a wave each 64
  static_assert(XROWS % 64 == 0 && XROWS <= 64 * NW, "one scale load a wave");
  static_assert((16 * NT) <= kF8Block && kF8Block % (16 * NT) == 0, "a wave's columns share a scale");
  constexpr int STAGE = ROWS * kF8Block;
  constexpr int OUT_BYTES = SPLIT ? 0 : NW * kOutBytes<OUT, NT, MT>;
  constexpr int RINGS = KG * S * STAGE, AFTER = OUT_BYTES + (KG - 1) * NW * NT * MT * 1024;   // (groups' sums)
  __shared__ __attribute__((aligned(1024))) uint8_t s_mem[RINGS > AFTER ? RINGS : AFTER];
  __shared__ __attribute__((aligned(1024))) float s_xs[KG][2][XROWS][4];

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wv = wave % NW, kg = wave / NW;
  uint8_t* const ring = s_mem + kg * (S * STAGE);
  int64_t tile_m;
  int tile_n;
  if (!tile_of_block<BM >= 128 ? 8 : 16>(count_row_tiles<BM>(p), p.tiles_n, &tile_m, &tile_n)) return;
  const RowTile rt = find_rows<BM>(p, tile_m);
  if (rt.expert < 0) return;
  const int n0 = tile_n * BN;
  const int wn = wv % WN, wm = wv / WN;
  const uint8_t* wq = p.wq + static_cast<size_t>(rt.expert) * p.N * p.K;
  // (a wave past N has no columns and takes the last scale row)
  // in the constant address space: scalar loads, which no vector load waits for
  typedef const __attribute__((address_space(4))) float* scalar_floats;
  const scalar_floats ws = (scalar_floats)(p.ws + (static_cast<size_t>(rt.expert) * p.nb +
                            min((n0 + wn * NT * 16) / kF8Block, p.nb - 1)) * p.kb);
  const int b_first = SPLIT ? static_cast<int>(blockIdx.y) * p.kb_split : 0;
  const int b_last = SPLIT ? min(b_first + p.kb_split, p.kb) : p.kb;
  const int steps = (b_last - b_first + KG - 1) / KG;   // of the block: its barriers
  const int b_begin = b_first + kg * steps;
  const int b_end = min(b_begin + steps, b_last);       // (a last group may have none)

  // load i of this wave: rows 8 (wv LOADS + i) .. + 7 of the step's BN weight
  // rows and BM activation rows; lane l fills position l % 8 of row l / 8.
  // The scale load's lane takes row 64 wv + lane, in the first waves (rows past
  // BM: padding of s_xs).  Rows past the tile's end are its last row again.
  int64_t from[LOADS + 1];
  int chunk[LOADS];
#pragma unroll
  for (int i = 0; i <= LOADS; ++i) {
    const int r = i == LOADS ? BN + min(64 * wv + lane, BM - 1) : 8 * (wv * LOADS + i) + (lane >> 3);
    if (i < LOADS) chunk[i] = (lane & 7) ^ swizzle(r);
    from[i] = r < BN ? min(n0 + r, p.N - 1) : min(rt.begin + (r - BN), rt.end - 1);
  }
  if (p.rows) {                        // (all index loads before the first use)
    int32_t at[LOADS + 1];
#pragma unroll
    for (int i = 0; i <= LOADS; ++i) {
      const bool x = i == LOADS || 8 * (wv * LOADS + i) + (lane >> 3) >= BN;
      at[i] = p.rows[x ? from[i] : rt.begin];
    }
#pragma unroll
    for (int i = 0; i <= LOADS; ++i) {
      const bool x = i == LOADS || 8 * (wv * LOADS + i) + (lane >> 3) >= BN;
      if (x) from[i] = at[i];
    }
  }
  const uint8_t* src[LOADS];
#pragma unroll
  for (int i = 0; i < LOADS; ++i) {
    const bool x = 8 * (wv * LOADS + i) + (lane >> 3) >= BN;
    const int64_t r = x && (from[i] < 0 || from[i] >= p.M) ? 0 : from[i];
    src[i] = (x ? p.xq : wq) + static_cast<size_t>(r) * p.K + 16 * chunk[i];
  }
  const bool xs_ok = from[LOADS] >= 0 && from[LOADS] < p.M;
  const float* xs = p.xs + (xs_ok ? from[LOADS] : 0) * p.kb;
  const int tail = (p.K & (kF8Block - 1)) / 16;         // chunks of a last, partial block (0: none)
  const uint32_t codes0 = lds_address(ring) + wv * LOADS * 8 * kF8Block;
  const uint32_t xs0 = lds_address(&s_xs[kg][0][0][0]) + wv * 64 * 16;
  auto load_step = [&](int b, int stage) {
    const uint32_t dst = codes0 + stage * STAGE;
    const size_t at = static_cast<size_t>(b) * kF8Block;
    if (tail != 0 && b == p.kb - 1) {
#pragma unroll
      for (int i = 0; i < LOADS; ++i) {
        const bool x = 8 * (wv * LOADS + i) >= BN;
        const uint8_t* past = x ? reinterpret_cast<const uint8_t*>(kZeroCodes) : src[i] + at - 16 * chunk[i];
        dma16(chunk[i] < tail ? src[i] + at : past, dst + i * 8 * kF8Block);
      }
    } else {
#pragma unroll
      for (int i = 0; i < LOADS; ++i) dma16(src[i] + at, dst + i * 8 * kF8Block);
    }
  };
  // Scales of four K blocks q .. q + 3 at once (a row's scales lie kb apart:
  // every lane reads a line of its own): one 16-byte load a lane, shifted back
  // inside the row at its end.
  auto xs_first = [&](int q) { return max(min(q, p.kb - 4), 0); };
  const bool has_xs = wv < XROWS / 64;
  auto load_scales = [&](int q, int half) {
    if (has_xs) dma16(xs_ok ? xs + xs_first(q) : kNanScales, xs0 + half * (XROWS * 16));
  };

  const int c16 = lane & 15, g = lane >> 4;
  f32x4_t acc[NT][MT];
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int j = 0; j < MT; ++j) acc[i][j] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};

  // chunks g and g + 4 (lane group g's K positions) of row 16 i + c16, whose
  // swizzle is that of row c16
  const int lo_at = c16 * kF8Block + 16 * (g ^ swizzle(c16));
  const int hi_at = c16 * kF8Block + 16 * ((g + 4) ^ swizzle(c16));
  auto compute = [&](int stage, const float* x_scale, float w_scale, auto&& meanwhile) {
    const uint8_t* wrow = ring + stage * STAGE + wn * NT * 16 * kF8Block;
    const uint8_t* xrow = ring + stage * STAGE + (BN + wm * MT * 16) * kF8Block;
    F8Fragment<EXACT> xf[MT];
    float s[MT];
#pragma unroll
    for (int j = 0; j < MT; ++j) {
      xf[j].set(*reinterpret_cast<const u32v4_t*>(xrow + lo_at + j * 16 * kF8Block),
                *reinterpret_cast<const u32v4_t*>(xrow + hi_at + j * 16 * kF8Block));
      s[j] = w_scale * x_scale[((wm * MT + j) * 16 + c16) * 4];
    }
    F8Fragment<EXACT> wf[NT];
#pragma unroll
    for (int i = 0; i < NT; ++i)
      wf[i].set(*reinterpret_cast<const u32v4_t*>(wrow + lo_at + i * 16 * kF8Block),
                *reinterpret_cast<const u32v4_t*>(wrow + hi_at + i * 16 * kF8Block));
    __builtin_amdgcn_sched_barrier(0);
    meanwhile();
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      f32x4_t P[MT];
#pragma unroll
      for (int j = 0; j < MT; ++j) P[j] = mfma_f8(wf[i], xf[j]);
#pragma unroll
      for (int j = 0; j < MT; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q) acc[i][j][q] = fmaf(s[j], P[j][q], acc[i][j][q]);
    }
  };

  if (p.kb >= 4) {
    load_scales(b_begin, 0);
  } else if (has_xs) {                 // rows shorter than one 16-byte load
    for (int q = 0; q < p.kb; ++q) s_xs[kg][0][64 * wv + lane][q] = xs_ok ? xs[q] : kNanScales[q];
  }
#pragma unroll
  for (int n = 0; n < S - 1; ++n)
    if (b_begin + n < b_end) load_step(b_begin + n, n);
  // four K blocks a round: what a round needs once is done once, and stages and
  // scale slots are constants
  static_assert(4 % S == 0, "the ring's stages repeat every round");
  int half = 0;
  for (int q = b_begin; q < b_begin + steps; q += 4, half ^= 1) {
    const float* x_scale = &s_xs[kg][half][0][q - xs_first(q)];
    float w_scale[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) w_scale[u] = ws[min(q + u, b_end - 1)];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int b = q + u;
      if (b >= b_begin + steps) break;
      // step b has landed (the code loads of the S - 2 steps after it may be in
      // flight, while there are that many) and every wave has read step b - 1
      if (b + S - 1 <= b_end) wait_loads_then_barrier<(S - 2) * LOADS>();
      else wait_loads_then_barrier<0>();
      if (KG > 1 && b >= b_end) continue;               // (the last group's: only the barrier)
      compute(u % S, x_scale + u, w_scale[u], [&]() {
        if (u == 0 && q + 4 < b_end) load_scales(q + 4, half ^ 1);
        if (b + S - 1 < b_end) load_step(b + S - 1, (u + S - 1) % S);
      });
    }
  }

  if constexpr (KG > 1) {              // the groups' sums meet in the first, in their order
    wait_loads_then_barrier<0>();      // every wave has read its last stage
    f32x4_t* const sums = reinterpret_cast<f32x4_t*>(s_mem + OUT_BYTES);
    if (kg > 0) {
#pragma unroll
      for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int j = 0; j < MT; ++j) sums[((((kg - 1) * NW + wv) * NT + i) * MT + j) * 64 + lane] = acc[i][j];
    }
    wait_loads_then_barrier<0>();
    if (kg > 0) return;
#pragma unroll
    for (int k = 1; k < KG; ++k)
#pragma unroll
      for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int j = 0; j < MT; ++j) acc[i][j] += sums[((((k - 1) * NW + wv) * NT + i) * MT + j) * 64 + lane];
  }
  if constexpr (SPLIT) {
    // planes of T rows of n_pad (a multiple of 4) columns
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      const int n = n0 + (wn * NT + i) * 16 + 4 * g;
#pragma unroll
      for (int j = 0; j < MT; ++j) {
        const int64_t m = rt.begin + (wm * MT + j) * 16 + c16;
        if (m < rt.end && n < p.N)
          *reinterpret_cast<f32x4_t*>(p.partials + (blockIdx.y * p.T + m) * p.n_pad + n) = acc[i][j];
      }
    }
  } else {
    if constexpr (KG == 1) wait_loads_then_barrier<0>();    // every wave has read the last stage
    store_outputs<OUT>(p, acc, s_mem + wv * kOutBytes<OUT, NT, MT>, rt.expert, rt.begin + wm * MT * 16, rt.end,
                       n0 + wn * NT * 16);
  }
}

// Many rows: 256 x 256 tiles, 8 waves of 128 (n) x 64 (t), the ring two
// stages of 64 KiB.  Direct loads through buffer descriptors: a lane offset per
// load (row and chunk) and a scalar base that moves on by 128 bytes a step, so
// that no wave keeps 64-bit addresses; rows past N or past the tile's end lie
// past the descriptor's end and read nothing.
// A step has 2048 MFMA cycles a CU and as many of LDS traffic (192 KiB read, 64
// KiB written, 128 bytes a cycle), and a scaling FMA a product in the MFMAs'
// shadow.  8192 rows of K = 4096 into N = 14336: 421-429 us, 2.2-2.3 PFLOP/s
// (a large unscaled e4m3 library product: 2.9-3.2); 352 us on codes of zero: the
// rest is the clock that the card's power leaves (1.8 to 2.0 of 2.4 GHz).  What
// each form measured (us, one card): one barrier a step and loads in pairs 452, a
// load a tile 436; without loads 354.  MFMAs of 32 x 32 x 64 are no faster beside
// the FMAs (registers only: 3.45 PFLOP/s against 3.80).
typedef int32_t i32x4_t __attribute__((ext_vector_type(4)));
__device__ __forceinline__ i32x4_t buffer_of(const void* base, uint64_t bytes) {
  const uint64_t a = reinterpret_cast<uint64_t>(base);
  const uint32_t size = (bytes >> 32) != 0 ? 0xffffffffu : static_cast<uint32_t>(bytes);
  return i32x4_t{__builtin_amdgcn_readfirstlane(static_cast<int32_t>(a)),
                 __builtin_amdgcn_readfirstlane(static_cast<int32_t>((a >> 32) & 0xffff)),
                 __builtin_amdgcn_readfirstlane(static_cast<int32_t>(size)), 0x00020000};
}
__device__ __forceinline__ void dma16_buffer(uint32_t voff, i32x4_t buf, uint32_t m0) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tbuffer_load_dwordx4 %0, %1, 0 offen lds"
               : : "v"(voff), "s"(buf), "s"(m0) : "memory", "m0");
}

// (K of four blocks or more)
template <int OUT>
__global__ __launch_bounds__(512, 2) void linear_f8_big_kernel(LinearF8Params p) {
  static_assert(OUT != ACT_F32, "fp8 MFMA sums are not fp32");
  constexpr int BN = 256, BM = 256, WN = 2, NT = 8, MT = 4;
  constexpr int STAGE = (BN + BM) * kF8Block;
  constexpr int OUT_BYTES = 8 * kOutBytes<OUT, NT, MT>;
  __shared__ __attribute__((aligned(1024))) uint8_t s_mem[2 * STAGE > OUT_BYTES ? 2 * STAGE : OUT_BYTES];
  __shared__ __attribute__((aligned(1024))) float s_xs[2][BM][4];

  const int lane = threadIdx.x & 63;
  const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  int64_t tile_m;
  int tile_n;
  if (!tile_of_block<8>(count_row_tiles<BM>(p), p.tiles_n, &tile_m, &tile_n)) return;
  const RowTile rt = find_rows<BM>(p, tile_m);
  if (rt.expert < 0) return;
  const int n0 = tile_n * BN;
  const int wn = wv % WN, wm = wv / WN;
  // the weights' scales of 64 K blocks, one a lane: a scalar load in the loop
  // would make every wait for LDS a wait for all of it
  const float* ws = p.ws + (static_cast<size_t>(rt.expert) * p.nb +
                            min((n0 + wn * NT * 16) / kF8Block, p.nb - 1)) * p.kb;
  float ws64 = ws[min(lane, p.kb - 1)];
  const uint8_t* wbase = p.wq + (static_cast<size_t>(rt.expert) * p.N + n0) * p.K;
  const uint8_t* xbase = p.rows ? p.xq : p.xq + static_cast<size_t>(rt.begin) * p.K;
  const uint64_t wbytes = static_cast<uint64_t>(p.N - n0) * p.K;
  const uint64_t xbytes = static_cast<uint64_t>(p.rows ? p.M : rt.end - rt.begin) * p.K;
  const int last_chunks = (p.K - (p.kb - 1) * kF8Block) / 16;   // of the last block: 1 .. 8

  // A wave loads 32 activation rows and 32 weight rows of a step, 8 rows a load:
  // activation rows 32 wv + 8 k; weight rows of pieces 0 and 1 in the upper half
  // of a column wave's 128 rows, of pieces 2 and 3 in the lower half.  Lane l
  // fills position l % 8 of row l / 8.
  const int sub = lane >> 3;
  const int chunk0 = (lane & 7) ^ swizzle(sub);         // of even pieces; odd ones: ^ 4
  const int wrow0 = (wv >> 2) * (BN / 2) + (wv & 3) * 16;
  const uint32_t woff = (wrow0 + sub) * p.K;
  uint32_t xoff[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int r = 32 * wv + 8 * k + sub;
    int from = r;
    if (p.rows) {
      from = p.rows[min(rt.begin + r, rt.end - 1)];
      if (from < 0 || from >= p.M) from = 0;
    }
    xoff[k] = static_cast<uint32_t>(from) * p.K;
  }
  const float* xs = kNanScales;        // of row 64 wv + lane; waves 0 .. 3 load them
  bool xs_ok = false;
  if (wv < BM / 64) {
    int64_t from = min(rt.begin + 64 * wv + lane, rt.end - 1);
    if (p.rows) from = p.rows[from];
    xs_ok = from >= 0 && from < p.M;
    if (xs_ok) xs = p.xs + from * p.kb;
  }
  const uint32_t wcodes0 = lds_address(s_mem) + wrow0 * kF8Block;
  const uint32_t xcodes0 = lds_address(s_mem) + (BN + wv * 32) * kF8Block;
  const uint32_t xs0 = lds_address(&s_xs[0][0][0]) + wv * 64 * 16;
  // (without branches, so that the loads can stand between a step's MFMAs: a
  // step past the last one reads nothing, from a descriptor of no bytes.  Past
  // the row's end in the last block: zeros for the activations (an offset past
  // the buffer), the block's first chunk for the weights they meet.)
  auto past_row = [&](int b, int chunk) { return b == p.kb - 1 && chunk >= last_chunks; };
  auto load_x = [&](int b, int k) {
    const uint64_t at = static_cast<uint64_t>(b) * kF8Block;
    const int chunk = k & 1 ? chunk0 ^ 4 : chunk0;
    dma16_buffer(past_row(b, chunk) ? 0xfffffff0u : xoff[k] + 16 * chunk,
                 buffer_of(xbase + at, b < p.kb ? xbytes - at : 0), xcodes0 + (b & 1) * STAGE + 8 * k * kF8Block);
  };
  auto load_w = [&](int b, int k) {
    const uint64_t at = static_cast<uint64_t>(b) * kF8Block;
    const int chunk = k & 1 ? chunk0 ^ 4 : chunk0, r = (k >> 1) * (BN / 4) + (k & 1) * 8;
    dma16_buffer(woff + r * p.K + (past_row(b, chunk) ? 0 : 16 * chunk),
                 buffer_of(wbase + at, b < p.kb ? wbytes - at : 0), wcodes0 + (b & 1) * STAGE + r * kF8Block);
  };
  auto xs_first = [&](int q) { return min(q, p.kb - 4); };
  auto load_four_scales = [&](int q, int half) {
    if (wv < BM / 64) dma16(xs_ok ? xs + xs_first(q) : xs, xs0 + half * (BM * 16));
  };

  const int c16 = lane & 15, g = lane >> 4;
  f32x4_t acc[NT][MT];
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int j = 0; j < MT; ++j) acc[i][j] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
  const int lo_at = c16 * kF8Block + 16 * (g ^ swizzle(c16));
  const int hi_at = c16 * kF8Block + 16 * ((g + 4) ^ swizzle(c16));
  F8Fragment<false> xf[MT], wf[3];
  f32x4_t P[4];                        // the products of the last four MFMAs
  float s[MT], s_last[MT];             // the scales of this step and of the one before
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    P[j] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
    s[j] = 0.0f;
  }
  auto read_x = [&](int j, int stage) {
    const uint8_t* xrow = s_mem + stage * STAGE + (BN + (wm * MT + j) * 16) * kF8Block;
    xf[j].set(*reinterpret_cast<const u32v4_t*>(xrow + lo_at), *reinterpret_cast<const u32v4_t*>(xrow + hi_at));
  };
  // (three fragments: the two last column tiles of a step and the first of the next)
  auto w_slot = [](int i) { return i == 4 || i == 7 ? 2 : i == 1 || i == 3 || i == 6 ? 1 : 0; };
  auto read_w = [&](int i, int stage) {
    const uint8_t* wrow = s_mem + stage * STAGE + (wn * NT + i) * 16 * kF8Block;
    wf[w_slot(i)].set(*reinterpret_cast<const u32v4_t*>(wrow + lo_at),
                      *reinterpret_cast<const u32v4_t*>(wrow + hi_at));
  };
  auto read_scales = [&](const float* x_scale, int b) {
    const float w_scale = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(ws64), b & 63));
#pragma unroll
    for (int j = 0; j < MT; ++j) {
      s_last[j] = s[j];
      s[j] = w_scale * x_scale[((wm * MT + j) * 16 + c16) * 4];
    }
  };
  // MFMA n of a step's 32: column tile by column tile, the last two together.
  // Each stands behind the scaling of the products that it replaces (those of
  // the fourth MFMA before it), in the shadow of the MFMA before.
  auto tile_i = [](int n) { return n < 24 ? n / 4 : 6 + (n & 1); };
  auto tile_j = [](int n) { return n < 24 ? n % 4 : (n - 24) / 2; };
  auto add_products = [&](int n, const float (&sc)[MT]) {
    const int i = tile_i(n), j = tile_j(n);
#pragma unroll
    for (int q = 0; q < 4; ++q) acc[i][j][q] = fmaf(sc[j], P[n & 3][q], acc[i][j][q]);
  };
  auto mfma = [&](int n) {
    if (n < 4) add_products(n + 28, s_last);
    else add_products(n - 4, s);
    P[n & 3] = mfma_f8(wf[w_slot(tile_i(n))], xf[tile_j(n)]);
    __builtin_amdgcn_sched_group_barrier(0x002, 4, 0);
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
  };

  // (keeps the compiler from sinking the sums below the branches that follow,
  // which would keep every product in a register until then)
  auto settle_sums = [&]() {
#pragma unroll
    for (int i = 0; i < NT; ++i)
      asm volatile("" : "+v"(acc[i][0]), "+v"(acc[i][1]), "+v"(acc[i][2]), "+v"(acc[i][3]));
  };

  // A step has two barriers.  Past the first, before its fourth column tile, its
  // lower weight rows have landed, and its activations and upper weight rows are
  // free for the step after next; past the second, before its last two tiles, the
  // next step's activations and upper weight rows have landed, and its lower
  // weight rows are free for the step after next.  So each wave issues one load a
  // column tile (a load holds up the wave that issues it for some 50 cycles, more
  // where all waves issue several at once), and six tiles or more pass before one
  // is waited for.  The next step's activations are read between the MFMAs of the
  // last two column tiles, each over a fragment that these need no more (all at
  // once they would hold up every wave).
  int half = 0, first = 0;
  load_four_scales(0, 0);
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    load_x(0, k);
    load_w(0, k);
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) load_x(1, k);
  load_w(1, 0);
  wait_loads_then_barrier<5>();
  if (p.kb > 4) load_four_scales(4, 1);
  read_w(0, 0);
#pragma unroll
  for (int j = 0; j < MT; ++j) read_x(j, 0);
  read_scales(&s_xs[0][0][0], 0);
  for (int b = 0; b < p.kb; ++b) {
    const int nb = b + 1, stage = b & 1;
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int i = 0; i < 6; ++i) {
      if (i == 0) load_w(nb, 1);
      if (i == 1 || i == 2) load_w(nb, 1 + i);
      if (i == 3) wait_loads_then_barrier<8>();
      if (i >= 3) load_x(nb + 1, i - 3);
      read_w(i + 1, stage);
      if (i == 5) read_w(7, stage);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int j = 0; j < MT; ++j) mfma(4 * i + j);
      __builtin_amdgcn_sched_barrier(0);
    }
    wait_loads_then_barrier<5>();
    load_x(nb + 1, 3);
#pragma unroll
    for (int j = 0; j < MT; ++j) {
      if (j == 2) load_w(nb + 1, 0);
      mfma(24 + 2 * j);
      mfma(25 + 2 * j);
      __builtin_amdgcn_sched_barrier(0);
      read_x(j, stage ^ 1);
      if (j == 1) read_w(0, stage ^ 1);
      __builtin_amdgcn_sched_barrier(0);
    }
    settle_sums();
    if ((nb & 3) == 0) {
      half ^= 1;
      first = xs_first(nb);
      if (nb + 4 < p.kb) load_four_scales(nb + 4, half ^ 1);
      if ((nb & 63) == 0) {
        ws64 = ws[min(nb + lane, p.kb - 1)];
        asm volatile("" : "+v"(ws64));                  // waited for here, not at each use
      }
    }
    read_scales(&s_xs[half][0][min(nb, p.kb - 1) - first], nb);
  }
#pragma unroll
  for (int n = 28; n < 32; ++n) add_products(n, s_last);
  settle_sums();

  wait_loads_then_barrier<0>();        // every wave has read the last stage
  store_outputs<OUT>(p, acc, s_mem + wv * kOutBytes<OUT, NT, MT>, rt.expert, rt.begin + wm * MT * 16, rt.end,
                     n0 + wn * NT * 16);
}

template <int OUT>
hipError_t launch_big(LinearF8Params p, hipStream_t s) {
  p.tiles_n = (p.N + 255) / 256;
  int64_t tiles_m = (p.T + 255) / 256;
  if (p.offsets) tiles_m = p.T / 256 + (p.T < p.E ? p.T : p.E);
  const int64_t blocks = tiles_m * p.tiles_n;
  if (blocks > kF8MaxThreads / 512) return hipErrorInvalidConfiguration;
  linear_f8_big_kernel<OUT><<<dim3(static_cast<unsigned>(blocks)), dim3(512), 0, s>>>(p);
  return hipGetLastError();
}

// Sum of the K splits' planes, in their order, and the bias, for the rows of the
// call (of the experts): four columns a thread.  128 x 4096 in four splits: 3.9 us
// of 21, most of it a launch (in two: 4.0).
template <int OUT>
__global__ __launch_bounds__(256) void linear_f8_reduce_kernel(LinearF8Params p, int splits) {
  int64_t lo = 0, hi = p.T;
  if (p.offsets) {
    lo = min(max(static_cast<int64_t>(p.offsets[0]), int64_t{0}), p.T);
    hi = min(max(static_cast<int64_t>(p.offsets[p.E]), lo), p.T);
  }
  const int quads = p.n_pad / 4;
  const int64_t id = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  const int64_t m = id / quads;
  if (m < lo || m >= hi) return;
  const int n = static_cast<int>(id - m * quads) * 4;
  f32x4_t sum = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int k = 0; k < splits; ++k)
    sum += *reinterpret_cast<const f32x4_t*>(p.partials + (k * p.T + m) * p.n_pad + n);
  if (p.bias) {
    int e = 0;                         // the last expert that begins at or before row m
    for (int end = p.offsets ? p.E : 1; end - e > 1;) {
      const int mid = (e + end) / 2;
      if (p.offsets[mid] <= m) e = mid;
      else end = mid;
    }
#pragma unroll
    for (int q = 0; q < 4; ++q)
      sum[q] += load_act<OUT>(p.bias, static_cast<size_t>(e) * p.N + min(n + q, p.N - 1));
  }
  const bool wide = p.N % 4 == 0 && reinterpret_cast<uintptr_t>(p.y) % (4 * Act<OUT>::bytes) == 0;
  const float v[4] = {sum[0], sum[1], sum[2], sum[3]};
  store4<OUT>(p, m, n, v, wide);
}

// Few rows: a block computes 16 NT columns of 16 MT rows over all of K, its W
// waves each a run of K blocks; their sums meet in LDS in a fixed order.  The
// weights go straight from memory to the MFMA operand (a step of a row is 128
// consecutive bytes, two 16-byte loads of four lanes each), U steps ahead.
// Bound by the weights' bytes: 64 tokens to 8 of 64 experts, 1408 x 2048, 38.7
// us, 4.8 TB/s; one row, 8192 x 2048, 5.3 us (a launch that does nothing takes
// about 2).
template <int NT, int MT, int W, int U, int OUT>
__global__ __launch_bounds__(64 * W) void linear_f8_rows_kernel(LinearF8Params p) {
  constexpr bool EXACT = OUT == ACT_F32;
  __shared__ f32x4_t s_acc[W][NT][MT][64];
  const int lane = threadIdx.x & 63;
  const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n0 = (blockIdx.x % p.tiles_n) * 16 * NT;
  const RowTile rt = find_rows<16 * MT>(p, blockIdx.x / p.tiles_n);
  if (rt.expert < 0) return;
  const int c16 = lane & 15, g = lane >> 4;
  const uint8_t* wrow[NT];
#pragma unroll
  for (int i = 0; i < NT; ++i)
    wrow[i] = p.wq + (static_cast<size_t>(rt.expert) * p.N + min(n0 + 16 * i + c16, p.N - 1)) * p.K;
  const float* ws = p.ws + (static_cast<size_t>(rt.expert) * p.nb + n0 / kF8Block) * p.kb;
  const uint8_t* xrow[MT];
  const float* xs[MT];
  bool ok[MT];
#pragma unroll
  for (int j = 0; j < MT; ++j) {
    const int64_t t = min(rt.begin + 16 * j + c16, rt.end - 1);
    int64_t r = p.rows ? p.rows[t] : t;
    ok[j] = r >= 0 && r < p.M;
    r = ok[j] ? r : 0;
    xrow[j] = p.xq + static_cast<size_t>(r) * p.K;
    xs[j] = p.xs + r * p.kb;
  }
  const int tail = (p.K & (kF8Block - 1)) / 16;
  const int per = (p.kb + W - 1) / W;
  const int begin = wv * per, end = min(begin + per, p.kb);

  struct Steps {
    u32v4_t w[U][NT][2], x[U][MT][2];
    float xs[U][MT], ws[U];
  };
  // (a step past the run loads the run's last block again, with scale 0)
  auto load = [&](int b0, Steps& st) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int b = min(b0 + u, end - 1);
      const int valid = (tail != 0 && b == p.kb - 1) ? tail : 8;
      const size_t at = static_cast<size_t>(b) * kF8Block;
      const int c0 = g < valid ? g : 0, c1 = g + 4 < valid ? g + 4 : 0;
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        st.w[u][i][0] = *reinterpret_cast<const u32v4_t*>(wrow[i] + at + 16 * c0);
        st.w[u][i][1] = *reinterpret_cast<const u32v4_t*>(wrow[i] + at + 16 * c1);
      }
      st.ws[u] = ws[b];
#pragma unroll
      for (int j = 0; j < MT; ++j) {
        st.x[u][j][0] = *reinterpret_cast<const u32v4_t*>(xrow[j] + at + 16 * c0);
        st.x[u][j][1] = *reinterpret_cast<const u32v4_t*>(xrow[j] + at + 16 * c1);
        st.xs[u][j] = xs[j][b];
      }
    }
  };
  f32x4_t acc[NT][MT];
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int j = 0; j < MT; ++j) acc[i][j] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
  if (begin < end) {
    Steps cur;
    load(begin, cur);
    for (int b0 = begin; b0 < end; b0 += U) {
      Steps nxt;
      if (b0 + U < end) load(b0 + U, nxt);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int b = b0 + u;
        const int valid = (tail != 0 && b >= p.kb - 1) ? tail : 8;
        F8Fragment<EXACT> wf[NT];
#pragma unroll
        for (int i = 0; i < NT; ++i) wf[i].set(cur.w[u][i][0], cur.w[u][i][1]);
#pragma unroll
        for (int j = 0; j < MT; ++j) {
          u32v4_t lo = cur.x[u][j][0], hi = cur.x[u][j][1];
          if (valid < 8) {
            if (g >= valid) lo = u32v4_t{0u, 0u, 0u, 0u};
            if (g + 4 >= valid) hi = u32v4_t{0u, 0u, 0u, 0u};
          }
          F8Fragment<EXACT> xf;
          xf.set(lo, hi);
          const float s = b < end ? cur.ws[u] * cur.xs[u][j] : 0.0f;
#pragma unroll
          for (int i = 0; i < NT; ++i) {
            const f32x4_t P = mfma_f8(wf[i], xf);
#pragma unroll
            for (int q = 0; q < 4; ++q) acc[i][j][q] = fmaf(s, P[q], acc[i][j][q]);
          }
        }
      }
      cur = nxt;
    }
  }
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int j = 0; j < MT; ++j) s_acc[wv][i][j][lane] = acc[i][j];
  __syncthreads();
  const bool wide = p.N % 4 == 0 && reinterpret_cast<uintptr_t>(p.y) % (4 * Act<OUT>::bytes) == 0;
#pragma unroll
  for (int f = 0; f < NT * MT; ++f) {
    if (f % W != wv) continue;
    const int i = f / MT, j = f % MT;
    const int n = n0 + 16 * i + 4 * g;
    const int64_t m = rt.begin + 16 * j + c16;
    if (n >= p.N || m >= rt.end) continue;
    f32x4_t sum = s_acc[0][i][j][lane];
#pragma unroll
    for (int w = 1; w < W; ++w) sum += s_acc[w][i][j][lane];
    float v[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      v[q] = sum[q];
      if (p.bias) v[q] += load_act<OUT>(p.bias, static_cast<size_t>(rt.expert) * p.N + min(n + q, p.N - 1));
      if (!ok[j]) v[q] = __builtin_nanf("");
    }
    store4<OUT>(p, m, n, v, wide);
  }
}

template <int NT, int MT, int W, int U, int OUT>
hipError_t launch_rows(LinearF8Params p, hipStream_t s) {
  p.tiles_n = (p.N + 16 * NT - 1) / (16 * NT);
  int64_t tiles_m = (p.T + 16 * MT - 1) / (16 * MT);
  if (p.offsets) tiles_m = p.T / (16 * MT) + (p.T < p.E ? p.T : p.E);
  const int64_t blocks = tiles_m * p.tiles_n;
  if (blocks > kF8MaxThreads / (64 * W)) return hipErrorInvalidConfiguration;
  linear_f8_rows_kernel<NT, MT, W, U, OUT><<<dim3(static_cast<unsigned>(blocks)), dim3(64 * W), 0, s>>>(p);
  return hipGetLastError();
}

template <int BN, int BM, int WN, int WM, int S, int KG, int OUT>
hipError_t launch_tile(LinearF8Params p, int splits, hipStream_t s) {
  p.tiles_n = (p.N + BN - 1) / BN;
  // row tiles: with experts, each adds less than one tile to T / BM
  int64_t tiles_m = (p.T + BM - 1) / BM;
  if (p.offsets) tiles_m = p.T / BM + (p.T < p.E ? p.T : p.E);
  const int64_t blocks = tiles_m * p.tiles_n;
  if (blocks > kF8MaxThreads / (64 * WN * WM * KG)) return hipErrorInvalidConfiguration;
  const dim3 block(64 * WN * WM * KG);
  if (splits <= 1) {
    linear_f8_tile_kernel<BN, BM, WN, WM, S, KG, false, OUT>
        <<<dim3(static_cast<unsigned>(blocks)), block, 0, s>>>(p);
    return hipGetLastError();
  }
  const int64_t quads = p.T * ((p.N + 3) / 4);
  if (quads > 0xffffff00ll) return hipErrorInvalidConfiguration;
  p.kb_split = (p.kb + splits - 1) / splits;
  splits = (p.kb + p.kb_split - 1) / p.kb_split;
  p.n_pad = (p.N + 3) / 4 * 4;
  linear_f8_tile_kernel<BN, BM, WN, WM, S, KG, true, OUT>
      <<<dim3(static_cast<unsigned>(blocks), splits), block, 0, s>>>(p);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  linear_f8_reduce_kernel<OUT><<<dim3(static_cast<unsigned>((quads + 255) / 256)), dim3(256), 0, s>>>(p, splits);
  return hipGetLastError();
}

// One entry per output type and variant (LinearF8Plan, chosen by the host).
template <int OUT>
hipError_t launch_out(const LinearF8Params& p, const LinearF8Plan& plan, hipStream_t s) {
  switch (plan.kind) {
    case F8_ROWS_NT1: return launch_rows<1, 1, 8, 2, OUT>(p, s);
    case F8_ROWS_NT2: return launch_rows<2, 1, 8, 1, OUT>(p, s);
    case F8_ROWS_NT4: return launch_rows<4, 1, 4, 1, OUT>(p, s);
    case F8_TILE_64X32: return launch_tile<64, 32, 4, 1, 4, 1, OUT>(p, plan.splits, s);
    case F8_TILE_64X32_K2: return launch_tile<64, 32, 4, 1, 4, 2, OUT>(p, plan.splits, s);
    case F8_TILE_64X64: return launch_tile<64, 64, 2, 2, 4, 1, OUT>(p, plan.splits, s);
    case F8_TILE_64X64_K2: return launch_tile<64, 64, 2, 2, 4, 2, OUT>(p, plan.splits, s);
    case F8_TILE_128X128: return launch_tile<128, 128, 2, 4, 2, 1, OUT>(p, plan.splits, s);
    default:                           // 16-bit outputs
      if constexpr (OUT == ACT_F32) return hipErrorInvalidValue;
      else if (plan.kind == F8_TILE_128X128_K2) return launch_tile<128, 128, 2, 4, 2, 2, OUT>(p, plan.splits, s);
      else return launch_big<OUT>(p, s);
  }
}

hipError_t launch_linear_f8(const LinearF8Params& p, const LinearF8Plan& plan, int out, hipStream_t s) {
  switch (out) {
    case ACT_F32: return launch_out<ACT_F32>(p, plan, s);
    case ACT_F16: return launch_out<ACT_F16>(p, plan, s);
    default: return launch_out<ACT_BF16>(p, plan, s);
  }
}

}  // namespace lowbit
