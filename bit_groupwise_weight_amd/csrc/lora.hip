// Low-rank adapters of many requests beside a shared projection:
//
//   y[m] = base[m] + scales[a] * (x[m] A_a^T) B_a^T,   a the adapter of row m
//
// with A_a [rank, K] and B_a [N, rank]; rows without an adapter keep base (or
// are 0 without one).  Rows come in the order of their adapter: position t of
// the call is row rows[t], and adapter a has positions offsets[a] ..
// offsets[a + 1] - 1; the positions before and behind are those without one.
//
// Two products, both on the matrix cores with fp32 sums: t = x A^T (shrink),
// K long and rank wide, split over K, and y = base + t B^T (expand), which is
// read and written once.  In both the adapter is the MFMA's A operand, so that
// a lane holds four consecutive outputs of one row.
//
// t enters the second product as two numbers of the call's type, t = hi + lo,
// which keep 16 bits of it in bf16 and 22 in fp16 where one would keep 8 and
// 11; the pair costs a second MFMA (none at rank 16, where both fill one), and
// the call is bound by memory.  fp16 pairs are taken of t times a power of two
// that brings a row's largest |t| to 1 .. 2, so that t may be any fp32 number.
// fp32 calls use the fp32 matrix instruction throughout.
//
// With an infinite element of B the pair's halves may meet it with unlike signs or
// as 0, where t itself gives an infinity: sums that are not a number are made
// again from t, one product at a time (sums_of_t).
#include "pieces.h"

#include <algorithm>

namespace lowbit {

namespace {

// 8 consecutive values of a row, K positions of one lane in a step of 32.
template <int ACT> struct Chunk {      // 16-bit types
  u32v4_t w;
  __device__ __forceinline__ void load(const void* p, size_t at) {
    w = *reinterpret_cast<const u32v4_t*>(static_cast<const uint16_t*>(p) + at);
  }
  __device__ __forceinline__ void keep(bool in) { w = in ? w : u32v4_t{0u, 0u, 0u, 0u}; }
};
template <> struct Chunk<ACT_F32> {
  f32x4_t v[2];
  __device__ __forceinline__ void load(const void* p, size_t at) {
    const f32x4_t* q = reinterpret_cast<const f32x4_t*>(static_cast<const float*>(p) + at);
    v[0] = q[0];
    v[1] = q[1];
  }
  __device__ __forceinline__ void keep(bool in) {
    if (!in) v[0] = v[1] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
  }
};

typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));

// acc += A . B over a step's 32 K positions: lane l supplies row (A) or column
// (B) l % 16 at K positions 8 (l / 16) .. + 7, and holds rows 4 (l / 16) + i of
// column l % 16 of the result.  (fp32: eight steps of four positions, the j-th
// of each lane's chunk.)
template <int ACT>
__device__ __forceinline__ f32x4_t mfma(const Chunk<ACT>& a, const Chunk<ACT>& b, f32x4_t acc) {
  if constexpr (ACT == ACT_F32) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      acc = __builtin_amdgcn_mfma_f32_16x16x4f32(a.v[j >> 2][j & 3], b.v[j >> 2][j & 3], acc, 0, 0, 0);
    return acc;
  } else if constexpr (ACT == ACT_F16) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8_t, a.w),
                                                  __builtin_bit_cast(f16x8_t, b.w), acc, 0, 0, 0);
  } else {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a.w),
                                                   __builtin_bit_cast(bf16x8_t, b.w), acc, 0, 0, 0);
  }
}

// The positions of group v: 0 those before the first adapter, 1 .. L the
// adapters', L + 1 those behind the last; clamped to 0 .. T.
__device__ __forceinline__ void group_bounds(const LoraParams& p, int v, int* lo, int* hi) {
  const int T = static_cast<int>(p.T);
  *lo = *hi = 0;
  if (v <= p.L + 1) {
    if (v > 0) *lo = min(max(p.offsets[v - 1], 0), T);
    *hi = v <= p.L ? min(max(p.offsets[v], *lo), T) : T;
  }
}

struct RowTile {
  int begin, end;         // positions
  int adapter;            // -1 or L: rows without one
  bool found;
};
// Tile `tile` of BM rows among all groups' tiles: the wave looks through the groups,
// PER of them a lane at a time.
template <int BM, int PER>
__device__ __forceinline__ RowTile search_rows(const LoraParams& p, int tile) {
  RowTile t{0, 0, -1, false};
  const int lane = threadIdx.x & 63;
  int before = 0;
  for (int v0 = 0; v0 < p.L + 2; v0 += 64 * PER) {
    int lo[PER], hi[PER], own = 0;
#pragma unroll
    for (int j = 0; j < PER; ++j) group_bounds(p, v0 + PER * lane + j, &lo[j], &hi[j]);
#pragma unroll
    for (int j = 0; j < PER; ++j) own += (hi[j] - lo[j] + BM - 1) / BM;
    int upto = own;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int u = __shfl_up(upto, o);
      if (lane >= o) upto += u;
    }
    const int first = before + upto - own;
    const uint64_t hit = __ballot(tile >= first && tile < first + own);
    if (hit != 0) {
      const int src = __builtin_ctzll(hit);
      int at = tile - first, begin = 0, end = 0, group = 0;   // of the lane that has it
#pragma unroll
      for (int j = 0; j < PER; ++j) {
        const int n = (hi[j] - lo[j] + BM - 1) / BM;
        if (at >= 0 && at < n) {
          begin = lo[j] + at * BM;
          end = min(begin + BM, hi[j]);
          group = j;
        }
        at -= n;
      }
      t.begin = __builtin_amdgcn_readlane(begin, src);
      t.end = __builtin_amdgcn_readlane(end, src);
      t.adapter = v0 + PER * src + __builtin_amdgcn_readlane(group, src) - 1;
      t.found = true;
      return t;
    }
    before += __builtin_amdgcn_readlane(upto, 63);
  }
  return t;
}
// (One group a lane / four, us: 64 rows of 1000 adapters, one launch, 13.2 / 10.3;
// 2000 rows of them, two launches, 45 / 37; 100 adapters the same.)
template <int BM>
__device__ __forceinline__ RowTile find_rows(const LoraParams& p, int tile) {
  return p.L + 2 <= 64 ? search_rows<BM, 1>(p, tile) : search_rows<BM, 4>(p, tile);
}

// Row of position t, -1 where it is no row.
__device__ __forceinline__ int row_of(const LoraParams& p, int t) {
  const int64_t r = p.rows ? p.rows[t] : t;
  return r >= 0 && r < p.M ? static_cast<int>(r) : -1;
}

// Direct global -> LDS loads of 16 bytes a lane, lane l to LDS at m0 + 16 l, and
// their waits.  Operands go through LDS because in an MFMA's layout neighbouring
// lanes hold different rows: loaded straight to registers, each lane's 16 bytes
// are a cache access of their own, four times as many as here (adapters of
// rank 64 on 8192 rows, 4096 -> 14336: 1.3 TB/s in the first product so).
__device__ __forceinline__ void dma16(const void* vaddr, uint32_t m0) {
  asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off"
               : : "v"(vaddr), "s"(m0) : "memory", "m0");
}
// At most N of this wave's loads and stores still in flight.
template <int N> __device__ __forceinline__ void wait_loads() {
  static_assert(N >= 0 && N < 64, "vmcnt range");
  asm volatile("s_waitcnt vmcnt(%0)" : : "n"(N) : "memory");
}
// This wave's LDS reads are done (before loads overwrite what they read).
__device__ __forceinline__ void wait_lds() { asm volatile("s_waitcnt lgkmcnt(0)" : : : "memory"); }
__device__ __forceinline__ void barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" : : : "memory"); }

template <typename T>
__device__ __forceinline__ uint32_t lds_address(T* p) {
  return static_cast<uint32_t>(reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) void*)p));
}

// What positions past K are read from.
__device__ __attribute__((aligned(16))) const uint32_t kZeros[4] = {0u, 0u, 0u, 0u};

// A unit: 128 bytes of each of 16 rows, 2 KiB in LDS from two loads.  Chunk c (16
// bytes) of row r sits at position c ^ ((r >> 1) & 7) of the row, so that the 16
// rows of a read at one chunk start in 16 different 4-bank groups.
constexpr int kUnitBytes = 2048;
template <int ACT> constexpr int kUnitK = 128 / Act<ACT>::bytes;       // positions
template <int ACT> constexpr int kUnitSteps = kUnitK<ACT> / 32;        // MFMA steps
template <int ACT> constexpr int kChunkK = 16 / Act<ACT>::bytes;       // positions of a chunk

// The lane's chunk of a step of a row's unit in LDS.
template <int ACT>
__device__ __forceinline__ void read_unit(const uint8_t* unit, int step, Chunk<ACT>& v) {
  const int c16 = threadIdx.x & 15, g = (threadIdx.x & 63) >> 4, swz = (c16 >> 1) & 7;
  const uint8_t* row = unit + c16 * 128;
  if constexpr (ACT == ACT_F32) {
    v.v[0] = *reinterpret_cast<const f32x4_t*>(row + 16 * ((2 * g) ^ swz));
    v.v[1] = *reinterpret_cast<const f32x4_t*>(row + 16 * ((2 * g + 1) ^ swz));
  } else {
    v.w = *reinterpret_cast<const u32v4_t*>(row + 16 * ((4 * step + g) ^ swz));
  }
}

// acc += A . x^T of a tile of 16 NT ranks (from r0) and 16 positions over the
// units first, first + WAVES, .. below last of K; ring: the wave's own STAGES
// stages of 1 + NT units.
template <int ACT, int NT, int WAVES, int STAGES>
__device__ __forceinline__ void shrink_tile(const LoraParams& p, const RowTile& rt, int r0, int first, int last,
                                            uint8_t* ring, f32x4_t (&acc)[NT]) {
  constexpr int LOADS = 2 * (1 + NT), STAGE = (1 + NT) * kUnitBytes;
  const int lane = threadIdx.x & 63;
  // load h of a unit: rows 8 h + lane / 8; the lane fills position lane % 8
  const uint8_t* from[LOADS];
  int chunk[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) chunk[h] = (lane & 7) ^ (((8 * h + (lane >> 3)) >> 1) & 7);
#pragma unroll
  for (int i = 0; i < LOADS; ++i) {
    const int tile = i / 2, r = 8 * (i & 1) + (lane >> 3);
    const uint8_t* base;
    size_t row;
    if (tile == 0) {                   // (positions past the tile: its last one again; rows that are none: row 0)
      base = static_cast<const uint8_t*>(p.x);
      row = static_cast<size_t>(max(row_of(p, min(rt.begin + r, rt.end - 1)), 0));
    } else {
      base = static_cast<const uint8_t*>(p.a);
      row = static_cast<size_t>(rt.adapter) * p.rank + min(r0 + 16 * (tile - 1) + r, p.rank - 1);
    }
    from[i] = base + row * p.K * Act<ACT>::bytes + 16 * chunk[i & 1];
  }
  const uint32_t to = lds_address(ring);
  auto load = [&](int unit, int stage) {
    const uint32_t dst = to + stage * STAGE;
    const size_t at = static_cast<size_t>(unit) * 128;
    const bool whole = (unit + 1) * kUnitK<ACT> <= p.K;
#pragma unroll
    for (int i = 0; i < LOADS; ++i)
      dma16(whole || unit * kUnitK<ACT> + chunk[i & 1] * kChunkK<ACT> < p.K
                ? from[i] + at : reinterpret_cast<const uint8_t*>(kZeros),
            dst + i * 1024);
  };
#pragma unroll
  for (int i = 0; i < NT; ++i) acc[i] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
  const int units = last > first ? (last - first + WAVES - 1) / WAVES : 0;
#pragma unroll
  for (int s = 0; s < STAGES - 1; ++s)
    if (s < units) load(first + s * WAVES, s);
  int stage = 0;
#pragma unroll 1
  for (int u = 0; u < units; ++u) {
    const int ahead = units - 1 - u;   // units behind this one: their loads may stay in flight
    if (ahead >= STAGES - 1) {
      int next = stage + STAGES - 1;
      if (next >= STAGES) next -= STAGES;
      wait_lds();
      load(first + (u + STAGES - 1) * WAVES, next);
      wait_loads<LOADS * (STAGES - 1)>();
    } else if (STAGES > 3 && ahead == 2) {
      wait_loads<LOADS * (STAGES > 3 ? 2 : 0)>();
    } else if (STAGES > 2 && ahead == 1) {
      wait_loads<LOADS * (STAGES > 2 ? 1 : 0)>();
    } else {
      wait_loads<0>();
    }
    const uint8_t* at = ring + stage * STAGE;
#pragma unroll
    for (int s = 0; s < kUnitSteps<ACT>; ++s) {
      Chunk<ACT> x, a[NT];
      read_unit<ACT>(at, s, x);
#pragma unroll
      for (int i = 0; i < NT; ++i) read_unit<ACT>(at + (1 + i) * kUnitBytes, s, a[i]);
#pragma unroll
      for (int i = 0; i < NT; ++i) acc[i] = mfma<ACT>(a[i], x, acc[i]);
    }
    if (++stage == STAGES) stage = 0;
  }
}

}  // namespace

// t of a tile of 16 positions and 16 NT ranks, over the units of K of blockIdx.y:
// the waves share them, their sums meet in LDS.  For adapters of few rows, whose
// A is most of what is read: many blocks with short ranges of K, bound by the
// latencies of offsets, rows and the first units (64 rows of 32 adapters of rank
// 32, 4096 bf16, 9 MB: 4.5 us, of rank 64 5.6).
template <int ACT, int NT, int WAVES, int STAGES>
__global__ __launch_bounds__(64 * WAVES) void lora_shrink_kernel(LoraParams p) {
  constexpr int RING = STAGES * (1 + NT) * kUnitBytes;
  static_assert(RING >= NT * 1024, "the sums fit the rings");
  __shared__ __attribute__((aligned(1024))) uint8_t s_ring[WAVES][RING];
  const int lane = threadIdx.x & 63, c16 = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const RowTile rt = find_rows<16>(p, static_cast<int>(blockIdx.x));
  if (!rt.found || rt.adapter < 0 || rt.adapter >= p.L) return;
  const int r0 = static_cast<int>(blockIdx.z) * 16 * NT;
  const int all = (p.K + kUnitK<ACT> - 1) / kUnitK<ACT>;
  const int first = static_cast<int>(blockIdx.y) * p.units_split, last = min(first + p.units_split, all);
  f32x4_t acc[NT];
  shrink_tile<ACT, NT, WAVES, STAGES>(p, rt, r0, first + wave, last, s_ring[wave], acc);
  // (a wave's own ring has no loads in flight and no reads that are not done)
  f32x4_t* sum = reinterpret_cast<f32x4_t*>(s_ring[wave]);
#pragma unroll
  for (int i = 0; i < NT; ++i) sum[i * 64 + lane] = acc[i];
  __syncthreads();
  float* plane = p.t + static_cast<size_t>(blockIdx.y) * p.T * p.rank_pad;
  for (int i = wave; i < NT; i += WAVES) {
    f32x4_t v = reinterpret_cast<const f32x4_t*>(s_ring[0])[i * 64 + lane];
#pragma unroll
    for (int w = 1; w < WAVES; ++w) v += reinterpret_cast<const f32x4_t*>(s_ring[w])[i * 64 + lane];
    const int t = rt.begin + c16, r = r0 + 16 * i + 4 * g;
    if (t < rt.end && r < p.rank_pad)
      *reinterpret_cast<f32x4_t*>(plane + static_cast<size_t>(t) * p.rank_pad + r) = v;
  }
}

// The same for many rows: each of the WAVES waves has 16 positions of its own
// and all share A's units, through a ring of STAGES stages.  A unit has one
// barrier, before which a wave waits for its own loads of it; the loads of later
// units go out behind it, into the stage that the unit before has left.  Bound by
// memory: x is read once for every 64 ranks, A once a tile (8192 rows of rank 64,
// 4096 bf16, 67 MB: 18 to 27 us; in tiles of 64 rows 33).
template <int ACT, int NT, int WAVES, int STAGES>
__global__ __launch_bounds__(64 * WAVES) void lora_shrink_rows_kernel(LoraParams p) {
  constexpr int A_LOADS = 2 * NT >= WAVES ? 2 * NT / WAVES : 1;   // of a wave (NT 1: two waves each the same)
  constexpr int LOADS = A_LOADS + 2, STAGE = (NT + WAVES) * kUnitBytes;
  static_assert(2 * NT % WAVES == 0 || WAVES % (2 * NT) == 0, "whole loads");
  __shared__ __attribute__((aligned(1024))) uint8_t s_ring[STAGES][STAGE];
  const int lane = threadIdx.x & 63, c16 = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const RowTile rt = find_rows<16 * WAVES>(p, static_cast<int>(blockIdx.x));
  if (!rt.found || rt.adapter < 0 || rt.adapter >= p.L) return;
  const int r0 = static_cast<int>(blockIdx.z) * 16 * NT;
  const int all = (p.K + kUnitK<ACT> - 1) / kUnitK<ACT>;
  const int first = static_cast<int>(blockIdx.y) * p.units_split, units = min(p.units_split, all - first);
  const int mine = rt.begin + 16 * wave;               // the wave's first position

  const uint8_t* from[LOADS];
  int chunk[LOADS], to[LOADS];
#pragma unroll
  for (int i = 0; i < LOADS; ++i) {
    // loads 0 and 1: the wave's x; then load `half` of A's 2 NT
    const int half = i < 2 ? i : (wave * A_LOADS + i - 2) % (2 * NT);
    const int r = 8 * (half & 1) + (lane >> 3);        // of the unit
    const uint8_t* base;
    size_t row;
    if (i < 2) {                       // (positions past the tile: its last one again; rows that are none: row 0)
      base = static_cast<const uint8_t*>(p.x);
      row = static_cast<size_t>(max(row_of(p, min(mine + r, rt.end - 1)), 0));
      to[i] = (NT + wave) * kUnitBytes + 1024 * i;
    } else {
      base = static_cast<const uint8_t*>(p.a);
      row = static_cast<size_t>(rt.adapter) * p.rank + min(r0 + 16 * (half / 2) + r, p.rank - 1);
      to[i] = 1024 * half;
    }
    chunk[i] = (lane & 7) ^ ((r >> 1) & 7);
    from[i] = base + row * p.K * Act<ACT>::bytes + 16 * chunk[i];
  }
  const uint32_t ring = lds_address(&s_ring[0][0]);
  auto load = [&](int unit, int stage) {
    const uint32_t dst = ring + stage * STAGE;
    const size_t at = static_cast<size_t>(unit) * 128;
    const bool whole = (unit + 1) * kUnitK<ACT> <= p.K;
#pragma unroll
    for (int i = 0; i < LOADS; ++i)
      dma16(whole || unit * kUnitK<ACT> + chunk[i] * kChunkK<ACT> < p.K ? from[i] + at
                                                                      : reinterpret_cast<const uint8_t*>(kZeros),
            dst + to[i]);
  };
  f32x4_t acc[NT];
#pragma unroll
  for (int i = 0; i < NT; ++i) acc[i] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int s = 0; s < STAGES - 1; ++s)
    if (s < units) load(first + s, s);
  int stage = 0;
#pragma unroll 1
  for (int u = 0; u < units; ++u) {
    const int ahead = units - 1 - u;   // units behind this one: their loads may stay in flight
    if (ahead >= STAGES - 2) wait_loads<LOADS * (STAGES - 2)>();
    else if (STAGES > 3 && ahead == 1) wait_loads<LOADS>();
    else wait_loads<0>();
    barrier();
    int next = stage + STAGES - 1;
    if (next >= STAGES) next -= STAGES;
    if (ahead >= STAGES - 1) load(first + u + STAGES - 1, next);
    const uint8_t* at = s_ring[stage];
#pragma unroll
    for (int s = 0; s < kUnitSteps<ACT>; ++s) {
      Chunk<ACT> x, a[NT];
      read_unit<ACT>(at + (NT + wave) * kUnitBytes, s, x);
#pragma unroll
      for (int i = 0; i < NT; ++i) read_unit<ACT>(at + i * kUnitBytes, s, a[i]);
#pragma unroll
      for (int i = 0; i < NT; ++i) acc[i] = mfma<ACT>(a[i], x, acc[i]);
    }
    if (++stage == STAGES) stage = 0;
  }
  float* plane = p.t + static_cast<size_t>(blockIdx.y) * p.T * p.rank_pad;
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    const int t = mine + c16, r = r0 + 16 * i + 4 * g;
    if (t < rt.end && r < p.rank_pad)
      *reinterpret_cast<f32x4_t*>(plane + static_cast<size_t>(t) * p.rank_pad + r) = acc[i];
  }
}

namespace {

// t of a tile's BM rows in LDS, ready for the second product: rows of RANKS + 8
// elements, an odd number of 16-byte pieces, so that the 16 rows of a read
// start in different banks; 16-bit types have the hi halves of all rows and
// then the lo halves.  put_t: eight ranks of row r.
template <int ACT, int BM, int RANKS> struct TileT {
  typedef typename Act<ACT>::bits_t T;
  static constexpr int PITCH = RANKS + 8, HALVES = ACT == ACT_F32 ? 1 : 2;
  T v[HALVES][BM][PITCH];
  float unscale[BM];                   // fp16
};
template <int ACT, int BM, int RANKS>
__device__ __forceinline__ void put_t(TileT<ACT, BM, RANKS>& t, int r, int k, float (&v)[8]) {
  constexpr int LANES = RANKS / 8;     // of a row, a power of two, which call together
  if constexpr (ACT == ACT_F32) {
    f32x4_t* to = reinterpret_cast<f32x4_t*>(&t.v[0][r][k]);
    to[0] = f32x4_t{v[0], v[1], v[2], v[3]};
    to[1] = f32x4_t{v[4], v[5], v[6], v[7]};
  } else {
    if constexpr (ACT == ACT_F16) {
      uint32_t top = 0;              // bits of the row's largest magnitude
#pragma unroll
      for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(v[i]) & 0x7fffffffu);
#pragma unroll
      for (int o = 1; o < LANES; o <<= 1)
        top = max(top, static_cast<uint32_t>(__shfl_xor(static_cast<int>(top), o)));
      // 2^-e with e the exponent of the largest, within fp32's normal powers
      const int e = min(max(static_cast<int>(top >> 23), 1), 253);
      const float by = __uint_as_float(static_cast<uint32_t>(254 - e) << 23);
      if (k == 0) t.unscale[r] = __uint_as_float(static_cast<uint32_t>(e) << 23);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] *= by;
    }
    constexpr float kMost = ACT == ACT_F16 ? 65504.0f : 0x1.fep127f;
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      // (hi is finite; an infinity and what is no number are lo's)
      hi[i] = pack2<ACT>(__builtin_amdgcn_fmed3f(v[2 * i], -kMost, kMost),
                         __builtin_amdgcn_fmed3f(v[2 * i + 1], -kMost, kMost));
      lo[i] = pack2<ACT>(v[2 * i] - act_bits_to_float<ACT>(hi[i] & 0xffffu),
                         v[2 * i + 1] - act_bits_to_float<ACT>(hi[i] >> 16));
    }
    *reinterpret_cast<u32v4_t*>(&t.v[0][r][k]) = u32v4_t{hi[0], hi[1], hi[2], hi[3]};
    *reinterpret_cast<u32v4_t*>(&t.v[1][r][k]) = u32v4_t{lo[0], lo[1], lo[2], lo[3]};
  }
}

// B of consecutive columns in LDS, the ranks of pass `pass` (128 bytes of each
// column, or what is left of the rank): chunk c of column n, of u chunks, is
// logical chunk n u + c, and logical chunk q sits at q ^ turn(q), within its 16:
// the 16 columns n, n + 8, ... of a read then start in different banks (for odd
// u: nearly).
template <int ACT> constexpr int kPassRanks = 128 / Act<ACT>::bytes;
struct BLayout {
  int u, inv, shift;
  __device__ __forceinline__ int turn(int q) const { return (q >> shift) & 15; }
};
template <int ACT> __device__ __forceinline__ BLayout b_layout(const LoraParams& p, int pass) {
  BLayout l;
  l.u = min(kPassRanks<ACT>, p.rank - pass * kPassRanks<ACT>) / kChunkK<ACT>;
  l.inv = (65536 + l.u - 1) / l.u;     // q / u == (q * inv) >> 16 for q < 2^13, u <= 8
  l.shift = 4 + ((l.u & 7) == 0 ? 2 : (l.u & 3) == 0 ? 1 : 0);
  return l;
}
// The share of wave `wave` of WAVES in loading COLS columns from n0 on.
template <int ACT, int COLS, int WAVES>
__device__ __forceinline__ void load_b(const LoraParams& p, int adapter, int n0, int pass, const BLayout& l,
                                       uint32_t to, int wave) {
  const uint8_t* b = static_cast<const uint8_t*>(p.b);
  const size_t col0 = static_cast<size_t>(adapter) * p.N;
  for (int i = wave; i < COLS * l.u / 64; i += WAVES) {
    const int at = 64 * i + static_cast<int>(threadIdx.x & 63), q = at ^ l.turn(at);
    const int n = (q * l.inv) >> 16, c = q - n * l.u;
    dma16(b + ((col0 + min(n0 + n, p.N - 1)) * p.rank + pass * kPassRanks<ACT> + c * kChunkK<ACT>) * Act<ACT>::bytes,
          to + 1024 * i);
  }
}

// acc += t B^T for 16 rows (from row m0 of the tile on) and 128 columns, ranks of
// one pass: MFMA tile j has the columns 8 c + j, c = 0 .. 15 (from column n0 of
// lds on), so that a lane ends with 8 consecutive columns of four rows, and 16
// lanes with 256 bytes of a row.
template <int ACT, int BM, int RANKS>
__device__ __forceinline__ void multiply_pass(const LoraParams& p, const TileT<ACT, BM, RANKS>& t, int m0,
                                              const uint8_t* lds, const BLayout& l, int n0, int pass,
                                              f32x4_t (&acc)[8]) {
  const int lane = threadIdx.x & 63, c16 = lane & 15, g = lane >> 4;
  const bool both = ACT != ACT_F32 && p.rank_pad == 16;       // hi and lo in one step
  auto read_b = [&](int j, int chunk, bool in) {
    const int q = (n0 + 8 * c16 + j) * l.u + (in ? chunk : 0);
    return *reinterpret_cast<const u32v4_t*>(lds + 16 * (q ^ l.turn(q)));
  };
  const int left = p.rank_pad - pass * kPassRanks<ACT>;
#pragma unroll
  for (int s = 0; s < kUnitSteps<ACT>; ++s) {
    if (32 * s >= left) break;
    const int k = both ? 8 * (g & 1) : 32 * s + 8 * g;        // of the pass
    const bool in = pass * kPassRanks<ACT> + k < p.rank;      // (B past the rank: zeros)
    Chunk<ACT> b[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if constexpr (ACT == ACT_F32) {
        b[j].v[0] = __builtin_bit_cast(f32x4_t, read_b(j, 2 * g, in));
        b[j].v[1] = __builtin_bit_cast(f32x4_t, read_b(j, 2 * g + 1, in));
      } else {
        b[j].w = read_b(j, k / 8, in);
      }
      b[j].keep(in);
    }
    const int kt = pass * kPassRanks<ACT> + k;
    const int r = m0 + c16;
    Chunk<ACT> v;
    v.load(ACT != ACT_F32 && both && g >= 2 ? &t.v[t.HALVES - 1][r][kt] : &t.v[0][r][kt], 0);
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[j] = mfma<ACT>(v, b[j], acc[j]);
    if constexpr (ACT != ACT_F32) {
      if (!both) {
        v.load(&t.v[1][r][kt], 0);
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[j] = mfma<ACT>(v, b[j], acc[j]);
      }
    }
  }
}

// Sums of a wave's 16 rows and 128 columns (from n0 on) that are not a number, made
// again; t_of(r, k): t of the tile's row r, rank k, with its scale.  (The look for
// them costs 0.1 us a launch, and 0.6 of 108 with 8192 rows.)
template <int ACT, int BM, int RANKS, class TOf>
__device__ __forceinline__ void sums_of_t(const LoraParams& p, const TileT<ACT, BM, RANKS>& t, int m0, int adapter,
                                          int n0, f32x4_t (&acc)[8], TOf t_of) {
  if constexpr (ACT != ACT_F32) {
    bool none = false;                 // (no number)
#pragma unroll
    for (int j = 0; j < 8; j += 2)
#pragma unroll
      for (int i = 0; i < 4; ++i) none |= __builtin_isunordered(acc[j][i], acc[j + 1][i]);
    if (__builtin_expect(__ballot(none) == 0, 1)) return;
    const int n = n0 + 8 * static_cast<int>(threadIdx.x & 15);
    const uint16_t* b = static_cast<const uint16_t*>(p.b) + (static_cast<size_t>(adapter) * p.N + n) * p.rank;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = m0 + 4 * static_cast<int>((threadIdx.x & 63) >> 4) + i;
      const float by = ACT == ACT_F16 ? 1.0f / t.unscale[r] : 1.0f;        // (a power of two)
      bool again = false;
#pragma unroll
      for (int j = 0; j < 8; ++j) again |= acc[j][i] != acc[j][i];
      float sum[8] = {};
#pragma unroll 1
      for (int k = 0; again && k < p.rank; ++k) {
        const float v = t_of(r, k) * by;
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (n + j < p.N) sum[j] += v * act_bits_to_float<ACT>(b[static_cast<size_t>(j) * p.rank + k]);
        again = v == v;                // (else none of the row's sums is a number)
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) acc[j][i] = acc[j][i] != acc[j][i] ? sum[j] : acc[j][i];
    }
  }
}

// The rows and columns that a lane ends with.
template <int ACT> struct Outputs {
  typedef typename Act<ACT>::bits_t T;
  static constexpr int LOADS = 4 * (ACT == ACT_F32 ? 2 : 1);   // or stores, of a full step
  int row[4];             // -1: none
  float unscale[4];       // fp16
  Piece<ACT> old[4];

  // rows 4 g + i of the wave's 16, from row m0 of the tile on
  __device__ __forceinline__ void set_rows(const int* rows, int m0) {
#pragma unroll
    for (int i = 0; i < 4; ++i) row[i] = rows[m0 + 4 * ((threadIdx.x & 63) >> 4) + i];
  }
  template <int BM, int RANKS> __device__ __forceinline__ void set_factors(const TileT<ACT, BM, RANKS>& t, int m0) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      unscale[i] = ACT == ACT_F16 ? t.unscale[m0 + 4 * ((threadIdx.x & 63) >> 4) + i] : 1.0f;
  }
  __device__ __forceinline__ bool all_rows() const {
    return __ballot(row[0] < 0 || row[1] < 0 || row[2] < 0 || row[3] < 0) == 0;
  }
  // FULL: every row and column of the step is there
  template <bool FULL> __device__ __forceinline__ void load(const LoraParams& p, int n0) {
    if (p.base == nullptr) return;
    const int n = n0 + 8 * static_cast<int>(threadIdx.x & 15);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (FULL || (row[i] >= 0 && n < p.N))
        load_piece<ACT>(static_cast<const T*>(p.base) + static_cast<size_t>(row[i]) * p.N + n, FULL ? 8 : p.N - n,
                        old[i]);
  }
  template <bool FULL> __device__ __forceinline__ void store(const LoraParams& p, int n0, const f32x4_t (&acc)[8]) {
    const int n = n0 + 8 * static_cast<int>(threadIdx.x & 15);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (!FULL && (row[i] < 0 || n >= p.N)) continue;
      float v[8] = {};
      if (p.base) piece_to_float<ACT>(old[i], v);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] += acc[j][i] * unscale[i];
      store_piece<ACT>(static_cast<T*>(p.y) + static_cast<size_t>(row[i]) * p.N + n, FULL ? 8 : p.N - n, v);
    }
  }
};

__device__ __forceinline__ void clear(f32x4_t (&acc)[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) acc[j] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
}

// Rows without an adapter: base, or 0, to another array.
template <int ACT>
__device__ __forceinline__ void copy_columns(const LoraParams& p, Outputs<ACT>& o, int n0, int n_end, int stride) {
  f32x4_t acc[8];
  clear(acc);
#pragma unroll
  for (int i = 0; i < 4; ++i) o.unscale[i] = 0.0f;
  for (; n0 < n_end; n0 += stride) {
    o.template load<false>(p, n0);
    o.template store<false>(p, n0, acc);
  }
}

}  // namespace

// y of a tile of BM = 16 WM positions: WN waves next to each other take 128
// columns each, and the block `cols` columns, 128 WN at a time, whose B the
// waves load together.  A step's B is asked for behind the products of the step
// before and ahead of that one's stores, its base behind them.  Bound by memory:
// base once in, y once out, past the caches (8192 rows, 14336 bf16 columns, rank
// 64, 470 MB: 107 to 117 us, 4.0 to 4.4 TB/s, a copy of the base alone 89; 777
// rows of 7 adapters, 5001 fp16 columns, rank 24: 10.5 us, most of it latencies
// that follow each other: offsets, then t, B and rows, then base).  Measured and
// left: the first base asked for with t (8192 rows 122), two row tiles a wave or
// the base a step further ahead (no faster, more registers), t four planes at a
// time behind the rows (777 rows 11.8, 8192 rows 113).
template <int ACT, int WM, int WN, int RANKS>
__global__ __launch_bounds__(64 * WM * WN) void lora_expand_kernel(LoraParams p, int cols) {
  constexpr int BM = 16 * WM, WAVES = WM * WN, COLS = 128 * WN;
  __shared__ __attribute__((aligned(1024))) uint8_t s_b[COLS * 128];
  __shared__ __attribute__((aligned(16))) TileT<ACT, BM, RANKS> s_t;
  __shared__ int s_row[BM];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), wm = wave / WN, wn = wave % WN;
  const unsigned across = static_cast<unsigned>((p.N + cols - 1) / cols), tile = blockIdx.x / across;
  const RowTile rt = find_rows<BM>(p, static_cast<int>(tile));
  if (!rt.found) return;
  const bool bare = rt.adapter < 0 || rt.adapter >= p.L;
  if (bare && p.base == p.y) return;
  const int first = static_cast<int>(blockIdx.x - tile * across) * cols, last = min(first + cols, p.N);
  const int passes = (p.rank + kPassRanks<ACT> - 1) / kPassRanks<ACT>;
  const uint32_t b_at = lds_address(s_b);
  BLayout l = b_layout<ACT>(p, 0);
  if (!bare) load_b<ACT, COLS, WAVES>(p, rt.adapter, first, 0, l, b_at, wave);
  // t, eight ranks a lane, all planes of a turn asked for at once, and the rows
  // behind those of the first
  constexpr int LANES = RANKS / 8, AT_ONCE = 64 * WAVES / LANES;
  const int k = threadIdx.x % LANES * 8;
  const float scale = !bare && p.scales ? p.scales[rt.adapter] : 1.0f;
  const bool one = threadIdx.x < BM && rt.begin + static_cast<int>(threadIdx.x) < rt.end;
  int row = -1;
  for (int r = threadIdx.x / LANES; r < BM; r += AT_ONCE) {
    f32x4_t planes[kLoraMaxSplits][2];
    if (!bare) {
      const float* from = p.t + static_cast<size_t>(min(rt.begin + r, rt.end - 1)) * p.rank_pad + min(k, p.rank_pad - 8);
#pragma unroll
      for (int s = 0; s < kLoraMaxSplits; ++s) {
        if (s >= p.splits) break;
        const f32x4_t* at = reinterpret_cast<const f32x4_t*>(from + static_cast<size_t>(s) * p.T * p.rank_pad);
        planes[s][0] = at[0];
        planes[s][1] = at[1];
      }
    }
    if (one && r == static_cast<int>(threadIdx.x) / LANES) row = row_of(p, rt.begin + threadIdx.x);
    if (bare) break;
    float v[8] = {};
#pragma unroll
    for (int s = 0; s < kLoraMaxSplits; ++s) {
      if (s >= p.splits) break;
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] += planes[s][i >> 2][i & 3];
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = k < p.rank && rt.begin + r < rt.end ? v[i] * scale : 0.0f;
    put_t<ACT, BM, RANKS>(s_t, r, k, v);
  }
  if (threadIdx.x < BM) s_row[threadIdx.x] = row;
  __syncthreads();
  Outputs<ACT> o;
  o.set_rows(s_row, 16 * wm);
  if (bare) {
    copy_columns<ACT>(p, o, first + 128 * wn, last, COLS);
    return;
  }
  o.set_factors(s_t, 16 * wm);
  const bool rows = o.all_rows() && p.base != nullptr;
  f32x4_t acc[8];
  for (int n0 = first; n0 < last; n0 += COLS) {
    const int n = n0 + 128 * wn;
    const bool full = rows && n + 128 <= p.N;
    if (full) o.template load<true>(p, n);
    else o.template load<false>(p, n);
    clear(acc);
    for (int pass = 0; pass < passes; ++pass) {
      // (behind a full first pass's B are the stores of the step before, which is
      // full, too, and the base: they stay in flight)
      if (full && pass == 0) {
        if (n0 == first) wait_loads<Outputs<ACT>::LOADS>();
        else wait_loads<2 * Outputs<ACT>::LOADS>();
      } else {
        wait_loads<0>();
      }
      barrier();
      multiply_pass<ACT, BM, RANKS>(p, s_t, 16 * wm, s_b, l, 128 * wn, pass, acc);
      barrier();
      const bool more = pass + 1 < passes;
      if (more || n0 + COLS < last) {
        l = b_layout<ACT>(p, more ? pass + 1 : 0);
        load_b<ACT, COLS, WAVES>(p, rt.adapter, more ? n0 : n0 + COLS, more ? pass + 1 : 0, l, b_at, wave);
      }
    }
    sums_of_t<ACT, BM, RANKS>(p, s_t, 16 * wm, rt.adapter, n, acc, [&](int r, int k) {
      const float* from = p.t + static_cast<size_t>(min(rt.begin + r, rt.end - 1)) * p.rank_pad + k;
      float v = 0.0f;
      for (int s = 0; s < p.splits; ++s) v += from[static_cast<size_t>(s) * p.T * p.rank_pad];
      return v * scale;
    });
    if (full) o.template store<true>(p, n, acc);
    else o.template store<false>(p, n, acc);
  }
}

// Both products of a tile of 16 positions in one launch, for few rows: every
// block of a tile's columns makes the tile's t by itself.  Each wave has 128
// columns at a time and loads their B alone, the first of it ahead of the first
// product.  Bound by latencies and by A, which every block of a tile reads whole
// (1 row of rank 16, 4096 -> 4096: 7.1 us, an empty launch 2.7; 64 rows of 32
// adapters of rank 16, 4096 -> 14336 bf16, 20 MB: 10.7 us; two launches 14.6, without
// the next step's B and base ahead of the products 0.7 more).  Measured and left: a
// fourth stage, x's rows past the tile not loaded (neither is faster).
template <int ACT, int NT, int WAVES, int STAGES>
__global__ __launch_bounds__(64 * WAVES) void lora_fused_kernel(LoraParams p, int cols) {
  constexpr int RANKS = 32, RING = STAGES * (1 + NT) * kUnitBytes, B = 128 * 16 * NT * Act<ACT>::bytes;
  __shared__ __attribute__((aligned(1024))) uint8_t s_ring[WAVES][RING];
  __shared__ __attribute__((aligned(1024))) uint8_t s_b[WAVES][B];
  __shared__ __attribute__((aligned(16))) TileT<ACT, 16, RANKS> s_t;
  __shared__ __attribute__((aligned(16))) float s_f[16][16 * NT + 4];
  __shared__ int s_row[16];
  const int lane = threadIdx.x & 63, c16 = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const RowTile rt = find_rows<16>(p, static_cast<int>(blockIdx.x));
  if (!rt.found) return;
  const bool bare = rt.adapter < 0 || rt.adapter >= p.L;
  if (bare && p.base == p.y) return;
  const int first = static_cast<int>(blockIdx.y) * cols + 128 * wave;
  const int last = min((static_cast<int>(blockIdx.y) + 1) * cols, p.N);
  const BLayout l = b_layout<ACT>(p, 0);
  const uint32_t b_at = lds_address(s_b[wave]);
  Outputs<ACT> o;
  if (threadIdx.x < 16) s_row[threadIdx.x] = rt.begin + static_cast<int>(threadIdx.x) < rt.end
                                                 ? row_of(p, rt.begin + threadIdx.x) : -1;
  if (!bare && first < last) load_b<ACT, 128, 1>(p, rt.adapter, first, 0, l, b_at, 0);
  __syncthreads();
  o.set_rows(s_row, 0);
  if (bare) {
    copy_columns<ACT>(p, o, first, last, 128 * WAVES);
    return;
  }
  o.template load<false>(p, first < last ? first : p.N);
  {
    f32x4_t acc[NT];
    shrink_tile<ACT, NT, WAVES, STAGES>(p, rt, 0, wave, (p.K + kUnitK<ACT> - 1) / kUnitK<ACT>, s_ring[wave], acc);
    f32x4_t* sum = reinterpret_cast<f32x4_t*>(s_ring[wave]);
#pragma unroll
    for (int i = 0; i < NT; ++i) sum[i * 64 + lane] = acc[i];
  }
  __syncthreads();
  {
    if (wave < NT) {
      f32x4_t v = reinterpret_cast<const f32x4_t*>(s_ring[0])[wave * 64 + lane];
#pragma unroll
      for (int w = 1; w < WAVES; ++w) v += reinterpret_cast<const f32x4_t*>(s_ring[w])[wave * 64 + lane];
      *reinterpret_cast<f32x4_t*>(&s_f[c16][16 * wave + 4 * g]) = v;
    }
    __syncthreads();
    const int r = threadIdx.x / (RANKS / 8), k = threadIdx.x % (RANKS / 8) * 8;
    if (r < 16) {
      const float scale = p.scales ? p.scales[rt.adapter] : 1.0f;
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = k < p.rank && rt.begin + r < rt.end ? s_f[r][k + i] * scale : 0.0f;
      put_t<ACT, 16, RANKS>(s_t, r, k, v);
    }
    __syncthreads();
  }
  o.set_factors(s_t, 0);
  // (B of the steps takes turns between its own place and the ring, which is free)
  static_assert(B <= RING, "a step's B fits a wave's ring");
  const uint8_t* b_now = s_b[wave];
  const uint8_t* b_next = s_ring[wave];
  for (int n0 = first; n0 < last; n0 += 128 * WAVES) {
    const int next = n0 + 128 * WAVES;
    Outputs<ACT> behind = o;
    wait_loads<0>();
    if (next < last) {
      load_b<ACT, 128, 1>(p, rt.adapter, next, 0, l, lds_address(b_next), 0);
      behind.template load<false>(p, next);
    }
    f32x4_t acc[8];
    clear(acc);
    multiply_pass<ACT, 16, RANKS>(p, s_t, 0, b_now, l, 0, 0, acc);
    sums_of_t<ACT, 16, RANKS>(p, s_t, 0, rt.adapter, n0, acc, [&](int r, int k) {
      return s_f[r][k] * (p.scales ? p.scales[rt.adapter] : 1.0f);
    });
    o.template store<false>(p, n0, acc);
    wait_lds();
    o = behind;
    const uint8_t* was = b_now;
    b_now = b_next;
    b_next = was;
  }
}

namespace {

unsigned row_tiles(const LoraParams& p, int bm) {
  return static_cast<unsigned>(p.T / bm + std::min<int64_t>(p.T, p.L + 2));
}

template <int ACT, int NT>
void launch_shrink(const LoraParams& p, int rows, hipStream_t stream) {
  const dim3 grid(row_tiles(p, rows), p.splits, (p.rank + 16 * NT - 1) / (16 * NT));
  if (rows == 128) lora_shrink_rows_kernel<ACT, NT, 8, 3><<<grid, 512, 0, stream>>>(p);
  else if (rows == 64) lora_shrink_rows_kernel<ACT, NT, 4, 3><<<grid, 256, 0, stream>>>(p);
  else lora_shrink_kernel<ACT, NT, 4, NT == 4 ? 3 : 4><<<grid, 256, 0, stream>>>(p);
}
template <int ACT, int WM, int WN>
void launch_expand(const LoraParams& p, int cols, hipStream_t stream) {
  const dim3 grid(row_tiles(p, 16 * WM) * ((p.N + cols - 1) / cols));
  constexpr int threads = 64 * WM * WN;
  if (p.rank <= 64) lora_expand_kernel<ACT, WM, WN, 64><<<grid, threads, 0, stream>>>(p, cols);
  else if (p.rank <= 128) lora_expand_kernel<ACT, WM, WN, 128><<<grid, threads, 0, stream>>>(p, cols);
  else lora_expand_kernel<ACT, WM, WN, 256><<<grid, threads, 0, stream>>>(p, cols);
}

template <int ACT>
hipError_t launch_lora_as(const LoraParams& p, const LoraPlan& plan, hipStream_t stream) {
  if (plan.fused) {                    // (the stages and the columns' B fill most of the LDS)
    const dim3 grid(row_tiles(p, 16), (p.N + plan.cols - 1) / plan.cols);
    if (p.rank <= 16) lora_fused_kernel<ACT, 1, 8, ACT == ACT_F32 ? 2 : 3><<<grid, 512, 0, stream>>>(p, plan.cols);
    else lora_fused_kernel<ACT, 2, 4, ACT == ACT_F32 ? 3 : 4><<<grid, 256, 0, stream>>>(p, plan.cols);
    return hipGetLastError();
  }
  if (p.rank <= 16) launch_shrink<ACT, 1>(p, plan.shrink_rows, stream);
  else if (p.rank <= 32) launch_shrink<ACT, 2>(p, plan.shrink_rows, stream);
  else launch_shrink<ACT, 4>(p, plan.shrink_rows, stream);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (plan.many) launch_expand<ACT, 2, 2>(p, plan.cols, stream);
  else launch_expand<ACT, 1, 2>(p, plan.cols, stream);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_lora(const LoraParams& p, const LoraPlan& plan, int act, hipStream_t stream) {
  switch (act) {
    case ACT_F32: return launch_lora_as<ACT_F32>(p, plan, stream);
    case ACT_F16: return launch_lora_as<ACT_F16>(p, plan, stream);
    default: return launch_lora_as<ACT_BF16>(p, plan, stream);
  }
}

}  // namespace lowbit
