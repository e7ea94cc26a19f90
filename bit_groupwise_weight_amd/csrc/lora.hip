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
#include "f8_common.h"

#include <algorithm>

namespace lowbit {

namespace {

// 8 consecutive values of a row, K positions of one lane in a step of 32.
template <int ACT> struct Chunk {      // 16-bit types
  u32v4_t w;
  __device__ __forceinline__ void load(const void* p, size_t at) {
    w = *reinterpret_cast<const u32v4_t*>(static_cast<const uint16_t*>(p) + at);
  }
  __device__ __forceinline__ void zero() { w = u32v4_t{0u, 0u, 0u, 0u}; }
};
template <> struct Chunk<ACT_F32> {
  f32x4_t v[2];
  __device__ __forceinline__ void load(const void* p, size_t at) {
    const f32x4_t* q = reinterpret_cast<const f32x4_t*>(static_cast<const float*>(p) + at);
    v[0] = q[0];
    v[1] = q[1];
  }
  __device__ __forceinline__ void zero() { v[0] = v[1] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f}; }
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
// Tile `tile` of BM rows among all groups' tiles.
template <int BM>
__device__ __forceinline__ RowTile find_rows(const LoraParams& p, int tile) {
  RowTile t{0, 0, -1, false};
  const int lane = threadIdx.x & 63;
  int before = 0;
  for (int v0 = 0; v0 < p.L + 2; v0 += 64) {
    int lo, hi;
    group_bounds(p, v0 + lane, &lo, &hi);
    const int own = (hi - lo + BM - 1) / BM;
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
      t.begin = __builtin_amdgcn_readlane(lo, src) + __builtin_amdgcn_readlane(tile - first, src) * BM;
      t.end = min(t.begin + BM, __builtin_amdgcn_readlane(hi, src));
      t.adapter = v0 + src - 1;
      t.found = true;
      return t;
    }
    before += __builtin_amdgcn_readlane(upto, 63);
  }
  return t;
}

// Row of position t, -1 where it is no row.
__device__ __forceinline__ int row_of(const LoraParams& p, int t) {
  const int64_t r = p.rows ? p.rows[t] : t;
  return r >= 0 && r < p.M ? static_cast<int>(r) : -1;
}

}  // namespace

constexpr int kLoraThreads = 256, kLoraWaves = 4;

// t of a tile of 16 MT positions and 16 NT ranks, over the K range of
// blockIdx.y: the waves take its steps of 32 in turn, their sums meet in LDS.
template <int ACT, int MT, int NT>
__global__ __launch_bounds__(kLoraThreads) void lora_shrink_kernel(LoraParams p) {
  __shared__ f32x4_t s_sum[kLoraWaves][NT * MT][64];
  const int lane = threadIdx.x & 63, c16 = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const RowTile rt = find_rows<16 * MT>(p, static_cast<int>(blockIdx.x));
  if (!rt.found || rt.adapter < 0 || rt.adapter >= p.L) return;
  const int r0 = static_cast<int>(blockIdx.z) * 16 * NT;
  const int k_begin = static_cast<int>(blockIdx.y) * p.k_split, k_end = min(k_begin + p.k_split, p.K);

  size_t x_at[MT], a_at[NT];
#pragma unroll
  for (int j = 0; j < MT; ++j) {
    const int row = row_of(p, min(rt.begin + 16 * j + c16, rt.end - 1));
    x_at[j] = static_cast<size_t>(max(row, 0)) * p.K;
  }
#pragma unroll
  for (int i = 0; i < NT; ++i)
    a_at[i] = (static_cast<size_t>(rt.adapter) * p.rank + min(r0 + 16 * i + c16, p.rank - 1)) * p.K;

  f32x4_t acc[NT][MT];
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int j = 0; j < MT; ++j) acc[i][j] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 2
  for (int k0 = k_begin + 32 * wave; k0 < k_end; k0 += 32 * kLoraWaves) {
    const int k = k0 + 8 * g;
    Chunk<ACT> x[MT], a[NT];
    if (k < p.K) {
#pragma unroll
      for (int j = 0; j < MT; ++j) x[j].load(p.x, x_at[j] + k);
#pragma unroll
      for (int i = 0; i < NT; ++i) a[i].load(p.a, a_at[i] + k);
    } else {                           // (K is a multiple of 16: the last step may be half)
#pragma unroll
      for (int j = 0; j < MT; ++j) x[j].zero();
#pragma unroll
      for (int i = 0; i < NT; ++i) a[i].zero();
    }
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int j = 0; j < MT; ++j) acc[i][j] = mfma<ACT>(a[i], x[j], acc[i][j]);
  }
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int j = 0; j < MT; ++j) s_sum[wave][i * MT + j][lane] = acc[i][j];
  __syncthreads();
  float* plane = p.t + static_cast<size_t>(blockIdx.y) * p.T * p.rank_pad;
  for (int q = wave; q < NT * MT; q += kLoraWaves) {
    const int i = q / MT, j = q % MT;
    f32x4_t v = s_sum[0][q][lane];
#pragma unroll
    for (int w = 1; w < kLoraWaves; ++w) v += s_sum[w][q][lane];
    const int t = rt.begin + 16 * j + c16, r = r0 + 16 * i + 4 * g;
    if (t < rt.end && r < p.rank_pad)
      *reinterpret_cast<f32x4_t*>(plane + static_cast<size_t>(t) * p.rank_pad + r) = v;
  }
}

namespace {

// t of a tile's BM rows in LDS, ready for the second product: rows of `pitch`
// elements, an odd number of 16-byte pieces, so that the 16 rows of a read
// start in different banks; 16-bit types have the hi halves of all rows and
// then the lo halves.
__device__ __forceinline__ int t_lanes(int rank) {   // lanes of a row, 8 ranks each
  int lanes = 4;
  while (lanes * 8 < rank) lanes *= 2;
  return lanes;
}
__device__ __forceinline__ int t_pitch(int rank) { return t_lanes(rank) * 8 + 8; }

// Eight values of t for row r from rank k on; the `lanes` lanes of a row call it
// together.
template <int ACT, int BM>
__device__ __forceinline__ void put_t(void* lds, float* unscale, int pitch, int r, int k, float (&v)[8],
                                      int lanes) {
  if constexpr (ACT == ACT_F32) {
    f32x4_t* to = reinterpret_cast<f32x4_t*>(static_cast<float*>(lds) + r * pitch + k);
    to[0] = f32x4_t{v[0], v[1], v[2], v[3]};
    to[1] = f32x4_t{v[4], v[5], v[6], v[7]};
  } else {
    if constexpr (ACT == ACT_F16) {
      uint32_t top = 0;                // bits of the row's largest magnitude
#pragma unroll
      for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(v[i]) & 0x7fffffffu);
      for (int o = 1; o < lanes; o <<= 1)
        top = max(top, static_cast<uint32_t>(__shfl_xor(static_cast<int>(top), o)));
      // 2^-e with e the exponent of the largest, within fp32's normal powers
      const int e = min(max(static_cast<int>(top >> 23), 1), 253);
      const float scale = __uint_as_float(static_cast<uint32_t>(254 - e) << 23);
      if (k == 0) unscale[r] = __uint_as_float(static_cast<uint32_t>(e) << 23);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] *= scale;
    }
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      hi[i] = pack2<ACT>(v[2 * i], v[2 * i + 1]);
      const float h0 = act_bits_to_float<ACT>(hi[i] & 0xffffu), h1 = act_bits_to_float<ACT>(hi[i] >> 16);
      // (an infinity has no rest)
      lo[i] = pack2<ACT>(fabsf(h0) <= 3.402823466e38f ? v[2 * i] - h0 : 0.0f,
                         fabsf(h1) <= 3.402823466e38f ? v[2 * i + 1] - h1 : 0.0f);
    }
    uint16_t* to = static_cast<uint16_t*>(lds) + r * pitch + k;
    *reinterpret_cast<u32v4_t*>(to) = u32v4_t{hi[0], hi[1], hi[2], hi[3]};
    *reinterpret_cast<u32v4_t*>(to + BM * pitch) = u32v4_t{lo[0], lo[1], lo[2], lo[3]};
  }
}

// base (or 0) + delta for 8 consecutive columns of a row.
template <int ACT>
__device__ __forceinline__ void add_row8(const LoraParams& p, int row, int n, const float (&d)[8], bool wide) {
  typedef typename Act<ACT>::bits_t T;
  const size_t at = static_cast<size_t>(row) * p.N + n;
  const T* base = static_cast<const T*>(p.base);
  T* y = static_cast<T*>(p.y);
  if (wide) {                          // (N % 8 == 0: all eight are columns)
    float v[8] = {};
    if (base) load8<ACT>(base + at, 0, v);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] += d[i];
    store8<ACT>(y + at, 0, v);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (n + i < p.N) store_act<ACT>(y, at + i, (base ? load_act<ACT>(base, at + i) : 0.0f) + d[i]);
  }
}

}  // namespace

// y of a tile of 16 MT positions and 256 columns, 64 a wave.
template <int ACT, int MT>
__global__ __launch_bounds__(kLoraThreads) void lora_expand_kernel(LoraParams p) {
  constexpr int BM = 16 * MT;
  extern __shared__ __attribute__((aligned(16))) uint8_t s_t[];
  __shared__ int s_row[BM];
  __shared__ float s_unscale[BM];
  const int lane = threadIdx.x & 63, c16 = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const RowTile rt = find_rows<BM>(p, static_cast<int>(blockIdx.x));
  if (!rt.found) return;
  const bool bare = rt.adapter < 0 || rt.adapter >= p.L;
  if (bare && p.base == p.y) return;
  const int n0 = (static_cast<int>(blockIdx.y) * kLoraWaves + wave) * 64;
  const bool wide = p.wide;

  for (int r = threadIdx.x; r < BM; r += kLoraThreads)
    s_row[r] = rt.begin + r < rt.end ? row_of(p, rt.begin + r) : -1;
  const int steps = (p.rank_pad + 31) / 32, pitch = t_pitch(p.rank);
  if (!bare) {
    const float scale = p.scales ? p.scales[rt.adapter] : 1.0f;
    const int lanes = t_lanes(p.rank);
    for (int r = threadIdx.x / lanes; r < BM; r += kLoraThreads / lanes) {
      const int k = threadIdx.x % lanes * 8;
      float v[8] = {};
      if (k < p.rank && rt.begin + r < rt.end) {
        for (int s = 0; s < p.splits; ++s) {
          const f32x4_t* from = reinterpret_cast<const f32x4_t*>(
              p.t + (static_cast<size_t>(s) * p.T + rt.begin + r) * p.rank_pad + k);
          const f32x4_t a = from[0], b = from[1];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            v[i] += a[i];
            v[4 + i] += b[i];
          }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] *= scale;
      }
      put_t<ACT, BM>(s_t, s_unscale, pitch, r, k, v, lanes);
    }
  }
  __syncthreads();

  // two MFMA tiles make 32 columns: row 4 g + i of tile j is column 8 g + 4 j + i,
  // so that a lane ends with 8 consecutive ones
#pragma unroll 1
  for (int h = 0; h < 2; ++h) {
    const int n = n0 + 32 * h;
    if (n >= p.N) break;
    f32x4_t acc[2][MT];
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int m = 0; m < MT; ++m) acc[j][m] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
    if (!bare) {
      size_t b_at[2];
#pragma unroll
      for (int j = 0; j < 2; ++j)
        b_at[j] = (static_cast<size_t>(rt.adapter) * p.N + min(n + 8 * (c16 >> 2) + 4 * j + (c16 & 3), p.N - 1)) *
                  p.rank;
      const bool both = ACT != ACT_F32 && p.rank_pad == 16;   // hi and lo in one step
#pragma unroll 1
      for (int s = 0; s < steps; ++s) {
        const int k = both ? 8 * (g & 1) : 32 * s + 8 * g;
        Chunk<ACT> b[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          if (k < p.rank) b[j].load(p.b, b_at[j] + k);
          else b[j].zero();
        }
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          const int t_at = (16 * m + c16) * pitch + k, t_lo = BM * pitch;
          Chunk<ACT> t;
          t.load(s_t, t_at + (both && g >= 2 ? t_lo : 0));
#pragma unroll
          for (int j = 0; j < 2; ++j) acc[j][m] = mfma<ACT>(b[j], t, acc[j][m]);
          if constexpr (ACT != ACT_F32) {
            if (!both) {
              t.load(s_t, t_at + t_lo);
#pragma unroll
              for (int j = 0; j < 2; ++j) acc[j][m] = mfma<ACT>(b[j], t, acc[j][m]);
            }
          }
        }
      }
    }
    if (n + 8 * g >= p.N) continue;
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      const int row = s_row[16 * m + c16];
      if (row < 0) continue;
      float by = 1.0f;
      if constexpr (ACT == ACT_F16) by = bare ? 1.0f : s_unscale[16 * m + c16];
      float d[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) d[i] = acc[i >> 2][m][i & 3] * by;
      add_row8<ACT>(p, row, n + 8 * g, d, wide);
    }
  }
}

namespace {

template <int ACT>
hipError_t launch_lora_as(const LoraParams& p, const LoraPlan& plan, hipStream_t stream) {
  auto tiles = [&](int bm) { return static_cast<unsigned>(p.T / bm + std::min<int64_t>(p.T, p.L + 2)); };
  if (plan.shrink_mt == 4) {
    const dim3 grid(tiles(64), p.splits, (p.rank + 63) / 64);
    lora_shrink_kernel<ACT, 4, 4><<<grid, kLoraThreads, 0, stream>>>(p);
  } else {
    const dim3 grid(tiles(16), p.splits, (p.rank + 63) / 64);
    lora_shrink_kernel<ACT, 1, 4><<<grid, kLoraThreads, 0, stream>>>(p);
  }
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const unsigned columns = static_cast<unsigned>((p.N + 255) / 256);
  int pitch = 32;                      // as t_pitch
  while (pitch < p.rank) pitch *= 2;
  const size_t row_bytes = static_cast<size_t>(pitch + 8) * 4;       // hi and lo, or fp32
  if (plan.expand_mt == 4)
    lora_expand_kernel<ACT, 4><<<dim3(tiles(64), columns), kLoraThreads, 64 * row_bytes, stream>>>(p);
  else
    lora_expand_kernel<ACT, 1><<<dim3(tiles(16), columns), kLoraThreads, 16 * row_bytes, stream>>>(p);
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
