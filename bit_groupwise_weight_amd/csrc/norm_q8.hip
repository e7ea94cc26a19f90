// Root-mean-square norm with the residual's addition and an 8-bit output,
// and the two quantizers of the fp8 format that stand without a norm.
//
// Per row of K values, in fp32:
//   h = round(x + residual)               (to the activation type; written out)
//   y = h / sqrt(sum_k h^2 / K + eps) * weight
//   int8:  one scale a row,          a = max |y| / 127, q = rint(y / a)
//   e4m3:  one scale a block of 128, s = max |y| / 448, q = e4m3(y / s)
// The norm is that of the rounded h, so that it normalizes what the residual
// stream carries on; y is not rounded before it is quantized.
//
// A row holding a NaN or an infinity: y is NaN throughout, its scales are NaN
// and its codes 0.  A finite row whose squares overflow fp32 is summed again
// from h * 2^-96 (exact), so that it is normalized as any other; it is divided
// in two steps, h * 2^-32 and the rest, as 1 / rms alone may be subnormal (what
// the first step loses of y is below fp32's smallest number).
#include "f8_common.h"

namespace lowbit {

namespace {

__device__ __forceinline__ uint32_t magnitude_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) v += __shfl_xor(v, o);
  return v;
}
template <int LANES>
__device__ __forceinline__ uint32_t lanes_max(uint32_t v) {
#pragma unroll
  for (int o = LANES / 2; o >= 1; o >>= 1) v = max(v, static_cast<uint32_t>(__shfl_xor(static_cast<int>(v), o)));
  return v;
}

// Sum and maximum over the T threads of a row (every thread gets them), in one
// fixed order; lds: T / 64 words that nothing else uses in the kernel.
template <int T>
__device__ __forceinline__ float row_sum(float v, float* lds) {
  v = wave_sum(v);
  if constexpr (T > 64) {
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
    __syncthreads();
    v = 0.0f;
#pragma unroll
    for (int w = 0; w < T / 64; ++w) v += lds[w];
  }
  return v;
}
template <int T>
__device__ __forceinline__ uint32_t row_max(uint32_t v, uint32_t* lds) {
  v = lanes_max<64>(v);
  if constexpr (T > 64) {
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
    __syncthreads();
    v = 0;
#pragma unroll
    for (int w = 0; w < T / 64; ++w) v = max(v, lds[w]);
  }
  return v;
}

// Eight codes of the values v / scale.
template <int FMT>
__device__ __forceinline__ u32v2_t codes8(const float (&v)[8], const SpanScale& s) {
  float t[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) t[i] = s.finite ? v[i] * s.factor : 0.0f;
  if constexpr (FMT == Q8_I8) return u32v2_t{pack4_i8(t[0], t[1], t[2], t[3]), pack4_i8(t[4], t[5], t[6], t[7])};
  else return u32v2_t{pack4_e4m3(t[0], t[1], t[2], t[3]), pack4_e4m3(t[4], t[5], t[6], t[7])};
}

}  // namespace

// T threads a row, each with the 8-value chunks tid, tid + T, ... of it in
// registers (C of them; C == 0: any number, read again from cache for each
// use).  The 16 lanes of an aligned group hold the chunks of one block of 128.
// Rows of one wave go four to a block.
// Bound by memory with many rows, by one round of latencies (load, row sum, row
// maximum, store) with few: a row is read once and its values wait in registers
// for the sum.  bf16 with residual to e4m3, MI355X: 8192 x 4096 43.5 us, 5.4 TB/s
// (a copy of 1 GiB: 5.1; a plain read of 4 GiB: 6.8); 1 x 4096 2.7 us.  int8, 128 x 14336: 4.1 us.
template <int ACT, int FMT, int T, int C>
__global__ __launch_bounds__(T == 64 ? 256 : T) void norm_q8_kernel(NormQ8Params p) {
  __shared__ float s_sum[2][T / 64];
  __shared__ uint32_t s_max[2][T / 64];
  const int64_t m = T == 64 ? static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 6) : blockIdx.x;
  if (T == 64 && m >= p.M) return;     // (no barrier in that form)
  const int tid = T == 64 ? threadIdx.x & 63 : threadIdx.x;
  const int chunks = p.K / 8;
  const int n = C ? C : (chunks + T - 1) / T;           // chunks of a thread, past the row's end included
  const size_t row_bytes = static_cast<size_t>(p.K) * Act<ACT>::bytes;
  const char* x = static_cast<const char*>(p.x) + m * row_bytes;
  const char* r = p.residual ? static_cast<const char*>(p.residual) + m * row_bytes : nullptr;
  char* sum = p.sum ? static_cast<char*>(p.sum) + m * row_bytes : nullptr;
  char* y = p.y ? static_cast<char*>(p.y) + m * row_bytes : nullptr;
  float kept[C ? C : 1][8];

  // h of chunk c: made and written once, then kept or read back (a thread reads
  // what it wrote itself)
  auto make_h = [&](int c, float (&v)[8]) {
    load8<ACT>(x, c, v);
    if (r) {
      float w[8];
      load8<ACT>(r, c, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] += w[i];
      store8<ACT>(sum, c, v);
    }
  };
  float ss = 0.0f;
  uint32_t top = 0;
#pragma unroll
  for (int k = 0; k < (C ? C : n); ++k) {
    float (&v)[8] = kept[C ? k : 0];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = 0.0f;
    if (tid + k * T < chunks) make_h(tid + k * T, v);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      ss = fmaf(v[i], v[i], ss);
      top = max(top, magnitude_bits(v[i]));
    }
  }
  auto h_of = [&](int k, float (&v)[8]) {
    if constexpr (C != 0) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = kept[k][i];
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = 0.0f;
      if (tid + k * T < chunks) load8<ACT>(sum ? sum : x, tid + k * T, v);
    }
  };
  ss = row_sum<T>(ss, s_sum[0]);
  float inv = 1.0f / sqrtf(ss / static_cast<float>(p.K) + p.eps);
  float down = 1.0f;                   // (of a row read again: kept ones are scaled in place)
  if (!(ss < __builtin_inff())) {      // the same for every thread of the row
    if (row_max<T>(top, s_max[0]) >= 0x7f800000u) {
      inv = __builtin_nanf("");
    } else {
      float s2 = 0.0f;
#pragma unroll
      for (int k = 0; k < (C ? C : n); ++k) {
        float v[8];
        h_of(k, v);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          s2 = fmaf(v[i] * 0x1p-96f, v[i] * 0x1p-96f, s2);
          if constexpr (C != 0) kept[k][i] *= 0x1p-32f;
        }
      }
      down = 0x1p-32f;
      inv = 0x1p-64f / sqrtf(row_sum<T>(s2, s_sum[1]) / static_cast<float>(p.K));
    }
  }

  auto normed = [&](int k, float (&v)[8]) {
    h_of(k, v);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = (C != 0 ? v[i] : v[i] * down) * inv;
    const int c = tid + k * T;
    if (p.weight && c < chunks) {
      float g[8];
      load8<ACT>(p.weight, c, g);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] *= g[i];
    }
  };
  auto top_of = [&](const float (&v)[8]) {
    uint32_t a = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) a = max(a, magnitude_bits(v[i]));
    return a;
  };
  auto write_y = [&](int c, const float (&v)[8]) {
    float t[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) t[i] = v[i];
    store8<ACT>(y, c, t);
  };
  uint8_t* q = static_cast<uint8_t*>(p.q) + m * p.K;
  if constexpr (FMT == Q8_I8) {
    uint32_t amax = 0;
#pragma unroll
    for (int k = 0; k < (C ? C : n); ++k) {
      float v[8];
      normed(k, v);
      // (lanes past the row hold 0 * inv: a NaN where the whole row is one)
      amax = max(amax, top_of(v));
      if constexpr (C != 0) {
#pragma unroll
        for (int i = 0; i < 8; ++i) kept[k][i] = v[i];
      }
    }
    const SpanScale s = span_scale(row_max<T>(amax, s_max[1]), kI8Max);
    if (tid == 0) p.qscale[m] = s.scale;
#pragma unroll
    for (int k = 0; k < (C ? C : n); ++k) {
      const int c = tid + k * T;
      float v[8];
      if constexpr (C != 0) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = kept[k][i];
      } else {
        normed(k, v);
      }
      if (c < chunks) {
        if (y) write_y(c, v);
        *reinterpret_cast<u32v2_t*>(q + 8 * c) = codes8<Q8_I8>(v, s);
      }
    }
  } else {
    const int kb = (p.K + kF8Block - 1) / kF8Block;
#pragma unroll
    for (int k = 0; k < (C ? C : n); ++k) {
      const int c = tid + k * T;
      float v[8];
      normed(k, v);
      if (y && c < chunks) write_y(c, v);
      if constexpr (FMT == Q8_F8) {
        // (lanes past the row's end take no part in the maximum of its last block)
        const SpanScale s = span_scale(lanes_max<16>(c < chunks ? top_of(v) : 0u), kE4m3Max);
        if ((tid & 15) == 0 && c < chunks) p.qscale[m * kb + (c >> 4)] = s.scale;
        if (c < chunks) *reinterpret_cast<u32v2_t*>(q + 8 * c) = codes8<Q8_F8>(v, s);
      }
    }
  }
}

template <int ACT, int FMT, int T, int C>
hipError_t launch_norm_rows(const NormQ8Params& p, hipStream_t s) {
  const int64_t blocks = T == 64 ? (p.M + 3) / 4 : p.M;
  norm_q8_kernel<ACT, FMT, T, C><<<dim3(static_cast<unsigned>(blocks)), dim3(T == 64 ? 256 : T), 0, s>>>(p);
  return hipGetLastError();
}

// The threads of a row by its length alone, so that a row's result does not
// depend on how many there are.  Up to 1024 values one wave a row, up to 8192 one
// chunk a thread: the smallest power of two that holds them, or 3/4 or 5/8 of it
// (in whole waves); beyond, 1024 threads with two or four chunks each.  us for
// many rows / one row, bf16 with residual to e4m3 (T x C), at each width's upper
// end and a little over it:
//   K = 512     64 x 1: 12.4 / 2.4     256 x 1: 19.9 / 2.5     (16384 rows)
//   K = 1024    64 x 2: 25.9 / 3.2     256 x 1: 30.8 / 2.5     (16384 rows)
//   K = 1056   192 x 1: 29.3 / 2.5     256 x 1: 33.1 / 2.6     (16384 rows)
//   K = 1536   192 x 1: 34.1           256 x 1: 36.8           (16384 rows)
//   K = 2048   256 x 1: 24.3 / 2.6     512 x 1: 30.7 / 2.6     (8192 rows)
//   K = 2080   320 x 1: 51.9 / 2.6     384 x 1: 55.9   512 x 1: 60.4 / 2.6   (16131 rows)
//   K = 2560   320 x 1: 46.1           384 x 1: 48.6   512 x 1: 52.1         (13107 rows)
//   K = 2576   384 x 1: 51.1           448 x 1: 53.3   512 x 1: 53.7         (13025 rows)
//   K = 3328   512 x 1: 46.2 / 2.7     448 x 1: 45.9 / 2.6     (10082 rows; int8 3360: 33.0 and 33.1)
//   K = 4096   512 x 1: 44.4 / 2.7     256 x 2: 46.9 / 3.5     (8192 rows)
//   K = 4128   640 x 1: 53.0 / 2.8     768 x 1: 58.5   1024 x 1: 61.2 / 2.8  (8128 rows; int8: 47.5, 48.4, 48.6)
//   K = 5120   640 x 1: 50.6 / 2.8     768 x 1: 51.1   1024 x 1: 52.5 / 2.8  (6553 rows)
//   K = 6144   768 x 1: 46.1 / 2.9     896 x 1: 46.8   1024 x 1: 47.4 / 2.9  (5461 rows)
//   K = 7168  1024 x 1: 45.6           896 x 1: 45.4           (4681 rows; int8: 35.7 and 36.5)
//   K = 8192  1024 x 1: 45.0 / 3.1     512 x 2: 46.9 / 3.6     (4096 rows)
//   K = 8224  1024 x 2: 51.7 / 3.5     640 x 2: 52.3 / 3.6     (4080 rows; fewer threads gain nothing)
//   K = 10240 1024 x 2: 49.6 / 3.5     640 x 2: 49.6 / 3.9     (3276 rows)
//   K = 14336 1024 x 2: 24.4 / 3.6     512 x 4: 22.0 / 4.0     (2048 rows, int8)
//   K = 16416 1024 x 4: 52.0 / 4.9     768 x 4: 51.6 / 5.0     (2044 rows)
//   K = 32768 1024 x 4: 50.5 / 6.6     re-read: 56.7 / 7.6     (1024 rows)
//   K = 65536  re-read: 60.7 / 13.0 of 1024, 92.3 / 35.2 of 256 (512 rows)
template <int ACT, int FMT>
hipError_t launch_norm(const NormQ8Params& p, hipStream_t s) {
  if (p.K > 32768) return launch_norm_rows<ACT, FMT, 1024, 0>(p, s);
  if (p.K > 16384) return launch_norm_rows<ACT, FMT, 1024, 4>(p, s);
  if (p.K > 8192) return launch_norm_rows<ACT, FMT, 1024, 2>(p, s);
  switch ((p.K + 511) / 512) {         // waves of one chunk a thread
    case 1: return launch_norm_rows<ACT, FMT, 64, 1>(p, s);
    case 2: return launch_norm_rows<ACT, FMT, 64, 2>(p, s);
    case 3: return launch_norm_rows<ACT, FMT, 192, 1>(p, s);
    case 4: return launch_norm_rows<ACT, FMT, 256, 1>(p, s);
    case 5: return launch_norm_rows<ACT, FMT, 320, 1>(p, s);
    case 6: return launch_norm_rows<ACT, FMT, 384, 1>(p, s);
    case 7: case 8: return launch_norm_rows<ACT, FMT, 512, 1>(p, s);
    case 9: case 10: return launch_norm_rows<ACT, FMT, 640, 1>(p, s);
    case 11: case 12: return launch_norm_rows<ACT, FMT, 768, 1>(p, s);
    default: return launch_norm_rows<ACT, FMT, 1024, 1>(p, s);
  }
}

template <int ACT>
hipError_t launch_norm_fmt(const NormQ8Params& p, int fmt, hipStream_t s) {
  switch (fmt) {
    case Q8_NONE: return launch_norm<ACT, Q8_NONE>(p, s);
    case Q8_I8: return launch_norm<ACT, Q8_I8>(p, s);
    default: return launch_norm<ACT, Q8_F8>(p, s);
  }
}

hipError_t launch_norm_q8(const NormQ8Params& p, int act, int fmt, hipStream_t s) {
  switch (act) {
    case ACT_F32: return launch_norm_fmt<ACT_F32>(p, fmt, s);
    case ACT_F16: return launch_norm_fmt<ACT_F16>(p, fmt, s);
    default: return launch_norm_fmt<ACT_BF16>(p, fmt, s);
  }
}

// e4m3 codes of the rows of x and the scale of each block of 128 of a row:
// 16 lanes a block, one 8-value chunk a lane, 16 blocks a thread block.  Bound
// by memory: bf16 8192 x 4096 21.5 us, 4.7 TB/s; 1 x 4096 2.0 us.
template <int ACT>
__global__ __launch_bounds__(256) void act_quant_f8_kernel(ActQuantF8Params p) {
  const int kb = (p.K + kF8Block - 1) / kF8Block;
  const int64_t blk = static_cast<int64_t>(blockIdx.x) * 16 + (threadIdx.x >> 4);
  if (blk >= p.M * kb) return;         // whole groups of 16 lanes leave together
  const int64_t m = blk / kb;
  const int b = static_cast<int>(blk - m * kb);
  const int c = 16 * b + (threadIdx.x & 15);
  const char* row = static_cast<const char*>(p.x) + static_cast<size_t>(m) * p.K * Act<ACT>::bytes;
  float v[8] = {};
  uint32_t amax = 0;
  const bool in = 8 * c < p.K;
  if (in) {
    load8<ACT>(row, c, v);
#pragma unroll
    for (int i = 0; i < 8; ++i) amax = max(amax, magnitude_bits(v[i]));
  }
  amax = lanes_max<16>(amax);
  const SpanScale s = span_scale(amax, kE4m3Max);
  if ((threadIdx.x & 15) == 0) p.xscale[blk] = s.scale;
  if (in) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = s.finite ? v[i] * s.factor : 0.0f;
    *reinterpret_cast<u32v2_t*>(p.xq + m * p.K + 8 * c) =
        u32v2_t{pack4_e4m3(v[0], v[1], v[2], v[3]), pack4_e4m3(v[4], v[5], v[6], v[7])};
  }
}

hipError_t launch_act_quant_f8(const ActQuantF8Params& p, int act, hipStream_t s) {
  const int64_t blocks = p.M * ((p.K + kF8Block - 1) / kF8Block);
  const dim3 grid(static_cast<unsigned>((blocks + 15) / 16)), block(256);
  switch (act) {
    case ACT_F32: act_quant_f8_kernel<ACT_F32><<<grid, block, 0, s>>>(p); break;
    case ACT_F16: act_quant_f8_kernel<ACT_F16><<<grid, block, 0, s>>>(p); break;
    default: act_quant_f8_kernel<ACT_BF16><<<grid, block, 0, s>>>(p); break;
  }
  return hipGetLastError();
}

// e4m3 codes of weights w[E, N, K] and the scale of each block of 128 x 128
// (rows of one matrix): one thread block a weight block; a thread takes one
// chunk of a row in each of 8 passes of 16 rows and keeps them in registers.
// Bound by memory: bf16 14336 x 4096 38 us, 4.6 TB/s.
template <int ACT>
__global__ __launch_bounds__(256) void weight_quant_f8_kernel(WeightQuantF8Params p) {
  __shared__ uint32_t s_max[4];
  const int kb = (p.K + kF8Block - 1) / kF8Block, nb = (p.N + kF8Block - 1) / kF8Block;
  const int64_t blk = blockIdx.x;
  const int64_t e = blk / (static_cast<int64_t>(nb) * kb);
  const int rest = static_cast<int>(blk - e * nb * kb);
  const int n0 = rest / kb * kF8Block, b = rest % kb;
  const int c = 16 * b + (threadIdx.x & 15);
  const int r0 = threadIdx.x >> 4;
  float v[8][8];
  uint32_t amax = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int n = n0 + 16 * i + r0;
    if (n < p.N && 8 * c < p.K) {
      const int64_t row = e * p.N + n;
      load8<ACT>(static_cast<const char*>(p.w) + static_cast<size_t>(row) * p.K * Act<ACT>::bytes, c, v[i]);
#pragma unroll
      for (int j = 0; j < 8; ++j) amax = max(amax, magnitude_bits(v[i][j]));
    }
  }
  amax = row_max<256>(amax, s_max);
  const SpanScale s = span_scale(amax, kE4m3Max);
  if (threadIdx.x == 0) p.wscale[blk] = s.scale;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int n = n0 + 16 * i + r0;
    if (n < p.N && 8 * c < p.K) {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] = s.finite ? v[i][j] * s.factor : 0.0f;
      *reinterpret_cast<u32v2_t*>(p.wq + (e * p.N + n) * p.K + 8 * c) =
          u32v2_t{pack4_e4m3(v[i][0], v[i][1], v[i][2], v[i][3]),
                  pack4_e4m3(v[i][4], v[i][5], v[i][6], v[i][7])};
    }
  }
}

hipError_t launch_weight_quant_f8(const WeightQuantF8Params& p, int act, hipStream_t s) {
  const int64_t kb = (p.K + kF8Block - 1) / kF8Block, nb = (p.N + kF8Block - 1) / kF8Block;
  const dim3 grid(static_cast<unsigned>(p.E * nb * kb)), block(256);
  switch (act) {
    case ACT_F32: weight_quant_f8_kernel<ACT_F32><<<grid, block, 0, s>>>(p); break;
    case ACT_F16: weight_quant_f8_kernel<ACT_F16><<<grid, block, 0, s>>>(p); break;
    default: weight_quant_f8_kernel<ACT_BF16><<<grid, block, 0, s>>>(p); break;
  }
  return hipGetLastError();
}

}  // namespace lowbit
