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
// from h * 2^-96 (exact), so that it is normalized as any other.
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

constexpr int kNormThreads = 256;

// Sum over the block's threads (every thread gets it), in one fixed order.
__device__ __forceinline__ float block_sum(float v, float* lds) {
  v = wave_sum(v);
  __syncthreads();                     // the array's last readers are done
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
  __syncthreads();
  float s = 0.0f;
#pragma unroll
  for (int w = 0; w < kNormThreads / 64; ++w) s += lds[w];
  return s;
}
__device__ __forceinline__ uint32_t block_max(uint32_t v, uint32_t* lds) {
  v = lanes_max<64>(v);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
  __syncthreads();
  uint32_t m = 0;
#pragma unroll
  for (int w = 0; w < kNormThreads / 64; ++w) m = max(m, lds[w]);
  return m;
}

}  // namespace

// One block per row; each thread takes 8-value chunks tid, tid + 256, ...;
// the chunks are read again (from cache) once the row's sum is known.  The 16
// lanes of an aligned group hold the 16 chunks of one block of 128.
template <int ACT, int FMT>
__global__ __launch_bounds__(kNormThreads) void norm_q8_kernel(NormQ8Params p) {
  __shared__ float s_sum[kNormThreads / 64];
  __shared__ uint32_t s_max[kNormThreads / 64];
  const int64_t m = blockIdx.x;
  const int tid = threadIdx.x;
  const int chunks = p.K / 8;
  const size_t row_bytes = static_cast<size_t>(p.K) * Act<ACT>::bytes;
  const char* x = static_cast<const char*>(p.x) + m * row_bytes;
  const char* r = p.residual ? static_cast<const char*>(p.residual) + m * row_bytes : nullptr;
  char* sum = p.sum ? static_cast<char*>(p.sum) + m * row_bytes : nullptr;
  const char* h_row = sum ? sum : x;   // a thread reads back what it wrote itself

  float ss = 0.0f;
  uint32_t top = 0;
  for (int c = tid; c < chunks; c += kNormThreads) {
    float v[8];
    load8<ACT>(x, c, v);
    if (r) {
      float w[8];
      load8<ACT>(r, c, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] += w[i];
      store8<ACT>(sum, c, v);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      ss = fmaf(v[i], v[i], ss);
      top = max(top, magnitude_bits(v[i]));
    }
  }
  ss = block_sum(ss, s_sum);
  float inv = 1.0f / sqrtf(ss / static_cast<float>(p.K) + p.eps);
  if (!(ss < __builtin_inff())) {      // the same for every thread of the block
    if (block_max(top, s_max) >= 0x7f800000u) {
      inv = __builtin_nanf("");
    } else {
      float s2 = 0.0f;
      for (int c = tid; c < chunks; c += kNormThreads) {
        float v[8];
        load8<ACT>(h_row, c, v);
#pragma unroll
        for (int i = 0; i < 8; ++i) s2 = fmaf(v[i] * 0x1p-96f, v[i] * 0x1p-96f, s2);
      }
      s2 = block_sum(s2, s_sum);
      inv = 0x1p-96f / sqrtf(s2 / static_cast<float>(p.K));
    }
  }

  auto normed = [&](int c, float (&v)[8]) {
    load8<ACT>(h_row, c, v);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] *= inv;
    if (p.weight) {
      float g[8];
      load8<ACT>(p.weight, c, g);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] *= g[i];
    }
  };
  auto write_y = [&](int c, const float (&v)[8]) {
    if (p.y) {
      float t[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) t[i] = v[i];
      store8<ACT>(static_cast<char*>(p.y) + m * row_bytes, c, t);
    }
  };
  uint8_t* q = static_cast<uint8_t*>(p.q) + m * p.K;
  if constexpr (FMT == Q8_I8) {
    uint32_t amax = 0;
    for (int c = tid; c < chunks; c += kNormThreads) {
      float v[8];
      normed(c, v);
#pragma unroll
      for (int i = 0; i < 8; ++i) amax = max(amax, magnitude_bits(v[i]));
    }
    amax = block_max(amax, s_max);
    const SpanScale s = span_scale(amax, kI8Max);
    if (tid == 0) p.qscale[m] = s.scale;
    for (int c = tid; c < chunks; c += kNormThreads) {
      float v[8];
      normed(c, v);
      write_y(c, v);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = s.finite ? v[i] * s.factor : 0.0f;
      *reinterpret_cast<u32v2_t*>(q + 8 * c) =
          u32v2_t{pack4_i8(v[0], v[1], v[2], v[3]), pack4_i8(v[4], v[5], v[6], v[7])};
    }
  } else {
    const int kb = (p.K + kF8Block - 1) / kF8Block;
    // whole groups of 16 lanes run each round; the last one's lanes past the
    // row take no part in its maximum
    for (int c0 = tid & ~15; c0 < chunks; c0 += kNormThreads) {
      const int c = c0 + (tid & 15);
      float v[8] = {};
      uint32_t amax = 0;
      if (c < chunks) {
        normed(c, v);
        write_y(c, v);
#pragma unroll
        for (int i = 0; i < 8; ++i) amax = max(amax, magnitude_bits(v[i]));
      }
      if constexpr (FMT == Q8_F8) {
        amax = lanes_max<16>(amax);
        const SpanScale s = span_scale(amax, kE4m3Max);
        if ((tid & 15) == 0) p.qscale[m * kb + (c0 >> 4)] = s.scale;
        if (c < chunks) {
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] = s.finite ? v[i] * s.factor : 0.0f;
          *reinterpret_cast<u32v2_t*>(q + 8 * c) =
              u32v2_t{pack4_e4m3(v[0], v[1], v[2], v[3]), pack4_e4m3(v[4], v[5], v[6], v[7])};
        }
      }
    }
  }
}

template <int ACT>
hipError_t launch_norm(const NormQ8Params& p, int fmt, hipStream_t s) {
  const dim3 grid(static_cast<unsigned>(p.M)), block(kNormThreads);
  switch (fmt) {
    case Q8_NONE: norm_q8_kernel<ACT, Q8_NONE><<<grid, block, 0, s>>>(p); break;
    case Q8_I8: norm_q8_kernel<ACT, Q8_I8><<<grid, block, 0, s>>>(p); break;
    default: norm_q8_kernel<ACT, Q8_F8><<<grid, block, 0, s>>>(p); break;
  }
  return hipGetLastError();
}

hipError_t launch_norm_q8(const NormQ8Params& p, int act, int fmt, hipStream_t s) {
  switch (act) {
    case ACT_F32: return launch_norm<ACT_F32>(p, fmt, s);
    case ACT_F16: return launch_norm<ACT_F16>(p, fmt, s);
    default: return launch_norm<ACT_BF16>(p, fmt, s);
  }
}

// e4m3 codes of the rows of x and the scale of each block of 128 of a row:
// 16 lanes a block, one 8-value chunk a lane, 16 blocks a thread block.
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
  amax = block_max(amax, s_max);
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
