// Rows in the order of their expert, and the experts' rows added up for each
// token again.
//
// group_rows: a stable counting sort of S = T x topk expert ids.
//   position[s] = (ids below ids[s]) + (earlier slots with the same id)
//   rows[position[s]] = s / topk,   offsets[e] = ids below e
// Slots whose id is no expert come behind all others, with position -1.
//
// combine: out[t] = sum_j weights[t, j] * y[position[t, j]] (+ residual[t]) in
// fp32, products rounded before they are added: four sums, of the slots j, j +
// 4, ..., which then meet in order, and the residual last.
#include "f8_common.h"

namespace lowbit {

namespace {

__device__ __forceinline__ int wave_sum(int v) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) v += __shfl_xor(v, o);
  return v;
}

}  // namespace

// Block e finds the slots of expert e by itself (block E: those of none): it
// reads all ids, which lie in cache, counts the smaller ones and its own, and
// then writes its own in order.  No block waits for another, and nothing hangs
// on the order of atomics.  Wave w has a run of the slots.
template <class ID, int WAVES>
__global__ __launch_bounds__(64 * WAVES) void group_rows_kernel(GroupRowsParams p) {
  __shared__ int s_below[WAVES], s_own[WAVES];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int e = static_cast<int>(blockIdx.x);
  const ID* ids = static_cast<const ID*>(p.ids);
  const int S = static_cast<int>(p.S);
  const int run = (S + WAVES * 64 - 1) / (WAVES * 64) * 64;
  const int begin = min(wave * run, S), end = min(begin + run, S);
  auto id_at = [&](int s) {
    const ID id = ids[s];
    return id >= 0 && id < p.E ? static_cast<int>(id) : p.E;
  };

  int below = 0, own = 0;
  for (int s = begin + lane; s < end; s += 64) {
    const int id = id_at(s);
    below += id < e;
    own += id == e;
  }
  below = wave_sum(below);
  own = wave_sum(own);
  if (lane == 0) {
    s_below[wave] = below;
    s_own[wave] = own;
  }
  __syncthreads();
  int first = 0, before = 0;
#pragma unroll
  for (int w = 0; w < WAVES; ++w) {
    first += s_below[w];
    before += w < wave ? s_own[w] : 0;
  }
  if (threadIdx.x == 0) p.offsets[e] = first;

  int at = first + before;
  for (int s0 = begin; s0 < end; s0 += 64) {
    const int s = s0 + lane;
    const bool hit = s < end && id_at(s) == e;
    const uint64_t hits = __ballot(hit);
    if (hit) {
      const int to = at + __popcll(hits & ((uint64_t{1} << lane) - 1));
      p.rows[to] = s / p.topk;
      if (p.position) p.position[s] = e < p.E ? to : -1;
    }
    at += __popcll(hits);
  }
}

hipError_t launch_group_rows(const GroupRowsParams& p, int id_bytes, hipStream_t stream) {
  const dim3 grid(static_cast<unsigned>(p.E + 1));
  if (p.S <= 1024) {
    if (id_bytes == 8) group_rows_kernel<int64_t, 1><<<grid, 64, 0, stream>>>(p);
    else group_rows_kernel<int32_t, 1><<<grid, 64, 0, stream>>>(p);
  } else {
    if (id_bytes == 8) group_rows_kernel<int64_t, 16><<<grid, 1024, 0, stream>>>(p);
    else group_rows_kernel<int32_t, 16><<<grid, 1024, 0, stream>>>(p);
  }
  return hipGetLastError();
}

// A block has a token's row, or a run of it: each thread PIECE columns at a
// time (16 bytes of them where rows are whole 16-byte pieces, one element
// otherwise).  Bound by the bytes of the experts' rows.
constexpr int kCombineThreads = 256;

template <int ACT, bool WIDE>
__global__ __launch_bounds__(kCombineThreads) void moe_combine_kernel(CombineParams p, int runs) {
  constexpr int PIECE = WIDE ? 8 : 1;
  typedef typename Act<ACT>::bits_t T;
  const int64_t t = blockIdx.x / static_cast<unsigned>(runs);
  const int run = static_cast<int>(blockIdx.x % static_cast<unsigned>(runs));
  const int n = (run * kCombineThreads + static_cast<int>(threadIdx.x)) * PIECE;
  if (n >= p.N) return;
  const T* y = static_cast<const T*>(p.y);
  float part[4][PIECE] = {};
  auto add = [&](int j, float (&sum)[PIECE]) {
    const int64_t at = p.position[t * p.topk + j];
    const float w = p.weights[t * p.topk + j];
    if (at < 0) return;
    float v[PIECE];
    if (at >= p.R) {
#pragma unroll
      for (int i = 0; i < PIECE; ++i) v[i] = __builtin_nanf("");
    } else if constexpr (WIDE) {
      load8<ACT>(y + at * p.N, n / 8, v);
    } else {
      v[0] = load_act<ACT>(y + at * p.N, n);
    }
#pragma unroll
    for (int i = 0; i < PIECE; ++i) sum[i] += w * v[i];
  };
  for (int j0 = 0; j0 < p.topk; j0 += 4) {
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (j0 + q < p.topk) add(j0 + q, part[q]);
  }
  float sum[PIECE];
#pragma unroll
  for (int i = 0; i < PIECE; ++i) sum[i] = ((part[0][i] + part[1][i]) + part[2][i]) + part[3][i];
  if (p.residual) {
    float v[PIECE];
    const T* r = static_cast<const T*>(p.residual) + t * p.N;
    if constexpr (WIDE) load8<ACT>(r, n / 8, v);
    else v[0] = load_act<ACT>(r, n);
#pragma unroll
    for (int i = 0; i < PIECE; ++i) sum[i] += v[i];
  }
  T* out = static_cast<T*>(p.out) + t * p.N;
  if constexpr (WIDE) store8<ACT>(out, n / 8, sum);
  else store_act<ACT>(out, n, sum[0]);
}

namespace {

template <int ACT>
void launch_combine_as(const CombineParams& p, bool wide, hipStream_t stream) {
  const int per = kCombineThreads * (wide ? 8 : 1);
  const int runs = (p.N + per - 1) / per;
  const dim3 grid(static_cast<unsigned>(p.T * runs));
  if (wide) moe_combine_kernel<ACT, true><<<grid, kCombineThreads, 0, stream>>>(p, runs);
  else moe_combine_kernel<ACT, false><<<grid, kCombineThreads, 0, stream>>>(p, runs);
}

}  // namespace

hipError_t launch_moe_combine(const CombineParams& p, int act, hipStream_t stream) {
  auto whole = [](const void* q) { return reinterpret_cast<uintptr_t>(q) % 16 == 0; };
  const bool wide = p.N % 8 == 0 && whole(p.y) && whole(p.residual) && whole(p.out);
  switch (act) {
    case ACT_F32: launch_combine_as<ACT_F32>(p, wide, stream); break;
    case ACT_F16: launch_combine_as<ACT_F16>(p, wide, stream); break;
    default: launch_combine_as<ACT_BF16>(p, wide, stream); break;
  }
  return hipGetLastError();
}

}  // namespace lowbit
