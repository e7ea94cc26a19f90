// Routing of tokens to experts.  Per row of E logits l:
//
//   softmax: s_e = exp(l_e) / sum exp(l)      sigmoid: s_e = 1 / (1 + exp(-l_e))
//   c_e = s_e + b_e (with a bias)             what the experts are chosen by
//   of G groups of E / G neighbours, those with the largest value (the largest
//   c, or the sum of the two largest) stay; of their experts the k largest c,
//   in that order, the lowest index first among equal ones
//   weight_j = scale * s_j (/ the sum of the chosen s)
//
// Which expert is chosen is a discrete answer, so it must not hang on a
// rounding.  Where only the order of the scores counts (no bias, groups by
// their largest), the logits themselves are compared, which have the same
// order; otherwise c is computed in 64 bits.  The weights, k a row, are
// computed in 64 bits too and rounded once; for the sum over all the exps that
// softmax without renormalization divides by, 32 bits do.
//
// -inf masks an expert.  A row with fewer experts left than k ends in experts
// -1 with weight 0; a row holding a NaN (softmax: or +inf) gets experts 0 ..
// k - 1 and weights NaN, so that what it is used for shows it.
#include "device_common.h"

namespace lowbit {

namespace {

constexpr float kNegInf = -__builtin_huge_valf();

template <int CTRL> __device__ __forceinline__ float dpp_move(float v) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xf, 0xf, true));
}
template <int CTRL> __device__ __forceinline__ double dpp_move(double v) {
  const int lo = __builtin_amdgcn_update_dpp(0, __double2loint(v), CTRL, 0xf, 0xf, true);
  const int hi = __builtin_amdgcn_update_dpp(0, __double2hiint(v), CTRL, 0xf, 0xf, true);
  return __hiloint2double(hi, lo);
}
__device__ __forceinline__ float read_lane(float v, int lane) {
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), lane));
}
__device__ __forceinline__ double read_lane(double v, int lane) {
  return __hiloint2double(__builtin_amdgcn_readlane(__double2hiint(v), lane),
                          __builtin_amdgcn_readlane(__double2loint(v), lane));
}
__device__ __forceinline__ float larger(float a, float b) { return a > b ? a : b; }
__device__ __forceinline__ double larger(double a, double b) { return a > b ? a : b; }

// Maximum and sum over the LANES (16 or 64) lanes of a row, in every lane, in a
// fixed order: rotations within 16 lanes, then the four sixteens.
template <int LANES, class C>
__device__ __forceinline__ C row_max(C v) {
  v = larger(v, dpp_move<0x128>(v));   // row_ror 8, 4, 2, 1
  v = larger(v, dpp_move<0x124>(v));
  v = larger(v, dpp_move<0x122>(v));
  v = larger(v, dpp_move<0x121>(v));
  if constexpr (LANES == 64)
    v = larger(larger(read_lane(v, 0), read_lane(v, 16)), larger(read_lane(v, 32), read_lane(v, 48)));
  return v;
}
template <int LANES, class C>
__device__ __forceinline__ C row_sum(C v) {
  v += dpp_move<0x128>(v);
  v += dpp_move<0x124>(v);
  v += dpp_move<0x122>(v);
  v += dpp_move<0x121>(v);
  if constexpr (LANES == 64) v = (read_lane(v, 0) + read_lane(v, 16)) + (read_lane(v, 32) + read_lane(v, 48));
  return v;
}
// Bits of this lane's row in a ballot.
template <int LANES>
__device__ __forceinline__ uint64_t row_bits(uint64_t ballot) {
  if constexpr (LANES == 64) return ballot;
  else return (ballot >> (threadIdx.x & 48)) & 0xffffu;
}

__device__ __forceinline__ double sigmoid64(double l) {
  const double e = exp(-fabs(l));
  return l > 0.0 ? 1.0 / (1.0 + e) : e / (1.0 + e);
}

}  // namespace

constexpr int kRouteThreads = 256;

// LANES lanes a row, each with up to V neighbouring experts of one group in
// registers: a group has LANES / (G rounded up to a power of two) lanes.  One
// round of the selection is a maximum over a lane's values and one over the
// row's lanes; the lane that holds it (the first, and there the first value)
// takes it out.  C: what is compared, float logits or 64-bit choices.
template <class C, int LANES, int V, int ACT>
__global__ __launch_bounds__(kRouteThreads) void moe_route_kernel(RouteParams p) {
  constexpr bool VALUED = sizeof(C) == 8;
  constexpr int ROWS = kRouteThreads / LANES;
  __shared__ int s_chosen[ROWS][kRouteMaxTopk];
  const int lane = threadIdx.x % LANES;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * ROWS + threadIdx.x / LANES;
  if (row >= p.T) return;              // (whole sets of 16 lanes, and nothing below meets at a barrier)
  int* chosen = s_chosen[threadIdx.x / LANES];
  const int per_group = p.E / p.groups;
  const int group_lanes = LANES >> p.groups_shift;
  const int group = lane / group_lanes;
  const int per_lane = (per_group + group_lanes - 1) / group_lanes;
  const int at = lane % group_lanes * per_lane;          // of the group
  const int held = group < p.groups ? min(max(per_group - at, 0), per_lane) : 0;
  const int first = group * per_group + at;
  const typename Act<ACT>::bits_t* logits =
      static_cast<const typename Act<ACT>::bits_t*>(p.logits) + row * p.E;

  float l[V];
  float top = kNegInf;
  bool bad = false;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    l[i] = i < held ? act_bits_to_float<ACT>(logits[first + i]) : kNegInf;
    bad |= l[i] != l[i] || (!p.sigmoid && l[i] > 3.402823466e38f);
    top = larger(top, l[i]);
  }
  C c[V];
  double total = 1.0;                  // softmax: the sum of exp(l - top)
  if constexpr (VALUED) {
    top = row_max<LANES>(top);
    const double shift = top == kNegInf ? 0.0 : static_cast<double>(top);
    if (!p.sigmoid) {
      double sum = 0.0;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        c[i] = exp(static_cast<double>(l[i]) - shift);
        sum += c[i];
      }
      total = row_sum<LANES>(sum);
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const double s = p.sigmoid ? sigmoid64(l[i]) : c[i] / total;
      const double b = p.bias != nullptr && i < held ? static_cast<double>(p.bias[first + i]) : 0.0;
      c[i] = l[i] == kNegInf ? static_cast<double>(kNegInf) : s + b;
      bad |= c[i] != c[i];
    }
  } else {
    if (!p.sigmoid && !p.renormalize) {
      top = row_max<LANES>(top);
      const float shift = top == kNegInf ? 0.0f : top;
      float sum = 0.0f;
#pragma unroll
      for (int i = 0; i < V; ++i) sum += expf(l[i] - shift);
      total = static_cast<double>(row_sum<LANES>(sum));
    }
#pragma unroll
    for (int i = 0; i < V; ++i) c[i] = l[i];
  }
  bad = row_bits<LANES>(__ballot(bad)) != 0;

  if (p.groups > 1) {
    C a = kNegInf, b = kNegInf;        // the lane's two largest
#pragma unroll
    for (int i = 0; i < V; ++i) {
      b = larger(b, c[i] > a ? a : c[i]);
      a = larger(a, c[i]);
    }
    for (int o = 1; o < group_lanes; o <<= 1) {
      const C x = __shfl_xor(a, o), y = __shfl_xor(b, o);
      b = larger(larger(b, y), x > a ? a : x);
      a = larger(a, x);
    }
    C value = a;
    if constexpr (VALUED) {
      if (p.group_best == 2 && b != static_cast<C>(kNegInf)) value = a + b;
    }
    int before = 0;                    // groups that come before this one
    for (int g = 0; g < p.groups; ++g) {
      const C v = __shfl(value, g * group_lanes, LANES);
      before += v > value || (v == value && g < group);
    }
    if (before >= p.topk_groups) {
#pragma unroll
      for (int i = 0; i < V; ++i) c[i] = kNegInf;
    }
  }

  C best = c[0];
#pragma unroll
  for (int i = 1; i < V; ++i) best = larger(best, c[i]);
  for (int j = 0; j < p.topk; ++j) {
    const C m = row_max<LANES>(best);
    const bool none = m == static_cast<C>(kNegInf);
    const bool mine = lane == __builtin_ctzll(row_bits<LANES>(__ballot(best == m)) | (uint64_t{1} << 63));
    int i_of = 0;
#pragma unroll
    for (int i = V - 1; i >= 0; --i) i_of = c[i] == m ? i : i_of;
    if (mine) chosen[j] = bad ? j : none ? -1 : first + i_of;
    best = kNegInf;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      c[i] = mine && i == i_of ? static_cast<C>(kNegInf) : c[i];
      best = larger(best, c[i]);
    }
  }
  if (bad && lane == 0) {              // (a NaN is no maximum: no lane may have written)
    for (int j = 0; j < p.topk; ++j) chosen[j] = j;
  }
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");

  // the weights: lane j, j + LANES, ... takes the choices j, ...
  constexpr int PER = (kRouteMaxTopk + LANES - 1) / LANES;
  double s[PER];
  int expert[PER];
  float lj[PER];
  float best_l = kNegInf;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int j = lane + i * LANES;
    expert[i] = j < p.topk ? chosen[j] : -1;
    lj[i] = expert[i] >= 0 ? act_bits_to_float<ACT>(logits[expert[i]]) : kNegInf;
    best_l = larger(best_l, lj[i]);
  }
  best_l = row_max<LANES>(best_l);
  // renormalized, a common factor of the scores cancels: they are taken times
  // exp(-best_l) (sigmoid: only while that is below 0), so that none of them
  // leaves the range
  const double shift = best_l == kNegInf ? 0.0
                       : p.renormalize ? (p.sigmoid ? fmin(static_cast<double>(best_l), 0.0) : static_cast<double>(best_l))
                       : p.sigmoid ? 0.0 : static_cast<double>(top);
  double sum = 0.0;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const double x = lj[i];
    s[i] = 0.0;
    if (expert[i] >= 0) {
      if (!p.sigmoid) s[i] = exp(x - shift);
      else s[i] = x > 0.0 ? 1.0 / (1.0 + exp(-x)) : exp(x - shift) / (1.0 + exp(x));
    }
    sum += s[i];
  }
  sum = row_sum<LANES>(sum);
  const double by = p.renormalize ? (sum > 0.0 ? sum : 1.0) : total;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int j = lane + i * LANES;
    if (j < p.topk) {
      p.experts[row * p.topk + j] = expert[i];
      p.weights[row * p.topk + j] =
          bad ? __builtin_nanf("")
              : expert[i] < 0 ? 0.0f : static_cast<float>(s[i] / by * static_cast<double>(p.scale));
    }
  }
}

namespace {

template <class C, int LANES, int V>
hipError_t launch_route_as(const RouteParams& p, int act, hipStream_t stream) {
  constexpr int ROWS = kRouteThreads / LANES;
  const dim3 grid(static_cast<unsigned>((p.T + ROWS - 1) / ROWS)), block(kRouteThreads);
  switch (act) {
    case ACT_F32: moe_route_kernel<C, LANES, V, ACT_F32><<<grid, block, 0, stream>>>(p); break;
    case ACT_F16: moe_route_kernel<C, LANES, V, ACT_F16><<<grid, block, 0, stream>>>(p); break;
    default: moe_route_kernel<C, LANES, V, ACT_BF16><<<grid, block, 0, stream>>>(p); break;
  }
  return hipGetLastError();
}
template <class C>
hipError_t launch_route_of(const RouteParams& p, int act, hipStream_t stream) {
  const int per_group = p.E / p.groups;
  auto held = [&](int lanes) {
    const int g = lanes >> p.groups_shift;
    return g == 0 ? kRouteMaxExperts : (per_group + g - 1) / g;
  };
  if (held(16) <= 4) return launch_route_as<C, 16, 4>(p, act, stream);
  if (held(16) <= 8) return launch_route_as<C, 16, 8>(p, act, stream);
  if (held(16) <= 16) return launch_route_as<C, 16, 16>(p, act, stream);
  if (held(64) <= 16) return launch_route_as<C, 64, 16>(p, act, stream);
  return launch_route_as<C, 64, 32>(p, act, stream);
}

}  // namespace

hipError_t launch_moe_route(const RouteParams& p, int act, hipStream_t stream) {
  const bool valued = p.bias != nullptr || (p.groups > 1 && p.group_best == 2);
  return valued ? launch_route_of<double>(p, act, stream) : launch_route_of<float>(p, act, stream);
}

}  // namespace lowbit
