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
// their largest), it is that of the logits; otherwise it is that of c in 64
// bits.  The weights, k a row, are computed in 64 bits too and rounded once; in
// the sum over all the exps that softmax without renormalization divides by, each
// is good to 32 bits.
//
// The selection itself runs on 32-bit keys that are cheap to compare: c in fp32
// with the expert's index in the low bits.  For 16-bit logits a key is exact.
// For others it brings three experts more than asked for, whose exact values
// then decide, and a row whose k-th expert and first left out are closer than
// the keys can tell is done again with exact values.
//
// -inf masks an expert.  A row with fewer experts left than k ends in experts
// -1 with weight 0; a row holding a NaN (softmax: or +inf) gets experts 0 ..
// k - 1 and weights NaN, so that what it is used for shows it.
#include "f8_common.h"

#include <type_traits>

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

__device__ __forceinline__ uint32_t row_max16(uint32_t v) {
  v = max(v, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(v), 0x128, 0xf, 0xf, true)));
  v = max(v, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(v), 0x124, 0xf, 0xf, true)));
  v = max(v, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(v), 0x122, 0xf, 0xf, true)));
  return max(v, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(v), 0x121, 0xf, 0xf, true)));
}
template <int LANES>
__device__ __forceinline__ uint32_t row_max_key(uint32_t v) {
  v = row_max16(v);
  if constexpr (LANES == 64) {
    const int w = static_cast<int>(v);
    v = max(max(static_cast<uint32_t>(__builtin_amdgcn_readlane(w, 0)), static_cast<uint32_t>(__builtin_amdgcn_readlane(w, 16))),
            max(static_cast<uint32_t>(__builtin_amdgcn_readlane(w, 32)), static_cast<uint32_t>(__builtin_amdgcn_readlane(w, 48))));
  }
  return v;
}

// Floats as unsigned integers of the same order (-inf: 0x007fffff).
__device__ __forceinline__ uint32_t ordered(float v) {
  const uint32_t b = __float_as_uint(v);
  return b ^ ((b >> 31) != 0 ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float unordered(uint32_t k) {
  return __uint_as_float((k >> 31) != 0 ? k ^ 0x80000000u : ~k);
}

__device__ __forceinline__ double sigmoid64(double l) {
  const double e = exp(-fabs(l));
  return (l > 0.0 ? 1.0 : e) / (1.0 + e);
}
// exp(l - top), l <= top, within 2^-32 of itself (of 2^-1000 below that, -inf too):
// 2^n times the series to f^8 / 8!, |f| <= ln(2) / 2, whose rest is less than 2^-32.
// (fp32 exponentials and sums left the weights errors as large as their rounding;
// us, those / these: 1237 x 60 fp16 4.35 / 4.37, 8192 x 256 bf16 6.5 / 6.9.)
__device__ __forceinline__ double exp_below(float l, float top) {
  const double x = fmax(static_cast<double>(l) - static_cast<double>(top), -700.0);
  const double n = rint(x * 1.4426950408889634);
  const double f = fma(n, -0.6931471805599453, x);
  double p = 1.0 / 40320.0;
  p = fma(p, f, 1.0 / 5040.0);
  p = fma(p, f, 1.0 / 720.0);
  p = fma(p, f, 1.0 / 120.0);
  p = fma(p, f, 1.0 / 24.0);
  p = fma(p, f, 1.0 / 6.0);
  p = fma(p, f, 0.5);
  p = fma(p, f, 1.0);
  return ldexp(fma(p, f, 1.0), static_cast<int>(n));
}
// The same within 2^-21: with e = exp(-l) the exponent's rounding makes |l|
// log2(e) 2^-24 of e, which is |l| 2^-23.4 s (1 - s) of s and less than 2^-25 (|l|
// s (1 - s) is below 0.23), the exponential and the reciprocal (good to a unit in
// the last place), the product and the sum at most 2^-23 s each.  (e may be
// infinite, s then 0.)
__device__ __forceinline__ float sigmoid32(float l) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-1.44269504f * l));
}

}  // namespace

constexpr int kRouteThreads = 256;

namespace {

// Where a lane's values stand: LANES lanes a row, each with up to V neighbouring
// experts of one group; a group has LANES / (G rounded up to a power of two)
// lanes.
struct RouteLane {
  int lane, group, group_lanes;
  int first, held;        // experts first .. first + held - 1
};
template <int LANES>
__device__ __forceinline__ RouteLane route_lane(const RouteParams& p) {
  RouteLane r;
  r.lane = threadIdx.x % LANES;
  const int per_group = p.E / p.groups;
  r.group_lanes = LANES >> p.groups_shift;
  r.group = r.lane / r.group_lanes;
  const int per_lane = (per_group + r.group_lanes - 1) / r.group_lanes;
  const int at = r.lane % r.group_lanes * per_lane;      // of the group
  r.held = r.group < p.groups ? min(max(per_group - at, 0), per_lane) : 0;
  r.first = r.group * per_group + at;
  return r;
}

// The two largest c of a lane, *a >= *b, and with one more.
__device__ __forceinline__ void add_to_two(double v, double* a, double* b) {
  *b = larger(*b, v > *a ? *a : v);
  *a = larger(*a, v);
}
__device__ __forceinline__ void add_to_two(float v, float* a, float* b) {
  *b = __builtin_amdgcn_fmed3f(*a, *b, v);
  *a = fmaxf(*a, v);
}
// The two largest of the group from those of its lanes, in every lane of it.
template <class C> __device__ __forceinline__ void two_of_group(const RouteLane& r, C* a, C* b) {
  for (int o = 1; o < r.group_lanes; o <<= 1) {
    const C x = __shfl_xor(*a, o), y = __shfl_xor(*b, o);
    *b = larger(larger(*b, y), x > *a ? *a : x);
    *a = larger(*a, x);
  }
}
// Whether the lane's group stays, from its two largest c; *gap: how far apart the
// values of the last that stays and the first that does not are.
template <class C, int LANES>
__device__ __forceinline__ bool group_stays(const RouteParams& p, const RouteLane& r, C a, C b, C* gap) {
  const C value = p.group_best == 2 && b != static_cast<C>(kNegInf) ? a + b : a;
  int before = 0;                      // groups that come before this one
  for (int g = 0; g < p.groups; ++g) {
    const C v = __shfl(value, g * r.group_lanes, LANES);
    before += v > value || (v == value && g < r.group);
  }
  const bool stays = before < p.topk_groups;
  const bool any = r.group < p.groups;
  const C last = -row_max<LANES>(any && stays ? -value : static_cast<C>(kNegInf));
  *gap = last - row_max<LANES>(any && !stays ? value : static_cast<C>(kNegInf));
  return stays;
}

// The topk experts of largest c, exactly and in order, into `chosen`.
template <class C, int LANES, int V>
__device__ __forceinline__ void select_exact(const RouteParams& p, const RouteLane& r, C (&c)[V], int* chosen) {
  C best = c[0];
#pragma unroll
  for (int i = 1; i < V; ++i) best = larger(best, c[i]);
  for (int j = 0; j < p.topk; ++j) {
    const C m = row_max<LANES>(best);
    const bool none = m == static_cast<C>(kNegInf);
    const bool mine = r.lane == __builtin_ctzll(row_bits<LANES>(__ballot(best == m)) | (uint64_t{1} << 63));
    int i_of = 0;
#pragma unroll
    for (int i = V - 1; i >= 0; --i) i_of = c[i] == m ? i : i_of;
    if (mine) chosen[j] = none ? -1 : r.first + i_of;
    best = kNegInf;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      c[i] = mine && i == i_of ? static_cast<C>(kNegInf) : c[i];
      best = larger(best, c[i]);
    }
  }
}

// The logits of a wave's rows (one or four, of at most 1024 in all) in LDS, as
// fp32: value j at j + 4 (j / 16), so that lanes that read neighbouring runs of 16,
// in pieces of four, do not meet in a bank.  Loaded in whole pieces, whatever the
// rows' alignment.
constexpr int kWaveLogits = 1024, kWaveLds = kWaveLogits + kWaveLogits / 4;
__device__ __forceinline__ int lds_at(int j) { return j + 4 * (j >> 4); }
template <int ACT>
__device__ __forceinline__ void stage_logits(const void* logits, int64_t first, int n, float* lds) {
  typedef typename Act<ACT>::bits_t T;
  struct __attribute__((packed, aligned(sizeof(T)))) Four { T v[4]; };
  const T* from = static_cast<const T*>(logits) + first;
#pragma unroll
  for (int i = 0; i < kWaveLogits / 256; ++i) {
    const int j = 256 * i + 4 * (threadIdx.x & 63);
    if (j + 4 <= n) {
      const Four f = *reinterpret_cast<const Four*>(from + j);
      f32x4_t v;
#pragma unroll
      for (int q = 0; q < 4; ++q) v[q] = act_bits_to_float<ACT>(f.v[q]);
      *reinterpret_cast<f32x4_t*>(lds + lds_at(j)) = v;
    } else {
#pragma unroll
      for (int q = 0; q < 4; ++q)
        if (j + q < n) lds[lds_at(j) + q] = act_bits_to_float<ACT>(from[j + q]);
    }
  }
}
// The values first .. first + held - 1 of a row that begins at `row` in such an
// LDS array, `none` behind them; whole: V of them in every lane, from a multiple of
// V on.
template <int V>
__device__ __forceinline__ void read_values(const float* lds, int row, const RouteLane& r, bool whole, float none,
                                            float (&v)[V]) {
  if (whole) {
#pragma unroll
    for (int i = 0; i < V; i += 4) {
      const f32x4_t f = *reinterpret_cast<const f32x4_t*>(lds + lds_at(row + r.first) + i + 4 * (i / 16));
#pragma unroll
      for (int q = 0; q < 4; ++q) v[i + q] = f[q];
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = i < r.held ? lds[lds_at(row + r.first + i)] : none;
  }
}

// The weights of the chosen experts, in 64 bits; logit(e): the row's logits;
// total: softmax's sum of exp(l - top) over all experts, where it is divided by.
// Lane j, j + LANES, .. takes the choices j, ..
template <int LANES, class Logit>
__device__ __forceinline__ void write_weights(const RouteParams& p, int64_t row, int lane, const int* chosen,
                                              bool bad, float top, double total, Logit logit) {
  constexpr int PER = (kRouteMaxTopk + LANES - 1) / LANES;
  double s[PER];
  int expert[PER];
  float lj[PER];
  float best_l = kNegInf;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int j = lane + i * LANES;
    expert[i] = j >= p.topk ? -1 : bad ? j : chosen[j];
    lj[i] = expert[i] >= 0 ? logit(expert[i]) : kNegInf;
    best_l = larger(best_l, lj[i]);
  }
  best_l = row_max<LANES>(best_l);
  // renormalized, a common factor of the scores cancels: they are taken times
  // exp(-best_l) (sigmoid: where they would leave the range), so that none of
  // them vanishes beside the others
  const double shift = best_l == kNegInf || (p.sigmoid && !(p.renormalize && best_l < -600.0f)) ? 0.0
                       : static_cast<double>(p.sigmoid || p.renormalize ? best_l : top);
  double sum = 0.0;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    s[i] = 0.0;
    if (expert[i] >= 0) {
      const double x = lj[i];
      const double e = exp(p.sigmoid && shift == 0.0 ? -fabs(x) : x - shift);
      s[i] = p.sigmoid && shift == 0.0 ? (x > 0.0 ? 1.0 : e) / (1.0 + e) : e;      // (1 + e^x is 1 below -600)
    }
    sum += s[i];
  }
  sum = row_sum<LANES>(sum);
  const double by = static_cast<double>(p.scale) / (p.renormalize ? (sum > 0.0 ? sum : 1.0) : total);
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int j = lane + i * LANES;
    if (j < p.topk) {
      p.experts[row * p.topk + j] = expert[i];
      p.weights[row * p.topk + j] =
          bad ? __builtin_nanf("") : expert[i] < 0 ? 0.0f : static_cast<float>(s[i] * by);
    }
  }
}

// What a wave's lanes wrote to LDS is there for its other lanes.
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

}  // namespace

// Everything in 64 bits: softmax scores that a bias or sums of two choose by, and
// more experts a token than the keys' lanes hold.  Bound by 64-bit exponentials, one
// for each expert, and by choices of 64-bit values (8 of 256, softmax with a bias: 1
// row 6.9 us, 1024 7.7, 8192 17.1; bf16, 8 of 4 of 8 groups by two: 7.8, 8.5, 18.1).
template <int LANES, int V, int ACT>
__global__ __launch_bounds__(kRouteThreads) void moe_route_exact_kernel(RouteParams p) {
  constexpr int ROWS = kRouteThreads / LANES;
  __shared__ int s_chosen[ROWS][kRouteMaxTopk];
  __shared__ __attribute__((aligned(16))) float s_logits[kRouteThreads / 64][kWaveLds], s_bias[kWaveLds];
  const RouteLane r = route_lane<LANES>(p);
  const int64_t row = static_cast<int64_t>(blockIdx.x) * ROWS + threadIdx.x / LANES;
  int* chosen = s_chosen[threadIdx.x / LANES];
  float* logits = s_logits[threadIdx.x / 64];
  {
    const int64_t first = static_cast<int64_t>(blockIdx.x) * ROWS + threadIdx.x / 64 * (64 / LANES);
    const int64_t rows = min(max(p.T - first, int64_t{0}), static_cast<int64_t>(64 / LANES));
    stage_logits<ACT>(p.logits, first * p.E, static_cast<int>(rows) * p.E, logits);
  }
  if (p.bias != nullptr)
    for (int e = threadIdx.x; e < p.E; e += kRouteThreads) s_bias[lds_at(e)] = p.bias[e];
  __syncthreads();
  if (row >= p.T) return;              // (whole sets of 16 lanes, and nothing below meets at a barrier)
  const int row_at = threadIdx.x % 64 / LANES * p.E;
  auto logit = [&](int e) { return logits[lds_at(row_at + e)]; };
  auto bias = [&](int e) { return p.bias != nullptr ? s_bias[lds_at(e)] : 0.0f; };
  const bool valued = p.bias != nullptr || p.group_best == 2;
  double c[V];
  float top = kNegInf;
  bool bad = false;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const float l = i < r.held ? logit(r.first + i) : kNegInf;
    bad |= l != l || (!p.sigmoid && l > 3.402823466e38f);
    top = larger(top, l);
    c[i] = l;
  }
  top = row_max<LANES>(top);
  const double shift = top == kNegInf ? 0.0 : static_cast<double>(top);
  double total = 1.0;                  // softmax: the sum of exp(l - top)
  if (!p.sigmoid && (valued || !p.renormalize)) {
    double sum = 0.0;
#pragma unroll
    for (int i = 0; i < V; ++i) sum += exp(c[i] - shift);
    total = row_sum<LANES>(sum);
  }
  if (valued) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const double b = i < r.held ? static_cast<double>(bias(r.first + i)) : 0.0;
      const double s = p.sigmoid ? sigmoid64(c[i]) : exp(c[i] - shift) / total;
      c[i] = c[i] == static_cast<double>(kNegInf) ? c[i] : s + b;
      bad |= c[i] != c[i];
    }
  }
  bad = row_bits<LANES>(__ballot(bad)) != 0;
  if (p.topk_groups < p.groups) {
    double a = kNegInf, b = kNegInf, gap;
#pragma unroll
    for (int i = 0; i < V; ++i) add_to_two(c[i], &a, &b);
    two_of_group(r, &a, &b);
    const bool stays = group_stays<double, LANES>(p, r, a, b, &gap);
#pragma unroll
    for (int i = 0; i < V; ++i) c[i] = stays ? c[i] : static_cast<double>(kNegInf);
  }
  select_exact<double, LANES, V>(p, r, c, chosen);
  wave_sync();
  write_weights<LANES>(p, row, r.lane, chosen, bad, top, total, logit);
}

// The selection on keys.  VALUED: sigmoid scores with a bias or groups by two;
// otherwise the logits' order.  A block stages its rows' logits in LDS with whole
// loads, each lane takes a run of neighbours from there (V of them, in registers
// throughout), and each choice is V comparisons and one maximum over the row's
// lanes.  Bound by instructions where there are many rows (8192 x 256 fp32,
// sigmoid, bias, 8 experts of 4 of 8 groups: 9.1 us, its 9 MB are 1.8; bf16 logits
// alone 5.2), by a launch and one row's chain of choices where there are few (1 x
// 256, 8 of 256 bf16 3.3 us, with groups 5.4, an empty launch 2.7).  The same with
// 64-bit values throughout took 20 us.  fp32 logits alone, with three candidates
// more than bf16's exact keys: 1 x 256 4.6 us, 8192 x 256 7.2.
template <bool VALUED, int LANES, int V, int ACT>
__global__ __launch_bounds__(kRouteThreads) void moe_route_kernel(RouteParams p) {
  constexpr int ROWS = kRouteThreads / LANES;
  constexpr bool EXACT_KEYS = !VALUED && ACT != ACT_F32;      // 16-bit logits leave at least 13 bits
  constexpr float kOff = 0x1p-20f;     // of a score: sigmoid32's error, doubled
  __shared__ int s_chosen[ROWS][kRouteMaxTopk];
  __shared__ __attribute__((aligned(16))) float s_logits[kRouteThreads / 64][kWaveLds], s_bias[kWaveLds];
  const RouteLane r = route_lane<LANES>(p);
  const int64_t row = static_cast<int64_t>(blockIdx.x) * ROWS + threadIdx.x / LANES;
  int* chosen = s_chosen[threadIdx.x / LANES];
  float* logits = s_logits[threadIdx.x / 64];
  {
    const int64_t first = static_cast<int64_t>(blockIdx.x) * ROWS + threadIdx.x / 64 * (64 / LANES);
    const int64_t rows = min(max(p.T - first, int64_t{0}), static_cast<int64_t>(64 / LANES));
    stage_logits<ACT>(p.logits, first * p.E, static_cast<int>(rows) * p.E, logits);
  }
  if (p.bias != nullptr)
    for (int e = threadIdx.x; e < p.E; e += kRouteThreads) s_bias[lds_at(e)] = p.bias[e];
  __syncthreads();
  if (row >= p.T) return;              // (whole sets of 16 lanes, and nothing below meets at a barrier)
  const int row_at = threadIdx.x % 64 / LANES * p.E;
  auto logit = [&](int e) { return logits[lds_at(row_at + e)]; };
  auto bias = [&](int e) { return p.bias != nullptr ? s_bias[lds_at(e)] : 0.0f; };

  float l[V], b[V], c[V];
  const bool whole = p.E == p.groups * r.group_lanes * V && (LANES >> p.groups_shift) * p.groups == LANES;
  read_values<V>(logits, row_at, r, whole, kNegInf, l);
  if (VALUED && p.bias != nullptr) {
    read_values<V>(s_bias, 0, r, whole, 0.0f, b);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) b[i] = 0.0f;
  }
  float top = kNegInf;
  double total = 1.0;
  bool bad = false;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    if constexpr (VALUED) {
      b[i] = l[i] == kNegInf ? kNegInf : b[i];                // (its score is 0)
      c[i] = sigmoid32(l[i]) + b[i];
      bad |= c[i] != c[i];
    } else {
      c[i] = l[i];
      bad |= l[i] != l[i] || (!p.sigmoid && l[i] > 3.402823466e38f);
      top = larger(top, l[i]);
    }
  }
  if (!VALUED && !p.sigmoid && !p.renormalize) {              // softmax's sum of exp(l - top)
    top = row_max<LANES>(top);
    const float shift = top == kNegInf ? 0.0f : top;
    double sum = 0.0;
#pragma unroll
    for (int i = 0; i < V; ++i) sum += exp_below(l[i], shift);
    total = row_sum<LANES>(sum);
  }
  bad = row_bits<LANES>(__ballot(bad)) != 0;

  auto exact = [&](int i) {            // (VALUED) c[i] in 64 bits
    return l[i] == kNegInf ? static_cast<double>(kNegInf) : sigmoid64(l[i]) + static_cast<double>(b[i]);
  };
  bool stays = true;
  if (p.topk_groups < p.groups) {
    float a = kNegInf, b2 = kNegInf, gap;
#pragma unroll
    for (int i = 0; i < V; ++i) add_to_two(c[i], &a, &b2);
    two_of_group(r, &a, &b2);
    stays = group_stays<float, LANES>(p, r, a, b2, &gap);
    if constexpr (VALUED) {
      // a value is the sum of up to two c, each within kOff + 2^-24 |c| (and 2^-24
      // of itself): where the border is narrower than the errors of two, the
      // groups are told apart in 64 bits, by those c that may be their largest
      // (which are as large as those that seem to be, within the errors)
      const float most = row_max<LANES>(larger(a == kNegInf ? 0.0f : fabsf(a), b2 == kNegInf ? 0.0f : fabsf(b2)));
      if (__ballot(gap <= 4.0f * kOff + 0x1p-20f * most) != 0) {
        const float from = (p.group_best == 2 ? b2 : a) - 2.0f * (kOff + 0x1p-22f * most);
        uint32_t left = 0;
#pragma unroll
        for (int i = 0; i < V; ++i) left |= c[i] != kNegInf && !(c[i] < from) ? 1u << i : 0u;
        double da = kNegInf, db = kNegInf, unused;
        while (__ballot(left != 0) != 0) {
          if (left != 0) {
            const int e = r.first + __builtin_ctz(left);
            add_to_two(sigmoid64(logit(e)) + static_cast<double>(bias(e)), &da, &db);
          }
          left &= left - 1;
        }
        two_of_group(r, &da, &db);
        stays = group_stays<double, LANES>(p, r, da, db, &unused);
      }
    }
  }

  // keys: c's order in the high bits, the lower index first in the low ones; none:
  // 0, or an infinity's, below kNoKey
  constexpr uint32_t kNoKey = 0x00800000u;
  const uint32_t mask = (1u << p.index_bits) - 1, keep = stays ? ~0u : 0u;
  uint32_t key[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const float v = VALUED ? c[i] : c[i] + 0.0f;              // (-0 is 0)
    key[i] = ((ordered(v) & ~mask) | (~static_cast<uint32_t>(r.first + i) & mask)) & keep;
  }
  const int count = EXACT_KEYS ? p.topk : p.topk + 3;         // at most LANES
  // The next one is the largest key below the one before, and so the largest of
  // key - before modulo 2^32: keys that were taken give less than those that were
  // not, as 2^32 is more than any two differ by.  (0, none, comes again for ever:
  // 0 - 1 is above all others.)
  uint32_t mine = 0;                   // the candidate of this lane: the lane-th largest
  uint32_t before = 0;
  for (int j = 0; j < count; ++j) {
    uint32_t m = key[0] - before;
#pragma unroll
    for (int i = 1; i < V; ++i) m = max(m, key[i] - before);
    m = row_max_key<LANES>(m) + before;
    mine = r.lane == j ? m : mine;
    before = max(m, 1u);
  }
  if (mine < kNoKey) mine = 0;
  const int expert = mine == 0 ? -1 : static_cast<int>(mask - (mine & mask));
  if constexpr (EXACT_KEYS) {
    if (r.lane < p.topk) chosen[r.lane] = expert;
  } else {
    // the candidates' exact values and their order (an expert that is none: last)
    typedef typename std::conditional<VALUED, double, float>::type C;
    C v = kNegInf;
    if (expert >= 0) {
      if constexpr (VALUED) v = sigmoid64(logit(expert)) + static_cast<double>(bias(expert));
      else v = logit(expert);
    }
    const bool real = r.lane < count && expert >= 0;
    const C v_before = __shfl_up(v, 1, LANES);
    const int e_before = __shfl_up(expert, 1, LANES);
    const bool wrong = real && r.lane > 0 && !(v_before > v || (v_before == v && e_before < expert));
    int rank = r.lane;
    if (__ballot(wrong) != 0) {
      rank = 0;
      for (int j = 0; j < count; ++j) {
        const C vj = __shfl(v, j, LANES);
        const int ej = __shfl(expert, j, LANES);
        rank += ej >= 0 && (vj > v || (vj == v && ej < expert));
      }
      if (!real) rank = r.lane;        // (behind all that are real)
    }
    if (r.lane < count && rank < p.topk) chosen[rank] = expert;
    // an expert that was left out has a key below the last candidate's: is its
    // value below the k-th's for sure?
    const uint32_t last = __shfl(mine, count - 1, LANES), kth = __shfl(mine, p.topk - 1, LANES);
    const float high = unordered(last | mask), low = unordered(kth & ~mask);
    float off = 0.0f;
    if constexpr (VALUED) off = kOff + 0x1p-22f * larger(fabsf(high), fabsf(low));
    const bool unsure = last != 0 && !(high + off < low - off) && !bad;
    if (__ballot(unsure) != 0) {
      wave_sync();
      C d[V];
#pragma unroll
      for (int i = 0; i < V; ++i) {
        if constexpr (VALUED) d[i] = stays ? exact(i) : static_cast<double>(kNegInf);
        else d[i] = stays ? c[i] : kNegInf;
      }
      select_exact<C, LANES, V>(p, r, d, chosen);
    }
  }
  wave_sync();
  write_weights<LANES>(p, row, r.lane, chosen, bad, top, total, logit);
}

namespace {

template <int KIND, int LANES, int V>
hipError_t launch_route_as(const RouteParams& p, int act, hipStream_t stream) {
  constexpr int ROWS = kRouteThreads / LANES;
  const dim3 grid(static_cast<unsigned>((p.T + ROWS - 1) / ROWS)), block(kRouteThreads);
  if constexpr (KIND == 2) {
    switch (act) {
      case ACT_F32: moe_route_exact_kernel<LANES, V, ACT_F32><<<grid, block, 0, stream>>>(p); break;
      case ACT_F16: moe_route_exact_kernel<LANES, V, ACT_F16><<<grid, block, 0, stream>>>(p); break;
      default: moe_route_exact_kernel<LANES, V, ACT_BF16><<<grid, block, 0, stream>>>(p); break;
    }
  } else {
    switch (act) {
      case ACT_F32: moe_route_kernel<KIND == 1, LANES, V, ACT_F32><<<grid, block, 0, stream>>>(p); break;
      case ACT_F16: moe_route_kernel<KIND == 1, LANES, V, ACT_F16><<<grid, block, 0, stream>>>(p); break;
      default: moe_route_kernel<KIND == 1, LANES, V, ACT_BF16><<<grid, block, 0, stream>>>(p); break;
    }
  }
  return hipGetLastError();
}
// 16 lanes a row where its values and its candidates fit them and there are rows
// enough, else 64 (us, 64 / 16 lanes, 256 experts: sigmoid, bias and groups by
// two, 1 row 5.4 / 6.5, 2048 rows 7.6 / 8.0, 4096 9.6 / 7.6; bf16 logits alone, 1
// row 3.3 / 4.0, 1024 3.8 / 4.4, 4096 5.4 / 4.5).  Rows of at most four values a
// lane have 16 lanes at any number of them: 64 experts, 8 chosen, bf16 logits alone,
// 1 row 3.9 / 4.1, 64 4.3 / 4.1, 2048 4.9 / 4.2, 8192 9.1 / 4.5; with sigmoid, bias and 4
// groups 5.7 / 5.7, 6.3 / 5.6, 7.1 / 6.3, 14.8 / 7.2.
template <int KIND>
hipError_t launch_route_of(const RouteParams& p, int candidates, int act, hipStream_t stream) {
  const int per_group = p.E / p.groups;
  auto held = [&](int lanes) {
    const int g = lanes >> p.groups_shift;
    return g == 0 || candidates > lanes ? kRouteMaxExperts : (per_group + g - 1) / g;
  };
  if (held(16) <= 4) return launch_route_as<KIND, 16, 4>(p, act, stream);
  if (p.T > 2048) {
    if (held(16) <= 8) return launch_route_as<KIND, 16, 8>(p, act, stream);
    if (held(16) <= 16) return launch_route_as<KIND, 16, 16>(p, act, stream);
  }
  if (held(64) <= 4) return launch_route_as<KIND, 64, 4>(p, act, stream);
  if (held(64) <= 8) return launch_route_as<KIND, 64, 8>(p, act, stream);
  if (held(64) <= 16) return launch_route_as<KIND, 64, 16>(p, act, stream);
  return launch_route_as<KIND, 64, 32>(p, act, stream);
}

}  // namespace

hipError_t launch_moe_route(const RouteParams& p, int act, hipStream_t stream) {
  const bool valued = p.bias != nullptr || p.group_best == 2;      // (as the exact kernel has it)
  const bool exact_keys = !valued && act != ACT_F32;
  const int candidates = exact_keys ? p.topk : p.topk + 3;
  if ((valued && !p.sigmoid) || candidates > 64) return launch_route_of<2>(p, 0, act, stream);
  return valued ? launch_route_of<1>(p, candidates, act, stream) : launch_route_of<0>(p, candidates, act, stream);
}

}  // namespace lowbit
