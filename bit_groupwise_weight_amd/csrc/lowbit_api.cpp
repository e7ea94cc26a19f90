// Host side of the C ABI declared in include/lowbit.h: argument validation,
// schedule selection and kernel dispatch.  Validation never touches the HIP
// runtime, so every argument error is reported identically with or without a
// GPU present.
#include "lowbit.h"
#include "lowbit_tuning.h"

#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <algorithm>
#include <atomic>
#include <limits>
#include <mutex>
#include <string>
#include <utility>

#include "kernels.h"

namespace {

thread_local std::string g_last_error;

lowbit_status fail(lowbit_status st, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
lowbit_status fail(lowbit_status st, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  g_last_error = buf;
  return st;
}

lowbit_status hip_fail(hipError_t e, const char* what) {
  return fail(LOWBIT_ERR_HIP, "%s: %s", what, hipGetErrorString(e));
}

bool valid_bits(int bits) { return bits >= 1 && bits <= 7; }
bool valid_group(int g) { return g == 32 || g == 64 || g == 128 || g == 256; }
bool valid_dtype(lowbit_dtype d) { return d == LOWBIT_F32 || d == LOWBIT_F16 || d == LOWBIT_BF16; }
size_t dtype_bytes(lowbit_dtype d) { return d == LOWBIT_F32 ? 4 : 2; }
bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// Shapes are limited so that every element index fits the kernels' 32-bit
// row/column counters and 64-bit offsets.
constexpr int64_t kMaxDim = int64_t(1) << 30;

lowbit_status check_common(int bits, int group, int64_t N, int64_t K) {
  if (!valid_bits(bits)) return fail(LOWBIT_ERR_INVALID_ARG, "bits=%d not in 1..7", bits);
  if (!valid_group(group))
    return fail(LOWBIT_ERR_INVALID_ARG, "group=%d not one of 32/64/128/256", group);
  if (N <= 0 || K <= 0 || N > kMaxDim || K > kMaxDim)
    return fail(LOWBIT_ERR_INVALID_ARG, "N=%lld K=%lld must be in 1..2^30", (long long)N,
                (long long)K);
  if (K % group != 0)
    return fail(LOWBIT_ERR_INVALID_ARG, "K=%lld is not a multiple of group=%d", (long long)K,
                group);
  return LOWBIT_OK;
}

// Arguments of one linear (shared by lowbit_linear_path and lowbit_linear_multi).
lowbit_status check_linear(const void* x, lowbit_dtype act_dtype, const uint8_t* packed,
                           const void* scales, const void* zeros, const void* bias, const void* y,
                           int bits, int group, int64_t M, int64_t N, int64_t K) {
  lowbit_status st = check_common(bits, group, N, K);
  if (st != LOWBIT_OK) return st;
  if (M < 0 || M > kMaxDim) return fail(LOWBIT_ERR_INVALID_ARG, "M=%lld", (long long)M);
  if (!valid_dtype(act_dtype)) return fail(LOWBIT_ERR_UNSUPPORTED, "act_dtype=%d", (int)act_dtype);
  if (!packed || !scales || !zeros) return fail(LOWBIT_ERR_INVALID_ARG, "NULL weight pointer");
  if (M > 0 && (!x || !y)) return fail(LOWBIT_ERR_INVALID_ARG, "NULL x or y");
  if (!aligned(packed, 16)) return fail(LOWBIT_ERR_MISALIGNED, "packed must be 16-byte aligned");
  if (!aligned(x, 16)) return fail(LOWBIT_ERR_MISALIGNED, "x must be 16-byte aligned");
  const size_t e = dtype_bytes(act_dtype);
  if (!aligned(scales, e) || !aligned(zeros, e) || !aligned(y, e) || (bias && !aligned(bias, e)))
    return fail(LOWBIT_ERR_MISALIGNED, "scales/zeros/bias/y must be aligned to their element size");
  return LOWBIT_OK;
}

// The quantizer's status words live in a device array that the library holds
// on every device (no allocation).  A call holds its device's mutex from
// clearing the words until it has read them back, so concurrent calls on one
// device (from any threads, on any streams) never see each other's flags.
constexpr int kMaxDevices = 64;
std::mutex g_status_mu[kMaxDevices];

// Current device's status words; on success *lock holds that device's mutex.
lowbit_status device_status_word(int** out, std::unique_lock<std::mutex>* lock) {
  int dev = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return hip_fail(e, "hipGetDevice");
  if (dev < 0 || dev >= kMaxDevices) return fail(LOWBIT_ERR_HIP, "device id %d out of range", dev);
  std::unique_lock<std::mutex> held(g_status_mu[dev]);
  e = lowbit::quant_status_words(out);
  if (e != hipSuccess) return hip_fail(e, "hipGetSymbolAddress(status)");
  *lock = std::move(held);
  return LOWBIT_OK;
}

int act_kind(lowbit_dtype d) {
  switch (d) {
    case LOWBIT_F32: return lowbit::ACT_F32;
    case LOWBIT_F16: return lowbit::ACT_F16;
    default: return lowbit::ACT_BF16;
  }
}

typedef hipError_t (*QmvLauncher)(const lowbit::QmvBatch&, const lowbit::QmvLaunch&, int, int,
                                  hipStream_t);
const QmvLauncher kQmv[8] = {nullptr,
                             lowbit::launch_qmv_b1,
                             lowbit::launch_qmv_b2,
                             lowbit::launch_qmv_b3,
                             lowbit::launch_qmv_b4,
                             lowbit::launch_qmv_b5,
                             lowbit::launch_qmv_b6,
                             lowbit::launch_qmv_b7};

// Largest M that the automatic choice sends to the decode kernel: measured
// on MI355X at K = N = 4096, group 64, fp16 and bf16, b = 1..5 and 7 (both
// paths forced, graph-timed on one box) -- the decode kernel is faster up to
// M = 4 at every width (e.g. b = 4, fp16, M = 4: 7.7 vs 10.6 us) and the MFMA
// kernel from M = 5 (b = 4: 10.5 vs 11.2 us; b = 7: 12.7 vs 15.8 us): the
// decode kernel serves four activation rows per pass and re-reads the
// weights for the next four.
// Largest M the decode kernel takes by default: fp32 activations always go
// to it; fp16 from M = 3 and bf16 from M = 5 go to the MFMA kernels (the
// small-M kernel for fp16 up to 16 rows; measured at K = N = 4096, decode /
// small-M kernel, us: M = 2 5.1-6.8 / 5.4-7.6, M = 4 7.3-9.9 / 5.5-7.4,
// M = 8 10.8-16.4 / 6.6-8.2).
inline int64_t qmv_max_m(lowbit_dtype act) { return act == LOWBIT_F16 ? 2 : 4; }
static_assert(LOWBIT_MAX_MULTI <= lowbit::kQmvMaxProblems, "one launch serves every desc");

typedef int (*QmvStageBytes)(int);
const QmvStageBytes kQmvStage[8] = {nullptr,
                                    lowbit::qmv_stage_bytes_b1,
                                    lowbit::qmv_stage_bytes_b2,
                                    lowbit::qmv_stage_bytes_b3,
                                    lowbit::qmv_stage_bytes_b4,
                                    lowbit::qmv_stage_bytes_b5,
                                    lowbit::qmv_stage_bytes_b6,
                                    lowbit::qmv_stage_bytes_b7};

// LDS budget of one decode block for its staged activations.
constexpr int64_t kQmvStageBudget = 64 * 1024 - 256;

// Overrides of the automatic schedule choices (lowbit_set_tuning; 0 = none),
// for tests and benchmarks.  Nothing reads the environment.
std::atomic<int> g_tuning[LOWBIT_TUNE_COUNT] = {};

int tuning(lowbit_tuning_key key, int dflt) {
  const int v = g_tuning[key].load(std::memory_order_relaxed);
  return v != 0 ? v : dflt;
}

// Compute units of the current device (cached per device; 256 if unknown).
int device_cus() {
  static std::atomic<int> cached[kMaxDevices] = {};
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= kMaxDevices) return 256;
  int v = cached[dev].load(std::memory_order_relaxed);
  if (v > 0) return v;
  int cus = 0;
  if (hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || cus <= 0)
    cus = 256;
  cached[dev].store(cus, std::memory_order_relaxed);
  return cus;
}

// One decode problem of a (possibly multi-problem) launch.
struct QmvProblem {
  const void* x;
  const uint8_t* packed;
  const void* scales;
  const void* zeros;
  const void* bias;
  void* y;
  int64_t N, K;
};

// All problems share bits, group, activation dtype and M; one launch serves
// them all (blocks are dealt out to the problems in order).
lowbit_status run_qmv_multi(const QmvProblem* probs, int count, lowbit_dtype act, int bits, int group,
                            int64_t M, hipStream_t stream) {
  lowbit::QmvBatch b{};
  int max_shift = 0;
  int64_t max_per_row = 0;
  for (int i = 0; i < count; ++i) {
    const QmvProblem& q = probs[i];
    lowbit::QmvParams& p = b.prob[i];
    p.x = q.x; p.packed = q.packed; p.scales = q.scales; p.zeros = q.zeros; p.bias = q.bias; p.y = q.y;
    p.M = static_cast<int>(M);
    p.N = static_cast<int>(q.N);
    p.K = static_cast<int>(q.K);
    p.groups = static_cast<int>(q.K / group);
    p.row_bytes = q.K * bits / 8;
    // lanes per row group: enough for four 32-code runs each, at most 64
    const int64_t units = (q.K + 127) / 128;
    int shift = 0;
    while ((int64_t(1) << shift) < units && shift < 6) ++shift;
    p.lpr_shift = shift;
    max_shift = std::max(max_shift, shift);
    max_per_row = std::max<int64_t>(max_per_row,
                                    static_cast<int64_t>(kQmvStage[bits](act_kind(act))) << shift);
  }

  // Activation rows per pass: as many as fit the LDS stage (at most 4).
  // max_per_row holds 4 * quads-per-run * 16 bytes per lane, times the lanes.
  auto stage_bytes = [&](int mt) {
    const int64_t qd = (max_per_row >> max_shift) / (4 * 16);
    return static_cast<int64_t>(lowbit::qmv_stage_quads_per_lane(mt, static_cast<int>(qd))) * 16
           << max_shift;
  };
  lowbit::QmvLaunch l{};
  l.mt = 1;
  if (M >= 2 && stage_bytes(2) <= kQmvStageBudget) l.mt = 2;
  if (M >= 3 && stage_bytes(4) <= kQmvStageBudget) l.mt = 4;
  if (stage_bytes(1) > kQmvStageBudget) return fail(LOWBIT_ERR_UNSUPPORTED, "activation stage too large");
  // Block size: 256 threads unless that leaves fewer blocks than CUs.
  int threads = tuning(LOWBIT_TUNE_QMV_BLOCK, 0);
  auto blocks_for = [&](int t, int i, int variant) {
    const int64_t rows_per_block =
        static_cast<int64_t>(t >> b.prob[i].lpr_shift) * lowbit::qmv_rows_per_group(bits, l.mt, variant);
    return (probs[i].N + rows_per_block - 1) / rows_per_block;
  };
  auto total_blocks = [&](int t, int variant) {
    int64_t n = 0;
    for (int i = 0; i < count; ++i) n += blocks_for(t, i, variant);
    return n;
  };
  if (threads != 64 && threads != 128 && threads != 256) {
    threads = 256;
    while (threads > 64 && total_blocks(threads, lowbit::QMV_DEFAULT) < device_cus() &&
           (threads >> 1) >= (1 << max_shift))
      threads >>= 1;
  }
  if (threads < (1 << max_shift)) threads = 1 << max_shift;
  const int64_t by = (M + l.mt - 1) / l.mt;
  // One activation row: with more than two blocks per CU the lean variant
  // (one more wave per SIMD) gains 7-9 % at b = 4 from 4096 x 14336 to
  // 16384 x 16384 and 12 % at b = 1, 4096 x 14336 (3.5 blocks per CU), and
  // where two rows per lane group still leave six or more blocks per CU,
  // LEAN2 gains another ~10 % (4096 x 28672, 16384 x 16384; at 3.5-4 blocks
  // per CU it loses 0-3 %).  With two blocks per CU or fewer the default is
  // ahead by 0-3 % (K = N = 4096).
  // Rows of more than one round per lane (K > 128 * lanes, e.g. K = 14336)
  // also take the lean variant: b = 1/4/7 at K = 14336, N = 4096 run 3/9/11 %
  // faster with it at two to four blocks per CU.
  const int64_t cus = device_cus();
  bool multi_round = false;
  for (int i = 0; i < count; ++i)
    multi_round |= probs[i].K > (int64_t{128} << b.prob[i].lpr_shift);
  // Otherwise (one round, at most two blocks per CU), widths with two rows
  // per lane group take one row per lane group, which doubles the waves,
  // unless that leaves the CUs between two and four waves each.  A/B on one
  // box, us: K = 4096, N = 1024, b = 1, 2, 3: 3.81/3.96/4.09 -> 3.59/3.67/3.77
  // and K = 2048, N = 1024, b = 1, 3: 3.12/3.47 -> 2.71/3.10 (one wave per CU
  // before); K = N = 4096, b = 1, 3: 3.74/4.31 -> 3.67/4.22 and K = 4096,
  // N = 8192, b = 2, 3: 5.07/5.77 -> 4.92/5.37 (four and eight waves per CU
  // before); K = 4096, N = 2048 (two waves per CU before) loses 3 %.
  l.variant = lowbit::QMV_DEFAULT;
  const int64_t waves = total_blocks(threads, lowbit::QMV_DEFAULT) * by * (threads / 64);
  if (l.mt == 1 && (total_blocks(threads, lowbit::QMV_DEFAULT) * by > 2 * cus || multi_round))
    l.variant = total_blocks(threads, lowbit::QMV_LEAN2) * by >= 6 * cus ? lowbit::QMV_LEAN2 : lowbit::QMV_LEAN;
  else if (l.mt == 1 && (waves < 2 * cus || waves >= 4 * cus) &&
           lowbit::qmv_rows_per_group(bits, 1, lowbit::QMV_DEFAULT) == 2)
    l.variant = lowbit::QMV_LEAN1;
  const int var_env = tuning(LOWBIT_TUNE_QMV_VARIANT, 0) - 1;   // (override: 1..4 forces variant 0..3)
  if (l.mt == 1 && var_env >= 0 && var_env <= 3) l.variant = var_env;
  int64_t bx = 0;
  for (int i = 0; i < count; ++i) bx = std::max<int64_t>(bx, blocks_for(threads, i, l.variant));
  if (bx > 0x7fffffff || by > 65535) return fail(LOWBIT_ERR_INVALID_ARG, "problem too large");
  l.grid = dim3(static_cast<unsigned>(bx), static_cast<unsigned>(by), static_cast<unsigned>(count));
  l.block = dim3(threads);
  hipError_t e = kQmv[bits](b, l, group, act_kind(act), stream);
  if (e != hipSuccess) return hip_fail(e, "qmv launch");
  return LOWBIT_OK;
}

lowbit_status run_qmv(const void* x, lowbit_dtype act, const uint8_t* packed, const void* scales,
                      const void* zeros, const void* bias, void* y, int bits, int group,
                      int64_t M, int64_t N, int64_t K, hipStream_t stream) {
  const QmvProblem q{x, packed, scales, zeros, bias, y, N, K};
  return run_qmv_multi(&q, 1, act, bits, group, M, stream);
}

typedef hipError_t (*QmmLauncher)(const lowbit::QmmParams&, const lowbit::QmmLaunch&, int,
                                  hipStream_t);
const QmmLauncher kQmm[8] = {nullptr,
                             lowbit::launch_qmm_b1,
                             lowbit::launch_qmm_b2,
                             lowbit::launch_qmm_b3,
                             lowbit::launch_qmm_b4,
                             lowbit::launch_qmm_b5,
                             lowbit::launch_qmm_b6,
                             lowbit::launch_qmm_b7};

typedef hipError_t (*QmmSmallLauncher)(const lowbit::QmmParams&, int, int, hipStream_t);
const QmmSmallLauncher kQmmSmall[8] = {nullptr,
                                       lowbit::launch_qmm_small_b1,
                                       lowbit::launch_qmm_small_b2,
                                       lowbit::launch_qmm_small_b3,
                                       lowbit::launch_qmm_small_b4,
                                       lowbit::launch_qmm_small_b5,
                                       lowbit::launch_qmm_small_b6,
                                       lowbit::launch_qmm_small_b7};

// Schedule of the MFMA kernel: block tile (16*mtt) x (16*nt*waves), K steps
// of 128, and a K split that fills the CUs with one block each.
struct QmmSchedule {
  bool small;             // the small-M kernel (fields below: nt, waves only)
  int mtt, nt, waves, kgroups, rgroups;
  int64_t tiles_n, tiles_m, ksteps;
  int splits, ksteps_per_split;
  size_t partial_bytes;   // fp32 partial planes (split-K)
};

// Block tiles and K split for column tile width 16*nt*waves: one block per
// CU (each block takes a whole CU's register file), K split just enough that
// the tiles times the splits fill the CUs without a second, partial wave of
// blocks (LOWBIT_TUNE_QMM_BLOCKS overrides the block target).
void qmm_split(QmmSchedule& sc, int64_t M, int64_t N, int64_t K) {
  const int64_t bn = 16 * sc.nt * sc.waves;
  sc.tiles_n = (N + bn - 1) / bn;
  sc.tiles_m = (M + 16 * sc.mtt - 1) / (16 * sc.mtt);
  sc.ksteps = (K + 127) / 128;
  const int64_t target = tuning(LOWBIT_TUNE_QMM_BLOCKS, device_cus());
  const int64_t tiles = sc.tiles_n * sc.tiles_m;
  int64_t s = std::max<int64_t>(1, target / tiles);
  const int64_t max_split = std::max<int64_t>(1, sc.ksteps / 2);   // >= 2 steps per split
  s = std::max<int64_t>(1, std::min<int64_t>(s, std::min<int64_t>(max_split, 64)));
  sc.ksteps_per_split = static_cast<int>((sc.ksteps + s - 1) / s);
  // with two K groups, an even step count per split keeps the groups equal
  if (sc.kgroups == 2 && sc.ksteps_per_split % 2 == 1 && sc.ksteps_per_split < sc.ksteps)
    ++sc.ksteps_per_split;
  sc.splits = static_cast<int>((sc.ksteps + sc.ksteps_per_split - 1) / sc.ksteps_per_split);
  // partial planes cover whole block tiles (the reduce kernel skips the
  // records past M or N)
  sc.partial_bytes = 0;
  if (sc.splits > 1)
    sc.partial_bytes = static_cast<size_t>(sc.splits) * static_cast<size_t>(sc.tiles_n * bn) *
                       static_cast<size_t>(sc.tiles_m * 16 * sc.mtt) * sizeof(float);
}

// Steps per block at or below which 64-column blocks (one column tile per
// wave) beat 128-column ones at M = 128: the narrower tile halves the K split
// (no reduce kernel at all for N = 14336 with K <= 4096) at the price of
// twice the LDS reads per MFMA, which only pays while the loop is short
// (measured, N = 14336: K = 1024 13.1 vs 21.2 us, K = 2048 20.1 vs 24.7,
// K = 4096 even, K = 8192 62.7 vs 55.7; N = 4096: K = 7168 22.7 vs 24.4,
// K = 14336 36.0 vs 33.3).
constexpr int kQmmNarrowMaxSteps = 16;

// Two K groups need enough steps per block for their two-step pipeline:
// measured (A/B in alternating processes on one box) K groups win with 14-16
// steps per block (M = 128, K = 14336, N = 4096: 34.2 vs 35.0 us; M = 64,
// K = 4096, N = 14336: 30.8 vs 33.1; M = 32: 27.1 vs 28.4) and lose with 4
// (M = 64, K = N = 4096: 17.25 vs 16.8).
constexpr int kQmmKGroupsMinSteps = 8;

// Largest M of the small-M kernel (fp16 activations): it streams the weights
// once per call whatever M is, while the tiled kernel pays a K split, its
// reduce and a pipeline fill.
constexpr int kQmmSmallMaxM = 16;

QmmSchedule qmm_schedule(int bits, lowbit_dtype act, int64_t M, int64_t N, int64_t K) {
  QmmSchedule sc{};
  sc.rgroups = 1;
  const int small_env = tuning(LOWBIT_TUNE_QMM_SMALL_M, kQmmSmallMaxM);
  if (act == LOWBIT_F16 && M <= std::min(small_env, 16)) {
    // blocks of 16 columns (32 when asked) over all of K; waves per block so
    // that each takes at least two K steps
    const int64_t ksteps = (K + 127) / 128;
    sc.small = true;
    sc.nt = tuning(LOWBIT_TUNE_QMM_NT, 1) == 2 ? 2 : 1;
    sc.waves = ksteps >= 32 ? 16 : ksteps >= 16 ? 8 : 4;
    const int wv_env = tuning(LOWBIT_TUNE_QMM_WAVES, 0);
    if (wv_env == 4 || wv_env == 8 || wv_env == 16) sc.waves = wv_env;
    if (sc.nt == 2 && sc.waves == 16) sc.waves = 8;
    sc.mtt = 1;
    sc.kgroups = 1;
    sc.tiles_n = (N + 16 * sc.nt - 1) / (16 * sc.nt);
    sc.tiles_m = 1;
    sc.ksteps = ksteps;
    sc.splits = 1;
    sc.ksteps_per_split = static_cast<int>(ksteps);
    sc.partial_bytes = 0;
    return sc;
  }
  sc.mtt = M <= 16 ? 1 : M <= 32 ? 2 : M <= 64 ? 4 : 8;
  const int mtt_env = tuning(LOWBIT_TUNE_QMM_MTT, 0);
  if (mtt_env == 1 || mtt_env == 2 || mtt_env == 4 || mtt_env == 8) sc.mtt = std::min(sc.mtt, mtt_env);
  sc.nt = 2;
  if (act == LOWBIT_BF16) {
    // bf16: the code-operand kernel, 4 column waves of two column tiles;
    // 128-row tiles split between two row groups of 4 waves (two waves per
    // SIMD; 64-row tiles only when asked)
    sc.waves = 4;
    sc.kgroups = 1;
    const int rg_env = tuning(LOWBIT_TUNE_QMM_RGROUPS, 0);
    sc.rgroups = ((sc.mtt == 8 && rg_env != 1) || (sc.mtt == 4 && rg_env == 2)) ? 2 : 1;
    if (tuning(LOWBIT_TUNE_QMM_NT, 0) == 1) {
      sc.nt = 1;
      sc.rgroups = 1;
    }
    qmm_split(sc, M, N, K);
    return sc;
  }
  // Two K groups of 4 column waves (8 waves, 128 columns) keep two waves per
  // SIMD at the tile width of a 4-wave block, so the K split across blocks
  // stays that of the 4-wave block: one wave's dequantization runs under the
  // other's MFMAs.  Up to 4 bits, with at least kQmmKGroupsMinSteps steps per
  // block; 128-row tiles may narrow to one column tile per wave (below).
  // Otherwise one K group: 8 column waves (256 columns) for full 128-row
  // tiles when N is wide enough that the K split stays small (1.6x more work
  // per CU than 4-wave blocks at M = 128, K = 4096, N = 14336; the wider tile
  // needs twice the K splits, whose partial planes cost more than that gain
  // once the split exceeds ~4), else 4 waves.
  // (LOWBIT_TUNE_QMM_MTT, _KGROUPS, _WAVES and _NT override the choices;
  // _WAVES applies with one K group, _NT with two at 128-row tiles.)
  const bool can8 = bits <= lowbit::qmm_max_bits_8waves;
  const bool can_kg = bits <= lowbit::qmm_max_bits_kgroups;
  const int kg_env = tuning(LOWBIT_TUNE_QMM_KGROUPS, 0);
  if (can_kg && kg_env != 1) {
    QmmSchedule kg = sc;
    kg.kgroups = 2;
    kg.waves = 4;
    if (kg.mtt == 8) {
      QmmSchedule narrow = kg;
      narrow.nt = 1;
      qmm_split(narrow, M, N, K);
      const int nt_env = tuning(LOWBIT_TUNE_QMM_NT, 0);
      if (nt_env == 1 || (nt_env != 2 && narrow.ksteps_per_split <= kQmmNarrowMaxSteps)) return narrow;
    }
    qmm_split(kg, M, N, K);
    if (kg_env == 2 || kg.ksteps_per_split >= kQmmKGroupsMinSteps) return kg;
  }
  sc.kgroups = 1;
  const int wv_default = (can8 && sc.mtt == 8 && (N + 255) / 256 >= device_cus() / 5) ? 8 : 4;
  sc.waves = (can8 && tuning(LOWBIT_TUNE_QMM_WAVES, wv_default) == 8) ? 8 : 4;
  qmm_split(sc, M, N, K);
  return sc;
}

lowbit_status run_qmm(const void* x, lowbit_dtype act, const uint8_t* packed, const void* scales,
                      const void* zeros, const void* bias, void* y, int bits, int group,
                      int64_t M, int64_t N, int64_t K, void* workspace, size_t workspace_bytes,
                      hipStream_t stream) {
  QmmSchedule sc = qmm_schedule(bits, act, M, N, K);
  if (sc.splits > 1 && (workspace == nullptr || workspace_bytes < sc.partial_bytes)) {
    sc.splits = 1;                               // no workspace: one block per tile over all K
    sc.ksteps_per_split = static_cast<int>(sc.ksteps);
  }
  if (sc.tiles_m > 65535 || sc.tiles_n > 0x7fffffff)
    return fail(LOWBIT_ERR_INVALID_ARG, "problem too large for qmm");
  // the bf16 kernel addresses activations and packed codes with 32-bit
  // lane offsets from a per-step base
  if (act == LOWBIT_BF16 && (M * K * 2 > int64_t{0xffffffff} || N * (K * bits / 8) > int64_t{0xffffffff}))
    return fail(LOWBIT_ERR_UNSUPPORTED, "bf16 qmm: activations and packed codes must each be below 4 GiB");
  if (sc.small) {
    lowbit::QmmParams p{};
    p.x = x; p.packed = packed; p.scales = scales; p.zeros = zeros; p.bias = bias; p.y = y;
    p.M = static_cast<int>(M);
    p.N = static_cast<int>(N);
    p.K = static_cast<int>(K);
    p.groups = static_cast<int>(K / group);
    int gs = 0;
    while ((1 << gs) < group) ++gs;
    p.group_shift = gs;
    p.row_bytes = K * bits / 8;
    p.ksteps_per_split = static_cast<int>(sc.ksteps);
    const hipError_t e = kQmmSmall[bits](p, sc.nt, sc.waves, stream);
    if (e != hipSuccess) return hip_fail(e, "small-M qmm launch");
    return LOWBIT_OK;
  }
  lowbit::QmmParams p{};
  p.x = x; p.packed = packed; p.scales = scales; p.zeros = zeros; p.bias = bias; p.y = y;
  p.M = static_cast<int>(M);
  p.N = static_cast<int>(N);
  p.K = static_cast<int>(K);
  p.groups = static_cast<int>(K / group);
  int gs = 0;
  while ((1 << gs) < group) ++gs;
  p.group_shift = gs;
  p.row_bytes = K * bits / 8;
  p.ksteps_per_split = sc.ksteps_per_split;
  if (sc.splits > 1) p.partials = static_cast<float*>(workspace);
  lowbit::QmmLaunch l{};
  l.mtt = sc.mtt;
  l.nt = sc.nt;
  l.waves = sc.waves;
  l.kgroups = sc.kgroups;
  l.rgroups = sc.rgroups;
  l.grid = dim3(static_cast<unsigned>(sc.tiles_n), static_cast<unsigned>(sc.tiles_m),
                static_cast<unsigned>(sc.splits));
  hipError_t e = kQmm[bits](p, l, act_kind(act), stream);
  if (e != hipSuccess) return hip_fail(e, "qmm launch");
  return LOWBIT_OK;
}

typedef hipError_t (*A8Launcher)(const lowbit::A8Params&, int, int, int, hipStream_t);
const A8Launcher kA8[8] = {nullptr,
                           lowbit::launch_qmm_a8_b1,
                           lowbit::launch_qmm_a8_b2,
                           lowbit::launch_qmm_a8_b3,
                           lowbit::launch_qmm_a8_b4,
                           lowbit::launch_qmm_a8_b5,
                           lowbit::launch_qmm_a8_b6,
                           lowbit::launch_qmm_a8_b7};

// Largest M of the int8-activation linear: 65535 blocks (the grid's y
// limit) of 16 rows.
constexpr int64_t kA8MaxM = int64_t(16) * 65535;

// Tiles of the int8-activation linear: 16-row tiles per block (mtt) and
// 16-column tiles per wave (nt).  The kernel is bound by its vector-memory
// instructions.  The block's waves share the activation fragments through
// LDS, so per 16 x 16 output tile and 64-wide K window a wave issues about
// 1/(4 nt) activation loads, 1/mtt code loads and 1/4 scale/zero loads: the
// row tiles matter most, and the largest tiles win as long as the launch
// keeps at least 3.5 waves per CU (measured at M = 128, bits 4, group 32:
// K = 4096, N = 14336 runs fastest with mtt 4, nt 1 at 7 waves per CU,
// 58 us, against 67 us for mtt 4, nt 2 at 3.5; K = 14336, N = 4096 with
// mtt 2, nt 1 at 4 waves per CU, 82 us, against 134-222 us for larger tiles
// at 2 waves per CU).
constexpr int kA8HalfWavesPerCu = 7;
void a8_tiles(int64_t M, int64_t N, int* mtt_out, int* nt_out) {
  static const int kOrder[][2] = {{4, 1}, {2, 1}, {4, 2}, {2, 2}, {1, 1}, {1, 2}};
  const int64_t target = (int64_t(kA8HalfWavesPerCu) * device_cus() + 1) / 2;
  int mtt = 1, nt = 1;
  for (const auto& c : kOrder) {
    if (c[0] > 1 && 16 * (c[0] / 2) >= M) continue;   // the rows fit in half the tiles
    const int64_t waves = ((N + 16 * c[1] - 1) / (16 * c[1])) * ((M + 16 * c[0] - 1) / (16 * c[0]));
    if (waves >= target) {
      mtt = c[0];
      nt = c[1];
      break;
    }
  }
  const int fm = tuning(LOWBIT_TUNE_A8_MTT, 0), fn = tuning(LOWBIT_TUNE_A8_NT, 0);
  if (fm == 1 || fm == 2 || fm == 4) mtt = fm;
  if (fn == 1 || fn == 2) nt = fn;
  *mtt_out = mtt;
  *nt_out = nt;
}

// Limits of the 8-bit path: row lengths whose block counts and lane offsets
// fit 32 bits, and launches of fewer than 2^32 threads (checked per call).
constexpr int64_t kQ8MaxK = int64_t(1) << 23;
constexpr int64_t kNormMaxM = (int64_t(1) << 22) - 1;
constexpr int64_t kActF8MaxBlocks = (int64_t(1) << 28) - 16;   // of 16 threads each
constexpr int64_t kF8MaxExperts = int64_t(1) << 16;
int64_t f8_blocks(int64_t n) { return (n + 127) / 128; }

lowbit_status check_q8_row(int64_t K, int unit) {
  if (K <= 0 || K > kQ8MaxK || K % unit != 0)
    return fail(LOWBIT_ERR_INVALID_ARG, "K=%lld must be a positive multiple of %d (at most 2^23)",
                (long long)K, unit);
  return LOWBIT_OK;
}

// Variant and K split of a block-scaled e4m3 product: T rows of y, E experts
// (0: dense), rows of xq gathered from M.  Times: us on MI355X, bf16 outputs,
// the variants forced in turn on one card (M, N, K; "64 x 8 of 64" is 64 tokens
// to 8 of 64 experts each).
//
// Up to 16 rows (10 an expert on average: grouped rows are uneven, and a second
// tile of 16 costs more than one of 32; 13 an expert: 44 against 42 of 64 x 32)
// the weights are streamed past them.  Wider blocks load the activations once
// for more weights, narrower ones are more:
// - 64 columns from 7/4 of a block a CU on (64 x 8 of 64, 1408, 2048: 39 against
//   48 of 32 columns; 16, 28672, 4096: 27 against 30);
// - 32 columns from 7/8 on (8, 8192, 2048: 5.7 against 6.3 of 16; 8, 4096, 4096,
//   half a block: 8.1 against 6.7);
// - 64 x 32 tiles, whose loads are further ahead, where they are 2/3 of a block
//   to one a CU (16, 14336, 4096: 11.5 against 13.3; 1 x 8 of 64, 1408, 2048: 8.0
//   against 8.5; 8, 4096, 4096, 1/4 of a block: 8.8 against 6.7; 8, 14336, 12288:
//   34.9 against 37.9 of 64 columns), but not where the rows they read side by
//   side lie a multiple of 8 KiB apart: there 64 columns, whose waves read
//   different parts of K (8, 14336: K = 8064 23.3 against 24.6, K = 8192 29.5
//   against 24.4, K = 8320 24.0 against 25.6; 16, 16384, 8192: 34.6 against 26.5;
//   8, 11264, 8192: 23.4 against 23.3; 8, 14336, 16384: 55.0 against 57.2; 1 x 8 of
//   64, 2048, 8192: 28.8 against 26.8, with 1536 columns 24.4 against 26.7);
// - 16 columns read more activations than they can hide from 9 rows on where K
//   is long (16, 4096, 14336: 18.4 against 14.4 of 64 x 32 tiles in splits).
//
// All other calls take the cheapest of the tiles by an estimate: a CU runs one
// block's K step in `one`, the steps of two blocks (or of two groups of waves of
// one) in `two`; splits of K of at least four steps add the write and the read of
// their partial sums and a launch; weights come at 5 TB/s at best.  The figures
// (us) are fitted to forced runs of 100 shapes (1 to 8192 rows, K of 1024 to
// 14336, dense and grouped), over which the choice is 2.4 % (root mean square)
// slower than the fastest variant, 13 % at worst (17, 1024, 1024: 4.4 against
// 3.9).  Where it changes over: 128, 4096, 4096: 9.4 of 64 x 32 in two groups
// against 11.1 of 64 x 64; 256, 4096, 4096: 16.9 against 11.5; 384, 4096, 4096:
// 20.6 of 64 x 64 in two groups against 16.3 in one; 512, 4096, 4096: 16.8 of 64 x
// 64 against 21.9 of 128 x 128 in two groups; 600, 4096, 4096: 26.0 against 21.8;
// 1500, 4096, 4096: 32 of 128 x 128 in one group against 49 of 256 x 256; 3000,
// 4096, 4096: 59 against 51; 128, 4096, 14336 in 64 x 64 tiles of one group: 20.4
// in four splits against 51 in one.
struct F8TileRate {
  lowbit::LinearF8Kind kind;
  int bn, bm, groups, threads;
  double one, two;
};
constexpr F8TileRate kF8Tiles[] = {{lowbit::F8_TILE_64X32, 64, 32, 1, 256, 0.36, 0.46},
                                   {lowbit::F8_TILE_64X64, 64, 64, 1, 256, 0.51, 0.57},
                                   {lowbit::F8_TILE_128X128, 128, 128, 1, 512, 1.04, 1.29},
                                   {lowbit::F8_TILE_64X32_K2, 64, 32, 2, 512, 0.51, 0.51},
                                   {lowbit::F8_TILE_64X64_K2, 64, 64, 2, 512, 0.72, 0.72},
                                   {lowbit::F8_TILE_128X128_K2, 128, 128, 2, 1024, 1.64, 1.64}};
constexpr double kF8JoinUs = 4.57, kF8JoinUsPerByte = 0.63e-6, kF8BytesPerUs = 5e6;
constexpr double kF8GroupsUs = 0.27;   // the sums of two groups
// 256 x 256: one block a CU, a round's start and end, a step of few and of all CUs
constexpr double kF8BigUs = 6.85, kF8BigStep = 1.28, kF8BigFullStep = 1.65;
constexpr int kF8MaxSplits = 16, kF8MinSplitSteps = 4;
lowbit::LinearF8Plan f8_plan(int64_t M, int64_t T, int64_t E, bool gather, int64_t N, int64_t K,
                             lowbit_dtype dtype) {
  using namespace lowbit;
  const int64_t cus = device_cus(), kb = f8_blocks(K);
  const bool grouped = E > 0;
  const int64_t used = grouped ? std::min(E, T) : 1;    // experts with rows, at most
  const int64_t per = (T + used - 1) / used;            // rows of one, on average
  // a variant's row tiles (with experts, each adds less than one to T / bm), and
  // whether a launch can hold its threads
  auto fits = [&](int64_t bn, int64_t bm, int64_t threads) {
    const int64_t tm = grouped ? T / bm + used : (T + bm - 1) / bm;
    return tm * ((N + bn - 1) / bn) <= kF8MaxThreads / threads;
  };
  if (per <= (grouped ? 10 : 16) && fits(64, 16, 256)) {
    const int64_t units = used * ((N + 15) / 16), wide = used * ((N + 63) / 64);
    if (wide * 3 >= cus * 2 && wide <= cus) return {K % 8192 != 0 ? F8_TILE_64X32_K2 : F8_ROWS_NT4, 1};
    if (units >= 4 * (cus * 7 / 4)) return {F8_ROWS_NT4, 1};
    if (units >= 2 * (cus * 7 / 8)) return {F8_ROWS_NT2, 1};
    if (per <= 8 || kb < 64) return {F8_ROWS_NT1, 1};
  }
  // blocks a CU (an expert's last row tile is half full, its first never missing)
  auto load = [&](int64_t bn, int64_t bm) {
    const int64_t tm = grouped ? std::max(used, T / bm + used / 2) : (T + bm - 1) / bm;
    return static_cast<double>(tm) * static_cast<double>((N + bn - 1) / bn) / static_cast<double>(cus);
  };
  const double codes = (static_cast<double>(used) * static_cast<double>(N) + static_cast<double>(T)) *
                       static_cast<double>(kb) * 128.0;
  LinearF8Plan plan{F8_TILE_128X128, 1};                // the fewest threads (16-bit outputs have fewer still)
  double best = std::numeric_limits<double>::infinity();
  for (const F8TileRate& t : kF8Tiles) {
    // (16 waves have 128 registers each: too few for fp32's bf16 copies of the codes)
    if (t.kind == F8_TILE_128X128_K2 && dtype == LOWBIT_F32) continue;
    if (!fits(t.bn, t.bm, t.threads)) continue;
    const double blocks = load(t.bn, t.bm);
    for (int splits = 1; splits <= kF8MaxSplits; ++splits) {
      const int64_t steps = (kb + splits - 1) / splits;
      if (splits > 1 && (kb < int64_t{kF8MinSplitSteps} * splits || (kb + steps - 1) / steps != splits)) continue;
      const double n = blocks * splits;
      double us;
      if (t.groups == 1) {
        const double rest = n - 2 * std::floor(n / 2);
        us = std::floor(n / 2) * t.two;
        if (rest > 0) us += t.one + std::max(rest - 1, 0.0) * (t.two - t.one);
        us *= static_cast<double>(steps);
      } else {                           // (eight steps or more)
        if (kb < int64_t{8} * splits) continue;
        us = std::ceil(n) * t.two * static_cast<double>((steps + 1) / 2) + kF8GroupsUs;
      }
      if (splits > 1)
        us = std::max(us, codes / kF8BytesPerUs) + kF8JoinUs +
             kF8JoinUsPerByte * 4 * splits * static_cast<double>(T) * static_cast<double>(N);
      if (us < best) {
        best = us;
        plan = {t.kind, splits};
      }
    }
  }
  // 256 x 256 tiles: their sums are those of the fp8 MFMA, their offsets into a
  // gathered xq 32 bits, and they load four blocks' scales at once
  if (dtype != LOWBIT_F32 && kb >= 4 && !(gather && M * K > int64_t{0xffffffff}) && fits(256, 256, 512)) {
    const double n = load(256, 256), whole = std::floor(n);
    double us = whole * (kF8BigUs + static_cast<double>(kb) * kF8BigFullStep);
    if (n > whole) us += kF8BigUs + static_cast<double>(kb) * kF8BigStep;
    if (us < best) plan = {F8_TILE_256X256, 1};
  }
  return plan;
}

size_t f8_partial_bytes(const lowbit::LinearF8Plan& plan, int64_t T, int64_t N) {
  if (plan.splits <= 1) return 0;
  return static_cast<size_t>(plan.splits) * static_cast<size_t>(T) * static_cast<size_t>((N + 3) / 4 * 4) *
         sizeof(float);
}

// The block-scaled e4m3 product (shared by the dense and the grouped call;
// offsets == nullptr with E == 0 is the dense one).
lowbit_status run_linear_f8(const uint8_t* xq, const float* xscale, const int32_t* rows,
                            const int32_t* offsets, const uint8_t* wq, const float* wscale,
                            const void* bias, void* y, lowbit_dtype dtype, int64_t M, int64_t T, int64_t E,
                            int64_t N, int64_t K, void* workspace, size_t workspace_bytes, void* stream) {
  lowbit_status st = check_q8_row(K, 16);
  if (st != LOWBIT_OK) return st;
  if (!valid_dtype(dtype)) return fail(LOWBIT_ERR_UNSUPPORTED, "dtype=%d", (int)dtype);
  if (N <= 0 || N > kMaxDim) return fail(LOWBIT_ERR_INVALID_ARG, "N=%lld must be in 1..2^30", (long long)N);
  if (M < 0 || M > kMaxDim || T < 0 || T > kMaxDim)
    return fail(LOWBIT_ERR_INVALID_ARG, "rows M=%lld, T=%lld must be in 0..2^30", (long long)M, (long long)T);
  if (!wq || !wscale) return fail(LOWBIT_ERR_INVALID_ARG, "NULL weight pointer");
  if (workspace == nullptr && workspace_bytes != 0)
    return fail(LOWBIT_ERR_WORKSPACE, "workspace_bytes > 0 with a NULL workspace");
  if (workspace != nullptr && !aligned(workspace, 256))
    return fail(LOWBIT_ERR_WORKSPACE, "workspace must be 256-byte aligned");
  if (T == 0) return LOWBIT_OK;
  if (M == 0) return fail(LOWBIT_ERR_INVALID_ARG, "M=0 rows of xq for T=%lld rows of y", (long long)T);
  if (!xq || !xscale || !y) return fail(LOWBIT_ERR_INVALID_ARG, "NULL xq, xscale or y");
  if (!aligned(xq, 16) || !aligned(wq, 16))
    return fail(LOWBIT_ERR_MISALIGNED, "xq and wq must be 16-byte aligned");
  const size_t e = dtype_bytes(dtype);
  if (!aligned(xscale, 4) || !aligned(wscale, 4) || !aligned(y, e) || (bias && !aligned(bias, e)) ||
      (rows && !aligned(rows, 4)) || (offsets && !aligned(offsets, 4)))
    return fail(LOWBIT_ERR_MISALIGNED,
                "scales, rows, offsets, bias and y must be aligned to their element size");
  lowbit::LinearF8Params p{};
  p.xq = xq;
  p.xs = xscale;
  p.rows = rows;
  p.offsets = offsets;
  p.wq = wq;
  p.ws = wscale;
  p.bias = bias;
  p.y = y;
  p.M = M;
  p.T = T;
  p.N = static_cast<int>(N);
  p.K = static_cast<int>(K);
  p.E = static_cast<int>(E);
  p.kb = static_cast<int>(f8_blocks(K));
  p.nb = static_cast<int>(f8_blocks(N));
  lowbit::LinearF8Plan plan = f8_plan(M, T, E, rows != nullptr, N, K, dtype);
  if (workspace_bytes < f8_partial_bytes(plan, T, N)) plan.splits = 1;   // one block a tile over all of K
  p.partials = static_cast<float*>(workspace);
  const hipError_t he = lowbit::launch_linear_f8(p, plan, act_kind(dtype), static_cast<hipStream_t>(stream));
  if (he == hipErrorInvalidConfiguration)
    return fail(LOWBIT_ERR_INVALID_ARG, "T=%lld N=%lld: the outputs have 2^23 tiles of 128 x 128 or more",
                (long long)T, (long long)N);
  if (he != hipSuccess) return hip_fail(he, "linear_f8 launch");
  return LOWBIT_OK;
}

// ------------------------------------------- around the experts, adapters --

constexpr int64_t kLoraMaxN = int64_t(1) << 23;
constexpr int64_t kRouteMaxT = int64_t(1) << 25;                 // (four rows a block of 256 threads)
constexpr int64_t kLaunchBlocks = lowbit::kF8MaxThreads / 256;   // of 256 threads

// Schedule of the adapters' two products.
struct LoraSchedule {
  lowbit::LoraPlan plan;
  int rank_pad, splits, units_split;
  size_t bytes;
};
LoraSchedule lora_schedule(int64_t T, int64_t L, int64_t rank, int64_t N, int64_t K, lowbit_dtype dtype) {
  LoraSchedule s{};
  const int64_t each = T / std::min(T, L), cus = device_cus();   // rows an adapter
  const int64_t units = (K * static_cast<int64_t>(dtype_bytes(dtype)) + 127) / 128;
  s.rank_pad = static_cast<int>((rank + 15) / 16 * 16);
  s.splits = 1;
  s.units_split = static_cast<int>(units);
  // tiles that hold rows: those of all rows, and a part of one for each adapter
  auto tiles = [&](int64_t rows) { return (T + rows - 1) / rows + std::min(T, L) / 2; };

  // One launch for few rows, whose blocks each make their tile's t: latencies, then
  // a wave's units of K one after another (8 waves share them up to rank 16, 4
  // beyond), up to 4.5 us more where every CU has a block, and a second turn of
  // `step` columns.  Two launches are latencies and the bytes.  The estimates, fitted
  // to both sides of 90 random shapes (1 to 200 rows, K 512 to 14336, N 256 to
  // 14336), cost 0.5 % over the better of the two on them.  us, one / two launches:
  // 1 row of rank 16, 4096 -> 4096 bf16 6.7 / 9.5; 4 rows of 1024 -> 256, rank 32 5.5
  // / 9.1; 64 rows of 32 adapters of rank 16, 4096 -> 14336 10.2 / 14.6; rank 32,
  // 200 rows of 16, 8192 -> 4096 16.2 / 10.5; 1 row, 14336 -> 1024 18 / 9.7; fp32,
  // 16 rows of rank 24, 512 -> 256 8.3 / 10.1, 32 rows, 5120 -> 1024 24 / 14.
  const bool fp32 = dtype == LOWBIT_F32;
  const int64_t step = rank <= 16 ? 1024 : 512, steps = (N + step - 1) / step;
  const int64_t across = std::max<int64_t>(1, std::min(steps, cus / tiles(16)));
  const int64_t turns = (steps + across - 1) / across;
  const double one_us = (fp32 ? 7.3 : 4.6) + (fp32 ? 0.42 : 0.24) * static_cast<double>(units) / (rank <= 16 ? 8 : 4) +
                        4.5 * static_cast<double>(tiles(16) * across) / static_cast<double>(cus) +
                        static_cast<double>(turns - 1);
  const double bytes = static_cast<double>(std::min(T, L) * rank * (K + N) + T * (2 * N + K)) *
                       static_cast<double>(dtype_bytes(dtype));
  const double two_us = (fp32 ? 10.0 : 8.7) + bytes / 6e6;
  if (each < 32 && rank <= 32 && turns <= 2 && tiles(16) <= cus / 2 && one_us < two_us) {
    s.plan.fused = true;
    s.plan.cols = static_cast<int>(turns * step);
    return s;
  }

  // Two launches.  Tiles of 16 rows whose K the waves share, or, where adapters
  // have rows for them, of 64 or 128 in the first product (8192 rows, rank 64:
  // 27 us in tiles of 128, 33 of 64) and of 32 in the second.  us, tiles of 16 and
  // 16 / of 64 and 32, 4096 -> 4096 bf16, rank 64: 24 rows an adapter of 16 adapters
  // 15.5 / 15.1, 32 rows 15.1 / 15.0, 64 rows 20.0 / 17.1, 128 rows 32 / 23; 1024 ->
  // 14336, 32 rows 22.3 / 18.3.  Few adapters in all gain by the waves' sharing of K
  // instead (32 rows of one 10.0 / 11.8, 64 of one 10.0 / 12.1, 64 of each of 4 11.2 /
  // 12.7), which this rule gives away.
  s.plan.many = each >= 32;
  s.plan.shrink_rows = each >= 256 ? 128 : each >= 32 ? 64 : 16;
  // as many K ranges as there are CUs for: the second product adds their sums up
  // (8192 rows: 111 us with 4 of them, 125 with 16)
  const int64_t want = std::max<int64_t>(cus / (tiles(s.plan.shrink_rows) * ((rank + 63) / 64)), 1);
  const int64_t splits = std::min<int64_t>({want, (units + 7) / 8, lowbit::kLoraMaxSplits});
  s.units_split = static_cast<int>((units + splits - 1) / splits);
  s.splits = static_cast<int>((units + s.units_split - 1) / s.units_split);
  // columns of a block: the most that leave each CU two blocks (64 rows of 32
  // adapters, 14336 columns: 512 10.4 us, 256 12.8, 1024 15.2; 777 rows of 7,
  // 5001 columns: 256 11.2, 512 14.0; 8192 rows: 1024 109, 2048 134)
  s.plan.cols = 1024;
  while (s.plan.cols > 256 && tiles(s.plan.many ? 32 : 16) * ((N + s.plan.cols - 1) / s.plan.cols) < 2 * cus)
    s.plan.cols /= 2;
  s.bytes = static_cast<size_t>(s.splits) * static_cast<size_t>(T) * s.rank_pad * sizeof(float);
  return s;
}

bool lora_sizes_ok(int64_t T, int64_t L, int64_t rank, int64_t N, int64_t K) {
  return T >= 0 && T <= kMaxDim && L >= 1 && L <= kF8MaxExperts && rank >= 8 && rank % 8 == 0 &&
         rank <= lowbit::kLoraMaxRank && N >= 1 && N <= kLoraMaxN && K >= 16 && K % 16 == 0 && K <= kQ8MaxK &&
         (T / 16 + std::min(T, L + 2)) * std::max((N + 255) / 256, (rank + 63) / 64) < kLaunchBlocks;
}

}  // namespace

extern "C" {

int lowbit_abi_version(void) { return LOWBIT_ABI_VERSION; }

size_t lowbit_packed_bytes(int bits, int64_t N, int64_t K) {
  if (!valid_bits(bits) || N <= 0 || K <= 0 || K % 32 != 0) return 0;
  return static_cast<size_t>(N) * static_cast<size_t>(K) * bits / 8;
}

int64_t lowbit_num_groups(int64_t K, int group) {
  if (!valid_group(group) || K <= 0 || K % group != 0) return 0;
  return K / group;
}

const char* lowbit_status_string(lowbit_status s) {
  switch (s) {
    case LOWBIT_OK: return "ok";
    case LOWBIT_ERR_INVALID_ARG: return "invalid argument";
    case LOWBIT_ERR_UNSUPPORTED: return "unsupported combination";
    case LOWBIT_ERR_MISALIGNED: return "misaligned pointer";
    case LOWBIT_ERR_NONFINITE: return "non-finite weight";
    case LOWBIT_ERR_RANGE: return "scale or zero out of range for its dtype";
    case LOWBIT_ERR_WORKSPACE: return "bad workspace";
    case LOWBIT_ERR_HIP: return "HIP runtime error";
  }
  return "unknown status";
}

const char* lowbit_last_error(void) { return g_last_error.c_str(); }

lowbit_status lowbit_set_tuning(lowbit_tuning_key key, int value) {
  g_last_error.clear();
  if (static_cast<int>(key) < 0 || key >= LOWBIT_TUNE_COUNT)
    return fail(LOWBIT_ERR_INVALID_ARG, "tuning key %d", (int)key);
  if (value < 0) return fail(LOWBIT_ERR_INVALID_ARG, "tuning value %d", value);
  g_tuning[key].store(value, std::memory_order_relaxed);
  return LOWBIT_OK;
}

lowbit_status lowbit_quantize_pack(const void* w, lowbit_dtype w_dtype, int bits, int group, int64_t N,
                                   int64_t K, lowbit_dtype sz_dtype, void* scales, void* zeros,
                                   uint8_t* packed, uint8_t* codes, void* stream) {
  g_last_error.clear();
  lowbit_status st = check_common(bits, group, N, K);
  if (st != LOWBIT_OK) return st;
  if (!valid_dtype(w_dtype)) return fail(LOWBIT_ERR_UNSUPPORTED, "w_dtype=%d", (int)w_dtype);
  if (!valid_dtype(sz_dtype)) return fail(LOWBIT_ERR_UNSUPPORTED, "sz_dtype=%d", (int)sz_dtype);
  if (!w || !scales || !zeros || !packed) return fail(LOWBIT_ERR_INVALID_ARG, "NULL pointer");
  if (!aligned(w, 16)) return fail(LOWBIT_ERR_MISALIGNED, "w must be 16-byte aligned");
  if (!aligned(packed, 16)) return fail(LOWBIT_ERR_MISALIGNED, "packed must be 16-byte aligned");
  const size_t e = dtype_bytes(sz_dtype);
  if (!aligned(scales, e) || !aligned(zeros, e))
    return fail(LOWBIT_ERR_MISALIGNED, "scales/zeros must be aligned to their element size");

  hipStream_t s = static_cast<hipStream_t>(stream);
  int* status = nullptr;
  std::unique_lock<std::mutex> status_lock;
  st = device_status_word(&status, &status_lock);
  if (st != LOWBIT_OK) return st;
  hipError_t he = hipMemsetAsync(status, 0, 2 * sizeof(int), s);
  if (he != hipSuccess) return hip_fail(he, "hipMemsetAsync(status)");
  lowbit::QuantParams p{};
  p.w = w; p.scales = scales; p.zeros = zeros; p.packed = packed; p.codes = codes;
  p.status = status; p.N = N; p.K = K; p.bits = bits; p.group = group;
  p.sz_act = act_kind(sz_dtype);
  p.w_act = act_kind(w_dtype);
  he = lowbit::launch_quant_pack(p, s);
  if (he != hipSuccess) return hip_fail(he, "quant_pack launch");
  int host[2] = {0, 0};
  he = hipMemcpyAsync(host, status, sizeof(host), hipMemcpyDeviceToHost, s);
  if (he != hipSuccess) return hip_fail(he, "hipMemcpyAsync(status)");
  he = hipStreamSynchronize(s);
  if (he != hipSuccess) return hip_fail(he, "hipStreamSynchronize");
  if (host[0]) return fail(LOWBIT_ERR_NONFINITE, "weight holds a NaN or infinity");
  if (host[1]) return fail(LOWBIT_ERR_RANGE, "a scale or zero is not finite in its dtype");
  return LOWBIT_OK;
}

size_t lowbit_linear_workspace_bytes(int bits, int group, int64_t M, int64_t N, int64_t K,
                                     lowbit_dtype act_dtype) {
  if (!valid_bits(bits) || !valid_group(group) || M <= 0 || N <= 0 || K <= 0 || K % group != 0 ||
      M > kMaxDim || N > kMaxDim || K > kMaxDim || !valid_dtype(act_dtype))
    return 0;
  if (act_dtype == LOWBIT_F32) return 0;         // fp32 runs the decode kernel only
  const QmmSchedule sc = qmm_schedule(bits, act_dtype, M, N, K);
  return sc.partial_bytes;
}

lowbit_status lowbit_linear_path(const void* x, lowbit_dtype act_dtype, const uint8_t* packed,
                                 const void* scales, const void* zeros, const void* bias, void* y,
                                 int bits, int group, int64_t M, int64_t N, int64_t K,
                                 void* workspace, size_t workspace_bytes, lowbit_path path,
                                 void* stream) {
  g_last_error.clear();
  lowbit_status st = check_linear(x, act_dtype, packed, scales, zeros, bias, y, bits, group, M, N, K);
  if (st != LOWBIT_OK) return st;
  if (path != LOWBIT_PATH_AUTO && path != LOWBIT_PATH_QMV && path != LOWBIT_PATH_QMM)
    return fail(LOWBIT_ERR_INVALID_ARG, "path=%d", (int)path);
  if (workspace == nullptr && workspace_bytes != 0)
    return fail(LOWBIT_ERR_WORKSPACE, "workspace_bytes > 0 with a NULL workspace");
  if (workspace != nullptr && !aligned(workspace, 256))
    return fail(LOWBIT_ERR_WORKSPACE, "workspace must be 256-byte aligned");
  if (path == LOWBIT_PATH_QMM && act_dtype == LOWBIT_F32)
    return fail(LOWBIT_ERR_UNSUPPORTED, "the MFMA path takes fp16 or bf16 activations");
  if (M == 0) return LOWBIT_OK;

  bool use_qmm;
  if (path == LOWBIT_PATH_QMV) use_qmm = false;
  else if (path == LOWBIT_PATH_QMM) use_qmm = true;
  else use_qmm = (M > qmv_max_m(act_dtype)) && act_dtype != LOWBIT_F32;

  hipStream_t s = static_cast<hipStream_t>(stream);
  if (use_qmm)
    return run_qmm(x, act_dtype, packed, scales, zeros, bias, y, bits, group, M, N, K, workspace,
                   workspace_bytes, s);
  return run_qmv(x, act_dtype, packed, scales, zeros, bias, y, bits, group, M, N, K, s);
}

lowbit_status lowbit_linear(const void* x, lowbit_dtype act_dtype, const uint8_t* packed,
                            const void* scales, const void* zeros, const void* bias, void* y,
                            int bits, int group, int64_t M, int64_t N, int64_t K, void* workspace,
                            size_t workspace_bytes, void* stream) {
  return lowbit_linear_path(x, act_dtype, packed, scales, zeros, bias, y, bits, group, M, N, K,
                            workspace, workspace_bytes, LOWBIT_PATH_AUTO, stream);
}

lowbit_status lowbit_linear_noalloc(const void* x, lowbit_dtype act_dtype, const uint8_t* packed,
                                    const void* scales, const void* zeros, const void* bias, void* y,
                                    int bits, int group, int64_t M, int64_t N, int64_t K,
                                    void* stream) {
  g_last_error.clear();
  lowbit_status st = check_linear(x, act_dtype, packed, scales, zeros, bias, y, bits, group, M, N, K);
  if (st != LOWBIT_OK) return st;
  if (M == 0) return LOWBIT_OK;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const bool use_qmm = (M > qmv_max_m(act_dtype)) && act_dtype != LOWBIT_F32;
  if (!use_qmm) return run_qmv(x, act_dtype, packed, scales, zeros, bias, y, bits, group, M, N, K, s);
  // the schedule lowbit_linear takes with a full workspace, its partial
  // planes in the library's device array
  const QmmSchedule sc = qmm_schedule(bits, act_dtype, M, N, K);
  void* scratch = nullptr;
  size_t scratch_bytes = 0;
  if (sc.partial_bytes > 0) {
    if (sc.partial_bytes > lowbit::kNoallocScratchBytes)
      return fail(LOWBIT_ERR_WORKSPACE,
                  "this problem's K split needs %zu bytes of scratch, more than the %zu bytes of the "
                  "library's device array; call lowbit_linear with a workspace",
                  sc.partial_bytes, lowbit::kNoallocScratchBytes);
    const hipError_t e = lowbit::noalloc_scratch(&scratch);
    if (e != hipSuccess) return hip_fail(e, "hipGetSymbolAddress(scratch)");
    scratch_bytes = lowbit::kNoallocScratchBytes;
  }
  return run_qmm(x, act_dtype, packed, scales, zeros, bias, y, bits, group, M, N, K, scratch,
                 scratch_bytes, s);
}

lowbit_status lowbit_linear_multi(const lowbit_linear_desc* descs, int count, lowbit_dtype act_dtype,
                                  int bits, int group, int64_t M, void* stream) {
  g_last_error.clear();
  if (count < 0 || count > LOWBIT_MAX_MULTI)
    return fail(LOWBIT_ERR_INVALID_ARG, "count=%d not in 0..%d", count, LOWBIT_MAX_MULTI);
  if (count > 0 && descs == nullptr) return fail(LOWBIT_ERR_INVALID_ARG, "NULL descs");
  QmvProblem probs[LOWBIT_MAX_MULTI];
  for (int i = 0; i < count; ++i) {
    const lowbit_linear_desc& d = descs[i];
    const lowbit_status st = check_linear(d.x, act_dtype, d.packed, d.scales, d.zeros, d.bias, d.y,
                                          bits, group, M, d.N, d.K);
    if (st != LOWBIT_OK) {
      const std::string detail = g_last_error;
      return fail(st, "desc %d: %s", i, detail.c_str());
    }
    probs[i] = QmvProblem{d.x, d.packed, d.scales, d.zeros, d.bias, d.y, d.N, d.K};
  }
  if (count == 0 || M == 0) return LOWBIT_OK;
  return run_qmv_multi(probs, count, act_dtype, bits, group, M, static_cast<hipStream_t>(stream));
}

lowbit_status lowbit_quantize_act_i8(const void* x, lowbit_dtype act_dtype, int64_t M, int64_t K,
                                     int8_t* xq, float* ascale, void* stream) {
  g_last_error.clear();
  if (!valid_dtype(act_dtype)) return fail(LOWBIT_ERR_UNSUPPORTED, "act_dtype=%d", (int)act_dtype);
  if (M < 0 || M > kMaxDim) return fail(LOWBIT_ERR_INVALID_ARG, "M=%lld", (long long)M);
  if (K <= 0 || K > kMaxDim || K % 32 != 0)
    return fail(LOWBIT_ERR_INVALID_ARG, "K=%lld must be a positive multiple of 32 (at most 2^30)",
                (long long)K);
  if (M == 0) return LOWBIT_OK;
  if (!x || !xq || !ascale) return fail(LOWBIT_ERR_INVALID_ARG, "NULL x, xq or ascale");
  if (!aligned(x, 16) || !aligned(xq, 16) || !aligned(ascale, 4))
    return fail(LOWBIT_ERR_MISALIGNED, "x and xq must be 16-byte aligned, ascale 4-byte aligned");
  lowbit::ActQuantParams p{x, xq, ascale, static_cast<int>(M), static_cast<int>(K)};
  const hipError_t e = lowbit::launch_act_quant_i8(p, act_kind(act_dtype), static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return hip_fail(e, "act_quant_i8 launch");
  return LOWBIT_OK;
}

lowbit_status lowbit_linear_a8(const int8_t* xq, const float* ascale, const uint8_t* packed,
                               const void* scales, const void* zeros, const void* bias, void* y,
                               lowbit_dtype dtype, int bits, int group, int64_t M, int64_t N,
                               int64_t K, void* stream) {
  g_last_error.clear();
  lowbit_status st = check_common(bits, group, N, K);
  if (st != LOWBIT_OK) return st;
  if (M < 0 || M > kA8MaxM)
    return fail(LOWBIT_ERR_INVALID_ARG, "M=%lld not in 0..%lld", (long long)M, (long long)kA8MaxM);
  if (!valid_dtype(dtype)) return fail(LOWBIT_ERR_UNSUPPORTED, "dtype=%d", (int)dtype);
  if (!packed || !scales || !zeros) return fail(LOWBIT_ERR_INVALID_ARG, "NULL weight pointer");
  if (M == 0) return LOWBIT_OK;
  if (!xq || !ascale || !y) return fail(LOWBIT_ERR_INVALID_ARG, "NULL xq, ascale or y");
  if (!aligned(packed, 16) || !aligned(xq, 16))
    return fail(LOWBIT_ERR_MISALIGNED, "packed and xq must be 16-byte aligned");
  const size_t e = dtype_bytes(dtype);
  if (!aligned(ascale, 4) || !aligned(scales, e) || !aligned(zeros, e) || !aligned(y, e) ||
      (bias && !aligned(bias, e)))
    return fail(LOWBIT_ERR_MISALIGNED, "ascale/scales/zeros/bias/y must be aligned to their element size");
  lowbit::A8Params p{};
  p.xq = xq;
  p.ascale = ascale;
  p.packed = packed;
  p.scales = scales;
  p.zeros = zeros;
  p.bias = bias;
  p.y = y;
  p.M = static_cast<int>(M);
  p.N = static_cast<int>(N);
  p.K = static_cast<int>(K);
  p.groups = static_cast<int>(K / group);
  p.group = group;
  p.row_bytes = K * bits / 8;
  int mtt = 1, nt = 1;
  a8_tiles(M, N, &mtt, &nt);
  const hipError_t he = kA8[bits](p, mtt, nt, act_kind(dtype), static_cast<hipStream_t>(stream));
  if (he != hipSuccess) return hip_fail(he, "qmm_a8 launch");
  return LOWBIT_OK;
}

lowbit_status lowbit_add_rmsnorm_q8(const void* x, const void* residual, const void* weight, float eps,
                                    lowbit_dtype dtype, int64_t M, int64_t K, lowbit_q8_format format,
                                    void* q, float* qscale, void* sum, void* y, void* stream) {
  g_last_error.clear();
  if (!valid_dtype(dtype)) return fail(LOWBIT_ERR_UNSUPPORTED, "dtype=%d", (int)dtype);
  if (format != LOWBIT_Q8_NONE && format != LOWBIT_Q8_I8 && format != LOWBIT_Q8_F8)
    return fail(LOWBIT_ERR_UNSUPPORTED, "format=%d", (int)format);
  const lowbit_status st = check_q8_row(K, format == LOWBIT_Q8_I8 ? 32 : 16);
  if (st != LOWBIT_OK) return st;
  if (M < 0 || M > kNormMaxM) return fail(LOWBIT_ERR_INVALID_ARG, "M=%lld not in 0..2^22 - 1", (long long)M);
  if (!(eps >= 1e-20f && eps <= 1.0f)) return fail(LOWBIT_ERR_INVALID_ARG, "eps=%g not in 1e-20..1", eps);
  if (M == 0) return LOWBIT_OK;
  if (!x) return fail(LOWBIT_ERR_INVALID_ARG, "NULL x");
  if ((residual != nullptr) != (sum != nullptr))
    return fail(LOWBIT_ERR_INVALID_ARG, "residual and sum go together");
  if ((format != LOWBIT_Q8_NONE) != (q != nullptr) || (format != LOWBIT_Q8_NONE) != (qscale != nullptr))
    return fail(LOWBIT_ERR_INVALID_ARG, "q and qscale are given with an 8-bit format and not without");
  if (format == LOWBIT_Q8_NONE && !y) return fail(LOWBIT_ERR_INVALID_ARG, "no output: NULL y without a format");
  if (!aligned(x, 16) || !aligned(residual, 16) || !aligned(weight, 16) || !aligned(sum, 16) ||
      !aligned(y, 16) || !aligned(q, 16) || !aligned(qscale, 4))
    return fail(LOWBIT_ERR_MISALIGNED, "arrays must be 16-byte aligned, qscale 4-byte aligned");
  lowbit::NormQ8Params p{};
  p.x = x;
  p.residual = residual;
  p.weight = weight;
  p.sum = sum;
  p.y = y;
  p.q = q;
  p.qscale = qscale;
  p.eps = eps;
  p.M = M;
  p.K = static_cast<int>(K);
  const hipError_t e =
      lowbit::launch_norm_q8(p, act_kind(dtype), static_cast<int>(format), static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return hip_fail(e, "norm_q8 launch");
  return LOWBIT_OK;
}

lowbit_status lowbit_quantize_act_f8(const void* x, lowbit_dtype dtype, int64_t M, int64_t K, uint8_t* xq,
                                     float* xscale, void* stream) {
  g_last_error.clear();
  if (!valid_dtype(dtype)) return fail(LOWBIT_ERR_UNSUPPORTED, "dtype=%d", (int)dtype);
  const lowbit_status st = check_q8_row(K, 16);
  if (st != LOWBIT_OK) return st;
  if (M < 0 || M > kMaxDim || M * f8_blocks(K) > kActF8MaxBlocks)
    return fail(LOWBIT_ERR_INVALID_ARG, "M=%lld: M * ceil(K / 128) must be at most 2^28 - 16", (long long)M);
  if (M == 0) return LOWBIT_OK;
  if (!x || !xq || !xscale) return fail(LOWBIT_ERR_INVALID_ARG, "NULL x, xq or xscale");
  if (!aligned(x, 16) || !aligned(xq, 16) || !aligned(xscale, 4))
    return fail(LOWBIT_ERR_MISALIGNED, "x and xq must be 16-byte aligned, xscale 4-byte aligned");
  const lowbit::ActQuantF8Params p{x, xq, xscale, M, static_cast<int>(K)};
  const hipError_t e = lowbit::launch_act_quant_f8(p, act_kind(dtype), static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return hip_fail(e, "act_quant_f8 launch");
  return LOWBIT_OK;
}

lowbit_status lowbit_quantize_weight_f8(const void* w, lowbit_dtype dtype, int64_t E, int64_t N, int64_t K,
                                        uint8_t* wq, float* wscale, void* stream) {
  g_last_error.clear();
  if (!valid_dtype(dtype)) return fail(LOWBIT_ERR_UNSUPPORTED, "dtype=%d", (int)dtype);
  const lowbit_status st = check_q8_row(K, 16);
  if (st != LOWBIT_OK) return st;
  if (E <= 0 || E > kF8MaxExperts || N <= 0 || N > kMaxDim ||
      E * f8_blocks(N) * f8_blocks(K) >= (int64_t(1) << 24))
    return fail(LOWBIT_ERR_INVALID_ARG,
                "E=%lld N=%lld: must be positive, E at most 2^16, fewer than 2^24 blocks of 128 x 128",
                (long long)E, (long long)N);
  if (!w || !wq || !wscale) return fail(LOWBIT_ERR_INVALID_ARG, "NULL w, wq or wscale");
  if (!aligned(w, 16) || !aligned(wq, 16) || !aligned(wscale, 4))
    return fail(LOWBIT_ERR_MISALIGNED, "w and wq must be 16-byte aligned, wscale 4-byte aligned");
  const lowbit::WeightQuantF8Params p{w, wq, wscale, E, static_cast<int>(N), static_cast<int>(K)};
  const hipError_t e = lowbit::launch_weight_quant_f8(p, act_kind(dtype), static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return hip_fail(e, "weight_quant_f8 launch");
  return LOWBIT_OK;
}

size_t lowbit_linear_f8_workspace_bytes(int64_t M, int64_t T, int64_t E, int64_t N, int64_t K,
                                        lowbit_dtype dtype) {
  if (K <= 0 || K > kQ8MaxK || K % 16 != 0 || N <= 0 || N > kMaxDim || T <= 0 || T > kMaxDim || M <= 0 ||
      M > kMaxDim || E < 0 || E > kF8MaxExperts || !valid_dtype(dtype))
    return 0;
  // (whether the rows are gathered is not said here, and decides the schedule of a large xq)
  const size_t plain = f8_partial_bytes(f8_plan(M, T, E, false, N, K, dtype), T, N);
  return E == 0 ? plain : std::max(plain, f8_partial_bytes(f8_plan(M, T, E, true, N, K, dtype), T, N));
}

lowbit_status lowbit_linear_f8(const uint8_t* xq, const float* xscale, const uint8_t* wq,
                               const float* wscale, const void* bias, void* y, lowbit_dtype dtype,
                               int64_t M, int64_t N, int64_t K, void* workspace, size_t workspace_bytes,
                               void* stream) {
  g_last_error.clear();
  return run_linear_f8(xq, xscale, nullptr, nullptr, wq, wscale, bias, y, dtype, M, M, 0, N, K, workspace,
                       workspace_bytes, stream);
}

lowbit_status lowbit_linear_f8_grouped(const uint8_t* xq, const float* xscale, const int32_t* rows,
                                       const int32_t* offsets, const uint8_t* wq, const float* wscale,
                                       const void* bias, void* y, lowbit_dtype dtype, int64_t M, int64_t T,
                                       int64_t E, int64_t N, int64_t K, void* workspace,
                                       size_t workspace_bytes, void* stream) {
  g_last_error.clear();
  if (E <= 0 || E > kF8MaxExperts) return fail(LOWBIT_ERR_INVALID_ARG, "E=%lld not in 1..2^16", (long long)E);
  if (!offsets) return fail(LOWBIT_ERR_INVALID_ARG, "NULL offsets");
  if (!rows && M != T && T != 0)
    return fail(LOWBIT_ERR_INVALID_ARG, "without rows, xq's M=%lld must be y's T=%lld", (long long)M, (long long)T);
  return run_linear_f8(xq, xscale, rows, offsets, wq, wscale, bias, y, dtype, M, T, E, N, K, workspace,
                       workspace_bytes, stream);
}

lowbit_status lowbit_moe_route(const void* logits, lowbit_dtype dtype, const float* bias, int64_t T,
                               int64_t E, int64_t topk, lowbit_route_score score, int64_t groups,
                               int64_t topk_groups, int group_best, int renormalize, float scale,
                               int32_t* experts, float* weights, void* stream) {
  g_last_error.clear();
  if (!valid_dtype(dtype)) return fail(LOWBIT_ERR_UNSUPPORTED, "dtype=%d", (int)dtype);
  if (score != LOWBIT_ROUTE_SOFTMAX && score != LOWBIT_ROUTE_SIGMOID)
    return fail(LOWBIT_ERR_UNSUPPORTED, "score=%d", (int)score);
  if (T < 0 || T > kRouteMaxT) return fail(LOWBIT_ERR_INVALID_ARG, "T=%lld not in 0..2^25", (long long)T);
  if (E < 1 || E > lowbit::kRouteMaxExperts)
    return fail(LOWBIT_ERR_INVALID_ARG, "E=%lld not in 1..%d", (long long)E, lowbit::kRouteMaxExperts);
  if (topk < 1 || topk > E || topk > lowbit::kRouteMaxTopk)
    return fail(LOWBIT_ERR_INVALID_ARG, "topk=%lld not in 1..min(E, %d)", (long long)topk, lowbit::kRouteMaxTopk);
  if (groups < 1 || groups > lowbit::kRouteMaxGroups || E % groups != 0)
    return fail(LOWBIT_ERR_INVALID_ARG, "groups=%lld must be a divisor of E=%lld, at most %d", (long long)groups,
                (long long)E, lowbit::kRouteMaxGroups);
  if (topk_groups < 1 || topk_groups > groups)
    return fail(LOWBIT_ERR_INVALID_ARG, "topk_groups=%lld not in 1..groups", (long long)topk_groups);
  if (group_best != 1 && group_best != 2) return fail(LOWBIT_ERR_INVALID_ARG, "group_best=%d not 1 or 2", group_best);
  if (!std::isfinite(scale)) return fail(LOWBIT_ERR_INVALID_ARG, "scale=%g is not finite", scale);
  if (T == 0) return LOWBIT_OK;
  if (!logits || !experts || !weights) return fail(LOWBIT_ERR_INVALID_ARG, "NULL logits, experts or weights");
  if (!aligned(logits, dtype_bytes(dtype)) || !aligned(bias, 4) || !aligned(experts, 4) || !aligned(weights, 4))
    return fail(LOWBIT_ERR_MISALIGNED, "arrays must be aligned to their element size");
  lowbit::RouteParams p{};
  p.logits = logits;
  p.bias = bias;
  p.experts = experts;
  p.weights = weights;
  p.T = T;
  p.E = static_cast<int>(E);
  p.topk = static_cast<int>(topk);
  p.sigmoid = score == LOWBIT_ROUTE_SIGMOID;
  p.groups = static_cast<int>(groups);
  while ((int64_t{1} << p.groups_shift) < groups) ++p.groups_shift;
  while ((int64_t{1} << p.index_bits) < E) ++p.index_bits;
  p.topk_groups = static_cast<int>(topk_groups);
  p.group_best = groups > 1 ? static_cast<int>(group_best) : 1;   // (one group has no value to compare)
  p.renormalize = renormalize != 0;
  p.scale = scale;
  const hipError_t e = lowbit::launch_moe_route(p, act_kind(dtype), static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return hip_fail(e, "moe_route launch");
  return LOWBIT_OK;
}

size_t lowbit_group_rows_workspace_bytes(int64_t T, int64_t topk, int64_t E) {
  if (T <= 0 || T > kMaxDim || topk < 1 || topk > kMaxDim || T * topk > kMaxDim || E < 1 || E > kF8MaxExperts) return 0;
  return lowbit::group_workspace(T * topk, E).bytes;
}

lowbit_status lowbit_group_rows(const void* ids, int id_bytes, int64_t T, int64_t topk, int64_t E,
                                int32_t* rows, int32_t* offsets, int32_t* position, void* workspace,
                                size_t workspace_bytes, void* stream) {
  g_last_error.clear();
  if (id_bytes != 4 && id_bytes != 8) return fail(LOWBIT_ERR_UNSUPPORTED, "id_bytes=%d not 4 or 8", id_bytes);
  if (T < 0 || T > kMaxDim || topk < 1 || topk > kMaxDim || T * topk > kMaxDim)
    return fail(LOWBIT_ERR_INVALID_ARG, "T=%lld topk=%lld: T * topk must be in 0..2^30, topk at least 1",
                (long long)T, (long long)topk);
  if (E < 1 || E > kF8MaxExperts) return fail(LOWBIT_ERR_INVALID_ARG, "E=%lld not in 1..2^16", (long long)E);
  if (!offsets || (T > 0 && (!ids || !rows))) return fail(LOWBIT_ERR_INVALID_ARG, "NULL ids, rows or offsets");
  if (!aligned(ids, id_bytes) || !aligned(rows, 4) || !aligned(offsets, 4) || !aligned(position, 4))
    return fail(LOWBIT_ERR_MISALIGNED, "arrays must be aligned to their element size");
  if (workspace == nullptr && workspace_bytes != 0)
    return fail(LOWBIT_ERR_WORKSPACE, "workspace_bytes > 0 with a NULL workspace");
  if (workspace != nullptr && !aligned(workspace, 256))
    return fail(LOWBIT_ERR_WORKSPACE, "workspace must be 256-byte aligned");
  // Division by topk: with m = floor(2^b / topk) + 1, b = 30 + ceil(log2(topk)),
  // s * m / 2^b is s / topk plus less than s * topk / (2^b topk) <= s / (2^30 topk),
  // too little to reach the next whole number for s < 2^30.
  int shift = 30;
  while ((int64_t{1} << (shift - 30)) < topk) ++shift;
  const uint32_t mul = static_cast<uint32_t>((uint64_t{1} << shift) / static_cast<uint64_t>(topk) + 1);
  lowbit::GroupRowsParams p{ids, rows, offsets, position, T * topk, static_cast<int>(E), mul, shift,
                            nullptr, nullptr, nullptr, nullptr};
  const lowbit::GroupWorkspace w = lowbit::group_workspace(T * topk, E);
  if (w.used && workspace_bytes >= w.bytes) {
    char* at = static_cast<char*>(workspace);
    p.counts = reinterpret_cast<int*>(at);
    if (w.scanned) p.totals = reinterpret_cast<int*>(at + w.totals);
    if (w.digits) {
      p.order = reinterpret_cast<int32_t*>(at + w.order);
      p.keys = reinterpret_cast<int32_t*>(at + w.keys);
    }
  }
  const hipError_t e = lowbit::launch_group_rows(p, id_bytes, static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return hip_fail(e, "group_rows launch");
  return LOWBIT_OK;
}

lowbit_status lowbit_moe_combine(const void* y, const int32_t* position, const float* weights,
                                 const void* residual, void* out, lowbit_dtype dtype, int64_t R, int64_t T,
                                 int64_t topk, int64_t N, void* stream) {
  g_last_error.clear();
  if (!valid_dtype(dtype)) return fail(LOWBIT_ERR_UNSUPPORTED, "dtype=%d", (int)dtype);
  if (T < 0 || T > kMaxDim || R < 0 || R > kMaxDim)
    return fail(LOWBIT_ERR_INVALID_ARG, "rows T=%lld, R=%lld must be in 0..2^30", (long long)T, (long long)R);
  if (topk < 1 || topk > (int64_t(1) << 16)) return fail(LOWBIT_ERR_INVALID_ARG, "topk=%lld not in 1..2^16", (long long)topk);
  if (N < 1 || N > kMaxDim) return fail(LOWBIT_ERR_INVALID_ARG, "N=%lld not in 1..2^30", (long long)N);
  if (T == 0) return LOWBIT_OK;
  if (!position || !weights || !out || (R > 0 && !y))
    return fail(LOWBIT_ERR_INVALID_ARG, "NULL y, position, weights or out");
  const size_t e = dtype_bytes(dtype);
  if (!aligned(y, e) || !aligned(residual, e) || !aligned(out, e) || !aligned(position, 4) || !aligned(weights, 4))
    return fail(LOWBIT_ERR_MISALIGNED, "arrays must be aligned to their element size");
  const lowbit::CombineParams p{y, position, weights, residual, out, R, T, static_cast<int>(N),
                                static_cast<int>(topk)};
  const hipError_t he = lowbit::launch_moe_combine(p, act_kind(dtype), static_cast<hipStream_t>(stream));
  if (he != hipSuccess) return hip_fail(he, "moe_combine launch");
  return LOWBIT_OK;
}

size_t lowbit_lora_workspace_bytes(int64_t T, int64_t L, int64_t rank, int64_t N, int64_t K,
                                   lowbit_dtype dtype) {
  if (!lora_sizes_ok(T, L, rank, N, K) || T == 0 || !valid_dtype(dtype)) return 0;
  return lora_schedule(T, L, rank, N, K, dtype).bytes;
}

lowbit_status lowbit_lora(const void* x, const void* a, const void* b, const float* scales,
                          const int32_t* rows, const int32_t* offsets, const void* base, void* y,
                          lowbit_dtype dtype, int64_t M, int64_t T, int64_t L, int64_t rank, int64_t N,
                          int64_t K, void* workspace, size_t workspace_bytes, void* stream) {
  g_last_error.clear();
  if (!valid_dtype(dtype)) return fail(LOWBIT_ERR_UNSUPPORTED, "dtype=%d", (int)dtype);
  if (M < 0 || M > kMaxDim || !lora_sizes_ok(T, L, rank, N, K))
    return fail(LOWBIT_ERR_INVALID_ARG,
                "M=%lld T=%lld L=%lld rank=%lld N=%lld K=%lld: rows in 0..2^30, L in 1..2^16, rank a multiple of 8 "
                "up to 256, K a multiple of 16 up to 2^23, N in 1..2^23, fewer than 2^24 tiles of 16 x 256 outputs or 16 x 64 "
                "of x . a",
                (long long)M, (long long)T, (long long)L, (long long)rank, (long long)N, (long long)K);
  if (!rows && M != T) return fail(LOWBIT_ERR_INVALID_ARG, "without rows, M=%lld must be T=%lld", (long long)M, (long long)T);
  if (!a || !b || !offsets) return fail(LOWBIT_ERR_INVALID_ARG, "NULL a, b or offsets");
  if (workspace == nullptr && workspace_bytes != 0)
    return fail(LOWBIT_ERR_WORKSPACE, "workspace_bytes > 0 with a NULL workspace");
  if (workspace != nullptr && !aligned(workspace, 256))
    return fail(LOWBIT_ERR_WORKSPACE, "workspace must be 256-byte aligned");
  if (T == 0 || M == 0) return LOWBIT_OK;
  if (!x || !y) return fail(LOWBIT_ERR_INVALID_ARG, "NULL x or y");
  const size_t e = dtype_bytes(dtype);
  if (!aligned(x, 16) || !aligned(a, 16) || !aligned(b, 16))
    return fail(LOWBIT_ERR_MISALIGNED, "x, a and b must be 16-byte aligned");
  if (!aligned(scales, 4) || !aligned(rows, 4) || !aligned(offsets, 4) || !aligned(base, e) || !aligned(y, e))
    return fail(LOWBIT_ERR_MISALIGNED, "scales, rows, offsets, base and y must be aligned to their element size");
  const LoraSchedule s = lora_schedule(T, L, rank, N, K, dtype);
  if (workspace_bytes < s.bytes)
    return fail(LOWBIT_ERR_WORKSPACE, "workspace of %zu bytes, %zu needed", workspace_bytes, s.bytes);
  lowbit::LoraParams p{};
  p.x = x;
  p.a = a;
  p.b = b;
  p.scales = scales;
  p.rows = rows;
  p.offsets = offsets;
  p.base = base;
  p.y = y;
  p.t = static_cast<float*>(workspace);
  p.M = M;
  p.T = T;
  p.L = static_cast<int>(L);
  p.N = static_cast<int>(N);
  p.K = static_cast<int>(K);
  p.rank = static_cast<int>(rank);
  p.rank_pad = s.rank_pad;
  p.splits = s.splits;
  p.units_split = s.units_split;
  const hipError_t he = lowbit::launch_lora(p, s.plan, act_kind(dtype), static_cast<hipStream_t>(stream));
  if (he != hipSuccess) return hip_fail(he, "lora launch");
  return LOWBIT_OK;
}

}  // extern "C"
