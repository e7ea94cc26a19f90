// Launch interface between the C-ABI host code and the HIP kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace lowbit {

// Activation (and scale/zero) element types.
enum ActKind : int { ACT_F32 = 0, ACT_F16 = 1, ACT_BF16 = 2 };

// ---------------------------------------------------------------- quantize --
struct QuantParams {
  const void* w;       // N x K, w_act (fp32, fp16 or bf16; upcast exactly to fp32)
  void* scales;        // N x G, sz dtype
  void* zeros;         // N x G, sz dtype
  uint8_t* packed;     // N x K*bits/8
  uint8_t* codes;      // N x K or nullptr
  int* status;         // [0] non-finite weight seen, [1] non-finite stored scale/zero
  int64_t N, K;
  int bits, group, sz_act, w_act;
};
hipError_t launch_quant_pack(const QuantParams& p, hipStream_t stream);

// --------------------------------------------------------------------- qmv --
struct QmvParams {
  const void* x;          // M x K act
  const uint8_t* packed;  // N x row_bytes
  const void* scales;     // N x groups act
  const void* zeros;      // N x groups act
  const void* bias;       // N act or nullptr
  void* y;                // M x N act
  int M, N, K;
  int lpr_shift;          // log2(lanes cooperating on one row group), <= 6
  int groups;             // K / group
  int64_t row_bytes;      // K * bits / 8
};
// Variants of the decode kernel for one activation row per pass (chosen at
// launch from the blocks per CU, the waves per CU and the row length): the
// default; LEAN, which keeps one staged fragment live at a time (fewer
// registers, one more wave per SIMD); LEAN2, LEAN with two rows per lane
// group at every bit width (more weight bytes in flight per wave); and LEAN1,
// LEAN with one row per lane group at every bit width (twice the waves where
// the default has two rows, for launches too small to fill the CUs).
enum QmvVariant { QMV_DEFAULT = 0, QMV_LEAN = 1, QMV_LEAN2 = 2, QMV_LEAN1 = 3 };
// Rows per row group of the decode kernel for one activation row per pass:
// two rows for 1, 2 and 3-bit codes, one for 4..7 bits (measured on MI355X at
// K = N = 4096, A/B of both builds on one box: two rows 0.15-0.18 us faster
// at b = 1, 2, equal at b = 3, 4, 6, 7, one row 0.35 us faster at b = 5),
// two for every width in LEAN2, one in LEAN1; one row whenever several
// activation rows share a pass.
constexpr int qmv_rows_per_group(int bits, int mt, int variant) {
  return mt == 1 && variant != QMV_LEAN1 && (variant == QMV_LEAN2 || bits <= 3) ? 2 : 1;
}
// LDS quads (16 bytes) per lane of a row group that the decode kernel stages
// for `mt` activation rows of `qd` quads per run (four runs per lane): rounded
// up to an odd count, so that the 16 lanes of one 16-byte LDS read, each at
// the same quad of its own runs, start in 16 distinct 4-bank groups.
constexpr int qmv_stage_quads_per_lane(int mt, int qd) { return (mt * 4 * qd) | 1; }
// Up to kQmvMaxProblems decode problems of one bit width, group size and
// activation dtype served by one launch: blocks with blockIdx.z == i work on
// problem i (grid.x is sized for the largest; blocks past a problem's rows
// exit at once); all share M (grid.y).
constexpr int kQmvMaxProblems = 8;
struct QmvBatch {
  QmvParams prob[kQmvMaxProblems];
};
struct QmvLaunch {
  dim3 grid, block;
  int mt;                 // activation rows per pass: 1, 2 or 4
  int variant;            // mt == 1: a QmvVariant
};
// One entry point per bit width (compiled as separate objects).
hipError_t launch_qmv_b1(const QmvBatch&, const QmvLaunch&, int group, int act, hipStream_t);
hipError_t launch_qmv_b2(const QmvBatch&, const QmvLaunch&, int group, int act, hipStream_t);
hipError_t launch_qmv_b3(const QmvBatch&, const QmvLaunch&, int group, int act, hipStream_t);
hipError_t launch_qmv_b4(const QmvBatch&, const QmvLaunch&, int group, int act, hipStream_t);
hipError_t launch_qmv_b5(const QmvBatch&, const QmvLaunch&, int group, int act, hipStream_t);
hipError_t launch_qmv_b6(const QmvBatch&, const QmvLaunch&, int group, int act, hipStream_t);
hipError_t launch_qmv_b7(const QmvBatch&, const QmvLaunch&, int group, int act, hipStream_t);
// LDS bytes the decode kernel stages per activation row and per lane of a
// round (four 32-code runs).
int qmv_stage_bytes_b1(int act);
int qmv_stage_bytes_b2(int act);
int qmv_stage_bytes_b3(int act);
int qmv_stage_bytes_b4(int act);
int qmv_stage_bytes_b5(int act);
int qmv_stage_bytes_b6(int act);
int qmv_stage_bytes_b7(int act);

// --------------------------------------------------------------------- qmm --
struct QmmParams {
  const void* x;          // M x K act (f16 / bf16)
  const uint8_t* packed;  // N x row_bytes
  const void* scales;     // N x groups act
  const void* zeros;      // N x groups act
  const void* bias;       // N act or nullptr
  void* y;                // M x N act
  float* partials;        // split-K: gridDim.z planes of fp32 tile records (workspace)
  int M, N, K;
  int groups;             // K / group
  int group_shift;        // log2(group)
  int ksteps_per_split;   // 128-wide K steps per grid.z slice
  int64_t row_bytes;      // K * bits / 8
};
// Layout of the split-K partial planes for the reduce kernel: records of
// 4 fp32 in (tile, wave, row tile, column tile, lane) order, one plane per
// K split (block tile 16*mtt x 16*nt*waves; mtt, nt, waves powers of two).
struct QmmReduceShape {
  int splits;
  int tiles_n;            // gridDim.x of the main kernel
  int mtt_shift, nt_shift, wv_shift;
  int64_t plane_recs;     // records per plane
};
// Largest bit widths with an 8-wave MFMA kernel instance: 8 column waves,
// and 4 column waves in two K groups (whose super-step activations take more
// registers).
constexpr int qmm_max_bits_8waves = 5;
constexpr int qmm_max_bits_kgroups = 4;
struct QmmLaunch {
  dim3 grid;              // (ceil(N/(16*nt*waves)), ceil(M/(16*mtt)), k-splits)
  int mtt;                // 16-row MFMA tiles per block: 1, 2, 4 or 8
  int nt;                 // 16-column MFMA tiles per wave (2)
  int waves;              // column waves per block: 4, or 8 (bits <= qmm_max_bits_8waves)
  int kgroups;            // K groups per block: 1, or 2 with 4 column waves
                          // (bits <= qmm_max_bits_kgroups); waves*kgroups waves in all
  int rgroups;            // bf16 kernel: row groups per block, 1 or 2 (each a set of
                          // `waves` column waves over its share of the row tiles)
};
hipError_t launch_qmm_b1(const QmmParams&, const QmmLaunch&, int act, hipStream_t);
hipError_t launch_qmm_b2(const QmmParams&, const QmmLaunch&, int act, hipStream_t);
hipError_t launch_qmm_b3(const QmmParams&, const QmmLaunch&, int act, hipStream_t);
hipError_t launch_qmm_b4(const QmmParams&, const QmmLaunch&, int act, hipStream_t);
hipError_t launch_qmm_b5(const QmmParams&, const QmmLaunch&, int act, hipStream_t);
hipError_t launch_qmm_b6(const QmmParams&, const QmmLaunch&, int act, hipStream_t);
hipError_t launch_qmm_b7(const QmmParams&, const QmmLaunch&, int act, hipStream_t);
// The small-M MFMA kernel (1 <= M <= 16, fp16 activations): blocks of
// 16*nt columns (nt 1 or 2) over all of K, `waves` (4, 8 or 16) waves per
// block splitting the K steps; no workspace, one launch.
hipError_t launch_qmm_small_b1(const QmmParams&, int nt, int waves, hipStream_t);
hipError_t launch_qmm_small_b2(const QmmParams&, int nt, int waves, hipStream_t);
hipError_t launch_qmm_small_b3(const QmmParams&, int nt, int waves, hipStream_t);
hipError_t launch_qmm_small_b4(const QmmParams&, int nt, int waves, hipStream_t);
hipError_t launch_qmm_small_b5(const QmmParams&, int nt, int waves, hipStream_t);
hipError_t launch_qmm_small_b6(const QmmParams&, int nt, int waves, hipStream_t);
hipError_t launch_qmm_small_b7(const QmmParams&, int nt, int waves, hipStream_t);
// The bf16 kernel's main launch (code operands; 4 column waves, nt == 2,
// one K group); launch_qmm_b<bits> calls it and adds the split-K reduce.
hipError_t launch_qmm_bf16_b1(const QmmParams&, const QmmLaunch&, hipStream_t);
hipError_t launch_qmm_bf16_b2(const QmmParams&, const QmmLaunch&, hipStream_t);
hipError_t launch_qmm_bf16_b3(const QmmParams&, const QmmLaunch&, hipStream_t);
hipError_t launch_qmm_bf16_b4(const QmmParams&, const QmmLaunch&, hipStream_t);
hipError_t launch_qmm_bf16_b5(const QmmParams&, const QmmLaunch&, hipStream_t);
hipError_t launch_qmm_bf16_b6(const QmmParams&, const QmmLaunch&, hipStream_t);
hipError_t launch_qmm_bf16_b7(const QmmParams&, const QmmLaunch&, hipStream_t);

// ------------------------------------------- int8 dynamic activations --
struct ActQuantParams {
  const void* x;          // M x K act (fp32, fp16 or bf16), 16-byte aligned
  int8_t* xq;             // M x K codes, 16-byte aligned
  float* ascale;          // M
  int M, K;               // K % 16 == 0
};
hipError_t launch_act_quant_i8(const ActQuantParams&, int act, hipStream_t);

struct A8Params {
  const int8_t* xq;       // M x K codes, 16-byte aligned
  const float* ascale;    // M
  const uint8_t* packed;  // N x row_bytes
  const void* scales;     // N x groups, sz dtype
  const void* zeros;      // N x groups, sz dtype
  const void* bias;       // N, sz dtype, or nullptr
  void* y;                // M x N, sz dtype
  int M, N, K;
  int groups;             // K / group
  int group;
  int64_t row_bytes;      // K * bits / 8
};
// Blocks of 4 waves, `nt` (1 or 2) 16-column MFMA tiles per wave, `mtt`
// (1, 2 or 4) 16-row tiles per block: grid (ceil(N / (64 nt)), ceil(M / (16 mtt))).
hipError_t launch_qmm_a8_b1(const A8Params&, int mtt, int nt, int sz, hipStream_t);
hipError_t launch_qmm_a8_b2(const A8Params&, int mtt, int nt, int sz, hipStream_t);
hipError_t launch_qmm_a8_b3(const A8Params&, int mtt, int nt, int sz, hipStream_t);
hipError_t launch_qmm_a8_b4(const A8Params&, int mtt, int nt, int sz, hipStream_t);
hipError_t launch_qmm_a8_b5(const A8Params&, int mtt, int nt, int sz, hipStream_t);
hipError_t launch_qmm_a8_b6(const A8Params&, int mtt, int nt, int sz, hipStream_t);
hipError_t launch_qmm_a8_b7(const A8Params&, int mtt, int nt, int sz, hipStream_t);

// ------------------------------------------------------ the 8-bit path --
// What a norm writes beside h and y (the values of lowbit_q8_format).
enum Q8Format : int { Q8_NONE = 0, Q8_I8 = 1, Q8_F8 = 2 };
struct NormQ8Params {
  const void* x;          // M x K act, 16-byte aligned
  const void* residual;   // M x K act, or nullptr (then sum is nullptr too)
  const void* weight;     // K act, or nullptr (ones)
  void* sum;              // M x K act: x + residual (may be x or residual itself)
  void* y;                // M x K act: the normalized rows, or nullptr
  void* q;                // M x K codes (int8 or e4m3), or nullptr (Q8_NONE)
  float* qscale;          // M (int8) or M x ceil(K / 128) (e4m3)
  float eps;
  int64_t M;
  int K;                  // K % 16 == 0
};
hipError_t launch_norm_q8(const NormQ8Params&, int act, int fmt, hipStream_t);

struct ActQuantF8Params {
  const void* x;          // M x K act, 16-byte aligned
  uint8_t* xq;            // M x K e4m3 codes, 16-byte aligned
  float* xscale;          // M x ceil(K / 128)
  int64_t M;
  int K;                  // K % 16 == 0
};
hipError_t launch_act_quant_f8(const ActQuantF8Params&, int act, hipStream_t);

struct WeightQuantF8Params {
  const void* w;          // E x N x K act, 16-byte aligned
  uint8_t* wq;            // E x N x K e4m3 codes, 16-byte aligned
  float* wscale;          // E x ceil(N / 128) x ceil(K / 128)
  int64_t E;
  int N, K;               // K % 16 == 0
};
hipError_t launch_weight_quant_f8(const WeightQuantF8Params&, int act, hipStream_t);

// Block-scaled e4m3 product, dense or grouped by expert.
struct LinearF8Params {
  const uint8_t* xq;      // M x K e4m3 codes, 16-byte aligned
  const float* xs;        // M x kb
  const int32_t* rows;    // T source rows of xq, or nullptr (row t reads row t)
  const int32_t* offsets; // E + 1 row bounds of the experts, or nullptr (dense)
  const uint8_t* wq;      // E x N x K e4m3 codes, 16-byte aligned
  const float* ws;        // E x nb x kb
  const void* bias;       // E x N, out type, or nullptr
  void* y;                // T x N, out type
  int64_t M, T;           // rows of xq, rows of y (equal without `rows`)
  int N, K, E;            // K % 16 == 0
  int kb, nb;             // ceil(K / 128), ceil(N / 128)
  int tiles_n;            // column tiles
  float* partials;        // K splits: planes of T x n_pad fp32 (workspace)
  int n_pad;              // N rounded up to a multiple of 4
  int kb_split;           // K blocks of a split
};
// Variants: few rows (16 rows and 16, 32 or 64 columns a block, the weights
// straight from memory); tiles of columns x rows through LDS, their K range
// split between two groups of a block's waves (_K2) and over the grid where
// there are few (partial sums in the workspace); and 256 x 256 tiles (16-bit
// outputs).
enum LinearF8Kind : int {
  F8_ROWS_NT1, F8_ROWS_NT2, F8_ROWS_NT4, F8_TILE_64X32, F8_TILE_64X32_K2, F8_TILE_64X64, F8_TILE_64X64_K2,
  F8_TILE_128X128, F8_TILE_128X128_K2, F8_TILE_256X256
};
constexpr int64_t kF8MaxThreads = 0xffffffff;   // of a launch (HIP counts them in 32 bits)
struct LinearF8Plan {
  LinearF8Kind kind;
  int splits;             // K splits (tiles below 256 x 256; 1: no partial sums)
};
hipError_t launch_linear_f8(const LinearF8Params&, const LinearF8Plan&, int out, hipStream_t);

// ------------------------------------------- around the experts, adapters --
constexpr int kRouteMaxExperts = 1024;
constexpr int kRouteMaxTopk = 64;
constexpr int kRouteMaxGroups = 64;
struct RouteParams {
  const void* logits;     // T x E, act
  const float* bias;      // E, or nullptr
  int32_t* experts;       // T x topk
  float* weights;         // T x topk
  int64_t T;
  int E, topk;
  int sigmoid;            // 0: softmax
  int groups;             // divides E
  int groups_shift;       // log2(groups), rounded up
  int topk_groups;
  int group_best;         // 1 or 2; 1 where there is one group
  int index_bits;         // of an expert's index
  int renormalize;
  float scale;
};
hipError_t launch_moe_route(const RouteParams&, int act, hipStream_t);

constexpr int kGroupChunkExperts = 900;   // 18 arrays of E + 2 in 64 KiB of LDS
constexpr int64_t kGroupAlone = 65536;    // slots that one launch without workspace sorts
constexpr int64_t kGroupOneByOne = int64_t(1) << 25;   // with more experts: slots x experts of a block an expert
// Slots of a block of group_rows' two launches.
constexpr int64_t group_chunk(int64_t S) { return S <= 128 * 1024 ? 1024 : 4096; }
struct GroupRowsParams {
  const void* ids;        // S = T x topk, int32 or int64
  int32_t* rows;          // S
  int32_t* offsets;       // E + 1
  int32_t* position;      // S, or nullptr
  int64_t S;              // at most 2^30
  int E;
  uint32_t topk_mul;      // s / topk == (s * topk_mul) >> topk_shift for 0 <= s < 2^30
  int topk_shift;
  // workspace, as GroupWorkspace has it, or nullptr
  int* counts;            // of each chunk; nullptr: one launch
  int* totals;            // of all chunks; nullptr: added up from the counts
  int32_t* order;         // S: slots by their id's low digit, and nullptr: one sort by whole ids
  int32_t* keys;          // S: the sorted ids
};
// What a call with a workspace uses, in bytes from its begin: one sort by whole ids or
// two by digits, and sums over the chunks taken ahead where there are many.
constexpr int kGroupDigits = 512;
struct GroupWorkspace {
  bool used, scanned, digits;
  size_t totals, order, keys, bytes;
};
constexpr GroupWorkspace group_workspace(int64_t S, int64_t E) {
  GroupWorkspace w{};
  w.digits = E > kGroupChunkExperts;
  w.used = w.digits ? S * E > kGroupOneByOne : S > kGroupAlone;
  if (!w.used) return w;
  const int64_t chunks = (S + group_chunk(S) - 1) / group_chunk(S), values = w.digits ? kGroupDigits : E + 1;
  w.scanned = w.digits || chunks > 512 || chunks * values > 32768;
  const auto whole = [](size_t bytes) { return (bytes + 255) / 256 * 256; };
  w.totals = static_cast<size_t>(chunks) * values * sizeof(int);
  w.bytes = w.totals;
  if (w.scanned) {
    w.totals = whole(w.totals);
    w.order = w.totals + whole(values * sizeof(int));
    w.keys = w.order + (w.digits ? whole(S * sizeof(int32_t)) : 0);
    w.bytes = w.keys + (w.digits ? S * sizeof(int32_t) : 0);
  }
  return w;
}
hipError_t launch_group_rows(const GroupRowsParams&, int id_bytes, hipStream_t);

struct CombineParams {
  const void* y;            // R x N, act
  const int32_t* position;  // T x topk rows of y
  const float* weights;     // T x topk
  const void* residual;     // T x N, act, or nullptr
  void* out;                // T x N, act (may be residual)
  int64_t R, T;
  int N, topk;
};
hipError_t launch_moe_combine(const CombineParams&, int act, hipStream_t);

constexpr int kLoraMaxRank = 256;
constexpr int kLoraMaxSplits = 8;
struct LoraParams {
  const void* x;            // M x K, act, 16-byte aligned
  const void* a;            // L x rank x K, act, 16-byte aligned
  const void* b;            // L x N x rank, act, 16-byte aligned
  const float* scales;      // L, or nullptr (ones)
  const int32_t* rows;      // T, or nullptr (T == M, position t is row t)
  const int32_t* offsets;   // L + 1
  const void* base;         // M x N, act, or nullptr (zeros)
  void* y;                  // M x N, act (may be base)
  float* t;                 // workspace: splits x T x rank_pad
  int64_t M, T;
  int L, N, K;              // K % 16 == 0
  int rank, rank_pad;       // rank % 8 == 0; rounded up to 16
  int splits, units_split;  // K ranges of the first product, in units of 128 bytes of a row
};
struct LoraPlan {
  bool fused;               // one launch (rank up to 32), no workspace
  bool many;                // two launches, of 32 rows a tile in the second (else 16)
  int shrink_rows;          // rows a tile in the first of two launches: 16, 64 or 128
  int cols;                 // columns of a block, a multiple of what its waves take at a time
};
hipError_t launch_lora(const LoraParams&, const LoraPlan&, int act, hipStream_t);

// ------------------------------------------------- library-owned scratch --
// Size of the device array behind lowbit_linear_noalloc (per device).  The
// largest K-split schedule of the MFMA path writes one fp32 partial per
// output of a block tile per block, at most (CUs) x (128 x 256) x 4 bytes =
// 32 MiB on a 256-CU device.
constexpr size_t kNoallocScratchBytes = size_t(32) << 20;
// Device address of this device's copy of the array (looked up once per
// device, with that device current).
hipError_t noalloc_scratch(void** out);
// Device address of this device's two status words of the quantizer (a
// second library-owned device array, looked up the same way).
hipError_t quant_status_words(int** out);

}  // namespace lowbit
