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
#include "pieces.h"

#include <algorithm>

namespace lowbit {

namespace {

// An id as an expert: E for one that is none.
__device__ __forceinline__ uint32_t expert_of(int32_t id, uint32_t E) {
  return min(static_cast<uint32_t>(id), E);              // (a negative one is large)
}
__device__ __forceinline__ uint32_t expert_of(int64_t id, uint32_t E) {
  return (static_cast<uint64_t>(id) >> 32) != 0 ? E : min(static_cast<uint32_t>(id), E);
}

}  // namespace

// Block e finds the slots of expert e by itself (block E: those of none): it
// reads all ids, which lie in cache, counts the smaller ones and its own, and
// then writes its own in order.  No block waits for another, nothing hangs on
// the order of atomics, and one launch does.  A wave takes runs of 64 steps of
// 64 slots; step i's own slots are a 64-bit mask that lane i keeps, so that the
// second pass costs a prefix sum and a turn for each bit of the fullest mask.
// (One run a wave where S allows it; otherwise the masks are made again.)
// Bound by a launch up to some 4096 slots (64 tokens of 8 in 64 experts: 3.1
// us, an empty launch 2.7), by every block's reading of all ids from there: taken
// up to 8192, and beyond for more experts than the chunks below count.  One wave
// up to 1024 slots, four to 8192 (us, 1 / 4 / 16 waves, 64 experts: 1024 slots 3.5
// / 4.3 / 5.5, 2048 4.2 / 4.3 / 5.5, 4096 5.4 / 4.0 / 5.6, 8192 12.5 / 4.7 / 5.7,
// 16384 23 / 6.1 / 5.3).
template <class ID, int WAVES>
__global__ __launch_bounds__(64 * WAVES) void group_rows_kernel(GroupRowsParams p) {
  __shared__ int s_below[WAVES], s_own[WAVES];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  constexpr int STEPS = 16;                  // asked for at once
  const uint32_t e = blockIdx.x, E = static_cast<uint32_t>(p.E);
  const int S = static_cast<int>(p.S);
  const int steps = (S + WAVES * 64 - 1) / (WAVES * 64);   // of a wave
  const int runs = (steps + 63) / 64;
  const int begin = wave * steps * 64;       // (may be past S: less than 2^30 + 2^10)

  int below = 0;
  uint64_t mask = 0;                         // of step `lane` of the run
  auto scan = [&](int run) {
    uint32_t lo = 0, hi = 0;
    const int last = min(steps, 64 * run + 64);
    const ID* ids = static_cast<const ID*>(p.ids);
    for (int i0 = 64 * run; i0 < last; i0 += STEPS) {
      const int s0 = begin + i0 * 64;
      ID v[STEPS];
      uint32_t x[STEPS];
      if (i0 + STEPS <= last && s0 + STEPS * 64 <= S) {
#pragma unroll
        for (int j = 0; j < STEPS; ++j) v[j] = ids[s0 + lane + j * 64];
#pragma unroll
        for (int j = 0; j < STEPS; ++j) x[j] = expert_of(v[j], E);
      } else {                               // past the wave's steps or the last slot: E + 1, no block's
#pragma unroll
        for (int j = 0; j < STEPS; ++j) v[j] = ids[min(s0 + lane + j * 64, S - 1)];
#pragma unroll
        for (int j = 0; j < STEPS; ++j)
          x[j] = i0 + j < last && s0 + lane + j * 64 < S ? expert_of(v[j], E) : E + 1;
      }
#pragma unroll
      for (int j = 0; j < STEPS; ++j) {
        below += __popcll(__ballot(x[j] < e));
        const uint64_t own = __ballot(x[j] == e);
        const bool keep = lane == ((i0 + j) & 63);
        lo = keep ? static_cast<uint32_t>(own) : lo;
        hi = keep ? static_cast<uint32_t>(own >> 32) : hi;
      }
    }
    mask = (static_cast<uint64_t>(hi) << 32) | lo;
  };
  int own = 0;                               // of this lane's masks
  for (int run = 0; run < runs; ++run) {
    scan(run);
    own += __popcll(mask);
  }
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) own += __shfl_xor(own, o);
  int first = below, at = below;
  if constexpr (WAVES > 1) {
    if (lane == 0) {
      s_below[wave] = below;
      s_own[wave] = own;
    }
    __syncthreads();
    first = at = 0;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) {
      first += s_below[w];
      at += w < wave ? s_own[w] : 0;
    }
    at += first;
  }
  if (threadIdx.x == 0) p.offsets[e] = first;

  for (int run = 0; run < runs; ++run) {
    if (runs > 1) scan(run);
    const int mine = __popcll(mask);
    int upto = mine;                         // inclusive prefix sum over the lanes
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int v = __shfl_up(upto, o);
      if (lane >= o) upto += v;
    }
    int to = at + upto - mine;
    at += __builtin_amdgcn_readlane(upto, 63);
    const int slot = begin + (64 * run + lane) * 64;
    for (; mask != 0; mask &= mask - 1) {
      const int s = slot + __builtin_ctzll(mask);
      p.rows[to] = static_cast<int>((static_cast<uint64_t>(s) * p.topk_mul) >> p.topk_shift);   // s / topk
      if (p.position) p.position[s] = e < E ? to : -1;
      ++to;
    }
  }
}

// For more slots, a chunk of 1024 STEPS of them a block: each chunk's places, from
// the counts of all chunks before it.  Up to 65536 slots every block counts all
// of them itself (bound by the LDS's atomic additions, some 8 us for 65536);
// beyond, a first launch counts each chunk into the workspace.  us, block an
// expert / one launch of chunks / two: 4096 slots, 256 experts 3.3 / 5.8 / 7.7;
// 16384 6.8 / 6.0 / 8.4; 32768 - / 7.7 / 9.7; 65536 14.1 / 11.2 / 9.1 (but an
// eager call takes 13 with two launches and a workspace); 131072 - / 18.5 /
// 11.0; 524288 141 / - / 17 (two empty launches are 4.9).  Chunks of 1024 slots
// up to 128 of them, of 4096 beyond (524288 slots 29 against 17): what a block
// adds up of the others' counts grows with their number.  Where that is more than
// 32768 of them, or past 512 chunks, a launch between the two turns the counts into
// those of the chunks before (us, without / with it: 64 experts, 2^20 slots 17 / 19,
// 2^21 32 / 31, 2^22 71 / 54; 256, 2^18 15.3 / 16.4, 2^19 18.0 / 17.4, 2^22 141 / 61;
// 900, 2^17 22.8 / 13.8, 2^20 42 / 26, 2^22 381 / 76).
//
// More experts than the LDS has counts for take two such sorts, by the low 9 bits of
// the id and then by the others, and their offsets from the sorted ids: seven
// launches, past 2^25 slots x experts (us, a block an expert / so: 1024 experts, 32768
// slots 22 / 26, 65536 35 / 28, 131072 92 / 30; 4096, 8192 slots 14 / 24, 16384 50 /
// 25, 131072 302 / 30; 65536, 1024 slots 26 / 21, 16384 701 / 26).
constexpr int kChunkWaves = 16;

enum : int { WHOLE, LOW, HIGH };             // the part of the id that a sort goes by
constexpr int kLowBits = 9;
static_assert(1 << kLowBits == kGroupDigits, "the low digit's values");
template <int PART> __device__ __forceinline__ uint32_t part_of(uint32_t x) {
  return PART == WHOLE ? x : PART == LOW ? x & (kGroupDigits - 1) : x >> kLowBits;
}
template <int PART> __host__ __device__ __forceinline__ int parts(int E) {      // how many values it has
  return PART == WHOLE ? E + 1 : PART == LOW ? kGroupDigits : (E >> kLowBits) + 1;
}
// The slot at place s of the sort before.
template <int PART> __device__ __forceinline__ int64_t slot_at(const GroupRowsParams& p, int64_t s) {
  return PART == HIGH ? p.order[s] : s;
}
// The part of the id at place s; past the last one, one more than there are.
template <class ID, int PART>
__device__ __forceinline__ uint32_t chunk_id(const GroupRowsParams& p, int64_t s) {
  if (s >= p.S) return parts<PART>(p.E);
  return part_of<PART>(expert_of(static_cast<const ID*>(p.ids)[slot_at<PART>(p, s)], static_cast<uint32_t>(p.E)));
}

// counts[x] += 1 for each lane's x.  (A wave of one id, as where all tokens go one
// way, would queue at its count.)
__device__ __forceinline__ void count_one(int* counts, uint32_t x) {
  const uint32_t one = __builtin_amdgcn_readfirstlane(x);
  if (__ballot(x == one) == ~uint64_t{0}) {
    if ((threadIdx.x & 63) == 0) atomicAdd(&counts[one], 64);
  } else {
    atomicAdd(&counts[x], 1);
  }
}

template <class ID, int STEPS, int PART>
__global__ __launch_bounds__(64 * kChunkWaves) void group_count_kernel(GroupRowsParams p) {
  extern __shared__ int s_count[];           // the parts, past the last slot
  const int values = parts<PART>(p.E);
  for (int e = threadIdx.x; e <= values; e += blockDim.x) s_count[e] = 0;
  __syncthreads();
  const int64_t begin = static_cast<int64_t>(blockIdx.x) * (1024 * STEPS);
  uint32_t x[STEPS];
#pragma unroll
  for (int i = 0; i < STEPS; ++i) x[i] = chunk_id<ID, PART>(p, begin + i * 64 * kChunkWaves + threadIdx.x);
#pragma unroll
  for (int i = 0; i < STEPS; ++i) {
    count_one(s_count, x[i]);
  }
  __syncthreads();
  int* to = p.counts + static_cast<size_t>(blockIdx.x) * values;
  for (int e = threadIdx.x; e < values; e += blockDim.x) to[e] = s_count[e];
}

// Each chunk's counts become those of the chunks before it, and their sums over all
// chunks go to p.totals: 64 values a block, whose waves share the chunks.
__global__ __launch_bounds__(64 * kChunkWaves) void group_scan_kernel(GroupRowsParams p, int values, int chunks) {
  __shared__ int s_sum[kChunkWaves][64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int e = static_cast<int>(blockIdx.x) * 64 + lane;
  const int each = (chunks + kChunkWaves - 1) / kChunkWaves;
  const int first = min(wave * each, chunks), last = min(first + each, chunks);
  int* counts = p.counts + e;
  int sum = 0;
  if (e < values) {
#pragma unroll 8
    for (int c = first; c < last; ++c) sum += counts[static_cast<size_t>(c) * values];
  }
  s_sum[wave][lane] = sum;
  __syncthreads();
  if (e >= values) return;
  int before = 0;
  for (int w = 0; w < wave; ++w) before += s_sum[w][lane];
  if (wave == kChunkWaves - 1) p.totals[e] = before + sum;
  for (int c0 = first; c0 < last; c0 += 8) {
    int v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = c0 + i < last ? counts[static_cast<size_t>(c0 + i) * values] : 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (c0 + i < last) counts[static_cast<size_t>(c0 + i) * values] = before;
      before += v[i];
    }
  }
}

// Four ids from slot s on, as experts (E + 1 past the last slot).
template <class ID>
__device__ __forceinline__ void load_four(const GroupRowsParams& p, int s, uint32_t (&x)[4]) {
  const uint32_t E = static_cast<uint32_t>(p.E);
  struct __attribute__((packed, aligned(sizeof(ID)))) Four { ID v[4]; };
  const ID* from = static_cast<const ID*>(p.ids) + s;
  if (s + 4 <= p.S) {
    const Four f = *reinterpret_cast<const Four*>(from);
#pragma unroll
    for (int q = 0; q < 4; ++q) x[q] = expert_of(f.v[q], E);
  } else {
#pragma unroll
    for (int q = 0; q < 4; ++q) x[q] = s + q < p.S ? expert_of(from[q], E) : E + 1;
  }
}

// ALONE: in one launch, each block counting all slots itself; SUM: from all chunks'
// counts; SCANNED: from the counts before its own.
enum : int { ALONE, SUM, SCANNED };
template <class ID, int STEPS, int FROM, int PART>
__global__ __launch_bounds__(64 * kChunkWaves) void group_place_kernel(GroupRowsParams p, int chunks, int bits) {
  extern __shared__ int s_mem[];
  const int values = parts<PART>(p.E), ids = values + 1;
  int* s_all = s_mem;                        // [ids] an id's slots in all chunks
  int* s_base = s_mem + ids;                 // [ids] in the chunks before this one, then its first place here
  int* s_wave = s_mem + 2 * ids;             // [kChunkWaves][ids] its slots by wave, then those of the waves before
  __shared__ int s_part[kChunkWaves];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t E = static_cast<uint32_t>(p.E);
  const int64_t begin = static_cast<int64_t>(blockIdx.x) * (1024 * STEPS) + wave * (64 * STEPS);
  uint32_t x[STEPS];
#pragma unroll
  for (int i = 0; i < STEPS; ++i) x[i] = chunk_id<ID, PART>(p, begin + i * 64 + lane);
  for (int i = threadIdx.x; i < (2 + kChunkWaves) * ids; i += blockDim.x) s_mem[i] = 0;
  __syncthreads();
  if constexpr (FROM == ALONE) {
    const int here = static_cast<int>(blockIdx.x) * (1024 * STEPS), S = static_cast<int>(p.S);
#pragma unroll 1
    for (int s0 = 0; s0 < S; s0 += 4 * 4096) {
      uint32_t v[4][4];
#pragma unroll
      for (int r = 0; r < 4; ++r) load_four<ID>(p, min(s0 + 4096 * r + 4 * static_cast<int>(threadIdx.x), S), v[r]);
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        // (a chunk begins at a multiple of 1024: a lane's four are all before it or none)
        int* to = s0 + 4096 * r + 4 * static_cast<int>(threadIdx.x) < here ? s_base : s_all;
#pragma unroll
        for (int q = 0; q < 4; ++q) count_one(to, v[r][q]);
      }
    }
    __syncthreads();
    for (int e = threadIdx.x; e <= p.E; e += blockDim.x) s_all[e] += s_base[e];
  } else if constexpr (FROM == SCANNED) {
    for (int e = threadIdx.x; e < values; e += blockDim.x) {
      s_all[e] = p.totals[e];
      s_base[e] = p.counts[static_cast<size_t>(blockIdx.x) * values + e];
    }
  } else {
    for (int e = lane; e < values; e += 64) {  // the waves take the chunks in turn
      int before = 0, all = 0;
      const int* from = p.counts + e;
#pragma unroll 4
      for (int c = wave; c < chunks; c += kChunkWaves) {
        const int v = from[static_cast<size_t>(c) * values];
        all += v;
        before += c < static_cast<int>(blockIdx.x) ? v : 0;
      }
      if (all != 0) atomicAdd(&s_all[e], all);
      if (before != 0) atomicAdd(&s_base[e], before);
    }
  }
  __syncthreads();
  int carry = 0;
  for (int e0 = 0; e0 < values; e0 += 64 * kChunkWaves) {
    const int e = e0 + static_cast<int>(threadIdx.x);
    const int all = e < values ? s_all[e] : 0;
    int upto = all;                          // inclusive prefix sum over the lanes
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int v = __shfl_up(upto, o);
      if (lane >= o) upto += v;
    }
    if (e0 > 0) __syncthreads();             // (s_part's last round is read)
    if (lane == 63) s_part[wave] = upto;
    __syncthreads();
    int less = carry;
#pragma unroll
    for (int w = 0; w < kChunkWaves; ++w) {
      less += w < wave ? s_part[w] : 0;
      carry += s_part[w];
    }
    if (e < values) {
      const int first = less + upto - all;
      s_base[e] += first;
      if (PART == WHOLE && blockIdx.x == 0) p.offsets[e] = first;
    }
  }

  // each slot's rank among the wave's slots of its id, step after step
  int* mine = s_wave + wave * ids;
  int rank[STEPS];
#pragma unroll
  for (int i = 0; i < STEPS; ++i) {
    uint64_t same = ~uint64_t{0};            // lanes with this lane's id
    for (int b = 0; b < bits; ++b) {
      const bool bit = (x[i] >> b) & 1;
      const uint64_t set = __ballot(bit);
      same &= bit ? set : ~set;
    }
    const int lower = __popcll(same & ((uint64_t{1} << lane) - 1));
    rank[i] = mine[x[i]] + lower;
    __builtin_amdgcn_wave_barrier();
    if (lower == 0) mine[x[i]] = rank[i] + __popcll(same);
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
  }
  __syncthreads();
  for (int e = threadIdx.x; e < values; e += blockDim.x) {
    int sum = 0;
#pragma unroll
    for (int w = 0; w < kChunkWaves; ++w) {
      const int v = s_wave[w * ids + e];
      s_wave[w * ids + e] = sum;
      sum += v;
    }
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < STEPS; ++i) {
    const int64_t s = begin + i * 64 + lane;
    if (s >= p.S) continue;
    const int to = s_base[x[i]] + mine[x[i]] + rank[i];
    if constexpr (PART == LOW) {
      p.order[to] = static_cast<int32_t>(s);
    } else {
      const int64_t slot = slot_at<PART>(p, s);
      const uint32_t id = PART == WHOLE ? x[i] : expert_of(static_cast<const ID*>(p.ids)[slot], E);
      p.rows[to] = static_cast<int>((static_cast<uint64_t>(slot) * p.topk_mul) >> p.topk_shift);
      if (p.position) p.position[slot] = id < E ? to : -1;
      if constexpr (PART == HIGH) p.keys[to] = static_cast<int32_t>(id);
    }
  }
}

// Where each expert's begin among the sorted ids: the first that is not below it.
__global__ __launch_bounds__(256) void group_bounds_kernel(GroupRowsParams p) {
  const int e = static_cast<int>(blockIdx.x * 256 + threadIdx.x);
  if (e > p.E) return;
  int lo = 0, hi = static_cast<int>(p.S);
  while (lo < hi) {
    const int at = lo + (hi - lo) / 2;
    if (p.keys[at] < e) lo = at + 1;
    else hi = at;
  }
  p.offsets[e] = lo;
}

namespace {

constexpr int bits_of(int values) {          // of the numbers 0 .. values
  int bits = 1;
  while ((1 << bits) < values + 1) ++bits;
  return bits;
}
template <class ID, int STEPS, int PART>
void launch_sort(const GroupRowsParams& p, bool scanned, hipStream_t stream) {
  const int chunks = static_cast<int>((p.S + 1024 * STEPS - 1) / (1024 * STEPS)), threads = 64 * kChunkWaves;
  const int values = parts<PART>(p.E), bits = bits_of(values);
  const size_t row = (values + 1) * sizeof(int);
  group_count_kernel<ID, STEPS, PART><<<chunks, threads, row, stream>>>(p);
  if (scanned) {
    group_scan_kernel<<<(values + 63) / 64, threads, 0, stream>>>(p, values, chunks);
    group_place_kernel<ID, STEPS, SCANNED, PART><<<chunks, threads, (kChunkWaves + 2) * row, stream>>>(p, chunks, bits);
  } else {
    group_place_kernel<ID, STEPS, SUM, PART><<<chunks, threads, (kChunkWaves + 2) * row, stream>>>(p, chunks, bits);
  }
}
template <class ID, int STEPS>
void launch_chunks_as(const GroupRowsParams& p, hipStream_t stream) {
  const bool scanned = p.totals != nullptr;
  if (p.order == nullptr) {
    launch_sort<ID, STEPS, WHOLE>(p, scanned, stream);
  } else {
    launch_sort<ID, STEPS, LOW>(p, scanned, stream);
    launch_sort<ID, STEPS, HIGH>(p, scanned, stream);
    group_bounds_kernel<<<p.E / 256 + 1, 256, 0, stream>>>(p);
  }
}
template <class ID>
void launch_group_as(const GroupRowsParams& p, hipStream_t stream) {
  const dim3 grid(static_cast<unsigned>(p.E + 1));
  if (p.counts) {
    if (group_chunk(p.S) == 1024) launch_chunks_as<ID, 1>(p, stream);
    else launch_chunks_as<ID, 4>(p, stream);
  } else if (p.S <= 1024) {
    group_rows_kernel<ID, 1><<<grid, 64, 0, stream>>>(p);
  } else if (p.S <= 8192) {
    group_rows_kernel<ID, 4><<<grid, 256, 0, stream>>>(p);
  } else if (p.S <= kGroupAlone && p.E <= kGroupChunkExperts) {
    const int chunks = static_cast<int>((p.S + 1023) / 1024);
    const size_t lds = (kChunkWaves + 2) * (p.E + 2) * sizeof(int);
    group_place_kernel<ID, 1, ALONE, WHOLE><<<chunks, 64 * kChunkWaves, lds, stream>>>(p, chunks, bits_of(p.E + 1));
  } else {
    group_rows_kernel<ID, 16><<<grid, 1024, 0, stream>>>(p);
  }
}

}  // namespace

hipError_t launch_group_rows(const GroupRowsParams& p, int id_bytes, hipStream_t stream) {
  if (id_bytes == 8) launch_group_as<int64_t>(p, stream);
  else launch_group_as<int32_t>(p, stream);
  return hipGetLastError();
}

// LX lanes a row, eight columns each (LX < 256: 256 / LX rows a block; wider
// rows: several blocks).  The rows of eight slots are all asked for before the
// first is used, each as whole 16-byte pieces; what is written goes past the
// caches, what is read does not (rows may be there still: loads past the caches
// 11.4 us where these take 8.2).  Bound by memory: each row once in, each sum once
// out (8192 tokens x 8 rows of 2048 bf16, 302 MB: 45 us with rows just written, 57
// without, 5.3 TB/s; 1500 x 4 x 2003 fp16, no row on 16 bytes: 8.2 us).
// The fewest lanes that hold a row, 64 from there on and 256 for rows of several
// blocks (us, 8 / 16 / 32 / 64 / 256 lanes, 8192 tokens of 8, bf16: N = 64 4.7 /
// 4.8 / 5.9 / 7.5 / 9.9, 128 6.0 / 5.9 / 6.7 / 7.7 / 10.4, 256 9.8 / 9.7 / 9.6 /
// 9.7 / 10.9, 512 17.0 / 16.7 / 16.5 / 13.8 / 14.5, 1024 31 / 30 / 29 / 24.4 / 24.9,
// 2048 76 / 67 / 65 / 55.4 / 56.2; one token 0.2 to 0.5 more with 8 to 32 lanes:
// N = 64 3.8 / 3.9 / 3.7 / 3.4 / 3.5, 4096 4.1 / 4.1 / 4.1 / 3.5 / 3.7).
constexpr int kCombineThreads = 256;

template <int ACT, int LX>
__global__ __launch_bounds__(kCombineThreads) void moe_combine_kernel(CombineParams p, int runs) {
  typedef typename Act<ACT>::bits_t T;
  const unsigned block = blockIdx.x / static_cast<unsigned>(runs);
  const int run = static_cast<int>(blockIdx.x - block * static_cast<unsigned>(runs));
  int row_of_block = static_cast<int>(threadIdx.x) / LX;
  if constexpr (LX >= 64) row_of_block = __builtin_amdgcn_readfirstlane(row_of_block);   // positions: scalar loads
  const int64_t t = static_cast<int64_t>(block) * (kCombineThreads / LX) + row_of_block;
  const int n = (run * LX + static_cast<int>(threadIdx.x) % LX) * 8, left = p.N - n;
  if (t >= p.T || left <= 0) return;
  const T* y = static_cast<const T*>(p.y) + n;
  const int32_t* position = p.position + t * p.topk;
  const float* weights = p.weights + t * p.topk;
  Piece<ACT> residual;
  if (p.residual) load_piece<ACT>(static_cast<const T*>(p.residual) + t * p.N + n, left, residual);

  float part[4][8] = {};
  for (int j0 = 0; j0 < p.topk; j0 += 8) {
    Piece<ACT> v[8];
    int64_t at[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) at[q] = j0 + q < p.topk ? position[j0 + q] : -1;
#pragma unroll
    for (int q = 0; q < 8; ++q)
      if (at[q] >= 0 && at[q] < p.R) load_piece<ACT>(y + at[q] * p.N, left, v[q]);
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      if (at[q] < 0) continue;
      const float w = at[q] < p.R ? weights[j0 + q] : __builtin_nanf("");
      float f[8];
      piece_to_float<ACT>(v[q], f);
#pragma unroll
      for (int i = 0; i < 8; ++i) part[q & 3][i] += w * f[i];
    }
  }
  float sum[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) sum[i] = ((part[0][i] + part[1][i]) + part[2][i]) + part[3][i];
  if (p.residual) {
    float f[8];
    piece_to_float<ACT>(residual, f);
#pragma unroll
    for (int i = 0; i < 8; ++i) sum[i] += f[i];
  }
  store_piece<ACT>(static_cast<T*>(p.out) + t * p.N + n, left, sum);
}

namespace {

template <int ACT, int LX>
void launch_combine_rows(const CombineParams& p, int pieces, hipStream_t stream) {
  typedef typename Act<ACT>::bits_t T;
  const int runs = (pieces + LX - 1) / LX;
  constexpr int ROWS = kCombineThreads / LX;
  const int64_t most = kF8MaxThreads / kCombineThreads / runs * ROWS;        // of a launch
  for (int64_t t = 0; t < p.T; t += most) {
    CombineParams q = p;
    q.T = std::min(p.T - t, most);
    q.position += t * p.topk;
    q.weights += t * p.topk;
    q.out = static_cast<T*>(p.out) + t * p.N;
    if (p.residual) q.residual = static_cast<const T*>(p.residual) + t * p.N;
    moe_combine_kernel<ACT, LX><<<static_cast<unsigned>((q.T + ROWS - 1) / ROWS * runs), kCombineThreads, 0, stream>>>(q, runs);
  }
}
template <int ACT>
void launch_combine_as(const CombineParams& p, hipStream_t stream) {
  const int pieces = (p.N + 7) / 8;
  if (pieces <= 8) launch_combine_rows<ACT, 8>(p, pieces, stream);
  else if (pieces <= 16) launch_combine_rows<ACT, 16>(p, pieces, stream);
  else if (pieces <= 32) launch_combine_rows<ACT, 32>(p, pieces, stream);
  else if (pieces <= 128) launch_combine_rows<ACT, 64>(p, pieces, stream);
  else launch_combine_rows<ACT, 256>(p, pieces, stream);
}

}  // namespace

hipError_t launch_moe_combine(const CombineParams& p, int act, hipStream_t stream) {
  switch (act) {
    case ACT_F32: launch_combine_as<ACT_F32>(p, stream); break;
    case ACT_F16: launch_combine_as<ACT_F16>(p, stream); break;
    default: launch_combine_as<ACT_BF16>(p, stream); break;
  }
  return hipGetLastError();
}

}  // namespace lowbit
