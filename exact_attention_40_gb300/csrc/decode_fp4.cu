// One-token paged decode over the 4-bit cache (layout in fp4.cuh) for sm_103a:
// split-KV partial attention plus a log-sum-exp merge, as the bf16 decode.
//
// decode_fp4_split_kernel: the work is units of 8 blocks (128 tokens) of one
//   (sequence, kv head, chunk of up to 8 NT query heads), its segment, numbered
//   through all segments in order.  Each CTA takes an equal, contiguous share of
//   them, so that the longest sequence of a ragged batch holds nobody up and one
//   wave of CTAs is enough; it finds its share from ctx_lens itself, so a
//   captured graph follows their contents.  One warp copies: units in order into
//   a ring in shared memory, one bulk copy for each block's span (18 d bytes:
//   codes and scales of keys and values), across segments.  Four warps compute,
//   two blocks of a unit each.  At a segment's end their states merge; a segment
//   that lies in one CTA is written to the output, any other leaves partial
//   outputs, at most two a CTA.
//   Everything is computed transposed, so that the 16 tokens of a block are
//   the rows of mma.sync m16n8k16 and the few query heads of the group its 8
//   columns (as rows, half or more of them would be padding):
//     S^T = K Q^T   A = keys [16 tokens x 16 columns], B = queries;
//     O^T += V^T P^T  A = values [16 columns x 16 tokens], B = weights.
//   Codes become fp16 by the cvt of packed e2m1 and are multiplied by their
//   scale there; the product has 6 significant bits, so keys and values enter
//   the tensor core exactly.  Queries are bf16: each is multiplied by a power of
//   two that brings its largest element to [1, 2), after which fp16 holds its
//   elements exactly down to 2^-17 and within 2^-25 below, and the power goes
//   into the score's factor.  Both products sum over their inner index
//   in any order, so which column or token an mma index stands for is free: it
//   is chosen so that a lane reads its codes as one vector each, from one or two
//   scale groups.  Weights are rounded to fp16 for the second product.  They are
//   taken 2^7 times as large as the softmax's, so that their largest lies between 2^7
//   and 2^15: fp16 then rounds those above 2^-21 of the reference by at most 2^-11
//   relative (the output is rounded to bf16, 2^-8), the smaller ones by at most
//   2^-32 of the reference, which many tokens beside one that dominates do not add up
//   to anything.  Their sums are fp32 and take them unrounded (a second sum, of the
//   rounded weights, cost 1 to 2% of the time).
//   What bounds it at d = 128 with up to 8 heads: conversions and the multiplications
//   by the scales, which share a pipe (4 + 4 of them and one mma take 15 cycles of an
//   SM's quarter, each of the three alone 8), then DRAM.  64 sequences of 8192 tokens,
//   32 heads over 8 of 128: 106.4 us = 5.68 TB/s; the copies alone take 94.  64 sequences
//   of 512 to 8192 tokens with the merge 62.7 us = 5.13 TB/s.  At d = 64 (64 heads over 8,
//   the same lengths: 44.8 us = 3.59 TB/s) and with 16 rows (32 sequences, 96 heads over
//   8: 54.3 us = 2.97 TB/s) no unit is full: the chain of products, vote, exponentials,
//   transposes and products of few warps is what takes the time.
//   Small calls (few segments, none long) take a cluster of 8 CTAs for each
//   segment instead, which take its units in turn and merge through distributed
//   shared memory: one launch and no workspace (six of up to 1500 tokens 3.9 us).
// decode_fp4_combine_kernel: merges the partial outputs of a segment.
#include <cuda_bf16.h>

#include <type_traits>

#include "fp4.cuh"
#include "launch.h"
#include "ptx.cuh"

namespace exattn {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;       // that compute; one warp more copies
constexpr int kCtaThreads = kThreads + 32;
constexpr int kMergeThreads = 256;
constexpr int kStages = 3;  // units in flight
constexpr int kBlk = kDecodeBlockSize;
constexpr int kUnit = kFp4UnitBlocks;
static_assert(kUnit == 2 * kWarps, "a pair of blocks per warp");
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.69314718055994531f;
constexpr int kWhole = static_cast<int>(0x80000000u);
constexpr float kNoScore = -3.0e38f;     // below any score; -inf would give inf - inf
// Weights are 2^(score - reference), the reference kLift below the running maximum that it
// was taken from, and a new one taken once a score passes it by more than kMost: fp16
// holds weights of up to 2^15.
constexpr float kLift = 7.f;
constexpr float kMost = 15.f;

struct Fp4SplitParams {
  const __nv_bfloat16* q;
  const uint8_t* cache;
  const int32_t* block_table;
  const int32_t* ctx_lens;
  Fp4Joint* joints;  // one per CTA: its last segment, where others go on with it; or NULL
  float* ws_o;    // [2 * ctas][rows][d]
  float* ws_lse;  // [2 * ctas][rows]
  __nv_bfloat16* out;
  float* lse;
  unsigned int* status;
  unsigned long long wait_ns;
  int num_seqs, Hq, Hkv, group, n_chunks, num_blocks, max_blocks_per_seq;
  float scale_log2;       // scale * k_scale * log2 e
  float v_scale;
};

__device__ __forceinline__ int clamp_ctx(int n, int max_ctx, unsigned int* status) {
  if (n < 0 || n > max_ctx) {
    atomicOr(status, 2u);  // EXATTN_DEVICE_BOUNDS_BIT
    n = n < 0 ? 0 : max_ctx;
  }
  return n;
}

__device__ __forceinline__ void mma_f16_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The same product without a sum before it.
__device__ __forceinline__ void mma_f16_16816_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                                    uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%10, %10, %10, %10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

// Transposes an 8x8 matrix of 16-bit elements held one row per four lanes.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// c0, c1 times f[0], f[1], rounded, and their distances x0, x1 from m[0], m[1].  (Packed,
// so that the products cost no more than the one fused operation for each score.)
__device__ __forceinline__ void scores_and_distances(float& c0, float& c1, const float (&f)[2], const float (&m)[2],
                                                     float& x0, float& x1) {
  const uint64_t p = f2_mul(f2_pack(c0, c1), f2_pack(f[0], f[1]));
  f2_unpack(p, c0, c1);
  f2_unpack(f2_sub(p, f2_pack(m[0], m[1])), x0, x1);
}

// Loads from shared memory at addr + kOff (the offset is part of the instruction).
template <int kOff, int W>
__device__ __forceinline__ void lds_words(uint32_t addr, uint32_t (&w)[W]) {
  if constexpr (W == 4) {
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4 + %5];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                 : "r"(addr), "n"(kOff));
  } else if constexpr (W == 2) {
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2 + %3];" : "=r"(w[0]), "=r"(w[1]) : "r"(addr), "n"(kOff));
  } else {
    asm volatile("ld.shared.b32 %0, [%1 + %2];" : "=r"(w[0]) : "r"(addr), "n"(kOff));
  }
}

template <int kOff>
__device__ __forceinline__ uint32_t lds_u8(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.u8 %0, [%1 + %2];" : "=r"(v) : "r"(addr), "n"(kOff));
  return v;
}

template <int kOff>
__device__ __forceinline__ uint32_t lds_u16(uint32_t addr) {
  uint32_t v;
  asm volatile("{\n\t.reg .u16 h;\n\tld.shared.u16 h, [%1 + %2];\n\tcvt.u32.u16 %0, h;\n\t}"
               : "=r"(v)
               : "r"(addr), "n"(kOff));
  return v;
}

template <int D, int NT>
struct Fp4Smem {
  static constexpr int kAccStride = D + 4;  // row of the merge staging, floats
  alignas(128) uint8_t ring[kStages][kUnit][Fp4Span<D>::kBytes];
  float acc[kWarps][8 * NT][kAccStride];
  uint64_t full[kStages];        // a unit's copies have landed
  uint64_t empty[kStages];       // the four warps have used it
  int present[kStages];          // bits of its blocks that were copied, kWhole where all are and are full
  float wm[2][kWarps][8 * NT];   // per-warp reference (log2 units)
  float wl[2][kWarps][8 * NT];   // per-warp sum of the weights
};

// Waits for the computing warps of the CTA.
__device__ __forceinline__ void compute_barrier() {
  __syncwarp();
  asm volatile("bar.sync 1, %0;" ::"n"(kThreads) : "memory");
}

// Equal contiguous shares of `total` places for `parts` CTAs, the first
// total % parts of them one larger.  (The host keeps totals below 2^31.)
struct Shares {
  int base, extra, parts;
  __device__ __forceinline__ Shares(int total, int n) : base(total / n), extra(total % n), parts(n) {}
  __device__ __forceinline__ int begin(int c) const { return c * base + min(c, extra); }
  __device__ __forceinline__ int owner(int place) const {
    const int large = extra * (base + 1);
    const int c = place < large ? place / (base + 1) : extra + (place - large) / max(1, base);
    return max(0, min(parts - 1, c));
  }
};

// A place in the numbering of all segments: unit k of `units` of segment (seq, head,
// chunk), or (k == units) the place that stands for the segment's end.
struct Place {
  int seq, head, chunk, k, units, ctx;
};

__device__ __forceinline__ int units_of(int ctx) { return (ctx + kUnit * kBlk - 1) / (kUnit * kBlk); }

// Places of a segment: its units and one for its end, whose merge and change of
// queries take a CTA 2400 cycles, about what a unit does (2100).  (With units alone the
// CTAs that got the short sequences of a batch were the last to finish: 128 sequences
// of 1 to 2000 tokens took 45.8 us, 38.4 with the ends counted.)
__device__ __forceinline__ int places_of(int ctx) { return units_of(ctx) + (ctx > 0 ? 1 : 0); }

// Sums over the sequences that a warp forms from ctx_lens, each lane holding those of a
// contiguous range of them.  In a large batch the warp reads 32 neighbours together: with
// every lane reading its own range, no two of a load's addresses share a line, and 4096
// sequences took each CTA 40 us before its first copy.  (Lengths are read more than
// once; if another stream changes them meanwhile the result is undefined, but every
// place that comes out is clamped to one that exists.)
struct Batch {
  const int32_t* ctx_lens;
  int max_ctx, num_seqs;
  int range;                     // sequences per lane; a multiple of 32 where the warp reads them together
  int lane_begin, before, mine;  // this lane's first sequence, the places before it, in its range
  int first_ctx;                 // of its first sequence (small batches)
  int per_segment;               // places of all sequences (of one segment of each)

  static constexpr int kAlone = 4;  // longest range that a lane reads by itself

  // Clamped without a word: whoever handles the sequence reports it.
  __device__ __forceinline__ int ctx_of(int s) const { return max(0, min(max_ctx, __ldg(ctx_lens + s))); }
  __device__ __forceinline__ int places_at(int s, int end) const { return s < end ? places_of(ctx_of(s)) : 0; }

  __device__ __forceinline__ Batch(const int32_t* lens, int seqs, int longest) {
    ctx_lens = lens;
    num_seqs = seqs;
    max_ctx = longest;
    const int lane = threadIdx.x & 31;
    const bool alone = seqs <= 32 * kAlone;
    range = alone ? (seqs + 31) / 32 : (seqs + 1023) / 1024 * 32;
    lane_begin = min(seqs, lane * range);
    first_ctx = mine = 0;
    if (alone) {
      const int end = min(seqs, lane_begin + range);
      if (lane_begin < end) first_ctx = ctx_of(lane_begin);
      mine = places_of(first_ctx);
#pragma unroll
      for (int i = 1; i < kAlone; ++i) mine += places_at(lane_begin + i, end);
    } else {
      const int groups = (seqs + 31) / 32, per_lane = range / 32;
      int owner = 0, left = per_lane;
#pragma unroll 8
      for (int i = 0; i < groups; ++i) {
        const int sum = __reduce_add_sync(0xffffffffu, places_at(32 * i + lane, seqs));
        if (lane == owner) mine += sum;
        if (--left == 0) {
          left = per_lane;
          ++owner;
        }
      }
    }
    int upto = mine;  // inclusive sum over the lanes
#pragma unroll
    for (int x = 1; x < 32; x *= 2) {
      const int v = __shfl_up_sync(0xffffffffu, upto, x);
      if (lane >= x) upto += v;
    }
    per_segment = __shfl_sync(0xffffffffu, upto, 31);
    before = upto - mine;
  }

  // The unit or end at a place (below per_segment * segs); whole warp, same place.
  __device__ __forceinline__ Place find(int place, int segs, int n_chunks) const {
    const int target = place / segs;
    const unsigned int owners = __ballot_sync(0xffffffffu, before <= target && target < before + mine);
    const int lane = max(0, __ffs(owners) - 1);
    Place p;
    int prefix;
    if (num_seqs <= 32 * kAlone) {
      int s = lane_begin, ctx = first_ctx;
      prefix = before;
      if ((threadIdx.x & 31) == lane)
        while (target >= prefix + places_of(ctx) && s + 1 < num_seqs) {
          prefix += places_of(ctx);
          ctx = ctx_of(++s);
        }
      p.seq = min(num_seqs - 1, __shfl_sync(0xffffffffu, s, lane));
      p.ctx = __shfl_sync(0xffffffffu, ctx, lane);
      prefix = __shfl_sync(0xffffffffu, prefix, lane);
    } else {
      const int end = min(num_seqs, (lane + 1) * range);
      int base = lane * range;
      prefix = __shfl_sync(0xffffffffu, before, lane);
      while (true) {  // 32 sequences at a time; one of the range has the place
        const int n = places_at(base + (threadIdx.x & 31), end);
        int upto = n;
#pragma unroll
        for (int x = 1; x < 32; x *= 2) {
          const int v = __shfl_up_sync(0xffffffffu, upto, x);
          if ((threadIdx.x & 31) >= x) upto += v;
        }
        const unsigned int past = __ballot_sync(0xffffffffu, target < prefix + upto);
        if (past != 0 || base + 32 >= end) {
          const int at = past != 0 ? __ffs(past) - 1 : 0;
          prefix += __shfl_sync(0xffffffffu, upto - n, at);
          p.seq = min(num_seqs - 1, base + at);
          break;
        }
        prefix += __shfl_sync(0xffffffffu, upto, 31);
        base += 32;
      }
      p.ctx = ctx_of(p.seq);
    }
    p.units = max(1, units_of(p.ctx));
    const int rest = max(0, place - prefix * segs);
    const int y = min(segs - 1, rest / (p.units + 1));
    p.k = min(p.units, rest - y * (p.units + 1));
    p.head = n_chunks == 1 ? y : y / n_chunks;
    p.chunk = y - p.head * n_chunks;
    return p;
  }

  // The places before a sequence, per segment; whole warp, same s.
  __device__ __forceinline__ int before_seq(int s) const {
    const int lane = s / range;
    int prefix = before, ctx = first_ctx;
    if (num_seqs <= 32 * kAlone) {
      if ((threadIdx.x & 31) == lane)
        for (int i = lane_begin; i < s; ctx = ctx_of(++i)) prefix += places_of(ctx);
      return __shfl_sync(0xffffffffu, prefix, lane);
    }
    int sum = 0;
    for (int i = lane * range + (threadIdx.x & 31); i < s; i += 32) sum += places_of(ctx_of(i));
    return __shfl_sync(0xffffffffu, prefix, lane) + __reduce_add_sync(0xffffffffu, sum);
  }
};

// Waits for every thread of the cluster; shared memory written before is seen after.
// Not the .aligned form: that needs the warp's lanes together, and after a loop
// that some of them left early nothing says they are.
__device__ __forceinline__ void cluster_barrier() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}

// Loads from the shared memory of the cluster's CTA `rank`, at an address of one's own.
__device__ __forceinline__ float4 cluster_load4(const void* own, uint32_t rank) {
  float4 v;
  asm volatile(
      "{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %4, %5;\n\t"
      "ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [a];\n\t}"
      : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
      : "r"(smem_u32(own)), "r"(rank)
      : "memory");
  return v;
}

__device__ __forceinline__ float cluster_load(const void* own, uint32_t rank) {
  float v;
  asm volatile("{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %1, %2;\n\tld.shared::cluster.f32 %0, [a];\n\t}"
               : "=f"(v)
               : "r"(smem_u32(own)), "r"(rank)
               : "memory");
  return v;
}

template <int D, int NT, bool kCluster>
__global__ void __launch_bounds__(kCtaThreads, fp4_decode_ctas(8 * NT)) decode_fp4_split_kernel(const Fp4SplitParams p) {
  using Span = Fp4Span<D>;
  using Smem = Fp4Smem<D, NT>;
  constexpr int kRows = 8 * NT;      // query heads per CTA
  constexpr int kKSteps = D / 16;    // mma steps of S^T
  constexpr int kMTiles = D / 16;    // mma row tiles of O^T
  constexpr int kKeyWords = D / 32;  // 32-bit words of a lane's key codes per token
  constexpr int kValWords = D / 64;  // ... value codes
  constexpr int kStep = kCluster ? kFp4ClusterCtas : 1;  // from a CTA's unit to its next

  extern __shared__ uint8_t smem_raw[];
  Smem& sm = *reinterpret_cast<Smem*>((reinterpret_cast<uintptr_t>(smem_raw) + 127) & ~static_cast<uintptr_t>(127));

  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);  // (the same in all lanes, for the compiler too)
  const int lane = threadIdx.x & 31;
  const int g = lane >> 2;  // mma group: rows g, g + 8 of A and the accumulator, column g of B
  const int t = lane & 3;   // thread in group
  const int cta = blockIdx.x;
  const int segs = p.Hkv * p.n_chunks;  // segments of a sequence

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&sm.full[s], kUnit);
      mbar_init(&sm.empty[s], kWarps);
    }
    fence_mbar_init();
  }
  cudaGridDependencySynchronize();
  cudaTriggerProgrammaticLaunchCompletion();  // the merge may launch and wait while this runs
  const int max_ctx = p.max_blocks_per_seq * kBlk;
  auto ctx_of = [&](int s) { return clamp_ctx(__ldg(p.ctx_lens + s), max_ctx, p.status); };
  // Queries as B fragments: column g = query head hq0 + 8 nt + g; step ks,
  // indices 2t, 2t + 1 and 2t + 8, 2t + 9 = columns (D/4) t + 4 ks + 0..3, the
  // columns of the lane's own key codes.
  uint32_t qb[NT][kKSteps][2];
  auto rows_of = [&](const Place& x) { return min(kRows, p.group - x.chunk * kRows); };
  auto row_of = [&](const Place& x) {  // first row of the queries and the output
    return static_cast<size_t>(x.seq) * p.Hq + x.head * p.group + x.chunk * kRows;
  };
  auto load_queries = [&](const Place& x) {
    const int rows = rows_of(x);
    const size_t row0 = row_of(x);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const bool real = 8 * nt + g < rows;
      const uint2* row = reinterpret_cast<const uint2*>(p.q + (row0 + (real ? 8 * nt + g : 0)) * D + (D / 4) * t);
#pragma unroll
      for (int ks = 0; ks < kKSteps; ++ks) {
        const uint2 w = real ? __ldg(row + ks) : make_uint2(0u, 0u);
        qb[nt][ks][0] = w.x;
        qb[nt][ks][1] = w.y;
      }
    }
  };
  Place at;             // the next unit to compute
  int left;             // units (in a cluster) or places of this CTA that are not yet computed
  int joint_parts = 0;  // CTAs after this one that its last segment goes on in (warp 0)
  const uint32_t rank = kCluster ? cta % kFp4ClusterCtas : 0;
  // Sequences without a cached token: o = 0, lse = -inf.  A lane looks at one, the
  // warp clears what is found.  (Every sequence's length passes here once, so that
  // one out of range is reported.)
  auto clear_empty = [&]() {
    for (int i = 32 * warp; cta + static_cast<int>(gridDim.x) * i < p.num_seqs; i += kCtaThreads) {
      const int s = cta + gridDim.x * (i + lane);
      for (uint32_t empty = __ballot_sync(0xffffffffu, s < p.num_seqs && ctx_of(s) == 0); empty != 0;
           empty &= empty - 1) {
        const size_t row0 = static_cast<size_t>(cta + gridDim.x * (i + __ffs(empty) - 1)) * p.Hq;
        for (int idx = lane; idx < p.Hq * (D / 8); idx += 32)
          reinterpret_cast<uint4*>(p.out + row0 * D)[idx] = make_uint4(0u, 0u, 0u, 0u);
        if (p.lse != nullptr)
          for (int h = lane; h < p.Hq; h += 32) p.lse[row0 + h] = -INFINITY;
        __syncwarp();
      }
    }
  };
  auto next_segment = [&](Place& x) {  // the following segment that has units
    x.k = 0;
    if (++x.chunk < p.n_chunks) return;
    x.chunk = 0;
    if (++x.head < p.Hkv) return;
    x.head = 0;
    do {
      x.seq = min(x.seq + 1, p.num_seqs - 1);
      x.ctx = ctx_of(x.seq);
    } while (x.ctx == 0 && x.seq < p.num_seqs - 1);
    x.units = max(1, units_of(x.ctx));
  };
  const bool copies = warp == kWarps;
  int phys_lane = -1;  // of the copying warp: physical block of block lane % 8 of a batch's unit lane / 8; -1: none
  auto check = [&](int ph) {
    if (ph >= 0 && ph < p.num_blocks) return ph;
    atomicOr(p.status, 2u);  // EXATTN_DEVICE_BOUNDS_BIT
    return -1;
  };
  if constexpr (kCluster) {
    // Every 8th unit, so that the table entries and queries need not wait for the
    // context length: the three loads are in flight together.
    static_assert(kFp4ClusterUnits / kFp4ClusterCtas <= 32 / kUnit, "one batch of table entries");
    const int seg = cta / kFp4ClusterCtas;
    at.seq = seg / segs;
    at.head = seg % segs / p.n_chunks;
    at.chunk = seg % p.n_chunks;
    at.k = rank;
    const int blk = (rank + kStep * (lane / kUnit)) * kUnit + lane % kUnit;
    const int entry = copies && blk < p.max_blocks_per_seq
                          ? __ldg(p.block_table + static_cast<size_t>(at.seq) * p.max_blocks_per_seq + blk)
                          : -1;
    if (!copies) load_queries(at);
    at.ctx = ctx_of(at.seq);
    at.units = units_of(at.ctx);
    left = (at.units - static_cast<int>(rank) + kStep - 1) / kStep;
    if (copies && blk * kBlk < at.ctx) phys_lane = check(entry);
  } else {
    // ---- this CTA's share; every warp finds it for itself
    const Batch seqs(p.ctx_lens, p.num_seqs, max_ctx);
    const Shares shares(seqs.per_segment * segs, gridDim.x);
    const int begin = shares.begin(cta), begin_next = shares.begin(cta + 1);
    left = begin_next - begin;
    if (p.joints != nullptr && threadIdx.x == 0) p.joints[cta].more = 0;
    if (left == 0) {
      clear_empty();
      return;
    }
    at = seqs.find(begin, segs, p.n_chunks);
    if (at.k == at.units) {  // the end of a segment that others compute
      if (--left == 0) {
        clear_empty();
        return;
      }
      next_segment(at);
    }
    if (!copies) load_queries(at);
    if (p.joints != nullptr && warp == 0) {
      const Place last = seqs.find(begin_next - 1, segs, p.n_chunks);
      joint_parts = shares.owner(begin_next - 1 + last.units - 1 - last.k) - cta;
    }
  }

  __syncthreads();  // the barriers are set up

  if (copies) {
    // ---- the copying warp: units in order, as stages come free; the lane that holds a
    // block's table entry copies it.  A block past the end, or whose entry is out of
    // range, arrives without a copy.
    const uint64_t stream_policy = l2_policy_evict_first();
    const uint32_t blk_bytes = static_cast<uint32_t>(p.Hkv) * Span::kBytes;
    Place to = at;
    int to_load = left;  // places whose table entries are not yet asked for
    // A batch: up to four units of one segment; lane 8 i + b has unit i's block b.
    struct Entries {
      int units, raw;  // raw: this lane's table entry, if it has one (`mine`)
      bool mine;
      int past;  // tokens of the context past the batch's first unit
      const uint8_t* head;
    };
    auto load_batch = [&]() {
      Entries e;
      if (to.k == to.units) {
        next_segment(to);
        // its queries into the L1 cache, for the computing warps
        if (lane < rows_of(to) * D / 64)
          asm volatile("prefetch.global.L1 [%0];" ::"l"(p.q + row_of(to) * D + lane * 64));
      }
      e.units = min(32 / kUnit, min(to.units - to.k, to_load));
      const int blk = to.k * kUnit + lane;
      e.mine = lane < e.units * kUnit && blk * kBlk < to.ctx;
      e.raw = e.mine ? __ldg(p.block_table + static_cast<size_t>(to.seq) * p.max_blocks_per_seq + blk) : -1;
      e.past = to.ctx - (to.k + 1) * kUnit * kBlk;
      e.head = p.cache + static_cast<size_t>(to.head) * Span::kBytes;
      to.k += e.units;
      to_load -= e.units;
      if (to.k == to.units && to_load > 0) --to_load;
      return e;
    };
    Entries now, next;  // the entries of the next batch are on their way while this one's blocks are copied
    if constexpr (kCluster)
      now = Entries{left, phys_lane, phys_lane >= 0, at.ctx - (at.k + 1) * kUnit * kBlk,
                    p.cache + static_cast<size_t>(at.head) * Span::kBytes};
    else
      next = load_batch();
    bool more = !kCluster;  // `next` holds a batch
    if (!kCluster) now.units = 0;
    int batch_at = 0;
    int i = 0;
    int st = 0;
    uint32_t parity = 1;  // of the stage's last use; the first round waits for none
#pragma unroll 1
    for (;; ++i) {
      if (batch_at == now.units) {
        if (!more) break;
        now = next;
        more = false;
        batch_at = 0;
        phys_lane = now.mine ? check(now.raw) : -1;
      }
      const bool waited = i < kStages || mbar_wait(&sm.empty[st], parity, p.wait_ns);
      if (!__all_sync(0xffffffffu, waited)) {
        if (lane == 0) atomicOr(p.status, 1u);  // EXATTN_DEVICE_TIMEOUT_BIT
        break;
      }
      const uint32_t present = (__ballot_sync(0xffffffffu, phys_lane >= 0) >> (batch_at * kUnit)) & ((1u << kUnit) - 1);
      if (lane / kUnit == batch_at) {
        const int b = lane % kUnit;
        if (b == 0) sm.present[st] = now.past >= 0 && present == (1u << kUnit) - 1 ? kWhole : static_cast<int>(present);
        if (phys_lane < 0) {
          mbar_arrive(&sm.full[st]);
        } else {
          mbar_arrive_expect_tx(&sm.full[st], Span::kBytes);
          bulk_load_hint(sm.ring[st][b], now.head + static_cast<uint64_t>(static_cast<uint32_t>(phys_lane)) * blk_bytes,
                         Span::kBytes, &sm.full[st], stream_policy);
        }
      }
      if (!kCluster && batch_at == 0 && to_load > 0) {
        next = load_batch();
        more = true;
      }
      ++batch_at;
      now.past -= kStep * kUnit * kBlk;
      if (++st == kStages) {
        st = 0;
        parity ^= 1u;
      }
    }
    for (int j = max(0, i - kStages); j < i; ++j)  // no copy is left in flight
      mbar_wait(&sm.full[j % kStages], (j / kStages) & 1, p.wait_ns);
    __syncwarp();
    if constexpr (kCluster) {
      cluster_barrier();
      cluster_barrier();
    } else {
      clear_empty();
    }
    return;
  }

  // mma token index r stands for token r ^ ((r >> 1) & 1): neighbouring pairs
  // swapped for odd t, so that the value loads of the four lanes of a group
  // fall on both halves of the banks.
  const int tok_s = g ^ ((g >> 1) & 1);    // this lane's score rows: tok_s, tok_s + 8
  const int tok_v0 = 2 * t + (t & 1);      // mma index 2t (and 2t + 8: + 8)
  const int tok_v1 = 2 * t + 1 - (t & 1);  // mma index 2t + 1 (and 2t + 9: + 8)
  const uint32_t ring0 = smem_u32(sm.ring[0][2 * warp]);
  const uint32_t key_at = ring0 + Span::kKeyCodes + tok_s * Span::kCodeRow + t * (D / 8);
  const uint32_t key_scale_at = ring0 + Span::kKeyScales + tok_s * Span::kScaleRow + t * (D / 64);
  const uint32_t val_at0 = ring0 + Span::kValueCodes + tok_v0 * Span::kCodeRow + g * (D / 16);
  const uint32_t val_at1 = ring0 + Span::kValueCodes + tok_v1 * Span::kCodeRow + g * (D / 16);
  const uint32_t val_scale_at0 = ring0 + Span::kValueScales + tok_v0 * Span::kScaleRow + g * D / 128;
  const uint32_t val_scale_at1 = ring0 + Span::kValueScales + tok_v1 * Span::kScaleRow + g * D / 128;
  constexpr int kCodes8 = 8 * Span::kCodeRow, kScales8 = 8 * Span::kScaleRow;  // eight tokens on
  bool ok = true;  // no wait has run out
  int st = 0;      // stage of the next unit
  uint32_t parity = 0;

  // In a cluster: this CTA's outcome, in the ring, which every copy has left by then.
  float* const cluster_o = reinterpret_cast<float*>(&sm.ring[0][0][0]);
  float* const cluster_lse = cluster_o + kRows * D;
  if constexpr (kCluster)
    if (left == 0)
      for (int idx = threadIdx.x; idx < kRows * D; idx += kThreads) {
        cluster_o[idx] = 0.f;
        if (idx < kRows) cluster_lse[idx] = -INFINITY;
      }

  const bool two_halves = p.group <= 4 * NT;  // staging rows for two segments
  int buf = 0;
#pragma unroll 1
  while (left > 0) {  // segments of this CTA's share
    const int rows_here = rows_of(at);
    const size_t row0 = row_of(at);
    const bool starts = at.k == 0;
    const int n_units = kCluster ? left : min(at.units - at.k, left);
    const bool ends = at.k + n_units == at.units;

    float factor[NT][2];  // score factor of heads 2t, 2t + 1
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float top = 0.f;
#pragma unroll
      for (int ks = 0; ks < kKSteps; ++ks)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const uint32_t v = qb[nt][ks][e];
          top = max3f(top, fabsf(__uint_as_float(v << 16)), fabsf(__uint_as_float(v & 0xFFFF0000u)));
        }
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      // the power of two of the largest element, within what its reciprocal
      // can be; zeros stay zeros and infinities infinities
      const int e = max(-120, min(126, static_cast<int>(__float_as_uint(top) >> 23) - 127));
      const float down = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
      const float up = __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
#pragma unroll
      for (int ks = 0; ks < kKSteps; ++ks)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const uint32_t v = qb[nt][ks][x];
          qb[nt][ks][x] = pack_f16x2(__uint_as_float(v << 16) * down, __uint_as_float(v & 0xFFFF0000u) * down);
        }
      // (at least the smallest normal number: a masked -inf stays one)
      factor[nt][0] = fmaxf(__shfl_sync(0xffffffffu, up, 8 * t) * p.scale_log2, 1.17549435e-38f);
      factor[nt][1] = fmaxf(__shfl_sync(0xffffffffu, up, 8 * t + 4) * p.scale_log2, 1.17549435e-38f);
    }

    float m[NT][2], l[NT][2];     // heads 2t, 2t + 1; l: this lane's tokens only
    float acc[kMTiles][NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      m[nt][0] = m[nt][1] = kNoScore;
      l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
      for (int mt = 0; mt < kMTiles; ++mt) acc[mt][nt][0] = acc[mt][nt][1] = acc[mt][nt][2] = acc[mt][nt][3] = 0.f;
    }

#pragma unroll 1
    for (int i = 0; i < n_units; ++i) {
      if (ok && !__all_sync(0xffffffffu, mbar_wait(&sm.full[st], parity, p.wait_ns))) {
        ok = false;  // nothing more is computed, the CTA's barriers are still met
        if (lane == 0) atomicOr(p.status, 1u);  // EXATTN_DEVICE_TIMEOUT_BIT
      }
      if (!ok) continue;
      const uint32_t stage = st * (kUnit * Span::kBytes);
      const int present = sm.present[st];
      // Whether all of this warp's two blocks' tokens count; else, how many of each.
      const bool full = present == kWhole;
      int n_valid[2] = {kBlk, kBlk};
      if (!full) {
        const int tokens = at.ctx - ((at.k + i * kStep) * kUnit + 2 * warp) * kBlk;
        n_valid[0] = present >> (2 * warp) & 1 ? tokens : 0;
        n_valid[1] = present >> (2 * warp) & 2 ? tokens - kBlk : 0;
      }
      if (full || max(n_valid[0], n_valid[1]) > 0) {
        // ---- S^T = K Q^T
        float c[2][NT][4];
        auto scores = [&](auto block) {
          constexpr int b = decltype(block)::value, kSpan = b * Span::kBytes;
          uint32_t ka[kKeyWords], kb[kKeyWords];
          lds_words<kSpan>(key_at + stage, ka);
          lds_words<kSpan + kCodes8>(key_at + stage, kb);
          uint32_t sa, sb;  // scales of the lane's groups, fp16 pairs
          if constexpr (D == 128) {
            sa = e4m3x2_to_f16(lds_u16<kSpan>(key_scale_at + stage));
            sb = e4m3x2_to_f16(lds_u16<kSpan + kScales8>(key_scale_at + stage));
          } else {
            sa = e4m3x2_to_f16(lds_u8<kSpan>(key_scale_at + stage));
            sb = e4m3x2_to_f16(lds_u8<kSpan + kScales8>(key_scale_at + stage));
          }
#pragma unroll
          for (int w = 0; w < kKeyWords; ++w) {
            // words 0, 1: the first group of 16 columns, words 2, 3: the second
            const uint32_t s0 = __byte_perm(sa, 0, w < 2 ? 0x1010 : 0x3232);
            const uint32_t s1 = __byte_perm(sb, 0, w < 2 ? 0x1010 : 0x3232);
            uint32_t h0[4], h1[4];
            e2m1x8_to_f16(ka[w], h0);
            e2m1x8_to_f16(kb[w], h1);
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              h0[x] = f16x2_mul(h0[x], s0);
              h1[x] = f16x2_mul(h1[x], s1);
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              if (w == 0)
                mma_f16_16816_first(c[b][nt], h0[0], h1[0], h0[1], h1[1], qb[nt][0][0], qb[nt][0][1]);
              else
                mma_f16_16816(c[b][nt], h0[0], h1[0], h0[1], h1[1], qb[nt][2 * w][0], qb[nt][2 * w][1]);
              mma_f16_16816(c[b][nt], h0[2], h1[2], h0[3], h1[3], qb[nt][2 * w + 1][0], qb[nt][2 * w + 1][1]);
            }
          }
        };
        scores(std::integral_constant<int, 0>());
        scores(std::integral_constant<int, 1>());
        // ---- online softmax: c[b][nt][j] is token tok_s, head 2t + j, c[b][nt][2 + j]
        // token tok_s + 8.  Tokens that do not count are masked here and their
        // value scales zeroed below (the slots may hold anything).
        if (!full) {
#pragma unroll
          for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int j = 0; j < 2; ++j) {
                if (tok_s >= n_valid[b]) c[b][nt][j] = -INFINITY;
                if (tok_s + 8 >= n_valid[b]) c[b][nt][2 + j] = -INFINITY;
              }
          __syncwarp();  // the lanes together again for the next mma
        }
        // Exponents relative to the reference m.  It follows the running maximum
        // only when that has grown by more than kMost - kLift, which is rare after the
        // first blocks: most pairs pay one vote.  A score is rounded before m is taken
        // from it, as it was when it gave m: in one fused operation the largest
        // itself would lie off by the rounding, which passes all that fp16 holds once
        // scores come to 2^28.
        float x[2][NT][4];
        float most = -INFINITY;
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int y = 0; y < 4; y += 2) {
              scores_and_distances(c[b][nt][y], c[b][nt][y + 1], factor[nt], m[nt], x[b][nt][y], x[b][nt][y + 1]);
              most = max3f(most, x[b][nt][y], x[b][nt][y + 1]);
            }
        if (__any_sync(0xffffffffu, most > kMost)) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              float top = fmaxf(fmaxf(c[0][nt][j], c[0][nt][2 + j]), fmaxf(c[1][nt][j], c[1][nt][2 + j]));
              top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
              top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
              top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
              const float mn = fmaxf(m[nt][j], top - kLift);
              const float alpha = ex2_approx(m[nt][j] - mn);
              m[nt][j] = mn;
              l[nt][j] *= alpha;
#pragma unroll
              for (int mt = 0; mt < kMTiles; ++mt) {
                acc[mt][nt][j] *= alpha;
                acc[mt][nt][2 + j] *= alpha;
              }
#pragma unroll
              for (int b = 0; b < 2; ++b) {
                x[b][nt][j] = c[b][nt][j] - mn;
                x[b][nt][2 + j] = c[b][nt][2 + j] - mn;
              }
            }
        }
        // ---- O^T += V^T P^T: row tile mt, row g = column (D/8) g + 2 mt, row
        // g + 8 the next one, all of one scale group
        auto products = [&](auto block) {
          constexpr int b = decltype(block)::value, kSpan = b * Span::kBytes;
          uint32_t va0[kValWords], va1[kValWords], vb0[kValWords], vb1[kValWords];
          lds_words<kSpan>(val_at0 + stage, va0);
          lds_words<kSpan>(val_at1 + stage, va1);
          lds_words<kSpan + kCodes8>(val_at0 + stage, vb0);
          lds_words<kSpan + kCodes8>(val_at1 + stage, vb1);
          uint32_t ea0 = lds_u8<kSpan>(val_scale_at0 + stage), ea1 = lds_u8<kSpan>(val_scale_at1 + stage);
          uint32_t eb0 = lds_u8<kSpan + kScales8>(val_scale_at0 + stage);
          uint32_t eb1 = lds_u8<kSpan + kScales8>(val_scale_at1 + stage);
          uint32_t pb[NT][2];
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            float w[4];
#pragma unroll
            for (int y = 0; y < 4; ++y) w[y] = ex2_approx(x[b][nt][y]);
            l[nt][0] += w[0] + w[2];
            l[nt][1] += w[1] + w[3];
            pb[nt][0] = transpose8x8(pack_f16x2(w[0], w[1]));
            pb[nt][1] = transpose8x8(pack_f16x2(w[2], w[3]));
          }
          if (!full) {
            if (tok_v0 >= n_valid[b]) ea0 = 0;
            if (tok_v1 >= n_valid[b]) ea1 = 0;
            if (tok_v0 + 8 >= n_valid[b]) eb0 = 0;
            if (tok_v1 + 8 >= n_valid[b]) eb1 = 0;
            __syncwarp();  // the lanes together again for the next mma
          }
          const uint32_t ta = e4m3x2_to_f16(__byte_perm(ea0, ea1, 0x0040));
          const uint32_t tb = e4m3x2_to_f16(__byte_perm(eb0, eb1, 0x0040));
#pragma unroll
          for (int w = 0; w < kValWords; ++w) {
            // bytes of (token 2t, token 2t + 1) pairs, even columns then odd ones
            const uint32_t ae = (va0[w] & 0x0F0F0F0Fu) | ((va1[w] << 4) & 0xF0F0F0F0u);
            const uint32_t ao = ((va0[w] >> 4) & 0x0F0F0F0Fu) | (va1[w] & 0xF0F0F0F0u);
            const uint32_t be = (vb0[w] & 0x0F0F0F0Fu) | ((vb1[w] << 4) & 0xF0F0F0F0u);
            const uint32_t bo = ((vb0[w] >> 4) & 0x0F0F0F0Fu) | (vb1[w] & 0xF0F0F0F0u);
            uint32_t h0[4], h1[4], h2[4], h3[4];
            e2m1x8_to_f16(ae, h0);
            e2m1x8_to_f16(ao, h1);
            e2m1x8_to_f16(be, h2);
            e2m1x8_to_f16(bo, h3);
#pragma unroll
            for (int y = 0; y < 4; ++y) {
              h0[y] = f16x2_mul(h0[y], ta);
              h1[y] = f16x2_mul(h1[y], ta);
              h2[y] = f16x2_mul(h2[y], tb);
              h3[y] = f16x2_mul(h3[y], tb);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
                mma_f16_16816(acc[4 * w + y][nt], h0[y], h1[y], h2[y], h3[y], pb[nt][0], pb[nt][1]);
            }
          }
        };
        products(std::integral_constant<int, 0>());
        products(std::integral_constant<int, 1>());
      }
      __syncwarp();  // all lanes are done with this stage
      if (lane == 0) mbar_arrive(&sm.empty[st]);
      if (++st == kStages) {
        st = 0;
        parity ^= 1u;
      }
    }

    // ---- the warps' states merge.  The staging of the segment before may still
    // be read, unless the two take turns with halves of it.
    if (!two_halves) compute_barrier();
    const int half = two_halves ? buf * 4 * NT : 0;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
#pragma unroll
        for (int y = 4; y < 32; y *= 2) l[nt][j] += __shfl_xor_sync(0xffffffffu, l[nt][j], y);
        const int r = 8 * nt + 2 * t + j;
        if (g == 0) {
          sm.wm[buf][warp][r] = m[nt][j];
          sm.wl[buf][warp][r] = l[nt][j];
        }
        if (r < rows_here)
#pragma unroll
          for (int mt = 0; mt < kMTiles; mt += 2)
            *reinterpret_cast<float4*>(&sm.acc[warp][half + r][(D / 8) * g + 2 * mt]) =
                make_float4(acc[mt][nt][j], acc[mt][nt][2 + j], acc[mt + 1][nt][j], acc[mt + 1][nt][2 + j]);
      }
    left -= n_units;
    if (!kCluster && ends && left > 0) --left;
    if (left > 0) {  // the next segment's queries arrive during the merge
      next_segment(at);
      load_queries(at);
    }
    compute_barrier();
    for (int idx = threadIdx.x; idx < rows_here * (D / 4); idx += kThreads) {
      const int r = idx / (D / 4), col = idx % (D / 4) * 4;
      float M = kNoScore;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) M = fmaxf(M, sm.wm[buf][w][r]);
      float L = 0.f;
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float wt = ex2_approx(sm.wm[buf][w][r] - M);
        L += wt * sm.wl[buf][w][r];
        const float4 a = *reinterpret_cast<const float4*>(&sm.acc[w][half + r][col]);
        o.x += wt * a.x;
        o.y += wt * a.y;
        o.z += wt * a.z;
        o.w += wt * a.w;
      }
      // a share all of whose scores are -inf, or whose blocks are all missing, sees nothing
      // (v_scale on its own: over the sum of the weights it could lose its bits)
      const float inv = L == 0.f ? 0.f : __fdividef(1.f, L);
      o = make_float4(o.x * inv * p.v_scale, o.y * inv * p.v_scale, o.z * inv * p.v_scale, o.w * inv * p.v_scale);
      const float ls = L == 0.f ? -INFINITY : (M + __log2f(L)) * kLn2;
      if constexpr (kCluster) {
        *reinterpret_cast<float4*>(cluster_o + r * D + col) = o;
        if (col == 0) cluster_lse[r] = ls;
      } else if (starts && ends) {
        *reinterpret_cast<uint2*>(p.out + (row0 + r) * D + col) =
            make_uint2(pack_bf16x2(o.x, o.y), pack_bf16x2(o.z, o.w));
        if (p.lse != nullptr && col == 0) p.lse[row0 + r] = ls;
      } else {
        const size_t row = static_cast<size_t>(2 * cta + (starts ? 1 : 0)) * kRows + r;
        *reinterpret_cast<float4*>(p.ws_o + row * D + col) = o;
        if (col == 0) p.ws_lse[row] = ls;
      }
    }
    if (left == 0) {
      // the only segment that can go on into further CTAs is the last
      if (!kCluster && p.joints != nullptr && starts && !ends && threadIdx.x == 0)
        p.joints[cta] = Fp4Joint{cta, joint_parts, static_cast<int>(row0), rows_here};
      break;
    }
    buf ^= 1;
  }
  __syncwarp();
  if constexpr (kCluster) {
    // ---- the cluster's CTAs merge: L = log sum_i exp(lse_i), o = sum_i exp(lse_i - L) O_i
    const int rows_here = rows_of(at);
    const size_t row0 = row_of(at);
    cluster_barrier();
    for (int idx = threadIdx.x * kFp4ClusterCtas + rank; idx < rows_here * (D / 4); idx += kThreads * kFp4ClusterCtas) {
      const int r = idx / (D / 4), col = idx % (D / 4) * 4;
      float ls[kFp4ClusterCtas];
      float4 part[kFp4ClusterCtas];
#pragma unroll
      for (int i = 0; i < kFp4ClusterCtas; ++i) {
        ls[i] = cluster_load(cluster_lse + r, i);
        part[i] = cluster_load4(cluster_o + r * D + col, i);
      }
      float M = ls[0];
#pragma unroll
      for (int i = 1; i < kFp4ClusterCtas; ++i) M = max_nan(M, ls[i]);
      const float ref = M == -INFINITY ? 0.f : M;
      float W = 0.f;
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int i = 0; i < kFp4ClusterCtas; ++i) {
        const float w = ex2_approx((ls[i] - ref) * kLog2e);
        W += w;
        o.x = fmaf(w, part[i].x, o.x);
        o.y = fmaf(w, part[i].y, o.y);
        o.z = fmaf(w, part[i].z, o.z);
        o.w = fmaf(w, part[i].w, o.w);
      }
      const float inv = W == 0.f ? 0.f : 1.f / W;
      *reinterpret_cast<uint2*>(p.out + (row0 + r) * D + col) =
          make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
      if (p.lse != nullptr && col == 0) p.lse[row0 + r] = W == 0.f ? -INFINITY : M + __logf(W);
    }
    cluster_barrier();  // nobody's shared memory goes away before the others have read it
  } else {
    clear_empty();
  }
}

struct Fp4CombineParams {
  const Fp4Joint* joints;  // one per CTA of the split kernel, or NULL (kFind): one CTA row per segment
  const int32_t* ctx_lens;
  const float* ws_o;
  const float* ws_lse;
  __nv_bfloat16* out;
  float* lse;
  int num_seqs, Hq, segs, n_chunks, group, max_blocks_per_seq, ctas;
  int rows;  // query heads per segment, at most
};

// One CTA per (row, segment that several CTAs share): its partial outputs O_i
// lie in the second place of the CTA where it starts and the first places of
// the `more` that follow; L = log sum_i exp(lse_i), o = sum_i exp(lse_i - L) O_i.
// Where segments are few (kFind) it finds them from ctx_lens, while the split kernel
// still runs; else it reads what that wrote down.  Registers: with 40, not 64, where it
// reads (64 sequences of 512 to 8192 tokens 62.7 us, 63.7); with 48 where it finds: 66
// would leave it no room beside a split kernel for 16 heads (32 sequences of 96 heads
// 59.7 us, 55.4 with 48), and fewer slow the search (one of 8000 tokens 8.4 us with 66,
// 8.8 with 48, 9.1 with 40).  The weights are formed once, one
// per thread; D/4 threads take four columns each of every kTeams-th partial output,
// the first ones' loads on their way before the weights are known.
template <int D, bool kFind>
__global__ void __launch_bounds__(kMergeThreads, kFind ? 5 : 6) decode_fp4_combine_kernel(const Fp4CombineParams p) {
  constexpr int kTeams = kMergeThreads / (D / 4);
  constexpr int kMergeWarps = kMergeThreads / 32;
  constexpr int kEarly = 3;
  __shared__ float weight[kFp4MaxCtas];
  __shared__ float top[kMergeWarps], sum[kMergeWarps];
  __shared__ float4 part[kTeams][D / 4];
  __shared__ Fp4Joint found;
  const int r = blockIdx.x;
  if constexpr (kFind) {
    if (threadIdx.x < 32) {
      const Batch seqs(p.ctx_lens, p.num_seqs, p.max_blocks_per_seq * kBlk);
      const Shares shares(seqs.per_segment * p.segs, p.ctas);
      const int seq = blockIdx.y / p.segs, y = blockIdx.y % p.segs;
      const int ctx = seqs.ctx_of(seq), units = units_of(ctx);
      const int unit = seqs.before_seq(seq) * p.segs + y * places_of(ctx);  // the place of its first
      if (threadIdx.x == 0) {
        found.cta = units > 0 ? shares.owner(unit) : 0;
        found.more = units > 0 ? shares.owner(unit + units - 1) - found.cta : 0;
        found.row = seq * p.Hq + y / p.n_chunks * p.group + y % p.n_chunks * p.rows;
        found.rows = min(p.rows, p.group - y % p.n_chunks * p.rows);
      }
    }
    __syncthreads();
  }
  cudaGridDependencySynchronize();  // launched while the split kernel runs, after all before that had ended
  const Fp4Joint joint = kFind ? found : p.joints[blockIdx.y];
  if (joint.more == 0 || r >= joint.rows) return;
  const int used = joint.more + 1;
  auto place = [&](int i) { return static_cast<size_t>(2 * (joint.cta + i) + (i == 0 ? 1 : 0)) * p.rows + r; };
  const int col = threadIdx.x % (D / 4), team = threadIdx.x / (D / 4);
  auto part_of = [&](int s) { return reinterpret_cast<const float4*>(p.ws_o + place(s) * D)[col]; };
  float4 early[kEarly];
#pragma unroll
  for (int i = 0; i < kEarly; ++i)
    early[i] = team + i * kTeams < used ? part_of(team + i * kTeams) : make_float4(0.f, 0.f, 0.f, 0.f);
  float M = -INFINITY;
  for (int s = threadIdx.x; s < used; s += kMergeThreads) {
    const float ls = p.ws_lse[place(s)];
    weight[s] = ls;
    M = max_nan(M, ls);
  }
#pragma unroll
  for (int x = 1; x < 32; x *= 2) M = max_nan(M, __shfl_xor_sync(0xffffffffu, M, x));
  if ((threadIdx.x & 31) == 0) top[threadIdx.x >> 5] = M;
  __syncthreads();
  M = top[0];
#pragma unroll
  for (int w = 1; w < kMergeWarps; ++w) M = max_nan(M, top[w]);
  const float ref = M == -INFINITY ? 0.f : M;  // all weights 0 where no part sees anything
  float W = 0.f;
  for (int s = threadIdx.x; s < used; s += kMergeThreads) {
    const float w = ex2_approx((weight[s] - ref) * kLog2e);
    weight[s] = w;
    W += w;
  }
#pragma unroll
  for (int x = 1; x < 32; x *= 2) W += __shfl_xor_sync(0xffffffffu, W, x);
  if ((threadIdx.x & 31) == 0) sum[threadIdx.x >> 5] = W;
  __syncthreads();
  W = 0.f;
#pragma unroll
  for (int w = 0; w < kMergeWarps; ++w) W += sum[w];
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  auto add = [&](float w, const float4& a) {
    o.x = fmaf(w, a.x, o.x);
    o.y = fmaf(w, a.y, o.y);
    o.z = fmaf(w, a.z, o.z);
    o.w = fmaf(w, a.w, o.w);
  };
#pragma unroll
  for (int i = 0; i < kEarly; ++i)
    if (team + i * kTeams < used) add(weight[team + i * kTeams], early[i]);
#pragma unroll 4
  for (int s = team + kEarly * kTeams; s < used; s += kTeams) add(weight[s], part_of(s));
  part[team][col] = o;
  __syncthreads();
  if (threadIdx.x < D / 4) {
#pragma unroll
    for (int x = 1; x < kTeams; ++x) {
      const float4 a = part[x][col];
      o.x += a.x;
      o.y += a.y;
      o.z += a.z;
      o.w += a.w;
    }
    const float inv = W == 0.f ? 0.f : 1.f / W;
    const size_t row = static_cast<size_t>(joint.row) + r;
    reinterpret_cast<uint2*>(p.out + row * D)[col] =
        make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
    if (p.lse != nullptr && col == 0) p.lse[row] = W == 0.f ? -INFINITY : M + __logf(W);
  }
}

template <int D, int NT, bool kCluster>
cudaError_t launch_split(const Fp4SplitParams& sp, int ctas, cudaStream_t stream) {
  const size_t smem = sizeof(Fp4Smem<D, NT>) + 128;
  static std::atomic<int> smem_set[64] = {};
  cudaError_t e = smem_limit_once(reinterpret_cast<const void*>(decode_fp4_split_kernel<D, NT, kCluster>),
                                  static_cast<int>(smem), smem_set);
  if (e != cudaSuccess) return e;
  return launch_overlapped(decode_fp4_split_kernel<D, NT, kCluster>, ctas, kCtaThreads, smem, stream,
                           kCluster ? kFp4ClusterCtas : 1, sp);
}

template <int D>
cudaError_t launch_d(const DecodeFp4Args& a, const DeviceGuard& g, cudaStream_t stream) {
  const Fp4Plan& plan = a.plan;
  Fp4SplitParams sp;
  sp.q = static_cast<const __nv_bfloat16*>(a.q);
  sp.cache = static_cast<const uint8_t*>(a.kv_cache);
  sp.block_table = a.block_table;
  sp.ctx_lens = a.ctx_lens;
  uint8_t* ws = static_cast<uint8_t*>(a.workspace);
  sp.joints = plan.joints > 0 ? reinterpret_cast<Fp4Joint*>(ws) : nullptr;
  sp.ws_o = reinterpret_cast<float*>(ws + plan.joint_bytes());
  sp.ws_lse = reinterpret_cast<float*>(ws + plan.joint_bytes() + plan.part_bytes(D));
  sp.out = static_cast<__nv_bfloat16*>(a.out);
  sp.lse = a.lse;
  sp.status = g.status;
  sp.wait_ns = g.wait_ns;
  sp.num_seqs = a.num_seqs;
  sp.Hq = a.Hq;
  sp.Hkv = a.Hkv;
  sp.group = a.Hq / a.Hkv;
  sp.n_chunks = plan.chunks;
  sp.num_blocks = a.num_blocks;
  sp.max_blocks_per_seq = a.max_blocks_per_seq;
  sp.scale_log2 = static_cast<float>(static_cast<double>(a.scale) * a.k_scale * 1.4426950408889634);
  sp.v_scale = a.v_scale;
  if (plan.cluster)
    return plan.rows == 8 ? launch_split<D, 1, true>(sp, plan.ctas, stream)
                          : launch_split<D, 2, true>(sp, plan.ctas, stream);
  const cudaError_t e = plan.rows == 8 ? launch_split<D, 1, false>(sp, plan.ctas, stream)
                                       : launch_split<D, 2, false>(sp, plan.ctas, stream);
  if (e != cudaSuccess || !plan.shared) return e;

  Fp4CombineParams cp;
  cp.joints = sp.joints;
  cp.ctx_lens = a.ctx_lens;
  cp.ws_o = sp.ws_o;
  cp.ws_lse = sp.ws_lse;
  cp.out = sp.out;
  cp.lse = a.lse;
  cp.num_seqs = a.num_seqs;
  cp.Hq = a.Hq;
  cp.segs = a.Hkv * plan.chunks;
  cp.n_chunks = plan.chunks;
  cp.group = sp.group;
  cp.max_blocks_per_seq = a.max_blocks_per_seq;
  cp.ctas = plan.ctas;
  cp.rows = plan.rows;
  const dim3 grid(sp.group < plan.rows ? sp.group : plan.rows, plan.joints > 0 ? plan.joints : a.num_seqs * cp.segs);
  return launch_overlapped(plan.joints > 0 ? decode_fp4_combine_kernel<D, false> : decode_fp4_combine_kernel<D, true>,
                           grid, kMergeThreads, 0, stream, 1, cp);
}

}  // namespace

cudaError_t launch_decode_fp4(const DecodeFp4Args& a, const DeviceGuard& g, cudaStream_t stream) {
  return a.d == 64 ? launch_d<64>(a, g, stream) : launch_d<128>(a, g, stream);
}

}  // namespace exattn
