// What the paged decode kernels over quantised caches share: how a call's work is
// divided among the CTAs of one wave, the merge of partial outputs, and the
// instructions that both use.  kUnit: blocks of 16 tokens in a unit of work; kEnd: units
// that the end of a segment, its merge and the change of queries, counts for.
#pragma once
#include <cuda_bf16.h>

#include "fp4.cuh"
#include "launch.h"
#include "ptx.cuh"

namespace exattn {

constexpr int kMergeThreads = 256;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.69314718055994531f;
constexpr float kNoScore = -3.0e38f;     // below any score; -inf would give inf - inf

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
// chunk), or (k >= units) a place that stands for the segment's end.
struct Place {
  int seq, head, chunk, k, units, ctx;
};

template <int kUnit>
__device__ __forceinline__ int units_of(int ctx) {
  return (ctx + kUnit * kDecodeBlockSize - 1) / (kUnit * kDecodeBlockSize);
}

// Places of a segment: its units and kEnd for its end, whose merge and change of
// queries take a CTA time too (4-bit cache: 2400 cycles where a unit takes 2100; with units
// alone the CTAs that got the short sequences of a batch were the last to finish, 128
// sequences of 1 to 2000 tokens took 45.8 us, 38.4 with the ends counted).
template <int kUnit, int kEnd>
__device__ __forceinline__ int places_of(int ctx) {
  return units_of<kUnit>(ctx) + (ctx > 0 ? kEnd : 0);
}

// Sums over the sequences that a warp forms from ctx_lens, each lane holding those of a
// contiguous range of them.  In a large batch the warp reads 32 neighbours together: with
// every lane reading its own range, no two of a load's addresses share a line, and 4096
// sequences took each CTA 40 us before its first copy.  (Lengths are read more than
// once; if another stream changes them meanwhile the result is undefined, but every
// place that comes out is clamped to one that exists.)
template <int kUnit, int kEnd>
struct BatchOf {
  const int32_t* ctx_lens;
  int max_ctx, num_seqs;
  int range;                     // sequences per lane; a multiple of 32 where the warp reads them together
  int lane_begin, before, mine;  // this lane's first sequence, the places before it, in its range
  int first_ctx;                 // of its first sequence (small batches)
  int per_segment;               // places of all sequences (of one segment of each)

  static constexpr int kAlone = 4;  // longest range that a lane reads by itself

  // Clamped without a word: whoever handles the sequence reports it.
  __device__ __forceinline__ int ctx_of(int s) const { return max(0, min(max_ctx, __ldg(ctx_lens + s))); }
  __device__ __forceinline__ int places_at(int s, int end) const { return s < end ? places_of<kUnit, kEnd>(ctx_of(s)) : 0; }

  __device__ __forceinline__ BatchOf(const int32_t* lens, int seqs, int longest) {
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
      mine = places_of<kUnit, kEnd>(first_ctx);
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
        while (target >= prefix + places_of<kUnit, kEnd>(ctx) && s + 1 < num_seqs) {
          prefix += places_of<kUnit, kEnd>(ctx);
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
    p.units = max(1, units_of<kUnit>(p.ctx));
    const int rest = max(0, place - prefix * segs);
    const int y = min(segs - 1, rest / (p.units + kEnd));
    p.k = min(p.units + kEnd - 1, rest - y * (p.units + kEnd));
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
        for (int i = lane_begin; i < s; ctx = ctx_of(++i)) prefix += places_of<kUnit, kEnd>(ctx);
      return __shfl_sync(0xffffffffu, prefix, lane);
    }
    int sum = 0;
    for (int i = lane * range + (threadIdx.x & 31); i < s; i += 32) sum += places_of<kUnit, kEnd>(ctx_of(i));
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

struct MergeParams {
  const SegmentJoint* joints;  // one per CTA of the split kernel, or NULL (kFind): one CTA row per segment
  const int32_t* ctx_lens;
  const float* ws_o;
  const float* ws_lse;
  const float2* ws_sum;  // in place of it (kMany)
  __nv_bfloat16* out;
  float* lse;
  int num_seqs, Hq, segs, n_chunks, group, max_blocks_per_seq, ctas;
  int queries;  // query tokens of a sequence
  int rows;     // columns (query heads of a token) per segment, at most
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
// per thread; kVecs threads take four columns each of every kTeams-th partial output,
// the first ones' loads on their way before the weights are known.
// kMany: a segment's columns are the heads of several query tokens (SegmentJoint), and its
// parts come with the reference m_i (log2 units) and the sum l_i of their weights instead of
// their lse: o = sum_i 2^(m_i - M) l_i O_i / sum_i 2^(m_i - M) l_i.  (An lse of 2^24 has no room
// for the logarithm of the sum: parts with equal scores would weigh by a power of e, not
// by their tokens.)
// kCuts: CTAs that share a row, each a part of its d columns.
template <int D, int kUnit, int kEnd, bool kFind, bool kMany, int kCuts = 1>
__device__ __forceinline__ void merge_segment(const MergeParams& p) {
  constexpr int kVecs = D / 4 / kCuts;  // vectors of four columns
  constexpr int kTeams = kMergeThreads / kVecs;
  constexpr int kMergeWarps = kMergeThreads / 32;
  constexpr int kEarly = 3;
  __shared__ float weight[kSplitMaxCtas];
  __shared__ float amount[kMany ? kSplitMaxCtas : 1];
  __shared__ float top[kMergeWarps], sum[kMergeWarps];
  constexpr int kSums = kCuts > 1 ? kMergeWarps : kTeams;  // (with cuts a warp's teams add up by shuffles first)
  __shared__ float4 part[kSums][kVecs];
  __shared__ SegmentJoint found;
  const int r = blockIdx.x;
  if constexpr (kFind) {
    if (threadIdx.x < 32) {
      const BatchOf<kUnit, kEnd> seqs(p.ctx_lens, p.num_seqs, p.max_blocks_per_seq * kDecodeBlockSize);
      const Shares shares(seqs.per_segment * p.segs, p.ctas);
      const int seq = blockIdx.y / p.segs, y = blockIdx.y % p.segs;
      const int ctx = seqs.ctx_of(seq), units = units_of<kUnit>(ctx);
      const int unit = seqs.before_seq(seq) * p.segs + y * places_of<kUnit, kEnd>(ctx);  // the place of its first
      if (threadIdx.x == 0) {
        found.cta = units > 0 ? shares.owner(unit) : 0;
        found.more = units > 0 ? shares.owner(unit + units - 1) - found.cta : 0;
        const int first = y % p.n_chunks * p.rows;  // the chunk's first column
        const int rows = min(p.rows, p.queries * p.group - first);
        if constexpr (kMany) {
          found.row = seq * p.queries * p.Hq + y / p.n_chunks * p.group;
          found.rows = SegmentJoint::pack(rows, first);
        } else {
          found.row = seq * p.Hq + y / p.n_chunks * p.group + first;
          found.rows = rows;
        }
      }
    }
    __syncthreads();
  }
  cudaGridDependencySynchronize();  // launched while the split kernel runs, after all before that had ended
  const SegmentJoint joint = kFind ? found : p.joints[blockIdx.y];
  if (joint.more == 0 || r >= (kMany ? joint.columns() : joint.rows)) return;
  const int used = joint.more + 1;
  auto place = [&](int i) { return static_cast<size_t>(2 * (joint.cta + i) + (i == 0 ? 1 : 0)) * p.rows + r; };
  const int vec = threadIdx.x % kVecs, team = threadIdx.x / kVecs;
  const int col = kCuts == 1 ? vec : blockIdx.z * kVecs + vec;
  auto part_of = [&](int s) { return reinterpret_cast<const float4*>(p.ws_o + place(s) * D)[col]; };
  float4 early[kEarly];
#pragma unroll
  for (int i = 0; i < kEarly; ++i)
    early[i] = team + i * kTeams < used ? part_of(team + i * kTeams) : make_float4(0.f, 0.f, 0.f, 0.f);
  float M = -INFINITY;
  for (int s = threadIdx.x; s < used; s += kMergeThreads) {
    if constexpr (kMany) {
      const float2 x = p.ws_sum[place(s)];
      weight[s] = x.x;
      amount[s] = x.y;
      M = fmaxf(M, x.x);
    } else {
      const float ls = p.ws_lse[place(s)];
      weight[s] = ls;
      M = max_nan(M, ls);
    }
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
    const float w = kMany ? ex2_approx(weight[s] - M) * amount[s] : ex2_approx((weight[s] - ref) * kLog2e);
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
  if constexpr (kCuts > 1) {
#pragma unroll
    for (int x = kVecs; x < 32; x *= 2) {
      o.x += __shfl_xor_sync(0xffffffffu, o.x, x);
      o.y += __shfl_xor_sync(0xffffffffu, o.y, x);
      o.z += __shfl_xor_sync(0xffffffffu, o.z, x);
      o.w += __shfl_xor_sync(0xffffffffu, o.w, x);
    }
    if ((threadIdx.x & 31) < kVecs) part[threadIdx.x >> 5][vec] = o;
  } else {
    part[team][vec] = o;
  }
  __syncthreads();
  if (threadIdx.x < kVecs) {
    if constexpr (kCuts > 1) o = part[0][vec];
#pragma unroll
    for (int x = 1; x < kSums; ++x) {
      const float4 a = part[x][vec];
      o.x += a.x;
      o.y += a.y;
      o.z += a.z;
      o.w += a.w;
    }
    const float inv = W == 0.f ? 0.f : 1.f / W;
    const int at = kMany ? joint.first() + r : r;
    const size_t row = static_cast<size_t>(joint.row) + (kMany ? at / p.group * p.Hq + at % p.group : r);
    reinterpret_cast<uint2*>(p.out + row * D)[col] =
        make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
    if (p.lse != nullptr && col == 0)
      p.lse[row] = W == 0.f ? -INFINITY : kMany ? (M + __log2f(W)) * kLn2 : M + __logf(W);
  }
}

}  // namespace exattn
