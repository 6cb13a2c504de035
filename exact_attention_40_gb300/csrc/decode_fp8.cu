// One-token paged decode over the 8-bit cache (layout in fp8.cuh) for sm_103a, and the
// decode of a few tokens of each sequence at once: split-KV partial attention plus a
// merge of the parts by the references and the sums of their weights.
//
//   s_ij = scale <q_i, kc_j> ks_j,   o_i = sum_j exp(s_ij - m_i) vs_j vc_j / sum_j exp(s_ij - m_i)
//   with kc, vc the codes and ks, vs the scales of j's block.
//
// decode_fp8_split_kernel: the frame of the 4-bit decode (decode_shares.cuh).  The work is
//   units of 16.5 KB, 64 tokens of heads of 128 or 128 of heads of 64, of one (sequence, KV
//   head, chunk of up to 8 NT columns), its segment; a column is a query head of one of the
//   query tokens.  Each CTA takes an equal, contiguous share of all segments' units, found
//   from ctx_lens.  One warp copies, a bulk copy for each block's span; four compute, a block
//   of each unit for a warp (two at d = 64), transposed, so that tokens are the rows of
//   mma.sync m16n8k16 and columns its 8 columns:
//     S^T = K Q^T      A = keys [16 tokens x 16 columns], B = queries
//     O^T += V^T P^T   A = values [16 columns x 16 tokens], B = weights.
//   The scales are kept out of the products: a block's key scale, a power of two, goes into
//   the factor of its scores, and its value scale into the exponent of the weights that the
//   second product takes.  So a code only has to become fp16, one cvt for two, and both enter
//   exactly.  The sum of the weights has a reference m of its own, the weighted values one (m + n)
//   that follows score + value exponent: whatever the blocks' scales, the largest weight of
//   the product lies between 2^7 and 2^15, where fp16 rounds those above 2^-21 of it by at
//   most 2^-11 of themselves and the rest by 2^-32 of it.  Only n, their distance, is held: it
//   has the size of the scales' exponents, so that a score of any size meets m alone, and what
//   the rounding of m brings is the same in both.  The sum takes the weights unrounded
//   in fp32.  (Two exponentials a score: with one reference for both, a block of large values
//   and small weights would be rounded away, or pass what fp16 holds.)
//   Query tokens before the last see fewer keys: their scores are masked in the units that
//   reach past what the first of them sees, and a value that only some see, if it is NaN,
//   is multiplied for each of them apart.
//   What bounds it: HBM for up to 8 columns and long contexts (64 sequences of 8192 tokens, 32
//   heads over 8 of 128: 164 to 168 us = 6.4 to 6.6 TB/s, 95 to 97% of a copy; 64 sequences of 512
//   to 8192 tokens 92.3 us = 6.2 TB/s with the merge).  A unit takes a warp 1100 cycles
//   (scores 370, distances and vote 100, products 360, the rest waits), which twelve warps an SM
//   overlap.  For 9 to 16 columns 168 registers (and, at d = 128, 88 bytes of spills a thread; 28
//   in a cluster) leave room for eight computing warps, whose units take 1390 cycles (440, 150,
//   485), and their latency bounds it: 32 sequences of 512 to 8192 tokens, 96 heads over 8:
//   59.3 us; four queries of 32 heads over 8: 63.6 us = 4.5 TB/s.  More than 16 columns are
//   chunks of 16, each of which reads, converts and multiplies all keys and values again
//   (64 columns, 16 sequences of 4000 tokens: 97.9 us, their bytes' time 20).  Short contexts pay
//   for the ends of their segments, 1450 to 4500 cycles (4096 sequences of 200 tokens, 8 heads
//   over 2: 90.2 us), few of them for the chain ctx_lens -> table -> copies -> merge (one of
//   32768 tokens 16.1 us, its bytes' time 9.9).
//   Small calls take a cluster of 8 CTAs for each segment, which take its units in turn and
//   merge through distributed shared memory: one launch, no workspace (six of up to 1500 tokens
//   4.3 us).
//   Measured and not taken (four queries 64.9 us then): the scores of a unit beside the products
//   of the one before (four queries 85 us, 4096 x 200 104), two chains of a score's products
//   (68, no change for 8 columns), two blocks a warp for 16 columns (68 to 77), the queries of
//   16 columns in shared memory and three CTAs (77, with spills), 16 columns as two chunks of 8
//   (91) or as two warps that read the same blocks (72), two warps that share their weights and
//   split the values' columns (73; both with three CTAs; the latter with 32 columns, for groups
//   of 64: 187 us, 97.9 in chunks of 16), scores by mma.sync on the e4m3 keys themselves with
//   each query as two e4m3 numbers (84: it is slower here than conversions and fp16), tcgen05
//   with units of 128 tokens (74: a unit's hand-overs between copies, conversions, scores,
//   softmax and products take longer than its bytes; at 64 columns 97).
// decode_fp8_combine_kernel: merges the partial outputs of a segment: 2 to 2.6 us of a
//   call, its launch included.
#include <cuda_bf16.h>

#include <cmath>
#include <type_traits>

#include "decode_shares.cuh"
#include "fp8.cuh"
#include "launch.h"
#include "ptx.cuh"

namespace exattn {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;       // that compute; one warp more copies
constexpr int kCtaThreads = kThreads + 32;
constexpr int kBlk = kDecodeBlockSize;
constexpr int kWhole = static_cast<int>(0x80000000u), kNever = 0x40000000;  // of `present`
// Weights are 2^(score - reference), the reference kLift below the running maximum that it
// was taken from, and a new one taken once a score passes it by more than kMost: fp16
// holds weights of up to 2^15.
constexpr float kLift = 7.f;
constexpr float kMost = 15.f;

struct Fp8SplitParams {
  const __nv_bfloat16* q;
  const uint8_t* cache;
  const int32_t* block_table;
  const int32_t* ctx_lens;
  SegmentJoint* joints;  // one per CTA: its last segment, where others go on with it; or NULL
  float* ws_o;    // [2 * ctas][rows][d]
  float2* ws_sum;  // [2 * ctas][rows]: reference (log2 units) and sum of the weights
  __nv_bfloat16* out;
  float* lse;
  unsigned int* status;
  unsigned long long wait_ns;
  int num_seqs, queries, Hq, Hkv, group, n_chunks, num_blocks, max_blocks_per_seq;
  int scale_exponent;     // scale * log2 e = scale_fraction * 2^scale_exponent
  float scale_fraction;   // in [1, 2)
};

template <int D, int NT>
struct Fp8Smem {
  static constexpr int kStages = NT == 1 ? 3 : 4;  // units in flight
  static constexpr int kAccStride = D + 4;  // row of the merge staging, floats
  alignas(128) uint8_t ring[kStages][fp8_unit_blocks(D)][Fp8Span<D>::kBytes];
  float acc[kWarps][8 * NT][kAccStride];
  uint64_t full[kStages];        // a unit's copies have landed
  uint64_t empty[kStages];       // the four warps have used it
  int present[kStages];          // bits of its blocks that were copied, kWhole where all are and are full
  float wm[2][kWarps][8 * NT];   // per-warp references (log2 units) of the weights
  float wn[2][kWarps][8 * NT];   // ... and how far that of the weighted values lies from it
  float wl[2][kWarps][8 * NT];   // per-warp sum of the weights
};

// Waits for the computing warps of the CTA.
__device__ __forceinline__ void compute_barrier() {
  __syncwarp();
  asm volatile("bar.sync 1, %0;" ::"n"(kThreads) : "memory");
}

template <int D, int NT, bool kCluster>
__global__ void __launch_bounds__(kCtaThreads, fp8_decode_ctas(8 * NT)) decode_fp8_split_kernel(const Fp8SplitParams p) {
  using Span = Fp8Span<D>;
  using Smem = Fp8Smem<D, NT>;
  constexpr int kRows = 8 * NT;      // columns (query heads of a token) per CTA
  constexpr int kKSteps = D / 16;    // mma steps of S^T
  constexpr int kMTiles = D / 16;    // mma row tiles of O^T
  constexpr int kKeyVecs = D / 64;   // 16-byte vectors of a lane's key codes per token
  constexpr int kValWords = D / 32;  // words of a lane's value codes per token
  constexpr int kUnit = fp8_unit_blocks(D);
  constexpr int kEnd = fp8_end_units(D, kRows);
  constexpr int kPer = kUnit / kWarps;  // blocks of a unit for each warp
  constexpr int kStages = Smem::kStages;
  constexpr int kStep = kCluster ? kSplitClusterCtas : 1;  // from a CTA's unit to its next
  constexpr int kUnitTokens = kUnit * kBlk;

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
  // Queries as B fragments: column g of the segment's 8 nt ..; step ks,
  // indices 2t, 2t + 1 and 2t + 8, 2t + 9 = columns (D/4) t + 4 ks + 0..3, the
  // columns of the lane's own key codes.
  uint32_t qb[NT][kKSteps][2];
  const int columns = p.queries * p.group;
  auto rows_of = [&](const Place& x) { return min(kRows, columns - x.chunk * kRows); };
  auto token_of = [&](int column) { return p.queries == 1 ? 0 : column / p.group; };  // its query token
  auto row_of = [&](const Place& x, int r) {  // row of the queries and the output of a segment's column
    const int column = x.chunk * kRows + r, token = token_of(column);
    return static_cast<size_t>(x.seq * p.queries + token) * p.Hq + x.head * p.group + (column - token * p.group);
  };
  // Tokens at the end of the context that a segment's column does not see.
  auto unseen = [&](const Place& x, int r) { return p.queries - 1 - token_of(min(columns - 1, x.chunk * kRows + r)); };
  auto load_queries = [&](const Place& x) {
    const int rows = rows_of(x);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const bool real = 8 * nt + g < rows;
      const uint2* row = reinterpret_cast<const uint2*>(p.q + row_of(x, real ? 8 * nt + g : 0) * D + (D / 4) * t);
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
  const uint32_t rank = kCluster ? cta % kSplitClusterCtas : 0;
  // Sequences without a cached token: o = 0, lse = -inf.  A lane looks at one, the
  // warp clears what is found.  (Every sequence's length passes here once, so that
  // one out of range is reported.)
  auto clear_empty = [&]() {
    for (int i = 32 * warp; cta + static_cast<int>(gridDim.x) * i < p.num_seqs; i += kCtaThreads) {
      const int s = cta + gridDim.x * (i + lane);
      for (uint32_t empty = __ballot_sync(0xffffffffu, s < p.num_seqs && ctx_of(s) == 0); empty != 0;
           empty &= empty - 1) {
        const int rows = p.queries * p.Hq;
        const size_t row0 = static_cast<size_t>(cta + gridDim.x * (i + __ffs(empty) - 1)) * rows;
        for (int idx = lane; idx < rows * (D / 8); idx += 32)
          reinterpret_cast<uint4*>(p.out + row0 * D)[idx] = make_uint4(0u, 0u, 0u, 0u);
        if (p.lse != nullptr)
          for (int h = lane; h < rows; h += 32) p.lse[row0 + h] = -INFINITY;
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
    x.units = max(1, units_of<kUnit>(x.ctx));
  };
  const bool copies = warp == kWarps;
  int phys_lane = -1;  // of the copying warp: physical block of block lane % kUnit of a batch's unit lane / kUnit; -1: none
  auto check = [&](int ph) {
    if (ph >= 0 && ph < p.num_blocks) return ph;
    atomicOr(p.status, 2u);  // EXATTN_DEVICE_BOUNDS_BIT
    return -1;
  };
  if constexpr (kCluster) {
    // Every kStep-th unit, so that the table entries and queries need not wait for the
    // context length: the three loads are in flight together.
    static_assert(kSplitClusterTokens / kUnitTokens / kSplitClusterCtas <= 32 / kUnit, "one batch of table entries");
    const int seg = cta / kSplitClusterCtas;
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
    at.units = units_of<kUnit>(at.ctx);
    left = (at.units - static_cast<int>(rank) + kStep - 1) / kStep;
    if (copies && blk * kBlk < at.ctx) phys_lane = check(entry);
  } else {
    // ---- this CTA's share; every warp finds it for itself
    const BatchOf<kUnit, kEnd> seqs(p.ctx_lens, p.num_seqs, max_ctx);
    const Shares shares(seqs.per_segment * segs, gridDim.x);
    const int begin = shares.begin(cta), begin_next = shares.begin(cta + 1);
    left = begin_next - begin;
    if (p.joints != nullptr && threadIdx.x == 0) p.joints[cta].more = 0;
    if (left == 0) {
      clear_empty();
      return;
    }
    at = seqs.find(begin, segs, p.n_chunks);
    if (at.k >= at.units) {  // the end of a segment that others compute
      left -= at.units + kEnd - at.k;
      if (left <= 0) {
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
    // A batch: as many units of one segment as lanes have blocks; lane kUnit i + b has unit i's block b.
    struct Entries {
      int units, raw;  // raw: this lane's table entry, if it has one (`mine`)
      bool mine;
      int past;  // tokens past the batch's first unit that the first of the queries sees
      const uint8_t* head;
    };
    auto load_batch = [&]() {
      Entries e;
      if (to.k == to.units) {
        next_segment(to);
        // its queries into the L1 cache, for the computing warps
        if (lane < rows_of(to) * D / 64)
          asm volatile("prefetch.global.L1 [%0];" ::"l"(p.q + row_of(to, lane / (D / 64)) * D + lane % (D / 64) * 64));
      }
      e.units = min(32 / kUnit, min(to.units - to.k, to_load));
      const int blk = to.k * kUnit + lane;
      e.mine = lane < e.units * kUnit && blk * kBlk < to.ctx;
      e.raw = e.mine ? __ldg(p.block_table + static_cast<size_t>(to.seq) * p.max_blocks_per_seq + blk) : -1;
      e.past = to.ctx - (p.queries - 1) - (to.k + 1) * kUnitTokens;
      e.head = p.cache + static_cast<size_t>(to.head) * Span::kBytes;
      to.k += e.units;
      to_load -= e.units;
      if (to.k == to.units) to_load = max(0, to_load - kEnd);
      return e;
    };
    Entries now, next;  // the entries of the next batch are on their way while this one's blocks are copied
    if constexpr (kCluster)
      now = Entries{left, phys_lane, phys_lane >= 0, at.ctx - (p.queries - 1) - (at.k + 1) * kUnitTokens,
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
      const uint32_t present = (__ballot_sync(0xffffffffu, phys_lane >= 0) >> (batch_at * kUnit)) & ((1u << kUnit) - 1u);
      if (lane / kUnit == batch_at) {
        const int b = lane % kUnit;
        if (b == 0) sm.present[st] = now.past >= 0 && present == (1u << kUnit) - 1u ? kWhole : static_cast<int>(present);
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
      now.past -= kStep * kUnitTokens;
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
  // swapped for odd t, so that the loads of eight lanes at a time fall on all banks.
  const int tok_s = g ^ ((g >> 1) & 1);    // this lane's score rows: tok_s, tok_s + 8
  const int tok_v0 = 2 * t + (t & 1);      // mma index 2t (and 2t + 8: + 8)
  const int tok_v1 = 2 * t + 1 - (t & 1);  // mma index 2t + 1 (and 2t + 9: + 8)
  const uint32_t ring0 = smem_u32(sm.ring[0][kPer * warp]);
  // (the turn of token n + 8 is that of n; the second chunk's place is the first's with
  // its lowest bit changed)
  const uint32_t key_at = ring0 + Span::kKeyCodes + tok_s * Span::kRow + ((kKeyVecs * t) ^ fp8_turn<D>(tok_s)) * 16;
  auto value_at = [&](int tok) {  // D/8 columns from column (D/8) g
    const int chunk = D == 128 ? g : g >> 1;
    return ring0 + Span::kValueCodes + tok * Span::kRow + (chunk ^ fp8_turn<D>(tok)) * 16 + (D == 128 ? 0 : (g & 1) * 8);
  };
  const uint32_t val_at0 = value_at(tok_v0), val_at1 = value_at(tok_v1);
  constexpr int kCodes8 = 8 * Span::kRow;  // eight tokens on
  bool ok = true;  // no wait has run out
  int st = 0;      // stage of the next unit
  uint32_t parity = 0;

  // In a cluster: this CTA's outcome, its weights' references and their sums, in the ring,
  // which every copy has left by then.
  float* const cluster_o = reinterpret_cast<float*>(&sm.ring[0][0][0]);
  float* const cluster_ref = cluster_o + kRows * D;
  float* const cluster_sum = cluster_ref + kRows;
  if constexpr (kCluster)
    if (left == 0)
      for (int idx = threadIdx.x; idx < kRows * D; idx += kThreads) {
        cluster_o[idx] = 0.f;
        if (idx < kRows) {
          cluster_ref[idx] = kNoScore;
          cluster_sum[idx] = 0.f;
        }
      }

  const bool two_halves = columns <= 4 * NT;  // staging rows for two segments
  int buf = 0;
#pragma unroll 1
  while (left > 0) {  // segments of this CTA's share
    const int n_units = kCluster ? left : min(at.units - at.k, left);

    int exponent[NT][2];  // of the power of two that columns 2t, 2t + 1 were divided by, and of the scores' factor
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
#pragma unroll
      for (int ks = 0; ks < kKSteps; ++ks)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const uint32_t v = qb[nt][ks][x];
          qb[nt][ks][x] = pack_f16x2(__uint_as_float(v << 16) * down, __uint_as_float(v & 0xFFFF0000u) * down);
        }
      exponent[nt][0] = __shfl_sync(0xffffffffu, e + p.scale_exponent, 8 * t);
      exponent[nt][1] = __shfl_sync(0xffffffffu, e + p.scale_exponent, 8 * t + 4);
    }
    // Whether a block of this segment can have a factor past what fp32 holds, though the scores
    // need not: a column's largest element may meet codes of 0, and the next lie far below it.
    // All units then go through the code with the masks, which takes such a factor in two
    // steps (4096 x 200 tokens, most units masked, 89.2 to 90.1 us; in the code of whole units four
    // queries of 32 sequences 63.5 to 64.8).
    int top_exponent = max(exponent[0][0], exponent[0][1]);
    if constexpr (NT == 2) top_exponent = max(top_exponent, max(exponent[NT - 1][0], exponent[NT - 1][1]));
    const int counts_whole = __any_sync(0xffffffffu, top_exponent + kFp8HighExponent > 127) ? kNever : kWhole;

    // Of columns 2t, 2t + 1: m, the reference of the weights, and n, what the weighted values'
    // lies above it; l, the sum of this lane's tokens' weights.
    float m[NT][2], n[NT][2], l[NT][2];
    float acc[kMTiles][NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      m[nt][0] = m[nt][1] = kNoScore;
      n[nt][0] = n[nt][1] = l[nt][0] = l[nt][1] = 0.f;
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
      // Whether all tokens of this warp's blocks count for every query; else, how many of
      // each block for the last one (each query before it sees one less).
      const bool full = present == counts_whole;
      int n_valid[kPer];
      int most_valid = kBlk;
#pragma unroll
      for (int b = 0; b < kPer; ++b) n_valid[b] = kBlk;
      if (!full) {
        const int tokens = at.ctx - ((at.k + i * kStep) * kUnit + kPer * warp) * kBlk;
        most_valid = 0;
#pragma unroll
        for (int b = 0; b < kPer; ++b) {
          n_valid[b] = present == kWhole || present >> (kPer * warp + b) & 1 ? tokens - b * kBlk : 0;
          most_valid = max(most_valid, n_valid[b]);
        }
      }
      // Units that count whole have code of their own, without the masks: the loop over
      // them then fits the instruction caches better (four queries of 32 sequences 64.9 us
      // with one code for both, 62.9 with two; 96 heads over 8 60.8 and 58.7).
      auto compute = [&](auto whole_unit) {
        constexpr bool full = decltype(whole_unit)::value;
        // ---- S^T = K Q^T, with the score's factor and the key scale
        float c[kPer][NT][4];
        float value_exp[kPer];  // exponent of the block's value scale
        auto scores = [&](auto block) {
          constexpr int b = decltype(block)::value, kSpan = b * Span::kBytes;
          uint32_t ka[kKeyVecs][4], kb[kKeyVecs][4], s[2];
          lds_words<kSpan>(key_at + stage, ka[0]);
          lds_words<kSpan + kCodes8>(key_at + stage, kb[0]);
          if constexpr (kKeyVecs == 2) {
            lds_words<kSpan>((key_at ^ 16u) + stage, ka[1]);
            lds_words<kSpan + kCodes8>((key_at ^ 16u) + stage, kb[1]);
          }
          lds_words<kSpan + Span::kScales>(ring0 + stage, s);
#pragma unroll
          for (int w = 0; w < kKSteps; ++w) {
            uint32_t h0, h1, h2, h3;
            e4m3x4_to_f16(ka[w / 4][w % 4], h0, h2);
            e4m3x4_to_f16(kb[w / 4][w % 4], h1, h3);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              if (w == 0)
                mma_f16_16816_first(c[b][nt], h0, h1, h2, h3, qb[nt][0][0], qb[nt][0][1]);
              else
                mma_f16_16816(c[b][nt], h0, h1, h2, h3, qb[nt][w][0], qb[nt][w][1]);
            }
          }
          const int key_exp = static_cast<int>(s[0] >> 23 & 255u);
          value_exp[b] = static_cast<float>(static_cast<int>(s[1] >> 23 & 255u) - 127);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            auto times = [&](float f0, float f1) {
#pragma unroll
              for (int y = 0; y < 4; y += 2)
                f2_unpack(f2_mul(f2_pack(c[b][nt][y], c[b][nt][y + 1]), f2_pack(f0, f1)), c[b][nt][y], c[b][nt][y + 1]);
            };
            auto power = [](int exponent) { return __uint_as_float(static_cast<uint32_t>(exponent) << 23); };
            // (a factor is kept finite and above zero: a product of 0 stays one, whatever the scales)
            const int e0 = exponent[nt][0] + key_exp, e1 = exponent[nt][1] + key_exp;
            times(p.scale_fraction * power(max(1, min(254, e0))), p.scale_fraction * power(max(1, min(254, e1))));
            // what its exponent lacked (2^254 takes the smallest product past fp32)
            if (!full) times(power(127 + max(0, min(127, e0 - 254))), power(127 + max(0, min(127, e1 - 254))));
          }
        };
        scores(std::integral_constant<int, 0>());
        if constexpr (kPer == 2) scores(std::integral_constant<int, 1>());
        // ---- online softmax: c[b][nt][j] is token tok_s, column 2t + j, c[b][nt][2 + j]
        // token tok_s + 8.  Tokens that do not count are masked here and their values
        // zeroed below (the slots may hold anything).
        if (!full) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const int less = unseen(at, 8 * nt + 2 * t + j);
#pragma unroll
              for (int b = 0; b < kPer; ++b) {
                if (tok_s >= n_valid[b] - less) c[b][nt][j] = -INFINITY;
                if (tok_s + 8 >= n_valid[b] - less) c[b][nt][2 + j] = -INFINITY;
              }
            }
          __syncwarp();  // the lanes together again for the next mma
        }
        // Exponents relative to the references, x of the weights and y of the weighted
        // values: a block's value scale is part of y, so that what fp16 rounds is the
        // token's part of the output.  The references follow the running maxima only
        // when these have grown by more than kMost - kLift, which is rare after the
        // first blocks: most blocks pay one vote.  A score is rounded before the
        // reference is taken from it, as it was when it gave that: in one fused
        // operation the largest itself would lie off by the rounding, which passes all
        // that fp16 holds once scores come to 2^28.  y is taken from x: a sum of the
        // score's size and the value exponent would be rounded to the score's last place.
        float x[kPer][NT][4], y[kPer][NT][4];
        auto distances = [&]() {
          float most = -INFINITY;
#pragma unroll
          for (int b = 0; b < kPer; ++b)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              const uint64_t mm = f2_pack(m[nt][0], m[nt][1]);
              const uint64_t up = f2_pack(value_exp[b] - n[nt][0], value_exp[b] - n[nt][1]);
#pragma unroll
              for (int z = 0; z < 4; z += 2) {
                const uint64_t above = f2_sub(f2_pack(c[b][nt][z], c[b][nt][z + 1]), mm);
                f2_unpack(above, x[b][nt][z], x[b][nt][z + 1]);
                f2_unpack(f2_add(above, up), y[b][nt][z], y[b][nt][z + 1]);
                most = max3f(most, max3f(x[b][nt][z], x[b][nt][z + 1], y[b][nt][z]), y[b][nt][z + 1]);
              }
            }
          return most;
        };
        if (__any_sync(0xffffffffu, distances() > kMost)) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              float top[kPer];  // of each block
#pragma unroll
              for (int b = 0; b < kPer; ++b) {
                top[b] = fmaxf(c[b][nt][j], c[b][nt][2 + j]);
#pragma unroll
                for (int z = 4; z < 32; z *= 2) top[b] = fmaxf(top[b], __shfl_xor_sync(0xffffffffu, top[b], z));
              }
              const float mn = fmaxf(m[nt][j], fmaxf(top[0], top[kPer - 1]) - kLift);
              const float top_value = fmaxf(top[0] - mn + value_exp[0], top[kPer - 1] - mn + value_exp[kPer - 1]);
              const float down = m[nt][j] - mn, kept = down + n[nt][j], nn = fmaxf(kept, top_value - kLift);
              l[nt][j] *= ex2_approx(down);
              const float alpha = ex2_approx(kept - nn);
              m[nt][j] = mn;
              n[nt][j] = nn;
#pragma unroll
              for (int mt = 0; mt < kMTiles; ++mt) {
                acc[mt][nt][j] *= alpha;
                acc[mt][nt][2 + j] *= alpha;
              }
            }
          distances();
        }
        // ---- O^T += V^T P^T: row tile mt, row g = column (D/8) g + 2 mt, row
        // g + 8 the next one
        auto products = [&](auto block) {
          constexpr int b = decltype(block)::value, kSpan = b * Span::kBytes;
          uint32_t va0[kValWords], va1[kValWords], vb0[kValWords], vb1[kValWords];
          lds_words<kSpan>(val_at0 + stage, va0);
          lds_words<kSpan>(val_at1 + stage, va1);
          lds_words<kSpan + kCodes8>(val_at0 + stage, vb0);
          lds_words<kSpan + kCodes8>(val_at1 + stage, vb1);
          uint32_t pb[NT][2];
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            float w[4];
#pragma unroll
            for (int z = 0; z < 4; ++z) {
              l[nt][z & 1] += ex2_approx(x[b][nt][z]);
              w[z] = ex2_approx(y[b][nt][z]);
            }
            pb[nt][0] = transpose8x8(pack_f16x2(w[0], w[1]));
            pb[nt][1] = transpose8x8(pack_f16x2(w[2], w[3]));
          }
          bool hidden_nan = false;  // a NaN among the values that some of the queries do not see
          auto keep_below = [&](int n_tokens) {
#pragma unroll
            for (int w = 0; w < kValWords; ++w) {
              if (tok_v0 >= n_tokens) va0[w] = 0u;
              if (tok_v1 >= n_tokens) va1[w] = 0u;
              if (tok_v0 + 8 >= n_tokens) vb0[w] = 0u;
              if (tok_v1 + 8 >= n_tokens) vb1[w] = 0u;
            }
          };
          if (!full) {
            keep_below(n_valid[b]);
            if (p.queries > 1) {
              const int all_see = n_valid[b] - (p.queries - 1);
              auto nan_at = [&](int tok, const uint32_t (&v)[kValWords]) {
#pragma unroll
                for (int w = 0; w < kValWords; ++w)
                  hidden_nan |= tok >= all_see && (((v[w] & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u) != 0u;
              };
              nan_at(tok_v0, va0);
              nan_at(tok_v1, va1);
              nan_at(tok_v0 + 8, vb0);
              nan_at(tok_v1 + 8, vb1);
            }
            hidden_nan = __any_sync(0xffffffffu, hidden_nan);
          }
          // into(mt, a, b, c, d): the mma of row tile mt
          auto tiles = [&](auto into) {
#pragma unroll
            for (int w = 0; w < kValWords; ++w) {
              // bytes of (token 2t, token 2t + 1) pairs of columns 4w, 4w + 1, then the next two
              uint32_t h0, h1, h2, h3;
              e4m3x4_to_f16(__byte_perm(va0[w], va1[w], 0x5140), h0, h1);
              e4m3x4_to_f16(__byte_perm(vb0[w], vb1[w], 0x5140), h2, h3);
              into(2 * w, h0, h1, h2, h3);
              e4m3x4_to_f16(__byte_perm(va0[w], va1[w], 0x7362), h0, h1);
              e4m3x4_to_f16(__byte_perm(vb0[w], vb1[w], 0x7362), h2, h3);
              into(2 * w + 1, h0, h1, h2, h3);
            }
          };
          if (!hidden_nan) {
            tiles([&](int mt, uint32_t h0, uint32_t h1, uint32_t h2, uint32_t h3) {
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) mma_f16_16816(acc[mt][nt], h0, h1, h2, h3, pb[nt][0], pb[nt][1]);
            });
          } else {
            // a weight of 0 would not keep the NaN out of the queries before it: each query's
            // sums are taken with only the values that it sees
#pragma unroll 1
            for (int less = 0; less < p.queries; ++less) {
              keep_below(n_valid[b] - less);
              __syncwarp();
              tiles([&](int mt, uint32_t h0, uint32_t h1, uint32_t h2, uint32_t h3) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                  float sum[4];
                  mma_f16_16816_first(sum, h0, h1, h2, h3, pb[nt][0], pb[nt][1]);
#pragma unroll
                  for (int z = 0; z < 4; ++z)
                    if (unseen(at, 8 * nt + 2 * t + (z & 1)) == less) acc[mt][nt][z] += sum[z];
                }
              });
            }
          }
        };
        products(std::integral_constant<int, 0>());
        if constexpr (kPer == 2) products(std::integral_constant<int, 1>());
      };
      if (full)
        compute(std::integral_constant<bool, true>());
      else if (most_valid > 0)
        compute(std::integral_constant<bool, false>());
      __syncwarp();  // all lanes are done with this stage
      if (lane == 0) mbar_arrive(&sm.empty[st]);
      if (++st == kStages) {
        st = 0;
        parity ^= 1u;
      }
    }

    const int rows_here = rows_of(at);
    const int chunk0 = at.chunk * kRows;  // the segment's first column
    const int segment_row = at.seq * p.queries * p.Hq + at.head * p.group;
    const Place here = at;
    const bool starts = at.k == 0;
    const bool ends = at.k + n_units == at.units;
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
          sm.wn[buf][warp][r] = n[nt][j];
          sm.wl[buf][warp][r] = l[nt][j];
        }
        if (r < rows_here)
#pragma unroll
          for (int mt = 0; mt < kMTiles; mt += 2)
            *reinterpret_cast<float4*>(&sm.acc[warp][half + r][(D / 8) * g + 2 * mt]) =
                make_float4(acc[mt][nt][j], acc[mt][nt][2 + j], acc[mt + 1][nt][j], acc[mt + 1][nt][2 + j]);
      }
    left -= n_units;
    if (!kCluster && ends) left = max(0, left - kEnd);
    if (left > 0) {  // the next segment's queries arrive during the merge
      next_segment(at);
      load_queries(at);
    }
    compute_barrier();
    // A lane forms one row's factors: of each warp's sums, then from the values' reference
    // back to the weights', in two steps as their distance may pass what fp32's exponents
    // hold.  A share all of whose scores are -inf, or whose blocks are all missing, sees nothing.
    const int own = lane % kRows;
    float M = kNoScore, N = -INFINITY, L = 0.f, part[kWarps];
#pragma unroll
    for (int w = 0; w < kWarps; ++w) M = fmaxf(M, sm.wm[buf][w][own]);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float down = sm.wm[buf][w][own] - M;
      part[w] = down + sm.wn[buf][w][own];  // of its values, the reference's distance from M
      N = fmaxf(N, part[w]);
      L += ex2_approx(down) * sm.wl[buf][w][own];
    }
#pragma unroll
    for (int w = 0; w < kWarps; ++w) part[w] = ex2_approx(part[w] - N);
    const float inv = L == 0.f ? 0.f : __fdividef(1.f, L), half_way = ex2_approx(0.5f * N);
    const bool whole = starts && ends;
    // the log-sum-exp, or the reference, which goes with the sum to where the parts merge
    const float own_ref = kCluster || !whole ? M : L == 0.f ? -INFINITY : (M + __log2f(L)) * kLn2;
    const int own_row = whole && own < rows_here ? static_cast<int>(row_of(here, own)) : 0;
    constexpr int kRowLanes = D / 4, kAtOnce = 32 / kRowLanes;  // lanes of a row, rows of a warp
#pragma unroll 1
    for (int r0 = warp * kAtOnce; r0 < rows_here; r0 += kWarps * kAtOnce) {
      const int r = r0 + lane / kRowLanes, col = lane % kRowLanes * 4;
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float wt = __shfl_sync(0xffffffffu, part[w], r);
        const float4 a = *reinterpret_cast<const float4*>(&sm.acc[w][half + r][col]);
        o.x += wt * a.x;
        o.y += wt * a.y;
        o.z += wt * a.z;
        o.w += wt * a.w;
      }
      const float by = __shfl_sync(0xffffffffu, inv, r), h = __shfl_sync(0xffffffffu, half_way, r);
      const float from = __shfl_sync(0xffffffffu, own_ref, r), sum = __shfl_sync(0xffffffffu, L, r);
      const int row_out = __shfl_sync(0xffffffffu, own_row, r);
      if (r >= rows_here) continue;
      auto scaled = [&](float x) { return x * by * h * h; };
      o = make_float4(scaled(o.x), scaled(o.y), scaled(o.z), scaled(o.w));
      if constexpr (kCluster) {
        *reinterpret_cast<float4*>(cluster_o + r * D + col) = o;
        if (col == 0) {
          cluster_ref[r] = from;
          cluster_sum[r] = sum;
        }
      } else if (whole) {
        const size_t row = row_out;
        *reinterpret_cast<uint2*>(p.out + row * D + col) = make_uint2(pack_bf16x2(o.x, o.y), pack_bf16x2(o.z, o.w));
        if (p.lse != nullptr && col == 0) p.lse[row] = from;
      } else {
        const size_t row = static_cast<size_t>(2 * cta + (starts ? 1 : 0)) * kRows + r;
        *reinterpret_cast<float4*>(p.ws_o + row * D + col) = o;
        if (col == 0) p.ws_sum[row] = make_float2(from, sum);
      }
    }
    __syncwarp();
    if (left == 0) {
      // the only segment that can go on into further CTAs is the last
      if (!kCluster && p.joints != nullptr && starts && !ends && threadIdx.x == 0)
        p.joints[cta] = SegmentJoint{cta, joint_parts, segment_row, SegmentJoint::pack(rows_here, chunk0)};
      break;
    }
    buf ^= 1;
  }
  __syncwarp();
  if constexpr (kCluster) {
    // ---- the cluster's CTAs merge: W = sum_i 2^(m_i - M) l_i, o = sum_i 2^(m_i - M) l_i O_i / W
    const int rows_here = rows_of(at);
    cluster_barrier();
    for (int idx = threadIdx.x * kSplitClusterCtas + rank; idx < rows_here * (D / 4); idx += kThreads * kSplitClusterCtas) {
      const int r = idx / (D / 4), col = idx % (D / 4) * 4;
      float from[kSplitClusterCtas], sum[kSplitClusterCtas];
      float4 part[kSplitClusterCtas];
#pragma unroll
      for (int i = 0; i < kSplitClusterCtas; ++i) {
        from[i] = cluster_load(cluster_ref + r, i);
        sum[i] = cluster_load(cluster_sum + r, i);
        part[i] = cluster_load4(cluster_o + r * D + col, i);
      }
      float M = from[0];
#pragma unroll
      for (int i = 1; i < kSplitClusterCtas; ++i) M = fmaxf(M, from[i]);
      float W = 0.f;
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int i = 0; i < kSplitClusterCtas; ++i) {
        const float w = ex2_approx(from[i] - M) * sum[i];
        W += w;
        o.x = fmaf(w, part[i].x, o.x);
        o.y = fmaf(w, part[i].y, o.y);
        o.z = fmaf(w, part[i].z, o.z);
        o.w = fmaf(w, part[i].w, o.w);
      }
      const float inv = W == 0.f ? 0.f : 1.f / W;
      const size_t row = row_of(at, r);
      *reinterpret_cast<uint2*>(p.out + row * D + col) =
          make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
      if (p.lse != nullptr && col == 0) p.lse[row] = W == 0.f ? -INFINITY : (M + __log2f(W)) * kLn2;
    }
    cluster_barrier();  // nobody's shared memory goes away before the others have read it
  } else {
    clear_empty();
  }
}

template <int D, int NT, bool kFind, int kCuts>
__global__ void __launch_bounds__(kMergeThreads, kFind ? 5 : 6) decode_fp8_combine_kernel(const MergeParams p) {
  merge_segment<D, fp8_unit_blocks(D), fp8_end_units(D, 8 * NT), kFind, true, kCuts>(p);
}

template <int D, int NT, bool kCluster>
cudaError_t launch_split(const Fp8SplitParams& sp, int ctas, cudaStream_t stream) {
  const size_t smem = sizeof(Fp8Smem<D, NT>) + 128;
  static std::atomic<int> smem_set[64] = {};
  cudaError_t e = smem_limit_once(reinterpret_cast<const void*>(decode_fp8_split_kernel<D, NT, kCluster>),
                                  static_cast<int>(smem), smem_set);
  if (e != cudaSuccess) return e;
  return launch_overlapped(decode_fp8_split_kernel<D, NT, kCluster>, ctas, kCtaThreads, smem, stream,
                           kCluster ? kSplitClusterCtas : 1, sp);
}

template <int D>
cudaError_t launch_d(const DecodeFp8Args& a, const DeviceGuard& g, cudaStream_t stream) {
  const Fp8Plan& plan = a.plan;
  Fp8SplitParams sp;
  sp.q = static_cast<const __nv_bfloat16*>(a.q);
  sp.cache = static_cast<const uint8_t*>(a.kv_cache);
  sp.block_table = a.block_table;
  sp.ctx_lens = a.ctx_lens;
  uint8_t* ws = static_cast<uint8_t*>(a.workspace);
  sp.joints = plan.joints > 0 ? reinterpret_cast<SegmentJoint*>(ws) : nullptr;
  sp.ws_o = reinterpret_cast<float*>(ws + plan.joint_bytes());
  sp.ws_sum = reinterpret_cast<float2*>(ws + plan.joint_bytes() + plan.part_bytes(D));
  sp.out = static_cast<__nv_bfloat16*>(a.out);
  sp.lse = a.lse;
  sp.status = g.status;
  sp.wait_ns = g.wait_ns;
  sp.num_seqs = a.num_seqs;
  sp.queries = a.queries;
  sp.Hq = a.Hq;
  sp.Hkv = a.Hkv;
  sp.group = a.Hq / a.Hkv;
  sp.n_chunks = plan.chunks;
  sp.num_blocks = a.num_blocks;
  sp.max_blocks_per_seq = a.max_blocks_per_seq;
  // (rounded once, also where the scale itself has fewer bits)
  sp.scale_fraction = static_cast<float>(2.0 * std::frexp(static_cast<double>(a.scale) * 1.4426950408889634, &sp.scale_exponent));
  sp.scale_exponent -= 1;
  if (sp.scale_fraction == 2.f) {
    sp.scale_fraction = 1.f;
    sp.scale_exponent += 1;
  }
  if (plan.cluster)
    return plan.rows == 8 ? launch_split<D, 1, true>(sp, plan.ctas, stream)
                          : launch_split<D, 2, true>(sp, plan.ctas, stream);
  const cudaError_t e = plan.rows == 8 ? launch_split<D, 1, false>(sp, plan.ctas, stream)
                                       : launch_split<D, 2, false>(sp, plan.ctas, stream);
  if (e != cudaSuccess || !plan.shared) return e;

  MergeParams cp;
  cp.joints = sp.joints;
  cp.ctx_lens = a.ctx_lens;
  cp.ws_o = sp.ws_o;
  cp.ws_sum = sp.ws_sum;
  cp.out = sp.out;
  cp.lse = a.lse;
  cp.num_seqs = a.num_seqs;
  cp.Hq = a.Hq;
  cp.segs = a.Hkv * plan.chunks;
  cp.n_chunks = plan.chunks;
  cp.group = sp.group;
  cp.queries = a.queries;
  cp.max_blocks_per_seq = a.max_blocks_per_seq;
  cp.ctas = plan.ctas;
  cp.rows = plan.rows;
  const int columns = a.queries * sp.group;
  const int rows = columns < plan.rows ? columns : plan.rows;
  auto merge = [&](auto kernel, int segments, int cuts) {
    return launch_overlapped(kernel, dim3(rows, segments, cuts), kMergeThreads, 0, stream, 1, cp);
  };
  auto merge_of = [&](auto nt) {
    constexpr int NT = decltype(nt)::value;
    const int segments = a.num_seqs * cp.segs;
    if (plan.joints > 0) return merge(decode_fp8_combine_kernel<D, NT, false, 1>, plan.joints, 1);
    // Few rows are cut, so that all their partial outputs are on their way at once: one
    // sequence of 8000 tokens (32 rows) 8.3 us with four cuts, 8.6 with two, 8.9 with none;
    // four queries of two (256 rows) 15.1, 13.0 and 13.4; nine sequences (288) 15.8, 13.5, 13.4.
    if (rows * segments <= 64) return merge(decode_fp8_combine_kernel<D, NT, true, 4>, segments, 4);
    if (rows * segments <= 256) return merge(decode_fp8_combine_kernel<D, NT, true, 2>, segments, 2);
    return merge(decode_fp8_combine_kernel<D, NT, true, 1>, segments, 1);
  };
  return plan.rows == 8 ? merge_of(std::integral_constant<int, 1>()) : merge_of(std::integral_constant<int, 2>());
}

}  // namespace

cudaError_t launch_decode_fp8(const DecodeFp8Args& a, const DeviceGuard& g, cudaStream_t stream) {
  return a.d == 64 ? launch_d<64>(a, g, stream) : launch_d<128>(a, g, stream);
}

}  // namespace exattn
