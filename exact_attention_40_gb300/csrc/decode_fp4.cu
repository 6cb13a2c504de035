// One-token paged decode over the 4-bit cache (layout in fp4.cuh) for sm_103a:
// split-KV partial attention plus a log-sum-exp merge, as the bf16 decode.
//
// decode_fp4_split_kernel: one CTA per (sequence, kv head, chunk of up to
//   8 NT query heads, split).  A sequence's blocks are shared out evenly over
//   the splits it uses.  Each warp owns every kWarps-th block of the split and
//   streams the blocks' spans (18 d bytes: codes and scales of keys and
//   values) through a private shared-memory ring, one bulk copy a block.
//   Everything is computed transposed, so that the 16 tokens of a block are
//   the rows of mma.sync m16n8k16 and the few query heads of the group its 8
//   columns (as rows, half or more of them would be padding):
//     S^T = K Q^T   A = keys [16 tokens x 16 columns], B = queries;
//     O^T += V^T P^T  A = values [16 columns x 16 tokens], B = weights.
//   Codes become fp16 by the cvt of packed e2m1 and are multiplied by their
//   scale there; the product has 6 significant bits, so keys and values enter
//   the tensor core exactly.  Queries are bf16: each is multiplied by a power of
//   two that brings its largest element to [1, 2), after which fp16 holds
//   every element that is not 2^-24 of the largest or less exactly, and the
//   power goes into the score's factor.  Both products sum over their inner index
//   in any order, so which column or token an mma index stands for is free: it
//   is chosen so that a lane reads its codes as one vector each, from one or two
//   scale groups.  Weights are rounded to fp16 (at most 2^-12 relative; the output is
//   rounded to bf16, 2^-9) and the output is divided by the sum of the
//   rounded weights, the log-sum-exp keeps the unrounded.
// decode_fp4_combine_kernel: merges the splits of a (sequence, head).
#include <cuda_bf16.h>

#include "fp4.cuh"
#include "launch.h"
#include "ptx.cuh"

namespace exattn {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kStages = 3;  // pairs of blocks in flight per warp
constexpr int kBlk = kDecodeBlockSize;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.69314718055994531f;
constexpr uint32_t kOnes = 0x3C003C00u;  // fp16 (1, 1)
constexpr float kNoScore = -3.0e38f;  // below any score; -inf would give inf - inf

struct Fp4SplitParams {
  const __nv_bfloat16* q;
  const uint8_t* cache;
  const int32_t* block_table;
  const int32_t* ctx_lens;
  float* ws_o;    // [num_seqs, Hq, splits, d]
  float* ws_lse;  // [num_seqs, Hq, splits]
  __nv_bfloat16* out;
  float* lse;
  unsigned int* status;
  unsigned long long wait_ns;
  int Hq, Hkv, group, n_chunks, num_blocks, max_blocks_per_seq, splits;
  float scale_log2;  // scale * k_scale * log2 e
  float v_scale;
};

__device__ __forceinline__ int clamp_ctx(int n, int max_ctx, unsigned int* status) {
  if (n < 0 || n > max_ctx) {
    atomicOr(status, 2u);  // EXATTN_DEVICE_BOUNDS_BIT
    n = n < 0 ? 0 : max_ctx;
  }
  return n;
}

// Blocks each used split of a sequence of n_blk blocks takes.
__device__ __forceinline__ int blocks_per_split(int n_blk, int splits) {
  const int per = (n_blk + splits - 1) / splits;
  return per > kFp4MinSplitBlocks ? per : kFp4MinSplitBlocks;
}

__device__ __forceinline__ void mma_f16_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Transposes an 8x8 matrix of 16-bit elements held one row per four lanes.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

template <int W>
__device__ __forceinline__ void lds_words(uint32_t addr, uint32_t (&w)[W]) {
  if constexpr (W == 4) {
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                 : "r"(addr));
  } else if constexpr (W == 2) {
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(addr));
  } else {
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(w[0]) : "r"(addr));
  }
}

__device__ __forceinline__ uint32_t lds_u8(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(addr));
  return v;
}

__device__ __forceinline__ uint32_t lds_u16(uint32_t addr) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(addr));
  return v;
}

template <int D>
struct Fp4Smem {
  alignas(128) uint8_t ring[kWarps][kStages][2 * Fp4Span<D>::kBytes];
  uint64_t full[kWarps][kStages];
  float wm[kWarps][16];   // per-warp running max (log2 units)
  float wl[kWarps][16];   // per-warp sum of the weights
  float wlr[kWarps][16];  // ... of the rounded weights
};

template <int D, int NT>
__global__ void __launch_bounds__(kThreads, NT == 1 ? 4 : 3) decode_fp4_split_kernel(const Fp4SplitParams p) {
  using Span = Fp4Span<D>;
  constexpr int kRows = 8 * NT;      // query heads per CTA
  constexpr int kKSteps = D / 16;    // mma steps of S^T
  constexpr int kMTiles = D / 16;    // mma row tiles of O^T
  constexpr int kKeyWords = D / 32;  // 32-bit words of a lane's key codes per token
  constexpr int kValWords = D / 64;  // ... value codes
  constexpr int kAccStride = D + 4;  // row of the merge staging, floats

  extern __shared__ uint8_t smem_raw[];
  Fp4Smem<D>& sm = *reinterpret_cast<Fp4Smem<D>*>((reinterpret_cast<uintptr_t>(smem_raw) + 127) &
                                                  ~static_cast<uintptr_t>(127));
  static_assert(sizeof(float) * kWarps * kRows * kAccStride <= sizeof(Fp4Smem<D>::ring), "merge staging");

  cudaTriggerProgrammaticLaunchCompletion();  // the merge may launch and wait while the last splits run
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int g = lane >> 2;  // mma group: rows g, g + 8 of A and the accumulator, column g of B
  const int t = lane & 3;   // thread in group
  const int split = blockIdx.x;
  const int hkv = blockIdx.y / p.n_chunks;
  const int chunk = blockIdx.y % p.n_chunks;
  const int seq = blockIdx.z;

  const int hq0 = hkv * p.group + chunk * kRows;
  const int rows_here = min(kRows, p.group - chunk * kRows);
  const int ctx = clamp_ctx(__ldg(p.ctx_lens + seq), p.max_blocks_per_seq * kBlk, p.status);
  const int seq_blk = (ctx + kBlk - 1) / kBlk;
  const int per = blocks_per_split(seq_blk, p.splits);
  const int blk0 = split * per;
  const int n_blk = min(per, seq_blk - blk0);
  if (n_blk <= 0) {  // whole CTA: nothing of this sequence here
    if (split == 0 && p.splits == 1) {
      for (int idx = threadIdx.x; idx < rows_here * D; idx += kThreads) {
        const size_t row = static_cast<size_t>(seq) * p.Hq + hq0 + idx / D;
        p.out[row * D + idx % D] = __float2bfloat16_rn(0.f);
        if (p.lse != nullptr && idx % D == 0) p.lse[row] = -INFINITY;
      }
    }
    return;
  }
  // This warp's pairs of blocks: pair i is blocks 2 (warp + kWarps i) and the next one.
  const int n_pairs = (n_blk + 1) / 2;
  const int my_n = n_pairs > warp ? (n_pairs - warp + kWarps - 1) / kWarps : 0;
  const int32_t* table = p.block_table + static_cast<size_t>(seq) * p.max_blocks_per_seq + blk0;
  const uint8_t* head = p.cache + static_cast<size_t>(hkv) * Span::kBytes;
  const size_t blk_bytes = static_cast<size_t>(p.Hkv) * Span::kBytes;

  if (lane == 0) {
    for (int s = 0; s < kStages; ++s) mbar_init(&sm.full[warp][s], 2);
    fence_mbar_init();
  }
  __syncwarp();

  const uint64_t stream_policy = l2_policy_evict_first();
  int phys_lane = -1;         // physical block of this warp's block ((2 i) & ~31) + lane
  uint32_t present = 0;       // bits of the issued, not yet consumed blocks, next first
  // Starts the copies of this warp's i-th pair into stage i % kStages (whole
  // warp calls, i ascending; lanes 0 and 1 copy a block each).  A block past the
  // end, or whose table entry is out of range, arrives without a copy.
  auto issue = [&](int i, int ahead) {
    if ((i & 15) == 0) {
      const int mine = i + (lane >> 1);  // pair of this lane
      const int at = 2 * (warp + kWarps * mine) + (lane & 1);
      phys_lane = -1;
      if (mine < my_n && at < n_blk) {
        phys_lane = __ldg(table + at);
        if (phys_lane < 0 || phys_lane >= p.num_blocks) {
          atomicOr(p.status, 2u);
          phys_lane = -1;
        }
      }
    }
    const int ph = __shfl_sync(0xffffffffu, phys_lane, 2 * (i & 15) + (lane & 1));
    present |= (__ballot_sync(0xffffffffu, ph >= 0) & 3u) << (2 * ahead);
    if (lane < 2) {
      uint64_t* bar = &sm.full[warp][i % kStages];
      if (ph < 0) {
        mbar_arrive(bar);
      } else {
        fence_proxy_async_smem();
        mbar_arrive_expect_tx(bar, Span::kBytes);
        bulk_load_hint(sm.ring[warp][i % kStages] + lane * Span::kBytes, head + ph * blk_bytes, Span::kBytes, bar,
                       stream_policy);
      }
    }
  };
  int issued = 0;
  for (; issued < min(my_n, kStages); ++issued) issue(issued, issued);

  // Queries as B fragments: column g = query head hq0 + 8 nt + g; step ks,
  // indices 2t, 2t + 1 and 2t + 8, 2t + 9 = columns (D/4) t + 4 ks + 0..3, the
  // columns of the lane's own key codes.
  uint32_t qb[NT][kKSteps][2];
  float factor[NT][2];  // score factor of heads 2t, 2t + 1
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const bool real = 8 * nt + g < rows_here;
    const uint2* src = reinterpret_cast<const uint2*>(
        p.q + (static_cast<size_t>(seq) * p.Hq + hq0 + (real ? 8 * nt + g : 0)) * D + (D / 4) * t);
    float top = 0.f;
#pragma unroll
    for (int ks = 0; ks < kKSteps; ++ks) {
      const uint2 w = real ? __ldg(src + ks) : make_uint2(0u, 0u);
      qb[nt][ks][0] = w.x;
      qb[nt][ks][1] = w.y;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const uint32_t v = qb[nt][ks][e];
        top = fmaxf(top, fmaxf(fabsf(__uint_as_float(v << 16)), fabsf(__uint_as_float(v & 0xFFFF0000u))));
      }
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
  float rounded[NT][4];         // sums of the rounded weights: the product with a row of ones
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    m[nt][0] = m[nt][1] = kNoScore;
    l[nt][0] = l[nt][1] = 0.f;
    rounded[nt][0] = rounded[nt][1] = rounded[nt][2] = rounded[nt][3] = 0.f;
#pragma unroll
    for (int mt = 0; mt < kMTiles; ++mt) acc[mt][nt][0] = acc[mt][nt][1] = acc[mt][nt][2] = acc[mt][nt][3] = 0.f;
  }

  // mma token index r stands for token r ^ ((r >> 1) & 1): neighbouring pairs
  // swapped for odd t, so that the value loads of the four lanes of a group
  // fall on both halves of the banks.
  const int tok_s = g ^ ((g >> 1) & 1);    // this lane's score rows: tok_s, tok_s + 8
  const int tok_v0 = 2 * t + (t & 1);      // mma index 2t (and 2t + 8: + 8)
  const int tok_v1 = 2 * t + 1 - (t & 1);  // mma index 2t + 1 (and 2t + 9: + 8)
  const uint32_t key_off = Span::kKeyCodes + tok_s * Span::kCodeRow + t * (D / 8);
  const uint32_t key_scale_off = Span::kKeyScales + tok_s * Span::kScaleRow + t * (D / 64);
  const uint32_t val_off0 = Span::kValueCodes + tok_v0 * Span::kCodeRow + g * (D / 16);
  const uint32_t val_off1 = Span::kValueCodes + tok_v1 * Span::kCodeRow + g * (D / 16);
  const uint32_t val_scale_off0 = Span::kValueScales + tok_v0 * Span::kScaleRow + g * D / 128;
  const uint32_t val_scale_off1 = Span::kValueScales + tok_v1 * Span::kScaleRow + g * D / 128;
  const uint32_t ring0 = smem_u32(sm.ring[warp][0]);

  int st = 0;
  uint32_t parity = 0;
#pragma unroll 1
  for (int i = 0; i < my_n; ++i) {
    const bool waited = mbar_wait(&sm.full[warp][st], parity, p.wait_ns);
    if (!__all_sync(0xffffffffu, waited)) {
      if (lane == 0) {
        atomicOr(p.status, 1u);  // EXATTN_DEVICE_TIMEOUT_BIT
        for (int j = i + 1; j < issued; ++j)  // let copies in flight land
          mbar_wait(&sm.full[warp][j % kStages], (j / kStages) & 1, p.wait_ns);
      }
      __syncwarp();
      break;
    }
    const uint32_t base = ring0 + st * (2 * Span::kBytes);
    // Tokens of the two blocks that count: a missing block has none.
    const int left = ctx - (blk0 + 2 * (warp + kWarps * i)) * kBlk;
    int n_valid[2] = {min(kBlk, left), min(kBlk, left - kBlk)};
    if (!(present & 1u)) n_valid[0] = 0;
    if (!(present & 2u)) n_valid[1] = 0;
    present >>= 2;
    const bool partial = min(n_valid[0], n_valid[1]) < kBlk;

    // ---- S^T = K Q^T
    float c[2][NT][4];
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      const uint32_t span = base + b * Span::kBytes;
      uint32_t ka[kKeyWords], kb[kKeyWords];
      lds_words(span + key_off, ka);
      lds_words(span + key_off + 8 * Span::kCodeRow, kb);
      uint32_t sa, sb;  // scales of the lane's groups, fp16 pairs
      if constexpr (D == 128) {
        sa = e4m3x2_to_f16(lds_u16(span + key_scale_off));
        sb = e4m3x2_to_f16(lds_u16(span + key_scale_off + 8 * Span::kScaleRow));
      } else {
        sa = e4m3x2_to_f16(lds_u8(span + key_scale_off));
        sb = e4m3x2_to_f16(lds_u8(span + key_scale_off + 8 * Span::kScaleRow));
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) c[b][nt][0] = c[b][nt][1] = c[b][nt][2] = c[b][nt][3] = 0.f;
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
          mma_f16_16816(c[b][nt], h0[0], h1[0], h0[1], h1[1], qb[nt][2 * w][0], qb[nt][2 * w][1]);
          mma_f16_16816(c[b][nt], h0[2], h1[2], h0[3], h1[3], qb[nt][2 * w + 1][0], qb[nt][2 * w + 1][1]);
        }
      }
    }
    // ---- online softmax: c[b][nt][j] is token tok_s, head 2t + j, c[b][nt][2 + j]
    // token tok_s + 8.  Tokens that do not count are masked here and their
    // value scales zeroed below (the slots may hold anything).
    if (partial) {
#pragma unroll
      for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            if (tok_s >= n_valid[b]) c[b][nt][j] = -INFINITY;
            if (tok_s + 8 >= n_valid[b]) c[b][nt][2 + j] = -INFINITY;
          }
    }
    // Exponents relative to the reference m.  It follows the running maximum
    // only when a score passes it by more than 8 (weights up to 2^8 fit fp16
    // and the fp32 sums), which is rare after the first blocks: most pairs pay
    // one vote.
    float x[2][NT][4];
    float most = -INFINITY;
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          x[b][nt][y] = fmaf(c[b][nt][y], factor[nt][y & 1], -m[nt][y & 1]);
          most = fmaxf(most, x[b][nt][y]);
        }
    if (__any_sync(0xffffffffu, most > 8.f)) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          float top = fmaxf(fmaxf(c[0][nt][j], c[0][nt][2 + j]), fmaxf(c[1][nt][j], c[1][nt][2 + j]));
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
          const float mn = fmaxf(m[nt][j], top * factor[nt][j]);
          const float alpha = ex2_approx(m[nt][j] - mn);
          m[nt][j] = mn;
          l[nt][j] *= alpha;
          rounded[nt][j] *= alpha;
#pragma unroll
          for (int mt = 0; mt < kMTiles; ++mt) {
            acc[mt][nt][j] *= alpha;
            acc[mt][nt][2 + j] *= alpha;
          }
#pragma unroll
          for (int b = 0; b < 2; ++b) {
            x[b][nt][j] = fmaf(c[b][nt][j], factor[nt][j], -mn);
            x[b][nt][2 + j] = fmaf(c[b][nt][2 + j], factor[nt][j], -mn);
          }
        }
    }
    // ---- O^T += V^T P^T: row tile mt, row g = column (D/8) g + 2 mt, row
    // g + 8 the next one, all of one scale group
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      const uint32_t span = base + b * Span::kBytes;
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
        mma_f16_16816(rounded[nt], kOnes, kOnes, kOnes, kOnes, pb[nt][0], pb[nt][1]);
      }
      uint32_t va0[kValWords], va1[kValWords], vb0[kValWords], vb1[kValWords];
      lds_words(span + val_off0, va0);
      lds_words(span + val_off1, va1);
      lds_words(span + val_off0 + 8 * Span::kCodeRow, vb0);
      lds_words(span + val_off1 + 8 * Span::kCodeRow, vb1);
      uint32_t ea0 = lds_u8(span + val_scale_off0), ea1 = lds_u8(span + val_scale_off1);
      uint32_t eb0 = lds_u8(span + val_scale_off0 + 8 * Span::kScaleRow);
      uint32_t eb1 = lds_u8(span + val_scale_off1 + 8 * Span::kScaleRow);
      if (partial) {
        if (tok_v0 >= n_valid[b]) ea0 = 0;
        if (tok_v1 >= n_valid[b]) ea1 = 0;
        if (tok_v0 + 8 >= n_valid[b]) eb0 = 0;
        if (tok_v1 + 8 >= n_valid[b]) eb1 = 0;
      }
      const uint32_t ta = e4m3x2_to_f16(__byte_perm(ea0, ea1, 0x0040)), tb = e4m3x2_to_f16(__byte_perm(eb0, eb1, 0x0040));
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
    }
    __syncwarp();  // all lanes done with this stage before it is refilled
    if (issued < my_n) {
      issue(issued, issued - i - 1);
      ++issued;
    }
    if (++st == kStages) {
      st = 0;
      parity ^= 1u;
    }
  }

  // ---- the warp's sums over the eight lanes that share a head
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
#pragma unroll
      for (int y = 4; y < 32; y *= 2) l[nt][j] += __shfl_xor_sync(0xffffffffu, l[nt][j], y);
      if (g == 0) {
        sm.wm[warp][8 * nt + 2 * t + j] = m[nt][j];
        sm.wl[warp][8 * nt + 2 * t + j] = l[nt][j];
        sm.wlr[warp][8 * nt + 2 * t + j] = rounded[nt][j];
      }
    }
  __syncthreads();  // every warp finished streaming: the rings are free
  float* wacc = reinterpret_cast<float*>(&sm.ring[0][0][0]);  // [warp][head][kAccStride]
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int j = 0; j < 2; ++j)
      if (8 * nt + 2 * t + j < rows_here)
#pragma unroll
        for (int mt = 0; mt < kMTiles; mt += 2)
          *reinterpret_cast<float4*>(&wacc[(warp * kRows + 8 * nt + 2 * t + j) * kAccStride + (D / 8) * g + 2 * mt]) =
              make_float4(acc[mt][nt][j], acc[mt][nt][2 + j], acc[mt + 1][nt][j], acc[mt + 1][nt][2 + j]);
  __syncthreads();

  // ---- merge the warps; thread -> (head, four columns) of real heads
  for (int idx = threadIdx.x; idx < rows_here * (D / 4); idx += kThreads) {
    const int r = idx / (D / 4), col = idx % (D / 4) * 4;
    float M = kNoScore;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) M = fmaxf(M, sm.wm[w][r]);
    float L = 0.f, Lr = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float wt = ex2_approx(sm.wm[w][r] - M);
      L += wt * sm.wl[w][r];
      Lr += wt * sm.wlr[w][r];
      const float4 a = *reinterpret_cast<const float4*>(&wacc[(w * kRows + r) * kAccStride + col]);
      o.x += wt * a.x;
      o.y += wt * a.y;
      o.z += wt * a.z;
      o.w += wt * a.w;
    }
    // a split all of whose scores are -inf, or whose blocks are all missing, sees nothing
    const float scale = L == 0.f ? 0.f : p.v_scale / Lr;
    const float ls = L == 0.f ? -INFINITY : (M + __log2f(L)) * kLn2;
    const size_t row = static_cast<size_t>(seq) * p.Hq + hq0 + r;
    if (p.splits == 1) {
      *reinterpret_cast<uint2*>(p.out + row * D + col) =
          make_uint2(pack_bf16x2(o.x * scale, o.y * scale), pack_bf16x2(o.z * scale, o.w * scale));
      if (p.lse != nullptr && col == 0) p.lse[row] = ls;
    } else {
      *reinterpret_cast<float4*>(p.ws_o + (row * p.splits + split) * D + col) =
          make_float4(o.x * scale, o.y * scale, o.z * scale, o.w * scale);
      if (col == 0) p.ws_lse[row * p.splits + split] = ls;
    }
  }
}

struct Fp4CombineParams {
  const float* ws_o;
  const float* ws_lse;
  const int32_t* ctx_lens;
  __nv_bfloat16* out;
  float* lse;
  unsigned int* status;
  int Hq, max_blocks_per_seq, splits;
};

// One CTA per (query head, sequence): L = log sum_s exp(lse_s),
// o = sum_s exp(lse_s - L) O_s.  The weights are formed once, a split per
// thread; then D/4 threads take four columns each of every kTeams-th split.
template <int D>
__global__ void __launch_bounds__(kThreads) decode_fp4_combine_kernel(const Fp4CombineParams p) {
  constexpr int kTeams = kThreads / (D / 4);
  __shared__ float weight[kFp4MaxSplits];
  __shared__ float top[kWarps], sum[kWarps];
  __shared__ float4 part[kTeams][D / 4];
  const int hq = blockIdx.x, seq = blockIdx.y;
  const int ctx = clamp_ctx(__ldg(p.ctx_lens + seq), p.max_blocks_per_seq * kBlk, p.status);
  const int seq_blk = (ctx + kBlk - 1) / kBlk;
  const int per = blocks_per_split(seq_blk, p.splits);
  const int used = (seq_blk + per - 1) / per;
  const size_t row = static_cast<size_t>(seq) * p.Hq + hq;
  const size_t base = row * p.splits;
  cudaGridDependencySynchronize();  // launched while the split kernel drains
  float M = -INFINITY;
  for (int s = threadIdx.x; s < used; s += kThreads) {
    const float ls = p.ws_lse[base + s];
    weight[s] = ls;
    M = max_nan(M, ls);
  }
#pragma unroll
  for (int x = 1; x < 32; x *= 2) M = max_nan(M, __shfl_xor_sync(0xffffffffu, M, x));
  if ((threadIdx.x & 31) == 0) top[threadIdx.x >> 5] = M;
  __syncthreads();
  M = top[0];
#pragma unroll
  for (int w = 1; w < kWarps; ++w) M = max_nan(M, top[w]);
  const float ref = M == -INFINITY ? 0.f : M;  // all weights 0 where no split sees anything
  float W = 0.f;
  for (int s = threadIdx.x; s < used; s += kThreads) {
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
  for (int w = 0; w < kWarps; ++w) W += sum[w];
  const int col = threadIdx.x % (D / 4), team = threadIdx.x / (D / 4);
  const float4* src = reinterpret_cast<const float4*>(p.ws_o + base * D) + col;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int s = team; s < used; s += kTeams) {
    const float w = weight[s];
    const float4 a = src[static_cast<size_t>(s) * (D / 4)];
    o.x = fmaf(w, a.x, o.x);
    o.y = fmaf(w, a.y, o.y);
    o.z = fmaf(w, a.z, o.z);
    o.w = fmaf(w, a.w, o.w);
  }
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
    reinterpret_cast<uint2*>(p.out + row * D)[col] =
        make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
    if (p.lse != nullptr && col == 0) p.lse[row] = W == 0.f ? -INFINITY : M + __logf(W);
  }
}

template <int D, int NT>
cudaError_t launch_split(const DecodeFp4Args& a, const Fp4SplitParams& sp, cudaStream_t stream) {
  const size_t smem = sizeof(Fp4Smem<D>) + 128;
  static std::atomic<int> smem_set[64] = {};
  cudaError_t e = smem_limit_once(reinterpret_cast<const void*>(decode_fp4_split_kernel<D, NT>),
                                  static_cast<int>(smem), smem_set);
  if (e != cudaSuccess) return e;
  dim3 grid(a.splits, a.Hkv * sp.n_chunks, a.num_seqs);
  decode_fp4_split_kernel<D, NT><<<grid, kThreads, smem, stream>>>(sp);
  return cudaGetLastError();
}

template <int D>
cudaError_t launch_d(const DecodeFp4Args& a, const DeviceGuard& g, cudaStream_t stream) {
  Fp4SplitParams sp;
  sp.q = static_cast<const __nv_bfloat16*>(a.q);
  sp.cache = static_cast<const uint8_t*>(a.kv_cache);
  sp.block_table = a.block_table;
  sp.ctx_lens = a.ctx_lens;
  sp.ws_o = a.ws_o;
  sp.ws_lse = a.ws_lse;
  sp.out = static_cast<__nv_bfloat16*>(a.out);
  sp.lse = a.lse;
  sp.status = g.status;
  sp.wait_ns = g.wait_ns;
  sp.Hq = a.Hq;
  sp.Hkv = a.Hkv;
  sp.group = a.Hq / a.Hkv;
  const int rows = fp4_decode_rows(sp.group);
  sp.n_chunks = (sp.group + rows - 1) / rows;
  sp.num_blocks = a.num_blocks;
  sp.max_blocks_per_seq = a.max_blocks_per_seq;
  sp.splits = a.splits;
  sp.scale_log2 = static_cast<float>(static_cast<double>(a.scale) * a.k_scale * 1.4426950408889634);
  sp.v_scale = a.v_scale;
  cudaError_t e = rows == 8 ? launch_split<D, 1>(a, sp, stream) : launch_split<D, 2>(a, sp, stream);
  if (e != cudaSuccess || a.splits == 1) return e;

  Fp4CombineParams cp;
  cp.ws_o = a.ws_o;
  cp.ws_lse = a.ws_lse;
  cp.ctx_lens = a.ctx_lens;
  cp.out = sp.out;
  cp.lse = a.lse;
  cp.status = g.status;
  cp.Hq = a.Hq;
  cp.max_blocks_per_seq = a.max_blocks_per_seq;
  cp.splits = a.splits;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(a.Hq, a.num_seqs);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, decode_fp4_combine_kernel<D>, cp);
}

}  // namespace

cudaError_t launch_decode_fp4(const DecodeFp4Args& a, const DeviceGuard& g, cudaStream_t stream) {
  return a.d == 64 ? launch_d<64>(a, g, stream) : launch_d<128>(a, g, stream);
}

}  // namespace exattn
