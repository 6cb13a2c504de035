// The 8-bit paged cache's append and read (layout in fp8.cuh) for sm_103a.
//
// rope_cache_fp8_kernel: a block's scale belongs to all its tokens, so the new tokens of one
//   sequence that fall into one block, a run, are handled together: a warp takes one head of
//   a run, 16 tokens at most, and finds the largest magnitude, the scale and the codes without
//   meeting another warp.  Where each sequence has one token (the step of a serving batch)
//   neighbouring sequences' tokens share a warp, each with a block of its own.  A CTA forms
//   its run's cosines and sines once for all heads; rows come through a ring in shared memory,
//   each lane's own (cp.async), one head ahead, through all runs of the CTA.  Keys are turned
//   twice, for their magnitude and for their codes, which costs less than registers that would
//   keep them.
//   Bound by HBM: 64 x 256 tokens (32 + 2 x 8 heads of 128; 202 MB read, 168 written): 60.1 us =
//   6.2 TB/s, 91% of a copy.  Long stretches of a token's row at once are worth more than
//   balance: with the heads of each run divided among CTAs 68 us and more, with those of the
//   last round of runs 69.  Small calls are one round of dependent loads (64 tokens of 64
//   sequences 2.7 us, one token 2.5; five chunks of 1 to 333 tokens, 14 + 2 x 2 heads of 64, whose
//   runs are counted first, 3.9).  Where a block's scale grows, its other codes are read and
//   written too, by the eight lanes of a token (four at d = 64) or by the warp of a run: 64 tokens
//   that all let both scales of their blocks grow 9.3 us, 3.1 without (512 of them 31 and 6.6; four
//   new tokens of each of 64 sequences 5.8 and 4.8).
// cache_read_fp8_kernel: below.
#include <cuda_bf16.h>

#include "fp8.cuh"
#include "launch.h"
#include "ptx.cuh"
#include "rope_rows.cuh"

namespace exattn {
namespace {

// CTAs of eight warps that share an SM: 72 registers, 73 KB each at d = 128.  (200 sequences of 16
// more tokens, 4000 + 63 tokens: 19.1 and 16.9 us; with 76 KB, so that only two of three
// fitted, 22.3 and 19.2; 2048 + 63 tokens 11.5 with both, 16.6 with five CTAs of four warps.)
constexpr int kAppendCtas = 3;
constexpr long long kAppendLarge = 16 << 20;  // bytes of rows of a large call
constexpr long long kAppendWide = 192 << 10;  // ... and of a run of 16 tokens with many heads
constexpr int kAppendStages = 2;  // heads of a warp on their way, and the one at hand
constexpr int kBlk = kDecodeBlockSize;
constexpr int kReadLanes = 4;

// Rows of the call that are handled together: new tokens of one sequence that fall into
// one block, or (kSingle) one token each of neighbouring sequences.
struct Run {
  int token, count;  // the call's tokens token .. token + count - 1
  int seq, place;    // of the first
  long long slot;    // of the first
};

// The new tokens of a sequence: tokens begin .. end - 1 of the call, the last ones of ctx.
struct Added {
  int begin, end, ctx;
  __device__ __forceinline__ int phase() const {  // place of the first
    return static_cast<int>((static_cast<unsigned int>(ctx) - (end - begin)) & (kBlk - 1));
  }
  __device__ __forceinline__ int runs() const { return end > begin ? (phase() + end - begin + kBlk - 1) / kBlk : 0; }
  __device__ __forceinline__ Run run(int seq, int r) const {
    const int from = max(0, r * kBlk - phase());
    Run x;
    x.seq = seq;
    x.token = begin + from;
    x.place = r == 0 ? phase() : 0;
    x.count = max(0, min(kBlk - x.place, end - x.token));  // (0 only where the numbers changed meanwhile)
    x.slot = static_cast<long long>(ctx) - (end - begin) + from;
    return x;
  }
};

template <int D, int kWarps>
struct AppendSmem {
  static constexpr int kThreads = 32 * kWarps;
  static constexpr int kPerTok = D / 16;              // lanes per token: 8 pairs each
  static constexpr int kSteps = kBlk * kPerTok / 32;  // rounds of a warp over 16 tokens
  uint4 ring[kWarps][kAppendStages][kSteps][2][32];  // a lane's two vectors of each round
  // Of a run: cosines and sines by token, then two pairs (float4) of each lane next to each
  // other, so that the lanes of a token read neighbouring vectors; and where each token lies.
  float4 angles[kBlk][4][kPerTok];
  int block[kBlk], place[kBlk];
  int upto[kThreads];  // runs of the sequences of this and earlier threads
  int warp_sum[kWarps];
};
static_assert(kAppendCtas * (sizeof(AppendSmem<128, 8>) + 1024) <= 228 * 1024, "CTAs of an SM by shared memory");

__device__ __forceinline__ bool is_finite(float x) { return fabsf(x) <= 3.4028234663852886e38f; }

// Largest of m and the magnitudes of a and b, NaN where one is.
__device__ __forceinline__ float max3_nan_abs(float m, float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(m), "f"(fabsf(a)), "f"(fabsf(b)));
  return r;
}

// Brings a block's codes from one scale to a larger one (biased exponents; 0: there was
// none, and all are 0), but for places first .. first + count - 1.  By `lanes` lanes.
template <int D>
__device__ __forceinline__ void rescale(uint8_t* codes, int from, int to, int first, int count, int lane, int lanes) {
  const int shift = from > 0 ? 127 + from - to : 0;
  const float factor = shift > 0 ? __uint_as_float(static_cast<uint32_t>(shift) << 23) : 0.f;
  auto moved = [&](uint32_t w) {
    uint32_t h0, h1;
    e4m3x4_to_f16(w, h0, h1);
    return f32x4_to_e4m3(f16_lo(h0) * factor, f16_hi(h0) * factor, f16_lo(h1) * factor, f16_hi(h1) * factor);
  };
#pragma unroll 1
  for (int v = lane; v < D; v += lanes) {
    const int place = v / (D / 16);
    if (place >= first && place < first + count) continue;
    uint4* at = reinterpret_cast<uint4*>(codes) + v;
    const uint4 old = *at;
    *at = make_uint4(moved(old.x), moved(old.y), moved(old.z), moved(old.w));
  }
}

// kSingle: each sequence has one token; runs are `tile` of them.
template <int D, bool kSingle, int kWarps>
__global__ void __launch_bounds__(32 * kWarps, kWarps == 8 ? kAppendCtas : 1)
    rope_cache_fp8_kernel(const RopeFp8Args a, const __grid_constant__ RopeAxesTable table, const int tile,
                          const int splits) {
  using Span = Fp8Span<D>;
  using Smem = AppendSmem<D, kWarps>;
  constexpr int kThreads = Smem::kThreads;
  constexpr int kHalf = D / 2, kApart = kHalf / 8;  // 16-byte vectors between the halves of a row
  constexpr int kPerTok = Smem::kPerTok, kSteps = Smem::kSteps;
  constexpr int kToks = 32 / kPerTok;               // tokens of a warp at once
  constexpr int kAtOnce = kThreads / kHalf;   // tokens whose angles the threads form at once
  constexpr int kAngles = (kBlk + kAtOnce - 1) / kAtOnce;
  extern __shared__ __align__(16) uint8_t append_smem[];
  Smem& sm = *reinterpret_cast<Smem*>(append_smem);

  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int j = lane % kPerTok, tok0 = lane / kPerTok;
  // this thread's pair of the angles
  const int pair = threadIdx.x % kHalf, angle_tok = threadIdx.x / kHalf;
  unsigned long long freq;
  uint32_t axis;
  asm volatile("ld.b64 %0, [%1];" : "=l"(freq) : "l"(table.u + pair));
  asm volatile("ld.u8 %0, [%1];" : "=r"(axis) : "l"(table.axis + pair));
  cudaGridDependencySynchronize();

  // ---- the runs: counted from token_starts, or `tile` sequences each
  const int per = (a.num_seqs + kThreads - 1) / kThreads;
  auto added_of = [&](int s) {
    return Added{__ldg(a.token_starts + s), __ldg(a.token_starts + s + 1), __ldg(a.ctx_lens + s)};
  };
  int total = (a.num_seqs + tile - 1) / tile;
  if constexpr (!kSingle) {
    int mine = 0;
    bool bad = false;
    for (int i = 0; i < per; ++i) {
      const int s = threadIdx.x * per + i;
      if (s >= a.num_seqs) break;
      const Added x = added_of(s);
      bad |= x.begin < 0 || x.end < x.begin || x.end > a.num_tokens;
      mine += bad ? 0 : x.runs();
    }
    int sum = mine;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
      const int v = __shfl_up_sync(0xffffffffu, sum, d);
      if (lane >= d) sum += v;
    }
    if (lane == 31) sm.warp_sum[warp] = sum;
    // starts that decrease or leave the call could name a token twice: nothing is done then
    if (__syncthreads_or(bad)) {
      if (blockIdx.x == 0 && threadIdx.x == 0) atomicOr(a.status, 2u);  // EXATTN_DEVICE_BOUNDS_BIT
      return;
    }
    total = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) sum += sm.warp_sum[w];
      total += sm.warp_sum[w];
    }
    sm.upto[threadIdx.x] = sum;
    __syncthreads();
  }
  auto find_run = [&](int r) {
    if constexpr (kSingle) return Run{r * tile, min(tile, a.num_seqs - r * tile), r * tile, 0, 0};
    // the first thread with upto > r, by the warp: its warp's place, then its own
    const int eighth = min(31, __popc(__ballot_sync(0xffffffffu, sm.upto[kWarps * lane + kWarps - 1] <= r)));
    const bool past = lane < kWarps && sm.upto[kWarps * eighth + min(lane, kWarps - 1)] <= r;
    const int lo = kWarps * eighth + min(kWarps - 1, __popc(__ballot_sync(0xffffffffu, past)));
    r -= lo > 0 ? sm.upto[lo - 1] : 0;
    int s = lo * per;
    // (the numbers are read a second time: if another stream changes them meanwhile the result is
    // undefined, but every row that comes out is one of the call)
    auto within = [&] {
      const Added x = added_of(s);
      return Added{max(0, x.begin), min(a.num_tokens, x.end), x.ctx};
    };
    Added x = within();
    while (r >= x.runs() && s + 1 < a.num_seqs) {
      r -= x.runs();
      ++s;
      x = within();
    }
    return x.run(s, r);
  };

  // ---- units of work: a run and a part of its items, which are key heads, value heads and
  // query heads in order.  (Runs hold a token each, and have several parts only where they
  // are fewer than the CTAs: the numbers stay far below 2^31.)
  const int first_value = a.Hkv, first_query = 2 * a.Hkv, items = first_query + a.Hq;
  const int units = total * splits;
  int unit = blockIdx.x;
  if (unit >= units) return;

  // Rows on their way into the ring: this warp's items in order, through all units.
  int to_unit = unit, to_item = unit % splits + splits * warp;
  Run to = find_run(unit / splits);
  auto fetch = [&](int stage) {
    while (to_item >= items) {
      to_unit += gridDim.x;
      if (to_unit >= units) break;
      to = find_run(to_unit / splits);
      to_item = to_unit % splits + splits * warp;
    }
    if (to_unit < units) {
      const HeadView& view = to_item < first_value ? a.k : to_item < first_query ? a.v : a.q;
      const int head = to_item - (to_item < first_value ? 0 : to_item < first_query ? first_value : first_query);
      const uint4* row = row_of(view, 0, head, to.token + tok0) + j;
      const uint32_t slot = smem_u32(&sm.ring[warp][stage][0][0][lane]);
#pragma unroll
      for (int s = 0; s < kSteps; ++s) {
        if (s * kToks + tok0 < to.count) {
          cp_async16(slot + s * 1024, row, true);
          cp_async16(slot + s * 1024 + 512, row + kApart, true);
        }
        row += kToks * view.token;
      }
      to_item += splits * kWarps;
    }
    cp_async_commit();
  };

  // What a run needs beside its rows: where thread n's token n lies, the positions of the
  // tokens whose angles a thread forms.  Asked for while the run before is worked on.
  int ahead_block = -1, ahead_place = 0;
  int ahead_pos[kAngles];
  auto ask = [&](const Run& run) {
    if (threadIdx.x < run.count) {
      int seq = run.seq;
      long long slot = run.slot;
      ahead_place = run.place + threadIdx.x;
      if constexpr (kSingle) {
        seq += threadIdx.x;
        slot = static_cast<long long>(__ldg(a.ctx_lens + seq)) - 1;
        ahead_place = static_cast<int>(slot & (kBlk - 1));
      }
      ahead_block = -1;
      if (slot >= 0 && slot < static_cast<long long>(a.max_blocks_per_seq) * kBlk) {
        ahead_block = __ldg(a.block_table + static_cast<long long>(seq) * a.max_blocks_per_seq + slot / kBlk);
        if (ahead_block >= a.num_blocks) ahead_block = -1;
      }
      if (ahead_block < 0) atomicOr(a.status, 2u);  // EXATTN_DEVICE_BOUNDS_BIT
    }
#pragma unroll
    for (int i = 0; i < kAngles; ++i) {
      const int tok = angle_tok + i * kAtOnce;
      ahead_pos[i] = tok < run.count ? __ldg(a.positions + axis * a.pos_axis + run.token + tok) : 0;
    }
  };
  auto put = [&](const Run& run) {
    if (threadIdx.x < run.count) {
      sm.block[threadIdx.x] = ahead_block;
      sm.place[threadIdx.x] = ahead_place;
    }
#pragma unroll
    for (int i = 0; i < kAngles; ++i) {
      const int tok = angle_tok + i * kAtOnce;
      if (tok < run.count)
        reinterpret_cast<float2*>(&sm.angles[tok][pair % 8 / 2][pair / 8])[pair & 1] =
            turn_cos_sin(static_cast<unsigned long long>(static_cast<long long>(ahead_pos[i])) * freq);
    }
  };

#pragma unroll
  for (int s = 0; s < kAppendStages - 1; ++s) fetch(s);
  Run run = find_run(unit / splits);
  ask(run);
  int stage = 0, behind = kAppendStages - 1;  // stages of the item at hand, and of the one before it
  for (;;) {
    put(run);
    __syncthreads();  // this run's angles are there
    const bool more = unit + static_cast<int>(gridDim.x) < units;
    const Run next = more ? find_run((unit + gridDim.x) / splits) : run;
    if (more) ask(next);
    for (int item = unit % splits + splits * warp; item < items; item += splits * kWarps) {
      const bool value = item >= first_value, query = item >= first_query;
      const int head = item - (query ? first_query : value ? first_value : 0);
      cp_async_wait<kAppendStages - 2>();
      const uint4* const rows = &sm.ring[warp][stage][0][0][lane];  // vector x of round s at rows[64 s + 32 x]
      fetch(behind);
      behind = stage;
      stage = stage + 1 == kAppendStages ? 0 : stage + 1;
      // A token's 8 low and 8 high columns, turned; `turns` is false for values.
      auto columns = [&](int s, bool turns, float (&ya)[8], float (&yb)[8]) {
        const uint4 lo = rows[64 * s], hi = rows[64 * s + 32];
        if (!turns) {
          unpack_bf16x8(lo, ya);
          unpack_bf16x8(hi, yb);
          return;
        }
        Turn8 t;
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const float4 v = sm.angles[s * kToks + tok0][x][j];
          t.c[2 * x] = v.x;
          t.s[2 * x] = v.y;
          t.c[2 * x + 1] = v.z;
          t.s[2 * x + 1] = v.w;
        }
        t.turn(lo, hi, ya, yb);
      };
      if (query) {
        uint4* out = const_cast<uint4*>(row_of(a.q_out, 0, head, run.token + tok0)) + j;
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
          if (s * kToks + tok0 < run.count) {
            float ya[8], yb[8];
            columns(s, true, ya, yb);
            out[0] = pack_bf16x8(ya);
            out[kApart] = pack_bf16x8(yb);
          }
          out += kToks * a.q_out.token;
        }
        continue;
      }
      // ---- a head's keys or values: their largest magnitude, the scale, the codes
      auto largest = [&](int s, bool all) {  // of a token's columns of this lane; of the finite ones, or NaN where one is
        float ya[8], yb[8];
        columns(s, !value, ya, yb);
        float m = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          if (all) {
            m = max3_nan_abs(m, ya[e], yb[e]);
          } else {
            m = fmaxf(m, is_finite(ya[e]) ? fabsf(ya[e]) : 0.f);
            m = fmaxf(m, is_finite(yb[e]) ? fabsf(yb[e]) : 0.f);
          }
        }
        return m;
      };
      auto store = [&](int s, float most, bool plain, int block, int place, int first, int count, uint32_t before) {
        uint8_t* const span = static_cast<uint8_t*>(a.kv_cache) +
                              (static_cast<size_t>(block) * a.Hkv + head) * Span::kBytes;
        uint8_t* const codes = span + (value ? Span::kValueCodes : Span::kKeyCodes);
        const int e_before = min(static_cast<int>(before >> 23), 127 + kFp8HighExponent);
        const int e = max(fp8_scale_exponent(most), e_before);
        if (s * kToks + tok0 < run.count) {
          const float down = __uint_as_float(static_cast<uint32_t>(254 - e) << 23);
          float ya[8], yb[8];
          columns(s, !value, ya, yb);
          if (!plain) {
#pragma unroll
            for (int x = 0; x < 8; ++x) {
              if (!is_finite(ya[x])) ya[x] = __int_as_float(0x7FC00000);
              if (!is_finite(yb[x])) yb[x] = __int_as_float(0x7FC00000);
            }
          }
          uint32_t w[4];
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            w[x] = f32x4_to_e4m3(ya[4 * x] * down, ya[4 * x + 1] * down, ya[4 * x + 2] * down, ya[4 * x + 3] * down);
            w[2 + x] = f32x4_to_e4m3(yb[4 * x] * down, yb[4 * x + 1] * down, yb[4 * x + 2] * down, yb[4 * x + 3] * down);
          }
          uint8_t* row = codes + place * Span::kRow + (j & 1) * 8;
          *reinterpret_cast<uint2*>(row + ((j / 2) ^ fp8_turn<D>(place)) * 16) = make_uint2(w[0], w[1]);
          *reinterpret_cast<uint2*>(row + ((j / 2 + D / 32) ^ fp8_turn<D>(place)) * 16) = make_uint2(w[2], w[3]);
        }
        if ((kSingle || s == 0) && e > e_before) {  // the scale, once for a block
          if (kSingle ? j == 0 : lane == 0)
            reinterpret_cast<uint32_t*>(span + Span::kScales)[value ? 1 : 0] = static_cast<uint32_t>(e) << 23;
          if (first > 0) rescale<D>(codes, e_before, e, first, count, kSingle ? j : lane, kSingle ? kPerTok : 32);
        }
      };
      auto scale_of = [&](int block) {
        return reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(a.kv_cache) +
                                                 (static_cast<size_t>(block) * a.Hkv + head) * Span::kBytes +
                                                 Span::kScales)[value ? 1 : 0];
      };
      if constexpr (kSingle) {
#pragma unroll 1
        for (int s = 0; s * kToks < run.count; ++s) {
          const int tok = s * kToks + tok0;
          const bool real = tok < run.count;
          const int block = real ? sm.block[tok] : -1, place = real ? sm.place[tok] : 0;
          const uint32_t before = block >= 0 && place > 0 ? scale_of(block) : 0u;
          float m = real ? largest(s, true) : 0.f;
          const bool plain = is_finite(m);
          if (!plain) m = largest(s, false);
          __syncwarp();
#pragma unroll
          for (int d = 1; d < kPerTok; d *= 2) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
          if (block >= 0) store(s, m, plain, block, place, place, 1, before);
          __syncwarp();
        }
      } else {
        const int block = sm.block[0];
        const uint32_t before = block >= 0 && run.place > 0 ? scale_of(block) : 0u;
        float m = 0.f;
#pragma unroll
        for (int s = 0; s < kSteps; ++s)
          if (s * kToks + tok0 < run.count) m = max_nan(m, largest(s, true));
        const bool plain = __all_sync(0xffffffffu, is_finite(m));
        if (!plain) {
          m = 0.f;
#pragma unroll 1
          for (int s = 0; s < kSteps; ++s)
            if (s * kToks + tok0 < run.count) m = fmaxf(m, largest(s, false));
          __syncwarp();
        }
        m = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(m)));
        if (block >= 0) {
#pragma unroll
          for (int s = 0; s < kSteps; ++s)
            if (s * kToks < run.count)
              store(s, m, plain, block, run.place + s * kToks + tok0, run.place, run.count, before);
        }
        __syncwarp();
      }
    }
    if (!more) break;
    __syncthreads();  // this run's angles are no longer read
    unit += gridDim.x;
    run = next;
  }
  cp_async_wait<0>();
}

// Read: thread j of a token takes chunk j of the keys and values of every head
// it visits: rows 0 .. Hkv - 1 are keys, the next Hkv values.  A code times its scale is a bf16
// number, so nothing is rounded.  Bound by its bytes, two thirds of them writes: 32,768 tokens of
// 8 heads of 128 (202 MB) 33.2 us = 6.1 TB/s; 34.0 with 2 or 8 lanes, 37.4 with 1, 35.6 with one
// row at a time, 33.1 with four and 64 x 256 tokens then 16.0 instead of 15.0.
template <int D>
__global__ void __launch_bounds__(kTileThreads, 8) cache_read_fp8_kernel(const ReadFp8Args a, const Tile tile) {
  using Span = Fp8Span<D>;
  constexpr int kPerTok = D / 16;
  constexpr int kUnroll = 2;
  const int j = threadIdx.x % kPerTok, rest = threadIdx.x / kPerTok;
  const int tok = rest % tile.toks, lane = rest / tile.toks;
  const long long n = static_cast<long long>(blockIdx.x) * tile.toks + tok;
  cudaGridDependencySynchronize();
  if (lane >= tile.lanes || n >= a.at.num_tokens) return;
  int off;
  const long long blk = find_block(a.at, n, &off);
  if (blk < 0 && j == 0 && lane == 0) atomicOr(a.at.status, 2u);  // EXATTN_DEVICE_BOUNDS_BIT
  const uint8_t* spans = static_cast<const uint8_t*>(a.kv_cache) + (blk < 0 ? 0 : blk) * a.Hkv * Span::kBytes;
  const int code_off = off * Span::kRow + (j ^ fp8_turn<D>(off)) * 16;
  uint4* k_out = const_cast<uint4*>(row_of(a.k_out, 0, 0, n)) + 2 * j;
  uint4* v_out = const_cast<uint4*>(row_of(a.v_out, 0, 0, n)) + 2 * j;
  for (int r0 = lane; r0 < 2 * a.Hkv; r0 += kUnroll * tile.lanes) {
    uint4 codes[kUnroll];
    float scale[kUnroll];
#pragma unroll
    for (int x = 0; x < kUnroll; ++x) {
      const int r = r0 + x * tile.lanes;
      codes[x] = make_uint4(0u, 0u, 0u, 0u);
      scale[x] = 0.f;
      if (r < 2 * a.Hkv && blk >= 0) {
        const uint8_t* span = spans + static_cast<size_t>(r >= a.Hkv ? r - a.Hkv : r) * Span::kBytes;
        codes[x] = *reinterpret_cast<const uint4*>(span + (r >= a.Hkv ? Span::kValueCodes : Span::kKeyCodes) + code_off);
        scale[x] = reinterpret_cast<const float*>(span + Span::kScales)[r >= a.Hkv ? 1 : 0];
      }
    }
#pragma unroll
    for (int x = 0; x < kUnroll; ++x) {
      const int r = r0 + x * tile.lanes;
      if (r >= 2 * a.Hkv) break;
      const uint32_t c[4] = {codes[x].x, codes[x].y, codes[x].z, codes[x].w};
      uint32_t w[8];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        uint32_t h0, h1;
        e4m3x4_to_f16(c[e], h0, h1);
        w[2 * e] = pack_bf16x2(f16_lo(h0) * scale[x], f16_hi(h0) * scale[x]);
        w[2 * e + 1] = pack_bf16x2(f16_lo(h1) * scale[x], f16_hi(h1) * scale[x]);
      }
      uint4* dst = r >= a.Hkv ? v_out + (r - a.Hkv) * a.v_out.head : k_out + r * a.k_out.head;
      if ((reinterpret_cast<uintptr_t>(dst) & 31) == 0) {  // (rows are on 16-byte boundaries)
        st_global_v8(dst, w);
      } else {
        dst[0] = make_uint4(w[0], w[1], w[2], w[3]);
        dst[1] = make_uint4(w[4], w[5], w[6], w[7]);
      }
    }
  }
}

template <int D, bool kSingle, int kWarps>
cudaError_t launch_append(const RopeFp8Args& a, const RopeAxesTable& table, int sms, long long runs, int tile,
                          cudaStream_t stream) {
  using Smem = AppendSmem<D, kWarps>;
  static std::atomic<int> smem_set[64] = {};
  const cudaError_t e = smem_limit_once(reinterpret_cast<const void*>(rope_cache_fp8_kernel<D, kSingle, kWarps>),
                                        static_cast<int>(sizeof(Smem)), smem_set);
  if (e != cudaSuccess) return e;
  // Few runs are divided among as many CTAs as fit under the end of a launch before (half of
  // the places on the SMs), down to an item for each warp.
  const int places = sms * (kWarps == 8 ? kAppendCtas : 1), few = kWarps == 8 ? places / 2 : places;
  const int most = (a.Hq + 2 * a.Hkv + kWarps - 1) / kWarps;
  const int splits = runs * most <= few ? most : runs < few ? static_cast<int>(few / runs) : 1;
  const long long units = runs * splits;
  return launch_overlapped(rope_cache_fp8_kernel<D, kSingle, kWarps>, static_cast<unsigned int>(units < places ? units : places),
                           Smem::kThreads, sizeof(Smem), stream, 1, a, table, tile, splits);
}

template <int D>
cudaError_t launch_append_d(const RopeFp8Args& a, const RopeAxesTable& table, int sms, cudaStream_t stream) {
  const long long items = a.Hq + 2 * a.Hkv;
  if (a.token_starts == nullptr) {
    const long long most = (items + 7) / 8;
    int tile = 32 / AppendSmem<D, 8>::kPerTok;  // tokens that a warp's lanes take at once
    while (tile < kBlk && (a.num_tokens + tile - 1) / tile * most > sms * kAppendCtas / 2) tile *= 2;
    return launch_append<D, true, 8>(a, table, sms, (a.num_tokens + tile - 1) / tile, tile, stream);
  }
  // About as many runs as the call can have.  Large calls whose runs fill one CTA an SM, or
  // many where the runs are wide, take CTAs of 16 warps, each run's tokens in longer stretches:
  // 64 x 256 tokens (32 + 2 x 8 heads of 128) 60.1 us, 65.6 with three of eight; 2048 tokens 9.7
  // and 11.0; but 2048 tokens and 63 single ones 13.7 and 11.5, and small calls lose the overlap
  // (64 tokens 3.0 and 2.7).  Beside the borders, 16 warps and eight: 80 runs of 192 KB 8.4 both, 100
  // 9.4 and 9.1, 128 9.2 and 10.0, 190 16.9 and 15.5, 456 28.7 and 27.9, 500 34.7 and 32.9, 608
  // 37.0 and 37.9; 1024 of 160 KB (64 + 2 x 8 heads of 64) 62.4 and 57.3, of 72 KB 36.4 and 26.4,
  // of 320 KB 107 both.
  const long long runs = a.num_tokens / kBlk + (a.num_seqs < a.num_tokens ? a.num_seqs : a.num_tokens);
  if (a.num_tokens * items * D * 2 > kAppendLarge &&
      (runs <= sms || (runs > sms * kAppendCtas && kBlk * items * D * 2 >= kAppendWide)))
    return launch_append<D, false, 16>(a, table, sms, runs, 1, stream);
  return launch_append<D, false, 8>(a, table, sms, runs, 1, stream);
}

}  // namespace

cudaError_t launch_rope_cache_write_fp8(const RopeFp8Args& a, const RopeAxesTable& table, cudaStream_t stream) {
  const int sms = device_sm_count();
  if (sms <= 0) return cudaErrorInvalidDevice;
  return a.d == 64 ? launch_append_d<64>(a, table, sms, stream) : launch_append_d<128>(a, table, sms, stream);
}

cudaError_t launch_cache_read_fp8(const ReadFp8Args& a, cudaStream_t stream) {
  const int sms = device_sm_count();
  if (sms <= 0) return cudaErrorInvalidDevice;
  const Tile t = make_tile(a.d, a.at.num_tokens, 2 * a.Hkv, kReadLanes, 1, 1, sms);
  return launch_overlapped(a.d == 64 ? cache_read_fp8_kernel<64> : cache_read_fp8_kernel<128>,
                           tiles(t, a.at.num_tokens), kTileThreads, 0, stream, 1, a, t);
}

}  // namespace exattn
