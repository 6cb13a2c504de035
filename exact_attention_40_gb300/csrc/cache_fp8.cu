// The 8-bit paged cache's append and read (layout in fp8.cuh) for sm_103a.
#include <cuda_bf16.h>

#include "fp8.cuh"
#include "launch.h"
#include "ptx.cuh"
#include "rope_rows.cuh"

namespace exattn {
namespace {

constexpr int kAppendThreads = 256;
constexpr int kAppendWarps = kAppendThreads / 32;
constexpr int kAppendCtas = 2;  // that share an SM
constexpr int kBlk = kDecodeBlockSize;
constexpr int kReadLanes = 4;

// New tokens of one sequence that fall into one block: `count` of them from the call's
// token `token` on, at places `place` and following.
struct Run {
  int seq, token, count, place;
  long long slot;  // of the first
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
    x.count = min(kBlk - x.place, end - x.token);
    x.slot = static_cast<long long>(ctx) - (end - begin) + from;
    return x;
  }
};

template <int D>
__global__ void __launch_bounds__(kAppendThreads, kAppendCtas)
    rope_cache_fp8_kernel(const RopeFp8Args a, const __grid_constant__ RopeAxesTable table, const int splits) {
  using Span = Fp8Span<D>;
  constexpr int kHalf = D / 2, kApart = kHalf / 8;  // 16-byte vectors between the halves of a row
  constexpr int kPerTok = D / 16;                   // lanes per token: 8 pairs each
  constexpr int kToks = 32 / kPerTok;               // tokens of a warp at once
  constexpr int kSteps = kBlk / kToks;
  // Cosines and sines by token, then two pairs (float4) of each lane next to each other:
  // the lanes of a token read neighbouring vectors.
  __shared__ float4 angles[kBlk][4][kPerTok];
  __shared__ int upto[kAppendThreads];       // runs of the sequences of this and earlier threads
  __shared__ Added added[kAppendThreads];    // where a thread has one sequence
  __shared__ int warp_sum[kAppendWarps];

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int j = lane % kPerTok, tok0 = lane / kPerTok;
  cudaGridDependencySynchronize();

  // ---- the runs: one for each sequence, or counted from token_starts
  const int per = a.token_starts == nullptr ? 1 : (a.num_seqs + kAppendThreads - 1) / kAppendThreads;
  auto added_of = [&](int s) {
    if (a.token_starts == nullptr) return Added{s, s + 1, __ldg(a.ctx_lens + s)};
    return Added{__ldg(a.token_starts + s), __ldg(a.token_starts + s + 1), __ldg(a.ctx_lens + s)};
  };
  int total = a.num_seqs;
  if (a.token_starts != nullptr) {
    int mine = 0;
    bool bad = false;
    Added x = {0, 0, 0};
    for (int i = 0; i < per; ++i) {
      const int s = threadIdx.x * per + i;
      if (s >= a.num_seqs) break;
      x = added_of(s);
      bad |= x.begin < 0 || x.end < x.begin || x.end > a.num_tokens;
      mine += bad ? 0 : x.runs();
    }
    added[threadIdx.x] = x;
    int sum = mine;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
      const int v = __shfl_up_sync(0xffffffffu, sum, d);
      if (lane >= d) sum += v;
    }
    if (lane == 31) warp_sum[warp] = sum;
    // starts that decrease or leave the call could name a token twice: nothing is done then
    if (__syncthreads_or(bad)) {
      if (blockIdx.x == 0 && threadIdx.x == 0) atomicOr(a.status, 2u);  // EXATTN_DEVICE_BOUNDS_BIT
      return;
    }
    total = 0;
#pragma unroll
    for (int w = 0; w < kAppendWarps; ++w) {
      if (w < warp) sum += warp_sum[w];
      total += warp_sum[w];
    }
    upto[threadIdx.x] = sum;
    __syncthreads();
  }
  auto find_run = [&](int r) {
    if (a.token_starts == nullptr) return added_of(r).run(r, 0);
    int lo = 0, hi = kAppendThreads - 1;  // the first thread with upto > r
    while (lo < hi) {
      const int mid = (lo + hi) / 2;
      if (upto[mid] > r)
        hi = mid;
      else
        lo = mid + 1;
    }
    r -= lo > 0 ? upto[lo - 1] : 0;
    if (per == 1) return added[lo].run(lo, r);
    int s = lo * per;
    Added x = added_of(s);
    while (r >= x.runs() && s + 1 < a.num_seqs) {
      r -= x.runs();
      x = added_of(++s);
    }
    return x.run(s, r);
  };

  // items of a run: key heads, value heads, query heads
  const int first_value = a.Hkv, first_query = 2 * a.Hkv, items = first_query + a.Hq;
  // (the grid has no more CTAs than fit at once: total * splits stays far below 2^31, runs
  // hold a token each and splits are few)
  for (long long unit = blockIdx.x; unit < static_cast<long long>(total) * splits; unit += gridDim.x) {
    const Run run = find_run(static_cast<int>(unit / splits));
    const int part = static_cast<int>(unit % splits);
    uint4 lo[kSteps], hi[kSteps];
    auto load = [&](int item) {
      if (item >= items) return;
      const HeadView& view = item < first_value ? a.k : item < first_query ? a.v : a.q;
      const int head = item < first_value ? item : item < first_query ? item - first_value : item - first_query;
#pragma unroll
      for (int s = 0; s < kSteps; ++s) {
        const int tok = s * kToks + tok0;
        if (tok < run.count) {
          const uint4* row = row_of(view, 0, head, run.token + tok) + j;
          lo[s] = row[0];
          hi[s] = row[kApart];
        } else {
          lo[s] = hi[s] = make_uint4(0u, 0u, 0u, 0u);
        }
      }
    };
    int item = part + splits * warp;
    load(item);
    int blk = -1;
    if (run.slot >= 0 && run.slot < static_cast<long long>(a.max_blocks_per_seq) * kBlk) {
      blk = __ldg(a.block_table + static_cast<long long>(run.seq) * a.max_blocks_per_seq + run.slot / kBlk);
      if (blk >= a.num_blocks) blk = -1;
    }
    if (blk < 0 && part == 0 && threadIdx.x == 0) atomicOr(a.status, 2u);  // EXATTN_DEVICE_BOUNDS_BIT
    __syncthreads();  // the angles of the run before are no longer read
    {
      constexpr int kAtOnce = kAppendThreads / kHalf;
      const int pair = threadIdx.x % kHalf;
      unsigned long long u;
      uint32_t axis;
      asm volatile("ld.b64 %0, [%1];" : "=l"(u) : "l"(table.u + pair));
      asm volatile("ld.u8 %0, [%1];" : "=r"(axis) : "l"(table.axis + pair));
      for (int tok = threadIdx.x / kHalf; tok < run.count; tok += kAtOnce) {
        const long long pos = a.positions[axis * a.pos_axis + run.token + tok];
        reinterpret_cast<float2*>(&angles[tok][pair % 8 / 2][pair / 8])[pair & 1] =
            turn_cos_sin(static_cast<unsigned long long>(pos) * u);
      }
    }
    __syncthreads();
    auto turn_of = [&](int tok) {
      Turn8 t;
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const float4 v = angles[tok][x][j];
        t.c[2 * x] = v.x;
        t.s[2 * x] = v.y;
        t.c[2 * x + 1] = v.z;
        t.s[2 * x + 1] = v.w;
      }
      return t;
    };
    uint8_t* const spans = static_cast<uint8_t*>(a.kv_cache) + static_cast<size_t>(max(blk, 0)) * a.Hkv * Span::kBytes;
    const bool anew = run.place == 0;

    for (; item < items; item += splits * kAppendWarps) {
      if (item >= first_query) {
        // ---- queries: turned and stored
        uint4* out = const_cast<uint4*>(row_of(a.q_out, 0, item - first_query, run.token)) + j;
        uint4 to_lo[kSteps], to_hi[kSteps];
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
          if (s * kToks >= run.count) break;
          float ya[8], yb[8];
          turn_of(s * kToks + tok0).turn(lo[s], hi[s], ya, yb);
          to_lo[s] = pack_bf16x8(ya);
          to_hi[s] = pack_bf16x8(yb);
        }
        load(item + splits * kAppendWarps);
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
          const int tok = s * kToks + tok0;
          if (tok < run.count) {
            out[tok * a.q_out.token] = to_lo[s];
            out[tok * a.q_out.token + kApart] = to_hi[s];
          }
        }
        continue;
      }
      // ---- a head's keys or values of the run
      const bool value = item >= first_value;
      uint8_t* const span = spans + static_cast<size_t>(value ? item - first_value : item) * Span::kBytes;
      uint8_t* const codes = span + (value ? Span::kValueCodes : Span::kKeyCodes);
      uint32_t* const scale = reinterpret_cast<uint32_t*>(span + Span::kScales) + (value ? 1 : 0);
      const uint32_t before = blk >= 0 && !anew ? *scale : 0u;
      float y[kSteps][16];
      float most = 0.f;
#pragma unroll
      for (int s = 0; s < kSteps; ++s) {
        if (s * kToks < run.count) {
          float ya[8], yb[8];
          if (value) {
            unpack_bf16x8(lo[s], ya);
            unpack_bf16x8(hi[s], yb);
          } else {
            turn_of(s * kToks + tok0).turn(lo[s], hi[s], ya, yb);
          }
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            y[s][e] = ya[e];
            y[s][8 + e] = yb[e];
          }
          const bool real = s * kToks + tok0 < run.count;
#pragma unroll
          for (int e = 0; e < 16; ++e) {  // (what is not finite becomes NaN, and has no part in the scale)
            const bool finite = fabsf(y[s][e]) <= 3.4028234663852886e38f;
            most = fmaxf(most, real && finite ? fabsf(y[s][e]) : 0.f);
            if (!finite) y[s][e] = __int_as_float(0x7FC00000);
          }
        }
      }
      load(item + splits * kAppendWarps);
      most = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(most)));
      const int e_before = min(static_cast<int>(before >> 23), 127 + kFp8HighExponent);
      const int e = max(fp8_scale_exponent(most), e_before);
      if (blk < 0) continue;
      const float down = __uint_as_float(static_cast<uint32_t>(254 - e) << 23);
#pragma unroll
      for (int s = 0; s < kSteps; ++s) {
        const int tok = s * kToks + tok0;
        if (tok < run.count) {
          const int place = run.place + tok;
          uint32_t w[4];
#pragma unroll
          for (int x = 0; x < 4; ++x)
            w[x] = f32x4_to_e4m3(y[s][4 * x] * down, y[s][4 * x + 1] * down, y[s][4 * x + 2] * down,
                                 y[s][4 * x + 3] * down);
          uint8_t* row = codes + place * Span::kRow + (j & 1) * 8;
          *reinterpret_cast<uint2*>(row + ((j / 2) ^ fp8_turn<D>(place)) * 16) = make_uint2(w[0], w[1]);
          *reinterpret_cast<uint2*>(row + ((j / 2 + D / 32) ^ fp8_turn<D>(place)) * 16) = make_uint2(w[2], w[3]);
        }
      }
      if (anew || e > e_before) {
        if (lane == 0) *scale = static_cast<uint32_t>(e) << 23;
        if (!anew) {
          // the block's other codes, at the larger scale
          const int shift = e_before > 0 ? 127 + e_before - e : 0;
          const float factor = shift > 0 ? __uint_as_float(static_cast<uint32_t>(shift) << 23) : 0.f;
#pragma unroll 1
          for (int v = lane; v < D; v += 32) {
            const int place = v / (D / 16);
            if (place >= run.place && place < run.place + run.count) continue;
            uint4* at = reinterpret_cast<uint4*>(codes) + v;
            const uint4 old = *at;
            auto moved = [&](uint32_t w) {
              uint32_t h0, h1;
              e4m3x4_to_f16(w, h0, h1);
              return f32x4_to_e4m3(f16_lo(h0) * factor, f16_hi(h0) * factor, f16_lo(h1) * factor, f16_hi(h1) * factor);
            };
            *at = make_uint4(moved(old.x), moved(old.y), moved(old.z), moved(old.w));
          }
          __syncwarp();
        }
      }
    }
  }
}

// Read: thread j of a token takes chunk j of the keys and values of every head
// it visits: rows 0 .. Hkv - 1 are keys, the next Hkv values.
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

}  // namespace

cudaError_t launch_rope_cache_write_fp8(const RopeFp8Args& a, const RopeAxesTable& table, cudaStream_t stream) {
  const int sms = device_sm_count();
  if (sms <= 0) return cudaErrorInvalidDevice;
  // About as many runs as the call can have; where they are fewer than the CTAs that fit at
  // once, several CTAs share the heads of each, down to one for each warp.
  const long long few = a.num_seqs < a.num_tokens ? a.num_seqs : a.num_tokens;
  const long long runs = a.token_starts == nullptr ? a.num_tokens : a.num_tokens / kBlk + few;
  const int fit = sms * kAppendCtas, most = (a.Hq + 2 * a.Hkv + kAppendWarps - 1) / kAppendWarps;
  const int wanted = static_cast<int>((fit + runs - 1) / runs);
  const int splits = wanted < 1 ? 1 : wanted < most ? wanted : most;
  const long long units = runs * splits;
  const int grid = static_cast<int>(units < fit ? units : fit);
  return launch_overlapped(a.d == 64 ? rope_cache_fp8_kernel<64> : rope_cache_fp8_kernel<128>, grid, kAppendThreads, 0,
                           stream, 1, a, table, splits);
}

cudaError_t launch_cache_read_fp8(const ReadFp8Args& a, cudaStream_t stream) {
  const int sms = device_sm_count();
  if (sms <= 0) return cudaErrorInvalidDevice;
  const Tile t = make_tile(a.d, a.at.num_tokens, 2 * a.Hkv, kReadLanes, 1, 1, sms);
  return launch_overlapped(a.d == 64 ? cache_read_fp8_kernel<64> : cache_read_fp8_kernel<128>,
                           tiles(t, a.at.num_tokens), kTileThreads, 0, stream, 1, a, t);
}

}  // namespace exattn
