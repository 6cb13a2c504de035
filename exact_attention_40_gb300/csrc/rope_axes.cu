// Rotary positions of several axes, and the 4-bit paged cache's append and read,
// for sm_103a.
//
// Pairs (i, i + d/2) of a head vector turn by position[axis(i)] * theta_i
// (rotary.cuh): with one axis the rotary embedding of text, with several (time,
// height, width) that of images and video.  The gradient of a rotation is the
// reverse rotation, the same kernel with the sines negated.
//
// All three kernels are bound by their bytes.  A CTA takes a tile of `toks`
// tokens; it forms the tile's cosines and sines once, in shared memory, and
// its threads then walk the heads.  Thread (token, j) of d/16 threads a token
// owns the 8 pairs 8 j .. 8 j + 7 of every head it visits (two 16-byte loads,
// two 16-byte stores), so its cosines and sines stay in registers; `lanes`
// such sets of threads share the heads.  Tiles shrink, and lanes grow, until
// there are two CTAs an SM.
#include <cuda_bf16.h>

#include "fp4.cuh"
#include "launch.h"
#include "ptx.cuh"
#include "rotary.cuh"

namespace exattn {
namespace {

constexpr int kTileThreads = 256;
constexpr int kUnroll = 4;  // heads whose loads are in flight together

// How a CTA's threads cover tokens and heads.
struct Tile {
  int per_tok;  // threads per token: d / 16
  int toks;     // tokens per CTA
  int lanes;    // threads that share a (token, j)
};

__device__ __forceinline__ const uint4* row_of(const HeadView& v, long long b, long long h, long long n) {
  return static_cast<const uint4*>(v.ptr) + b * v.batch + h * v.head + n * v.token;
}

// Cosines and sines of the tile's tokens into cs[token][pair]: pos(token, axis)
// gives the position.
template <typename Pos>
__device__ __forceinline__ void tile_angles(float2* cs, const RopeAxesTable& table, int half, int count, Pos pos) {
  for (int idx = threadIdx.x; idx < count * half; idx += kTileThreads) {
    const int tok = idx / half, i = idx - tok * half;
    const long long p = pos(tok, table.axis[i]);
    cs[idx] = turn_cos_sin(static_cast<unsigned long long>(p) * table.u[i]);
  }
}

__device__ __forceinline__ void load_cs(const float2* cs, float (&c)[8], float (&s)[8], float sign) {
#pragma unroll
  for (int e = 0; e < 8; e += 2) {
    const float4 x = *reinterpret_cast<const float4*>(cs + e);
    c[e] = x.x;
    s[e] = sign * x.y;
    c[e + 1] = x.z;
    s[e + 1] = sign * x.w;
  }
}

__device__ __forceinline__ void turn8(const uint4 lo, const uint4 hi, const float (&c)[8], const float (&s)[8],
                                      float (&a)[8], float (&b)[8]) {
  unpack_bf16x8(lo, a);
  unpack_bf16x8(hi, b);
#pragma unroll
  for (int e = 0; e < 8; ++e) turn_pair(a[e], b[e], c[e], s[e]);
}

__global__ void __launch_bounds__(kTileThreads) rope_axes_kernel(const RopeAxesArgs a,
                                                                 const __grid_constant__ RopeAxesTable table,
                                                                 const Tile tile) {
  extern __shared__ __align__(16) uint8_t rope_axes_smem[];
  float2* cs = reinterpret_cast<float2*>(rope_axes_smem);
  const int half = a.d / 2, vec_half = half / 8;
  const unsigned int total = static_cast<unsigned int>(a.B) * a.N, n0 = blockIdx.x * tile.toks;
  const int count = static_cast<int>(min(total - n0, static_cast<unsigned int>(tile.toks)));
  tile_angles(cs, table, half, count, [&](int tok, int axis) {
    const unsigned int b = (n0 + tok) / a.N, n = n0 + tok - b * a.N;
    return static_cast<long long>(a.positions[axis * a.pos_axis + b * a.pos_batch + n * a.pos_token]);
  });
  __syncthreads();
  const int j = threadIdx.x % tile.per_tok, rest = threadIdx.x / tile.per_tok;
  const int tok = rest % tile.toks, lane = rest / tile.toks;
  if (lane >= tile.lanes || tok >= count) return;
  float c[8], s[8];
  load_cs(cs + tok * half + 8 * j, c, s, a.inverse ? -1.f : 1.f);
  const unsigned int b = (n0 + tok) / a.N, n = n0 + tok - b * a.N;
  const int heads = a.Hq + a.Hkv;
  for (int h0 = lane; h0 < heads; h0 += kUnroll * tile.lanes) {
    uint4 lo[kUnroll], hi[kUnroll];
#pragma unroll
    for (int x = 0; x < kUnroll; ++x) {
      const int h = h0 + x * tile.lanes;
      if (h < heads) {
        const uint4* src = (h < a.Hq ? row_of(a.q, b, h, n) : row_of(a.k, b, h - a.Hq, n)) + j;
        lo[x] = src[0];
        hi[x] = src[vec_half];
      }
    }
#pragma unroll
    for (int x = 0; x < kUnroll; ++x) {
      const int h = h0 + x * tile.lanes;
      if (h < heads) {
        float ya[8], yb[8];
        turn8(lo[x], hi[x], c, s, ya, yb);
        uint4* dst =
            const_cast<uint4*>(h < a.Hq ? row_of(a.q_out, b, h, n) : row_of(a.k_out, b, h - a.Hq, n)) + j;
        dst[0] = pack_bf16x8(ya);
        dst[vec_half] = pack_bf16x8(yb);
      }
    }
  }
}

// Span index (block * Hkv) and offset of a token in the cache, or -1.
__device__ __forceinline__ long long find_block(const Fp4Slots& at, long long n, int* off) {
  const int seq = at.seq_ids[n], slot = at.slots[n];
  *off = slot & 15;
  if (seq < 0 || seq >= at.num_seqs || slot < 0 || slot / 16 >= at.max_blocks_per_seq) return -1;
  const int blk = at.block_table[static_cast<long long>(seq) * at.max_blocks_per_seq + slot / 16];
  return blk >= 0 && blk < at.num_blocks ? blk : -1;
}

// Largest magnitude of 8 values, NaN if one is.
__device__ __forceinline__ float amax8(const float (&x)[8]) {
  float m = fabsf(x[0]);
#pragma unroll
  for (int e = 1; e < 8; ++e) m = max_nan(m, fabsf(x[e]));
  return m;
}

// Append: heads in the order q, k, v.  A rotated key's 8 low (and 8 high)
// columns are half of a scale group; the neighbouring thread has the other
// half.  A value's thread takes a whole group.
template <int D>
__global__ void __launch_bounds__(kTileThreads) rope_cache_fp4_kernel(const RopeFp4Args a,
                                                                      const __grid_constant__ RopeAxesTable table,
                                                                      const Tile tile) {
  using Span = Fp4Span<D>;
  constexpr int kHalf = D / 2, kVecHalf = kHalf / 8, kPerTok = D / 16;
  extern __shared__ __align__(16) uint8_t rope_axes_smem[];
  float2* cs = reinterpret_cast<float2*>(rope_axes_smem);
  const long long n0 = static_cast<long long>(blockIdx.x) * tile.toks;
  const int count = static_cast<int>(a.at.num_tokens - n0 < tile.toks ? a.at.num_tokens - n0 : tile.toks);
  tile_angles(cs, table, kHalf, count,
              [&](int tok, int axis) { return static_cast<long long>(a.positions[axis * a.pos_axis + n0 + tok]); });
  __syncthreads();
  const int j = threadIdx.x % kPerTok, rest = threadIdx.x / kPerTok;
  const int tok = rest % tile.toks, lane = rest / tile.toks;
  if (lane >= tile.lanes || tok >= count) return;
  const unsigned int pair_mask = 3u << (threadIdx.x & 30);  // this thread and its neighbour: same token and heads
  const long long n = n0 + tok;
  float c[8], s[8];
  load_cs(cs + tok * kHalf + 8 * j, c, s, 1.f);
  int off;
  const long long blk = find_block(a.at, n, &off);
  if (blk < 0 && j == 0 && lane == 0) atomicOr(a.at.status, 2u);  // EXATTN_DEVICE_BOUNDS_BIT
  uint8_t* spans = static_cast<uint8_t*>(a.kv_cache) + (blk < 0 ? 0 : blk) * a.Hkv * Span::kBytes;
  const int heads = a.Hq + 2 * a.Hkv;
  for (int h0 = lane; h0 < heads; h0 += kUnroll * tile.lanes) {
    uint4 lo[kUnroll], hi[kUnroll];
#pragma unroll
    for (int x = 0; x < kUnroll; ++x) {
      const int h = h0 + x * tile.lanes;
      if (h < a.Hq + a.Hkv) {
        const uint4* src = (h < a.Hq ? row_of(a.q, 0, h, n) : row_of(a.k, 0, h - a.Hq, n)) + j;
        lo[x] = src[0];
        hi[x] = src[kVecHalf];
      } else if (h < heads) {
        const uint4* src = row_of(a.v, 0, h - a.Hq - a.Hkv, n) + 2 * j;
        lo[x] = src[0];
        hi[x] = src[1];
      }
    }
#pragma unroll
    for (int x = 0; x < kUnroll; ++x) {
      const int h = h0 + x * tile.lanes;
      float ya[8], yb[8];
      if (h < a.Hq) {
        turn8(lo[x], hi[x], c, s, ya, yb);
        uint4* dst = const_cast<uint4*>(row_of(a.q_out, 0, h, n)) + j;
        dst[0] = pack_bf16x8(ya);
        dst[kVecHalf] = pack_bf16x8(yb);
      } else if (h < a.Hq + a.Hkv) {
        turn8(lo[x], hi[x], c, s, ya, yb);
        float ma = amax8(ya), mb = amax8(yb);
        ma = max_nan(ma, __shfl_xor_sync(pair_mask, ma, 1));
        mb = max_nan(mb, __shfl_xor_sync(pair_mask, mb, 1));
        float da, db;
        const uint32_t sa = fp4_group_scale(ma, a.k_scale, &da), sb = fp4_group_scale(mb, a.k_scale, &db);
        if (blk >= 0) {
          uint8_t* span = spans + static_cast<size_t>(h - a.Hq) * Span::kBytes;
          uint32_t* codes = reinterpret_cast<uint32_t*>(span + Span::kKeyCodes + off * Span::kCodeRow) + j;
          codes[0] = fp4_encode8(ya, da);
          codes[kPerTok] = fp4_encode8(yb, db);
          // the even thread of a pair stores the low group's scale, the odd one the high one's
          span[Span::kKeyScales + off * Span::kScaleRow + j / 2 + (j & 1) * (Span::kScaleRow / 2)] =
              static_cast<uint8_t>(j & 1 ? sb : sa);
        }
      } else if (h < heads && blk >= 0) {
        unpack_bf16x8(lo[x], ya);
        unpack_bf16x8(hi[x], yb);
        float dv;
        const uint32_t sv = fp4_group_scale(max_nan(amax8(ya), amax8(yb)), a.v_scale, &dv);
        uint8_t* span = spans + static_cast<size_t>(h - a.Hq - a.Hkv) * Span::kBytes;
        reinterpret_cast<uint2*>(span + Span::kValueCodes + off * Span::kCodeRow)[j] =
            make_uint2(fp4_encode8(ya, dv), fp4_encode8(yb, dv));
        span[Span::kValueScales + off * Span::kScaleRow + j] = static_cast<uint8_t>(sv);
      }
    }
  }
}

// Read: thread j of a token takes group j of the keys and values of every head
// it visits.
template <int D>
__global__ void __launch_bounds__(kTileThreads) cache_read_fp4_kernel(const ReadFp4Args a, const Tile tile) {
  using Span = Fp4Span<D>;
  constexpr int kPerTok = D / 16;
  const int j = threadIdx.x % kPerTok, rest = threadIdx.x / kPerTok;
  const int tok = rest % tile.toks, lane = rest / tile.toks;
  const long long n = static_cast<long long>(blockIdx.x) * tile.toks + tok;
  if (lane >= tile.lanes || n >= a.at.num_tokens) return;
  int off;
  const long long blk = find_block(a.at, n, &off);
  if (blk < 0 && j == 0 && lane == 0) atomicOr(a.at.status, 2u);  // EXATTN_DEVICE_BOUNDS_BIT
  const uint8_t* spans = static_cast<const uint8_t*>(a.kv_cache) + (blk < 0 ? 0 : blk) * a.Hkv * Span::kBytes;
  // rows 2 h: key of head h, rows 2 h + 1: its value
  for (int r0 = lane; r0 < 2 * a.Hkv; r0 += kUnroll * tile.lanes) {
    uint2 codes[kUnroll];
    uint32_t scale[kUnroll];
#pragma unroll
    for (int x = 0; x < kUnroll; ++x) {
      const int r = r0 + x * tile.lanes;
      codes[x] = make_uint2(0u, 0u);
      scale[x] = 0u;
      if (r < 2 * a.Hkv && blk >= 0) {
        const uint8_t* span = spans + static_cast<size_t>(r >> 1) * Span::kBytes;
        codes[x] = reinterpret_cast<const uint2*>(span + (r & 1 ? Span::kValueCodes : Span::kKeyCodes) +
                                                  off * Span::kCodeRow)[j];
        scale[x] = span[(r & 1 ? Span::kValueScales : Span::kKeyScales) + off * Span::kScaleRow + j];
      }
    }
#pragma unroll
    for (int x = 0; x < kUnroll; ++x) {
      const int r = r0 + x * tile.lanes;
      if (r >= 2 * a.Hkv) break;
      const uint32_t s8 = e4m3x2_to_f16(scale[x] | (scale[x] << 8));
      const float g = r & 1 ? a.v_scale : a.k_scale;
      uint32_t h[8], w[8];
      {
        uint32_t h0[4], h1[4];
        e2m1x8_to_f16(codes[x].x, h0);
        e2m1x8_to_f16(codes[x].y, h1);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          h[e] = h0[e];
          h[4 + e] = h1[e];
        }
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const uint32_t v = f16x2_mul(h[e], s8);
        w[e] = pack_bf16x2(__fmul_rn(f16_lo(v), g), __fmul_rn(f16_hi(v), g));
      }
      uint4* dst = const_cast<uint4*>(row_of(r & 1 ? a.v_out : a.k_out, 0, r >> 1, n)) + 2 * j;
      dst[0] = make_uint4(w[0], w[1], w[2], w[3]);
      dst[1] = make_uint4(w[4], w[5], w[6], w[7]);
    }
  }
}

// Tokens per CTA: as many as the threads hold, halved while there are fewer
// than two CTAs an SM; the other threads share the `rows` heads of a token.
Tile make_tile(int d, long long tokens, int rows, int sms) {
  Tile t;
  t.per_tok = d / 16;
  const int slots = kTileThreads / t.per_tok;
  t.toks = 1;
  while (2 * t.toks <= slots) t.toks *= 2;
  while (t.toks > 1 && (tokens + t.toks - 1) / t.toks < 2ll * sms && slots / t.toks < rows) t.toks /= 2;
  t.lanes = slots / t.toks;
  return t;
}

unsigned int tiles(const Tile& t, long long tokens) {
  return static_cast<unsigned int>((tokens + t.toks - 1) / t.toks);
}

}  // namespace

cudaError_t launch_rope_axes(const RopeAxesArgs& a, const RopeAxesTable& table, cudaStream_t stream) {
  const int sms = device_sm_count();
  if (sms <= 0) return cudaErrorInvalidDevice;
  const long long tokens = static_cast<long long>(a.B) * a.N;
  const Tile t = make_tile(a.d, tokens, a.Hq + a.Hkv, sms);
  rope_axes_kernel<<<tiles(t, tokens), kTileThreads, sizeof(float2) * t.toks * (a.d / 2), stream>>>(a, table, t);
  return cudaGetLastError();
}

cudaError_t launch_rope_cache_write_fp4(const RopeFp4Args& a, const RopeAxesTable& table, cudaStream_t stream) {
  const int sms = device_sm_count();
  if (sms <= 0) return cudaErrorInvalidDevice;
  const Tile t = make_tile(a.d, a.at.num_tokens, a.Hq + 2 * a.Hkv, sms);
  const unsigned int grid = tiles(t, a.at.num_tokens);
  const size_t smem = sizeof(float2) * t.toks * (a.d / 2);
  if (a.d == 64)
    rope_cache_fp4_kernel<64><<<grid, kTileThreads, smem, stream>>>(a, table, t);
  else
    rope_cache_fp4_kernel<128><<<grid, kTileThreads, smem, stream>>>(a, table, t);
  return cudaGetLastError();
}

cudaError_t launch_cache_read_fp4(const ReadFp4Args& a, cudaStream_t stream) {
  const int sms = device_sm_count();
  if (sms <= 0) return cudaErrorInvalidDevice;
  const Tile t = make_tile(a.d, a.at.num_tokens, 2 * a.Hkv, sms);
  const unsigned int grid = tiles(t, a.at.num_tokens);
  if (a.d == 64)
    cache_read_fp4_kernel<64><<<grid, kTileThreads, 0, stream>>>(a, t);
  else
    cache_read_fp4_kernel<128><<<grid, kTileThreads, 0, stream>>>(a, t);
  return cudaGetLastError();
}

}  // namespace exattn
