// What the kernels that walk tokens' head vectors share (rotations, appends to and reads
// of the quantised caches): rows by their strides, a thread's part of a rotation, a token's
// block in a paged cache, and how a CTA's threads cover tokens and heads.
#pragma once
#include "launch.h"
#include "ptx.cuh"
#include "rotary.cuh"

namespace exattn {

constexpr int kTileThreads = 256;

// How a CTA's threads cover tokens and heads.
struct Tile {
  int per_tok;  // threads per token: d / 16
  int toks;     // tokens per CTA
  int lanes;    // threads that share a (token, j)
};

__device__ __forceinline__ const uint4* row_of(const HeadView& v, long long b, long long h, long long n) {
  return static_cast<const uint4*>(v.ptr) + b * v.batch + h * v.head + n * v.token;
}

// A thread's 8 cosines and sines.
struct Turn8 {
  float c[8], s[8];
  __device__ __forceinline__ void load(const float2* cs, float sign) {
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
      const float4 x = *reinterpret_cast<const float4*>(cs + e);
      c[e] = x.x;
      s[e] = sign * x.y;
      c[e + 1] = x.z;
      s[e + 1] = sign * x.w;
    }
  }
  // The turned pairs of the vectors (lo, hi).  Products are rounded before they are
  // added, so that the fp32 result, and with it every 4-bit code, is the one
  // that the definition's plain fp32 operations give.  (Packed f32x2
  // operations do not keep that: their products end up fused into the sums.)
  __device__ __forceinline__ void turn(const uint4 lo, const uint4 hi, float (&ya)[8], float (&yb)[8]) const {
    float a[8], b[8];
    unpack_bf16x8(lo, a);
    unpack_bf16x8(hi, b);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      ya[e] = __fsub_rn(__fmul_rn(a[e], c[e]), __fmul_rn(b[e], s[e]));
      yb[e] = __fadd_rn(__fmul_rn(b[e], c[e]), __fmul_rn(a[e], s[e]));
    }
  }
};

// Span index (block * Hkv) and offset of a token in the cache, or -1.
__device__ __forceinline__ long long find_block(const PagedSlots& at, long long n, int* off) {
  const int seq = at.seq_ids[n], slot = at.slots[n];
  *off = slot & 15;
  if (seq < 0 || seq >= at.num_seqs || slot < 0 || slot / 16 >= at.max_blocks_per_seq) return -1;
  const int blk = at.block_table[static_cast<long long>(seq) * at.max_blocks_per_seq + slot / 16];
  return blk >= 0 && blk < at.num_blocks ? blk : -1;
}

// A tile of as many tokens as the threads hold with `lanes` heads of each walked at
// once: fewer where a token has fewer rows, so that a thread gets `each` of them (2 + 2
// heads of 64, 258,842 tokens: 69 us with four, 95 with one), but no fewer than `least`.
// Halved while there are fewer than two CTAs an SM and a token still has rows for the
// threads that frees (3 x 1001 tokens of 16 heads: 4.2 us; 4.5 with one, 5.5 with four).
inline Tile make_tile(int d, long long tokens, int rows, int lanes, int each, int least, int sms) {
  Tile t;
  t.per_tok = d / 16;
  const int slots = kTileThreads / t.per_tok;
  while (lanes > least && each * lanes > rows) lanes /= 2;
  t.toks = 1;
  while (2 * t.toks * lanes <= slots) t.toks *= 2;
  while (t.toks > 1 && (tokens + t.toks - 1) / t.toks < 2 * sms && 2 * (slots / t.toks) <= rows) t.toks /= 2;
  t.lanes = slots / t.toks;
  return t;
}

inline unsigned int tiles(const Tile& t, long long tokens) {
  return static_cast<unsigned int>((tokens + t.toks - 1) / t.toks);
}

}  // namespace exattn
