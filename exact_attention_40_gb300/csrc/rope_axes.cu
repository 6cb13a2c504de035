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
// such sets of threads share the heads.  Its loads run three or four heads ahead,
// through shared memory, and start before the angles are formed.  Rates are at the
// constants below and at the kernels.
#include <cuda_bf16.h>

#include "fp4.cuh"
#include "launch.h"
#include "ptx.cuh"
#include "rotary.cuh"

namespace exattn {
namespace {

constexpr int kTileThreads = 256;
// Measured choices (heads of a token in flight together, rows of a thread in the ring
// with the one at hand, CTAs an SM).  Rotation of 8 x 4096 tokens, 32 + 32 heads of 128:
// 156 us = 6.88 TB/s with 8 lanes, 4 or 5 stages and 4 CTAs, 157 with 4 lanes, 166 with
// 5 CTAs of 3 stages, 157 with two rows in registers and no ring.  Append of 16,384
// tokens, 32 + 2 * 8 heads: 56.6 us = 6.26 TB/s with 4 lanes, 5 stages and 3 CTAs; 1 us more
// with 4 stages, 4 with 4 CTAs, 9 with 8 lanes, 3 with 2, 9 without the ring.
constexpr int kRopeLanes = 8;
constexpr int kRopeStages = 4;  // rows of a thread on their way, and the one at hand
constexpr int kFp4Lanes = 4;
constexpr int kFp4Stages = 5;
constexpr int kReadLanes = 4;  // of the read

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
// gives the position.  A thread keeps to one pair, and takes its entry of the table by
// an ordinary load: as an operand of the constant bank it would be served to one
// lane after the other.
template <typename Pos>
__device__ __forceinline__ void tile_angles(float2* cs, const RopeAxesTable& table, int half, int count, Pos pos) {
  const int per = kTileThreads / half, i = threadIdx.x % half;
  if (threadIdx.x >= per * half) return;
  unsigned long long u;
  uint32_t axis;
  asm volatile("ld.b64 %0, [%1];" : "=l"(u) : "l"(table.u + i));
  asm volatile("ld.u8 %0, [%1];" : "=r"(axis) : "l"(table.axis + i));
  for (int tok = threadIdx.x / half; tok < count; tok += per)
    cs[tok * half + i] = turn_cos_sin(static_cast<unsigned long long>(static_cast<long long>(pos(tok, axis))) * u);
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

// Two 16-byte vectors of one row.
struct Vecs {
  uint4 lo, hi;
};

// Rows of a token on their way into shared memory, where a thread finds its own two
// vectors of each; only it reads them, so no barrier is needed.  A stage is filled
// again after the row after it has been waited for, when its vectors are long in
// registers.
template <int kStages>
struct RowRing {
  uint4* slot;  // this thread's: vector x of stage s at slot[(2 s + x) * kTileThreads]
  static constexpr size_t kBytes = sizeof(uint4) * 2 * kStages * kTileThreads;
  __device__ __forceinline__ void fetch(int stage, const uint4* src, int apart) const {
    cp_async16(smem_u32(slot + 2 * stage * kTileThreads), src, true);
    cp_async16(smem_u32(slot + (2 * stage + 1) * kTileThreads), src + apart, true);
  }
  __device__ __forceinline__ Vecs take(int stage) const {
    return Vecs{slot[2 * stage * kTileThreads], slot[(2 * stage + 1) * kTileThreads]};
  }
};

__global__ void __launch_bounds__(kTileThreads, 4) rope_axes_kernel(const RopeAxesArgs a,
                                                                    const __grid_constant__ RopeAxesTable table,
                                                                    const Tile tile) {
  using Ring = RowRing<kRopeStages>;
  extern __shared__ __align__(16) uint8_t rope_axes_smem[];
  float2* cs = reinterpret_cast<float2*>(rope_axes_smem + Ring::kBytes);
  const Ring ring{reinterpret_cast<uint4*>(rope_axes_smem) + threadIdx.x};
  const int half = a.d / 2, apart = half / 8;
  const unsigned int total = static_cast<unsigned int>(a.B) * a.N, n0 = blockIdx.x * tile.toks;
  const int count = static_cast<int>(min(total - n0, static_cast<unsigned int>(tile.toks)));
  const int j = threadIdx.x % tile.per_tok, rest = threadIdx.x / tile.per_tok;
  const int tok = rest % tile.toks, lane = rest / tile.toks;
  const bool works = lane < tile.lanes && tok < count;
  const unsigned int b = (n0 + tok) / a.N, n = n0 + tok - b * a.N;
  const int step = tile.lanes;
  // rows of a token: query heads, key heads
  const int rows = works ? a.Hq + a.Hkv : 0;
  const uint4* q = row_of(a.q, b, 0, n) + j;
  const uint4* k = row_of(a.k, b, -a.Hq, n) + j;
  int next = lane;  // row to fetch
  auto fetch = [&](int stage) {
    if (next < rows) ring.fetch(stage, next < a.Hq ? q + next * a.q.head : k + next * a.k.head, apart);
    cp_async_commit();
    next += step;
  };
  cudaGridDependencySynchronize();
#pragma unroll
  for (int s = 0; s < kRopeStages - 1; ++s) fetch(s);
  tile_angles(cs, table, half, count, [&](int at, int axis) {
    const unsigned int pb = (n0 + at) / a.N, pn = n0 + at - pb * a.N;
    return static_cast<long long>(a.positions[axis * a.pos_axis + pb * a.pos_batch + pn * a.pos_token]);
  });
  __syncthreads();
  if (!works) return;
  Turn8 turn;
  turn.load(cs + tok * half + 8 * j, a.inverse ? -1.f : 1.f);
  uint4* q_out = const_cast<uint4*>(row_of(a.q_out, b, 0, n)) + j;
  uint4* k_out = const_cast<uint4*>(row_of(a.k_out, b, -a.Hq, n)) + j;
  int stage = 0, behind = kRopeStages - 1;  // of the row at hand, and of the one before it
  for (int r = lane; r < rows; r += step) {
    cp_async_wait<kRopeStages - 2>();
    const Vecs x = ring.take(stage);
    fetch(behind);
    behind = stage;
    stage = stage + 1 == kRopeStages ? 0 : stage + 1;
    float ya[8], yb[8];
    turn.turn(x.lo, x.hi, ya, yb);
    uint4* to = r < a.Hq ? q_out + r * a.q_out.head : k_out + r * a.k_out.head;
    to[0] = pack_bf16x8(ya);
    to[apart] = pack_bf16x8(yb);
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

// Quantises groups of one tensor with fp32 scale g.
//
// Values of a few bits often lie exactly between two codes, so the quotients
// have to be the correctly rounded ones; a product with the reciprocal would not
// see those ties.  They come from the correctly rounded reciprocal r by one
// step: q = x r, q + (x - q y) r with fused multiply-adds is x / y correctly
// rounded (Markstein, IBM Journal of Research and Development 34, 1990).
// Written as q - (q y - x) r it also keeps the sign of a zero x, as the
// division does: the residual of an exact quotient is +0, and adding +0 to -0
// would lose it.  That holds while nothing over- or underflows; the rare rest takes
// the division itself.
struct Quantiser {
  float g, six_g, inv_six_g;
  bool plain;  // 6 g and its reciprocal are of an ordinary size
  __device__ __forceinline__ explicit Quantiser(float scale) {
    g = scale;
    six_g = __fmul_rn(6.f, scale);
    inv_six_g = __frcp_rn(six_g);
    plain = six_g > 1e-25f && six_g < 1e25f;
  }

  // Scale of a group with largest magnitude `amax` (NaN when it holds one):
  // e4m3(amax / (6 g)), NaN when the group holds a NaN or an infinity, so that
  // the whole group reads back as NaN.
  __device__ __forceinline__ uint32_t scale(float amax) const {
    if (!(amax <= 3.4028234663852886e38f)) return 0x7Fu;
    float t = __fmul_rn(amax, inv_six_g);
    if (plain && t < 1000.f)
      t = __fmaf_rn(__fmaf_rn(-t, six_g, amax), inv_six_g, t);
    else
      t = __fdiv_rn(amax, six_g);
    return f32_to_e4m3(t);
  }

  // Codes of 16 values with that scale, in order.
  __device__ __forceinline__ uint2 codes(const float (&x)[16], float amax, uint32_t s8) const {
    const float y = __fmul_rn(f16_lo(e4m3x2_to_f16(s8)), g);
    float q[16];
    // (a scale below the saturated one keeps every quotient under 8)
    if (plain && s8 < 0x7Eu && s8 > 0u && amax < 1e25f) {
      const float r = __frcp_rn(y);
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const float q0 = __fmul_rn(x[e], r);
        q[e] = __fmaf_rn(__fmaf_rn(q0, y, -x[e]), -r, q0);
      }
    } else {
#pragma unroll
      for (int e = 0; e < 16; ++e) q[e] = y == 0.f ? 0.f : __fdiv_rn(x[e], y);
    }
    return make_uint2(f32x8_to_e2m1(q), f32x8_to_e2m1(q + 8));
  }
};

// Largest magnitude of 16 values, NaN if one is.
__device__ __forceinline__ float amax16(const float (&x)[16]) {
  float m = fabsf(x[0]);
#pragma unroll
  for (int e = 1; e < 16; ++e) m = max_nan(m, fabsf(x[e]));
  return m;
}

// Append.  A rotated key's thread has 8 low and 8 high columns, half of a scale
// group each; neighbouring threads swap halves, so that the even one has the
// low group and the odd one the high group.  A value's thread loads a whole
// group.
template <int D>
__global__ void __launch_bounds__(kTileThreads, 3) rope_cache_fp4_kernel(const RopeFp4Args a,
                                                                         const __grid_constant__ RopeAxesTable table,
                                                                         const Tile tile) {
  using Span = Fp4Span<D>;
  using Ring = RowRing<kFp4Stages>;
  constexpr int kHalf = D / 2, kApart = kHalf / 8, kPerTok = D / 16;
  extern __shared__ __align__(16) uint8_t rope_axes_smem[];
  float2* cs = reinterpret_cast<float2*>(rope_axes_smem + Ring::kBytes);
  const Ring ring{reinterpret_cast<uint4*>(rope_axes_smem) + threadIdx.x};
  const long long n0 = static_cast<long long>(blockIdx.x) * tile.toks;
  const int count = static_cast<int>(a.at.num_tokens - n0 < tile.toks ? a.at.num_tokens - n0 : tile.toks);
  const int j = threadIdx.x % kPerTok, rest = threadIdx.x / kPerTok;
  const int tok = rest % tile.toks, lane = rest / tile.toks;
  const bool works = lane < tile.lanes && tok < count;
  const long long n = n0 + tok;
  const int step = tile.lanes;
  // rows of a token: query heads, key heads, value heads
  const int first_key = a.Hq, first_value = a.Hq + a.Hkv, rows = works ? a.Hq + 2 * a.Hkv : 0;
  const uint4* q = row_of(a.q, 0, 0, n) + j;
  const uint4* k = row_of(a.k, 0, -first_key, n) + j;
  const uint4* v = row_of(a.v, 0, -first_value, n) + 2 * j;
  int next = lane;  // row to fetch
  auto fetch = [&](int stage) {
    if (next < first_value) {
      if (next < rows) ring.fetch(stage, next < first_key ? q + next * a.q.head : k + next * a.k.head, kApart);
    } else if (next < rows) {
      ring.fetch(stage, v + next * a.v.head, 1);
    }
    cp_async_commit();
    next += step;
  };
  cudaGridDependencySynchronize();
#pragma unroll
  for (int s = 0; s < kFp4Stages - 1; ++s) fetch(s);
  int off = 0;
  long long blk = -1;
  if (works) {
    blk = find_block(a.at, n, &off);
    if (blk < 0 && j == 0 && lane == 0) atomicOr(a.at.status, 2u);  // EXATTN_DEVICE_BOUNDS_BIT
  }
  tile_angles(cs, table, kHalf, count,
              [&](int at, int axis) { return static_cast<long long>(a.positions[axis * a.pos_axis + n0 + at]); });
  __syncthreads();
  if (!works) return;
  uint8_t* spans = static_cast<uint8_t*>(a.kv_cache) + (blk < 0 ? 0 : blk) * a.Hkv * Span::kBytes;
  int stage = 0, behind = kFp4Stages - 1;  // of the row at hand, and of the one before it
  auto take = [&]() {
    cp_async_wait<kFp4Stages - 2>();
    const Vecs x = ring.take(stage);
    fetch(behind);
    behind = stage;
    stage = stage + 1 == kFp4Stages ? 0 : stage + 1;
    return x;
  };
  int r = lane;
  {
    Turn8 turn;
    turn.load(cs + tok * kHalf + 8 * j, 1.f);
    uint4* dst = const_cast<uint4*>(row_of(a.q_out, 0, 0, n)) + j;
    for (; r < first_key; r += step) {
      const Vecs x = take();
      float ya[8], yb[8];
      turn.turn(x.lo, x.hi, ya, yb);
      uint4* to = dst + r * a.q_out.head;
      to[0] = pack_bf16x8(ya);
      to[kApart] = pack_bf16x8(yb);
    }
    const Quantiser quant(a.k_scale);
    const bool odd = j & 1;
    const unsigned int pair_mask = 3u << (threadIdx.x & 30);  // this thread and its neighbour: same token and rows
    // the group this thread ends up with: j / 2 of the low half, or of the high one
    const int group = j / 2 + (odd ? kPerTok / 2 : 0);
    uint8_t* code = spans + Span::kKeyCodes + off * Span::kCodeRow + group * 8;
    uint8_t* scale = spans + Span::kKeyScales + off * Span::kScaleRow + group;
    for (; r < first_value; r += step) {
      const Vecs x = take();
      float ya[8], yb[8];
      turn.turn(x.lo, x.hi, ya, yb);
      float y[16];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        // the even thread gives its high half for the odd one's low half
        const float mine = odd ? yb[e] : ya[e];
        const float other = __shfl_xor_sync(pair_mask, odd ? ya[e] : yb[e], 1);
        y[e] = odd ? other : mine;
        y[8 + e] = odd ? mine : other;
      }
      const float m = amax16(y);
      const uint32_t s8 = quant.scale(m);
      if (blk >= 0) {
        const int at = (r - first_key) * Span::kBytes;
        *reinterpret_cast<uint2*>(code + at) = quant.codes(y, m, s8);
        scale[at] = static_cast<uint8_t>(s8);
      }
    }
  }
  const Quantiser quant(a.v_scale);
  uint8_t* code = spans + Span::kValueCodes + off * Span::kCodeRow + j * 8;
  uint8_t* scale = spans + Span::kValueScales + off * Span::kScaleRow + j;
  for (; r < rows; r += step) {
    const Vecs x = take();
    float y[16];
    const uint32_t w[8] = {x.lo.x, x.lo.y, x.lo.z, x.lo.w, x.hi.x, x.hi.y, x.hi.z, x.hi.w};
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      y[2 * e] = __uint_as_float(w[e] << 16);
      y[2 * e + 1] = __uint_as_float(w[e] & 0xFFFF0000u);
    }
    const float m = amax16(y);
    const uint32_t s8 = quant.scale(m);
    if (blk >= 0) {
      const int at = (r - first_value) * Span::kBytes;
      *reinterpret_cast<uint2*>(code + at) = quant.codes(y, m, s8);
      scale[at] = static_cast<uint8_t>(s8);
    }
  }
}

// Read: thread j of a token takes group j of the keys and values of every head
// it visits: rows 0 .. Hkv - 1 are keys, the next Hkv values.  Bound by its writes and
// by the chain from a token's place through the block table to its codes, which many
// small CTAs overlap best.  32,768 tokens of 8 heads of 128 (172 MB): 28.7 us = 6.0 TB/s;
// 30.0 with six CTAs an SM instead of eight, 32.9 with 8 lanes, 34.8 with 1, and two
// us more with each group stored as two vectors of 16 bytes, which touch a sector twice.
template <int D>
__global__ void __launch_bounds__(kTileThreads, 8) cache_read_fp4_kernel(const ReadFp4Args a, const Tile tile) {
  using Span = Fp4Span<D>;
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
  const int code_off = off * Span::kCodeRow + 8 * j, scale_off = off * Span::kScaleRow + j;
  uint4* k_out = const_cast<uint4*>(row_of(a.k_out, 0, 0, n)) + 2 * j;
  uint4* v_out = const_cast<uint4*>(row_of(a.v_out, 0, 0, n)) + 2 * j;
  for (int r0 = lane; r0 < 2 * a.Hkv; r0 += kUnroll * tile.lanes) {
    uint2 codes[kUnroll];
    uint32_t scale[kUnroll];
#pragma unroll
    for (int x = 0; x < kUnroll; ++x) {
      const int r = r0 + x * tile.lanes;
      codes[x] = make_uint2(0u, 0u);
      scale[x] = 0u;
      if (r < 2 * a.Hkv && blk >= 0) {
        const uint8_t* span = spans + static_cast<size_t>(r >= a.Hkv ? r - a.Hkv : r) * Span::kBytes;
        codes[x] = *reinterpret_cast<const uint2*>(span + (r >= a.Hkv ? Span::kValueCodes : Span::kKeyCodes) + code_off);
        scale[x] = span[(r >= a.Hkv ? Span::kValueScales : Span::kKeyScales) + scale_off];
      }
    }
#pragma unroll
    for (int x = 0; x < kUnroll; ++x) {
      const int r = r0 + x * tile.lanes;
      if (r >= 2 * a.Hkv) break;
      const uint32_t s8 = e4m3x2_to_f16(__byte_perm(scale[x], 0, 0x4400));
      const float g = r >= a.Hkv ? a.v_scale : a.k_scale;
      uint32_t h0[4], h1[4], w[8];
      e2m1x8_to_f16(codes[x].x, h0);
      e2m1x8_to_f16(codes[x].y, h1);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const uint32_t v = f16x2_mul(e < 4 ? h0[e & 3] : h1[e & 3], s8);
        w[e] = pack_bf16x2(__fmul_rn(f16_lo(v), g), __fmul_rn(f16_hi(v), g));
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

// A tile of as many tokens as the threads hold with `lanes` heads of each walked at
// once: fewer where a token has fewer rows, so that a thread gets `each` of them (2 + 2
// heads of 64, 258,842 tokens: 69 us with four, 95 with one), but no fewer than `least`.
// Halved while there are fewer than two CTAs an SM and a token still has rows for the
// threads that frees (3 x 1001 tokens of 16 heads: 4.2 us; 4.5 with one, 5.5 with four).
Tile make_tile(int d, long long tokens, int rows, int lanes, int each, int least, int sms) {
  Tile t;
  t.per_tok = d / 16;
  const int slots = kTileThreads / t.per_tok;
  while (lanes > least && each * lanes > rows) lanes /= 2;
  // A ring and the cosines and sines, 4 d bytes a token and so 64 for each of its d/16
  // threads, divided by the lanes: within the 48 KB that a launch has without asking (an
  // append has two lanes or more).
  static_assert(RowRing<kRopeStages>::kBytes + 64 * kTileThreads <= 48 * 1024, "shared memory of the rotation");
  static_assert(RowRing<kFp4Stages>::kBytes + 32 * kTileThreads <= 48 * 1024, "shared memory of the append");
  t.toks = 1;
  while (2 * t.toks * lanes <= slots) t.toks *= 2;
  while (t.toks > 1 && (tokens + t.toks - 1) / t.toks < 2 * sms && 2 * (slots / t.toks) <= rows) t.toks /= 2;
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
  const Tile t = make_tile(a.d, tokens, a.Hq + a.Hkv, kRopeLanes, 4, 1, sms);
  const size_t smem = RowRing<kRopeStages>::kBytes + sizeof(float2) * t.toks * (a.d / 2);
  return launch_overlapped(rope_axes_kernel, tiles(t, tokens), kTileThreads, smem, stream, 1, a, table, t);
}

cudaError_t launch_rope_cache_write_fp4(const RopeFp4Args& a, const RopeAxesTable& table, cudaStream_t stream) {
  const int sms = device_sm_count();
  if (sms <= 0) return cudaErrorInvalidDevice;
  const Tile t = make_tile(a.d, a.at.num_tokens, a.Hq + 2 * a.Hkv, kFp4Lanes, 4, 2, sms);
  const size_t smem = RowRing<kFp4Stages>::kBytes + sizeof(float2) * t.toks * (a.d / 2);
  return launch_overlapped(a.d == 64 ? rope_cache_fp4_kernel<64> : rope_cache_fp4_kernel<128>,
                           tiles(t, a.at.num_tokens), kTileThreads, smem, stream, 1, a, table, t);
}

cudaError_t launch_cache_read_fp4(const ReadFp4Args& a, cudaStream_t stream) {
  const int sms = device_sm_count();
  if (sms <= 0) return cudaErrorInvalidDevice;
  const Tile t = make_tile(a.d, a.at.num_tokens, 2 * a.Hkv, kReadLanes, 1, 1, sms);
  return launch_overlapped(a.d == 64 ? cache_read_fp4_kernel<64> : cache_read_fp4_kernel<128>,
                           tiles(t, a.at.num_tokens), kTileThreads, 0, stream, 1, a, t);
}

}  // namespace exattn
