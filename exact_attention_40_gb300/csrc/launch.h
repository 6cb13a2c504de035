// Internal launch interface between the C-ABI layer (api.cu) and the kernel
// translation units.  Not part of the public ABI.
#pragma once
#include <atomic>
#include <cstddef>
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

namespace exattn {

// Streaming multiprocessors of the current device (cached per device; 0 on
// error).  Grids of the persistent and grid-stride kernels are sized by it.
inline int device_sm_count() {
  // Launchers run outside the API lock: callers racing on a device's first
  // query store the same value.
  static std::atomic<int> cached[64] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
  int n = cached[dev].load(std::memory_order_relaxed);
  if (n == 0) {
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
    cached[dev].store(n, std::memory_order_relaxed);
  }
  return n;
}

// Launches a kernel that may take its place on the SMs while the last CTAs of the one before
// it on the stream end (programmatic dependent launch): about 1 us of a launch's 2
// to 3.  Every thread of it calls cudaGridDependencySynchronize before it reads or writes
// any tensor.  The 4-bit decode lets the next kernel (its merge, or what follows a
// small call) in earlier, after its own wait, so that what came before both has ended
// by then.  The others do not: CTAs of the next call would take slots that the present
// one's last CTAs want (rotation of 3 x 1001 tokens 5.5 us against 4.6; the same trigger
// in the merge, decode of 9 sequences of 1000 to 4000 tokens, 15.0 against 12.4).
// `cluster`: CTAs of a cluster.
template <typename... Params, typename... Args>
cudaError_t launch_overlapped(void (*kernel)(Params...), dim3 grid, int threads, size_t smem, cudaStream_t stream,
                              int cluster, const Args&... args) {
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// Raises `func`'s dynamic shared-memory limit to `bytes` once per device:
// `done` is the calling launcher's own per-device record of the value set
// (callers racing on a device's first launch set the same attribute).
inline cudaError_t smem_limit_once(const void* func, int bytes, std::atomic<int> (&done)[64]) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (done[dev].load(std::memory_order_acquire) == bytes) return cudaSuccess;
  e = cudaFuncSetAttribute(func, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done[dev].store(bytes, std::memory_order_release);
  return e;
}

// Wait budget for every bounded pipeline wait inside the kernels.
struct DeviceGuard {
  unsigned int* status;        // device status word (OR of EXATTN_DEVICE_*_BIT)
  unsigned long long wait_ns;  // per-wait time budget
};

struct PrefillArgs {
  const CUtensorMap* tm_q;
  const CUtensorMap* tm_k;
  const CUtensorMap* tm_v;
  const CUtensorMap* tm_o;  // out, stored one 128-row tile at a time with TMA
  void* out;  // [B, Hq, Nq, d] bf16
  float* lse;
  int B, Hq, Hkv, Nq, Nk, d;
  int causal;
  float scale;
};

cudaError_t launch_prefill(const PrefillArgs& a, const DeviceGuard& g, cudaStream_t stream);
size_t prefill_smem_bytes(int d);

constexpr int kDecodeSplitTokens = 512;
constexpr int kDecodeBlockSize = 16;

struct DecodeArgs {
  const CUtensorMap* tm_k;  // cache viewed as [num_blocks * Hkv * 16 rows, d], 16-row boxes
  const CUtensorMap* tm_v;
  const void* q;
  const void* k_cache;
  const void* v_cache;
  const int32_t* block_table;
  const int32_t* ctx_lens;
  void* out;
  float* lse;
  float* ws_o;    // [num_seqs, Hq, max_splits, d]
  float* ws_lse;  // [num_seqs, Hq, max_splits]
  int num_seqs, Hq, Hkv, d, num_blocks, max_blocks_per_seq, max_splits;
  float scale;
};

cudaError_t launch_decode(const DecodeArgs& a, const DeviceGuard& g, cudaStream_t stream);

struct NormArgs {
  const void* x;          // [n_rows, hidden] bf16
  const void* residual;   // [n_rows, hidden] bf16
  const void* weight;     // [hidden] bf16
  void* out;              // [n_rows, hidden] bf16
  void* residual_out;     // [n_rows, hidden] bf16: x + residual
  long long n_rows;
  int hidden;             // multiple of 8, at most kNormMaxHidden
  float inv_hidden;       // 1 / hidden
  float eps;
};

constexpr int kNormMaxHidden = 16384;

cudaError_t launch_add_rms_norm(const NormArgs& a, cudaStream_t stream);

constexpr int kRopeMaxDim = 256;

struct RopeArgs {
  void* q;                    // [num_tokens, Hq, d] bf16, rotated in place
  const void* k;              // [num_tokens, Hkv, d] bf16
  const void* v;              // [num_tokens, Hkv, d] bf16
  const int32_t* seq_ids;     // [num_tokens]
  const int32_t* positions;   // [num_tokens]
  const int32_t* block_table; // [num_seqs, max_blocks_per_seq]
  void* k_cache;              // [num_blocks, Hkv, 16, d] bf16
  void* v_cache;
  unsigned int* status;       // device status word
  long long num_tokens;
  int Hq, Hkv, d, num_seqs, num_blocks, max_blocks_per_seq;
  double log2_base;
};

cudaError_t launch_rope_cache_write(const RopeArgs& a, cudaStream_t stream);

// Positions of several axes: strides (in elements) of [axes][batch][token], or
// of [axes][token] with batch stride 0.
struct RopeAxesTable {
  unsigned long long u[kRopeMaxDim / 2];  // theta_i / (2 pi), in units of 2^-64 turn
  unsigned char axis[kRopeMaxDim / 2];    // position axis of pair i
};

constexpr int kRopeMaxAxes = 4;

// A [batch, heads, tokens, d] bf16 tensor by its strides, in 16-byte vectors.
struct HeadView {
  const void* ptr;
  long long batch, head, token;
};

struct RopeAxesArgs {
  HeadView q, k, q_out, k_out;
  const int32_t* positions;
  long long pos_axis, pos_batch, pos_token;
  unsigned int B, N;  // B * N < 2^31
  int Hq, Hkv, d, inverse;
};

cudaError_t launch_rope_axes(const RopeAxesArgs& a, const RopeAxesTable& table, cudaStream_t stream);

// Where the tokens of the 4-bit cache calls lie.
struct Fp4Slots {
  const int32_t* seq_ids;      // [num_tokens]
  const int32_t* slots;        // [num_tokens]: token index within its sequence
  const int32_t* block_table;  // [num_seqs, max_blocks_per_seq]
  unsigned int* status;        // device status word
  long long num_tokens;
  int num_seqs, num_blocks, max_blocks_per_seq;
};

struct RopeFp4Args {
  HeadView q, k, v, q_out;  // batch stride unused
  const int32_t* positions;
  long long pos_axis;       // stride between axes, in elements
  void* kv_cache;           // [num_blocks, Hkv, 18 d]
  Fp4Slots at;
  int Hq, Hkv, d;
  float k_scale, v_scale;
};

cudaError_t launch_rope_cache_write_fp4(const RopeFp4Args& a, const RopeAxesTable& table, cudaStream_t stream);

struct ReadFp4Args {
  const void* kv_cache;
  HeadView k_out, v_out;  // batch stride unused
  Fp4Slots at;
  int Hkv, d;
  float k_scale, v_scale;
};

cudaError_t launch_cache_read_fp4(const ReadFp4Args& a, cudaStream_t stream);

constexpr int kFp4UnitBlocks = 8;       // blocks in a unit of the 4-bit decode's work
constexpr int kFp4Sms = 152;
constexpr int kFp4MaxCtas = kFp4Sms * 3;  // no grid of the batch's shares is larger

// CTAs of the 4-bit decode that share an SM, for segments of `rows` query heads.
// Three of four computing warps, though registers and shared memory would hold
// four at d = 64: a batch of 64 x 8192 tokens takes 67.4 us with three, 73.1 with
// four and 78.2 with two (d = 128, where four would spill: 106, 132 and 109).  Two for
// 16 heads, whose accumulators fill the registers: 168 of them at d = 128, with four
// words spilled in the form for small calls and none in the other.
constexpr __host__ __device__ int fp4_decode_ctas(int rows) { return rows > 8 ? 2 : 3; }

constexpr int kFp4ClusterCtas = 8;      // CTAs of a segment in a small call (the portable cluster size)
constexpr int kFp4ClusterUnits = 32;    // units of the longest segment of a small call

// A segment (the query heads of one sequence that share a KV head, in chunks
// of `rows`) that starts in CTA `cta` and goes on through `more` further CTAs.
struct Fp4Joint {
  int cta, more;
  int row;   // its first row of the output
  int rows;  // and how many
};

// How the 4-bit decode divides a call.  By the call's sizes alone, so that the
// workspace can be sized on any host and a captured graph stays good.
struct Fp4Plan {
  int rows;               // query heads per segment: 8 columns of an mma, or 16 for larger groups
  int chunks;             // segments per KV head
  int ctas;               // shares: one wave, but no more than there can be places
  int joints;             // entries of the list of shared segments; 0 where the merge finds them itself
  bool cluster;           // a cluster of CTAs for each segment
  bool shared;            // whether a segment's partial outputs can lie in several CTAs' workspace
  bool fits;              // the numbers of the work's places fit 32 bits
  Fp4Plan(int num_seqs, int Hkv, int group, int max_blocks_per_seq) {
    rows = group <= 8 ? 8 : 16;
    chunks = (group + rows - 1) / rows;
    const long long segments = static_cast<long long>(num_seqs) * Hkv * chunks;
    const long long units = segments * ((max_blocks_per_seq + kFp4UnitBlocks - 1) / kFp4UnitBlocks);
    const int wave = kFp4Sms * fp4_decode_ctas(rows);
    const bool split = units > segments;
    // (with a place more for each segment's end, which a CTA may get alone, where that
    // leaves every other CTA a single unit)
    const long long shares = split ? units + segments : units;
    ctas = static_cast<int>(shares < wave ? shares : wave);
    cluster = split && segments * kFp4ClusterCtas <= wave && units <= segments * kFp4ClusterUnits;
    if (cluster) ctas = static_cast<int>(segments * kFp4ClusterCtas);
    shared = split && !cluster;
    joints = shared && segments > ctas ? ctas : 0;
    fits = units + segments <= 0x7FFFFFFF;  // the places of units and of segments' ends
  }
  size_t joint_bytes() const { return sizeof(Fp4Joint) * joints; }
  size_t part_bytes(int d) const { return sizeof(float) * 2 * ctas * rows * d; }
  // of the workspace: joints, partial outputs, their log-sum-exp
  size_t bytes(int d) const {
    return shared ? joint_bytes() + part_bytes(d) + sizeof(float) * 2 * ctas * rows : 0;
  }
};

struct DecodeFp4Args {
  const void* q;
  const void* kv_cache;
  const int32_t* block_table;
  const int32_t* ctx_lens;
  void* out;
  float* lse;
  void* workspace;  // joints, then partial outputs [2 ctas][rows][d] and their lse
  Fp4Plan plan;
  int num_seqs, Hq, Hkv, d, num_blocks, max_blocks_per_seq;
  float scale, k_scale, v_scale;
};

cudaError_t launch_decode_fp4(const DecodeFp4Args& a, const DeviceGuard& g, cudaStream_t stream);

struct BwdArgs {
  // tensor maps (3-D views (d, rows, planes), 64-column boxes, 128-byte
  // swizzle) of q, dout (planes B*Hq) and k, v (planes B*Hkv), with 64-row
  // and 128-row boxes
  const CUtensorMap* tm_q64;
  const CUtensorMap* tm_do64;
  const CUtensorMap* tm_k128;
  const CUtensorMap* tm_v128;
  const CUtensorMap* tm_q128;
  const CUtensorMap* tm_do128;
  const CUtensorMap* tm_k64;
  const CUtensorMap* tm_v64;
  const CUtensorMap* tm_o128;   // out, 128-row boxes
  const CUtensorMap* tm_dq128;  // dq, 128-row boxes (TMA stores)
  const CUtensorMap* tm_ldp;    // ldp as [B*Hq][1][2 Nq] fp32, 64-pair boxes
  const void* q;     // [B, Hq, Nq, d] bf16
  const void* k;     // [B, Hkv, Nk, d] bf16
  const void* v;
  const void* out;   // forward output [B, Hq, Nq, d] bf16
  const void* dout;  // [B, Hq, Nq, d] bf16
  const float* lse;  // forward log-sum-exp [B, Hq, Nq]
  float* ldp;        // workspace: (lse * log2 e, D) pairs [B*Hq][Nq rounded up to even][2]
  float* part;       // workspace (Hq > Hkv): dK, dV partials per query head, fp32
  void* dq;          // [B, Hq, Nq, d] bf16
  void* dk;          // [B, Hkv, Nk, d] bf16
  void* dv;
  int B, Hq, Hkv, Nq, Nk, d, causal;
  float scale;
};

cudaError_t launch_bwd(const BwdArgs& a, const DeviceGuard& g, cudaStream_t stream);

}  // namespace exattn
