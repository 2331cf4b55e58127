// mea_internal.h -- launch descriptions shared between the C-ABI translation unit
// and the kernel translation units (host side only; no kernel code here).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

namespace mea {

// Raises kernel KERN's dynamic shared-memory limit to `bytes` on the current
// device, once per device (the attribute lasts as long as the device's
// context); later calls only test a bit.  If the context is destroyed and
// created again (cudaDeviceReset), the bit stays set and the kernel's launch
// then fails with an error status instead of running.
template <auto KERN>
cudaError_t set_smem_once(int bytes) {
  static std::atomic<unsigned long long> done{0};  // bit d: done on device d (d < 64)
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = (dev >= 0 && dev < 64) ? (1ull << dev) : 0ull;
  if (bit != 0 && (done.load(std::memory_order_acquire) & bit) != 0) return cudaSuccess;
  e = cudaFuncSetAttribute(KERN, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess && bit != 0) done.fetch_or(bit, std::memory_order_acq_rel);
  return e;
}

// Launches `kern` so that its blocks may start while the stream's previous kernel is
// still running (programmatic dependent launch): the kernel waits for that kernel's
// results itself (grid_dependency_wait), and the launch's own latency is hidden.
template <typename... KArgs, typename... Args>
cudaError_t launch_after(void (*kern)(KArgs...), dim3 grid, int threads, size_t smem,
                         cudaStream_t stream, const Args&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

// Prefill: one CTA computes two 128-row query tiles of one (sequence, head).
constexpr int kFwdRowsPerCta = 256;

struct FwdArgs {
  void* out;
  float* lse;                  // [B, Hq, M] or nullptr
  const int32_t* seqstart_q;   // packed batches only
  const int32_t* seqstart_k;
  int* status;                 // device status word
  long long o_sb, o_sm, o_sh;  // out strides (elements)
  int B, M, N, Hq, Hkv, group;
  int num_units;    // B for dense batches, num_seqs for packed ones
  int num_mblocks;  // ceil(max query rows per unit / kFwdRowsPerCta)
  float scale_log2; // scale * log2(e)
  // Block-sparse only (nullptr otherwise): byte [b * bm_sb + h * bm_sh +
  // (query row / 128) * bm_nk + key / 128], zero = block left out.
  const uint8_t* block_mask;
  long long bm_sb, bm_sh;
  int bm_nk;        // ceil(N / 128)
  // Prefill chunk against a cache only (cache_len nullptr otherwise): the
  // chunk's q/out/lse have M rows per sequence, of which q_lens[b] (nullptr: M)
  // are real; the caches [B, cap, Hkv, K] hold cache_len[b] rows before the call.
  const int32_t* cache_len;
  const int32_t* q_lens;
  const void* k_new;
  const void* v_new;
  void* k_cache;
  void* v_cache;
  long long kn_s[3], vn_s[3], kc_s[3], vc_s[3];  // element strides (b, row, head)
  int cap;
};

constexpr int kSparseBlock = 128;  // rows and keys per block-mask entry

struct FwdLaunch {
  CUtensorMap tmQ, tmK, tmV;
  CUtensorMap tmKn, tmVn;  // new keys / values of a prefill chunk (cache mode only)
  FwdArgs args;
  int head_dim;   // 64 or 128
  bool bf16;
  int mask;       // mea_bias_t value
  bool alibi;
};

cudaError_t launch_fwd(const FwdLaunch& launch, cudaStream_t stream);

// Rows with no visible key (or an empty key set): out = 0, lse = -inf.
cudaError_t launch_fill_empty(void* out, float* lse, int B, int M, int Hq, int K, long long o_sb,
                              long long o_sm, long long o_sh, cudaStream_t stream);

// Decode: split-KV partial kernel + log-sum-exp merge.
constexpr int kDecodeChunk = 512;  // cache rows per split

struct DecodeArgs {
  const void* q;               // [B, Hq, K]
  void* out;                   // [B, Hq, K]
  float* lse;                  // [B, Hq] or nullptr
  const int32_t* kv_seqstart;  // [B + 1]
  float* part_o;               // [B, Hq, max_splits, K]
  float* part_lse;             // [B, Hq, max_splits] (log2 domain)
  int* status;
  int B, Hq, Hkv, group, max_splits, cache_rows;
  float scale_log2;
};

struct DecodeLaunch {
  CUtensorMap tmK, tmV;
  DecodeArgs args;
  int head_dim;
  bool bf16;
  bool alibi;
};

cudaError_t launch_decode(const DecodeLaunch& launch, cudaStream_t stream);

// Backward: dq, dk, dv from q, k, v, out, dout and the forward's lse.
constexpr int kBwdBlock = 128;  // keys per CTA

struct BwdArgs {
  const void *q, *k, *v, *out, *dout;  // contiguous [B,M,Hq,K] / [B,N,Hkv,K]
  const float* lse;                    // [B, Hq, M] natural log (from mea_fwd)
  void *dq, *dk, *dv;
  float* dq_acc;                       // [B, M, Hq, K] fp32 workspace
  float* delta;                        // [B, Hq, M] fp32 workspace: <dout_i, out_i>
  const int32_t* seqstart_q;
  const int32_t* seqstart_k;
  int* status;
  int B, M, N, Hq, Hkv, group, num_units, num_kblocks;
  float scale, scale_log2;
};

struct BwdLaunch {
  CUtensorMap tmQ, tmK, tmV, tmDO;  // boxes: bwd_query_block rows (q, dout), kBwdBlock rows (k, v)
  CUtensorMap tmDQ;                 // fp32 dq accumulator, 32 x 1 x bwd_dq_box_rows boxes
  BwdArgs args;
  int head_dim;
  bool bf16;
  int mask;
  bool alibi;
};

// stages: bit 0 the D / accumulator preparation, bit 1 the main kernel, bit 2
// the dq conversion (the three launches of one backward, in that order).
cudaError_t launch_bwd(const BwdLaunch& launch, cudaStream_t stream, int stages = 7);

// Query rows per step of the backward kernel for head dimension 64 or 128.
int bwd_query_block(int head_dim);
int bwd_dq_box_rows(int head_dim);  // rows of the dq accumulator's TMA reduction boxes

// ---------------------------------------------------------------------------
// Shared by the C-ABI translation units (defined in mea_api.cu).
// ---------------------------------------------------------------------------
int* device_status_word();  // nullptr if the lookup fails

// A [batch, rows, heads, K] 16-bit tensor with element strides st = {b, row,
// head} as a rank-4 TMA map with boxes of 64 elements x 1 head x box_rows.
bool encode_rows(CUtensorMap* map, const void* base, bool bf16, int batch, int rows, int heads,
                 int K, const int64_t st[3], int box_rows);

// ---------------------------------------------------------------------------
// 4-bit cache (mea_kv4_sm100.cu): planes [B, Hkv, cap, ...], contiguous.
// ---------------------------------------------------------------------------
// x / d for x < 2^31: (hi32(x m) + x) >> s.
struct FastDiv {
  uint32_t d, m, s;
};
inline FastDiv fast_div(uint32_t d) {
  FastDiv f{d, 0, 0};
  while ((uint64_t(1) << f.s) < d) ++f.s;
  f.m = static_cast<uint32_t>(((uint64_t(1) << 32) * ((uint64_t(1) << f.s) - d)) / d + 1);
  return f;
}

// Flat order of (sequence, row group, head), the head fastest.
struct RowOrder {
  FastDiv heads, tiles;  // heads; row groups of a sequence
  uint32_t total;        // < 2^31
};

struct Kv4AppendArgs {
  const void *k_new, *v_new;
  void *k_codes, *k_params, *v_codes, *v_params;
  const int32_t* cache_len;
  const int32_t* q_lens;  // nullptr: M
  int* status;
  long long kn_s[3], vn_s[3];
  RowOrder order;
  int M, Hkv, cap;
};

struct Kv4ReadArgs {
  const void *k_codes, *k_params, *v_codes, *v_params;
  void *k_out, *v_out;
  const int32_t* rows;   // [B]
  const int32_t* first;  // [B] or nullptr: 0
  int* status;
  long long ko_s[3], vo_s[3];
  RowOrder order;
  int out_rows, Hkv, cap;
};

struct Kv4DecodeArgs {
  const void* q;
  const void *k_codes, *k_params, *v_codes, *v_params;
  const int32_t* kv_lens;
  void* out;
  float* lse;       // or nullptr
  float* part_o;    // [B, Hq, max_splits, K], nullptr with a single split
  float* part_lse;  // [B, Hq, max_splits] (log2 units) or nullptr
  float* scores;    // [B, Hq, score_stride] (log2 units) or nullptr: no weights wanted
  const float* w_in;
  float* w_out;     // [B, Hkv, cap] or nullptr
  int* status;
  long long score_stride;
  int B, Hq, Hkv, group, cap, max_len, chunk, max_splits;
  int head_blocks;    // ceil(group / 8)
  int merge_blocks;   // blocks of the merge launch that join splits
  int weight_blocks;  // blocks per (sequence, kv head) that gather weights
  float scale_log2;
};

int kv4_weight_rows();  // rows of one weight block of the merge launch
int kv4_row_group();    // rows of one head a group of lanes stores or loads
cudaError_t launch_kv4_append(const Kv4AppendArgs& a, int head_dim, bool bf16,
                              cudaStream_t stream);
cudaError_t launch_kv4_read(const Kv4ReadArgs& a, int head_dim, bool bf16, cudaStream_t stream);
cudaError_t launch_kv4_decode(const Kv4DecodeArgs& a, int head_dim, bool bf16, bool alibi,
                              cudaStream_t stream);

// ---------------------------------------------------------------------------
// Gathered key weights (mea_weights_sm100.cu).
// ---------------------------------------------------------------------------
constexpr int kWeightKeys = 128;  // keys per A operand

struct WeightArgs {
  const float* lse;          // [B, Hq, M]
  const float* w_in;         // [B, Hkv, N] or nullptr
  float* w_out;              // [B, Hkv, N]
  const int32_t* cache_len;  // [B] or nullptr: N - M
  const int32_t* q_lens;     // [B] or nullptr: M
  int* status;
  int B, M, N, Hq, Hkv, group;
  float scale_log2;
  int parts;                 // many rows only: CTAs (a cluster) that share a key block
  int few_chunk;             // few rows only: keys per CTA (a multiple of 64)
  long long q_s[3], k_s[3];  // few rows only: element strides (b, row, head)
};

struct WeightLaunch {
  CUtensorMap tmQ, tmK;
  const void *q, *k;
  WeightArgs args;
  int head_dim;
  bool bf16, causal, alibi;
  bool few;  // few query rows: K read once, mma.sync
};

cudaError_t launch_weights(const WeightLaunch& launch, cudaStream_t stream);

// ---------------------------------------------------------------------------
// Eviction (mea_evict_sm100.cu).
// ---------------------------------------------------------------------------
constexpr int kMaxPlanes = 5;

struct EvictPlane {
  const uint8_t* src;
  uint8_t* dst;
  long long src_s[3], dst_s[3];  // bytes: b, row, head
  int row_bytes;
  int piece_bytes;  // bytes of a row one block moves
  int access;       // bytes of one load: 16, 8 or 4
};

struct EvictArgs {
  EvictPlane planes[kMaxPlanes];
  int first_block[kMaxPlanes + 1];  // plane p: pieces first_block[p] .. first_block[p + 1] - 1
  int n_planes;
  int seg_rows;              // kept rows one move block takes (budget when anything is in place)
  bool in_place;             // some plane or the weights
  int parts;                 // CTAs (a cluster) that choose for one (sequence, kv head)
  const float* weights;      // [B, Hkv, cap]
  float* w_out;              // [B, Hkv, out_rows]
  const int32_t* lens;       // [B]
  int32_t* new_lens;         // [B]
  int32_t* kept;             // [B, Hkv, budget]
  int* status;
  int B, Hkv, cap, out_rows, budget, recent;
};

cudaError_t launch_evict(const EvictArgs& a, cudaStream_t stream);

}  // namespace mea
