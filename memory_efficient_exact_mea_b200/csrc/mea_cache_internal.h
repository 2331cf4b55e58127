// mea_cache_internal.h -- launch descriptions of the cache operators (4-bit cache, gathered
// key weights, eviction), shared between their C-ABI and kernel translation units.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "mea_internal.h"

namespace mea {

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

// Waits until the kernels before this one in the stream have finished and their
// writes can be read (a kernel launched with launch_after).
__device__ __forceinline__ void grid_dependency_wait() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

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
// x / d for x < 2^31: (hi32(x m) + x) >> s (division by an invariant through a
// multiplication; Granlund and Montgomery, 1994).
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

// Shared memory of the few-row kernel: per (row, query head) pair, in blocks of 8, what its
// column needs and its row of q.
struct FewColumn {
  float nl;     // -lse log2(e); -inf: takes no weight
  float slope;  // ALiBi, log2 units
  int pos;      // position of the row
  int last;     // last key it sees
};
inline int64_t few_row_bytes(int64_t pairs, int head_dim) {
  return (pairs + 7) / 8 * 8 * (static_cast<int64_t>(sizeof(FewColumn)) + 2 * head_dim);
}

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
