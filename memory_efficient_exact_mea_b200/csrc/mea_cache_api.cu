// mea_cache_api.cu -- C ABI of the cache operators declared in include/mea.h
// (4-bit cache, gathered key weights, eviction): host-side validation, launch
// plans and dispatch.  No allocation, no state.
#include <stdint.h>

#include <algorithm>

#include "mea.h"
#include "mea_cache_internal.h"

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

bool strides_ok(const int64_t s[3]) {
  for (int i = 0; i < 3; ++i)
    if (s[i] <= 0 || (s[i] & 7) != 0 || s[i] >= (int64_t(1) << 38)) return false;
  return true;
}

size_t align256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

// ---------------------------------------------------------------------------
// Where outputs may lie.  Blocks write rows in no order, so two rows of outputs in one
// place would leave whichever came last.
// ---------------------------------------------------------------------------
bool ranges_meet(const void* a, int64_t a_bytes, const void* b, int64_t b_bytes) {
  const uint8_t *p = static_cast<const uint8_t*>(a), *q = static_cast<const uint8_t*>(b);
  return p < q + b_bytes && q < p + a_bytes;
}

// Rows of `bytes` bytes at base + sum of i_k step_k: the axes longer than one, longest step
// first, and the bytes from the first row to the last one's end.
struct RowSet {
  const uint8_t* base = nullptr;
  int64_t n[3], step[3], bytes = 0, extent = 0;
  int axes = 0;
};

// False if rows meet one another (a step shorter than what it steps over) or lie too far
// apart for the arithmetic below.
bool row_set(RowSet* r, const void* base, const int64_t n[3], const int64_t step[3],
             int64_t bytes) {
  r->base = static_cast<const uint8_t*>(base);
  r->bytes = r->extent = bytes;
  for (int k = 0; k < 3; ++k) {
    if (n[k] <= 1) continue;
    int at = r->axes++;
    for (; at > 0 && r->step[at - 1] < step[k]; --at) {
      r->step[at] = r->step[at - 1];
      r->n[at] = r->n[at - 1];
    }
    r->step[at] = step[k];
    r->n[at] = n[k];
  }
  for (int k = r->axes - 1; k >= 0; --k) {
    if (r->step[k] < r->extent || r->n[k] - 1 > (int64_t(1) << 60) / r->step[k]) return false;
    r->extent += (r->n[k] - 1) * r->step[k];
    if (r->extent > int64_t(1) << 60) return false;
  }
  return true;
}

// Whether a row of b, which begins `apart` bytes after a's row with the same indices, meets
// a row of a in the axes from k on.  The rest of the axes spans less than one step, so only
// the two nearest steps can bring them together.
bool rows_meet(const RowSet& a, const RowSet& b, int64_t apart, int k) {
  if (k == a.axes) return apart < a.bytes && -apart < b.bytes;
  const int64_t i = apart >= 0 ? apart / a.step[k] : -((-apart + a.step[k] - 1) / a.step[k]);
  for (const int64_t j : {i, i + 1})
    if (j < a.n[k] && -j < a.n[k] && rows_meet(a, b, apart - j * a.step[k], k + 1)) return true;
  return false;
}

// True if rows of a and b meet, or if their steps differ and they lie within one another.
bool sets_meet(const RowSet& a, const RowSet& b) {
  if (!ranges_meet(a.base, a.extent, b.base, b.extent)) return false;
  if (a.axes != b.axes) return true;
  for (int k = 0; k < a.axes; ++k)
    if (a.n[k] != b.n[k] || a.step[k] != b.step[k]) return true;
  return rows_meet(a, b, b.base - a.base, 0);
}

constexpr int64_t kMaxRows = (int64_t(1) << 31) - 1;
constexpr int kMaxLen = 1 << 30;  // rows of one sequence: tile arithmetic stays in 32 bits

// False if the batch has 2^31 rows or more.
bool row_order(mea::RowOrder* o, int B, int M, int Hkv) {
  const int64_t tiles = (static_cast<int64_t>(M) + mea::kv4_row_group() - 1) / mea::kv4_row_group();
  if (static_cast<int64_t>(B) * Hkv > kMaxRows / (tiles * mea::kv4_row_group())) return false;
  o->total = static_cast<uint32_t>(tiles * B * Hkv);
  o->heads = mea::fast_div(static_cast<uint32_t>(Hkv));
  o->tiles = mea::fast_div(static_cast<uint32_t>(tiles));
  return true;
}

// mea_key_weights with fewer query rows than a tile has (128) goes to the kernel that reads
// K once with mma.sync, as long as its (row, query head) pairs fit the 48 KB that a block
// may use as it is: 176 pairs at K = 128, 336 at K = 64.  8 x 8 heads x 8192 keys, us here /
// with 128-row tiles, K = 128: one head a kv head 52 / 86 (64 rows), 73 / 87 (100), 85 / 81
// (128); two 85 / 108 (64), 101 / 107 (80); four 101 / 153 (40); eight 98 / 245 (20).
// K = 64: one head 48 / 68 (100); two 78 / 85 (100), 94 / 75 (128); four 114 / 126 (80);
// eight 112 / 212 (40).  (4 x 2 heads x 4096 keys, too few to fill the GPU: 9 / 9 with 64
// rows, 13 / 9 with 100.)  Past the limit a tile a head is taken however few its rows.
constexpr int kFewRows = 127, kFewBytes = 48 * 1024;

// Splits of one decode call.  A split is a whole number of 128-row steps (four
// warps of 32 rows); long enough that its partial state (K floats a head) and
// its start-up stay small beside the rows it reads, short enough that the grid
// fills the GPU's resident CTAs a few times over: at most 768 / 1024 / 1536 / 2048
// rows took 94.1 / 88.7 / 84.5 / 83.7 us for 64 sequences of up to 8192 rows and
// 91.2 / 85.1 / 82.2 / 81.6 us for four of up to 65521.
struct DecodePlan {
  int head_blocks, chunk, splits;
};

DecodePlan decode_plan(int B, int Hq, int Hkv, int max_len) {
  DecodePlan p{};
  p.head_blocks = (Hq / Hkv + 7) / 8;
  const int64_t units = static_cast<int64_t>(B) * Hkv * p.head_blocks;
  const int64_t want = std::max<int64_t>(1, 148 * 6 / std::max<int64_t>(1, units));
  int64_t chunk = (max_len + want - 1) / want;
  chunk = std::min<int64_t>(2048, std::max<int64_t>(128, (chunk + 127) / 128 * 128));
  chunk = std::max<int64_t>(chunk, ((max_len + int64_t(65534)) / 65535 + 127) / 128 * 128);
  p.chunk = static_cast<int>(chunk);
  p.splits = static_cast<int>((static_cast<int64_t>(max_len) + chunk - 1) / chunk);
  return p;
}

}  // namespace

extern "C" {

int mea_kv4_append(const void* k_new, const void* v_new, void* k_codes, void* k_params,
                   void* v_codes, void* v_params, const int32_t* cache_seqlens,
                   const int32_t* q_seqlens, int B, int M, int cache_rows, int Hkv, int K,
                   const int64_t kn_strides[3], const int64_t vn_strides[3], mea_dtype_t dtype,
                   cudaStream_t stream) {
  if (B < 0 || M < 0 || cache_rows < 0 || Hkv <= 0) return MEA_ERR_INVALID_ARG;
  if (dtype != MEA_F16 && dtype != MEA_BF16) return MEA_ERR_INVALID_ARG;
  if (!kn_strides || !vn_strides) return MEA_ERR_INVALID_ARG;
  if (B == 0 || M == 0) return MEA_OK;
  if (!k_new || !v_new || !k_codes || !k_params || !v_codes || !v_params || !cache_seqlens)
    return MEA_ERR_INVALID_ARG;
  if (K != 64 && K != 128) return MEA_ERR_UNSUPPORTED;
  if (M > kMaxLen || cache_rows > kMaxLen) return MEA_ERR_UNSUPPORTED;
  for (const void* p : {k_new, v_new, static_cast<const void*>(k_codes),
                        static_cast<const void*>(k_params), static_cast<const void*>(v_codes),
                        static_cast<const void*>(v_params)})
    if (!aligned16(p)) return MEA_ERR_UNSUPPORTED;
  if (!strides_ok(kn_strides) || !strides_ok(vn_strides)) return MEA_ERR_UNSUPPORTED;
  mea::Kv4AppendArgs a{};
  if (!row_order(&a.order, B, M, Hkv)) return MEA_ERR_UNSUPPORTED;
  const int64_t rows = static_cast<int64_t>(B) * Hkv * cache_rows;
  const void* planes[4] = {k_codes, v_codes, k_params, v_params};
  for (int i = 0; i < 4; ++i)
    for (int j = 0; j < i; ++j)
      if (ranges_meet(planes[i], rows * (i < 2 ? K / 2 : K / 16), planes[j],
                      rows * (j < 2 ? K / 2 : K / 16)))
        return MEA_ERR_INVALID_ARG;
  a.k_new = k_new;
  a.v_new = v_new;
  a.k_codes = k_codes;
  a.k_params = k_params;
  a.v_codes = v_codes;
  a.v_params = v_params;
  a.cache_len = cache_seqlens;
  a.q_lens = q_seqlens;
  a.status = mea::device_status_word();
  if (!a.status) return MEA_ERR_CUDA;
  for (int i = 0; i < 3; ++i) {
    a.kn_s[i] = kn_strides[i];
    a.vn_s[i] = vn_strides[i];
  }
  a.M = M;
  a.Hkv = Hkv;
  a.cap = cache_rows;
  return mea::launch_kv4_append(a, K, dtype == MEA_BF16, stream) == cudaSuccess ? MEA_OK
                                                                                : MEA_ERR_CUDA;
}

int mea_kv4_read(const void* k_codes, const void* k_params, const void* v_codes,
                 const void* v_params, const int32_t* rows, const int32_t* first_rows,
                 void* k_out, void* v_out, int B, int cache_rows, int out_rows, int Hkv, int K,
                 const int64_t ko_strides[3], const int64_t vo_strides[3], mea_dtype_t dtype,
                 cudaStream_t stream) {
  if (B < 0 || out_rows < 0 || cache_rows < 0 || Hkv <= 0) return MEA_ERR_INVALID_ARG;
  if (dtype != MEA_F16 && dtype != MEA_BF16) return MEA_ERR_INVALID_ARG;
  if (!ko_strides || !vo_strides) return MEA_ERR_INVALID_ARG;
  if (B == 0 || out_rows == 0) return MEA_OK;
  if (!k_codes || !k_params || !v_codes || !v_params || !rows || !k_out || !v_out)
    return MEA_ERR_INVALID_ARG;
  if (K != 64 && K != 128) return MEA_ERR_UNSUPPORTED;
  if (out_rows > kMaxLen || cache_rows > kMaxLen) return MEA_ERR_UNSUPPORTED;
  for (const void* p : {k_codes, k_params, v_codes, v_params, static_cast<const void*>(k_out),
                        static_cast<const void*>(v_out)})
    if (!aligned16(p)) return MEA_ERR_UNSUPPORTED;
  if (!strides_ok(ko_strides) || !strides_ok(vo_strides)) return MEA_ERR_UNSUPPORTED;
  mea::Kv4ReadArgs a{};
  if (!row_order(&a.order, B, out_rows, Hkv)) return MEA_ERR_UNSUPPORTED;
  const int64_t n[3] = {B, out_rows, Hkv};
  const int64_t ko[3] = {2 * ko_strides[0], 2 * ko_strides[1], 2 * ko_strides[2]};
  const int64_t vo[3] = {2 * vo_strides[0], 2 * vo_strides[1], 2 * vo_strides[2]};
  RowSet kr, vr;
  if (!row_set(&kr, k_out, n, ko, 2 * K) || !row_set(&vr, v_out, n, vo, 2 * K) ||
      sets_meet(kr, vr))
    return MEA_ERR_INVALID_ARG;
  a.k_codes = k_codes;
  a.k_params = k_params;
  a.v_codes = v_codes;
  a.v_params = v_params;
  a.k_out = k_out;
  a.v_out = v_out;
  a.rows = rows;
  a.first = first_rows;
  a.status = mea::device_status_word();
  if (!a.status) return MEA_ERR_CUDA;
  for (int i = 0; i < 3; ++i) {
    a.ko_s[i] = ko_strides[i];
    a.vo_s[i] = vo_strides[i];
  }
  a.out_rows = out_rows;
  a.Hkv = Hkv;
  a.cap = cache_rows;
  return mea::launch_kv4_read(a, K, dtype == MEA_BF16, stream) == cudaSuccess ? MEA_OK
                                                                              : MEA_ERR_CUDA;
}

// Scores of one head: rows rounded up to whole 16-byte loads.
static size_t score_stride(int max_len) { return (static_cast<size_t>(max_len) + 3) & ~size_t(3); }

// Workspace: partial outputs, partial log-sum-exps (both only with several
// splits or weights), scores (weights only), each 256-byte aligned.
static size_t kv4_workspace(int B, int Hq, int Hkv, int K, int max_len, bool weights,
                            size_t* lse_at, size_t* score_at) {
  const DecodePlan p = decode_plan(B, Hq, Hkv, max_len);
  const size_t rows = static_cast<size_t>(B) * Hq;
  size_t at = 0;
  if (p.splits > 1) at += align256(rows * p.splits * K * sizeof(float));
  *lse_at = at;
  if (p.splits > 1 || weights) at += align256(rows * p.splits * sizeof(float));
  *score_at = at;
  if (weights) at += align256(rows * score_stride(max_len) * sizeof(float));
  return at;
}

size_t mea_decode_kv4_workspace_size(int B, int Hq, int Hkv, int K, int max_kv_len, int weights) {
  if (B < 0 || Hq <= 0 || Hkv <= 0 || Hq % Hkv != 0 || K <= 0 || max_kv_len < 0) return 0;
  size_t l, s;
  return kv4_workspace(B, Hq, Hkv, K, max_kv_len, weights != 0, &l, &s);
}

int mea_decode_kv4(const void* q, const void* k_codes, const void* k_params, const void* v_codes,
                   const void* v_params, const int32_t* kv_seqlens, void* out, float* lse,
                   const float* weights_in, float* weights_out, int B, int Hq, int Hkv, int K,
                   int cache_rows, int max_kv_len, mea_dtype_t dtype, int alibi, float scale,
                   void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  if (B < 0 || Hq <= 0 || Hkv <= 0 || Hq % Hkv != 0 || cache_rows < 0 || max_kv_len < 0)
    return MEA_ERR_INVALID_ARG;
  if (dtype != MEA_F16 && dtype != MEA_BF16) return MEA_ERR_INVALID_ARG;
  if (!(scale == scale)) return MEA_ERR_INVALID_ARG;
  if (weights_in && !weights_out) return MEA_ERR_INVALID_ARG;
  if (B == 0) return MEA_OK;
  if (!q || !out || !kv_seqlens) return MEA_ERR_INVALID_ARG;
  if (cache_rows > 0 && (!k_codes || !k_params || !v_codes || !v_params))
    return MEA_ERR_INVALID_ARG;
  if (K != 64 && K != 128) return MEA_ERR_UNSUPPORTED;
  if (cache_rows > kMaxLen || max_kv_len > kMaxLen) return MEA_ERR_UNSUPPORTED;
  for (const void* p : {q, k_codes, k_params, v_codes, v_params, static_cast<const void*>(out)})
    if (!aligned16(p)) return MEA_ERR_UNSUPPORTED;
  size_t lse_at, score_at;
  const size_t need =
      kv4_workspace(B, Hq, Hkv, K, max_kv_len, weights_out != nullptr, &lse_at, &score_at);
  if (need > 0 && (!workspace || workspace_bytes < need ||
                   (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0))
    return MEA_ERR_WORKSPACE;
  const int64_t weight_bytes = static_cast<int64_t>(B) * Hkv * cache_rows * 4;
  if (weights_in && weights_in != weights_out &&
      ranges_meet(weights_in, weight_bytes, weights_out, weight_bytes))
    return MEA_ERR_INVALID_ARG;
  mea::Kv4DecodeArgs a{};
  const DecodePlan p = decode_plan(B, Hq, Hkv, max_kv_len);
  if (static_cast<int64_t>(Hkv) * p.head_blocks > 65535 || B > 65535) return MEA_ERR_UNSUPPORTED;
  a.weight_blocks =
      weights_out ? (cache_rows + mea::kv4_weight_rows() - 1) / mea::kv4_weight_rows() : 0;
  a.merge_blocks = static_cast<int>((static_cast<int64_t>(B) * Hq + 7) / 8);
  if (static_cast<int64_t>(B) * Hkv * a.weight_blocks + a.merge_blocks > kMaxRows ||
      static_cast<int64_t>(B) * Hq > kMaxRows)
    return MEA_ERR_UNSUPPORTED;
  a.status = mea::device_status_word();
  if (!a.status) return MEA_ERR_CUDA;
  a.q = q;
  a.k_codes = k_codes;
  a.k_params = k_params;
  a.v_codes = v_codes;
  a.v_params = v_params;
  a.kv_lens = kv_seqlens;
  a.out = out;
  a.lse = lse;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  a.part_o = p.splits > 1 ? static_cast<float*>(workspace) : nullptr;
  a.part_lse = p.splits > 1 || weights_out ? reinterpret_cast<float*>(ws + lse_at) : nullptr;
  a.scores = weights_out ? reinterpret_cast<float*>(ws + score_at) : nullptr;
  a.score_stride = static_cast<long long>(score_stride(max_kv_len));
  a.w_in = weights_in;
  a.w_out = weights_out;
  a.B = B;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.group = Hq / Hkv;
  a.cap = cache_rows;
  a.max_len = std::min(max_kv_len, cache_rows);
  a.chunk = p.chunk;
  a.max_splits = p.splits;
  a.head_blocks = p.head_blocks;
  // one split writes the result itself: the merge launch has only weights to gather
  if (p.splits == 1) a.merge_blocks = 0;
  a.scale_log2 = scale * 1.4426950408889634f;
  return mea::launch_kv4_decode(a, K, dtype == MEA_BF16, alibi != 0, stream) == cudaSuccess
             ? MEA_OK
             : MEA_ERR_CUDA;
}

int mea_key_weights(const void* q, const void* k, const float* lse, const int32_t* cache_seqlens,
                    const int32_t* q_seqlens, const float* weights_in, float* weights_out, int B,
                    int M, int N, int Hq, int Hkv, int K, const int64_t q_strides[3],
                    const int64_t k_strides[3], mea_dtype_t dtype, int causal, int alibi,
                    float scale, cudaStream_t stream) {
  if (B < 0 || M < 0 || N < 0 || Hq <= 0 || Hkv <= 0 || Hq % Hkv != 0) return MEA_ERR_INVALID_ARG;
  if (dtype != MEA_F16 && dtype != MEA_BF16) return MEA_ERR_INVALID_ARG;
  if (causal != 0 && causal != 1) return MEA_ERR_INVALID_ARG;
  if (!q_strides || !k_strides) return MEA_ERR_INVALID_ARG;
  if (!(scale == scale)) return MEA_ERR_INVALID_ARG;
  if (q_seqlens && !cache_seqlens) return MEA_ERR_INVALID_ARG;
  if (B == 0 || N == 0) return MEA_OK;
  if (M < 1) return MEA_ERR_INVALID_ARG;
  if (!q || !k || !lse || !weights_out) return MEA_ERR_INVALID_ARG;
  if (K != 64 && K != 128) return MEA_ERR_UNSUPPORTED;
  if (scale < 0.f || M > kMaxLen || N > kMaxLen) return MEA_ERR_UNSUPPORTED;
  if (!aligned16(q) || !aligned16(k)) return MEA_ERR_UNSUPPORTED;
  if (!strides_ok(q_strides) || !strides_ok(k_strides)) return MEA_ERR_UNSUPPORTED;
  const int64_t blocks = (static_cast<int64_t>(N) + mea::kWeightKeys - 1) / mea::kWeightKeys;
  if (static_cast<int64_t>(B) * Hkv > kMaxRows / blocks) return MEA_ERR_UNSUPPORTED;
  const int64_t weight_bytes = static_cast<int64_t>(B) * Hkv * N * 4;
  if (weights_in && weights_in != weights_out &&
      ranges_meet(weights_in, weight_bytes, weights_out, weight_bytes))
    return MEA_ERR_INVALID_ARG;
  mea::WeightLaunch L{};
  mea::WeightArgs& a = L.args;
  a.status = mea::device_status_word();
  if (!a.status) return MEA_ERR_CUDA;
  a.group = Hq / Hkv;
  // Few (row, head) pairs to a key: the kernel that is bound by reading K.
  L.few = M <= kFewRows && mea::few_row_bytes(static_cast<int64_t>(M) * a.group, K) <= kFewBytes &&
          Hkv <= 65535 && B <= 65535;
  const bool bf16 = dtype == MEA_BF16;
  if (L.few) {
    const int64_t units = static_cast<int64_t>(B) * Hkv;
    const int64_t chunk = (units * N / (148 * 8) + 63) / 64 * 64;
    a.few_chunk = static_cast<int>(std::min<int64_t>(512, std::max<int64_t>(64, chunk)));
    for (int i = 0; i < 3; ++i) {
      a.q_s[i] = q_strides[i];
      a.k_s[i] = k_strides[i];
    }
    L.q = q;
    L.k = k;
  } else if (!mea::encode_rows(&L.tmQ, q, bf16, B, M, Hq, K, q_strides, 128) ||
             !mea::encode_rows(&L.tmK, k, bf16, B, N, Hkv, K, k_strides, mea::kWeightKeys)) {
    return MEA_ERR_CUDA;
  }
  a.lse = lse;
  a.w_in = weights_in;
  a.w_out = weights_out;
  a.cache_len = cache_seqlens;
  a.q_lens = q_seqlens;
  a.B = B;
  a.M = M;
  a.N = N;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.scale_log2 = scale * 1.4426950408889634f;
  L.head_dim = K;
  L.bf16 = bf16;
  L.causal = causal != 0;
  L.alibi = alibi != 0;
  return mea::launch_weights(L, stream) == cudaSuccess ? MEA_OK : MEA_ERR_CUDA;
}

int mea_cache_evict(const mea_plane_t* planes, int n_planes, const float* weights,
                    float* weights_out, const int32_t* cache_seqlens, int32_t* new_seqlens,
                    int32_t* kept, int B, int Hkv, int cache_rows, int out_rows, int budget,
                    int recent, cudaStream_t stream) {
  if (B < 0 || Hkv <= 0 || cache_rows < 0 || out_rows < 0) return MEA_ERR_INVALID_ARG;
  if (n_planes < 1 || n_planes > 4 || !planes) return MEA_ERR_INVALID_ARG;
  if (budget < 1 || budget > out_rows || recent < 0 || recent > budget) return MEA_ERR_INVALID_ARG;
  if (B == 0) return MEA_OK;
  if (!cache_seqlens || !new_seqlens || cache_seqlens == new_seqlens || !kept || !weights_out ||
      !weights || cache_rows < 1)
    return MEA_ERR_INVALID_ARG;
  if (static_cast<int64_t>(B) * Hkv > 65535 || cache_rows > kMaxLen || out_rows > kMaxLen)
    return MEA_ERR_UNSUPPORTED;

  mea_plane_t all[mea::kMaxPlanes];
  for (int p = 0; p < n_planes; ++p) all[p] = planes[p];
  mea_plane_t& w = all[n_planes];
  w.src = weights;
  w.dst = weights_out;
  w.row_bytes = 4;
  const int64_t rows[2] = {cache_rows, out_rows};
  for (int side = 0; side < 2; ++side) {
    int64_t* st = side == 0 ? w.src_strides : w.dst_strides;
    st[0] = rows[side] * Hkv * 4;
    st[1] = 4;
    st[2] = rows[side] * 4;
  }
  const int total = n_planes + 1;
  mea::EvictArgs a{};
  bool in_place = false;
  for (int p = 0; p < total; ++p) {
    const mea_plane_t& x = all[p];
    if (!x.src || !x.dst || x.row_bytes < 4) return MEA_ERR_INVALID_ARG;
    int64_t bits = x.row_bytes | static_cast<int64_t>(reinterpret_cast<uintptr_t>(x.src) & 15u) |
                   static_cast<int64_t>(reinterpret_cast<uintptr_t>(x.dst) & 15u);
    for (int i = 0; i < 3; ++i) {
      if (x.src_strides[i] < 0 || x.dst_strides[i] < 0) return MEA_ERR_INVALID_ARG;
      if ((x.src_strides[i] | x.dst_strides[i]) >= (int64_t(1) << 40)) return MEA_ERR_UNSUPPORTED;
      bits |= x.src_strides[i] | x.dst_strides[i];
    }
    if (bits & 3) return MEA_ERR_UNSUPPORTED;
    mea::EvictPlane& e = a.planes[p];
    e.access = (bits & 15) == 0 ? 16 : (bits & 7) == 0 ? 8 : 4;
    e.src = static_cast<const uint8_t*>(x.src);
    e.dst = static_cast<uint8_t*>(x.dst);
    e.row_bytes = x.row_bytes;
    for (int i = 0; i < 3; ++i) {
      e.src_s[i] = x.src_strides[i];
      e.dst_s[i] = x.dst_strides[i];
    }
    if (x.src == x.dst) {
      if (out_rows != cache_rows) return MEA_ERR_INVALID_ARG;
      for (int i = 0; i < 3; ++i)
        if (x.src_strides[i] != x.dst_strides[i]) return MEA_ERR_INVALID_ARG;
      in_place = true;
    }
  }
  // Destinations: the planes', each row in a place of its own (the rows of several planes
  // of one array may interleave), away from every source but, in place, their own and
  // those cut in place with it.
  RowSet dst[mea::kMaxPlanes];
  const uint8_t *s0[mea::kMaxPlanes], *s1[mea::kMaxPlanes];  // what the sources span
  const int64_t dst_n[3] = {B, out_rows, Hkv}, src_n[3] = {B, cache_rows, Hkv};
  for (int p = 0; p < total; ++p) {
    if (!row_set(&dst[p], all[p].dst, dst_n, all[p].dst_strides, all[p].row_bytes))
      return MEA_ERR_INVALID_ARG;
    int64_t span = all[p].row_bytes;
    for (int i = 0; i < 3; ++i) {
      const int64_t step = all[p].src_strides[i];
      if (step > 0 && src_n[i] - 1 > (int64_t(1) << 60) / step) return MEA_ERR_INVALID_ARG;
      span += (src_n[i] - 1) * step;
    }
    s0[p] = a.planes[p].src;
    s1[p] = s0[p] + span;
  }
  for (int d = 0; d < total; ++d)
    for (int s = 0; s < total; ++s) {
      if (d < s && sets_meet(dst[d], dst[s])) return MEA_ERR_INVALID_ARG;
      const bool same_array = all[d].src == all[d].dst && all[s].src == all[s].dst;
      if (!same_array && ranges_meet(dst[d].base, dst[d].extent, s0[s], s1[s] - s0[s]))
        return MEA_ERR_INVALID_ARG;
    }
  // kept and new_seqlens: away from all of these, and from the lengths
  const int64_t kept_bytes = static_cast<int64_t>(B) * Hkv * budget * 4, len_bytes = int64_t(4) * B;
  if (ranges_meet(kept, kept_bytes, new_seqlens, len_bytes) ||
      ranges_meet(kept, kept_bytes, cache_seqlens, len_bytes) ||
      ranges_meet(new_seqlens, len_bytes, cache_seqlens, len_bytes))
    return MEA_ERR_INVALID_ARG;
  for (int p = 0; p < total; ++p) {
    const int64_t span = s1[p] - s0[p];
    if (ranges_meet(kept, kept_bytes, dst[p].base, dst[p].extent) ||
        ranges_meet(kept, kept_bytes, s0[p], span) ||
        ranges_meet(new_seqlens, len_bytes, dst[p].base, dst[p].extent) ||
        ranges_meet(new_seqlens, len_bytes, s0[p], span) ||
        ranges_meet(cache_seqlens, len_bytes, dst[p].base, dst[p].extent))
      return MEA_ERR_INVALID_ARG;
  }

  // Blocks: (column piece of a plane) x (sequence, kv head) x row segment.  Into
  // other memory the rows are shared out; in place a piece's rows are one block's,
  // so narrow pieces make the parallelism when there are few (sequence, head)s.
  const int64_t bh = static_cast<int64_t>(B) * Hkv;
  a.in_place = in_place;
  // 32 KB of the widest plane a block, at least 128 rows: 8 x 8192 rows of 256 bytes
  // took 29 us with 128 rows and 32 with 64, rows of 64 bytes 36 us with 128, 27 with 256.
  int widest = 4;
  for (int p = 0; p < n_planes; ++p) widest = std::max(widest, planes[p].row_bytes);
  a.seg_rows = in_place ? budget
                        : std::max({128, 32768 / widest, (budget + 65534) / 65535});
  const int64_t segs = (budget + a.seg_rows - 1) / a.seg_rows;
  int pieces = 0;
  for (int p = 0; p < total; ++p) {
    mea::EvictPlane& e = a.planes[p];
    e.piece_bytes = e.row_bytes;
    // at most 256 lanes of `access` bytes; halved further while the grid is small
    while (e.piece_bytes % (2 * e.access) == 0 &&
           (e.piece_bytes / e.access > 256 ||
            (e.piece_bytes > 32 && bh * segs * n_planes * (e.row_bytes / e.piece_bytes) < 148 * 4)))
      e.piece_bytes /= 2;
    if (e.piece_bytes / e.access > 256) return MEA_ERR_UNSUPPORTED;
    a.first_block[p] = pieces;
    pieces += e.row_bytes / e.piece_bytes;
  }
  a.first_block[total] = pieces;
  a.n_planes = total;
  a.weights = weights;
  a.w_out = weights_out;
  a.lens = cache_seqlens;
  a.new_lens = new_seqlens;
  a.kept = kept;
  a.status = mea::device_status_word();
  if (!a.status) return MEA_ERR_CUDA;
  a.B = B;
  a.Hkv = Hkv;
  a.cap = cache_rows;
  a.out_rows = out_rows;
  a.budget = budget;
  a.recent = recent;
  return mea::launch_evict(a, stream) == cudaSuccess ? MEA_OK : MEA_ERR_CUDA;
}

}  // extern "C"
