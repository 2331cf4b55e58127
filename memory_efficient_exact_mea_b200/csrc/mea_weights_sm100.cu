// mea_weights_sm100.cu -- the attention weight each cached key has gathered:
//     w_j += sum over the query heads of j's group and the rows i that see j of
//            exp(scale q_i.k_j + b_ij - lse_i)
// (the weights of "FlashAttention (2022)", section "Il trucco della softmax che
// non ha bisogno di vedere tutto", recomputed from the log-sum-exp as a backward
// pass does, and summed over the queries instead of multiplied with V).
//
// One CTA holds 128 or 256 keys of one kv head as A operands in shared memory and
// walks the (query head, query block) pairs that can see them: S^T = K Q_i^T in
// tensor memory has a key per lane, so the sum over queries is a sum along each
// thread's own row -- no reduction across lanes, no atomics, the same order every
// time.  For each 128 keys, two groups of four warps take alternate tiles (one TMEM
// buffer each), so one group's exponentials overlap the other's MMA and TMEM read.
// Bound by the exponential unit (16 a clock per SM; 74 % busy at K = 128, 71 % at 64).
//
// A few query rows (a decode step, a short chunk) go to weights_few_kernel: the same
// sum with mma.sync straight from global memory, bound by reading K once.
#include <cooperative_groups.h>
#include <math.h>

#include <type_traits>

#include "mea_cache_internal.h"
#include "sm100.cuh"

namespace mea {
namespace {

namespace cg = cooperative_groups;

constexpr int kMaxWeightParts = 8;  // CTAs of a cluster that share a key block
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float neg_inf() { return __int_as_float(0xff800000); }

// acc + 2^x for a pair, on the FMA pipe: 2^x = 2^n 2^f with n the integer next to x
// (added into the low mantissa bits of 1.5 2^23) and 2^f, |f| <= 1/2, by a polynomial
// of degree 5 fitted here for the least relative error (7.5e-8; 2.2e-7 with fp32's
// roundings).  x < -126.5 gives 0, x > 127.5 infinity (2^n is then no number; exp2 itself
// ends half a step later), a NaN stays a NaN.
__device__ __forceinline__ float clamp_exponent(float x) {
  float y;
  asm("max.NaN.f32 %0, %1, 0fC2FE0000;" : "=f"(y) : "f"(x));  // -127
  asm("min.NaN.f32 %0, %1, 0f43000000;" : "=f"(y) : "f"(y));  // 128
  return y;
}
__device__ __forceinline__ f2 exp2_add(f2 x, f2 acc) {
  constexpr float kRound = 12582912.f;  // 1.5 * 2^23
  x = {clamp_exponent(x.x), clamp_exponent(x.y)};
  const f2 r = add2(x, {kRound, kRound});
  const f2 n = add2(r, {-kRound, -kRound});
  const f2 f = fma2(n, {-1.f, -1.f}, x);
  f2 p = fma2(f, {0.0013276470116741828f, 0.0013276470116741828f},
              {0.009675541319485738f, 0.009675541319485738f});
  p = fma2(p, f, {0.05550713279300344f, 0.05550713279300344f});
  p = fma2(p, f, {0.24022119724212534f, 0.24022119724212534f});
  p = fma2(p, f, {0.6931469670612077f, 0.6931469670612077f});
  p = fma2(p, f, {1.0000000716545692f, 1.0000000716545692f});
  const f2 two_n = {__uint_as_float((__float_as_uint(r.x) << 23) + 0x3F800000u),
                    __uint_as_float((__float_as_uint(r.y) << 23) + 0x3F800000u)};
  return fma2(p, two_n, acc);
}

// Which of a chunk's 16 pairs take the polynomial, spread evenly: 0 / 2 / 3 / 4 / 5 of 16
// measured 350 / 330 / 325 / 328 / 334 us (causal 4 x 4096) and 168 / 157 / 153 / 153 /
// 153 us (two-sided 8 x 2048).
constexpr int kPolyOf16 = 3;
__device__ __forceinline__ constexpr bool on_fma_pipe(int pair) {
  return (pair * kPolyOf16) % 16 < kPolyOf16;
}

// A query tile is used against kHalves x 128 keys, 2 halves at K = 128 (one
// CTA per SM), 1 at K = 64 (two CTAs): 1 byte of Q read from L2 per score either way.
// Query tiles are released as soon as their MMAs have read them, so the ring runs
// four or five tiles ahead; lse has a ring of its own that lives until the tile's
// sums are done.
template <int D>
struct WCfg {
  static constexpr int NQ = 128;  // query rows per tile
  static constexpr int kHalves = D == 128 ? 2 : 1;
  static constexpr int kKeys = kHalves * kWeightKeys;
  static constexpr int kParity = 2;  // consumer groups per half
  static constexpr int kGroups = kHalves * kParity;  // of four warps
  static constexpr int kWarps = 4 * kGroups;
  static constexpr int kThreads = (kWarps + 2) * 32;
  static constexpr int kMmaWarp = kWarps, kLoadWarp = kWarps + 1;
  static constexpr int kStages = D == 128 ? 4 : 5;
  static constexpr int kLseSlots = 8;
  static constexpr int kCtas = kHalves == 2 ? 1 : 2;  // per SM
  static constexpr int kChunks = D / 64;
  static constexpr int kKChunk = kWeightKeys * 128;
  static constexpr int kQChunk = NQ * 128;
  static constexpr int kKTile = kChunks * kKChunk;  // one half
  static constexpr int kQTile = kChunks * kQChunk;
  static constexpr int kQ = kHalves * kKTile;
  static constexpr int kLse = kQ + kStages * kQTile;      // [slot][NQ] -lse * log2(e)
  static constexpr int kSlope = kLse + kLseSlots * NQ * 4;  // [slot] the tile's ALiBi slope
  static constexpr int kOpen = kSlope + kLseSlots * 4;     // [slot] every row takes weight
  static constexpr int kSum = kOpen + kLseSlots * 4;       // [kKeys]
  static constexpr int kPart = kSum + kKeys * 4;           // [kMaxWeightParts][kKeys]
  static constexpr int kBar = kPart + kMaxWeightParts * kKeys * 4;
  static constexpr int kNumBars = 2 + 2 * kStages + 2 * kLseSlots + 4 * kHalves;
  static constexpr int kTmemSlot = kBar + kNumBars * 8;
  static constexpr int kAbort = kTmemSlot + 4;
  static constexpr int kBytes = kAbort + 4 + 1024;
  static_assert(kCtas * (kBytes + 1024) <= 228 * 1024, "shared memory");
  static constexpr uint32_t kTmemCols = 2 * kHalves * NQ;  // two buffers a half
};

template <int D, bool BF16, bool CAUSAL, bool ALIBI>
__global__ void __launch_bounds__(WCfg<D>::kThreads, WCfg<D>::kCtas)
    weights_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                   const WeightArgs a) {
  using C = WCfg<D>;
  constexpr int NQ = C::NQ;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint64_t* k_full = reinterpret_cast<uint64_t*>(smem + C::kBar);
  uint64_t* q_full = k_full + 1;
  uint64_t* q_empty = q_full + C::kStages;      // the tile's MMAs are done
  uint64_t* l_full = q_empty + C::kStages;      // [kLseSlots] lse of a tile is staged
  uint64_t* l_empty = l_full + C::kLseSlots;    // its sums are done
  uint64_t* s_full = l_empty + C::kLseSlots;    // [half][2] scores of a tile are in TMEM
  uint64_t* s_free = s_full + 2 * C::kHalves;   // [half][2] read out of TMEM
  uint64_t* mma_done = s_free + 2 * C::kHalves;
  float* s_lse = reinterpret_cast<float*>(smem + C::kLse);
  float* s_slope = reinterpret_cast<float*>(smem + C::kSlope);
  int* s_open = reinterpret_cast<int*>(smem + C::kOpen);
  float* s_sum = reinterpret_cast<float*>(smem + C::kSum);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kTmemSlot);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kAbort);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // The key block varies slowest: under a causal mask the first blocks, seen by
  // the most query rows, start first.  The a.parts CTAs of a cluster share a block's
  // (head, row block) pairs.
  const int per = a.Hkv * a.B;
  const int unit = blockIdx.x / a.parts, part = blockIdx.x - unit * a.parts;
  const int nb = unit / per;
  const int bh = unit - nb * per;
  const int b = bh / a.Hkv, kvh = bh - b * a.Hkv;
  const int n0 = nb * C::kKeys;

  const int m = a.q_lens ? a.q_lens[b] : a.M;
  const int past = a.cache_len ? a.cache_len[b] : a.N - a.M;
  const long long wrow = static_cast<long long>(bh) * a.N;
  if (m < 0 || m > a.M || (a.cache_len && past < 0) || past > a.N - m) {
    if (nb == 0 && kvh == 0 && part == 0 && threadIdx.x == 0)
      record_error(a.status, kErrInvalidArg);
    return;
  }
  // without cache_len the N keys are all there, whatever m is
  const int n = a.cache_len ? past + m : a.N;
  // (head, row block) pairs; a causal key block starts at the first row that sees it
  int m_first = 0;
  if constexpr (CAUSAL) m_first = max(0, n0 - past) / NQ * NQ;
  const int mblocks = m > m_first ? (m - m_first + NQ - 1) / NQ : 0;
  const int total = n0 < n ? a.group * mblocks : 0;
  if (total == 0) {  // no query sees these keys (the same for the whole cluster)
    if (part == 0 && threadIdx.x < C::kKeys && n0 + static_cast<int>(threadIdx.x) < a.N) {
      const int j = n0 + threadIdx.x;
      a.w_out[wrow + j] = (j < n && a.w_in) ? a.w_in[wrow + j] : 0.f;
    }
    return;
  }

  const int s_first = static_cast<int>(static_cast<long long>(total) * part / a.parts);
  const int steps = static_cast<int>(static_cast<long long>(total) * (part + 1) / a.parts) - s_first;

  if (threadIdx.x == 0) {
    mbar_init(k_full, 1);
    mbar_init(mma_done, 1);
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(&q_full[s], 1);
      mbar_init(&q_empty[s], 1);
    }
    for (int s = 0; s < C::kLseSlots; ++s) {
      mbar_init(&l_full[s], 1);
      mbar_init(&l_empty[s], 4 * C::kHalves);  // the warps that took the tile
    }
    for (int s = 0; s < 2 * C::kHalves; ++s) {
      mbar_init(&s_full[s], 1);
      mbar_init(&s_free[s], 4);
    }
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == C::kMmaWarp) {
    tmem_alloc(tmem_slot, C::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (a.parts > 1) cg::this_cluster().sync();  // every CTA runs before any reaches into another
  const uint32_t tmem_base = *tmem_slot;

  float sum = 0.f;
  if (warp == C::kLoadWarp) {
    // ===================== loads =============================================
    if (lane == 0) {
      mbar_arrive_expect_tx(k_full, C::kHalves * C::kKTile);
      for (int c = 0; c < C::kHalves * C::kChunks; ++c)
        tma_load_4d(smem + c * C::kKChunk, &tmK, k_full, c % C::kChunks * 64, kvh,
                    n0 + c / C::kChunks * kWeightKeys, b);
    }
    int issued = 0;
    for (int s = 0; s < steps; ++s) {
      const int g = (s_first + s) / mblocks, m0 = m_first + (s_first + s - g * mblocks) * NQ;
      const int slot = s % C::kStages, ls = s % C::kLseSlots;
      const int h = kvh * a.group + g;
      float l2[NQ / 32];
#pragma unroll
      for (int u = 0; u < NQ / 32; ++u) {  // in flight during the waits
        const int i = m0 + u * 32 + lane;
        l2[u] = i < m ? a.lse[(static_cast<long long>(b) * a.Hq + h) * a.M + i] : neg_inf();
      }
      if (!mbar_wait_warp(&q_empty[slot], ((s / C::kStages) & 1) ^ 1, abort_flag, a.status)) break;
      if (lane == 0) {
        mbar_arrive_expect_tx(&q_full[slot], C::kQTile);
        for (int c = 0; c < C::kChunks; ++c)
          tma_load_4d(smem + C::kQ + slot * C::kQTile + c * C::kQChunk, &tmQ, &q_full[slot],
                      c * 64, h, m0, b);
      }
      ++issued;
      if (!mbar_wait_warp(&l_empty[ls], ((s / C::kLseSlots) & 1) ^ 1, abort_flag, a.status)) break;
      bool open = true;
#pragma unroll
      for (int u = 0; u < NQ / 32; ++u) {  // -inf: the row takes no weight
        const float nl = l2[u] == neg_inf() ? l2[u] : -l2[u] * kLog2e;
        s_lse[ls * NQ + u * 32 + lane] = nl;
        open = open && nl != neg_inf();
      }
      open = __all_sync(0xffffffffu, open);
      if (lane == 0) s_open[ls] = open;
      if (ALIBI && lane == 0)
        s_slope[ls] = exp2f(-8.0f * static_cast<float>(h + 1) / a.Hq) * kLog2e;
      mbar_arrive_warp(&l_full[ls]);
    }
    if (lane == 0) {  // no copy may be in flight when the CTA ends
      mbar_wait_drain(k_full, 0, a.status);
      for (int j = max(0, issued - C::kStages); j < issued; ++j)
        mbar_wait_drain(&q_full[j % C::kStages], (j / C::kStages) & 1, a.status);
    }
  } else if (warp == C::kMmaWarp) {
    // ===================== S^T = K Q^T =======================================
    constexpr uint32_t idesc = idesc_f16(BF16, kWeightKeys, NQ, false);
    const uint32_t sk = smem_u32(smem), sq = smem_u32(smem + C::kQ);
    bool ok = mbar_wait_warp(k_full, 0, abort_flag, a.status);
    for (int s = 0; s < steps && ok; ++s) {
      const int slot = s % C::kStages, buf = s & 1;
      ok = mbar_wait_warp(&q_full[slot], (s / C::kStages) & 1, abort_flag, a.status);
      for (int h = 0; h < C::kHalves && ok; ++h) {
        ok = mbar_wait_warp(&s_free[2 * h + buf], ((s >> 1) & 1) ^ 1, abort_flag, a.status);
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int c = 0; c < C::kChunks; ++c)
#pragma unroll
          for (int k = 0; k < 4; ++k)
            umma_ss_warp(tmem_base + (2 * h + buf) * NQ,
                         sdesc_sw128(sk + h * C::kKTile + c * C::kKChunk + k * 32, 16, 1024),
                         sdesc_sw128(sq + slot * C::kQTile + c * C::kQChunk + k * 32, 16, 1024),
                         idesc, c + k > 0);
        umma_commit_warp(&s_full[2 * h + buf]);
      }
      if (!ok) break;
      umma_commit_warp(&q_empty[slot]);
    }
    // every MMA has completed before the tensor memory is given back
    umma_commit_warp(mma_done);
    mbar_wait_drain(mma_done, 0, a.status);
  } else {
    // ===================== exponentials and sums =============================
    const int grp = warp >> 2, half = grp / C::kParity;
    const int key = n0 + half * kWeightKeys + (warp & 3) * 32 + lane;
    const uint32_t lane_addr = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const f2 sc2 = {a.scale_log2, a.scale_log2};
    for (int s = grp % C::kParity; s < steps; s += C::kParity) {
      const int g = (s_first + s) / mblocks, m0 = m_first + (s_first + s - g * mblocks) * NQ;
      const int ls = s % C::kLseSlots, buf = 2 * half + (s & 1);
      // row i = m0 + row(c) sees this key iff i >= key - past
      const int first = CAUSAL ? max(0, key - past - m0) : 0;
      const bool seen = !CAUSAL || n0 + (half + 1) * kWeightKeys - 1 - past <= m0;
      if (!mbar_wait_warp(&l_full[ls], (s / C::kLseSlots) & 1, abort_flag, a.status) ||
          !mbar_wait_warp(&s_full[buf], (s >> 1) & 1, abort_flag, a.status))
        break;
      tc_fence_after();
      const float* lse = s_lse + ls * NQ;
      [[maybe_unused]] const float slope = ALIBI ? s_slope[ls] : 0.f;
      f2 acc = {0.f, 0.f};  // of this tile: the total takes one term a tile, whatever M and G
      // `open`: every column of the tile counts for every key of it (rows past m have an
      // lse of -inf here; a row that takes no weight may hold anything, NaN too)
      auto add_tile = [&](auto open) {
#pragma unroll 2
        for (int c0 = 0; c0 < NQ; c0 += 32) {
          uint32_t r[32];
          tmem_ld32(tmem_base + buf * NQ + c0 + lane_addr, r);
          tmem_ld_wait(r);
          if (c0 + 32 >= NQ) {
            tc_fence_before();
            mbar_arrive_warp(&s_free[buf]);
          }
          [[maybe_unused]] const float dist =
              ALIBI ? static_cast<float>(past + m0 + c0 - key) : 0.f;
#pragma unroll
          for (int c = 0; c < 32; c += 2) {
            const f2 nl = *reinterpret_cast<const f2*>(lse + c0 + c);
            f2 x = fma2({__uint_as_float(r[c]), __uint_as_float(r[c + 1])}, sc2, nl);
            if constexpr (ALIBI) {
              x.x = fmaf(-slope, fabsf(dist + c), x.x);
              x.y = fmaf(-slope, fabsf(dist + (c + 1)), x.y);
            }
            if constexpr (open) {
              if (on_fma_pipe(c / 2)) {
                acc = exp2_add(x, acc);
              } else {
                acc = add2(acc, {ex2(x.x), ex2(x.y)});
              }
            } else {
              f2 e = {ex2(x.x), ex2(x.y)};
              if (nl.x == neg_inf() || c0 + c < first) e.x = 0.f;
              if (nl.y == neg_inf() || c0 + c + 1 < first) e.y = 0.f;
              acc = add2(acc, e);
            }
          }
        }
      };
      if (seen && s_open[ls]) add_tile(std::true_type{});
      else add_tile(std::false_type{});
      mbar_arrive_warp(&l_empty[ls]);
      sum += acc.x + acc.y;
    }
    if (grp % C::kParity == 1) s_sum[key - n0] = sum;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == C::kMmaWarp) tmem_dealloc(tmem_base, C::kTmemCols);
  const bool sums = warp < C::kWarps && (warp >> 2) % C::kParity == 0;
  if (a.parts > 1) {
    // Every CTA leaves its sums in the first one's shared memory, which adds them up
    // in order.  (All get here: each wait above is bounded.)
    float* s_part = reinterpret_cast<float*>(smem + C::kPart);  // [part][kKeys]
    cg::cluster_group cluster = cg::this_cluster();
    if (sums) {
      const int at = (warp >> 2) / C::kParity * kWeightKeys + (warp & 3) * 32 + lane;
      sum += s_sum[at];
      if (*abort_flag) sum = __int_as_float(0x7fc00000);
      cluster.map_shared_rank(s_part, 0)[part * C::kKeys + at] = sum;
    }
    cluster.sync();
    if (part != 0 || !sums) return;
    const int at = (warp >> 2) / C::kParity * kWeightKeys + (warp & 3) * 32 + lane, j = n0 + at;
    sum = 0.f;
    for (int p = 0; p < a.parts; ++p) sum += s_part[p * C::kKeys + at];
    if (j < a.N) a.w_out[wrow + j] = j < n ? sum + (a.w_in ? a.w_in[wrow + j] : 0.f) : 0.f;
    return;
  }
  if (sums) {
    const int at = (warp >> 2) / C::kParity * kWeightKeys + (warp & 3) * 32 + lane, j = n0 + at;
    sum += s_sum[at];
    if (*abort_flag) sum = __int_as_float(0x7fc00000);  // a wait gave up
    if (j < a.N) a.w_out[wrow + j] = j < n ? sum + (a.w_in ? a.w_in[wrow + j] : 0.f) : 0.f;
  }
}

// ---------------------------------------------------------------------------
// Few query rows: the (row, head) pairs of a kv head's group are the columns of
// S^T = K Q^T, 8 to a product; a warp takes 16 keys at a time straight from global
// memory into the A fragment (16 bytes of a row a thread and load: the order of the
// contraction index is free, so a thread's 8 consecutive dimensions are two of its
// operand pairs in two steps), the next 16 in flight; Q and lse wait in shared
// memory in fragment order.  Bound by reading K.
// ---------------------------------------------------------------------------
constexpr int kFewWarps = 4;
constexpr int kFewThreads = kFewWarps * 32;

template <bool BF16>
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  if constexpr (BF16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, "
        "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, "
        "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

template <int D, bool BF16, bool ALIBI>
__global__ void __launch_bounds__(kFewThreads, 4)
    weights_few_kernel(const WeightArgs a, const uint16_t* q, const uint16_t* k, bool causal,
                       int blocks) {
  constexpr int J = D / 32;  // 16-byte loads of a row a thread
  extern __shared__ __align__(16) uint8_t smem[];
  FewColumn* s_col = reinterpret_cast<FewColumn*>(smem);               // [blocks * 8]
  uint4* s_q = reinterpret_cast<uint4*>(smem + blocks * 8 * sizeof(FewColumn));  // [blocks][J][32]
  const int kvh = blockIdx.y, b = blockIdx.z;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int gid = lane >> 2, tig = lane & 3;
  const int m = a.q_lens ? a.q_lens[b] : a.M;
  const int past = a.cache_len ? a.cache_len[b] : a.N - a.M;
  if (m < 0 || m > a.M || (a.cache_len && past < 0) || past > a.N - m) {
    if (blockIdx.x == 0 && kvh == 0 && threadIdx.x == 0) record_error(a.status, kErrInvalidArg);
    return;
  }
  const int n = a.cache_len ? past + m : a.N;
  const int c0 = blockIdx.x * a.few_chunk, c1 = min(a.N, c0 + a.few_chunk);
  const int k1 = min(c1, n);  // keys [c0, k1) are there
  float* w_out = a.w_out + (static_cast<long long>(b) * a.Hkv + kvh) * a.N;
  const float* w_in = a.w_in ? a.w_in + (static_cast<long long>(b) * a.Hkv + kvh) * a.N : nullptr;
  for (int j = max(c0, n) + threadIdx.x; j < c1; j += kFewThreads) w_out[j] = 0.f;
  if (c0 >= k1) return;

  const uint16_t* kb = k + b * a.k_s[0] + kvh * a.k_s[2] + 8 * tig;
  auto fetch = [&](int t, uint4(&r)[2][J]) {  // rows gid, gid + 8; past the end the last again
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint4* row = reinterpret_cast<const uint4*>(
          kb + static_cast<long long>(min(t + gid + 8 * h, k1 - 1)) * a.k_s[1]);
#pragma unroll
      for (int j = 0; j < J; ++j) r[h][j] = __ldg(row + 4 * j);
    }
  };
  int t = c0 + warp * 16;
  uint4 cur[2][J];
  if (t < k1) fetch(t, cur);

  const int cols = a.M * a.group;
  for (int c = threadIdx.x; c < blocks * 8; c += kFewThreads) {
    const int i = c / a.group, h = kvh * a.group + c % a.group;
    FewColumn x{neg_inf(), 0.f, 0, 0x7fffffff};
    if (c < cols && i < m) {
      const float l = a.lse[(static_cast<long long>(b) * a.Hq + h) * a.M + i];
      if (l != neg_inf()) x.nl = -l * kLog2e;
      x.slope = exp2f(-8.0f * static_cast<float>(h + 1) / a.Hq) * kLog2e;
      x.pos = past + i;
      if (causal) x.last = past + i;
    }
    s_col[c] = x;
  }
  for (int e = threadIdx.x; e < blocks * J * 32; e += kFewThreads) {
    const int l = e & 31, j = (e >> 5) % J, c = (e >> 5) / J * 8 + (l >> 2);
    const int i = c / a.group, h = kvh * a.group + c % a.group;
    uint4 x = make_uint4(0, 0, 0, 0);
    if (c < cols && i < m)
      x = __ldg(reinterpret_cast<const uint4*>(q + b * a.q_s[0] + i * a.q_s[1] + h * a.q_s[2] +
                                               32 * j + 8 * (l & 3)));
    s_q[e] = x;
  }
  __syncthreads();

  for (; t < k1; t += kFewWarps * 16) {
    uint4 nxt[2][J];
    if (t + kFewWarps * 16 < k1) fetch(t + kFewWarps * 16, nxt);
    float sum[2] = {0.f, 0.f};
    for (int blk = 0; blk < blocks; ++blk) {
      float sc[2][4];  // two chains, half of the dimensions each
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int e = 0; e < 4; ++e) sc[h][e] = 0.f;
#pragma unroll
      for (int j = 0; j < J; ++j) {
        const uint4 x = s_q[(blk * J + j) * 32 + lane];
        mma16816<BF16>(sc[0], cur[0][j].x, cur[1][j].x, cur[0][j].y, cur[1][j].y, x.x, x.y);
        mma16816<BF16>(sc[1], cur[0][j].z, cur[1][j].z, cur[0][j].w, cur[1][j].w, x.z, x.w);
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const FewColumn c = s_col[blk * 8 + 2 * tig + e];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int key = t + gid + 8 * h;
          float x = fmaf(sc[0][2 * h + e] + sc[1][2 * h + e], a.scale_log2, c.nl);
          if constexpr (ALIBI) x = fmaf(-c.slope, fabsf(static_cast<float>(c.pos - key)), x);
          sum[h] += (c.nl == neg_inf() || key > c.last) ? 0.f : ex2(x);
        }
      }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      sum[h] += __shfl_xor_sync(0xffffffffu, sum[h], 1);
      sum[h] += __shfl_xor_sync(0xffffffffu, sum[h], 2);
      const int key = t + gid + 8 * h;
      if (tig == 0 && key < k1) w_out[key] = sum[h] + (w_in ? w_in[key] : 0.f);
#pragma unroll
      for (int j = 0; j < J; ++j) cur[h][j] = nxt[h][j];
    }
  }
}

template <int D, bool BF16>
cudaError_t launch_few(const WeightLaunch& L, cudaStream_t stream) {
  const WeightArgs& a = L.args;
  const int blocks = (a.M * a.group + 7) / 8;
  const int smem = static_cast<int>(few_row_bytes(static_cast<int64_t>(a.M) * a.group, D));
  const dim3 grid((a.N + a.few_chunk - 1) / a.few_chunk, a.Hkv, a.B);
  const uint16_t* q = static_cast<const uint16_t*>(L.q);
  const uint16_t* k = static_cast<const uint16_t*>(L.k);
  if (L.alibi)
    weights_few_kernel<D, BF16, true><<<grid, kFewThreads, smem, stream>>>(a, q, k, L.causal, blocks);
  else
    weights_few_kernel<D, BF16, false><<<grid, kFewThreads, smem, stream>>>(a, q, k, L.causal, blocks);
  return cudaGetLastError();
}

template <int D, bool BF16, bool CAUSAL, bool ALIBI>
cudaError_t launch_t(const WeightLaunch& L, cudaStream_t stream) {
  constexpr auto kern = weights_kernel<D, BF16, CAUSAL, ALIBI>;
  constexpr int smem = WCfg<D>::kBytes, keys = WCfg<D>::kKeys;
  const cudaError_t e = set_smem_once<kern>(smem);
  if (e != cudaSuccess) return e;
  const WeightArgs& a = L.args;
  const long long blocks = static_cast<long long>((a.N + keys - 1) / keys) * a.Hkv * a.B;
  // Fewer key blocks than the GPU holds CTAs: clusters of up to 8 share a block's
  // queries, as long as each has two tiles or more.
  const long long tiles = static_cast<long long>(a.group) * ((a.M + WCfg<D>::NQ - 1) / WCfg<D>::NQ);
  WeightArgs args = a;
  args.parts = 1;
  while (args.parts < kMaxWeightParts && blocks * args.parts * 2 <= 148 * WCfg<D>::kCtas &&
         tiles >= args.parts * 4)
    args.parts *= 2;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks * args.parts));
  cfg.blockDim = dim3(WCfg<D>::kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = args.parts;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = args.parts > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kern, L.tmQ, L.tmK, args);
}

template <int D, bool BF16>
cudaError_t launch_d(const WeightLaunch& L, cudaStream_t stream) {
  if (L.few) return launch_few<D, BF16>(L, stream);
  if (L.causal) return L.alibi ? launch_t<D, BF16, true, true>(L, stream)
                               : launch_t<D, BF16, true, false>(L, stream);
  return L.alibi ? launch_t<D, BF16, false, true>(L, stream)
                 : launch_t<D, BF16, false, false>(L, stream);
}

}  // namespace

cudaError_t launch_weights(const WeightLaunch& L, cudaStream_t stream) {
  if (L.head_dim == 64)
    return L.bf16 ? launch_d<64, true>(L, stream) : launch_d<64, false>(L, stream);
  return L.bf16 ? launch_d<128, true>(L, stream) : launch_d<128, false>(L, stream);
}

}  // namespace mea
