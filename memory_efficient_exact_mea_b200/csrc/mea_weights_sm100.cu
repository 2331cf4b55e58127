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
// buffer each), so one group's exponentials overlap the other's MMA and TMEM read.  Bound by
// the exponential unit (16 a clock per SM) for long query blocks, by reading K
// for a single query row.
//
// Query tiles: 128 rows of one head; or 16 columns of box_heads heads x box_rows
// rows when there are few rows (a decode step's group of heads shares one tile).
#include <math.h>

#include <type_traits>

#include "mea_internal.h"
#include "sm100.cuh"

namespace mea {
namespace {

constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float neg_inf() { return __int_as_float(0xff800000); }

// 32 lanes x 16 columns (thread t: lane quarter + t) and the wait for them.
__device__ __forceinline__ void tmem_ld16_wait(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}

// acc + 2^x for a pair, on the FMA pipe: 2^x = 2^n 2^f with n the integer next to x
// (added into the low mantissa bits of 1.5 2^23) and 2^f, |f| <= 1/2, by a polynomial
// of degree 5 fitted here for the least relative error (7.5e-8; 2.2e-7 with fp32's
// roundings).  x <= -126.5 gives 0, x >= 127 stays there, a NaN stays a NaN.
__device__ __forceinline__ float clamp_exponent(float x) {
  float y;
  asm("max.NaN.f32 %0, %1, 0fC2FE0000;" : "=f"(y) : "f"(x));  // -127
  asm("min.NaN.f32 %0, %1, 0f42FE0000;" : "=f"(y) : "f"(y));  // 127
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

#ifndef MEA_POLY_OF_16
#define MEA_POLY_OF_16 6
#endif
// Which of a chunk's 16 pairs take the polynomial, spread evenly.
__device__ __forceinline__ constexpr bool on_fma_pipe(int pair) {
  return (pair * MEA_POLY_OF_16) % 16 < MEA_POLY_OF_16;
}

// NQ = 128: a query tile is used against kHalves x 128 keys, 2 halves at K = 128 (one
// CTA per SM), 1 at K = 64 (two CTAs): 1 byte of Q read from L2 per score either way.
// Query tiles are released as soon as their MMAs have read them, so the ring runs
// four or five tiles ahead; lse has a ring of its own that lives until the tile's
// sums are done.
template <int D, int NQ>
struct WCfg {
  static constexpr int kHalves = (NQ == 128 && D == 128) ? 2 : 1;
  static constexpr int kKeys = kHalves * kWeightKeys;
  static constexpr int kParity = NQ == 16 ? 1 : 2;  // consumer groups per half
  static constexpr int kGroups = kHalves * kParity;  // of four warps
  static constexpr int kWarps = 4 * kGroups;
  static constexpr int kThreads = (kWarps + 2) * 32;
  static constexpr int kMmaWarp = kWarps, kLoadWarp = kWarps + 1;
  static constexpr int kStages = NQ == 16 ? 2 : (D == 128 ? 4 : 5);
  static constexpr int kLseSlots = 8;
  static constexpr int kCtas = NQ == 16 ? 4 : (kHalves == 2 ? 1 : 2);  // per SM
  static constexpr int kChunks = D / 64;
  static constexpr int kKChunk = kWeightKeys * 128;
  static constexpr int kQChunk = NQ * 128;
  static constexpr int kKTile = kChunks * kKChunk;  // one half
  static constexpr int kQTile = kChunks * kQChunk;
  static constexpr int kQ = kHalves * kKTile;
  static constexpr int kLse = kQ + kStages * kQTile;      // [slot][NQ] -lse * log2(e)
  static constexpr int kSlope = kLse + kLseSlots * NQ * 4;  // [slot][NQ] (narrow), [slot] (wide)
  static constexpr int kSum = kSlope + kLseSlots * (NQ == 16 ? 16 : 1) * 4;  // [kKeys]
  static constexpr int kBar = kSum + kKeys * 4;
  static constexpr int kNumBars = 2 + 2 * kStages + 2 * kLseSlots + 4 * kHalves;
  static constexpr int kTmemSlot = kBar + kNumBars * 8;
  static constexpr int kAbort = kTmemSlot + 4;
  static constexpr int kBytes = kAbort + 4 + 1024;
  static_assert(kCtas * (kBytes + 1024) <= 228 * 1024, "shared memory");
  static constexpr uint32_t kTmemCols = 2 * kHalves * NQ;  // two buffers a half
};

template <int D, bool BF16, int NQ, bool CAUSAL, bool ALIBI>
__global__ void __launch_bounds__(WCfg<D, NQ>::kThreads, WCfg<D, NQ>::kCtas)
    weights_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                   const WeightArgs a) {
  using C = WCfg<D, NQ>;
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
  float* s_sum = reinterpret_cast<float*>(smem + C::kSum);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kTmemSlot);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kAbort);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // The key block varies slowest: under a causal mask the first blocks, seen by
  // the most query rows, start first; CTAs of one (kv head, sequence) read the
  // same query tiles from L2 at about the same time.
  const int per = a.Hkv * a.B;
  const int nb = blockIdx.x / per;
  const int bh = blockIdx.x - nb * per;
  const int b = bh / a.Hkv, kvh = bh - b * a.Hkv;
  const int n0 = nb * C::kKeys;

  const int m = a.q_lens ? a.q_lens[b] : a.M;
  const int past = a.cache_len ? a.cache_len[b] : a.N - a.M;
  const long long wrow = static_cast<long long>(bh) * a.N;
  if (m < 0 || m > a.M || (a.cache_len && past < 0) || past > a.N - m) {
    if (nb == 0 && kvh == 0 && threadIdx.x == 0) record_error(a.status, kErrInvalidArg);
    return;
  }
  // without cache_len the N keys are all there, whatever m is
  const int n = a.cache_len ? past + m : a.N;
  // (head block, row block) pairs; a causal key block starts at the first row that sees it
  const int rows = NQ == 16 ? a.box_rows : NQ;
  const int hblocks = (a.group + a.box_heads - 1) / a.box_heads;
  int m_first = 0;
  if constexpr (CAUSAL) m_first = max(0, n0 - past) / rows * rows;
  const int mblocks = m > m_first ? (m - m_first + rows - 1) / rows : 0;
  const int steps = n0 < n ? hblocks * mblocks : 0;
  if (steps == 0) {  // no query sees these keys
    if (threadIdx.x < C::kKeys && n0 + static_cast<int>(threadIdx.x) < a.N) {
      const int j = n0 + threadIdx.x;
      a.w_out[wrow + j] = (j < n && a.w_in) ? a.w_in[wrow + j] : 0.f;
    }
    return;
  }

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
      const int hb = s / mblocks, m0 = m_first + (s - hb * mblocks) * rows;
      const int slot = s % C::kStages, ls = s % C::kLseSlots;
      float l2[(NQ + 31) / 32], sl[(NQ + 31) / 32];
#pragma unroll
      for (int u = 0; u < (NQ + 31) / 32; ++u) {  // in flight during the waits
        const int c = u * 32 + lane;
        const int g = hb * a.box_heads + (NQ == 16 ? c & (a.box_heads - 1) : 0);
        const int i = m0 + (NQ == 16 ? c >> a.box_shift : c);
        l2[u] = neg_inf();
        sl[u] = 0.f;
        if (c < NQ && i < m && g < a.group) {
          const int h = kvh * a.group + g;
          l2[u] = a.lse[(static_cast<long long>(b) * a.Hq + h) * a.M + i];
          if constexpr (ALIBI) sl[u] = exp2f(-8.0f * static_cast<float>(h + 1) / a.Hq) * kLog2e;
        }
      }
      if (!mbar_wait_warp(&q_empty[slot], ((s / C::kStages) & 1) ^ 1, abort_flag, a.status)) break;
      if (lane == 0) {
        mbar_arrive_expect_tx(&q_full[slot], C::kQTile);
        for (int c = 0; c < C::kChunks; ++c)
          tma_load_4d(smem + C::kQ + slot * C::kQTile + c * C::kQChunk, &tmQ, &q_full[slot],
                      c * 64, kvh * a.group + hb * a.box_heads, m0, b);
      }
      ++issued;
      if (!mbar_wait_warp(&l_empty[ls], ((s / C::kLseSlots) & 1) ^ 1, abort_flag, a.status)) break;
#pragma unroll
      for (int u = 0; u < (NQ + 31) / 32; ++u) {
        const int c = u * 32 + lane;
        if (c < NQ) {  // -inf: the row takes no weight
          s_lse[ls * NQ + c] = l2[u] == neg_inf() ? l2[u] : -l2[u] * kLog2e;
          if (ALIBI && NQ == 16) s_slope[ls * NQ + c] = sl[u];
          if (ALIBI && NQ == 128 && c == 0) s_slope[ls] = sl[u];
        }
      }
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
    f2 acc = {0.f, 0.f};
    const f2 sc2 = {a.scale_log2, a.scale_log2};
    for (int s = grp % C::kParity; s < steps; s += C::kParity) {
      const int hb = s / mblocks, m0 = m_first + (s - hb * mblocks) * rows;
      const int ls = s % C::kLseSlots, buf = 2 * half + (s & 1);
      // row i = m0 + row(c) sees this key iff i >= key - past
      const int first = CAUSAL ? max(0, key - past - m0) : 0;
      const bool whole = NQ == 128 && m0 + NQ <= m &&
                         (!CAUSAL || n0 + (half + 1) * kWeightKeys - 1 - past <= m0);
      if (!mbar_wait_warp(&l_full[ls], (s / C::kLseSlots) & 1, abort_flag, a.status) ||
          !mbar_wait_warp(&s_full[buf], (s >> 1) & 1, abort_flag, a.status))
        break;
      tc_fence_after();
      const float* lse = s_lse + ls * NQ;
      const float slope = ALIBI && NQ == 128 ? s_slope[ls] : 0.f;
      // `open`: every column of the tile counts for every key of it
      auto add_tile = [&](auto open) {
#pragma unroll 1
        for (int c0 = 0; c0 < NQ; c0 += 32) {
          uint32_t r[32];
          if constexpr (NQ == 16) {
            tmem_ld16_wait(tmem_base + buf * NQ + lane_addr, r);
          } else {
            tmem_ld32(tmem_base + buf * NQ + c0 + lane_addr, r);
            tmem_ld_wait(r);
          }
          if (c0 + 32 >= NQ) {
            tc_fence_before();
            mbar_arrive_warp(&s_free[buf]);
          }
          [[maybe_unused]] const float dist =
              ALIBI ? static_cast<float>(past + m0 + (NQ == 16 ? 0 : c0) - key) : 0.f;
#pragma unroll
          for (int c = 0; c < (NQ == 16 ? 16 : 32); c += 2) {
            const f2 nl = *reinterpret_cast<const f2*>(lse + c0 + c);
            f2 x = fma2({__uint_as_float(r[c]), __uint_as_float(r[c + 1])}, sc2, nl);
            const int r0 = NQ == 16 ? c >> a.box_shift : c0 + c;
            const int r1 = NQ == 16 ? (c + 1) >> a.box_shift : c0 + c + 1;
            if constexpr (ALIBI) {
              const float sl0 = NQ == 16 ? s_slope[ls * NQ + c] : slope;
              const float sl1 = NQ == 16 ? s_slope[ls * NQ + c + 1] : slope;
              const float d0 = NQ == 16 ? dist + r0 : dist + c,
                          d1 = NQ == 16 ? dist + r1 : d0 + 1.f;
              x.x = fmaf(-sl0, fabsf(d0), x.x);
              x.y = fmaf(-sl1, fabsf(d1), x.y);
            }
            if constexpr (open) {
              if (on_fma_pipe(c / 2)) {
                acc = exp2_add(x, acc);
              } else {
                acc = add2(acc, {ex2(x.x), ex2(x.y)});
              }
            } else {
              f2 e = {ex2(x.x), ex2(x.y)};
              if (nl.x == neg_inf() || r0 < first) e.x = 0.f;
              if (nl.y == neg_inf() || r1 < first) e.y = 0.f;
              acc = add2(acc, e);
            }
          }
        }
      };
      if (whole) add_tile(std::true_type{});
      else add_tile(std::false_type{});
      mbar_arrive_warp(&l_empty[ls]);
    }
    sum = acc.x + acc.y;
    if (grp % C::kParity == 1) s_sum[key - n0] = sum;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == C::kMmaWarp) tmem_dealloc(tmem_base, C::kTmemCols);
  if (warp < C::kWarps && (warp >> 2) % C::kParity == 0) {
    const int at = (warp >> 2) / C::kParity * kWeightKeys + (warp & 3) * 32 + lane, j = n0 + at;
    if (C::kParity == 2) sum += s_sum[at];
    if (*abort_flag) sum = __int_as_float(0x7fc00000);  // a wait gave up
    if (j < a.N) a.w_out[wrow + j] = j < n ? sum + (a.w_in ? a.w_in[wrow + j] : 0.f) : 0.f;
  }
}

template <int D, bool BF16, int NQ, bool CAUSAL, bool ALIBI>
cudaError_t launch_t(const WeightLaunch& L, cudaStream_t stream) {
  constexpr auto kern = weights_kernel<D, BF16, NQ, CAUSAL, ALIBI>;
  constexpr int smem = WCfg<D, NQ>::kBytes;
  const cudaError_t e = set_smem_once<kern>(smem);
  if (e != cudaSuccess) return e;
  const WeightArgs& a = L.args;
  constexpr int keys = WCfg<D, NQ>::kKeys;
  const long long blocks = static_cast<long long>((a.N + keys - 1) / keys) * a.Hkv * a.B;
  kern<<<static_cast<unsigned>(blocks), WCfg<D, NQ>::kThreads, smem, stream>>>(L.tmQ, L.tmK, a);
  return cudaGetLastError();
}

template <int D, bool BF16, int NQ>
cudaError_t launch_m(const WeightLaunch& L, cudaStream_t stream) {
  if (L.causal) return L.alibi ? launch_t<D, BF16, NQ, true, true>(L, stream)
                               : launch_t<D, BF16, NQ, true, false>(L, stream);
  return L.alibi ? launch_t<D, BF16, NQ, false, true>(L, stream)
                 : launch_t<D, BF16, NQ, false, false>(L, stream);
}

template <int D, bool BF16>
cudaError_t launch_n(const WeightLaunch& L, cudaStream_t stream) {
  return L.narrow ? launch_m<D, BF16, 16>(L, stream) : launch_m<D, BF16, 128>(L, stream);
}

}  // namespace

cudaError_t launch_weights(const WeightLaunch& L, cudaStream_t stream) {
  if (L.head_dim == 64)
    return L.bf16 ? launch_n<64, true>(L, stream) : launch_n<64, false>(L, stream);
  return L.bf16 ? launch_n<128, true>(L, stream) : launch_n<128, false>(L, stream);
}

}  // namespace mea
