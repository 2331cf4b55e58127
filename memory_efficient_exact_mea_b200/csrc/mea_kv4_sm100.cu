// mea_kv4_sm100.cu -- a key/value cache held in 4 bits: store, load, decode.
//
// A decode step is bound by reading the cache ("Transformer : comprendre
// l'entrainement et l'inference", section "Pre-remplissage et decodage"), so a
// cache of K/2 + K/16 bytes per row, head and plane instead of 2 K is read in
// little over a quarter of the time.  Per row and head, 64 dimensions x share a
// zero z = min x and a step s = (max x - min x) / 15 (both rounded to the input's
// 16-bit type; z is one of the inputs, so it is exact); c = nearest integer to
// (x - z) / s in 0..15, and the cache stands for z + s c.  The codes and the
// step are chosen against the rounded z and s, so rounding them costs nothing
// beyond |z + s c - x| <= s/2 (and 15 half steps of s's rounding at c = 15).
#include <math.h>

#include "mea_internal.h"
#include "sm100.cuh"

namespace mea {
namespace {

constexpr float kLn2 = 0.6931471805599453f;
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float neg_inf() { return __int_as_float(0xff800000); }
__device__ __forceinline__ float nan_f() { return __int_as_float(0x7fc00000); }

template <bool BF16>
__device__ __forceinline__ float to_f(uint32_t x) {  // low 16 bits
  if constexpr (BF16) return __uint_as_float(x << 16);
  else return __half2float(__ushort_as_half(static_cast<unsigned short>(x)));
}

template <bool BF16>
__device__ __forceinline__ uint32_t to_16(float x) {
  if constexpr (BF16) return __bfloat16_as_ushort(__float2bfloat16_rn(x));
  else return __half_as_ushort(__float2half_rn(x));
}

// ---------------------------------------------------------------------------
// Store.  Eight lanes hold one group of 64 (16 bytes each); minimum and maximum
// by shuffles.  Consecutive lanes walk rows of one head, so the 16-bit rows are
// read in segments of K * 2 bytes and the codes are written contiguously.
// Bound by memory: 4.6 bytes per element pair against ~12 instructions.
// ---------------------------------------------------------------------------
constexpr int kRowThreads = 256;
constexpr int kRowUnroll = 4;

// The nearest integer to (x - z) / s, ties to even, decided exactly: the fp32
// quotient is right unless it lies next to a half, and there x is compared with
// z + s (k + 1/2), which a double holds exactly for 16-bit z and s.
__device__ __noinline__ float code_exact(float x, float z, float s) {
  const double q = (static_cast<double>(x) - z) / s;
  const double k = floor(q);
  const double edge = static_cast<double>(z) + static_cast<double>(s) * (k + 0.5);
  const double xd = x;
  if (fabs(q - k - 0.5) < 1e-6)
    return static_cast<float>(xd > edge ? k + 1.0 : xd < edge ? k : rint(k + 0.5));
  return static_cast<float>(rint(q));
}

template <int D, bool BF16>
__global__ void __launch_bounds__(kRowThreads) kv4_append_kernel(const Kv4AppendArgs a) {
  constexpr int kLanes = D / 8;  // lanes per row
  constexpr int kRows = kRowThreads / kLanes;
  const int part = threadIdx.x % kLanes;
  const bool value = blockIdx.y != 0;
  const uint16_t* src = static_cast<const uint16_t*>(value ? a.v_new : a.k_new);
  const long long* st = value ? a.vn_s : a.kn_s;
  uint32_t* codes = static_cast<uint32_t*>(value ? a.v_codes : a.k_codes);
  uint32_t* params = static_cast<uint32_t*>(value ? a.v_params : a.k_params);

  uint4 raw[kRowUnroll];
  long long dst[kRowUnroll];  // row of the [B, Hkv, cap] planes, or -1
#pragma unroll
  for (int u = 0; u < kRowUnroll; ++u) {
    const long long idx = (static_cast<long long>(blockIdx.x) * kRowUnroll + u) * kRows +
                          threadIdx.x / kLanes;
    dst[u] = -1;
    raw[u] = make_uint4(0, 0, 0, 0);
    if (idx < a.rows) {
      const unsigned i = static_cast<unsigned>(idx);
      const unsigned bh = i / static_cast<unsigned>(a.M), r = i - bh * a.M;
      const unsigned b = bh / static_cast<unsigned>(a.Hkv), h = bh - b * a.Hkv;
      const int n = a.q_lens ? a.q_lens[b] : a.M;
      const int past = a.cache_len[b];
      if (n < 0 || n > a.M || past < 0 || past > a.cap - n) {
        if (r == 0 && h == 0 && part == 0) record_error(a.status, kErrInvalidArg);
      } else if (static_cast<int>(r) < n) {
        dst[u] = static_cast<long long>(bh) * a.cap + past + r;
        raw[u] = *reinterpret_cast<const uint4*>(src + b * st[0] + r * st[1] + h * st[2] +
                                                 part * 8);
      }
    }
  }
#pragma unroll
  for (int u = 0; u < kRowUnroll; ++u) {
    const uint32_t w[4] = {raw[u].x, raw[u].y, raw[u].z, raw[u].w};
    float x[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = to_f<BF16>(w[i] & 0xffffu);
      x[2 * i + 1] = to_f<BF16>(w[i] >> 16);
    }
    float mn = x[0], mx = x[0], bad = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      mn = fminf(mn, x[i]);
      mx = fmaxf(mx, x[i]);
      bad = fmaf(x[i], 0.f, bad);  // NaN once a value is not finite
    }
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) {
      mn = fminf(mn, __shfl_xor_sync(0xffffffffu, mn, o));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
      bad += __shfl_xor_sync(0xffffffffu, bad, o);
    }
    const float range = mx - mn;  // may pass fp32's largest value for bf16 inputs
    const float s_raw = isinf(range) ? (0.5f * mx - 0.5f * mn) / 15.f * 2.f : range / 15.f;
    uint32_t s16 = to_16<BF16>(s_raw), z16 = to_16<BF16>(mn);
    const float s = to_f<BF16>(s16), z = mn;
    uint32_t word = 0;
    if (bad != bad) {
      s16 = z16 = BF16 ? 0x7fc0u : 0x7e00u;  // a group with a NaN or infinity stands for NaN
    } else if (s > 0.f) {
      float c[8], worst = 0.f;
      // outside this range 1/s or x - z could leave fp32's range
      const bool plain = s >= 0x1p-100f && s <= 0x1p100f;
      const float inv = plain ? 1.f / s : 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float t = (x[i] - z) * inv;
        c[i] = rintf(t);
        worst = fmaxf(worst, fabsf(t - c[i]));
      }
      if (!plain || worst > 0.4999f) {
#pragma unroll
        for (int i = 0; i < 8; ++i) c[i] = code_exact(x[i], z, s);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i)
        word |= static_cast<uint32_t>(fminf(fmaxf(c[i], 0.f), 15.f)) << (4 * i);
    }
    if (dst[u] >= 0) {
      codes[dst[u] * kLanes + part] = word;
      if (part % 8 == 0) params[dst[u] * (D / 64) + part / 8] = s16 | (z16 << 16);
    }
  }
}

// ---------------------------------------------------------------------------
// Load: rows [first_b, first_b + count_b) of every head back into 16 bits.
// ---------------------------------------------------------------------------
template <int D, bool BF16>
__global__ void __launch_bounds__(kRowThreads) kv4_read_kernel(const Kv4ReadArgs a) {
  constexpr int kLanes = D / 8;
  constexpr int kRows = kRowThreads / kLanes;
  const int part = threadIdx.x % kLanes;
  const bool value = blockIdx.y != 0;
  const uint32_t* codes = static_cast<const uint32_t*>(value ? a.v_codes : a.k_codes);
  const uint32_t* params = static_cast<const uint32_t*>(value ? a.v_params : a.k_params);
  uint16_t* out = static_cast<uint16_t*>(value ? a.v_out : a.k_out);
  const long long* st = value ? a.vo_s : a.ko_s;

  uint32_t word[kRowUnroll], sz[kRowUnroll];
  long long dst[kRowUnroll];
#pragma unroll
  for (int u = 0; u < kRowUnroll; ++u) {
    const long long idx = (static_cast<long long>(blockIdx.x) * kRowUnroll + u) * kRows +
                          threadIdx.x / kLanes;
    dst[u] = -1;
    word[u] = sz[u] = 0;
    if (idx < a.total) {
      const unsigned i = static_cast<unsigned>(idx);
      const unsigned bh = i / static_cast<unsigned>(a.out_rows), r = i - bh * a.out_rows;
      const unsigned b = bh / static_cast<unsigned>(a.Hkv), h = bh - b * a.Hkv;
      const int n = a.rows[b];
      const int first = a.first ? a.first[b] : 0;
      if (n < 0 || n > a.out_rows || first < 0 || first > a.cap - n) {
        if (r == 0 && h == 0 && part == 0) record_error(a.status, kErrInvalidArg);
      } else if (static_cast<int>(r) < n) {
        const long long row = static_cast<long long>(bh) * a.cap + first + r;
        word[u] = codes[row * kLanes + part];
        sz[u] = params[row * (D / 64) + part / 8];
        dst[u] = b * st[0] + r * st[1] + h * st[2] + part * 8;
      }
    }
  }
#pragma unroll
  for (int u = 0; u < kRowUnroll; ++u) {
    const float s = to_f<BF16>(sz[u] & 0xffffu), z = to_f<BF16>(sz[u] >> 16);
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      o[i] = pack2<BF16>(fmaf(static_cast<float>((word[u] >> (8 * i)) & 15u), s, z),
                         fmaf(static_cast<float>((word[u] >> (8 * i + 4)) & 15u), s, z));
    if (dst[u] >= 0)
      *reinterpret_cast<uint4*>(out + dst[u]) = make_uint4(o[0], o[1], o[2], o[3]);
  }
}

// ---------------------------------------------------------------------------
// Decode.  With the group's sums kept apart,
//   q.k^_j = sum_g s_jg (sum_{d in g} q_d c_jd) + z_jg (sum_{d in g} q_d)
//   out_d  = sum_j (p_j s_jg) c_jd + sum_j p_j z_jg          (d in group g)
// so the codes go into the tensor cores as they are: a 16-bit number 16 + c is
// made from a nibble by one shift and one and-or (its mantissa field), exact in
// fp16 and bf16, and 16 times the other operand's sum is taken off again in
// fp32.  No dequantised value is ever rounded; p s goes in as bf16 hi + lo.
//
// A warp takes 32 rows at a time straight from global memory into the fragment
// layout of mma.sync m16n8k16 (rows x heads and dimensions x heads, heads
// padded to 8): a thread's nibbles for one row are whole words of the row, and
// since the order of the contraction index is free, the pairs (i, i + 4) of a
// word serve as the operand's pairs.  V pairs two rows: one byte permute joins
// the halves of the two rows' words.  The next 32 rows are fetched while the
// current ones are computed.  The running maximum is raised only when a score
// passes it by 2^8, so the accumulators are rarely rescaled.
// ---------------------------------------------------------------------------
constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kTile = 32;        // rows per warp and iteration
constexpr int kHeads = 8;        // query heads per CTA (MMA n)
constexpr float kLazy = 8.f;     // log2 units a score may pass the running maximum

template <bool BF16>
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  if constexpr (BF16) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, "
        "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  } else {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, "
        "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  }
}

__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// Nibbles N and N + 4 of w as a pair of 16-bit numbers 16 + c: bf16 has the
// unit at mantissa bit 3 of [16, 32), fp16 at bit 6.
template <bool BF16, int N>
__device__ __forceinline__ uint32_t code_pair(uint32_t w) {
  constexpr int kUp = (BF16 ? 3 : 6) - 4 * N;
  const uint32_t x = kUp >= 0 ? w << (kUp >= 0 ? kUp : 0) : w >> (kUp < 0 ? -kUp : 0);
  return BF16 ? ((x & 0x00780078u) | 0x41804180u) : ((x & 0x03C003C0u) | 0x4C004C00u);
}

template <int BYTES>
__device__ __forceinline__ void load_words(const void* p, uint32_t* r) {
  if constexpr (BYTES == 8)
    asm volatile("ld.global.nc.v2.u32 {%0, %1}, [%2];" : "=r"(r[0]), "=r"(r[1]) : "l"(p));
  else
    asm volatile("ld.global.nc.u32 %0, [%1];" : "=r"(r[0]) : "l"(p));
}

template <int D>
struct KSmem {
  float m[kWarps][kHeads];
  float l[kWarps][kHeads];
  float acc[kWarps][kHeads][D];
};

template <int D, bool BF16, bool ALIBI>
__global__ void __launch_bounds__(kThreads, 3) kv4_decode_kernel(const Kv4DecodeArgs a) {
  constexpr int NG = D / 64;  // groups of a row
  __shared__ KSmem<D> sm;
  const int split = blockIdx.x, b = blockIdx.z;
  const int kvh = blockIdx.y / a.head_blocks;
  const int g0 = (blockIdx.y - kvh * a.head_blocks) * kHeads;  // first head within the group
  const int heads = min(kHeads, a.group - g0);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int gid = lane >> 2, tig = lane & 3;
  const int n = a.kv_lens[b];
  const int h0 = kvh * a.group + g0;
  const bool ok = n >= 0 && n <= a.max_len;
  if (!ok && split == 0 && blockIdx.y == 0 && threadIdx.x == 0)
    record_error(a.status, kErrInvalidArg);
  if (!ok || n == 0) {
    if (a.part_o == nullptr) {  // no merge follows
      for (int idx = threadIdx.x; idx < heads * D; idx += kThreads)
        static_cast<uint16_t*>(a.out)[(static_cast<long long>(b) * a.Hq + h0) * D + idx] = 0;
      if (threadIdx.x < heads && a.lse != nullptr)
        a.lse[static_cast<long long>(b) * a.Hq + h0 + threadIdx.x] = ok ? neg_inf() : nan_f();
    }
    return;
  }
  const int s0 = split * a.chunk;
  if (s0 >= n) return;
  const int s1 = min(n, s0 + a.chunk);

  // rows of this (sequence, head) in the four planes
  const long long plane = (static_cast<long long>(b) * a.Hkv + kvh) * a.cap;
  const uint8_t* kc = static_cast<const uint8_t*>(a.k_codes) + plane * (D / 2);
  const uint8_t* vc = static_cast<const uint8_t*>(a.v_codes) + plane * (D / 2);
  const uint32_t* kp = static_cast<const uint32_t*>(a.k_params) + plane * NG;
  const uint32_t* vp = static_cast<const uint32_t*>(a.v_params) + plane * NG;

  uint32_t kw[4][NG][2], kq[4][NG];  // rows gid + 8 i: 16 codes a group; (s, z)
  uint32_t vw[8][NG], vq[4][NG];     // rows 16 (i / 4) + 2 tig + (0, 1, 8, 9)[i % 4]: 8 codes a group
  auto load_k = [&](int t) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const long long row = min(t + gid + 8 * i, s1 - 1);
#pragma unroll
      for (int g = 0; g < NG; ++g)
        load_words<8>(kc + row * (D / 2) + 32 * g + 8 * tig, kw[i][g]);
      load_words<4 * NG>(kp + row * NG, kq[i]);
    }
  };
  auto load_v = [&](int t) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const long long row =
          min(t + 16 * (i / 4) + 2 * tig + (i & 1) + 8 * ((i >> 1) & 1), s1 - 1);
#pragma unroll
      for (int g = 0; g < NG; ++g)
        load_words<4>(vc + row * (D / 2) + 32 * g + 4 * gid, &vw[i][g]);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
      load_words<4 * NG>(vp + static_cast<long long>(min(t + gid + 8 * i, s1 - 1)) * NG, vq[i]);
  };
  int t = s0 + warp * kTile;
  if (t < s1) {
    load_k(t);
    load_v(t);
  }

  // Q^T as the B operand (head gid), and 2^x-scaled sums of q over each group
  // for this thread's two heads.
  uint32_t qb[NG][4][2];
  float qsum[NG][2];
  {
    const uint16_t* qrow = static_cast<const uint16_t*>(a.q) +
                           (static_cast<long long>(b) * a.Hq + h0 + gid) * D;
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      float sum = 0.f;
#pragma unroll
      for (int ks = 0; ks < 4; ++ks)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int d = 64 * g + 16 * tig + 8 * (ks >> 1) + 2 * (ks & 1) + e;
          const uint32_t lo = gid < heads ? qrow[d] : 0u;
          const uint32_t hi = gid < heads ? qrow[d + 4] : 0u;
          qb[g][ks][e] = lo | (hi << 16);
          sum += to_f<BF16>(lo) + to_f<BF16>(hi);
        }
      sum += __shfl_xor_sync(0xffffffffu, sum, 1);
      sum += __shfl_xor_sync(0xffffffffu, sum, 2);
      qsum[g][0] = __shfl_sync(0xffffffffu, sum, 8 * tig) * a.scale_log2;
      qsum[g][1] = __shfl_sync(0xffffffffu, sum, 8 * tig + 4) * a.scale_log2;
    }
  }
  float slope[2] = {0.f, 0.f};
  if constexpr (ALIBI) {
#pragma unroll
    for (int e = 0; e < 2; ++e)
      slope[e] = exp2f(-8.0f * static_cast<float>(h0 + 2 * tig + e + 1) / a.Hq) * kLog2e;
  }

  float m_run[2] = {neg_inf(), neg_inf()}, l_part[2] = {0.f, 0.f};
  float zacc[NG][2], acc[D / 16][4];
#pragma unroll
  for (int g = 0; g < NG; ++g) zacc[g][0] = zacc[g][1] = 0.f;
#pragma unroll
  for (int i = 0; i < D / 16; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[i][e] = 0.f;

  for (; t < s1; t += kWarps * kTile) {
    const int next = t + kWarps * kTile;
    float x[2][4];
#pragma unroll
    for (int blk = 0; blk < 2; ++blk) {
#pragma unroll
      for (int e = 0; e < 4; ++e) x[blk][e] = 0.f;
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        float sc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          const uint32_t lo = kw[2 * blk][g][w], hi = kw[2 * blk + 1][g][w];
          mma16816<BF16>(sc, code_pair<BF16, 0>(lo), code_pair<BF16, 0>(hi),
                         code_pair<BF16, 1>(lo), code_pair<BF16, 1>(hi), qb[g][2 * w][0],
                         qb[g][2 * w][1]);
          mma16816<BF16>(sc, code_pair<BF16, 2>(lo), code_pair<BF16, 2>(hi),
                         code_pair<BF16, 3>(lo), code_pair<BF16, 3>(hi), qb[g][2 * w + 1][0],
                         qb[g][2 * w + 1][1]);
        }
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const float s = to_f<BF16>(kq[2 * blk + r][g] & 0xffffu);
          const float z = to_f<BF16>(kq[2 * blk + r][g] >> 16);
          const float corr = fmaf(-16.f, s, z), ss = s * a.scale_log2;
#pragma unroll
          for (int e = 0; e < 2; ++e)
            x[blk][2 * r + e] += fmaf(ss, sc[2 * r + e], corr * qsum[g][e]);
        }
      }
    }
    if (next < s1) load_k(next);
    if constexpr (ALIBI) {
#pragma unroll
      for (int blk = 0; blk < 2; ++blk)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          x[blk][e] = fmaf(-slope[e & 1],
                           static_cast<float>(n - 1 - (t + 16 * blk + 8 * (e >> 1) + gid)),
                           x[blk][e]);
    }
    if (t + kTile > s1) {
#pragma unroll
      for (int blk = 0; blk < 2; ++blk)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (t + 16 * blk + 8 * (e >> 1) + gid >= s1) x[blk][e] = neg_inf();
    }
    if (a.scores != nullptr) {  // kept for the gathered weights, log2 units
#pragma unroll
      for (int e = 0; e < 2; ++e)
        if (2 * tig + e < heads) {
          float* out = a.scores + (static_cast<long long>(b) * a.Hq + h0 + 2 * tig + e) *
                                      a.score_stride + t + gid;
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (t + 8 * i + gid < s1) out[8 * i] = x[i >> 1][2 * (i & 1) + e];
        }
    }
    float mx[2];
#pragma unroll
    for (int e = 0; e < 2; ++e)
      mx[e] = fmaxf(fmaxf(x[0][e], x[0][e + 2]), fmaxf(x[1][e], x[1][e + 2]));
    if (__any_sync(0xffffffffu, mx[0] > m_run[0] + kLazy || mx[1] > m_run[1] + kLazy)) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], 4));
        mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], 8));
        mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], 16));
        const float m_new = fmaxf(m_run[e], mx[e]);
        const float alpha = m_new == m_run[e] ? 1.f : ex2(m_run[e] - m_new);
        m_run[e] = m_new;
        l_part[e] *= alpha;
#pragma unroll
        for (int g = 0; g < NG; ++g) zacc[g][e] *= alpha;
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          acc[i][e] *= alpha;
          acc[i][e + 2] *= alpha;
        }
      }
    }
#pragma unroll
    for (int blk = 0; blk < 2; ++blk) {
      float p[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        // a row of -inf scores alone leaves m_run at -inf: no weight yet
        p[e] = x[blk][e] == neg_inf() ? 0.f : ex2(x[blk][e] - m_run[e & 1]);
        l_part[e & 1] += p[e];
      }
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        uint32_t hi[2], lo[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const float s = to_f<BF16>(vq[2 * blk + r][g] & 0xffffu);
          const float z = to_f<BF16>(vq[2 * blk + r][g] >> 16);
          const float p0 = p[2 * r] * s, p1 = p[2 * r + 1] * s;
          const uint32_t h = pack2<true>(p0, p1);
          const float h0f = __uint_as_float(h << 16), h1f = __uint_as_float(h & 0xffff0000u);
          const uint32_t l = pack2<true>(p0 - h0f, p1 - h1f);
          const float r0 = h0f + __uint_as_float(l << 16);
          const float r1 = h1f + __uint_as_float(l & 0xffff0000u);
          // what the tensor cores add for the code offset is 16 x the rounded p s
          zacc[g][0] += fmaf(p[2 * r], z, -16.f * r0);
          zacc[g][1] += fmaf(p[2 * r + 1], z, -16.f * r1);
          hi[r] = movmatrix_trans(h);
          lo[r] = movmatrix_trans(l);
        }
        // rows 2 tig, 2 tig + 1 (first pair) and + 8 (second): words of 8 dimensions
        const uint32_t w0 = vw[4 * blk][g], w1 = vw[4 * blk + 1][g];
        const uint32_t w2 = vw[4 * blk + 2][g], w3 = vw[4 * blk + 3][g];
        const uint32_t xa = __byte_perm(w0, w1, 0x5410), ya = __byte_perm(w0, w1, 0x7632);
        const uint32_t xb = __byte_perm(w2, w3, 0x5410), yb = __byte_perm(w2, w3, 0x7632);
#define MEA_KV4_PV(N)                                                                       \
  {                                                                                         \
    const uint32_t a0 = code_pair<true, N>(xa), a1 = code_pair<true, N>(ya);                \
    const uint32_t a2 = code_pair<true, N>(xb), a3 = code_pair<true, N>(yb);                \
    mma16816<true>(acc[4 * g + N], a0, a1, a2, a3, hi[0], hi[1]);                           \
    mma16816<true>(acc[4 * g + N], a0, a1, a2, a3, lo[0], lo[1]);                           \
  }
        MEA_KV4_PV(0)
        MEA_KV4_PV(1)
        MEA_KV4_PV(2)
        MEA_KV4_PV(3)
#undef MEA_KV4_PV
      }
    }
    if (next < s1) load_v(next);
  }

#pragma unroll
  for (int e = 0; e < 2; ++e)
#pragma unroll
    for (int o = 4; o <= 16; o <<= 1) {
      l_part[e] += __shfl_xor_sync(0xffffffffu, l_part[e], o);
#pragma unroll
      for (int g = 0; g < NG; ++g) zacc[g][e] += __shfl_xor_sync(0xffffffffu, zacc[g][e], o);
    }
  if (gid == 0) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      sm.m[warp][2 * tig + e] = m_run[e];
      sm.l[warp][2 * tig + e] = l_part[e];
    }
  }
#pragma unroll
  for (int i = 0; i < D / 16; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e)  // tile i: dimension 64 (i/4) + 8 gid + i % 4 (+ 4)
      sm.acc[warp][2 * tig + (e & 1)][64 * (i >> 2) + 8 * gid + (i & 3) + 4 * (e >> 1)] =
          acc[i][e] + zacc[i >> 2][e & 1];
  __syncthreads();

  for (int idx = threadIdx.x; idx < heads * D; idx += kThreads) {
    const int g = idx / D, d = idx - g * D;
    float mx = neg_inf();
#pragma unroll
    for (int w = 0; w < kWarps; ++w) mx = fmaxf(mx, sm.m[w][g]);
    float lsum = 0.f, o = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float wgt = sm.m[w][g] == neg_inf() ? (sm.l[w][g] == 0.f ? 0.f : 1.f)
                                                : ex2(sm.m[w][g] - mx);
      lsum += wgt * sm.l[w][g];
      o += wgt * sm.acc[w][g][d];
    }
    const long long row = static_cast<long long>(b) * a.Hq + h0 + g;
    const float val = lsum == 0.f ? 0.f : o / lsum;  // a NaN stays a NaN
    const float lse2 = lsum == 0.f ? neg_inf() : mx + __log2f(lsum);
    if (a.part_o == nullptr) {  // the only split
      static_cast<uint16_t*>(a.out)[row * D + d] = static_cast<uint16_t>(to_16<BF16>(val));
    } else {
      a.part_o[(row * a.max_splits + split) * D + d] = val;
    }
    if (d == 0) {
      if (a.part_lse != nullptr) a.part_lse[row * a.max_splits + split] = lse2;
      if (a.part_o == nullptr && a.lse != nullptr) a.lse[row] = lse2 * kLn2;
    }
  }
}

// Joins the splits of a (sequence, query head) by their log-sum-exp (one warp a
// head), and adds the gathered weights: blocks from merge_blocks on take
// kWeightRows rows of one (sequence, kv head) each and sum 2^(x - lse) over the
// group's heads, in head order.
constexpr int kWeightRows = 1024;

__device__ __forceinline__ float merged_lse2(const float* pl, int ns, int lane) {
  float mx = neg_inf();
  for (int s = lane; s < ns; s += 32) mx = fmaxf(mx, pl[s]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  float sum = 0.f;
  const float base = mx == neg_inf() ? 0.f : mx;
  for (int s = lane; s < ns; s += 32) sum += ex2(pl[s] - base);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  return sum == 0.f ? neg_inf() : base + __log2f(sum);
}

template <int D, bool BF16>
__global__ void __launch_bounds__(256) kv4_merge_kernel(const Kv4DecodeArgs a) {
  __shared__ float s_lse[256];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (static_cast<int>(blockIdx.x) < a.merge_blocks) {
    const int row = blockIdx.x * 8 + warp;
    if (row >= a.B * a.Hq) return;
    const int b = row / a.Hq;
    const int n = a.kv_lens[b];
    uint16_t* out = static_cast<uint16_t*>(a.out) + static_cast<long long>(row) * D;
    const bool ok = n >= 0 && n <= a.max_len;
    if (!ok || n == 0) {
      if (!ok && lane == 0 && row % a.Hq == 0) record_error(a.status, kErrInvalidArg);
#pragma unroll
      for (int i = 0; i < D / 32; ++i) out[lane + 32 * i] = 0;
      if (lane == 0 && a.lse != nullptr) a.lse[row] = ok ? neg_inf() : nan_f();
      return;
    }
    const int ns = (n + a.chunk - 1) / a.chunk;
    const float* pl = a.part_lse + static_cast<long long>(row) * a.max_splits;
    const float* po = a.part_o + static_cast<long long>(row) * a.max_splits * D;
    const float lse2 = merged_lse2(pl, ns, lane);
    const float base = lse2 == neg_inf() ? 0.f : lse2;
    float o[D / 32];
#pragma unroll
    for (int i = 0; i < D / 32; ++i) o[i] = 0.f;
#pragma unroll 4
    for (int s = 0; s < ns; ++s) {
      const float w = ex2(pl[s] - base);
#pragma unroll
      for (int i = 0; i < D / 32; ++i) o[i] = fmaf(w, po[s * D + lane + 32 * i], o[i]);
    }
#pragma unroll
    for (int i = 0; i < D / 32; ++i)
      out[lane + 32 * i] = static_cast<uint16_t>(to_16<BF16>(o[i]));
    if (lane == 0 && a.lse != nullptr) a.lse[row] = lse2 * kLn2;
    return;
  }
  // weights
  const int blk = blockIdx.x - a.merge_blocks;
  const int bh = blk / a.weight_blocks, c0 = (blk - bh * a.weight_blocks) * kWeightRows;
  const int b = bh / a.Hkv, kvh = bh - b * a.Hkv;
  const int n = a.kv_lens[b];
  if (n < 0 || n > a.max_len) return;
  const long long wrow = static_cast<long long>(bh) * a.cap;
  const int ns = (n + a.chunk - 1) / a.chunk;
  const int c1 = min(a.cap, c0 + kWeightRows);
  float sum[kWeightRows / 256];
#pragma unroll
  for (int u = 0; u < kWeightRows / 256; ++u) sum[u] = 0.f;
  for (int g0 = 0; g0 < a.group && c0 < n; g0 += 256) {
    const int gn = min(256, a.group - g0);
    __syncthreads();
    for (int g = warp; g < gn; g += 8) {
      const long long row = static_cast<long long>(b) * a.Hq + kvh * a.group + g0 + g;
      const float l = merged_lse2(a.part_lse + row * a.max_splits, ns, lane);
      if (lane == 0) s_lse[g] = l;
    }
    __syncthreads();
    for (int g = 0; g < gn; ++g) {
      const float* x = a.scores + (static_cast<long long>(b) * a.Hq + kvh * a.group + g0 + g) *
                                      a.score_stride;
      const float l = s_lse[g];
#pragma unroll
      for (int u = 0; u < kWeightRows / 256; ++u) {
        const int j = c0 + u * 256 + threadIdx.x;
        if (j < n && l != neg_inf()) sum[u] += ex2(x[j] - l);
      }
    }
  }
#pragma unroll
  for (int u = 0; u < kWeightRows / 256; ++u) {
    const int j = c0 + u * 256 + threadIdx.x;
    if (j < c1)
      a.w_out[wrow + j] = j < n ? sum[u] + (a.w_in ? a.w_in[wrow + j] : 0.f) : 0.f;
  }
}

template <int D, bool BF16>
cudaError_t decode_t(const Kv4DecodeArgs& a, bool alibi, cudaStream_t stream) {
  if (a.max_splits > 0) {
    const dim3 grid(a.max_splits, a.Hkv * a.head_blocks, a.B);
    if (alibi) kv4_decode_kernel<D, BF16, true><<<grid, kThreads, 0, stream>>>(a);
    else kv4_decode_kernel<D, BF16, false><<<grid, kThreads, 0, stream>>>(a);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  if (a.part_o == nullptr && a.max_splits > 0 && a.w_out == nullptr) return cudaSuccess;
  const long long blocks =
      a.merge_blocks + static_cast<long long>(a.B) * a.Hkv * a.weight_blocks;
  if (blocks == 0) return cudaSuccess;
  kv4_merge_kernel<D, BF16><<<static_cast<unsigned>(blocks), 256, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace

int kv4_weight_rows() { return kWeightRows; }

cudaError_t launch_kv4_append(const Kv4AppendArgs& a, int head_dim, bool bf16,
                              cudaStream_t stream) {
  const long long per = static_cast<long long>(kRowUnroll) * kRowThreads * 8 / head_dim;
  const dim3 grid(static_cast<unsigned>((a.rows + per - 1) / per), 2);
  if (head_dim == 64 && !bf16) kv4_append_kernel<64, false><<<grid, kRowThreads, 0, stream>>>(a);
  else if (head_dim == 64) kv4_append_kernel<64, true><<<grid, kRowThreads, 0, stream>>>(a);
  else if (!bf16) kv4_append_kernel<128, false><<<grid, kRowThreads, 0, stream>>>(a);
  else kv4_append_kernel<128, true><<<grid, kRowThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_kv4_read(const Kv4ReadArgs& a, int head_dim, bool bf16, cudaStream_t stream) {
  const long long per = static_cast<long long>(kRowUnroll) * kRowThreads * 8 / head_dim;
  const dim3 grid(static_cast<unsigned>((a.total + per - 1) / per), 2);
  if (head_dim == 64 && !bf16) kv4_read_kernel<64, false><<<grid, kRowThreads, 0, stream>>>(a);
  else if (head_dim == 64) kv4_read_kernel<64, true><<<grid, kRowThreads, 0, stream>>>(a);
  else if (!bf16) kv4_read_kernel<128, false><<<grid, kRowThreads, 0, stream>>>(a);
  else kv4_read_kernel<128, true><<<grid, kRowThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_kv4_decode(const Kv4DecodeArgs& a, int head_dim, bool bf16, bool alibi,
                              cudaStream_t stream) {
  if (head_dim == 64) return bf16 ? decode_t<64, true>(a, alibi, stream)
                                  : decode_t<64, false>(a, alibi, stream);
  return bf16 ? decode_t<128, true>(a, alibi, stream) : decode_t<128, false>(a, alibi, stream);
}

}  // namespace mea
