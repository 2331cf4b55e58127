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

#include "mea_cache_internal.h"
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
__device__ __forceinline__ float step_of(uint32_t w) {  // low 16 bits of a pair
  if constexpr (BF16) return __uint_as_float(w << 16);
  else return __low2float(*reinterpret_cast<const __half2*>(&w));
}

template <bool BF16>
__device__ __forceinline__ float zero_of(uint32_t w) {  // high 16 bits of a pair
  if constexpr (BF16) return __uint_as_float(w & 0xffff0000u);
  else return __high2float(*reinterpret_cast<const __half2*>(&w));
}

template <bool BF16>
__device__ __forceinline__ uint32_t to_16(float x) {
  if constexpr (BF16) return __bfloat16_as_ushort(__float2bfloat16_rn(x));
  else return __half_as_ushort(__float2half_rn(x));
}

// ---------------------------------------------------------------------------
// Rows of a [B, M, Hkv] batch in one flat order: kRowGroup rows of one head (one
// group of lanes takes them all), then the next head, then the next rows.  A
// block's share is one contiguous piece of the 16-bit side ([B, M, Hkv, K]) and
// runs of a few whole rows on the 4-bit side ([B, Hkv, rows, ...]).  (Head by head,
// 2 KB apart on the 16-bit side, loading 300 MB took 87 us instead of 78; a row at
// a time, its place divided out for each, left the kernels bound by that
// arithmetic.)
// ---------------------------------------------------------------------------
constexpr int kRowThreads = 256;
constexpr int kRowGroup = 4;

__device__ __forceinline__ unsigned divide(unsigned x, const FastDiv& d) {
  return (__umulhi(x, d.m) + x) >> d.s;
}

// ---------------------------------------------------------------------------
// Store.  Eight lanes hold one group of 64 (16 bytes each); minimum and maximum
// by packed 16-bit comparisons and shuffles.
// ---------------------------------------------------------------------------
// c = nearest integer to (x - z) / s, ties to even, decided exactly.  Adding 1.5 2^23
// to d / s (in one fused step, d = x - z) rounds it to an integer in the low mantissa
// bits; that is right unless the quotient lies next to a half.  There the sign of
// x - (z + s (k + 1/2)) decides: s (k + 1/2) has at most 16 bits, d lies within a
// factor of two of it, and the part of x - z that d lost is known (the error term of
// Knuth's two-sum), so the sign is exact.
constexpr float kRound = 12582912.f;  // 1.5 * 2^23

// In fp32 with q = d / s to within 1e-4; in doubles (q = d / s) for steps outside
// [2^-100, 2^100], where fp32's products could leave its range.
template <typename T>
__device__ __forceinline__ float code_near_half(T x, T z, T s, T inv) {
  const T d = x - z;
  const T bb = d - x;
  const T lost = (x - (d - bb)) + (-z - bb);  // x - z = d + lost
  T q;
  if constexpr (sizeof(T) == 8) q = d / s;
  else q = d * inv;
  const T k = floor(q);
  if (fabs(q - k - T(0.5)) > T(1e-3)) return static_cast<float>(rint(q));
  const T over = (d - s * (k + T(0.5))) + lost;
  return static_cast<float>(over > 0 ? k + 1 : over < 0 ? k : rint(k + T(0.5)));
}
__device__ __noinline__ float code_wide(float x, float z, float s) {
  return code_near_half<double>(x, z, s, 0.0);
}

// Packed minimum and maximum; a NaN stays one.
template <bool BF16>
__device__ __forceinline__ uint32_t min2(uint32_t a, uint32_t b) {
  if constexpr (BF16) {
    const __nv_bfloat162 r = __hmin2_nan(*reinterpret_cast<const __nv_bfloat162*>(&a),
                                         *reinterpret_cast<const __nv_bfloat162*>(&b));
    return *reinterpret_cast<const uint32_t*>(&r);
  } else {
    const __half2 r =
        __hmin2_nan(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
    return *reinterpret_cast<const uint32_t*>(&r);
  }
}
template <bool BF16>
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
  if constexpr (BF16) {
    const __nv_bfloat162 r = __hmax2_nan(*reinterpret_cast<const __nv_bfloat162*>(&a),
                                         *reinterpret_cast<const __nv_bfloat162*>(&b));
    return *reinterpret_cast<const uint32_t*>(&r);
  } else {
    const __half2 r =
        __hmax2_nan(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
    return *reinterpret_cast<const uint32_t*>(&r);
  }
}

template <int D, bool BF16>
__global__ void __launch_bounds__(kRowThreads, 5) kv4_append_kernel(const Kv4AppendArgs a) {
  constexpr int kLanes = D / 8;  // lanes per row
  const unsigned group =
      blockIdx.x * (kRowThreads / kLanes) + threadIdx.x / kLanes;  // of kRowGroup rows
  const int part = threadIdx.x % kLanes;
  const bool value = blockIdx.y != 0;
  const unsigned q = divide(group, a.order.heads), h = group - q * a.order.heads.d;
  const unsigned b = divide(q, a.order.tiles), r0 = (q - b * a.order.tiles.d) * kRowGroup;
  int rows = 0;  // of this group
  long long dst = 0;
  if (group < a.order.total) {
    const int n = a.q_lens ? a.q_lens[b] : a.M;
    const int past = a.cache_len[b];
    if (n < 0 || n > a.M || past < 0 || past > a.cap - n) {
      if (r0 == 0 && h == 0 && part == 0) record_error(a.status, kErrInvalidArg);
    } else {
      rows = min(n - static_cast<int>(r0), kRowGroup);
      dst = (static_cast<long long>(b) * a.Hkv + h) * a.cap + past + r0;
    }
  }
  const long long step = value ? a.vn_s[1] : a.kn_s[1];
  const uint16_t* src = static_cast<const uint16_t*>(value ? a.v_new : a.k_new) +
                        b * (value ? a.vn_s[0] : a.kn_s[0]) + r0 * step +
                        h * (value ? a.vn_s[2] : a.kn_s[2]) + part * 8;
  uint32_t* codes = static_cast<uint32_t*>(value ? a.v_codes : a.k_codes) + dst * kLanes + part;
  uint32_t* params =
      static_cast<uint32_t*>(value ? a.v_params : a.k_params) + dst * (D / 64) + part / 8;
  static_assert(kRowGroup <= 8, "a lane of the eight for each row");

  uint4 raw[kRowGroup];
#pragma unroll
  for (int u = 0; u < kRowGroup; ++u) {
    raw[u] = make_uint4(0, 0, 0, 0);
    if (u < rows) raw[u] = *reinterpret_cast<const uint4*>(src + u * step);
  }
  // Least and greatest value of each row's group, in all its eight lanes; lane u of
  // the eight then keeps those of row u and works out its step alone.
  float z_row[kRowGroup], top = 0.f, low = 0.f;
  const int lane8 = threadIdx.x & 7;
#pragma unroll
  for (int u = 0; u < kRowGroup; ++u) {
    uint32_t lo = min2<BF16>(min2<BF16>(raw[u].x, raw[u].y), min2<BF16>(raw[u].z, raw[u].w));
    uint32_t hi = max2<BF16>(max2<BF16>(raw[u].x, raw[u].y), max2<BF16>(raw[u].z, raw[u].w));
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) {
      lo = min2<BF16>(lo, __shfl_xor_sync(0xffffffffu, lo, o));
      hi = max2<BF16>(hi, __shfl_xor_sync(0xffffffffu, hi, o));
    }
    lo = min2<BF16>(lo, lo >> 16);  // (the high half is not used)
    hi = max2<BF16>(hi, hi >> 16);
    z_row[u] = to_f<BF16>(lo & 0xffffu);
    if (lane8 == u) {
      low = z_row[u];
      top = to_f<BF16>(hi & 0xffffu);
    }
  }
  const float range = top - low;  // may pass fp32's largest value for bf16 inputs
  const float s_raw = isinf(range) ? (0.5f * top - 0.5f * low) / 15.f * 2.f : range / 15.f;
  uint32_t s16 = to_16<BF16>(s_raw), z16 = to_16<BF16>(low);
  const float s_mine = to_f<BF16>(s16);
  // 1/s within 2 ulp, like the 1e-4 next to a half below; 0: codes of zero; negative:
  // steps whose reciprocal or whose x - z could leave fp32's range
  float inv_mine = 0.f;
  if (!(fabsf(low) < __int_as_float(0x7f800000) && fabsf(top) < __int_as_float(0x7f800000)))
    s16 = z16 = BF16 ? 0x7fc0u : 0x7e00u;  // a group with a NaN or infinity stands for NaN
  else if (s_mine > 0.f)
    inv_mine = s_mine >= 0x1p-100f && s_mine <= 0x1p100f ? __fdividef(1.f, s_mine) : -1.f;
  if (lane8 < rows) params[lane8 * (D / 64)] = s16 | (z16 << 16);

#pragma unroll
  for (int u = 0; u < kRowGroup; ++u) {
    const float inv = __shfl_sync(0xffffffffu, inv_mine, u, 8);
    const float s = __shfl_sync(0xffffffffu, s_mine, u, 8), z = z_row[u];
    if (u >= rows) continue;
    const uint32_t w[4] = {raw[u].x, raw[u].y, raw[u].z, raw[u].w};
    float x[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = step_of<BF16>(w[i]);
      x[2 * i + 1] = zero_of<BF16>(w[i]);
    }
    uint32_t word = 0;
    if (inv > 0.f) {
      float worst = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float d = x[i] - z;
        const float m = fminf(fmaf(d, inv, kRound), kRound + 15.f);
        worst = fmaxf(worst, fabsf(fmaf(d, inv, kRound - m)));
        // the mantissa's low bits are the code; kRound's own bits come off below
        word += __float_as_uint(m) << (4 * i);
      }
      constexpr uint32_t kBits = 0x4B400000u;
      word -= kBits + (kBits << 4) + (kBits << 8) + (kBits << 12) + (kBits << 16) +
              (kBits << 20) + (kBits << 24) + (kBits << 28);
      if (worst > 0.4999f) {  // some quotient lies next to a half, or past 15
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float d = x[i] - z;
          const float m = fminf(fmaf(d, inv, kRound), kRound + 15.f);
          if (fabsf(fmaf(d, inv, kRound - m)) > 0.4999f) {
            const uint32_t c =
                static_cast<uint32_t>(fminf(code_near_half<float>(x[i], z, s, inv), 15.f));
            word = (word & ~(15u << (4 * i))) | (c << (4 * i));
          }
        }
      }
    } else if (inv < 0.f) {
      for (int i = 0; i < 8; ++i)
        word |= static_cast<uint32_t>(fminf(fmaxf(code_wide(x[i], z, s), 0.f), 15.f)) << (4 * i);
    }
    codes[u * kLanes] = word;
  }
}

// Results: rounded to 16 bits and held to the type's finite range (z + 15 s may pass it
// by a step's rounding; an infinity is never stored), a NaN stays one.
template <bool BF16>
__device__ __forceinline__ uint32_t pack2_finite(float lo, float hi) {
  uint32_t r;
  if constexpr (BF16) asm("cvt.rn.satfinite.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  else asm("cvt.rn.satfinite.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
template <bool BF16>
__device__ __forceinline__ uint16_t to_16_finite(float x) {
  return static_cast<uint16_t>(pack2_finite<BF16>(x, x));
}

// ---------------------------------------------------------------------------
// Load: rows [first_b, first_b + count_b) of every head back into 16 bits.
// ---------------------------------------------------------------------------
// c s + z in fp32 with c and s 16-bit (exact product, one rounding).
template <bool BF16>
__device__ __forceinline__ float fma_16(uint16_t c, uint16_t s, float z) {
  float d;
  if constexpr (BF16)
    asm("fma.rn.f32.bf16 %0, %1, %2, %3;" : "=f"(d) : "h"(c), "h"(s), "f"(z));
  else
    asm("fma.rn.f32.f16 %0, %1, %2, %3;" : "=f"(d) : "h"(c), "h"(s), "f"(z));
  return d;
}

template <int D, bool BF16>
__global__ void __launch_bounds__(kRowThreads) kv4_read_kernel(const Kv4ReadArgs a) {
  constexpr int kLanes = D / 8;
  const unsigned group =
      blockIdx.x * (kRowThreads / kLanes) + threadIdx.x / kLanes;  // of kRowGroup rows
  const int part = threadIdx.x % kLanes;
  const bool value = blockIdx.y != 0;
  if (group >= a.order.total) return;
  const unsigned q = divide(group, a.order.heads), h = group - q * a.order.heads.d;
  const unsigned b = divide(q, a.order.tiles), r0 = (q - b * a.order.tiles.d) * kRowGroup;
  const int n = a.rows[b];
  const int skip = a.first ? a.first[b] : 0;
  if (n < 0 || n > a.out_rows || skip < 0 || skip > a.cap - n) {
    if (r0 == 0 && h == 0 && part == 0) record_error(a.status, kErrInvalidArg);
    return;
  }
  const int rows = min(n - static_cast<int>(r0), kRowGroup);
  if (rows <= 0) return;
  const long long row = (static_cast<long long>(b) * a.Hkv + h) * a.cap + skip + r0;
  const uint32_t* codes =
      static_cast<const uint32_t*>(value ? a.v_codes : a.k_codes) + row * kLanes + part;
  const uint32_t* params =
      static_cast<const uint32_t*>(value ? a.v_params : a.k_params) + row * (D / 64) + part / 8;
  const long long step = value ? a.vo_s[1] : a.ko_s[1];
  uint16_t* out = static_cast<uint16_t*>(value ? a.v_out : a.k_out) +
                  b * (value ? a.vo_s[0] : a.ko_s[0]) + r0 * step +
                  h * (value ? a.vo_s[2] : a.ko_s[2]) + part * 8;

  uint32_t word[kRowGroup], sz[kRowGroup];
#pragma unroll
  for (int u = 0; u < kRowGroup; ++u) {
    word[u] = sz[u] = 0;
    if (u < rows) {
      word[u] = codes[u * kLanes];
      sz[u] = params[u * (D / 64)];
    }
  }
#pragma unroll
  for (int u = 0; u < kRowGroup; ++u) {
    const uint16_t s = static_cast<uint16_t>(sz[u]);
    const float z = BF16 ? __uint_as_float(sz[u] & 0xffff0000u) : to_f<BF16>(sz[u] >> 16);
    float v[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {  // nibbles i and i + 4 as a pair of numbers 16 + c, then c
      uint32_t c;
      if constexpr (BF16) {
        const uint32_t y = i == 0 ? word[u] << 3 : word[u] >> (4 * i - 3);
        const uint32_t m = (y & 0x00780078u) | 0x41804180u;
        const __nv_bfloat162 k = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&m),
                                         __float2bfloat162_rn(16.f));
        c = *reinterpret_cast<const uint32_t*>(&k);
      } else {
        const uint32_t y = i < 2 ? word[u] << (6 - 4 * i) : word[u] >> (4 * i - 6);
        const uint32_t m = (y & 0x03C003C0u) | 0x4C004C00u;
        const __half2 k = __hsub2(*reinterpret_cast<const __half2*>(&m), __float2half2_rn(16.f));
        c = *reinterpret_cast<const uint32_t*>(&k);
      }
      v[i] = fma_16<BF16>(static_cast<uint16_t>(c), s, z);
      v[i + 4] = fma_16<BF16>(static_cast<uint16_t>(c >> 16), s, z);
    }
    if (u < rows)
      *reinterpret_cast<uint4*>(out + u * step) =
          make_uint4(pack2_finite<BF16>(v[0], v[1]), pack2_finite<BF16>(v[2], v[3]),
                     pack2_finite<BF16>(v[4], v[5]), pack2_finite<BF16>(v[6], v[7]));
  }
}

// ---------------------------------------------------------------------------
// Decode.  With the group's sums kept apart,
//   q.k^_j = sum_g s_jg (sum_{d in g} q_d c_jd) + z_jg (sum_{d in g} q_d)
//   out_d  = sum_j (p_j s_jg) c_jd + sum_j p_j z_jg          (d in group g)
// so the codes go into the tensor cores as they are, and no dequantised value is
// ever formed.  A nibble alone in the low byte of an fp16 number is a subnormal: in
// bits 0-3 the number c 2^-24, in bits 4-7 the number c 2^-20, both exact.  So one
// shift and four ands turn a word into four operand pairs, and the powers of two go
// into q (one half of its operand is 16 times larger) and into the final scaling.
// (With 16 + c and 256 + c in the mantissa instead -- two shifts, four and-ors whose
// second constant costs a register or an instruction, one more product for the sum
// of the weights -- the decode of B = 64 took 101 us.)
//
// Both products run in fp16 whatever the input type.  q is scaled by a power of two to
// a largest magnitude below 256, exact but for values 2^-22 of that and less.
// p s goes in as two fp16 numbers, high and low (22 bits): with one, a fifth of the bf16
// results of the B = 64 decode differed from those of fp32 weights (2 % with two), at
// 79 instead of 84 us.  p = 2^(y - ref), ref the running maximum of a head's scores; what
// goes in is p s F, F a power of two for each (head, group of 64 dimensions) that puts
// the largest p s so far at 2^4, so that a group keeps its bits however small its steps
// are beside the other group's.  fp16's range then ends 28 powers of two below a group's
// largest p s; a row that far below adds less than the sum's own rounding.  ref and F
// move only when some p s F passes 2^15 or some p 2^11 (so the accumulators are rarely
// rescaled), or when p z F, kept in fp32, passes 2^100.
//
// A warp takes 32 rows at a time in the fragment layout of mma.sync m16n8k16 (rows
// x heads and dimensions x heads, heads padded to 8): a thread's nibbles for one
// row are whole words of the row, and since the order of the contraction index is
// free, the pairs (i, i + 4) of a word serve as the operand's pairs.  V pairs two
// rows: one byte permute joins the halves of the two rows' words.  Each warp copies
// its own tiles into a ring of its own (cp.async, 16-byte chunks, no barrier but
// __syncwarp), two tiles ahead.
//
// PAIR (K = 128, at most four heads): the columns that would be padding take the
// second group of dimensions, so a thread works for one group only -- half the
// arithmetic between the products (scores, p s, sums), one exchange of the scores'
// halves.  In the product of a group's codes of V the other group's columns take this
// group's low parts, so the low parts cost no product of their own.
// ---------------------------------------------------------------------------
constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kTile = 32;        // rows per warp and iteration
constexpr int kHeads = 8;        // query heads per CTA (MMA n)
constexpr float kNoRef = -3.0e38f;     // reference of a warp that has seen no score
constexpr float kMaxWeight = 32768.f;  // largest p s F before ref and F are set anew
constexpr float kTarget = 4.f;         // log2 of the largest p s F then
constexpr float kPerPlain = 16.f;      // a p of 2^11 counts as much as a p s F of 2^15,
constexpr float kPerZero = 0x1p-85f;   // and a p z F of 2^100
// F <= 2^112, so that p F stays in fp32's range: groups whose steps are all below
// 2^-108 reach fp16's subnormals earlier.
constexpr float kLeastFactor = -126.f, kMostFactor = 112.f;  // log2

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1, float c0, float c1,
                                        float c2, float c3) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, "
      "{%4, %5, %6, %7}, {%8, %9}, {%10, %11, %12, %13};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
}

__device__ __forceinline__ void mma_f16_acc(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                            uint32_t a3, uint32_t b0, uint32_t b1) {
  mma_f16(d, a0, a1, a2, a3, b0, b1, d[0], d[1], d[2], d[3]);
}

__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// Nibbles N and N + 4 of a word as fp16 pairs: c 2^-24 for even N, c 2^-20 for odd.
struct CodePairs {
  uint32_t n[4];
};
__device__ __forceinline__ CodePairs code_pairs(uint32_t w) {
  const uint32_t hi = w >> 8;
  return {{w & 0x000F000Fu, w & 0x00F000F0u, hi & 0x000F000Fu, hi & 0x00F000F0u}};
}
constexpr float kUnitEven = 0x1p24f, kUnitOdd = 0x1p20f;  // what brings them back to c

// log2 of a normal power of two, and back.
__device__ __forceinline__ float log2_of(float f) {
  return static_cast<float>((__float_as_int(f) >> 23) - 127);
}
__device__ __forceinline__ float power_of_two(float e) {
  return __int_as_float((static_cast<int>(e) + 127) << 23);
}

template <int BYTES>
__device__ __forceinline__ void copy_async(uint32_t dst, const void* src) {
  if constexpr (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(BYTES)
                 : "memory");
}

template <int BYTES>
__device__ __forceinline__ void lds(const uint8_t* p, uint32_t* r) {
  if constexpr (BYTES == 8) {
    const uint2 x = *reinterpret_cast<const uint2*>(p);
    r[0] = x.x;
    r[1] = x.y;
  } else {
    r[0] = *reinterpret_cast<const uint32_t*>(p);
  }
}

constexpr int kStages = 3;  // ring of one warp: one tile in use, two in flight

template <int D>
struct KSmem {
  static constexpr int NG = D / 64;
  static constexpr int kCodes = kTile * D / 2;       // one plane's codes of a tile
  static constexpr int kParams = kTile * 4 * NG;
  static constexpr int kStage = 2 * (kCodes + kParams);  // K codes, V codes, K params, V params
  static constexpr int kWarp = kStages * kStage;
  static constexpr int kBytes = kWarps * kWarp;
  // after the ring: ref, l [kWarps][kHeads], log2 F [kWarps][kHeads][NG],
  // acc [kWarps][kHeads][D]
  static_assert(kWarps * kHeads * (D + 2 + NG) * 4 <= kBytes, "combine area");
};

// Where 16-byte chunk c of row r of a tile lies: 128-byte lines, the chunk's slot
// in the line turned by the line number, so that both the K reads (4 or 8 rows x
// 32 bytes) and the V reads (every other row) touch every bank once.
template <int D>
__device__ __forceinline__ int chunk_at(int r, int c) {
  if constexpr (D == 128)
    return (r >> 1) * 128 + (((((r & 1) << 2) | c) ^ (((r >> 1) & 3) << 1)) << 4);
  else
    return (r >> 2) * 128 + (((((r & 3) << 1) | c) ^ (((r >> 2) & 1) << 1)) << 4);
}

template <int D, bool BF16, bool ALIBI, bool PAIR>
__global__ void __launch_bounds__(kThreads, PAIR ? 4 : 3) kv4_decode_kernel(const Kv4DecodeArgs a) {
  using L = KSmem<D>;
  constexpr int NG = L::NG;  // groups of a row
  static_assert(!PAIR || NG == 2, "a column for each group and head");
  constexpr int NT = PAIR ? 1 : NG;  // groups a thread's columns stand for
  extern __shared__ __align__(128) uint8_t smem[];
  // The split varies slowest: whole chunks start first, the ragged last ones fill the end.
  const int split = blockIdx.z, b = blockIdx.y;
  const int kvh = blockIdx.x / a.head_blocks;
  const int g0 = (blockIdx.x - kvh * a.head_blocks) * kHeads;  // first head within the group
  const int heads = min(kHeads, a.group - g0);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int gid = lane >> 2, tig = lane & 3;
  // columns 2 tig, 2 tig + 1 of a product: heads hp, hp + 1 (of the thread's group)
  const int own = PAIR ? tig >> 1 : 0, hp = PAIR ? 2 * (tig & 1) : 2 * tig;
  const int n = a.kv_lens[b];
  const int h0 = kvh * a.group + g0;
  const bool ok = n >= 0 && n <= a.max_len;
  if (!ok && split == 0 && blockIdx.x == 0 && threadIdx.x == 0)
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
  const uint8_t* kp = static_cast<const uint8_t*>(a.k_params) + plane * (4 * NG);
  const uint8_t* vp = static_cast<const uint8_t*>(a.v_params) + plane * (4 * NG);
  uint8_t* const ring = smem + warp * L::kWarp;
  const uint32_t ring_u32 = smem_u32(ring);

  // One tile into stage `slot`; in the last tile, rows past the end take the last
  // row again (their weight is zero).
  constexpr int kPer = D / 32;  // 16-byte chunks of a row's codes; 8 or 16 rows a copy
  const int chunk0 = chunk_at<D>(lane / kPer, lane % kPer);
  auto fetch = [&](int tile, int slot) {
    const uint32_t st = ring_u32 + slot * L::kStage, to = st + chunk0;
    const uint32_t top = st + 2 * L::kCodes + lane * 4 * NG;
    if (tile + kTile <= s1) {
      const long long off = static_cast<long long>(tile) * (D / 2) + lane * 16;
      const long long poff = static_cast<long long>(tile + lane) * (4 * NG);
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        copy_async<16>(to + 512 * j, kc + off + 512 * j);
        copy_async<16>(to + 512 * j + L::kCodes, vc + off + 512 * j);
      }
      copy_async<4 * NG>(top, kp + poff);
      copy_async<4 * NG>(top + L::kParams, vp + poff);
    } else if (tile < s1) {
      const int left = s1 - 1 - tile;
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        const int r = min(lane / kPer + 32 / kPer * j, left);
        const long long off = static_cast<long long>(tile + r) * (D / 2) + lane % kPer * 16;
        copy_async<16>(to + 512 * j, kc + off);
        copy_async<16>(to + 512 * j + L::kCodes, vc + off);
      }
      const long long poff = static_cast<long long>(tile + min(lane, left)) * (4 * NG);
      copy_async<4 * NG>(top, kp + poff);
      copy_async<4 * NG>(top + L::kParams, vp + poff);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  int t = s0 + warp * kTile;
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) fetch(t + i * kWarps * kTile, i);

  // This thread's words within a stage: K rows gid + 8 i, 8 bytes at 8 tig of a
  // group; V rows 16 blk + 2 tig + (0, 1, 8, 9), 4 bytes at 4 gid.
  int k_at[NG], v_at[2][NG];
#pragma unroll
  for (int g = 0; g < NG; ++g) {
    k_at[g] = chunk_at<D>(gid, 2 * g + (tig >> 1)) + 8 * (tig & 1);
    v_at[0][g] = L::kCodes + chunk_at<D>(2 * tig, 2 * g + (gid >> 2)) + 4 * (gid & 3);
    v_at[1][g] = L::kCodes + chunk_at<D>(2 * tig + 1, 2 * g + (gid >> 2)) + 4 * (gid & 3);
  }

  // Q^T as the B operand (head gid), scaled; the sums of q that go with the zeros,
  // for this thread's two columns.  Column gid is head gid, or (PAIR) head gid % 4 with
  // the dimensions of group gid / 4 alone.
  uint32_t qb[NG][4][2];
  float qsum[NT][2], scl[2];
  bool wide;  // see `up` below; the same in the whole warp
  {
    const int head = PAIR ? gid & 3 : gid;
    const uint4* qrow = reinterpret_cast<const uint4*>(
        static_cast<const uint16_t*>(a.q) +
        (static_cast<long long>(b) * a.Hq + h0 + (head < heads ? head : 0)) * D + 16 * tig);
    uint32_t big2 = 0u;  // largest magnitudes, as pairs of bit patterns
#pragma unroll
    for (int g = 0; g < NG; ++g)
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        uint4 x = qrow[8 * g + w];  // dimensions 64 g + 16 tig + 8 w + 0..7
        if (head >= heads) x = make_uint4(0, 0, 0, 0);
        big2 = __vmaxu2(__vmaxu2(big2, __vmaxu2(x.x & 0x7fff7fffu, x.y & 0x7fff7fffu)),
                        __vmaxu2(x.z & 0x7fff7fffu, x.w & 0x7fff7fffu));
        qb[g][2 * w][0] = __byte_perm(x.x, x.z, 0x5410);  // pairs (d, d + 4)
        qb[g][2 * w][1] = __byte_perm(x.x, x.z, 0x7632);
        qb[g][2 * w + 1][0] = __byte_perm(x.y, x.w, 0x5410);
        qb[g][2 * w + 1][1] = __byte_perm(x.y, x.w, 0x7632);
      }
    big2 = __vmaxu2(big2, __shfl_xor_sync(0xffffffffu, big2, 1));
    big2 = __vmaxu2(big2, __shfl_xor_sync(0xffffffffu, big2, 2));
    const uint32_t big = max(big2 & 0xffffu, big2 >> 16);
    // 2^k with the largest |q| 2^k in [128, 256), 1 where q is zero or not finite (16
    // times that must fit fp16)
    int k = 0;
    if (BF16 && big != 0u && big < 0x7f80u) k = 134 - static_cast<int>(big >> 7);
    if (!BF16 && big != 0u && big < 0x7c00u) k = min(22 - static_cast<int>(big >> 10), 15);
    k = min(max(k, -126), 126);
    const float f = __int_as_float((127 + k) << 23), inv = __int_as_float((127 - k) << 23);
    float col_sum = 0.f;  // PAIR: of the column's own group
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      float sum = 0.f;
#pragma unroll
      for (int ks = 0; ks < 4; ++ks)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          if constexpr (BF16)
            qb[g][ks][e] = pack2<false>(step_of<true>(qb[g][ks][e]) * f,
                                        zero_of<true>(qb[g][ks][e]) * f);
          __half2 x = *reinterpret_cast<const __half2*>(&qb[g][ks][e]);
          if constexpr (!BF16) x = __hmul2(x, __float2half2_rn(f));
          sum += __low2float(x) + __high2float(x);
          if (e == 0) x = __hmul2(x, __float2half2_rn(kUnitEven / kUnitOdd));
          qb[g][ks][e] = *reinterpret_cast<const uint32_t*>(&x);
          if (PAIR && (gid >> 2) != g) qb[g][ks][e] = 0u;
        }
#pragma unroll
      for (int o = 1; o <= 2; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      if (PAIR && (gid >> 2) == g) col_sum = sum;
      if constexpr (!PAIR) {
#pragma unroll
        for (int e = 0; e < 2; ++e) qsum[g][e] = __shfl_sync(0xffffffffu, sum, 8 * tig + 4 * e);
      }
    }
    if constexpr (PAIR) {
#pragma unroll
      for (int e = 0; e < 2; ++e) qsum[0][e] = __shfl_sync(0xffffffffu, col_sum, 8 * tig + 4 * e);
    }
    // Scores are summed in units of kUnitOdd, which goes into their scale (and out of the
    // sums of q), so that s sum(q c) stays in range for any step; with a q so large (about
    // 2^107) that its scale would leave the range, they take it tile by tile.
    wide = __any_sync(0xffffffffu, inv > 0x1p100f);
    const float up = wide ? 1.f : kUnitOdd;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      scl[e] = __shfl_sync(0xffffffffu, inv, 8 * tig + 4 * e) * up * a.scale_log2;
#pragma unroll
      for (int g = 0; g < NT; ++g) qsum[g][e] *= 1.f / kUnitOdd;
    }
  }
  float slope[2] = {0.f, 0.f};
  if constexpr (ALIBI) {
#pragma unroll
    for (int e = 0; e < 2; ++e)
      slope[e] = exp2f(-8.0f * static_cast<float>(h0 + hp + e + 1) / a.Hq) * kLog2e;
  }

  float ref[2] = {kNoRef, kNoRef}, l_part[2] = {0.f, 0.f};
  float fac[NT][2], zacc[NT][2], acc[D / 16][4];
#pragma unroll
  for (int g = 0; g < NT; ++g) {
    fac[g][0] = fac[g][1] = 1.f;
    zacc[g][0] = zacc[g][1] = 0.f;
  }
#pragma unroll
  for (int i = 0; i < D / 16; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[i][e] = 0.f;

  // Scores of the tile in `slot`, log2 units.
  auto score = [&](int slot, float(&y)[2][4]) {
    const uint8_t* st = ring + slot * L::kStage;
    float sc[2][NT][4];
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      uint32_t kw[4][2];
#pragma unroll
      for (int i = 0; i < 4; ++i) lds<8>(st + k_at[g] + i * 4 * D, kw[i]);
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        CodePairs c[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) c[i] = code_pairs(kw[i][w]);
#pragma unroll
        for (int half = 0; half < 2; ++half)
#pragma unroll
          for (int blk = 0; blk < 2; ++blk) {
            const CodePairs &lo = c[2 * blk], &hi = c[2 * blk + 1];
            const uint32_t(&q2)[2] = qb[g][2 * w + half];
            float(&s4)[4] = sc[blk][PAIR ? 0 : g];
            if (w + half == 0 && (!PAIR || g == 0))
              mma_f16(s4, lo.n[0], hi.n[0], lo.n[1], hi.n[1], q2[0], q2[1], 0.f, 0.f, 0.f, 0.f);
            else
              mma_f16_acc(s4, lo.n[2 * half], hi.n[2 * half], lo.n[2 * half + 1],
                          hi.n[2 * half + 1], q2[0], q2[1]);
          }
      }
    }
    uint32_t kq[4][NT];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      lds<4 * NT>(st + 2 * L::kCodes + (gid + 8 * i) * 4 * NG + 4 * own, kq[i]);
#pragma unroll
    for (int blk = 0; blk < 2; ++blk) {
#pragma unroll
      for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int g = 0; g < NT; ++g) {
          const float s = step_of<BF16>(kq[2 * blk + r][g]);
          const float z = zero_of<BF16>(kq[2 * blk + r][g]);
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float& yy = y[blk][2 * r + e];
            yy = fmaf(s, sc[blk][g][2 * r + e], g == 0 ? z * qsum[g][e] : fmaf(z, qsum[g][e], yy));
          }
        }
    }
    if constexpr (PAIR) {  // the other group's share, two columns of tig on
#pragma unroll
      for (int blk = 0; blk < 2; ++blk)
#pragma unroll
        for (int e = 0; e < 4; ++e) y[blk][e] += __shfl_xor_sync(0xffffffffu, y[blk][e], 2);
    }
    // The scale is taken here and not together with the reference: the two roundings of
    // y scl, here and in a fused y scl - ref, are 2^-24 y apart, which past scores of
    // 2^24 is no longer a weight near one.
#pragma unroll
    for (int blk = 0; blk < 2; ++blk)
#pragma unroll
      for (int e = 0; e < 4; ++e) y[blk][e] *= scl[e & 1];
    if (wide) {
#pragma unroll
      for (int blk = 0; blk < 2; ++blk)
#pragma unroll
        for (int e = 0; e < 4; ++e) y[blk][e] *= kUnitOdd;
    }
  };

  int slot = 0;
  for (; t < s1; t += kWarps * kTile) {
    asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
    __syncwarp();  // the tile is there for every lane, and the one before is read
    fetch(t + (kStages - 1) * kWarps * kTile, slot == 0 ? kStages - 1 : slot - 1);
    const uint8_t* st = ring + slot * L::kStage;
    float y[2][4];
    score(slot, y);
    slot = slot == kStages - 1 ? 0 : slot + 1;
    uint32_t vq[4][NT];  // (s, z) of the V rows gid + 8 i
#pragma unroll
    for (int i = 0; i < 4; ++i)
      lds<4 * NT>(st + 2 * L::kCodes + L::kParams + (gid + 8 * i) * 4 * NG + 4 * own, vq[i]);
    const bool last = t + kTile > s1;
    if constexpr (ALIBI) {
      // y - slope (n - 1 - row)
#pragma unroll
      for (int blk = 0; blk < 2; ++blk)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          y[blk][e] = fmaf(
              -slope[e & 1],
              static_cast<float>(n - 1 - min(t + 16 * blk + 8 * (e >> 1) + gid, s1 - 1)),
              y[blk][e]);
    }
    if (a.scores != nullptr) {  // kept for the gathered weights
#pragma unroll
      for (int e = 0; e < 2; ++e)
        if (own == 0 && hp + e < heads) {
          float* out = a.scores + (static_cast<long long>(b) * a.Hq + h0 + hp + e) *
                                      a.score_stride + t + gid;
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (t + 8 * i + gid < s1) out[8 * i] = y[i >> 1][2 * (i & 1) + e];
        }
    }
    // Weights of the tile against the present reference: p s F in fp16, and the sums
    // of p, p s F and p z F (an overflow shows in a sum of numbers >= 0).
    uint32_t pk[2][NT][2][2];  // [..][high, low]
    float sum[2], heavy[2], zsum[NT][2];
    auto weigh = [&] {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        sum[e] = heavy[e] = 0.f;
#pragma unroll
        for (int g = 0; g < NT; ++g) zsum[g][e] = 0.f;
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {  // row gid + 8 i
        float p[2];
#pragma unroll
        for (int e = 0; e < 2; ++e)
          p[e] = ex2(y[i >> 1][2 * (i & 1) + e] - ref[e]);
        if (last) {
          asm volatile("");  // a branch, not selects in every tile
          if (t + 8 * i + gid >= s1) p[0] = p[1] = 0.f;
        }
#pragma unroll
        for (int g = 0; g < NT; ++g) {
          const float s = step_of<BF16>(vq[i][g]), z = zero_of<BF16>(vq[i][g]);
          const float pf0 = p[0] * fac[g][0], pf1 = p[1] * fac[g][1];
          const float ps0 = pf0 * s, ps1 = pf1 * s;
          heavy[0] += ps0;
          heavy[1] += ps1;
          zsum[g][0] = fmaf(pf0, z, zsum[g][0]);
          zsum[g][1] = fmaf(pf1, z, zsum[g][1]);
          uint32_t(&out)[2] = pk[i >> 1][g][i & 1];
          out[0] = pack2<false>(ps0, ps1);
          constexpr uint16_t kMinusOne = 0xBC00;
          out[1] = pack2<false>(fma_16<false>(static_cast<uint16_t>(out[0]), kMinusOne, ps0),
                                fma_16<false>(static_cast<uint16_t>(out[0] >> 16), kMinusOne, ps1));
        }
        sum[0] += p[0];
        sum[1] += p[1];
      }
    };
    weigh();
    // One sum tells of them all (a NaN hides the others, so it counts as an overflow).
    float over = heavy[0] + heavy[1] + kPerPlain * (sum[0] + sum[1]);
#pragma unroll
    for (int g = 0; g < NT; ++g)
      over = fmaf(kPerZero, fabsf(zsum[g][0]) + fabsf(zsum[g][1]), over);
    if (__any_sync(0xffffffffu, !(over <= kMaxWeight))) {
      // Set ref and F anew.  A row whose step is small beside its zero counts with
      // 2^-12 of the zero, so that p z F stays in range too.
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        auto over_rows = [](float v) {  // the warp's rows of a column
          v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
          v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
          return fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16));
        };
        float v = neg_inf();
#pragma unroll
        for (int i = 0; i < 4; ++i) v = fmaxf(v, y[i >> 1][2 * (i & 1) + e]);
        const float r_new = fmaxf(ref[e], over_rows(v));
        const float drop = r_new == ref[e] ? 0.f : ref[e] - r_new;
        l_part[e] *= ex2(drop);
#pragma unroll
        for (int g = 0; g < NT; ++g) {
          float m = neg_inf();  // log2 of the largest p s against the new reference
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float mag = fmaxf(step_of<BF16>(vq[i][g]),
                                    fabsf(zero_of<BF16>(vq[i][g])) * 0x1p-12f);
            m = fmaxf(m, (y[i >> 1][2 * (i & 1) + e] - r_new) + __log2f(mag));
          }
          const float f_old = log2_of(fac[g][e]);
          m = fmaxf(over_rows(m), drop + (kTarget - f_old));
          const float f_new = fminf(fmaxf(rintf(kTarget - m), kLeastFactor), kMostFactor);
          fac[g][e] = power_of_two(f_new);
          const float alpha = ex2(drop + (f_new - f_old));
          // PAIR: this thread's columns of the other group's products hold its low parts
          const float other = PAIR ? __shfl_xor_sync(0xffffffffu, alpha, 2) : alpha;
          zacc[g][e] *= alpha;
#pragma unroll
          for (int i = 0; i < D / 16; ++i) {
            if (!PAIR && (i >> 2) != g) continue;
            const float by = PAIR && (i >> 2) != own ? other : alpha;
            acc[i][e] *= by;
            acc[i][e + 2] *= by;
          }
        }
        ref[e] = r_new;
      }
      weigh();
    }
    l_part[0] += sum[0];
    l_part[1] += sum[1];
#pragma unroll
    for (int g = 0; g < NT; ++g) {
      zacc[g][0] += zsum[g][0];
      zacc[g][1] += zsum[g][1];
    }
    // B operands of the products with V's codes.  PAIR: of a group, the high parts in its
    // own columns and the low parts in the other's.
    constexpr int kOps = PAIR ? 1 : 2;
    uint32_t pb[2][NG][kOps][2];
#pragma unroll
    for (int blk = 0; blk < 2; ++blk)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        if constexpr (PAIR) {
          const uint32_t high = pk[blk][0][r][0];
          const uint32_t low = __shfl_xor_sync(0xffffffffu, pk[blk][0][r][1], 2);
          pb[blk][0][0][r] = movmatrix_trans(own == 0 ? high : low);
          pb[blk][1][0][r] = movmatrix_trans(own == 0 ? low : high);
        } else {
#pragma unroll
          for (int g = 0; g < NG; ++g)
#pragma unroll
            for (int op = 0; op < kOps; ++op)
              pb[blk][g][op][r] = movmatrix_trans(pk[blk][g][r][op]);
        }
      }
#pragma unroll
    for (int g = 0; g < NG; ++g) {
#pragma unroll
      for (int blk = 0; blk < 2; ++blk) {
        // rows 2 tig, 2 tig + 1 (first pair) and + 8 (second): words of 8 dimensions
        uint32_t w0, w1, w2, w3;
        lds<4>(st + v_at[0][g] + blk * 8 * D, &w0);
        lds<4>(st + v_at[1][g] + blk * 8 * D, &w1);
        lds<4>(st + v_at[0][g] + blk * 8 * D + 4 * D, &w2);
        lds<4>(st + v_at[1][g] + blk * 8 * D + 4 * D, &w3);
        const CodePairs xa = code_pairs(__byte_perm(w0, w1, 0x5410));
        const CodePairs ya = code_pairs(__byte_perm(w0, w1, 0x7632));
        const CodePairs xb = code_pairs(__byte_perm(w2, w3, 0x5410));
        const CodePairs yb = code_pairs(__byte_perm(w2, w3, 0x7632));
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int op = 0; op < kOps; ++op)
            mma_f16_acc(acc[4 * g + i], xa.n[i], ya.n[i], xb.n[i], yb.n[i], pb[blk][g][op][0],
                        pb[blk][g][op][1]);
      }
    }
  }

#pragma unroll
  for (int e = 0; e < 2; ++e)
#pragma unroll
    for (int o = 4; o <= 16; o <<= 1) {
      l_part[e] += __shfl_xor_sync(0xffffffffu, l_part[e], o);
#pragma unroll
      for (int g = 0; g < NT; ++g) zacc[g][e] += __shfl_xor_sync(0xffffffffu, zacc[g][e], o);
    }
  asm volatile("cp.async.wait_all;" ::: "memory");
  __syncthreads();  // the rings are read: their memory joins the warps' states
  float* c_ref = reinterpret_cast<float*>(smem);
  float* c_l = c_ref + kWarps * kHeads;
  float* c_fac = c_l + kWarps * kHeads;
  float* c_acc = c_fac + kWarps * kHeads * NG;
  if (gid == 0) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int at = warp * kHeads + hp + e;
      if (own == 0) {
        c_ref[at] = ref[e];
        c_l[at] = l_part[e];
      }
#pragma unroll
      for (int g = 0; g < NT; ++g) c_fac[at * NG + own + g] = log2_of(fac[g][e]);
    }
  }
#pragma unroll
  for (int i = 0; i < D / 16; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) {  // tile i: dimension 64 (i/4) + 8 gid + i % 4 (+ 4)
      float x = acc[i][e];
      if constexpr (PAIR) x += __shfl_xor_sync(0xffffffffu, x, 2);  // high and low parts
      if (!PAIR || own == (i >> 2))
        c_acc[(warp * kHeads + hp + (e & 1)) * D + 64 * (i >> 2) + 8 * gid + (i & 3) +
              4 * (e >> 1)] =
            fmaf(x, (i & 1) ? kUnitOdd : kUnitEven, zacc[PAIR ? 0 : i >> 2][e & 1]);
    }
  __syncthreads();

  for (int idx = threadIdx.x; idx < heads * D; idx += kThreads) {
    const int g = idx / D, d = idx - g * D;
    float mx = kNoRef, top = neg_inf(), unit[kWarps];
#pragma unroll
    for (int w = 0; w < kWarps; ++w) mx = fmaxf(mx, c_ref[w * kHeads + g]);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {  // log2 of what one of acc stands for, against mx
      unit[w] = (c_ref[w * kHeads + g] - mx) - c_fac[(w * kHeads + g) * NG + d / 64];
      top = fmaxf(top, unit[w]);
    }
    float lsum = 0.f, o = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {  // factors of 1 if no warp has a reference
      lsum = fmaf(ex2(c_ref[w * kHeads + g] - mx), c_l[w * kHeads + g], lsum);
      o = fmaf(ex2(unit[w] - top), c_acc[(w * kHeads + g) * D + d], o);
    }
    const long long row = static_cast<long long>(b) * a.Hq + h0 + g;
    // (a NaN stays a NaN; top lies in -kMostFactor .. -kLeastFactor)
    const float val = lsum == 0.f ? 0.f : o / lsum * ex2(top);
    const float lse2 = lsum == 0.f ? neg_inf() : mx + log2f(lsum);
    if (a.part_o == nullptr) {  // the only split
      static_cast<uint16_t*>(a.out)[row * D + d] = to_16_finite<BF16>(val);
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
  return sum == 0.f ? neg_inf() : base + log2f(sum);
}

template <int D, bool BF16>
__global__ void __launch_bounds__(256) kv4_merge_kernel(const Kv4DecodeArgs a) {
  __shared__ float s_lse[256];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  grid_dependency_wait();
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
      out[lane + 32 * i] = to_16_finite<BF16>(o[i]);
    if (lane == 0 && a.lse != nullptr) a.lse[row] = lse2 * kLn2;
    return;
  }
  // weights: four consecutive rows a thread (score_stride is a multiple of 4)
  const int blk = blockIdx.x - a.merge_blocks;
  const int bh = blk / a.weight_blocks, c0 = (blk - bh * a.weight_blocks) * kWeightRows;
  const int b = bh / a.Hkv, kvh = bh - b * a.Hkv;
  const int n = a.kv_lens[b];
  if (n < 0 || n > a.max_len) return;
  const long long wrow = static_cast<long long>(bh) * a.cap;
  const int ns = (n + a.chunk - 1) / a.chunk;
  const int j0 = c0 + 4 * threadIdx.x;
  float sum[4] = {0.f, 0.f, 0.f, 0.f}, w_in[4] = {0.f, 0.f, 0.f, 0.f};
  const long long row0 = static_cast<long long>(b) * a.Hq + kvh * a.group;
  if (a.w_in != nullptr) {
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (j0 + u < n) w_in[u] = a.w_in[wrow + j0 + u];
  }
  constexpr int kAhead = 4;  // heads whose scores are fetched before their lse is joined
  for (int g0 = 0; g0 < a.group && c0 < n; g0 += 256) {
    const int gn = min(256, a.group - g0);
    const float* x = a.scores + (row0 + g0) * a.score_stride + j0;
    float4 v[kAhead];
#pragma unroll
    for (int g = 0; g < kAhead; ++g)
      v[g] = g < gn && j0 < n ? *reinterpret_cast<const float4*>(x + g * a.score_stride)
                              : make_float4(0.f, 0.f, 0.f, 0.f);
    __syncthreads();
    for (int g = warp; g < gn; g += 8) {
      const float l = merged_lse2(a.part_lse + (row0 + g0 + g) * a.max_splits, ns, lane);
      if (lane == 0) s_lse[g] = l;
    }
    __syncthreads();
    auto add = [&](const float4& y, float l) {
      if (l == neg_inf()) return;
      sum[0] += ex2(y.x - l);
      sum[1] += ex2(y.y - l);
      sum[2] += ex2(y.z - l);
      sum[3] += ex2(y.w - l);
    };
#pragma unroll
    for (int g = 0; g < kAhead; ++g)
      if (g < gn) add(v[g], s_lse[g]);
    if (j0 < n)
      for (int g = kAhead; g < gn; ++g)
        add(*reinterpret_cast<const float4*>(x + g * a.score_stride), s_lse[g]);
  }
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const int j = j0 + u;
    if (j < min(a.cap, c0 + kWeightRows))
      a.w_out[wrow + j] = j < n ? sum[u] + w_in[u] : 0.f;
  }
}

template <int D, bool BF16, bool ALIBI, bool PAIR>
cudaError_t decode_run(const Kv4DecodeArgs& a, dim3 grid, cudaStream_t stream) {
  constexpr auto kern = kv4_decode_kernel<D, BF16, ALIBI, PAIR>;
  const cudaError_t e = set_smem_once<kern>(KSmem<D>::kBytes);
  if (e != cudaSuccess) return e;
  kern<<<grid, kThreads, KSmem<D>::kBytes, stream>>>(a);
  return cudaGetLastError();
}

template <int D, bool BF16>
cudaError_t decode_t(const Kv4DecodeArgs& a, bool alibi, cudaStream_t stream) {
  if (a.max_splits > 0) {
    const dim3 grid(a.Hkv * a.head_blocks, a.B, a.max_splits);
    // Up to four heads at K = 128: a column for each (group, head) (84 us at B = 64,
    // 82 us for four long contexts with weights; without, 96 and 90 us).
    cudaError_t e;
    if (D == 128 && a.group <= 4)
      e = alibi ? decode_run<D, BF16, true, D == 128>(a, grid, stream)
                : decode_run<D, BF16, false, D == 128>(a, grid, stream);
    else
      e = alibi ? decode_run<D, BF16, true, false>(a, grid, stream)
                : decode_run<D, BF16, false, false>(a, grid, stream);
    if (e != cudaSuccess) return e;
  }
  if (a.part_o == nullptr && a.max_splits > 0 && a.w_out == nullptr) return cudaSuccess;
  const long long blocks =
      a.merge_blocks + static_cast<long long>(a.B) * a.Hkv * a.weight_blocks;
  if (blocks == 0) return cudaSuccess;
  return launch_after(kv4_merge_kernel<D, BF16>, dim3(static_cast<unsigned>(blocks)), 256, 0,
                      stream, a);
}

}  // namespace

int kv4_weight_rows() { return kWeightRows; }
int kv4_row_group() { return kRowGroup; }

cudaError_t launch_kv4_append(const Kv4AppendArgs& a, int head_dim, bool bf16,
                              cudaStream_t stream) {
  const unsigned per = kRowThreads * 8 / head_dim;  // row groups a block
  const dim3 grid((a.order.total + per - 1) / per, 2);
  if (head_dim == 64 && !bf16) kv4_append_kernel<64, false><<<grid, kRowThreads, 0, stream>>>(a);
  else if (head_dim == 64) kv4_append_kernel<64, true><<<grid, kRowThreads, 0, stream>>>(a);
  else if (!bf16) kv4_append_kernel<128, false><<<grid, kRowThreads, 0, stream>>>(a);
  else kv4_append_kernel<128, true><<<grid, kRowThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_kv4_read(const Kv4ReadArgs& a, int head_dim, bool bf16, cudaStream_t stream) {
  const unsigned per = kRowThreads * 8 / head_dim;  // row groups a block
  const dim3 grid((a.order.total + per - 1) / per, 2);
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
