// mea_evict_sm100.cu -- eviction from a cache by gathered attention weight.
//
// Of a sequence's n rows a kv head keeps, when n > budget, the newest `recent`
// and the budget - recent heaviest of the others (equal weights: the lowest row;
// NaN: as the lightest), in their old order.  Two launches:
//   evict_select  a block (or a cluster) per (sequence, kv head): the weight of the last row
//                 to keep by three counting passes over 11, 11 and 10 bits of an
//                 order-preserving integer, then the kept row numbers by counting
//                 in row order (ballots and a scan: no atomic decides an order);
//   evict_move    rows kept[r] -> r of every plane.  In place a block owns a
//                 column strip of one (sequence, head) and walks the tiles of
//                 rows upwards: kept[r] >= r, so a tile's sources lie at or past
//                 it, and one barrier between a tile's loads and its stores is
//                 all the order there is to keep.  Into another cache, blocks
//                 also share out the rows.
#include <cooperative_groups.h>
#include <math.h>

#include "mea_cache_internal.h"
#include "sm100.cuh"

namespace mea {
namespace {

namespace cg = cooperative_groups;

constexpr int kSelThreads = 1024;
constexpr int kSelTile = 4 * kSelThreads;
constexpr int kSelHeld = 8;  // keys a thread holds: up to 8192 rows are read once
constexpr int kBins = 2048;

// An unsigned integer ordered as the float is; NaN below everything, -0 as 0.
__device__ __forceinline__ uint32_t order_key(float x) {
  if (x != x) return 0u;
  const uint32_t u = __float_as_uint(x + 0.f);
  return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

// The a.parts CTAs of a cluster take a (sequence, kv head)'s rows in equal runs, add
// up their counts in each other's shared memory and all find the same last key.
template <bool CLUSTER>
__global__ void __launch_bounds__(kSelThreads, CLUSTER ? 1 : 2)
    evict_select_kernel(const __grid_constant__ EvictArgs a) {
  __shared__ uint32_t hist[kBins];
  __shared__ uint32_t whole[CLUSTER ? kBins : 1];  // the cluster's sum of hist
  __shared__ uint32_t warp_sum[32];
  __shared__ uint32_t s_bin, s_above;
  __shared__ uint32_t counts[128];
  __shared__ uint32_t s_rows[2];  // this CTA's rows above the last key, and equal to it
  const int parts = CLUSTER ? a.parts : 1;
  const int bh = blockIdx.x / parts, part = blockIdx.x - bh * parts;
  const int b = bh / a.Hkv, kvh = bh - b * a.Hkv;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int n = a.lens[b];
  int32_t* kept = a.kept + static_cast<long long>(bh) * a.budget;
  if (n < 0 || n > a.cap) {
    if (part != 0) return;
    if (kvh == 0 && tid == 0) {
      record_error(a.status, kErrInvalidArg);
      a.new_lens[b] = 0;
    }
    for (int r = tid; r < a.budget; r += kSelThreads) kept[r] = -1;
    return;
  }
  if (kvh == 0 && part == 0 && tid == 0) a.new_lens[b] = min(n, a.budget);
  if (n <= a.budget) {
    for (int r = part * kSelThreads + tid; r < a.budget; r += parts * kSelThreads)
      kept[r] = r < n ? r : -1;
    return;
  }
  const int rows = n - a.recent;         // candidates
  const int take = a.budget - a.recent;  // < rows
  for (int r = part * kSelThreads + tid; r < a.recent; r += parts * kSelThreads)
    kept[take + r] = rows + r;
  if (take == 0) return;
  // this CTA's rows [lo, lo + m); every exit above is the whole cluster's
  const int per = (rows + parts - 1) / parts;
  const int lo = min(rows, part * per), m = min(rows, lo + per) - lo;
  const float* w = a.weights + static_cast<long long>(bh) * a.cap + lo;
  [[maybe_unused]] cg::cluster_group cluster = cg::this_cluster();

  const bool held = m <= kSelHeld * kSelThreads;
  uint32_t mine[kSelHeld];
  if (held) {
#pragma unroll
    for (int u = 0; u < kSelHeld; ++u) {
      const int j = u * kSelThreads + tid;
      mine[u] = j < m ? order_key(w[j]) : 0u;
    }
  }
  uint32_t prefix = 0, need = take;  // rows still to find among those with this prefix
#pragma unroll 1
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
    const uint32_t mask = pass == 2 ? 1023u : 2047u;
    const int above = pass == 0 ? 0 : pass == 1 ? 21 : 10;  // bits already fixed start here
    for (int i = tid; i < kBins; i += kSelThreads) hist[i] = 0;
    __syncthreads();
    auto count = [&](uint32_t key) {
      if (pass == 0 || (key >> above) == prefix) atomicAdd(&hist[(key >> shift) & mask], 1u);
    };
    if (held) {
#pragma unroll
      for (int u = 0; u < kSelHeld; ++u)
        if (u * kSelThreads + tid < m) count(mine[u]);
    } else {
      for (int j0 = tid; j0 < m; j0 += kSelHeld * kSelThreads) {
        float x[kSelHeld];  // all in flight before the first is counted
#pragma unroll
        for (int u = 0; u < kSelHeld; ++u)
          x[u] = j0 + u * kSelThreads < m ? w[j0 + u * kSelThreads] : 0.f;
#pragma unroll
        for (int u = 0; u < kSelHeld; ++u)
          if (j0 + u * kSelThreads < m) count(order_key(x[u]));
      }
    }
    __syncthreads();
    if constexpr (CLUSTER) {
      cluster.sync();  // all have counted
      for (int i = tid; i < kBins; i += kSelThreads) {
        uint32_t sum = 0;
        for (int r = 0; r < parts; ++r) sum += cluster.map_shared_rank(hist, r)[i];
        whole[i] = sum;
      }
      cluster.sync();  // all have read: hist may be cleared
    }
    const uint32_t* bins = CLUSTER ? whole : hist;
    // bins from the top: thread t holds bins 2047 - 2t and 2046 - 2t
    const uint32_t c0 = bins[kBins - 1 - 2 * tid], c1 = bins[kBins - 2 - 2 * tid];
    uint32_t sum = c0 + c1;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += y;
    }
    if (lane == 31) warp_sum[warp] = sum;
    __syncthreads();
    uint32_t before = lane < warp ? warp_sum[lane] : 0u;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) before += __shfl_xor_sync(0xffffffffu, before, o);
    const uint32_t excl = before + sum - c0 - c1;  // keys in higher bins
    if (excl < need && need <= excl + c0) {
      s_bin = kBins - 1 - 2 * tid;
      s_above = excl;
    } else if (excl + c0 < need && need <= excl + c0 + c1) {
      s_bin = kBins - 2 - 2 * tid;
      s_above = excl + c0;
    }
    __syncthreads();
    prefix = pass == 0 ? s_bin : pass == 1 ? (prefix << 11) | s_bin : (prefix << 10) | s_bin;
    need -= s_above;
    __syncthreads();
  }

  // Rows above the key `prefix` are kept, and the first `need` equal to it.
  uint32_t base = 0, base_eq = 0;  // rows before this tile: above, and equal
  if constexpr (CLUSTER) {
    if (tid < 2) s_rows[tid] = 0;
    __syncthreads();
    uint32_t above = 0, equal = 0;
    auto tally = [&](uint32_t key) {
      above += key > prefix;
      equal += key == prefix;
    };
    if (held) {
#pragma unroll
      for (int u = 0; u < kSelHeld; ++u)
        if (u * kSelThreads + tid < m) tally(mine[u]);
    } else {
      for (int j = tid; j < m; j += kSelThreads) tally(order_key(w[j]));
    }
    above = __reduce_add_sync(0xffffffffu, above);
    equal = __reduce_add_sync(0xffffffffu, equal);
    if (lane == 0) {  // whole numbers: the order of the additions does not matter
      atomicAdd(&s_rows[0], above);
      atomicAdd(&s_rows[1], equal);
    }
    cluster.sync();
    for (int r = 0; r < part; ++r) {
      base += cluster.map_shared_rank(s_rows, r)[0];
      base_eq += cluster.map_shared_rank(s_rows, r)[1];
    }
    cluster.sync();  // no CTA ends while another reads its counts
  }
  auto place = [&](int t0, const uint32_t(&keys)[4]) {
    uint32_t gt[4], eq[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int j = t0 + u * kSelThreads + tid;
      const uint32_t key = keys[u];
      gt[u] = __ballot_sync(0xffffffffu, j < m && key > prefix);
      eq[u] = __ballot_sync(0xffffffffu, j < m && key == prefix);
      if (lane == 0) counts[u * 32 + warp] = __popc(gt[u]) | (__popc(eq[u]) << 16);
    }
    __syncthreads();
    if (warp == 0) {  // exclusive scan of the 128 counts (at most 4096 each: no carry)
      uint32_t v[4], run = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[i] = run;
        run += counts[lane * 4 + i];
      }
      uint32_t incl = run;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) counts[lane * 4 + i] = v[i] + incl - run;
      if (lane == 31) warp_sum[0] = incl;
    }
    __syncthreads();
    const uint32_t lower = (1u << lane) - 1u;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const uint32_t c = counts[u * 32 + warp];
      const uint32_t ngt = base + (c & 0xffffu) + __popc(gt[u] & lower);
      const uint32_t neq = base_eq + (c >> 16) + __popc(eq[u] & lower);
      const bool is_eq = (eq[u] >> lane) & 1u;
      if (((gt[u] >> lane) & 1u) || (is_eq && neq < need))
        kept[ngt + min(neq, need)] = lo + t0 + u * kSelThreads + tid;
    }
    base += warp_sum[0] & 0xffffu;
    base_eq += warp_sum[0] >> 16;
    __syncthreads();
  };
  static_assert(kSelHeld == 8, "two tiles are held");
  if (held) {
    place(0, {mine[0], mine[1], mine[2], mine[3]});
    if (m > kSelTile) place(kSelTile, {mine[4], mine[5], mine[6], mine[7]});
  } else {
#pragma unroll 1
    for (int t0 = 0; t0 < m; t0 += kSelTile) {
      uint32_t keys[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int j = t0 + u * kSelThreads + tid;
        keys[u] = j < m ? order_key(w[j]) : 0u;
      }
      place(t0, keys);
    }
  }
}

constexpr int kMoveThreads = 256;

template <int A>
struct Word;
template <>
struct Word<16> { uint32_t v[4]; };
template <>
struct Word<8> { uint32_t v[2]; };
template <>
struct Word<4> { uint32_t v[1]; };

// Plain (not read-only-cache) accesses: the planes may be rewritten in place.
template <int A>
__device__ __forceinline__ Word<A> load_word(const uint8_t* p) {
  Word<A> w;
  if constexpr (A == 16)
    asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(w.v[0]), "=r"(w.v[1]), "=r"(w.v[2]), "=r"(w.v[3]) : "l"(p) : "memory");
  else if constexpr (A == 8)
    asm volatile("ld.global.v2.u32 {%0, %1}, [%2];"
                 : "=r"(w.v[0]), "=r"(w.v[1]) : "l"(p) : "memory");
  else
    asm volatile("ld.global.u32 %0, [%1];" : "=r"(w.v[0]) : "l"(p) : "memory");
  return w;
}

template <int A>
__device__ __forceinline__ void store_word(uint8_t* p, const Word<A>& w) {
  if constexpr (A == 16)
    *reinterpret_cast<uint4*>(p) = make_uint4(w.v[0], w.v[1], w.v[2], w.v[3]);
  else if constexpr (A == 8)
    *reinterpret_cast<uint2*>(p) = make_uint2(w.v[0], w.v[1]);
  else
    *reinterpret_cast<uint32_t*>(p) = w.v[0];
}

// Rows [r_begin, r_end) of one column piece.  In place, a tile's sources lie at or
// past the tile, so one barrier between its loads and its stores orders everything;
// the next tile's loads go out before this one's stores.
template <int A, bool IN_PLACE>
__device__ __forceinline__ void move_rows(const EvictPlane& pl, const uint8_t* src, uint8_t* dst,
                                          const int32_t* kept, int r_begin, int r_end) {
  constexpr int U = IN_PLACE ? 8 : 4;
  const int lanes = pl.piece_bytes / A;
  const int part = threadIdx.x % lanes, sub = threadIdx.x / lanes;
  const int per = kMoveThreads / lanes;  // rows per unroll step
  const bool mine = sub < per;
  src += part * A;
  dst += part * A;
  if constexpr (!IN_PLACE) {
    for (int r0 = r_begin; r0 < r_end; r0 += per * U) {
      int32_t from[U];
      Word<A> w[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int r = r0 + u * per + sub;
        from[u] = mine && r < r_end ? kept[r] : -1;
      }
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (from[u] >= 0) w[u] = load_word<A>(src + from[u] * pl.src_s[1]);
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (from[u] >= 0) store_word<A>(dst + (r0 + u * per + sub) * pl.dst_s[1], w[u]);
    }
  } else {
    Word<A> cur[U], nxt[U];
    auto fetch = [&](Word<A>(&w)[U], int r0) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int r = r0 + u * per + sub;
        if (mine && r < r_end) w[u] = load_word<A>(src + kept[r] * pl.src_s[1]);
      }
    };
    fetch(cur, r_begin);
    for (int r0 = r_begin; r0 < r_end; r0 += per * U) {
      fetch(nxt, r0 + per * U);
      __syncthreads();
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int r = r0 + u * per + sub;
        if (mine && r < r_end) store_word<A>(dst + r * pl.dst_s[1], cur[u]);
        cur[u] = nxt[u];
      }
    }
  }
}

template <bool IN_PLACE>
__global__ void __launch_bounds__(kMoveThreads)
    evict_move_kernel(const __grid_constant__ EvictArgs a) {
  grid_dependency_wait();
  int p = 0;
  while (p + 1 < a.n_planes && static_cast<int>(blockIdx.x) >= a.first_block[p + 1]) ++p;
  const EvictPlane& pl = a.planes[p];
  const int piece = blockIdx.x - a.first_block[p];
  const int bh = blockIdx.y, b = bh / a.Hkv, kvh = bh - b * a.Hkv;
  const int n = a.lens[b];
  if (n < 0 || n > a.cap) return;  // evict_select has recorded it
  const int count = min(n, a.budget);
  const int r_begin = blockIdx.z * a.seg_rows;
  const int r_end = min(count, r_begin + a.seg_rows);
  const uint8_t* src = pl.src + b * pl.src_s[0] + kvh * pl.src_s[2] + piece * pl.piece_bytes;
  uint8_t* dst = pl.dst + b * pl.dst_s[0] + kvh * pl.dst_s[2] + piece * pl.piece_bytes;
  // in place, a sequence within its budget stays where it is
  if (r_begin < r_end && !(pl.src == pl.dst && n <= a.budget)) {
    const int32_t* kept = a.kept + static_cast<long long>(bh) * a.budget;
    if (pl.access == 16) move_rows<16, IN_PLACE>(pl, src, dst, kept, r_begin, r_end);
    else if (pl.access == 8) move_rows<8, IN_PLACE>(pl, src, dst, kept, r_begin, r_end);
    else move_rows<4, IN_PLACE>(pl, src, dst, kept, r_begin, r_end);
  }
  if (pl.dst == reinterpret_cast<uint8_t*>(a.w_out) && blockIdx.z == 0) {
    __syncthreads();  // in place: after the weights have moved down
    float* w = a.w_out + static_cast<long long>(bh) * a.out_rows;
    for (int r = count + threadIdx.x; r < a.out_rows; r += kMoveThreads) w[r] = 0.f;
  }
}

}  // namespace

cudaError_t launch_evict(const EvictArgs& a, cudaStream_t stream) {
  // Long caches of few (sequence, head)s: clusters share the rows, down to the number
  // a CTA holds (131072 rows of 8 heads took one CTA each 117 us).
  EvictArgs args = a;
  args.parts = 1;
  while (args.parts < 8 && a.cap > args.parts * kSelHeld * kSelThreads &&
         a.B * a.Hkv * args.parts * 2 <= 148 * 2)
    args.parts *= 2;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(a.B * a.Hkv * args.parts);
  cfg.blockDim = dim3(kSelThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = args.parts;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = args.parts > 1 ? 1 : 0;
  const cudaError_t e = args.parts > 1 ? cudaLaunchKernelEx(&cfg, evict_select_kernel<true>, args)
                                       : cudaLaunchKernelEx(&cfg, evict_select_kernel<false>, args);
  if (e != cudaSuccess) return e;
  const dim3 grid(a.first_block[a.n_planes], a.B * a.Hkv,
                  (a.budget + a.seg_rows - 1) / a.seg_rows);
  return launch_after(a.in_place ? evict_move_kernel<true> : evict_move_kernel<false>, grid,
                      kMoveThreads, 0, stream, a);
}

}  // namespace mea
