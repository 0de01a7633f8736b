// paged_kv_evict_rows and paged_kv_evict_pages: which keys of each sequence stay,
// by their accumulated attention weight (paged_attention_decode_mass).
//
// Units are rows, or pages (their weight: the sum of their rows' by adding halves
// again and again, so that it is the same whoever computes it).  A sequence of more
// units than its budget keeps its first ones (sinks), its last ones (recent) and the
// heaviest of the others, ties by the lower index.
//
// A cluster of CTAs shares a sequence, each a stretch of its units, whose keys (floats
// as ordered integers) stay in shared memory where they fit.  The threshold comes from
// histograms of its digits (a radix select; integer counts, so the result is the same on
// every run), added up over the cluster through distributed shared memory; a digit that
// takes all of its keys ends the search.  Then each CTA knows how many units
// before its stretch are kept, and one pass ranks and moves its own.  What a digit costs
// in a cluster is what each CTA reads of the others' counts: digits of 11 bits, 8 KB a
// CTA, took 4.2 us a digit on 8 CTAs and 8 us on 16, 8 bits 2.7 on 16 (one sequence of
// 131,072 rows: 25, 32 and 17 us in all).  Alone, a CTA takes 11 (32 sequences of
// 512-4096 rows: 8.5 us, with 8 bits 9.4).
// Bytes: the masses once read and once written (and the re-reads of units that do not
// fit in shared memory).  256 sequences of 1k to 32k rows by pages of 16 take 22 us
// (55 MB; 8 us at the rate of a copy): one wave of CTAs, as long as its longest
// sequences.  One long sequence is latency on its few CTAs: the loads, each digit's
// counts and barriers, the moves.
#include <algorithm>

#include "cluster.cuh"
#include "common.cuh"
#include "inputs.cuh"
#include "internal.h"

namespace pa {

namespace {

constexpr int kEvictThreads = 512;
constexpr int kEvictWarps = kEvictThreads / 32;
constexpr int kCacheUnits = kMaxEvictPages / 8 + 32;  // keys in shared memory: 160 KB
constexpr int kAhead = 4;                             // vectors of a thread in flight
constexpr int kMaxCtas = 16;                          // of a cluster (more than 8 are opted in to)
constexpr int kRowsAhead = 16;                        // masses of a lane in flight as they move

// A float as an integer of the same order; NaN lowest, -0 as 0.
__device__ __forceinline__ uint32_t order_key(float x) {
  const uint32_t b = __float_as_uint(x == 0.f ? 0.f : x);
  return x != x ? 0u : ((b >> 31) ? ~b : b | 0x80000000u);
}

__device__ __forceinline__ float ld_float(const float* p) {
  return __uint_as_float(ld_input(reinterpret_cast<const uint32_t*>(p)));
}
__device__ __forceinline__ float4 ld_float4(const float* p) {
  const uint4 v = ld_input(reinterpret_cast<const uint4*>(p));
  return make_float4(__uint_as_float(v.x), __uint_as_float(v.y), __uint_as_float(v.z), __uint_as_float(v.w));
}

template <bool CL>
struct EvictShared {
  // CL: this CTA's counts of four digits of 8 bits (one barrier of the cluster a digit)
  // and behind them the cluster's; one CTA: of digits of 11, 11 and 10 bits
  static constexpr int kBins = CL ? 256 : 2048, kHists = CL ? 8 : 3;
  uint32_t hist[kHists][kBins];
  uint32_t above, ties;        // this CTA's units above the threshold (or kept anyway), and at it
  uint32_t digit, left, here;  // the threshold's digit, units still to be taken at it, and all units at it
  uint32_t warp_sum[kEvictWarps];
  uint32_t warp_above[kEvictWarps], warp_ties[kEvictWarps];
  int32_t count;
};

__device__ __forceinline__ float plus(float a, float b) { return __fadd_rn(a, b); }

// The weight of a page, for the warp's pages: rows [u * ps, + ps) below L.  M: rows a lane.
template <int M>
__device__ __forceinline__ float page_weight(const float* mass, int64_t row, int L, int step) {
  float v[M];
#pragma unroll
  for (int k = 0; k < M; ++k) v[k] = row + 32 * k < L ? ld_float(mass + row + 32 * k) : 0.f;
#pragma unroll
  for (int h = M / 2; h > 0; h >>= 1)
#pragma unroll
    for (int k = 0; k < M / 2; ++k)
      if (k < h) v[k] = plus(v[k], v[k + h]);
  float x = v[0];
  for (int o = step; o > 0; o >>= 1) x = plus(x, __shfl_xor_sync(0xffffffffu, x, o));
  return x;
}

// The same from vectors of four rows, pages of 4 to 128 rows: lanes o / 4 apart add
// rows o apart, then the vector's own.
__device__ __forceinline__ float page_weight4(float4 v, int ps) {
  for (int o = ps / 8; o > 0; o >>= 1) {
    v.x = plus(v.x, __shfl_xor_sync(0xffffffffu, v.x, o));
    v.y = plus(v.y, __shfl_xor_sync(0xffffffffu, v.y, o));
    v.z = plus(v.z, __shfl_xor_sync(0xffffffffu, v.z, o));
    v.w = plus(v.w, __shfl_xor_sync(0xffffffffu, v.w, o));
  }
  return plus(plus(v.x, v.z), plus(v.y, v.w));
}

// The warp's inclusive sums.
__device__ __forceinline__ uint32_t warp_sums(uint32_t x, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t t = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += t;
  }
  return x;
}

// Which of the digits highest, highest - 1, .. the left-th key has: n their counts,
// *before the keys of higher digits (and of all above the one found), *here its count.
template <int N>
__device__ __forceinline__ uint32_t find_digit(const uint32_t (&n)[N], uint32_t highest, uint32_t left, uint32_t* before,
                                               uint32_t* here) {
  uint32_t d = highest;
  *here = n[0];
#pragma unroll
  for (int k = 0; k + 1 < N; ++k)
    if (d == highest - k && *before + n[k] < left) {
      *before += n[k];
      *here = n[k + 1];
      --d;
    }
  return d;
}

// CL: a cluster of csize CTAs a sequence; else one CTA.
template <bool PAGES, bool CL>
__global__ void __launch_bounds__(kEvictThreads) evict_kernel(const __grid_constant__ EvictParams p, int csize) {
  using Shared = EvictShared<CL>;
  extern __shared__ uint4 cache4[];
  uint32_t* cache = reinterpret_cast<uint32_t*>(cache4);
  __shared__ __align__(16) Shared sh;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if constexpr (!CL) csize = 1;
  const int b = blockIdx.x / csize, rank = blockIdx.x - b * csize;
  griddep_wait();
  const int L = ld_seq_len(p.seq_lens, b, p.max_len, rank == 0 && tid == 0 ? p.err : nullptr);
  const int ps = PAGES ? p.page_size : 1;
  const int units = PAGES ? (L + ps - 1) / ps : L;
  const bool over = units > p.budget;
  const float* mass = p.mass + (int64_t)b * p.mass_stride;
  float* new_mass = p.new_mass + (int64_t)b * p.new_mass_stride;
  // units [0, front) and [back, units) stay
  const int front = over ? (PAGES ? (p.num_sinks + ps - 1) / ps : p.num_sinks) : units;
  const int back = over ? (PAGES ? max(0, L - max(1, p.num_recent)) / ps : L - p.num_recent) : units;
  const uint32_t want = over ? (uint32_t)(p.budget - front - (units - back)) : 0u;  // of [front, back)
  const int per = ((units + csize - 1) / csize + 31) / 32 * 32;
  const int lo = min(units, rank * per), hi = min(units, lo + per);
  const int cached = min(hi - lo, kCacheUnits);
  const bool select = over && want > 0u;
  // ---- the keys of this stretch ----
  if (select) {
    for (int i = tid; i < Shared::kHists * Shared::kBins / 4; i += kEvictThreads)
      reinterpret_cast<uint4*>(sh.hist[0])[i] = make_uint4(0u, 0u, 0u, 0u);
    if constexpr (PAGES) {
      if (p.vec && ps >= 4 && ps <= 128) {
        const int pages = 128 / ps, lanes = ps / 4;  // of a warp's vectors
        const int step = kEvictWarps * pages;
        for (int u0 = lo + warp * pages; u0 < hi; u0 += step * kAhead) {
          float4 v[kAhead];
#pragma unroll
          for (int k = 0; k < kAhead; ++k) {
            const int u = u0 + k * step + lane / lanes;
            const int64_t row = (int64_t)u * ps + lane % lanes * 4;
            v[k] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (u < hi && row + 3 < L) {
              v[k] = ld_float4(mass + row);
            } else if (u < hi) {
              if (row < L) v[k].x = ld_float(mass + row);
              if (row + 1 < L) v[k].y = ld_float(mass + row + 1);
              if (row + 2 < L) v[k].z = ld_float(mass + row + 2);
            }
          }
#pragma unroll
          for (int k = 0; k < kAhead; ++k) {
            const int u = u0 + k * step + lane / lanes;
            const float x = page_weight4(v[k], ps);
            if (u < hi && lane % lanes == 0) cache[u - lo] = order_key(x);
          }
        }
      } else {
        const int lanes = min(ps, 32), pages = 32 / lanes, m = ps > 32 ? ps / 32 : 1;
        for (int u0 = lo + warp * pages; u0 < hi; u0 += kEvictWarps * pages) {
          const int u = u0 + lane / lanes;
          const int64_t row = (int64_t)u * ps + lane % lanes;
          const int end = u < hi ? L : 0;
          float x;
          switch (m) {
            case 1: x = page_weight<1>(mass, row, end, lanes / 2); break;
            case 2: x = page_weight<2>(mass, row, end, 16); break;
            case 4: x = page_weight<4>(mass, row, end, 16); break;
            case 8: x = page_weight<8>(mass, row, end, 16); break;
            case 16: x = page_weight<16>(mass, row, end, 16); break;
            default: x = page_weight<32>(mass, row, end, 16); break;
          }
          if (u < hi && lane % lanes == 0) cache[u - lo] = order_key(x);
        }
      }
    } else {
      const int vecs = p.vec ? cached / 4 : 0;  // lo is a multiple of 32
      for (int i0 = tid; i0 < vecs; i0 += kAhead * kEvictThreads) {
        float4 v[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
          if (i0 + k * kEvictThreads < vecs) v[k] = ld_float4(mass + lo + 4 * (i0 + k * kEvictThreads));
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
          if (i0 + k * kEvictThreads < vecs)
            cache4[i0 + k * kEvictThreads] =
                make_uint4(order_key(v[k].x), order_key(v[k].y), order_key(v[k].z), order_key(v[k].w));
      }
      for (int i = 4 * vecs + tid; i < cached; i += kEvictThreads) cache[i] = order_key(ld_float(mass + lo + i));
    }
  }
  // f(key) for the units of [a, e), four a thread and step, in any order
  auto each = [&](int a, int e, auto f) {
    const int vecs = (cached + 3) / 4;
#pragma unroll 4
    for (int i = tid; i < vecs; i += kEvictThreads) {
      const uint4 k = cache4[i];
      const int u = lo + 4 * i;
      if (u >= a && u + 3 < e) {
        f(k.x);
        f(k.y);
        f(k.z);
        f(k.w);
      } else {
        if (u >= a && u < e) f(k.x);
        if (u + 1 >= a && u + 1 < e) f(k.y);
        if (u + 2 >= a && u + 2 < e) f(k.z);
        if (u + 3 >= a && u + 3 < e) f(k.w);
      }
    }
    for (int u = max(a, lo + cached) + tid; u < e; u += kEvictThreads) f(order_key(ld_float(mass + u)));
  };
  auto key = [&](int u) { return PAGES || u - lo < kCacheUnits ? cache[u - lo] : order_key(ld_float(mass + u)); };
  __syncthreads();
  // ---- the threshold: the want-th largest key of [front, back) ----
  uint32_t prefix = 0u, left = want;  // digits so far; units still to be found below them
  if (select) {
    const int a = max(lo, front), e = min(hi, back);
    for (int pass = 0; pass < (CL ? 4 : 3); ++pass) {
      // the digit's lowest bit, and the one above its highest
      const int shift = CL ? 24 - 8 * pass : max(0, 21 - 11 * pass), top = CL ? shift + 8 : (pass == 0 ? 32 : 32 - 11 * pass);
      uint32_t* hist = sh.hist[pass];
      each(a, e, [&](uint32_t k) {
        if (((uint64_t)(k ^ prefix) >> top) == 0) atomicAdd(&hist[(k >> shift) & ((1u << (top - shift)) - 1u)], 1u);
      });
      uint32_t here;
      if constexpr (CL) {
        cluster_sync();
        // 64 threads to a CTA's histogram
        uint32_t* total = sh.hist[4 + pass];
        const int g = 31 - lane;
        for (int c = tid >> 6; c < csize; c += kEvictThreads / 64) {
          const int at = 4 * (tid & 63);
          const float4 x = ld_cluster4(map_rank(smem_u32(hist + at), c));
          if (__float_as_uint(x.x) != 0u) atomicAdd(total + at, __float_as_uint(x.x));
          if (__float_as_uint(x.y) != 0u) atomicAdd(total + at + 1, __float_as_uint(x.y));
          if (__float_as_uint(x.z) != 0u) atomicAdd(total + at + 2, __float_as_uint(x.z));
          if (__float_as_uint(x.w) != 0u) atomicAdd(total + at + 3, __float_as_uint(x.w));
        }
        __syncthreads();
        // each warp by itself: lane i has digits 8 (31 - i) .. + 7, the highest first
        const uint4 n0 = reinterpret_cast<const uint4*>(total)[2 * g], n1 = reinterpret_cast<const uint4*>(total)[2 * g + 1];
        const uint32_t n[8] = {n1.w, n1.z, n1.y, n1.x, n0.w, n0.z, n0.y, n0.x};
        const uint32_t mine = n[0] + n[1] + n[2] + n[3] + n[4] + n[5] + n[6] + n[7];
        const uint32_t incl = warp_sums(mine, lane);
        uint32_t before = incl - mine, d = find_digit(n, 8u * (uint32_t)g + 7u, left, &before, &here);
        // the first lane whose digits reach `left`
        const int at = __ffs(__ballot_sync(0xffffffffu, incl >= left)) - 1;
        prefix |= __shfl_sync(0xffffffffu, d, at) << shift;
        left -= __shfl_sync(0xffffffffu, before, at);
        here = __shfl_sync(0xffffffffu, here, at);
      } else {
        __syncthreads();
        // thread i: digits 4 (511 - i) .. + 3, the highest first
        const int g = kEvictThreads - 1 - tid;
        const uint4 v = reinterpret_cast<const uint4*>(hist)[g];
        const uint32_t n[4] = {v.w, v.z, v.y, v.x};
        const uint32_t mine = v.x + v.y + v.z + v.w;
        uint32_t incl = warp_sums(mine, lane);
        if (lane == 31) sh.warp_sum[warp] = incl;
        __syncthreads();
        for (int w = 0; w < warp; ++w) incl += sh.warp_sum[w];
        uint32_t before = incl - mine;
        if (incl >= left && before < left) {  // one thread
          sh.digit = find_digit(n, 4u * (uint32_t)g + 3u, left, &before, &here);
          sh.left = left - before;
          sh.here = here;
        }
        __syncthreads();
        prefix |= sh.digit << shift;
        left = sh.left;
        here = sh.here;
      }
      if (here == left && prefix != 0u) {
        --prefix;  // every key that begins with these digits stays: no more of them are needed
        left = 0u;
        break;
      }
    }
  }
  // ---- this stretch's units above the threshold and at it ----
  // a warp walks a stretch of its own, 32 units at a time
  const int wper = (((hi - lo) + kEvictWarps - 1) / kEvictWarps + 31) / 32 * 32;
  const int wlo = min(hi, lo + warp * wper), whi = min(hi, wlo + wper);
  const bool inside = select && wlo >= front && whi <= back;  // the key alone says whether a unit stays
  auto classify = [&](int u, uint32_t k, bool* above, bool* tie) {
    const bool may = select && u >= front && u < back;
    *above = u < whi && (may ? k > prefix : u < front || u >= back);
    *tie = u < whi && may && k == prefix;
  };
  __syncthreads();
  uint32_t n_above = 0u, n_ties = 0u;
  auto count = [&](int u, uint32_t k) {
    bool ab, ti;
    classify(u, k, &ab, &ti);
    n_above += ab ? 1u : 0u;
    n_ties += ti ? 1u : 0u;
  };
  if (!select) {  // all of them, or those at the ends
    for (int u = wlo + lane; u < whi; u += 32) count(u, 0u);
  } else if (whi - lo <= cached) {  // four units a lane and step
#pragma unroll 2
    for (int i = (wlo - lo + 3) / 4 + lane; 4 * i < whi - lo; i += 32) {  // wlo: a multiple of 32 past lo, or hi
      const uint4 k = cache4[i];
      const int u = lo + 4 * i;
      if (inside && u + 3 < whi) {
        n_above += (k.x > prefix ? 1u : 0u) + (k.y > prefix ? 1u : 0u) + (k.z > prefix ? 1u : 0u) + (k.w > prefix ? 1u : 0u);
        n_ties += (k.x == prefix ? 1u : 0u) + (k.y == prefix ? 1u : 0u) + (k.z == prefix ? 1u : 0u) + (k.w == prefix ? 1u : 0u);
      } else {
        count(u, k.x);
        count(u + 1, k.y);
        count(u + 2, k.z);
        count(u + 3, k.w);
      }
    }
  } else {
    for (int u = wlo + lane; u < whi; u += 32) count(u, key(u));
  }
  n_above = __reduce_add_sync(0xffffffffu, n_above);
  n_ties = __reduce_add_sync(0xffffffffu, n_ties);
  if (lane == 0) {
    sh.warp_above[warp] = n_above;
    sh.warp_ties[warp] = n_ties;
  }
  if (tid == 0) sh.count = 0;
  __syncthreads();
  if (tid == 0) {
    uint32_t x = 0u, y = 0u;
    for (int w = 0; w < kEvictWarps; ++w) {
      x += sh.warp_above[w];
      y += sh.warp_ties[w];
    }
    sh.above = x;
    sh.ties = y;
  }
  // where this sequence's list begins
  if constexpr (!PAGES) {
    int n = 0;
    for (int i = tid; i < b; i += kEvictThreads) n += ld_seq_len(p.seq_lens, i, p.max_len, nullptr) > p.budget ? 1 : 0;
    n = __reduce_add_sync(0xffffffffu, n);
    if (lane == 0 && n != 0) atomicAdd(&sh.count, n);
  }
  if constexpr (CL) cluster_sync(); else __syncthreads();
  uint32_t above = 0u, ties = 0u, all_above = 0u;
  if constexpr (CL) {
    // lane c reads the counts of CTA c (above and ties lie side by side)
    const float2 v = lane < csize ? ld_cluster2(map_rank(smem_u32(&sh.above), lane)) : make_float2(0.f, 0.f);
    const uint32_t x = lane < csize ? __float_as_uint(v.x) : 0u, y = lane < csize ? __float_as_uint(v.y) : 0u;
    all_above = __reduce_add_sync(0xffffffffu, x);
    above = __reduce_add_sync(0xffffffffu, lane < rank ? x : 0u);
    ties = __reduce_add_sync(0xffffffffu, lane < rank ? y : 0u);
  } else {
    all_above = sh.above;
  }
  for (int w = 0; w < warp; ++w) {
    above += sh.warp_above[w];
    ties += sh.warp_ties[w];
  }
  const uint32_t kept_total = select ? all_above + left : all_above;
  const int share = PAGES ? 0 : p.budget - p.num_sinks;
  const int64_t list = (int64_t)sh.count * share;
  if (!PAGES && rank == 0 && tid == 0) {
    if (b == 0) p.keep_indptr[0] = 0;
    p.keep_indptr[b + 1] = (int32_t)(list + (over ? share : 0));
    p.base[b] = over ? p.num_sinks : L;
  }
  // ---- ranks, and the moves ----
  // The rank of unit u0 + lane among those kept, 0xFFFFFFFF if it goes; `before`: the
  // kept ones in front of it.
  auto rank_of = [&](int u, uint32_t k, uint32_t* before) {
    bool ab, ti;
    classify(u, k, &ab, &ti);
    const unsigned ma = __ballot_sync(0xffffffffu, ab), mt = __ballot_sync(0xffffffffu, ti);
    const unsigned below = (1u << lane) - 1u;
    const uint32_t tr = ties + __popc(mt & below);
    *before = above + __popc(ma & below) + min(tr, select ? left : 0u);
    above += __popc(ma);
    ties += __popc(mt);
    return ab || (ti && tr < left) ? *before : 0xFFFFFFFFu;
  };
  if constexpr (PAGES) {
    const int64_t table = (int64_t)b * p.max_blocks;
    for (int u0 = wlo; u0 < whi; u0 += 32) {
      const int u = u0 + lane;
      uint32_t before;
      const uint32_t r = rank_of(u, select && u < whi ? key(u) : 0u, &before);
      if (u < whi) {
        p.new_block_table[table + (r != 0xFFFFFFFFu ? r : kept_total + ((uint32_t)u - before))] =
            ld_input(p.block_table + table + u);
        cache[u - lo] = r;  // its key is done with: each warp reads its own stretch alone
      }
    }
    __syncthreads();
    // the rows of the stretch that stay, four at a time where pages and rows allow
    const int64_t row0 = (int64_t)lo * ps, row1 = min((int64_t)L, (int64_t)hi * ps);
    const int shift = 31 - __clz(ps);
    if (p.vec && ps >= 4) {
      for (int64_t i0 = row0 / 4 + tid; 4 * i0 + 3 < row1; i0 += kAhead * kEvictThreads) {
        float4 v[kAhead];
        int64_t to[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
          const int64_t row = 4 * (i0 + k * kEvictThreads);
          to[k] = -1;
          if (row + 3 < row1) {
            const uint32_t r = cache[(int)(row >> shift) - lo];
            if (r != 0xFFFFFFFFu) {
              to[k] = (int64_t)r * ps + (row & (ps - 1));
              v[k] = ld_float4(mass + row);
            }
          }
        }
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
          if (to[k] >= 0) *reinterpret_cast<float4*>(new_mass + to[k]) = v[k];
      }
    }
    const int64_t rest = p.vec && ps >= 4 ? row1 / 4 * 4 : row0;  // (lo * ps is a multiple of 32)
    for (int64_t row = max(rest, row0) + tid; row < row1; row += kEvictThreads) {
      const uint32_t r = cache[(int)(row >> shift) - lo];
      if (r != 0xFFFFFFFFu) new_mass[(int64_t)r * ps + (row & (ps - 1))] = ld_float(mass + row);
    }
  } else {
    for (int u0 = wlo; u0 < whi; u0 += 32 * kRowsAhead) {
      float v[kRowsAhead];
#pragma unroll
      for (int k = 0; k < kRowsAhead; ++k) v[k] = u0 + 32 * k + lane < whi ? ld_float(mass + u0 + 32 * k + lane) : 0.f;
      if (inside && left == 0u) {  // and no tie does
#pragma unroll
        for (int k = 0; k < kRowsAhead; ++k) {
          const int u = u0 + 32 * k + lane;
          const bool stays = u < whi && order_key(v[k]) > prefix;
          const unsigned m = __ballot_sync(0xffffffffu, stays);
          const uint32_t r = above + __popc(m & ((1u << lane) - 1u));
          above += __popc(m);
          if (stays) {
            new_mass[r] = v[k];
            p.keep[list + (int)r - p.num_sinks] = u;
          }
        }
        continue;
      }
#pragma unroll
      for (int k = 0; k < kRowsAhead; ++k) {
        uint32_t before;
        const uint32_t r = rank_of(u0 + 32 * k + lane, order_key(v[k]), &before);
        if (r != 0xFFFFFFFFu) {
          new_mass[r] = v[k];
          if (over && (int)r >= p.num_sinks) p.keep[list + (int)r - p.num_sinks] = u0 + 32 * k + lane;
        }
      }
    }
  }
  const int new_len = PAGES ? L - ps * (units - (int)kept_total) : (int)kept_total;
  int zero = new_len;
  if (p.vec) {  // whole vectors of zeros behind the next multiple of 4
    const int z4 = (new_len + 3) / 4;
    for (int i = z4 + rank * kEvictThreads + tid; 4 * i + 3 < p.width; i += csize * kEvictThreads)
      reinterpret_cast<float4*>(new_mass)[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (rank == 0 && tid < 4 && new_len + tid < min(4 * z4, p.width)) new_mass[new_len + tid] = 0.f;
    zero = max(new_len, p.width / 4 * 4);
  }
  for (int i = zero + rank * kEvictThreads + tid; i < p.width; i += csize * kEvictThreads) new_mass[i] = 0.f;
  if constexpr (PAGES) {
    for (int i = units + rank * kEvictThreads + tid; i < p.max_blocks; i += csize * kEvictThreads)
      p.new_block_table[(int64_t)b * p.max_blocks + i] = ld_input(p.block_table + (int64_t)b * p.max_blocks + i);
    if (rank == 0 && tid == 0) p.new_seq_lens[b] = new_len;
  }
  if constexpr (CL) cluster_sync();  // no CTA leaves while another reads its counts
}

// Whether a cluster of kMaxCtas CTAs, more than the 8 that every GPU takes, finds its SMs
// beside one another (on a part of a GPU it may not).
template <typename Kernel>
bool most_fit(Kernel kern, size_t smem) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(kMaxCtas);
  cfg.blockDim = dim3(kEvictThreads);
  cfg.dynamicSmemBytes = smem;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = kMaxCtas;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int n = 0;
  const bool ok = cudaOccupancyMaxActiveClusters(&n, kern, &cfg) == cudaSuccess;
  if (!ok) (void)cudaGetLastError();
  return ok && n > 0;
}

}  // namespace

// CTAs of a sequence, `most` at most: as many as find an SM, with 4096 rows each or more;
// enough that their stretches fit in shared memory, where `most` can.  One sequence of
// 131,072 rows: 21 us on 8 CTAs, 16 on 16; of 8192 rows, where one CTA would do: 11.4 us on
// two, 9.8 on one; of 32,768: 11.9 us on eight, 13.9 on four.
int evict_cluster(int num_sms, int32_t batch, int64_t units, int64_t rows, int most) {
  int c = 1;
  while (c < most && ((int64_t)batch * c * 2 <= num_sms && rows >= 4096 * 2 * (int64_t)c)) c *= 2;
  while (c < most && units > (int64_t)c * (kCacheUnits - 32)) c *= 2;
  return c;
}

cudaError_t launch_evict(const EvictParams& p, bool pages, int num_sms, cudaStream_t s) {
  if (p.batch <= 0) return cudaSuccess;
  const int64_t units = pages ? std::min<int64_t>(p.max_blocks, (p.max_len + p.page_size - 1) / p.page_size) : p.max_len;
  if (pages && units > kMaxEvictPages) return cudaErrorInvalidValue;  // their weights have no place
  const int64_t rows = pages ? units * p.page_size : units;
  int csize = evict_cluster(num_sms, p.batch, units, rows, kMaxCtas);
  auto kern = csize > 1 ? (pages ? evict_kernel<true, true> : evict_kernel<false, true>)
                        : (pages ? evict_kernel<true, false> : evict_kernel<false, false>);
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kCacheUnits * 4 + 16);
  if (e == cudaSuccess && csize > 8) e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e != cudaSuccess) return e;
  auto smem_of = [&](int c) {
    const int64_t stretch = (units + c - 1) / c + 32;
    return (size_t)(stretch < kCacheUnits ? stretch : kCacheUnits) * 4 + 16;
  };
  if (csize > 8 && !most_fit(kern, smem_of(csize))) csize = evict_cluster(num_sms, p.batch, units, rows, 8);
  return launch_pdl_cluster(kern, dim3((unsigned)(p.batch * csize)), dim3(kEvictThreads), smem_of(csize), csize, s, p, csize);
}

}  // namespace pa
