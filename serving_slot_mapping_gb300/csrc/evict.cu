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
// four histograms of 8 bits each (a radix select; integer counts, so the result is the
// same on every run), added up over the cluster through distributed shared memory; then
// each CTA knows how many units before its stretch are kept, and one pass ranks and
// moves its own.
// Bytes: the masses once read and once written (and the re-reads of units that do not
// fit in shared memory).
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

// A float as an integer of the same order; NaN lowest, -0 as 0.
__device__ __forceinline__ uint32_t order_key(float x) {
  const uint32_t b = __float_as_uint(x == 0.f ? 0.f : x);
  return x != x ? 0u : ((b >> 31) ? ~b : b | 0x80000000u);
}

__device__ __forceinline__ float ld_float(const float* p) {
  return __uint_as_float(ld_input(reinterpret_cast<const uint32_t*>(p)));
}

struct EvictShared {
  uint32_t hist[256];
  uint32_t sums[256];          // of the cluster
  uint32_t above, ties;        // this CTA's units above the threshold (or kept anyway), and at it
  uint32_t digit, left;        // the threshold's digit, units still to be taken at it
  uint32_t warp_above[kEvictWarps], warp_ties[kEvictWarps];
  int32_t count;
};

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
      if (k < h) v[k] += v[k + h];
  float x = v[0];
  for (int o = step; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

template <bool PAGES>
__global__ void __launch_bounds__(kEvictThreads) evict_kernel(const __grid_constant__ EvictParams p, int csize) {
  extern __shared__ uint32_t cache[];
  __shared__ EvictShared sh;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
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
  auto key_of = [&](int u) { return order_key(ld_float(mass + u)); };  // rows
  const int cached = min(hi - lo, kCacheUnits);
  if (over) {
    if constexpr (PAGES) {
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
    } else {
      for (int i = tid; i < cached; i += kEvictThreads) cache[i] = key_of(lo + i);
    }
  }
  auto key = [&](int u) { return PAGES || u - lo < kCacheUnits ? cache[u - lo] : key_of(u); };
  // ---- the threshold: the want-th largest key of [front, back) ----
  uint32_t prefix = 0u, left = want;  // digits so far; units still to be found below them
  const bool select = over && want > 0u;
  if (select) {
    const int a = max(lo, front), e = min(hi, back);
    for (int shift = 24; shift >= 0; shift -= 8) {
      if (tid < 256) sh.hist[tid] = 0u;
      __syncthreads();
      for (int u = a + tid; u < e; u += kEvictThreads) {
        const uint32_t k = key(u);
        if (shift == 24 || (k >> (shift + 8)) == (prefix >> (shift + 8))) atomicAdd(&sh.hist[(k >> shift) & 255u], 1u);
      }
      if (csize > 1) cluster_sync(); else __syncthreads();
      if (tid < 256) {
        uint32_t n = 0u;
        if (csize > 1)
          for (int c = 0; c < csize; ++c) n += ld_cluster(map_rank(smem_u32(&sh.hist[tid]), c));
        else
          n = sh.hist[tid];
        sh.sums[tid] = n;
      }
      if (csize > 1) cluster_sync(); else __syncthreads();  // every histogram is read
      if (warp == 0) {  // lane i: digits 255 - 8 i down to 248 - 8 i
        uint32_t n = 0u;
        for (int k = 0; k < 8; ++k) n += sh.sums[255 - 8 * lane - k];
        uint32_t incl = n;
        for (int o = 1; o < 32; o <<= 1) {
          const uint32_t t = __shfl_up_sync(0xffffffffu, incl, o);
          if (lane >= o) incl += t;
        }
        if (incl >= left && incl - n < left) {
          uint32_t before = incl - n;
          int d = 255 - 8 * lane;
          while (before + sh.sums[d] < left) before += sh.sums[d--];
          sh.digit = (uint32_t)d;
          sh.left = left - before;
        }
      }
      __syncthreads();
      prefix |= sh.digit << shift;
      left = sh.left;
    }
  }
  // ---- this stretch's units above the threshold and at it ----
  auto classify = [&](int u, bool* above, bool* tie) {
    *above = *tie = false;
    if (u >= hi) return;
    if (u < front || u >= back) {
      *above = true;
    } else if (select) {
      const uint32_t k = key(u);
      *above = k > prefix;
      *tie = k == prefix;
    }
  };
  // a warp walks a stretch of its own, 32 units at a time
  const int wper = (((hi - lo) + kEvictWarps - 1) / kEvictWarps + 31) / 32 * 32;
  const int wlo = min(hi, lo + warp * wper), whi = min(hi, wlo + wper);
  __syncthreads();
  uint32_t n_above = 0u, n_ties = 0u;
  for (int u0 = wlo; u0 < whi; u0 += 32) {
    bool ab, ti;
    classify(u0 + lane, &ab, &ti);
    ab &= u0 + lane < whi;
    ti &= u0 + lane < whi;
    n_above += __popc(__ballot_sync(0xffffffffu, ab));
    n_ties += __popc(__ballot_sync(0xffffffffu, ti));
  }
  if (lane == 0) {
    sh.warp_above[warp] = n_above;
    sh.warp_ties[warp] = n_ties;
  }
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
  if (csize > 1) cluster_sync(); else __syncthreads();
  uint32_t above = 0u, ties = 0u, all_above = 0u;
  for (int c = 0; c < csize; ++c) {
    const uint32_t x = csize > 1 ? ld_cluster(map_rank(smem_u32(&sh.above), c)) : sh.above;
    const uint32_t y = csize > 1 ? ld_cluster(map_rank(smem_u32(&sh.ties), c)) : sh.ties;
    if (c < rank) {
      above += x;
      ties += y;
    }
    all_above += x;
  }
  for (int w = 0; w < warp; ++w) {
    above += sh.warp_above[w];
    ties += sh.warp_ties[w];
  }
  const uint32_t kept_total = select ? all_above + left : all_above;
  // ---- where this sequence's list begins ----
  int64_t list = 0;
  if constexpr (!PAGES) {
    if (tid == 0) sh.count = 0;
    __syncthreads();
    const int share = p.budget - p.num_sinks;
    int n = 0;
    for (int i = tid; i < b; i += kEvictThreads) n += ld_seq_len(p.seq_lens, i, p.max_len, nullptr) > p.budget ? 1 : 0;
    n = __reduce_add_sync(0xffffffffu, n);
    if (lane == 0 && n != 0) atomicAdd(&sh.count, n);
    __syncthreads();
    list = (int64_t)sh.count * share;
    if (rank == 0 && tid == 0) {
      if (b == 0) p.keep_indptr[0] = 0;
      p.keep_indptr[b + 1] = (int32_t)(list + (over ? share : 0));
      p.base[b] = over ? p.num_sinks : L;
    }
  }
  // ---- ranks, and the moves ----
  for (int u0 = wlo; u0 < whi; u0 += 32) {
    const int u = u0 + lane;
    bool ab, ti;
    classify(u, &ab, &ti);
    ab &= u < whi;
    ti &= u < whi;
    const unsigned ma = __ballot_sync(0xffffffffu, ab), mt = __ballot_sync(0xffffffffu, ti);
    const unsigned below = (1u << lane) - 1u;
    const uint32_t tr = ties + __popc(mt & below);
    const bool kept = ab || (ti && tr < left);
    const uint32_t at = above + __popc(ma & below) + min(tr, select ? left : 0u);
    if constexpr (PAGES) {
      if (u < whi) {
        const int page = ld_input(p.block_table + (int64_t)b * p.max_blocks + u);
        p.new_block_table[(int64_t)b * p.max_blocks + (kept ? at : kept_total + ((uint32_t)u - at))] = page;
      }
      for (unsigned m = __ballot_sync(0xffffffffu, kept); m != 0u; m &= m - 1u) {
        const int src = __ffs(m) - 1;
        const int64_t to = (int64_t)__shfl_sync(0xffffffffu, at, src) * ps, from = (int64_t)(u0 + src) * ps;
        for (int r = lane; r < ps && from + r < L; r += 32) new_mass[to + r] = ld_float(mass + from + r);
      }
    } else if (kept) {
      new_mass[at] = ld_float(mass + u);
      if (over && (int)at >= p.num_sinks) p.keep[list + (int)at - p.num_sinks] = u;
    }
    above += __popc(ma);
    ties += __popc(mt);
  }
  const int new_len = PAGES ? L - ps * (units - (int)kept_total) : (int)kept_total;
  for (int i = new_len + rank * kEvictThreads + tid; i < p.width; i += csize * kEvictThreads) new_mass[i] = 0.f;
  if constexpr (PAGES) {
    for (int i = units + rank * kEvictThreads + tid; i < p.max_blocks; i += csize * kEvictThreads)
      p.new_block_table[(int64_t)b * p.max_blocks + i] = ld_input(p.block_table + (int64_t)b * p.max_blocks + i);
    if (rank == 0 && tid == 0) p.new_seq_lens[b] = new_len;
  }
  if (csize > 1) cluster_sync();  // no CTA leaves while another reads its counts
}

}  // namespace

cudaError_t launch_evict(const EvictParams& p, bool pages, int num_sms, cudaStream_t s) {
  if (p.batch <= 0) return cudaSuccess;
  const int64_t units = pages ? std::min<int64_t>(p.max_blocks, (p.max_len + p.page_size - 1) / p.page_size) : p.max_len;
  if (pages && units > kMaxEvictPages) return cudaErrorInvalidValue;  // their weights have no place
  // CTAs of a sequence: as many as find an SM, with 4096 units each or more; enough
  // that their stretches fit in shared memory, where 8 can
  int csize = 1;
  while (csize < 8 && ((int64_t)p.batch * csize * 2 <= num_sms && units >= 4096 * 2 * (int64_t)csize)) csize *= 2;
  while (csize < 8 && units > (int64_t)csize * (kCacheUnits - 32)) csize *= 2;
  const int64_t stretch = (units + csize - 1) / csize + 32;
  const int smem = (int)(stretch < kCacheUnits ? stretch : kCacheUnits) * 4;
  auto kern = pages ? evict_kernel<true> : evict_kernel<false>;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kCacheUnits * 4);
  if (e != cudaSuccess) return e;
  return launch_pdl_cluster(kern, dim3((unsigned)(p.batch * csize)), dim3(kEvictThreads), (size_t)smem, csize, s, p, csize);
}

}  // namespace pa
