// paged_kv_copy_pages and paged_kv_compact: moves of cached rows inside the
// page pools of all layers, one launch each.
//
// Copy: page dst[i] of every pool becomes page src[i] (a fork of a sequence
// shares its full pages and copies the one that both will go on writing).
// Compact: row base_b + i of sequence b becomes its old row keep_b[i]
// (ascending old positions), in place: eviction keeps a part of the keys, a
// verified draft keeps the accepted tokens.
//
// Both are bound by memory: 2 bytes of traffic per byte moved, rows read with
// 16-byte accesses and several in flight per thread.  1900 pages of 32 KB in 4
// layers: 149 us, 6.7 TB/s; half of 16 sequences of 1024 - 4096 keys moved in 4
// layers: 99 us, 6.1 TB/s (the barrier between a tile's reads and its writes).
#include "common.cuh"
#include "inputs.cuh"
#include "internal.h"

namespace pa {

namespace {

// ---- copy ---------------------------------------------------------------------
constexpr int kCopyThreads = 256;
constexpr int kCopyAhead = 4;  // vectors of a thread in flight

// Units (pair i, pool tensor, chunk of a page), chunk fastest.
template <typename V>
__global__ void __launch_bounds__(kCopyThreads) copy_pages_kernel(const __grid_constant__ CopyPagesParams p,
                                                                  int chunks) {
  griddep_wait();
  const int64_t nvec = p.page_bytes / (int64_t)sizeof(V);
  const int tensors = 2 * p.pools.count;
  const int64_t units = p.n * tensors * chunks;
  const int64_t per = (int64_t)blockDim.x * kCopyAhead;
  for (int64_t w = blockIdx.x; w < units; w += gridDim.x) {
    const int64_t pt = w / chunks;
    const int chunk = (int)(w - pt * chunks);
    const int64_t i = pt / tensors;
    const int tensor = (int)(pt - i * tensors);
    const int src = ld_input(p.src + i), dst = ld_input(p.dst + i);
    if (src < 0 || dst < 0 || src == dst) continue;  // padding pair, or nothing to do
    if (src >= p.num_pages || dst >= p.num_pages) {
      if (threadIdx.x == 0 && tensor == 0 && chunk == 0)
        record_error(p.err, ERR_BLOCK_TABLE, src >= p.num_pages ? src : dst);
      continue;
    }
    char* pool = (tensor & 1) ? p.pools.value_pool[tensor >> 1] : p.pools.key_pool[tensor >> 1];
    const V* s = reinterpret_cast<const V*>(pool + src * p.page_bytes);
    V* d = reinterpret_cast<V*>(pool + dst * p.page_bytes);
    const int64_t x0 = chunk * per + threadIdx.x;
    V v[kCopyAhead];
#pragma unroll
    for (int k = 0; k < kCopyAhead; ++k)
      if (x0 + k * blockDim.x < nvec) v[k] = ld_stream(s + x0 + k * blockDim.x);
#pragma unroll
    for (int k = 0; k < kCopyAhead; ++k)
      if (x0 + k * blockDim.x < nvec) d[x0 + k * blockDim.x] = v[k];
  }
}

template <typename V>
cudaError_t launch_copy(const CopyPagesParams& p, cudaStream_t s) {
  const int64_t nvec = p.page_bytes / (int64_t)sizeof(V);
  int64_t threads = (nvec + kCopyAhead - 1) / kCopyAhead;
  threads = threads >= kCopyThreads ? kCopyThreads : (threads + 31) / 32 * 32;
  const int64_t per = threads * kCopyAhead;
  const int64_t chunks = (nvec + per - 1) / per;
  int64_t blocks = p.n * 2 * p.pools.count * chunks;
  if (blocks > INT32_MAX) blocks = INT32_MAX;
  return launch_pdl(copy_pages_kernel<V>, dim3((unsigned)blocks), dim3((unsigned)threads), 0, s, p, (int)chunks);
}

// ---- compact --------------------------------------------------------------------
constexpr int kCompactThreads = 256;
constexpr int kRowsAhead = 8;  // rows of a thread in flight
constexpr int kMinCols = 16;   // vectors of a row a block moves, at least
constexpr int kMaxTile = kCompactThreads / kMinCols * kRowsAhead;

// One block moves a segment of `cols` vectors of every listed row of one
// sequence in one pool tensor, a tile of rows at a time: all reads of a tile
// are done (barrier) before its first write.  A write of row base + i can hit
// the source of a later row only (keep is ascending, so keep[j] >= base + j >
// base + i for j > i) inside the same tile, and no other block touches the
// segment, so the move needs no second buffer.
template <typename V>
__global__ void __launch_bounds__(kCompactThreads) compact_kernel(const __grid_constant__ CompactParams p, int cols) {
  // No early trigger: the attention kernels read seq_lens ahead of their own
  // wait, and new_seq_lens is written here.
  __shared__ int64_t from[kMaxTile], to[kMaxTile];
  const int tensor = blockIdx.y, b = blockIdx.z;
  const int rows = kCompactThreads / cols;  // rows a pass of the block covers
  const int tile = rows * kRowsAhead;
  const int col = threadIdx.x & (cols - 1), r0 = threadIdx.x / cols;
  const int64_t nvec = p.row_bytes / (int64_t)sizeof(V);
  const int64_t x = (int64_t)blockIdx.x * cols + col;  // this thread's vector of a row
  griddep_wait();
  const bool first = blockIdx.x == 0 && tensor == 0;  // records errors, writes the new length
  const int max_len = p.max_blocks * p.page_size;
  const int L0 = ld_input(p.seq_lens + b);
  const int base = p.base != nullptr ? ld_input(p.base + b) : 0;
  const int s0 = ld_input(p.keep_indptr + b), s1 = ld_input(p.keep_indptr + b + 1);
  const bool bad_len = L0 < 0 || L0 > max_len || base < 0 || base > L0;
  const bool bad_list = s0 < 0 || s1 < s0 || s1 > p.num_keep || (!bad_len && s1 - s0 > L0 - base);
  if (bad_len || bad_list) {
    if (first && threadIdx.x == 0) {
      record_error(p.err, bad_len ? ERR_SEQ_LEN : ERR_KEEP, bad_len ? (base < 0 || base > L0 ? base : L0) : s1);
      if (p.new_seq_lens != nullptr) p.new_seq_lens[b] = L0;
    }
    return;
  }
  const int count = s1 - s0;
  if (first && threadIdx.x == 0 && p.new_seq_lens != nullptr) p.new_seq_lens[b] = base + count;
  const int32_t* bt = p.block_table + (int64_t)b * p.max_blocks;
  char* pool = (tensor & 1) ? p.pools.value_pool[tensor >> 1] : p.pools.key_pool[tensor >> 1];
  for (int i0 = 0; i0 < count; i0 += tile) {
    // slots of the tile's rows; -1: nothing to move
    for (int r = threadIdx.x; r < tile; r += kCompactThreads) {
      int64_t f = -1, d = -1;
      const int i = i0 + r;
      if (i < count) {
        const int old = ld_input(p.keep + s0 + i), now = base + i;
        const int before = i > 0 ? ld_input(p.keep + s0 + i - 1) : now - 1;
        if (old < now || old >= L0 || old <= before) {
          if (first) record_error(p.err, ERR_KEEP, old);
        } else if (old != now) {
          const int pf = ld_input(bt + old / p.page_size), pt = ld_input(bt + now / p.page_size);
          if (pf < 0 || pf >= p.num_pages || pt < 0 || pt >= p.num_pages) {
            if (first) record_error(p.err, ERR_BLOCK_TABLE, pf < 0 || pf >= p.num_pages ? pf : pt);
          } else {
            f = (int64_t)pf * p.page_size + old % p.page_size;
            d = (int64_t)pt * p.page_size + now % p.page_size;
          }
        }
      }
      from[r] = f;
      to[r] = d;
    }
    __syncthreads();
    V v[kRowsAhead];
    if (x < nvec) {
#pragma unroll
      for (int k = 0; k < kRowsAhead; ++k) {
        const int64_t f = from[r0 + k * rows];
        if (f >= 0) v[k] = reinterpret_cast<const V*>(pool + f * p.row_bytes)[x];
      }
    }
    __syncthreads();  // every read of the tile before its first write
    if (x < nvec) {
#pragma unroll
      for (int k = 0; k < kRowsAhead; ++k) {
        const int64_t d = to[r0 + k * rows];
        if (d >= 0) reinterpret_cast<V*>(pool + d * p.row_bytes)[x] = v[k];
      }
    }
    __syncthreads();  // the slots are read: the next tile may write them
  }
}

template <typename V>
cudaError_t launch_compact_v(const CompactParams& p, int num_sms, cudaStream_t s) {
  const int64_t nvec = p.row_bytes / (int64_t)sizeof(V);
  const int64_t lists = 2 * (int64_t)p.pools.count * p.batch;
  // Wide segments while a tile still holds an average list, or while the grid
  // stays large enough to fill the GPU; else narrow ones (256 bytes at least)
  // that split a row over more blocks.
  int cols = kCompactThreads;
  while (cols > kMinCols && (cols / 2 >= nvec || (lists * ((nvec + cols - 1) / cols) < 8 * (int64_t)num_sms &&
                                            (int64_t)(kCompactThreads / cols) * kRowsAhead * p.batch < p.num_keep)))
    cols /= 2;
  const int64_t segs = (nvec + cols - 1) / cols;
  return launch_pdl(compact_kernel<V>, dim3((unsigned)segs, 2u * p.pools.count, (unsigned)p.batch),
                    dim3(kCompactThreads), 0, s, p, cols);
}

}  // namespace

cudaError_t launch_copy_pages(const CopyPagesParams& p, int vec_bytes, cudaStream_t s) {
  if (p.n <= 0 || p.pools.count <= 0) return cudaSuccess;
  switch (vec_bytes) {
    case 16: return launch_copy<uint4>(p, s);
    case 8: return launch_copy<uint2>(p, s);
    case 4: return launch_copy<uint32_t>(p, s);
    case 2: return launch_copy<unsigned short>(p, s);
    default: return launch_copy<unsigned char>(p, s);
  }
}

cudaError_t launch_compact(const CompactParams& p, int vec_bytes, int num_sms, cudaStream_t s) {
  if (p.batch <= 0 || p.pools.count <= 0) return cudaSuccess;
  switch (vec_bytes) {
    case 16: return launch_compact_v<uint4>(p, num_sms, s);
    case 8: return launch_compact_v<uint2>(p, num_sms, s);
    case 4: return launch_compact_v<uint32_t>(p, num_sms, s);
    case 2: return launch_compact_v<unsigned short>(p, num_sms, s);
    default: return launch_compact_v<unsigned char>(p, num_sms, s);
  }
}

}  // namespace pa
