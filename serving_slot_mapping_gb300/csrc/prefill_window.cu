// paged_attention_prefill_window: tcgen05 / TMEM varlen causal attention over a
// sliding window and the first tokens of each sequence, bf16 and e4m3 pools.
//
// Row i of sequence b is at position p = L_b - n_b + i and sees the keys
// j <= p with j > p - window or j < num_sinks.
//
// A CTA's work item is what it is in prefill_tc.cuh -- 256 packed rows of one
// (sequence, KV head) as two 128-row query tiles that share every staged tile of
// 128 keys, one TMA warp, one MMA thread, two softmax warpgroups (and two
// converter warps for e4m3 pools) -- with what short key ranges ask for:
// * The grid is persistent, one CTA per SM, and walks items w = blockIdx.x,
//   + gridDim.x, ... (KV head fastest, then 256-row tiles, then sequences).
//   A window of 1024 keys leaves an item ~10 key tiles; with a CTA for each item,
//   as the plain kernel has it, its start, first loads and last writes took 11 us
//   beside tiles of 1.9 us.  Here the TMA warp runs ahead into the next item's keys, the query
//   rows of the next item are copied in while the last key tile's softmax runs,
//   and its first S is multiplied while this item's rows are written.
// * Keys are staged as a list of page boxes, not as aligned tiles: the sinks'
//   boxes, then those from the first key the item's first row sees through
//   the window on.  A key's place in that list is its "logical" position:
//   key - gap for keys behind the skipped boxes, the key itself for the sinks;
//   the masks are ranges of logical positions.  So four sinks cost a box, not a
//   tile, and a window starts at a box, not at a multiple of 128.
// * Few items (a short chunk of one request): the SPLIT instantiations give an item
//   to a cluster of CTAs, each a part of its key tiles, and merge their rows
//   through distributed shared memory (see window_split).
// * The masks of a row of a 128-key tile are four 32-bit words, built once per
//   tile that needs any.
// Boxes whose page holds no key that a row of the sequence sees are never looked
// up; slots of loaded pages that no row of the sequence sees (between the sinks
// and the sequence's first window key, or at and past L_b) are zeroed in V.
// A block_table entry out of range is noted by the TMA warp; a CTA that met one
// computes the rows of its items with such a page again at its end, without their
// keys (redo_bad_items).  The loop knows nothing of them: masks told to the softmax by
// tile took 12 % (8 chunks of 512-2048, window 1024: 220 against 196 us).
#include <algorithm>
#include <type_traits>

#include "cluster.cuh"
#include "inputs.cuh"
#include "prefill_tc.cuh"

namespace pa {

namespace {

constexpr int kItems = 4;        // items whose geometry is in shared memory
constexpr int kItemBytes = 52;
constexpr int kWBars = 32;

enum { W_QFULL = 0, W_KFULL = W_QFULL + kQT, W_KEMPTY = W_KFULL + kNSK, W_VFULL = W_KEMPTY + kNSK,
       W_VEMPTY = W_VFULL + kNSV, W_SFULL = W_VEMPTY + kNSV, W_PFULL = W_SFULL + kQT, W_ODONE = W_PFULL + kQT,
       W_VLAND = W_ODONE + kQT, W_KREADY = W_VLAND + 1, W_VREADY = W_KREADY + kNSK, W_IFULL = W_VREADY + kNSV,
       W_IEMPTY = W_IFULL + kItems, W_COUNT = W_IEMPTY + kItems };
static_assert(W_COUNT <= kWBars, "barrier slots");

template <int D, bool KV8>
struct WCfg : PCfg<D, KV8> {
  using Base = PCfg<D, KV8>;
  // Three warpgroups of 168 registers a thread at launch (two idle warps fill the
  // third where there are no converters).  The third gives registers to the two
  // of the softmax, whose threads hold a whole row of S (128 fp32): 2 x 200 + 104
  // (2 x 192 + 120) = 3 x 168.
  static constexpr int kThreads = 384;
  static constexpr int kSoftmaxRegs = KV8 ? 192 : 200, kOtherRegs = KV8 ? 120 : 104;
  static_assert(2 * kSoftmaxRegs + kOtherRegs <= 3 * 168, "more registers than the launch has");
  // 8 tiles in flight: {KV head, valid, hid0, hid1} after the first slots of their boxes
  static constexpr int kMetaOff = Base::kPageOff + 8 * 32 * 4;
  static constexpr int kItemOff = kMetaOff + 8 * 16;
  static constexpr int kWBarOff = kItemOff + kItems * kItemBytes;
  static constexpr int kTmemOff = kWBarOff + kWBars * 8;  // the word that tcgen05.alloc writes, behind every barrier
  static_assert(kTmemOff >= kWBarOff + 8 * W_COUNT, "the TMEM base lies on a barrier");
  static constexpr int kBadOff = kTmemOff + 8;  // a page out of range was met
  static constexpr int kWSmem = kTmemOff + 16 + 1024;
  // SPLIT, once the item's products are done: its rows of O, fp32, padded against
  // bank conflicts, and their (reference max, sum) over the K and V rings
  static constexpr int kPartRow = D + 4;
  static constexpr int kPartMl = kQT * kBM * kPartRow * 4;
  static_assert(kPartMl + kQT * kBM * 8 <= (kNSK + kNSV) * Base::kKVTile, "an item's rows fit over the rings");
};

// Sequence b's rows [qs, qs + n) of q; n = 0 where query_start_loc is inconsistent.
__device__ __forceinline__ int seq_rows(const PrefillParams& p, int b, int* qs) {
  const int s0 = ld_input(p.query_start_loc + b), s1 = ld_input(p.query_start_loc + b + 1);
  *qs = s0;
  return (s0 < 0 || s1 < s0 || (int64_t)s1 > p.total_q) ? 0 : s1 - s0;
}

__host__ __device__ __forceinline__ int row_tiles(int64_t rows) { return (int)((rows + kQT * kBM - 1) / (kQT * kBM)); }

// One work item.  One warp derives it and hands it to the others through a ring
// in shared memory (deriving it takes ~1.4 us of dependent loads and divisions,
// which the softmax warps would add to every item): warp 10 for bf16 pools, the
// TMA warp for e4m3 pools, where warps 10 and 11 convert and clear the tiles.
struct Item {
  int b, hk, qs, L;
  int n;                  // new rows of the sequence; -1: no more items
  int first;              // position of the sequence's first new row
  int row0;               // the item's first packed row
  int head_keys, gap;     // logical position of key j: j below head_keys, else j - gap
  int seq_start;          // first key that the sequence's first row sees through the window
  int nt0, nt1;           // key tiles that the query tiles see
  int base;               // logical position of the first (SPLIT: this CTA's part of them)
  __device__ int nt() const { return max(nt0, nt1); }
};
static_assert(sizeof(Item) == kItemBytes, "ring entry");

// Walks the items of one CTA in order (whole warps only): 32 sequences at a
// time, lane i knows the row tiles of sequence base + i.
struct Walker {
  int base, total, incl;  // of the chunk; incl: tiles of its sequences up to this lane's
  int64_t before;         // tiles of the sequences before the chunk
  int64_t w;              // next item

  __device__ void load(const PrefillParams& p) {
    const int lane = threadIdx.x & 31, b = base + lane;
    int qs, c = 0;
    if (b < p.batch) c = row_tiles((int64_t)min(seq_rows(p, b, &qs), p.max_q_len) * p.group);
    incl = c;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int t = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += t;
    }
    total = __shfl_sync(0xffffffffu, incl, 31);
  }
  __device__ void start(const PrefillParams& p, int csize) {
    base = 0;
    before = 0;
    w = blockIdx.x / csize;
    load(p);
  }
  // The next item; false at the end.
  __device__ bool next(const PrefillParams& p, int kpo, int csize, Item* it) {
    const int Hkv = p.pool.num_kv_heads;
    const int64_t gt = w / Hkv;
    while (gt >= before + total) {
      if (base + 32 >= p.batch) return false;
      before += total;
      base += 32;
      load(p);
    }
    const int rel = (int)(gt - before);
    const int i = __popc(__ballot_sync(0xffffffffu, incl <= rel));  // < 32: rel < total
    const int tile = rel - (i > 0 ? __shfl_sync(0xffffffffu, incl, i - 1) : 0);
    it->b = base + i;
    it->hk = (int)(w - gt * Hkv);
    w += gridDim.x / csize;
    const int ps = p.pool.page_size;
    it->n = seq_rows(p, it->b, &it->qs);
    it->L = ld_seq_len(p.seq_lens, it->b, p.max_blocks * ps, nullptr);
    it->first = it->L - it->n;
    it->row0 = tile * kQT * kBM;
    const int G = p.group;
    const int rows = it->n * G;
    const int start = max(0, max(0, it->first + it->row0 / G) - p.window + 1);
    const int head_boxes = min((p.num_sinks + kpo - 1) / kpo, start / kpo);
    it->head_keys = head_boxes * kpo;
    it->gap = start / kpo * kpo - it->head_keys;
    it->seq_start = max(0, max(0, it->first) - p.window + 1);
    auto tiles = [&](int r0) {  // tiles up to the last row's own key
      if (r0 >= rows) return 0;
      const int pmax = it->first + (min(r0 + kBM, rows) - 1) / G;
      return pmax < 0 ? 0 : (pmax - it->gap) / kBN + 1;
    };
    it->nt0 = tiles(it->row0);
    it->nt1 = tiles(it->row0 + kBM);
    it->base = 0;
    if (csize > 1) {  // this CTA's part of the key tiles
      const int per = (it->nt() + csize - 1) / csize, j0 = (int)(blockIdx.x % csize) * per;
      it->nt0 = min(max(it->nt0 - j0, 0), per);
      it->nt1 = min(max(it->nt1 - j0, 0), per);
      it->base = j0 * kBN;
    }
    return true;
  }
};

// Bits 0 .. k of a word (none for k < 0).
__device__ __forceinline__ uint32_t bits_to(int k) {
  return k < 0 ? 0u : (k >= 31 ? 0xFFFFFFFFu : 0xFFFFFFFFu >> (31 - k));
}

// The larger of three; pairs of floats (first in the low half) for the packed
// fp32 instructions of sm_100+, each half rounded as the scalar one.
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ uint64_t pair(float lo, float hi) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(lo), "f"(hi));
  return d;
}
__device__ __forceinline__ float2 unpair(uint64_t x) {
  float2 d;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(d.x), "=f"(d.y) : "l"(x));
  return d;
}
__device__ __forceinline__ uint64_t fma_pair(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t add_pair(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// The items of this CTA (SPLIT: of its cluster) that have a page out of range in one
// of their key tiles, once all their rows are written: each row anew over the keys
// whose pages are in range, a warp a row and a key at a time.  An error path, slow.
template <int D, bool KV8>
__device__ __forceinline__ void redo_bad_items(const PrefillParams& p, int kpo, int csize) {
  constexpr int E = D / 32;  // a lane's dims
  const int lane = threadIdx.x & 31, warps = blockDim.x >> 5, ps = p.pool.page_size, G = p.group;
  const int worker = (int)(blockIdx.x % csize) * warps + (threadIdx.x >> 5), workers = csize * warps;
  auto element = [&](const void* pool, int64_t at) {
    if (KV8) {
      const uint32_t f = e4m3x2_lo_to_f16x2(static_cast<const unsigned char*>(pool)[at]);
      return __half2float(__ushort_as_half((unsigned short)(f & 0xFFFFu)));
    }
    return __bfloat162float(static_cast<const __nv_bfloat16*>(pool)[at]);
  };
  Walker wk;
  wk.start(p, csize);
  Item x;
  while (wk.next(p, kpo, csize, &x)) {
    const int32_t* bt = p.block_table + (int64_t)x.b * p.max_blocks;
    auto in_range = [&](int key) {
      const int page = ld_input(bt + (key >> p.pool.page_shift));
      return page >= 0 && page < p.pool.num_pages;
    };
    const int rows = min(kQT * kBM, x.n * G - x.row0);
    // its key tiles reach from the window of the first row to less than a tile past
    // the last row's own key; the keys there are seen by later rows at least
    const int lo = x.first + x.row0 / G, hi = x.first + (x.row0 + rows - 1) / G;
    bool bad = false;
    for (int m = lane; hi >= 0 && m * ps < min(x.L, hi + kBN); m += 32) {
      const int key = m * ps;
      if (key < p.num_sinks || key + ps > max(0, lo) - p.window + 1) bad |= !in_range(key);
    }
    if (!__any_sync(0xffffffffu, bad)) continue;
#pragma unroll 1
    for (int r = worker; r < rows; r += workers) {
      const int R = x.row0 + r, tok = R / G, pos = x.first + tok;
      const int64_t row = ((int64_t)(x.qs + tok) * p.num_q_heads + (int64_t)x.hk * G + (R - tok * G)) * D + lane * E;
      float q[E], o[E] = {}, m = -INFINITY, l = 0.f;
#pragma unroll
      for (int e = 0; e < E; ++e) q[e] = __bfloat162float(static_cast<const __nv_bfloat16*>(p.q)[row + e]) * p.scale_log2;
#pragma unroll 1
      for (int j = 0; j <= pos; ++j) {
        if (j >= p.num_sinks && j <= pos - p.window) j = pos - p.window + 1;
        if (!in_range(j)) continue;
        const int64_t page = ld_input(bt + (j >> p.pool.page_shift));
        const int64_t at = ((page * ps + (j & (ps - 1))) * p.pool.num_kv_heads + x.hk) * D + lane * E;
        float s = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) s = fmaf(q[e], element(p.pool.key_pool, at + e), s);
#pragma unroll
        for (int i = 16; i > 0; i >>= 1) s += __shfl_xor_sync(0xffffffffu, s, i);
        const float mn = fmaxf(m, s), a = fast_exp2(m - mn), w = fast_exp2(s - mn);
        m = mn;
        l = fmaf(l, a, w);
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = fmaf(o[e], a, w * element(p.pool.value_pool, at + e));
      }
      const float inv = l > 0.f ? p.v_scale / l : 0.f;
#pragma unroll
      for (int e = 0; e < E; ++e) static_cast<__nv_bfloat16*>(p.out)[row + e] = __float2bfloat16_rn(o[e] * inv);
    }
  }
}

// SPLIT: csize CTAs of a cluster share an item, and there are clusters for all
// items (a CTA has one item at most); else csize is 1.
template <int D, bool KV8, bool SPLIT>
__global__ void __launch_bounds__(WCfg<D, KV8>::kThreads, 1)
    prefill_window_kernel(const __grid_constant__ CUtensorMap tmap_k, const __grid_constant__ CUtensorMap tmap_v,
                          const __grid_constant__ PrefillParams p, int csize_arg) {
  const int csize = SPLIT ? csize_arg : 1;
  using C = WCfg<D, KV8>;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const int G = p.group, Hq = p.num_q_heads;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int ps = p.pool.page_size, pshift = p.pool.page_shift;
  const int kpo = ps < kBN ? ps : kBN;  // keys per box
  const int ops = kBN / kpo;
  unsigned char* q_s = smem + C::kQOff;
  const uint32_t k_base = smem_u32(smem + C::kKOff);
  const uint32_t v_base = smem_u32(smem + C::kVOff);
  const uint32_t bars = smem_u32(smem + C::kWBarOff);
  auto bar = [&](int i) { return bars + 8u * i; };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kTmemOff);
  int* slot_ring = reinterpret_cast<int*>(smem + C::kPageOff);  // [8 tiles][32 lanes] first slot of each box, -1: none
  volatile Item* item_ring = reinterpret_cast<volatile Item*>(smem + C::kItemOff);
  int4* meta = reinterpret_cast<int4*>(smem + C::kMetaOff);     // [8 tiles] {KV head, valid, hid0, hid1}

  volatile int* bad_page = reinterpret_cast<volatile int*>(smem + C::kBadOff);

  if (tid == 0) {
    *bad_page = 0;
    for (int t = 0; t < kQT; ++t) {
      mbar_init(bar(W_QFULL + t), kBM);
      mbar_init(bar(W_SFULL + t), 1);
      mbar_init(bar(W_PFULL + t), kBM);
      mbar_init(bar(W_ODONE + t), 1);
    }
    for (int s = 0; s < kNSK; ++s) {
      mbar_init(bar(W_KFULL + s), 1);
      mbar_init(bar(W_KEMPTY + s), 1);
      mbar_init(bar(W_KREADY + s), 1);
    }
    for (int s = 0; s < kNSV; ++s) {
      mbar_init(bar(W_VFULL + s), 1);
      mbar_init(bar(W_VEMPTY + s), 1);
      mbar_init(bar(W_VREADY + s), 1);
    }
    mbar_init(bar(W_VLAND), 1);
    for (int s = 0; s < kItems; ++s) {
      mbar_init(bar(W_IFULL + s), 1);
      mbar_init(bar(W_IEMPTY + s), 4 * kQT + 2 + (KV8 ? 2 : 0));  // each warp with a role
    }
    fence_mbar_init();
  }
  if (warp == kMmaWarp) tmem_alloc(smem_u32(tmem_slot), C::kTmemCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  // A scale below 0 is taken by the queries (negated as they are staged), a scale
  // of 0 too (zeros): the softmax then always has a positive one, and takes the max
  // over raw S and one fused multiply-add per exponential.
  const float sl2 = p.scale_log2 == 0.f ? 1.f : fabsf(p.scale_log2);
  griddep_launch_dependents();
  // before the first read of an input: any of them, the lengths and tables too, may
  // come from the kernel before (read ahead of this wait: 0.5 to 1.5 us less)
  griddep_wait();
  // inconsistent inputs are recorded once, whatever items there are
  for (int b = blockIdx.x * C::kThreads + tid; b < p.batch; b += gridDim.x * C::kThreads) {
    int qs;
    const int n = seq_rows(p, b, &qs);
    if (n == 0 && qs != ld_input(p.query_start_loc + b + 1)) record_error(p.err, ERR_QUERY_LOC, qs);
    if (n > p.max_q_len) record_error(p.err, ERR_QUERY_LOC, n);
    ld_seq_len(p.seq_lens, b, p.max_blocks * ps, p.err);
  }
  bool alive = true;
  Item it = {};
  // The i-th item of this CTA, for a whole warp (in order, each item once).
  auto read_item = [&](int i, Item* x) {
    const int s = i % kItems;
    if (alive) alive = mbar_wait(bar(W_IFULL + s), (uint32_t)((i / kItems) & 1), p.err);
    const volatile int* src = reinterpret_cast<const volatile int*>(item_ring + s);
    int* dst = reinterpret_cast<int*>(x);
#pragma unroll
    for (int k = 0; k < kItemBytes / 4; ++k) dst[k] = src[k];
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(W_IEMPTY + s));
    return alive && x->n >= 0;
  };
  // Derive the next item and hand it out as entry i (whole warp); false at the end.
  auto publish_next = [&](Walker& wk, int i) {
    Item x = {};
    const bool got = (!SPLIT || i == 0) && wk.next(p, kpo, csize, &x);
    if (!got) x.n = -1;
    if (lane == 0) {
      volatile int* dst = reinterpret_cast<volatile int*>(item_ring + i % kItems);
      const int* src = reinterpret_cast<const int*>(&x);
#pragma unroll
      for (int k = 0; k < kItemBytes / 4; ++k) dst[k] = src[k];
      mbar_arrive(bar(W_IFULL + i % kItems));
    }
    __syncwarp();
    return got;
  };
  if (warp >= 4 * kQT) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(C::kOtherRegs));
  if (warp == kTmaWarp) {
    // ======================= TMA producer (one warp) =======================
    // K tiles of all items in order, each as soon as its ring slot is free, and
    // the V tiles behind them (a V tile reuses the slots its K tile looked up).
    // The page ids of the next K tile are read while this one is issued.
    const uint32_t box_bytes = (uint32_t)kpo * D * (KV8 ? 1 : 2);
    auto box_key = [&](int j) {  // first key of this lane's box of tile j
      const int l = it.base + j * kBN + lane * kpo;
      return l < it.head_keys ? l : l + it.gap;
    };
    auto box_used = [&](int key) {  // a box with a key that some row of the sequence sees
      return lane < ops && key < it.L && (key < p.num_sinks || key + kpo > it.seq_start);
    };
    const int32_t* bt = nullptr;
    auto fetch = [&](int j) {  // raw block_table entry of this lane's box of tile j
      const int key = box_key(j);
      return box_used(key) ? ld_input(bt + (key >> pshift)) : -1;
    };
    auto issue = [&](const CUtensorMap* map, uint32_t dst, int hk, int slot, uint32_t full) {
      const bool ok = slot >= 0;
      const int cnt = __popc(__ballot_sync(0xffffffffu, ok));
      if (lane == 0) mbar_arrive_expect_tx(full, (uint32_t)cnt * box_bytes);
      __syncwarp();
      if (ok) {
        if (KV8)  // codes in the ring slot's upper half, [keys][D B]
          tma_load_3d(dst + (uint32_t)(kBN * D + lane * kpo * D), map, 0, slot, hk, full);
        else
          tma_load_5d(dst + (uint32_t)(lane * (kpo / 8)) * C::kRowBlock, map, 0, 0, 0, slot >> 3, hk, full);
      }
    };
    auto phase_done = [&](int b, uint32_t parity) {  // lane 0 polls, the warp agrees
      int t = 0;
      if (lane == 0) t = mbar_test(bar(b), parity) ? 1 : 0;
      return __shfl_sync(0xffffffffu, t, 0) != 0;
    };
    Walker wk;
    if (KV8) wk.start(p, csize);
    int pub = 0, seen = 0;      // items handed out, items taken for their K tiles
    bool all_out = !KV8;        // the last entry says that there are no more
    int j = 0, raw = -1;
    bool more = false, end = false;  // `it` has a K tile j left to issue; no item is left
    int kt = 0, vt = 0;  // tiles issued so far, over all items
    int land_slot = -1;  // ring slot of a V tile whose rows are to be cleared when it has landed
    int4 land = make_int4(0, 0, 0, 0);
    uint32_t land_phase = 0;
    unsigned long long t_last = global_ns();
    while ((!end || vt < kt || land_slot >= 0) && alive) {
      bool progressed = false;
      if (!all_out && (pub < kItems || phase_done(W_IEMPTY + pub % kItems, (uint32_t)((pub / kItems - 1) & 1)))) {
        all_out = !publish_next(wk, pub);
        ++pub;
        progressed = true;
      }
      if (!more && !end && (KV8 ? seen < pub : phase_done(W_IFULL + seen % kItems, (uint32_t)((seen / kItems) & 1)))) {
        end = !read_item(seen, &it);
        ++seen;
        more = !end && it.nt() > 0;
        j = 0;
        if (more) {
          bt = p.block_table + (int64_t)it.b * p.max_blocks;
          raw = fetch(0);
        }
        progressed = true;
      }
      if (more && (kt < kNSK || phase_done(W_KEMPTY + kt % kNSK, (uint32_t)((kt / kNSK - 1) & 1)))) {
        const int key = box_key(j);
        int slot = -1;
        if (box_used(key)) {
          if (raw < 0 || raw >= p.pool.num_pages) {
            record_error(p.err, ERR_BLOCK_TABLE, raw);
            *bad_page = 1;
          } else {
            slot = (int)(((int64_t)raw << pshift) + (key & (ps - 1)));
          }
        }
        slot_ring[(kt & 7) * 32 + lane] = slot;
        if (lane == 0) {
          const int l0 = it.base + j * kBN;  // rows of the tile: valid ones, and those no row of the sequence sees
          const int end = it.seq_start <= it.head_keys ? it.seq_start : max(it.head_keys, it.seq_start - it.gap);
          meta[kt & 7] = make_int4(it.hk, min(it.L - it.gap - l0, kBN), max(0, p.num_sinks - l0), min(end - l0, kBN));
        }
        issue(&tmap_k, k_base + (kt % kNSK) * C::kKVTile, it.hk, slot, bar(W_KFULL + kt % kNSK));
        ++kt;
        more = ++j < it.nt();
        if (more) raw = fetch(j);
        progressed = true;
      }
      if (vt < kt && (vt < kNSV || phase_done(W_VEMPTY + vt % kNSV, (uint32_t)((vt / kNSV - 1) & 1)))) {
        const int4 m = meta[vt & 7];
        // rows that may hold anything meet P = 0 and must be zeros (e4m3: the converter writes them)
        const bool clear = !KV8 && (m.y < kBN || m.z < m.w);
        if (!clear || land_slot < 0) {
          const int s = vt % kNSV;
          issue(&tmap_v, v_base + s * C::kKVTile, m.x, slot_ring[(vt & 7) * 32 + lane],
                bar(clear ? (int)W_VLAND : W_VFULL + s));
          if (clear) {
            land_slot = s;
            land = m;
          }
          ++vt;
          progressed = true;
        }
      }
      if (land_slot >= 0 && phase_done(W_VLAND, land_phase)) {
        unsigned char* vtile = smem + C::kVOff + land_slot * C::kKVTile;
        auto clear_rows = [&](int lo, int hi) {
          for (int i = lane; i < (hi - lo) * (D / 8); i += 32) {
            const int k = lo + i / (D / 8), c = i % (D / 8);
            *reinterpret_cast<uint4*>(vtile + (k >> 3) * C::kRowBlock + (c >> 3) * 1024 + (k & 7) * 128 +
                                      (c & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
          }
        };
        clear_rows(land.y, kBN);
        clear_rows(land.z, land.w);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(W_VFULL + land_slot));
        land_slot = -1;
        land_phase ^= 1u;
        progressed = true;
      }
      int give_up = 0;
      if (lane == 0) {
        const unsigned long long now = global_ns();
        if (progressed) {
          t_last = now;
        } else if (now - t_last > kWaitLimitNs) {
          record_error(p.err, ERR_TIMEOUT, vt);
          give_up = 1;
        }
      }
      if (__shfl_sync(0xffffffffu, give_up, 0)) alive = false;
      if (!progressed) __nanosleep(32);
    }
  }

  if (!KV8 && warp == kCvtWarp) {
    // ======================= items, bf16 pools =======================
    Walker wk;
    wk.start(p, csize);
    for (int i = 0;; ++i) {
      if (i >= kItems)
        alive = __all_sync(0xffffffffu, mbar_wait(bar(W_IEMPTY + i % kItems), (uint32_t)((i / kItems - 1) & 1), p.err));
      if (!publish_next(wk, i) || !alive) break;
    }
  }

  if (KV8 && (warp == kCvtWarp || warp == kCvtWarp + 1)) {
    // ======================= e4m3 -> f16 converters (K: warp 10, V: warp 11) =======================
    const bool isv = warp == kCvtWarp + 1;
    const int nslots = isv ? kNSV : kNSK;
    for (int i = 0, kt = 0; read_item(i, &it); ++i) {
      for (int j = 0; j < it.nt() && alive; ++j, ++kt) {
        const int sl = kt % nslots;
        alive = __all_sync(0xffffffffu, mbar_wait(bar((isv ? W_VFULL : W_KFULL) + sl),
                                                  (uint32_t)((kt / nslots) & 1), p.err));
        const int4 m = meta[kt & 7];
        convert_tile_e4m3<D>(smem + (isv ? C::kVOff : C::kKOff) + sl * C::kKVTile, m.y, lane, m.z, m.w);
        fence_proxy_async_smem();  // the f16 tile before the tensor core reads it
        __syncwarp();
        if (lane == 0) mbar_arrive(bar((isv ? W_VREADY : W_KREADY) + sl));
      }
    }
  }

  if (warp == kMmaWarp) {
    // ======================= MMA issuer (lane 0) =======================
    // Per item S_A(0) S_B(0), then per key tile j: PV_A(j) S_A(j+1) PV_B(j)
    // S_B(j+1), as in prefill_tc.cuh, with the next item's S_A(0) and S_B(0) in the
    // places of S_A and S_B past this item's last tiles.  tcgen05 operations of
    // one thread execute in order, so the next item's S may overwrite this item's
    // last P; its first PV overwrites O only after the softmax threads, which
    // write its P, have read this item's O.
    constexpr uint32_t idesc_s = KV8 ? umma_idesc_f16(kBM, kBN, false) : umma_idesc_bf16(kBM, kBN, false);
    constexpr uint32_t idesc_o = KV8 ? umma_idesc_f16(kBM, D, true) : umma_idesc_bf16(kBM, D, true);
    constexpr int kKWait = KV8 ? W_KREADY : W_KFULL, kVWait = KV8 ? W_VREADY : W_VFULL;
    const uint64_t q_desc = umma_desc_sw128(smem_u32(q_s), 16, 1024);
    const uint64_t k_desc = umma_desc_sw128(k_base, 16, C::kRowBlock);
    const uint64_t v_desc = umma_desc_sw128(v_base, 1024, C::kRowBlock);
    int kt0 = 0;                                         // key tiles of the items before
    uint32_t items[kQT] = {0u, 0u}, sp[kQT] = {0u, 0u};  // per query tile: items with keys, P tiles awaited
    bool begun[kQT] = {false, false};                    // the item's S_t(0) is issued
    Item nx;
    int taken = 1;
    bool have = read_item(0, &nx);
    while (have) {
      it = nx;
      have = read_item(taken++, &nx);
      if (lane == 0) {
        const int nt0 = it.nt0, nt1 = it.nt1, nt = it.nt();
        // S_t of key tile j of an item whose tiles start at k0: wait for K where
        // this is the first S of the tile, free its stage where it is the last
        auto issue_s = [&](const Item& x, int k0, int t, int j) {
          const int kt = k0 + j, sk = kt % kNSK;
          if (t == 0 || j >= x.nt0) {
            if (alive) alive = mbar_wait(bar(kKWait + sk), (uint32_t)((kt / kNSK) & 1), p.err);
          }
          tc_fence_after();
          const uint64_t qd = q_desc + (uint64_t)((t * C::kQBytes) >> 4);
          const uint64_t kd = k_desc + (uint64_t)((sk * C::kKVTile) >> 4);
          const uint32_t s_tm = tmem + C::kSCol + t * 128;
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)  // S_t = Q_t K^T over 16-dim steps
            umma_bf16(s_tm, qd + (uint64_t)(((kk >> 2) * kSlab + (kk & 3) * 32) >> 4),
                      kd + (uint64_t)(((kk >> 2) * 1024 + (kk & 3) * 32) >> 4), idesc_s, kk > 0);
          umma_commit(bar(W_SFULL + t));
          if (t == 1 || j >= x.nt1) umma_commit(bar(W_KEMPTY + sk));
        };
        auto issue_pv = [&](int t, int j) {
          const int kt = kt0 + j, sv = kt % kNSV;
          if (alive) alive = mbar_wait(bar(W_PFULL + t), sp[t] & 1u, p.err);
          ++sp[t];
          if (t == 0 || j >= nt0) {  // first PV of key tile j
            if (alive) alive = mbar_wait(bar(kVWait + sv), (uint32_t)((kt / kNSV) & 1), p.err);
          }
          tc_fence_after();
          const uint64_t vd = v_desc + (uint64_t)((sv * C::kKVTile) >> 4);
          const uint32_t s_tm = tmem + C::kSCol + t * 128;
          const uint32_t o_tm = tmem + C::kOCol + t * 128;
#pragma unroll
          for (int kk = 0; kk < kBN / 16; ++kk)  // O_t += P_t V over 16-key steps (two 8-key blocks each)
            umma_bf16_ts(o_tm, s_tm + kk * 8, vd + (uint64_t)((kk * 2 * C::kRowBlock) >> 4), idesc_o,
                         (j > 0 || kk > 0) ? 1u : 0u);
          if (j == (t ? nt1 : nt0) - 1) umma_commit(bar(W_ODONE + t));
          if (t == 1 || j >= nt1) umma_commit(bar(W_VEMPTY + sv));  // last PV of key tile j
        };
        auto begin = [&](const Item& x, int k0, int t) {
          if (alive) alive = mbar_wait(bar(W_QFULL + t), items[t] & 1u, p.err);
          ++items[t];
          issue_s(x, k0, t, 0);
        };
        for (int t = 0; t < kQT; ++t) {
          if (!begun[t] && (t ? nt1 : nt0) > 0) begin(it, kt0, t);
          begun[t] = false;
        }
        for (int j = 0; j < nt; ++j) {
          if (j < nt0) {
            issue_pv(0, j);
            if (j + 1 < nt0) {
              issue_s(it, kt0, 0, j + 1);
            } else if (have && nx.nt0 > 0) {
              begin(nx, kt0 + nt, 0);
              begun[0] = true;
            }
          }
          if (j < nt1) {
            issue_pv(1, j);
            if (j + 1 < nt1) {
              issue_s(it, kt0, 1, j + 1);
            } else if (have && nx.nt1 > 0 && (begun[0] || nx.nt0 == 0)) {  // never ahead of S_A(0)
              begin(nx, kt0 + nt, 1);
              begun[1] = true;
            }
          }
        }
        kt0 += nt;
      }
      __syncwarp();
    }
  }

  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(C::kSoftmaxRegs));
    // ======================= softmax: one TMEM lane (row) per thread =======================
    const int t = warp >> 2;                 // query tile
    const int r = tid & (kBM - 1);           // row within the tile == TMEM lane
    const __nv_bfloat16* qp = static_cast<const __nv_bfloat16*>(p.q);
    __nv_bfloat16* outp = static_cast<__nv_bfloat16*>(p.out);
    unsigned char* qt = q_s + t * C::kQBytes;
    const uint32_t lane_base = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t s_col = lane_base + C::kSCol + t * 128;
    const uint32_t o_col = lane_base + C::kOCol + t * 128;
    auto tiles_of = [&](const Item& x) { return t ? x.nt1 : x.nt0; };
    auto row_of = [&](const Item& x) { return x.row0 + t * kBM + r; };
    auto row_off = [&](const Item& x, int R) {  // packed row -> element offset of its q / out row
      const int i = R / G, g = R - (R / G) * G;
      return ((int64_t)(x.qs + i) * Hq + (int64_t)x.hk * G + g) * D;
    };
    auto q_chunk = [&](int row, int c) { return qt + (c >> 3) * kSlab + row * 128 + (((c & 7) ^ (row & 7)) << 4); };
    // the warp's 32 Q rows into the UMMA A layout (K-major, 128-byte swizzle),
    // whole rows of D / 8 chunks a time; zeros past the last row
    constexpr int kRowLanes = D / 8, kRowsPerCopy = 32 / kRowLanes;
    auto copy_q = [&](const Item& x) {
      const int R = row_of(x);
      const long long off = R < x.n * G ? row_off(x, R) : -1;
#pragma unroll
      for (int i = 0; i < 32; i += kRowsPerCopy) {
        const int src_lane = i + lane / kRowLanes, c = lane % kRowLanes;
        const long long o = __shfl_sync(0xffffffffu, off, src_lane);
        cp_async_16(smem_u32(q_chunk((warp & 3) * 32 + src_lane, c)), qp + (o < 0 ? 0 : o) + c * 8, o < 0 ? 0 : 16);
      }
      cp_async_commit();
    };
    auto publish_q = [&]() {
      cp_async_wait<0>();
      if (KV8) {  // f16 operands: bf16 -> f16 in place, each thread its row
        __syncwarp();
#pragma unroll 4
        for (int c = 0; c < D / 8; ++c) {
          uint4* x = reinterpret_cast<uint4*>(q_chunk(r, c));
          const uint4 v = *x;
          *x = make_uint4(bf16x2_to_f16x2(v.x), bf16x2_to_f16x2(v.y), bf16x2_to_f16x2(v.z), bf16x2_to_f16x2(v.w));
        }
      }
      if (p.scale_log2 <= 0.f) {
        __syncwarp();
#pragma unroll 1
        for (int c = 0; c < D / 8; ++c) {
          uint4* x = reinterpret_cast<uint4*>(q_chunk(r, c));
          const uint32_t keep = p.scale_log2 < 0.f ? 0xFFFFFFFFu : 0u, flip = p.scale_log2 < 0.f ? 0x80008000u : 0u;
          const uint4 v = *x;
          *x = make_uint4((v.x & keep) ^ flip, (v.y & keep) ^ flip, (v.z & keep) ^ flip, (v.w & keep) ^ flip);
        }
      }
      fence_proxy_async_smem();
      mbar_arrive(bar(W_QFULL + t));
    };
    Item nx;
    int taken = 1;
    bool have = read_item(0, &nx);
    if (have && tiles_of(nx) > 0) {
      copy_q(nx);
      publish_q();
    }
    uint32_t sn = 0, on = 0;  // S tiles and finished O's awaited so far
    while (have) {
      it = nx;
      const int ntt = tiles_of(it);
      have = read_item(taken++, &nx);
      const bool next_q = have && tiles_of(nx) > 0;
      const int R = row_of(it);
      const int rows = it.n * G;
      const bool valid_row = R < rows;
      // logical positions: this row's own key, the first key of its window; the
      // least own key and the last window start among the tile's rows
      const int pos = valid_row ? it.first + R / G : -1;
      const int lim = pos - it.gap;
      const int wlo = max(0, max(0, pos) - p.window + 1) - it.gap;
      const int lim_min = it.first + (it.row0 + t * kBM) / G - it.gap;
      const int pos_max = it.first + (min(it.row0 + (t + 1) * kBM, rows) - 1) / G;
      const int wlo_max = max(0, max(0, pos_max) - p.window + 1) - it.gap;
      float m_ref = -INFINITY, l = 0.f;
      for (int j = 0; j < ntt; ++j) {
        if (alive) alive = mbar_wait(bar(W_SFULL + t), sn & 1u, p.err);
        ++sn;
        tc_fence_after();
        // every S of this item is done: Q may be replaced
        if (j == ntt - 1 && next_q) copy_q(nx);
        const int l0 = it.base + j * kBN;
        // some row does not see some key of the tile
        const bool masked = l0 + kBN - 1 > lim_min || (l0 < wlo_max && l0 + kBN > p.num_sinks);
        // the row of S, and its max
        uint32_t v[4][32];
#pragma unroll
        for (int i = 0; i < 4; ++i) tmem_ld32(s_col + i * 32, v[i]);
        tmem_wait_ld();
        if (masked) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int c0 = l0 + 32 * i;
            const uint32_t see = bits_to(lim - c0) & (~bits_to(wlo - 1 - c0) | bits_to(p.num_sinks - 1 - c0));
#pragma unroll
            for (int e = 0; e < 32; ++e) v[i][e] = ((see >> e) & 1u) ? v[i][e] : 0xFF800000u;
          }
        }
        float mx[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          mx[i] = __uint_as_float(v[i][0]);
#pragma unroll
          for (int e = 1; e < 31; e += 2) mx[i] = max3(mx[i], __uint_as_float(v[i][e]), __uint_as_float(v[i][e + 1]));
          mx[i] = fmaxf(mx[i], __uint_as_float(v[i][31]));
        }
        float tmax = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
        tmax *= sl2;
        // reference max: moved only when the row max grows by more than 2^8
        float alpha = 1.f;
        bool rescale = false;
        if (tmax > m_ref + kRescaleThreshold) {
          alpha = m_ref == -INFINITY ? 0.f : fast_exp2(m_ref - tmax);
          m_ref = tmax;
          l *= alpha;
          rescale = j > 0;
        }
        const float mbase = m_ref == -INFINITY ? 0.f : m_ref;
        // P = exp2(x - m) as bf16 (f16) pairs, written over the S columns: V's type, the one that the product takes
        // beside it; l sums the fp32 ones.  Against 64 bits an output is off by 0.0023 of its norm so (codes:
        // 0.0017), by 0.0017 with its own rounding alone
        const uint64_t mul = pair(sl2, sl2), sub = pair(-mbase, -mbase);
        uint64_t rs[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t w[32];
#pragma unroll
          for (int cb = 0; cb < 2; ++cb)
#pragma unroll
            for (int e = 0; e < 32; e += 2) {
              const float2 x = unpair(fma_pair(
                  pair(__uint_as_float(v[2 * h + cb][e]), __uint_as_float(v[2 * h + cb][e + 1])), mul, sub));
              const float p0 = fast_exp2(x.x), p1 = fast_exp2(x.y);
              rs[(e >> 1) & 3] = add_pair(rs[(e >> 1) & 3], pair(p0, p1));
              w[cb * 16 + (e >> 1)] = KV8 ? pack_f16(p0, p1) : pack_bf16(p0, p1);
            }
          tmem_st32(s_col + h * 32, w);
        }
        const float2 sum = unpair(add_pair(add_pair(rs[0], rs[1]), add_pair(rs[2], rs[3])));
        l += sum.x + sum.y;
        // O is rescaled in place only when some row of the warp moved its
        // reference max.  PV_t(j-1) is complete: S_t(j) was issued after it.
        if (__any_sync(0xffffffffu, rescale)) {
#pragma unroll 1
          for (int cb = 0; cb < D / 32; ++cb) {
            uint32_t o[32];
            tmem_ld32(o_col + cb * 32, o);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
            tmem_st32(o_col + cb * 32, o);
          }
        }
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(bar(W_PFULL + t));
      }
      if (next_q) {
        if (ntt == 0) copy_q(nx);
        publish_q();
      }
      // ---- O / l -> bf16 (zeros for a tile that sees no key) ----
      if (ntt > 0) {
        if (alive) alive = mbar_wait(bar(W_ODONE + t), on & 1u, p.err);
        ++on;
        tc_fence_after();
      }
      if constexpr (SPLIT) {
        // the row unnormalised over the rings, once the other query tile's
        // products have read them too
        named_barrier(1, kQT * kBM);
        float* row = reinterpret_cast<float*>(smem + C::kKOff) + (t * kBM + r) * C::kPartRow;
        reinterpret_cast<float2*>(smem + C::kKOff + C::kPartMl)[t * kBM + r] = make_float2(m_ref, l);
        if (ntt > 0) {
#pragma unroll
          for (int cb = 0; cb < D / 32; ++cb) {
            uint32_t o[32];
            tmem_ld32(o_col + cb * 32, o);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; e += 4)
              *reinterpret_cast<uint4*>(row + cb * 32 + e) = make_uint4(o[e], o[e + 1], o[e + 2], o[e + 3]);
          }
        }
        continue;
      }
      // A quad of lanes holds four rows of 64 bytes per 32 columns; they are
      // transposed within the quad (16-byte units), so that a store covers 64
      // contiguous bytes of 8 rows and not 16 of 32.
      const float inv = l > 0.f ? p.v_scale / l : 0.f;  // v_scale: 1 for bf16 pools
      const long long off = valid_row ? row_off(it, R) : -1;
      long long dst[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) dst[k] = __shfl_sync(0xffffffffu, off, (lane & ~3) + k);
      uint32_t oall[D / 32][32];
#pragma unroll
      for (int cb = 0; cb < D / 32; ++cb)
        if (ntt > 0) {
          tmem_ld32(o_col + cb * 32, oall[cb]);
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e) oall[cb][e] = 0u;
        }
      if (ntt > 0) tmem_wait_ld();
#pragma unroll
      for (int cb = 0; cb < D / 32; ++cb) {
        const uint32_t (&o)[32] = oall[cb];
        uint32_t w[4][4];  // unit u: columns 8u .. 8u + 7
#pragma unroll
        for (int u = 0; u < 4; ++u)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            w[u][i] = pack_bf16(__uint_as_float(o[8 * u + 2 * i]) * inv, __uint_as_float(o[8 * u + 2 * i + 1]) * inv);
#pragma unroll
        for (int s = 1; s < 4; s <<= 1) {
          const bool odd = (lane & s) != 0;
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            if (u & s) continue;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint32_t got = __shfl_xor_sync(0xffffffffu, odd ? w[u][i] : w[u | s][i], s);
              if (odd) w[u][i] = got; else w[u | s][i] = got;
            }
          }
        }
#pragma unroll
        for (int k = 0; k < 4; ++k)  // row k of the quad, this lane's unit of it
          if (dst[k] >= 0)
            *reinterpret_cast<uint4*>(outp + dst[k] + cb * 32 + (lane & 3) * 8) =
                make_uint4(w[k][0], w[k][1], w[k][2], w[k][3]);
      }
      tc_fence_before();  // O is read before this thread's next P lets PV write it again
    }
  }

  // ---- teardown: every warp reaches this point; TMEM is freed by its allocator warp ----
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kMmaWarp) tmem_dealloc(tmem, C::kTmemCols);
  bool redo = *bad_page != 0;
  if constexpr (SPLIT) {
    // ======================= the cluster's parts joined =======================
    // o = v_scale sum_c 2^(m_c - M) o_c / sum_c 2^(m_c - M) l_c; each CTA a part of
    // the item's rows, 4 dims a thread.
    cluster_sync();
    const Item x = *const_cast<const Item*>(item_ring);
    const int rank = (int)(blockIdx.x % csize);
    if (x.n >= 0) {
      const uint32_t part = smem_u32(smem + C::kKOff), part_ml = part + C::kPartMl;
      const int rows = min(kQT * kBM, x.n * G - x.row0);
      // 16 loads of a thread in flight whatever the cluster's size
      auto join = [&](auto size) {
        constexpr int N = decltype(size)::value, U = 8 / N;
        const int total = rows * (D / 4), step = N * C::kThreads;
        for (int i0 = rank * C::kThreads + tid; i0 < total; i0 += U * step) {
          float2 ml[U][N];
          float4 v[U][N];
#pragma unroll
          for (int k = 0; k < U; ++k) {
            const int i = min(i0 + k * step, total - 1), r = i / (D / 4), c = i - r * (D / 4);
#pragma unroll
            for (int q = 0; q < N; ++q) {
              ml[k][q] = ld_cluster2(map_rank(part_ml + 8u * r, q));
              v[k][q] = ld_cluster4(map_rank(part + 4u * (r * C::kPartRow + 4 * c), q));
            }
          }
#pragma unroll
          for (int k = 0; k < U; ++k) {
            const int i = i0 + k * step, r = i / (D / 4), c = i - r * (D / 4);
            if (i >= total) break;
            float M = -INFINITY, den = 0.f;
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int q = 0; q < N; ++q) M = fmaxf(M, ml[k][q].x);
#pragma unroll
            for (int q = 0; q < N; ++q) {
              if (ml[k][q].x == -INFINITY) continue;  // a part without a visible key: its row is not written
              const float f = fast_exp2(ml[k][q].x - M);
              den += f * ml[k][q].y;
              acc.x += f * v[k][q].x; acc.y += f * v[k][q].y; acc.z += f * v[k][q].z; acc.w += f * v[k][q].w;
            }
            const float inv = den > 0.f ? p.v_scale / den : 0.f;
            const int R = x.row0 + r, tok = R / G;
            const int64_t at = ((int64_t)(x.qs + tok) * Hq + (int64_t)x.hk * G + (R - tok * G)) * D + 4 * c;
            *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.out) + at) =
                make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
          }
        }
      };
      if (csize == 2) join(std::integral_constant<int, 2>());
      else if (csize == 4) join(std::integral_constant<int, 4>());
      else join(std::integral_constant<int, 8>());
    }
    for (int c = 0; c < csize; ++c) redo |= ld_cluster(map_rank(smem_u32(smem + C::kBadOff), c)) != 0u;
    cluster_sync();  // no CTA leaves while another reads its memory; every row of the item is written
  }
  if (__builtin_expect(redo, 0)) redo_bad_items<D, KV8>(p, kpo, csize);
}

// CTAs of an item: one where the items fill the SMs; else as many (a power of two
// up to 8, with two key tiles each at least) as the SMs hold at once (four fifths
// of them for clusters of 4 and 8, which do not fill every SM).  32 / 8 heads of 128 on one CTA an item
// and so split: 512 tokens, window 1024 25.2 and 22.8 us (2 CTAs); 128 tokens 25.0
// and 18.4 us (4); 64 tokens, window 4096 71.7 and 22.7 us (4).
int window_split(int num_sms, int64_t items, int64_t max_keys) {
  const int64_t tiles = (max_keys + kBN - 1) / kBN;
  int c = 1;
  while (c < 8 && items * 2 * c <= (c == 1 ? (int64_t)num_sms : (int64_t)num_sms * 4 / 5) && tiles >= 4 * c) c *= 2;
  return c;
}

template <int D, bool KV8, bool SPLIT>
cudaError_t launch_items(const PrefillParams& p, const CUtensorMap& tk, const CUtensorMap& tv, unsigned grid, int csize,
                         cudaStream_t s) {
  using C = WCfg<D, KV8>;
  auto kern = prefill_window_kernel<D, KV8, SPLIT>;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kWSmem);
  if (e != cudaSuccess) return e;
  if (!SPLIT) return launch_pdl(kern, dim3(grid), dim3(C::kThreads), (size_t)C::kWSmem, s, tk, tv, p, 1);
  return launch_pdl_cluster(kern, dim3(grid), dim3(C::kThreads), (size_t)C::kWSmem, csize, s, tk, tv, p, csize);
}

template <int D, bool KV8>
cudaError_t launch_window(const PrefillParams& p, int num_sms, cudaStream_t s) {
  CUtensorMap tk, tv;
  if (!encode_prefill_tmaps<D, KV8>(p, &tk, &tv)) return cudaErrorInvalidValue;
  // items: at most a partial tile per sequence beside the full ones, and at most
  // the longest sequence's for each
  const int64_t tiles = std::min<int64_t>(p.total_q * p.group / (kQT * kBM) + p.batch,
                                          (int64_t)p.batch * row_tiles((int64_t)p.max_q_len * p.group));
  const int64_t items = tiles * p.pool.num_kv_heads;
  const int64_t keys = std::min<int64_t>((int64_t)p.max_blocks * p.pool.page_size,
                                         (int64_t)p.window + p.num_sinks + kQT * kBM / p.group);
  const int csize = window_split(num_sms, items, keys);
  if (csize > 1) return launch_items<D, KV8, true>(p, tk, tv, (unsigned)(items * csize), csize, s);
  return launch_items<D, KV8, false>(p, tk, tv, (unsigned)(items < num_sms ? items : num_sms), 1, s);
}

}  // namespace

cudaError_t launch_prefill_window(const PrefillParams& p, int num_sms, cudaStream_t s) {
  if (p.max_q_len <= 0 || p.batch <= 0) return cudaSuccess;
  if (p.pool.page_size < 8 || p.pool.page_shift < 0) return cudaErrorInvalidValue;
  if (p.kv8) return p.pool.head_dim == 128 ? launch_window<128, true>(p, num_sms, s) : launch_window<64, true>(p, num_sms, s);
  return p.pool.head_dim == 128 ? launch_window<128, false>(p, num_sms, s) : launch_window<64, false>(p, num_sms, s);
}

}  // namespace pa
