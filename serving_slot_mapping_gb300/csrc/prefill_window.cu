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
// int8 pools (SC; paged_attention_prefill_int8, a window that reaches every key): the
// codes land as they are, in stages of their own, and become f16 exactly.  A tile's 16-key
// blocks each have a scale for K and one for V, k and v, which reach a row only through
// the columns that it sees:
// * warp 10 looks the scales up ahead and hands out, per tile, {scale * k, log2 v, 1 / v}
//   of its 8 blocks (a ring of four tiles);
// * four converter warps take the tiles in the order that the products ask for them,
//   K(0), then K(t + 1), V(t);
// * k goes into the factor of S that the softmax has anyway, log2 v into the exponent, as
//   in decode_split.cuh: y = x + log2 v, the reference max m follows y, P = 2^(y - m)
//   stays in f16's range whatever the scales of the visible blocks are, and l sums P / v.
//   y is rounded before m is taken off it, so that the largest P is 1 however large the
//   scores are: an addition for two elements of S, beside the fused multiply-add (8 chunks
//   of 512-2048 after 0-8192 tokens, 32 / 8 heads of 128: 933 us, without it 919; behind a
//   branch that only large scores take 997 where the plain addition took 957).
//   (Scales multiplied into the codes, relative to their tile's largest, took 940 us where
//   this takes 958, and cost a row its keys' last bits for the sake of blocks that it does
//   not see.)
// Sixteen warps for that: 2 x 144 + 2 x 112 registers a thread, and the softmax in loops
// of 32 columns: written out, it and the conversion did not fit in the instruction cache.
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
constexpr int kWBars = 40;
constexpr int kScaleTiles = 4;   // int8: tiles whose scales are in shared memory
constexpr int kScaleBytes = 128;
constexpr int kI8Warps = 4;      // int8: converter warps 12 .. 15; warp 10 hands out items and scales

enum { W_QFULL = 0, W_KFULL = W_QFULL + kQT, W_KEMPTY = W_KFULL + kNSK, W_VFULL = W_KEMPTY + kNSK,
       W_VEMPTY = W_VFULL + kNSV, W_SFULL = W_VEMPTY + kNSV, W_PFULL = W_SFULL + kQT, W_ODONE = W_PFULL + kQT,
       W_VLAND = W_ODONE + kQT, W_KREADY = W_VLAND + 1, W_VREADY = W_KREADY + kNSK, W_IFULL = W_VREADY + kNSV,
       W_IEMPTY = W_IFULL + kItems, W_CFULL = W_IEMPTY + kItems, W_CEMPTY = W_CFULL + kScaleTiles,
       W_COUNT = W_CEMPTY + kScaleTiles };
static_assert(W_COUNT <= kWBars, "barrier slots");

template <int D, bool KV8, bool SC = false>
struct WCfg : PCfg<D, KV8> {
  using Base = PCfg<D, KV8>;
  // Three warpgroups of 168 registers a thread at launch (two idle warps fill the
  // third where there are no converters).  The third gives registers to the two
  // of the softmax, whose threads hold a whole row of S (128 fp32): 2 x 200 + 104
  // (2 x 192 + 120) = 3 x 168.
  // int8: a fourth one, 128 registers a thread at launch.
  static constexpr int kThreads = SC ? 512 : 384;
  static constexpr int kSoftmaxRegs = SC ? 144 : (KV8 ? 192 : 200), kOtherRegs = SC ? 112 : (KV8 ? 120 : 104);
  static_assert(SC ? 2 * kSoftmaxRegs + 2 * kOtherRegs <= 4 * 128 : 2 * kSoftmaxRegs + kOtherRegs <= 3 * 168,
                "more registers than the launch has");
  // 8 tiles in flight: {KV head, valid, hid0, hid1} after the first slots of their boxes
  static constexpr int kMetaOff = Base::kPageOff + 8 * 32 * 4;
  static constexpr int kItemOff = kMetaOff + 8 * 16;
  static constexpr int kWBarOff = kItemOff + kItems * kItemBytes;
  static constexpr int kTmemOff = kWBarOff + kWBars * 8;  // the word that tcgen05.alloc writes, behind every barrier
  static_assert(kTmemOff >= kWBarOff + 8 * W_COUNT, "the TMEM base lies on a barrier");
  static constexpr int kBadOff = kTmemOff + 8;  // a page out of range was met
  // int8: K and V rings of two f16 tiles each, then two stages of codes (16 KB for 128
  // dims), in the space of the others' three and two tiles.  Codes that land in the slot
  // of their f16 tile (as e4m3 ones do) can be loaded only once the products on that
  // slot's last tile are done, and load and conversion then lie in a row: 1426 us for 19
  // chunks of 512 after 4096 tokens, 32 / 8 heads; with stages of their own 1370.
  static constexpr int kNK = SC ? 2 : kNSK;
  static constexpr int kVRing = SC ? Base::kKOff + 2 * Base::kKVTile : Base::kVOff;
  static constexpr int kCodeOff = Base::kKOff + (2 + kNSV) * Base::kKVTile;
  static constexpr int kCodeTile = kBN * D;
  static_assert(!SC || kCodeOff + 2 * kCodeTile <= Base::kPageOff, "the stages of codes");
  // int8: pages of 16 slots or more, so a tile has 8 boxes at most, and the scales take what
  // the first slots of 32 have left
  static constexpr int kBoxes = SC ? 8 : 32;
  static constexpr int kScaleOff = Base::kPageOff + 8 * 8 * 4;
  static_assert(!SC || (kScaleOff % 16 == 0 && kScaleOff + kScaleTiles * kScaleBytes <= kMetaOff), "the tiles' scales");
  static constexpr int kWSmem = kTmemOff + 16 + 1024;
  static_assert(kWSmem <= 232448, "shared memory");
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

// int8: the scales of a key tile, for each 16 keys.
struct TileScales {
  float4 of[8];  // factor of S (the first one below 0: no such tile, nor any after it), log2 v, 1 / 2^(log2 v), 0
};
static_assert(sizeof(TileScales) == kScaleBytes, "ring entry");

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
    fill(p, kpo, csize, tile, it);
    return true;
  }
  // The rest of item `it` = (b, hk, row tile).
  static __device__ void fill(const PrefillParams& p, int kpo, int csize, int tile, Item* it) {
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
  }
};

// The same items with the ones of most keys first, dealt out to the CTAs forwards and
// backwards in turn (ranks c, 2N - 1 - c, 2N + c, ...), so that the sums of keys come
// out even: without a window an item has from one key tile to all of its sequence's.
// Items are ranked by level = key tiles up to their last row's own key, then by sequence;
// count(b, level), the row tiles of sequence b at a level or above, is a closed form, so
// a rank is found by stepping the level down, a lane a sequence.  No window.
struct SortedWalker {
  int level, round;
  int64_t above, upto;  // row tiles of levels > level, >= level

  // Row tiles of sequence b with at least `level` key tiles (none past the batch).
  __device__ int count(const PrefillParams& p, int b, int level_) const {
    if (b >= p.batch) return 0;
    int qs;
    const int n = seq_rows(p, b, &qs);
    const int T = row_tiles((int64_t)min(n, p.max_q_len) * p.group);
    if (level_ <= 0 || T == 0) return T;
    const int L = ld_seq_len(p.seq_lens, b, p.max_blocks * p.pool.page_size, nullptr);
    const int64_t key = (int64_t)(level_ - 1) * kBN;  // a row at this position or behind it
    if (L - 1 < key) return 0;
    const int64_t x = key - (L - n);
    return T - (int)min(x <= 0 ? (int64_t)0 : x * p.group / (kQT * kBM), (int64_t)T - 1);
  }
  __device__ int64_t total(const PrefillParams& p, int level_) const {
    int sum = 0;  // at most 2^31 tokens of 32 heads make 2^28 row tiles
#pragma unroll 4
    for (int b = threadIdx.x & 31; b < p.batch; b += 32) sum += count(p, b, level_);
    return __reduce_add_sync(0xffffffffu, sum);
  }
  __device__ void start(const PrefillParams& p, int) {
    int top = 0;
#pragma unroll 4
    for (int b = threadIdx.x & 31; b < p.batch; b += 32)
      top = max(top, ld_seq_len(p.seq_lens, b, p.max_blocks * p.pool.page_size, nullptr) / kBN + 1);
    level = __reduce_max_sync(0xffffffffu, top);
    round = 0;
    above = 0;
    upto = total(p, level);
  }
  __device__ bool next(const PrefillParams& p, int kpo, int csize, Item* it) {
    const int N = gridDim.x / csize, c = blockIdx.x / csize, Hkv = p.pool.num_kv_heads;
    const int64_t rank = (int64_t)round * N + ((round & 1) ? N - 1 - c : c);
    ++round;
    const int64_t g = rank / Hkv;
    while (upto <= g) {
      if (level == 0) return false;
      above = upto;
      upto = total(p, --level);
    }
    int rel = (int)(g - above);  // among the row tiles of this level
    it->hk = (int)(rank - g * Hkv);
    for (int base = 0; base < p.batch; base += 32) {
      const int b = base + (threadIdx.x & 31), more = count(p, b, level + 1), mine = count(p, b, level) - more;
      int incl = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int t = __shfl_up_sync(0xffffffffu, incl, o);
        if ((threadIdx.x & 31) >= o) incl += t;
      }
      const int all = __shfl_sync(0xffffffffu, incl, 31);
      if (rel < all) {
        const int i = __popc(__ballot_sync(0xffffffffu, incl <= rel));
        it->b = base + i;
        const int before = __shfl_sync(0xffffffffu, incl - mine, i);
        // the tiles of sequence b at this level: [T - count(level), T - count(level + 1))
        const int first = __shfl_sync(0xffffffffu, count(p, b, 0) - more - mine, i);
        Walker::fill(p, kpo, csize, first + rel - before, it);
        return true;
      }
      rel -= all;
    }
    return false;  // (lengths that changed since they were counted)
  }
};

// int8: sorted up to 256 sequences, whose ranks a warp finds in eight steps.  8 chunks of
// 512-2048 after 0-8192 tokens: 1898 us in plain order, 1040 sorted; 256 of 24 after 200:
// 134 sorted; 2048 of 16 after 100: 2704 us sorted (64 steps an item).
struct AnyWalker {
  bool sorted;
  SortedWalker s;
  Walker w;
  __device__ void start(const PrefillParams& p, int csize) {
    sorted = p.batch <= 256;
    if (sorted) s.start(p, csize); else w.start(p, csize);
  }
  __device__ bool next(const PrefillParams& p, int kpo, int csize, Item* it) {
    return sorted ? s.next(p, kpo, csize, it) : w.next(p, kpo, csize, it);
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
template <int D, bool KV8, bool SC>
__device__ __forceinline__ void redo_bad_items(const PrefillParams& p, int kpo, int csize) {
  constexpr int E = D / 32;  // a lane's dims
  const int lane = threadIdx.x & 31, warps = blockDim.x >> 5, ps = p.pool.page_size, G = p.group;
  const int worker = (int)(blockIdx.x % csize) * warps + (threadIdx.x >> 5), workers = csize * warps;
  auto element = [&](const void* pool, int64_t at) {
    if (SC) return (float)static_cast<const signed char*>(pool)[at];
    if (KV8) {
      const uint32_t f = e4m3x2_lo_to_f16x2(static_cast<const unsigned char*>(pool)[at]);
      return __half2float(__ushort_as_half((unsigned short)(f & 0xFFFFu)));
    }
    return __bfloat162float(static_cast<const __nv_bfloat16*>(pool)[at]);
  };
  std::conditional_t<SC, AnyWalker, Walker> wk;  // this CTA's items
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
        float s = 0.f, ks = 1.f, vs = 1.f;
        if constexpr (SC) {
          const int64_t c = ((page * ps + (j & (ps - 1))) >> p.scale_shift) * p.pool.num_kv_heads + x.hk;
          ks = clamp_scale(__uint_as_float(ld_input(reinterpret_cast<const uint32_t*>(p.key_scales) + c)));
          vs = clamp_scale(__uint_as_float(ld_input(reinterpret_cast<const uint32_t*>(p.value_scales) + c)));
        }
#pragma unroll
        for (int e = 0; e < E; ++e) s = fmaf(q[e], element(p.pool.key_pool, at + e) * ks, s);
#pragma unroll
        for (int i = 16; i > 0; i >>= 1) s += __shfl_xor_sync(0xffffffffu, s, i);
        const float mn = fmaxf(m, s), a = fast_exp2(m - mn), w = fast_exp2(s - mn);
        m = mn;
        l = fmaf(l, a, w);
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = fmaf(o[e], a, w * (element(p.pool.value_pool, at + e) * vs));
      }
      const float inv = l > 0.f ? p.v_scale / l : 0.f;
#pragma unroll
      for (int e = 0; e < E; ++e) static_cast<__nv_bfloat16*>(p.out)[row + e] = __float2bfloat16_rn(o[e] * inv);
    }
  }
}

// SPLIT: csize CTAs of a cluster share an item, and there are clusters for all
// items (a CTA has one item at most); else csize is 1.
template <int D, bool KV8, bool SPLIT, bool SC = false>
__global__ void __launch_bounds__(WCfg<D, KV8, SC>::kThreads, 1)
    prefill_window_kernel(const __grid_constant__ CUtensorMap tmap_k, const __grid_constant__ CUtensorMap tmap_v,
                          const __grid_constant__ PrefillParams p, int csize_arg) {
  const int csize = SPLIT ? csize_arg : 1;
  using C = WCfg<D, KV8, SC>;
  static_assert(!SC || KV8, "int8 codes land as e4m3 ones do");
  constexpr int NK = C::kNK;
  constexpr bool kItemWarp = !KV8 || SC;  // warp 10 derives the items, else the TMA warp
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
  const uint32_t v_base = smem_u32(smem + C::kVRing);
  const uint32_t bars = smem_u32(smem + C::kWBarOff);
  auto bar = [&](int i) { return bars + 8u * i; };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kTmemOff);
  int* slot_ring = reinterpret_cast<int*>(smem + C::kPageOff);  // [8 tiles][kBoxes] first slot of each box, -1: none
  volatile Item* item_ring = reinterpret_cast<volatile Item*>(smem + C::kItemOff);
  int4* meta = reinterpret_cast<int4*>(smem + C::kMetaOff);     // [8 tiles] {KV head, valid, hid0, hid1}

  TileScales* scale_ring = reinterpret_cast<TileScales*>(smem + C::kScaleOff);
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
      mbar_init(bar(W_KREADY + s), SC ? kI8Warps : 1);
    }
    for (int s = 0; s < kNSV; ++s) {
      mbar_init(bar(W_VFULL + s), SC ? kI8Warps : 1);  // (int8: the stage of codes is free)
      mbar_init(bar(W_VEMPTY + s), 1);
      mbar_init(bar(W_VREADY + s), SC ? kI8Warps : 1);
    }
    mbar_init(bar(W_VLAND), 1);
    for (int s = 0; SC && s < kScaleTiles; ++s) {
      mbar_init(bar(W_CFULL + s), 1);
      mbar_init(bar(W_CEMPTY + s), 4 * kQT + kI8Warps);
    }
    for (int s = 0; s < kItems; ++s) {
      mbar_init(bar(W_IFULL + s), 1);
      mbar_init(bar(W_IEMPTY + s), 4 * kQT + 2 + (KV8 && !SC ? 2 : 0));  // each warp that reads items
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
  auto publish_next = [&](auto& wk, int i, Item* item = nullptr) {
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
    if (item != nullptr) *item = x;
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
        if (KV8)  // codes [keys][D B] in the ring slot's upper half (int8: in a stage of their own)
          tma_load_3d(dst + (uint32_t)((SC ? 0 : kBN * D) + lane * kpo * D), map, 0, slot, hk, full);
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
    if (!kItemWarp) wk.start(p, csize);
    int pub = 0, seen = 0;      // items handed out, items taken for their K tiles
    bool all_out = kItemWarp;   // the last entry says that there are no more
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
      if (!more && !end && (!kItemWarp ? seen < pub : phase_done(W_IFULL + seen % kItems, (uint32_t)((seen / kItems) & 1)))) {
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
      // int8: stage (kt + vt) % 2 of the codes, in the converters' order
      const int stage = (kt + vt) & 1;
      const bool stage_free = SC && (kt + vt < 2 || phase_done(W_VFULL + stage, (uint32_t)(((kt + vt) / 2 - 1) & 1)));
      const uint32_t code_dst = smem_u32(smem + C::kCodeOff) + stage * C::kCodeTile;
      const bool v_turn = SC && stage_free && vt < kt && (kt - vt == 2 || (end && !more));
      if (more && (SC ? stage_free && kt - vt < 2
                      : (kt < kNSK || phase_done(W_KEMPTY + kt % kNSK, (uint32_t)((kt / kNSK - 1) & 1))))) {
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
        if (lane < C::kBoxes) slot_ring[(kt & 7) * C::kBoxes + lane] = slot;
        if (lane == 0) {
          const int l0 = it.base + j * kBN;  // rows of the tile: valid ones, and those no row of the sequence sees
          const int end = it.seq_start <= it.head_keys ? it.seq_start : max(it.head_keys, it.seq_start - it.gap);
          meta[kt & 7] = make_int4(it.hk, min(it.L - it.gap - l0, kBN), max(0, p.num_sinks - l0), min(end - l0, kBN));
        }
        if constexpr (SC)
          issue(&tmap_k, code_dst, it.hk, slot, bar(W_KFULL + stage));
        else
          issue(&tmap_k, k_base + (kt % kNSK) * C::kKVTile, it.hk, slot, bar(W_KFULL + kt % kNSK));
        ++kt;
        more = ++j < it.nt();
        if (more) raw = fetch(j);
        progressed = true;
      }
      if constexpr (SC) {
        if (v_turn) {
          issue(&tmap_v, code_dst, meta[vt & 7].x, lane < C::kBoxes ? slot_ring[(vt & 7) * C::kBoxes + lane] : -1,
                bar(W_KFULL + stage));
          ++vt;
          progressed = true;
        }
      } else if (vt < kt && (vt < kNSV || phase_done(W_VEMPTY + vt % kNSV, (uint32_t)((vt / kNSV - 1) & 1)))) {
        const int4 m = meta[vt & 7];
        // rows that may hold anything meet P = 0 and must be zeros (e4m3: the converter writes them)
        const bool clear = !KV8 && (m.y < kBN || m.z < m.w);
        if (!clear || land_slot < 0) {
          const int s = vt % kNSV;
          issue(&tmap_v, v_base + s * C::kKVTile, m.x, slot_ring[(vt & 7) * C::kBoxes + lane],
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

  if constexpr (SC) {
    if (warp == kCvtWarp) {
      // ======================= items and scales, int8 pools =======================
      AnyWalker wk;
      wk.start(p, csize);
      const int per = 1 << p.scale_shift;                   // tokens of a scale: 16 or more
      const int lanes = per < kBN ? kBN / per : 1;          // scales of a tile
      int kt = 0;
      auto hand_out = [&](float4 mine) {                    // lanes 0 .. 7: of a block each
        const int s = kt % kScaleTiles;
        if (kt >= kScaleTiles && alive)  // each lane writes, so each waits
          alive = mbar_wait(bar(W_CEMPTY + s), (uint32_t)((kt / kScaleTiles - 1) & 1), p.err);
        alive = __all_sync(0xffffffffu, alive);
        if (lane < 8) scale_ring[s].of[lane] = mine;
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(W_CFULL + s));
      };
      // an item ahead of the scales: the others take the next item before they begin one
      Item nx = {};
      bool more = publish_next(wk, 0, &nx);
      for (int i = 0; more && alive; ++i) {
        const Item x = nx;
        if (i + 1 >= kItems)
          alive = __all_sync(0xffffffffu, mbar_wait(bar(W_IEMPTY + (i + 1) % kItems),
                                                    (uint32_t)(((i + 1) / kItems - 1) & 1), p.err));
        more = publish_next(wk, i + 1, &nx);
        const int32_t* bt = p.block_table + (int64_t)x.b * p.max_blocks;
        auto page_of = [&](int j) {  // of this lane's scale of tile j
          const int l = x.base + j * kBN + lane * per, key = l < x.head_keys ? l : l + x.gap;
          return lane < lanes && key < x.L ? ld_input(bt + (key >> pshift)) : -1;
        };
        int page = x.nt() > 0 ? page_of(0) : -1;
        for (int j = 0; j < x.nt(); ++j, ++kt) {
          const int l = x.base + j * kBN + lane * per, key = l < x.head_keys ? l : l + x.gap;
          float ks = kScaleMin, vs = kScaleMin;  // (no key, or a page out of range: any value)
          if (page >= 0 && page < p.pool.num_pages) {
            const int64_t slot = ((int64_t)page << pshift) + (key & (ps - 1));
            const int64_t c = (slot >> p.scale_shift) * p.pool.num_kv_heads + x.hk;
            ks = clamp_scale(__uint_as_float(ld_input(reinterpret_cast<const uint32_t*>(p.key_scales) + c)));
            vs = clamp_scale(__uint_as_float(ld_input(reinterpret_cast<const uint32_t*>(p.value_scales) + c)));
          }
          if (j + 1 < x.nt()) page = page_of(j + 1);
          const int from = ((lane & 7) * 16) >> p.scale_shift;  // the lane with the scales of block `lane`
          const float v_log2 = __log2f(__shfl_sync(0xffffffffu, vs, from));
          // (a factor of 0 would make NaN of a masked column)
          hand_out(make_float4(fmaxf(sl2 * __shfl_sync(0xffffffffu, ks, from), 0x1p-126f), v_log2,
                               fast_exp2(-v_log2), 0.f));  // the inverse of the very power that P carries
          if (!alive) break;
        }
      }
      hand_out(make_float4(-1.f, 0.f, 0.f, 0.f));
    }
    if (warp >= 16 - kI8Warps) {
      // ======================= int8 -> f16 converters (warps 12 .. 15) =======================
      const int part = warp - (16 - kI8Warps);
      int ct = 0;  // tiles of codes taken
      constexpr int kChunks = D / 16, kKeysPerLoad = 32 / kChunks, kLoads = 8 / kKeysPerLoad, kAtOnce = 2 / kLoads;
      const int q4 = lane >> 3, j8 = lane & 7;  // (bank-conflict-free as in convert_tile_e4m3)
      const int m = D == 128 ? (j8 & 3) + 4 * (j8 >> 2) : lane % kChunks;
      const int r0 = D == 128 ? 2 * (q4 >> 1) + ((j8 >> 2) ^ (q4 & 1)) : lane / kChunks;
      auto tile = [&](int t, bool isv) {
        const int n = isv ? kNSV : NK, sl = t % n, stage = ct & 1;
        if (alive) alive = mbar_wait(bar(W_KFULL + stage), (uint32_t)((ct >> 1) & 1), p.err);
        ++ct;
        if (t >= n && alive)  // the products on the slot's last tile are done
          alive = mbar_wait(bar((isv ? W_VEMPTY : W_KEMPTY) + sl), (uint32_t)((t / n - 1) & 1), p.err);
        // this warp's quarter of the tile: four 8-key blocks, two loads of a lane at a time (four
        // were more code than the instruction cache has room for: 762 us where these take 702)
        const unsigned char* codes = smem + C::kCodeOff + stage * C::kCodeTile + (part * 32 + r0) * D + m * 16;
        unsigned char* slot = smem + (isv ? C::kVRing : C::kKOff) + sl * C::kKVTile + part * 4 * C::kRowBlock;
#pragma unroll 1
        for (int k0 = 0; k0 < 4; k0 += kAtOnce) {
          uint4 raw[kAtOnce][kLoads];
#pragma unroll
          for (int kb = 0; kb < kAtOnce; ++kb)
#pragma unroll
            for (int x = 0; x < kLoads; ++x)
              raw[kb][x] = *reinterpret_cast<const uint4*>(codes + ((k0 + kb) * 8 + x * kKeysPerLoad) * D);
#pragma unroll
          for (int kb = 0; kb < kAtOnce; ++kb)
#pragma unroll
            for (int x = 0; x < kLoads; ++x) {
              const int kr = r0 + x * kKeysPerLoad;
              const uint4 w = raw[kb][x];
              unsigned char* blk = slot + (k0 + kb) * C::kRowBlock + kr * 128;
              const int c0 = 2 * m, c1 = 2 * m + 1;  // 8-dim chunks over D
              *reinterpret_cast<uint4*>(blk + (c0 >> 3) * 1024 + (((c0 & 7) ^ kr) << 4)) =
                  make_uint4(i8x2_to_f16x2<0, 1>(w.x), i8x2_to_f16x2<2, 3>(w.x), i8x2_to_f16x2<0, 1>(w.y),
                             i8x2_to_f16x2<2, 3>(w.y));
              *reinterpret_cast<uint4*>(blk + (c1 >> 3) * 1024 + (((c1 & 7) ^ kr) << 4)) =
                  make_uint4(i8x2_to_f16x2<0, 1>(w.z), i8x2_to_f16x2<2, 3>(w.z), i8x2_to_f16x2<0, 1>(w.w),
                             i8x2_to_f16x2<2, 3>(w.w));
            }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(W_VFULL + stage));  // the codes are read
        fence_proxy_async_smem();  // the f16 tile before the tensor core reads it
        __syncwarp();
        if (lane == 0) mbar_arrive(bar((isv ? W_VREADY : W_KREADY) + sl));
      };
      auto there = [&](int t) {  // the tile exists (its scales are handed out)
        const int s = t % kScaleTiles;
        if (alive) alive = mbar_wait(bar(W_CFULL + s), (uint32_t)((t / kScaleTiles) & 1), p.err);
        return alive && scale_ring[s].of[0].x >= 0.f;
      };
      int kt = 0, vt = 0;
      bool ended = false;
      for (;;) {  // (one call: see kHeld below)
        bool isv = kt - vt == 2 || ended;
        if (!isv && !__all_sync(0xffffffffu, there(kt))) {
          ended = true;
          isv = true;
        }
        if (isv && vt == kt) break;
        if (!isv && lane == 0) mbar_arrive(bar(W_CEMPTY + kt % kScaleTiles));  // that it exists is all that is read
        tile(isv ? vt : kt, isv);
        if (isv) ++vt; else ++kt;
      }
    }
  }

  if (KV8 && !SC && (warp == kCvtWarp || warp == kCvtWarp + 1)) {
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
          const int kt = k0 + j, sk = kt % NK;
          if (t == 0 || j >= x.nt0) {
            if (alive) alive = mbar_wait(bar(kKWait + sk), (uint32_t)((kt / NK) & 1), p.err);
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
    int cn = 0;               // SC: tiles whose scales are taken
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
      const float4* of = nullptr;  // SC: the tile's scales, of each 16 columns
      auto take_scales = [&]() {
        const int s = cn % kScaleTiles;
        if (alive) alive = mbar_wait(bar(W_CFULL + s), (uint32_t)((cn / kScaleTiles) & 1), p.err);
        of = scale_ring[s].of;
      };
      auto leave_scales = [&]() {
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(W_CEMPTY + cn % kScaleTiles));
        ++cn;
      };
      for (int j = 0; j < ntt; ++j) {
        if constexpr (SC) take_scales();
        if (alive) alive = mbar_wait(bar(W_SFULL + t), sn & 1u, p.err);
        ++sn;
        tc_fence_after();
        // every S of this item is done: Q may be replaced
        if (j == ntt - 1 && next_q) copy_q(nx);
        const int l0 = it.base + j * kBN;
        // some row does not see some key of the tile
        const bool masked = l0 + kBN - 1 > lim_min || (l0 < wlo_max && l0 + kBN > p.num_sinks);
        // The row of S, and its max.  Held whole where the code allows; int8 (SC) reads it
        // again for P, 32 columns at a time in loops: with the converters' and the scales'
        // code beside it, the unrolled form had warps wait for instructions (4.2 per issue)
        // and took 1258 us where the loops take 740 (19 chunks of 512 after 4096 tokens,
        // 32 / 8 heads of 128).
        constexpr int kHeld = SC ? 1 : 4;
        auto load = [&](auto& v, int first, int n) {
#pragma unroll
          for (int i = 0; i < n; ++i) tmem_ld32(s_col + (first + i) * 32, v[i]);
          tmem_wait_ld();
          if (masked) {
#pragma unroll
            for (int i = 0; i < n; ++i) {
              const int c0 = l0 + 32 * (first + i);
              const uint32_t see = bits_to(lim - c0) & (~bits_to(wlo - 1 - c0) | bits_to(p.num_sinks - 1 - c0));
#pragma unroll
              for (int e = 0; e < 32; ++e) v[i][e] = ((see >> e) & 1u) ? v[i][e] : 0xFF800000u;
            }
          }
        };
        float tmax = -INFINITY;
        uint32_t v[kHeld][32];
        // The loads find the max where nothing is masked: less code again (heads of 64: 661 -> 592
        // us).  Max and P in one pass, done again where the reference moves, needs P held in
        // registers and the loop written out: 1239 us for 770.
        const bool by_load = SC && !masked;
        if (by_load) {
#pragma unroll 1
          for (int cb = 0; cb < 4; ++cb) {
            const float2 c0 = *reinterpret_cast<const float2*>(of + 2 * cb), c1 = *reinterpret_cast<const float2*>(of + 2 * cb + 1);
            const float2 x = tmem_max16x2(s_col + cb * 32);
            tmax = max3(tmax, fmaf(x.x, c0.x, c0.y), fmaf(x.y, c1.x, c1.y));
          }
        }
#pragma unroll 1
        for (int first = by_load ? 4 : 0; first < 4; first += kHeld) {
          load(v, first, kHeld);
          if constexpr (SC) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint32_t* c = v[0] + 16 * h;
              float x = __uint_as_float(c[0]);
#pragma unroll
              for (int e = 1; e < 15; e += 2) x = max3(x, __uint_as_float(c[e]), __uint_as_float(c[e + 1]));
              x = fmaxf(x, __uint_as_float(c[15]));
              tmax = fmaxf(tmax, fmaf(x, of[2 * first + h].x, of[2 * first + h].y));
            }
          } else {
            float mx[kHeld];
#pragma unroll
            for (int i = 0; i < kHeld; ++i) {
              float& x = mx[i];
              x = __uint_as_float(v[i][0]);
#pragma unroll
              for (int e = 1; e < 31; e += 2) x = max3(x, __uint_as_float(v[i][e]), __uint_as_float(v[i][e + 1]));
              x = fmaxf(x, __uint_as_float(v[i][31]));
            }
#pragma unroll
            for (int i = 0; i < kHeld; ++i) tmax = fmaxf(tmax, mx[i]);
          }
        }
        if constexpr (!SC) tmax *= sl2;
        // reference max: moved only when the row max grows by more than 2^8
        float alpha = 1.f;
        bool rescale = false;
        // (int8: by the difference, which is exact: a sum rounded up would let P past f16's range)
        if (SC ? tmax - m_ref > kRescaleThreshold : tmax > m_ref + kRescaleThreshold) {
          alpha = m_ref == -INFINITY ? 0.f : fast_exp2(m_ref - tmax);
          m_ref = tmax;
          l *= alpha;
          rescale = j > 0;
        }
        const float mbase = m_ref == -INFINITY ? 0.f : m_ref;
        // P = exp2(x - m) as bf16 (f16) pairs, written over the S columns: V's type, the one that the product takes
        // beside it; l sums the fp32 ones.  Against 64 bits an output is off by 0.0023 of its norm so (codes:
        // 0.0017), by 0.0017 with its own rounding alone
        const uint64_t sub = pair(-mbase, -mbase);
        uint64_t rs[4] = {0ull, 0ull, 0ull, 0ull};
        if constexpr (SC) {
#pragma unroll 1
          for (int cb = 0; cb < 4; ++cb) {
            uint32_t x[1][32], w[16];
            const float4 c2[2] = {of[2 * cb], of[2 * cb + 1]};  // read ahead of the columns: 1002 -> 933 us
            load(x, cb, 1);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const float4 c = c2[h];
              const uint64_t mul = pair(c.x, c.x), add = pair(c.y, c.y), inv = pair(c.z, c.z);
#pragma unroll
              for (int e = 16 * h; e < 16 * h + 16; e += 2) {
                const uint64_t y = fma_pair(pair(__uint_as_float(x[0][e]), __uint_as_float(x[0][e + 1])), mul, add);
                const float2 d = unpair(add_pair(y, sub));
                const float p0 = fast_exp2(d.x), p1 = fast_exp2(d.y);
                rs[(e >> 1) & 3] = fma_pair(pair(p0, p1), inv, rs[(e >> 1) & 3]);
                w[e >> 1] = pack_f16(p0, p1);
              }
            }
            tmem_st16(s_col + cb * 16, w);
          }
        } else {
          const uint64_t mul = pair(sl2, sl2);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t w[32];
#pragma unroll
            for (int cb = 0; cb < 2; ++cb)
#pragma unroll
              for (int e = 0; e < 32; e += 2) {
                const uint32_t (&c)[32] = v[(2 * h + cb) % kHeld];
                const float2 x = unpair(fma_pair(pair(__uint_as_float(c[e]), __uint_as_float(c[e + 1])), mul, sub));
                const float p0 = fast_exp2(x.x), p1 = fast_exp2(x.y);
                rs[(e >> 1) & 3] = add_pair(rs[(e >> 1) & 3], pair(p0, p1));
                w[cb * 16 + (e >> 1)] = KV8 ? pack_f16(p0, p1) : pack_bf16(p0, p1);
              }
            tmem_st32(s_col + h * 32, w);
          }
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
        if constexpr (SC) leave_scales();
      }
      if constexpr (SC)
        for (int j = ntt; j < it.nt(); ++j) {  // tiles of the other query tile alone
          take_scales();
          leave_scales();
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
      constexpr int kOut = SC ? 1 : D / 32;  // 32 columns each, held at once
#pragma unroll 1
      for (int first = 0; first < D / 32; first += kOut) {
        uint32_t oall[kOut][32];
#pragma unroll
        for (int cb = 0; cb < kOut; ++cb)
          if (ntt > 0) {
            tmem_ld32(o_col + (first + cb) * 32, oall[cb]);
          } else {
#pragma unroll
            for (int e = 0; e < 32; ++e) oall[cb][e] = 0u;
          }
        if (ntt > 0) tmem_wait_ld();
#pragma unroll
        for (int cb = 0; cb < kOut; ++cb) {
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
              *reinterpret_cast<uint4*>(outp + dst[k] + (first + cb) * 32 + (lane & 3) * 8) =
                  make_uint4(w[k][0], w[k][1], w[k][2], w[k][3]);
        }
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
  if (__builtin_expect(redo, 0)) redo_bad_items<D, KV8, SC>(p, kpo, csize);
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

template <int D, bool KV8, bool SPLIT, bool SC>
cudaError_t launch_items(const PrefillParams& p, const CUtensorMap& tk, const CUtensorMap& tv, unsigned grid, int csize,
                         cudaStream_t s) {
  using C = WCfg<D, KV8, SC>;
  auto kern = prefill_window_kernel<D, KV8, SPLIT, SC>;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kWSmem);
  if (e != cudaSuccess) return e;
  if (!SPLIT) return launch_pdl(kern, dim3(grid), dim3(C::kThreads), (size_t)C::kWSmem, s, tk, tv, p, 1);
  return launch_pdl_cluster(kern, dim3(grid), dim3(C::kThreads), (size_t)C::kWSmem, csize, s, tk, tv, p, csize);
}

template <int D, bool KV8, bool SC = false>
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
  if (csize > 1) return launch_items<D, KV8, true, SC>(p, tk, tv, (unsigned)(items * csize), csize, s);
  return launch_items<D, KV8, false, SC>(p, tk, tv, (unsigned)(items < num_sms ? items : num_sms), 1, s);
}

}  // namespace

cudaError_t launch_prefill_window(const PrefillParams& p, int num_sms, cudaStream_t s) {
  if (p.max_q_len <= 0 || p.batch <= 0) return cudaSuccess;
  if (p.pool.page_size < 8 || p.pool.page_shift < 0) return cudaErrorInvalidValue;
  if (p.key_scales != nullptr)
    return p.pool.head_dim == 128 ? launch_window<128, true, true>(p, num_sms, s) : launch_window<64, true, true>(p, num_sms, s);
  if (p.kv8) return p.pool.head_dim == 128 ? launch_window<128, true>(p, num_sms, s) : launch_window<64, true>(p, num_sms, s);
  return p.pool.head_dim == 128 ? launch_window<128, false>(p, num_sms, s) : launch_window<64, false>(p, num_sms, s);
}

}  // namespace pa
