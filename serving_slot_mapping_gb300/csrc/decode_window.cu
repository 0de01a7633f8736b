// paged_attention_decode_window: decode over a sliding window and the first
// tokens of each sequence, split over the CTAs of a thread-block cluster.
//
//   out[b, h] = softmax_j(scale * q[b,h] . K_b[j, h/G]) V_b[j, h/G],
//   j < L_b with j >= L_b - window or j < num_sinks
//
// A window bounds every sequence's work, so the batch needs no common cut: a
// cluster of c CTAs takes one (sequence, KV head) and each CTA a c-th of its
// 16-key blocks (WinSpan: the sinks' blocks, then the window's; the blocks
// between are not looked up).  The parts are merged through distributed shared
// memory: no workspace, no counters, no cooperative launch.
// * A CTA is four teams of one warp (two for 17 to 32 query heads per KV head, one
//   per 16 heads) and a producer warp.  A team takes every fourth block of
//   the CTA's range through a ring of its own; two lanes of the producer issue
//   the TMA boxes of a team's block, its K and V rows (one page, or half-blocks
//   of 8-slot pages).  No warp waits for another team before the end.
// * Per block S^T = K Q^T and O^T += V^T P^T with mma.sync m16n8k16 (keys, then
//   dims, as the 16 rows, query heads as the 8 columns), online softmax in the
//   log2 domain; e4m3 codes become f16 fragments in registers.
// * Keys hidden by the window or past L_b are masked in S and zeroed in V.  A
//   block_table entry out of range is noted by the producer, and a CTA that met
//   one computes its part again without the keys of such pages (skip_bad_pages).
//   The loop itself knows nothing of them: a word that says which keys of a block
//   are there, read for each block or for each 8, took 117 and 113.5 us for 256 MQA
//   sequences with a window of 4096 (so: 110.6) and 40.3 and 40.8 us for 256
//   sequences with a window of 128 (37.5; with no such check 107.2 and 37.2).
// * End: teams merge in shared memory, then each CTA of the cluster finishes a
//   slice of the G x D outputs over the c partial rows.
#include <math.h>

#include <algorithm>

#include "cluster.cuh"
#include "common.cuh"
#include "inputs.cuh"
#include "internal.h"
#include "tma.cuh"

namespace pa {

namespace {

constexpr int kTeams = 4;

// The keys of a sequence of L keys that are visible: those below num_sinks and
// those from `start` on.  Its blocks are the 16-key blocks 0 .. head - 1 (the
// sinks') and then head + gap, head + gap + 1, ... (the window's); gap is 0
// where the two meet.
struct WinSpan {
  int start, head, gap;
};

__device__ __forceinline__ WinSpan win_span(const DecodeParams& p, int L) {
  WinSpan w;
  w.start = max(0, L - p.window);
  w.head = (min(p.num_sinks, w.start) + 15) >> 4;
  w.gap = max(0, (w.start >> 4) - w.head);
  return w;
}

// Block of the sequence that its k-th one with a visible key is.
__device__ __forceinline__ int win_block(const WinSpan& w, int k) { return k < w.head ? k : k + w.gap; }

// Byte offset of 16-byte chunk `chunk` of row `row` of an e4m3 tile ([16 rows][D
// B]) as TMA lands it: the 128-byte swizzle (D = 128) or the 64-byte one (D = 64).
template <int D>
__device__ __forceinline__ uint32_t code_chunk(int row, int chunk) {
  return D == 128 ? row * 128 + ((chunk ^ (row & 7)) << 4) : row * 64 + ((chunk ^ ((row >> 1) & 3)) << 4);
}

// CTAs of an SM that the ring of a team is sized for: 128 registers a thread
// leave room for three of 160 threads (up to 8 query heads per KV head), 168 for
// two of 160 (16) or one of 288 (32).
__host__ __device__ constexpr int ctas_per_sm(int heads) { return heads <= 8 ? 3 : (heads <= 16 ? 2 : 1); }

// Up to 8 heads: with up to 4 CTAs for each SM, a ring half as long again and two
// CTAs an SM (32 sequences, 8 KV heads, a window of 1024: 23.4 against 24.2 us; 64
// sequences: 43.1 against 46.6 us); with more, the third CTA hides more than the
// ring (256 sequences, a window of 128: 38.1 against 43.9 us).
bool deep_rings(int num_sms, int64_t ctas) { return ctas <= 4 * (int64_t)num_sms; }

// RT: warps per team, each with NT tiles of 8 query heads of the group; DEEP: see
// deep_rings.
template <int D, bool KV8, int RT, int NT, bool DEEP>
struct DCfg {
  static constexpr int kConsumers = kTeams * RT;           // warps
  static constexpr int kThreads = 32 * (kConsumers + 1);   // + the producer warp
  static constexpr int kSlabs = KV8 ? 1 : D / 64;          // TMA slabs per row
  static constexpr int kRowBytes = KV8 ? D : 128;          // bytes of one slot row of one slab
  static constexpr int kSlabBytes = 16 * kRowBytes;
  static constexpr int kTensorBytes = kSlabs * kSlabBytes;  // K or V of one block
  static constexpr int kBlockBytes = 2 * kTensorBytes;
  static constexpr int kHeads = 8 * NT * RT;
  static constexpr int kPerSm = DEEP ? 2 : ctas_per_sm(kHeads);
  static constexpr int kTeamRing = (kPerSm == 3 ? 16 : (kPerSm == 2 ? 24 : 40)) * 1024;
  static constexpr int kStages = kTeamRing / kBlockBytes;
  static constexpr int kRing = kTeams * kStages * kBlockBytes;
  // after the ring has drained: the teams' partial rows [team][head][kRow], their
  // (m, l) and the CTA's; its partial rows go over team 0's.  Rows are padded so
  // that the lanes of a quad, which hold different heads, hit different banks.
  static constexpr int kRow = D + 4;
  static constexpr int kPartMl = kTeams * kHeads * kRow * 4;
  static constexpr int kParts = kPartMl + (kTeams + 1) * kHeads * 8;
  static constexpr int kBarOff = kRing > kParts ? kRing : (kParts + 127) / 128 * 128;
  static constexpr int kSmem = kBarOff + 2 * kTeams * kStages * 8 + 1024;
  static_assert(kTeams * kStages <= 32 * (kTeams + 1), "one thread sets up each stage's barriers");
};

// The 8x8 matrix of 16-bit elements that the warp holds, row lane / 4, columns
// 2 (lane % 4) and the next, transposed.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(x));
  return d;
}

// The part of a CTA over the keys whose pages are in range, a warp a query head and
// a key at a time: team 0's partial rows and (m, l), the other teams' empty.  An
// error path, slow, which works out its blocks anew so that the loop before it holds
// no register for it.
template <int D, bool KV8, int HEADS, int ROW>
__device__ __forceinline__ void skip_bad_pages(const DecodeParams& p, int csize, float* part, float2* part_ml) {
  constexpr int E = D / 32;  // a lane's dims
  const int lane = threadIdx.x & 31, ps = p.pool.page_size, G = p.group;
  const int seg = blockIdx.x / csize, rank = blockIdx.x - seg * csize;
  const int b = seg / p.pool.num_kv_heads, hk = seg - b * p.pool.num_kv_heads;
  const int L = ld_seq_len(p.seq_lens, b, p.max_blocks * ps, nullptr);
  const WinSpan win = win_span(p, L);
  const int nblk = ((L + 15) >> 4) - win.gap, per = (nblk + csize - 1) / csize;
  const int k0 = rank * per, k1 = min(nblk, k0 + per);
  const int32_t* bt = p.block_table + (int64_t)b * p.max_blocks;
  for (int i = threadIdx.x; i < kTeams * HEADS * ROW; i += blockDim.x) part[i] = 0.f;
  for (int i = threadIdx.x; i < kTeams * HEADS; i += blockDim.x) part_ml[i] = make_float2(-INFINITY, 0.f);
  __syncthreads();
  auto element = [&](const void* pool, int64_t at) {
    if (KV8) {
      const uint32_t f = e4m3x2_lo_to_f16x2(static_cast<const unsigned char*>(pool)[at]);
      return __half2float(__ushort_as_half((unsigned short)(f & 0xFFFFu)));
    }
    return __bfloat162float(static_cast<const __nv_bfloat16*>(pool)[at]);
  };
  for (int head = threadIdx.x >> 5; head < G; head += blockDim.x >> 5) {
    const __nv_bfloat16* q =
        static_cast<const __nv_bfloat16*>(p.q) + ((int64_t)b * p.num_q_heads + (int64_t)hk * G + head) * D;
    float qv[E], o[E] = {}, m = -INFINITY, l = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) qv[e] = __bfloat162float(q[lane * E + e]) * p.scale_log2;
#pragma unroll 1
    for (int i = k0 * 16; i < k1 * 16; ++i) {
      const int j = win_block(win, i >> 4) * 16 + (i & 15);
      if (j >= L || (j >= p.num_sinks && j < win.start)) continue;
      const int page = ld_input(bt + (j >> p.pool.page_shift));
      if (page < 0 || page >= p.pool.num_pages) continue;
      const int64_t at = (((int64_t)page * ps + (j & (ps - 1))) * p.pool.num_kv_heads + hk) * D + lane * E;
      float s = 0.f;
#pragma unroll
      for (int e = 0; e < E; ++e) s = fmaf(qv[e], element(p.pool.key_pool, at + e), s);
#pragma unroll
      for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
      const float mn = fmaxf(m, s), a = fast_exp2(m - mn), w = fast_exp2(s - mn);
      m = mn;
      l = fmaf(l, a, w);
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] = fmaf(o[e], a, w * element(p.pool.value_pool, at + e));
    }
#pragma unroll
    for (int e = 0; e < E; ++e) part[head * ROW + lane * E + e] = o[e];
    if (lane == 0) part_ml[head] = make_float2(m, l);
  }
}

template <int D, bool KV8, int RT, int NT, bool DEEP>
__global__ void __launch_bounds__(DCfg<D, KV8, RT, NT, DEEP>::kThreads, DCfg<D, KV8, RT, NT, DEEP>::kPerSm)
    decode_window_kernel(const __grid_constant__ CUtensorMap tmap_k, const __grid_constant__ CUtensorMap tmap_v,
                          const __grid_constant__ DecodeParams p, int csize) {
  using C = DCfg<D, KV8, RT, NT, DEEP>;
  constexpr int S = C::kStages;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int G = p.group, Hkv = p.pool.num_kv_heads, Hq = p.num_q_heads;
  const int ps = p.pool.page_size, pshift = p.pool.page_shift;
  const int seg = blockIdx.x / csize, rank = blockIdx.x - seg * csize;
  const int b = seg / Hkv, hk = seg - b * Hkv;
  const uint32_t bars = smem_u32(smem + C::kBarOff);
  auto full_bar = [&](int team, int s) { return bars + 8u * (team * S + s); };
  auto empty_bar = [&](int team, int s) { return bars + 8u * ((kTeams + team) * S + s); };
  __shared__ volatile int bad_page;  // one out of range was met
  if (tid == 0) bad_page = 0;
  if (tid < kTeams * S) {
    mbar_init(bars + 8u * tid, 2);  // full: the lanes that issue K and V
    mbar_init(bars + 8u * (kTeams * S + tid), RT);  // empty: the team's warps
    fence_mbar_init();
  }
  griddep_launch_dependents();
  // Before the first read of an input: any of them, the lengths and the table too,
  // may come from the kernel before.  Read ahead of this wait they save 0.4 to 0.9 us
  // a call among decodes alone and nothing behind an append (32 sequences, append and
  // decode 26.3 us either way).
  griddep_wait();
  const int L = ld_seq_len(p.seq_lens, b, p.max_blocks * ps, tid == 0 && rank == 0 && hk == 0 ? p.err : nullptr);
  const WinSpan win = win_span(p, L);
  const int nblk = ((L + 15) >> 4) - win.gap;  // the sequence's blocks with a visible key
  const int per = (nblk + csize - 1) / csize;
  // the blocks of this CTA, every kTeams-th one a team's: block i of team t is
  // the sequence's k0 + t + i * kTeams
  const int k0 = rank * per, k1 = min(nblk, k0 + per);
  auto team_blocks = [&](int team) { return max(0, (k1 - k0 - team + kTeams - 1) / kTeams); };
  __syncthreads();  // the barriers are set up
  bool alive = true;

  if (warp == C::kConsumers) {
    // ======================= producer warp =======================
    // Lane t + kTeams * r knows the page (of each half, 8-slot pages) of block
    // i0 + r of team t; the next 8 blocks' are read while these are issued.  Two
    // lanes a team issue its K and its V box.
    const int32_t* bt = p.block_table + (int64_t)b * p.max_blocks;
    const int R = ps < 16 ? ps : 16;  // rows per box (page_size >= 8)
    constexpr int kAhead = 32 / kTeams;
    auto half_used = [&](int kk) { return kk < L && (kk < p.num_sinks || kk + R > win.start); };
    const int team = lane % kTeams, T = (lane / kTeams) & 1;
    const int mine = team_blocks(team), most = team_blocks(0);
    int pg0 = -1, pg1 = -1, next0 = -1, next1 = -1;
    auto fetch = [&](int i0) {
      const int k = k0 + team + (i0 + lane / kTeams) * kTeams;
      if (k >= k1) return;
      const int kk = win_block(win, k) * 16;
      if (half_used(kk)) next0 = ld_input(bt + (kk >> pshift));
      if (R < 16 && half_used(kk + 8)) next1 = ld_input(bt + ((kk + 8) >> pshift));
    };
    fetch(0);
    const CUtensorMap* map = T ? &tmap_v : &tmap_k;
    const uint32_t ring = smem_u32(smem) + (uint32_t)(team * S * C::kBlockBytes + T * C::kTensorBytes);
    int slot = 0;
    uint32_t phase = 1;  // of the empty barriers' previous lap (passes at once in the first)
    for (int i = 0; i < most; ++i) {
      if (i % kAhead == 0) {
        pg0 = next0;
        pg1 = next1;
        fetch(i + kAhead);
      }
      const int from = team + kTeams * (i % kAhead);
      const int pages[2] = {__shfl_sync(0xffffffffu, pg0, from), __shfl_sync(0xffffffffu, pg1, from)};
      if (i < mine && lane < 2 * kTeams) {
        const int kk0 = win_block(win, k0 + team + i * kTeams) * 16;
        const uint32_t bar = full_bar(team, slot);
        int rows[2] = {-1, -1}, boxes = 0;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int kk = kk0 + h * 8;
          if ((h == 1 && R == 16) || !half_used(kk)) continue;
          if (pages[h] < 0 || pages[h] >= p.pool.num_pages) {
            if (T == 0) {
              record_error(p.err, ERR_BLOCK_TABLE, pages[h]);
              bad_page = 1;
            }
            continue;
          }
          rows[h] = pages[h] * ps + (kk & (ps - 1));
          ++boxes;
        }
        if (alive) alive = mbar_wait(empty_bar(team, slot), phase, p.err);
        mbar_arrive_expect_tx(bar, (uint32_t)(boxes * C::kSlabs * R * C::kRowBytes));
        const uint32_t dst = ring + (uint32_t)(slot * C::kBlockBytes);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (rows[h] < 0) continue;
          const uint32_t to = dst + h * 8 * C::kRowBytes;
          if (KV8) {
            tma_load_3d(to, map, 0, rows[h], hk, bar);
          } else if (R == 16) {  // one box covers every slab
            tma_load_4d(to, map, 0, rows[h], hk, 0, bar);
          } else {
            for (int sl = 0; sl < C::kSlabs; ++sl) tma_load_4d(to + sl * C::kSlabBytes, map, 0, rows[h], hk, sl, bar);
          }
        }
      }
      __syncwarp();
      if (++slot == S) {
        slot = 0;
        phase ^= 1u;
      }
    }
  }

  // ======================= consumer warps =======================
  const int team = warp / RT, rt = warp % RT;
  const bool consumer = warp < C::kConsumers;
  const int mine = consumer ? team_blocks(team) : 0;
  unsigned char* ring = smem + team * S * C::kBlockBytes;
  // ---- queries: B fragments of m16n8k16 (columns are heads; those >= G are zero) ----
  const int c4 = lane & 3, r8 = lane >> 2;
  uint32_t qf[NT][D / 16][2];
  {
    const uint32_t* qg = reinterpret_cast<const uint32_t*>(static_cast<const __nv_bfloat16*>(p.q) +
                                                           ((int64_t)b * Hq + (int64_t)hk * G) * D);
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int head = (rt * NT + n) * 8 + r8;
      auto ld = [&](int d) { return head < G && mine > 0 ? ld_input(qg + ((head * D + d) >> 1)) : 0u; };
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        // e4m3 pools: f16, dims permuted to match the K fragments: MMA k = 2c, 2c + 1
        // are dims 4c, 4c + 1 of a 16-dim step and k = 2c + 8, 2c + 9 are 4c + 2, 4c + 3
        qf[n][kk][0] = ld(kk * 16 + c4 * (KV8 ? 4 : 2));
        qf[n][kk][1] = ld(kk * 16 + c4 * (KV8 ? 4 : 2) + (KV8 ? 2 : 8));
        if (KV8) {
          qf[n][kk][0] = bf16x2_to_f16x2(qf[n][kk][0]);
          qf[n][kk][1] = bf16x2_to_f16x2(qf[n][kk][1]);
        }
      }
    }
  }
  const float sl2 = p.scale_log2;
  const bool up = sl2 > 0.f;  // the usual scale: the max is taken over raw S, exp2 takes one fused multiply-add
  const float mul = up ? sl2 : 1.f;
  // O^T: tile x of 16 dims; elements 0, 1: dim r8 of the tile (e4m3: 2 r8), heads
  // 2c and 2c + 1; 2, 3: dim r8 + 8 (2 r8 + 1)
  float o[NT][D / 16][4];
  float m[NT][2], l[NT][2];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    m[n][0] = m[n][1] = -INFINITY;
    l[n][0] = l[n][1] = 0.f;
#pragma unroll
    for (int x = 0; x < D / 16; ++x) o[n][x][0] = o[n][x][1] = o[n][x][2] = o[n][x][3] = 0.f;
  }
  // Byte offsets of this lane's ldmatrix rows in a K and a V tile: chunk x of a
  // 128-byte slab row is XOR-ed with the row, so the chunks of one slab take an
  // offset each, the next slab a constant more.  K: keys (mi & 1) * 8 + rr, dims
  // chunk (mi >> 1); V (transposed): keys (mi >> 1) * 8 + rr, dims chunk (mi & 1);
  // a chunk is 16 bytes, 8 bf16 dims or 16 codes.
  constexpr int kFrags = KV8 ? D / 32 : D / 16;
  constexpr int kOffs = KV8 ? kFrags : 4;
  const int mi = lane >> 3, rr = lane & 7;
  uint32_t koff[kOffs], voff[kOffs];
#pragma unroll
  for (int x = 0; x < kOffs; ++x) {
    koff[x] = KV8 ? code_chunk<D>((mi & 1) * 8 + rr, 2 * x + (mi >> 1)) : sw128((mi & 1) * 8 + rr, 2 * x + (mi >> 1), C::kSlabBytes);
    voff[x] = KV8 ? koff[x] : sw128((mi >> 1) * 8 + rr, 2 * x + (mi & 1), C::kSlabBytes);
  }
  int slot = 0;
  uint32_t phase = 0;
  for (int i = 0; i < mine; ++i) {
    if (alive) alive = mbar_wait(full_bar(team, slot), phase, p.err);
    unsigned char* kt = ring + slot * C::kBlockBytes;
    unsigned char* vt = kt + C::kTensorBytes;
    const uint32_t kbase = smem_u32(kt), vbase = smem_u32(vt);
    const int key0 = win_block(win, k0 + team + i * kTeams) * 16;
    const int valid = L - key0;  // >= 1
    const int hid0 = max(0, p.num_sinks - key0), hid1 = min(16, win.start - key0);  // rows between sinks and window
    const bool edge = valid < 16 || hid0 < hid1;
    if (edge) {
      // hidden rows may hold anything (NaN would survive P = 0): zero them in V
      // (by the team's first warp; the second waits); a row's chunks stay in the
      // row under either swizzle
      if (rt == 0) {
        constexpr int kCh = C::kRowBytes / 16;
        for (int e = lane; e < 16 * C::kSlabs * kCh; e += 32) {
          const int row = e / (C::kSlabs * kCh), rem = e % (C::kSlabs * kCh);
          if (row >= valid || (row >= hid0 && row < hid1))
            *reinterpret_cast<uint4*>(vt + (rem / kCh) * C::kSlabBytes + row * C::kRowBytes + (rem % kCh) * 16) =
                make_uint4(0, 0, 0, 0);
        }
      }
      if (RT == 2) named_barrier(1 + team, 64);
      else __syncwarp();
    }
    // S^T = K Q^T: keys are the rows of the product and query heads its 8 columns
    // a tile, so a group of up to 8 heads costs one tile (heads as the 16 rows
    // would leave most of them empty).  All K fragments are loaded before the
    // first product; V's as they are used (loaded before the softmax their
    // registers cost more than the wait: 12 % for MQA, 256 x 4096 keys, 111.6 us now).
    float s[NT][4];
    uint32_t f[kFrags][4];
#pragma unroll
    for (int x = 0; x < kFrags; ++x)
      ldmatrix_x4(kbase + koff[x % kOffs] + (x / kOffs) * C::kSlabBytes, f[x][0], f[x][1], f[x][2], f[x][3]);
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      float s0[4] = {0.f, 0.f, 0.f, 0.f}, s1[4] = {0.f, 0.f, 0.f, 0.f};  // two halves of the dims, for latency
#pragma unroll
      for (int x = 0; x < kFrags; ++x) {
        if (KV8) {
          const uint32_t a[4] = {e4m3x2_lo_to_f16x2(f[x][0]), e4m3x2_lo_to_f16x2(f[x][1]), e4m3x2_hi_to_f16x2(f[x][0]),
                                 e4m3x2_hi_to_f16x2(f[x][1])};
          const uint32_t a2[4] = {e4m3x2_lo_to_f16x2(f[x][2]), e4m3x2_lo_to_f16x2(f[x][3]),
                                  e4m3x2_hi_to_f16x2(f[x][2]), e4m3x2_hi_to_f16x2(f[x][3])};
          mma_f16_16816(s0, a, qf[n][2 * x][0], qf[n][2 * x][1]);
          mma_f16_16816(s1, a2, qf[n][2 * x + 1][0], qf[n][2 * x + 1][1]);
        } else {
          mma_bf16_16816((x & 1) ? s1 : s0, f[x], qf[n][x][0], qf[n][x][1]);
        }
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) s[n][e] = up ? s0[e] + s1[e] : (s0[e] + s1[e]) * sl2;
    }
    if (edge) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int key = r8 + 8 * h;
        if (key >= valid || (key >= hid0 && key < hid1)) {
#pragma unroll
          for (int n = 0; n < NT; ++n) s[n][2 * h] = s[n][2 * h + 1] = -INFINITY;
        }
      }
    }
    float mn[NT][2];
    bool moved = false;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {  // heads 2c and 2c + 1
        float mx = fmaxf(s[n][e], s[n][2 + e]);
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
        mn[n][e] = fmaxf(m[n][e], mx * mul);  // finite: a block has a visible key
        moved |= mn[n][e] != m[n][e];
      }
    if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const float a0 = fast_exp2(m[n][0] - mn[n][0]), a1 = fast_exp2(m[n][1] - mn[n][1]);
        l[n][0] *= a0;
        l[n][1] *= a1;
        m[n][0] = mn[n][0];
        m[n][1] = mn[n][1];
#pragma unroll
        for (int x = 0; x < D / 16; ++x) {
          o[n][x][0] *= a0; o[n][x][1] *= a1;
          o[n][x][2] *= a0; o[n][x][3] *= a1;
        }
      }
    }
    // O^T += V^T P^T; P^T is the transpose of the weights as they stand.  They are
    // rounded to V's type (f16 for codes), the one that the matrix instruction takes
    // beside it; their sum is of the fp32 ones.  Against 64 bits an output is off by
    // 0.0021 to 0.0022 of its norm so (codes: 0.0017), by 0.0017 with its own
    // rounding alone.
    uint32_t pb[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      float w[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) w[e] = fast_exp2(fmaf(s[n][e], mul, -mn[n][e & 1]));
      l[n][0] += w[0] + w[2];
      l[n][1] += w[1] + w[3];
      pb[n][0] = transpose8(KV8 ? pack_f16(w[0], w[1]) : pack_bf16(w[0], w[1]));
      pb[n][1] = transpose8(KV8 ? pack_f16(w[2], w[3]) : pack_bf16(w[2], w[3]));
    }
#pragma unroll
    for (int x = 0; x < kFrags; ++x) {
      ldmatrix_x4_trans(vbase + voff[x % kOffs] + (x / kOffs) * C::kSlabBytes, f[x][0], f[x][1], f[x][2], f[x][3]);
      if (KV8) {
        // codes of keys 2c, 2c + 1 and dims 2j, 2j + 1 (j = lane / 4), regrouped by dim:
        // the even dims of the chunk are the tile's rows 0 - 7, the odd ones 8 - 15
#pragma unroll
        for (int r = 0; r < 4; ++r) f[x][r] = __byte_perm(f[x][r], 0u, 0x3120);
        const uint32_t a[4] = {e4m3x2_lo_to_f16x2(f[x][0]), e4m3x2_hi_to_f16x2(f[x][0]), e4m3x2_lo_to_f16x2(f[x][1]),
                               e4m3x2_hi_to_f16x2(f[x][1])};
        const uint32_t a2[4] = {e4m3x2_lo_to_f16x2(f[x][2]), e4m3x2_hi_to_f16x2(f[x][2]), e4m3x2_lo_to_f16x2(f[x][3]),
                                e4m3x2_hi_to_f16x2(f[x][3])};
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          mma_f16_16816(o[n][2 * x], a, pb[n][0], pb[n][1]);
          mma_f16_16816(o[n][2 * x + 1], a2, pb[n][0], pb[n][1]);
        }
      } else {
#pragma unroll
        for (int n = 0; n < NT; ++n) mma_bf16_16816(o[n][x], f[x], pb[n][0], pb[n][1]);
      }
    }
    if (edge) fence_proxy_async_smem();  // our stores precede the next TMA into this slot
    __syncwarp();
    if (lane == 0) mbar_arrive(empty_bar(team, slot));
    if (++slot == S) {
      slot = 0;
      phase ^= 1u;
    }
  }

  // ---- merge: the teams of the CTA, then the CTAs of the cluster ----
  float* part = reinterpret_cast<float*>(smem);                      // [team][kHeads][kRow]
  float2* part_ml = reinterpret_cast<float2*>(smem + C::kPartMl);    // [team][kHeads]
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      l[n][e] += __shfl_xor_sync(0xffffffffu, l[n][e], 4);
      l[n][e] += __shfl_xor_sync(0xffffffffu, l[n][e], 8);
      l[n][e] += __shfl_xor_sync(0xffffffffu, l[n][e], 16);
    }
  __syncthreads();  // every ring has drained
  if (consumer) {
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int head = (rt * NT + n) * 8 + 2 * c4 + e;
        if (head >= G) continue;
        float* to = part + (team * C::kHeads + head) * C::kRow;
#pragma unroll
        for (int x = 0; x < D / 16; ++x) {
          to[x * 16 + (KV8 ? 2 * r8 : r8)] = o[n][x][e];
          to[x * 16 + (KV8 ? 2 * r8 + 1 : r8 + 8)] = o[n][x][2 + e];
        }
        if (r8 == 0) part_ml[team * C::kHeads + head] = make_float2(m[n][e], l[n][e]);
      }
  }
  __syncthreads();
  if (__builtin_expect(bad_page != 0, 0)) {
    skip_bad_pages<D, KV8, C::kHeads, C::kRow>(p, csize, part, part_ml);
    __syncthreads();
  }
  const int items = G * (D / 4);  // float4s of the output
  __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.out) + ((int64_t)b * Hq + (int64_t)hk * G) * D;
  auto store = [&](int x, float4 acc, float den) {
    const float inv = den > 0.f ? p.v_scale / den : 0.f;  // v_scale: 1 for bf16 pools
    uint2 packed;
    packed.x = pack_bf16(acc.x * inv, acc.y * inv);
    packed.y = pack_bf16(acc.z * inv, acc.w * inv);
    *reinterpret_cast<uint2*>(out + 4 * (int64_t)x) = packed;
  };
  for (int x = tid; x < items; x += C::kThreads) {
    const int row = x / (D / 4), c = x - row * (D / 4);
    float M = -INFINITY;
#pragma unroll
    for (int t = 0; t < kTeams; ++t) M = fmaxf(M, part_ml[t * C::kHeads + row].x);
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    float den = 0.f;
#pragma unroll
    for (int t = 0; t < kTeams; ++t) {
      const float2 ml = part_ml[t * C::kHeads + row];
      const float f = ml.x == -INFINITY ? 0.f : fast_exp2(ml.x - M);
      const float4 v = *reinterpret_cast<const float4*>(part + (t * C::kHeads + row) * C::kRow + 4 * c);
      den += f * ml.y;
      acc.x += f * v.x; acc.y += f * v.y; acc.z += f * v.z; acc.w += f * v.w;
    }
    if (csize == 1) {
      store(x, acc, den);
    } else {  // the CTA's partial over team 0's place; (M, den) after the teams' (m, l)
      *reinterpret_cast<float4*>(part + row * C::kRow + 4 * c) = acc;
      if (c == 0) part_ml[kTeams * C::kHeads + row] = make_float2(M, den);
    }
  }
  if (csize > 1) {
    cluster_sync();
    const uint32_t part_at = smem_u32(part), ml_at = smem_u32(part_ml + kTeams * C::kHeads);
    for (int x = rank + csize * tid; x < items; x += csize * C::kThreads) {
      const int row = x / (D / 4), c = x - row * (D / 4);
      float M = -INFINITY, den = 0.f;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
      float2 ml[8];
      float4 v[8];
#pragma unroll
      for (int r = 0; r < 8; ++r) {
        ml[r] = make_float2(-INFINITY, 0.f);
        v[r] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (r < csize) {
          ml[r] = ld_cluster2(map_rank(ml_at + 8u * row, r));
          v[r] = ld_cluster4(map_rank(part_at + 4u * (row * C::kRow + 4 * c), r));
        }
      }
#pragma unroll
      for (int r = 0; r < 8; ++r) M = fmaxf(M, ml[r].x);
#pragma unroll
      for (int r = 0; r < 8; ++r) {
        const float f = ml[r].x == -INFINITY ? 0.f : fast_exp2(ml[r].x - M);
        den += f * ml[r].y;
        acc.x += f * v[r].x; acc.y += f * v[r].y; acc.z += f * v[r].z; acc.w += f * v[r].w;
      }
      store(x, acc, den);
    }
    cluster_sync();  // no CTA leaves while another reads its memory
  }
}

template <int D, bool KV8, int RT, int NT, bool DEEP>
cudaError_t launch_window(const DecodeParams& p, const CUtensorMap& tk, const CUtensorMap& tv, int csize,
                           cudaStream_t s) {
  using C = DCfg<D, KV8, RT, NT, DEEP>;
  auto kern = decode_window_kernel<D, KV8, RT, NT, DEEP>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  if (e != cudaSuccess) return e;
  const unsigned grid = (unsigned)((int64_t)p.batch * p.pool.num_kv_heads * csize);
  return launch_pdl_cluster(kern, dim3(grid), dim3(C::kThreads), (size_t)C::kSmem, csize, s, tk, tv, p, csize);
}

template <int D, bool KV8>
cudaError_t launch_group(const DecodeParams& p, const CUtensorMap& tk, const CUtensorMap& tv, int num_sms, int csize,
                         cudaStream_t s) {
  if (p.group <= 8)
    return deep_rings(num_sms, (int64_t)p.batch * p.pool.num_kv_heads * csize)
               ? launch_window<D, KV8, 1, 1, true>(p, tk, tv, csize, s)
               : launch_window<D, KV8, 1, 1, false>(p, tk, tv, csize, s);
  return p.group <= 16 ? launch_window<D, KV8, 1, 2, false>(p, tk, tv, csize, s)
                       : launch_window<D, KV8, 2, 2, false>(p, tk, tv, csize, s);
}

}  // namespace

// As many CTAs a (sequence, KV head) as are resident at once, and each with a
// block at least for every team: a cluster whose CTAs wait for a second wave
// loses more than the shorter parts gain (1024 keys, on clusters of 1, 2, 4 and
// 8 CTAs: 32 sequences of 2 KV heads of 64 dims 14.7, 10.5, 7.7 and 12.5 us; of 8
// heads of 128 dims 24.6, 29.3, 33.8 and 45.0 us).  Clusters get the deep rings (a
// grid of them is never past deep_rings' bound), so two CTAs are resident on an SM
// at most: counted as three, 12 and 24 sequences of 8 heads of 128 dims got clusters
// of 4 and 2 and took 17.8 and 26.4 us; on 2 and 1 they take 12.9 and 19.3 us.
int decode_window_cluster(int num_sms, int32_t batch, int32_t num_kv_heads, int32_t group, int64_t max_keys) {
  const int64_t segments = (int64_t)batch * num_kv_heads, slots = (int64_t)num_sms * std::min(2, ctas_per_sm(group));
  const int64_t blocks = (max_keys + 15) / 16;
  int c = 1;
  while (c < 8 && segments * 2 * c <= slots && blocks >= 2 * kTeams * c) c *= 2;
  return c;
}

cudaError_t launch_decode_window(const DecodeParams& p, int num_sms, int csize, cudaStream_t s) {
  const int D = p.pool.head_dim;
  const int R = p.pool.page_size < 16 ? p.pool.page_size : 16;
  const int64_t rows = p.pool.num_pages * (int64_t)p.pool.page_size;
  CUtensorMap tk, tv;
  if (p.kv8) {
    if (!encode_pool_tmap_u8(&tk, p.pool.key_pool, rows, p.pool.num_kv_heads, D, R, 1, true) ||
        !encode_pool_tmap_u8(&tv, p.pool.value_pool, rows, p.pool.num_kv_heads, D, R, 1, true))
      return cudaErrorInvalidValue;
    return D == 128 ? launch_group<128, true>(p, tk, tv, num_sms, csize, s) : launch_group<64, true>(p, tk, tv, num_sms, csize, s);
  }
  const int slabs = R == 16 ? D / 64 : 1;
  if (!encode_pool_tmap(&tk, p.pool.key_pool, rows, p.pool.num_kv_heads, D, R, 1, slabs) ||
      !encode_pool_tmap(&tv, p.pool.value_pool, rows, p.pool.num_kv_heads, D, R, 1, slabs))
    return cudaErrorInvalidValue;
  return D == 128 ? launch_group<128, false>(p, tk, tv, num_sms, csize, s) : launch_group<64, false>(p, tk, tv, num_sms, csize, s);
}

}  // namespace pa
