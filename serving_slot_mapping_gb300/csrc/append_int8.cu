// paged_kv_append_int8: the append of new K/V rows into int8 pools, which sets the
// scale of each block of tokens and KV head as it goes.
//
// For a block of which the call writes rows, a head and a tensor, with a the largest
// magnitude of those rows there:
//   n  = clamp(a / 127, 2^-40, 2^40)
//   s' = n                    if the block's first slot is among the rows (a new block)
//      = max(clamp(s), n)     else; where s' > s the block's other rows, whose codes
//                             stand for c s, become rint(c (s / s'))
//   c  = rint(x / s'), at most 127 in magnitude (NaN: 0)
// all in fp32, a division's quotient and one rounding (to nearest even) a row element.
//
// A run is the consecutive tokens whose slots lie in one block, padding tokens between
// them aside (31 at most in a row).  A team takes a run for one head and tensor: one warp,
// two where a block has 32 tokens, four from 64 on.  16 rows a warp stay in registers
// between their maximum and their codes, so they are read once.  (Blocks of 64, 10,304
// tokens, 8 heads of 128: 24.1 us, with one warp a run 36.4.)  A re-encoded block is rewritten
// whole before the run's own rows, so the team need not know which rows are its own.
// Six CTAs of an SM (80 registers a thread) hide each other's chains of slots, rows,
// maximum and codes: 15.3-15.8 us for 10,304 tokens of sequences that begin a block of 16
// (9.3 of bytes); five 18.0, eight, which spill, 15.4.  Where the sequences begin inside a
// block (10,648 tokens after 0-8192, 9.6 of bytes) it is 17.2 us, and 18 with five as with six.
#include <algorithm>

#include "common.cuh"
#include "inputs.cuh"
#include "internal.h"
#include "tma.cuh"

namespace pa {

namespace {

constexpr int kAppendWarps = 4;

// The rounded quotient of x by the block's scale, in the low byte: RN(x / s) by the
// reciprocal y = RN(1 / s) and one correction of the product with its remainder
// (Markstein's division), then rounding to an integer by adding 1.5 2^23, whose low bits
// the integer is in.  The same as the division's code for bf16 values of less than 127.5
// scales (the tests compare every quotient of a new block, and a sample of the scales of
// blocks in use); 127.5 itself is a tie that would become 128.  Not for NaN.
__device__ __forceinline__ uint32_t code_of(float x, float s, float y) {
  const float q = __fmul_rn(x, y);
  return __float_as_uint(__fadd_rn(__fmaf_rn(__fmaf_rn(-s, q, x), y, q), 12582912.f));
}
// The same for any x, by the division: infinities saturate, NaN becomes 0.
__device__ __forceinline__ uint32_t code_of_any(float x, float s) {
  return (uint32_t)min(max(__float2int_rn(__fdiv_rn(x, s)), -127), 127);
}

// Eight bf16 elements -> eight codes.  `plain`: they are finite.
__device__ __forceinline__ uint2 codes8(uint4 v, float s, float y, bool plain) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t c[8];
  if (plain) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      c[2 * i] = code_of(__uint_as_float(w[i] << 16), s, y);
      c[2 * i + 1] = code_of(__uint_as_float(w[i] & 0xFFFF0000u), s, y);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      c[2 * i] = code_of_any(__uint_as_float(w[i] << 16), s);
      c[2 * i + 1] = code_of_any(__uint_as_float(w[i] & 0xFFFF0000u), s);
    }
  }
  auto four = [&](int i) {
    return __byte_perm(__byte_perm(c[i], c[i + 1], 0x0040), __byte_perm(c[i + 2], c[i + 3], 0x0040), 0x5410);
  };
  return make_uint2(four(0), four(4));
}

// Four codes times r, rounded.
__device__ __forceinline__ uint32_t rescale4(uint32_t w, float r) {
  uint32_t o = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int c = (int)(signed char)((w >> (8 * i)) & 0xFFu);
    o |= (uint32_t)(__float2int_rn(__fmul_rn((float)c, r)) & 0xFF) << (8 * i);
  }
  return o;
}

// The larger magnitudes, element by element (first in the low half); NaN wins in `any`
// and loses in `number`.
__device__ __forceinline__ void max_abs8(__nv_bfloat162* any, uint4 v) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t m = w[i] & 0x7FFF7FFFu;
    *any = __hmax2_nan(*any, *reinterpret_cast<const __nv_bfloat162*>(&m));
  }
}
__device__ __forceinline__ float max_number8(float a, uint4 v) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i)
    a = fmaxf(a, fmaxf(fabsf(__uint_as_float(w[i] << 16)), fabsf(__uint_as_float(w[i] & 0xFFFF0000u))));
  return a;
}

// Tokens [blockIdx.x * per_cta, + per_cta), at most 32: the runs that begin there.  W:
// warps of a team.
// blockIdx.y: a share of the (run, tensor, head) tasks.  Every warp finds the runs by
// itself, from the slots of these tokens and of the 32 before them, a lane each.
template <int D, int W>
__global__ void __launch_bounds__(kAppendWarps * 32, 6) append_int8_kernel(const __grid_constant__ AppendInt8Params p,
                                                                        int per_cta) {
  constexpr int kLanes = D / 8;            // lanes of a row
  constexpr int kRows = 32 / kLanes;       // rows of a pass
  constexpr int kPasses = 16 / kRows;      // passes whose rows stay in registers
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int sub = lane / kLanes, col = lane % kLanes;
  const int64_t first = (int64_t)blockIdx.x * per_cta;
  const int pairs = 2 * p.num_kv_heads;
  const unsigned kAll = 0xffffffffu;
  constexpr int kTeams = kAppendWarps / W;
  __shared__ float most[kAppendWarps];
  const int team = warp / W, w0 = warp % W * 16;  // w0: this warp's first row of the span
  auto team_sync = [&]() {
    if constexpr (W == 1) __syncwarp();
    else named_barrier(1 + team, W * 32);
  };
  // the largest of the team's values (NaN wins), for every warp of it
  auto team_max = [&](float a) {
    if constexpr (W == 1) return a;
    if (lane == 0) most[warp] = a;
    team_sync();
    a = most[team * W];
#pragma unroll
    for (int i = 1; i < W; ++i) {
      const float x = most[team * W + i];
      a = a != a || x != x ? a + x : fmaxf(a, x);
    }
    team_sync();  // read before the next one is written
    return a;
  };
  griddep_wait();
  auto slot_at = [&](int64_t t) {  // -1: no token, or one without a place
    const int64_t s = t >= 0 && t < p.num_tokens ? ld_input(p.slot_mapping + t) : -1;
    return s < 0 || s >= p.num_slots ? -1 : (int)s;
  };
  auto block_of = [&](int s) { return s >> p.scale_shift; };  // -1: none
  const int slot = slot_at(first + lane), blk = block_of(slot);
  const int blk0 = block_of(slot_at(first - 32 + lane));
  if (blockIdx.y == 0 && warp == 0 && lane < per_cta && first + lane < p.num_tokens) {
    const int64_t s = ld_input(p.slot_mapping + first + lane);
    if (s >= p.num_slots) record_error(p.err, ERR_SLOT, s);
  }
  // the first token of a run: the last token with a slot before it, among 32, is of
  // another block
  const unsigned there = __ballot_sync(kAll, blk >= 0), there0 = __ballot_sync(kAll, blk0 >= 0);
  const unsigned lower = there & ((1u << lane) - 1u);
  const int last = lower != 0u ? 31 - __clz(lower) : 31 - __clz(there0 | 1u);
  const int pb = __shfl_sync(kAll, blk, last), pb0 = __shfl_sync(kAll, blk0, last);
  const int before = lower != 0u ? pb : (there0 != 0u && last >= lane ? pb0 : -1);
  const unsigned leaders = __ballot_sync(kAll, lane < per_cta && blk >= 0 && before != blk);
  const int tasks = __popc(leaders) * pairs;
  for (int task = blockIdx.y * kTeams + team; task < tasks; task += gridDim.y * kTeams) {
    const int pair = task % pairs;
    unsigned m = leaders;
    for (int i = task / pairs; i > 0; --i) m &= m - 1u;
    const int l = __ffs(m) - 1;
    const int64_t t0 = first + l;
    const int b = __shfl_sync(kAll, blk, l);
    const int head_slot = b << p.scale_shift;
    // the span (the run's tokens, and padding), and whether it holds the block's first slot
    auto members = [&](int x, unsigned from, bool* ends) {
      const unsigned same = __ballot_sync(kAll, x == b) & from, other = __ballot_sync(kAll, x >= 0 && x != b) & from;
      *ends = other != 0u;
      return same & (other == 0u ? kAll : (1u << (__ffs(other) - 1)) - 1u);
    };
    bool ends;
    unsigned mine = members(blk, kAll << l, &ends);
    bool fresh = __any_sync(kAll, ((mine >> lane) & 1u) && slot == head_slot);
    int64_t n = 32 - __clz(mine) - l;
    while (!ends) {
      const int s = slot_at(t0 + n + lane);
      mine = members(block_of(s), kAll, &ends);
      if (mine == 0u) break;  // (32 padding tokens end a run)
      fresh |= __any_sync(kAll, ((mine >> lane) & 1u) && s == head_slot) != 0;
      n += 32 - __clz(mine);
    }
    const bool isv = pair >= p.num_kv_heads;
    const int h = isv ? pair - p.num_kv_heads : pair;
    const int64_t stride = isv ? p.value_stride : p.key_stride;
    const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(isv ? p.value : p.key) + t0 * stride + h * D + col * 8;
    signed char* pool = static_cast<signed char*>(isv ? p.value_pool : p.key_pool) + h * D + col * 8;
    float* scale = (isv ? p.value_scales : p.key_scales) + (int64_t)b * p.num_kv_heads + h;
    const int64_t pitch = (int64_t)p.num_kv_heads * D;
    auto row = [&](int64_t r) { return ld_stream(reinterpret_cast<const uint4*>(src + r * stride)); };
    uint4 v[kPasses];
#pragma unroll
    for (int x = 0; x < kPasses; ++x) {
      const int r = w0 + x * kRows + sub;
      v[x] = r < n ? row(r) : make_uint4(0u, 0u, 0u, 0u);
    }
    const float old = fresh ? 0.f : clamp_scale(__uint_as_float(ld_input(reinterpret_cast<const uint32_t*>(scale))));
    // the slot of span row r; -1: a padding token
    auto mine_of = [&](int64_t r) {
      const int s = r < n ? slot_at(t0 + r) : -1;
      return block_of(s) == b ? s : -1;
    };
    int at[kPasses];
#pragma unroll
    for (int x = 0; x < kPasses; ++x) {
      const int r = w0 + x * kRows + sub, s = __shfl_sync(kAll, slot, (l + r) & 31);
      at[x] = l + r < 32 ? (r < n && block_of(s) == b ? s : -1) : mine_of(r);
    }
    // f(row, slot) for this warp's rows of the span from `first` on that are the run's
    auto each = [&](int64_t from, auto f) {
      for (int64_t c = from + w0; c < n; c += 16 * W)
        for (int64_t r = c + sub; r < min(n, c + 16); r += kRows) {
          const int to = mine_of(r);
          if (to >= 0) f(r, to);
        }
    };
    __nv_bfloat162 any = __float2bfloat162_rn(0.f);
#pragma unroll
    for (int x = 0; x < kPasses; ++x)
      if (at[x] >= 0) max_abs8(&any, v[x]);
    each(16 * W, [&](int64_t r, int) { max_abs8(&any, row(r)); });
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) any = __hmax2_nan(any, __shfl_xor_sync(kAll, any, o));
    float a = team_max(__bfloat162float(__hmax_nan(any.x, any.y)));
    const bool plain = a <= 3.3e38f;  // neither infinities nor NaN
    if (a != a) {                     // the largest of the numbers
      a = 0.f;
      each(0, [&](int64_t r, int) { a = max_number8(a, row(r)); });
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) a = fmaxf(a, __shfl_xor_sync(kAll, a, o));
      a = team_max(a);
    }
    const float s = fmaxf(old, clamp_scale(__fdiv_rn(a, 127.f)));
    // values of 127.5 scales and more, which the largest scale leaves, need saturating too
    const bool fast = plain && a < 127.5f * kScaleMax;
    const float y = __frcp_rn(s);
    if (!fresh && s > old) {
      const float ratio = __fdiv_rn(old, s);
      const int rows = 1 << p.scale_shift;
      for (int c = w0; c < rows; c += 16 * W)
        for (int r = c + sub; r < c + 16; r += kRows) {  // (a block has 16 tokens or a multiple)
          uint2* to = reinterpret_cast<uint2*>(pool + (int64_t)(head_slot + r) * pitch);
          const uint2 w = ld_input(to);
          *to = make_uint2(rescale4(w.x, ratio), rescale4(w.y, ratio));
        }
    }
    team_sync();  // the rows below land over the re-encoded ones
    if (lane == 0 && w0 == 0) *scale = s;
#pragma unroll
    for (int x = 0; x < kPasses; ++x)
      if (at[x] >= 0) *reinterpret_cast<uint2*>(pool + (int64_t)at[x] * pitch) = codes8(v[x], s, y, fast);
    each(16 * W, [&](int64_t r, int to) {
      *reinterpret_cast<uint2*>(pool + (int64_t)to * pitch) = codes8(row(r), s, y, fast);
    });
  }
}

template <int W>
cudaError_t launch_teams(const AppendInt8Params& p, int num_sms, cudaStream_t s) {
  constexpr int kTeams = kAppendWarps / W;
  const int shares = (2 * p.num_kv_heads + kTeams - 1) / kTeams;
  // one token a CTA while that fills the SMs four times at most (a decode step: every
  // token is a run), else 16
  const int per_cta = p.num_tokens * shares <= 4 * (int64_t)num_sms ? 1 : 16;
  const int64_t ctas = (p.num_tokens + per_cta - 1) / per_cta;
  auto kern = p.head_dim == 128 ? append_int8_kernel<128, W> : append_int8_kernel<64, W>;
  return launch_pdl(kern, dim3((unsigned)ctas, (unsigned)std::min(shares, 65535)), dim3(kAppendWarps * 32), 0, s, p, per_cta);
}

}  // namespace

cudaError_t launch_append_int8(const AppendInt8Params& p, int num_sms, cudaStream_t s) {
  if (p.num_tokens <= 0) return cudaSuccess;
  if (p.scale_shift == 4) return launch_teams<1>(p, num_sms, s);
  return p.scale_shift == 5 ? launch_teams<2>(p, num_sms, s) : launch_teams<4>(p, num_sms, s);
}

}  // namespace pa
