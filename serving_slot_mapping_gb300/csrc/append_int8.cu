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
// all in fp32, one division and one rounding (to nearest even) a row element.
//
// A run is the consecutive tokens whose slots lie in one block, padding tokens between
// them aside (31 at most in a row); a warp takes a run for one head and tensor: up to 16
// rows stay in registers between their maximum and their codes, so they are read once.  A re-encoded block is rewritten whole before
// the run's own rows (__syncwarp orders the two), so the warp need not know which
// rows are its own.
#include <algorithm>

#include "common.cuh"
#include "inputs.cuh"
#include "internal.h"

namespace pa {

namespace {

constexpr int kAppendWarps = 4;

// bf16 pair -> two codes' bytes (low 16 bits).
__device__ __forceinline__ uint32_t codes2(uint32_t w, float s) {
  const int a = min(max(__float2int_rn(__fdiv_rn(__uint_as_float(w << 16), s)), -127), 127);
  const int b = min(max(__float2int_rn(__fdiv_rn(__uint_as_float(w & 0xFFFF0000u), s)), -127), 127);
  return (uint32_t)(a & 0xFF) | ((uint32_t)(b & 0xFF) << 8);
}

__device__ __forceinline__ uint2 codes8(uint4 v, float s) {
  return make_uint2(codes2(v.x, s) | (codes2(v.y, s) << 16), codes2(v.z, s) | (codes2(v.w, s) << 16));
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

__device__ __forceinline__ float max_abs8(float a, uint4 v) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i)
    a = fmaxf(a, fmaxf(fabsf(__uint_as_float(w[i] << 16)), fabsf(__uint_as_float(w[i] & 0xFFFF0000u))));
  return a;
}

// Tokens [blockIdx.x * per_cta, + per_cta): the runs that begin there.  blockIdx.y:
// a share of the (head, tensor) pairs.
template <int D>
__global__ void __launch_bounds__(kAppendWarps * 32) append_int8_kernel(const __grid_constant__ AppendInt8Params p,
                                                                        int per_cta) {
  constexpr int kLanes = D / 8;            // lanes of a row
  constexpr int kRows = 32 / kLanes;       // rows of a pass
  constexpr int kPasses = 16 / kRows;      // passes whose rows stay in registers
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int sub = lane / kLanes, col = lane % kLanes;
  const int64_t first = (int64_t)blockIdx.x * per_cta;
  const int pairs = 2 * p.num_kv_heads;
  griddep_wait();
  auto slot_at = [&](int64_t t) -> int64_t { return t < p.num_tokens ? ld_input(p.slot_mapping + t) : -1; };
  auto block_of = [&](int64_t s) -> int64_t { return s < 0 || s >= p.num_slots ? -1 : s >> p.scale_shift; };
  for (int i = 0; i < per_cta; ++i) {
    const int64_t t0 = first + i;
    if (t0 >= p.num_tokens) return;
    const int64_t s0 = slot_at(t0), blk = block_of(s0);
    if (s0 >= p.num_slots && blockIdx.y == 0 && threadIdx.x == 0) record_error(p.err, ERR_SLOT, s0);
    if (blk < 0) continue;
    // the first token of a run: the last token with a slot before it, among 32, is of
    // another block
    {
      const int64_t before = t0 - 1 - lane >= 0 ? block_of(slot_at(t0 - 1 - lane)) : -1;
      const unsigned there = __ballot_sync(0xffffffffu, before >= 0);
      if (there != 0u && __shfl_sync(0xffffffffu, before, __ffs(there) - 1) == blk) continue;
    }
    // its span (the run's tokens, and padding), and whether it holds the block's first slot
    int64_t n = 1;
    bool fresh = s0 == (blk << p.scale_shift);
    for (;;) {
      const int64_t s = slot_at(t0 + n + lane), x = block_of(s);
      const unsigned same = __ballot_sync(0xffffffffu, x == blk), other = __ballot_sync(0xffffffffu, x >= 0 && x != blk);
      const unsigned mine = same & (other == 0u ? 0xffffffffu : (1u << (__ffs(other) - 1)) - 1u);
      if (mine == 0u) break;  // (32 padding tokens end a run)
      fresh |= __any_sync(0xffffffffu, ((mine >> lane) & 1u) && s == (blk << p.scale_shift));
      n += 32 - __clz(mine);
      if (other != 0u) break;
    }
    for (int pair = blockIdx.y * kAppendWarps + warp; pair < pairs; pair += gridDim.y * kAppendWarps) {
      const bool isv = pair >= p.num_kv_heads;
      const int h = isv ? pair - p.num_kv_heads : pair;
      const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(isv ? p.value : p.key) + h * D + col * 8;
      const int64_t stride = isv ? p.value_stride : p.key_stride;
      signed char* pool = static_cast<signed char*>(isv ? p.value_pool : p.key_pool) + h * D;
      float* scale = (isv ? p.value_scales : p.key_scales) + blk * p.num_kv_heads + h;
      const int64_t pitch = (int64_t)p.num_kv_heads * D;
      auto row = [&](int64_t r) {
        return ld_stream(reinterpret_cast<const uint4*>(src + (t0 + r) * stride));
      };
      // the slot of span row r; -1: a padding token
      auto slot_of = [&](int64_t r) -> int64_t {
        const int64_t s = r < n ? slot_at(t0 + r) : -1;
        return block_of(s) == blk ? s : -1;
      };
      const float old = fresh ? 0.f : clamp_scale(__uint_as_float(ld_input(reinterpret_cast<const uint32_t*>(scale))));
      uint4 v[kPasses];
      int64_t at[kPasses];
      float a = 0.f;
#pragma unroll
      for (int x = 0; x < kPasses; ++x) {
        const int64_t r = x * kRows + sub;
        v[x] = r < n ? row(r) : make_uint4(0u, 0u, 0u, 0u);
        at[x] = slot_of(r);
      }
#pragma unroll
      for (int x = 0; x < kPasses; ++x)
        if (at[x] >= 0) a = max_abs8(a, v[x]);
      for (int64_t r = 16 + sub; r < n; r += kRows)
        if (slot_of(r) >= 0) a = max_abs8(a, row(r));
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
      const float s = fmaxf(old, clamp_scale(__fdiv_rn(a, 127.f)));
      if (!fresh && s > old) {
        const float ratio = __fdiv_rn(old, s);
        const int rows = 1 << p.scale_shift;
        for (int r = sub; r < rows; r += kRows) {
          uint2* c = reinterpret_cast<uint2*>(pool + ((blk << p.scale_shift) + r) * pitch + col * 8);
          const uint2 w = ld_input(c);
          *c = make_uint2(rescale4(w.x, ratio), rescale4(w.y, ratio));
        }
      }
      __syncwarp();  // the rows below land over the re-encoded ones
      if (lane == 0) *scale = s;
#pragma unroll
      for (int x = 0; x < kPasses; ++x)
        if (at[x] >= 0) *reinterpret_cast<uint2*>(pool + at[x] * pitch + col * 8) = codes8(v[x], s);
      for (int64_t r = 16 + sub; r < n; r += kRows) {
        const int64_t to = slot_of(r);
        if (to >= 0) *reinterpret_cast<uint2*>(pool + to * pitch + col * 8) = codes8(row(r), s);
      }
    }
  }
}

}  // namespace

cudaError_t launch_append_int8(const AppendInt8Params& p, int num_sms, cudaStream_t s) {
  if (p.num_tokens <= 0) return cudaSuccess;
  const int shares = (2 * p.num_kv_heads + kAppendWarps - 1) / kAppendWarps;
  // one token a CTA while that fills the SMs four times at most (a decode step: every
  // token is a run), else 16
  const int per_cta = p.num_tokens * shares <= 4 * (int64_t)num_sms ? 1 : 16;
  const int64_t ctas = (p.num_tokens + per_cta - 1) / per_cta;
  auto kern = p.head_dim == 128 ? append_int8_kernel<128> : append_int8_kernel<64>;
  return launch_pdl(kern, dim3((unsigned)ctas, (unsigned)std::min(shares, 65535)), dim3(kAppendWarps * 32), 0, s, p, per_cta);
}

}  // namespace pa
