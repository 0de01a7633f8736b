// paged_qk_norm_rope_append: per-head RMS norm of queries and keys, position
// rotation, and the write of keys and values into the page pool, in one pass.
//
// For a token t at position p and a head row x of head_dim elements:
//   y = x / sqrt(mean(x^2) + eps) * w          (no norm: y = x)
//   (y_a, y_b) -> (y_a cos - y_b sin, y_b cos + y_a sin)  for each pair (a, b)
// of the first rotary_dim dims, with cos / sin row p of the table; q rows go
// to q_out, k rows to slot_mapping[t] of the key pool, v rows (untouched) to the
// value pool.  Everything is fp32 until the one rounding to the output type
// (e4m3 pools: the IEEE quotient by the scale, as paged_kv_append).
//
// Bound by memory: each row is read once and written once, and by the
// instructions between: a first form with a thread's heads converted, normed and
// rotated one operation at a time issued 315 instructions per 4 heads and ran at
// half the copy rate.  On a GB300, 10,496 tokens of 32 + 8 + 8 heads of 128 bf16
// dims (262 MB): 45 us, 5.8 TB/s (75 us in the first form); one token: 2.3 us.
// * A thread holds V elements of each half of a head (16-byte accesses for bf16 V
//   = 8 and fp32 V = 4), placed so that both elements of every rotated pair are
//   its own; a head takes LPH lanes (8 for 128 bf16 dims), its sum of squares
//   LPH-wide shuffles.
// * A warp walks a token's heads (two warps share them in the ring below, several
//   where there are few tokens), 32 / LPH at a time: a thread's dims stay the same, so
//   weight, cosine and sine are multiplied into four factors per dim pair once per
//   token, and a head costs two packed fp32 instructions per pair and one more for
//   1 / sqrt(mean).
// * Many tokens whose rows fit the ring go through shared memory; few tokens, and
//   wider or unaligned rows, straight to registers.  10,496 tokens of 40 + 8 + 8, 64 +
//   8 + 8 and 32 + 32 + 32 heads of 128 that way: 63, 88 and 98 us, 0.71 to 0.78 of
//   the copy rate.
#include <cmath>

#include "common.cuh"
#include "inputs.cuh"
#include "internal.h"
#include "tma.cuh"

namespace pa {

namespace {

constexpr int kThreads = 128;
constexpr int kAhead = 2;  // heads of a thread whose loads are in flight together

// Pairs of floats (first in the low half): the packed fp32 instructions of
// sm_100+, each half rounded as the scalar one.
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
__device__ __forceinline__ uint64_t swap_pair(uint64_t x) {
  const float2 v = unpair(x);
  return pair(v.y, v.x);
}
__device__ __forceinline__ uint64_t mul_pair(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t fma_pair(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}

// V consecutive elements as loaded: 32-bit words.
template <typename T, int V>
struct Raw {
  static constexpr int kWords = V * (int)sizeof(T) / 4;
  uint32_t w[kWords];
};

// VEC: the address is aligned to the whole vector, else element by element.
// Rows are read once (streaming); a norm weight by every token.
template <typename T, int V, bool VEC, bool STREAM>
__device__ __forceinline__ Raw<T, V> load_raw(const T* src) {
  Raw<T, V> r;
  if constexpr (VEC && Raw<T, V>::kWords == 4) {
    const uint4* s = reinterpret_cast<const uint4*>(src);
    const uint4 v = STREAM ? ld_stream(s) : ld_input(s);
    r.w[0] = v.x; r.w[1] = v.y; r.w[2] = v.z; r.w[3] = v.w;
  } else if constexpr (VEC) {
    const uint2* s = reinterpret_cast<const uint2*>(src);
    const uint2 v = STREAM ? ld_stream(s) : ld_input(s);
    r.w[0] = v.x; r.w[1] = v.y;
  } else if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < V; ++i) r.w[i] = reinterpret_cast<const uint32_t*>(src)[i];
  } else {
    const unsigned short* s = reinterpret_cast<const unsigned short*>(src);
#pragma unroll
    for (int i = 0; i < V / 2; ++i) r.w[i] = (uint32_t)s[2 * i] | ((uint32_t)s[2 * i + 1] << 16);
  }
  return r;
}

template <typename T, int V, bool VEC>
__device__ __forceinline__ void store_raw(T* dst, const Raw<T, V>& r) {
  if constexpr (VEC && Raw<T, V>::kWords == 4) {
    *reinterpret_cast<uint4*>(dst) = make_uint4(r.w[0], r.w[1], r.w[2], r.w[3]);
  } else if constexpr (VEC) {
    *reinterpret_cast<uint2*>(dst) = make_uint2(r.w[0], r.w[1]);
  } else if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < V; ++i) reinterpret_cast<uint32_t*>(dst)[i] = r.w[i];
  } else {
    unsigned short* d = reinterpret_cast<unsigned short*>(dst);
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
      d[2 * i] = (unsigned short)(r.w[i] & 0xFFFFu);
      d[2 * i + 1] = (unsigned short)(r.w[i] >> 16);
    }
  }
}

// Elements 2i and 2i + 1 as a pair of floats, and back with one rounding.
template <int V>
__device__ __forceinline__ uint64_t get_pair(const Raw<__nv_bfloat16, V>& r, int i) {
  return pair(__uint_as_float(r.w[i] << 16), __uint_as_float(r.w[i] & 0xFFFF0000u));
}
template <int V>
__device__ __forceinline__ uint64_t get_pair(const Raw<float, V>& r, int i) {
  return pair(__uint_as_float(r.w[2 * i]), __uint_as_float(r.w[2 * i + 1]));
}
template <int V>
__device__ __forceinline__ void set_pair(Raw<__nv_bfloat16, V>& r, int i, uint64_t x) {
  const float2 v = unpair(x);
  r.w[i] = pack_bf16(v.x, v.y);
}
template <int V>
__device__ __forceinline__ void set_pair(Raw<float, V>& r, int i, uint64_t x) {
  const float2 v = unpair(x);
  r.w[2 * i] = __float_as_uint(v.x);
  r.w[2 * i + 1] = __float_as_uint(v.y);
}

// V values as e4m3 codes of x / scale (the correctly rounded quotient, nearest
// even, saturating).  With inv = the rounded reciprocal of the scale, q = x inv
// and q + (x - q scale) inv, both fused, is the correctly rounded quotient unless
// the scale's significand is all ones (Markstein, IBM J. Res. Dev. 34, 1990); the
// host gives inv = 0 for those scales and for ones so small (below 2^-90) that the
// remainder x - q scale would not be exact, or near the other end of fp32's range.
// Quotients outside 2^-12 .. 2^12 round to 0 or saturate as they stand (and
// infinities and NaN pass).  A division each took the e4m3 append from 61 to 72 us
// for 10,496 tokens.
template <int V, bool VEC>
__device__ __forceinline__ void store_codes(unsigned char* dst, const uint64_t (&x)[V / 2], float scale, float inv) {
  uint32_t c[V / 2];
  auto quotient = [&](float v) {
    const float q = v * inv, r = fmaf(fmaf(-q, scale, v), inv, q);
    return fabsf(q) >= 0x1p-12f && fabsf(q) <= 0x1p12f ? r : q;
  };
  if (inv != 0.f) {
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
      const float2 v = unpair(x[i]);
      c[i] = f32x2_to_e4m3x2(quotient(v.x), quotient(v.y));
    }
  } else {
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
      const float2 v = unpair(x[i]);
      c[i] = f32x2_to_e4m3x2(__fdiv_rn(v.x, scale), __fdiv_rn(v.y, scale));
    }
  }
  if constexpr (VEC) {
    const uint32_t lo = c[0] | (c[1] << 16);
    if constexpr (V == 8)
      *reinterpret_cast<uint2*>(dst) = make_uint2(lo, c[2] | (c[3] << 16));
    else
      *reinterpret_cast<uint32_t*>(dst) = lo;
  } else {
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
      dst[2 * i] = (unsigned char)(c[i] & 0xFFu);
      dst[2 * i + 1] = (unsigned char)(c[i] >> 8);
    }
  }
}

// A lane's place in the heads of a pass: which head of the pass, and its dims a ..
// a + V - 1 and b .. b + V - 1: the two halves of the rotated dims, then of the rest.
template <int V>
struct Lane {
  int g, a, b;
  bool on, turn;
  __device__ Lane(const NormRopeParams& p, int lane) {
    const int lph = p.lanes_per_head, rot = p.rotary_dim, D = p.head_dim;  // lph: power of two >= D / (2 V)
    const int u = lane & (lph - 1);
    g = lane / lph;
    on = u < D / (2 * V);
    turn = u < rot / (2 * V);
    a = turn ? u * V : rot + (u - rot / (2 * V)) * V;
    b = a + (turn ? rot / 2 : (D - rot) / 2);
  }
};

// Cosines and sines of a lane's pairs (1 and 0 where nothing turns): half-split,
// those of dims a + e (and b + e); interleaved, those of the pairs of a, then of
// the pairs of b.  `row`: a position's row of the table (global or shared memory).
template <int V, bool VEC, bool INTER>
struct Turn {
  float cs[V], sn[V];
  __device__ __forceinline__ Turn(const NormRopeParams& p, const Lane<V>& ln, const float* row) {
#pragma unroll
    for (int e = 0; e < V; ++e) {
      cs[e] = 1.f;
      sn[e] = 0.f;
    }
    if (!ln.on || !ln.turn) return;
    const float* srow = row + p.rotary_dim / 2;
    if constexpr (VEC && V == 8) {
      const int lo = INTER ? ln.a / 2 : ln.a, hi = INTER ? ln.b / 2 : ln.a + 4;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float4 c = *reinterpret_cast<const float4*>(row + (h ? hi : lo));
        const float4 s = *reinterpret_cast<const float4*>(srow + (h ? hi : lo));
        cs[4 * h] = c.x; cs[4 * h + 1] = c.y; cs[4 * h + 2] = c.z; cs[4 * h + 3] = c.w;
        sn[4 * h] = s.x; sn[4 * h + 1] = s.y; sn[4 * h + 2] = s.z; sn[4 * h + 3] = s.w;
      }
    } else {
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const int i = !INTER ? ln.a + e : (e < V / 2 ? ln.a / 2 + e : ln.b / 2 + e - V / 2);
        cs[e] = row[i];
        sn[e] = srow[i];
      }
    }
  }
};

// Rotated, normed values are r (X * P + X' * Q) by pairs, r = 1 / sqrt(mean + eps):
// half-split, (za, zb) = r (xa wa c - xb wb s, xb wb c + xa wa s), X' the other
// half; interleaved, (z0, z1) = r (x0 w0 c - x1 w1 s, x1 w1 c + x0 w0 s), X' the
// pair swapped.
template <typename T, int V, bool VEC, bool INTER>
struct Factors {
  uint64_t Pa[V / 2], Qa[V / 2], Pb[V / 2], Qb[V / 2];
  __device__ __forceinline__ void set(const NormRopeParams& p, const Lane<V>& ln, const Turn<V, VEC, INTER>& tr,
                                      const T* w) {
    const bool norm = w != nullptr && ln.on;
    Raw<T, V> ra = {}, rb = {};
    if (norm) {
      ra = load_raw<T, V, VEC, false>(w + ln.a);
      rb = load_raw<T, V, VEC, false>(w + ln.b);
    }
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
      const float2 wa = norm ? unpair(get_pair(ra, i)) : make_float2(1.f, 1.f);
      const float2 wb = norm ? unpair(get_pair(rb, i)) : make_float2(1.f, 1.f);
      if constexpr (!INTER) {
        const float c0 = tr.cs[2 * i], c1 = tr.cs[2 * i + 1], s0 = tr.sn[2 * i], s1 = tr.sn[2 * i + 1];
        Pa[i] = pair(wa.x * c0, wa.y * c1);
        Qa[i] = pair(-wb.x * s0, -wb.y * s1);
        Pb[i] = pair(wb.x * c0, wb.y * c1);
        Qb[i] = pair(wa.x * s0, wa.y * s1);
      } else {
        const float ca = tr.cs[i], cb = tr.cs[V / 2 + i], sa = tr.sn[i], sb = tr.sn[V / 2 + i];
        Pa[i] = pair(wa.x * ca, wa.y * ca);
        Qa[i] = pair(-wa.y * sa, wa.x * sa);
        Pb[i] = pair(wb.x * cb, wb.y * cb);
        Qb[i] = pair(-wb.y * sb, wb.x * sb);
      }
    }
  }
  // One pass of heads (whole warp): za, zb of the halves xa, xb.
  __device__ __forceinline__ void apply(const NormRopeParams& p, const Lane<V>& ln, bool norm, const Raw<T, V>& xa,
                                        const Raw<T, V>& xb, uint64_t (&za)[V / 2], uint64_t (&zb)[V / 2]) const {
    uint64_t A[V / 2], B[V / 2];
#pragma unroll
    for (int e = 0; e < V / 2; ++e) {
      A[e] = get_pair(xa, e);
      B[e] = get_pair(xb, e);
    }
    uint64_t r2 = 0ull;
    if (norm) {
      uint64_t s0 = 0ull, s1 = 0ull;
#pragma unroll
      for (int e = 0; e < V / 2; ++e) {
        s0 = fma_pair(A[e], A[e], s0);
        s1 = fma_pair(B[e], B[e], s1);
      }
      const float2 sa = unpair(s0), sb = unpair(s1);
      float ss = (sa.x + sa.y) + (sb.x + sb.y);
      for (int o = p.lanes_per_head >> 1; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      const float r = rsqrtf(fmaf(ss, p.inv_dim, p.eps));
      r2 = pair(r, r);
    }
#pragma unroll
    for (int e = 0; e < V / 2; ++e) {
      za[e] = mul_pair(A[e], Pa[e]);
      zb[e] = mul_pair(B[e], Pb[e]);
    }
    if (ln.turn) {  // (not where nothing turns: 0 times an infinite partner is no 0)
#pragma unroll
      for (int e = 0; e < V / 2; ++e) {
        za[e] = fma_pair(INTER ? swap_pair(A[e]) : B[e], Qa[e], za[e]);
        zb[e] = fma_pair(INTER ? swap_pair(B[e]) : A[e], Qb[e], zb[e]);
      }
    }
    if (norm) {
#pragma unroll
      for (int e = 0; e < V / 2; ++e) {
        za[e] = mul_pair(za[e], r2);
        zb[e] = mul_pair(zb[e], r2);
      }
    }
  }
};

template <typename T, int V, bool VEC>
__device__ __forceinline__ void store_pairs(T* dst, const uint64_t (&z)[V / 2]) {
  Raw<T, V> y;
#pragma unroll
  for (int e = 0; e < V / 2; ++e) set_pair(y, e, z[e]);
  store_raw<T, V, VEC>(dst, y);
}

// A token's slot, or -1 where there is nothing to write: padding, or a slot or
// position out of range (recorded by the lane that gets `err`).
__device__ __forceinline__ int64_t live_slot(const NormRopeParams& p, int64_t slot, int pos, unsigned long long* err) {
  if (slot < 0) return -1;
  if (slot >= p.num_slots) {
    if (err != nullptr) record_error(err, ERR_SLOT, slot);
    return -1;
  }
  if (p.rotary_dim > 0 && (pos < 0 || pos >= p.max_position)) {
    if (err != nullptr) record_error(err, ERR_POSITION, pos);
    return -1;
  }
  return slot;
}

// T: element type of q, key and value rows; KV8: the pools hold e4m3 codes
// (else T); V: elements of one half of a thread's share of a head; VEC: every
// row address is aligned to a vector of V elements.
template <typename T, bool KV8, int V, bool VEC>
__device__ __forceinline__ void store_key(const NormRopeParams& p, const Lane<V>& ln, int64_t at,
                                          const uint64_t (&za)[V / 2], const uint64_t (&zb)[V / 2]) {
  if constexpr (KV8) {
    store_codes<V, VEC>(static_cast<unsigned char*>(p.key_pool) + at + ln.a, za, p.k_scale, p.k_inv);
    store_codes<V, VEC>(static_cast<unsigned char*>(p.key_pool) + at + ln.b, zb, p.k_scale, p.k_inv);
  } else {
    store_pairs<T, V, VEC>(static_cast<T*>(p.key_pool) + at + ln.a, za);
    store_pairs<T, V, VEC>(static_cast<T*>(p.key_pool) + at + ln.b, zb);
  }
}

template <typename T, bool KV8, int V, bool VEC>
__device__ __forceinline__ void store_value(const NormRopeParams& p, const Lane<V>& ln, int64_t at, const Raw<T, V>& xa,
                                            const Raw<T, V>& xb) {
  if constexpr (KV8) {
    uint64_t za[V / 2], zb[V / 2];
#pragma unroll
    for (int e = 0; e < V / 2; ++e) {
      za[e] = get_pair(xa, e);
      zb[e] = get_pair(xb, e);
    }
    store_codes<V, VEC>(static_cast<unsigned char*>(p.value_pool) + at + ln.a, za, p.v_scale, p.v_inv);
    store_codes<V, VEC>(static_cast<unsigned char*>(p.value_pool) + at + ln.b, zb, p.v_scale, p.v_inv);
  } else {
    store_raw<T, V, VEC>(static_cast<T*>(p.value_pool) + at + ln.a, xa);
    store_raw<T, V, VEC>(static_cast<T*>(p.value_pool) + at + ln.b, xb);
  }
}

// Few tokens, or rows that no bulk copy takes: rows straight to registers, the
// passes over a token's heads spread over p.slices warps.
template <typename T, bool KV8, int V, bool VEC, bool INTER>
__global__ void __launch_bounds__(kThreads) qk_norm_rope_append_kernel(const __grid_constant__ NormRopeParams p) {
  // No early trigger: the attention kernels read their queries and tables ahead
  // of their own wait, and q_out is written here.
  const int64_t unit = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  const int64_t t = unit / p.slices;
  if (t >= p.num_tokens) return;
  const int slice = (int)(unit - t * p.slices);
  const int hpw = 32 / p.lanes_per_head;  // heads of one pass
  const int D = p.head_dim;
  const Lane<V> ln(p, threadIdx.x & 31);
  const int q_passes = (p.num_q_heads + hpw - 1) / hpw, kv_passes = (p.num_kv_heads + hpw - 1) / hpw;
  const T* q = static_cast<const T*>(p.q) + t * p.q_stride;
  const T* k = static_cast<const T*>(p.key) + t * p.key_stride;
  const T* v = static_cast<const T*>(p.value) + t * p.value_stride;
  T* qo = static_cast<T*>(p.q_out) + t * (int64_t)p.num_q_heads * D;
  Raw<T, V> xa[kAhead], xb[kAhead];
  // the halves of head (pass + i * slices) * hpw + g of a row of heads
  auto load = [&](const T* row, int heads, int pass) {
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int h = (pass + i * p.slices) * hpw + ln.g;
      if (h < heads && ln.on) {
        xa[i] = load_raw<T, V, VEC, true>(row + h * D + ln.a);
        xb[i] = load_raw<T, V, VEC, true>(row + h * D + ln.b);
      } else {
        xa[i] = xb[i] = Raw<T, V>{};
      }
    }
  };
  griddep_wait();
  // this slice's first passes over q, k and v (a token's passes are counted
  // through all three)
  auto first_pass = [&](int before) { return (slice - before % p.slices + p.slices) % p.slices; };
  const int q0 = slice, k0 = first_pass(q_passes), v0 = first_pass(q_passes + kv_passes);
  if (q0 < q_passes) load(q, p.num_q_heads, q0);  // in flight while slot, position and table are read
  const int pos = p.rotary_dim > 0 ? ld_input(p.positions + t) : 0;
  const int64_t slot =
      live_slot(p, ld_input(p.slot_mapping + t), pos, slice == 0 && (threadIdx.x & 31) == 0 ? p.err : nullptr);
  if (slot < 0) return;
  const Turn<V, VEC, INTER> tr(p, ln, p.cos_sin + (int64_t)pos * p.rotary_dim);
  Factors<T, V, VEC, INTER> f;
  const int step = kAhead * p.slices;
  if (q0 < q_passes) {
    f.set(p, ln, tr, static_cast<const T*>(p.q_weight));
    for (int pass = q0; pass < q_passes; pass += step) {
      if (pass != q0) load(q, p.num_q_heads, pass);
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        if (pass + i * p.slices >= q_passes) break;
        uint64_t za[V / 2], zb[V / 2];
        f.apply(p, ln, p.q_weight != nullptr, xa[i], xb[i], za, zb);
        const int h = (pass + i * p.slices) * hpw + ln.g;
        if (h < p.num_q_heads && ln.on) {
          store_pairs<T, V, VEC>(qo + h * D + ln.a, za);
          store_pairs<T, V, VEC>(qo + h * D + ln.b, zb);
        }
      }
    }
  }
  const int64_t pool_row = slot * (int64_t)p.num_kv_heads * D;
  if (k0 < kv_passes) {
    load(k, p.num_kv_heads, k0);
    f.set(p, ln, tr, static_cast<const T*>(p.k_weight));
    for (int pass = k0; pass < kv_passes; pass += step) {
      if (pass != k0) load(k, p.num_kv_heads, pass);
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        if (pass + i * p.slices >= kv_passes) break;
        uint64_t za[V / 2], zb[V / 2];
        f.apply(p, ln, p.k_weight != nullptr, xa[i], xb[i], za, zb);
        const int h = (pass + i * p.slices) * hpw + ln.g;
        if (h < p.num_kv_heads && ln.on) store_key<T, KV8, V, VEC>(p, ln, pool_row + (int64_t)h * D, za, zb);
      }
    }
  }
  for (int pass = v0; pass < kv_passes; pass += step) {
    load(v, p.num_kv_heads, pass);
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int h = (pass + i * p.slices) * hpw + ln.g;
      if (h < p.num_kv_heads && ln.on) store_value<T, KV8, V, VEC>(p, ln, pool_row + (int64_t)h * D, xa[i], xb[i]);
    }
  }
}

// Many tokens: a team of two warps walks tokens w, w + teams, ... through a ring of
// its own of kSlots tokens in shared memory, filled by bulk copies of the token's
// q, k, v and cos / sin rows, so that every team always has a token's 12 KB in
// flight (in registers the bytes in flight cost occupancy: 55 us at best for the
// same rows).  The warps share a token's passes: one warp a token left 8 warps an
// SM, whose latency bound the call (49 us).
constexpr int kSlots = 2;
constexpr int kTeamWarps = 2;
constexpr int kTeams = 4;  // a block
constexpr int kBulkThreads = 32 * kTeamWarps * kTeams;

template <typename T, bool KV8, int V, bool INTER>
__global__ void __launch_bounds__(kBulkThreads, 2) qk_norm_rope_append_bulk_kernel(const __grid_constant__ NormRopeParams p) {
  extern __shared__ __align__(128) unsigned char smem[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int team = warp / kTeamWarps, part = warp % kTeamWarps;  // this warp's passes: part, part + kTeamWarps, ...
  const bool leads = part == 0 && lane == 0;                     // issues the team's copies, records errors
  const int D = p.head_dim, rot = p.rotary_dim, hpw = 32 / p.lanes_per_head;
  const Lane<V> ln(p, lane);
  const int q_bytes = p.num_q_heads * D * (int)sizeof(T), kv_bytes = p.num_kv_heads * D * (int)sizeof(T);
  const int stage = p.stage_bytes;
  unsigned char* ring = smem + team * kSlots * stage;
  const uint32_t bars = smem_u32(smem + kTeams * kSlots * stage) + 8u * (team * kSlots);
  if (threadIdx.x < kTeams * kSlots) {
    mbar_init(smem_u32(smem + kTeams * kSlots * stage) + 8u * threadIdx.x, 1);
    fence_mbar_init();
  }
  __syncthreads();
  const int64_t teams = (int64_t)gridDim.x * kTeams;
  int64_t t = (int64_t)blockIdx.x * kTeams + team;
  griddep_wait();
  // slot and position of a token (every lane the same)
  auto look_up = [&](int64_t x, int64_t* slot, int* pos) {
    *slot = -1;
    *pos = 0;
    if (x >= p.num_tokens) return;
    *slot = ld_input(p.slot_mapping + x);
    if (rot > 0) *pos = ld_input(p.positions + x);
  };
  auto issue = [&](int64_t x, int pos, int s) {  // one thread
    const uint32_t dst = smem_u32(ring + s * stage), bar = bars + 8u * s;
    mbar_arrive_expect_tx(bar, (uint32_t)(q_bytes + 2 * kv_bytes + rot * 4));
    bulk_load(dst, static_cast<const T*>(p.q) + x * p.q_stride, q_bytes, bar);
    bulk_load(dst + q_bytes, static_cast<const T*>(p.key) + x * p.key_stride, kv_bytes, bar);
    bulk_load(dst + q_bytes + kv_bytes, static_cast<const T*>(p.value) + x * p.value_stride, kv_bytes, bar);
    if (rot > 0) bulk_load(dst + q_bytes + 2 * kv_bytes, p.cos_sin + (int64_t)pos * rot, rot * 4, bar);
  };
  int64_t slot, next_slot, raw;
  int raw_pos;
  look_up(t, &raw, &raw_pos);
  slot = live_slot(p, raw, raw_pos, leads ? p.err : nullptr);
  if (slot >= 0 && leads) issue(t, raw_pos, 0);
  look_up(t + teams, &raw, &raw_pos);
  uint32_t phases = 0;  // bit s: parity of slot s's next phase
  bool alive = true;
  for (int s = 0; t < p.num_tokens; t += teams, s ^= 1) {
    // the next token's copies, the one after's slot and position
    next_slot = t + teams < p.num_tokens ? live_slot(p, raw, raw_pos, leads ? p.err : nullptr) : -1;
    if (next_slot >= 0 && leads) issue(t + teams, raw_pos, s ^ 1);
    look_up(t + 2 * teams, &raw, &raw_pos);
    if (slot >= 0) {
      if (alive) alive = mbar_wait(bars + 8u * s, (phases >> s) & 1u, p.err);
      phases ^= 1u << s;
      const unsigned char* row = ring + s * stage;
      const T* q = reinterpret_cast<const T*>(row);
      const T* k = reinterpret_cast<const T*>(row + q_bytes);
      const T* v = reinterpret_cast<const T*>(row + q_bytes + kv_bytes);
      const Turn<V, true, INTER> tr(p, ln, reinterpret_cast<const float*>(row + q_bytes + 2 * kv_bytes));
      T* qo = static_cast<T*>(p.q_out) + t * (int64_t)p.num_q_heads * D;
      Factors<T, V, true, INTER> f;
      auto half = [&](const T* base, int h, int d) {
        Raw<T, V> x = {};
        if (ln.on) {
          const uint4 w = *reinterpret_cast<const uint4*>(base + h * D + d);
          x.w[0] = w.x; x.w[1] = w.y; x.w[2] = w.z; x.w[3] = w.w;
        }
        return x;
      };
      f.set(p, ln, tr, static_cast<const T*>(p.q_weight));
#pragma unroll 2
      for (int h0 = part * hpw; h0 < p.num_q_heads; h0 += kTeamWarps * hpw) {
        const int h = min(h0 + ln.g, p.num_q_heads - 1);
        uint64_t za[V / 2], zb[V / 2];
        f.apply(p, ln, p.q_weight != nullptr, half(q, h, ln.a), half(q, h, ln.b), za, zb);
        if (h0 + ln.g < p.num_q_heads && ln.on) {
          store_pairs<T, V, true>(qo + h * D + ln.a, za);
          store_pairs<T, V, true>(qo + h * D + ln.b, zb);
        }
      }
      const int64_t pool_row = slot * (int64_t)p.num_kv_heads * D;
      f.set(p, ln, tr, static_cast<const T*>(p.k_weight));
      for (int h0 = part * hpw; h0 < p.num_kv_heads; h0 += kTeamWarps * hpw) {
        const int h = min(h0 + ln.g, p.num_kv_heads - 1);
        const bool mine = h0 + ln.g < p.num_kv_heads && ln.on;
        const int64_t at = pool_row + (int64_t)h * D;
        uint64_t za[V / 2], zb[V / 2];
        f.apply(p, ln, p.k_weight != nullptr, half(k, h, ln.a), half(k, h, ln.b), za, zb);
        if (mine) {
          store_key<T, KV8, V, true>(p, ln, at, za, zb);
          store_value<T, KV8, V, true>(p, ln, at, half(v, h, ln.a), half(v, h, ln.b));
        }
      }
      named_barrier(1 + team, 32 * kTeamWarps);  // the token is read: its slot may be filled again
    }
    slot = next_slot;
  }
}

template <typename T, bool KV8, int V, bool VEC, bool INTER>
cudaError_t launch_style(NormRopeParams p, int num_sms, cudaStream_t s) {
  int lph = 1;
  while (lph < p.head_dim / (2 * V)) lph *= 2;
  p.lanes_per_head = lph;
  p.inv_dim = 1.f / (float)p.head_dim;
  auto reciprocal = [](float scale) {
    int e = 0;
    const float f = std::frexp(scale, &e);  // in [1/2, 1)
    // q >= 2^-12 ends at 2^-35 and scale at 2^(e - 24): their product at 2^-149 or above
    return e > -90 && e < 100 && f != 1.f - 0x1p-24f ? 1.f / scale : 0.f;
  };
  p.k_inv = KV8 ? reciprocal(p.k_scale) : 0.f;
  p.v_inv = KV8 ? reciprocal(p.v_scale) : 0.f;
  if constexpr (VEC && V * sizeof(T) == 16) {
    // bulk copies: 16-byte rows, two blocks an SM, and tokens for half the teams
    // (2048 tokens of 48 bf16 heads of 128: 9.7 us, straight to registers 14.0; 512
    // tokens, fewer than half: 6.4 us straight)
    const int64_t row = (int64_t)(p.num_q_heads + 2 * p.num_kv_heads) * p.head_dim * (int)sizeof(T) + p.rotary_dim * 4;
    const int64_t stage = (row + 127) / 128 * 128;
    const int64_t smem = kTeams * kSlots * (stage + 8);
    const int64_t teams = 2 * (int64_t)num_sms * kTeams;
    if (p.bulk && smem <= 113 * 1024 && p.num_tokens >= teams / 2) {
      p.stage_bytes = (int32_t)stage;
      auto kern = qk_norm_rope_append_bulk_kernel<T, KV8, V, INTER>;
      const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
      if (e != cudaSuccess) return e;
      return launch_pdl(kern, dim3((unsigned)(2 * num_sms)), dim3(kBulkThreads), (size_t)smem, s, p);
    }
  }
  const int hpw = 32 / lph;
  const int passes = (p.num_q_heads + hpw - 1) / hpw + 2 * ((p.num_kv_heads + hpw - 1) / hpw);
  // a token a warp once that fills the SMs (32 warps each); with fewer tokens
  // the passes of a token go to several warps
  const int64_t want = (32 * (int64_t)num_sms + p.num_tokens - 1) / p.num_tokens;
  p.slices = (int)(want < passes ? want : passes);
  const int64_t warps = p.num_tokens * p.slices;
  const int64_t blocks = (warps + kThreads / 32 - 1) / (kThreads / 32);
  return launch_pdl(qk_norm_rope_append_kernel<T, KV8, V, VEC, INTER>, dim3((unsigned)blocks), dim3(kThreads), 0, s, p);
}

template <typename T, bool KV8, int V, bool VEC>
cudaError_t launch(const NormRopeParams& p, int num_sms, cudaStream_t s) {
  return p.interleaved ? launch_style<T, KV8, V, VEC, true>(p, num_sms, s)
                       : launch_style<T, KV8, V, VEC, false>(p, num_sms, s);
}

}  // namespace

cudaError_t launch_qk_norm_rope_append(const NormRopeParams& p, int num_sms, cudaStream_t s) {
  if (p.num_tokens <= 0) return cudaSuccess;
  if (p.f32) return p.vec ? launch<float, false, 4, true>(p, num_sms, s) : launch<float, false, 4, false>(p, num_sms, s);
  if (p.kv8) {
    if (p.vec == 8) return launch<__nv_bfloat16, true, 8, true>(p, num_sms, s);
    return p.vec ? launch<__nv_bfloat16, true, 4, true>(p, num_sms, s) : launch<__nv_bfloat16, true, 4, false>(p, num_sms, s);
  }
  if (p.vec == 8) return launch<__nv_bfloat16, false, 8, true>(p, num_sms, s);
  return p.vec ? launch<__nv_bfloat16, false, 4, true>(p, num_sms, s) : launch<__nv_bfloat16, false, 4, false>(p, num_sms, s);
}

}  // namespace pa
