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
// Bound by memory: each row is read once and written once.  A thread holds V
// elements of each half of a head (16-byte accesses for bf16 V = 8 and fp32 V
// = 4), placed so that both elements of every rotated pair are its own; a head
// takes LPH lanes (8 for 128 bf16 dims), its sum of squares LPH-wide shuffles.
// A block serves one token, so the cos / sin values of a thread's dims are read
// once and used for all its heads.
#include "common.cuh"
#include "internal.h"

namespace pa {

namespace {

constexpr int kThreads = 128;
constexpr int kHeadsAhead = 3;  // heads of a thread whose loads are in flight together

// N consecutive elements as floats; VEC: the address is aligned to the whole
// vector (16 bytes, or 8 for N = 4 bf16), else element by element.
template <int N, bool VEC>
__device__ __forceinline__ void load_row(const __nv_bfloat16* src, float (&x)[N]) {
  if constexpr (VEC) {
    uint32_t w[N / 2];
    if constexpr (N == 8) {
      const uint4 v = __ldcs(reinterpret_cast<const uint4*>(src));
      w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
    } else {
      const uint2 v = __ldcs(reinterpret_cast<const uint2*>(src));
      w[0] = v.x; w[1] = v.y;
    }
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = __bfloat162float(src[i]);
  }
}

template <int N, bool VEC>
__device__ __forceinline__ void load_row(const float* src, float (&x)[N]) {
  if constexpr (VEC) {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      const float4 v = __ldcs(reinterpret_cast<const float4*>(src + i));
      x[i] = v.x; x[i + 1] = v.y; x[i + 2] = v.z; x[i + 3] = v.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = src[i];
  }
}

template <int N, bool VEC>
__device__ __forceinline__ void store_row(__nv_bfloat16* dst, const float (&x)[N]) {
  if constexpr (VEC) {
    uint32_t w[N / 2];
#pragma unroll
    for (int i = 0; i < N / 2; ++i) w[i] = pack_bf16(x[2 * i], x[2 * i + 1]);
    if constexpr (N == 8)
      *reinterpret_cast<uint4*>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
    else
      *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[1]);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) dst[i] = __float2bfloat16_rn(x[i]);
  }
}

template <int N, bool VEC>
__device__ __forceinline__ void store_row(float* dst, const float (&x)[N]) {
  if constexpr (VEC) {
#pragma unroll
    for (int i = 0; i < N; i += 4)
      *reinterpret_cast<float4*>(dst + i) = make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) dst[i] = x[i];
  }
}

// N elements of a norm weight (read by every head: kept in the caches)
template <int N, bool VEC, typename T>
__device__ __forceinline__ void load_weight(const T* src, float (&x)[N]) {
  if constexpr (VEC && sizeof(T) * N >= 16) {
    static_assert(sizeof(T) * N == 16, "one 16-byte vector");
    const uint4 v = __ldg(reinterpret_cast<const uint4*>(src));
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (sizeof(T) == 4) {
        x[i] = __uint_as_float(w[i]);
      } else {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = (float)src[i];
  }
}

// N values as e4m3 codes of x / scale (IEEE division, nearest even, saturating)
template <int N, bool VEC>
__device__ __forceinline__ void store_codes(unsigned char* dst, const float (&x)[N], float scale) {
  uint32_t c[N / 2];
#pragma unroll
  for (int i = 0; i < N / 2; ++i) c[i] = f32x2_to_e4m3x2(__fdiv_rn(x[2 * i], scale), __fdiv_rn(x[2 * i + 1], scale));
  if constexpr (VEC) {
    const uint32_t lo = c[0] | (c[1] << 16);
    if constexpr (N == 8)
      *reinterpret_cast<uint2*>(dst) = make_uint2(lo, c[2] | (c[3] << 16));
    else
      *reinterpret_cast<uint32_t*>(dst) = lo;
  } else {
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
      dst[2 * i] = (unsigned char)(c[i] & 0xFFu);
      dst[2 * i + 1] = (unsigned char)(c[i] >> 8);
    }
  }
}

// T: element type of q, key and value rows; KV8: the pools hold e4m3 codes
// (else T); V: elements of one half of a thread's share of a head; VEC: every
// row address is aligned to a vector of V elements.
template <typename T, bool KV8, int V, bool VEC>
__global__ void __launch_bounds__(kThreads) qk_norm_rope_append_kernel(NormRopeParams p) {
  // No early trigger: the attention kernels read their queries and tables ahead
  // of their own wait, and q_out is written here.
  const int lph = p.lanes_per_head;                  // power of two >= D / (2 V)
  const int D = p.head_dim, rot = p.rotary_dim;
  const int u = threadIdx.x & (lph - 1);             // this thread's chunk of a head
  const int g0 = threadIdx.x / lph;                  // head within a pass of the block
  const int per_pass = kThreads / lph;
  const int heads = p.num_q_heads + 2 * p.num_kv_heads;  // q, then k, then v
  const bool on = u < D / (2 * V);
  // dims a .. a + V - 1 and b .. b + V - 1: the two halves of the rotated
  // dims, then of the rest
  const bool turn = u < rot / (2 * V);
  const int a = turn ? u * V : rot + (u - rot / (2 * V)) * V;
  const int b = a + (turn ? rot / 2 : (D - rot) / 2);
  griddep_wait();
  const int64_t t = blockIdx.x;
  const int64_t slot = __ldg(p.slot_mapping + t);
  if (slot < 0) return;  // padding token
  if (slot >= p.num_slots) {
    if (threadIdx.x == 0 && blockIdx.y == 0) record_error(p.err, ERR_SLOT, slot);
    return;
  }
  float cs[V], sn[V];  // half-split pairs: of dims a + e (and b + e); interleaved: pairs of a, then of b
  if (rot > 0) {
    const int pos = __ldg(p.positions + t);
    if (pos < 0 || pos >= p.max_position) {
      if (threadIdx.x == 0 && blockIdx.y == 0) record_error(p.err, ERR_POSITION, pos);
      return;
    }
    const float* row = p.cos_sin + (int64_t)pos * rot;
    if (on && turn) {
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const int i = !p.interleaved ? a + e : (e < V / 2 ? a / 2 + e : b / 2 + e - V / 2);
        cs[e] = __ldg(row + i);
        sn[e] = __ldg(row + rot / 2 + i);
      }
    }
  }
  const int64_t pool_row = slot * (int64_t)p.num_kv_heads * D;
  const T* q = static_cast<const T*>(p.q) + t * p.q_stride;
  const T* k = static_cast<const T*>(p.key) + t * p.key_stride;
  const T* v = static_cast<const T*>(p.value) + t * p.value_stride;
  T* qo = static_cast<T*>(p.q_out) + t * (int64_t)p.num_q_heads * D;
  const int step = per_pass * gridDim.y;
  for (int h0 = blockIdx.y * per_pass; h0 < heads; h0 += kHeadsAhead * step) {
    float x[kHeadsAhead][2][V];
#pragma unroll
    for (int i = 0; i < kHeadsAhead; ++i) {
      const int h = h0 + i * step + g0;
      if (h < heads && on) {
        const T* src = h < p.num_q_heads ? q + h * D
                       : h < p.num_q_heads + p.num_kv_heads ? k + (h - p.num_q_heads) * D
                                                            : v + (h - p.num_q_heads - p.num_kv_heads) * D;
        load_row<V, VEC>(src + a, x[i][0]);
        load_row<V, VEC>(src + b, x[i][1]);
      } else {
#pragma unroll
        for (int e = 0; e < V; ++e) x[i][0][e] = x[i][1][e] = 0.f;
      }
    }
#pragma unroll
    for (int i = 0; i < kHeadsAhead; ++i) {
      const int h = h0 + i * step + g0;
      const bool is_q = h < p.num_q_heads, is_v = h >= p.num_q_heads + p.num_kv_heads;
      const T* w = static_cast<const T*>(is_q ? p.q_weight : p.k_weight);
      float ss = 0.f;
#pragma unroll
      for (int e = 0; e < V; ++e) ss += x[i][0][e] * x[i][0][e] + x[i][1][e] * x[i][1][e];
      for (int o = lph >> 1; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      if (h >= heads || !on) continue;
      if (!is_v) {
        if (w != nullptr) {
          const float r = 1.f / sqrtf(ss / (float)D + p.eps);
          float wa[V], wb[V];
          load_weight<V, VEC>(w + a, wa);
          load_weight<V, VEC>(w + b, wb);
#pragma unroll
          for (int e = 0; e < V; ++e) {
            x[i][0][e] *= r * wa[e];
            x[i][1][e] *= r * wb[e];
          }
        }
        if (rot > 0 && turn) {
          if (!p.interleaved) {
#pragma unroll
            for (int e = 0; e < V; ++e) {
              const float xa = x[i][0][e], xb = x[i][1][e];
              x[i][0][e] = xa * cs[e] - xb * sn[e];
              x[i][1][e] = xb * cs[e] + xa * sn[e];
            }
          } else {
#pragma unroll
            for (int s = 0; s < 2; ++s)
#pragma unroll
              for (int e = 0; e < V / 2; ++e) {
                const float c = cs[s * (V / 2) + e], sv = sn[s * (V / 2) + e];
                const float xa = x[i][s][2 * e], xb = x[i][s][2 * e + 1];
                x[i][s][2 * e] = xa * c - xb * sv;
                x[i][s][2 * e + 1] = xb * c + xa * sv;
              }
          }
        }
      }
      if (is_q) {
        store_row<V, VEC>(qo + h * D + a, x[i][0]);
        store_row<V, VEC>(qo + h * D + b, x[i][1]);
      } else {
        const int hk = h - p.num_q_heads - (is_v ? p.num_kv_heads : 0);
        void* pool = is_v ? p.value_pool : p.key_pool;
        const int64_t at = pool_row + (int64_t)hk * D;
        if constexpr (KV8) {
          const float scale = is_v ? p.v_scale : p.k_scale;
          store_codes<V, VEC>(static_cast<unsigned char*>(pool) + at + a, x[i][0], scale);
          store_codes<V, VEC>(static_cast<unsigned char*>(pool) + at + b, x[i][1], scale);
        } else {
          store_row<V, VEC>(static_cast<T*>(pool) + at + a, x[i][0]);
          store_row<V, VEC>(static_cast<T*>(pool) + at + b, x[i][1]);
        }
      }
    }
  }
}

template <typename T, bool KV8, int V, bool VEC>
cudaError_t launch(NormRopeParams p, int num_sms, cudaStream_t s) {
  int lph = 1;
  while (lph < p.head_dim / (2 * V)) lph *= 2;
  p.lanes_per_head = lph;
  const int per_pass = kThreads / lph;
  const int passes = (p.num_q_heads + 2 * p.num_kv_heads + per_pass - 1) / per_pass;
  // few tokens: one pass of heads a block, to spread them over the SMs
  const int gy = p.num_tokens < 4 * (int64_t)num_sms ? (passes < 65535 ? passes : 65535) : 1;
  return launch_pdl(qk_norm_rope_append_kernel<T, KV8, V, VEC>, dim3((unsigned)p.num_tokens, (unsigned)gy),
                    dim3(kThreads), 0, s, p);
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
