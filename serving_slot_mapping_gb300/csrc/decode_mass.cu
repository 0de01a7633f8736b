// paged_attention_decode_mass: the attention weight of every key, summed over the
// query heads and added to what the key had before.
//
// A weight needs its row's whole sum, which is known when the decode ends: the
// decode kernel (decode_split.cuh, kExtMass) leaves the scaled scores x [B, Hq, keys]
// and each row's lse = log2 sum_j 2^x, and key_mass_kernel computes
//   mass_out[b, j] = decay mass_in[b, j] + sum_h 2^(x[b, h, j] - lse[b, h]).
// A block takes 128 or 256 keys of a sequence, four a lane and tile; its warps share the
// heads, each with all its loads in flight (32 heads in one round trip), and their sums are
// added in the order of the warps: the same on every run.
//
// 4 Hq bytes a key read (mostly from L2, where the decode has just put them) beside
// 4 to 8 of mass.
#include "common.cuh"
#include "inputs.cuh"
#include "internal.h"

namespace pa {

namespace {

constexpr int kMassWarps = 8;
constexpr int kMassKeys = 128;   // of a tile: four a lane
constexpr int kMassAhead = 4;    // heads of a warp and tile in flight

// T: tiles of a block.
template <int T>
__global__ void __launch_bounds__(kMassWarps * 32) key_mass_kernel(const __grid_constant__ KeyMassParams p) {
  __shared__ float4 part[kMassWarps][T * 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  griddep_wait();
  const int b = blockIdx.y, L = ld_seq_len(p.seq_lens, b, p.max_len, nullptr);
  const int j0 = blockIdx.x * T * kMassKeys;
  if (j0 >= L) return;
  const int Hq = p.num_q_heads;
  const float* x = p.scores + (int64_t)b * Hq * p.score_stride + j0 + 4 * lane;
  const uint32_t* lse = reinterpret_cast<const uint32_t*>(p.lse) + (int64_t)b * Hq;
  float4 a[T];
#pragma unroll
  for (int t = 0; t < T; ++t) a[t] = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int h0 = warp; h0 < Hq; h0 += kMassWarps * kMassAhead) {
    uint4 v[kMassAhead][T];
    float m[kMassAhead];
#pragma unroll
    for (int k = 0; k < kMassAhead; ++k) {
      const int h = h0 + k * kMassWarps;
      if (h >= Hq) break;
#pragma unroll
      for (int t = 0; t < T; ++t)  // (rows of the scores are padded to 16 keys)
        if (j0 + t * kMassKeys + 4 * lane < L)
          v[k][t] = ld_input(reinterpret_cast<const uint4*>(x + h * p.score_stride + t * kMassKeys));
      m[k] = __uint_as_float(ld_input(lse + h));
    }
#pragma unroll
    for (int k = 0; k < kMassAhead; ++k) {
      if (h0 + k * kMassWarps >= Hq) break;
#pragma unroll
      for (int t = 0; t < T; ++t) {
        if (j0 + t * kMassKeys + 4 * lane >= L) break;
        a[t].x += fast_exp2(__uint_as_float(v[k][t].x) - m[k]);
        a[t].y += fast_exp2(__uint_as_float(v[k][t].y) - m[k]);
        a[t].z += fast_exp2(__uint_as_float(v[k][t].z) - m[k]);
        a[t].w += fast_exp2(__uint_as_float(v[k][t].w) - m[k]);
      }
    }
  }
#pragma unroll
  for (int t = 0; t < T; ++t) part[warp][t * 32 + lane] = a[t];
  __syncthreads();
  const int key = j0 + threadIdx.x;
  if (threadIdx.x >= T * kMassKeys || key >= L) return;
  float sum = 0.f;
#pragma unroll
  for (int w = 0; w < kMassWarps; ++w) sum += reinterpret_cast<const float*>(part[w])[threadIdx.x];
  const int64_t at = b * p.mass_stride + key;
  p.mass_out[at] =
      p.mass_in != nullptr ? fmaf(p.decay, __uint_as_float(ld_input(reinterpret_cast<const uint32_t*>(p.mass_in) + at)), sum)
                           : sum;
}

template <int T>
cudaError_t launch_mass(const KeyMassParams& p, cudaStream_t s) {
  const int per = T * kMassKeys;
  return launch_pdl(key_mass_kernel<T>, dim3((unsigned)((p.max_keys + per - 1) / per), (unsigned)p.batch),
                    dim3(kMassWarps * 32), 0, s, p);
}

}  // namespace

// Two tiles a block past 8 single ones an SM, the most whose threads it holds.  It sees the
// bound of the lengths: blocks past a sequence's end return at once.
int key_mass_tiles(int num_sms, int32_t batch, int32_t max_keys) {
  const int64_t tiles = (int64_t)batch * (((int64_t)max_keys + kMassKeys - 1) / kMassKeys);
  return tiles <= 8 * (int64_t)num_sms ? 1 : 2;
}

cudaError_t launch_key_mass(const KeyMassParams& p, int num_sms, cudaStream_t s) {
  if (p.max_keys <= 0) return cudaSuccess;
  return key_mass_tiles(num_sms, p.batch, p.max_keys) == 1 ? launch_mass<1>(p, s) : launch_mass<2>(p, s);
}

cudaError_t launch_decode_scores(const DecodeParams& p, cudaStream_t s) {
  if (p.key_scales != nullptr) return launch_decode_scores_int8(p, s);
  return p.kv8 ? launch_decode_scores_e4m3(p, s) : launch_decode_scores_bf16(p, s);
}

}  // namespace pa
