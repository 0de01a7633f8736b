// paged_attention_decode_mass: the attention weight of every key, summed over the
// query heads and added to what the key had before.
//
// A weight needs its row's whole sum, which is known when the decode ends: the
// decode kernel (decode_split.cuh, kExtMass) leaves the scaled scores x [B, Hq, keys]
// and each row's lse = log2 sum_j 2^x, and key_mass_kernel computes
//   mass_out[b, j] = decay mass_in[b, j] + sum_h 2^(x[b, h, j] - lse[b, h]),
// heads in ascending order, so the sums are the same on every run.
//
// 4 Hq bytes a key read (mostly from L2, where the decode has just put them) beside
// 4 to 8 of mass.
#include "common.cuh"
#include "inputs.cuh"
#include "internal.h"

namespace pa {

namespace {

constexpr int kMassThreads = 128;
constexpr int kMaxMassHeads = 1024;  // lse staged this many heads at a time

__global__ void __launch_bounds__(kMassThreads) key_mass_kernel(const __grid_constant__ KeyMassParams p) {
  __shared__ float lse[kMaxMassHeads];
  griddep_wait();
  const int b = blockIdx.y, L = ld_seq_len(p.seq_lens, b, p.max_len, nullptr);
  const int j = (blockIdx.x * kMassThreads + threadIdx.x) * 2;
  if (blockIdx.x * kMassThreads * 2 >= L) return;
  float a0 = 0.f, a1 = 0.f;
  for (int h0 = 0; h0 < p.num_q_heads; h0 += kMaxMassHeads) {
    const int heads = min(kMaxMassHeads, p.num_q_heads - h0);
    if (h0 > 0) __syncthreads();
    for (int h = threadIdx.x; h < heads; h += kMassThreads)
      lse[h] = __uint_as_float(ld_input(reinterpret_cast<const uint32_t*>(p.lse) + (int64_t)b * p.num_q_heads + h0 + h));
    __syncthreads();
    if (j < L) {
      const float* x = p.scores + ((int64_t)b * p.num_q_heads + h0) * p.score_stride + j;
#pragma unroll 8
      for (int h = 0; h < heads; ++h) {
        const uint2 v = ld_input(reinterpret_cast<const uint2*>(x + h * p.score_stride));
        a0 += fast_exp2(__uint_as_float(v.x) - lse[h]);
        a1 += fast_exp2(__uint_as_float(v.y) - lse[h]);
      }
    }
  }
  float* out = p.mass_out + b * p.mass_stride;
  const uint32_t* in = reinterpret_cast<const uint32_t*>(p.mass_in) + b * p.mass_stride;
  if (j < L) out[j] = p.mass_in != nullptr ? fmaf(p.decay, __uint_as_float(ld_input(in + j)), a0) : a0;
  if (j + 1 < L) out[j + 1] = p.mass_in != nullptr ? fmaf(p.decay, __uint_as_float(ld_input(in + j + 1)), a1) : a1;
}

}  // namespace

cudaError_t launch_key_mass(const KeyMassParams& p, cudaStream_t s) {
  if (p.max_keys <= 0) return cudaSuccess;
  const int per = kMassThreads * 2;
  return launch_pdl(key_mass_kernel, dim3((unsigned)((p.max_keys + per - 1) / per), (unsigned)p.batch),
                    dim3(kMassThreads), 0, s, p);
}

cudaError_t launch_decode_scores(const DecodeParams& p, cudaStream_t s) {
  if (p.key_scales != nullptr) return launch_decode_scores_int8(p, s);
  return p.kv8 ? launch_decode_scores_e4m3(p, s) : launch_decode_scores_bf16(p, s);
}

}  // namespace pa
