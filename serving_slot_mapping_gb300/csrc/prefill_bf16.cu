// paged_attention_prefill, bf16 and e4m3 pools: the instantiations of the
// tensor-core prefill kernel in prefill_tc.cuh.
#include "prefill_tc.cuh"

namespace pa {

cudaError_t launch_prefill_bf16(const PrefillParams& p, cudaStream_t s) {
  if (p.max_q_len <= 0 || p.batch <= 0) return cudaSuccess;
  if (p.kv8) return p.pool.head_dim == 128 ? launch_prefill_tc<128, true>(p, s) : launch_prefill_tc<64, true>(p, s);
  return p.pool.head_dim == 128 ? launch_prefill_tc<128, false>(p, s) : launch_prefill_tc<64, false>(p, s);
}

}  // namespace pa
