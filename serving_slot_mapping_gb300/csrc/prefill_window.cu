// paged_attention_prefill_window: the sliding-window instantiations of the
// tensor-core prefill kernel in prefill_tc.cuh, in a translation unit of their
// own so that they leave the plain ones' code generation untouched.
#include "prefill_tc.cuh"

namespace pa {

cudaError_t launch_prefill_window(const PrefillParams& p, cudaStream_t s) {
  if (p.kv8)
    return p.pool.head_dim == 128 ? launch_prefill_tc<128, true, true>(p, s) : launch_prefill_tc<64, true, true>(p, s);
  return p.pool.head_dim == 128 ? launch_prefill_tc<128, false, true>(p, s) : launch_prefill_tc<64, false, true>(p, s);
}

}  // namespace pa
