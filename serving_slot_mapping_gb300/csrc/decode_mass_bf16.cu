// paged_attention_decode_mass, bf16 pools: the split-KV decode kernel of decode_split.cuh
// that also keeps its scores.
#include "decode_ext.cuh"

namespace pa {

cudaError_t launch_decode_scores_bf16(const DecodeParams& p, cudaStream_t s) {
  return launch_decode_ext<false, kExtMass>(p, s);
}

}  // namespace pa
