// paged_attention_decode_mass, e4m3 pools: the split-KV decode kernel of decode_split.cuh
// that also keeps its scores.
#include "decode_ext.cuh"

namespace pa {

cudaError_t launch_decode_scores_e4m3(const DecodeParams& p, cudaStream_t s) {
  return launch_decode_ext<true, kExtMass>(p, s);
}

}  // namespace pa
