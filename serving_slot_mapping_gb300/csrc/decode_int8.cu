// paged_attention_decode_int8: the split-KV decode kernel of decode_split.cuh over
// int8 codes with a scale for each block of tokens and KV head.
#include "decode_ext.cuh"

namespace pa {

cudaError_t launch_decode_int8(const DecodeParams& p, cudaStream_t s) {
  return launch_decode_ext<true, kExtScales>(p, s);
}

}  // namespace pa
