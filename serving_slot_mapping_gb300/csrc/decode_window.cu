// paged_attention_decode_window, bf16 pools: the sliding-window instantiations
// of the split-KV decode kernel in decode_split.cuh (see there), in a
// translation unit of their own so that they compile in parallel with the
// others and leave their code generation untouched.
#include "decode_split.cuh"

namespace pa {

cudaError_t launch_split_window_bf16(const DecodeParams& p, const CUtensorMap& tk, const CUtensorMap& tv, int rt,
                                     cudaStream_t s) {
  return p.pool.head_dim == 128 ? launch_split_d<128, false, false, true>(p, tk, tv, rt, s)
                                : launch_split_d<64, false, false, true>(p, tk, tv, rt, s);
}

}  // namespace pa
