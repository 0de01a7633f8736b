// Host side of the decode_split.cuh instantiations with EXT: tensor maps and
// dispatch.  Included by one translation unit for each (pool type, EXT).
#pragma once
#include "decode_split.cuh"

namespace pa {

namespace {

template <bool KV8, int EXT>
cudaError_t launch_decode_ext(const DecodeParams& p, cudaStream_t s) {
  const int D = p.pool.head_dim, rt = p.group <= 16 ? 1 : 2;
  const int R = p.pool.page_size < 16 ? p.pool.page_size : 16;
  const int64_t rows = p.pool.num_pages * (int64_t)p.pool.page_size;
  CUtensorMap tk, tv;
  if (KV8) {
    if (!encode_pool_tmap_u8(&tk, p.pool.key_pool, rows, p.pool.num_kv_heads, D, R, p.heads_per_box, true) ||
        !encode_pool_tmap_u8(&tv, p.pool.value_pool, rows, p.pool.num_kv_heads, D, R, p.heads_per_box, true))
      return cudaErrorInvalidValue;
  } else {
    const int slabs = R == 16 ? D / 64 : 1;
    if (!encode_pool_tmap(&tk, p.pool.key_pool, rows, p.pool.num_kv_heads, D, R, p.heads_per_box, slabs) ||
        !encode_pool_tmap(&tv, p.pool.value_pool, rows, p.pool.num_kv_heads, D, R, p.heads_per_box, slabs))
      return cudaErrorInvalidValue;
  }
  return D == 128 ? launch_split_d<128, KV8, false, EXT>(p, tk, tv, rt, s)
                  : launch_split_d<64, KV8, false, EXT>(p, tk, tv, rt, s);
}

}  // namespace

}  // namespace pa
