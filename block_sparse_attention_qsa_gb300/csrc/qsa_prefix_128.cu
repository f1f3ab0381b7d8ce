// Attention over a shared prefix for head dim 128 (one translation unit a head
// dim: they compile side by side).
#include "qsa_prefix.cuh"

namespace qsa {

cudaError_t launch_prefix_128(const qsa_dims& d, const PrefixArgs& a, const void* k, const void* v, bool short_k,
                              cudaStream_t s) {
  const bool fp8 = d.kv_dtype == QSA_KV_FP8_E4M3;
  if (a.row_tiles == 1)
    return fp8 ? launch_prefix<128, true, 1>(d, a, k, v, short_k, s)
               : launch_prefix<128, false, 1>(d, a, k, v, short_k, s);
  return fp8 ? launch_prefix<128, true, 2>(d, a, k, v, short_k, s) : launch_prefix<128, false, 2>(d, a, k, v, short_k, s);
}

}  // namespace qsa
