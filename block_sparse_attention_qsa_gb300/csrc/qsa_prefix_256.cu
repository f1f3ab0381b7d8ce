// Attention over a shared prefix for head dim 256 (one translation unit a head
// dim: they compile side by side).
#include "qsa_prefix.cuh"

namespace qsa {

cudaError_t launch_prefix_256(const qsa_dims& d, const PrefixArgs& a, const void* k, const void* v, bool short_k,
                              cudaStream_t s) {
  const bool fp8 = d.kv_dtype == QSA_KV_FP8_E4M3;
  return fp8 ? launch_prefix<256, true, 1>(d, a, k, v, short_k, s) : launch_prefix<256, false, 1>(d, a, k, v, short_k, s);
}

}  // namespace qsa
