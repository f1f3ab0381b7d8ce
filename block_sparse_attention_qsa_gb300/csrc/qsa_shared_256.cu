// Dense attention for head dim 256 where requests share a prefix.
#include "qsa_dense_tc.cuh"

namespace qsa {

cudaError_t launch_dense_256(int rows, const qsa_dims& d, const SharedArgs& a, const void* k_cache, const void* v_cache,
                            bool short_k, cudaStream_t s) {
  return d.kv_dtype == QSA_KV_FP8_E4M3 ? launch_tc<256, true>(rows, d, a, k_cache, v_cache, short_k, s)
                                       : launch_tc<256, false>(rows, d, a, k_cache, v_cache, short_k, s);
}

}  // namespace qsa
