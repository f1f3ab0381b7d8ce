// Dense attention for head dim 64 (one translation unit a head dim: they
// compile side by side).
#include "qsa_dense_tc.cuh"

namespace qsa {

cudaError_t launch_dense_64(int rows, const qsa_dims& d, const DenseArgs& a, const void* k_cache, const void* v_cache,
                            bool short_k, cudaStream_t s) {
  return d.kv_dtype == QSA_KV_FP8_E4M3 ? launch_tc<64, true>(rows, d, a, k_cache, v_cache, short_k, s)
                                       : launch_tc<64, false>(rows, d, a, k_cache, v_cache, short_k, s);
}

}  // namespace qsa
