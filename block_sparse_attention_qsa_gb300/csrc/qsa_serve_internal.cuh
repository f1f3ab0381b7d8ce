// Declarations shared by the translation units of the entry points in qsa_serve.h.
#pragma once

#include "qsa_kv_internal.cuh"
#include "qsa_serve.h"

namespace qsa {

constexpr int kErrToken = 7;   // qsa_verify_drafts: a drafted token outside the vocabulary
constexpr int kErrLength = 8;  // qsa_kv_evict: a length outside the page table
constexpr int kErrHeavy = 9;   // qsa_verify_drafts: weights that sum to 16 or more

// short_k: the failure-detection test (qsa_test_kv_weight_timeout)
cudaError_t launch_kv_weight(const qsa_dims& d, float decay, const void* q, const void* k_cache, const float* k_scale,
                             const int32_t* page_table, const int32_t* q_pos, const float* lse, float* weight,
                             int32_t* err, cudaStream_t s, bool short_k);

struct EvictArgs {
  const int32_t* len;
  const float* weight;
  const int32_t* page_table;
  const int32_t* page_table_out;
  uint8_t* k_cache;
  uint8_t* v_cache;
  float* weight_out;
  int32_t* kept;
  int32_t* new_len;
  int32_t* err;
  int batch, keep, sinks, recent, out_pages;
  int hk, row_bytes, page_size, max_pages, num_pages;
  unsigned held;  // weights of a CTA's slice in shared memory (set by the launcher)
};
cudaError_t launch_kv_evict(EvictArgs a, cudaStream_t s);

struct VerifyArgs {
  const void* target;
  const void* draft;  // null: the drafts were not sampled
  long long target_batch, target_row, draft_batch, draft_row;
  const int32_t* tokens;
  const float* uniform;
  int32_t* accepted;
  int32_t* out_tokens;
  int32_t* err;
  int batch, n_draft, vocab;
};
cudaError_t launch_verify(const VerifyArgs& a, bool bf16, cudaStream_t s);

// launch_k with thread-block clusters of `cluster` CTAs (along x)
template <typename... KArgs, typename... Args>
cudaError_t launch_clusters(void (*kern)(KArgs...), dim3 grid, dim3 block, unsigned cluster, size_t smem,
                            cudaStream_t s, Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kern, std::forward<Args>(args)...);
}

}  // namespace qsa
