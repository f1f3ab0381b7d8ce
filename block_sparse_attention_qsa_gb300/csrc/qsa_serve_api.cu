// C ABI of the entry points in qsa_serve.h: argument checks and launches.
#include <math.h>

#include "qsa_serve_internal.cuh"

using namespace qsa;

namespace {

bool needs_scales(const qsa_dims& d) { return d.kv_dtype == QSA_KV_FP8_E4M3; }

qsa_status prefix_attn(const qsa_dims* dims, int32_t alone, int32_t prefix_pages, const int32_t* prefix_table,
                       const void* q, const void* k_cache, const void* v_cache, const float* k_scale,
                       const float* v_scale, const int32_t* page_table, const int32_t* q_pos, void* out, float* lse,
                       void* ws, size_t ws_bytes, void* stream, bool short_k = false) {
  const qsa_status st = check_kv_dims(dims);
  if (st != QSA_OK) return st;
  if (prefix_pages < 0 || prefix_pages > dims->max_pages || (prefix_pages > 0 && !prefix_table))
    return QSA_ERR_INVALID_ARG;
  if (!q || !k_cache || !v_cache || !page_table || !q_pos || !out) return QSA_ERR_INVALID_ARG;
  if (needs_scales(*dims) && (!k_scale || !v_scale)) return QSA_ERR_INVALID_ARG;
  if (!aligned_all(16, {q, k_cache, v_cache, out}) ||
      !aligned_all(4, {k_scale, v_scale, prefix_table, page_table, q_pos, lse}))
    return QSA_ERR_INVALID_ARG;
  size_t need = 0;
  qsa_prefix_workspace_size(dims, prefix_pages, &need);
  if (!ws || !aligned(ws, 256) || ws_bytes < need) return QSA_ERR_WORKSPACE;
  return from_cuda(launch_paged_attn(*dims, 0, q, k_cache, v_cache, k_scale, v_scale, page_table, q_pos, out, lse, ws,
                                 static_cast<cudaStream_t>(stream), short_k,
                                 Prefix{prefix_table, prefix_pages * dims->page_size, alone}));
}

qsa_status kv_weight(const qsa_dims* dims, float decay, const void* q, const void* k_cache, const float* k_scale,
                     const int32_t* page_table, const int32_t* q_pos, const float* lse, float* weight, void* ws,
                     size_t ws_bytes, void* stream, bool short_k) {
  const qsa_status st = check_kv_dims(dims);
  if (st != QSA_OK) return st;
  if (!(decay >= 0.f && decay <= 1.f)) return QSA_ERR_INVALID_ARG;
  if (!q || !k_cache || !page_table || !q_pos || !lse || !weight) return QSA_ERR_INVALID_ARG;
  if (needs_scales(*dims) && !k_scale) return QSA_ERR_INVALID_ARG;
  if (!aligned_all(16, {q, k_cache}) || !aligned_all(4, {k_scale, page_table, q_pos, lse, weight}))
    return QSA_ERR_INVALID_ARG;
  if (!check_header(ws, ws_bytes)) return QSA_ERR_WORKSPACE;
  return from_cuda(launch_kv_weight(*dims, decay, q, k_cache, k_scale, page_table, q_pos, lse, weight,
                                    static_cast<int32_t*>(ws), static_cast<cudaStream_t>(stream), short_k));
}

}  // namespace

extern "C" {

qsa_status qsa_prefix_workspace_size(const qsa_dims* dims, int32_t prefix_pages, size_t* bytes) {
  const qsa_status st = check_kv_dims(dims);
  if (st != QSA_OK) return st;
  if (!bytes || prefix_pages < 0 || prefix_pages > dims->max_pages) return QSA_ERR_INVALID_ARG;
  *bytes = prefix_ws(*dims, prefix_pages * dims->page_size, device_sm_count());
  return QSA_OK;
}

qsa_status qsa_prefix_attn(const qsa_dims* dims, int32_t prefix_pages, const int32_t* prefix_table, const void* q,
                           const void* k_cache, const void* v_cache, const float* k_scale, const float* v_scale,
                           const int32_t* page_table, const int32_t* q_pos, void* out, float* lse, void* ws,
                           size_t ws_bytes, void* stream) {
  return prefix_attn(dims, -1, prefix_pages, prefix_table, q, k_cache, v_cache, k_scale, v_scale, page_table, q_pos,
                     out, lse, ws, ws_bytes, stream);
}

qsa_status qsa_test_prefix_attn(const qsa_dims* dims, int32_t alone, int32_t prefix_pages, const int32_t* prefix_table,
                                const void* q, const void* k_cache, const void* v_cache, const float* k_scale,
                                const float* v_scale, const int32_t* page_table, const int32_t* q_pos, void* out,
                                float* lse, void* ws, size_t ws_bytes, void* stream) {
  if (alone != 0 && alone != 1) return QSA_ERR_INVALID_ARG;
  return prefix_attn(dims, alone, prefix_pages, prefix_table, q, k_cache, v_cache, k_scale, v_scale, page_table, q_pos,
                     out, lse, ws, ws_bytes, stream);
}

qsa_status qsa_test_prefix_attn_timeout(const qsa_dims* dims, int32_t prefix_pages, const int32_t* prefix_table,
                                        const void* q, const void* k_cache, const void* v_cache, const float* k_scale,
                                        const float* v_scale, const int32_t* page_table, const int32_t* q_pos,
                                        void* out, float* lse, void* ws, size_t ws_bytes, void* stream) {
  if (prefix_pages < 1) return QSA_ERR_INVALID_ARG;
  return prefix_attn(dims, 0, prefix_pages, prefix_table, q, k_cache, v_cache, k_scale, v_scale, page_table, q_pos,
                     out, lse, ws, ws_bytes, stream, true);
}

qsa_status qsa_kv_weight(const qsa_dims* dims, float decay, const void* q, const void* k_cache, const float* k_scale,
                         const int32_t* page_table, const int32_t* q_pos, const float* lse, float* weight, void* ws,
                         size_t ws_bytes, void* stream) {
  return kv_weight(dims, decay, q, k_cache, k_scale, page_table, q_pos, lse, weight, ws, ws_bytes, stream, false);
}

qsa_status qsa_test_kv_weight_timeout(const qsa_dims* dims, float decay, const void* q, const void* k_cache,
                                      const float* k_scale, const int32_t* page_table, const int32_t* q_pos,
                                      const float* lse, float* weight, void* ws, size_t ws_bytes, void* stream) {
  return kv_weight(dims, decay, q, k_cache, k_scale, page_table, q_pos, lse, weight, ws, ws_bytes, stream, true);
}

qsa_status qsa_kv_evict(const qsa_dims* dims, int32_t keep, int32_t sinks, int32_t recent, int32_t out_pages,
                        const int32_t* len, const float* weight, const int32_t* page_table,
                        const int32_t* page_table_out, void* k_cache, void* v_cache, float* weight_out, int32_t* kept,
                        int32_t* new_len, void* ws, size_t ws_bytes, void* stream) {
  const qsa_status st = check_kv_dims(dims);
  if (st != QSA_OK) return st;
  if (out_pages < 1 || keep < 1 || sinks < 0 || recent < 0) return QSA_ERR_INVALID_ARG;
  const long long cap = (long long)out_pages * dims->page_size;
  if (cap >= (1LL << 31) || dims->batch * ((keep + 31LL) / 32) >= (1LL << 31)) return QSA_ERR_UNSUPPORTED;
  if (keep > cap || (long long)sinks + recent > keep) return QSA_ERR_INVALID_ARG;
  if (!len || !weight || !page_table || !page_table_out || !k_cache || !v_cache || !weight_out || !kept || !new_len)
    return QSA_ERR_INVALID_ARG;
  if (!aligned_all(16, {k_cache, v_cache}) ||
      !aligned_all(4, {len, weight, page_table, page_table_out, weight_out, kept, new_len}))
    return QSA_ERR_INVALID_ARG;
  // (a request's new weights are written while others' old ones are still read)
  if (weight < weight_out + dims->batch * cap &&
      weight_out < weight + (long long)dims->batch * dims->max_pages * dims->page_size)
    return QSA_ERR_INVALID_ARG;
  if (!check_header(ws, ws_bytes)) return QSA_ERR_WORKSPACE;
  EvictArgs a = {};
  a.len = len;
  a.weight = weight;
  a.page_table = page_table;
  a.page_table_out = page_table_out;
  a.k_cache = static_cast<uint8_t*>(k_cache);
  a.v_cache = static_cast<uint8_t*>(v_cache);
  a.weight_out = weight_out;
  a.kept = kept;
  a.new_len = new_len;
  a.err = static_cast<int32_t*>(ws);
  a.batch = dims->batch;
  a.keep = keep;
  a.sinks = sinks;
  a.recent = recent;
  a.out_pages = out_pages;
  a.hk = dims->n_kv_heads;
  a.row_bytes = dims->head_dim * (needs_scales(*dims) ? 1 : 2);
  a.page_size = dims->page_size;
  a.max_pages = dims->max_pages;
  a.num_pages = dims->num_pages;
  return from_cuda(launch_kv_evict(a, static_cast<cudaStream_t>(stream)));
}

qsa_status qsa_verify_drafts(int32_t batch, int32_t n_draft, int32_t vocab, int32_t prob_dtype, const void* target,
                             const qsa_prob_strides* target_strides, const void* draft,
                             const qsa_prob_strides* draft_strides, const int32_t* tokens, const float* uniform,
                             int32_t* accepted, int32_t* out_tokens, void* ws, size_t ws_bytes, void* stream) {
  if (batch < 1 || n_draft < 1 || vocab < 1) return QSA_ERR_INVALID_ARG;
  if (batch > (1 << 22) || n_draft > QSA_MAX_DRAFTS || vocab > QSA_MAX_VOCAB) return QSA_ERR_UNSUPPORTED;
  if (prob_dtype != QSA_PROB_F32 && prob_dtype != QSA_PROB_BF16) return QSA_ERR_UNSUPPORTED;
  if (!target || !tokens || !uniform || !accepted || !out_tokens) return QSA_ERR_INVALID_ARG;
  if (!aligned_all(prob_dtype == QSA_PROB_F32 ? 4 : 2, {target, draft}) ||
      !aligned_all(4, {tokens, uniform, accepted, out_tokens}))
    return QSA_ERR_INVALID_ARG;
  if (!check_header(ws, ws_bytes)) return QSA_ERR_WORKSPACE;
  VerifyArgs a = {};
  a.target = target;
  a.draft = draft;
  a.target_row = target_strides ? target_strides->row : vocab;
  a.target_batch = target_strides ? target_strides->batch : (long long)(n_draft + 1) * vocab;
  a.draft_row = draft_strides ? draft_strides->row : vocab;
  a.draft_batch = draft_strides ? draft_strides->batch : (long long)n_draft * vocab;
  a.tokens = tokens;
  a.uniform = uniform;
  a.accepted = accepted;
  a.out_tokens = out_tokens;
  a.err = static_cast<int32_t*>(ws);
  a.batch = batch;
  a.n_draft = n_draft;
  a.vocab = vocab;
  return from_cuda(launch_verify(a, prob_dtype == QSA_PROB_BF16, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
