#include "qsa_dense.cuh"

namespace qsa {

EncodeTiled encode_tiled() {
  static EncodeTiled fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<EncodeTiled>(p);
  }();
  return fn;
}

// Rows of a unit: a softmax thread's work grows with its warpgroup's rows, so
// the smallest of 8, 16, 32 (two warpgroups of 16) and 64 (two of 32) that
// holds them; more rows are several units, which each read K and V. Rows of
// 512 bytes leave no shared memory for 64.
static int unit_rows(const qsa_dims& d) {
  const int rows = d.n_q * (d.n_q_heads / d.n_kv_heads);
  const bool wide = d.head_dim == 256 && d.kv_dtype == QSA_KV_BF16;
  return rows <= 8 ? 8 : rows <= 16 ? 16 : rows <= 32 || wide ? 32 : 64;
}

DenseWs dense_ws(const qsa_dims& d, int num_sms) {
  DenseWs w;
  const int rows = d.n_q * (d.n_q_heads / d.n_kv_heads), per = unit_rows(d);
  const size_t units = (size_t)d.batch * d.n_kv_heads * ((rows + per - 1) / per);
  w.units = 256 + align_up((size_t)d.batch * d.n_q * d.n_kv_heads * sizeof(int32_t), 256);
  w.parts = align_up(w.units + units * sizeof(long long), 256);
  w.total = align_up(w.parts + (size_t)num_sms * 2 * per * (d.head_dim + 2) * sizeof(float), 256);
  return w;
}

cudaError_t launch_paged_attn(const qsa_dims& d, int window, const void* q, const void* k_cache, const void* v_cache,
                              const float* k_scale, const float* v_scale, const int32_t* page_table,
                              const int32_t* q_pos, void* out, float* lse, void* ws, cudaStream_t s, bool short_k) {
  const int sms = device_sm_count();
  const DenseWs w = dense_ws(d, sms);
  uint8_t* base = static_cast<uint8_t*>(ws);
  DenseArgs a = {};
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  a.page_table = page_table;
  a.q_pos = q_pos;
  a.out = static_cast<__nv_bfloat16*>(out);
  a.lse = lse;
  a.unit_desc = reinterpret_cast<long long*>(base + w.units);
  a.parts = reinterpret_cast<float*>(base + w.parts);
  a.err = static_cast<int32_t*>(ws);
  a.batch = d.batch;
  a.n_q = d.n_q;
  a.n_q_heads = d.n_q_heads;
  a.n_kv_heads = d.n_kv_heads;
  a.group = d.n_q_heads / d.n_kv_heads;
  a.page_size = d.page_size;
  while ((1 << a.page_shift) < d.page_size) ++a.page_shift;
  a.max_pages = d.max_pages;
  a.num_pages = d.num_pages;
  a.window = window;
  a.grid = sms;
  a.sm_scale = d.sm_scale > 0.f ? d.sm_scale : 1.f / sqrtf((float)d.head_dim);
  a.one = 1.f;
  const int rows = unit_rows(d);
  switch (d.head_dim) {
    case 64: return launch_dense_64(rows, d, a, k_cache, v_cache, short_k, s);
    case 128: return launch_dense_128(rows, d, a, k_cache, v_cache, short_k, s);
    default: return launch_dense_256(rows, d, a, k_cache, v_cache, short_k, s);
  }
}

}  // namespace qsa
