// C ABI of the entry points in qsa_kv.h: argument checks and launches, and the
// host side of the rotary frequencies.
#include <math.h>

#include <initializer_list>

#include "qsa_kv_internal.cuh"

using namespace qsa;

namespace {

constexpr double kPi = 3.14159265358979323846;

qsa_status check_kv_dims(const qsa_dims* d) {
  if (!d) return QSA_ERR_INVALID_ARG;
  if (d->batch < 1 || d->n_q < 1 || d->max_pages < 1 || d->num_pages < 1 || d->n_kv_heads < 1 ||
      d->n_q_heads < 1 || d->page_size < 1)
    return QSA_ERR_INVALID_ARG;
  if (d->head_dim != 64 && d->head_dim != 128 && d->head_dim != 256) return QSA_ERR_UNSUPPORTED;
  if (d->n_q_heads % d->n_kv_heads != 0 || d->n_q_heads > QSA_MAX_KV_HEADS) return QSA_ERR_UNSUPPORTED;
  if (d->n_q > kMaxNq) return QSA_ERR_UNSUPPORTED;
  if (d->page_size < 16 || d->page_size > 256 || (d->page_size & (d->page_size - 1)) != 0)
    return QSA_ERR_UNSUPPORTED;
  if (d->kv_dtype != QSA_KV_BF16 && d->kv_dtype != QSA_KV_FP8_E4M3) return QSA_ERR_UNSUPPORTED;
  if (!(d->sm_scale >= 0.f) || isinf(d->sm_scale)) return QSA_ERR_INVALID_ARG;
  if (d->batch > (1 << 22)) return QSA_ERR_UNSUPPORTED;  // the kernels' request counters
  // 32-bit position and row indexes of the kernels
  if ((long long)d->max_pages * d->page_size >= (1LL << 31)) return QSA_ERR_UNSUPPORTED;
  if ((long long)d->batch * d->n_q * d->n_q_heads >= (1LL << 31)) return QSA_ERR_UNSUPPORTED;
  return QSA_OK;
}

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

bool aligned_all(uintptr_t a, std::initializer_list<const void*> ps) {
  for (const void* p : ps)
    if (!aligned(p, a)) return false;
  return true;
}

bool check_header(const void* ws, size_t bytes) { return ws && aligned(ws, 256) && bytes >= 256; }

qsa_status from_cuda(cudaError_t e) { return e == cudaSuccess ? QSA_OK : QSA_ERR_CUDA; }

// (a dimension of one element has no stride, whatever the caller's says)
Strided strided(const void* p, const qsa_strides* s, int batch, int n_tok, int heads, int dim) {
  Strided t;
  t.p = static_cast<__nv_bfloat16*>(const_cast<void*>(p));
  t.head = heads == 1 ? 0 : s ? s->head : dim;
  t.token = n_tok == 1 ? 0 : s ? s->token : (long long)heads * dim;
  t.batch = batch == 1 ? 0 : s ? s->batch : (long long)n_tok * heads * dim;
  return t;
}

// an output's strides must move it to other elements in every dimension it has
bool writable(const Strided& t, int batch, int n_tok, int heads) {
  return (t.batch != 0 || batch == 1) && (t.token != 0 || n_tok == 1) && (t.head != 0 || heads == 1);
}

// an output that starts where an input does must be that input, in place
bool in_place_or_apart(const Strided& in, const Strided& out) {
  return in.p != out.p || (in.batch == out.batch && in.token == out.token && in.head == out.head);
}

qsa_status check_rope(const qsa_rope_args* r, int head_dim, Rope* out) {
  if (!r) {
    *out = Rope{nullptr, 1.f, 0, 0};
    return QSA_OK;
  }
  if (!r->turns || !aligned(r->turns, 8)) return QSA_ERR_INVALID_ARG;
  if (r->rot_dim < 2 || r->rot_dim % 2 != 0 || r->rot_dim > head_dim) return QSA_ERR_INVALID_ARG;
  if (r->layout != QSA_ROPE_HALF && r->layout != QSA_ROPE_INTERLEAVED) return QSA_ERR_INVALID_ARG;
  if (!(r->amplitude > 0.f) || isinf(r->amplitude)) return QSA_ERR_INVALID_ARG;
  *out = Rope{r->turns, r->amplitude, r->rot_dim, r->layout == QSA_ROPE_INTERLEAVED};
  return QSA_OK;
}

qsa_status paged_attn(const qsa_dims* dims, int32_t window, const void* q, const void* k_cache,
                      const void* v_cache, const float* k_scale, const float* v_scale,
                      const int32_t* page_table, const int32_t* q_pos, void* out, float* lse, void* ws,
                      size_t ws_bytes, void* stream, bool short_k) {
  const qsa_status st = check_kv_dims(dims);
  if (st != QSA_OK) return st;
  if (window < 0 || !q || !k_cache || !v_cache || !page_table || !q_pos || !out) return QSA_ERR_INVALID_ARG;
  if (dims->kv_dtype == QSA_KV_FP8_E4M3 && (!k_scale || !v_scale)) return QSA_ERR_INVALID_ARG;
  if (!aligned_all(16, {q, k_cache, v_cache, out}) || !aligned_all(4, {k_scale, v_scale, page_table, q_pos, lse}))
    return QSA_ERR_INVALID_ARG;
  if (!ws || !aligned(ws, 256) || ws_bytes < dense_ws(*dims, device_sm_count()).total) return QSA_ERR_WORKSPACE;
  return from_cuda(launch_paged_attn(*dims, window, q, k_cache, v_cache, k_scale, v_scale, page_table, q_pos, out,
                                     lse, ws, static_cast<cudaStream_t>(stream), short_k));
}

}  // namespace

extern "C" {

qsa_status qsa_rope_table(const qsa_rope_spec* s, uint64_t* turns, float* amplitude) {
  if (!s || !turns || !amplitude) return QSA_ERR_INVALID_ARG;
  const int R = s->rot_dim;
  if (R < 2 || R % 2 != 0 || R > 256) return QSA_ERR_INVALID_ARG;
  if (s->layout != QSA_ROPE_HALF && s->layout != QSA_ROPE_INTERLEAVED) return QSA_ERR_INVALID_ARG;
  if (s->scaling < QSA_ROPE_NONE || s->scaling > QSA_ROPE_YARN) return QSA_ERR_INVALID_ARG;
  double base = s->base == 0 ? 10000.0 : s->base;
  const double f = s->scaling == QSA_ROPE_NONE || s->factor == 0 ? 1.0 : s->factor;
  // (comparisons written so that a NaN is refused)
  if (!(base > 1.0) || isinf(base) || !(f >= 1.0) || isinf(f)) return QSA_ERR_INVALID_ARG;
  double alpha = s->alpha, beta = s->beta;
  if (alpha == 0 && beta == 0) alpha = 1, beta = 32;
  const bool yarn = s->scaling == QSA_ROPE_YARN;
  if (yarn && (!(s->orig_len >= 1.0) || isinf(s->orig_len) || !(alpha >= 0) || !(beta > alpha) || isinf(beta)))
    return QSA_ERR_INVALID_ARG;
  if (!(s->amplitude >= 0) || isinf(s->amplitude)) return QSA_ERR_INVALID_ARG;
  if (s->scaling == QSA_ROPE_NTK) {
    if (R == 2) return QSA_ERR_INVALID_ARG;
    base *= pow(f, (double)R / (R - 2));
    if (isinf(base)) return QSA_ERR_INVALID_ARG;
  }
  for (int i = 0; i < R / 2; ++i) {
    double w = pow(base, -2.0 * i / R);
    if (s->scaling == QSA_ROPE_LINEAR) w /= f;
    if (yarn) {
      const double g = fmin(1.0, fmax(0.0, (s->orig_len * w / (2 * kPi) - alpha) / (beta - alpha)));
      w = g * w + (1 - g) * w / f;
    }
    turns[i] = (uint64_t)nearbyint(ldexp(w / (2 * kPi), 64));  // w <= 1: below 2^62
  }
  const double amp = s->amplitude > 0 ? s->amplitude : yarn ? 0.1 * log(f) + 1.0 : 1.0;
  *amplitude = (float)amp;
  return *amplitude > 0.f && !isinf(*amplitude) ? QSA_OK : QSA_ERR_INVALID_ARG;
}

qsa_status qsa_rope(const qsa_rope_args* rope, int32_t batch, int32_t n_tok, int32_t n_heads, int32_t head_dim,
                    int32_t inverse, const void* x, const qsa_strides* xs, const int32_t* pos, void* y,
                    const qsa_strides* ys, void* stream) {
  if (!rope || !x || !pos || !y || batch < 1 || n_tok < 1 || n_heads < 1) return QSA_ERR_INVALID_ARG;
  if (inverse != 0 && inverse != 1) return QSA_ERR_INVALID_ARG;
  if (head_dim != 64 && head_dim != 128 && head_dim != 256) return QSA_ERR_UNSUPPORTED;
  if (n_heads > QSA_MAX_KV_HEADS || (long long)batch * n_tok >= (1LL << 31)) return QSA_ERR_UNSUPPORTED;
  Rope ro;
  qsa_status st = check_rope(rope, head_dim, &ro);
  if (st != QSA_OK) return st;
  if (!aligned_all(2, {x, y}) || !aligned(pos, 4)) return QSA_ERR_INVALID_ARG;
  const Strided xi = strided(x, xs, batch, n_tok, n_heads, head_dim);
  const Strided yo = strided(y, ys, batch, n_tok, n_heads, head_dim);
  if (!writable(yo, batch, n_tok, n_heads) || !in_place_or_apart(xi, yo)) return QSA_ERR_INVALID_ARG;
  return from_cuda(launch_rope(ro, batch, n_tok, n_heads, head_dim, inverse != 0, xi, pos, yo,
                               static_cast<cudaStream_t>(stream)));
}

qsa_status qsa_kv_workspace_size(const qsa_dims* dims, size_t* bytes) {
  const qsa_status st = check_kv_dims(dims);
  if (st != QSA_OK) return st;
  if (!bytes) return QSA_ERR_INVALID_ARG;
  *bytes = dense_ws(*dims, device_sm_count()).total;
  return QSA_OK;
}

qsa_status qsa_kv_append(const qsa_dims* dims, int32_t n_tok, const qsa_rope_args* rope, const void* k,
                         const qsa_strides* ks, const void* v, const qsa_strides* vs, const void* q,
                         const qsa_strides* qs, void* q_out, const qsa_strides* qos, const int32_t* pos,
                         const int32_t* page_table, void* k_cache, void* v_cache, const float* k_scale,
                         const float* v_scale, void* ws, size_t ws_bytes, void* stream) {
  qsa_status st = check_kv_dims(dims);
  if (st != QSA_OK) return st;
  if (n_tok < 1 || n_tok > QSA_MAX_CHUNK) return QSA_ERR_INVALID_ARG;
  if (!k || !v || !pos || !page_table || !k_cache || !v_cache) return QSA_ERR_INVALID_ARG;
  if ((q != nullptr) != (q_out != nullptr) || (q && !rope)) return QSA_ERR_INVALID_ARG;
  if (dims->kv_dtype == QSA_KV_FP8_E4M3 && (!k_scale || !v_scale)) return QSA_ERR_INVALID_ARG;
  if ((long long)dims->batch * n_tok >= (1LL << 31)) return QSA_ERR_UNSUPPORTED;
  Rope ro;
  if ((st = check_rope(rope, dims->head_dim, &ro)) != QSA_OK) return st;
  if (!aligned_all(16, {k_cache, v_cache}) || !aligned_all(2, {k, v, q, q_out}) ||
      !aligned_all(4, {pos, page_table, k_scale, v_scale}))
    return QSA_ERR_INVALID_ARG;
  const int B = dims->batch, D = dims->head_dim, hk = dims->n_kv_heads, hq = dims->n_q_heads;
  const Strided qo = strided(q_out, qos, B, n_tok, hq, D);
  const Strided qi = strided(q, qs, B, n_tok, hq, D);
  if (q && (!writable(qo, B, n_tok, hq) || !in_place_or_apart(qi, qo))) return QSA_ERR_INVALID_ARG;
  if (!check_header(ws, ws_bytes)) return QSA_ERR_WORKSPACE;
  return from_cuda(launch_kv_append(*dims, n_tok, ro, strided(k, ks, B, n_tok, hk, D),
                                    strided(v, vs, B, n_tok, hk, D), qi, qo, pos, page_table, k_cache, v_cache,
                                    k_scale, v_scale, static_cast<int32_t*>(ws), static_cast<cudaStream_t>(stream)));
}

qsa_status qsa_kv_gather(const qsa_dims* dims, int32_t n_tok, const void* k_cache, const void* v_cache,
                         const float* k_scale, const float* v_scale, const int32_t* page_table, const int32_t* pos,
                         void* k_out, void* v_out, void* ws, size_t ws_bytes, void* stream) {
  const qsa_status st = check_kv_dims(dims);
  if (st != QSA_OK) return st;
  if (n_tok < 1 || n_tok > QSA_MAX_CHUNK) return QSA_ERR_INVALID_ARG;
  if (!k_cache || !v_cache || !page_table || !pos || !k_out || !v_out) return QSA_ERR_INVALID_ARG;
  if (dims->kv_dtype == QSA_KV_FP8_E4M3 && (!k_scale || !v_scale)) return QSA_ERR_INVALID_ARG;
  if ((long long)dims->batch * n_tok >= (1LL << 31)) return QSA_ERR_UNSUPPORTED;
  if (!aligned_all(16, {k_cache, v_cache, k_out, v_out}) || !aligned_all(4, {pos, page_table, k_scale, v_scale}))
    return QSA_ERR_INVALID_ARG;
  if (!check_header(ws, ws_bytes)) return QSA_ERR_WORKSPACE;
  return from_cuda(launch_kv_gather(*dims, n_tok, k_cache, v_cache, k_scale, v_scale, page_table, pos, k_out, v_out,
                                    static_cast<int32_t*>(ws), static_cast<cudaStream_t>(stream)));
}

qsa_status qsa_paged_attn(const qsa_dims* dims, int32_t window, const void* q, const void* k_cache,
                          const void* v_cache, const float* k_scale, const float* v_scale,
                          const int32_t* page_table, const int32_t* q_pos, void* out, float* lse, void* ws,
                          size_t ws_bytes, void* stream) {
  return paged_attn(dims, window, q, k_cache, v_cache, k_scale, v_scale, page_table, q_pos, out, lse, ws, ws_bytes,
                    stream, false);
}

qsa_status qsa_test_paged_attn_timeout(const qsa_dims* dims, int32_t window, const void* q, const void* k_cache,
                                       const void* v_cache, const float* k_scale, const float* v_scale,
                                       const int32_t* page_table, const int32_t* q_pos, void* out, float* lse, void* ws,
                                       size_t ws_bytes, void* stream) {
  return paged_attn(dims, window, q, k_cache, v_cache, k_scale, v_scale, page_table, q_pos, out, lse, ws, ws_bytes,
                    stream, true);
}

}  // extern "C"
