/*
 * qsa_kv.h -- the operators of libqsa.so round the paged KV cache: rotary
 * positions, writing new keys and values into the pages, reading them back,
 * and dense attention over them.
 *
 * qsa.h's step reads a paged cache and attends over at most 2,051 selected
 * positions. These entry points fill that cache (qsa_kv_append: rotary
 * positions, E4M3 quantisation and the page lookup in one launch), read it
 * back (qsa_kv_gather), and attend over all of it, or over a sliding window
 * (qsa_paged_attn: short contexts, dense layers, and the result the sparse
 * step approximates). qsa_rope is the rotation alone, in both directions.
 *
 * Cache, page table, scales, positions, error record and execution rules are
 * those of qsa.h: every call is asynchronous on `stream`, allocates nothing,
 * returns argument errors before anything is launched, and records errors
 * found on the device in the workspace header for qsa_check_errors. Of
 * qsa_dims these entry points use batch, n_q_heads, n_kv_heads, head_dim,
 * page_size, max_pages, num_pages, kv_dtype and, in qsa_paged_attn, n_q and
 * sm_scale; the other fields are not looked at.
 *
 * Supported geometry: head_dim 64, 128 or 256; n_q_heads any multiple of
 * n_kv_heads (1..1024 heads); page_size a power of two in 16..256; BF16 or
 * E4M3 cache; n_q 1..4; at most 2^22 requests. Anything else returns
 * QSA_ERR_UNSUPPORTED.
 *
 * A position of -1 stands for no token (a padded batch): nothing is read,
 * written or reported for it, except that qsa_paged_attn writes its output
 * row as zeros.
 */
#ifndef QSA_KV_H_
#define QSA_KV_H_

#include "qsa.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Strides, in elements, of a tensor [batch][token][head][head_dim] whose last
 * dimension is contiguous. A NULL pointer to it means a contiguous tensor. A
 * stride of an input may be 0 (a broadcast input); the elements of an output
 * must not overlap, and one of its strides may be 0 only where its dimension
 * has one element (the stride of such a dimension is not looked at). */
typedef struct {
  int64_t batch, token, head;
} qsa_strides;

/* Which components form a pair: HALF pairs i with i + rot_dim / 2,
 * INTERLEAVED 2 i with 2 i + 1. */
typedef enum { QSA_ROPE_HALF = 0, QSA_ROPE_INTERLEAVED = 1 } qsa_rope_layout;

/* How the frequencies w_i = base^(-2 i / rot_dim) are scaled for contexts
 * longer than the ones trained on, by `factor` f >= 1:
 *   NONE    w_i
 *   LINEAR  w_i / f
 *   NTK     the frequencies of the base base * f^(rot_dim / (rot_dim - 2))
 *           (rot_dim > 2)
 *   YARN    g_i w_i + (1 - g_i) w_i / f with
 *           g_i = clamp((orig_len w_i / 2 pi - alpha) / (beta - alpha), 0, 1):
 *           pairs that turn more than beta times over the original length
 *           keep their frequency, those below alpha turns are interpolated
 *           (Peng et al., "YaRN", 2023); amplitude 0.1 ln f + 1 unless given */
typedef enum {
  QSA_ROPE_NONE = 0, QSA_ROPE_LINEAR = 1, QSA_ROPE_NTK = 2, QSA_ROPE_YARN = 3
} qsa_rope_scaling;

typedef struct {
  int32_t rot_dim; /* rotated components, even, 2..256: the first of each head */
  int32_t layout;  /* qsa_rope_layout */
  int32_t scaling; /* qsa_rope_scaling */
  double base;     /* > 1 (0 selects 10,000) */
  double factor;   /* f >= 1 (0 selects 1); not looked at for NONE */
  double orig_len; /* YARN: the original context length, >= 1 */
  double alpha;    /* YARN: 0 <= alpha < beta (both 0 selects 1 and 32) */
  double beta;
  double amplitude; /* factor of cos and sin; 0 selects the scaling's own
                     * (1, or YARN's), else > 0 */
} qsa_rope_spec;

/* Host function: fills turns[0 .. rot_dim / 2) (host memory) with each pair's
 * frequency in turns per position, w_i / 2 pi, as a 64-bit binary fraction
 * (times 2^64, modulo 2^64), and *amplitude. A position times such an entry,
 * in 64-bit integer arithmetic, is the rotation's angle as a fraction of a
 * turn, with whole turns dropped exactly: angles of far positions lose
 * nothing. The caller copies the table to the device once. */
qsa_status qsa_rope_table(const qsa_rope_spec* spec, uint64_t* turns, float* amplitude);

/* A rotation as the kernels take it. */
typedef struct {
  int32_t rot_dim; /* as in the spec; at most head_dim */
  int32_t layout;
  float amplitude;       /* qsa_rope_table's */
  const uint64_t* turns; /* device copy of qsa_rope_table's table */
} qsa_rope_args;

/* Most heads in one call of the entry points below. */
#define QSA_MAX_KV_HEADS 1024

/* Rotary positions. For request r, token j at position t = pos[r][j] >= 0,
 * every head of x and pair (a, b) at angle t w_i (times -1 with inverse):
 *   y_a = A (x_a cos - x_b sin),  y_b = A (x_b cos + x_a sin);
 * components from rot_dim on are copied. With inverse = 1 the call is the
 * gradient of the one with inverse = 0 (the transpose of its matrix, with the
 * same amplitude; for A = 1 also its inverse). FP32 arithmetic, one rounding
 * to BF16. Tokens with pos < 0 are left as they are in y. x is bf16
 * [batch][n_tok][n_heads][head_dim] with strides xs, y the same with ys; y
 * may be x with the same strides, else it must not overlap it. pos is int32
 * [batch][n_tok]. batch, n_tok, n_heads >= 1, n_heads <= QSA_MAX_KV_HEADS. */
qsa_status qsa_rope(const qsa_rope_args* rope, int32_t batch, int32_t n_tok, int32_t n_heads, int32_t head_dim,
                    int32_t inverse, const void* x, const qsa_strides* xs, const int32_t* pos, void* y,
                    const qsa_strides* ys, void* stream);

/* Bytes of workspace for the entry points below (n_q as in qsa_paged_attn).
 * It starts with qsa.h's error record; qsa_workspace_init zeroes it once. A
 * workspace may be shared with qsa.h's entry points called with the same
 * dims, if it has the larger of the two sizes. */
qsa_status qsa_kv_workspace_size(const qsa_dims* dims, size_t* bytes);

/* New keys and values into the cache. Token j of request r, at position
 * t = pos[r][j], is written to page page_table[r][t / page_size], slot
 * t % page_size, for every KV head g: K after the rotation (rope NULL: none),
 * V as it is. BF16 cache: one rounding of the rotated key. E4M3 cache:
 * code = x / scale[g], rounded to nearest even and clamped to +-448 (NaN
 * stays NaN). With q, the queries of the same tokens (n_q_heads of them) are
 * rotated into q_out; q needs a rope.
 *
 * The tokens of a request are consecutive: pos[r][j] is pos[r][0] + j, or -1
 * for no token (a padded batch has its padding behind the tokens, not in front
 * of them). One that is neither is reported (kind 6), one past the page
 * table is reported (kind 1), and both are skipped, their q_out row too. A
 * page id outside the cache is reported (kind 2) and the token's K and V are
 * not written. Requests must not share a page that the call writes to.
 *
 * k, v: bf16 [batch][n_tok][n_kv_heads][head_dim] (strides ks, vs); q, q_out:
 * bf16 [batch][n_tok][n_q_heads][head_dim] (strides qs, qos); q_out may be q
 * with the same strides, else it must not overlap an input. k_scale and
 * v_scale are read only for E4M3. ws needs 256 bytes (its header). n_tok is
 * 1..QSA_MAX_CHUNK. */
qsa_status qsa_kv_append(const qsa_dims* dims, int32_t n_tok, const qsa_rope_args* rope, const void* k,
                         const qsa_strides* ks, const void* v, const qsa_strides* vs, const void* q,
                         const qsa_strides* qs, void* q_out, const qsa_strides* qos, const int32_t* pos,
                         const int32_t* page_table, void* k_cache, void* v_cache, const float* k_scale,
                         const float* v_scale, void* ws, size_t ws_bytes, void* stream);

/* Reads cache rows back: k_out[r][j] and v_out[r][j] (bf16, contiguous
 * [batch][n_tok][n_kv_heads][head_dim]) = the values at position pos[r][j] of
 * request r, code * scale[g] rounded to BF16 for an E4M3 cache. Positions may
 * come in any order and repeat; a row whose position is -1 is left as it is,
 * and so is one that is reported: a position below -1 or past the page table
 * (kind 1), a page id outside the cache (kind 2). ws needs 256 bytes. n_tok
 * is 1..QSA_MAX_CHUNK. */
qsa_status qsa_kv_gather(const qsa_dims* dims, int32_t n_tok, const void* k_cache, const void* v_cache,
                         const float* k_scale, const float* v_scale, const int32_t* page_table, const int32_t* pos,
                         void* k_out, void* v_out, void* ws, size_t ws_bytes, void* stream);

/* Dense attention over the paged cache (decode and verify). For request r,
 * query j at p = q_pos[r][j] and query head h with KV head
 * g = h / (n_q_heads / n_kv_heads): out = softmax(sm_scale * q K^T) V over the
 * positions max(0, p - window + 1) .. p (window 0: 0 .. p), and
 * lse[r][j][h] = ln(sum of exp) of those scores where lse is not NULL (fp32
 * [batch][n_q][n_q_heads]). K and V outside a query's positions never reach
 * its output, whatever they hold. A row without positions (p = -1, or p below
 * -1 or past the page table, which is reported as kind 1) gives zeros and an
 * lse of -infinity, as does a row whose scores are all -infinity. A page id
 * outside the cache is reported (kind 2) and its positions are left out. The
 * cache's positions are split over the GPU and the pieces joined in a fixed
 * order: the same call gives the same bits. q and out are contiguous, as for
 * qsa_sparse_attn.
 *
 * FP32 softmax statistics and accumulation, BF16 out. The sums before the
 * division by the softmax's have weights up to 2^8: values of 2^(119 - log2 of
 * the positions) or more may overflow in them. What has fewer bits:
 *  - the weights of the second product (not those in the softmax's sum), each
 *    off by at most 2^-8 of itself. With an E4M3 cache that holds from 2^-12 of
 *    a row's largest weight on; smaller ones are off by less than 2^-20 of it,
 *    as often up as down, so that a long tail of them keeps its sum: what it
 *    adds to the output's error has a standard deviation of at most 2^-11 of
 *    the largest |V|, at any length;
 *  - with an E4M3 cache, the queries: a component is off by at most 2^-22 of
 *    its head's largest. */
qsa_status qsa_paged_attn(const qsa_dims* dims, int32_t window, const void* q, const void* k_cache,
                          const void* v_cache, const float* k_scale, const float* v_scale,
                          const int32_t* page_table, const int32_t* q_pos, void* out, float* lse, void* ws,
                          size_t ws_bytes, void* stream);

/* Test hook for failure detection: qsa_paged_attn with copies of K that bring
 * half of the bytes its kernel waits for. Every CTA's bounded wait runs out
 * (about a second), the kernel stops, frees what it holds and records a timeout
 * (kind 5, QSA_ERR_TIMEOUT); out and lse hold nothing of meaning. The next call
 * on the same workspace is complete again. */
qsa_status qsa_test_paged_attn_timeout(const qsa_dims* dims, int32_t window, const void* q, const void* k_cache,
                                       const void* v_cache, const float* k_scale, const float* v_scale,
                                       const int32_t* page_table, const int32_t* q_pos, void* out, float* lse,
                                       void* ws, size_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* QSA_KV_H_ */
