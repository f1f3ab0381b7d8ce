/*
 * qsa_serve.h -- the operators of libqsa.so for serving a batch in a bounded
 * cache: dense attention of requests that share a long prefix, the attention
 * weight that each cached position gets, eviction of the positions with the
 * least of it, and verification of drafted tokens.
 *
 * A serving loop over qsa_kv.h's cache uses them together: requests branched
 * from one context attend with qsa_prefix_attn (which also gives their lse),
 * qsa_verify_drafts turns the target's probabilities of the verified tokens
 * into the tokens that stay, qsa_kv_weight keeps account of which positions
 * are attended to (by the tokens that stay: see there), and qsa_kv_evict brings
 * a request that has grown too long back to its bound (how its later tokens are
 * rotated: see there).
 *
 * Cache, page table, scales, positions, error record and execution rules are
 * those of qsa.h and qsa_kv.h, the fields of qsa_dims that are looked at and
 * the supported geometry those of qsa_kv.h. Errors found on the device go to
 * the workspace header (qsa_check_errors): kinds as in qsa.h, and
 *   7  a drafted token outside the vocabulary (request, draft, token),
 *   8  a request's length outside its page table (request, 0, length),
 *   9  weights to sample from that sum to 16 or more (request, row, 0).
 */
#ifndef QSA_SERVE_H_
#define QSA_SERVE_H_

#include "qsa_kv.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Bytes of workspace for qsa_prefix_attn with these dims and this many shared
 * pages (at least qsa_kv_workspace_size's, so that qsa_kv.h's entry points can
 * be called on the same one; enough for fewer shared pages too). Where a long
 * prefix is read in parts there is room for the pieces of three waves of them: 3
 * to 6 pieces of 128 query rows an SM, head_dim + 2 floats a row (30 to 60 MB
 * with head dim 128, more with the batch from about 250 requests x 4 queries over
 * 8 KV heads on). A call mostly fills a third of it. */
qsa_status qsa_prefix_workspace_size(const qsa_dims* dims, int32_t prefix_pages, size_t* bytes);

/* Dense attention of a batch that shares a prefix: qsa_paged_attn (window 0)
 * where the first prefix_pages * page_size positions of every request live in
 * the pages prefix_table[0 .. prefix_pages) and the others, as there, in the
 * pages that the request's page_table row names. A row's first prefix_pages
 * entries are not looked at (a table that names the shared pages there too is
 * fine). prefix_pages is 0..max_pages; with 0 the call is qsa_paged_attn.
 *
 * The shared positions are read once for all requests, whose query rows are
 * worked on together, and each request's own positions once for the request;
 * a request one of whose queries does not see the whole prefix is worked on by
 * itself, and so are all of them where the prefix's bytes are few. The pieces
 * are joined in a fixed order: the same call gives the same bits. Out, lse,
 * empty rows and errors are as for qsa_paged_attn; a page id of the prefix
 * outside the cache is reported (kind 2) for request -1.
 *
 * FP32 softmax statistics and accumulation, BF16 out. What has fewer bits over
 * a request's own positions (and over the prefix, where it is read alone) is
 * said at qsa_paged_attn. Over a prefix read once, the weights of the second
 * product (not those in the softmax's sum) are BF16 (off by at most 2^-8 of
 * themselves) with a BF16 cache and FP16 (2^-11 of themselves, or 2^-31 of the
 * largest weight so far) with an E4M3 cache, whose queries are FP16 then too,
 * scaled by a power of two: a component is off by at most 2^-39 of its head's
 * largest. The sums before the division by the softmax's have weights up to
 * 2^24 (BF16) or 2^15 there: values of 2^(103 - log2 of the positions) or more
 * may overflow in them. */
qsa_status qsa_prefix_attn(const qsa_dims* dims, int32_t prefix_pages, const int32_t* prefix_table, const void* q,
                           const void* k_cache, const void* v_cache, const float* k_scale, const float* v_scale,
                           const int32_t* page_table, const int32_t* q_pos, void* out, float* lse, void* ws,
                           size_t ws_bytes, void* stream);

/* Test hook: qsa_prefix_attn with the choice made for it that it makes by the
 * prefix's bytes: alone 0, the prefix is read once for all requests; 1, each
 * request reads it by itself (what it does for small ones). */
qsa_status qsa_test_prefix_attn(const qsa_dims* dims, int32_t alone, int32_t prefix_pages, const int32_t* prefix_table,
                                const void* q, const void* k_cache, const void* v_cache, const float* k_scale,
                                const float* v_scale, const int32_t* page_table, const int32_t* q_pos, void* out,
                                float* lse, void* ws, size_t ws_bytes, void* stream);

/* Test hook for failure detection: qsa_prefix_attn with the prefix read once (at
 * least one page) and copies of its K that bring half of the bytes its kernel
 * waits for, as qsa_test_paged_attn_timeout (kind 5, QSA_ERR_TIMEOUT). */
qsa_status qsa_test_prefix_attn_timeout(const qsa_dims* dims, int32_t prefix_pages, const int32_t* prefix_table,
                                        const void* q, const void* k_cache, const void* v_cache, const float* k_scale,
                                        const float* v_scale, const int32_t* page_table, const int32_t* q_pos,
                                        void* out, float* lse, void* ws, size_t ws_bytes, void* stream);

/* The attention weight that each cached position gets from the newest tokens:
 *   weight[r][t] = decay * weight[r][t]
 *                + sum over j with t <= q_pos[r][j], and over query heads h, of
 *                  exp(sm_scale q[r][j][h] . k[r][t][g] - lse[r][j][h])
 * with g = h / (n_q_heads / n_kv_heads), for the positions t that at least one
 * query of the request sees (t <= max_j q_pos[r][j]); the others are left as
 * they are. q, k_cache, k_scale, page_table and q_pos are those of the call of
 * qsa_paged_attn (window 0) or qsa_prefix_attn that gave lse (fp32
 * [batch][n_q][n_q_heads]); the prefix's pages have to be in page_table here.
 * weight is fp32 [batch][max_pages * page_size]. decay is in 0..1; with 0 what
 * weight holds is not read. A row whose lse is -infinity, or whose position is
 * -1 (or outside the page table: reported, kind 1), adds nothing. A position
 * whose page id is outside the cache is reported (kind 2) and gets no new
 * weight. Called behind qsa_verify_drafts, with a q_pos of -1 for the drafts that
 * were not accepted, it leaves them out, and their places' weights as they were:
 * a later token takes what weight holds at its place, so that has to be 0 where
 * no token is (weight starts as zeros; an eviction leaves 0). FP32 scores, exponentials and sums, added in a fixed order (the same
 * call gives the same bits); with an E4M3 cache a component of q is off by at
 * most 2^-22 of its head's largest. ws needs 256 bytes (its header). */
qsa_status qsa_kv_weight(const qsa_dims* dims, float decay, const void* q, const void* k_cache, const float* k_scale,
                         const int32_t* page_table, const int32_t* q_pos, const float* lse, float* weight, void* ws,
                         size_t ws_bytes, void* stream);

/* Test hook for failure detection: qsa_kv_weight with copies of K that bring
 * half of the bytes its kernel waits for, as qsa_test_paged_attn_timeout (kind
 * 5, QSA_ERR_TIMEOUT). weight holds nothing of meaning where a query sees it;
 * the next call on the same workspace is complete again. */
qsa_status qsa_test_kv_weight_timeout(const qsa_dims* dims, float decay, const void* q, const void* k_cache,
                                      const float* k_scale, const int32_t* page_table, const int32_t* q_pos,
                                      const float* lse, float* weight, void* ws, size_t ws_bytes, void* stream);

/* Eviction: of the len[r] tokens that request r has cached (positions 0 ..
 * len[r] - 1), at most `keep` stay: the first `sinks`, the last `recent`, and
 * of those between the ones with the largest weight[r][t], the lower position
 * first where they are equal (-0 equals 0; NaN is the least). Those that stay,
 * in their order, become the positions 0 .. new_len[r] - 1, new_len[r] =
 * min(len[r], keep):
 *   kept[r][i]       = the old position of the token now at i, -1 from new_len on
 *   weight_out[r][i] = weight[r][kept[r][i]], 0 from new_len on
 * and K and V of every KV head are copied, bit for bit, to the pages that
 * page_table_out[r] (out_pages entries a row) names for positions 0 ..
 * new_len - 1. A token whose new place is its old one is not copied, so a page
 * of both tables at the same index whose positions all stay where they are (a
 * shared prefix below `sinks`) may be in both; every other page that the call
 * writes to must not be read by it or written for another request.
 *
 * Keys stay as they were rotated, at the tokens' true positions, which from here
 * on are no longer their places (the caller keeps the number of tokens that a
 * request has had). So the tokens that follow are rotated and placed apart:
 * qsa_rope of their queries and keys at the true positions, then qsa_kv_append
 * without a rope at new_len and on (a rotated key is rounded to BF16 on the way,
 * in front of an E4M3 code too), then attention and weights with these places as
 * q_pos. qsa_kv_append's own rotation is at the place, which is wrong here, and
 * nothing can report it.
 *
 * K, V and weights move, and nothing else: the call is for the dense attention
 * (qsa_paged_attn, qsa_prefix_attn). qsa.h's sparse step chooses through a
 * compressed key of each 4 neighbouring positions, held beside the cache or in
 * its pages, and 4 places that are neighbours now were other blocks before. A
 * caller who wants that step on an evicted request puts the tokens' index keys
 * into their new order by `kept` and compresses all of them anew
 * (qsa_compress_keys or _paged, block_lo NULL); a block is then 4 tokens that
 * have become neighbours.
 *
 * keep is 1..out_pages * page_size, sinks and recent at least 0 with sinks +
 * recent <= keep. weight is fp32 [batch][max_pages * page_size], weight_out
 * fp32 [batch][out_pages * page_size] (they must not overlap), kept int32
 * [batch][keep], new_len int32 [batch] (it may be len); no other output may
 * overlap an input. A length below 0 or past the page table is reported (kind
 * 8) and taken as 0, a page id outside the cache is reported (kind 2) and its
 * tokens are not copied. ws needs 256 bytes (its header). */
qsa_status qsa_kv_evict(const qsa_dims* dims, int32_t keep, int32_t sinks, int32_t recent, int32_t out_pages,
                        const int32_t* len, const float* weight, const int32_t* page_table,
                        const int32_t* page_table_out, void* k_cache, void* v_cache, float* weight_out, int32_t* kept,
                        int32_t* new_len, void* ws, size_t ws_bytes, void* stream);

typedef enum { QSA_PROB_F32 = 0, QSA_PROB_BF16 = 1 } qsa_prob_dtype;

/* Most drafts of a request and largest vocabulary of qsa_verify_drafts. */
#define QSA_MAX_DRAFTS 31
#define QSA_MAX_VOCAB (1 << 24)

/* Strides, in elements, of probabilities [batch][row][vocab] whose last
 * dimension is contiguous; may be 0 (broadcast). NULL: a contiguous tensor. */
typedef struct {
  int64_t batch, row;
} qsa_prob_strides;

/* Verification of drafted tokens (speculative sampling). Request r has drafted
 * x[j] = tokens[r][j], j < n_draft; a token of -1 ends its drafts. With the
 * target's probabilities p_j = target[r][j] (row j is the distribution behind
 * draft j - 1; n_draft + 1 rows), those the drafts were sampled from, q_j =
 * draft[r][j] (n_draft rows), and given random numbers u[r][0 .. n_draft] in
 * [0, 1):
 *   draft j is accepted while  u[j] q_j(x[j]) < p_j(x[j]);
 *   with m the number accepted, the next token y is sampled with u[n_draft]
 *     from max(p_m - q_m, 0) where draft m was rejected, and from p_m where
 *     there was none left (or where that difference, rounded as below, is 0
 *     everywhere);
 *   sampled: the lowest y with  u[n_draft] sum_v w(v) < sum_{v <= y} w(v).
 * draft NULL: the drafts were not sampled; q_j is 1 at x[j] and 0 elsewhere.
 * Writes accepted[r] = m and out_tokens[r] = x[0 .. m - 1], y, then -1
 * (n_draft + 1 entries). The distribution so sampled is the target's.
 *
 * The test is exact. For the sampling every probability is rounded to a multiple
 * of 2^-54; the sums of those are exact, so that the result does not depend on an
 * order and is the formula's for probabilities so rounded. Against the ones given
 * a weight is off by at most 2^-54, and all of them together by vocab times that
 * (2^-36 with 150,001 tokens): where the weights sum to S, what is sampled is off
 * by at most vocab 2^-54 / S. A token whose p - q is less than 2^-54 may have no
 * weight, a row of nothing but values of 2^-55 or less none at all. A
 * probability that is negative or NaN counts as 0, one above 1 as 1; a row's
 * need not sum to 1, but weights to sample from that sum to 16 or more are
 * reported (kind 9), and y is -1. A u below 0 or NaN counts as 0, one of 1 or
 * more as the largest below 1. Where p_m so rounded is 0 everywhere, y is -1.
 *
 * A token outside 0..vocab - 1 other than -1 ends the drafts too; it is
 * reported (kind 7), but for -2 as a request's first token, which stands for
 * no request (a padded batch): accepted[r] = 0, out_tokens[r] = -1 everywhere.
 * Of target and draft, only the rows of a request's drafts up to their end, and
 * target's one behind them, are read: a request that is none needs no rows. Its
 * other tokens and random numbers have no effect.
 *
 * target and draft are fp32 or bf16 (prob_dtype), tokens int32
 * [batch][n_draft], uniform fp32 [batch][n_draft + 1], accepted int32 [batch],
 * out_tokens int32 [batch][n_draft + 1], neither of which may overlap an input.
 * n_draft is 1..QSA_MAX_DRAFTS, vocab 1..QSA_MAX_VOCAB, batch 1..2^22. ws needs
 * 256 bytes (its header): any workspace of the library. */
qsa_status qsa_verify_drafts(int32_t batch, int32_t n_draft, int32_t vocab, int32_t prob_dtype, const void* target,
                             const qsa_prob_strides* target_strides, const void* draft,
                             const qsa_prob_strides* draft_strides, const int32_t* tokens, const float* uniform,
                             int32_t* accepted, int32_t* out_tokens, void* ws, size_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* QSA_SERVE_H_ */
