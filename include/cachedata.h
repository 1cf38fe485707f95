/*
 * cachedata.h -- what the pages of a paged cache hold, part of libdescbuild.so
 * (CUDA, sm_103a): keys and values written to their slots and read back, as
 * they are or as 8-bit codes; attention of drafted tokens over the cache; the
 * verification of the drafts; and the accepted tokens moved together.
 *
 * Beside pagecache.h, whose tables say which pages hold a sequence's tokens.
 * A speculative step is
 *   db_page_extend   room for the drafted tokens (db_page_copy: its copies)
 *   db_cache_write   their keys and values, layer by layer
 *   db_cache_attention   what they see, layer by layer
 *   db_draft_verify  which of them stay, and one more token
 *   db_cache_keep    the kept ones move behind the tokens before the step
 *   db_page_free     the others' slots go back (the cuts of db_cache_keep)
 * with no host round trip between the calls.
 *
 * Conventions are those of descbuild.h and pagecache.h: device pointers owned
 * by the caller, asynchronous on `stream`, negative errno returns for bad
 * arguments, data-dependent results in per-request status and db_counters.
 * Structs of this header are HOST structs, read during the call only. Nothing
 * but what a call names as its output is written.
 *
 * A batch (db_cache_batch) names sequences and the rows that come with them:
 * rows start[i] to start[i+1] of the arrays beside it belong to request i.
 * start ascends; rows before start[0] and from start[n] on are neither read
 * nor written. In calls on new tokens (write, attention, keep) a request's m
 * rows are the sequence's last m tokens, positions length - m to length - 1,
 * as db_page_extend has made room for them. A request is DB_PAGE_INVALID, and
 * does nothing, when
 *   - its seq is not below n_seqs, its sequence has more tokens than a row of
 *     the table has places for, or 2^31,
 *   - start[i] > start[i+1] or start[i+1] > rows, or
 *   - (new tokens) it has more rows than the sequence tokens.
 * Every other request is done by itself, whatever is wrong beside it; where
 * start does not ascend and valid requests share rows, each reads them, and
 * what several write is any one's (write and read take longer then: they look
 * for a row's request by its place among the starts first).
 * No sequence may be named twice where a call writes to the cache: what two
 * requests both write is then either's (nothing else is touched).
 *
 * status  NULL or [n] out: DB_PAGE_OK or DB_PAGE_INVALID
 * ctr     NULL or counters: total = rows of valid requests, n_invalid =
 *         invalid requests, err = DB_ERR_PAGE_TABLE where a valid request met
 *         a table entry outside [0, n_pages). Such an entry's tokens are not
 *         written, read as zeros, and seen by nobody.
 *
 * Limits: width a multiple of 16, 16 to 256; heads and page_tokens from 1,
 * their product times width below 2^31; pools and rows start on multiples of
 * 16 bytes and have strides that are multiples of 16 bytes; scales, indexes
 * and other 32-bit arrays on multiples of 4, counters of 8.
 */
#ifndef CACHEDATA_H
#define CACHEDATA_H

#include <stddef.h>
#include <stdint.h>

#include "pagecache.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Types of cached values and of rows outside the cache. */
#define DB_BF16 0u
#define DB_F16 1u
#define DB_F32 2u  /* rows and probabilities only */
#define DB_E4M3 3u /* cached values only: 4 exponent and 3 mantissa bits, no infinities */
#define DB_I8 4u   /* cached values only: -127 to 127 */

typedef struct db_cache_batch {
  const int32_t* seq;   /* [n] */
  const int32_t* start; /* [n + 1] */
  uint32_t n;
  uint32_t rows;        /* of the arrays that come with the batch */
} db_cache_batch;

/* The keys and the values of one layer: page p of the keys starts at
 * k + p*k_stride (bytes) and holds heads * page_tokens rows of `width` values
 * without gaps, [token][head] or (heads_first) [head][token]. The 8-bit types
 * have a scale for each row, page p's at k_scale + p*k_scale_stride (bytes) in
 * the same order; a row's values are its codes times its scale. */
typedef struct db_cache_layer {
  void* k;
  void* v;
  float* k_scale; /* NULL for 16-bit types */
  float* v_scale;
  uint64_t k_stride;
  uint64_t v_stride;
  uint64_t k_scale_stride;
  uint64_t v_scale_stride;
  uint32_t heads;
  uint32_t width;
  uint32_t type; /* DB_BF16, DB_F16, DB_E4M3 or DB_I8 */
  uint32_t heads_first;
} db_cache_layer;

/* Rows outside the cache: head h of row r is `width` neighbouring values at
 * base + r*row_stride + h*head_stride (bytes). */
typedef struct db_cache_rows {
  void* base;
  uint64_t row_stride;
  uint64_t head_stride;
} db_cache_rows;

/* New tokens' keys and values go to their slots. `type` is that of the rows
 * (DB_BF16, DB_F16, DB_F32); 16-bit caches hold them rounded to nearest even.
 * 8-bit ones hold, for each row, with a its largest magnitude and L = 448
 * (E4M3) or 127 (I8): scale = a / L, codes = x * (L / a) rounded to nearest
 * even, in 32-bit floating point (a = 0, or so small that a / L is 0 or L / a
 * infinite: scale and codes 0). A row with an infinity or a NaN gets the scale
 * NaN and codes 0: all of it reads back as NaN. */
int db_cache_write(const db_page_tables* t, const db_cache_batch* b, const db_cache_layer* c,
                   const db_cache_rows* k, const db_cache_rows* v, uint32_t type, uint8_t* status,
                   db_counters* ctr, void* stream);

/* Tokens come back: row start[i] + j of request i gets position first[i] + j
 * of its sequence (first NULL: position j) in type `type` (DB_BF16, DB_F16,
 * DB_F32; products in 32 bits, rounded once). Rows past the sequence's last
 * token are zeros. first[] is read as u32. */
int db_cache_read(const db_page_tables* t, const db_cache_batch* b, const int32_t* first,
                  const db_cache_layer* c, const db_cache_rows* k, const db_cache_rows* v,
                  uint32_t type, uint8_t* status, db_counters* ctr, void* stream);

/* Attention of each request's m tokens, its last, over its sequence's cache.
 * Query head x attends with key head x / (q_heads / heads). Node j of a
 * request (row start[i] + j) sees all tokens before the request's, and of the
 * request's own
 *   mask NULL: nodes 0 to j (a chain, or a single token)
 *   mask: the nodes whose bit is set: bit (b % 32) of
 *         mask[(start[i] + j) * mask_words + b / 32] for node b.
 * With s the scaled products of the query with the keys that it sees, out =
 * sum exp(s) v / sum exp(s) and lse (NULL or [rows][q_heads]) = log sum
 * exp(s). A row that sees nothing (or only scores of -infinity) has out 0 and
 * lse -infinity. What a row does not see does not reach it, whatever the
 * slots hold (infinities and NaN included).
 * `type` is that of q and out, DB_BF16 or DB_F16; 16-bit caches are of the
 * same type. Statistics and sums are held in 32 bits. Weights are rounded to
 * `type`, or held finer, for the product with 16-bit values; with codes
 * weights times scales are rounded to f16 or held finer, each off by 2^-11 of
 * itself or by 2^-29 of the largest among the tokens that the row sees,
 * whichever is more (where scales below 2^-80, 0 too, count as that), and bf16
 * queries are taken as f16 times a power of two that is each row's own (off by
 * 2^-38 of the row's largest value at most).
 * Sums of weights times values have to stay within 32 bits' range: values up
 * to 2^100 do, and those of codes above 2^-90 keep their precision.
 *   max_tokens  no request has more rows (one that has is DB_PAGE_INVALID);
 *               with a mask at most 32 * mask_words. It chooses the kernel for
 *               all requests of the call: single tokens go faster in a call of
 *               their own than beside requests of many
 *   ws          of db_cache_attention_workspace_size bytes for these heads,
 *               width and max_tokens (or larger ones of the same heads and
 *               width); the size is that of the current device. Zeros at
 *               first, and left ready for the next call; calls that may run at
 *               the same time (on two streams, in two graphs) need one each.
 *               After DB_ERR_TIMEOUT in ctr (a kernel gave up waiting, out is not
 *               valid, and status is DB_PAGE_INVALID for all requests) it has to
 *               be zeros again.
 * q may be out. n <= 65536, q_heads a multiple of heads and at most 64 of
 * them to a key head. */
int db_cache_attention_workspace_size(uint32_t n, uint32_t q_heads, uint32_t heads, uint32_t width,
                                      uint32_t max_tokens, size_t* bytes);
int db_cache_attention(const db_page_tables* t, const db_cache_batch* b, const db_cache_layer* c,
                       const db_cache_rows* q, const db_cache_rows* out, uint32_t type,
                       uint32_t q_heads, uint32_t max_tokens, float scale, const uint32_t* mask,
                       uint32_t mask_words, float* lse, uint8_t* status, db_counters* ctr, void* ws,
                       size_t ws_bytes, void* stream);

/* Drafted tokens against the target's probabilities. The m nodes of request i
 * (rows start[i] on, of which node 0 is the root: the last token that is
 * certain) form a tree: parent[r] is the node that row r's token follows,
 * below its own (the root's is not read). p [rows][vocab] are the target's
 * probabilities after each node, q (NULL or [rows][vocab]) the drafter's, from
 * which a node's children were drawn one by one, each from all tokens.
 * The walk starts at the root. At node j, with w = p_j and W = 1, its children
 * are tried in ascending order: child c with token t is accepted when
 * u[c] * q_j(t) * W < w(t), and the walk goes on from it. Otherwise w becomes
 * max(w / W - q_j, 0) and W its sum. Without q a child stands for itself alone
 * (q_j is 1 at t): w(t) becomes 0 and W loses it. When no child is left, the
 * next token is the first t whose w(0) + ... + w(t) exceeds u[root] times the
 * sum of all (w = p_j where that sum is 0). So each token is distributed as
 * the target's, u being uniform on [0, 1).
 *   parent, token  i32 [rows]; token from 0 to vocab - 1 (the root's is not read)
 *   u        f32 [rows], 0 <= u < 1
 *   path     out i32 [rows]: the accepted nodes, ascending, from start[i] on
 *            (the root, 0, is the first), then -1
 *   accepted out i32 [n]: how many (the root included)
 *   next     out i32 [n]
 * type is that of p and q (DB_BF16, DB_F16, DB_F32), p_stride and q_stride
 * elements from row to row. Probabilities are from 0 to 1; others (NaN too)
 * count as 0 when below 0 or NaN, as 1 above. Sums are exact sums of weights
 * rounded to multiples of 2^-44, so they depend on no order; w / W - q is
 * computed in 32 bits, the test of a child in 64.
 * DB_PAGE_INVALID: no rows or more than 1024, start as in a batch, a node's
 * parent not below it or its token outside. Then accepted = 0, next = -1, and
 * the rows' path -1 (unless start is what is wrong). A step goes on with that:
 * db_cache_keep keeps none of the request's tokens and cuts to base, so that
 * db_page_free leaves the sequence as it was before the step's db_page_extend,
 * the root not in it; the step can be taken again. next is -1 as well where
 * all of p_j is 0. vocab <= 2^19. */
int db_draft_verify(const int32_t* start, uint32_t n, uint32_t rows, const int32_t* parent,
                    const int32_t* token, const void* p, uint64_t p_stride, const void* q,
                    uint64_t q_stride, uint32_t type, uint32_t vocab, const float* u, int32_t* path,
                    int32_t* accepted, int32_t* next, uint8_t* status, db_counters* ctr,
                    void* stream);

/* The accepted tokens move together: with base = length - m, the token at
 * position base + path[start[i] + k] goes to base + k, for k < accepted[i], in
 * every plane of the pool (one call for the codes, one for their scales).
 * Other slots keep what they hold, lengths are not changed.
 *   cut  NULL or [n] out (8-byte aligned): {seq, base + accepted[i]}, requests
 *        of db_page_free; of an invalid request {seq, 0xFFFFFFFF}, which keeps
 *        everything
 * DB_PAGE_INVALID also: accepted[i] > m (read as u32), or the path not
 * ascending below m. Pool and shape as in db_page_copy, page_tokens that of
 * t. */
int db_cache_keep(const db_page_tables* t, const db_cache_batch* b, const int32_t* path,
                  const int32_t* accepted, const db_page_pool* pool, const db_page_shape* shape,
                  db_page_cut* cut, uint8_t* status, db_counters* ctr, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* CACHEDATA_H */
