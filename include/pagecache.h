/*
 * pagecache.h -- a paged cache in the device heap, part of libdescbuild.so
 * (CUDA, sm_103a): batched extension, forking, freeing and compaction of
 * sequences held in pages, and the copies of pages these ask for.
 *
 * A model's key/value cache lives in fixed-size pages of the device heap; the
 * ranges that db_prp_build reads or writes and that db_wqe_bucket puts to a
 * peer are such pages. The calls here keep the page tables on the device, in
 * stream order with the kernels that read them, with no host round trip
 * between them. No call makes the requests of db_prp_build or db_wqe_bucket
 * from a row or from a list of moves: that is the caller's to do, on the
 * device or by way of the host.
 *
 * Conventions are those of descbuild.h: device pointers owned by the caller,
 * asynchronous on `stream`, negative errno returns for bad arguments,
 * data-dependent results in per-request status and db_counters, n == 0 only
 * zeroes the counters, a zero-filled workspace that every call leaves ready
 * for the next. db_page_tables and db_page_pool are HOST structs of device
 * pointers, read during the call only.
 *
 * The state of a cache of n_seqs sequences and n_pages pages, both below
 * 2^31 (no size may be 0; the free words start on a multiple of 16 bytes, the
 * other arrays of 4):
 *   table  i32 [n_seqs][columns]: page of tokens [c*T, (c+1)*T) of the
 *          sequence, T = page_tokens; DB_PAGE_NONE past its last page
 *   length u32 [n_seqs]: tokens held; the first ceil(length/T) columns of the
 *          row are pages, each named once in a row
 *   refs   u32 [n_pages]: the rows that name the page
 *   free   u32 [ceil(n_pages/32)]: bit p%32 of word p/32 set <=> refs[p] == 0
 *          (bits past n_pages are ignored and written 0)
 * An empty cache has table all DB_PAGE_NONE, length and refs 0, free bits 1.
 *
 * Which pages a call takes depends on the set of free pages alone: the lowest
 * free index first. So results do not depend on the order in which pages
 * were freed, pages freed together come back as the same runs of
 * neighbours, and the cache keeps to the low end of its region.
 *
 * In a batch, the first request that names a sequence (a fork: a child) is
 * the one that counts; later ones naming it are DB_PAGE_INVALID.
 *
 * A row that names a page outside [0, n_pages), or a page with fewer
 * references than rows, is not a state these calls leave. The entry of a page
 * outside is skipped, and DB_ERR_PAGE_TABLE is set in ctr->err; a row that
 * frees a page without references, when it looks, is reported so too, while
 * rows of one batch that look together and then drop more references than
 * there are go unreported. Nothing outside the arrays is read or written in
 * either case; the cache's contents are then undefined.
 */
#ifndef PAGECACHE_H
#define PAGECACHE_H

#include <stddef.h>
#include <stdint.h>

#include "descbuild.h"

#ifdef __cplusplus
extern "C" {
#endif

#define DB_PAGE_NONE (-1)
#define DB_PAGE_ALL 0xFFFFFFFFu /* db_page_move::tokens: the whole page */

#define DB_PAGE_OK 0
#define DB_PAGE_INVALID 1 /* the request is malformed and did nothing              */
#define DB_PAGE_SHORT 2   /* db_page_extend: too few free pages; the batch did nothing */

#define DB_ERR_PAGE_TABLE 8u /* a row names a page that does not exist or is free */

typedef struct db_page_tables {
  int32_t* table;
  uint32_t* length;
  uint32_t* refs;
  uint32_t* free;
  uint32_t n_seqs;
  uint32_t columns;     /* entries of a row */
  uint32_t n_pages;
  uint32_t page_tokens; /* T */
} db_page_tables;

/* `tokens` more tokens for sequence `seq`. */
typedef struct db_page_grow {
  uint32_t seq;
  uint32_t tokens;
} db_page_grow;  /* 8 bytes */

/* Sequence `child` gets the first `tokens` tokens of `parent`. */
typedef struct db_page_fork_req {
  uint32_t parent;
  uint32_t child;
  uint32_t tokens;
  uint32_t rsvd; /* ignored */
} db_page_fork_req; /* 16 bytes */

/* Sequence `seq` keeps its first `keep` tokens. */
typedef struct db_page_cut {
  uint32_t seq;
  uint32_t keep;
} db_page_cut;   /* 8 bytes */

/* The first `tokens` tokens of page `src` go to page `dst`. */
typedef struct db_page_move {
  uint32_t src;
  uint32_t dst;
  uint32_t tokens; /* DB_PAGE_ALL (or any number >= T): the whole page */
  uint32_t rsvd;   /* written 0, ignored when read */
} db_page_move;  /* 16 bytes */

/* One workspace serves every call of this header on a cache of this size, and
 * of no other: its parts lie where these two sizes put them, and one that
 * calls on a cache of other sizes have used must be zero-filled again. */
int db_page_workspace_size(uint32_t n_seqs, uint32_t n_pages, size_t* bytes);

/* Sequences grow. Request i needs ceil((length + tokens)/T) - ceil(length/T)
 * new pages, and one more, copy on write, when it adds tokens to a partly
 * filled last page that others hold: as if requests ran in order, a page all
 * of whose holders are in the batch stays with the last of them, and every
 * other one gets a page of its own in its place. Pages go to the requests in
 * order (a copy's page first), the lowest free index first.
 *   req     [n] requests (8-byte aligned)
 *   moves   [n] out (16-byte aligned): the copies to make, in request order:
 *           the shared page, its replacement, and the tokens it holds for the
 *           sequence
 *   n_moves [1] out (4-byte aligned): how many
 *   status  NULL or [n] out: DB_PAGE_INVALID when seq >= n_seqs, named
 *           before, or length + tokens > columns * T (or >= 2^32)
 *   ctr     NULL or counters: total = pages the valid requests need. With
 *           fewer free pages than that the batch changes nothing: n_overflow
 *           = the valid requests, their status DB_PAGE_SHORT, *n_moves = 0.
 * n <= n_seqs, n * columns < 2^32. */
int db_page_extend(const db_page_tables* t, const db_page_grow* req, uint32_t n,
                   db_page_move* moves, uint32_t* n_moves, uint8_t* status, db_counters* ctr,
                   void* ws, size_t ws_bytes, void* stream);

/* Sequences that share the first tokens of others: the child's row is the
 * parent's first ceil(tokens/T) pages, which each get one more reference (a
 * page that `tokens` fills partly too: the one that extends it first copies).
 * Lengths are those before the call. DB_PAGE_INVALID: parent or child >=
 * n_seqs, parent == child, child named before or not empty, tokens >
 * length[parent]. ctr: total = references taken. n <= n_seqs,
 * n * columns < 2^32, req 16-byte aligned. */
int db_page_fork(const db_page_tables* t, const db_page_fork_req* req, uint32_t n,
                 uint8_t* status, db_counters* ctr, void* ws, size_t ws_bytes, void* stream);

/* Sequences cut back to their first `keep` tokens (0: all go; keep >= length:
 * nothing does). Each page past ceil(keep/T) loses one reference and its
 * entry becomes DB_PAGE_NONE; a page without references is free.
 * DB_PAGE_INVALID: seq >= n_seqs or named before. ctr: total = pages that
 * became free. n <= n_seqs, n * columns < 2^32, req 8-byte aligned. */
int db_page_free(const db_page_tables* t, const db_page_cut* req, uint32_t n, uint8_t* status,
                 db_counters* ctr, void* ws, size_t ws_bytes, void* stream);

/* Live pages move down: with L live pages, the k-th lowest free page below L
 * gets the k-th highest live page, for k < min(M, cap), M being the free pages
 * below L. With cap >= M (n_pages/2 is always enough) the live pages are then
 * exactly [0, L). The cache as it is after the moves goes to `out`, whose
 * arrays may be t's own (any of them); sizes and page_tokens must be t's.
 * The bytes are the caller's to move with db_page_copy. Sources are not
 * overwritten, so until then the cache at `t`, when kept, stays readable.
 *   moves   [cap] out (16-byte aligned): {source, destination, DB_PAGE_ALL}
 *   n_moves [1] out (4-byte aligned): how many
 *   ctr     NULL or counters: total = M, n_overflow = M - *n_moves. */
int db_page_compact(const db_page_tables* t, const db_page_tables* out, db_page_move* moves,
                    uint32_t cap, uint32_t* n_moves, db_counters* ctr, void* ws, size_t ws_bytes,
                    void* stream);

/* The storage of pages: `planes` arrays of pages (keys and values of each
 * layer, say). Page p of plane l starts at base + l*plane_stride +
 * p*page_stride (bytes) and holds `segments` runs of page_tokens slots of
 * token_bytes each, without gaps: segments = 1 for [token][head] pages, the
 * heads for [head][token] ones. Data without a token axis (a scale for each
 * page and head) is one segment of one slot. base may be device memory or
 * pinned host memory. */
typedef struct db_page_pool {
  void* base;
  uint64_t n_pages;
  uint64_t plane_stride;
  uint64_t page_stride;
} db_page_pool;

typedef struct db_page_shape {
  uint32_t planes;
  uint32_t segments;
  uint32_t page_tokens;
  uint32_t token_bytes;
} db_page_shape;

/* The moves' bytes, in every plane: of each segment the first min(tokens,
 * page_tokens) slots. Slots past them keep what they hold. src and dst may be
 * the same pool, or different ones of one shape.
 *   moves   [max_moves] records (16-byte aligned), in device or pinned host
 *           memory
 *   n_moves [1] how many of them there are (4-byte aligned; more than
 *           max_moves: max_moves)
 * No page may be the destination of two records or of one and the source of
 * another (in one pool): its bytes are then undefined. A record naming a page
 * outside its pool is skipped; ctr (NULL or counters): total = records
 * copied, n_invalid = records skipped. One CTA counts them after its share of
 * the copying, at about a nanosecond a record: long lists of small pages
 * copy faster without counters (a million pages of 64 bytes in 52 us, and in
 * 853 with them). Launches are sized by max_moves: many more of them than
 * *n_moves cost time where segments are small (6 copies of 64 planes and 8
 * segments take 4 us in a list of 6, 27 in one of 4,096 and 516 in one of
 * 100,000). Strides must keep pages of one pool
 * apart; they and the bases need no alignment, but 16 bytes copy fastest. A
 * page's bytes in all planes are at most 2^31, planes at most 65536. */
int db_page_copy(const db_page_move* moves, uint32_t max_moves, const uint32_t* n_moves,
                 const db_page_pool* src, const db_page_pool* dst, const db_page_shape* shape,
                 db_counters* ctr, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* PAGECACHE_H */
