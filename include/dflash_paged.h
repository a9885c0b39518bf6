/*
 * dflash_paged.h — a paged key/value pool, the operations on its pages, and
 * attention over it; sliding-window attention for the draft step.
 *
 * dflash_cache (dflash.h) gives every request one slab of `capacity` positions.
 * A pool gives memory out in pages of page_size positions instead: a sequence
 * owns the positions [0, len) through a table of page ids, sequences with a
 * common prefix hold the same pages, and a page that others still hold is copied
 * before it is written.  dflash_pages_store / dflash_pages_load move a request's
 * rows between a dflash_cache and a sequence, so contexts that dflash_inject_kv
 * wrote can be kept, shared and brought back; dflash_paged_attention reads the
 * pages in place (one new token, a draft block, or a chunk of a prompt).
 *
 * A sequence s has len[s] positions and the table row table[s][0..max_pages):
 * entry i is the page of positions [i * page_size, (i+1) * page_size), entries
 * form a prefix and -1 follows them.  refs[x] counts the entries that hold page
 * x; a page is free when its count is 0.  A page stands at the same index i in
 * every table that holds it.  All of it lives in device memory and every call
 * below is a fixed sequence of kernels on the given stream, so calls can be
 * captured in a CUDA graph, and lengths, counts and sequence lists may have been
 * computed on the device.
 *
 * Conventions (beside those of dflash.h)
 *   - seqs: device int32[n] of sequence ids, or NULL for 0..n-1.  An entry of -1
 *     is padding: nothing is done for it.  n <= max_seqs (attention, which may list a
 *     sequence more than once: n <= 1024); n == 0 is a no-op.
 *   - A sequence that occurs again later in a list of a call that changes
 *     sequences is processed for its first entry only (device error INVALID_ARG);
 *     ids outside [-1, max_seqs) likewise are skipped with INVALID_ARG.
 *   - Device errors go to the pool's sticky first-error-wins status word
 *     (dflash_pool_status); the affected sequences are skipped unless a call says
 *     otherwise, the others proceed.
 *   - A pool is used from one stream at a time (it holds the calls' scratch), and
 *     with its own device current: otherwise calls return DFLASH_INVALID_ARG.
 */
#ifndef DFLASH_PAGED_H_
#define DFLASH_PAGED_H_

#include "dflash.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct {
    int n_layers;      /* >= 1 */
    int n_q_heads;     /* query heads of dflash_paged_attention, a multiple of n_kv_heads */
    int n_kv_heads;
    int head_dim;      /* 64 or 128 */
    int dtype;         /* DFLASH_BF16 or DFLASH_F32 */
    int n_pages;
    int page_size;     /* 16, 32, 64, 128 or 256 positions */
    int max_seqs;      /* 1..1024 */
    int max_len;       /* positions of a sequence, 1..2^30; a table has ceil(max_len / page_size) entries */
    int reserved;
} dflash_pool_config;

typedef struct dflash_pool dflash_pool;

typedef struct {
    int max_pages;        /* entries of a table row */
    int32_t* status;      /* device */
    int32_t* len;         /* device [max_seqs] */
    int32_t* table;       /* device [max_seqs][max_pages] */
    int32_t* refs;        /* device [n_pages] */
    void* slab;           /* device, storage type, [n_pages][n_layers][2 (K, V)][n_kv_heads][page_size][head_dim] */
    int64_t stride_page;  /* elements between pages */
    int64_t stride_layer; /* elements between layers of a page */
    int64_t stride_kind;  /* elements between K and V */
    int64_t stride_kv;    /* elements between kv heads */
} dflash_pool_info;

/* Bytes of device memory of a pool: tables, scratch of the calls, and the slab.
 * DFLASH_INVALID_ARG / DFLASH_UNSUPPORTED (page_size or head_dim not listed above;
 * more than 128 query heads per kv head; more than 2^31 - 1 rows of one head's K
 * or V in the slab; max_seqs * max_pages of 2^31 or more). */
int dflash_pool_bytes(const dflash_pool_config* cfg, size_t* bytes);

/* Bind caller memory (1024-byte aligned, borrowed) on the current device as an
 * empty pool (cleared on `stream`; the slab is left as it is). */
int dflash_pool_init(const dflash_pool_config* cfg, void* mem, size_t bytes, dflash_pool** out, dflash_stream stream);
void dflash_pool_release(dflash_pool* p);
int dflash_pool_get_info(const dflash_pool* p, dflash_pool_info* info);

/* Synchronise `stream`, then return and clear the pool's status word. */
int dflash_pool_status(dflash_pool* p, dflash_stream stream);

/* Kernel launches enqueued for this pool since it was bound (host counter). */
int64_t dflash_pool_launch_count(const dflash_pool* p);

/* Replace every table and length: lens device int32[max_seqs], table device
 * int32[max_seqs][max_pages] (they may be the pool's own arrays).  Counts are
 * taken from the tables.  For callers that filled the slab themselves or resume
 * from a saved state.  Device error: INVALID_ARG when a length is outside
 * [0, max_len], an id outside [-1, n_pages), entries are no prefix or too few for
 * the length, or a page stands at two different indices; every sequence is empty
 * then. */
int dflash_pool_set_tables(dflash_pool* p, const int32_t* lens, const int32_t* table, dflash_stream stream);

/* Make the positions [len, len + grow[i]) of each listed sequence writable: an
 * entry that is missing gets the lowest-numbered free page, and an entry whose
 * page another sequence still holds is replaced by a free page, the rows before
 * len copied into it (copy on write).  Entries are served in list order, table
 * index ascending, free pages ascending; of the listed sequences that share a
 * page and would write it, the last keeps it if no other sequence holds it.
 * grow: device int32[n], >= 0 (INVALID_ARG), len + grow <= max_len (CAPACITY).
 * When the free pages do not suffice for the whole call, CAPACITY is recorded and
 * nothing is changed for any sequence. */
int dflash_pages_reserve(dflash_pool* p, const int32_t* seqs, const int32_t* grow, int n, dflash_stream stream);

/* dst[i] becomes src[i]'s context: the same pages up to ceil(len / page_size)
 * (deep == 0), or copies of them in free pages (deep != 0; taken as in reserve,
 * CAPACITY and nothing changed when they do not suffice).  src and dst: device
 * int32[n]; a pair with src or dst -1 is padding: what stands beside the -1 is not
 * looked at, except that no destination may stand in src, beside a dst of -1 either.
 * A source may occur any number of times.  A destination must be empty (len 0 and no
 * pages: STATE otherwise), occur once, and not stand in src (INVALID_ARG). */
int dflash_pages_fork(dflash_pool* p, const int32_t* src, const int32_t* dst, int n, int deep, dflash_stream stream);

/* Cut each listed sequence back to keep[i] positions (device int32[n], NULL = 0:
 * free it) and give back the pages past ceil(keep / page_size), reserved ones
 * included.  0 <= keep[i] <= len (INVALID_ARG). */
int dflash_pages_free(dflash_pool* p, const int32_t* seqs, const int32_t* keep, int n, dflash_stream stream);

/* Move pages so that the ones in use are 0..used-1: with `used` pages in use, the
 * j-th page in use numbered >= used moves to the j-th free page below used.
 * Tables and counts follow.  used: device int32[1], written. */
int dflash_pages_compact(dflash_pool* p, int32_t* used, dflash_stream stream);

/* Write new rows of one layer at the positions len, len + 1, ... of each listed
 * sequence (lengths are not changed: dflash_pages_advance).  Entry i owns the rows
 * row_start[i] .. row_start[i] + row_count[i) of k and v (device int32[n], ranges
 * inside [0, total_rows): INVALID_ARG; both NULL: entry i owns row i).  k, v:
 * device, storage type, row r at k + r * stride (elements; rows 16-byte aligned),
 * a row is [n_kv_heads][head_dim], K already rotated.  max_rows: host bound of
 * row_count (larger counts: INVALID_ARG).  Device errors: CAPACITY (positions not
 * reserved), STATE (a page that another sequence holds: reserve first). */
int dflash_pages_write(dflash_pool* p, const int32_t* seqs, int n, int layer, const void* k, const void* v,
                       int64_t stride, const int32_t* row_start, const int32_t* row_count, int total_rows,
                       int max_rows, dflash_stream stream);

/* len += row_count[i] (device int32[n]; NULL = 1) for each listed sequence, e.g.
 * accepted rows after dflash_accept.  INVALID_ARG when negative, CAPACITY when the
 * positions are not reserved. */
int dflash_pages_advance(dflash_pool* p, const int32_t* seqs, const int32_t* row_count, int n, dflash_stream stream);

/* Keep a request's context: append the positions [len of seqs[i], len of request
 * reqs[i]) of every layer from the cache (reqs: device int32[n] or NULL for
 * 0..n-1; the cache's shape and type must match the pool's) and set the sequence's
 * len.  The positions must be reserved (CAPACITY, STATE as in write).  Nothing is
 * done where the sequence is at least as long.  The caller vouches that both hold
 * the same context up to the shorter length.  A pair with seqs or reqs -1 is padding:
 * what stands beside the -1 is not looked at (here and in dflash_pages_load). */
int dflash_pages_store(dflash_pool* p, const int32_t* seqs, const dflash_cache* c, const int32_t* reqs, int n,
                       dflash_stream stream);

/* Bring a context back: append the positions [len of request reqs[i], len of
 * seqs[i]) to the cache and set the request's len and committed to the sequence's
 * length.  CAPACITY when the cache is too short; a request that occurs twice is
 * processed once (INVALID_ARG).  Nothing is done where the request is longer. */
int dflash_pages_load(dflash_pool* p, const int32_t* seqs, dflash_cache* c, const int32_t* reqs, int n,
                      dflash_stream stream);

/* Attention of new rows over one layer of the pool.  Entry i owns the query rows
 * row_start[i] .. row_start[i] + row_count[i) (as in dflash_pages_write; both NULL:
 * one row each, row i), at the positions len, len + 1, ...; their keys and values
 * are in the pool (dflash_pages_write before this, dflash_pages_advance after it).
 * A row at position p sees the keys k <= p (causal) or k < len + row_count (not
 * causal, a block whose rows see one another), and with window > 0 of those only
 * k > p - window and k < sinks.  window == 0: no window (sinks is not used).
 * With t_k = q.k log2(e) / sqrt(head_dim),
 *   out = R( sum_k P_k v_k / sum_k 2^(t_k - b) ),  P_k = 2^(t_k - b),
 * for an integer b; bf16 pools round P_k to bf16 before it weights v (as
 * dflash_draft_block) in calls with max_rows * n_q_heads / n_kv_heads > 16, and
 * keep 16 bits of it (two bf16 terms) in smaller ones; fp32 pools do not round it.
 * The keys of an entry may be split over the device in a way that depends on the
 * whole call, so a row's result can differ in its last bits when other entries
 * do; the same call gives the same bits every time.
 * q: device, storage type, row r at q + r * q_stride elements (>= n_q_heads *
 * head_dim, rows 16-byte aligned), a row is [n_q_heads][head_dim].  out: device
 * [total_rows][n_q_heads][head_dim], 16-byte aligned, no part of q; rows that no entry owns are
 * not written, rows of a skipped entry are zero (of an entry whose row range or row_count is
 * refused: not written).  Entries may list the same sequence and must not own the same row.
 * max_rows or total_rows 0: a no-op, whatever row_count holds (here and in
 * dflash_pages_write).
 * Cached rows past the last position, and rows that no query row of the call sees,
 * may hold anything, NaN included; a V row that one query row of an entry sees and
 * another does not must be finite.  bf16 pools want |t_k| below 2^31: beyond, one
 * rounding of t_k in fp32 is a factor of 2^128, and rows may come out as NaN.
 * Device errors: INVALID_ARG (row ranges, row_count > max_rows or negative),
 * CAPACITY (positions without a page), UNSUPPORTED (bf16: 2^31 or more tiles of 64
 * keys over all rows and heads of the call; no result is written). */
int dflash_paged_attention(dflash_pool* p, const int32_t* seqs, int n, int layer, const void* q, int64_t q_stride,
                           const int32_t* row_start, const int32_t* row_count, int total_rows, int max_rows,
                           int causal, int window, int sinks, void* out, dflash_stream stream);

/* Sliding-window attention for the draft step of one cache (bf16 handles): from
 * now on dflash_draft_block on c lets the block row at position p see, of the
 * context, only the keys k > p - window and k < sinks (all of the block's own rows
 * k >= len stay subject to the same rule and are otherwise visible), and
 * dflash_ingest_fused_input the causal form of it.  window == 0 turns it off.
 * The cached rows are kept whole, so the window may change between calls.
 * scratch: device memory of dflash_window_scratch_bytes, 256-byte aligned,
 * borrowed until the window is turned off or the cache released (and while a graph
 * captured with it may still be replayed), and cleared here on `stream`; one cache
 * uses it at a time.  DFLASH_UNSUPPORTED: fp32 handles, more than 1024 requests, or
 * a slab of 2^31 or more rows of one head's K or V. */
int dflash_window_scratch_bytes(size_t* bytes);
int dflash_cache_set_window(dflash_cache* c, int window, int sinks, void* scratch, size_t bytes, dflash_stream stream);

#ifdef __cplusplus
}
#endif
#endif /* DFLASH_PAGED_H_ */
