/*
 * dspark_cache.h -- C ABI of the paged key/value cache that the target's forward
 * pass reads between dspark_schedule and dspark_verify, for AMD Instinct MI355X
 * (gfx950).
 *
 *   dspark_cache_append  -- the keys and values of the scheduled rows, into pages
 *   dspark_cache_attend  -- attention of the scheduled rows over those pages
 *   dspark_cache_update  -- every slot's next sequence: grow by the schedule, drop
 *                           the rejected tokens, fork, reorder, free
 *   dspark_cache_compact -- live pages moved to the lowest ids
 *
 * One cycle of a serving loop, all of it on one stream and without the host
 * reading anything back:
 *   dspark_draft, dspark_schedule,
 *   dspark_cache_update (length + n_sched + 1),
 *   per layer: dspark_cache_append, dspark_cache_attend,
 *   dspark_verify,
 *   dspark_cache_update (the accepted length).
 * A request gets n_new = length_out - length rows from the first update: fewer than
 * n_sched + 1 at the end of its row of the page table, none where the pool has no room.
 * Those are the counts for append and attend, and dspark_verify may judge n_new - 1
 * drafts at most: the target has no logits for more.
 *
 * The cache.  Request slot b holds length[b] tokens in the pages
 * table[b][0 .. ceil(length[b] / page) - 1]; token j lies in page table[b][j / page]
 * at offset j % page.  A page id names the same page in every layer of both pools;
 * ref[p] counts the slots that hold page p (0: free).  Several slots may hold one
 * page (forks of one prompt).  Pools:
 *   k_pool [n_layers][n_pages][Hkv][page][D]       a key is one row
 *   v_pool [n_layers][n_pages][Hkv][page/8][D][8]  8 tokens of one coordinate together,
 *     so that the product with the softmax weights reads its operand (8 consecutive
 *     tokens per lane) with one load, and a token's write stays within 8 * D elements.
 * What no sequence holds (other pages, offsets past a length) may contain anything,
 * NaN and infinities included.
 *
 * Conventions are those of dspark.h: device pointers, host struct, caller-owned
 * buffers, host-side validation before anything is enqueued, no allocation, no
 * synchronisation, no state between calls; every call can be captured in a HIP
 * graph.  Calls that share a workspace, or of which one writes what the other
 * reads, have to be ordered (one stream, or events).  Results are bit-reproducible
 * for given inputs.  Values in device memory cannot be checked on the host: a page
 * id outside [0, n_pages) is never dereferenced (attend reads another page of the
 * pool in its place, append skips the token, update and compact leave it out),
 * lengths are clamped to [0, max_pages * page], row counts to [0, max_new], and
 * rows outside [0, n_rows) are skipped.
 *
 * Supported: 1 <= B <= 65536; page in {16, 32, 64, 128, 256}; 1 <= max_pages with
 * max_pages * page <= 2^24; 1 <= n_pages <= 2^24; 1 <= n_layers <= 1024;
 * Hq a multiple of Hkv, 1 <= Hkv, Hq <= 1024; D in {64, 128, 256}; 1 <= max_new <=
 * 2^20, for attend with B * ceil(max_new * Hq / Hkv / 16) <= 2^24.  Types (data = q,
 * k, v, out): fp32 data with an fp32 cache, bf16 data with a bf16 or an e4m3 cache.
 * Pools, q, k, v, out 16-byte aligned; other arrays 4-byte aligned.
 */
#ifndef DSPARK_CACHE_H
#define DSPARK_CACHE_H

#include "dspark.h"

#ifdef __cplusplus
extern "C" {
#endif

/* cache_dtype only: 8-bit floats (4 exponent, 3 mantissa bits, no infinities), with a
 * scale per kv head: value = stored * scale[head]. */
enum { DSPARK_F8E4M3 = 2 };

typedef struct {
  int32_t B;           /* request slots */
  int32_t n_pages;     /* pages of the pool */
  int32_t page;        /* tokens of a page */
  int32_t max_pages;   /* entries of a slot's row of the page table */
  int32_t n_layers;
  int32_t Hq, Hkv, D;  /* query heads, key/value heads, head size; query head i reads kv head i / (Hq / Hkv) */
  int32_t data_dtype;  /* dspark_dtype of q, k, v and out */
  int32_t cache_dtype; /* dspark_dtype of the pools, or DSPARK_F8E4M3 */
} dspark_cache;

/* Bytes of workspace for dspark_cache_attend with up to max_new rows a request,
 * dspark_cache_update and dspark_cache_compact; 0 if C or max_new is invalid.
 * Host-only: makes no HIP call.  256-byte aligned, contents need no initialising. */
size_t dspark_cache_workspace_bytes(const dspark_cache* C, int32_t max_new);

/*
 * dspark_cache_append -- token i (0 <= i < n_new[b]) of request b, row
 * row_start[b] + i of k and v, becomes position length[b] - n_new[b] + i of its
 * sequence (length counts the new tokens already; negative positions are skipped).
 *
 * Inputs:  k, v [n_rows][Hkv][D] (data_dtype; rows k_stride and v_stride elements
 *          apart, each a multiple of 16 bytes); n_new [B] int32 or NULL (max_new
 *          everywhere); row_start [B] int32 or NULL (b * max_new); length [B];
 *          table [B][max_pages]; k_scale, v_scale [Hkv] fp32, finite and positive,
 *          for an e4m3 cache (ignored otherwise).
 * In/out:  k_pool, v_pool: layer `layer` receives the tokens; nothing else changes.
 * An e4m3 cache stores x / scale rounded to nearest (ties to even), values past
 * +-448 as +-448, NaN as NaN.  A page that several slots hold must not be written
 * (dspark_cache_update gives every growing slot a private one).  Of 8 neighbouring
 * tokens that are not all new the others' values are read and written back as they
 * are: two calls that append to one page have to be ordered.  n_rows = 0 does
 * nothing.
 */
dspark_status dspark_cache_append(const dspark_cache* C, int32_t layer, const void* k, int64_t k_stride, const void* v,
                                  int64_t v_stride, int32_t n_rows, const int32_t* n_new, const int32_t* row_start,
                                  int32_t max_new, const int32_t* length, const int32_t* table, const float* k_scale,
                                  const float* v_scale, void* k_pool, void* v_pool, hipStream_t stream);

/*
 * dspark_cache_attend -- for every new token i of request b, at position
 * pos = length[b] - n_new[b] + i, and every query head:
 *   out = sum_j w_j v_j / sum_j w_j,  w_j = exp(scale * q . k_j),  lse = ln sum_j w_j,
 * over the positions j that it sees: 0 <= j < length[b]; with causal != 0 also
 * j <= pos; with window > 0 also j > pos - window.  A row that sees no position (or
 * only weights of 0) gets out = 0 and lse = -inf.  Keys and values that a row does
 * not see have no influence on it, not even as NaN.
 *
 * Inputs:  q [n_rows][Hq][D] (data_dtype, rows q_stride elements apart, a multiple
 *          of 16 bytes); n_new, row_start, length, table, k_scale, v_scale as above;
 *          scale > 0, scale * log2(e) finite (with an e4m3 cache also times k_scale).
 * Outputs: out [n_rows][Hq][D] (rows out_stride elements apart); lse
 *          [n_rows][Hq] fp32 or NULL.  Rows that belong to no request are left as
 *          they were.  Outputs must not overlap the inputs or each other.
 * Products and sums are fp32.  With bf16 data the softmax weights enter their product
 * with the values in two bf16 terms (2^-16 relative) where max_new * Hq / Hkv <= 16, and
 * rounded to bf16 (2^-8) beyond, where products are what a call waits for.  causal = 0 is
 * the mask of a parallel drafter's block.  n_rows = 0 does nothing.
 * Work is launched for max_new rows of all B slots and for the width of the page
 * table, whatever n_new and length hold: prompts are better in a call over their own
 * slots (a dspark_cache of fewer B, table and length from the first of them on), single
 * tokens in one with a small max_new, where the prompts' n_new is 0.
 */
dspark_status dspark_cache_attend(const dspark_cache* C, int32_t layer, const void* q, int64_t q_stride, int32_t n_rows,
                                  const int32_t* n_new, const int32_t* row_start, int32_t max_new,
                                  const int32_t* length, const int32_t* table, const void* k_pool, const void* v_pool,
                                  const float* k_scale, const float* v_scale, float scale, int32_t causal,
                                  int32_t window, void* out, int64_t out_stride, float* lse, void* workspace,
                                  size_t workspace_bytes, hipStream_t stream);

/*
 * dspark_cache_update -- every slot's next sequence, from the slots' present ones:
 * slot b starts with the first keep = min(length[parent[b]], new_len[b]) tokens of
 * slot parent[b] (its own with parent[b] = b or parent = NULL; none with parent[b]
 * outside [0, B)) and is extended to new_len[b] tokens (clamped to
 * [0, max_pages * page]), whose content dspark_cache_append writes.  One call forks,
 * reorders, grows, shrinks and frees:
 *   1. references of all present sequences go, those of the kept pages come;
 *   2. a slot that grows while its last kept page is partly filled and held by
 *      others too gets a private copy of that page (all layers, both pools);
 *   3. new pages are the free pages (ref 0 after step 1), lowest ids first, to the
 *      slots in ascending order, a slot's copy before its further pages.
 * When the free pages run out, the first slot whose pages do not fit, and every
 * later slot that needs any, stays at its kept tokens (length_out tells), and
 * n_short is the number of pages that were missing.
 *
 * Inputs:  parent [B] or NULL; new_len [B]; table [B][max_pages]; length [B];
 *          ref [n_pages].
 * Outputs: table_out, length_out, ref_out (entries of table_out past a sequence's
 *          pages are -1); n_short [1].  They must not overlap the inputs.
 * In/out:  k_pool, v_pool (step 2's copies; other pages are left alone).
 */
dspark_status dspark_cache_update(const dspark_cache* C, const int32_t* parent, const int32_t* new_len,
                                  const int32_t* table, const int32_t* length, const int32_t* ref, int32_t* table_out,
                                  int32_t* length_out, int32_t* ref_out, int32_t* n_short, void* k_pool, void* v_pool,
                                  void* workspace, size_t workspace_bytes, hipStream_t stream);

/*
 * dspark_cache_compact -- with n_live pages in use, those with ids >= n_live move
 * (all layers, both pools) to the free ids below n_live, both in ascending order,
 * so that the pool's first n_live pages are the live ones.  Lengths do not change.
 * A caller that wants a smaller pool copies the first n_live (or more) pages of every
 * layer of both pools into it, and goes on with the same table and the first entries
 * of ref, under a dspark_cache with that n_pages; the same pages are a snapshot's.
 *
 * Inputs:  table [B][max_pages], length [B], ref [n_pages].
 * Outputs: table_out (entries past a sequence's pages, and ids that ref calls free,
 *          are -1), ref_out, n_live [1].  They must not overlap the inputs.
 * In/out:  k_pool, v_pool (the pages below n_live that were free are written).
 */
dspark_status dspark_cache_compact(const dspark_cache* C, const int32_t* table, const int32_t* length,
                                   const int32_t* ref, int32_t* table_out, int32_t* ref_out, int32_t* n_live,
                                   void* k_pool, void* v_pool, void* workspace, size_t workspace_bytes,
                                   hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* DSPARK_CACHE_H */
