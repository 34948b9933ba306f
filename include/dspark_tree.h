/*
 * dspark_tree.h -- C ABI of drafts that form a tree, over the paged key/value cache of
 * dspark_cache.h, for AMD Instinct MI355X (gfx950).
 *
 *   dspark_tree_mask   -- every node's ancestors and depth, from the nodes' parents
 *   dspark_tree_attend -- attention of the nodes over their context and their ancestors
 *   dspark_tree_keep   -- the accepted nodes' keys and values to the front of the tree
 *
 * A tree's nodes are the new tokens of a request, in an order in which a parent comes
 * before its children (node 0, for instance, the anchor, which hangs from the context
 * alone).  Node i is row row_start[b] + i, and its key and value lie at position
 * length[b] - n_new[b] + i of the request's sequence until the accepted path is kept.
 * One cycle, without the host reading anything back:
 *   dspark_cache_update (length + the number of nodes),
 *   n_new = length_out - length, on the device,
 *   dspark_tree_mask,
 *   per layer: dspark_cache_append, dspark_tree_attend,
 *   the caller's choice of a path, dspark_tree_keep, dspark_cache_update (length_out).
 * n_new is what the update gave a request, in every call of the cycle: fewer than its nodes at
 * the end of its row of the page table (the first nodes, a tree again), none where the pool has no
 * room.  With a larger count the nodes would begin among the tokens that the sequence already
 * holds: those would be overwritten, in pages that others may share, and dropped.  The path has
 * to be cut to nodes below n_new, which in an ascending path come first.
 * A node is at position length - n_new + depth of its branch's text; encodings of
 * positions are the caller's, as they are with dspark_cache_append.
 *
 * Conventions, limits, types and status codes are those of dspark_cache.h.
 */
#ifndef DSPARK_TREE_H
#define DSPARK_TREE_H

#include "dspark_cache.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * dspark_tree_mask -- for node i of request b: bit j of mask[row] (word j / 32, bit j % 32)
 * is set iff j is i or one of its ancestors, with window > 0 only those nearer than window
 * (i itself at distance 0); depth[row] is the number of its ancestors.
 *
 * Inputs:  parent [n_rows] int32: the node's parent among the request's nodes, -1 (or
 *          any value outside [0, i)) for a node without one; n_new [B], row_start [B]
 *          int32 or NULL as for dspark_cache_append.
 * Outputs: mask [n_rows][ceil(max_new / 32)] uint32; depth [n_rows] int32 or NULL.  Rows
 *          that belong to no request are left as they were.  They must not overlap the
 *          inputs or each other.
 * 1 <= B <= 65536, 1 <= max_new <= 1024, window >= 0; 4-byte aligned.  n_rows = 0 does
 * nothing.
 */
dspark_status dspark_tree_mask(int32_t B, const int32_t* parent, int32_t n_rows, const int32_t* n_new,
                               const int32_t* row_start, int32_t max_new, int32_t window, uint32_t* mask,
                               int32_t* depth, hipStream_t stream);

/*
 * dspark_tree_attend -- dspark_cache_attend with another choice of what a row sees: node i
 * of request b sees the positions j < length[b] - n_new[b] of its context, with window > 0
 * only j > length[b] - n_new[b] + depth[row] - window, and the nodes k <= i whose bit is
 * set in mask[row].  Any bits will do; those of other nodes are ignored.  With a window,
 * mask is to be one made with it.
 *
 * Inputs:  as for dspark_cache_attend; mask [n_rows][ceil(max_new / 32)] uint32; depth
 *          [n_rows] int32 (clamped to [0, i]; may be NULL with window = 0).
 * Outputs, types, precision, workspace and limits as for dspark_cache_attend.
 */
dspark_status dspark_tree_attend(const dspark_cache* C, int32_t layer, const void* q, int64_t q_stride, int32_t n_rows,
                                 const int32_t* n_new, const int32_t* row_start, int32_t max_new, const uint32_t* mask,
                                 const int32_t* depth, const int32_t* length, const int32_t* table,
                                 const void* k_pool, const void* v_pool, const float* k_scale, const float* v_scale,
                                 float scale, int32_t window, void* out, int64_t out_stride, float* lse,
                                 void* workspace, size_t workspace_bytes, hipStream_t stream);

/*
 * dspark_tree_keep -- for i < n_keep[b], in this order: the key and the value at position
 * length[b] - n_new[b] + path[b][i] go to position length[b] - n_new[b] + i, in all layers
 * of both pools (with their scales, if tokens have their own).  length_out[b] =
 * length[b] - n_new[b] + n_keep[b], the new_len of the update that drops the rest.
 *
 * Inputs:  path [B][max_path] int32, ascending within a request, in [0, n_new[b]): entries
 *          outside are skipped, and an order that does not ascend leaves unspecified
 *          tokens among those written; n_keep [B] int32 (clamped to [0, max_path] and to
 *          n_new[b]); n_new [B] int32 or NULL (max_new everywhere); length [B]; table
 *          [B][max_pages].  (Entries that are skipped count in n_keep: a path that may hold nodes
 *          that did not run is to be cut first.)
 * Outputs: length_out [B] int32, which must not overlap the inputs.
 * In/out:  k_pool, v_pool.  Pages of a request's new tokens must be its own (as after the
 *          update that made room for them).
 * 1 <= max_path <= 1024, 1 <= max_new <= 2^20.
 */
dspark_status dspark_tree_keep(const dspark_cache* C, const int32_t* path, const int32_t* n_keep, int32_t max_path,
                               const int32_t* n_new, int32_t max_new, const int32_t* length, const int32_t* table,
                               int32_t* length_out, void* k_pool, void* v_pool, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* DSPARK_TREE_H */
