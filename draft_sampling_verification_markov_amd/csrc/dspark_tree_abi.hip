// C ABI of drafted trees over the paged cache: argument validation and the launch of each
// call.  See include/dspark_tree.h for the contract.
#include "../../include/dspark_tree.h"

#include "dspark_cache_checks.hpp"

using namespace dspark;

extern "C" dspark_status dspark_tree_mask(int32_t B, const int32_t* parent, int32_t n_rows, const int32_t* n_new,
                                          const int32_t* row_start, int32_t max_new, int32_t window, uint32_t* mask,
                                          int32_t* depth, hipStream_t stream) {
  const AbiRange range("dspark_tree_mask");
  if (B < 1 || B > 65536 || n_rows < 0 || max_new < 1 || max_new > kMaxNodes || window < 0) return DSPARK_E_INVALID;
  if (n_rows == 0) return DSPARK_OK;
  if (!parent || !mask) return DSPARK_E_POINTER;
  for (const void* p : {(const void*)parent, (const void*)n_new, (const void*)row_start, (const void*)mask,
                        (const void*)depth})
    if (!aligned(p, 4)) return DSPARK_E_POINTER;
  const int32_t words = (max_new + 31) / 32;
  const size_t nb = (size_t)B * 4, nr = (size_t)n_rows * 4, nm = nr * words;
  const struct { const void* p; size_t n; } in[] = {{parent, nr}, {n_new, n_new ? nb : 0}, {row_start, row_start ? nb : 0}};
  for (const auto& x : in)
    if (x.n && (overlap(x.p, x.n, mask, nm) || (depth && overlap(x.p, x.n, depth, nr)))) return DSPARK_E_POINTER;
  if (depth && overlap(mask, nm, depth, nr)) return DSPARK_E_POINTER;
  (void)hipGetLastError();
  const TreeMaskArgs a{parent, n_new, row_start, mask, depth, B, n_rows, max_new, window, words};
  return launch_tree_mask(a, stream) == hipSuccess ? DSPARK_OK : DSPARK_E_LAUNCH;
}

extern "C" dspark_status dspark_tree_attend(const dspark_cache* C, int32_t layer, const void* q, int64_t q_stride,
                                            int32_t n_rows, const int32_t* n_new, const int32_t* row_start,
                                            int32_t max_new, const uint32_t* mask, const int32_t* depth,
                                            const int32_t* length, const int32_t* table, const void* k_pool,
                                            const void* v_pool, const float* k_scale, const float* v_scale,
                                            float scale, int32_t window, void* out, int64_t out_stride, float* lse,
                                            void* workspace, size_t workspace_bytes, hipStream_t stream) {
  const AbiRange range("dspark_tree_attend");
  AttendArgs a;
  const dspark_status st =
      attend_args(C, layer, q, q_stride, n_rows, n_new, row_start, max_new, length, table, k_pool, v_pool, k_scale, v_scale,
                  scale, 1, window, out, out_stride, lse, workspace, workspace_bytes, a);
  if (st != DSPARK_OK || n_rows == 0) return st;
  if (!mask || !aligned(mask, 4) || !aligned(depth, 4) || (window > 0 && !depth)) return DSPARK_E_POINTER;
  a.mask = mask;
  a.depth = window > 0 ? depth : nullptr;
  a.mask_words = (max_new + 31) / 32;
  (void)hipGetLastError();
  return launch_tree_attend(*C, a, stream) == hipSuccess ? DSPARK_OK : DSPARK_E_LAUNCH;
}

extern "C" dspark_status dspark_tree_keep(const dspark_cache* C, const int32_t* path, const int32_t* n_keep,
                                          int32_t max_path, const int32_t* n_new, int32_t max_new,
                                          const int32_t* length, const int32_t* table, int32_t* length_out,
                                          void* k_pool, void* v_pool, hipStream_t stream) {
  const AbiRange range("dspark_tree_keep");
  const dspark_status st = check_cache(C);
  if (st != DSPARK_OK) return st;
  if (max_path < 1 || max_path > kMaxPath || max_new < 1 || max_new > kMaxNew) return DSPARK_E_INVALID;
  if (!path || !n_keep || !length || !table || !length_out || !k_pool || !v_pool) return DSPARK_E_POINTER;
  if (!aligned(k_pool, 16) || !aligned(v_pool, 16)) return DSPARK_E_POINTER;
  for (const void* p : {(const void*)path, (const void*)n_keep, (const void*)n_new, (const void*)length,
                        (const void*)table, (const void*)length_out})
    if (!aligned(p, 4)) return DSPARK_E_POINTER;
  const size_t nb = (size_t)C->B * 4;
  const struct { const void* p; size_t n; } in[] = {{path, nb * max_path}, {n_keep, nb}, {n_new, n_new ? nb : 0},
                                                    {length, nb}, {table, nb * C->max_pages}};
  for (const auto& x : in)
    if (x.n && overlap(x.p, x.n, length_out, nb)) return DSPARK_E_POINTER;
  (void)hipGetLastError();
  KeepArgs a{};
  a.c = view(*C, 0, n_new, nullptr, max_new, length, table);
  a.path = path;
  a.n_keep = n_keep;
  a.length_out = length_out;
  a.k_pool = static_cast<char*>(k_pool);
  a.v_pool = static_cast<char*>(v_pool);
  a.layer_bytes = page_bytes(*C) * C->n_pages;
  a.max_path = max_path;
  return launch_tree_keep(*C, a, stream) == hipSuccess ? DSPARK_OK : DSPARK_E_LAUNCH;
}
