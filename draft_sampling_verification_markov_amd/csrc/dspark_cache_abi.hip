// C ABI of the paged cache: argument validation, workspace layout and the kernel
// sequence of each call.  See include/dspark_cache.h for the contract.
#include "dspark_cache_checks.hpp"

namespace dspark {
namespace {

template <typename T>
T* at(void* ws, size_t off) {
  return reinterpret_cast<T*>(static_cast<char*>(ws) + off);
}

dspark_status check_pages(const dspark_cache* C, void* k_pool, void* v_pool, void* ws, size_t bytes) {
  if (!k_pool || !v_pool || !aligned(k_pool, 16) || !aligned(v_pool, 16)) return DSPARK_E_POINTER;
  if (!ws || !aligned(ws, 256) || bytes < pages_layout(*C).total) return DSPARK_E_WORKSPACE;
  return DSPARK_OK;
}

PagesArgs pages_args(const dspark_cache& C, const int32_t* table, const int32_t* length, const int32_t* ref,
                     int32_t* table_out, int32_t* ref_out, int32_t* count, void* ws) {
  const PagesLayout L = pages_layout(C);
  PagesArgs a{};
  a.table = table;
  a.length = length;
  a.ref = ref;
  a.table_out = table_out;
  a.ref_out = ref_out;
  a.count = count;
  a.block_count = at<int32_t>(ws, L.block_count);
  a.need = at<int32_t>(ws, L.need);
  a.base = at<int32_t>(ws, L.base);
  a.ids = at<int32_t>(ws, L.ids);
  a.src = at<int32_t>(ws, L.src);
  a.dst = at<int32_t>(ws, L.dst);
  a.rank = at<int32_t>(ws, L.rank);
  a.n_copies = at<int32_t>(ws, L.n_copies);
  a.B = C.B;
  a.n_pages = C.n_pages;
  a.page_shift = log2_page(C.page);
  a.max_pages = C.max_pages;
  return a;
}

}  // namespace
}  // namespace dspark

using namespace dspark;

extern "C" size_t dspark_cache_workspace_bytes(const dspark_cache* C, int32_t max_new) {
  if (check_cache(C) != DSPARK_OK || max_new < 1 || max_new > kMaxNew) return 0;
  const size_t a = attend_workspace_bytes(*C, max_new), p = pages_layout(*C).total;
  return a > p ? a : p;
}

extern "C" dspark_status dspark_cache_append(const dspark_cache* C, int32_t layer, const void* k, int64_t k_stride,
                                             const void* v, int64_t v_stride, int32_t n_rows, const int32_t* n_new,
                                             const int32_t* row_start, int32_t max_new, const int32_t* length,
                                             const int32_t* table, const float* k_scale, const float* v_scale,
                                             void* k_pool, void* v_pool, hipStream_t stream) {
  const AbiRange range("dspark_cache_append");
  dspark_status st = check_cache(C);
  if (st != DSPARK_OK) return st;
  st = check_tokens(*C, layer, n_rows, n_new, row_start, max_new, length, table, k_pool, v_pool, k_scale, v_scale);
  if (st != DSPARK_OK) return st;
  if (n_rows == 0) return DSPARK_OK;
  const int es = element_bytes(C->data_dtype);
  st = check_rows(k, k_stride, (int64_t)C->Hkv * C->D, n_rows, es);
  if (st == DSPARK_OK) st = check_rows(v, v_stride, (int64_t)C->Hkv * C->D, n_rows, es);
  if (st != DSPARK_OK) return st;
  (void)hipGetLastError();
  const size_t layer_bytes = page_bytes(*C) * C->n_pages;
  AppendArgs a{};
  a.c = view(*C, n_rows, n_new, row_start, max_new, length, table);
  a.k = k;
  a.v = v;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  a.k_pool = static_cast<char*>(k_pool) + layer * layer_bytes;
  a.v_pool = static_cast<char*>(v_pool) + layer * layer_bytes;
  return launch_cache_append(*C, a, stream) == hipSuccess ? DSPARK_OK : DSPARK_E_LAUNCH;
}

extern "C" dspark_status dspark_cache_attend(const dspark_cache* C, int32_t layer, const void* q, int64_t q_stride,
                                             int32_t n_rows, const int32_t* n_new, const int32_t* row_start,
                                             int32_t max_new, const int32_t* length, const int32_t* table,
                                             const void* k_pool, const void* v_pool, const float* k_scale,
                                             const float* v_scale, float scale, int32_t causal, int32_t window,
                                             void* out, int64_t out_stride, float* lse, void* workspace,
                                             size_t workspace_bytes, hipStream_t stream) {
  const AbiRange range("dspark_cache_attend");
  AttendArgs a;
  const dspark_status st =
      attend_args(C, layer, q, q_stride, n_rows, n_new, row_start, max_new, length, table, k_pool, v_pool, k_scale, v_scale,
                  scale, causal, window, out, out_stride, lse, workspace, workspace_bytes, a);
  if (st != DSPARK_OK || n_rows == 0) return st;
  (void)hipGetLastError();
  return launch_cache_attend(*C, a, stream) == hipSuccess ? DSPARK_OK : DSPARK_E_LAUNCH;
}

extern "C" dspark_status dspark_cache_update(const dspark_cache* C, const int32_t* parent, const int32_t* new_len,
                                             const int32_t* table, const int32_t* length, const int32_t* ref,
                                             int32_t* table_out, int32_t* length_out, int32_t* ref_out,
                                             int32_t* n_short, void* k_pool, void* v_pool, void* workspace,
                                             size_t workspace_bytes, hipStream_t stream) {
  const AbiRange range("dspark_cache_update");
  dspark_status st = check_cache(C);
  if (st != DSPARK_OK) return st;
  if (!new_len || !table || !length || !ref || !table_out || !length_out || !ref_out || !n_short)
    return DSPARK_E_POINTER;
  for (const void* p : {(const void*)parent, (const void*)new_len, (const void*)table, (const void*)length,
                        (const void*)ref, (const void*)table_out, (const void*)length_out, (const void*)ref_out,
                        (const void*)n_short})
    if (!aligned(p, 4)) return DSPARK_E_POINTER;
  const size_t nb = (size_t)C->B * 4, nt = nb * C->max_pages, nr = (size_t)C->n_pages * 4;
  const struct { const void* p; size_t n; } in[] = {{parent, parent ? nb : 0}, {new_len, nb}, {table, nt}, {length, nb},
                                                    {ref, nr}},
      to[] = {{table_out, nt}, {length_out, nb}, {ref_out, nr}, {n_short, 4}};
  for (const auto& x : in)
    for (const auto& y : to)
      if (x.n && overlap(x.p, x.n, y.p, y.n)) return DSPARK_E_POINTER;
  st = check_pages(C, k_pool, v_pool, workspace, workspace_bytes);
  if (st != DSPARK_OK) return st;
  (void)hipGetLastError();
  PagesArgs a = pages_args(*C, table, length, ref, table_out, ref_out, n_short, workspace);
  a.parent = parent;
  a.new_len = new_len;
  a.length_out = length_out;
  return launch_cache_update(*C, a, k_pool, v_pool, stream) == hipSuccess ? DSPARK_OK : DSPARK_E_LAUNCH;
}

extern "C" dspark_status dspark_cache_compact(const dspark_cache* C, const int32_t* table, const int32_t* length,
                                              const int32_t* ref, int32_t* table_out, int32_t* ref_out,
                                              int32_t* n_live, void* k_pool, void* v_pool, void* workspace,
                                              size_t workspace_bytes, hipStream_t stream) {
  const AbiRange range("dspark_cache_compact");
  dspark_status st = check_cache(C);
  if (st != DSPARK_OK) return st;
  if (!table || !length || !ref || !table_out || !ref_out || !n_live) return DSPARK_E_POINTER;
  for (const void* p : {(const void*)table, (const void*)length, (const void*)ref, (const void*)table_out,
                        (const void*)ref_out, (const void*)n_live})
    if (!aligned(p, 4)) return DSPARK_E_POINTER;
  const size_t nb = (size_t)C->B * 4, nt = nb * C->max_pages, nr = (size_t)C->n_pages * 4;
  const struct { const void* p; size_t n; } in[] = {{table, nt}, {length, nb}, {ref, nr}},
      to[] = {{table_out, nt}, {ref_out, nr}, {n_live, 4}};
  for (const auto& x : in)
    for (const auto& y : to)
      if (overlap(x.p, x.n, y.p, y.n)) return DSPARK_E_POINTER;
  st = check_pages(C, k_pool, v_pool, workspace, workspace_bytes);
  if (st != DSPARK_OK) return st;
  (void)hipGetLastError();
  const PagesArgs a = pages_args(*C, table, length, ref, table_out, ref_out, n_live, workspace);
  return launch_cache_compact(*C, a, k_pool, v_pool, stream) == hipSuccess ? DSPARK_OK : DSPARK_E_LAUNCH;
}
