// Paged cache: what the ABI layers of dspark_cache.h and dspark_tree.h check alike.
#pragma once

#include <math.h>

#include "dspark_cache_internal.hpp"
#include "dspark_internal.hpp"

namespace dspark {
namespace {

bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

dspark_status check_cache(const dspark_cache* C) {
  if (!C) return DSPARK_E_POINTER;
  if (C->B < 1 || C->B > 65536 || C->n_pages < 1 || C->n_pages > (1 << 24) || C->n_layers < 1 || C->n_layers > 1024)
    return DSPARK_E_INVALID;
  if (C->page < 1 || C->max_pages < 1 || (long long)C->max_pages * C->page > (1 << 24)) return DSPARK_E_INVALID;
  if (C->Hkv < 1 || C->Hq < C->Hkv || C->Hq > 1024 || C->Hq % C->Hkv != 0 || C->D < 1) return DSPARK_E_INVALID;
  if (C->data_dtype != DSPARK_F32 && C->data_dtype != DSPARK_BF16) return DSPARK_E_DTYPE;
  if (C->cache_dtype != DSPARK_F32 && C->cache_dtype != DSPARK_BF16 && !is_f8(C->cache_dtype)) return DSPARK_E_DTYPE;
  if (C->page != 16 && C->page != 32 && C->page != 64 && C->page != 128 && C->page != 256) return DSPARK_E_UNSUPPORTED;
  if (C->D != 64 && C->D != 128 && C->D != 256) return DSPARK_E_UNSUPPORTED;
  if ((C->data_dtype == DSPARK_F32) != (C->cache_dtype == DSPARK_F32)) return DSPARK_E_UNSUPPORTED;
  return DSPARK_OK;
}

// largest max_new: rows are counted in 31 bits, also after the heads of a group are folded in
constexpr int32_t kMaxNew = 1 << 20;
constexpr long long kMaxTiles = 1 << 24;
// a window that hides nothing: positions lie in [-2^20, 2^24)
constexpr int32_t kNoWindow = 1 << 26;

// What append and attend have in common.  rows: strided arrays of `heads` heads.
dspark_status check_tokens(const dspark_cache& C, int32_t layer, int32_t n_rows, const int32_t* n_new,
                           const int32_t* row_start, int32_t max_new, const int32_t* length, const int32_t* table,
                           const void* k_pool, const void* v_pool, const float* k_scale, const float* v_scale) {
  if (layer < 0 || layer >= C.n_layers || n_rows < 0 || max_new < 1 || max_new > kMaxNew) return DSPARK_E_INVALID;
  if (!length || !table || !k_pool || !v_pool) return DSPARK_E_POINTER;
  if (C.cache_dtype == DSPARK_F8E4M3 && (!k_scale || !v_scale)) return DSPARK_E_POINTER;
  if (!aligned(k_pool, 16) || !aligned(v_pool, 16)) return DSPARK_E_POINTER;
  for (const void* p : {(const void*)n_new, (const void*)row_start, (const void*)length, (const void*)table,
                        (const void*)k_scale, (const void*)v_scale})
    if (!aligned(p, 4)) return DSPARK_E_POINTER;
  return DSPARK_OK;
}

// a strided array of n_rows rows of `width` elements, rows a multiple of 16 bytes apart
dspark_status check_rows(const void* x, int64_t stride, int64_t width, int32_t n_rows, int element) {
  if (!x || !aligned(x, 16)) return DSPARK_E_POINTER;
  if (n_rows > 1 && (stride < width || stride > ((int64_t)1 << 40) || (stride * element) % 16 != 0))
    return DSPARK_E_INVALID;
  return DSPARK_OK;
}

CacheView view(const dspark_cache& C, int32_t n_rows, const int32_t* n_new, const int32_t* row_start, int32_t max_new,
               const int32_t* length, const int32_t* table) {
  CacheView v{};
  v.n_new = n_new;
  v.row_start = row_start;
  v.length = length;
  v.table = table;
  v.B = C.B;
  v.n_pages = C.n_pages;
  v.page_shift = log2_page(C.page);
  v.max_pages = C.max_pages;
  v.Hq = C.Hq;
  v.Hkv = C.Hkv;
  v.max_new = max_new;
  v.n_rows = n_rows;
  return v;
}

// do [a, a + na) and [b, b + nb) share a byte?
bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
  return x < y + nb && y < x + na;
}

// What an attention over the cache checks, and its argument block (the mask of a tree aside).
// Nothing is left to do where n_rows is 0.
dspark_status attend_args(const dspark_cache* C, int32_t layer, const void* q, int64_t q_stride, int32_t n_rows,
                          const int32_t* n_new, const int32_t* row_start, int32_t max_new, const int32_t* length,
                          const int32_t* table, const void* k_pool, const void* v_pool, const float* k_scale,
                          const float* v_scale, float scale, int32_t causal, int32_t window, void* out,
                          int64_t out_stride, float* lse, void* workspace, size_t workspace_bytes, AttendArgs& a) {
  dspark_status st = check_cache(C);
  if (st != DSPARK_OK) return st;
  st = check_tokens(*C, layer, n_rows, n_new, row_start, max_new, length, table, k_pool, v_pool, k_scale, v_scale);
  if (st != DSPARK_OK) return st;
  const float scale2 = (float)((double)scale * 1.4426950408889634);  // times log2(e)
  if (!(scale > 0.0f) || !isfinite(scale2) || window < 0) return DSPARK_E_INVALID;
  // row tiles (of 16 rows or more) over which the workers look for their share
  if ((((long long)max_new * (C->Hq / C->Hkv) + 15) / 16) * C->B > kMaxTiles) return DSPARK_E_INVALID;
  if (!aligned(lse, 4)) return DSPARK_E_POINTER;
  if (!workspace || !aligned(workspace, 256) || workspace_bytes < dspark_cache_workspace_bytes(C, max_new))
    return DSPARK_E_WORKSPACE;
  if (n_rows == 0) return DSPARK_OK;
  const int es = element_bytes(C->data_dtype);
  st = check_rows(q, q_stride, (int64_t)C->Hq * C->D, n_rows, es);
  if (st == DSPARK_OK) st = check_rows(out, out_stride, (int64_t)C->Hq * C->D, n_rows, es);
  if (st != DSPARK_OK) return st;
  const size_t layer_bytes = page_bytes(*C) * C->n_pages;
  a = AttendArgs{};
  a.c = view(*C, n_rows, n_new, row_start, max_new, length, table);
  a.q = q;
  a.out = out;
  a.lse = lse;
  a.q_stride = q_stride;
  a.out_stride = out_stride;
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  a.k_pool = static_cast<const char*>(k_pool) + layer * layer_bytes;
  a.v_pool = static_cast<const char*>(v_pool) + layer * layer_bytes;
  a.scale2 = scale2;
  a.causal = causal != 0;
  a.window = window < kNoWindow ? window : kNoWindow;
  a.workspace = workspace;
  return DSPARK_OK;
}

}  // namespace
}  // namespace dspark
