// Internal interfaces of the paged cache: argument blocks and launchers shared by the ABI
// layers (dspark_cache_abi.hip, dspark_tree_abi.hip) and the kernels (k_pages.hip,
// k_attend.hip, k_attend_tree.hip, k_tree.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/dspark_cache.h"
#include "dspark_device.hpp"

namespace dspark {

constexpr size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

inline int element_bytes(int dtype) { return dtype == DSPARK_F32 ? 4 : dtype == DSPARK_BF16 ? 2 : 1; }
constexpr bool is_f8(int dtype) { return dtype == DSPARK_F8E4M3 || dtype == DSPARK_F8E4M3_TOKEN; }
// bytes of a token's scale, which follow the entries of its page and head
constexpr int scale_bytes(int dtype) { return dtype == DSPARK_F8E4M3_TOKEN ? 4 : 0; }
// bytes of one page in one layer of one pool
inline size_t page_bytes(const dspark_cache& C) {
  return (size_t)C.Hkv * C.page * (C.D * element_bytes(C.cache_dtype) + scale_bytes(C.cache_dtype));
}
inline int log2_page(int page) { return 31 - __builtin_clz((unsigned)page); }

// The sequences' geometry, as every kernel clamps it.
struct CacheView {
  const int32_t* n_new;      // or null
  const int32_t* row_start;  // or null
  const int32_t* length;
  const int32_t* table;
  int32_t B, n_pages, page_shift, max_pages, Hq, Hkv, max_new, n_rows;

  __device__ __forceinline__ int len(int b) const {
    const int cap = max_pages << page_shift, l = length[b];
    return l < 0 ? 0 : l > cap ? cap : l;
  }
  __device__ __forceinline__ int rows(int b) const {
    if (!n_new) return max_new;
    const int n = n_new[b];
    return n < 0 ? 0 : n > max_new ? max_new : n;
  }
  __device__ __forceinline__ long long first_row(int b) const {
    return row_start ? (long long)row_start[b] : (long long)b * max_new;
  }
  __device__ __forceinline__ bool has_row(long long r) const { return r >= 0 && r < n_rows; }
};

// ---- k_pages.hip
struct AppendArgs {
  CacheView c;
  const void *k, *v;
  long long k_stride, v_stride;  // elements
  const float *k_scale, *v_scale;
  void *k_pool, *v_pool;  // of the layer
};
hipError_t launch_cache_append(const dspark_cache& C, const AppendArgs& a, hipStream_t s);

// Pages of one block of the free-page scan.
constexpr int kPageBlock = 1024;
inline int page_blocks(int n_pages) { return (n_pages + kPageBlock - 1) / kPageBlock; }

struct PagesArgs {
  const int32_t *parent, *new_len;  // update only; parent may be null
  const int32_t *table, *length, *ref;
  int32_t *table_out, *length_out, *ref_out;
  int32_t* count;  // update: n_short; compact: n_live
  // workspace
  int32_t *block_count;      // [page_blocks]
  int32_t *need, *base;      // [B]
  int32_t *ids;              // [n_pages]: the free ids in order (update); the holes (compact)
  int32_t *src, *dst;        // copies, -1: none ([B] for update, [n_pages] for compact)
  int32_t *rank;             // [n_pages], compact
  int32_t *n_copies;         // compact
  int32_t B, n_pages, page_shift, max_pages;
};
struct PagesLayout {
  size_t block_count, need, base, ids, src, dst, rank, n_copies, total;
};
PagesLayout pages_layout(const dspark_cache& C);
hipError_t launch_cache_update(const dspark_cache& C, const PagesArgs& a, void* k_pool, void* v_pool, hipStream_t s);
hipError_t launch_cache_compact(const dspark_cache& C, const PagesArgs& a, void* k_pool, void* v_pool, hipStream_t s);

// ---- k_attend.hip
struct AttendArgs {
  CacheView c;
  const void* q;
  void* out;
  float* lse;  // or null
  long long q_stride, out_stride;  // elements
  const float *k_scale, *v_scale;
  const void *k_pool, *v_pool;  // of the layer
  float scale2;                 // softmax scale * log2(e)
  int32_t causal, window;
  void* workspace;
  // a tree's nodes (null otherwise)
  const uint32_t* mask;  // [n_rows][mask_words]
  const int32_t* depth;  // [n_rows], or null without a window
  int32_t mask_words;
};
size_t attend_workspace_bytes(const dspark_cache& C, int32_t max_new);
hipError_t launch_cache_attend(const dspark_cache& C, const AttendArgs& a, hipStream_t s);

// ---- k_attend_tree.hip
hipError_t launch_tree_attend(const dspark_cache& C, const AttendArgs& a, hipStream_t s);

// ---- k_tree.hip
struct TreeMaskArgs {
  const int32_t *parent, *n_new, *row_start;  // n_new, row_start: or null
  uint32_t* mask;                             // [n_rows][words]
  int32_t* depth;                             // or null
  int32_t B, n_rows, max_new, window, words;
};
constexpr int kMaxNodes = 1024;
hipError_t launch_tree_mask(const TreeMaskArgs& a, hipStream_t s);

struct KeepArgs {
  CacheView c;
  const int32_t *path, *n_keep;  // [B][max_path], [B]
  int32_t* length_out;
  char *k_pool, *v_pool;
  size_t layer_bytes;
  int32_t max_path;
};
constexpr int kMaxPath = 1024;
hipError_t launch_tree_keep(const dspark_cache& C, const KeepArgs& a, hipStream_t s);

}  // namespace dspark
