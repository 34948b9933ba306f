// Host-only driver of the argument validation of drafted trees and of caches whose tokens
// carry their own scales, built with AddressSanitizer over the ABI layers' host code
// (tests/test_tree_asan.py).  Every call below is rejected before any device work, or has
// nothing to do; the launchers are stubs that say so if one is reached.
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>

#include "../../draft_sampling_verification_markov_amd/csrc/dspark_cache_internal.hpp"
#include "../../include/dspark_tree.h"

static int failures = 0;

static void expect(const char* what, long long got, long long want) {
  if (got != want) {
    printf("FAIL %s: got %lld, want %lld\n", what, got, want);
    ++failures;
  }
}

namespace dspark {
static hipError_t reached(const char* what) {
  printf("FAIL launch of %s\n", what);
  ++failures;
  return hipErrorUnknown;
}
hipError_t launch_cache_append(const dspark_cache&, const AppendArgs&, hipStream_t) { return reached("append"); }
hipError_t launch_cache_attend(const dspark_cache&, const AttendArgs&, hipStream_t) { return reached("attend"); }
hipError_t launch_cache_update(const dspark_cache&, const PagesArgs&, void*, void*, hipStream_t) { return reached("update"); }
hipError_t launch_cache_compact(const dspark_cache&, const PagesArgs&, void*, void*, hipStream_t) { return reached("compact"); }
hipError_t launch_tree_attend(const dspark_cache&, const AttendArgs&, hipStream_t) { return reached("tree attend"); }
hipError_t launch_tree_mask(const TreeMaskArgs&, hipStream_t) { return reached("mask"); }
hipError_t launch_tree_keep(const dspark_cache&, const KeepArgs&, hipStream_t) { return reached("keep"); }
size_t attend_workspace_bytes(const dspark_cache&, int32_t) { return 4096; }
PagesLayout pages_layout(const dspark_cache&) {
  PagesLayout l{};
  l.total = 1024;
  return l;
}
}  // namespace dspark

// Arguments of the calls; addresses that validation accepts and never reads.
struct Args {
  const dspark_cache* C;
  int32_t B = 4, layer = 0, n_rows = 4, max_new = 3, window = 0, max_path = 2;
  int64_t q_stride = 1024, out_stride = 1024;
  float scale = 0.1f;
  size_t bytes = 4096;
  char *q, *out, *k_pool, *v_pool, *ws;
  int32_t *parent, *n_new, *row_start, *depth, *length, *table, *path, *n_keep, *length_out;
  uint32_t* mask;
  float *k_scale, *v_scale, *lse;

  explicit Args(const dspark_cache* c) : C(c) {
    uintptr_t at = (uintptr_t)1 << 40;
    auto next = [&] { return at += (uintptr_t)1 << 32; };
    for (char** p : {&q, &out, &k_pool, &v_pool, &ws}) *p = (char*)next();
    for (int32_t** p : {&parent, &n_new, &row_start, &depth, &length, &table, &path, &n_keep, &length_out}) *p = (int32_t*)next();
    mask = (uint32_t*)next();
    for (float** p : {&k_scale, &v_scale, &lse}) *p = (float*)next();
  }
  int tree_mask() const {
    return dspark_tree_mask(B, parent, n_rows, n_new, row_start, max_new, window, mask, depth, nullptr);
  }
  int attend() const {
    return dspark_tree_attend(C, layer, q, q_stride, n_rows, n_new, row_start, max_new, mask, depth, length, table, k_pool,
                              v_pool, k_scale, v_scale, scale, window, out, out_stride, lse, ws, bytes, nullptr);
  }
  int keep() const {
    return dspark_tree_keep(C, path, n_keep, max_path, n_new, max_new, length, table, length_out, k_pool, v_pool, nullptr);
  }
};

int main() {
  // in memory of its own size, so that a read past its end is seen
  dspark_cache* C = (dspark_cache*)malloc(sizeof(dspark_cache));
  const dspark_cache good = {4, 100, 16, 10, 2, 8, 2, 128, DSPARK_BF16, DSPARK_F8E4M3_TOKEN};
  *C = good;

  Args a(nullptr);
  expect("attend without a cache", a.attend(), DSPARK_E_POINTER);
  expect("keep without a cache", a.keep(), DSPARK_E_POINTER);

  for (int32_t dtype : {3, 5, -1, INT32_MAX, INT32_MIN}) {
    C->cache_dtype = dtype;
    a = Args(C);
    expect("attend type", a.attend(), DSPARK_E_DTYPE);
    expect("keep type", a.keep(), DSPARK_E_DTYPE);
    expect("workspace type", (long long)dspark_cache_workspace_bytes(C, 3), 0);
  }
  *C = good;
  C->data_dtype = DSPARK_F32;
  a = Args(C);
  expect("attend of fp32 data over quantised tokens", a.attend(), DSPARK_E_UNSUPPORTED);
  expect("keep of fp32 data over quantised tokens", a.keep(), DSPARK_E_UNSUPPORTED);
  *C = good;

  a = Args(C);
  a.n_rows = 0;
  a.mask = nullptr;
  a.parent = nullptr;
  expect("mask of no rows", a.tree_mask(), DSPARK_OK);
  expect("attend of no rows", a.attend(), DSPARK_OK);
  a = Args(C);
  a.k_scale = a.v_scale = nullptr;  // (not asked for)
  a.mask = nullptr;
  expect("attend without a mask", a.attend(), DSPARK_E_POINTER);
  a = Args(C);
  a.window = 1;
  a.depth = nullptr;
  expect("attend with a window, without depths", a.attend(), DSPARK_E_POINTER);
  a = Args(C);
  a.bytes = 4095;
  expect("attend's workspace", a.attend(), DSPARK_E_WORKSPACE);
  for (int32_t n : {0, -1, 1025, INT32_MAX}) {
    a = Args(C);
    a.max_new = n;
    expect("mask's nodes", a.tree_mask(), DSPARK_E_INVALID);
    a = Args(C);
    a.max_path = n;
    expect("keep's path", a.keep(), DSPARK_E_INVALID);
  }
  for (int32_t n : {0, (1 << 20) + 1, INT32_MIN}) {
    a = Args(C);
    a.max_new = n;
    expect("attend's nodes", a.attend(), DSPARK_E_INVALID);
    expect("keep's nodes", a.keep(), DSPARK_E_INVALID);
  }
  // the largest sizes: buffers' ends are computed without overflow
  a = Args(C);
  a.B = 65536;
  a.n_rows = INT32_MAX;
  a.max_new = 1024;
  a.parent = (int32_t*)((uintptr_t)1 << 50);
  a.depth = (int32_t*)((uintptr_t)1 << 51);
  a.mask = (uint32_t*)((uintptr_t)1 << 52);
  a.row_start = (int32_t*)((uintptr_t)a.mask + ((uintptr_t)INT32_MAX * 128) - 4);
  expect("mask over row_start", a.tree_mask(), DSPARK_E_POINTER);
  const dspark_cache large = {65536, 1 << 24, 16, 1 << 20, 1024, 1024, 1024, 256, DSPARK_BF16, DSPARK_F8E4M3_TOKEN};
  *C = large;
  expect("workspace of the largest cache", dspark_cache_workspace_bytes(C, 1 << 20) > 0, 1);
  a = Args(C);
  a.length_out = a.table + (size_t)65536 * (1 << 20) - 1;
  expect("keep over the table's end", a.keep(), DSPARK_E_POINTER);

  free(C);
  if (failures) return 1;
  printf("ok\n");
  return 0;
}
