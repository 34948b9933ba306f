// Host-only driver of the paged cache's argument validation, built with
// AddressSanitizer over the cache's host code (tests/test_cache_asan.py).  Every
// call below is rejected before any device work, or has no rows.  The driver
// checks each status and prints "ok" at the end; AddressSanitizer reports any
// invalid memory access in the validation code itself.
#include <math.h>
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>

#include "../../include/dspark_cache.h"

static int failures = 0;

static void expect(const char* what, long long got, long long want) {
  if (got != want) {
    printf("FAIL %s: got %lld, want %lld\n", what, got, want);
    ++failures;
  }
}

// The arguments of all four calls; addresses that validation accepts and never reads.
struct Args {
  const dspark_cache* C;
  int32_t layer = 0, n_rows = 4, max_new = 3, window = 0;
  int64_t k_stride = 256, v_stride = 256, q_stride = 1024, out_stride = 1024;
  float scale = 0.1f;
  size_t bytes = (size_t)1 << 32;
  char *k, *v, *q, *out, *k_pool, *v_pool, *ws;
  int32_t *n_new, *row_start, *length, *table, *ref, *new_len, *parent, *table_out, *length_out, *ref_out, *count;
  float *k_scale, *v_scale, *lse;

  explicit Args(const dspark_cache* c) : C(c) {
    uintptr_t at = (uintptr_t)1 << 40;
    auto next = [&] { return at += (uintptr_t)1 << 32; };
    for (char** p : {&k, &v, &q, &out, &k_pool, &v_pool, &ws}) *p = (char*)next();
    for (int32_t** p : {&n_new, &row_start, &length, &table, &ref, &new_len, &parent, &table_out, &length_out, &ref_out,
                        &count})
      *p = (int32_t*)next();
    for (float** p : {&k_scale, &v_scale, &lse}) *p = (float*)next();
  }
  int append() const {
    return dspark_cache_append(C, layer, k, k_stride, v, v_stride, n_rows, n_new, row_start, max_new, length, table,
                               k_scale, v_scale, k_pool, v_pool, nullptr);
  }
  int attend() const {
    return dspark_cache_attend(C, layer, q, q_stride, n_rows, n_new, row_start, max_new, length, table, k_pool, v_pool,
                               k_scale, v_scale, scale, 1, window, out, out_stride, lse, ws, bytes, nullptr);
  }
  int update() const {
    return dspark_cache_update(C, parent, new_len, table, length, ref, table_out, length_out, ref_out, count, k_pool,
                               v_pool, ws, bytes, nullptr);
  }
  int compact() const {
    return dspark_cache_compact(C, table, length, ref, table_out, ref_out, count, k_pool, v_pool, ws, bytes, nullptr);
  }
  void all(const char* what, int want) const {
    expect(what, append(), want);
    expect(what, attend(), want);
    expect(what, update(), want);
    expect(what, compact(), want);
  }
};

int main() {
  // on the heap, of its exact size: a read past the struct is seen
  dspark_cache* C = (dspark_cache*)malloc(sizeof(dspark_cache));
  const dspark_cache good = {4, 100, 16, 10, 2, 8, 2, 128, DSPARK_BF16, DSPARK_BF16};
  *C = good;
  expect("workspace", dspark_cache_workspace_bytes(C, 3) > 0, 1);
  expect("workspace of no rows", dspark_cache_workspace_bytes(C, 0), 0);
  expect("workspace of no cache", dspark_cache_workspace_bytes(nullptr, 3), 0);
  Args(nullptr).all("no cache", DSPARK_E_POINTER);

  const struct {
    int32_t dspark_cache::*field;
    int32_t value;
    int want;
  } bad[] = {{&dspark_cache::B, 0, DSPARK_E_INVALID},           {&dspark_cache::B, 65537, DSPARK_E_INVALID},
             {&dspark_cache::n_pages, -1, DSPARK_E_INVALID},    {&dspark_cache::n_pages, INT32_MAX, DSPARK_E_INVALID},
             {&dspark_cache::page, 0, DSPARK_E_INVALID},        {&dspark_cache::page, 24, DSPARK_E_UNSUPPORTED},
             {&dspark_cache::max_pages, INT32_MAX, DSPARK_E_INVALID}, {&dspark_cache::max_pages, 0, DSPARK_E_INVALID},
             {&dspark_cache::n_layers, 1025, DSPARK_E_INVALID}, {&dspark_cache::Hq, INT32_MIN, DSPARK_E_INVALID},
             {&dspark_cache::Hq, 9, DSPARK_E_INVALID},          {&dspark_cache::Hkv, 0, DSPARK_E_INVALID},
             {&dspark_cache::D, 96, DSPARK_E_UNSUPPORTED},      {&dspark_cache::D, INT32_MIN, DSPARK_E_INVALID},
             {&dspark_cache::data_dtype, 7, DSPARK_E_DTYPE},    {&dspark_cache::cache_dtype, -1, DSPARK_E_DTYPE},
             {&dspark_cache::data_dtype, DSPARK_F32, DSPARK_E_UNSUPPORTED}};
  for (const auto& b : bad) {
    *C = good;
    C->*b.field = b.value;
    Args(C).all("geometry", b.want);
    expect("workspace of a bad geometry", dspark_cache_workspace_bytes(C, 3), 0);
  }

  *C = good;
  Args a(C);
  a.length = nullptr;
  a.all("no lengths", DSPARK_E_POINTER);
  a = Args(C);
  a.k_pool += 8;
  a.all("a pool off its alignment", DSPARK_E_POINTER);
  for (int32_t layer : {-1, 2, INT32_MAX}) {
    a = Args(C);
    a.layer = layer;
    expect("append layer", a.append(), DSPARK_E_INVALID);
    expect("attend layer", a.attend(), DSPARK_E_INVALID);
  }
  for (int64_t stride : {(int64_t)255, (int64_t)0, (int64_t)-1024, INT64_MAX, INT64_MIN, ((int64_t)1 << 40) + 8}) {
    a = Args(C);
    a.k_stride = stride;
    expect("k stride", a.append(), DSPARK_E_INVALID);
    a = Args(C);
    a.v_stride = stride;
    expect("v stride", a.append(), DSPARK_E_INVALID);
    a = Args(C);
    a.q_stride = stride;
    expect("q stride", a.attend(), DSPARK_E_INVALID);
    a = Args(C);
    a.out_stride = stride;
    expect("out stride", a.attend(), DSPARK_E_INVALID);
  }
  for (float scale : {0.0f, -1.0f, INFINITY, NAN, 3e38f}) {
    a = Args(C);
    a.scale = scale;
    expect("scale", a.attend(), DSPARK_E_INVALID);
  }
  a = Args(C);
  a.window = INT32_MIN;
  expect("window", a.attend(), DSPARK_E_INVALID);
  a = Args(C);
  a.n_rows = -1;
  expect("append rows", a.append(), DSPARK_E_INVALID);
  expect("attend rows", a.attend(), DSPARK_E_INVALID);
  a.n_rows = 0;
  a.k = a.v = a.q = a.out = nullptr;
  expect("append of no rows", a.append(), DSPARK_OK);
  expect("attend of no rows", a.attend(), DSPARK_OK);
  for (size_t bytes : {(size_t)0, dspark_cache_workspace_bytes(C, 3) - 1}) {
    a = Args(C);
    a.bytes = bytes;
    expect("attend workspace", a.attend(), DSPARK_E_WORKSPACE);
  }
  a = Args(C);
  a.bytes = 255;
  expect("update workspace", a.update(), DSPARK_E_WORKSPACE);
  expect("compact workspace", a.compact(), DSPARK_E_WORKSPACE);
  a = Args(C);
  a.table_out = a.table + 39;  // the last entry
  expect("update over its input", a.update(), DSPARK_E_POINTER);
  expect("compact over its input", a.compact(), DSPARK_E_POINTER);
  a = Args(C);
  a.count = a.ref + 99;
  expect("update's count over its input", a.update(), DSPARK_E_POINTER);
  expect("compact's count over its input", a.compact(), DSPARK_E_POINTER);

  C->cache_dtype = DSPARK_F8E4M3;
  a = Args(C);
  a.v_scale = nullptr;
  expect("append without a scale", a.append(), DSPARK_E_POINTER);
  expect("attend without a scale", a.attend(), DSPARK_E_POINTER);

  // the largest sizes that a cache may have: the sizes of buffers are computed without overflow
  const dspark_cache large = {65536, 1 << 24, 16, 1 << 20, 1024, 1024, 1024, 256, DSPARK_F32, DSPARK_F32};
  *C = large;
  expect("workspace of the largest cache", dspark_cache_workspace_bytes(C, 1 << 20) > ((size_t)1 << 27), 1);
  a = Args(C);
  a.max_new = 1 << 20;
  expect("attend of the most rows", a.attend(), DSPARK_E_INVALID);

  free(C);
  if (failures) return 1;
  printf("ok\n");
  return 0;
}
