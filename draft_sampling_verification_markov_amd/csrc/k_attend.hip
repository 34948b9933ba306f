// Paged cache: attention of each request's new tokens over its pages.  See
// include/dspark_cache.h for the contract, attend_core.hpp for the mathematics,
// attend_launch.hpp for the choice of kernel and split.
#include "attend_launch.hpp"

namespace dspark {

size_t attend_workspace_bytes(const dspark_cache& C, int32_t max_new) {
  // the records and two partial results a worker
  const int workers = 2 * kCUs, rows = max_rows(C, max_new) <= 16 ? 16 : C.cache_dtype == DSPARK_F32 ? 32 : 128;
  return records_bytes(workers) + (size_t)2 * workers * rows * (C.D + 2) * sizeof(float);
}

hipError_t launch_cache_attend(const dspark_cache& C, const AttendArgs& a, hipStream_t s) {
  return launch_attend<false>(C, a, s);
}

}  // namespace dspark
