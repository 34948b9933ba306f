// Paged cache: attention of each request's new tokens over its pages -- the choice of
// kernel and split.  See include/dspark_cache.h for the contract, attend_core.hpp for
// the mathematics.
#include "attend_keys.hpp"
#include "attend_rows.hpp"

namespace dspark {
namespace {

// Workgroups that the chip holds at once decide how many workers share the units.
struct Plan {
  Split split;
  int rows;     // of a tile
  int slots;    // partial results
};

constexpr int kDirectKeys = 1024;

int max_rows(const dspark_cache& C, int32_t max_new) { return max_new * (C.Hq / C.Hkv); }

Plan plan_for(const dspark_cache& C, int32_t max_new, int window, int rows, int unit_shift, int occupancy) {
  Plan pl{};
  pl.rows = rows;
  pl.split.row_tiles = (max_rows(C, max_new) + rows - 1) / rows;
  pl.split.unit_shift = unit_shift;
  long long keys = (long long)C.max_pages * C.page;
  if (window > 0 && (long long)window + max_new < keys) keys = (long long)window + max_new;
  const long long segments = (long long)C.B * pl.split.row_tiles * C.Hkv;
  // few keys a segment: nothing to share out
  const bool direct = keys <= kDirectKeys && segments <= (1 << 22);
  pl.split.workers = direct ? 0 : kCUs * occupancy;
  return pl;
}

template <int CT, int D, int NB, int OCC>
hipError_t run_keys(const dspark_cache& C, const AttendArgs& a, hipStream_t s) {
  const Plan pl = plan_for(C, a.c.max_new, a.window, NB * 32, 7, OCC);
  if (!pl.split.workers) {
    k_attend_keys<CT, D, NB, OCC><<<C.B * pl.split.row_tiles * C.Hkv, kAttendThreads, 0, s>>>(a, pl.split);
    return hipGetLastError();
  }
  k_attend_keys<CT, D, NB, OCC><<<pl.split.workers, kAttendThreads, 0, s>>>(a, pl.split);
  k_attend_join<CT, D, NB * 32><<<dim3(pl.split.workers, kJoinY), kAttendThreads, 0, s>>>(a, pl.split);
  return hipGetLastError();
}

template <int CT, int D, int NB, int OCC>
hipError_t run_rows(const dspark_cache& C, const AttendArgs& a, hipStream_t s) {
  constexpr int kRows = NB * 128;
  const Plan pl = plan_for(C, a.c.max_new, a.window, kRows, RowsShape<CT, D, NB>::kKeys == 64 ? 6 : 5, OCC);
  if (!pl.split.workers) {
    k_attend_rows<CT, D, NB, OCC><<<C.B * pl.split.row_tiles * C.Hkv, kAttendThreads, 0, s>>>(a, pl.split);
    return hipGetLastError();
  }
  k_attend_rows<CT, D, NB, OCC><<<pl.split.workers, kAttendThreads, 0, s>>>(a, pl.split);
  k_attend_join<CT, D, kRows><<<dim3(pl.split.workers, kJoinY), kAttendThreads, 0, s>>>(a, pl.split);
  return hipGetLastError();
}

template <int CT, int D>
hipError_t run(const dspark_cache& C, const AttendArgs& a, hipStream_t s) {
  const int rows = max_rows(C, a.c.max_new);
  constexpr int kOne = CT != DSPARK_F32 && D <= 128 ? 2 : 1;
  if (rows <= 32) return run_keys<CT, D, 1, kOne>(C, a, s);
  if constexpr (CT == DSPARK_F32) {
    return run_keys<CT, D, D == 256 ? 1 : 2, 1>(C, a, s);
  } else if constexpr (D == 256) {
    return run_rows<CT, D, 1, 1>(C, a, s);
  } else {
    if (rows <= 128) return run_rows<CT, D, 1, 2>(C, a, s);
    return run_rows<CT, D, 2, 1>(C, a, s);
  }
}

template <int CT>
hipError_t run_type(const dspark_cache& C, const AttendArgs& a, hipStream_t s) {
  return C.D == 64 ? run<CT, 64>(C, a, s) : C.D == 128 ? run<CT, 128>(C, a, s) : run<CT, 256>(C, a, s);
}

}  // namespace

size_t attend_workspace_bytes(const dspark_cache& C, int32_t max_new) {
  // the records and two partial results a worker: 2 workers a CU with up to 128 rows, one with up to 256
  const int rows = max_rows(C, max_new) <= 32 ? 32 : C.cache_dtype == DSPARK_F32 ? 64 : 128;
  return records_bytes(2 * kCUs) + (size_t)2 * 2 * kCUs * rows * (C.D + 2) * sizeof(float);
}

hipError_t launch_cache_attend(const dspark_cache& C, const AttendArgs& a, hipStream_t s) {
  switch (C.cache_dtype) {
    case DSPARK_F32: return run_type<DSPARK_F32>(C, a, s);
    case DSPARK_BF16: return run_type<DSPARK_BF16>(C, a, s);
    default: return run_type<DSPARK_F8E4M3>(C, a, s);
  }
}

}  // namespace dspark
