// Paged cache: attention of each request's new tokens over its pages -- the choice of
// kernel and split.  See include/dspark_cache.h for the contract, attend_core.hpp for
// the mathematics.
#include "attend_keys.hpp"
#include "attend_rows.hpp"

namespace dspark {
namespace {

int max_rows(const dspark_cache& C, int32_t max_new) { return max_new * (C.Hq / C.Hkv); }

// Whole segments or dealt units.  Whole segments need no partial results, and the row
// tiles of a head run side by side through one L2; but they leave the chip idle where they
// are few or of unequal length.  Whole are:
//   segments of few keys, where partial results would cost more than a longer loop (120
//     segments of 128 rows over 969 keys, head size 128: 24 us whole, 34 dealt; 128
//     segments of a token over 900 keys 15 / 22);
//   `whole` segments or more;
//   with several row tiles a head, whose lengths differ little, one a CU and not many keys
//     (376 segments of 128 rows over 4096 keys 96 / 105, over 1500 43 / 75; 352 over 16000
//     354 / 320).
// Whole segments of unequal length end at unequal times: where they do not all run at once,
// the longest requests go first (100 requests of up to 17 rows over up to 3000 keys 103 ->
// 78 us, 256 over 2048 192 -> 184, 8 x 300 rows fp32 over 2000 279 -> 230); each workgroup
// counts out its request, about 1 us, so not for few keys, nor with a window.
// The host knows no lengths: a segment's keys are what its request's row of the page table
// (or the window) holds, its rows what max_new allows.  Short requests in a long table are
// dealt out (16 tokens over 500 keys 11.8 us, in rows of 131072 tokens 18.8; 64 x 17 rows
// over 1000 52.0 / 53.4), and one prompt of 2048 rows among 255 tokens has the row tiles of
// all of them launched (1957 us; in calls of their own 121 + 391).
// Dealt ones go to one worker a CU, or to two where there are enough keys (`twice`): the
// second hides the other's waits, but doubles the partial results and halves their shares.
constexpr int kFewKeys = 1024, kSomeKeys = 4096;
struct Rule {
  int few;          // keys of a segment, of fewer than half as many as CUs (kFewKeys for more)
  long long whole;  // segments
  long long twice;  // keys of all segments
};
// Keys that a request can see, from what the host knows: its row of the page table, or the window.
long long most_keys(const dspark_cache& C, int32_t max_new, int window) {
  const long long row = (long long)C.max_pages * C.page, seen = (long long)window + max_new;
  return window > 0 && seen < row ? seen : row;
}
Split plan_for(const dspark_cache& C, int32_t max_new, int window, int rows, int unit_shift, int per_cu, const Rule& r) {
  Split pl{};
  pl.row_tiles = (max_rows(C, max_new) + rows - 1) / rows;
  pl.unit_shift = unit_shift;
  const long long keys = most_keys(C, max_new, window);
  const long long segments = (long long)C.B * pl.row_tiles * C.Hkv;
  const bool direct = segments <= (1 << 22) && (keys <= (segments < kCUs / 2 ? r.few : kFewKeys) || segments >= r.whole ||
                                                (pl.row_tiles > 1 && segments >= kCUs && keys <= kSomeKeys));
  pl.longest_first = C.B > 1 && C.B <= kAttendThreads && segments > 2 * kCUs && keys > kFewKeys && window == 0;
  pl.workers = direct ? 0 : per_cu > 1 && segments * keys >= r.twice ? 2 * kCUs : kCUs;
  return pl;
}

// Keys that one workgroup reads, and that the 256 MB last-level cache does not hold until
// the next call, are read with the streaming policy: 256 requests x 17 rows 191 -> 182 us,
// 256 x 1 402 -> 374.  For others it costs: prompts, whose row tiles meet in L2, 563 -> 589,
// 64 tokens over 2000 keys x 2 heads (72 MB) 27.8 -> 29.6, a window of 512 keys of 64
// requests x 8 heads in a pool of 2 GB 25.9 -> 27.9.  How much a call reads at most, from
// what the host knows: the pool, or what its requests can see.
bool read_once(const dspark_cache& C, const Split& pl, int32_t max_new, int window) {
  const size_t page = 2 * page_bytes(C), pool = page * C.n_pages;
  const size_t seen = page / C.page * C.B * (size_t)most_keys(C, max_new, window);
  return pl.row_tiles == 1 && (seen < pool ? seen : pool) > ((size_t)256 << 20);
}

template <int CT, int D, int ROWS, typename Kernel>
hipError_t run_plan(const dspark_cache& C, const AttendArgs& a, Split pl, Kernel kernel, hipStream_t s) {
  if (!pl.workers) {
    const int grid = whole_grid(C, pl);
    kernel<<<grid, kAttendThreads, 0, s>>>(a, pl);
    return hipGetLastError();
  }
  kernel<<<pl.workers, kAttendThreads, 0, s>>>(a, pl);
  k_attend_join<CT, D, ROWS><<<dim3(pl.workers, join_groups(ROWS)), kAttendThreads, 0, s>>>(a, pl);
  return hipGetLastError();
}

template <int CT, int D, int NB, int OCC>
hipError_t run_keys(const dspark_cache& C, const AttendArgs& a, hipStream_t s) {
  // `few`: wide fp32 products make the loop longer: 32 segments of 1000 keys, head size 256,
  // 46 us whole, 24 dealt, but 512 segments of 900 keys 121 / 126, head size 128 61 / 72.
  // `twice`: for a few rows (memory bound) one worker a CU suffices for long: a token over
  // 20000 keys 15.9 us with one, 18.8 with two, 3 requests over 150000 keys x 4 heads
  // 108 / 111, 200 over 3000 x 8 heads 250 / 244; for more rows, 608 segments of 3000 keys,
  // 133 / 111.
  // `whole`: as many as the chip holds, where the longest go first (256 tokens over up to
  // 4096 keys x 8 heads 375 us whole, 402 dealt; 256 over 2000 x 4, e4m3, 58 / 84); many more
  // where they cannot be ordered.
  constexpr int kHeld = (OCC > 2 ? OCC : 2) * kCUs;
  const Rule rule{CT == DSPARK_F32 && D >= 128 ? kFewKeys / 2 : kFewKeys, C.B <= kAttendThreads ? kHeld : 16 * kHeld,
                  NB == 1 ? 1 << 22 : 1 << 20};
  const Split pl = plan_for(C, a.c.max_new, a.window, NB * 16, 7, OCC, rule);
  const bool once = read_once(C, pl, a.c.max_new, a.window);
  return run_plan<CT, D, NB * 16>(
      C, a, pl, once ? k_attend_keys<CT, D, NB, OCC, NB == 1> : k_attend_keys<CT, D, NB, OCC, false>, s);
}

template <int CT, int D>
hipError_t run_rows(const dspark_cache& C, const AttendArgs& a, hipStream_t s) {
  using S = RowsShape<CT, D>;
  // `twice`: 12 segments of 17123 keys 42 us with one worker a CU, 50 with two; 20 of 132768
  // 159 / 115
  constexpr Rule kRule{kFewKeys, 2 * kCUs, 1 << 20};
  const Split pl = plan_for(C, a.c.max_new, a.window, S::kRows, S::kKeys == 64 ? 6 : 5, 2, kRule);
  const bool once = read_once(C, pl, a.c.max_new, a.window);
  return run_plan<CT, D, S::kRows>(C, a, pl, once ? k_attend_rows<CT, D, true> : k_attend_rows<CT, D, false>, s);
}

// Workgroups of k_attend_keys that a CU holds, by their registers.
template <int CT, int D, int NB>
constexpr int keys_per_cu() {
  if (CT == DSPARK_F32) return D == 64 ? 5 - NB : D == 128 ? 2 : 1;
  return D == 64 ? 4 : D == 128 ? 3 : 2;
}

template <int CT, int D>
hipError_t run(const dspark_cache& C, const AttendArgs& a, hipStream_t s) {
  const int rows = max_rows(C, a.c.max_new);
  if (rows <= 16) return run_keys<CT, D, 1, keys_per_cu<CT, D, 1>()>(C, a, s);
  if constexpr (CT == DSPARK_F32) {
    // fp32 products take 8 to 16 times as long as bf16 ones: no kernel that shares loads
    // through LDS is needed.  32 rows a workgroup read the keys half as often as 16, with
    // fewer workgroups a CU; head size 128: where they fill the chip (1024 rows x 4 heads
    // over 4096 keys 294 us against 343), not for fewer (482 rows over 1302 keys 70 against
    // 64); head size 256: no room.
    constexpr int kNB = D == 256 ? 1 : 2, kOcc = keys_per_cu<CT, D, kNB>();
    if (D == 64 || (long long)C.B * C.Hkv * ((rows + 31) / 32) >= kOcc * kCUs) return run_keys<CT, D, kNB, kOcc>(C, a, s);
    return run_keys<CT, D, 1, keys_per_cu<CT, D, 1>()>(C, a, s);
  } else {
    // (k_attend_keys with 32 rows: 256 requests of 28 rows over 2000 keys 226 us against 172,
    // 8 of 32 rows 29 against 24; only at 20 rows it gains a little, 40 against 42)
    return run_rows<CT, D>(C, a, s);
  }
}

template <int CT>
hipError_t run_type(const dspark_cache& C, const AttendArgs& a, hipStream_t s) {
  return C.D == 64 ? run<CT, 64>(C, a, s) : C.D == 128 ? run<CT, 128>(C, a, s) : run<CT, 256>(C, a, s);
}

}  // namespace

size_t attend_workspace_bytes(const dspark_cache& C, int32_t max_new) {
  // the records and two partial results a worker
  const int workers = 2 * kCUs, rows = max_rows(C, max_new) <= 16 ? 16 : C.cache_dtype == DSPARK_F32 ? 32 : 128;
  return records_bytes(workers) + (size_t)2 * workers * rows * (C.D + 2) * sizeof(float);
}

hipError_t launch_cache_attend(const dspark_cache& C, const AttendArgs& a, hipStream_t s) {
  switch (C.cache_dtype) {
    case DSPARK_F32: return run_type<DSPARK_F32>(C, a, s);
    case DSPARK_BF16: return run_type<DSPARK_BF16>(C, a, s);
    default: return run_type<DSPARK_F8E4M3>(C, a, s);
  }
}

}  // namespace dspark
