// Paged cache: writing tokens into pages (append), and the bookkeeping of pages
// (update: fork, grow, shrink, free, private copies; compact).  See
// include/dspark_cache.h for the contract.
//
// The page bookkeeping is integer work over the table, the lengths and the
// reference counts; every result is independent of the order in which workgroups
// or atomics run (sums of references, ranks from prefix sums, lowest free ids
// first).  Device-wide dependencies are launch boundaries: a launch of the next
// kernel costs about 2 us on the stream, a grid barrier over 8 XCDs no less.
#include <type_traits>

#include "dspark_cache_internal.hpp"

namespace dspark {
namespace {

constexpr int kThreads = 256;

// ------------------------------------------------------------------ append
// e4m3 bits of x (round to nearest, ties to even; past +-448: +-448; NaN: NaN)
__device__ __forceinline__ uint32_t f8_pair(float x, float y) {
  x = x != x ? x : fminf(fmaxf(x, -448.f), 448.f);
  y = y != y ? y : fminf(fmaxf(y, -448.f), 448.f);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(x, y, 0, false) & 0xFFFFu;
}

// One thread carries 2 coordinates of the 8 tokens of a value group (the v_pool's
// unit [D][8]): it reads 8 rows, neighbouring threads neighbouring coordinates, and
// writes 2 x 8 tokens, so a full group leaves as whole 16-byte pieces and a single
// token as 2-element stores inside one 8 * D element region.  The keys of the
// same 8 tokens are copied row by row.  Bound by the bytes of the new rows (read
// once, written once); for a few tokens by the latency of table -> page -> store.
template <int CT>
struct CacheType;
template <>
struct CacheType<DSPARK_F32> { using T = uint32_t; };
template <>
struct CacheType<DSPARK_BF16> { using T = uint16_t; };
template <>
struct CacheType<DSPARK_F8E4M3> { using T = uint8_t; };

// two neighbouring data elements, and what the cache stores for them
template <int CT>
struct DataPair {
  using T = typename std::conditional<CT == DSPARK_F32, uint2, uint32_t>::type;
  __device__ __forceinline__ static T load(const void* x, long long i) {
    return *reinterpret_cast<const T*>(static_cast<const char*>(x) + i * (CT == DSPARK_F32 ? 4 : 2));
  }
};
template <int CT>
__device__ __forceinline__ void store_type(const typename DataPair<CT>::T& w, float scale,
                                           typename CacheType<CT>::T (&o)[2]) {
  if constexpr (CT == DSPARK_F32) {
    o[0] = w.x;
    o[1] = w.y;
  } else if constexpr (CT == DSPARK_BF16) {
    o[0] = (uint16_t)w;
    o[1] = (uint16_t)(w >> 16);
  } else {
    const uint32_t p = f8_pair(bf16_lo(w) / scale, bf16_hi(w) / scale);
    o[0] = (uint8_t)p;
    o[1] = (uint8_t)(p >> 8);
  }
}

template <int CT, int D>
__device__ __forceinline__ void append_group(const AppendArgs& a, int b, int gi) {
  using T = typename CacheType<CT>::T;
  constexpr int kPerHead = D / 2;  // threads of one head
  const CacheView& c = a.c;
  const int n = c.rows(b), len = c.len(b);
  const int pos0 = len - n;                       // of token 0; may be negative
  const int first = pos0 < 0 ? 0 : pos0;
  const int j0 = ((first >> 3) + gi) << 3;        // the group's first position
  const int lo = j0 > first ? j0 : first, hi = j0 + 8 < len ? j0 + 8 : len;
  if (n == 0 || lo >= hi) return;
  const int head = blockIdx.y * (kThreads / kPerHead) + threadIdx.x / kPerHead;
  if (head >= c.Hkv) return;
  const int d = (threadIdx.x % kPerHead) * 2;
  const int page = c.table[(size_t)b * c.max_pages + (j0 >> c.page_shift)];
  if ((unsigned)page >= (unsigned)c.n_pages) return;
  const int off = j0 & ((1 << c.page_shift) - 1);
  const size_t block = ((size_t)page * c.Hkv + head) << c.page_shift;  // tokens
  T* const kd = static_cast<T*>(a.k_pool) + (block + off) * D + d;
  T* const vd = static_cast<T*>(a.v_pool) + (block + off) * D + (size_t)d * 8;
  const float ks = CT == DSPARK_F8E4M3 ? a.k_scale[head] : 1.f, vs = CT == DSPARK_F8E4M3 ? a.v_scale[head] : 1.f;
  const long long row0 = c.first_row(b) + (j0 - pos0);
  // all loads at once: rows that are not there are read as the nearest one that is
  typename DataPair<CT>::T kw[8], vw[8];
  bool has[8], all = true;
#pragma unroll
  for (int t = 0; t < 8; ++t) {
    const long long r = row0 + t, near = row0 + min(max(t, lo - j0), hi - 1 - j0);
    has[t] = j0 + t >= lo && j0 + t < hi && c.has_row(r);
    all = all && has[t];
    const long long safe = near < 0 ? 0 : near < c.n_rows ? near : c.n_rows - 1;
    kw[t] = DataPair<CT>::load(a.k, safe * a.k_stride + head * D + d);
    vw[t] = DataPair<CT>::load(a.v, safe * a.v_stride + head * D + d);
  }
  T kx[8][2], vx[8][2];
#pragma unroll
  for (int t = 0; t < 8; ++t) {
    store_type<CT>(kw[t], ks, kx[t]);
    store_type<CT>(vw[t], vs, vx[t]);
  }
#pragma unroll
  for (int t = 0; t < 8; ++t)
    if (has[t]) {
      if constexpr (CT == DSPARK_F32)
        *reinterpret_cast<uint2*>(kd + t * D) = make_uint2(kx[t][0], kx[t][1]);
      else if constexpr (CT == DSPARK_BF16)
        *reinterpret_cast<uint32_t*>(kd + t * D) = kx[t][0] | (uint32_t)kx[t][1] << 16;
      else
        *reinterpret_cast<uint16_t*>(kd + t * D) = (uint16_t)(kx[t][0] | kx[t][1] << 8);
    }
  if (all) {
    T line[16];
#pragma unroll
    for (int t = 0; t < 8; ++t) {
      line[t] = vx[t][0];
      line[8 + t] = vx[t][1];
    }
    constexpr int kPieces = (int)sizeof(line) / 16;
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      uint4 w;
      __builtin_memcpy(&w, reinterpret_cast<const char*>(line) + 16 * i, 16);
      reinterpret_cast<uint4*>(vd)[i] = w;
    }
  } else {
#pragma unroll
    for (int t = 0; t < 8; ++t)
      if (has[t]) {
        vd[t] = vx[t][0];
        vd[8 + t] = vx[t][1];
      }
  }
}

// 8-token groups that a request's new positions can touch
int append_groups(const dspark_cache& C, const CacheView& v) {
  long long n = v.max_new;
  const long long cap = (long long)C.max_pages * C.page;
  n = n < cap ? n : cap;
  return (int)((n + 14) >> 3);
}

template <int CT, int D>
__global__ __launch_bounds__(kThreads) void k_append(AppendArgs a, int groups) {
  for (long long u = blockIdx.x; u < (long long)a.c.B * groups; u += gridDim.x)
    append_group<CT, D>(a, (int)(u / groups), (int)(u % groups));
}

template <int CT>
hipError_t append_typed(const dspark_cache& C, const AppendArgs& a, hipStream_t s) {
  const int groups = append_groups(C, a.c);
  const long long units = (long long)C.B * groups;
  const dim3 grid(units < 65536 ? (unsigned)units : 65536u, (C.Hkv * (C.D / 2) + kThreads - 1) / kThreads);
  if (C.D == 64)
    k_append<CT, 64><<<grid, kThreads, 0, s>>>(a, groups);
  else if (C.D == 128)
    k_append<CT, 128><<<grid, kThreads, 0, s>>>(a, groups);
  else
    k_append<CT, 256><<<grid, kThreads, 0, s>>>(a, groups);
  return hipGetLastError();
}

// ------------------------------------------------------------------ block scans
// Sum over the workgroup (every thread gets it); sh holds one int per wave.
__device__ __forceinline__ int block_sum(int v, int* sh) {
  for (int o = 32; o; o >>= 1) v += __shfl_xor(v, o);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = v;
  __syncthreads();
  int t = 0;
  for (int w = 0; w < (int)(blockDim.x >> 6); ++w) t += sh[w];
  return t;
}
// Exclusive prefix over the workgroup; total receives the sum.
__device__ __forceinline__ int block_prefix(int v, int* sh, int& total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int x = v;
  for (int o = 1; o < 64; o <<= 1) {
    const int y = __shfl_up(x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();
  if (lane == 63) sh[wave] = x;
  __syncthreads();
  int before = 0;
  total = 0;
  for (int w = 0; w < (int)(blockDim.x >> 6); ++w) {
    if (w < wave) before += sh[w];
    total += sh[w];
  }
  return before + x - v;
}

// A slot's present sequence and its next one, before pages are given out.
struct Slot {
  int source;  // row of the kept pages
  int keep, kept, old, want, next;
};
__device__ __forceinline__ int clamp_len(const PagesArgs& a, int l) {
  const int cap = a.max_pages << a.page_shift;
  return l < 0 ? 0 : l > cap ? cap : l;
}
__device__ __forceinline__ int pages_of(const PagesArgs& a, int tokens) {
  return (tokens + (1 << a.page_shift) - 1) >> a.page_shift;
}
__device__ __forceinline__ Slot slot_of(const PagesArgs& a, int b) {
  Slot s;
  s.next = clamp_len(a, a.new_len[b]);
  const int p = a.parent ? a.parent[b] : b;
  const bool has = (unsigned)p < (unsigned)a.B;
  s.source = has ? p : b;
  const int l = has ? clamp_len(a, a.length[p]) : 0;
  s.keep = l < s.next ? l : s.next;
  s.kept = pages_of(a, s.keep);
  s.old = pages_of(a, clamp_len(a, a.length[b]));
  s.want = pages_of(a, s.next);
  return s;
}

__global__ __launch_bounds__(kThreads) void k_ref_copy(PagesArgs a) {
  const int i = blockIdx.x * kThreads + threadIdx.x;
  if (i < a.n_pages) a.ref_out[i] = a.ref[i];
}

// References of the present sequences go, those of the kept pages come.  Integer
// atomics: their sum does not depend on their order.
__global__ __launch_bounds__(kThreads) void k_ref_move(PagesArgs a) {
  const int b = blockIdx.x;
  const Slot s = slot_of(a, b);
  const bool self = s.source == b && s.keep > 0;
  const int32_t* mine = a.table + (size_t)b * a.max_pages;
  const int32_t* from = a.table + (size_t)s.source * a.max_pages;
  for (int i = threadIdx.x + (self ? s.kept : 0); i < s.old; i += kThreads)
    if ((unsigned)mine[i] < (unsigned)a.n_pages) atomicSub(a.ref_out + mine[i], 1);
  if (!self)
    for (int i = threadIdx.x; i < s.kept; i += kThreads)
      if ((unsigned)from[i] < (unsigned)a.n_pages) atomicAdd(a.ref_out + from[i], 1);
}

// Pages of the block that are free (LIVE: in use), and, in the further workgroups
// of an update, what each slot needs.
template <bool LIVE>
__device__ __forceinline__ bool counts(int ref) { return LIVE ? ref > 0 : ref == 0; }

// A thread's consecutive pages of a block: their references (-1 past the pool), all
// loads in flight at once.
constexpr int kPerThread = kPageBlock / kThreads;
__device__ __forceinline__ void load_refs(const int32_t* ref, int n_pages, int block, int (&r)[kPerThread]) {
  const int p0 = block * kPageBlock + threadIdx.x * kPerThread;
#pragma unroll
  for (int i = 0; i < kPerThread; ++i) r[i] = ref[min(p0 + i, n_pages - 1)];
#pragma unroll
  for (int i = 0; i < kPerThread; ++i) r[i] = p0 + i < n_pages ? r[i] : -1;
}

template <bool LIVE>
__global__ __launch_bounds__(kThreads) void k_count(PagesArgs a, const int32_t* ref, int blocks) {
  __shared__ int sh[kThreads / 64];
  if ((int)blockIdx.x < blocks) {
    int r[kPerThread];
    load_refs(ref, a.n_pages, blockIdx.x, r);
    int n = 0;
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) n += counts<LIVE>(r[i]);
    n = block_sum(n, sh);
    if (threadIdx.x == 0) a.block_count[blockIdx.x] = n;
    return;
  }
  if constexpr (!LIVE) {
    const int b = (blockIdx.x - blocks) * kThreads + threadIdx.x;
    if (b >= a.B) return;
    const Slot s = slot_of(a, b);
    int need = 0, from = -1;
    if (s.next > s.keep) {
      need = s.want - s.kept;
      if (s.keep & ((1 << a.page_shift) - 1)) {
        const int last = a.table[(size_t)s.source * a.max_pages + s.kept - 1];
        if ((unsigned)last < (unsigned)a.n_pages && ref[last] > 1) {
          ++need;
          from = last;
        }
      }
    }
    a.need[b] = need;
    a.src[b] = from;
  }
}

// Pages before the block, and the total, from the blocks' counts.
__device__ __forceinline__ int counted_before(const PagesArgs& a, int block, int blocks, int* sh, int& total) {
  int before = 0, all = 0;
  for (int i = threadIdx.x; i < blocks; i += kThreads) {
    const int n = a.block_count[i];
    all += n;
    if (i < block) before += n;
  }
  total = block_sum(all, sh);
  return block_sum(before, sh);
}

// The free ids in ascending order; the last workgroup gives every slot its place
// in that list.
__global__ __launch_bounds__(kThreads) void k_free_list(PagesArgs a, int blocks) {
  __shared__ int sh[kThreads / 64];
  int mine[kPerThread];
  if ((int)blockIdx.x < blocks) load_refs(a.ref_out, a.n_pages, blockIdx.x, mine);
  int total;
  int at = counted_before(a, blockIdx.x, blocks, sh, total);
  if ((int)blockIdx.x < blocks) {
    int n = 0;
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) n += counts<false>(mine[i]);
    at += block_prefix(n, sh, n);
    const int p0 = blockIdx.x * kPageBlock + threadIdx.x * kPerThread;
#pragma unroll
    for (int i = 0; i < kPerThread; ++i)
      if (counts<false>(mine[i])) a.ids[at++] = p0 + i;
    return;
  }
  long long base = 0;  // requests may ask for more pages than 31 bits count
  for (int b0 = 0; b0 < a.B; b0 += kThreads) {
    const int b = b0 + threadIdx.x;
    const int need = b < a.B ? a.need[b] : 0;
    int n;
    const long long r = base + block_prefix(need, sh, n);
    if (b < a.B) a.base[b] = need == 0 ? 0 : r + need > total ? -1 : (int)r;  // -1: the pages do not fit
    base += n;
  }
  const long long missing = base - total;
  if (threadIdx.x == 0) *a.count = missing < 0 ? 0 : missing > INT32_MAX ? INT32_MAX : (int)missing;
}

__global__ __launch_bounds__(kThreads) void k_table(PagesArgs a) {
  const int b = blockIdx.x;
  const Slot s = slot_of(a, b);
  const int base = a.base[b], from = a.src[b];
  const bool fits = base >= 0;
  const bool copy = fits && from >= 0;
  const int want = s.next > s.keep && fits ? s.want : s.kept;
  const int32_t* kept = a.table + (size_t)s.source * a.max_pages;
  int32_t* row = a.table_out + (size_t)b * a.max_pages;
  for (int i = threadIdx.x; i < a.max_pages; i += kThreads) {
    int id = -1;
    if (i < s.kept && !(copy && i == s.kept - 1))
      id = kept[i];
    else if (i < want) {  // the private copy, or a further page
      id = a.ids[base + (i < s.kept ? 0 : copy + i - s.kept)];
      a.ref_out[id] = 1;
    }
    row[i] = id;
  }
  if (threadIdx.x == 0) {
    a.length_out[b] = s.next > s.keep && fits ? s.next : s.keep;
    if (copy) atomicSub(a.ref_out + from, 1);
    a.src[b] = copy ? from : -1;
    a.dst[b] = copy ? a.ids[base] : -1;
  }
}

// ------------------------------------------------------------------ compact
// Ranks: a hole is a free id below n_live, a source a live id at or above it;
// there are equally many.  `rank` of a source, `ids` the holes, `src` the sources.
__global__ __launch_bounds__(kThreads) void k_compact_rank(PagesArgs a, int blocks) {
  __shared__ int sh[kThreads / 64];
  int mine[kPerThread], edge_refs[kPerThread];
  load_refs(a.ref, a.n_pages, blockIdx.x, mine);
  int n_live;
  int at = counted_before(a, blockIdx.x, blocks, sh, n_live);
  // live ids below n_live: the whole blocks before n_live's, and the part of it
  const int edge = n_live / kPageBlock;  // n_live < n_pages, or every page is live and below
  int unused, part = 0;
  const int whole = counted_before(a, edge, blocks, sh, unused);
  load_refs(a.ref, a.n_pages, edge, edge_refs);
  const int e0 = edge * kPageBlock + threadIdx.x * kPerThread;
#pragma unroll
  for (int i = 0; i < kPerThread; ++i) part += e0 + i < n_live && edge_refs[i] > 0;
  const int below = whole + block_sum(part, sh);
  int n = 0;
#pragma unroll
  for (int i = 0; i < kPerThread; ++i) n += mine[i] > 0;
  at += block_prefix(n, sh, n);  // live ids before this thread's first
  const int p0 = blockIdx.x * kPageBlock + threadIdx.x * kPerThread;
#pragma unroll
  for (int i = 0; i < kPerThread; ++i) {
    const int p = p0 + i, ref = mine[i];
    const bool live = ref > 0;
    if (p < a.n_pages) {
      if (p >= n_live) {
        a.ref_out[p] = 0;
        a.rank[p] = live ? at - below : -1;
        if (live) a.src[at - below] = p;
      } else if (live) {
        a.ref_out[p] = ref;
      } else {
        a.ids[p - at] = p;
      }
    }
    at += live;
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    *a.count = n_live;
    *a.n_copies = n_live - below;
  }
}

// The renamed tables (one workgroup a slot); the further workgroups give the holes
// the references of the pages that move there.
__global__ __launch_bounds__(kThreads) void k_compact_table(PagesArgs a) {
  if ((int)blockIdx.x >= a.B) {
    const int r = (blockIdx.x - a.B) * kThreads + threadIdx.x;
    if (r < *a.n_copies) {
      a.ref_out[a.ids[r]] = a.ref[a.src[r]];
      a.dst[r] = a.ids[r];
    }
    return;
  }
  const int b = blockIdx.x;
  const int held = pages_of(a, clamp_len(a, a.length[b])), n_live = *a.count;
  const int32_t* from = a.table + (size_t)b * a.max_pages;
  int32_t* row = a.table_out + (size_t)b * a.max_pages;
  for (int i = threadIdx.x; i < a.max_pages; i += kThreads) {
    int id = -1;
    if (i < held) {
      const int p = from[i];
      if ((unsigned)p < (unsigned)a.n_pages && a.ref[p] > 0) id = p < n_live ? p : a.ids[a.rank[p]];
    }
    row[i] = id;
  }
}

// ------------------------------------------------------------------ page copies
// Copies src[i] -> dst[i] of both pools in every layer (entries of -1: nothing).
// Destinations are free pages, so no copy reads what another writes.  A workgroup
// moves pieces of 16 KiB, 4 x 16 bytes a thread in flight; bound by HBM.
constexpr int kPiece = 16384;
__global__ __launch_bounds__(kThreads) void k_copy_pages(const int32_t* src, const int32_t* dst, const int32_t* count,
                                                         int n, char* k_pool, char* v_pool, size_t bytes,
                                                         size_t layer_bytes) {
  if (count) n = *count;
  char* const pool = (blockIdx.z & 1 ? v_pool : k_pool) + (size_t)(blockIdx.z >> 1) * layer_bytes;
  const size_t at = (size_t)blockIdx.y * kPiece;
  for (int i = blockIdx.x; i < n; i += gridDim.x) {
    const int from = src[i], to = dst[i];
    if (from < 0 || to < 0) continue;
    const uint4* x = reinterpret_cast<const uint4*>(pool + (size_t)from * bytes + at);
    uint4* y = reinterpret_cast<uint4*>(pool + (size_t)to * bytes + at);
    const int m = (int)((bytes - at < (size_t)kPiece ? bytes - at : (size_t)kPiece) / 16);
    uint4 w[4];
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (u * kThreads + (int)threadIdx.x < m) w[u] = x[u * kThreads + threadIdx.x];
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (u * kThreads + (int)threadIdx.x < m) y[u * kThreads + threadIdx.x] = w[u];
  }
}

hipError_t copy_pages(const dspark_cache& C, const int32_t* src, const int32_t* dst, const int32_t* count, int n,
                      void* k_pool, void* v_pool, hipStream_t s) {
  const size_t bytes = page_bytes(C);
  const int pieces = (int)((bytes + kPiece - 1) / kPiece);
  const int per = pieces * 2 * C.n_layers;  // workgroups of one page
  int x = 16384 / per < 64 ? 64 : 16384 / per;
  x = x < n ? x : n;
  const dim3 grid(x, pieces, 2 * C.n_layers);
  k_copy_pages<<<grid, kThreads, 0, s>>>(src, dst, count, n, static_cast<char*>(k_pool), static_cast<char*>(v_pool),
                                         bytes, bytes * C.n_pages);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_cache_append(const dspark_cache& C, const AppendArgs& a, hipStream_t s) {
  switch (C.cache_dtype) {
    case DSPARK_F32: return append_typed<DSPARK_F32>(C, a, s);
    case DSPARK_BF16: return append_typed<DSPARK_BF16>(C, a, s);
    default: return append_typed<DSPARK_F8E4M3>(C, a, s);
  }
}

PagesLayout pages_layout(const dspark_cache& C) {
  PagesLayout L{};
  const size_t B = (size_t)C.B, N = (size_t)C.n_pages, w = sizeof(int32_t), M = B > N ? B : N;
  size_t off = 0;
  L.block_count = off; off = align256(off + page_blocks(C.n_pages) * w);
  L.need = off;        off = align256(off + B * w);
  L.base = off;        off = align256(off + B * w);
  L.ids = off;         off = align256(off + N * w);
  L.src = off;         off = align256(off + M * w);
  L.dst = off;         off = align256(off + M * w);
  L.rank = off;        off = align256(off + N * w);
  L.n_copies = off;    off = align256(off + w);
  L.total = off;
  return L;
}

hipError_t launch_cache_update(const dspark_cache& C, const PagesArgs& a, void* k_pool, void* v_pool, hipStream_t s) {
  const int blocks = page_blocks(C.n_pages);
  k_ref_copy<<<(C.n_pages + kThreads - 1) / kThreads, kThreads, 0, s>>>(a);
  k_ref_move<<<C.B, kThreads, 0, s>>>(a);
  k_count<false><<<blocks + (C.B + kThreads - 1) / kThreads, kThreads, 0, s>>>(a, a.ref_out, blocks);
  k_free_list<<<blocks + 1, kThreads, 0, s>>>(a, blocks);
  k_table<<<C.B, kThreads, 0, s>>>(a);
  const hipError_t e = hipGetLastError();
  return e != hipSuccess ? e : copy_pages(C, a.src, a.dst, nullptr, C.B, k_pool, v_pool, s);
}

hipError_t launch_cache_compact(const dspark_cache& C, const PagesArgs& a, void* k_pool, void* v_pool, hipStream_t s) {
  const int blocks = page_blocks(C.n_pages);
  k_count<true><<<blocks, kThreads, 0, s>>>(a, a.ref, blocks);
  k_compact_rank<<<blocks, kThreads, 0, s>>>(a, blocks);
  // at most half of the pages can move
  k_compact_table<<<C.B + (C.n_pages / 2 + kThreads) / kThreads, kThreads, 0, s>>>(a);
  const hipError_t e = hipGetLastError();
  return e != hipSuccess ? e : copy_pages(C, a.src, a.dst, a.n_copies, C.n_pages / 2 + 1, k_pool, v_pool, s);
}

}  // namespace dspark
