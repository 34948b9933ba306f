// Paged-cache attention: what its kernels share -- operand types, the geometry of a
// segment, the split of the work, the softmax of a tile, the join of partial results.
//
// Mathematics.  For a kv head, the G query heads that read it and the new tokens of
// a request form the rows of one product: row rho = (token rho / G, head rho % G).
// A tile of keys gives S^T = K Q^T (keys x rows) and O^T += V^T P^T with
// P = exp2(c S - m), c the softmax scale times log2(e), m the row's running maximum,
// l the running sum of P.  Transposed, a row is one MFMA column, that is one lane and
// its partners 32 (or 16) lanes on: the maximum and the sum of a row need one or two
// lane swaps, a rescaling of O is one factor per lane, and the registers that S^T
// leaves are, once exponentiated and rounded, the B operand of the second product as
// they stand.  The last holds because the rows of K are read in an order chosen for it
// (key_of_row): the product sums over keys, so their order within the tile is free.
//
// Running maximum.  m only moves when some row's maximum rises by more than 2^8 in
// weight; until then P may reach 2^8, which costs no precision (fp32 sums, and a rounding
// to bf16 is relative to the value), and O is not rescaled.
//
// What a row does not see must not reach it, not even as NaN times a weight of 0.
// Scores are replaced before the exponential.  In the tiles that some rows see in part
// or not at all (the sequence's end, the diagonal, a window's edge) values that are not
// finite are replaced by 0; if a row does see one, the coordinate's result is made NaN
// or infinite when it is stored (add_nonfinite), from the values themselves, by a walk over
// the keys of these tiles.  One that no row sees (behind the sequence's end) starts no walk
// in the row kernel; in the other the walk is short, and a check would cost registers.
// All other tiles are seen whole by all rows and need no such care.  These branches are
// marked as unlikely: without that their code costs the loops registers (256 x up to 17
// tokens over up to 2048 keys fp32 562 us, with it 517).
#pragma once

#include <type_traits>

#include "dspark_cache_internal.hpp"

namespace dspark {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef __attribute__((__vector_size__(2 * sizeof(float)))) float f32x2_t;

constexpr int kAttendThreads = 256;
constexpr float kRescale = 8.f;  // log2 of the weight up to which the maximum may lag
constexpr int kCUs = 256;

// How the work of a call is dealt out.  A segment is one (request, kv head, row tile),
// in that order, so that neighbours read the same keys; a unit is `unit` keys of a
// segment.  With `workers` 0 every workgroup takes one whole segment; else the units of
// all segments, in order, are dealt evenly to the workers, whose first and last
// segments may be partial.
struct Split {
  int row_tiles;  // of a request, at most
  int workers;
  int unit_shift;
  int spread_shift, xcd_tiles;  // of whole segments: XCDs (log2) that share a pair's row tiles, and each one's number
  bool longest_first;           // of whole segments: requests in descending order of their length
};

// A partial segment: O (unnormalised) [rows][D], then (m, l) [rows]; two a worker.
struct Record {  // of a worker whose first unit lies inside a segment (b -1: it does not)
  int b, head, row_tile;
  int first, last;  // workers that share the segment
  int slot;         // of the first one's part; the others' is twice their number
};

struct Geometry {
  int b, row_tile;
  int row0, rows;         // first row of the tile among the request's; rows in it
  int n, pos0;            // new tokens; position of token 0
  int lo, hi;             // keys that some row sees
  int all_lo, all_hi;     // keys in [all_lo, all_hi) are seen by every row
  int tile0, tiles;       // units
};

struct Masks {
  int causal, window, len;
  __device__ __forceinline__ int hi(int pos) const { return causal ? max(0, min(len, pos + 1)) : len; }
  __device__ __forceinline__ int lo(int pos) const { return window > 0 ? max(0, pos - window + 1) : 0; }
};

template <int ROWS>
__device__ __forceinline__ Geometry geometry(const AttendArgs& a, const Split& p, int b, int rt) {
  Geometry g;
  const int G = a.c.Hq / a.c.Hkv;
  g.b = b;
  g.row_tile = rt;
  g.n = a.c.rows(g.b);
  const int len = a.c.len(g.b);
  g.pos0 = len - g.n;
  g.row0 = rt * ROWS;
  g.rows = min(ROWS, g.n * G - g.row0);
  if (g.rows <= 0) {
    g.rows = g.tiles = g.tile0 = g.lo = g.hi = g.all_lo = g.all_hi = 0;
    return g;
  }
  const Masks m{a.causal, a.window, len};
  const int first = g.pos0 + g.row0 / G, last = g.pos0 + (g.row0 + g.rows - 1) / G;
  g.hi = m.hi(last);
  g.lo = min(m.lo(first), g.hi);
  g.all_hi = m.hi(first);
  g.all_lo = m.lo(last);
  g.tile0 = g.lo >> p.unit_shift;
  g.tiles = max(1, ((g.hi + (1 << p.unit_shift) - 1) >> p.unit_shift) - g.tile0);  // 1: its rows are written
  return g;
}

// Position in the dealt work: the segment that holds a worker's first unit.
struct Start {
  int b, head, row_tile;
  int skip;   // units of the segment before the worker's first
  long long count;  // the worker's units
  int workers;  // that have any
  long long unit, total;
};

// Exclusive prefix over the workgroup's THREADS threads; all receives the sum.
template <int THREADS>
__device__ __forceinline__ int wg_prefix(int v, int* sh, int& all) {
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
  all = 0;
#pragma unroll
  for (int w = 0; w < THREADS / 64; ++w) {
    const int s = sh[w];
    all += s;
    before += w < wave ? s : 0;
  }
  return x - v + before;
}

// Every worker finds its own start.  (Request, row tile) pairs are summed a
// chunk at a time, one a thread; the request is the last one whose units begin at or before the
// worker's, and within it the head and then the row tile follow.  For the batches that
// are dealt (up to a few thousand pairs) that is cheaper than a launch of its own.
template <int ROWS, int THREADS>
__device__ __forceinline__ Start find_start(const AttendArgs& a, const Split& p, int worker, int* sh) {
  const int RT = p.row_tiles, Hkv = a.c.Hkv;
  const long long pairs = (long long)a.c.B * RT;
  __shared__ int found_b, found_rt, found_skip;
  __shared__ long long found_before;
  auto tiles_of = [&](long long i) __attribute__((always_inline)) {
    return i < pairs ? geometry<ROWS>(a, p, RT == 1 ? (int)i : (int)(i / RT), RT == 1 ? 0 : (int)(i % RT)).tiles : 0;
  };
  Start s{};
  long long total = 0;
  int all, mine = 0;
  for (long long c = 0; c < pairs; c += THREADS) {
    mine = tiles_of(c + threadIdx.x);
    wg_prefix<THREADS>(mine, sh, all);
    total += all;
  }
  s.total = total * Hkv;
  s.workers = (int)(s.total < p.workers ? s.total : p.workers);
  if (worker >= s.workers) return s;
  s.unit = worker * s.total / s.workers;
  s.count = (worker + 1) * s.total / s.workers - s.unit;
  long long before = 0;
  for (long long c = 0; c < pairs; c += THREADS) {
    const long long i = c + threadIdx.x;
    if (pairs > THREADS) mine = tiles_of(i);
    const int ahead = wg_prefix<THREADS>(mine, sh, all);
    // the last pair, if any, that opens a request with units at or before the worker's first
    if (threadIdx.x == 0) found_rt = -1;
    __syncthreads();
    const bool opens = i < pairs && (RT == 1 || i % RT == 0) && (before + ahead) * Hkv <= s.unit;
    if (opens) atomicMax(&found_rt, (int)threadIdx.x);
    __syncthreads();
    if (opens && found_rt == (int)threadIdx.x) {
      found_b = RT == 1 ? (int)i : (int)(i / RT);
      found_before = before + ahead;
    }
    before += all;
    __syncthreads();
    if (before * Hkv > s.unit) break;
  }
  s.b = found_b;
  long long in = s.unit - found_before * Hkv;  // units into the request
  if (RT == 1) {
    const int t = geometry<ROWS>(a, p, s.b, 0).tiles;
    s.head = (int)(in / t);
    s.skip = (int)(in % t);
    return s;
  }
  long long per_head = 0;
  for (int c = 0; c < RT; c += THREADS) {
    mine = c + (int)threadIdx.x < RT ? geometry<ROWS>(a, p, s.b, c + threadIdx.x).tiles : 0;
    wg_prefix<THREADS>(mine, sh, all);
    per_head += all;
  }
  s.head = (int)(in / per_head);
  in %= per_head;
  for (int c = 0; c < RT; c += THREADS) {
    if (RT > THREADS) mine = c + (int)threadIdx.x < RT ? geometry<ROWS>(a, p, s.b, c + threadIdx.x).tiles : 0;
    const int ahead = wg_prefix<THREADS>(mine, sh, all);
    if (mine > 0 && in >= ahead && in < ahead + mine) {
      found_rt = c + threadIdx.x;
      found_skip = (int)(in - ahead);
    }
    in -= all;
    if (in < 0) break;
  }
  __syncthreads();
  s.row_tile = found_rt;
  s.skip = found_skip;
  return s;
}

// The request with the n-th largest length (of equal ones the first), by counting: every
// thread ranks its own.  Up to kAttendThreads requests.
__device__ __forceinline__ int nth_longest(const AttendArgs& a, int n) {
  static_assert(kAttendThreads == 256, "a length (24 bits) and the thread's number share a word");
  __shared__ __attribute__((aligned(16))) uint32_t key[kAttendThreads];
  __shared__ int found;
  const int t = threadIdx.x, B = a.c.B;
  const int len = t < B && a.c.rows(t) > 0 ? min(a.c.len(t), (1 << 24) - 1) : 0;
  const uint32_t mine = t < B ? ((uint32_t)len << 8) + (255 - t) : 0;
  key[t] = mine;
  __syncthreads();
  int rank = 0;
  for (int i = 0; i < B; i += 4) {  // (keys past B are 0: not larger than any)
    const uint4 k = *reinterpret_cast<const uint4*>(key + i);
    rank += (k.x > mine) + (k.y > mine) + (k.z > mine) + (k.w > mine);
  }
  if (t < B && rank == n) found = t;
  __syncthreads();
  return found;
}

// The segment of a workgroup that takes a whole one (none: b = B or row_tile < 0).
// Workgroups go round the 8 XCDs; a (request, head) pair's row tiles go to one XCD, next to
// each other, so that they read the keys through one L2 at about the same time; the last
// ones, which see the most keys, go first.  Pairs that would not fill the XCDs evenly are
// spread over 2, 4 or 8 of them (2 pairs of 2000 rows x 8 heads, fp32, on 2 XCDs: 630 us).
__device__ __forceinline__ Start whole_segment(const AttendArgs& a, const Split& p) {
  Start s{};
  const unsigned slot = blockIdx.x >> 3;
  const unsigned share = (slot / p.xcd_tiles << 3) + (blockIdx.x & 7), pair = share >> p.spread_shift;
  const int turn = (int)((slot % p.xcd_tiles << p.spread_shift) + (share & ((1u << p.spread_shift) - 1)));
  s.row_tile = p.row_tiles - 1 - turn;
  s.head = (int)(pair % a.c.Hkv);
  s.b = (int)(pair / a.c.Hkv);
  s.count = 0x7fffffffffffffffLL;
  if (p.longest_first && s.b < a.c.B && s.row_tile >= 0) s.b = nth_longest(a, s.b);
  return s;
}
// workgroups of such a launch: the pairs' shares rounded up to whole rounds of the XCDs
inline int whole_grid(const dspark_cache& C, Split& p) {
  const int pairs = C.B * C.Hkv;
  p.spread_shift = 0;
  // a pair more or less on an XCD is an eighth of its work or less from 64 pairs on
  while (pairs < 64 && ((pairs << p.spread_shift) & 7) && (2 << p.spread_shift) <= p.row_tiles) ++p.spread_shift;
  p.xcd_tiles = (p.row_tiles + (1 << p.spread_shift) - 1) >> p.spread_shift;
  return (((pairs << p.spread_shift) + 7) & ~7) * p.xcd_tiles;
}

// The next segment that has units (there is one).
template <int ROWS>
__device__ __forceinline__ Geometry next_segment(const AttendArgs& a, const Split& p, Start& s) {
  s.skip = 0;
  ++s.row_tile;
  while (true) {
    Geometry g;
    if (s.row_tile < p.row_tiles && (g = geometry<ROWS>(a, p, s.b, s.row_tile)).tiles > 0) return g;
    // the request's row tiles are done (or it has none): its next head, or the next request
    if (s.row_tile > 0 && ++s.head < a.c.Hkv) {
      s.row_tile = 0;
      continue;
    }
    s.head = s.row_tile = 0;
    ++s.b;
  }
}

// A request's row of the page table, read over the scalar cache (uniform addresses).
struct TableRow {
  const __attribute__((address_space(4))) int32_t* row;
  int shift, last, n_pages;
  __device__ __forceinline__ TableRow(const CacheView& c, int b)
      : row((const __attribute__((address_space(4))) int32_t*)(uintptr_t)(c.table + (size_t)b * c.max_pages)),
        shift(c.page_shift), last(c.max_pages - 1), n_pages(c.n_pages) {}
  __device__ __forceinline__ int raw(int key) const { return row[min(key >> shift, last)]; }
  __device__ __forceinline__ unsigned id(int raw) const { return min((unsigned)raw, (unsigned)n_pages - 1u); }
};

// ---- operands
// Element types of the two products: bf16 MFMA for bf16 and e4m3 caches (an e4m3
// value is a bf16 value; its scale is a factor of the scores and of the result),
// fp32 MFMA for fp32.
template <int CT>
struct Operand {
  static constexpr bool kF32 = CT == DSPARK_F32;
  static constexpr int kBytes = CT == DSPARK_F32 ? 4 : CT == DSPARK_BF16 ? 2 : 1;
  using Data = typename std::conditional<kF32, float, uint16_t>::type;
};

__device__ __forceinline__ bf16x8_t as_bf16x8(uint4 w) { return __builtin_bit_cast(bf16x8_t, w); }
__device__ __forceinline__ bf16x8_t f8_to_bf16x8(uint32_t lo, uint32_t hi) {
  bf16x2_t r[4] = {__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.f, false), __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.f, true),
                   __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.f, false), __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.f, true)};
  bf16x8_t o;
  __builtin_memcpy(&o, r, 16);
  return o;
}

// One row's running state in a lane: m is common to the row's lanes, l is the lane's
// share of the sum.
struct Running {
  float m, l;
};

// From scores to exponents of 2.  Not 0, so that a score of -inf stays one.
template <int CT>
__device__ __forceinline__ float score_factor(const AttendArgs& a, int head) {
  return fmaxf(CT == DSPARK_F8E4M3 ? a.scale2 * a.k_scale[head] : a.scale2, 0x1p-126f);
}

// The running maximum moves to include `top`; returns the factor by which O and l fade.
__device__ __forceinline__ float fade_to(Running& r, float top) {
  const float m = fmaxf(r.m, top);
  const float fade = m == -INFINITY ? 1.f : __builtin_amdgcn_exp2f(r.m - m);
  r.m = m;
  r.l *= fade;
  return fade;
}

// ---- values that a tile's rows see in part or not at all
template <int CT>
__device__ __forceinline__ uint32_t finite_word(uint32_t w) {
  if constexpr (CT == DSPARK_F32) {
    return (w & 0x7F800000u) == 0x7F800000u ? 0u : w;
  } else if constexpr (CT == DSPARK_BF16) {
    return ((w & 0x7F80u) == 0x7F80u ? 0u : w & 0xFFFFu) | ((w & 0x7F800000u) == 0x7F800000u ? 0u : w & 0xFFFF0000u);
  } else {
    uint32_t o = w;
#pragma unroll
    for (int e = 0; e < 32; e += 8)
      if ((w >> e & 0x7Fu) == 0x7Fu) o &= ~(0xFFu << e);
    return o;
  }
}
// kOdd bits are left in `odd` if an element of x is not finite: all exponent bits set
// (e4m3: all bits but the sign), where adding one carries into the element's top bit.
template <int CT>
constexpr uint32_t kOdd = CT == DSPARK_F32 ? 0x80000000u : CT == DSPARK_BF16 ? 0x80008000u : 0x80808080u;
template <int CT, typename V>
__device__ __forceinline__ void find_nonfinite(const V& x, uint32_t& odd) {
  constexpr uint32_t kExp = CT == DSPARK_F32 ? 0x7F800000u : CT == DSPARK_BF16 ? 0x7F807F80u : 0x7F7F7F7Fu;
  constexpr uint32_t kOne = CT == DSPARK_F32 ? 0x00800000u : CT == DSPARK_BF16 ? 0x00800080u : 0x01010101u;
  uint32_t w[sizeof(V) / 4];
  __builtin_memcpy(w, &x, sizeof(V));
#pragma unroll
  for (int i = 0; i < (int)(sizeof(V) / 4); ++i) odd |= (w[i] & kExp) + kOne;
}
template <int CT, typename V>
__device__ __forceinline__ V finite_part(V x) {
  uint32_t w[sizeof(V) / 4];
  __builtin_memcpy(w, &x, sizeof(V));
#pragma unroll
  for (int i = 0; i < (int)(sizeof(V) / 4); ++i) w[i] = finite_word<CT>(w[i]);
  __builtin_memcpy(&x, w, sizeof(V));
  return x;
}
// All bits of the elements of a word, neighbouring tokens from key `first` on, whose keys lie
// in [lo, hi).
template <int CT>
__device__ __forceinline__ uint32_t keys_within(int first, int lo, int hi) {
  constexpr int kOf = 4 / Operand<CT>::kBytes, kBits = 32 / kOf;  // elements of a word
  uint32_t mask = 0;
#pragma unroll
  for (int e = 0; e < kOf; ++e)
    if (first + e >= lo && first + e < hi) mask |= 0xFFFFFFFFu >> (32 - kBits) << (kBits * e);
  return mask;
}

template <int CT, typename V>
__device__ __forceinline__ bf16x8_t value_operand(const V& v) {
  if constexpr (CT == DSPARK_BF16)
    return as_bf16x8(v);
  else
    return f8_to_bf16x8(v.x, v.y);
}

// ---- results
// out and lse of one row from its sums
__device__ __forceinline__ float row_factor(float l, float vs) { return l == 0.f ? 0.f : vs / l; }

template <int CT>
__device__ __forceinline__ void store4(void* out, size_t at, float4 y) {
  if constexpr (CT == DSPARK_F32) {
    *reinterpret_cast<float4*>(static_cast<float*>(out) + at) = y;
  } else {
    uint2 w;
    const bf16x2_t p = __builtin_convertvector(f32x2_t{y.x, y.y}, bf16x2_t);
    const bf16x2_t q = __builtin_convertvector(f32x2_t{y.z, y.w}, bf16x2_t);
    __builtin_memcpy(&w.x, &p, 4);
    __builtin_memcpy(&w.y, &q, 4);
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(out) + at) = w;
  }
}

template <int CT>
__device__ __forceinline__ float cached(const char* p) {
  if constexpr (CT == DSPARK_F32)
    return *reinterpret_cast<const float*>(p);
  else if constexpr (CT == DSPARK_BF16)
    return bf16_to_f32(*reinterpret_cast<const uint16_t*>(p));
  else
    return __builtin_amdgcn_cvt_f32_fp8(*reinterpret_cast<const uint8_t*>(p), 0);
}

// What the values that are not finite make of coordinates d .. d + 3 of the row at
// position pos: those of the keys in [k0, k1) that it sees, in tiles of TILE keys that
// are not wholly in [all_lo, all_hi) (the others' products took them as they are).  A walk
// over groups of 8 keys, whose values of 4 coordinates lie together.
template <int CT, int D, int TILE>
__device__ __forceinline__ void add_nonfinite(const AttendArgs& a, const Geometry& g, const Masks& mask, int head,
                                              int pos, int d, int k0, int k1, float4& y) {
  constexpr int kEs = Operand<CT>::kBytes;
  const CacheView& c = a.c;
  const int lo = max(k0, mask.lo(pos)), hi = min(k1, mask.hi(pos));
  const int whole0 = (g.all_lo + TILE - 1) & ~(TILE - 1), whole1 = g.all_hi & ~(TILE - 1);  // the others' tiles
  for (int j0 = lo & ~7; j0 < hi; j0 += 8) {
    if (j0 >= whole0 && j0 < whole1) {
      j0 = whole1 - 8;
      continue;
    }
    const unsigned page = min((unsigned)c.table[(size_t)g.b * c.max_pages + (j0 >> c.page_shift)], (unsigned)c.n_pages - 1u);
    const size_t token = (((size_t)page * c.Hkv + head) << c.page_shift) + (j0 & ((1 << c.page_shift) - 1));
    const char* src = static_cast<const char*>(a.v_pool) + (token * D + (size_t)d * 8) * kEs;
    uint4 w[2 * kEs];
#pragma unroll
    for (int i = 0; i < 2 * kEs; ++i) w[i] = reinterpret_cast<const uint4*>(src)[i];
    uint32_t bits = 0;
#pragma unroll
    for (int i = 0; i < 2 * kEs; ++i) find_nonfinite<CT>(w[i], bits);
    if (!(bits & kOdd<CT>)) continue;
    float* const out = &y.x;
#pragma unroll 1
    for (int key = max(j0, lo); key < min(j0 + 8, hi); ++key)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float x = cached<CT>(src + (8 * i + (key & 7)) * kEs);
        if (!(fabsf(x) < INFINITY)) out[i] += x;
      }
  }
}

constexpr float kLn2f = 0.6931471805599453f;

// Row rho of the tile: its row of q and out, or -1
__device__ __forceinline__ long long global_row(const AttendArgs& a, const Geometry& g, int rho, int head, int& hq) {
  const int G = a.c.Hq / a.c.Hkv;
  const int t = (g.row0 + rho) / G;
  hq = head * G + (g.row0 + rho) - t * G;
  const long long r = a.c.first_row(g.b) + t;
  return a.c.has_row(r) ? r : -1;
}

template <int D>
constexpr size_t slot_floats(int rows) { return (size_t)rows * (D + 2); }

inline size_t records_bytes(int workers) { return align256((size_t)workers * sizeof(Record)); }

// The workspace of a dealt call
struct Partials {
  Record* records;
  float* slots;
  template <int D, int ROWS>
  __device__ __forceinline__ float* slot(int i) const { return slots + (size_t)i * slot_floats<D>(ROWS); }
};
__device__ __forceinline__ Partials partials(const AttendArgs& a, const Split& p) {
  return {static_cast<Record*>(a.workspace),
          reinterpret_cast<float*>(static_cast<char*>(a.workspace) + align256((size_t)p.workers * sizeof(Record)))};
}

// Worker `worker`'s record (one thread writes it)
__device__ __forceinline__ void put_record(const Partials& ws, const Start& s, int worker, int tiles) {
  Record r{-1, 0, 0, 0, 0, 0};
  if (s.count > 0 && s.skip > 0) {
    const long long u0 = s.unit - s.skip;  // a unit u is worker ((u + 1) W - 1) / total's
    r.b = s.b;
    r.head = s.head;
    r.row_tile = s.row_tile;
    r.first = (int)(((u0 + 1) * s.workers - 1) / s.total);
    r.last = (int)(((u0 + tiles) * s.workers - 1) / s.total);
    r.slot = 2 * r.first + (r.first * s.total / s.workers == u0 ? 0 : 1);
  }
  ws.records[worker] = r;
}

// Joins the partial results of the segment that a worker's first unit lies in, if the
// worker is the segment's second one.  Equal segments have equally many workers, often a
// multiple of the 8 XCDs: a segment's workgroups (blockIdx.y) take turns with the XCDs (16
// segments of 32 parts and 128 rows, all on one XCD: 71 us).  A row's parts (m, l, O) add up as
// sum exp2(m - M) (l, O), M the largest m, in a fixed order.  Groups of D / 4 threads
// take a row each; where there are many parts and few rows (tokens over a long context
// dealt to many workers) the workgroup takes a row, its groups the parts in turn.
constexpr int join_groups(int rows) { return rows > 64 ? 16 : 8; }  // workgroups of a segment
constexpr int kFewParts = 8, kMaxParts = 2 * kCUs;  // (the most workers)
template <int CT, int D, int ROWS>
__global__ __launch_bounds__(kAttendThreads) void k_attend_join(AttendArgs a, Split p) {
  constexpr int kLanes = D / 4, kGroups = kAttendThreads / kLanes;  // a float4 a lane
  const Partials ws = partials(a, p);
  const int worker = (blockIdx.x + blockIdx.y) % gridDim.x;
  const Record rec = ws.records[worker];
  if (rec.b < 0 || worker != rec.first + 1) return;
  const int parts = rec.last - rec.first + 1;
  const Geometry g = geometry<ROWS>(a, p, rec.b, rec.row_tile);
  const int group = threadIdx.x / kLanes, lane = threadIdx.x % kLanes;
  const float vs = CT == DSPARK_F8E4M3 ? a.v_scale[rec.head] : 1.f;
  auto slot = [&](int i) __attribute__((always_inline)) { return ws.template slot<D, ROWS>(i == 0 ? rec.slot : 2 * (rec.first + i)); };
  auto weight = [](float m, float top) __attribute__((always_inline)) { return m == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(m - top); };
  // (the l of such an m is 0 or NaN)
  auto share = [](float m, float l, float f) __attribute__((always_inline)) { return m == -INFINITY ? l : l * f; };
  auto add = [](float4& o, const float4& x, float f) __attribute__((always_inline)) {
    o.x = fmaf(x.x, f, o.x);
    o.y = fmaf(x.y, f, o.y);
    o.z = fmaf(x.z, f, o.z);
    o.w = fmaf(x.w, f, o.w);
  };
  auto store = [&](int rho, float top, float l, float4 o) __attribute__((always_inline)) {
    int hq;
    const long long row = global_row(a, g, rho, rec.head, hq);
    if (row < 0) return;
    const float f = row_factor(l, vs);
    if (l == 0.f) o = make_float4(0.f, 0.f, 0.f, 0.f);
    store4<CT>(a.out, row * a.out_stride + (size_t)hq * D + 4 * lane, make_float4(o.x * f, o.y * f, o.z * f, o.w * f));
    if (a.lse && lane == 0) a.lse[row * a.c.Hq + hq] = l == 0.f ? -INFINITY : (top + log2f(l)) * kLn2f;
  };
  if (parts <= kFewParts || g.rows > (int)gridDim.y) {
    for (int rho = blockIdx.y * kGroups + group; rho < g.rows; rho += gridDim.y * kGroups) {
      float top = -INFINITY, l = 0.f;
#pragma unroll 8
      for (int i = 0; i < parts; ++i) top = fmaxf(top, slot(i)[(size_t)ROWS * D + 2 * rho]);
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
      for (int i = 0; i < parts; ++i) {
        const float* s = slot(i);
        const float2 ml = *reinterpret_cast<const float2*>(s + (size_t)ROWS * D + 2 * rho);
        const float f = weight(ml.x, top);
        l += share(ml.x, ml.y, f);
        add(o, *reinterpret_cast<const float4*>(s + (size_t)rho * D + 4 * lane), f);
      }
      store(rho, top, l, o);
    }
    return;
  }
  __shared__ float factor[kMaxParts], sh[kAttendThreads / 64];
  __shared__ float4 so[kGroups][kLanes];
  for (int rho = blockIdx.y; rho < g.rows; rho += gridDim.y) {
    float2 ml[kMaxParts / kAttendThreads];
#pragma unroll
    for (int e = 0; e < kMaxParts / kAttendThreads; ++e) {
      const int i = e * kAttendThreads + threadIdx.x;
      ml[e] = i < parts ? *reinterpret_cast<const float2*>(slot(i) + (size_t)ROWS * D + 2 * rho)
                        : make_float2(-INFINITY, 0.f);
    }
    float top = ml[0].x;
#pragma unroll
    for (int e = 1; e < kMaxParts / kAttendThreads; ++e) top = fmaxf(top, ml[e].x);
    top = wave_max(top);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = top;
    __syncthreads();
    top = fmaxf(fmaxf(sh[0], sh[1]), fmaxf(sh[2], sh[3]));
    float l = 0.f;
#pragma unroll
    for (int e = 0; e < kMaxParts / kAttendThreads; ++e) {
      const float f = weight(ml[e].x, top);
      factor[e * kAttendThreads + threadIdx.x] = f;
      l += share(ml[e].x, ml[e].y, f);
    }
    l = wave_sum(l);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = l;
    __syncthreads();
    l = sh[0] + sh[1] + sh[2] + sh[3];
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int i0 = group; i0 < parts; i0 += 8 * kGroups) {
      float4 x[8];
#pragma unroll
      for (int u = 0; u < 8; ++u)
        x[u] = *reinterpret_cast<const float4*>(slot(min(i0 + u * kGroups, parts - 1)) + (size_t)rho * D + 4 * lane);
#pragma unroll
      for (int u = 0; u < 8; ++u)
        if (i0 + u * kGroups < parts) add(o, x[u], factor[i0 + u * kGroups]);
    }
    so[group][lane] = o;
    __syncthreads();
    if (group == 0) {
      for (int i = 1; i < kGroups; ++i) add(o, so[i][lane], 1.f);
      store(rho, top, l, o);
    }
  }
}

}  // namespace dspark
