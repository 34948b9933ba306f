// Paged cache: writing tokens into pages (append), and the bookkeeping of pages
// (update: fork, grow, shrink, free, private copies; compact).  See
// include/dspark_cache.h for the contract.
//
// The page bookkeeping is integer work over the table, the lengths and the
// reference counts; every result is independent of the order in which workgroups
// or atomics run (sums of references, ranks from prefix sums, lowest free ids
// first).  Device-wide dependencies are launch boundaries: a launch of the next
// kernel costs about 2 us on the stream, a grid barrier over 8 XCDs no less.  An update of
// 256 slots and 68,125 pages takes 2.5 + 2.4 + 3.0 + 4.4 + 3.2 us in its five kernels.
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

// A workgroup writes 8-token groups (the v_pool's unit [D][8]) of a few heads, D / 2
// threads each.  Values: a thread carries 2 coordinates, reads 8 rows (neighbouring
// threads neighbouring coordinates) and writes 2 x 8 tokens as whole 16-byte pieces; of
// a group that is new in part it merges with the old pieces (read for every group), since
// 2-byte stores cost more (256 x 17 rows of 8 x 128, bf16, 13.6 us with them, 8.4 so).
// Keys: rows copied in 16-byte pieces.  All loads are issued before the first use.  Bound
// by memory and the way to it, length -> table -> rows and old values -> store: of those
// 8.4 us the waves wait 59% (25 MB read and written), of the 15.6 of 8192 rows of 8 x 128
// into an e4m3 cache 33%, and 41% for the issue of an instruction (59 MB, 8 of them old
// values; a reciprocal with a correction in place of the divisions gained nothing, vector
// instructions issue in 17% of the waves' cycles).
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
  constexpr int kData = CT == DSPARK_F32 ? 4 : 2;
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
  T* const kd = static_cast<T*>(a.k_pool) + (block + off) * D;
  T* const vd = static_cast<T*>(a.v_pool) + (block + off) * D + (size_t)d * 8;
  const float ks = CT == DSPARK_F8E4M3 ? a.k_scale[head] : 1.f, vs = CT == DSPARK_F8E4M3 ? a.v_scale[head] : 1.f;
  const long long row0 = c.first_row(b) + (j0 - pos0);
  // tokens of the group that are new and have a row; the others read the nearest row that is there
  auto has = [&](int t) { return j0 + t >= lo && j0 + t < hi && c.has_row(row0 + t); };
  auto row_of = [&](int t) {
    const long long near = row0 + min(max(t, lo - j0), hi - 1 - j0);
    return near < 0 ? 0 : near < c.n_rows ? near : (long long)c.n_rows - 1;
  };
  constexpr int kEs = sizeof(T), kPieces = D * kEs / 16;  // 16-byte pieces of a key
  constexpr int kWords = CT == DSPARK_F8E4M3 ? 2 : 1;     // 16-byte words of data for one
  uint4 kw[kEs][kWords];
#pragma unroll
  for (int i = 0; i < kEs; ++i) {
    const int at = i * kPerHead + threadIdx.x % kPerHead;
    const uint4* src = reinterpret_cast<const uint4*>(static_cast<const char*>(a.k) +
                                                      (row_of(at / kPieces) * a.k_stride + head * D) * kData) +
                       at % kPieces * kWords;
#pragma unroll
    for (int w = 0; w < kWords; ++w) kw[i][w] = src[w];
  }
  typename DataPair<CT>::T vw[8];
  bool all = true;
#pragma unroll
  for (int t = 0; t < 8; ++t) {
    all = all && has(t);
    vw[t] = DataPair<CT>::load(a.v, row_of(t) * a.v_stride + head * D + d);
  }
  constexpr int kLine = 16 * kEs / 16;  // 16-byte words of 2 coordinates x 8 tokens
  uint4 old[kLine];
#pragma unroll
  for (int i = 0; i < kLine; ++i) old[i] = reinterpret_cast<const uint4*>(vd)[i];

#pragma unroll
  for (int i = 0; i < kEs; ++i) {
    const int at = i * kPerHead + threadIdx.x % kPerHead, t = at / kPieces;
    uint4 x = kw[i][0];
    if constexpr (CT == DSPARK_F8E4M3) {
      const uint32_t in[8] = {kw[i][0].x, kw[i][0].y, kw[i][0].z, kw[i][0].w,
                              kw[i][1].x, kw[i][1].y, kw[i][1].z, kw[i][1].w};
      uint32_t o[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        o[j] = f8_pair(bf16_lo(in[2 * j]) / ks, bf16_hi(in[2 * j]) / ks) |
               f8_pair(bf16_lo(in[2 * j + 1]) / ks, bf16_hi(in[2 * j + 1]) / ks) << 16;
      x = make_uint4(o[0], o[1], o[2], o[3]);
    }
    if (has(t)) reinterpret_cast<uint4*>(kd)[at] = x;
  }
  T line[16];
  __builtin_memcpy(line, old, sizeof(line));
#pragma unroll
  for (int t = 0; t < 8; ++t) {
    T x[2];
    store_type<CT>(vw[t], vs, x);
    const bool is = all || has(t);
    line[t] = is ? x[0] : line[t];
    line[8 + t] = is ? x[1] : line[8 + t];
  }
#pragma unroll
  for (int i = 0; i < kLine; ++i) {
    uint4 w;
    __builtin_memcpy(&w, reinterpret_cast<const char*>(line) + 16 * i, 16);
    reinterpret_cast<uint4*>(vd)[i] = w;
  }
}

// The same with a scale for every token and head, taken from the token: the largest size
// of its D finite elements goes to 448.  A thread quantises 16 elements of a token's key and
// of its value; the token's D / 16 threads, neighbours in a row of 16 lanes, agree on the
// scale.  The values then change hands through LDS, from a token's elements to a coordinate's
// tokens.  Old pieces are read only where a group is new in part.
//   256 x up to 17 rows of 8 x 128: 7.9 us (11.5 MB; 10.6 read, 5.4 written), the chain length ->
// table -> rows -> scale -> LDS -> store; 4 x 2048 rows 11.5 us (51 MB, 4.4 TB/s), with divisions
// and reductions through LDS 18.1.
constexpr uint32_t kInf16 = 0x7F80;  // bf16

// The larger of x and another lane's, by a data-parallel primitive.
template <int CTRL>
__device__ __forceinline__ uint32_t max_with(uint32_t x) {
  const uint32_t y = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, CTRL, 0xF, 0xF, true);
  return x > y ? x : y;
}
// Largest size of the elements of a token's THREADS threads, as bf16 bits: sizes of bf16
// numbers are ordered as their bits are.  odd: an element is not finite (and left out).
template <int THREADS>
__device__ __forceinline__ uint32_t token_top(const uint32_t (&w)[8], bool& odd) {
  typedef uint16_t u16x2_t __attribute__((ext_vector_type(2)));
  u16x2_t top = {0, 0};
#pragma unroll
  for (int i = 0; i < 8; ++i) top = __builtin_elementwise_max(top, __builtin_bit_cast(u16x2_t, w[i] & 0x7FFF7FFFu));
  uint32_t t = top[0] > top[1] ? top[0] : top[1];
  odd = t >= kInf16;
  if (__builtin_expect(odd, 0)) {
    t = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const uint32_t x = w[i >> 1] >> (16 * (i & 1)) & 0x7FFFu;
      if (x < kInf16 && x > t) t = x;
    }
  }
  t = max_with<0xB1>(t);   // lanes 1, 0, 3, 2
  t = max_with<0x4E>(t);   // lanes 2, 3, 0, 1
  if constexpr (THREADS > 4) t = max_with<0x141>(t);  // lanes 7 .. 0 of each 8
  if constexpr (THREADS > 8) t = max_with<0x140>(t);  // lanes 15 .. 0 of each 16
  return t;
}
__device__ __forceinline__ float token_scale(uint32_t top) {
  return top ? fmaxf(__uint_as_float(top << 16) / 448.f, 0x1p-126f) : 1.f;
}
// e4m3 of the 16 quotients x / scale.  With r the rounded reciprocal of the scale and q = x r,
// the rest x - q scale is exact in an fma, and q plus the rest times r is the rounded quotient
// (Markstein, 1990): three instructions where a division takes ten.  Scales so small that the
// rest could fall among the subnormal numbers, and elements that are not finite, are divided.
// (No quotient of a finite element lies above 448 by more than a rounding, which goes to 448.)
__device__ __forceinline__ uint4 token_entries(const uint32_t (&w)[8], float scale, bool odd) {
  uint32_t o[4] = {0, 0, 0, 0};
  if (__builtin_expect(odd || scale < 0x1p-90f, 0)) {
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i >> 1] |= f8_pair(bf16_lo(w[i]) / scale, bf16_hi(w[i]) / scale) << (16 * (i & 1));
  } else {
    const float r = 1.f / scale;
    auto quotient = [&](float x) __attribute__((always_inline)) {
      const float q = x * r;
      return fmaf(fmaf(-q, scale, x), r, q);
    };
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int x = __builtin_amdgcn_cvt_pk_fp8_f32(quotient(bf16_lo(w[2 * i])), quotient(bf16_hi(w[2 * i])), 0, false);
      o[i] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(quotient(bf16_lo(w[2 * i + 1])), quotient(bf16_hi(w[2 * i + 1])), x, true);
    }
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

template <int D>
__global__ __launch_bounds__(kThreads) void k_append_token(AppendArgs a, int groups) {
  constexpr int kPerHead = D / 2, kPieces = D / 16, kHeads = kThreads / kPerHead;
  __shared__ __attribute__((aligned(16))) uint8_t turn[kHeads][8][D];
  const CacheView& c = a.c;
  const int slot = threadIdx.x / kPerHead, at = threadIdx.x % kPerHead;
  const int head = min((int)blockIdx.y * kHeads + slot, c.Hkv - 1);
  const bool mine = (int)blockIdx.y * kHeads + slot < c.Hkv;
  for (long long u = blockIdx.x; u < (long long)c.B * groups; u += gridDim.x) {
    const int b = (int)(u / groups), gi = (int)(u % groups);
    const int n = c.rows(b), len = c.len(b);
    const int pos0 = len - n;  // of token 0; may be negative
    const int first = pos0 < 0 ? 0 : pos0;
    const int j0 = ((first >> 3) + gi) << 3;
    const int lo = j0 > first ? j0 : first, hi = j0 + 8 < len ? j0 + 8 : len;
    if (n == 0 || lo >= hi) continue;
    const int page = c.table[(size_t)b * c.max_pages + (j0 >> c.page_shift)];
    const long long row0 = c.first_row(b) + (j0 - pos0);
    auto has = [&](int t) { return j0 + t >= lo && j0 + t < hi && c.has_row(row0 + t); };
    // this thread's 16 elements; a token that is not new reads the nearest row that is there
    const int t = at / kPieces, piece = at % kPieces;
    const long long near = row0 + min(max(t, lo - j0), hi - 1 - j0);
    const long long row = near < 0 ? 0 : near < c.n_rows ? near : (long long)c.n_rows - 1;
    auto load = [&](const void* x, long long stride, uint32_t(&w)[8]) {
      const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(x) + row * stride + head * D) + 2 * piece;
      const uint4 p = src[0], q = src[1];
      __builtin_memcpy(w, &p, 16);
      __builtin_memcpy(w + 4, &q, 16);
    };
    uint32_t kw[8], vw[8];
    load(a.k, a.k_stride, kw);
    load(a.v, a.v_stride, vw);
    if ((unsigned)page >= (unsigned)c.n_pages) continue;
    const int off = j0 & ((1 << c.page_shift) - 1);
    const size_t block = ((size_t)page * c.Hkv + head) << c.page_shift;  // tokens
    uint8_t* const kb = static_cast<uint8_t*>(a.k_pool) + block * (D + 4);
    uint8_t* const vb = static_cast<uint8_t*>(a.v_pool) + block * (D + 4);
    uint4* const line = reinterpret_cast<uint4*>(vb + (size_t)off * D) + at;  // 8 tokens of 2 coordinates
    bool all = true;
#pragma unroll
    for (int i = 0; i < 8; ++i) all = all && has(i);
    uint4 old{};
    if (!all) old = *line;
    bool k_odd, v_odd;
    const uint32_t k_top = token_top<kPieces>(kw, k_odd), v_top = token_top<kPieces>(vw, v_odd);
    const float ks = token_scale(k_top), vs = token_scale(v_top);
    const uint4 ke = token_entries(kw, ks, k_odd), ve = token_entries(vw, vs, v_odd);
    __syncthreads();  // the last group's values are read
    *reinterpret_cast<uint4*>(&turn[slot][t][16 * piece]) = ve;
    if (mine && has(t)) {
      reinterpret_cast<uint4*>(kb + (size_t)off * D)[at] = ke;
      if (piece == 0) {
        const size_t scales = (size_t)D << c.page_shift;
        reinterpret_cast<float*>(kb + scales)[off + t] = ks;
        reinterpret_cast<float*>(vb + scales)[off + t] = vs;
      }
    }
    __syncthreads();
    // two coordinates of a token are 16 bits; of 4 tokens the low bytes, and the high ones
    uint32_t x[8], y[4];
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = *reinterpret_cast<const uint16_t*>(&turn[slot][i][2 * at]);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t p = x[4 * i] | x[4 * i + 1] << 16, q = x[4 * i + 2] | x[4 * i + 3] << 16;
      y[i] = __builtin_amdgcn_perm(q, p, 0x06040200);
      y[2 + i] = __builtin_amdgcn_perm(q, p, 0x07050301);
    }
    if (!all) {
      uint32_t is[2] = {0, 0};  // the new tokens' bytes
#pragma unroll
      for (int i = 0; i < 8; ++i) is[i >> 2] |= has(i) ? 0xFFu << (8 * (i & 3)) : 0u;
      y[0] = (y[0] & is[0]) | (old.x & ~is[0]);
      y[1] = (y[1] & is[1]) | (old.y & ~is[1]);
      y[2] = (y[2] & is[0]) | (old.z & ~is[0]);
      y[3] = (y[3] & is[1]) | (old.w & ~is[1]);
    }
    if (mine) *line = make_uint4(y[0], y[1], y[2], y[3]);
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
  auto run = [&](auto d) {
    constexpr int D = decltype(d)::value;
    if constexpr (CT == DSPARK_F8E4M3_TOKEN)
      k_append_token<D><<<grid, kThreads, 0, s>>>(a, groups);
    else
      k_append<CT, D><<<grid, kThreads, 0, s>>>(a, groups);
  };
  if (C.D == 64)
    run(std::integral_constant<int, 64>());
  else if (C.D == 128)
    run(std::integral_constant<int, 128>());
  else
    run(std::integral_constant<int, 256>());
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

// Pages that slot b needs, and the shared page that it has to copy (-1: none); ref as
// after the sequences' change.
__device__ __forceinline__ void need_of(const PagesArgs& a, const int32_t* ref, int b, int32_t& need, int32_t& from) {
  const Slot s = slot_of(a, b);
  int n = 0, f = -1;
  if (s.next > s.keep) {
    n = s.want - s.kept;
    if (s.keep & ((1 << a.page_shift) - 1)) {
      const int last = a.table[(size_t)s.source * a.max_pages + s.kept - 1];
      if ((unsigned)last < (unsigned)a.n_pages && ref[last] > 1) {
        ++n;
        f = last;
      }
    }
  }
  need = n;
  from = f;
}

// Slot b's next row and length, and its pages' references.
__device__ __forceinline__ void write_slot(const PagesArgs& a, int b, int base, bool fits, int from, bool copy) {
  const Slot s = slot_of(a, b);
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
  }
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
    if (b < a.B) need_of(a, ref, b, a.need[b], a.src[b]);
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

// ------------------------------------------------------------------ small pools
// The whole bookkeeping of a call in one workgroup, with the references, the lists and
// the slots in LDS: what several launches do above, separated by barriers in place of
// launches.  One CU then reads and writes the tables, so this is for small ones: on the
// stream, update 9.2 us against 13.4 for 2,176 entries, 11.3 / 14.3 for 4,352, 15.8 / 14.3
// for 8,448; compact 5.9 / 10.7 for 512 pages, 9.3 / 12.5 for 4,096, 14.5 / 14.2 for 8,192.
constexpr int kSmallThreads = 1024;
constexpr int kSmallPages = 8192, kSmallEntries = 8192;
bool small_pool(const dspark_cache& C) {
  return C.n_pages <= kSmallPages && C.B <= kSmallThreads && (long long)C.B * C.max_pages <= kSmallEntries;
}

struct SmallPool {
  int ref[kSmallPages];
  uint16_t ids[kSmallPages];
  int source[kSmallThreads], kept[kSmallThreads], old[kSmallThreads], want[kSmallThreads];
  int from[kSmallThreads], base[kSmallThreads];
  int sh[kSmallThreads / 64];
};

// Pages of this thread, consecutive ones: each goes to put(page, rank among those with
// pred before it, pred).  Returns how many there are in the pool.
template <typename Pred, typename Put>
__device__ __forceinline__ int rank_pages(SmallPool& m, int n_pages, Pred pred, Put put) {
  const int per = (n_pages + kSmallThreads - 1) / kSmallThreads, p0 = threadIdx.x * per;
  const int p1 = min(p0 + per, n_pages);
  int n = 0;
  for (int p = p0; p < p1; ++p) n += pred(m.ref[p]);
  int total;
  int at = block_prefix(n, m.sh, total);
  for (int p = p0; p < p1; ++p) {
    const bool is = pred(m.ref[p]);
    put(p, at, is);
    at += is;
  }
  return total;
}

__device__ __forceinline__ void load_pool(SmallPool& m, const PagesArgs& a) {
  int r[kSmallPages / kSmallThreads];
#pragma unroll
  for (int u = 0; u < kSmallPages / kSmallThreads; ++u)
    r[u] = a.ref[min((int)threadIdx.x + u * kSmallThreads, a.n_pages - 1)];
#pragma unroll
  for (int u = 0; u < kSmallPages / kSmallThreads; ++u)
    if ((int)threadIdx.x + u * kSmallThreads < a.n_pages) m.ref[threadIdx.x + u * kSmallThreads] = r[u];
}

// all entries (slot, place) of the tables, kFlight of a thread at a time: get(slot,
// place) for all of them, then put(slot, place, what get gave)
constexpr int kFlight = 4;
template <typename Get, typename Put>
__device__ __forceinline__ void entries(const PagesArgs& a, Get get, Put put) {
  const int n = a.B * a.max_pages;
  for (int e0 = threadIdx.x; e0 < n; e0 += kFlight * kSmallThreads) {
    decltype(get(0, 0)) x[kFlight];
#pragma unroll
    for (int u = 0; u < kFlight; ++u) {
      const int e = min(e0 + u * kSmallThreads, n - 1);
      x[u] = get(e / a.max_pages, e % a.max_pages);
    }
#pragma unroll
    for (int u = 0; u < kFlight; ++u) {
      const int e = e0 + u * kSmallThreads;
      if (e < n) put(e / a.max_pages, e % a.max_pages, x[u]);
    }
  }
}

__global__ __launch_bounds__(kSmallThreads) void k_update_small(PagesArgs a) {
  __shared__ SmallPool m;
  const int b = threadIdx.x;  // this thread's slot
  const bool mine = b < a.B;
  Slot s{};
  int last = -1;  // its last kept page, if it is partly filled and the slot grows
  if (mine) {
    s = slot_of(a, b);
    if (s.next > s.keep && (s.keep & ((1 << a.page_shift) - 1)))
      last = a.table[(size_t)s.source * a.max_pages + s.kept - 1];
  }
  load_pool(m, a);
  if (mine) {
    m.source[b] = s.source;
    m.kept[b] = s.kept;
    m.old[b] = s.old;
  }
  __syncthreads();
  // a slot's own pages go, unless it keeps them; its source's kept pages come
  entries(
      a,
      [&](int t, int i) {
        const int src = m.source[t];
        return make_int2(a.table[t * a.max_pages + i], a.table[src * a.max_pages + i]);
      },
      [&](int t, int i, int2 id) {
        const bool self = m.source[t] == t, kept = i < m.kept[t];
        if (i < m.old[t] && !(self && kept) && (unsigned)id.x < (unsigned)a.n_pages) atomicSub(m.ref + id.x, 1);
        if (!self && kept && (unsigned)id.y < (unsigned)a.n_pages) atomicAdd(m.ref + id.y, 1);
      });
  __syncthreads();
  const int total = rank_pages(
      m, a.n_pages, [](int ref) { return ref == 0; },
      [&](int p, int at, bool is) {
        if (is) m.ids[at] = (uint16_t)p;
      });
  const int from = (unsigned)last < (unsigned)a.n_pages && m.ref[last] > 1 ? last : -1;
  const int need = mine && s.next > s.keep ? s.want - s.kept + (from >= 0) : 0;
  int all;
  const int at = block_prefix(need, m.sh, all);  // (at most kSmallEntries, and a copy a slot)
  if (mine) {
    const bool fits = need == 0 || at + need <= total, grows = s.next > s.keep && fits;
    const int copy = grows ? from : -1;
    m.want[b] = grows ? s.want : s.kept;
    m.from[b] = copy;
    m.base[b] = at;
    a.length_out[b] = grows ? s.next : s.keep;
    a.src[b] = copy;
    a.dst[b] = copy >= 0 ? (int)m.ids[at] : -1;
  }
  if (b == 0) *a.count = max(0, all - total);
  __syncthreads();  // (the list is whole, and every slot has read its page's references)
  if (mine && m.from[b] >= 0) atomicSub(m.ref + m.from[b], 1);
  entries(
      a, [&](int t, int i) { return a.table[m.source[t] * a.max_pages + i]; },
      [&](int t, int i, int id) {
        const int kept = m.kept[t];
        const bool copy = m.from[t] >= 0;
        if (i >= kept || (copy && i == kept - 1)) {
          id = -1;
          if (i < m.want[t]) {  // the private copy, or a further page
            id = m.ids[m.base[t] + (i < kept ? 0 : copy + i - kept)];
            m.ref[id] = 1;
          }
        }
        a.table_out[t * a.max_pages + i] = id;
      });
  __syncthreads();
  for (int p = threadIdx.x; p < a.n_pages; p += kSmallThreads) a.ref_out[p] = m.ref[p];
}

__global__ __launch_bounds__(kSmallThreads) void k_compact_small(PagesArgs a) {
  __shared__ SmallPool m;
  const int b = threadIdx.x;
  if (b < a.B) m.kept[b] = pages_of(a, clamp_len(a, a.length[b]));
  load_pool(m, a);
  __syncthreads();
  const int n_live = rank_pages(m, a.n_pages, [](int ref) { return ref > 0; },
                                [&](int p, int at, bool) { m.ids[p] = (uint16_t)at; });  // live pages before p
  __syncthreads();
  const int below = n_live < a.n_pages ? m.ids[n_live] : n_live;  // live ids below n_live
  const int holes = n_live - below;
  for (int p = threadIdx.x; p < a.n_pages; p += kSmallThreads) {
    const int ref = m.ref[p], before = m.ids[p];
    if (p >= n_live)
      a.ref_out[p] = 0;
    else if (ref > 0)
      a.ref_out[p] = ref;
    if (p < n_live && ref <= 0) a.dst[p - before] = p;
    if (p >= n_live && ref > 0) a.src[before - below] = p;
  }
  if (b == 0) {
    *a.count = n_live;
    *a.n_copies = holes;
  }
  __syncthreads();
  for (int r = threadIdx.x; r < holes; r += kSmallThreads) a.ref_out[a.dst[r]] = m.ref[a.src[r]];
  entries(
      a, [&](int t, int i) { return a.table[t * a.max_pages + i]; },
      [&](int t, int i, int p) {
        int id = -1;
        if (i < m.kept[t] && (unsigned)p < (unsigned)a.n_pages && m.ref[p] > 0)
          id = p < n_live ? p : a.dst[m.ids[p] - below];
        a.table_out[t * a.max_pages + i] = id;
      });
}

// ------------------------------------------------------------------ page copies
// A page moves in pieces of 16 KiB, 4 x 16 bytes a thread in flight; bound by HBM: 0.54 GB
// moved, read and written, 206 us, 5.2 TB/s, the rate of a large copy.
constexpr int kPiece = 16384;
struct Pools {
  char *k, *v;
  size_t bytes, layer_bytes;  // of a page in a layer; of a layer
  int pieces, parts;          // of a page in a layer; of a page in both pools and all layers
};
Pools pools_of(const dspark_cache& C, void* k_pool, void* v_pool) {
  Pools p{static_cast<char*>(k_pool), static_cast<char*>(v_pool), page_bytes(C), page_bytes(C) * C.n_pages, 0, 0};
  p.pieces = (int)((p.bytes + kPiece - 1) / kPiece);
  p.parts = p.pieces * 2 * C.n_layers;
  return p;
}
__device__ __forceinline__ void copy_part(const Pools& p, int part, int from, int to) {
  const int piece = part % p.pieces, pool = part / p.pieces;
  char* const base = ((pool & 1) ? p.v : p.k) + (size_t)(pool >> 1) * p.layer_bytes;
  const size_t at = (size_t)piece * kPiece;
  const int m = (int)((p.bytes - at < (size_t)kPiece ? p.bytes - at : (size_t)kPiece) / 16);  // 16-byte words
  const uint4* x = reinterpret_cast<const uint4*>(base + (size_t)from * p.bytes + at);
  uint4* y = reinterpret_cast<uint4*>(base + (size_t)to * p.bytes + at);
  const int t = threadIdx.x;
  if (m == 4 * kThreads) {
    const uint4 w0 = x[t], w1 = x[t + kThreads], w2 = x[t + 2 * kThreads], w3 = x[t + 3 * kThreads];
    y[t] = w0;
    y[t + kThreads] = w1;
    y[t + 2 * kThreads] = w2;
    y[t + 3 * kThreads] = w3;
  } else {
    for (int j = t; j < m; j += kThreads) y[j] = x[j];
  }
}

// Copies src[i] -> dst[i] of both pools in every layer (entries of -1: nothing).
// Destinations are free pages, so no copy reads what another writes.
__global__ __launch_bounds__(kThreads) void k_copy_pages(const int32_t* src, const int32_t* dst, const int32_t* count,
                                                         int n, Pools p) {
  if (count) n = *count;
  for (int i = blockIdx.x; i < n; i += gridDim.x) {
    const int from = src[i], to = dst[i];
    if (from < 0 || to < 0) continue;
    for (int part = blockIdx.y; part < p.parts; part += gridDim.y) copy_part(p, part, from, to);
  }
}

// The end of an update: row 0 of the workgroups writes the slots' rows, all of them
// copy the slots' shared last pages.
__global__ __launch_bounds__(kThreads) void k_table(PagesArgs a, Pools p) {
  const int b = blockIdx.x, base = a.base[b], from = a.src[b];
  const bool fits = base >= 0, copy = fits && from >= 0;
  if (blockIdx.y == 0) write_slot(a, b, base, fits, from, copy);
  if (copy) {
    const int to = a.ids[base];
    for (int part = blockIdx.y; part < p.parts; part += gridDim.y) copy_part(p, part, from, to);
  }
}

// workgroups to a page's parts, so that n pages make about 16384 of them
int part_groups(const Pools& p, int n) {
  const int want = 16384 / n < 1 ? 1 : 16384 / n;
  return want < p.parts ? want : p.parts;
}

hipError_t copy_pages(const dspark_cache& C, const int32_t* src, const int32_t* dst, const int32_t* count, int n,
                      void* k_pool, void* v_pool, hipStream_t s) {
  const Pools p = pools_of(C, k_pool, v_pool);
  const int x = n < 4096 ? n : 4096;
  k_copy_pages<<<dim3(x, part_groups(p, x)), kThreads, 0, s>>>(src, dst, count, n, p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_cache_append(const dspark_cache& C, const AppendArgs& a, hipStream_t s) {
  switch (C.cache_dtype) {
    case DSPARK_F32: return append_typed<DSPARK_F32>(C, a, s);
    case DSPARK_BF16: return append_typed<DSPARK_BF16>(C, a, s);
    case DSPARK_F8E4M3: return append_typed<DSPARK_F8E4M3>(C, a, s);
    default: return append_typed<DSPARK_F8E4M3_TOKEN>(C, a, s);
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
  if (small_pool(C)) {
    k_update_small<<<1, kSmallThreads, 0, s>>>(a);
    const hipError_t e = hipGetLastError();
    return e != hipSuccess ? e : copy_pages(C, a.src, a.dst, nullptr, C.B, k_pool, v_pool, s);
  }
  const int blocks = page_blocks(C.n_pages);
  k_ref_copy<<<(C.n_pages + kThreads - 1) / kThreads, kThreads, 0, s>>>(a);
  k_ref_move<<<C.B, kThreads, 0, s>>>(a);
  k_count<false><<<blocks + (C.B + kThreads - 1) / kThreads, kThreads, 0, s>>>(a, a.ref_out, blocks);
  k_free_list<<<blocks + 1, kThreads, 0, s>>>(a, blocks);
  const Pools p = pools_of(C, k_pool, v_pool);
  k_table<<<dim3(C.B, part_groups(p, C.B)), kThreads, 0, s>>>(a, p);
  return hipGetLastError();
}

hipError_t launch_cache_compact(const dspark_cache& C, const PagesArgs& a, void* k_pool, void* v_pool, hipStream_t s) {
  if (small_pool(C)) {
    k_compact_small<<<1, kSmallThreads, 0, s>>>(a);
    const hipError_t e = hipGetLastError();
    return e != hipSuccess ? e : copy_pages(C, a.src, a.dst, a.n_copies, C.n_pages / 2 + 1, k_pool, v_pool, s);
  }
  const int blocks = page_blocks(C.n_pages);
  k_count<true><<<blocks, kThreads, 0, s>>>(a, a.ref, blocks);
  k_compact_rank<<<blocks, kThreads, 0, s>>>(a, blocks);
  // at most half of the pages can move
  k_compact_table<<<C.B + (C.n_pages / 2 + kThreads) / kThreads, kThreads, 0, s>>>(a);
  const hipError_t e = hipGetLastError();
  return e != hipSuccess ? e : copy_pages(C, a.src, a.dst, a.n_copies, C.n_pages / 2 + 1, k_pool, v_pool, s);
}

}  // namespace dspark
