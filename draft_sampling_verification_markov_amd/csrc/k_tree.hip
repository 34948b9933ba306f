// Drafted trees over the paged cache: the nodes' ancestors, and the accepted path's move to
// the front of the tree.  See include/dspark_tree.h for the contract.
#include <type_traits>

#include "dspark_cache_internal.hpp"

namespace dspark {
namespace {

constexpr int kThreads = 256;

// ------------------------------------------------------------------ ancestors
// A workgroup a request, a thread a node: it walks up to the root through the parents in
// LDS.  Ancestors come in descending order, so the row's words are finished from the last
// one down.  The walk ends: a parent that is not an earlier node is none.  One tree of 16 takes
// 2.1 us, 256 of up to 64 3.7: a launch, two loads and a few dozen steps in LDS.
__global__ __launch_bounds__(kThreads) void k_tree_mask(TreeMaskArgs a) {
  __shared__ int16_t up[kMaxNodes];
  const int b = blockIdx.x;
  const int n = a.n_new ? min(max(a.n_new[b], 0), a.max_new) : a.max_new;
  const long long row0 = a.row_start ? (long long)a.row_start[b] : (long long)b * a.max_new;
  auto has = [&](int i) { return row0 + i >= 0 && row0 + i < a.n_rows; };
  for (int i = threadIdx.x; i < n; i += kThreads) {
    const int p = has(i) ? a.parent[row0 + i] : -1;
    up[i] = (int16_t)((unsigned)p < (unsigned)i ? p : -1);
  }
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += kThreads) {
    if (!has(i)) continue;
    uint32_t* const row = a.mask + (row0 + i) * a.words;
    int w = a.words - 1, depth = 0;
    uint32_t bits = 0;
    for (int node = i; node >= 0; node = up[node], ++depth) {
      for (; w > node >> 5; --w) {
        row[w] = bits;
        bits = 0;
      }
      if (a.window == 0 || depth < a.window) bits |= 1u << (node & 31);
    }
    for (; w >= 0; --w) {
      row[w] = bits;
      bits = 0;
    }
    if (a.depth) a.depth[row0 + i] = depth - 1;
  }
}

// ------------------------------------------------------------------ the accepted path
// A thread owns a piece of every token: 16 bytes of a key, one coordinate of a value, or a
// scale.  It moves the path's tokens in order, eight at a time: a node's place is at or
// before the place that it comes from, and before those of all later nodes, so eight loads
// may go ahead of their stores.  Values are written as whole groups of 8 tokens of the
// coordinate, merged with what the group holds.  Few bytes, in small pieces: a value's token is
// every eighth element of 2 KB (bf16, head size 128), and each thread waits for lengths -> path ->
// table -> tokens.  256 paths of up to 8 among up to 32 nodes, 4 layers of 8 x 128: 17 us (29 MB
// in and out, 35 counted); one of 5, 2 layers 2.5.  A workgroup over several layers, its places
// looked up once and two layers in flight, took 18.
constexpr uint32_t kNone = 0xFFFFFFFFu;

template <int CT, int D>
__global__ __launch_bounds__(kThreads) void k_tree_keep(KeepArgs a, int key_parts) {
  using T = typename std::conditional<CT == DSPARK_F32, uint32_t, typename std::conditional<CT == DSPARK_BF16, uint16_t, uint8_t>::type>::type;
  constexpr int kEs = sizeof(T), kPieces = D * kEs / 16, kSb = scale_bytes(CT), kAhead = 8;
  // page << 8 | offset of the path's nodes; kNone: not there (a pool of 2^24 pages of 256 tokens
  // would be larger than the card's memory)
  __shared__ uint32_t from[kMaxPath];
  const CacheView& c = a.c;
  const int b = blockIdx.x;
  const int n = c.rows(b), len = c.len(b), base = len - n;
  const int m = min(min(max(a.n_keep[b], 0), a.max_path), n);
  if (blockIdx.y == 0 && blockIdx.z == 0 && threadIdx.x == 0) a.length_out[b] = max(0, base + m);
  const int32_t* const pages = c.table + (size_t)b * c.max_pages;
  const int off_mask = (1 << c.page_shift) - 1;
  auto place = [&](int pos) {  // of a position that the sequence has
    const int page = pages[pos >> c.page_shift];
    return (unsigned)page < (unsigned)c.n_pages ? (uint32_t)page << 8 | (uint32_t)(pos & off_mask) : kNone;
  };
  for (int i = threadIdx.x; i < m; i += kThreads) {
    const int node = a.path[(size_t)b * a.max_path + i];
    // (a node that is already in its place stays)
    from[i] = (unsigned)node < (unsigned)n && node != i && base + node >= 0 && base + i >= 0 ? place(base + node) : kNone;
  }
  __syncthreads();
  if (m == 0) return;
  const size_t layer = (size_t)blockIdx.z * a.layer_bytes;
  auto block = [&](char* pool, uint32_t at, int head) {
    return pool + layer + ((size_t)((at >> 8) * (unsigned)c.Hkv + head) << c.page_shift) * (D * kEs + kSb);
  };
  const bool keys = (int)blockIdx.y < key_parts;
  int unit = ((int)blockIdx.y - (keys ? 0 : key_parts)) * kThreads + threadIdx.x;
  if (keys) {
    if (unit < c.Hkv * kPieces) {
      const int head = unit / kPieces, piece = unit % kPieces;
      auto key = [&](uint32_t at) {
        return reinterpret_cast<uint4*>(block(a.k_pool, at, head) + (at & 255) * (D * kEs)) + piece;
      };
      for (int i0 = 0; i0 < m; i0 += kAhead) {
        uint4 x[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
          if (i0 + i < m && from[i0 + i] != kNone) x[i] = *key(from[i0 + i]);
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
          if (i0 + i < m && from[i0 + i] != kNone) {
            const uint32_t to = place(base + i0 + i);
            if (to != kNone) *key(to) = x[i];
          }
      }
    } else if (kSb && (unit -= c.Hkv * kPieces) < 2 * c.Hkv) {
      char* const pool = unit < c.Hkv ? a.k_pool : a.v_pool;
      const int head = unit % c.Hkv;
      for (int i = 0; i < m; ++i) {
        if (from[i] == kNone) continue;
        const uint32_t to = place(base + i);
        auto scale = [&](uint32_t at) {
          return reinterpret_cast<float*>(block(pool, at, head) + ((size_t)(D * kEs) << c.page_shift)) + (at & 255);
        };
        if (to != kNone) *scale(to) = *scale(from[i]);
      }
    }
    return;
  }
  if (unit >= c.Hkv * D) return;
  const int head = unit / D, d = unit % D;
  auto line = [&](uint32_t at) {  // the group of 8 tokens that `at` lies in
    return reinterpret_cast<T*>(block(a.v_pool, at, head) + (size_t)((at & 255 & ~7u) * D + d * 8) * kEs);
  };
  struct __attribute__((aligned(8 * sizeof(T) < 16 ? 8 * sizeof(T) : 16))) Line { T x[8]; };
  for (int g0 = max(base, 0) & ~7; g0 < base + m; g0 += 8) {
    const uint32_t to = place(g0);
    if (to == kNone) continue;
    T x[8];
    bool any = false, has[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int k = g0 + i - base;  // of the path
      has[i] = k >= 0 && k < m && from[k] != kNone;
      any |= has[i];
      if (has[i]) x[i] = line(from[k])[from[k] & 7];
    }
    if (!any) continue;
    Line w = *reinterpret_cast<const Line*>(line(to));
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (has[i]) w.x[i] = x[i];
    *reinterpret_cast<Line*>(line(to)) = w;
  }
}

template <int CT, int D>
hipError_t keep(const dspark_cache& C, const KeepArgs& a, hipStream_t s) {
  const int pieces = D * element_bytes(CT) / 16 + (scale_bytes(CT) ? 2 : 0);  // of the keys, and the scales
  const int key_parts = (C.Hkv * pieces + kThreads - 1) / kThreads, value_parts = (C.Hkv * D + kThreads - 1) / kThreads;
  k_tree_keep<CT, D><<<dim3(C.B, key_parts + value_parts, C.n_layers), kThreads, 0, s>>>(a, key_parts);
  return hipGetLastError();
}

template <int CT>
hipError_t keep_type(const dspark_cache& C, const KeepArgs& a, hipStream_t s) {
  return C.D == 64 ? keep<CT, 64>(C, a, s) : C.D == 128 ? keep<CT, 128>(C, a, s) : keep<CT, 256>(C, a, s);
}

}  // namespace

hipError_t launch_tree_mask(const TreeMaskArgs& a, hipStream_t s) {
  k_tree_mask<<<a.B, kThreads, 0, s>>>(a);
  return hipGetLastError();
}

hipError_t launch_tree_keep(const dspark_cache& C, const KeepArgs& a, hipStream_t s) {
  switch (C.cache_dtype) {
    case DSPARK_F32: return keep_type<DSPARK_F32>(C, a, s);
    case DSPARK_BF16: return keep_type<DSPARK_BF16>(C, a, s);
    case DSPARK_F8E4M3: return keep_type<DSPARK_F8E4M3>(C, a, s);
    default: return keep_type<DSPARK_F8E4M3_TOKEN>(C, a, s);
  }
}

}  // namespace dspark
