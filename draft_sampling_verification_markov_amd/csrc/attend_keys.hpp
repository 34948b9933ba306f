// Paged-cache attention for few rows: the four waves of a workgroup hold the same
// rows (NB blocks of 16) and take turns over the keys, so that every key and value is
// loaded by one wave, straight into the registers that the matrix instructions read.
//
// Bound by HBM for a few rows (a decoding token of a group of 4 or 8 query heads):
// nothing is shared between waves, so LDS would only add a trip.  A wave keeps the next
// tile's keys and this tile's values in flight.  Blocks of 16 rows, not 32: half of the
// registers of O and Q, so that more waves are in flight, and half of the softmax's
// work on rows that are not there.  At a segment's end the waves' sums meet in LDS.
// Measured: 256 tokens over up to 4096 keys, 8 heads of 128, bf16 (2.37 GB) 361 us, 6.6 TB/s;
// 2 tokens over up to 200,000 keys, 4 heads of 128, e4m3 (318 MB) 55 us and 5 for the join;
// 256 tokens over up to 4096 keys with scales of their own (1.23 GB) 204 us, 6.0 TB/s.
//
// Weights: the product with bf16 values takes a weight in two bf16 terms, the rounded one
// and the rest (2^-16 of the weight is lost, not 2^-8).  The matrix units wait for memory
// here, so the second product costs next to nothing: 256 tokens over up to 4096 keys bf16
// 373.8 -> 374.2 us, 2 over up to 200,000 e4m3 59.5 -> 60.3.
//
// A tile of keys is two S^T tiles of 16 keys x 16 rows, for fp32 one (two need twice the
// registers of K and V: 64 tokens over 4000 keys, head size 128, 148 -> 106 us; head size
// 256, where they spill, a few hundred keys 37 -> 21).  With lane l = 16 g + c (c < 16):
// S^T register (t, i) holds row (of Q) c, key row 4 g + i of S tile t.  The bf16 product
// with the values takes 8 consecutive keys of each g, so K row m of tile t is read from
// key 8 (m / 4) + 4 t + m % 4; the fp32 product takes one key of each g at a time, 4 g + i
// for i = 0 .. 3, and K row m is key m.
#pragma once

#include "attend_core.hpp"

namespace dspark {

typedef float f32x4_t __attribute__((ext_vector_type(4)));

__device__ __forceinline__ float lane4(const uint4& w, int e) {
  return __uint_as_float(e == 0 ? w.x : e == 1 ? w.y : e == 2 ? w.z : w.w);
}
__device__ __forceinline__ f32x4_t mma16(bf16x8_t x, bf16x8_t y, f32x4_t c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(x, y, c, 0, 0, 0);
}
__device__ __forceinline__ f32x4_t mma16(float x, float y, f32x4_t c) {
  return __builtin_amdgcn_mfma_f32_16x16x4f32(x, y, c, 0, 0, 0);
}

template <int CT, int D>
struct KeysTile {
  static constexpr bool kF32 = CT == DSPARK_F32;
  static constexpr int kEs = Operand<CT>::kBytes;
  static constexpr int kK = D * kEs / 64;  // 16-byte loads of a K row's part in a lane
  static constexpr int kQ = kF32 ? D / 16 : D / 32;
  static constexpr int kS = kF32 ? 1 : 2;  // S^T tiles of 16 keys
  static constexpr int kKeys = 16 * kS;
  static constexpr int kBlocks = D / 16;
  using V = typename std::conditional<is_f8(CT), uint2, uint4>::type;
  // first coordinate of Q register x in lane group g: where K's load has it
  __device__ __forceinline__ static int coord(int x, int g) {
    return kF32 ? 16 * x + 4 * g : CT == DSPARK_BF16 ? 32 * x + 8 * g : 64 * (x >> 1) + 16 * g + 8 * (x & 1);
  }
  __device__ __forceinline__ static int key_of_row(int t, int m) {
    return kF32 ? m : 8 * (m >> 2) + 4 * t + (m & 3);
  }
  // key of S register (t, i) in lane group 0; group g adds kGroupKeys * g
  static constexpr int kGroupKeys = kF32 ? 4 : 8;
  __device__ __forceinline__ static constexpr int key_of_reg(int t, int i) { return 4 * t + i; }
};

// A load of keys or values; ONCE: with the streaming policy.
template <typename V, bool ONCE>
__device__ __forceinline__ V load_key(const char* p) {
  typedef unsigned words_t __attribute__((ext_vector_type(sizeof(V) / 4)));
  const words_t* q = reinterpret_cast<const words_t*>(p);
  return __builtin_bit_cast(V, ONCE ? __builtin_nontemporal_load(q) : *q);
}

// The largest, or the sum, of the four lanes that hold a row.
__device__ __forceinline__ float groups_max(float x) {
  const float2 a = rows16(x);
  return halves32_max(fmaxf(a.x, a.y));
}
__device__ __forceinline__ float groups_sum(float x) {
  const float2 a = rows16(x);
  return halves32_sum(a.x + a.y);
}

template <int CT, int D, int NB, int OCC, bool ONCE, bool TREE>
__global__ __launch_bounds__(kAttendThreads, OCC) void k_attend_keys(AttendArgs a, Split p) {
  using TT = KeysTile<CT, D>;
  constexpr bool kF32 = TT::kF32, kToken = Operand<CT>::kToken;
  constexpr int kRows = NB * 16, kEs = TT::kEs;
  using Data = typename Operand<CT>::Data;
  __shared__ int sh[4];
  __shared__ int odd;  // a value that is not finite was left out
  __shared__ float sm[4][16], sl[4][16];
  __shared__ float4 so[4][D / 4][16];
  const int lane = threadIdx.x & 63, col = lane & 15, g16 = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const CacheView& c = a.c;

  Start s;
  int worker = 0;
  if (p.workers) {
    // neighbouring workers on one XCD (workgroups go round the 8 of them)
    worker = (blockIdx.x & 7) * (p.workers >> 3) + (blockIdx.x >> 3);
    s = find_start<kRows, kAttendThreads, TREE>(a, p, worker, sh);
    if (s.count == 0) {
      if (threadIdx.x == 0) put_record(partials(a, p), s, worker, 0);
      return;
    }
  } else {
    s = whole_segment(a, p);
    if (s.b >= c.B || s.row_tile < 0) return;
  }
  long long left = s.count;
  bool first_segment = true;
  Geometry g = p.workers ? geometry<kRows, TREE>(a, p, s.b, s.row_tile)
                         : geometry<kRows, TREE>(a, p, s.b, s.row_tile, s.n, s.len);
  if (p.workers && threadIdx.x == 0) put_record(partials(a, p), s, worker, g.tiles);
  if (g.tiles == 0) return;  // a direct workgroup without rows

  while (true) {
    const int t0 = g.tile0 + s.skip, take = (int)min(left, (long long)(g.tiles - s.skip)), t1 = t0 + take;
    const int head = s.head, blocks = (g.rows + 15) >> 4;

    // ---- keys: this wave's tiles, every fourth one of the units that some row sees.
    // Page ids come over the scalar cache two tiles ahead, keys one tile ahead; past the
    // last tile the last one is loaded again, so that the loop has no branch that would
    // make the waits for its loads inexact.
    constexpr int kTurn = 4 * TT::kKeys;  // keys that the four waves take
    int key0 = (t0 << 7) + TT::kKeys * wave, last = (t1 << 7) - kTurn + TT::kKeys * wave;
    while (key0 + TT::kKeys <= g.lo && key0 <= last) key0 += kTurn;
    while (last >= g.hi && last >= key0) last -= kTurn;
    const int off_mask = (1 << c.page_shift) - 1;
    const char* const kp = static_cast<const char*>(a.k_pool);
    const char* const vp = static_cast<const char*>(a.v_pool);
    const TableRow row(c, g.b);
    struct Ids { int a, b; };  // of each 16 keys of the tile
    auto ids_of = [&](int key) __attribute__((always_inline)) { return Ids{row.raw(key), TT::kS == 2 ? row.raw(key + 16) : 0}; };
    auto token = [&](int id, int key) __attribute__((always_inline)) {  // first byte of 16 consecutive tokens
      return token_at<CT, D>(c, row.id(id), head, key & off_mask);
    };
    // scales of the lane's 8 keys of the tile, those of its scores and weights
    auto load_scales = [&](const char* pool, int key0_, Ids id, float4(&s)[2]) __attribute__((always_inline)) {
      const int key = key0_ + 8 * g16;
      const char* src = pool + scale_at<D>(c, row.id(g16 < 2 ? id.a : id.b), head, key & off_mask);
#pragma unroll
      for (int t = 0; t < 2; ++t) s[t] = load_key<float4, ONCE>(src + 16 * t);
    };
    auto load_k = [&](int key0_, Ids id, uint4(&k)[TT::kS][TT::kK]) __attribute__((always_inline)) {
      const size_t half[2] = {token(id.a, key0_), token(id.b, key0_ + 16)};
#pragma unroll
      for (int t = 0; t < TT::kS; ++t) {
        const int key = TT::key_of_row(t, col);
        const char* src = kp + (kF32 || col < 8 ? half[0] : half[1]) + (key & 15) * (D * kEs) + 16 * g16;
#pragma unroll
        for (int x = 0; x < TT::kK; ++x) k[t][x] = load_key<uint4, ONCE>(src + 64 * x);
      }
    };
    uint4 k[TT::kS][TT::kK];
    float4 k_scale[2], v_scale[2];
    Ids id0{}, id1{};
    if (key0 <= last) {
      id0 = ids_of(key0);
      id1 = ids_of(min(key0 + kTurn, last));
      load_k(key0, id0, k);
      if constexpr (kToken) load_scales(kp, key0, id0, k_scale);
    }

    // ---- rows
    const Masks mask{a.causal, a.window, g.pos0 + g.n};
    const int G = c.Hq / c.Hkv;
    uint4 q[NB][TT::kQ];
    RowKeys<TREE> keys[NB];
    if (threadIdx.x == 0) odd = 0;
    Running run[NB];
    f32x4_t acc[NB][TT::kBlocks];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      run[nb].m = -INFINITY;
      run[nb].l = 0.f;
#pragma unroll
      for (int db = 0; db < TT::kBlocks; ++db) acc[nb][db] = f32x4_t{};
      const int rho = nb * 16 + col;
      keys[nb] = {0, 0x7fffffff};  // a column without a row sees everything and is left out at the end
      int hq = 0;
      long long r = -1;
      if (rho < g.rows) {
        r = global_row(a, g, rho, head, hq);
        keys[nb] = row_keys<TREE>(a, g, mask, (g.row0 + rho) / G, r);
      }
      const Data* src = static_cast<const Data*>(a.q) + (r >= 0 ? r * a.q_stride + (size_t)hq * D : 0);
#pragma unroll
      for (int x = 0; x < TT::kQ; ++x) q[nb][x] = *reinterpret_cast<const uint4*>(src + TT::coord(x, g16));
      const uint32_t there = r >= 0 ? ~0u : 0u;
#pragma unroll
      for (int x = 0; x < TT::kQ; ++x)
        q[nb][x] = make_uint4(q[nb][x].x & there, q[nb][x].y & there, q[nb][x].z & there, q[nb][x].w & there);
    }
    const float ks = score_factor<CT>(a, head);
    __syncthreads();

    for (; key0 <= last; key0 += kTurn) {
      const int next = min(key0 + kTurn, last);
      const Ids id2 = ids_of(min(key0 + 2 * kTurn, last));
      typename TT::V v[TT::kBlocks];
      {
        // the lane's 8 (fp32: 4) keys of coordinate 16 db + col
        const size_t half[2] = {token(id0.a, key0), token(id0.b, key0 + 16)};
        const char* src = kF32 ? vp + half[0] + ((g16 >> 1) * D + col) * 32 + 16 * (g16 & 1)
                               : vp + (g16 < 2 ? half[0] : half[1]) + ((g16 & 1) * D + col) * (8 * kEs);
#pragma unroll
        for (int db = 0; db < TT::kBlocks; ++db) v[db] = load_key<typename TT::V, ONCE>(src + db * (16 * 8 * kEs));
        if constexpr (kToken) load_scales(vp, key0, id0, v_scale);
      }
      f32x4_t w[NB][TT::kS];
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int t = 0; t < TT::kS; ++t) {
          w[nb][t] = f32x4_t{};
          if (nb < blocks) {
#pragma unroll
            for (int x = 0; x < TT::kK; ++x) {
              if constexpr (kF32) {
#pragma unroll
                for (int e = 0; e < 4; ++e) w[nb][t] = mma16(lane4(k[t][x], e), lane4(q[nb][x], e), w[nb][t]);
              } else if constexpr (CT == DSPARK_BF16) {
                w[nb][t] = mma16(as_bf16x8(k[t][x]), as_bf16x8(q[nb][x]), w[nb][t]);
              } else {
                w[nb][t] = mma16(f8_to_bf16x8(k[t][x].x, k[t][x].y), as_bf16x8(q[nb][2 * x]), w[nb][t]);
                w[nb][t] = mma16(f8_to_bf16x8(k[t][x].z, k[t][x].w), as_bf16x8(q[nb][2 * x + 1]), w[nb][t]);
              }
            }
          }
        }
      if constexpr (kToken) {
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int t = 0; t < TT::kS; ++t) w[nb][t] *= f32x4_t{k_scale[t].x, k_scale[t].y, k_scale[t].z, k_scale[t].w};
        load_scales(kp, next, id1, k_scale);
      }
      load_k(next, id1, k);
      id0 = id1;
      id1 = id2;
      if (key0 < g.all_lo || key0 + TT::kKeys > g.all_hi) {  // not every row sees the whole tile
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          if constexpr (TREE) {
            const uint32_t seen = tree_seen(a, g, keys[nb], key0) >> (TT::kGroupKeys * g16);
#pragma unroll
            for (int t = 0; t < TT::kS; ++t)
#pragma unroll
              for (int i = 0; i < 4; ++i)
                w[nb][t][i] = seen >> TT::key_of_reg(t, i) & 1u ? w[nb][t][i] : -INFINITY;
            continue;
          }
          const int from = keys[nb].lo - key0 - TT::kGroupKeys * g16;
          const unsigned n = max(0, keys[nb].hi - keys[nb].lo);
#pragma unroll
          for (int t = 0; t < TT::kS; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              w[nb][t][i] = (unsigned)(TT::key_of_reg(t, i) - from) < n ? w[nb][t][i] : -INFINITY;
        }
        if constexpr (kToken) {
#pragma unroll
          for (int t = 0; t < TT::kS; ++t) v_scale[t] = finite_scales(v_scale[t]);
        }
        uint32_t bits = 0;
#pragma unroll
        for (int db = 0; db < TT::kBlocks; ++db) find_nonfinite<CT>(v[db], bits);
        if (__builtin_expect(__any(bits & kOdd<CT>), 0)) {
          odd = 1;
#pragma unroll
          for (int db = 0; db < TT::kBlocks; ++db) v[db] = finite_part<CT>(v[db]);
        }
      }
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
        if (nb < blocks) {
          float top = w[nb][0][0];
#pragma unroll
          for (int t = 0; t < TT::kS; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) top = fmaxf(top, w[nb][t][i]);
          top = groups_max(top) * ks;
          if (__any(top > run[nb].m + kRescale)) {
            const float fade = fade_to(run[nb], top);
#pragma unroll
            for (int db = 0; db < TT::kBlocks; ++db) acc[nb][db] *= fade;
          }
          const float ref = run[nb].m == -INFINITY ? 0.f : run[nb].m;
          float sum = 0.f;
#pragma unroll
          for (int t = 0; t < TT::kS; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              w[nb][t][i] = __builtin_amdgcn_exp2f(fmaf(w[nb][t][i], ks, -ref));
              sum += w[nb][t][i];
            }
          run[nb].l += sum;
          if constexpr (kF32) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
#pragma unroll
              for (int db = 0; db < TT::kBlocks; ++db)
                acc[nb][db] = mma16(lane4(v[db], e), w[nb][0][e], acc[nb][db]);
          } else {
            bf16x8_t pw, rest;  // the weights in bf16, and what that leaves of them
#pragma unroll
            for (int t = 0; t < TT::kS; ++t) {
              if constexpr (kToken) w[nb][t] *= f32x4_t{v_scale[t].x, v_scale[t].y, v_scale[t].z, v_scale[t].w};
#pragma unroll
              for (int i = 0; i < 4; i += 2) {
                const f32x2_t x{w[nb][t][i], w[nb][t][i + 1]};
                const bf16x2_t y = __builtin_convertvector(x, bf16x2_t);
                const bf16x2_t z = __builtin_convertvector(f32x2_t{x[0] - (float)y[0], x[1] - (float)y[1]}, bf16x2_t);
                pw[4 * t + i] = y[0];
                pw[4 * t + i + 1] = y[1];
                rest[4 * t + i] = z[0];
                rest[4 * t + i + 1] = z[1];
              }
            }
#pragma unroll
            for (int db = 0; db < TT::kBlocks; ++db) {
              const bf16x8_t x = value_operand<CT>(v[db]);
              acc[nb][db] = mma16(x, pw, acc[nb][db]);
              acc[nb][db] = mma16(x, rest, acc[nb][db]);
            }
          }
        }
    }

    // ---- the four waves' sums
    const bool whole = take == g.tiles;
    const float vs = CT == DSPARK_F8E4M3 ? a.v_scale[head] : 1.f;
    float* const slot = whole ? nullptr : partials(a, p).template slot<D, kRows>(2 * worker + (first_segment ? 0 : 1));
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
      if (nb < blocks) {
        const float l = groups_sum(run[nb].l);
        if (g16 == 0) {
          sm[wave][col] = run[nb].m;
          sl[wave][col] = l;
        }
        __syncthreads();
        const float m = fmaxf(fmaxf(sm[0][col], sm[1][col]), fmaxf(sm[2][col], sm[3][col]));
        const float f = run[nb].m == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(run[nb].m - m);
#pragma unroll
        for (int db = 0; db < TT::kBlocks; ++db)
          so[wave][4 * db + g16][col] = make_float4(acc[nb][db][0] * f, acc[nb][db][1] * f, acc[nb][db][2] * f,
                                                    acc[nb][db][3] * f);
        __syncthreads();
#pragma unroll 1
        for (int at = threadIdx.x; at < 16 * (D / 4); at += kAttendThreads) {
          const int d4 = at % (D / 4), r = at / (D / 4), rho = nb * 16 + r;
          if (rho >= g.rows) break;
          const float top = fmaxf(fmaxf(sm[0][r], sm[1][r]), fmaxf(sm[2][r], sm[3][r]));
          float sum = 0.f;
#pragma unroll
          for (int w4 = 0; w4 < 4; ++w4)
            sum += sm[w4][r] == -INFINITY ? sl[w4][r] : sl[w4][r] * __builtin_amdgcn_exp2f(sm[w4][r] - top);
          const float4 o0 = so[0][d4][r], o1 = so[1][d4][r], o2 = so[2][d4][r], o3 = so[3][d4][r];
          float4 y = make_float4(o0.x + o1.x + o2.x + o3.x, o0.y + o1.y + o2.y + o3.y, o0.z + o1.z + o2.z + o3.z,
                                 o0.w + o1.w + o2.w + o3.w);
          if (__builtin_expect(odd, 0)) {
            int hq;
            const long long at_row = global_row(a, g, rho, head, hq);
            if (!TREE || at_row >= 0)
              add_nonfinite<CT, D, TT::kKeys, TREE>(a, g, row_keys<TREE>(a, g, mask, (g.row0 + rho) / G, at_row), head,
                                                    4 * d4, t0 << 7, t1 << 7, y);
          }
          if (whole) {
            int hq;
            const long long to = global_row(a, g, rho, head, hq);
            if (to >= 0) {
              const float fr = row_factor(sum, vs);
              if (sum == 0.f) y = make_float4(0.f, 0.f, 0.f, 0.f);
              store4<CT>(a.out, to * a.out_stride + (size_t)hq * D + 4 * d4,
                         make_float4(y.x * fr, y.y * fr, y.z * fr, y.w * fr));
              if (a.lse && d4 == 0) a.lse[to * c.Hq + hq] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * kLn2f;
            }
          } else {
            *reinterpret_cast<float4*>(slot + (size_t)rho * D + 4 * d4) = y;
            if (d4 == 0) *reinterpret_cast<float2*>(slot + (size_t)kRows * D + 2 * rho) = make_float2(top, sum);
          }
        }
        __syncthreads();
      }

    // ---- next segment
    if (!p.workers) return;
    left -= take;
    if (left <= 0) return;
    first_segment = false;
    g = next_segment<kRows, TREE>(a, p, s);
  }
}

}  // namespace dspark
