// Paged-cache attention for few rows: the four waves of a workgroup hold the same
// rows (NB blocks of 32) and take turns over the keys, so that every key and value is
// loaded by one wave, straight into the registers that the matrix instructions read.
//
// Bound by HBM for a few rows (a decoding token of a group of 4 or 8 query heads, a
// verification block): nothing is shared between waves, so LDS would only add a trip.
// A wave keeps the next tile's keys and this tile's values in flight.  At a segment's
// end the waves' sums meet in LDS.
#pragma once

#include "attend_core.hpp"

namespace dspark {

template <int CT, int D, int NB, int OCC>
__global__ __launch_bounds__(kAttendThreads, OCC) void k_attend_keys(AttendArgs a, Split p) {
  using TT = Tile<CT, D>;
  constexpr bool kF32 = TT::kF32;
  constexpr int kQ = q_regs<CT, D>(), kRows = NB * 32, kEs = Operand<CT>::kBytes;
  using Data = typename Operand<CT>::Data;
  __shared__ int sh[4];
  __shared__ int odd;  // a value that is not finite was left out
  __shared__ float sm[4][32], sl[4][32];
  __shared__ float4 so[4][D / 4][32];
  const int lane = threadIdx.x & 63, col = lane & 31, h = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const CacheView& c = a.c;

  Start s;
  int worker = 0;
  if (p.workers) {
    // neighbouring workers on one XCD (workgroups go round the 8 of them)
    worker = (blockIdx.x & 7) * (p.workers >> 3) + (blockIdx.x >> 3);
    s = find_start<kRows, kAttendThreads>(a, p, worker, sh);
    if (s.count == 0) {
      if (threadIdx.x == 0) put_record(partials(a, p), s, worker, 0);
      return;
    }
  } else {
    s = whole_segment(a, p);
    if (s.b >= c.B) return;
  }
  int left = s.count;
  bool first_segment = true;
  Geometry g = geometry<kRows>(a, p, s.b, s.row_tile);
  if (p.workers && threadIdx.x == 0) put_record(partials(a, p), s, worker, g.tiles);
  if (g.tiles == 0) return;  // a direct workgroup without rows

  while (true) {
    const int t0 = g.tile0 + s.skip, take = min(left, g.tiles - s.skip), t1 = t0 + take;
    const int head = s.head, blocks = (g.rows + 31) >> 5;

    // ---- rows
    const Masks mask{a.causal, a.window, c.len(g.b)};
    const int G = c.Hq / c.Hkv;
    uint4 q[NB][kQ];
    int row_lo[NB], row_hi[NB];
    if (threadIdx.x == 0) odd = 0;
    __syncthreads();
    Running run[NB];
    f32x16_t acc[NB][TT::kBlocks];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      run[nb].m = -INFINITY;
      run[nb].l = 0.f;
#pragma unroll
      for (int db = 0; db < TT::kBlocks; ++db) acc[nb][db] = f32x16_t{};
      const int rho = nb * 32 + col;
      row_lo[nb] = 0;  // a column without a row sees everything and is left out at the end
      row_hi[nb] = 0x7fffffff;
      int hq;
      long long r = -1;
      if (rho < g.rows) {
        r = global_row(a, g, rho, head, hq);
        const int pos = g.pos0 + (g.row0 + rho) / G;
        row_lo[nb] = mask.lo(pos);
        row_hi[nb] = mask.hi(pos);
      }
      const Data* src = static_cast<const Data*>(a.q) + (r >= 0 ? r * a.q_stride + (size_t)hq * D : 0);
#pragma unroll
      for (int x = 0; x < kQ; ++x) q[nb][x] = *reinterpret_cast<const uint4*>(src + coord<CT>(x, h));
      const uint32_t there = r >= 0 ? ~0u : 0u;
#pragma unroll
      for (int x = 0; x < kQ; ++x)
        q[nb][x] = make_uint4(q[nb][x].x & there, q[nb][x].y & there, q[nb][x].z & there, q[nb][x].w & there);
    }
    const float ks = CT == DSPARK_F8E4M3 ? a.scale2 * a.k_scale[head] : a.scale2;

    // ---- keys
    // This wave's tiles: every fourth one of the units that some row sees.  Page ids come
    // over the scalar cache two tiles ahead, keys one tile ahead; past the last tile the
    // last one is loaded again, so that the loop has no branch that would make the waits
    // for its loads inexact.
    int key0 = (t0 << 7) + 32 * wave, last = ((t1 - 1) << 7) + 32 * wave;
    if (key0 + 32 <= g.lo) key0 += 128;
    while (last >= g.hi && last >= key0) last -= 128;
    const int off_mask = (1 << c.page_shift) - 1;
    const char* const kp = static_cast<const char*>(a.k_pool);
    const char* const vp = static_cast<const char*>(a.v_pool);
    const TableRow row(c, g.b);
    struct Ids { int a, b; };  // of the tile's two halves of 16 keys
    auto ids_of = [&](int key) __attribute__((always_inline)) { return Ids{row.raw(key), row.raw(key + 16)}; };
    auto token = [&](int id, int key) __attribute__((always_inline)) {  // first byte of 16 consecutive tokens
      return (((size_t)(row.id(id) * (unsigned)c.Hkv + head) << c.page_shift) + (key & off_mask)) * (D * kEs);
    };
    auto load_k = [&](int key0_, Ids id, uint4(&k)[TT::kK]) __attribute__((always_inline)) {
      const size_t ta = token(id.a, key0_), tb = token(id.b, key0_ + 16);
      const int key = key_of_row<kF32>(col) & 15;
      const char* src = kp + (col < 16 ? ta : tb) + key * (D * kEs) + 16 * h;
#pragma unroll
      for (int x = 0; x < TT::kK; ++x) k[x] = *reinterpret_cast<const uint4*>(src + 32 * x);
    };
    uint4 k[TT::kK];
    Ids id0{}, id1{};
    if (key0 <= last) {
      id0 = ids_of(key0);
      id1 = ids_of(min(key0 + 128, last));
      load_k(key0, id0, k);
    }
    for (; key0 <= last; key0 += 128) {
      const int next = min(key0 + 128, last);
      const Ids id2 = ids_of(min(key0 + 256, last));
      typename TT::V v[TT::kSlabs][TT::kBlocks];
      {
        const size_t tok[2] = {token(id0.a, key0), token(id0.b, key0 + 16)};
#pragma unroll
        for (int sl_ = 0; sl_ < TT::kSlabs; ++sl_) {
          // fp32: slab j is the 8-token group j, half h its tokens 4 h ..; else slab s has the groups 2 s + h
          const char* src = kF32 ? vp + tok[sl_ >> 1] + ((sl_ & 1) * D + col) * 32 + 16 * h
                                 : vp + tok[sl_] + (h * D + col) * (8 * kEs);
#pragma unroll
          for (int db = 0; db < TT::kBlocks; ++db)
            v[sl_][db] = *reinterpret_cast<const typename TT::V*>(src + db * (32 * 8 * kEs));
        }
      }
      f32x16_t w[NB];
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
        w[nb] = nb < blocks ? scores<CT, D>(k, q[nb]) : f32x16_t{};
      load_k(next, id1, k);
      id0 = id1;
      id1 = id2;
      const bool full = key0 >= g.all_lo && key0 + 32 <= g.all_hi;
      if (!full) {
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) mask_scores<kF32>(w[nb], row_lo[nb] - key0, row_hi[nb] - key0, h);
        uint32_t bits = 0;
#pragma unroll
        for (int sl_ = 0; sl_ < TT::kSlabs; ++sl_)
#pragma unroll
          for (int db = 0; db < TT::kBlocks; ++db) find_nonfinite<CT>(v[sl_][db], bits);
        if (__any(bits & kOdd<CT>)) {
          odd = 1;
#pragma unroll
          for (int sl_ = 0; sl_ < TT::kSlabs; ++sl_)
#pragma unroll
            for (int db = 0; db < TT::kBlocks; ++db) v[sl_][db] = finite_part<CT>(v[sl_][db]);
        }
      }
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
        if (nb < blocks) {
          const f32x16_t(&one)[1] = reinterpret_cast<const f32x16_t(&)[1]>(w[nb]);
          const float fade = raise_max(one, run[nb], ks);
          if (__any(fade != 1.f)) {
#pragma unroll
            for (int db = 0; db < TT::kBlocks; ++db) acc[nb][db] *= fade;
          }
          weights(w[nb], run[nb], ks);
          add_values<CT, D>(v, w[nb], acc[nb]);
        }
    }

    // ---- the four waves' sums
    const bool whole = take == g.tiles;
    const float vs = CT == DSPARK_F8E4M3 ? a.v_scale[head] : 1.f;
    float* const slot = whole ? nullptr : partials(a, p).template slot<D, kRows>(2 * worker + (first_segment ? 0 : 1));
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
      if (nb < blocks) {
        const float l = halves32_sum(run[nb].l);
        if (h == 0) {
          sm[wave][col] = run[nb].m;
          sl[wave][col] = l;
        }
        __syncthreads();
        const float m = fmaxf(fmaxf(sm[0][col], sm[1][col]), fmaxf(sm[2][col], sm[3][col]));
        const float f = run[nb].m == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(run[nb].m - m);
#pragma unroll
        for (int db = 0; db < TT::kBlocks; ++db)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            so[wave][8 * db + 2 * j + h][col] = make_float4(acc[nb][db][4 * j] * f, acc[nb][db][4 * j + 1] * f,
                                                            acc[nb][db][4 * j + 2] * f, acc[nb][db][4 * j + 3] * f);
        __syncthreads();
#pragma unroll 1
        for (int i = 0; i < 32 * (D / 4) / kAttendThreads; ++i) {
          const int at = i * kAttendThreads + threadIdx.x, d4 = at % (D / 4), r = at / (D / 4), rho = nb * 32 + r;
          if (rho < g.rows) {
            float top = fmaxf(fmaxf(sm[0][r], sm[1][r]), fmaxf(sm[2][r], sm[3][r])), sum = 0.f;
#pragma unroll
            for (int w4 = 0; w4 < 4; ++w4)
              sum += sm[w4][r] == -INFINITY ? sl[w4][r] : sl[w4][r] * __builtin_amdgcn_exp2f(sm[w4][r] - top);
            const float4 o0 = so[0][d4][r], o1 = so[1][d4][r], o2 = so[2][d4][r], o3 = so[3][d4][r];
            float4 y = make_float4(o0.x + o1.x + o2.x + o3.x, o0.y + o1.y + o2.y + o3.y, o0.z + o1.z + o2.z + o3.z,
                                   o0.w + o1.w + o2.w + o3.w);
            if (odd) {
              const int pos = g.pos0 + (g.row0 + rho) / G;
              add_nonfinite<CT, D, 32>(a, g, mask, head, pos, 4 * d4, t0 << 7, t1 << 7, y);
            }
            if (whole) {
              int hq;
              const long long row = global_row(a, g, rho, head, hq);
              if (row >= 0) {
                const float fr = row_factor(sum, vs);
                if (sum == 0.f) y = make_float4(0.f, 0.f, 0.f, 0.f);
                store4<CT>(a.out, row * a.out_stride + (size_t)hq * D + 4 * d4,
                           make_float4(y.x * fr, y.y * fr, y.z * fr, y.w * fr));
                if (a.lse && d4 == 0) a.lse[row * c.Hq + hq] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * kLn2f;
              }
            } else {
              *reinterpret_cast<float4*>(slot + (size_t)rho * D + 4 * d4) = y;
              if (d4 == 0) *reinterpret_cast<float2*>(slot + (size_t)kRows * D + 2 * rho) = make_float2(top, sum);
            }
          }
        }
        __syncthreads();
      }

    // ---- next segment
    if (!p.workers) return;
    left -= take;
    if (left <= 0) return;
    first_segment = false;
    g = next_segment<kRows>(a, p, s);
  }
}

}  // namespace dspark
