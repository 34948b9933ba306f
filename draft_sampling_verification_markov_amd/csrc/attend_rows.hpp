// Paged-cache attention for many rows (prompt chunks, verification blocks of wide
// groups): every wave of a workgroup has its own NB blocks of 32 rows, and the key
// tiles pass through LDS once for all four waves.
//
// Bound by the matrix units (and, next to them, by the exponentials of the softmax).
// A tile of kKeys keys and values comes by LDS DMA (16 bytes a lane) into one of two
// buffers while the other is used; the buffers are distinct __shared__ objects, so that
// the compiler lets reads of one pass the DMA into the other.  Reading a fragment from
// LDS serves NB products.
//
// LDS layout.  Keys: 16-byte pieces, row m of the tile's 32-key halves holding key
// key_of_row(m); piece c of row r lies at c ^ swizzle(r), which spreads the 16 rows that
// one LDS cycle reads over all banks.  Values: as in the pool, (8-key group, coordinate)
// pieces in order, read without conflicts.
#pragma once

#include "attend_core.hpp"

namespace dspark {

template <int CT, int D, int NB>
struct RowsShape {
  static constexpr int kEs = Operand<CT>::kBytes;
  static constexpr int kKeys = D == 256 ? 32 : 64;           // of a tile
  static constexpr int kSubs = kKeys / 32;
  static constexpr int kRows = 4 * NB * 32;                  // of a workgroup
  static constexpr int kBytes = kKeys * D * kEs;             // of the keys (or the values) of a tile
  static constexpr int kPieces = D * kEs / 16;               // of a key
  static constexpr int kOps = kBytes / 1024 / 4;             // DMA instructions a wave, keys (or values)
  // 64 banks of 4 bytes: 16 pieces a cycle, one or more rows of keys
  __device__ __forceinline__ static int swizzle(int r) { return kPieces >= 16 ? r & 15 : (r / (16 / kPieces)) & (kPieces - 1); }
};

// 64 lanes x 16 bytes from each lane's own address to 1 KB of LDS, in lane order
__device__ __forceinline__ void dma_1k(const char* src, unsigned char* lds) {
  __builtin_amdgcn_global_load_lds(src, (__attribute__((address_space(3))) void*)lds, 16, 0, 0);
}

template <int CT, int D, int NB, int OCC>
__global__ __launch_bounds__(kAttendThreads, OCC) void k_attend_rows(AttendArgs a, Split p) {
  using S = RowsShape<CT, D, NB>;
  using TT = Tile<CT, D>;
  constexpr int kQ = q_regs<CT, D>(), kRows = S::kRows, kEs = S::kEs;
  constexpr int kWavesPerSub16 = 4 / (S::kKeys / 16);  // waves that share the DMA of 16 keys
  __shared__ __attribute__((aligned(1024))) unsigned char k0[S::kBytes], k1[S::kBytes], v0[S::kBytes], v1[S::kBytes];
  __shared__ int sh[4];
  __shared__ int odd;  // a value that is not finite was replaced
  const int lane = threadIdx.x & 63, col = lane & 31, h = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const CacheView& c = a.c;

  Start s;
  int worker = 0;
  if (p.workers) {
    worker = (blockIdx.x & 7) * (p.workers >> 3) + (blockIdx.x >> 3);
    s = find_start<kRows>(a, p, worker, sh);
    if (s.count == 0) {
      if (threadIdx.x == 0) put_record(partials(a, p), s, worker, 0);
      return;
    }
  } else {
    s = Start{};
    s.row_tile = blockIdx.x % p.row_tiles;
    s.head = blockIdx.x / p.row_tiles % c.Hkv;
    s.b = blockIdx.x / p.row_tiles / c.Hkv;
    s.count = 0x7fffffff;
  }
  int left = s.count;
  bool first_segment = true;
  Geometry g = geometry<kRows>(a, p, s.b, s.row_tile);
  if (p.workers && threadIdx.x == 0) put_record(partials(a, p), s, worker, g.tiles);
  if (g.tiles == 0) return;

  // DMA: this wave brings 16 keys (or a part of them) of each tile: instruction i fills
  // LDS bytes (wave * kOps + i) * 1024 .., lane l the l-th 16 bytes.  Byte offsets of the
  // lane's source pieces from the first of the 16 keys:
  const int sub16 = wave / kWavesPerSub16;
  int k_src[S::kOps], v_src[S::kOps];
#pragma unroll
  for (int i = 0; i < S::kOps; ++i) {
    const int at = (wave * S::kOps + i) * 64 + lane;  // piece of the tile's keys
    const int r = at / S::kPieces, piece = (at % S::kPieces) ^ S::swizzle(r);
    k_src[i] = (key_of_row<false>(r & 31) & 15) * (D * kEs) + piece * 16;
    v_src[i] = (at % (S::kPieces * 16)) * 16;
  }
  // reading: this lane's K row is col of each half tile, pieces 2 x + h
  const int k_row = col * (S::kPieces * 16), k_swz = S::swizzle(col);

  while (true) {
    const int t0 = g.tile0 + s.skip, take = min(left, g.tiles - s.skip), t1 = t0 + take;
    const int head = s.head;
    const Masks mask{a.causal, a.window, c.len(g.b)};
    const int G = c.Hq / c.Hkv;
    const TableRow row(c, g.b);

    // ---- this wave's rows, and the keys that all or some of them see
    const int wrow = wave * NB * 32;
    const int wrows = min(NB * 32, g.rows - wrow);  // may be <= 0: the wave only helps with the DMA
    const int blocks = wrows <= 0 ? 0 : (wrows + 31) >> 5;
    int some_lo = 0, some_hi = 0, all_lo = 0, all_hi = 0;
    if (wrows > 0) {
      const int first = g.pos0 + (g.row0 + wrow) / G, last = g.pos0 + (g.row0 + wrow + wrows - 1) / G;
      some_lo = mask.lo(first);
      some_hi = mask.hi(last);
      all_lo = mask.lo(last);
      all_hi = mask.hi(first);
    }
    uint4 q[NB][kQ];
    int row_lo[NB], row_hi[NB];
    Running run[NB];
    f32x16_t acc[NB][TT::kBlocks];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      run[nb].m = -INFINITY;
      run[nb].l = 0.f;
#pragma unroll
      for (int db = 0; db < TT::kBlocks; ++db) acc[nb][db] = f32x16_t{};
      const int rho = wrow + nb * 32 + col;
      row_lo[nb] = 0;  // a column without a row sees everything and is left out at the end
      row_hi[nb] = 0x7fffffff;
      int hq = 0;
      long long r = -1;
      if (rho < g.rows) {
        r = global_row(a, g, rho, head, hq);
        const int pos = g.pos0 + (g.row0 + rho) / G;
        row_lo[nb] = mask.lo(pos);
        row_hi[nb] = mask.hi(pos);
      }
      const uint16_t* src = static_cast<const uint16_t*>(a.q) + (r >= 0 ? r * a.q_stride + (size_t)hq * D : 0);
#pragma unroll
      for (int x = 0; x < kQ; ++x) q[nb][x] = *reinterpret_cast<const uint4*>(src + coord<CT>(x, h));
      const uint32_t there = r >= 0 ? ~0u : 0u;
#pragma unroll
      for (int x = 0; x < kQ; ++x)
        q[nb][x] = make_uint4(q[nb][x].x & there, q[nb][x].y & there, q[nb][x].z & there, q[nb][x].w & there);
    }
    const float ks = CT == DSPARK_F8E4M3 ? a.scale2 * a.k_scale[head] : a.scale2;

    auto dma = [&](int raw_id, int t, unsigned char* kb, unsigned char* vb) {
      const int key = t * S::kKeys + 16 * sub16;
      const size_t token = ((size_t)(row.id(raw_id) * (unsigned)c.Hkv + head) << c.page_shift) + (key & ((1 << c.page_shift) - 1));
      const char* const ks_ = static_cast<const char*>(a.k_pool) + token * (D * kEs);
      const char* const vs_ = static_cast<const char*>(a.v_pool) + token * (D * kEs);
#pragma unroll
      for (int i = 0; i < S::kOps; ++i)
        dma_1k(ks_ + k_src[i], kb + (wave * S::kOps + i) * 1024);
#pragma unroll
      for (int i = 0; i < S::kOps; ++i)
        dma_1k(vs_ + v_src[i], vb + (wave * S::kOps + i) * 1024);
    };
    auto raw_id = [&](int t) { return row.raw(min(t, t1 - 1) * S::kKeys + 16 * sub16); };

    auto tile_scores = [&](const unsigned char* kb, int sub, f32x16_t(&w)[NB]) {
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) w[nb] = f32x16_t{};
#pragma unroll
      for (int x = 0; x < TT::kK; ++x) {
        const uint4 k = *reinterpret_cast<const uint4*>(kb + sub * 32 * (D * kEs) + k_row + (((2 * x + h) ^ k_swz) << 4));
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          if constexpr (CT == DSPARK_BF16) {
            w[nb] = mma(as_bf16x8(k), as_bf16x8(q[nb][x]), w[nb]);
          } else {
            w[nb] = mma(f8_to_bf16x8(k.x, k.y), as_bf16x8(q[nb][2 * x]), w[nb]);
            w[nb] = mma(f8_to_bf16x8(k.z, k.w), as_bf16x8(q[nb][2 * x + 1]), w[nb]);
          }
        }
      }
    };
    auto soften = [&](f32x16_t(&w)[NB]) {
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        const float fade = weights(w[nb], run[nb], ks);
        if (__any(fade != 1.f)) {
#pragma unroll
          for (int db = 0; db < TT::kBlocks; ++db) acc[nb][db] *= fade;
        }
      }
    };
    auto value = [&](const unsigned char* vb, int sub, int sl, int db) {
      return *reinterpret_cast<const typename TT::V*>(vb + ((sub * 4 + 2 * sl + h) * D + 32 * db + col) * (8 * kEs));
    };
    auto step = [&](int t, int id_next, unsigned char* kb, unsigned char* vb, unsigned char* kn, unsigned char* vn) {
      wait_vmem();         // this wave's part of the tile has landed
      barrier_lds_only();  // everybody's has, and nobody reads the other buffer any more
      if (t + 1 < t1) dma(id_next, t + 1, kn, vn);
      const int key0 = t * S::kKeys;
      if (key0 < g.all_lo || key0 + S::kKeys > g.all_hi) {
        // a tile that not all rows see whole: its values are made finite, in place
        uint4* const mine = reinterpret_cast<uint4*>(vb) + threadIdx.x;
        uint32_t bits = 0;
#pragma unroll
        for (int i = 0; i < S::kBytes / 16 / kAttendThreads; ++i) find_nonfinite<CT>(mine[i * kAttendThreads], bits);
        if (__any(bits & kOdd<CT>)) {
          odd = 1;
#pragma unroll 1
          for (int i = 0; i < S::kBytes / 16 / kAttendThreads; ++i)
            mine[i * kAttendThreads] = finite_part<CT>(mine[i * kAttendThreads]);
        }
        barrier_lds_only();
      }
      if (key0 >= some_hi || key0 + S::kKeys <= some_lo) return;  // nothing that this wave's rows see
      f32x16_t w[S::kSubs][NB];
#pragma unroll
      for (int sub = 0; sub < S::kSubs; ++sub) tile_scores(kb, sub, w[sub]);
      if (key0 < all_lo || key0 + S::kKeys > all_hi) {
#pragma unroll
        for (int sub = 0; sub < S::kSubs; ++sub)
#pragma unroll
          for (int nb = 0; nb < NB; ++nb)
            mask_scores<false>(w[sub][nb], row_lo[nb] - (key0 + 32 * sub), row_hi[nb] - (key0 + 32 * sub), h);
      }
#pragma unroll
      for (int sub = 0; sub < S::kSubs; ++sub) {
        soften(w[sub]);
#pragma unroll
        for (int sl = 0; sl < 2; ++sl) {
          bf16x8_t pw[NB];
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) pw[nb] = pack8(w[sub][nb], 8 * sl);
#pragma unroll
          for (int db = 0; db < TT::kBlocks; ++db) {
            const bf16x8_t v = value_operand<CT>(value(vb, sub, sl, db));
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) acc[nb][db] = mma(v, pw[nb], acc[nb][db]);
          }
        }
      }
    };

    // ---- tiles; page ids come over the scalar cache two tiles ahead
    int id = raw_id(t0), id1 = raw_id(t0 + 1);
    barrier_lds_only();  // the last segment's tiles are read
    if (threadIdx.x == 0) odd = 0;
    dma(id, t0, k0, v0);
    for (int t = t0; t < t1; t += 2) {
      id = raw_id(t + 2);
      step(t, id1, k0, v0, k1, v1);
      if (t + 1 == t1) break;
      id1 = raw_id(t + 3);
      step(t + 1, id, k1, v1, k0, v0);
    }

    // ---- results
    const bool whole = take == g.tiles;
    barrier_lds_only();
    const bool any_odd = odd != 0;
    const float vs = CT == DSPARK_F8E4M3 ? a.v_scale[head] : 1.f;
    float* const slot = whole ? nullptr : partials(a, p).template slot<D, kRows>(2 * worker + (first_segment ? 0 : 1));
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
      if (nb < blocks) {
        const int rho = wrow + nb * 32 + col;
        const float l = halves32_sum(run[nb].l);
        if (rho < g.rows) {
          int hq;
          const long long r = global_row(a, g, rho, head, hq);
          const float f = whole ? row_factor(l, vs) : 1.f;
          const bool none = whole && l == 0.f;
#pragma unroll
          for (int db = 0; db < TT::kBlocks; ++db)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              float4 y = make_float4(acc[nb][db][4 * j] * f, acc[nb][db][4 * j + 1] * f, acc[nb][db][4 * j + 2] * f,
                                     acc[nb][db][4 * j + 3] * f);
              if (none) y = make_float4(0.f, 0.f, 0.f, 0.f);
              const int d = 32 * db + 8 * j + 4 * h;
              if (!whole)
                *reinterpret_cast<float4*>(slot + (size_t)rho * D + d) = y;
              else if (r >= 0)
                store4<CT>(a.out, r * a.out_stride + (size_t)hq * D + d, y);
            }
          if (any_odd) {
            const int pos = g.pos0 + (g.row0 + rho) / G;
#pragma unroll 1
            for (int d = 4 * h; d < D; d += 8) {
              float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
              add_nonfinite<CT, D, S::kKeys>(a, g, mask, head, pos, d, t0 * S::kKeys, t1 * S::kKeys, y);
              const size_t at = whole ? r * a.out_stride + (size_t)hq * D + d : 0;
              float4* const part = reinterpret_cast<float4*>(slot + (size_t)rho * D + d);
              if (whole && r < 0) continue;
              const float4 x = whole ? load4<CT>(a.out, at) : *part;
              y = make_float4(x.x + y.x, x.y + y.y, x.z + y.z, x.w + y.w);
              if (whole)
                store4<CT>(a.out, at, y);
              else
                *part = y;
            }
          }
          if (h == 0) {
            if (!whole)
              *reinterpret_cast<float2*>(slot + (size_t)kRows * D + 2 * rho) = make_float2(run[nb].m, l);
            else if (r >= 0 && a.lse)
              a.lse[r * c.Hq + hq] = l == 0.f ? -INFINITY : (run[nb].m + log2f(l)) * kLn2f;
          }
        }
      }

    if (!p.workers) return;
    left -= take;
    if (left <= 0) return;
    first_segment = false;
    g = next_segment<kRows>(a, p, s);
  }
}

}  // namespace dspark
