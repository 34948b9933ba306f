// Paged-cache attention for many rows (prompt chunks, verification blocks): every wave
// of a workgroup has its own block of 32 rows, and the key tiles pass through LDS once
// for all waves.
//
// Bound by the matrix units and by LDS, whose reads (one a product) run a few products
// ahead of their use; two workgroups a CU hide one's softmax and waits behind the
// other's products.  Measured: 4 x 2048 tokens over up to 8192 keys, 32 heads reading 8 of
// 128, bf16 (590 GFLOP) 557 us, 1.06 PFLOP/s, the matrix units busy in 52% of the cycles
// (8 waves, half of them in their products and half in the softmax by barriers, 706; 64
// rows a wave 1272, for the moves between its registers); 256 x up to 17 tokens over up to
// 2048 keys (0.98 GB) 183 us, 5.4 TB/s.
//
// Weights are rounded to bf16 for their product with the values (half a step, 2^-8 of a
// weight; sums, maxima and results stay fp32): in two terms, as k_attend_keys takes them,
// the second product doubles, and the prompt takes 765 us in place of 563, the 256 x up to
// 17 tokens 188 for 184, with e4m3 values 145 for 126.
//
// A tile of kKeys keys and values comes by LDS DMA (16 bytes a lane) into one of two
// buffers while the other is used; the buffers are distinct __shared__ objects, so that
// the compiler lets reads of one pass the DMA into the other.
//
// LDS layout.  Keys: 16-byte pieces, row m of the tile's 32-key halves holding key
// key_of_row(m); piece c of row r lies at c ^ swizzle(r), which spreads the 16 rows that
// one LDS cycle reads over all banks.  Values: as in the pool, (8-key group, coordinate)
// pieces in order, read without conflicts.
#pragma once

#include "attend_core.hpp"

namespace dspark {

typedef float f32x16_t __attribute__((ext_vector_type(16)));

__device__ __forceinline__ f32x16_t mma(bf16x8_t x, bf16x8_t y, f32x16_t c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(x, y, c, 0, 0, 0);
}

// Row m of the K operand holds this key of the tile.  S^T row m = 8 j + 4 h + i sits in
// register 4 j + i of half-wave h; the product with the values takes 8 consecutive keys
// of a 16-key slab from each half, so those rows are the keys
// 16 (j / 2) + 8 h + 4 (j % 2) + i.
__device__ __forceinline__ int key_of_row(int m) {
  const int j = m >> 3, h = (m >> 2) & 1, i = m & 3;
  return 16 * (j >> 1) + 8 * h + 4 * (j & 1) + i;
}
// The key of score register r in half-wave 0; half-wave 1 holds the key 8 on.
__device__ __forceinline__ constexpr int key_of_reg(int r) { return 16 * (r >> 3) + (r & 7); }

// The first of the 8 consecutive coordinates that half h of Q register x holds: where
// K's pieces of 16 bytes (e4m3: of 16 coordinates) have them.
template <int CT>
__device__ __forceinline__ constexpr int coord(int x, int h) {
  return CT == DSPARK_BF16 ? 16 * x + 8 * h : 32 * (x >> 1) + 16 * h + 8 * (x & 1);
}

// Leaves the scores of the tile's keys that the row sees (lo <= key < hi).  The half's
// offset goes into the bounds, so that a key is a constant.
__device__ __forceinline__ void mask_scores(f32x16_t& s, int lo, int hi, int h) {
  const int from = lo - 8 * h;
  const unsigned n = max(0, hi - lo);
#pragma unroll
  for (int i = 0; i < 16; ++i) s[i] = (unsigned)(key_of_reg(i) - from) < n ? s[i] : -INFINITY;
}

// The running maximum over N score tiles of a row; returns the factor by which O and l
// fade (1 for most tiles).
template <int N>
__device__ __forceinline__ float raise_max(const f32x16_t (&s)[N], Running& r, float c) {
  float top = s[0][0];
#pragma unroll
  for (int n = 0; n < N; ++n)
#pragma unroll
    for (int i = 0; i < 16; ++i) top = fmaxf(top, s[n][i]);
  top = halves32_max(top) * c;
  if (!__any(top > r.m + kRescale)) return 1.f;
  return fade_to(r, top);
}
// Scores to weights; l grows by their sum.
__device__ __forceinline__ void weights(f32x16_t& s, Running& r, float c) {
  const float ref = r.m == -INFINITY ? 0.f : r.m;
  float sum0 = 0.f, sum1 = 0.f;
#pragma unroll
  for (int i = 0; i < 16; i += 2) {
    s[i] = __builtin_amdgcn_exp2f(fmaf(s[i], c, -ref));
    s[i + 1] = __builtin_amdgcn_exp2f(fmaf(s[i + 1], c, -ref));
    sum0 += s[i];
    sum1 += s[i + 1];
  }
  r.l += sum0 + sum1;
}

__device__ __forceinline__ bf16x8_t pack8(const f32x16_t& s, int at) {
  bf16x8_t o;
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    const bf16x2_t p = __builtin_convertvector(f32x2_t{s[at + i], s[at + i + 1]}, bf16x2_t);
    o[i] = p[0];
    o[i + 1] = p[1];
  }
  return o;
}

// four bf16 values of a result that this lane stored
__device__ __forceinline__ float4 load4(const void* out, size_t at) {
  const uint2 w = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(out) + at);
  return make_float4(bf16_lo(w.x), bf16_hi(w.x), bf16_lo(w.y), bf16_hi(w.y));
}

template <int CT, int D>
struct RowsShape {
  static constexpr int kEs = Operand<CT>::kBytes;
  static constexpr int kKeys = D == 256 ? 32 : 64;           // of a tile
  static constexpr int kSubs = kKeys / 32;
  static constexpr int kRows = 4 * 32;                      // of a workgroup
  static constexpr int kBytes = kKeys * D * kEs;             // of the keys (or the values) of a tile
  static constexpr int kPieces = D * kEs / 16;               // of a key
  static constexpr int kOps = kBytes / 1024 / 4;               // DMA instructions a wave, keys (or values)
  static constexpr int kAhead = D == 256 ? 3 : 4;            // LDS reads before their products (more spill at 256)
  static constexpr int kQ = D / 16;                          // registers of Q (16 bytes a lane)
  static constexpr int kBlocks = D / 32;                     // of 32 coordinates
  using V = typename std::conditional<is_f8(CT), uint2, uint4>::type;  // 8 tokens of a coordinate
  // 64 banks of 4 bytes: 16 pieces a cycle, one or more rows of keys
  __device__ __forceinline__ static int swizzle(int r) { return kPieces >= 16 ? r & 15 : (r / (16 / kPieces)) & (kPieces - 1); }
};

// Order of instructions that the scheduler is asked for: the next `n` of a kind.
constexpr int kValu = 0x2, kMfma = 0x8, kLdsRead = 0x100;
template <int KIND, int N>
__device__ __forceinline__ void schedule() {
  __builtin_amdgcn_sched_group_barrier(KIND, N, 0);
}

// 64 lanes x 16 bytes at the lanes' offsets + AT of the buffer to the 1 KB of LDS at AT, in
// lane order (the instruction's offset counts on both sides)
template <int AT, bool ONCE>
__device__ __forceinline__ void dma_1k(__amdgpu_buffer_rsrc_t src, int offset, unsigned char* lds) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(src, (__attribute__((address_space(3))) void*)lds, 16, offset, 0, AT,
                                           ONCE ? 2 : 0);
}

// ONCE: keys and values with the streaming policy
template <int CT, int D, bool ONCE>
__global__ __launch_bounds__(kAttendThreads, D == 256 ? 2 : 1) void k_attend_rows(AttendArgs a, Split p) {
  using S = RowsShape<CT, D>;
  constexpr int kQ = S::kQ, kRows = S::kRows, kEs = S::kEs;
  constexpr int kOps = S::kOps;
  constexpr int kWavesPerSub16 = 4 / (S::kKeys / 16);  // waves that share the DMA of 16 keys
  __shared__ __attribute__((aligned(1024))) unsigned char k0[S::kBytes], k1[S::kBytes], v0[S::kBytes], v1[S::kBytes];
  __shared__ int sh[4];
  __shared__ int odd;  // a value that is not finite, and that a row sees, was replaced
  const int lane = threadIdx.x & 63, col = lane & 31, h = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const CacheView& c = a.c;

  Start s;
  int worker = 0;
  if (p.workers) {
    worker = (blockIdx.x & 7) * (p.workers >> 3) + (blockIdx.x >> 3);
    s = find_start<kRows, kAttendThreads, false>(a, p, worker, sh);
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
  Geometry g = p.workers ? geometry<kRows, false>(a, p, s.b, s.row_tile)
                         : geometry<kRows, false>(a, p, s.b, s.row_tile, s.n, s.len);
  if (p.workers && threadIdx.x == 0) put_record(partials(a, p), s, worker, g.tiles);
  if (g.tiles == 0) return;

  // DMA: this wave brings 16 keys (or a part of them) of each tile: instruction i fills
  // LDS bytes (wave * kOps + i) * 1024 .., lane l the l-th 16 bytes.  Byte offsets of the
  // lane's source pieces from the first of the 16 keys:
  const int sub16 = wave / kWavesPerSub16;
  int k_src[kOps], v_src;
#pragma unroll
  for (int i = 0; i < kOps; ++i) {
    const int at = (wave * kOps + i) * 64 + lane;  // piece of the tile's keys
    const int r = at / S::kPieces, piece = (at % S::kPieces) ^ S::swizzle(r);
    k_src[i] = (key_of_row(r & 31) & 15) * (D * kEs) + piece * 16;
  }
  v_src = ((wave * kOps * 64 + lane) % (S::kPieces * 16)) * 16;
  // reading: this lane's K row is col of each half tile, pieces 2 x + h, at k_at ^ 32 x
  const int k_at = col * (S::kPieces * 16) + ((h ^ S::swizzle(col)) << 4);

  while (true) {
    const int t0 = g.tile0 + s.skip, take = (int)min(left, (long long)(g.tiles - s.skip)), t1 = t0 + take;
    const int head = s.head;
    // The length from memory again with e4m3, so that the tile loop's registers suffice (with g.pos0 + g.n head size 256
    // reloads a spilled register in every tile, behind all DMA: 32 x 9 rows, window 128, 21.0 us, so 16.7; head size 64
    // loses its order of LDS reads: 4 x 512 rows over 4096 keys 77.4, so 69.2).  bf16 is faster without (256 x 17 rows
    // over up to 1000 keys, head size 256, 99 us, with it 104).
    const Masks mask{a.causal, a.window, CT == DSPARK_BF16 ? g.pos0 + g.n : c.len(g.b)};
    const int G = c.Hq / c.Hkv;
    const TableRow row(c, g.b);

    // ---- this wave's rows, and the keys that all or some of them see
    const int wrow = wave * 32;
    const int wrows = min(32, g.rows - wrow);  // may be <= 0: the wave only helps with the DMA
    int some_lo = 0, some_hi = 0, all_lo = 0, all_hi = 0;
    if (wrows > 0) {
      const int first = g.pos0 + (g.row0 + wrow) / G, last = g.pos0 + (g.row0 + wrow + wrows - 1) / G;
      some_lo = mask.lo(first);
      some_hi = mask.hi(last);
      all_lo = mask.lo(last);
      all_hi = mask.hi(first);
    }
    uint4 q[kQ];
    int row_lo = 0, row_hi = 0x7fffffff;  // a column without a row sees everything and is left out at the end
    Running run{-INFINITY, 0.f};
    f32x16_t acc[S::kBlocks];
    const int rho = wrow + col;
    {
#pragma unroll
      for (int db = 0; db < S::kBlocks; ++db) acc[db] = f32x16_t{};
      int hq = 0;
      long long r = -1;
      if (rho < g.rows) {
        r = global_row(a, g, rho, head, hq);
        const int pos = g.pos0 + (g.row0 + rho) / G;
        row_lo = mask.lo(pos);
        row_hi = mask.hi(pos);
      }
      const uint16_t* src = static_cast<const uint16_t*>(a.q) + (r >= 0 ? r * a.q_stride + (size_t)hq * D : 0);
#pragma unroll
      for (int x = 0; x < kQ; ++x) q[x] = *reinterpret_cast<const uint4*>(src + coord<CT>(x, h));
      const uint32_t there = r >= 0 ? ~0u : 0u;
#pragma unroll
      for (int x = 0; x < kQ; ++x)
        q[x] = make_uint4(q[x].x & there, q[x].y & there, q[x].z & there, q[x].w & there);
    }
    const float ks = score_factor<CT>(a, head);

    // the 16 keys (or values) of tile t that this wave brings, as a buffer
    auto source = [&](const void* pool, int raw, int t) __attribute__((always_inline)) {
      const int key = min(t, t1 - 1) * S::kKeys + 16 * sub16;
      const size_t token = ((size_t)(row.id(raw) * (unsigned)c.Hkv + head) << c.page_shift) + (key & ((1 << c.page_shift) - 1));
      return make_rsrc(static_cast<const char*>(pool) + token * (D * kEs), 16 * D * kEs);
    };
    auto dma_k = [&](int raw, int t, unsigned char* to) __attribute__((always_inline)) {
      const __amdgpu_buffer_rsrc_t src = source(a.k_pool, raw, t);
#pragma unroll
      for (int i = 0; i < kOps; ++i) dma_1k<0, ONCE>(src, k_src[i], to + (wave * kOps + i) * 1024);
    };
    auto dma_v = [&](int raw, int t, unsigned char* to) __attribute__((always_inline)) {
      const __amdgpu_buffer_rsrc_t src = source(a.v_pool, raw, t);
      unsigned char* const at = to + wave * kOps * 1024;
      dma_1k<0, ONCE>(src, v_src, at);
      if constexpr (kOps > 1) dma_1k<1024, ONCE>(src, v_src, at);
      if constexpr (kOps > 2) dma_1k<2 * 1024, ONCE>(src, v_src, at);
      if constexpr (kOps > 3) dma_1k<3 * 1024, ONCE>(src, v_src, at);
    };
    auto raw_id = [&](int t) __attribute__((always_inline)) { return row.raw(min(t, t1 - 1) * S::kKeys + 16 * sub16); };

    auto scores = [&](const unsigned char* kb, int sub, f32x16_t& w) __attribute__((always_inline)) {
      w = f32x16_t{};
      int at = k_at;
      if (D == 256) asm volatile("" : "+v"(at));  // no room for 16 addresses kept from tile to tile
#pragma unroll
      for (int x = 0; x < S::kPieces / 2; ++x) {
        const uint4 k = *reinterpret_cast<const uint4*>(kb + sub * 32 * (D * kEs) + (at ^ (32 * x)));
        if constexpr (CT == DSPARK_BF16) {
          w = mma(as_bf16x8(k), as_bf16x8(q[x]), w);
        } else {
          w = mma(f8_to_bf16x8(k.x, k.y), as_bf16x8(q[2 * x]), w);
          w = mma(f8_to_bf16x8(k.z, k.w), as_bf16x8(q[2 * x + 1]), w);
        }
      }
    };
    auto value = [&](const unsigned char* vb, int sub, int sl, int db) __attribute__((always_inline)) {
      return value_operand<CT>(
          *reinterpret_cast<const typename S::V*>(vb + ((sub * 4 + 2 * sl + h) * D + 32 * db + col) * (8 * kEs)));
    };
    // Waits until at most the youngest two of this wave's DMA groups (of keys or of values)
    // are on their way.  Past the last tile the last one is brought again, so that there
    // are always as many and the compiler, which counts too, adds no waits of its own.
    auto landed = [&]() __attribute__((always_inline)) { wait_vmem_n<2 * kOps>(); };
    // One tile, keys in kb and values in vb; v_next receives the next tile's values and kb,
    // once read, the keys of the one after.  Every group of DMA is sent one and a half
    // tiles before it is used.
    auto step = [&](int t, int id1, int id2, unsigned char* kb, unsigned char* vb, unsigned char* v_next) __attribute__((always_inline)) {
      landed();            // this wave's part of the keys
      barrier_lds_only();  // everybody's, and the last tile's values are read
      dma_v(id1, t + 1, v_next);
      const int key0 = t * S::kKeys;
      const bool on = key0 < some_hi && key0 + S::kKeys > some_lo;  // something that this wave's rows see
      f32x16_t w[S::kSubs];
      if (on) {
#pragma unroll
        for (int sub = 0; sub < S::kSubs; ++sub) scores(kb, sub, w[sub]);
        // LDS reads run kAhead fragments before their products
        constexpr int kReads = S::kSubs * S::kPieces / 2, kMma = CT == DSPARK_BF16 ? 1 : 2;
        schedule<kLdsRead, S::kAhead>();
#pragma unroll
        for (int i = 0; i < kReads - S::kAhead; ++i) {
          schedule<kMfma, kMma>();
          schedule<kLdsRead, 1>();
        }
        schedule<kMfma, S::kAhead * kMma>();
        if (key0 < all_lo || key0 + S::kKeys > all_hi) {
#pragma unroll
          for (int sub = 0; sub < S::kSubs; ++sub)
            mask_scores(w[sub], row_lo - (key0 + 32 * sub), row_hi - (key0 + 32 * sub), h);
        }
        const float fade = raise_max(w, run, ks);
        if (__any(fade != 1.f)) {
#pragma unroll
          for (int db = 0; db < S::kBlocks; ++db) acc[db] *= fade;
        }
      }
      landed();            // this wave's part of the values
      barrier_lds_only();  // everybody's, and the keys are read
      dma_k(id2, t + 2, kb);
      if (key0 < g.all_lo || key0 + S::kKeys > g.all_hi) {
        // a tile that not all rows see whole: its values are made finite, in place
        uint4* const mine = reinterpret_cast<uint4*>(vb) + threadIdx.x;
        uint32_t bits = 0;
#pragma unroll
        for (int i = 0; i < S::kBytes / 16 / kAttendThreads; ++i) find_nonfinite<CT>(mine[i * kAttendThreads], bits);
        if (__builtin_expect(__any(bits & kOdd<CT>), 0)) {  // word by word, for few registers
          uint32_t seen = 0;
#pragma unroll 1
          for (int i = 0; i < S::kBytes / 4 / kAttendThreads; ++i) {
            const int at = 4 * (threadIdx.x + (i >> 2) * kAttendThreads) + (i & 3);  // 8 tokens are 2 kEs words
            uint32_t* const word = reinterpret_cast<uint32_t*>(vb) + at;
            const int key = key0 + at / (2 * kEs * D) * 8 + at % (2 * kEs) * (4 / kEs);
            find_nonfinite<CT>(*word & keys_within<CT>(key, g.lo, g.hi), seen);
            *word = finite_word<CT>(*word);
          }
          if (seen & kOdd<CT>) odd = 1;
        }
        barrier_lds_only();
      }
      if (!on) return;
      // the weights of the first half, then its product with the values next to the
      // weights of the second half
#pragma unroll
      for (int sub = 0; sub < S::kSubs; ++sub) {
        weights(w[sub], run, ks);
#pragma unroll
        for (int sl = 0; sl < 2; ++sl) {
          const bf16x8_t pw = pack8(w[sub], 8 * sl);
#pragma unroll
          for (int db = 0; db < S::kBlocks; ++db) acc[db] = mma(value(vb, sub, sl, db), pw, acc[db]);
        }
      }
      constexpr int kValues = 2 * S::kBlocks, kSoft = 58;
      schedule<kLdsRead, S::kAhead>();
      schedule<kValu, kSoft>();
#pragma unroll
      for (int sub = 0; sub < S::kSubs; ++sub)
#pragma unroll
        for (int i = 0; i < kValues; ++i) {
          schedule<kMfma, 1>();
          if (sub * kValues + i + S::kAhead < S::kSubs * kValues) schedule<kLdsRead, 1>();
          if (sub + 1 < S::kSubs) schedule<kValu, kSoft / kValues>();
        }
    };

    // ---- tiles; page ids come over the scalar cache ahead of their use
    int id0 = raw_id(t0), id1 = raw_id(t0 + 1), id2 = raw_id(t0 + 2);
    barrier_lds_only();  // the last segment's tiles are read
    if (threadIdx.x == 0) odd = 0;
    dma_k(id0, t0, k0);
    dma_v(id0, t0, v0);
    dma_k(id1, t0 + 1, k1);
    for (int t = t0; t < t1; t += 2) {
      const int id3 = raw_id(t + 3), id4 = raw_id(t + 4);
      step(t, id1, id2, k0, v0, v1);
      if (t + 1 == t1) break;
      step(t + 1, id2, id3, k1, v1, v0);
      id1 = id3;
      id2 = id4;
    }
    wait_vmem();  // what was brought again

    // ---- results
    const bool whole = take == g.tiles;
    barrier_lds_only();
    const bool any_odd = odd != 0;
    const float vs = CT == DSPARK_F8E4M3 ? a.v_scale[head] : 1.f;
    float* const slot = whole ? nullptr : partials(a, p).template slot<D, kRows>(2 * worker + (first_segment ? 0 : 1));
    const float l = halves32_sum(run.l);
    if (rho < g.rows) {
      int hq;
      const long long r = global_row(a, g, rho, head, hq);
      const float f = whole ? row_factor(l, vs) : 1.f;
      const bool none = whole && l == 0.f;
#pragma unroll
      for (int db = 0; db < S::kBlocks; ++db)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float4 y = make_float4(acc[db][4 * j] * f, acc[db][4 * j + 1] * f, acc[db][4 * j + 2] * f,
                                 acc[db][4 * j + 3] * f);
          if (none) y = make_float4(0.f, 0.f, 0.f, 0.f);
          const int d = 32 * db + 8 * j + 4 * h;
          if (!whole)
            *reinterpret_cast<float4*>(slot + (size_t)rho * D + d) = y;
          else if (r >= 0)
            store4<CT>(a.out, r * a.out_stride + (size_t)hq * D + d, y);
        }
      if (__builtin_expect(any_odd && !none, 0)) {
        const RowKeys<false> sees = row_keys<false>(a, g, mask, (g.row0 + rho) / G, r);
#pragma unroll 1
        for (int d = 4 * h; d < D; d += 8) {
          float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
          add_nonfinite<CT, D, S::kKeys, false>(a, g, sees, head, d, t0 * S::kKeys, t1 * S::kKeys, y);
          const size_t at = whole ? r * a.out_stride + (size_t)hq * D + d : 0;
          float4* const part = reinterpret_cast<float4*>(slot + (size_t)rho * D + d);
          if (whole && r < 0) continue;
          const float4 x = whole ? load4(a.out, at) : *part;
          y = make_float4(x.x + y.x, x.y + y.y, x.z + y.z, x.w + y.w);
          if (whole)
            store4<CT>(a.out, at, y);
          else
            *part = y;
        }
      }
      if (h == 0) {
        if (!whole)
          *reinterpret_cast<float2*>(slot + (size_t)kRows * D + 2 * rho) = make_float2(run.m, l);
        else if (r >= 0 && a.lse)
          a.lse[r * c.Hq + hq] = l == 0.f ? -INFINITY : (run.m + log2f(l)) * kLn2f;
      }
    }

    if (!p.workers) return;
    left -= take;
    if (left <= 0) return;
    first_segment = false;
    g = next_segment<kRows, false>(a, p, s);
  }
}

}  // namespace dspark
