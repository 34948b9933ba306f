// Paged-cache attention for many rows, over a cache whose tokens carry their own scales
// and for the nodes of trees: the tiles, products and softmax of k_attend_rows
// (attend_rows.hpp, which calls over the other types keep as it is), and
//
// - scales of tokens.  A key's scale is a factor of its column of scores, a value's of its
//   weights on their way to the second product (not of their sum); the product of the two is
//   what is rounded to bf16 there, by half a step as the weights of attend_rows.hpp, for its
//   reason.  Both come by DMA next to their tiles, 64 bytes for each 16 keys.  Their products are
//   vector instructions where the call waits for those (4 x 2048 tokens over up to 8192 keys, 32
//   heads reading 8 of 128: 635 us, 0.93 PFLOP/s; 548 with the two products left out);
// - a tree's bits in the tiles that hold its nodes (two words of the row's mask for each 32
//   keys; 64 requests of up to 33 nodes x 4 query heads over up to 500 keys 37.0 us, as a
//   sequence 35.1);
// - rows that several waves share.
//
// Of few rows and keys a segment's start counts: 2048 segments of 68 rows or less over up to
// 2048 keys take 147 us (3.5 TB/s), over up to 4096 222 (6.4 TB/s between the two), over none 32.
// (The rows' loads behind the first DMA, and a third or fourth pair of buffers, changed nothing.)
#pragma once

#include "attend_rows.hpp"

namespace dspark {

// Leaves the scores of the tile's keys whose bit is set, a bit for each of the tile's 32 keys.
__device__ __forceinline__ void mask_scores(f32x16_t& s, uint32_t seen, int h) {
  seen >>= 8 * h;
#pragma unroll
  for (int i = 0; i < 16; ++i) s[i] = seen >> key_of_reg(i) & 1u ? s[i] : -INFINITY;
}

// s[i] times lane i's x, of the 16 lanes that a lane is among.
template <int I = 0>
__device__ __forceinline__ void times_row16(f32x16_t& s, float x) {
  constexpr int kRowBroadcast = 0x150;  // + the lane
  s[I] *= __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), kRowBroadcast + I, 0xF, 0xF, true));
  if constexpr (I < 15) times_row16<I + 1>(s, x);
}

// 64 lanes x 4 bytes, in lane order; past the buffer's end zeros
template <bool ONCE>
__device__ __forceinline__ void dma_words(__amdgpu_buffer_rsrc_t src, int offset, float* lds) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(src, (__attribute__((address_space(3))) void*)lds, 4, offset, 0, 0, ONCE ? 2 : 0);
}

// ONCE: keys and values with the streaming policy
template <int CT, int D, bool ONCE, bool TREE>
__global__ __launch_bounds__(kAttendThreads, D == 256 ? 2 : 1) void k_attend_parts(AttendArgs a, Split p) {
  using S = RowsShape<CT, D>;
  constexpr int kQ = S::kQ, kRows = S::kRows, kEs = S::kEs;
  constexpr int kOps = S::kOps, kGroup = kOps + Operand<CT>::kToken;  // DMA instructions of a wave, and with the scales
  constexpr int kWavesPerSub16 = 4 / (S::kKeys / 16);  // waves that share the DMA of 16 keys
  __shared__ __attribute__((aligned(1024))) unsigned char k0[S::kBytes], k1[S::kBytes], v0[S::kBytes], v1[S::kBytes];
  // scales of a token: each wave brings those of its 16 keys into 64 words of its own
  constexpr bool kToken = Operand<CT>::kToken;
  constexpr int kScales = kToken ? kAttendThreads : 1;
  __shared__ __attribute__((aligned(256))) float ks0[kScales], ks1[kScales], vs0[kScales], vs1[kScales];
  __shared__ int sh[4];
  __shared__ int odd;  // a value that is not finite, and that a row sees, was replaced
  // Waves share rows where there are few (below) with head size 64: 64 trees of up to 30 nodes
  // x 2 query heads over up to 4000 keys 76 us without, 63 with; head size 128 98 / 101, over
  // e4m3 92 / 84, a prompt of 128 rows over tokens' scales 643 / 658 (the code for both takes
  // registers), 256 197 / 219.
  constexpr bool kShares = D == 64;
  // LDS reads before their products: with tokens' scales and head size 256 registers are short
  // (4 prompts of 1024 over up to 4096 keys x 4 heads 291 us with 3, 264 with 1; trees 241 / 221)
  constexpr int kAhead = kToken && D == 256 ? 1 : S::kAhead;
  constexpr int kSoft = kToken ? 74 : 58;  // vector instructions of a half tile's weights
  __shared__ float2 shared_ml[kShares ? 4 : 1][64];  // of shared rows
  const int lane = threadIdx.x & 63, col = lane & 31, h = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const CacheView& c = a.c;

  Start s;
  int worker = 0;
  if (p.workers) {
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
    const Masks mask{a.causal, a.window, g.pos0 + g.n};
    const int G = c.Hq / c.Hkv;
    const TableRow row(c, g.b);

    // ---- this wave's rows, and the keys that all or some of them see.  Where half or all but
    // one of the waves would have no rows, 2 or 4 waves take the same 32 and share the tiles:
    // a wave's part is every second or fourth half tile (whole tile of 32 keys).
    const int shares = !kShares || g.rows > 64 ? 1 : g.rows > 32 ? 2 : 4;
    const int share = shares == 1 ? 0 : shares == 2 ? wave >> 1 : wave;
    const int wrow = (shares == 1 ? wave : shares == 2 ? wave & 1 : 0) * 32;
    const int wrows = min(32, g.rows - wrow);  // may be <= 0: the wave only helps with the DMA
    int some_lo = 0, some_hi = 0, all_lo = 0, all_hi = 0;
    if (wrows > 0) {
      const int first = g.pos0 + (g.row0 + wrow) / G, last = g.pos0 + (g.row0 + wrow + wrows - 1) / G;
      some_lo = mask.lo(TREE ? g.pos0 : first);
      some_hi = mask.hi(last);
      all_lo = mask.lo(last);
      all_hi = TREE ? g.all_hi : mask.hi(first);
    }
    uint4 q[kQ];
    RowKeys<TREE> keys{0, 0x7fffffff};  // a column without a row sees everything and is left out at the end
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
        keys = row_keys<TREE>(a, g, mask, (g.row0 + rho) / G, r);
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
      const size_t at = token_at<CT, D>(c, row.id(raw), head, key & ((1 << c.page_shift) - 1));
      return make_rsrc(static_cast<const char*>(pool) + at, 16 * D * kEs);
    };
    auto dma_scales = [&](const void* pool, int raw, int t, float* to) __attribute__((always_inline)) {
      const int key = min(t, t1 - 1) * S::kKeys + 16 * sub16;
      const size_t at = scale_at<D>(c, row.id(raw), head, key & ((1 << c.page_shift) - 1));
      dma_words<ONCE>(make_rsrc(static_cast<const char*>(pool) + at, 16 * 4), 4 * lane, to + 64 * wave);
    };
    auto dma_k = [&](int raw, int t, unsigned char* to, float* scales) __attribute__((always_inline)) {
      const __amdgpu_buffer_rsrc_t src = source(a.k_pool, raw, t);
#pragma unroll
      for (int i = 0; i < kOps; ++i) dma_1k<0, ONCE>(src, k_src[i], to + (wave * kOps + i) * 1024);
      if constexpr (kToken) dma_scales(a.k_pool, raw, t, scales);
    };
    auto dma_v = [&](int raw, int t, unsigned char* to, float* scales) __attribute__((always_inline)) {
      const __amdgpu_buffer_rsrc_t src = source(a.v_pool, raw, t);
      if constexpr (kToken) dma_scales(a.v_pool, raw, t, scales);
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
    // Score register i of a lane belongs to key key_of_reg(i) + 8 h of its half tile.  Lane i of
    // each 16 holds that key's scale, and the product takes it from there (all 16 read from LDS by
    // every lane: a prompt chunk 671 us, 548 without scales).
    auto scales_of = [&](const float* sc, int sub) __attribute__((always_inline)) {
      return sc[(2 * sub + ((lane >> 3) & 1)) * kWavesPerSub16 * 64 + 8 * h + (lane & 7)];
    };
    // Waits until at most the youngest two of this wave's DMA groups (of keys or of values)
    // are on their way.  Past the last tile the last one is brought again, so that there
    // are always as many and the compiler, which counts too, adds no waits of its own.
    auto landed = [&]() __attribute__((always_inline)) { wait_vmem_n<2 * kGroup>(); };
    // The keys of a half tile that begins at key `first` and that the lane's row does not see
    auto hide = [&](int first, f32x16_t& w) __attribute__((always_inline)) {
      if constexpr (TREE)
        mask_scores(w, tree_seen(a, g, keys, first), h);
      else
        mask_scores(w, keys.lo - first, keys.hi - first, h);
    };
    // A wave that shares its rows: the scores of half tile `sub` ...
    auto half_scores = [&](int sub, int key0, const unsigned char* kb, const float* kc, f32x16_t(&w)[1])
                           __attribute__((always_inline)) {
      scores(kb, sub, w[0]);
      constexpr int kReads = S::kPieces / 2, kMma = CT == DSPARK_BF16 ? 1 : 2, kFirst = kAhead < kReads ? kAhead : kReads;
      schedule<kLdsRead, kFirst>();
#pragma unroll
      for (int i = 0; i < kReads - kFirst; ++i) {
        schedule<kMfma, kMma>();
        schedule<kLdsRead, 1>();
      }
      schedule<kMfma, kFirst * kMma>();
      if constexpr (kToken) times_row16(w[0], scales_of(kc, sub));
      if (key0 < all_lo || key0 + S::kKeys > all_hi) hide(key0 + 32 * sub, w[0]);
      const float fade = raise_max(w, run, ks);
      if (__any(fade != 1.f)) {
#pragma unroll
        for (int db = 0; db < S::kBlocks; ++db) acc[db] *= fade;
      }
    };
    // ... and its weights with the values
    auto half_values = [&](int sub, const unsigned char* vb, const float* vc, f32x16_t& w) __attribute__((always_inline)) {
      weights(w, run, ks);
      if constexpr (kToken) times_row16(w, scales_of(vc, sub));
#pragma unroll
      for (int sl = 0; sl < 2; ++sl) {
        const bf16x8_t pw = pack8(w, 8 * sl);
#pragma unroll
        for (int db = 0; db < S::kBlocks; ++db) acc[db] = mma(value(vb, sub, sl, db), pw, acc[db]);
      }
      constexpr int kValues = 2 * S::kBlocks;
      schedule<kLdsRead, kAhead>();
      schedule<kValu, kSoft>();
#pragma unroll
      for (int i = 0; i < kValues; ++i) {
        schedule<kMfma, 1>();
        if (i + kAhead < kValues) schedule<kLdsRead, 1>();
      }
    };
    // One tile, keys in kb and values in vb; v_next receives the next tile's values and kb,
    // once read, the keys of the one after.  Every group of DMA is sent one and a half
    // tiles before it is used.  Scales of a token go with their entries: kc with kb, ...
    auto step = [&](auto part, int t, int id1, int id2, unsigned char* kb, unsigned char* vb, unsigned char* v_next, float* kc,
                    float* vc, float* vc_next) __attribute__((always_inline)) {
      constexpr bool kPart = decltype(part)::value;
      landed();            // this wave's part of the keys
      barrier_lds_only();  // everybody's, and the last tile's values are read
      dma_v(id1, t + 1, v_next, vc_next);
      const int key0 = t * S::kKeys;
      bool on = key0 < some_hi && key0 + S::kKeys > some_lo;  // something that this wave's rows see
      f32x16_t w[kPart ? 1 : S::kSubs];
      const int sub0 = share & (S::kSubs - 1);  // the half tile of a wave that shares its rows
      if constexpr (kPart) {
        on = on && ((t * S::kSubs + sub0 - share) & (shares - 1)) == 0;
        if (on) half_scores(sub0, key0, kb, kc, w);
      } else if (on) {
#pragma unroll
        for (int sub = 0; sub < S::kSubs; ++sub) scores(kb, sub, w[sub]);
        // LDS reads run kAhead fragments before their products
        constexpr int kReads = S::kSubs * S::kPieces / 2, kMma = CT == DSPARK_BF16 ? 1 : 2;
        schedule<kLdsRead, kAhead>();
#pragma unroll
        for (int i = 0; i < kReads - kAhead; ++i) {
          schedule<kMfma, kMma>();
          schedule<kLdsRead, 1>();
        }
        schedule<kMfma, kAhead * kMma>();
        if constexpr (kToken) {
#pragma unroll
          for (int sub = 0; sub < S::kSubs; ++sub) times_row16(w[sub], scales_of(kc, sub));
        }
        if (key0 < all_lo || key0 + S::kKeys > all_hi) {
#pragma unroll
          for (int sub = 0; sub < S::kSubs; ++sub) hide(key0 + 32 * sub, w[sub]);
        }
        const float fade = raise_max(w, run, ks);
        if (__any(fade != 1.f)) {
#pragma unroll
          for (int db = 0; db < S::kBlocks; ++db) acc[db] *= fade;
        }
      }
      landed();            // this wave's part of the values
      barrier_lds_only();  // everybody's, and the keys are read
      dma_k(id2, t + 2, kb, kc);
      if (key0 < g.all_lo || key0 + S::kKeys > g.all_hi) {
        // a tile that not all rows see whole: its values are made finite, in place
        if constexpr (kToken) vc[threadIdx.x] = finite_scale(vc[threadIdx.x]);
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
      if constexpr (kPart) {
        half_values(sub0, vb, vc, w[0]);
        return;
      } else {
        // the weights of the first half, then its product with the values next to the
        // weights of the second half
#pragma unroll
        for (int sub = 0; sub < S::kSubs; ++sub) {
          weights(w[sub], run, ks);
          if constexpr (kToken) times_row16(w[sub], scales_of(vc, sub));
#pragma unroll
          for (int sl = 0; sl < 2; ++sl) {
            const bf16x8_t pw = pack8(w[sub], 8 * sl);
#pragma unroll
            for (int db = 0; db < S::kBlocks; ++db) acc[db] = mma(value(vb, sub, sl, db), pw, acc[db]);
          }
        }
        constexpr int kValues = 2 * S::kBlocks;
        schedule<kLdsRead, kAhead>();
        schedule<kValu, kSoft>();
#pragma unroll
        for (int sub = 0; sub < S::kSubs; ++sub)
#pragma unroll
          for (int i = 0; i < kValues; ++i) {
            schedule<kMfma, 1>();
            if (sub * kValues + i + kAhead < S::kSubs * kValues) schedule<kLdsRead, 1>();
            if (sub + 1 < S::kSubs) schedule<kValu, kSoft / kValues>();
          }
      }
    };

    // ---- tiles; page ids come over the scalar cache ahead of their use
    int id0 = raw_id(t0), id1 = raw_id(t0 + 1), id2 = raw_id(t0 + 2);
    barrier_lds_only();  // the last segment's tiles are read
    if (threadIdx.x == 0) odd = 0;
    dma_k(id0, t0, k0, ks0);
    dma_v(id0, t0, v0, vs0);
    dma_k(id1, t0 + 1, k1, ks1);
    auto tiles = [&](auto part) __attribute__((always_inline)) {
      for (int t = t0; t < t1; t += 2) {
        const int id3 = raw_id(t + 3), id4 = raw_id(t + 4);
        step(part, t, id1, id2, k0, v0, v1, ks0, vs0, vs1);
        if (t + 1 == t1) break;
        step(part, t + 1, id2, id3, k1, v1, v0, ks1, vs1, vs0);
        id1 = id3;
        id2 = id4;
      }
    };
    if (kShares && shares > 1)
      tiles(std::integral_constant<bool, kShares>());
    else
      tiles(std::false_type());
    wait_vmem();  // what was brought again

    // ---- results
    const bool whole = take == g.tiles;
    barrier_lds_only();
    const bool any_odd = odd != 0;
    if (kShares && shares > 1) {
      // The parts of shared rows meet in the tiles' buffers, lane by lane, in the order of the
      // shares: a part (m, l, O) counts exp2(m - M) (l, O), M the largest m.
      shared_ml[wave][lane] = make_float2(run.m, run.l);
      barrier_lds_only();
      const int step = shares == 2 ? 2 : 1;  // from one share's wave to the next's
      float top = run.m;
      for (int i = 1; i < shares; ++i) top = fmaxf(top, shared_ml[(wave + i * step) & 3][lane].x);
      const float f = run.m == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(run.m - top);
#pragma unroll
      for (int db = 0; db < S::kBlocks; ++db) acc[db] *= f;
      if (share == 0) {
        run.l = run.m == -INFINITY ? run.l : run.l * f;
        for (int i = 1; i < shares; ++i) {
          const float2 ml = shared_ml[wave + i * step][lane];
          run.l += ml.x == -INFINITY ? ml.y : ml.y * __builtin_amdgcn_exp2f(ml.x - top);
        }
        run.m = top;
      }
      auto buffer = [&](int w) __attribute__((always_inline)) {
        return reinterpret_cast<float4*>(w == 0 ? k0 : w == 1 ? k1 : w == 2 ? v0 : v1) + lane;
      };
      constexpr int kRound = S::kBytes / 4096 < S::kBlocks ? S::kBytes / 4096 : S::kBlocks;  // blocks that fit
#pragma unroll
      for (int db0 = 0; db0 < S::kBlocks; db0 += kRound) {
        if (share > 0) {
          float4* const to = buffer(wave);
#pragma unroll
          for (int i = 0; i < 4 * kRound; ++i) {
            const f32x16_t& x = acc[db0 + i / 4];
            to[64 * i] = make_float4(x[4 * (i & 3)], x[4 * (i & 3) + 1], x[4 * (i & 3) + 2], x[4 * (i & 3) + 3]);
          }
        }
        barrier_lds_only();
        if (share == 0) {
#pragma unroll 1
          for (int i = 1; i < shares; ++i) {
            const float4* const from = buffer(wave + i * step);
#pragma unroll
            for (int j = 0; j < 4 * kRound; ++j) {
              const float4 y = from[64 * j];
              f32x16_t& x = acc[db0 + j / 4];
              x[4 * (j & 3)] += y.x;
              x[4 * (j & 3) + 1] += y.y;
              x[4 * (j & 3) + 2] += y.z;
              x[4 * (j & 3) + 3] += y.w;
            }
          }
        }
        barrier_lds_only();
      }
    }
    const float vs = CT == DSPARK_F8E4M3 ? a.v_scale[head] : 1.f;
    float* const slot = whole ? nullptr : partials(a, p).template slot<D, kRows>(2 * worker + (first_segment ? 0 : 1));
    const float l = halves32_sum(run.l);
    if (rho < g.rows && share == 0) {
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
        const RowKeys<TREE> sees = row_keys<TREE>(a, g, mask, (g.row0 + rho) / G, r);
#pragma unroll 1
        for (int d = 4 * h; d < D; d += 8) {
          float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
          if (!TREE || r >= 0) add_nonfinite<CT, D, S::kKeys, TREE>(a, g, sees, head, d, t0 * S::kKeys, t1 * S::kKeys, y);
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
    g = next_segment<kRows, TREE>(a, p, s);
  }
}

}  // namespace dspark
