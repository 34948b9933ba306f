// Paged cache: attention of each request's new tokens over its pages.  See
// include/dspark_cache.h for the contract.
#include "dspark_cache_internal.hpp"

namespace dspark {
namespace {

template <int CT>
__device__ __forceinline__ float load_cached(const void* p, size_t i) {
  if constexpr (CT == DSPARK_F32)
    return static_cast<const float*>(p)[i];
  else if constexpr (CT == DSPARK_BF16)
    return bf16_to_f32(static_cast<const uint16_t*>(p)[i]);
  else
    return __builtin_amdgcn_cvt_f32_fp8(static_cast<const uint8_t*>(p)[i], 0);
}

// One wave a (row, query head): 64 positions at a time, one a lane, with the
// running maximum and sum of the softmax; then every lane adds the 64 weighted
// values of its D / 64 coordinates.
template <int CT, int D>
__global__ __launch_bounds__(64) void k_attend_rows(AttendArgs a) {
  const CacheView& c = a.c;
  const int b = blockIdx.x / c.max_new, i = blockIdx.x % c.max_new, hq = blockIdx.y, lane = threadIdx.x;
  const int n = c.rows(b), len = c.len(b);
  const long long row = c.first_row(b) + i;
  if (i >= n || !c.has_row(row)) return;
  const int head = hq / (c.Hq / c.Hkv);
  const float ks = CT == DSPARK_F8E4M3 ? a.k_scale[head] : 1.f, vs = CT == DSPARK_F8E4M3 ? a.v_scale[head] : 1.f;
  const int pos = len - n + i;
  const int hi = a.causal && pos + 1 < len ? pos + 1 : len;
  const int lo = a.window > 0 && pos - a.window + 1 > 0 ? pos - a.window + 1 : 0;
  __shared__ float q[D];
  for (int d = lane; d < D; d += 64)
    q[d] = load_cached<CT == DSPARK_F32 ? DSPARK_F32 : DSPARK_BF16>(a.q, row * a.q_stride + (size_t)hq * D + d);
  __syncthreads();
  float m = -INFINITY, l = 0.f, o[D / 64] = {};
  for (int j0 = lo; j0 < hi; j0 += 64) {
    const int j = j0 + lane;
    float x = -INFINITY;
    if (j < hi) {
      const int page = min((unsigned)c.table[(size_t)b * c.max_pages + (j >> c.page_shift)], (unsigned)c.n_pages - 1);
      const size_t at = ((((size_t)page * c.Hkv + head) << c.page_shift) + (j & ((1 << c.page_shift) - 1))) * D;
      float dot = 0.f;
      for (int d = 0; d < D; ++d) dot += q[d] * load_cached<CT>(a.k_pool, at + d);
      x = dot * ks * a.scale2;
    }
    const float top = fmaxf(m, wave_max(x));
    const float ref = top == -INFINITY ? 0.f : top;
    const float p = j < hi ? __builtin_amdgcn_exp2f(x - ref) : 0.f;
    const float fade = __builtin_amdgcn_exp2f(m - ref);
    l = l * fade + wave_sum(p);
    for (int e = 0; e < D / 64; ++e) o[e] *= fade;
    m = top;
    for (int t = 0; t < 64 && j0 + t < hi; ++t) {
      const int jt = j0 + t;
      const int page = min((unsigned)c.table[(size_t)b * c.max_pages + (jt >> c.page_shift)], (unsigned)c.n_pages - 1);
      const int off = jt & ((1 << c.page_shift) - 1);
      const size_t at = ((((size_t)page * c.Hkv + head) << c.page_shift) + (off & ~7)) * D + (off & 7);
      const float w = __shfl(p, t);
      for (int e = 0; e < D / 64; ++e) o[e] += w * load_cached<CT>(a.v_pool, at + (size_t)(e * 64 + lane) * 8);
    }
  }
  const float inv = l > 0.f ? vs / l : l == 0.f ? 0.f : l;  // NaN stays
  for (int e = 0; e < D / 64; ++e) {
    const float y = l == 0.f ? 0.f : o[e] * inv;
    const size_t at = row * a.out_stride + (size_t)hq * D + e * 64 + lane;
    if constexpr (CT == DSPARK_F32)
      static_cast<float*>(a.out)[at] = y;
    else
      static_cast<uint16_t*>(a.out)[at] = (uint16_t)f32_to_bf16_bits(y);
  }
  if (a.lse && lane == 0) a.lse[row * c.Hq + hq] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
}

template <int CT>
hipError_t attend_typed(const dspark_cache& C, const AttendArgs& a, hipStream_t s) {
  const dim3 grid((unsigned)C.B * a.c.max_new, C.Hq);
  if (C.D == 64)
    k_attend_rows<CT, 64><<<grid, 64, 0, s>>>(a);
  else if (C.D == 128)
    k_attend_rows<CT, 128><<<grid, 64, 0, s>>>(a);
  else
    k_attend_rows<CT, 256><<<grid, 64, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace

size_t attend_workspace_bytes(const dspark_cache&, int32_t) { return 0; }

hipError_t launch_cache_attend(const dspark_cache& C, const AttendArgs& a, hipStream_t s) {
  switch (C.cache_dtype) {
    case DSPARK_F32: return attend_typed<DSPARK_F32>(C, a, s);
    case DSPARK_BF16: return attend_typed<DSPARK_BF16>(C, a, s);
    default: return attend_typed<DSPARK_F8E4M3>(C, a, s);
  }
}

}  // namespace dspark
