// Merging partial softmax results of one row: O = sum_p e^(L_p - L) O_p,
// L = log sum_p e^(L_p). O_p is already normalised by its own sum; L_p is
// -inf where part p saw no key.
#pragma once

#include <math_constants.h>

#include "sm100.cuh"

namespace fa {

// Loads 2 or 4 consecutive floats (8- or 16-byte aligned) into registers.
__device__ __forceinline__ void load_vec(const float* p, float (&x)[4]) {
  const float4 t = *reinterpret_cast<const float4*>(p);
  x[0] = t.x;
  x[1] = t.y;
  x[2] = t.z;
  x[3] = t.w;
}
__device__ __forceinline__ void load_vec(const float* p, float (&x)[2]) {
  const float2 t = *reinterpret_cast<const float2*>(p);
  x[0] = t.x;
  x[1] = t.y;
}

// One warp merges one row of n_parts partials, the p-th at rows
// row0 + p * stride of part_o [..][D] and part_l; writes dst[D] and *lse. 32
// partials a step: each lane takes one logsumexp, whose max and sum go
// through the warp; the weighted sum of the partial rows runs over d across
// lanes, eight partials at a time so that their loads overlap.
template <int D>
__device__ __forceinline__ void merge_row(const float* __restrict__ part_o, const float* __restrict__ part_l,
                                          long long row0, long long stride, int n_parts, __nv_bfloat16* dst,
                                          float* lse, int lane) {
  constexpr int VW = D / 32;
  float acc[VW], m = -CUDART_INF_F, den = 0.f;
#pragma unroll
  for (int i = 0; i < VW; ++i) acc[i] = 0.f;
#pragma unroll 1
  for (int p0 = 0; p0 < n_parts; p0 += 32) {
    const int cnt = min(32, n_parts - p0);
    const float pl = lane < cnt ? part_l[row0 + (p0 + lane) * stride] : -CUDART_INF_F;
    float top = pl;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
    top = fmaxf(top, m);
    const float ref = top == -CUDART_INF_F ? 0.f : top;  // no key so far: every weight 0
    const float old = expf(m - ref);
    const float wl = expf(pl - ref);
    float sum = wl;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
    den = den * old + sum;
    m = top;
#pragma unroll
    for (int k = 0; k < VW; ++k) acc[k] *= old;
#pragma unroll 1
    for (int i = 0; i < cnt; i += 8) {
      float x[8][VW];
#pragma unroll
      for (int q = 0; q < 8; ++q)
        if (i + q < cnt) load_vec(part_o + (row0 + (p0 + i + q) * stride) * D + lane * VW, x[q]);
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const float wq = __shfl_sync(0xffffffffu, wl, (i + q) & 31);
        if (i + q < cnt && wq != 0.f)
#pragma unroll
          for (int k = 0; k < VW; ++k) acc[k] = fmaf(wq, x[q][k], acc[k]);
      }
    }
  }
  const float inv = den == 0.f ? 0.f : 1.f / den;
  if constexpr (VW == 4) {
    *reinterpret_cast<uint2*>(dst + lane * VW) =
        make_uint2(pack_bf16x2(acc[0] * inv, acc[1] * inv), pack_bf16x2(acc[2] * inv, acc[3] * inv));
  } else {
    *reinterpret_cast<uint32_t*>(dst + lane * VW) = pack_bf16x2(acc[0] * inv, acc[1] * inv);
  }
  if (lane == 0) *lse = den == 0.f ? -CUDART_INF_F : m + logf(den);
}

}  // namespace fa
