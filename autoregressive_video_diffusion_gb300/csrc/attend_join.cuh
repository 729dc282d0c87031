// Attention whose keys are split over CTAs: the partial results and how the last CTA joins them.
#pragma once

#include "serve.cuh"

namespace dcp {

// A split leaves for each of its rows [m, l, o_0 .. o_{D-1}] in fp32: the running maximum in units of log2, and the
// sums of weights and weighted values relative to it.  An item's parts are [split][rows][D + 2].
__device__ __forceinline__ float* part_of(float* parts, int64_t item, int splits, int split, int rows, int D, int r) {
  return parts + ((item * splits + split) * rows + r) * (int64_t)(D + 2);
}

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// lse of a row from its maximum (in units of log2) and sum.
__device__ __forceinline__ float row_lse(float m, float l) {
  return l != 0.f ? (m + __log2f(l)) * 0.6931471805599453f : -INFINITY;
}

// Called by a whole CTA after its part is written; true for the item's last CTA.  The parts are read in the order of
// the splits, so the result does not depend on which CTA comes last.
__device__ __forceinline__ bool last_of(uint32_t* done, int splits, int* s_last) {
  __threadfence();
  __syncthreads();
  if (threadIdx.x == 0) {
    const uint32_t before = atomicAdd(done, 1);
    *s_last = before == (uint32_t)splits - 1;
    if (*s_last) *done = 0;
    __threadfence();
  }
  __syncthreads();
  return *s_last;
}

// Joins `splits` parts of `rows` rows (`stride` rows a part) whose first is row `row0` of (token, head of the KV
// head) rows, sequence start lo.
template <typename T>
__device__ __forceinline__ void join_parts(const AttendParams& a, const float* part, int splits, int stride, int rows,
                                           int row0, int lo, int kh) {
  const int D = a.pool.D, quads = D / 4;
  const int64_t step = (int64_t)stride * (D + 2);
  for (int u = threadIdx.x; u < rows * quads; u += blockDim.x) {
    const int r = u / quads, d = (u - r * quads) * 4;
    const float* at = part + (int64_t)r * (D + 2);
    float top = -INFINITY;
    for (int k = 0; k < splits; ++k) top = fmaxf(top, __ldcg(at + k * step));
    float l = 0.f, o[4] = {};
#pragma unroll 4
    for (int k = 0; k < splits; ++k) {
      const float* x = at + k * step;
      const float2 ml = __ldcg(reinterpret_cast<const float2*>(x));
      if (ml.y == 0.f) continue;  // the split saw no key of this row
      const float w = exp2_fast(ml.x - top);
      const float2 x0 = __ldcg(reinterpret_cast<const float2*>(x + 2 + d));
      const float2 x1 = __ldcg(reinterpret_cast<const float2*>(x + 4 + d));
      l += w * ml.y;
      o[0] += w * x0.x, o[1] += w * x0.y, o[2] += w * x1.x, o[3] += w * x1.y;
    }
    const float inv = l != 0.f ? 1.f / l : 0.f;
    const int R = row0 + r, tok = R / a.G;
    const int64_t row = (int64_t)(lo + tok) * a.Hq + kh * a.G + (R - tok * a.G);
    if (sizeof(T) == 2)
      *reinterpret_cast<uint2*>(a.out + (row * D + d) * 2) =
          make_uint2(pack_bf16x2(o[0] * inv, o[1] * inv), pack_bf16x2(o[2] * inv, o[3] * inv));
    else
      *reinterpret_cast<float4*>(a.out + (row * D + d) * 4) =
          make_float4(o[0] * inv, o[1] * inv, o[2] * inv, o[3] * inv);
    if (a.lse && d == 0) a.lse[row] = row_lse(top, l);
  }
}

}  // namespace dcp
