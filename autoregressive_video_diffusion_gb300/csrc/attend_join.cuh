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
// head) rows, sequence start lo.  Called by a whole CTA; scratch: join_scratch(rows, splits) bytes of shared memory.
// First every part's maximum and sum, all at once, then the weights of the parts, then the values with many loads in
// flight: a loop that reads a part after the other pays a memory latency for each.
__host__ __device__ constexpr int64_t join_scratch(int rows, int splits) { return ((int64_t)rows * splits * 2 + rows) * 4; }

template <typename T>
__device__ __forceinline__ void join_parts(const AttendParams& a, const float* part, int splits, int stride, int rows,
                                           int row0, int lo, int kh, float* scratch) {
  const int D = a.pool.D, quads = D / 4;
  const int64_t step = (int64_t)stride * (D + 2);
  float* const weight = scratch;                 // [rows][splits]: the maximum, then the part's weight
  float* const sum = weight + rows * splits;     // [rows][splits]
  float* const inv = sum + rows * splits;        // [rows]
  __syncthreads();
  for (int u = threadIdx.x; u < rows * splits; u += blockDim.x) {
    const int r = u / splits, k = u - r * splits;
    const float2 ml = __ldcg(reinterpret_cast<const float2*>(part + k * step + (int64_t)r * (D + 2)));
    weight[u] = ml.x;
    sum[u] = ml.y;
  }
  __syncthreads();
  for (int r = threadIdx.x; r < rows; r += blockDim.x) {
    float top = -INFINITY, l = 0.f;
    for (int k = 0; k < splits; ++k) top = fmaxf(top, weight[r * splits + k]);
    for (int k = 0; k < splits; ++k) {
      // a split that saw no key of this row has the sum 0
      const float w = sum[r * splits + k] == 0.f ? 0.f : exp2_fast(weight[r * splits + k] - top);
      weight[r * splits + k] = w;
      if (w != 0.f) l += w * sum[r * splits + k];
    }
    inv[r] = l != 0.f ? 1.f / l : 0.f;
    const int R = row0 + r, tok = R / a.G;
    if (a.lse) a.lse[(int64_t)(lo + tok) * a.Hq + kh * a.G + (R - tok * a.G)] = row_lse(top, l);
  }
  __syncthreads();
  for (int u = threadIdx.x; u < rows * quads; u += blockDim.x) {
    const int r = u / quads, d = (u - r * quads) * 4;
    const float* at = part + (int64_t)r * (D + 2) + 2 + d;
    const float* w = weight + r * splits;
    float o[4] = {};
#pragma unroll 8
    for (int k = 0; k < splits; ++k) {
      const float2 x0 = __ldcg(reinterpret_cast<const float2*>(at + k * step));
      const float2 x1 = __ldcg(reinterpret_cast<const float2*>(at + k * step + 2));
      const float wk = w[k];
      if (wk != 0.f) o[0] += wk * x0.x, o[1] += wk * x0.y, o[2] += wk * x1.x, o[3] += wk * x1.y;
    }
    const int R = row0 + r, tok = R / a.G;
    const int64_t row = (int64_t)(lo + tok) * a.Hq + kh * a.G + (R - tok * a.G);
    const float n = inv[r];
    if (sizeof(T) == 2)
      *reinterpret_cast<uint2*>(a.out + (row * D + d) * 2) =
          make_uint2(pack_bf16x2(o[0] * n, o[1] * n), pack_bf16x2(o[2] * n, o[3] * n));
    else
      *reinterpret_cast<float4*>(a.out + (row * D + d) * 4) = make_float4(o[0] * n, o[1] * n, o[2] * n, o[3] * n);
  }
}

}  // namespace dcp
