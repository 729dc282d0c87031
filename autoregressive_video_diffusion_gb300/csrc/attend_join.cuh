// Attention whose keys are split over CTAs: the partial results and how the last CTA joins them.
#pragma once

#include "serve.cuh"

namespace dcp {

// A split leaves for each of its rows [m, l, -, -, o_0 .. o_{D-1}] in fp32: the running maximum of the scores before
// scaling (scaled maxima lose the bits that tell large ones apart), and the sums of weights and weighted values relative
// to it.  An item's parts are [split][rows][kPartHead + D].
constexpr int kPartHead = 4;

__device__ __forceinline__ float* part_of(float* parts, int64_t item, int splits, int split, int rows, int D, int r) {
  return parts + ((item * splits + split) * rows + r) * (int64_t)(kPartHead + D);
}

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// lse of a row from its maximum (before scaling) and sum.
__device__ __forceinline__ float row_lse(const AttendParams& a, float m, float l) {
  return l != 0.f ? m * fabsf(a.scale) + __log2f(l) * 0.6931471805599453f : -INFINITY;
}

// Called by a whole CTA after its part is written; true for the item's last CTA.  The parts are read in the order of
// the splits, so the result does not depend on which CTA comes last.
__device__ __forceinline__ bool last_of(uint32_t* done, int splits, int* s_last) {
  __syncthreads();  // the other threads' writes are ordered before this thread's release
  if (threadIdx.x == 0) {
    uint32_t before;
    asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], 1;" : "=r"(before) : "l"(done) : "memory");
    *s_last = before == (uint32_t)splits - 1;
    if (*s_last) *done = 0;
  }
  __syncthreads();
  return *s_last;
}

// Joins `splits` parts of `rows` rows whose first is row `row0` of (token, head of the KV
// head) rows, sequence start lo.  Called by a whole CTA; scratch: `room` bytes of shared memory, at least
// join_scratch(rows, splits).  Everything is fetched at once where it fits the scratch (a loop over the parts in global
// memory pays a memory latency every few of them: 5 us for 12 parts of 5 rows, 1 us this way), else the maxima and sums
// first and the values with several loads in flight.
__host__ __device__ constexpr int64_t join_scratch(int rows, int splits) {
  return (int64_t)rows * (2 * splits + 1) * 4;
}

// The first part is at `part0`, the others from `part1` on, `step` floats apart.
template <typename T>
__device__ __forceinline__ void join_parts(const AttendParams& a, const float* part0, const float* part1, int64_t step,
                                           int splits, int rows, int row0, int lo, int kh, uint8_t* scratch,
                                           int64_t room) {
  const int D = a.pool.D, quads = D / 4, width = kPartHead + D;
  auto part = [&](int k) { return k ? part1 + (k - 1) * step : part0; };
  float* const weight = reinterpret_cast<float*>(scratch);  // [rows][splits]: the maximum, then the part's weight
  float* const sum = weight + rows * splits;                // [rows][splits]
  float* const inv = sum + rows * splits;                   // [rows]
  const int64_t used = (join_scratch(rows, splits) + 15) & ~(int64_t)15;
  __syncthreads();
  const bool local = used + (int64_t)rows * splits * width * 4 <= room;
  if (local) {
    const int chunks = rows * width / 4;
    const uint32_t to = smem_u32(scratch + used);
    for (int u = threadIdx.x; u < splits * chunks; u += blockDim.x) {
      const int k = u / chunks;
      cp_async16(to + u * 16, part(k) + (u - k * chunks) * 4);
    }
    cp_async_commit();
    cp_async_wait<0>();
    __syncthreads();
    step = (int64_t)rows * width;
    part0 = reinterpret_cast<const float*>(scratch + used);
    part1 = part0 + step;
  }
  for (int u = threadIdx.x; u < rows * splits; u += blockDim.x) {
    const int r = u / splits;
    const float2* at = reinterpret_cast<const float2*>(part(u - r * splits) + (int64_t)r * width);
    const float2 ml = local ? *at : __ldcg(at);
    weight[u] = ml.x;
    sum[u] = ml.y;
  }
  __syncthreads();
  // a warp a row: the parts' weights (a split that saw no key of the row has the sum 0)
  for (int r = threadIdx.x >> 5; r < rows; r += blockDim.x >> 5) {
    const int lane = threadIdx.x & 31;
    float* const w = weight + r * splits;
    const float* const ls = sum + r * splits;
    float top = -INFINITY, l = 0.f;
    for (int k = lane; k < splits; k += 32)
      if (ls[k] != 0.f) top = fmaxf(top, w[k]);
#pragma unroll
    for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
    for (int k = lane; k < splits; k += 32) {
      const float wk = ls[k] == 0.f ? 0.f : exp2_fast((w[k] - top) * a.scale_log2);
      w[k] = wk;
      if (wk != 0.f) l += wk * ls[k];
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) l += __shfl_xor_sync(~0u, l, o);
    if (lane == 0) {
      inv[r] = l != 0.f ? 1.f / l : 0.f;
      const int R = row0 + r, tok = R / a.G;
      if (a.lse) a.lse[(int64_t)(lo + tok) * a.Hq + kh * a.G + (R - tok * a.G)] = row_lse(a, top, l);
    }
  }
  __syncthreads();
  for (int u = threadIdx.x; u < rows * quads; u += blockDim.x) {
    const int r = u / quads, d = (u - r * quads) * 4;
    const int64_t at = (int64_t)r * width + kPartHead + d;
    const float* w = weight + r * splits;
    float o[4] = {};
#pragma unroll 8
    for (int k = 0; k < splits; ++k) {
      const float4* from = reinterpret_cast<const float4*>(part(k) + at);
      const float4 x = local ? *from : __ldcg(from);
      const float wk = w[k];
      if (wk != 0.f) o[0] += wk * x.x, o[1] += wk * x.y, o[2] += wk * x.z, o[3] += wk * x.w;
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
