// Attention of the new tokens over the paged cache.
#include "serve.cuh"

namespace dcp {

namespace {

template <typename T>
__device__ __forceinline__ float load_f(const T* x);
template <>
__device__ __forceinline__ float load_f(const __nv_bfloat16* x) { return __bfloat162float(*x); }
template <>
__device__ __forceinline__ float load_f(const float* x) { return *x; }

// One warp a row (new token, query head): 32 keys at a time, a key a lane, with the running maximum and sum of the
// softmax; then each lane adds up its own dims of the weighted values.
template <typename T>
__global__ void __launch_bounds__(128) rows_kernel(const __grid_constant__ AttendParams p) {
  __shared__ float qs[4][128];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int s = blockIdx.y, D = p.pool.D;
  int lo, len;
  if (!seq_rows(p.b, s, lo, len)) return;
  const int64_t r = (int64_t)blockIdx.x * 4 + warp;
  if (r >= (int64_t)len * p.Hq) return;
  const int i = (int)(r / p.Hq), h = (int)(r % p.Hq), kh = h / p.G;
  int64_t kv;
  if (!seq_kv(p.b, p.pool.bs, p.pool.H, s, kh, kv)) return;
  const int64_t c = kv - len + i;
  const int64_t hi = p.causal ? min(kv, c + 1) : kv;
  const int64_t first = p.window >= 0 ? max((int64_t)0, c - p.window) : 0;
  const T* q = (const T*)p.q + (lo + i) * p.q_stride + (int64_t)h * D;
  for (int d = lane; d < D; d += 32) qs[warp][d] = load_f(q + d) * p.scale;
  __syncwarp();
  float m = -INFINITY, l = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
  for (int64_t j0 = first; j0 < hi; j0 += 32) {
    const int64_t j = j0 + lane;
    int64_t off = -1;
    float x = -INFINITY;
    if (j < hi) {
      const int64_t blk = p.b.tables[s * p.b.table_stride + j / p.pool.bs];
      if (blk >= 0 && blk < p.pool.n_blocks) {
        off = blk * p.pool.s_block + (int64_t)kh * p.pool.s_head + (j % p.pool.bs) * p.pool.s_row;
        x = 0.f;
        for (int d = 0; d < D; ++d) x = fmaf(qs[warp][d], load_f((const T*)p.pool.k + off + d), x);
      } else {
        set_status(p.b.status, DCP_EDEVICE);
      }
    }
    float top = x;
    for (int b = 16; b; b >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, b));
    const float m2 = fmaxf(m, top), keep = m == m2 ? 1.f : expf(m - m2);
    m = m2;
    const float w = x == -INFINITY ? 0.f : expf(x - m);
    float sum = w;
    for (int b = 16; b; b >>= 1) sum += __shfl_xor_sync(~0u, sum, b);
    l = l * keep + sum;
    for (int e = 0; e < 4; ++e) o[e] *= keep;
    for (int k = 0; k < 32; ++k) {
      const float wk = __shfl_sync(~0u, w, k);
      const int64_t at = __shfl_sync(~0u, off, k);
      if (at < 0) continue;
      for (int e = 0; e < 4; ++e)
        if (lane + 32 * e < D) o[e] = fmaf(wk, load_f((const T*)p.pool.v + at + lane + 32 * e), o[e]);
    }
  }
  const int64_t row = (int64_t)(lo + i) * p.Hq + h;
  for (int e = 0; e < 4; ++e) {
    if (lane + 32 * e >= D) continue;
    const float y = l != 0.f ? o[e] / l : 0.f;
    if (p.pool.dtype == DCP_BF16)
      ((__nv_bfloat16*)p.out)[row * D + lane + 32 * e] = __float2bfloat16_rn(y);
    else
      ((float*)p.out)[row * D + lane + 32 * e] = y;
  }
  if (p.lse && lane == 0) p.lse[row] = l != 0.f ? m + logf(l) : -INFINITY;
}

}  // namespace

cudaError_t launch_attend_rows(const AttendParams& p, cudaStream_t s) {
  const dim3 grid((unsigned)(((int64_t)p.b.max_q * p.Hq + 3) / 4), p.b.n_seqs);
  if (p.pool.dtype == DCP_BF16)
    rows_kernel<__nv_bfloat16><<<grid, 128, 0, s>>>(p);
  else
    rows_kernel<float><<<grid, 128, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace dcp
