// Rotary turn of the new tokens' q and k, and k, v into the cache's pages.
#include "serve.cuh"

namespace dcp {

namespace {

constexpr int kTok = 4;  // tokens a CTA

struct Where {
  int64_t off;   // element offset of the token's row in head 0 of the pool, -1: not stored
  int32_t phase;
  int32_t seq;   // -1: no sequence owns the row
};

template <typename T>
__device__ __forceinline__ float to_f(T x);
template <>
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
template <>
__device__ __forceinline__ float to_f(float x) { return x; }
template <typename T>
__device__ __forceinline__ T from_f(float x);
template <>
__device__ __forceinline__ __nv_bfloat16 from_f(float x) { return __float2bfloat16_rn(x); }
template <>
__device__ __forceinline__ float from_f(float x) { return x; }

template <typename T>
__global__ void __launch_bounds__(kThreads) append_kernel(const __grid_constant__ AppendParams p) {
  extern __shared__ float2 cs[];  // [kTok][half]
  __shared__ Where where[kTok];
  const int t0 = blockIdx.x * kTok;
  const int n = min(kTok, p.b.total_q - t0);
  if (threadIdx.x < kTok) where[threadIdx.x].seq = -1;
  __syncthreads();
  for (int s = threadIdx.x; s < p.b.n_seqs; s += blockDim.x) {
    int lo, len;
    if (!seq_rows(p.b, s, lo, len)) continue;
    for (int t = max(lo, t0); t < min(lo + len, t0 + n); ++t) where[t - t0].seq = s;
  }
  __syncthreads();
  if (threadIdx.x < n) {
    Where& w = where[threadIdx.x];
    w.off = -1;
    w.phase = 0;
    int lo, len;
    int64_t kv;
    if (w.seq >= 0 && seq_rows(p.b, w.seq, lo, len) && seq_kv(p.b, p.pool.bs, p.pool.H, w.seq, 0, kv)) {
      const int64_t c = kv - len + (t0 + threadIdx.x - lo);
      w.phase = p.positions ? p.positions[t0 + threadIdx.x] : (int32_t)c;
      if (c >= 0) {
        const int64_t blk = p.b.tables[w.seq * p.b.table_stride + c / p.pool.bs];
        if (blk >= 0 && blk < p.pool.n_blocks)
          w.off = blk * p.pool.s_block + (c % p.pool.bs) * p.pool.s_row;
        else
          set_status(p.b.status, DCP_EDEVICE);
      }
    } else {
      w.seq = -1;
    }
  }
  __syncthreads();
  // the phase in turns is an integer product modulo 2^64: whole turns drop out exactly at any distance
  for (int i = threadIdx.x; i < n * p.half; i += blockDim.x) {
    const uint64_t turn = (uint64_t)(int64_t)where[i / p.half].phase * p.turns[i % p.half];
    float s, c;
    sincospif((float)(int32_t)(turn >> 32) * 0x1p-31f, &s, &c);
    cs[i] = make_float2(c * p.amplitude, s * p.amplitude);
  }
  __syncthreads();
  const int D = p.pool.D, heads = p.Hq + 2 * p.pool.H, half = p.half;
  // a thread reads both dims of its pair before it writes either (q_out may be q)
  const int units = half + (D - 2 * half);
  for (int i = threadIdx.x; i < n * heads * units; i += blockDim.x) {
    const int u = i % units, h = i / units % heads, t = i / (units * heads);
    const Where w = where[t];
    if (w.seq < 0) continue;
    const bool is_q = h < p.Hq, is_v = h >= p.Hq + p.pool.H;
    const int kh = is_v ? h - p.Hq - p.pool.H : h - p.Hq;
    const T* src = is_q ? (const T*)p.q + (t0 + t) * p.q_stride + (int64_t)h * D
                        : (const T*)(is_v ? p.v : p.k) + (t0 + t) * p.kv_stride + (int64_t)kh * D;
    T* dst = is_q ? (T*)p.q_out + (int64_t)(t0 + t) * p.Hq * D + (int64_t)h * D
                  : (T*)(is_v ? p.pool.v : p.pool.k) + w.off + kh * p.pool.s_head;
    if (!is_q && w.off < 0) continue;
    if (u >= half) {
      dst[half + u] = src[half + u];
      continue;
    }
    const int d0 = p.half_layout ? u : 2 * u, d1 = p.half_layout ? u + half : 2 * u + 1;
    T y0 = src[d0], y1 = src[d1];
    if (!is_v) {
      const float2 r = cs[t * half + u];
      const float a = to_f(y0), b = to_f(y1);
      y0 = from_f<T>(a * r.x - b * r.y);
      y1 = from_f<T>(a * r.y + b * r.x);
    }
    dst[d0] = y0;
    dst[d1] = y1;
  }
}

}  // namespace

cudaError_t launch_append(const AppendParams& p, cudaStream_t s) {
  const size_t smem = sizeof(float2) * kTok * p.half;
  const int grid = (p.b.total_q + kTok - 1) / kTok;
  if (p.pool.dtype == DCP_BF16)
    append_kernel<__nv_bfloat16><<<grid, kThreads, smem, s>>>(p);
  else
    append_kernel<float><<<grid, kThreads, smem, s>>>(p);
  return cudaGetLastError();
}

}  // namespace dcp
