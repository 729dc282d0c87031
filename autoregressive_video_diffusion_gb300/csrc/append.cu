// Rotary turn of the new tokens' q and k, and k, v into the cache's pages, in one pass over the data.
//
// A CTA takes a few tokens: each thread first loads its first vectors of q, k, v (they depend on nothing), then the
// CTA finds the tokens' sequences, phases and page rows and builds their cos/sin in shared memory, then turns and
// stores.  The phase in turns is an integer product modulo 2^64, so whole turns drop out exactly at any distance; cos
// and sin are taken of the remaining fraction, once per token and pair, and shared by all heads.
// The bound is HBM (each of q, k, v read and written once); a few tokens are bound by the chain launch -> q_start,
// kv_len -> table -> store.
#include "serve.cuh"

namespace dcp {

namespace {

constexpr int kUnits = 4;  // units (one or two 16-byte vectors) a thread has in flight

struct Where {
  int64_t off;   // element offset of the token's row in head 0 of the pool, -1: not stored
  int32_t phase;
  int32_t seq;   // -1: no sequence owns the row
};

// Elements of a 16-byte vector in fp32 and back (bf16: round to nearest even, once).
template <typename T>
struct Elems;
template <>
struct Elems<__nv_bfloat16> {
  static constexpr int kN = 8;
  static __device__ __forceinline__ void get(const uint4& x, float (&y)[8]) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      y[2 * i] = bf16lo(w[i]);
      y[2 * i + 1] = bf16hi(w[i]);
    }
  }
  static __device__ __forceinline__ uint4 put(const float (&y)[8]) {
    return make_uint4(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]), pack_bf16x2(y[4], y[5]),
                      pack_bf16x2(y[6], y[7]));
  }
  static __device__ __forceinline__ float one(const uint4* row, int d) {
    return __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(row)[d]);
  }
};
template <>
struct Elems<float> {
  static constexpr int kN = 4;
  static __device__ __forceinline__ void get(const uint4& x, float (&y)[4]) {
    y[0] = __uint_as_float(x.x), y[1] = __uint_as_float(x.y), y[2] = __uint_as_float(x.z), y[3] = __uint_as_float(x.w);
  }
  static __device__ __forceinline__ uint4 put(const float (&y)[4]) {
    return make_uint4(__float_as_uint(y[0]), __float_as_uint(y[1]), __float_as_uint(y[2]), __float_as_uint(y[3]));
  }
  static __device__ __forceinline__ float one(const uint4* row, int d) {
    return reinterpret_cast<const float*>(row)[d];
  }
};

enum Pairs {
  kInterleaved,  // pair (2p, 2p + 1): inside a vector
  kHalfVec,      // pair (p, p + half), half a whole number of vectors: a unit is the two vectors of its pairs
  kHalfAny,      // any other half: partners are read from a copy of the rows in shared memory
};

template <typename T, int PAIRS, int TOK>
__global__ void __launch_bounds__(kThreads) append_kernel(const __grid_constant__ AppendParams p) {
  using E = Elems<T>;
  constexpr int N = E::kN;
  __shared__ Where where[TOK];
  __shared__ float2 cs[TOK][DCP_ROPE_MAX_PAIRS];
  __shared__ uint4 rows[PAIRS == kHalfAny ? kUnits * kThreads : 1];
  const int t0 = blockIdx.x * TOK, n = min(TOK, p.b.total_q - t0);
  const int D = p.pool.D, vecs = D / N, half = p.half, heads = p.Hq + 2 * p.pool.H;
  const int pair_vecs = PAIRS == kHalfVec ? half / N : 0;   // units of two vectors in a head
  const int per_head = vecs - pair_vecs;
  const int per_token = heads * per_head;
  // units of a token a thread holds at once; whole heads where they pass through shared memory
  const int batch = PAIRS == kHalfAny ? kUnits * kThreads / per_head * per_head : kUnits * kThreads;

  uint4 x[kUnits], y[kUnits];
  auto source = [&](int t, int h) {
    return h < p.Hq ? (const uint4*)((const T*)p.q + (t0 + t) * p.q_stride + (int64_t)h * D)
           : h < p.Hq + p.pool.H
               ? (const uint4*)((const T*)p.k + (t0 + t) * p.kv_stride + (int64_t)(h - p.Hq) * D)
               : (const uint4*)((const T*)p.v + (t0 + t) * p.kv_stride + (int64_t)(h - p.Hq - p.pool.H) * D);
  };
  auto load = [&](int t, int u0) {
#pragma unroll
    for (int j = 0; j < kUnits; ++j) {
      const int i = threadIdx.x + j * kThreads, u = u0 + i;
      if (i >= batch || u >= per_token) continue;
      const int h = u / per_head, e = u - h * per_head;
      const uint4* src = source(t, h);
      x[j] = src[e < pair_vecs ? e : e + pair_vecs];
      if (e < pair_vecs) y[j] = src[e + pair_vecs];
    }
  };

  load(0, 0);
  if (threadIdx.x < TOK) where[threadIdx.x].seq = -1;
  __syncthreads();
  for (int s = threadIdx.x; s < p.b.n_seqs; s += kThreads) {
    int lo, len;
    int64_t kv;
    const bool sound = seq_rows(p.b, s, lo, len) & seq_kv(p.b, p.pool.bs, p.pool.H, s, 0, kv);
    if (!sound) continue;
    for (int t = max(lo, t0); t < min(lo + len, t0 + n); ++t) {
      const int64_t c = kv - len + (t - lo);
      Where w{-1, (int32_t)c, s};
      if (c >= 0) {
        const int64_t page = c / p.pool.bs;
        const int64_t blk = p.b.tables[s * p.b.table_stride + page];
        if (blk >= 0 && blk < p.pool.n_blocks)
          w.off = blk * p.pool.s_block + (c - page * p.pool.bs) * p.pool.s_row;
        else
          set_status(p.b.status, DCP_EDEVICE);
      }
      where[t - t0] = w;
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < n * half; i += kThreads) {
    const int t = i / half, q = i - t * half;
    const int32_t phase = p.positions ? p.positions[t0 + t] : where[t].phase;
    const uint64_t turn = (uint64_t)(int64_t)phase * p.turns[q];
    float s, c;
    sincospif((float)(int32_t)(turn >> 32) * 0x1p-31f, &s, &c);
    cs[t][q] = make_float2(c * p.amplitude, s * p.amplitude);
  }
  __syncthreads();

  for (int t = 0; t < n; ++t) {
    const Where w = where[t];
    for (int u0 = 0; u0 < per_token; u0 += batch) {
      if (t || u0) load(t, u0);
      if (PAIRS == kHalfAny) {
        __syncthreads();
#pragma unroll
        for (int j = 0; j < kUnits; ++j)
          if (threadIdx.x + j * kThreads < batch) rows[threadIdx.x + j * kThreads] = x[j];
        __syncthreads();
      }
#pragma unroll
      for (int j = 0; j < kUnits; ++j) {
        const int i = threadIdx.x + j * kThreads, u = u0 + i;
        if (i >= batch || u >= per_token || w.seq < 0) continue;
        const int h = u / per_head, e = u - h * per_head;
        const bool is_q = h < p.Hq, is_v = h >= p.Hq + p.pool.H;
        if (!is_q && w.off < 0) continue;
        T* to = is_q ? (T*)p.q_out + (int64_t)(t0 + t) * p.Hq * D + (int64_t)h * D
                     : is_v ? (T*)p.pool.v + w.off + (h - p.Hq - p.pool.H) * p.pool.s_head
                            : (T*)p.pool.k + w.off + (h - p.Hq) * p.pool.s_head;
        uint4* dst = (uint4*)to;
        if (PAIRS == kHalfVec && e < pair_vecs) {
          if (!is_v) {
            float a[N], b[N];
            E::get(x[j], a);
            E::get(y[j], b);
#pragma unroll
            for (int k = 0; k < N; ++k) {
              const float2 r = cs[t][e * N + k];
              const float a2 = a[k] * r.x - b[k] * r.y;
              b[k] = a[k] * r.y + b[k] * r.x;
              a[k] = a2;
            }
            x[j] = E::put(a);
            y[j] = E::put(b);
          }
          dst[e] = x[j];
          dst[e + pair_vecs] = y[j];
          continue;
        }
        const int v = e + pair_vecs;
        if (PAIRS == kInterleaved && !is_v && v * N < 2 * half) {
          float a[N];
          E::get(x[j], a);
#pragma unroll
          for (int k = 0; k < N; k += 2) {
            const int q = v * (N / 2) + k / 2;
            if (q >= half) continue;
            const float2 r = cs[t][q];
            const float a2 = a[k] * r.x - a[k + 1] * r.y;
            a[k + 1] = a[k] * r.y + a[k + 1] * r.x;
            a[k] = a2;
          }
          x[j] = E::put(a);
        }
        if (PAIRS == kHalfAny && !is_v && v * N < 2 * half) {
          float a[N];
          E::get(x[j], a);
          const uint4* row = rows + i - e;
#pragma unroll
          for (int k = 0; k < N; ++k) {
            const int d = v * N + k;
            if (d >= 2 * half) continue;
            const float2 r = cs[t][d < half ? d : d - half];
            a[k] = d < half ? a[k] * r.x - E::one(row, d + half) * r.y : a[k] * r.x + E::one(row, d - half) * r.y;
          }
          x[j] = E::put(a);
        }
        dst[v] = x[j];
      }
    }
  }
}

template <typename T, int PAIRS>
void launch_tokens(const AppendParams& p, cudaStream_t s) {
  // one token a CTA until the SMs have several CTAs each, then four, so that the look-up is shared
  if (p.b.total_q <= 8 * sm_count())
    append_kernel<T, PAIRS, 1><<<p.b.total_q, kThreads, 0, s>>>(p);
  else
    append_kernel<T, PAIRS, 4><<<(p.b.total_q + 3) / 4, kThreads, 0, s>>>(p);
}

template <typename T>
cudaError_t launch_pairs(const AppendParams& p, cudaStream_t s) {
  if (!p.half_layout)
    launch_tokens<T, kInterleaved>(p, s);
  else if (p.half % Elems<T>::kN == 0)
    launch_tokens<T, kHalfVec>(p, s);
  else
    launch_tokens<T, kHalfAny>(p, s);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_append(const AppendParams& p, cudaStream_t s) {
  return p.pool.dtype == DCP_BF16 ? launch_pairs<__nv_bfloat16>(p, s) : launch_pairs<float>(p, s);
}

}  // namespace dcp
