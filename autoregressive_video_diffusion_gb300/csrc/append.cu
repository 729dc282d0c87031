// Rotary turn of the new tokens' q and k, and k, v into the cache's pages, in one pass over the data.
//
// A CTA takes a token: each thread first loads its first vectors of q, k, v (they depend on nothing), then the CTA
// finds the token's sequence, phase and page row and builds its cos/sin in shared memory, then turns and stores.  The
// phase in turns is an integer product modulo 2^64, so whole turns drop out exactly at any distance; cos and sin are
// taken of 32 bits of the remaining fraction, once per token and pair, and shared by all heads.  (The plan's fractions
// are good to 2^-62 of a turn and the cut is one of 2^-32, so the phase is off by less than 2^-30 turns at the ends of
// the int32 range.)
// The bound is HBM (each of q, k, v read and written once); a few tokens are bound by the chain launch -> q_start,
// kv_len -> table -> store.  Measured: 6240 tokens of 40 + 40 + 40 heads of 128 in bf16 68 us (5.7 TB/s), 3375 tokens
// of 32 + 8 + 8 fp32 heads of 96 25 us (5.0 TB/s), 32 tokens 4.0 us in a graph.
#include "serve.cuh"

namespace dcp {

namespace {

constexpr int kTurners = 128;  // threads of a CTA

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

template <typename T, int PAIRS>
__global__ void __launch_bounds__(kTurners) append_kernel(const __grid_constant__ AppendParams p) {
  using E = Elems<T>;
  constexpr int N = E::kN;
  constexpr int kUnits = PAIRS == kHalfVec ? 2 : 4;  // units (one or two vectors) a thread has in flight, twice
  __shared__ Where where;
  __shared__ float2 cs[DCP_ROPE_MAX_PAIRS];
  __shared__ uint4 rows[PAIRS == kHalfAny ? kUnits * kTurners : 1];
  const int64_t tok = blockIdx.x;
  const int D = p.pool.D, vecs = D / N, half = p.half, heads = p.Hq + 2 * p.pool.H;
  const int pair_vecs = PAIRS == kHalfVec ? half / N : 0;   // units of two vectors in a head
  const int per_head = vecs - pair_vecs;
  const int per_token = heads * per_head;
  // units of a token a thread holds at once; whole heads where they pass through shared memory
  const int batch = PAIRS == kHalfAny ? kUnits * kTurners / per_head * per_head : kUnits * kTurners;

  // A thread's units are kTurners apart: their head and place follow one another without a division.
  const int head_step = kTurners / per_head, unit_step = kTurners - head_step * per_head;
  uint4 x[2][kUnits], y[2][kUnits];
  struct Unit {
    int i, h, e;  // place in the batch, head (q, then k, then v), unit of the head
  };
  auto first = [&](int u0) {
    const int u = u0 + threadIdx.x, h = u / per_head;
    return Unit{(int)threadIdx.x, h, u - h * per_head};
  };
  auto next = [&](Unit& u) {
    u.i += kTurners;
    u.h += head_step;
    u.e += unit_step;
    if (u.e >= per_head) {
      u.e -= per_head;
      ++u.h;
    }
  };
  auto there = [&](const Unit& u) { return u.i < batch && u.h < heads; };
  auto load = [&](Unit u, uint4 (&a)[kUnits], uint4 (&b)[kUnits]) {
    const T* q = (const T*)p.q + tok * p.q_stride;
    const T* k = (const T*)p.k + tok * p.kv_stride - p.Hq * D;
    const T* v = (const T*)p.v + tok * p.kv_stride - (p.Hq + p.pool.H) * D;
#pragma unroll
    for (int j = 0; j < kUnits; ++j, next(u)) {
      if (!there(u)) continue;
      const uint4* src = (const uint4*)((u.h < p.Hq ? q : u.h < p.Hq + p.pool.H ? k : v) + u.h * D);
      a[j] = src[u.e < pair_vecs ? u.e : u.e + pair_vecs];
      if (PAIRS == kHalfVec && u.e < pair_vecs) b[j] = src[u.e + pair_vecs];
    }
  };

  allow_dependents();
  wait_for_predecessor();
  load(first(0), x[0], y[0]);
  if (threadIdx.x == 0) where.seq = -1;
  __syncthreads();
  for (int s = threadIdx.x; s < p.b.n_seqs; s += kTurners) {
    int lo, len;
    int64_t kv;
    const bool sound = seq_rows(p.b, s, lo, len) & seq_kv(p.b, p.pool.bs, p.pool.H, s, 0, kv);
    if (!sound || tok < lo || tok >= lo + len) continue;
    const int64_t c = kv - len + (tok - lo);
    Where w{-1, (int32_t)c, s};
    if (c >= 0) {
      const int64_t page = c / p.pool.bs;
      const int64_t blk = p.b.tables[s * p.b.table_stride + page];
      if (blk >= 0 && blk < p.pool.n_blocks)
        w.off = blk * p.pool.s_block + (c - page * p.pool.bs) * p.pool.s_row;
      else
        set_status(p.b.status, DCP_EDEVICE);
    }
    where = w;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < half; i += kTurners) {
    const int32_t phase = p.positions ? p.positions[tok] : where.phase;
    const uint64_t turn = (uint64_t)(int64_t)phase * p.turns[i];
    // the fraction of a turn, 32 bits: what fp32 holds of it, and the rest as a first-order correction
    const int32_t fraction = (int32_t)(turn >> 32);
    const float most = (float)fraction;
    const float rest = (float)((int64_t)fraction - (int64_t)most) * (float)(3.14159265358979323846 * 0x1p-31);
    float s, c;
    sincospif(most * 0x1p-31f, &s, &c);
    cs[i] = make_float2(fmaf(-s, rest, c) * p.amplitude, fmaf(c, rest, s) * p.amplitude);
  }
  __syncthreads();

  const int batches = (per_token + batch - 1) / batch;
  auto turn_and_store = [&](Unit u, uint4 (&a)[kUnits], uint4 (&b)[kUnits]) {
    const Where w = where;
    if (PAIRS == kHalfAny) {
      __syncthreads();
#pragma unroll
      for (int j = 0; j < kUnits; ++j)
        if (threadIdx.x + j * kTurners < batch) rows[threadIdx.x + j * kTurners] = a[j];
      __syncthreads();
    }
    if (w.seq < 0) return;
    T* const q_to = (T*)p.q_out + (int64_t)tok * p.Hq * D;
#pragma unroll
    for (int j = 0; j < kUnits; ++j, next(u)) {
      if (!there(u)) continue;
      const int h = u.h, e = u.e;
      const bool is_q = h < p.Hq, is_v = h >= p.Hq + p.pool.H;
      if (!is_q && w.off < 0) continue;
      uint4* dst = (uint4*)(is_q ? q_to + h * D
                                 : (T*)(is_v ? p.pool.v : p.pool.k) + w.off +
                                       (h - (is_v ? p.Hq + p.pool.H : p.Hq)) * p.pool.s_head);
      const int v = e + pair_vecs;  // of a unit of one vector
      if (PAIRS == kHalfVec && e < pair_vecs) {
        if (!is_v) {
          float f[N], g[N];
          E::get(a[j], f);
          E::get(b[j], g);
#pragma unroll
          for (int k = 0; k < N; ++k) {
            const float2 r = cs[e * N + k];
            const float f2 = f[k] * r.x - g[k] * r.y;
            g[k] = f[k] * r.y + g[k] * r.x;
            f[k] = f2;
          }
          a[j] = E::put(f);
          b[j] = E::put(g);
        }
        dst[e] = a[j];
        dst[v] = b[j];
        continue;
      }
      if (PAIRS == kInterleaved && !is_v && v * N < 2 * half) {
        float f[N];
        E::get(a[j], f);
#pragma unroll
        for (int k = 0; k < N; k += 2) {
          const int q = v * (N / 2) + k / 2;
          if (q >= half) continue;
          const float2 r = cs[q];
          const float f2 = f[k] * r.x - f[k + 1] * r.y;
          f[k + 1] = f[k] * r.y + f[k + 1] * r.x;
          f[k] = f2;
        }
        a[j] = E::put(f);
      }
      if (PAIRS == kHalfAny && !is_v && v * N < 2 * half) {
        float f[N];
        E::get(a[j], f);
        const uint4* row = rows + u.i - e;
#pragma unroll
        for (int k = 0; k < N; ++k) {
          const int d = v * N + k;
          if (d >= 2 * half) continue;
          const float2 r = cs[d < half ? d : d - half];
          f[k] = d < half ? f[k] * r.x - E::one(row, d + half) * r.y : f[k] * r.x + E::one(row, d - half) * r.y;
        }
        a[j] = E::put(f);
      }
      dst[v] = a[j];
    }
  };
  // the next batch's loads are in flight while a batch is turned and stored
  for (int b = 0; b < batches; b += 2) {
    if (b + 1 < batches) load(first((b + 1) * batch), x[1], y[1]);
    turn_and_store(first(b * batch), x[0], y[0]);
    if (b + 1 == batches) break;
    if (b + 2 < batches) load(first((b + 2) * batch), x[0], y[0]);
    turn_and_store(first((b + 1) * batch), x[1], y[1]);
  }
}

template <typename T, int PAIRS>
cudaError_t launch_tokens(const AppendParams& p, cudaStream_t s) {
  // A token a CTA of 128 threads, so that many CTAs are at different places of their chain.  (6240 tokens of 120
  // heads / 3375 of 48 fp32 heads whose units are two vectors: 4 units a thread 67 / 35 us, 2 units 71 / 26; two
  // tokens a CTA of 256 threads 74 / 29, four 81 / 35.)
  return launch_behind(append_kernel<T, PAIRS>, dim3((unsigned)p.b.total_q), kTurners, 0, s, p);
}

template <typename T>
cudaError_t launch_pairs(const AppendParams& p, cudaStream_t s) {
  if (!p.half_layout) return launch_tokens<T, kInterleaved>(p, s);
  if (p.half % Elems<T>::kN == 0) return launch_tokens<T, kHalfVec>(p, s);
  return launch_tokens<T, kHalfAny>(p, s);
}

}  // namespace

cudaError_t launch_append(const AppendParams& p, cudaStream_t s) {
  return p.pool.dtype == DCP_BF16 ? launch_pairs<__nv_bfloat16>(p, s) : launch_pairs<float>(p, s);
}

}  // namespace dcp
