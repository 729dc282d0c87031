// Root-mean-square norms of the new tokens' q and k, their rotary turn by up to three position axes, and k, v into the
// cache's pages, in one pass over the data.
//
//   y = x / sqrt(mean x^2 + eps) * w,  then each pair (a, b) of axis a turns by position[a] * theta: one rounding at the end
//
// The mean goes over a head, or over all heads of a token (q and k apart).  A CTA takes a token: its loads are issued
// first (they depend on nothing), under them it finds the token's place and builds its cos/sin.  A head lies in the
// registers of a power of two of neighbouring lanes, a 16-byte vector each (two where the pairs are a whole number of
// vectors apart), so a head's sum is a few shuffles and a token's one barrier; the values are still in registers when
// the sum is known, which makes it one pass (tokens of more than 128 heads of 128 are read again behind the first ones).
//
// Squares leave fp32 for values past 2^60 or below 2^-50 with an eps as small: such a sum is taken again of values scaled
// by a power of two, which every norm of the row shares, so that any finite values give what the formula says.
#include <algorithm>

#include "append.cuh"

namespace dcp {

namespace {

constexpr int kNormThreads = 512;     // of a CTA at most
constexpr int kNormResident = 1024;   // of an SM, by registers
constexpr int kUnits = 4;             // vectors of q and k a thread has in flight
constexpr int kBlock = 16;    // tokens whose places a CTA looks up at a time

// The factors of a norm: y = (x * up) * r; up is 1 but for values that are taken scaled.
struct Norm {
  float up, r;
};
constexpr float kMostSum = 0x1p120f, kLeastMean = 0x1p-100f;

// The scale at which a sum that left fp32's comfortable range is taken again, 1 where it did not.
__device__ __forceinline__ float rescale(float sum, float inv, float eps) {
  return !(sum <= kMostSum) ? 0x1p-80f : fmaf(sum, inv, eps) < kLeastMean ? 0x1p100f : 1.f;
}
// The sum was taken of values times c.
__device__ __forceinline__ Norm norm_of(float sum, float inv, float eps, float c) {
  const float m = fmaf(sum, inv, eps * c * c), r = rsqrtf(m);
  const float better = fmaf(0.5f * r, fmaf(-m * r, r, 1.f), r);  // a step of Newton's: 2 ulp to half of one
  return Norm{fmaxf(c, 1.f), (m > 0.f && m < INFINITY ? better : r) * fminf(c, 1.f)};
}

// A vector that is read once.
__device__ __forceinline__ uint4 load_once(const uint4* p) {
  uint4 x;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w)
               : "l"(p));
  return x;
}

// A vector's elements in pairs, and back.
template <typename T, int N>
__device__ __forceinline__ void pairs_of(const uint4& x, uint64_t (&y)[N / 2]) {
  float f[N];
  Elems<T>::get(x, f);
#pragma unroll
  for (int k = 0; k < N / 2; ++k) y[k] = pair(f[2 * k], f[2 * k + 1]);
}
template <typename T, int N>
__device__ __forceinline__ uint4 vector_of(const uint64_t (&y)[N / 2]) {
  float f[N];
#pragma unroll
  for (int k = 0; k < N / 2; ++k) unpair(y[k], f[2 * k], f[2 * k + 1]);
  return Elems<T>::put(f);
}

// y times consecutive weights of a head, from element `at` on.
template <int N>
__device__ __forceinline__ void weigh(const NormParams& n, const char* weight, int at, uint64_t (&y)[N / 2]) {
  if (!weight) return;
  if (n.weight_bf16) {
    uint32_t w[N / 2];
    if constexpr (N == 8)
      *reinterpret_cast<uint4*>(w) = __ldg(reinterpret_cast<const uint4*>(weight + (int64_t)at * 2));
    else
      *reinterpret_cast<uint2*>(w) = __ldg(reinterpret_cast<const uint2*>(weight + (int64_t)at * 2));
#pragma unroll
    for (int k = 0; k < N / 2; ++k) y[k] = mul2(y[k], pair(bf16lo(w[k]), bf16hi(w[k])));
  } else {
#pragma unroll
    for (int k = 0; k < N / 2; k += 2) {
      const float4 w = __ldg(reinterpret_cast<const float4*>(weight + ((int64_t)at + 2 * k) * 4));
      y[k] = mul2(y[k], pair(w.x, w.y));
      y[k + 1] = mul2(y[k + 1], pair(w.z, w.w));
    }
  }
}

// Where element d of a row of LENGTH lies in shared memory: quads of a vector's elements apart, those of neighbouring
// vectors side by side, so that the lanes' reads of a quad hit no bank twice.
template <int N, int LENGTH>
__device__ __forceinline__ int place(int d) {
  return (d % N / 4 * (LENGTH / N) + d / N) * 4 + d % 4;
}

template <typename T, int PAIRS, bool TOKEN, bool WEIGHTS>
__global__ void __launch_bounds__(kNormThreads, kNormResident / kNormThreads)
    norm_kernel(const __grid_constant__ NormParams n) {
  using E = Elems<T>;
  constexpr int N = E::kN, kWarps = kNormThreads / 32, kEs = sizeof(T);
  constexpr int kTwo = PAIRS == kHalfVec ? 2 : 1;  // vectors of a unit (a head's part in a lane)
  constexpr int kHeads = kUnits / kTwo;            // units of as many q and k heads that a thread has in flight
  constexpr int kValues = kTwo == 2 ? 1 : 2;       // and of v heads
  __shared__ Where where[kBlock];
  // cos and sin of a token's pairs: (c, s) in the places of the pair's elements, or all cosines, then all sines
  __shared__ __align__(16) float cs[kBlock][2 * DCP_ROPE_MAX_PAIRS];
  __shared__ float2 sums[3][kWarps];
  __shared__ __align__(16) float ws[WEIGHTS ? 1 : 2][WEIGHTS ? 4 : 128];  // weights that all heads share
  __shared__ uint4 rows[PAIRS == kHalfAny ? kNormThreads : 1];
  const AppendParams& p = n.a;
  const int D = p.pool.D, half = p.half, turned = p.Hq + p.pool.H;
  const int pair_vecs = PAIRS == kHalfVec ? half / N : 0;  // units of two vectors in a head
  const int per_head = D / N - pair_vecs;
  const int threads = blockDim.x, e = threadIdx.x & ((1 << n.lanes_log2) - 1), step = threads >> n.lanes_log2;
  const int h0 = threadIdx.x >> n.lanes_log2;  // the thread's heads: h0, h0 + step, ...
  const bool there = e < per_head, two = PAIRS == kHalfVec && e < pair_vecs;
  const int vec = two ? e : e + pair_vecs;  // the unit's (first) vector
  const int begin = (int)((int64_t)p.b.total_q * blockIdx.x / gridDim.x);  // the CTA's tokens
  const int end = (int)((int64_t)p.b.total_q * (blockIdx.x + 1) / gridDim.x);

  // The thread's vector of head h0 as a q, a k and a v head, of the token to be loaded, and where they go.  (Heads follow
  // one another by the same distance, so that a unit's address is a sum.)
  const int from_k = (h0 - p.Hq) * D * kEs, vec_at = vec * 16;
  const char* q_src = p.q + (begin * p.q_stride + h0 * D) * kEs + vec_at;
  const char* k_src = p.k + begin * p.kv_stride * kEs + from_k + vec_at;
  const char* v_src = p.v + (begin * p.kv_stride + h0 * D) * kEs + vec_at;
  char* q_dst = p.q_out + (begin * (int64_t)p.Hq + h0) * D * kEs + vec_at;
  char* const k_dst = p.pool.k + (h0 - p.Hq) * p.pool.s_head * kEs + vec_at;
  char* const v_dst = p.pool.v + h0 * p.pool.s_head * kEs + vec_at;
  const int next_head = step * D * kEs;
  const int64_t next_page_head = step * p.pool.s_head * kEs;

  auto fetch = [&](uint4 (&to)[kTwo], const char* from, bool real) {
#pragma unroll
    for (int i = 0; i < kTwo; ++i) to[i] = make_uint4(0, 0, 0, 0);
    if (!real) return;
    to[0] = load_once((const uint4*)from);
    if constexpr (kTwo == 2)
      if (two) to[1] = load_once((const uint4*)from + pair_vecs);
  };
  auto put = [&](char* to, const uint4& a, int which) {
    if (which == 0)
      *(uint4*)to = a;
    else
      ((uint4*)to)[pair_vecs] = a;
  };
  auto squares = [&](const uint4 (&a)[kTwo]) {
    uint64_t s = 0;
#pragma unroll
    for (int i = 0; i < kTwo; ++i) {
      uint64_t f[N / 2];
      pairs_of<T, N>(a[i], f);
#pragma unroll
      for (int k = 0; k < N / 2; ++k) s = fma2(f[k], f[k], s);
    }
    float s0, s1;
    unpair(s, s0, s1);
    return s0 + s1;
  };
  auto scaled_squares = [&](const uint4 (&a)[kTwo], float c) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < kTwo; ++i) {
      float f[N];
      E::get(a[i], f);
#pragma unroll
      for (int k = 0; k < N; ++k) s = fmaf(f[k] * c, f[k] * c, s);
    }
    return s;
  };
  // the places and phases of the tokens [first, first + kBlock) of the CTA's
  auto look_up = [&](int first) {
    const int last = min(first + kBlock, end);
    __syncthreads();
    if (threadIdx.x < kBlock) where[threadIdx.x] = Where{-1, 0, -1};
    __syncthreads();
    for (int s = threadIdx.x; s < p.b.n_seqs; s += threads) {
      int lo, len;
      int64_t kv;
      const bool sound = seq_rows(p.b, s, lo, len) & seq_kv(p.b, p.pool.bs, p.pool.H, s, 0, kv);
      if (!sound) continue;
      for (int t = max(lo, first); t < min(lo + len, last); ++t) where[t - first] = Where{kv - len + (t - lo), 0, s};
    }
    __syncthreads();
    for (int i = threadIdx.x; i < (last - first) * half; i += threads) {
      const int t = i / half, pair = i - t * half, axis = (pair >= n.first[1]) + (pair >= n.first[2]);
      const int32_t phase =
          p.positions ? p.positions[axis * (int64_t)p.b.total_q + first + t] : (int32_t)where[t].off;
      const float2 r =
          turn_at(phase, p.turns[pair], axis == 0 ? n.amplitude[0] : axis == 1 ? n.amplitude[1] : n.amplitude[2]);
      if constexpr (PAIRS == kInterleaved) {
        *reinterpret_cast<float2*>(&cs[t][place<N, 128>(2 * pair)]) = r;
      } else {
        cs[t][place<N, 64>(pair)] = r.x;
        cs[t][64 + place<N, 64>(pair)] = r.y;
      }
    }
    Where w{-1, 0, -1};
    if (threadIdx.x < last - first) {
      w = where[threadIdx.x];
      const int64_t c = w.off;
      w.off = -1;
      if (w.seq >= 0 && c >= 0) {
        const int64_t page = c / p.pool.bs;
        const int64_t blk = p.b.tables[w.seq * p.b.table_stride + page];
        if (blk >= 0 && blk < p.pool.n_blocks)
          w.off = blk * p.pool.s_block + (c - page * p.pool.bs) * p.pool.s_row;
        else
          set_status(p.b.status, DCP_EDEVICE);
      }
    }
    __syncthreads();
    if (threadIdx.x < last - first) where[threadIdx.x] = w;
    __syncthreads();
  };
  // a unit of a q or k head: norm, weights (of the head whose first element is number `at`), turn by `t`
  auto turn = [&](const uint4 (&raw)[kTwo], bool real, bool is_q, const Norm& f, int at, const float* t, char* to) {
    if constexpr (PAIRS == kHalfAny) {  // a head's lanes are in one warp
      __syncwarp();
      rows[threadIdx.x] = raw[0];
      __syncwarp();
    }
    if (!real) return;
    const char* weight = is_q ? n.q_weight : n.k_weight;
    uint64_t a[kTwo][N / 2];
    const uint64_t r2 = pair(f.r, f.r);
#pragma unroll
    for (int j = 0; j < kTwo; ++j) {
      if (j && !two) continue;
      pairs_of<T, N>(raw[j], a[j]);
      if (f.up != 1.f) {
#pragma unroll
        for (int k = 0; k < N / 2; ++k) a[j][k] = mul2(a[j][k], pair(f.up, f.up));
      }
#pragma unroll
      for (int k = 0; k < N / 2; ++k) a[j][k] = mul2(a[j][k], r2);
      const int d = (vec + j * pair_vecs) * N;
      if constexpr (WEIGHTS) {
        weigh<N>(n, weight, at + d, a[j]);
      } else {
#pragma unroll
        for (int k = 0; k < N / 2; k += 2) {
          const float4 w = *reinterpret_cast<const float4*>(&ws[!is_q][place<N, 128>(d + 2 * k)]);
          a[j][k] = mul2(a[j][k], pair(w.x, w.y));
          a[j][k + 1] = mul2(a[j][k + 1], pair(w.z, w.w));
        }
      }
    }
    if constexpr (PAIRS == kHalfVec) {
      if (two) {
#pragma unroll
        for (int k = 0; k < N / 2; k += 2) {
          const float4 c = *reinterpret_cast<const float4*>(&t[place<N, 64>(e * N + 2 * k)]);
          const float4 s = *reinterpret_cast<const float4*>(&t[64 + place<N, 64>(e * N + 2 * k)]);
          const uint64_t c2[2] = {pair(c.x, c.y), pair(c.z, c.w)}, s2[2] = {pair(s.x, s.y), pair(s.z, s.w)};
          const uint64_t minus[2] = {pair(-s.x, -s.y), pair(-s.z, -s.w)};
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const uint64_t x0 = a[0][k + u], x1 = a[1][k + u];
            a[0][k + u] = fma2(x0, c2[u], mul2(x1, minus[u]));
            a[1][k + u] = fma2(x1, c2[u], mul2(x0, s2[u]));
          }
        }
        put(to, vector_of<T, N>(a[1]), 1);
      }
    } else if constexpr (PAIRS == kInterleaved) {
      if (vec * N < 2 * half) {
#pragma unroll
        for (int k = 0; k < N / 2; k += 2) {
          const float4 r = *reinterpret_cast<const float4*>(&t[place<N, 128>(vec * N + 2 * k)]);
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            if (vec * N + 2 * (k + u) >= 2 * half) continue;
            const float c = u ? r.z : r.x, s = u ? r.w : r.y;
            float x0, x1;
            unpair(a[0][k + u], x0, x1);
            a[0][k + u] = pair(x0 * c - x1 * s, x0 * s + x1 * c);
          }
        }
      }
    } else if (vec * N < 2 * half) {
      const uint4* row = rows + threadIdx.x - e;
      float y[N];
#pragma unroll
      for (int k = 0; k < N / 2; ++k) unpair(a[0][k], y[2 * k], y[2 * k + 1]);
#pragma unroll
      for (int k = 0; k < N; ++k) {
        const int d = vec * N + k;
        if (d >= 2 * half) continue;
        const int o = d < half ? d + half : d - half;
        float b = E::one(row, o) * f.up * f.r;
        if constexpr (!WEIGHTS)
          b *= ws[!is_q][place<N, 128>(o)];
        else if (weight)
          b *= n.weight_bf16 ? __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(weight)[at + o])
                             : reinterpret_cast<const float*>(weight)[at + o];
        const int at_pair = place<N, 64>(d < half ? d : o);
        const float c = t[at_pair], s = t[64 + at_pair];
        y[k] = d < half ? y[k] * c - b * s : y[k] * c + b * s;
      }
#pragma unroll
      for (int k = 0; k < N / 2; ++k) a[0][k] = pair(y[2 * k], y[2 * k + 1]);
    }
    put(to, vector_of<T, N>(a[0]), 0);
  };
  // the norm of the head whose units this warp's lanes hold
  auto norm_of_head = [&](const uint4 (&a)[kTwo]) {
    auto of_head = [&](float s) {
      for (int o = 1 << n.lanes_log2 >> 1; o; o >>= 1) s += __shfl_xor_sync(~0u, s, o);
      return s;
    };
    float s = of_head(squares(a));
    const float c = rescale(s, n.inv_head, n.eps);
    if (__any_sync(~0u, c != 1.f)) s = of_head(scaled_squares(a, c));
    return norm_of(s, n.inv_head, n.eps, c);
  };

  allow_dependents();
  wait_for_predecessor();
  uint4 x[kHeads][kTwo], v[kValues][kTwo];
  auto load = [&](int j, bool real) {
    const int h = h0 + j * step;
    fetch(x[j], (h < p.Hq ? q_src : k_src) + j * next_head, real && there && h < turned);
  };
  auto load_value = [&](int j, bool real) {
    fetch(v[j], v_src + j * next_head, real && there && h0 + j * step < p.pool.H);
  };
#pragma unroll
  for (int j = 0; j < kHeads; ++j) load(j, true);
#pragma unroll
  for (int j = 0; j < kValues; ++j) load_value(j, true);
  if constexpr (!WEIGHTS) {
    for (int i = threadIdx.x; i < 2 * D; i += threads) {
      const int k = i >= D, d = i - k * D;
      const char* w = k ? n.k_weight : n.q_weight;
      ws[k][place<N, 128>(d)] =
          !w ? 1.f : n.weight_bf16 ? __bfloat162float(((const __nv_bfloat16*)w)[d]) : ((const float*)w)[d];
    }
  }

  for (int tok = begin; tok < end; ++tok) {
    const int i = (tok - begin) % kBlock;
    if (i == 0) look_up(tok);
    const Where w = where[i];
    Norm whole[2];  // of q and k, where the heads share one
    if constexpr (TOKEN) {
      float c[2] = {1.f, 1.f};
#pragma unroll 1
      for (int again = 0; again < 2; ++again) {
        float s[2] = {0.f, 0.f};
        auto add = [&](int h, const uint4 (&a)[kTwo]) {
          const float t = !again ? squares(a) : scaled_squares(a, h < p.Hq ? c[0] : c[1]);
          if (h < p.Hq)
            s[0] += t;
          else
            s[1] += t;  // past the last head: zeros
        };
#pragma unroll
        for (int j = 0; j < kHeads; ++j) add(h0 + j * step, x[j]);
        for (int j = kHeads; h0 + j * step < turned; ++j) {
          uint4 a[kTwo];
          fetch(a, (h0 + j * step < p.Hq ? q_src : k_src) + (int64_t)j * next_head, there);
          add(h0 + j * step, a);
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) {
          s[0] += __shfl_xor_sync(~0u, s[0], o);
          s[1] += __shfl_xor_sync(~0u, s[1], o);
        }
        float2* const to = sums[again ? 2 : tok & 1];  // in turns: a barrier a token is enough
        if ((threadIdx.x & 31) == 0) to[threadIdx.x >> 5] = make_float2(s[0], s[1]);
        __syncthreads();
        const int lane = threadIdx.x & 31;
        const float2 other = lane < threads >> 5 ? to[lane] : make_float2(0.f, 0.f);
        s[0] = other.x;
        s[1] = other.y;
        float scale[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
#pragma unroll
          for (int o = kWarps / 2; o; o >>= 1) s[k] += __shfl_xor_sync(~0u, s[k], o);
          s[k] = __shfl_sync(~0u, s[k], 0);
          const float inv = k ? n.inv_k : n.inv_q;
          scale[k] = k == 0 && p.Hq == 0 ? 1.f : rescale(s[k], inv, n.eps);
          whole[k] = norm_of(s[k], inv, n.eps, c[k]);
        }
        if (again || (scale[0] == 1.f && scale[1] == 1.f)) break;  // the same in every thread
        c[0] = scale[0];
        c[1] = scale[1];
      }
    }
    auto unit = [&](int j, const uint4 (&a)[kTwo]) {
      const int h = h0 + j * step;
      const bool is_q = h < p.Hq;
      Norm f;
      if constexpr (TOKEN)
        f = is_q ? whole[0] : whole[1];
      else
        f = norm_of_head(a);
      char* const to = is_q ? q_dst + (int64_t)j * next_head : k_dst + w.off * kEs + j * next_page_head;
      turn(a, there && h < turned && (is_q ? w.seq >= 0 : w.off >= 0), is_q, f, (is_q ? h : h - p.Hq) * D, cs[i], to);
    };
    auto value = [&](int j, const uint4 (&a)[kTwo]) {
      if (!there || h0 + j * step >= p.pool.H || w.off < 0) return;
      char* const to = v_dst + w.off * kEs + j * next_page_head;
      put(to, a[0], 0);
      if constexpr (kTwo == 2)
        if (two) put(to, a[1], 1);
    };
    // heads past the registers first: the next token is loaded where this one's units were
    for (int j = kHeads; j * step < turned; ++j) {
      uint4 a[kTwo];
      fetch(a, (h0 + j * step < p.Hq ? q_src : k_src) + (int64_t)j * next_head, there && h0 + j * step < turned);
      unit(j, a);
    }
    for (int j = kValues; h0 + j * step < p.pool.H; ++j) {
      uint4 a[kTwo];
      fetch(a, v_src + (int64_t)j * next_head, there);
      value(j, a);
    }
    q_src += p.q_stride * kEs;
    k_src += p.kv_stride * kEs;
    v_src += p.kv_stride * kEs;
#pragma unroll
    for (int j = 0; j < kValues; ++j) {
      value(j, v[j]);
      load_value(j, tok + 1 < end);
    }
#pragma unroll
    for (int j = 0; j < kHeads; ++j) {
      unit(j, x[j]);
      load(j, tok + 1 < end);
    }
    q_dst += (int64_t)p.Hq * D * kEs;
  }
}

template <typename T, int PAIRS, bool TOKEN, bool WEIGHTS>
cudaError_t launch(const NormParams& n, cudaStream_t s) {
  // No more threads than hold a token's q and k heads in kUnits vectors each: so many tokens are in flight on an SM.
  const int turned = n.a.Hq + n.a.pool.H, lanes = 1 << n.lanes_log2, each = kUnits / (PAIRS == kHalfVec ? 2 : 1);
  const int threads = (int)std::max<int64_t>(64, std::min<int64_t>(kNormThreads, ((int64_t)(turned + each - 1) / each * lanes + 31) / 32 * 32));
  const int64_t room = (int64_t)(kNormResident / threads) * sm_count();
  return launch_behind(norm_kernel<T, PAIRS, TOKEN, WEIGHTS>, dim3((unsigned)std::min<int64_t>(n.a.b.total_q, room)),
                       threads, 0, s, n);
}

template <typename T, int PAIRS>
cudaError_t launch_span(NormParams& n, cudaStream_t s) {
  const int units = n.a.pool.D / Elems<T>::kN - (PAIRS == kHalfVec ? n.a.half / Elems<T>::kN : 0);
  n.lanes_log2 = 0;
  while (1 << n.lanes_log2 < units) ++n.lanes_log2;
  const bool weights = n.weight_heads && (n.q_weight || n.k_weight);
  if (n.token_span) return weights ? launch<T, PAIRS, true, true>(n, s) : launch<T, PAIRS, true, false>(n, s);
  return weights ? launch<T, PAIRS, false, true>(n, s) : launch<T, PAIRS, false, false>(n, s);
}

template <typename T>
cudaError_t launch_pairs(NormParams& n, cudaStream_t s) {
  if (!n.a.half_layout) return launch_span<T, kInterleaved>(n, s);
  if (n.a.half % Elems<T>::kN == 0) return launch_span<T, kHalfVec>(n, s);
  return launch_span<T, kHalfAny>(n, s);
}

}  // namespace

cudaError_t launch_norm_append(const NormParams& p, cudaStream_t s) {
  NormParams n = p;
  return n.a.pool.dtype == DCP_BF16 ? launch_pairs<__nv_bfloat16>(n, s) : launch_pairs<float>(n, s);
}

}  // namespace dcp
