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
#include "append.cuh"

namespace dcp {

namespace {

constexpr int kNormThreads = 256;

// The factors of a norm: y = (x * up) * r.
struct Norm {
  float up, r;
};
constexpr float kMostSum = 0x1p120f, kLeastMean = 0x1p-100f;

// The scale at which a sum that left fp32's comfortable range is taken again, 1 where it did not.
__device__ __forceinline__ float rescale(float sum, float count, float eps) {
  if (!(sum <= kMostSum)) return 0x1p-80f;
  return sum / count + eps < kLeastMean ? 0x1p100f : 1.f;
}
__device__ __forceinline__ Norm norm_of(float sum, float count, float eps, float c) {
  return Norm{fmaxf(c, 1.f), __frsqrt_rn(sum / count + eps * c * c) * fminf(c, 1.f)};
}

template <typename T, int PAIRS, bool TOKEN>
__global__ void __launch_bounds__(kNormThreads) norm_kernel(const __grid_constant__ NormParams n) {
  using E = Elems<T>;
  constexpr int N = E::kN;
  constexpr int kUnits = PAIRS == kHalfVec ? 4 : 8;  // units (one or two vectors) of as many heads a thread holds
  constexpr int kWarps = kNormThreads / 32;
  __shared__ Where where;
  __shared__ float2 cs[DCP_ROPE_MAX_PAIRS];
  __shared__ float sums[2][kWarps][2];
  __shared__ uint4 rows[PAIRS == kHalfAny ? kNormThreads : 1];
  const AppendParams& p = n.a;
  const int64_t tok = blockIdx.x;
  const int D = p.pool.D, half = p.half, turned = p.Hq + p.pool.H, heads = turned + p.pool.H;
  const int pair_vecs = PAIRS == kHalfVec ? half / N : 0;  // units of two vectors in a head
  const int per_head = D / N - pair_vecs;
  const int e = threadIdx.x & ((1 << n.lanes_log2) - 1), step = kNormThreads >> n.lanes_log2;
  const int h0 = threadIdx.x >> n.lanes_log2;
  const bool there = e < per_head, two = PAIRS == kHalfVec && e < pair_vecs;
  const int vec = two ? e : e + pair_vecs;  // the unit's (first) vector

  uint4 x[kUnits], y[PAIRS == kHalfVec ? kUnits : 1];
  auto source = [&](int h) {
    return (const uint4*)(h < p.Hq ? (const T*)p.q + tok * p.q_stride + h * D
                          : h < turned ? (const T*)p.k + tok * p.kv_stride + (h - p.Hq) * D
                                       : (const T*)p.v + tok * p.kv_stride + (h - turned) * D);
  };
  auto load = [&](int first) {
#pragma unroll
    for (int j = 0; j < kUnits; ++j) {
      const int h = first + j * step;
      x[j] = make_uint4(0, 0, 0, 0);
      if constexpr (PAIRS == kHalfVec) y[j] = make_uint4(0, 0, 0, 0);
      if (!there || h >= heads) continue;
      const uint4* src = source(h);
      x[j] = src[vec];
      if constexpr (PAIRS == kHalfVec)
        if (two) y[j] = src[vec + pair_vecs];
    }
  };
  auto squares = [&](const uint4& a, float c) {
    float f[N], s = 0.f;
    E::get(a, f);
#pragma unroll
    for (int k = 0; k < N; ++k) s = fmaf(f[k] * c, f[k] * c, s);
    return s;
  };
  auto unit_squares = [&](int j, float c) {
    float s = squares(x[j], c);
    if constexpr (PAIRS == kHalfVec) s += squares(y[j], c);
    return s;
  };

  allow_dependents();
  wait_for_predecessor();
  load(h0);
  if (threadIdx.x == 0) where.seq = -1;
  __syncthreads();
  find_token<kNormThreads>(p.b, p.pool, tok, where);
  __syncthreads();
  for (int i = threadIdx.x; i < half; i += kNormThreads) {
    const int axis = (i >= n.first[1]) + (i >= n.first[2]);
    cs[i] = turn_at(p.positions ? p.positions[axis * (int64_t)p.b.total_q + tok] : where.phase, p.turns[i],
                    n.amplitude[axis]);
  }
  Norm whole[2];  // of q and k, where the heads share one
  if constexpr (TOKEN) {
    float c[2] = {1.f, 1.f};
#pragma unroll 1
    for (int again = 0; again < 2; ++again) {
      float s[2] = {0.f, 0.f};
#pragma unroll
      for (int j = 0; j < kUnits; ++j) {
        const int h = h0 + j * step;
        if (h < p.Hq)
          s[0] += unit_squares(j, c[0]);
        else if (h < turned)
          s[1] += unit_squares(j, c[1]);
      }
      for (int h = h0 + kUnits * step; h < turned; h += step) {
        if (!there) continue;
        const bool is_q = h < p.Hq;
        const uint4* src = source(h);
        float t = squares(src[vec], is_q ? c[0] : c[1]);
        if (two) t += squares(src[vec + pair_vecs], is_q ? c[0] : c[1]);
        if (is_q)
          s[0] += t;
        else
          s[1] += t;
      }
#pragma unroll
      for (int o = 16; o; o >>= 1) {
        s[0] += __shfl_xor_sync(~0u, s[0], o);
        s[1] += __shfl_xor_sync(~0u, s[1], o);
      }
      if ((threadIdx.x & 31) == 0) {
        sums[again][threadIdx.x >> 5][0] = s[0];
        sums[again][threadIdx.x >> 5][1] = s[1];
      }
      __syncthreads();
      float next[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float count = (float)(i ? p.pool.H : p.Hq) * D;
        s[i] = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) s[i] += sums[again][w][i];
        next[i] = i == 0 && p.Hq == 0 ? 1.f : rescale(s[i], count, n.eps);
        whole[i] = norm_of(s[i], count, n.eps, c[i]);
      }
      if (again || (next[0] == 1.f && next[1] == 1.f)) break;  // the same in every thread
      c[0] = next[0];
      c[1] = next[1];
    }
  } else {
    __syncthreads();
  }
  const Where w = where;
  if (w.seq < 0) return;

  // a vector of a head times its norm and weights
  auto normalise = [&](const uint4& a, const Norm& f, const char* weight, int at, float (&out)[N]) {
    E::get(a, out);
#pragma unroll
    for (int k = 0; k < N; ++k) out[k] = out[k] * f.up * f.r;
    if (!weight) return;
    if (n.weight_bf16) {
      if constexpr (N == 8) {
        float g[8];
        Elems<__nv_bfloat16>::get(*reinterpret_cast<const uint4*>(weight + (int64_t)at * 2), g);
#pragma unroll
        for (int k = 0; k < 8; ++k) out[k] *= g[k];
      } else {
        const uint2 g = *reinterpret_cast<const uint2*>(weight + (int64_t)at * 2);
        out[0] *= bf16lo(g.x), out[1] *= bf16hi(g.x), out[2] *= bf16lo(g.y), out[3] *= bf16hi(g.y);
      }
    } else {
#pragma unroll
      for (int k = 0; k < N; k += 4) {
        const float4 g = *reinterpret_cast<const float4*>(weight + ((int64_t)at + k) * 4);
        out[k] *= g.x, out[k + 1] *= g.y, out[k + 2] *= g.z, out[k + 3] *= g.w;
      }
    }
  };
  const float count = (float)D;
  T* const q_to = (T*)p.q_out + tok * p.Hq * D;
  for (int first = 0; first < heads; first += kUnits * step) {
    if (first) load(first + h0);
#pragma unroll
    for (int j = 0; j < kUnits; ++j) {
      if (first + j * step >= heads) break;  // the same in every thread
      const int h = first + h0 + j * step;
      const bool is_q = h < p.Hq, is_v = h >= turned;
      Norm f;
      if constexpr (TOKEN) {
        f = is_q ? whole[0] : whole[1];
      } else {
        auto sum = [&](float c) {
          float s = unit_squares(j, c);
          for (int o = 1 << n.lanes_log2 >> 1; o; o >>= 1) s += __shfl_xor_sync(~0u, s, o);
          return s;
        };
        float s = sum(1.f), c = rescale(s, count, n.eps);
        if (__any_sync(~0u, c != 1.f)) s = sum(c);
        f = norm_of(s, count, n.eps, c);
      }
      if constexpr (PAIRS == kHalfAny) {  // a head's lanes are in one warp
        __syncwarp();
        rows[threadIdx.x] = x[j];
        __syncwarp();
      }
      if (!there || h >= heads || (!is_q && w.off < 0)) continue;
      uint4* dst = (uint4*)(is_q ? q_to + h * D
                                 : (T*)(is_v ? p.pool.v : p.pool.k) + w.off + (h - (is_v ? turned : p.Hq)) * p.pool.s_head);
      if (is_v) {
        dst[vec] = x[j];
        if constexpr (PAIRS == kHalfVec)
          if (two) dst[vec + pair_vecs] = y[j];
        continue;
      }
      const char* weight = is_q ? n.q_weight : n.k_weight;
      const int at = n.weight_heads ? (is_q ? h : h - p.Hq) * D : 0;
      float a[N];
      normalise(x[j], f, weight, at + vec * N, a);
      if constexpr (PAIRS == kHalfVec) {
        if (two) {
          float b[N];
          normalise(y[j], f, weight, at + (vec + pair_vecs) * N, b);
#pragma unroll
          for (int k = 0; k < N; ++k) {
            const float2 r = cs[e * N + k];
            const float a2 = a[k] * r.x - b[k] * r.y;
            b[k] = a[k] * r.y + b[k] * r.x;
            a[k] = a2;
          }
          dst[vec + pair_vecs] = E::put(b);
        }
      } else if constexpr (PAIRS == kInterleaved) {
        if (vec * N < 2 * half)
#pragma unroll
          for (int k = 0; k < N; k += 2) {
            const int i = vec * (N / 2) + k / 2;
            if (i >= half) continue;
            const float2 r = cs[i];
            const float a2 = a[k] * r.x - a[k + 1] * r.y;
            a[k + 1] = a[k] * r.y + a[k + 1] * r.x;
            a[k] = a2;
          }
      } else if (vec * N < 2 * half) {
        const uint4* row = rows + threadIdx.x - e;
#pragma unroll
        for (int k = 0; k < N; ++k) {
          const int d = vec * N + k;
          if (d >= 2 * half) continue;
          const int o = d < half ? d + half : d - half;
          float b = E::one(row, o) * f.up * f.r;
          if (weight)
            b *= n.weight_bf16 ? __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(weight)[at + o])
                               : reinterpret_cast<const float*>(weight)[at + o];
          const float2 r = cs[d < half ? d : o];
          a[k] = d < half ? a[k] * r.x - b * r.y : a[k] * r.x + b * r.y;
        }
      }
      dst[vec] = E::put(a);
    }
  }
}

template <typename T, int PAIRS>
cudaError_t launch_span(NormParams& n, cudaStream_t s) {
  const int units = n.a.pool.D / Elems<T>::kN - (PAIRS == kHalfVec ? n.a.half / Elems<T>::kN : 0);
  n.lanes_log2 = 0;
  while (1 << n.lanes_log2 < units) ++n.lanes_log2;
  const dim3 grid((unsigned)n.a.b.total_q);
  return n.token_span ? launch_behind(norm_kernel<T, PAIRS, true>, grid, kNormThreads, 0, s, n)
                      : launch_behind(norm_kernel<T, PAIRS, false>, grid, kNormThreads, 0, s, n);
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
