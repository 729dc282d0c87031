// Root-mean-square norms of the new tokens' q and k, their rotary turn by up to three position axes, and k, v into the
// cache's pages, in one pass over the data.
//
//   y = x / sqrt(mean x^2 + eps) * w,  then each pair (a, b) of axis a turns by position[a] * theta: one rounding at the end
//
// The mean goes over a head, or over all heads of a token (q and k apart).  A CTA takes a few tokens at a time: their rows
// travel to shared memory while it looks up their places and builds their cos/sin, the sums are taken from there, and what
// is written is computed from there again, so that the data cross HBM once and nothing has to stay in registers in
// between.  A head is a power of two of neighbouring lanes, two 16-byte vectors each, so its sum is a few shuffles; a warp
// takes a few heads of one kind at a time.  A token that does not fit shared memory goes through it in pieces, twice where
// the mean is the token's.
//
// Squares leave fp32 for values past 2^60 or below 2^-50 with an eps as small: such a sum is taken again of values scaled
// by a power of two, which every norm of the row shares, so that any values give what the formula says.
//
// The bytes would take 57 us for the first case below; what bounds it is the instructions around the arithmetic (59 million
// warp instructions, issued at 57 % of the schedulers' rate).  Measured: 6240 tokens of 40 + 40 + 40 heads of 128 in
// bf16, means of tokens, three axes, fp32 weights of each head 92 us (4.2 TB/s); 5875 tokens of 20 + 4 + 4 fp32 heads of 96
// 43 us; 32 tokens 7.8 us.  Steps, us of these two: a token a CTA, its heads in registers 135 / 51; persistent CTAs with the
// next token's loads in flight 114 / 40; rows through shared memory 116 / 51; two vectors a lane 101 / 52; the head's size a
// constant 91 / 54; several small tokens at a time 90 / 44; three
// CTAs an SM without spills instead of four 92 / 43 (and 1045 tokens of 20 heads of 80 13 instead of 16 us).  In bulk copies
// instead of the threads' 16-byte ones 94 / 43 (fewer instructions, but the weights' loads wait longer).
#include <algorithm>

#include "append.cuh"

namespace dcp {

namespace {

constexpr int kNormThreads = 256;
constexpr int kNormWarps = kNormThreads / 32;
constexpr int kNormCtas = 3;             // of an SM, by registers
constexpr int kSharedOfSm = 228 << 10;  // and by shared memory, of which a CTA takes some for itself
constexpr int kSharedOfCta = 3 << 10;
constexpr int kBlock = 16;              // tokens whose places a CTA looks up at a time
constexpr int kBlockBytes = 40 << 10;   // it takes as many of them at a time as have about this in rows
constexpr int kMostBytes = 64 << 10;    // of a CTA's rows: a larger token goes through in pieces

constexpr float kMostSum = 0x1p120f, kLeastMean = 0x1p-100f;

// The scale at which a sum that left fp32's comfortable range is taken again, 1 where it did not.
__device__ __forceinline__ float rescale(float sum, float inv, float eps) {
  return !(sum <= kMostSum) ? 0x1p-80f : fmaf(sum, inv, eps) < kLeastMean ? 0x1p100f : 1.f;
}
// The factor of a norm, y = x * factor, from a sum that was taken of values times c.  (It is a number for a root mean square
// of 2^-126 and more.)
__device__ __forceinline__ float norm_of(float sum, float inv, float eps, float c) {
  const float m = fmaf(sum, inv, eps * c * c), r = rsqrtf(m);
  const float better = fmaf(0.5f * r, fmaf(-m * r, r, 1.f), r);  // a step of Newton's: 2 ulp to half of one
  return (m > 0.f && m < INFINITY ? better : r) * c;
}

// Where element d of a row of LENGTH lies in shared memory: quads of a vector's elements apart, those of neighbouring
// vectors side by side, so that the lanes' reads of a quad hit no bank twice.
template <int N, int LENGTH>
__device__ __forceinline__ int place(int d) {
  return (d % N / 4 * (LENGTH / N) + d / N) * 4 + d % 4;
}

// Shared memory beside the rows, for each token of a block.
struct Token {
  Where where;
  float2 sums[kNormWarps];                // of squares of q and k, by warp
  float scale[2], factor[2];              // at which they are taken; of the norms where the heads share one
  // cos and sin of the pairs: (c, s) in the places of the pair's elements, or all cosines, then all sines
  __align__(16) float cs[2 * DCP_ROPE_MAX_PAIRS];
};

template <typename T, int PAIRS, bool TOKEN, bool WEIGHTS, bool WIDE>
__global__ void __launch_bounds__(kNormThreads, kNormCtas) norm_kernel(const __grid_constant__ NormParams n) {
  using E = Elems<T>;
  constexpr int N = E::kN, kEs = sizeof(T);
  extern __shared__ __align__(16) uint8_t rows[];          // [token of the block][head of the piece][D]
  __shared__ __align__(16) float ws[WEIGHTS ? 1 : 2][WEIGHTS ? 4 : 128];  // weights that all heads share
  const AppendParams& p = n.a;
  Token* const tokens = reinterpret_cast<Token*>(rows + n.rows_bytes);
  constexpr int kVecs = 16;                                // of a head, where WIDE
  const int D = WIDE ? kVecs * N : p.pool.D, half = p.half, turned = p.Hq + p.pool.H, heads = turned + p.pool.H;
  // A lane has two vectors of a head, as far apart as the pairs where that is a whole number of vectors, else half a head
  // apart, so that neighbouring lanes' vectors are neighbours; those left over are one lane's each.
  const int pair_vecs = WIDE ? kVecs / 2 : PAIRS == kHalfVec ? half / N : D / N / 2, per_head = D / N - pair_vecs, row_bytes = D * kEs;
  const int lane = threadIdx.x & 31, warp = __shfl_sync(~0u, threadIdx.x >> 5, 0);
  const int lanes_log2 = WIDE ? 3 : n.lanes_log2, e = lane & ((1 << lanes_log2) - 1), h0 = lane >> lanes_log2;
  const int step = 32 >> lanes_log2;                       // heads that a warp has at a time
  const bool there = WIDE || e < per_head, two = WIDE || e < pair_vecs;
  const int vec = two ? e : e + pair_vecs;                 // the unit's (first) vector
  const int begin = (int)((int64_t)p.b.total_q * blockIdx.x / gridDim.x);  // the CTA's tokens
  const int end = (int)((int64_t)p.b.total_q * (blockIdx.x + 1) / gridDim.x);

  auto unit_at = [&](const uint8_t* row, uint4 (&to)[2]) {
    to[0] = reinterpret_cast<const uint4*>(row)[vec];
    to[1] = two ? reinterpret_cast<const uint4*>(row)[vec + pair_vecs] : make_uint4(0, 0, 0, 0);
  };
  auto squares = [&](const uint4 (&a)[2]) {
    float s[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float f[N];
      E::get(a[i], f);
#pragma unroll
      for (int k = 0; k < N; ++k) s[k & 1] = fmaf(f[k], f[k], s[k & 1]);
    }
    return s[0] + s[1];
  };
  auto scaled_squares = [&](const uint4 (&a)[2], float c) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float f[N];
      E::get(a[i], f);
#pragma unroll
      for (int k = 0; k < N; ++k) s = fmaf(f[k] * c, f[k] * c, s);
    }
    return s;
  };
  // heads [h, h + count) of tokens [first, last) on their way to shared memory
  auto load = [&](int first, int last, int h, int count) {
    const uint32_t to = smem_u32(rows);
    for (int t = first; t < last; ++t) {
      auto copy = [&](const char* from, int lo, int hi) {  // heads lo .. hi - 1 of all, head lo at `from`
        const int a = max(lo, h), b = min(hi, h + count);
        const char* src = from + (a - lo) * row_bytes + threadIdx.x * 16;
        uint32_t dst = to + ((t - first) * count + a - h) * row_bytes + threadIdx.x * 16;
#pragma unroll 1
        for (int left = (b - a) * row_bytes - (int)threadIdx.x * 16; left > 0; left -= kNormThreads * 16) {
          cp_async16(dst, src);
          dst += kNormThreads * 16;
          src += kNormThreads * 16;
        }
      };
      copy(p.q + t * p.q_stride * kEs, 0, p.Hq);
      copy(p.k + t * p.kv_stride * kEs, p.Hq, turned);
      copy(p.v + t * p.kv_stride * kEs, turned, heads);
    }
    cp_async_commit();
  };
  // the places and phases of tokens [first, last)
  auto look_up = [&](int first, int last) {
    if (threadIdx.x < last - first) {
      tokens[threadIdx.x].where = Where{-1, 0, -1};
      tokens[threadIdx.x].scale[0] = tokens[threadIdx.x].scale[1] = 1.f;
    }
    __syncthreads();
    for (int s = threadIdx.x; s < p.b.n_seqs; s += kNormThreads) {
      int lo, len;
      int64_t kv;
      const bool sound = seq_rows(p.b, s, lo, len) & seq_kv(p.b, p.pool.bs, p.pool.H, s, 0, kv);
      if (!sound) continue;
      for (int t = max(lo, first); t < min(lo + len, last); ++t)
        tokens[t - first].where = Where{kv - len + (t - lo), 0, s};
    }
    __syncthreads();
    for (int i = threadIdx.x; i < (last - first) * half; i += kNormThreads) {
      const int t = i / half, pair = i - t * half, axis = (pair >= n.first[1]) + (pair >= n.first[2]);
      const int32_t phase =
          p.positions ? p.positions[axis * (int64_t)p.b.total_q + first + t] : (int32_t)tokens[t].where.off;
      const float2 r =
          turn_at(phase, p.turns[pair], axis == 0 ? n.amplitude[0] : axis == 1 ? n.amplitude[1] : n.amplitude[2]);
      float* const cs = tokens[t].cs;
      if constexpr (PAIRS == kInterleaved) {
        *reinterpret_cast<float2*>(&cs[place<N, 128>(2 * pair)]) = r;
      } else {
        cs[place<N, 64>(pair)] = r.x;
        cs[64 + place<N, 64>(pair)] = r.y;
      }
    }
    Where w{-1, 0, -1};
    if (threadIdx.x < last - first) {
      w = tokens[threadIdx.x].where;
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
    if (threadIdx.x < last - first) tokens[threadIdx.x].where = w;
  };
  // Heads [h, h + count) of all: those that are heads lo .. hi - 1, from the first of these on.
  struct Part {
    int first, heads, rounds;  // rounds of a warp
  };
  auto part = [&](int h, int count, int lo, int hi) {
    const int first = max(lo, h), some = max(0, min(hi, h + count) - first);
    return Part{first - lo, some, (some + step - 1) / step};
  };
  // each warp's share of the sums of a token's q and k heads [h, h + count), which lie at `row`
  auto add_squares = [&](Token& tk, const uint8_t* row, int h, int count, bool more, bool scaled) {
    float s[2];
#pragma unroll
    for (int which = 0; which < 2; ++which) {
      const Part now = part(h, count, which ? p.Hq : 0, which ? turned : p.Hq);
      const uint8_t* at = row + (now.first + (which ? p.Hq : 0) - h + warp * step + h0) * row_bytes;
      s[which] = 0.f;
      for (int k = warp * step + h0; k < now.heads; k += kNormWarps * step, at += kNormWarps * step * row_bytes) {
        if (!there) continue;
        uint4 x[2];
        unit_at(at, x);
        s[which] += scaled ? scaled_squares(x, tk.scale[which]) : squares(x);
      }
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      s[0] += __shfl_xor_sync(~0u, s[0], o);
      s[1] += __shfl_xor_sync(~0u, s[1], o);
    }
    if (lane == 0) {
      float2& to = tk.sums[warp];
      to = more ? make_float2(to.x + s[0], to.y + s[1]) : make_float2(s[0], s[1]);
    }
  };
  // the factors of tokens [place, place + n_tokens) of the block; true where a sum has to be taken again, at another scale
  auto make_factors = [&](int place, int n_tokens, bool last_time) {
    __syncthreads();
    bool again = false;
    if (threadIdx.x < 2 * n_tokens) {
      Token& tk = tokens[place + (threadIdx.x >> 1)];
      const int k = threadIdx.x & 1;
      float s = 0.f;
#pragma unroll
      for (int w = 0; w < kNormWarps; ++w) s += k ? tk.sums[w].y : tk.sums[w].x;
      const float inv = k ? n.inv_k : n.inv_q;
      tk.factor[k] = norm_of(s, inv, n.eps, tk.scale[k]);
      if (!last_time && (k || p.Hq)) {
        tk.scale[k] = rescale(s, inv, n.eps);
        again = tk.scale[k] != 1.f;
      }
    }
    return __syncthreads_or(again);
  };
  // weights of a vector's elements, the first of which is element d of a head, and of one element; `own` is where the
  // head's own weights begin, where each has its own (null: ones)
  auto weights_at = [&](bool is_q, const char* own, uint32_t d, float (&g)[N]) {
    if constexpr (!WEIGHTS) {
#pragma unroll
      for (int u = 0; u < N; u += 4) {
        const float4 w = *reinterpret_cast<const float4*>(&ws[!is_q][place<N, 128>(d + u)]);
        g[u] = w.x, g[u + 1] = w.y, g[u + 2] = w.z, g[u + 3] = w.w;
      }
    } else if (!own) {
#pragma unroll
      for (int u = 0; u < N; ++u) g[u] = 1.f;
    } else if (n.weight_bf16) {
#pragma unroll
      for (int u = 0; u < N; u += 4) {
        const uint2 w = __ldg(reinterpret_cast<const uint2*>(own + 2 * d) + u / 4);
        g[u] = bf16lo(w.x), g[u + 1] = bf16hi(w.x), g[u + 2] = bf16lo(w.y), g[u + 3] = bf16hi(w.y);
      }
    } else {
#pragma unroll
      for (int u = 0; u < N; u += 4) {
        const float4 w = __ldg(reinterpret_cast<const float4*>(own + 4 * d) + u / 4);
        g[u] = w.x, g[u + 1] = w.y, g[u + 2] = w.z, g[u + 3] = w.w;
      }
    }
  };
  auto weight_at = [&](bool is_q, const char* own, int d) {
    if constexpr (!WEIGHTS) return ws[!is_q][place<N, 128>(d)];
    return !own ? 1.f : n.weight_bf16 ? __bfloat162float(((const __nv_bfloat16*)own)[d]) : ((const float*)own)[d];
  };
  // a unit: norm, weights, turn
  auto put = [&](const bool is_q, const uint4 (&x)[2], float f, const float* cs, const uint8_t* at, const char* own,
                 uint4* to) {
    float a[2][N];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      E::get(x[j], a[j]);
      float g[N];
      weights_at(is_q, own, (j && !two ? vec : vec + j * pair_vecs) * N, g);
#pragma unroll
      for (int u = 0; u < N; ++u) a[j][u] *= f * g[u];
    }
    if constexpr (PAIRS == kHalfVec) {
      if (two) {
#pragma unroll
        for (int q4 = 0; q4 < N; q4 += 4) {
          const float4 c4 = *reinterpret_cast<const float4*>(&cs[place<N, 64>(e * N + q4)]);
          const float4 s4 = *reinterpret_cast<const float4*>(&cs[64 + place<N, 64>(e * N + q4)]);
          const float c[4] = {c4.x, c4.y, c4.z, c4.w}, s[4] = {s4.x, s4.y, s4.z, s4.w};
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const float x0 = a[0][q4 + u], x1 = a[1][q4 + u];
            a[0][q4 + u] = x0 * c[u] - x1 * s[u];
            a[1][q4 + u] = x0 * s[u] + x1 * c[u];
          }
        }
      }
    } else {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int d0 = (vec + j * pair_vecs) * N;
        if (d0 >= 2 * half) continue;
        const bool whole = 2 * half % N == 0;  // no vector is turned in part
        if constexpr (PAIRS == kInterleaved) {
#pragma unroll
          for (int u = 0; u < N; u += 4) {
            const float4 r = *reinterpret_cast<const float4*>(&cs[place<N, 128>(d0 + u)]);
            const float x0 = a[j][u], x1 = a[j][u + 1], x2 = a[j][u + 2], x3 = a[j][u + 3];
            a[j][u] = x0 * r.x - x1 * r.y, a[j][u + 1] = x0 * r.y + x1 * r.x;
            a[j][u + 2] = x2 * r.z - x3 * r.w, a[j][u + 3] = x2 * r.w + x3 * r.z;
            if (whole) continue;
            if (d0 + u >= 2 * half) a[j][u] = x0, a[j][u + 1] = x1;
            if (d0 + u + 2 >= 2 * half) a[j][u + 2] = x2, a[j][u + 3] = x3;
          }
        } else {
#pragma unroll
          for (int u = 0; u < N; ++u) {
            const int d = d0 + u;
            if (d >= 2 * half) continue;
            const int o = d < half ? d + half : d - half;
            const float b = E::one(reinterpret_cast<const uint4*>(at), o) * (f * weight_at(is_q, own, o));
            const int at_pair = place<N, 64>(d < half ? d : o);
            const float c = cs[at_pair], s = cs[64 + at_pair];
            a[j][u] = d < half ? a[j][u] * c - b * s : a[j][u] * c + b * s;
          }
        }
      }
    }
    if (two) to[vec + pair_vecs] = E::put(a[1]);
    to[vec] = E::put(a[0]);
  };
  // Heads [h, h + count) of n_tokens tokens: norm, weights, turn; values as they are.  A warp takes a few heads at a time,
  // and its next ones kNormWarps further; who begins goes round, from kind to kind and token to token.
  const char* const q_weight = WEIGHTS && n.q_weight ? n.q_weight + h0 * D * n.weight_bytes : nullptr;
  const char* const k_weight = WEIGHTS && n.k_weight ? n.k_weight + h0 * D * n.weight_bytes : nullptr;
  auto finish = [&](int first, int place, int n_tokens, int h, int count) {
    const Part qs = part(h, count, 0, p.Hq), ks = part(h, count, p.Hq, turned), vs = part(h, count, turned, heads);
    const uint8_t* row = rows + h0 * row_bytes;
    int turn_of = warp;  // rounds before this warp's first of a kind
    auto next_kind = [&](int rounds) { turn_of = (turn_of - rounds) & (kNormWarps - 1); };
    auto heads_of = [&](const bool is_q, const Part& now, const Token& tk, const uint8_t* at, char* to, int64_t next,
                        bool wanted) {
      const char* own = is_q ? q_weight : k_weight;
      if constexpr (WEIGHTS)
        if (own) own += (now.first + turn_of * step) * D * n.weight_bytes;
      at += turn_of * step * row_bytes;
      to += (now.first + turn_of * step + h0) * next;
      float f;
      if constexpr (TOKEN) f = tk.factor[!is_q];
      for (int r = turn_of; r < now.rounds; r += kNormWarps) {
        const bool real = there && r * step + h0 < now.heads;
        uint4 x[2] = {};
        if (real) unit_at(at, x);
        if constexpr (!TOKEN) {
          auto of_head = [&](float s) {
            for (int o = 1 << lanes_log2 >> 1; o; o >>= 1) s += __shfl_xor_sync(~0u, s, o);
            return s;
          };
          float s = of_head(squares(x));
          const float c = rescale(s, n.inv_head, n.eps);
          if (__any_sync(~0u, c != 1.f)) s = of_head(scaled_squares(x, c));
          f = norm_of(s, n.inv_head, n.eps, c);
        }
        if (real && wanted) put(is_q, x, f, tk.cs, at, own, reinterpret_cast<uint4*>(to));
        at += kNormWarps * step * row_bytes;
        to += kNormWarps * step * next;
        if constexpr (WEIGHTS)
          if (own) own += kNormWarps * step * D * n.weight_bytes;
      }
      next_kind(now.rounds);
    };
    const int64_t page_head = p.pool.s_head * kEs;
    for (int t = 0; t < n_tokens; ++t, row += count * row_bytes) {
      const Token& tk = tokens[place + t];
      const Where w = tk.where;
      heads_of(true, qs, tk, row, p.q_out + (first + t) * (int64_t)p.Hq * row_bytes, row_bytes, w.seq >= 0);
      heads_of(false, ks, tk, row + qs.heads * row_bytes, p.pool.k + w.off * kEs, page_head, w.off >= 0);
      const uint8_t* at = row + (qs.heads + ks.heads + turn_of * step) * row_bytes;
      char* to = p.pool.v + w.off * kEs + (vs.first + turn_of * step + h0) * page_head;
      for (int r = turn_of; r < vs.rounds; r += kNormWarps) {
        if (there && r * step + h0 < vs.heads && w.off >= 0) {
          uint4 x[2];
          unit_at(at, x);
          reinterpret_cast<uint4*>(to)[vec] = x[0];
          if (two) reinterpret_cast<uint4*>(to)[vec + pair_vecs] = x[1];
        }
        at += kNormWarps * step * row_bytes;
        to += kNormWarps * step * page_head;
      }
      next_kind(vs.rounds);
    }
  };

  allow_dependents();
  wait_for_predecessor();
  load(begin, min(begin + n.tokens, end), 0, n.heads);
  if constexpr (!WEIGHTS) {
    for (int i = threadIdx.x; i < 2 * D; i += kNormThreads) {
      const int k = i >= D, d = i - k * D;
      const char* w = k ? n.k_weight : n.q_weight;
      ws[k][place<N, 128>(d)] =
          !w ? 1.f : n.weight_bf16 ? __bfloat162float(((const __nv_bfloat16*)w)[d]) : ((const float*)w)[d];
    }
  }
  int held = 0;  // first head of the piece that is in shared memory or on its way
  for (int first = begin; first < end; first += n.tokens) {
    const int last = min(first + n.tokens, end), place0 = (first - begin) % n.block;  // among the tokens looked up
    auto have = [&](int h) {  // heads from h on
      if (held != h) {
        __syncthreads();
        load(first, last, h, min(n.heads, heads - h));
        held = h;
      }
      cp_async_wait<0>();
      __syncthreads();
    };
    if (place0 == 0) look_up(first, min(first + n.block, end));
    if constexpr (TOKEN) {
      auto add = [&](bool scaled) {
        for (int h = 0; h < turned; h += n.heads) {
          const int count = min(n.heads, heads - h);
          have(h);
          for (int t = first; t < last; ++t)
            add_squares(tokens[place0 + t - first], rows + (t - first) * count * row_bytes, h, count, h > 0, scaled);
        }
      };
      add(false);
      if (make_factors(place0, last - first, false)) {
        add(true);
        make_factors(place0, last - first, true);
      }
    }
    for (int h = 0; h < heads; h += n.heads) {
      const int count = min(n.heads, heads - h);
      have(h);
      finish(first, place0, last - first, h, count);
    }
    if (last == end) break;
    __syncthreads();
    load(last, min(last + n.tokens, end), 0, n.heads);
    held = 0;
  }
}

template <typename T, int PAIRS, bool TOKEN, bool WEIGHTS, bool WIDE>
cudaError_t launch(NormParams& n, cudaStream_t s) {
  static LaunchCache lc;
  // A block's tokens, and their places behind the rows.
  const int heads = n.a.Hq + 2 * n.a.pool.H, row = n.a.pool.D * (int)sizeof(T);
  n.heads = (int)std::min<int64_t>(heads, kMostBytes / row);
  n.tokens = std::max(1, std::min(kBlock, kBlockBytes / (n.heads * row)));
  // no more than leave every CTA that the SMs hold something to do
  n.tokens = (int)std::min<int64_t>(n.tokens, std::max(1, n.a.b.total_q / (kNormCtas * sm_count())));
  n.rows_bytes = n.tokens * n.heads * row;
  n.block = kBlock / n.tokens * n.tokens;
  const size_t smem = n.rows_bytes + n.block * sizeof(Token);
  int unused;
  const cudaError_t e = launch_setup(lc, norm_kernel<T, PAIRS, TOKEN, WEIGHTS, WIDE>, kNormThreads,
                                     kMostBytes + kBlock * sizeof(Token), &unused);
  if (e != cudaSuccess) return e;
  const int64_t ctas = std::min<int64_t>(kNormCtas, kSharedOfSm / (int64_t)(smem + kSharedOfCta));
  const int64_t room = ctas * sm_count();
  return launch_behind(norm_kernel<T, PAIRS, TOKEN, WEIGHTS, WIDE>, dim3((unsigned)std::min<int64_t>(n.a.b.total_q, room)),
                       kNormThreads, smem, s, n);
}

template <typename T, int PAIRS, bool WIDE>
cudaError_t launch_span(NormParams& n, cudaStream_t s) {
  const bool weights = n.weight_heads && (n.q_weight || n.k_weight);
  if (n.token_span) return weights ? launch<T, PAIRS, true, true, WIDE>(n, s) : launch<T, PAIRS, true, false, WIDE>(n, s);
  return weights ? launch<T, PAIRS, false, true, WIDE>(n, s) : launch<T, PAIRS, false, false, WIDE>(n, s);
}

// Heads of 16 vectors, 8 lanes each, have a kernel to which all that depends on the head's size is a constant.
template <typename T, int PAIRS>
cudaError_t launch_width(NormParams& n, cudaStream_t s) {
  const int vecs = n.a.pool.D / Elems<T>::kN, pairs = PAIRS == kHalfVec ? n.a.half / Elems<T>::kN : vecs / 2;
  n.lanes_log2 = 0;
  while (1 << n.lanes_log2 < vecs - pairs) ++n.lanes_log2;
  return vecs == 16 && pairs == 8 ? launch_span<T, PAIRS, true>(n, s) : launch_span<T, PAIRS, false>(n, s);
}

template <typename T>
cudaError_t launch_pairs(NormParams& n, cudaStream_t s) {
  if (!n.a.half_layout) return launch_width<T, kInterleaved>(n, s);
  if (n.a.half % Elems<T>::kN == 0) return launch_width<T, kHalfVec>(n, s);
  return launch_width<T, kHalfAny>(n, s);
}

}  // namespace

cudaError_t launch_norm_append(const NormParams& p, cudaStream_t s) {
  NormParams n = p;
  return n.a.pool.dtype == DCP_BF16 ? launch_pairs<__nv_bfloat16>(n, s) : launch_pairs<float>(n, s);
}

}  // namespace dcp
