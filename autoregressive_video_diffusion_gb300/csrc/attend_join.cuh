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

// A piece of a group's prefix, and the rows that see it.
struct PrefixPiece {
  GroupRows of;
  int split, splits;            // the piece's number among the group's
};
__device__ __forceinline__ float* prefix_part(const PrefixPlan& pre, int D, int slot, int kh, int tile, int r) {
  return pre.part + ((((int64_t)slot * pre.heads + kh) * pre.tiles + tile) * pre.rows + r) * (kPartHead + D);
}

// The piece of slot `slot`, by a whole warp.  All pieces are at most L tiles long, L (2 at least) as small as the slots
// allow among 31 lengths from their even share up (a lane tries one each; the last, a piece a group, always fits).  A group
// without rows or prefix has none.  (A slot without a piece: len = 0.)  With `note` the groups' slots go to the table.
__device__ __forceinline__ PrefixPiece prefix_piece(const AttendParams& a, const PrefixPlan& pre, int slot, bool note) {
  const int lane = threadIdx.x & 31, n = a.groups.n;
  auto units = [&](int g, GroupRows& of) -> uint32_t {
    if (g >= n || !group_at(a, g, of) || of.len == 0) return 0;
    return ((uint32_t)of.prefix + pre.unit - 1) / pre.unit;
  };
  GroupRows of{};
  const uint32_t mine = units(lane, of);  // of group `lane`: most calls have no more groups than a warp has lanes
  int64_t total = 0;
  uint32_t most = 0;
  for (int g = lane; g < n; g += 32) {
    GroupRows other;
    const uint32_t w = g == lane ? mine : units(g, other);
    total += w;
    most = max(most, w);
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    total += __shfl_xor_sync(~0u, total, o);
    most = max(most, __shfl_xor_sync(~0u, most, o));
  }
  const uint32_t even = (uint32_t)((total + pre.slots - 1) / pre.slots);
  const uint32_t length = lane == 31 ? max(most, 1u) : max(2u, (uint32_t)(even + (uint64_t)even * lane * lane / 64));
  int64_t pieces = 0;
  for (int g0 = 0; g0 < n; g0 += 32) {
    GroupRows other;
    const uint32_t w = g0 ? units(g0 + lane, other) : mine;
    for (int k = 0; k < min(32, n - g0); ++k) pieces += (__shfl_sync(~0u, w, k) + length - 1) / length;
  }
  const bool fits = lane == 31 || (pieces <= pre.slots && (most + length - 1) / length <= (uint32_t)pre.cap);
  const uint32_t chosen = __shfl_sync(~0u, length, __ffs(__ballot_sync(~0u, fits)) - 1);
  PrefixPiece found{};
  int first = 0;  // slots of the groups before
  for (int g0 = 0; g0 < n; g0 += 32) {
    const uint32_t w = g0 ? units(g0 + lane, of) : mine;
    const int count = (int)((w + chosen - 1) / chosen);
    int end = count;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(~0u, end, o);
      if (lane >= o) end += y;
    }
    const int at = first + end - count;
    if (note && g0 + lane < n) pre.table[g0 + lane] = make_int2(at, count);
    const uint32_t hit = __ballot_sync(~0u, slot >= at && slot < at + count);
    if (hit) {
      const int who = __ffs(hit) - 1;
      found.of.g = __shfl_sync(~0u, of.g, who);
      found.of.s = __shfl_sync(~0u, of.s, who);
      found.of.lo = __shfl_sync(~0u, of.lo, who);
      found.of.len = __shfl_sync(~0u, of.len, who);
      found.of.prefix = __shfl_sync(~0u, of.prefix, who);
      found.split = slot - __shfl_sync(~0u, at, who);
      found.splits = __shfl_sync(~0u, count, who);
      if (!note) break;
    }
    first += __shfl_sync(~0u, end, 31);
  }
  return found;
}

// Joins `splits` parts of `rows` rows whose first is row `row0` of (token, head of the KV
// head) rows, sequence start lo.  Called by a whole CTA; scratch: `room` bytes of shared memory, at least
// join_scratch(rows, splits).  Everything is fetched at once where it fits the scratch (a loop over the parts in global
// memory pays a memory latency every few of them: 5 us for 12 parts of 5 rows, 1 us this way), else the maxima and sums
// first and the values with several loads in flight.
// parts.row(k, r): part k's row r.
__host__ __device__ constexpr int64_t join_scratch(int rows, int splits) {
  return (int64_t)rows * (2 * splits + 1) * 4;
}

// The parts of a row's own keys: the first is at `part0`, the others from `part1` on, `step` floats apart.
struct OwnParts {
  const float* part0;
  const float* part1;
  int64_t step;
  int width;
  __device__ __forceinline__ const float* part(int k) const { return k ? part1 + (k - 1) * step : part0; }
  __device__ __forceinline__ const float* row(int k, int r) const { return part(k) + (int64_t)r * width; }
  static constexpr bool kByRow = false;  // a part's rows lie one behind the other
};

// The parts' maxima and sums into join_rows' scratch.
template <typename Parts, typename Get>
__device__ __forceinline__ void join_heads(const Parts& parts, int splits, int rows, float* weight, Get get) {
  float* const sum = weight + rows * splits;
  for (int u = threadIdx.x; u < rows * splits; u += blockDim.x) {
    const int r = u / splits;
    const float2 ml = get(reinterpret_cast<const float2*>(parts.row(u - r * splits, r)));
    weight[u] = ml.x;
    sum[u] = ml.y;
  }
  __syncthreads();
}

// join_rows once the parts' values are where `get` reads them; `weight` is its scratch, with their maxima and sums.
template <typename T, typename Parts, typename Get>
__device__ __forceinline__ void join_values(const AttendParams& a, const Parts& parts, int splits, int rows, int row0,
                                            int lo, int kh, float* weight, Get get) {
  const int D = a.pool.D, quads = D / 4;
  float* const sum = weight + rows * splits;
  float* const inv = sum + rows * splits;
  // a warp a row: the parts' weights (a split that saw no key of the row has the sum 0)
  for (int r = threadIdx.x >> 5; r < rows; r += blockDim.x >> 5) {
    const int lane = threadIdx.x & 31;
    float* const w = weight + r * splits;
    const float* const ls = sum + r * splits;
    float top = -INFINITY, l = 0.f;
    bool tiny = false;
    for (int k = lane; k < splits; k += 32)
      if (ls[k] != 0.f) top = fmaxf(top, w[k]);
#pragma unroll
    for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
    for (int k = lane; k < splits; k += 32) {
      const float wk = ls[k] == 0.f ? 0.f : exp2_fast((w[k] - top) * a.scale_log2);
      w[k] = wk;
      if (wk != 0.f) l += wk * ls[k];
      tiny |= wk == 0.f && ls[k] != 0.f;
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) l += __shfl_xor_sync(~0u, l, o);
    tiny = __any_sync(~0u, tiny);
    if (lane == 0) {
      inv[r] = l != 0.f ? (tiny ? -1.f / l : 1.f / l) : 0.f;  // below 0: see below
      const int R = row0 + r, tok = R / a.G;
      if (a.lse) a.lse[(int64_t)(lo + tok) * a.Hq + kh * a.G + (R - tok * a.G)] = row_lse(a, top, l);
    }
  }
  __syncthreads();
  for (int u = threadIdx.x; u < rows * quads; u += blockDim.x) {
    const int r = u / quads, d = (u - r * quads) * 4;
    const float* w = weight + r * splits;
    float o[4] = {};
#pragma unroll 8
    for (int k = 0; k < splits; ++k) {
      const float4 x = get(reinterpret_cast<const float4*>(parts.row(k, r) + kPartHead + d));
      const float wk = w[k];
      if (wk != 0.f) o[0] += wk * x.x, o[1] += wk * x.y, o[2] += wk * x.z, o[3] += wk * x.w;
    }
    if (inv[r] < 0.f) {  // a part whose weight is too small for fp32: an infinity or NaN in it is the row's all the same
      for (int k = 0; k < splits; ++k) {
        if (w[k] != 0.f || sum[r * splits + k] == 0.f) continue;
        const float4 x = get(reinterpret_cast<const float4*>(parts.row(k, r) + kPartHead + d));
        if (!isfinite(x.x)) o[0] += x.x;
        if (!isfinite(x.y)) o[1] += x.y;
        if (!isfinite(x.z)) o[2] += x.z;
        if (!isfinite(x.w)) o[3] += x.w;
      }
    }
    const int R = row0 + r, tok = R / a.G;
    const int64_t row = (int64_t)(lo + tok) * a.Hq + kh * a.G + (R - tok * a.G);
    const float n = fabsf(inv[r]);
    if (sizeof(T) == 2)
      *reinterpret_cast<uint2*>(a.out + (row * D + d) * 2) =
          make_uint2(pack_bf16x2(o[0] * n, o[1] * n), pack_bf16x2(o[2] * n, o[3] * n));
    else
      *reinterpret_cast<float4*>(a.out + (row * D + d) * 4) = make_float4(o[0] * n, o[1] * n, o[2] * n, o[3] * n);
  }
}

template <typename T, typename Parts>
__device__ __forceinline__ void join_rows(const AttendParams& a, const Parts& parts, int splits, int rows, int row0,
                                          int lo, int kh, uint8_t* scratch, int64_t room) {
  const int width = kPartHead + a.pool.D;
  // [rows][splits] the parts' maxima, then their weights, [rows][splits] their sums, [rows] the row's factor
  float* const weight = reinterpret_cast<float*>(scratch);
  auto near = [](const auto* x) { return *x; };
  auto far = [](const auto* x) { return __ldcg(x); };
  auto used_by = [&](int some) { return (join_scratch(some, splits) + 15) & ~(int64_t)15; };
  if constexpr (Parts::kByRow) {
    // The rows lie apart: their places are found once, a thread a row, then a warp fetches a row (each of its threads
    // finding it anew made a join of 5 rows of 21 parts take 13 us).  As many rows at a time as fit (read from global memory
    // 5 rows of 39 parts took 30 us).
    const int some = (int)min((int64_t)rows, (room - 16) / ((int64_t)splits * (width * 4 + 16) + 4));
    for (int r0 = 0; some && r0 < rows; r0 += some) {
      const int now = min(some, rows - r0);
      const int64_t used = used_by(now);
      const float* const values = reinterpret_cast<const float*>(scratch + used);
      const float** const place = reinterpret_cast<const float**>(scratch + used + (int64_t)now * splits * width * 4);
      float* const sum = weight + now * splits;
      __syncthreads();
      for (int u = threadIdx.x; u < now * splits; u += blockDim.x) {
        const int k = u / now, r = u - k * now;
        const float* const at = parts.row(k, r0 + r);
        place[u] = at + kPartHead;
        const float2 ml = far(reinterpret_cast<const float2*>(at));
        weight[r * splits + k] = ml.x;
        sum[r * splits + k] = ml.y;
      }
      __syncthreads();
      const uint32_t to = smem_u32(values);
      const int c = threadIdx.x & 31, warps = blockDim.x >> 5;
      for (int u0 = threadIdx.x >> 5; u0 < splits * now; u0 += 8 * warps) {
        const float* from[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) from[j] = place[min(u0 + j * warps, splits * now - 1)];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int u = u0 + j * warps;
          if (u < splits * now && c < a.pool.D / 4) cp_async16(to + (u * width + kPartHead + c * 4) * 4, from[j] + c * 4);
        }
      }
      cp_async_commit();
      cp_async_wait<0>();
      __syncthreads();
      join_values<T>(a, OwnParts{values, values + now * width, (int64_t)now * width, width}, splits, now, row0 + r0, lo, kh,
                     weight, near);
    }
    if (some) return;
  } else {
    const int64_t used = used_by(rows);
    __syncthreads();
    if (used + (int64_t)rows * splits * width * 4 <= room) {
      const int chunks = rows * width / 4;
      const uint32_t to = smem_u32(scratch + used);
      for (int u = threadIdx.x; u < splits * chunks; u += blockDim.x) {
        const int k = u / chunks;
        cp_async16(to + u * 16, parts.part(k) + (u - k * chunks) * 4);
      }
      cp_async_commit();
      cp_async_wait<0>();
      __syncthreads();
      const float* const values = reinterpret_cast<const float*>(scratch + used);
      const OwnParts here{values, values + rows * width, (int64_t)rows * width, width};
      join_heads(here, splits, rows, weight, near);
      join_values<T>(a, here, splits, rows, row0, lo, kh, weight, near);
      return;
    }
  }
  __syncthreads();
  join_heads(parts, splits, rows, weight, far);
  join_values<T>(a, parts, splits, rows, row0, lo, kh, weight, far);
}

template <typename T>
__device__ __forceinline__ void join_parts(const AttendParams& a, const float* part0, const float* part1, int64_t step,
                                           int splits, int rows, int row0, int lo, int kh, uint8_t* scratch,
                                           int64_t room) {
  join_rows<T>(a, OwnParts{part0, part1, step, kPartHead + a.pool.D}, splits, rows, row0, lo, kh, scratch, room);
}

// The same and, behind them, those of the group's prefix, whose rows are counted from the group's first one on.
struct AllParts {
  OwnParts own;
  PrefixPlan pre;
  int n, first, kh, row0;       // own parts; the prefix's first slot; the item's first row among the group's
  __device__ __forceinline__ const float* row(int k, int r) const {
    if (k < n) return own.row(k, r);
    const int R = row0 + r, tile = R / pre.rows;
    return prefix_part(pre, own.width - kPartHead, first + k - n, kh, tile, R - tile * pre.rows);
  }
  static constexpr bool kByRow = true;
};
template <typename T>
__device__ __forceinline__ void join_with_prefix(const AttendParams& a, const PrefixPlan& pre, const GroupRows& of,
                                                 const float* part0, const float* part1, int64_t step, int splits,
                                                 int rows, int row0, int lo, int kh, uint8_t* scratch, int64_t room) {
  const int2 slots = of.g < 0 ? make_int2(0, 0) : pre.table[of.g];
  const AllParts all{OwnParts{part0, part1, step, kPartHead + a.pool.D}, pre, splits, slots.x, kh,
                     (lo - of.lo) * a.G + row0};
  join_rows<T>(a, all, splits + slots.y, rows, row0, lo, kh, scratch, room);
}

}  // namespace dcp
