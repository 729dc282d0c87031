// Attention of few rows a KV head (single tokens, drafts) over a bf16 cache, and of any number of rows over an fp32
// cache, in warp-level matrix products (16 rows a warp).
//
// Rows are (new token, query head of the KV head) pairs.  The warps share tiles of keys that travel page row by page
// row through shared memory (asynchronous copies, several tiles in flight).  With MW = 4 or 8 each warp (of as many)
// has 16 rows of its own and sees every key; with MW = 1 four warps have the same 16 rows and a quarter of each tile's
// keys, and join their results at the end.  Few rows read every key once, so the bound is HBM and the work is spread
// over the keys: an item's keys are split over CTAs, the last of which joins the parts.
//
// fp32: each factor x is x_hi + x_lo, both with 11 significant bits, and x y = x_hi y_hi + x_hi y_lo + x_lo y_hi up
// to 2^-22: three tensor products for one.  A tile is taken apart once, for all warps (each warp doing it for itself
// made the conversions the bound: 331 us for what now takes 200).  The large and the small products of a score are
// summed apart, and a tile's weighted values start from 0 and are added to the running ones by one fma, so that the
// tensor cores' accumulation (which may truncate) never runs over more than a tile.
//
// Measured: 48 sequences' tokens, 40 query heads over 8 KV heads of 128, 200 .. 16000 keys (2.02 GB): 307-324 us,
// 6.2-6.6 TB/s; one token over 1531 keys 12.1 us (launch and look-ups 3, keys 2, two tiles 1.2, parts and join 3);
// fp32, 3 sequences of 100 .. 513 tokens, 8 heads of 64, 513 .. 3001 keys: 195 us, bound by the tf32 products (40 % of
// their rate while a CTA runs).
#pragma once

#include <type_traits>

#include "attend_join.cuh"

namespace dcp {

constexpr int kMaxSplits = 64;
constexpr int kEvenItems = 512;       // items whose tiles can be shared evenly,
constexpr int kEvenItemsSink = 1024;  // and under a window whose first positions stay visible (768 items of 4200 keys at
                                      // most: 251 us, against 256 in pieces of a fixed span)

constexpr int kMaxSms = 160;       // the join's scratch holds a part of two CTAs on each,
constexpr int kLeastSlots = 32;    // and at least so many of a shared prefix

struct RowParams {
  AttendParams a;
  int even;                     // 1: the CTAs share all items' key tiles evenly
  int splits, span, row_tiles;  // else keys of an item are cut into pieces of `span`
  uint32_t flip;                // sign bit of a scale below 0, put into q
  float* part;
  uint32_t* done;
  PrefixPlan pre;               // kPrefix, kRest
};

namespace {

// What a kernel is built for; each form has a translation unit of its own, so that none pays for another's tests.
enum Form {
  kPlain,   // a causal mask, a window
  kSink,    // a window whose first positions stay visible
  kPrefix,  // the rows of all sequences of a group against the prefix they share; leaves parts
  kRest,    // sequences against what they hold behind the shared prefix, joined with the prefix's parts
};

template <typename T, int DP, int MW>
struct Rows {
  static constexpr bool kHalf = sizeof(T) == 2;
  static constexpr int kWarps = MW == 8 ? 8 : 4, kThreads = 32 * kWarps;
  static constexpr int kCtas = MW == 8 && DP == 128 ? 1 : 2;  // of an SM, by shared memory
  static constexpr int kKeys = kHalf ? 64 : 32;         // keys of a tile
  static constexpr int kMine = kKeys * MW / kWarps;     // of them, a warp's
  static constexpr int kTiles = kMine / 8;              // in columns of 8
  static constexpr int kRow = DP * sizeof(T) + 16;      // bytes of a row in shared memory: no bank is hit twice
  static constexpr int kStages = kHalf ? 3 : 2;  // with 2, two CTAs of an fp32 kernel fit an SM
  static constexpr int kStage = 2 * kKeys * kRow;
  // fp32 taken apart: (hi, lo) pairs, rows padded so that a product's operands hit every bank once
  static constexpr int kPairK = DP * 8 + 32, kPairV = DP * 8 + 16;
  static constexpr int kQ = kHalf ? 0 : 16 * MW * kRow;
  static constexpr int kPairs = kHalf ? 0 : kKeys * (kPairK + kPairV);
  static constexpr int kJoin = MW == 1 ? kWarps * 16 * (DP + 2) * 4 : 0;
  static constexpr int kBuffers = kStages * kStage > kJoin ? kStages * kStage : kJoin;
  static constexpr int kSmem = kBuffers + kQ + kPairs;
  static constexpr int kRoom = (kSmem / 4 / (16 * MW) - 1) / 2;  // parts of a row that the join's scratch holds
  static_assert(kRoom >= (MW == 1 ? 2 * kMaxSms : kMaxSplits) + kLeastSlots,
                "the join's scratch fits where the tiles were");
  static_assert(kWarps * 16 * kMine * (int)sizeof(T) <= kKeys * (kHalf ? kRow : kPairK),
                "a tile's weights fit where its keys were");
};

__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool real) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(real ? 16 : 0) : "memory");
}
__device__ __forceinline__ void ldm4(uint32_t (&r)[4], uint32_t at) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(at));
}
__device__ __forceinline__ void ldm4t(uint32_t (&r)[4], uint32_t at) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(at));
}
__device__ __forceinline__ void mma_bf16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_tf32(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// x = hi + lo: hi the upper 11 significant bits, lo the rest, rounded where the products cut it (they read 11 bits).
// An infinity or NaN is (0, x): of the three products, only the one with the other factor's large part then sees it.
// (As (x, 0) it met the other's low part too, which is 0 for a factor of few bits, a weight of 1 among them: 0 times
// infinity is NaN.)  A NaN has all its bits set, lest the cut make it an infinity.
__device__ __forceinline__ uint2 halves(uint32_t x) {
  if ((x & 0x7F800000u) == 0x7F800000u) return make_uint2(0, x & 0x007FFFFFu ? 0x7FFFFFFFu : x);
  const uint32_t hi = x & 0xFFFFE000u;
  return make_uint2(hi, __float_as_uint(__uint_as_float(x) - __uint_as_float(hi)) + 0x1000u);
}
// Four consecutive values taken apart.
__device__ __forceinline__ void store_halves(uint8_t* to, const uint4& x) {
  const uint2 a = halves(x.x), b = halves(x.y), c = halves(x.z), d = halves(x.w);
  *reinterpret_cast<uint4*>(to) = make_uint4(a.x, a.y, b.x, b.y);
  *reinterpret_cast<uint4*>(to + 16) = make_uint4(c.x, c.y, d.x, d.y);
}

// The keys some of an item's rows see, by place: place x stands for position x from `seam` on, and for position x - gap
// before it (the first positions, which stay visible behind a window that has left them).
struct Seen {
  int begin, end, seam, gap;
  template <int FORM>
  __device__ __forceinline__ int pos(int x) const {
    return FORM == kSink && x < seam ? x - gap : x;
  }
};

// Rows [row0, row0 + rows) of (token, head of the KV head) of sequence s, which has `len` new tokens from row lo of q
// on and `kv` cached positions, against the keys at the places of `keys`.  The result goes to out and lse, or to `part`.
// (kPrefix: `s` is the group's first sequence, the rows are those of all of the group's.)
template <typename T, int DP, int MW, int FORM>
__device__ __forceinline__ void attend_piece(const RowParams& p, uint8_t* smem,
                                             int64_t (*s_off)[Rows<T, DP, MW>::kKeys], int s, int kh, int lo,
                                             int len, int kv, int row0, int rows, const Seen& keys, float* part) {
  using R = Rows<T, DP, MW>;
  const AttendParams& a = p.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  const int D = a.pool.D, bs = a.pool.bs;
  const int c_lo = kv - len + row0 / a.G, c_hi = kv - len + (row0 + rows - 1) / a.G;  // first and last row's position
  const int begin = keys.begin, end = keys.end;
  const int n_tiles = (end - begin + R::kKeys - 1) / R::kKeys;
  const int32_t* table = a.b.tables + (int64_t)s * a.b.table_stride;

  // A key's table entry is read a tile before its place is needed: nothing waits for the one that was asked for last.
  struct Key {
    int blk, row;  // row -1: no key
  };
  auto find = [&](int t) -> Key {
    const int x = begin + t * R::kKeys + threadIdx.x;
    if (threadIdx.x >= R::kKeys || x >= end) return Key{0, -1};
    const int pos = keys.pos<FORM>(x), page = pos / bs;
    return Key{table[page], pos - page * bs};
  };
  auto place = [&](const Key& k) -> int64_t {
    if (k.row < 0) return -1;
    if (k.blk < 0 || k.blk >= a.pool.n_blocks) {
      set_status(a.b.status, DCP_EDEVICE);
      return -1;
    }
    return k.blk * a.pool.s_block + kh * a.pool.s_head + (int64_t)k.row * a.pool.s_row;
  };
  const uint32_t base = smem_u32(smem);
  const int chunks = D * (int)sizeof(T) / 16;
  constexpr int kChunks = DP * sizeof(T) / 16;
  auto fetch = [&](int t) {
    if (t < n_tiles) {
      const uint32_t k_at = base + (t % R::kStages) * R::kStage, v_at = k_at + R::kKeys * R::kRow;
      constexpr int kEach = R::kKeys * kChunks / R::kThreads, kAtOnce = kEach < 4 ? kEach : 4;
#pragma unroll
      for (int j0 = 0; j0 < kEach; j0 += kAtOnce) {  // (the copies are not reordered: their places first)
        int64_t off[kAtOnce];
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j) off[j] = s_off[t & 3][(threadIdx.x + (j0 + j) * R::kThreads) / kChunks];
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j) {
          const int u = threadIdx.x + (j0 + j) * R::kThreads, row = u / kChunks, ch = u % kChunks;
          const bool real = off[j] >= 0 && ch < chunks;
          const int64_t at = real ? off[j] * (int64_t)sizeof(T) + ch * 16 : 0;
          copy16(k_at + row * R::kRow + ch * 16, a.pool.k + at, real);
          copy16(v_at + row * R::kRow + ch * 16, a.pool.v + at, real);
        }
      }
    }
    cp_async_commit();
  };
  Key f[R::kStages];
#pragma unroll
  for (int t = 0; t < R::kStages; ++t) f[t] = find(t);
  // ---- q: bf16 in registers as the products want it, on its way while the keys are looked up; fp32 in shared memory
  const int first = MW == 1 ? 0 : warp * 16;  // the warp's first row of the item
  uint32_t qa[R::kHalf ? DP / 16 : 1][4];
  auto q_row = [&](int r) {
    const int tok = (row0 + r) / a.G;
    return a.q + ((int64_t)(lo + tok) * a.q_stride + (int64_t)(kh * a.G + (row0 + r) - tok * a.G) * D) *
                     (int64_t)sizeof(T);
  };
  if constexpr (R::kHalf) {
    const char* q0 = first + g < rows ? q_row(first + g) : nullptr;
    const char* q1 = first + g + 8 < rows ? q_row(first + g + 8) : nullptr;
#pragma unroll
    for (int k = 0; k < DP / 16; ++k) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const char* q = e & 1 ? q1 : q0;
        const int d = 16 * k + 2 * c + (e >> 1) * 8;
        qa[k][e] = q && d < D ? *reinterpret_cast<const uint32_t*>(q + d * 2) : 0;
      }
    }
  }
  if (threadIdx.x < R::kKeys)
#pragma unroll
    for (int t = 0; t < R::kStages; ++t) s_off[t][threadIdx.x] = place(f[t]);
  __syncthreads();
#pragma unroll
  for (int t = 0; t < R::kStages - 1; ++t) fetch(t);

  if constexpr (R::kHalf) {
    const uint32_t flip = p.flip | p.flip >> 16;
#pragma unroll
    for (int k = 0; k < DP / 16; ++k)
#pragma unroll
      for (int e = 0; e < 4; ++e) qa[k][e] ^= flip;
  } else {
    uint8_t* qs = smem + R::kBuffers;
    for (int u = threadIdx.x; u < 16 * MW * (DP / 4); u += R::kThreads) {
      const int r = u / (DP / 4), d = u % (DP / 4) * 4;
      uint4 x = make_uint4(0, 0, 0, 0);
      if (r < rows && d < D) {
        x = *reinterpret_cast<const uint4*>(q_row(r) + d * 4);
        x = make_uint4(x.x ^ p.flip, x.y ^ p.flip, x.z ^ p.flip, x.w ^ p.flip);
      }
      *reinterpret_cast<uint4*>(qs + r * R::kRow + d * 4) = x;
    }
  }

  // ---- the keys
  float o[DP / 8][4];
#pragma unroll
  for (int j = 0; j < DP / 8; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};  // rows g and g + 8; l is this lane's share
  int pos_of[2];
#pragma unroll
  for (int e = 0; e < 2; ++e) pos_of[e] = kv - len + (row0 + first + g + 8 * e) / a.G;
  const int k0 = MW == 1 ? warp * R::kMine : 0;  // the warp's first key of a tile
  const bool idle = first >= rows;

  for (int t = 0; t < n_tiles; ++t) {
    const Key ahead = t + R::kStages < n_tiles ? find(t + R::kStages) : Key{0, -1};
    cp_async_wait<R::kStages - 2>();
    __syncthreads();
    fetch(t + R::kStages - 1);
    const uint32_t k_at = base + (t % R::kStages) * R::kStage, v_at = k_at + R::kKeys * R::kRow;
    const uint8_t* kp = smem + (t % R::kStages) * R::kStage;
    const uint8_t* vp = kp + R::kKeys * R::kRow;
    const int p0 = begin + t * R::kKeys;
    bool all;  // no row's mask hides a key
    if constexpr (FORM == kPrefix)
      all = p0 + R::kKeys <= end;
    else if constexpr (FORM == kSink)  // first positions lie before every row
      all = p0 + R::kKeys <= keys.seam || (p0 + R::kKeys <= end && p0 >= keys.seam && p0 + R::kKeys - 1 <= c_lo &&
                                           p0 >= c_hi - a.window);
    else
      all = p0 + R::kKeys <= end && (!a.causal || p0 + R::kKeys - 1 <= c_lo) && (a.window < 0 || p0 >= c_hi - a.window);
    // a masked tile whose values hold infinities or NaN: 0 times those must not reach a row that does not see them
    bool poison = false;
    uint8_t* const pk = smem + R::kBuffers + R::kQ;
    uint8_t* const pv = pk + R::kKeys * R::kPairK;
    if constexpr (!R::kHalf) {
#pragma unroll 4
      for (int u = threadIdx.x; u < R::kKeys * kChunks; u += R::kThreads) {
        const int row = u / kChunks, ch = u % kChunks;
        store_halves(pk + row * R::kPairK + ch * 32, *reinterpret_cast<const uint4*>(kp + row * R::kRow + ch * 16));
        store_halves(pv + row * R::kPairV + ch * 32, *reinterpret_cast<const uint4*>(vp + row * R::kRow + ch * 16));
      }
      __syncthreads();
    }
    if (!all) {
      for (int u = threadIdx.x; u < R::kKeys * kChunks; u += R::kThreads) {
        const uint4 x = *reinterpret_cast<const uint4*>(vp + u / kChunks * R::kRow + u % kChunks * 16);
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int e = 0; e < 4; ++e)
          poison |= (w[e] & 0x7F800000u) == 0x7F800000u || (R::kHalf && (w[e] & 0x7F80u) == 0x7F80u);
      }
      poison = __syncthreads_or(poison);
    }
    float x[R::kTiles][4], keep[2];
#pragma unroll
    for (int n = 0; n < R::kTiles; ++n) x[n][0] = x[n][1] = x[n][2] = x[n][3] = 0.f;
    if (!idle) {
      if constexpr (R::kHalf) {
        float y[R::kTiles][4];  // every other step's products, so that none waits for the one before it
#pragma unroll
        for (int n = 0; n < R::kTiles; ++n) y[n][0] = y[n][1] = y[n][2] = y[n][3] = 0.f;
#pragma unroll
        for (int k = 0; k < DP / 32; ++k)
#pragma unroll
          for (int n = 0; n < R::kTiles; ++n) {
            uint32_t b[4];
            ldm4(b, k_at + (k0 + 8 * n + (lane & 7)) * R::kRow + k * 64 + (lane >> 3) * 16);
            mma_bf16(x[n], qa[2 * k], b[0], b[1]);
            mma_bf16(y[n], qa[2 * k + 1], b[2], b[3]);
          }
#pragma unroll
        for (int n = 0; n < R::kTiles; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) x[n][e] += y[n][e];
      } else {
        float y[R::kTiles][4];
#pragma unroll
        for (int n = 0; n < R::kTiles; ++n) y[n][0] = y[n][1] = y[n][2] = y[n][3] = 0.f;
        const uint8_t* qp = smem + R::kBuffers + (first + g) * R::kRow + c * 4;
        const uint8_t* kq = pk + (k0 + g) * R::kPairK + c * 8;
#pragma unroll
        for (int k = 0; k < DP / 8; ++k) {
          uint32_t ah[4], al[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint2 f = halves(*reinterpret_cast<const uint32_t*>(qp + (e & 1) * 8 * R::kRow +
                                                                      (8 * k + (e >> 1) * 4) * 4));
            ah[e] = f.x;
            al[e] = f.y;
          }
          uint2 f[R::kTiles][2];
#pragma unroll
          for (int n = 0; n < R::kTiles; ++n) {
            f[n][0] = *reinterpret_cast<const uint2*>(kq + 8 * n * R::kPairK + 64 * k);
            f[n][1] = *reinterpret_cast<const uint2*>(kq + 8 * n * R::kPairK + 64 * k + 32);
          }
          // no product right behind one it adds to: it would wait for it
#pragma unroll
          for (int n = 0; n < R::kTiles; ++n) mma_tf32(y[n], ah, f[n][0].y, f[n][1].y);
#pragma unroll
          for (int n = 0; n < R::kTiles; ++n) mma_tf32(x[n], ah, f[n][0].x, f[n][1].x);
#pragma unroll
          for (int n = 0; n < R::kTiles; ++n) mma_tf32(y[n], al, f[n][0].x, f[n][1].x);
        }
#pragma unroll
        for (int n = 0; n < R::kTiles; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) x[n][e] += y[n][e];
      }
      if (!all) {
#pragma unroll
        for (int n = 0; n < R::kTiles; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int x_at = p0 + k0 + 8 * n + 2 * c + (e & 1), pos = keys.pos<FORM>(x_at), at = pos_of[e >> 1];
            bool hidden = x_at >= end;
            if constexpr (FORM == kSink)
              hidden |= !sees(a, at, pos);
            else if constexpr (FORM != kPrefix)
              hidden |= (a.causal && pos > at) || (a.window >= 0 && pos < at - a.window);
            if (hidden) x[n][e] = -INFINITY;
          }
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float top = m[e];
#pragma unroll
        for (int n = 0; n < R::kTiles; ++n) top = fmaxf(top, fmaxf(x[n][2 * e], x[n][2 * e + 1]));
        top = fmaxf(top, __shfl_xor_sync(~0u, top, 1));
        top = fmaxf(top, __shfl_xor_sync(~0u, top, 2));
        keep[e] = m[e] == top ? 1.f : exp2_fast((m[e] - top) * a.scale_log2);
        m[e] = top;
        // the maximum comes off before the scaling: the scaled one is rounded by more than fp32's exponents from 2^31 on
        const float base = top == -INFINITY ? 0.f : top;
        float sum = 0.f;
#pragma unroll
        for (int n = 0; n < R::kTiles; ++n)
#pragma unroll
          for (int b = 2 * e; b < 2 * e + 2; ++b) {
            const bool hidden = x[n][b] == -INFINITY;
            x[n][b] = exp2_fast((x[n][b] - base) * a.scale_log2);
            sum += x[n][b];
            if (poison && hidden) x[n][b] = -1.f;
          }
        l[e] = l[e] * keep[e] + sum;
      }
    }
    if (poison) __syncthreads();  // every warp is done with the keys: the weights take their place
    if (!idle) {
      if (poison) {  // in plain arithmetic, skipping what a row does not see
        T* ps = reinterpret_cast<T*>(R::kHalf ? smem + (t % R::kStages) * R::kStage : pk) + warp * 16 * R::kMine;
#pragma unroll
        for (int n = 0; n < R::kTiles; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) ps[(g + 8 * (e >> 1)) * R::kMine + 8 * n + 2 * c + (e & 1)] = (T)x[n][e];
        __syncwarp();
#pragma unroll
        for (int j = 0; j < DP / 8; ++j) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float sum = o[j][e] * keep[e >> 1];
            for (int n = 0; n < R::kMine; ++n) {
              const float w = (float)ps[(g + 8 * (e >> 1)) * R::kMine + n];
              if (w < 0.f) continue;
              sum = fmaf(w, (float)*reinterpret_cast<const T*>(vp + (k0 + n) * R::kRow +
                                                               (8 * j + 2 * c + (e & 1)) * (int)sizeof(T)), sum);
            }
            o[j][e] = sum;
          }
        }
      } else if constexpr (R::kHalf) {
#pragma unroll
        for (int j = 0; j < DP / 8; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[j][e] *= keep[e >> 1];
#pragma unroll
        for (int n = 0; n < R::kTiles; n += 2) {
          const uint32_t w[4] = {pack_bf16x2(x[n][0], x[n][1]), pack_bf16x2(x[n][2], x[n][3]),
                                 pack_bf16x2(x[n + 1][0], x[n + 1][1]), pack_bf16x2(x[n + 1][2], x[n + 1][3])};
#pragma unroll
          for (int j = 0; j < DP / 8; j += 2) {
            uint32_t b[4];
            ldm4t(b, v_at + (k0 + 8 * n + (lane & 15)) * R::kRow + (j + (lane >> 4)) * 16);
            mma_bf16(o[j], w, b[0], b[1]);
            mma_bf16(o[j + 1], w, b[2], b[3]);
          }
        }
      } else {
        // weight columns in the order (0, 2, 4, 6, 1, 3, 5, 7): a lane's own scores are its factors
        uint32_t wh[R::kTiles][4], wl[R::kTiles][4];
#pragma unroll
        for (int n = 0; n < R::kTiles; ++n) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint2 f = halves(__float_as_uint(x[n][(e & 1) * 2 + (e >> 1)]));
            wh[n][e] = f.x;
            wl[n][e] = f.y;
          }
        }
        const uint8_t* vq = pv + (k0 + 2 * c) * R::kPairV + g * 8;
#pragma unroll
        for (int j = 0; j < DP / 8; j += 4) {
          float y[4][4];
#pragma unroll
          for (int b = 0; b < 4; ++b) y[b][0] = y[b][1] = y[b][2] = y[b][3] = 0.f;
#pragma unroll
          for (int n = 0; n < R::kTiles; ++n) {
            uint2 f[4][2];
#pragma unroll
            for (int b = 0; b < 4; ++b) {
              f[b][0] = *reinterpret_cast<const uint2*>(vq + 8 * n * R::kPairV + 64 * (j + b));
              f[b][1] = *reinterpret_cast<const uint2*>(vq + (8 * n + 1) * R::kPairV + 64 * (j + b));
            }
#pragma unroll
            for (int b = 0; b < 4; ++b) mma_tf32(y[b], wl[n], f[b][0].x, f[b][1].x);
#pragma unroll
            for (int b = 0; b < 4; ++b) mma_tf32(y[b], wh[n], f[b][0].y, f[b][1].y);
#pragma unroll
            for (int b = 0; b < 4; ++b) mma_tf32(y[b], wh[n], f[b][0].x, f[b][1].x);
          }
#pragma unroll
          for (int b = 0; b < 4; ++b)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[j + b][e] = fmaf(o[j + b][e], keep[e >> 1], y[b][e]);
        }
      }
    }
    if (threadIdx.x < R::kKeys) s_off[(t + R::kStages) & 3][threadIdx.x] = place(ahead);
  }
  cp_async_wait<0>();
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    l[e] += __shfl_xor_sync(~0u, l[e], 1);
    l[e] += __shfl_xor_sync(~0u, l[e], 2);
  }

  // ---- results
  auto put = [&](int r, int d, float y0, float y1, float mr, float lr) {  // two dims of a row of the item
    if (d >= D) return;
    if (part) {
      float* at = part + (int64_t)r * (kPartHead + D);
      if (d == 0) *reinterpret_cast<float2*>(at) = make_float2(mr, lr);
      *reinterpret_cast<float2*>(at + kPartHead + d) = make_float2(y0, y1);
      return;
    }
    const float inv = lr != 0.f ? 1.f / lr : 0.f;
    const int tok = (row0 + r) / a.G;
    const int64_t row = (int64_t)(lo + tok) * a.Hq + kh * a.G + (row0 + r) - tok * a.G;
    if constexpr (R::kHalf)
      *reinterpret_cast<uint32_t*>(a.out + (row * D + d) * 2) = pack_bf16x2(y0 * inv, y1 * inv);
    else
      *reinterpret_cast<float2*>(a.out + (row * D + d) * 4) = make_float2(y0 * inv, y1 * inv);
    if (a.lse && d == 0) a.lse[row] = row_lse(a, mr, lr);
  };
  if constexpr (MW > 1) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int r = first + g + 8 * e;
      if (r >= rows) continue;
#pragma unroll
      for (int j = 0; j < DP / 8; ++j) put(r, 8 * j + 2 * c, o[j][2 * e], o[j][2 * e + 1], m[e], l[e]);
    }
  } else {
    __syncthreads();
    float* join = reinterpret_cast<float*>(smem);  // [warp][16][DP + 2]
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int r = g + 8 * e;
      if (r >= rows) continue;
      float* at = join + (warp * 16 + r) * (DP + 2);
      if (c == 0) *reinterpret_cast<float2*>(at) = make_float2(m[e], l[e]);
#pragma unroll
      for (int j = 0; j < DP / 8; ++j)
        *reinterpret_cast<float2*>(at + 2 + 8 * j + 2 * c) = make_float2(o[j][2 * e], o[j][2 * e + 1]);
    }
    __syncthreads();
    for (int u = threadIdx.x; u < rows * (DP / 2); u += R::kThreads) {
      const int r = u / (DP / 2), d = u % (DP / 2) * 2;
      float top = -INFINITY;
#pragma unroll
      for (int w = 0; w < R::kWarps; ++w) top = fmaxf(top, join[(w * 16 + r) * (DP + 2)]);
      float sum = 0.f, y0 = 0.f, y1 = 0.f;
#pragma unroll
      for (int w = 0; w < R::kWarps; ++w) {
        const float* at = join + (w * 16 + r) * (DP + 2);
        if (at[1] == 0.f) continue;
        const float k = exp2_fast((at[0] - top) * a.scale_log2);
        sum += k * at[1];
        y0 += k * at[2 + d];
        y1 += k * at[3 + d];
      }
      put(r, d, y0, y1, top, sum);
    }
  }
}

// The keys some of the rows see, from position `from` on.
template <int FORM>
__device__ __forceinline__ Seen seen_range(const AttendParams& a, int from, int kv, int len, int row0, int rows) {
  const int c_lo = kv - len + row0 / a.G, c_hi = kv - len + (row0 + rows - 1) / a.G;
  Seen k;
  k.seam = FORM != kPrefix && a.window >= 0 ? max(0, c_lo - a.window) : from;
  k.begin = k.gap = FORM == kSink ? k.seam - min(a.sink, k.seam) : k.seam;
  k.end = max(FORM != kPrefix && a.causal ? min(kv, c_hi + 1) : kv, k.begin);
  return k;
}

// What a sequence holds behind its group's prefix (kRest); without slots it is worked on alone, its group only checked.
__device__ __forceinline__ bool rest_of(const RowParams& p, int s, int lo, int len, int kv, GroupRows& of, int& from) {
  const bool sound = group_of(p.a, s, lo, len, kv, of, from);
  if (p.pre.slots == 0) {
    from = 0;
    of.g = -1;
  }
  return sound;
}

// An item is a tile of rows of one sequence and KV head.
template <typename T, int DP, int MW, int FORM>
__global__ void __launch_bounds__(Rows<T, DP, MW>::kThreads, Rows<T, DP, MW>::kCtas)
    rows_kernel(const __grid_constant__ RowParams p) {
  using R = Rows<T, DP, MW>;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ int64_t s_off[4][R::kKeys];  // element offset of a key's row in the pool, -1: not read
  __shared__ int s_last;
  const AttendParams& a = p.a;
  const int D = a.pool.D, width = kPartHead + D;
  allow_dependents();
  wait_for_predecessor();

  if constexpr (MW == 1 && FORM != kPrefix) {
    if (p.even) {
      // Every CTA takes the same number of consecutive key tiles of all items together: the sums of the items' tiles,
      // then the pieces of the items that lie in the CTA's share.  At most its first and its last piece are parts.
      // Where items are joined with a prefix's parts, an item counts kBegin tiles more, for its look-ups and its join (of
      // single tiles a CTA had up to 13 items, and 32 branches of 20 .. 700 positions behind their prefix took 103 us);
      // a share that would end among these leaves the item to the next CTA.
      constexpr int kBegin = FORM == kRest ? 10 : 0;
      constexpr int kItems = FORM == kSink ? kEvenItemsSink : kEvenItems;
      __shared__ int64_t s_first[kItems + 1];  // tiles before an item
      __shared__ int64_t s_warp[R::kWarps];
      const int items = a.b.n_seqs * a.pool.H, each = (items + R::kThreads - 1) / R::kThreads;
      const int i0 = min(items, (int)threadIdx.x * each), i1 = min(items, i0 + each);
      auto look = [&](int i, int& lo, int& len, int& kv, Seen& seen, GroupRows& of) -> int64_t {
        int64_t kv64;
        const bool sound = seq_rows(a.b, i / a.pool.H, lo, len) &
                           seq_kv(a.b, a.pool.bs, a.pool.H, i / a.pool.H, i % a.pool.H, kv64);
        if (!sound || len == 0) return 0;
        kv = (int)kv64;
        int from = 0;
        if constexpr (FORM == kRest)
          if (!rest_of(p, i / a.pool.H, lo, len, kv, of, from)) return 0;
        seen = seen_range<FORM>(a, from, kv, len, 0, len * a.G);
        // rows that see nothing have their result too
        return max(1, (seen.end - seen.begin + R::kKeys - 1) / R::kKeys) + kBegin;
      };
      int lo, len, kv;
      Seen seen;
      GroupRows of{};
      int64_t mine = 0;
      for (int i = i0; i < i1; ++i) {
        s_first[i] = mine;
        mine += look(i, lo, len, kv, seen, of);
      }
      int64_t before = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(~0u, before, o);
        if ((threadIdx.x & 31) >= o) before += y;
      }
      if ((threadIdx.x & 31) == 31) s_warp[threadIdx.x >> 5] = before;
      __syncthreads();
      int64_t total = 0;
#pragma unroll
      for (int w = 0; w < R::kWarps; ++w) {
        if (w < threadIdx.x >> 5) before += s_warp[w];
        total += s_warp[w];
      }
      for (int i = i0; i < i1; ++i) s_first[i] += before - mine;
      if (threadIdx.x == 0) s_first[items] = total;
      __syncthreads();
      // Two tiles a CTA at least, and no fewer CTAs than items (a piece costs as much to begin as several tiles).
      const int64_t ctas = max((int64_t)1, min((int64_t)gridDim.x, max((total + 1) / 2, min((int64_t)items, total))));
      if (blockIdx.x >= ctas) return;
      auto item_at = [&](int64_t x) {  // the last item that begins at or before x
        int item = 0;
        for (int step = kItems; step; step >>= 1)
          if (item + step < items && s_first[item + step] <= x) item += step;
        return item;
      };
      auto share = [&](int64_t c) {  // where CTA c's share begins
        const int64_t x = c * total / ctas;
        if constexpr (kBegin == 0) return x;
        if (c == ctas) return total;
        const int64_t f0 = s_first[item_at(x)];
        return x - f0 <= kBegin ? f0 : x;
      };
      int64_t at = share(blockIdx.x);
      const int64_t to = share(blockIdx.x + 1);
      int item = item_at(at);
      for (; at < to; ++item) {
        const int64_t f0 = s_first[item], f1 = s_first[item + 1];
        if (f1 <= at) continue;
        look(item, lo, len, kv, seen, of);
        const int64_t stop = min(to, f1);
        const bool opens = at == f0, closes = stop == f1;
        const int s = item / a.pool.H, kh = item % a.pool.H, rows = len * a.G;
        Seen piece = seen;
        if (!opens) piece.begin += (int)(at - f0 - kBegin) * R::kKeys;
        if (!closes) piece.end = seen.begin + (int)(stop - f0 - kBegin) * R::kKeys;
        const int64_t slot = (int64_t)16 * width;  // parts of a CTA: of an item it goes on with, of one it begins
        const bool parted = !opens || !closes || (FORM == kRest && p.pre.slots);
        float* const part = parted ? p.part + (2 * (int64_t)blockIdx.x + opens) * slot : nullptr;
        attend_piece<T, DP, 1, FORM>(p, smem, s_off, s, kh, lo, len, kv, 0, rows, piece, part);
        if (part) {
          const int64_t c0 = ((f0 + kBegin + 1) * ctas - 1) / total, c1 = (f1 * ctas - 1) / total;
          const int n = (int)(c1 - c0 + 1);
          float* const part0 = opens ? part : p.part + (2 * c0 + 1) * slot;
          if (FORM == kRest && n == 1)
            __syncthreads();
          else if (!last_of(p.done + item, n, &s_last))
            goto next;
          if constexpr (FORM == kRest)
            join_with_prefix<T>(a, p.pre, of, part0, p.part + 2 * (c0 + 1) * slot, 2 * slot, n, rows, 0, lo, kh, smem,
                                R::kSmem);
          else
            join_parts<T>(a, part0, p.part + 2 * (c0 + 1) * slot, 2 * slot, n, rows, 0, lo, kh, smem, R::kSmem);
        }
      next:
        at = stop;
        __syncthreads();
      }
      return;
    }
  }

  const int kh = blockIdx.y;
  int lo, len;
  if constexpr (FORM == kPrefix) {
    __shared__ PrefixPiece s_piece;
    if (threadIdx.x < 32) {
      const PrefixPiece piece = prefix_piece(a, p.pre, blockIdx.z, (blockIdx.x | blockIdx.y | blockIdx.z) == 0);
      if (threadIdx.x == 0) s_piece = piece;
    }
    __syncthreads();
    const PrefixPiece piece = s_piece;
    const GroupRows& of = piece.of;
    const int row0 = blockIdx.x * 16 * MW;
    if (row0 >= of.len * a.G) return;
    const int rows = min(16 * MW, of.len * a.G - row0);
    const int whole = ((of.prefix + piece.splits - 1) / piece.splits + R::kKeys - 1) / R::kKeys * R::kKeys;
    Seen seen{};
    seen.begin = (int)min((int64_t)of.prefix, (int64_t)piece.split * whole);
    seen.end = (int)min((int64_t)of.prefix, (int64_t)seen.begin + whole);
    attend_piece<T, DP, MW, FORM>(p, smem, s_off, of.s, kh, of.lo, of.len, of.prefix, row0, rows, seen,
                                  prefix_part(p.pre, D, blockIdx.z, kh, blockIdx.x, 0));
    return;
  }
  const int s = blockIdx.z / p.splits, split = blockIdx.z % p.splits;
  const int tile = p.row_tiles - 1 - blockIdx.x;
  int64_t kv64;
  const bool sound = seq_rows(a.b, s, lo, len) & seq_kv(a.b, a.pool.bs, a.pool.H, s, kh, kv64);
  if (!sound) return;
  const int kv = (int)kv64, n_rows = len * a.G, row0 = tile * 16 * MW;
  if (row0 >= n_rows) return;
  const int rows = min(16 * MW, n_rows - row0);
  GroupRows of{};
  int from = 0;
  if constexpr (FORM == kRest)
    if (!rest_of(p, s, lo, len, kv, of, from)) return;
  Seen seen = seen_range<FORM>(a, from, kv, len, row0, rows);
  if (p.splits > 1) {
    // as even pieces of whole tiles as the splits allow (a longer sequence than max_kv has longer pieces)
    const int span = max((int64_t)p.span, ((int64_t)(seen.end - seen.begin) + p.splits - 1) / p.splits);
    const int whole = (span + R::kKeys - 1) / R::kKeys * R::kKeys;
    seen.begin = (int)min((int64_t)seen.end, seen.begin + (int64_t)split * whole);
    seen.end = (int)min((int64_t)seen.end, (int64_t)seen.begin + whole);
  }
  const int64_t item = ((int64_t)s * a.pool.H + kh) * p.row_tiles + tile;
  float* const parts =
      p.splits > 1 || (FORM == kRest && p.pre.slots) ? part_of(p.part, item, p.splits, 0, 16 * MW, D, 0) : nullptr;
  const int64_t step = (int64_t)16 * MW * width;
  attend_piece<T, DP, MW, FORM>(p, smem, s_off, s, kh, lo, len, kv, row0, rows, seen,
                                parts ? parts + split * step : nullptr);
  if (!parts) return;
  if (FORM == kRest && p.splits == 1)
    __syncthreads();
  else if (!last_of(p.done + item, p.splits, &s_last))
    return;
  if constexpr (FORM == kRest)
    join_with_prefix<T>(a, p.pre, of, parts, parts + step, step, p.splits, rows, row0, lo, kh, smem, R::kSmem);
  else
    join_parts<T>(a, parts, parts + step, step, p.splits, rows, row0, lo, kh, smem, R::kSmem);
}

template <typename T, int DP, int MW, int FORM>
cudaError_t launch(const RowParams& p, cudaStream_t s) {
  static LaunchCache lc;
  int blocks;
  using R = Rows<T, DP, MW>;
  const cudaError_t e = launch_setup(lc, rows_kernel<T, DP, MW, FORM>, R::kThreads, R::kSmem, &blocks);
  if (e != cudaSuccess) return e;
  const dim3 grid = FORM == kPrefix ? dim3(p.pre.tiles, p.a.pool.H, p.pre.slots)
                    : p.even        ? dim3(p.splits)
                                    : dim3(p.row_tiles, p.a.pool.H, p.a.b.n_seqs * p.splits);
  return launch_behind(rows_kernel<T, DP, MW, FORM>, grid, R::kThreads, R::kSmem, s, p);
}

// `rows` of a CTA.
template <int FORM>
cudaError_t launch_form(const RowParams& p, int rows, cudaStream_t s) {
  const bool one = rows == 16, wide = p.a.pool.D > 64;
  if (p.a.pool.dtype == DCP_BF16) {
    if (one) return wide ? launch<__nv_bfloat16, 128, 1, FORM>(p, s) : launch<__nv_bfloat16, 64, 1, FORM>(p, s);
    return wide ? launch<__nv_bfloat16, 128, 4, FORM>(p, s) : launch<__nv_bfloat16, 64, 4, FORM>(p, s);
  }
  if (one) return wide ? launch<float, 128, 1, FORM>(p, s) : launch<float, 64, 1, FORM>(p, s);
  return wide ? launch<float, 128, 8, FORM>(p, s) : launch<float, 64, 8, FORM>(p, s);
}

}  // namespace

// The forms' launches, each in its own translation unit.
cudaError_t launch_rows_plain(const RowParams& p, int rows, cudaStream_t s);
cudaError_t launch_rows_sink(const RowParams& p, int rows, cudaStream_t s);
cudaError_t launch_rows_prefix(const RowParams& p, int rows, cudaStream_t s);
cudaError_t launch_rows_rest(const RowParams& p, int rows, cudaStream_t s);

}  // namespace dcp
