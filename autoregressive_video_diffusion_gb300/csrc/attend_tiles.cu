// Attention of the new tokens over the paged bf16 cache in tiles of 128 rows x 128 keys on the 5th-generation tensor
// cores.
//
// Rows are (new token, query head of the KV head) pairs in that order, so the heads that share a KV head share its
// tiles.  A CTA owns 256 rows (two tiles of 128) of one sequence and KV head and walks the keys they see:
//   scores   S = Q K^T      Q, K in shared memory, S (fp32) in tensor memory
//   softmax  P = exp(S - m), m a running maximum; P (bf16) goes back over S in tensor memory
//   values   O += P V       P from tensor memory, V from shared memory, O (fp32) stays in tensor memory
// Each row tile has its own 8 warps, so one tile's softmax runs under the other's matrix products; a row is two threads'
// work, half of its scores each, so that an SM quarter always has several warps to choose from.  The weights are taken
// relative to a level m that the earlier tiles have set: the maximum of the first tile, and from then on what the sums
// of the weights say (a sum of 64 weights is within 2^6 of its largest).  m follows at the next tile, and only when a
// tile's weights have added up to more than 2^8, which leaves O untouched in almost every step; m has moved or not, the
// quotient O / l is the same (weights keep their relative precision in bf16, sums are held in 32 bits).  Only a row
// whose scores rise by more than 2^64 within one tile, or lie beyond 2^8192 (levels travel between a row's threads in
// bf16), or whose O has passed fp32's range by the weights of a level left behind, needs more care: its item is then done
// again with each tile's own maximum, in fp32, taken off before the scaling.
//
// Warps 0-7 and 8-15: softmax of row tile 0 and 1.  Warps 16, 17: issue the matrix products of row tile 0 and 1 (one
// warp for both was busy for 3600 clocks a step of 2048 clocks of products).  Warps 18, 19: copy the pages of the keys
// and of the values with TMA (a page of block_size positions is a box; 128-byte swizzle).
//
// A weight of 0 times a value of infinity or NaN is NaN.  So in the tiles where some row must not see some key, the
// softmax warps put zeros for rows past the sequence (page rows never written hold anything) and for infinities and
// NaN before they hand over their weights; rows that do see those get them back in the epilogue, from the cache.
//
// Measured: 6240 tokens, 40 query heads over 8 KV heads of 128, 25907 keys: 2155-2180 us, 1520-1540 TFLOP/s.  Causal
// chunks of 130 .. 2048 tokens behind up to 12000 keys: 700-721 us, 1330-1370 TFLOP/s.  What bounds it is the chain of
// a row tile (products 1100 clocks, scores ready 300, weights 1150, products awake 300), of which the other row tile's
// products cover 1100.
#include <cuda.h>

#include "attend_join.cuh"

namespace dcp {

namespace {

constexpr int kRows = 128;             // rows of a tile (lanes of tensor memory)
constexpr int kKeys = 128;             // keys of a tile
constexpr int kTileThreads = 640;
constexpr int kSoftWarps = 16;
constexpr int kMaxSplits = 92;         // of an item: what the join's scratch holds
constexpr float kGrow = 8.f;           // log2 of how far a row's maximum may grow before m follows,
constexpr float kFar = 64.f;           // and within one tile before the item is done again
constexpr float kSteep = 0x1p15f;      // sum of half a tile's weights that only a rise within the tile brings about
constexpr float kHuge = 8192.f;        // log2 of a weight whose level, heard in bf16, is too coarse for kFar
constexpr long long kPatience = 4000000000ll;  // limit of every wait, in SM clocks (two seconds)

struct Item {                          // what a CTA works on
  int s, kh, lo, len;                  // sequence, KV head, first row of q, new tokens
  int row0;                            // first (token, head) row
  int kv;                              // cached positions
  int rows[2];                         // rows of each tile
  int t0[2], t1[2];                    // key tiles each row tile sees
  int c0[2], c1[2];                    // cache positions of its first and last row
};

// How key tiles lie over pages: pages of up to 128 positions are gathered, pages_per_tile of them, each `box` rows
// of the tile (a multiple of 8, so that the swizzle's 8-row groups line up; rows past block_size stay masked); larger
// pages are cut into `subs` tiles.
struct Tiling {
  int bs, box, pages, subs;
  int span;                            // positions of every tile where all have as many, else 0
  __device__ __forceinline__ int tile_of(int pos) const {
    if (span == kKeys) return pos / kKeys;
    return subs == 1 ? pos / (pages * bs) : pos / bs * subs + pos % bs / kKeys;
  }
  __device__ __forceinline__ int first(int t) const {
    if (span) return t * span;
    return subs == 1 ? t * pages * bs : t / subs * bs + t % subs * kKeys;
  }
  __device__ __forceinline__ int count(int t) const {
    if (span) return span;
    return subs == 1 ? pages * bs : min(kKeys, bs - t % subs * kKeys);
  }
  __device__ __forceinline__ int columns() const { return pages * box; }  // of a tile, the rest stays empty
  __device__ __forceinline__ bool gaps() const { return subs == 1 && box != bs; }
  // position of column c relative to first(t), -1 where no position stands
  __device__ __forceinline__ int place(int t, int c) const {
    if (subs > 1) return c < count(t) ? c : -1;
    const int g = c / box, r = c - g * box;
    return g < pages && r < bs ? g * bs + r : -1;
  }
};

struct TileParams {
  AttendParams a;
  Tiling tl;
  int splits, q_tiles;
  int whole;                           // items of one CTA each before those that are split
  uint32_t idesc_qk, idesc_pv;
  float* part;                         // [item][split][256][kPartHead + D] partial results
  uint32_t* done;                      // [item] splits finished, 0 between calls
};

// ------------------------------------------------------------------------------------------ PTX
__device__ __forceinline__ void bar_init(uint32_t bar, int count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count));
}
__device__ __forceinline__ void bar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void bar_expect(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ bool bar_try(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok;
}
// False once any wait of the CTA has run out (`dead`).  (The limit goes by the SM's clock: reading the global timer
// between tries cost hundreds of cycles a wait.)
__device__ __forceinline__ bool bar_wait(uint32_t bar, uint32_t parity, volatile int* dead) {
  if (bar_try(bar, parity)) return true;
  const long long start = clock64();
  while (!bar_try(bar, parity)) {
    if (*dead) return false;
    if (clock64() - start > kPatience) {
      *dead = 1;
      return false;
    }
  }
  return true;
}
// The same for a whole warp: its lanes agree.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int* dead) {
  return __all_sync(~0u, bar_wait(bar, parity, dead));
}
// Issued by one lane of a converged warp.
__device__ __forceinline__ void tma_page(uint32_t dst, const CUtensorMap* map, int x, int row, int h, int blk,
                                         uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\t"
      "@q cp.async.bulk.tensor.4d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], "
      "[%6];\n\t}" ::"r"(dst), "l"(map), "r"(x), "r"(row), "r"(h), "r"(blk), "r"(bar)
      : "memory");
}
// The products are issued by the lane with `lead`, inside the instruction sequence: the warp's control flow stays uniform and
// the operands stay in uniform registers (a branch on the lane made eight products take 720 cycles to issue).
// Descriptors share their high word; `a`, `b` are the low words.
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a, uint32_t a_hi, uint32_t b, uint32_t b_hi,
                                       uint32_t idesc, bool add, uint32_t lead) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .b64 x, y;\n\tmov.b64 x, {%1, %2};\n\tmov.b64 y, {%3, %4};\n\t"
      "setp.ne.b32 p, %6, 0;\n\tsetp.ne.b32 q, %7, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %5, p;\n\t}" ::"r"(d), "r"(a), "r"(a_hi), "r"(b), "r"(b_hi),
      "r"(idesc), "r"((uint32_t)add), "r"(lead)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t b_hi, uint32_t idesc, bool add,
                                       uint32_t lead) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .b64 y;\n\tmov.b64 y, {%2, %3};\n\t"
      "setp.ne.b32 p, %5, 0;\n\tsetp.ne.b32 q, %6, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %4, p;\n\t}" ::"r"(d), "r"(a), "r"(b), "r"(b_hi),
      "r"(idesc), "r"((uint32_t)add), "r"(lead)
      : "memory");
}
__device__ __forceinline__ void mma_commit(uint32_t bar, uint32_t lead) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar), "r"(lead)
      : "memory");
}
// 1 in one lane of a converged warp.
__device__ __forceinline__ uint32_t elected() {
  uint32_t x;
  asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\tselp.u32 %0, 1, 0, q;\n\t}" : "=r"(x));
  return x;
}
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// The loaded registers pass through the wait, so that nothing reads them before it.
__device__ __forceinline__ void wait_ld(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]),
                 "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]),
                 "+r"(r[22]), "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]),
                 "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
               :
               : "memory");
}
__device__ __forceinline__ void wait_ld(uint32_t (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
               :
               : "memory");
}
__device__ __forceinline__ void tm_ld32(uint32_t (&r)[32], uint32_t at) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
      "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(at));
}
__device__ __forceinline__ void tm_ld16(uint32_t (&r)[16], uint32_t at) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(at));
}
__device__ __forceinline__ void tm_st16(uint32_t at, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::"r"(
          r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
      "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(at)
      : "memory");
}
// Two fp32 in a register pair.
__device__ __forceinline__ uint64_t pair(float x, float y) {
  uint64_t z;
  asm("mov.b64 %0, {%1, %2};" : "=l"(z) : "f"(x), "f"(y));
  return z;
}
__device__ __forceinline__ void unpair(uint64_t z, float& x, float& y) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(z));
}
__device__ __forceinline__ uint64_t fma2(uint64_t x, uint64_t y, uint64_t z) {
  uint64_t w;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(w) : "l"(x), "l"(y), "l"(z));
  return w;
}
__device__ __forceinline__ uint64_t add2(uint64_t x, uint64_t y) {
  uint64_t w;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(w) : "l"(x), "l"(y));
  return w;
}
__device__ __forceinline__ float max3(float x, uint32_t y, uint32_t z) {
  float w;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(w) : "f"(x), "f"(__uint_as_float(y)), "f"(__uint_as_float(z)));
  return w;
}
// The n lowest bits (n clamped to 0 .. 32).
__device__ __forceinline__ uint32_t low_bits(int n) { return n >= 32 ? ~0u : n <= 0 ? 0u : (1u << n) - 1; }
// x = -inf where keep is 0, in place: a select over 128 registers in two branches costs the compiler copies.
__device__ __forceinline__ void hide_unless(uint32_t& x, uint32_t keep) {
  asm volatile("{\n\t.reg .pred p;\n\tsetp.eq.u32 p, %1, 0;\n\t@p mov.b32 %0, 0xFF800000;\n\t}" : "+r"(x) : "r"(keep));
}

// Shared-memory matrix descriptor, 128-byte swizzle: low word the start and the leading stride in units of 16 bytes,
// high word the other stride, bit 46 = 1 and the swizzle at bits 61-63.
__device__ __forceinline__ uint32_t desc_lo(uint32_t addr, uint32_t leading) {
  return (addr >> 4 & 0x3FFF) | (leading >> 4) << 16;
}
constexpr uint32_t kDescHi = 1024 >> 4 | 1u << 14 | 2u << 29;

template <int HALVES>
struct Shape {
  static constexpr int kD = 64 * HALVES;                 // head dims, padded with zeros
  static constexpr int kHalf = kRows * 128;              // bytes of 128 rows x 64 dims
  static constexpr int kTile = kHalf * HALVES;
  static constexpr int kSlots = HALVES == 2 ? 5 : 10;    // ring of K and V tiles in turn
  static constexpr int kHead = 3 * 1024;                    // barriers and the like, before the tiles
  static constexpr int kSmem = kHead + (2 + kSlots) * kTile;
  static_assert(join_scratch(2 * kRows, kMaxSplits) <= kSmem - kHead, "the join's scratch fits where the tiles were");
};

// Two bf16: bit 15 or 31 where one is an infinity or NaN (its exponent's bits all set carry into it); and the two with
// 0 in such a place.
__device__ __forceinline__ uint32_t specials(uint32_t w) { return (w & 0x7F807F80u) + 0x00800080u; }
__device__ __forceinline__ uint32_t no_special(uint32_t w) {
  if ((w & 0x7F80u) == 0x7F80u) w &= 0xFFFF0000u;
  if ((w & 0x7F800000u) == 0x7F800000u) w &= 0xFFFFu;
  return w;
}

__device__ __forceinline__ bool visible(const AttendParams& a, int kv, int c, int pos) {
  return pos < kv && (!a.causal || pos <= c) && (a.window < 0 || pos >= c - a.window);
}

// The key tiles [x, y) of which every row at cache positions c_lo .. c_hi sees every key.
__device__ __forceinline__ int2 open_tiles(const AttendParams& a, const Tiling& tl, int kv, int c_lo, int c_hi) {
  if (!tl.span) return make_int2(0, 0);
  const int end = a.causal ? min(kv, c_lo + 1) : kv, begin = a.window >= 0 ? max(0, c_hi - a.window) : 0;
  return make_int2((begin + tl.span - 1) / tl.span, max(end, 0) / tl.span);
}
__device__ __forceinline__ bool within(int2 range, int t) { return t >= range.x && t < range.y; }

// A place in the ring and the parity of its fill.
template <int SLOTS>
struct Ring {
  int slot;
  uint32_t phase;
  __device__ __forceinline__ void step() {
    if (++slot == SLOTS) {
      slot = 0;
      phase ^= 1;
    }
  }
  __device__ __forceinline__ void back() {
    if (slot-- == 0) {
      slot = SLOTS - 1;
      phase ^= 1;
    }
  }
};

template <int HALVES>
__global__ void __launch_bounds__(kTileThreads, 1)
    tile_kernel(const __grid_constant__ TileParams p, const __grid_constant__ CUtensorMap map_k,
                const __grid_constant__ CUtensorMap map_v) {
  using Sh = Shape<HALVES>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  struct Head {
    uint64_t bars[2 * Sh::kSlots + 17];
    union {                   // what the two threads of a row tell each other
      __nv_bfloat16 top[2][2][2][kRows];
      float sum[2][2][kRows];
    } swap;
    uint32_t tmem;
    int dead, poison, last, far, steep;
  };
  static_assert(sizeof(Head) <= Sh::kHead, "the head fits before the tiles");
  Head& sh = *reinterpret_cast<Head*>(smem_raw);
  const AttendParams& a = p.a;
  const Tiling tl = p.tl;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  // ---- set-up that needs nothing of the predecessor's
  const uint32_t base = smem_u32(smem_raw) + Sh::kHead;
  const uint32_t q_smem = base, ring = base + 2 * Sh::kTile;
  uint8_t* const gbase = smem_raw + Sh::kHead;
  const uint32_t bars = smem_u32(sh.bars);
  auto full = [&](int i) { return bars + 8 * i; };
  auto empty = [&](int i) { return bars + 8 * (Sh::kSlots + i); };
  auto s_full = [&](int i) { return bars + 8 * (2 * Sh::kSlots + i); };
  auto p_full = [&](int i) { return bars + 8 * (2 * Sh::kSlots + 2 + i); };
  auto finished = [&](int i) { return bars + 8 * (2 * Sh::kSlots + 4 + i); };
  auto pair_met = [&](int i) { return bars + 8 * (2 * Sh::kSlots + 6 + i); };
  const uint32_t q_full = bars + 8 * (2 * Sh::kSlots + 14);
  auto turn = [&](int i) { return bars + 8 * (2 * Sh::kSlots + 15 + i); };
  if (warp == 0) {
    for (int i = lane; i < 2 * Sh::kSlots + 17; i += 32) {
      const int own = i - 2 * Sh::kSlots;  // past the ring: the order of the functions above
      // an empty slot: the products of both row tiles; weights of a row tile: its 8 warps; a pair: its two
      const int count = own < -Sh::kSlots ? 1 : own < 0 ? 2 : own < 2 ? 1 : own < 4 ? kSoftWarps / 2 : own < 6 ? 1
                        : own < 14 ? 2 : own < 15 ? 32 * kSoftWarps : 1;
      bar_init(bars + 8 * i, count);
    }
    if (lane == 0) sh.dead = sh.poison = sh.far = sh.steep = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }

  // ---- the item
  Item it;
  // blocks in the order: row tile, KV head, sequence; the first `whole` items are one CTA's, the others are split
  const int cut = max(0, (int)blockIdx.x - p.whole), item = cut ? p.whole + cut / p.splits : min(blockIdx.x, p.whole);
  const int splits = item < p.whole ? 1 : p.splits, split = item < p.whole ? 0 : cut % p.splits;
  const int qt = p.q_tiles - 1 - item % p.q_tiles;  // the rows that see most keys first
  it.kh = item / p.q_tiles % a.pool.H;
  it.s = item / p.q_tiles / a.pool.H;
  allow_dependents();
  wait_for_predecessor();
  int64_t kv64;
  const bool sound = seq_rows(a.b, it.s, it.lo, it.len) & seq_kv(a.b, tl.bs, a.pool.H, it.s, it.kh, kv64);
  if (!sound) return;
  const int n_rows = it.len * a.G;
  it.row0 = qt * 2 * kRows;
  if (it.row0 >= n_rows) return;
  it.kv = (int)kv64;
  const int32_t* table = a.b.tables + (int64_t)it.s * a.b.table_stride;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int r0 = it.row0 + i * kRows;
    it.rows[i] = max(0, min(kRows, n_rows - r0));
    it.t0[i] = it.t1[i] = 0;
    it.c0[i] = it.kv - it.len + r0 / a.G;
    it.c1[i] = it.kv - it.len + (r0 + max(it.rows[i], 1) - 1) / a.G;
    if (!it.rows[i]) continue;
    const int end = a.causal ? min(it.kv, it.c1[i] + 1) : it.kv;
    const int begin = a.window >= 0 ? max(0, it.c0[i] - a.window) : 0;
    if (begin < end) {
      it.t0[i] = tl.tile_of(begin);
      it.t1[i] = tl.tile_of(end - 1) + 1;
    }
  }
  if (splits > 1) {  // this split's share of the tiles the item's rows see
    const bool one = it.t1[1] <= it.t0[1];
    const int lo = it.t0[0] < it.t1[0] ? it.t0[0] : it.t0[1], hi = one ? it.t1[0] : it.t1[1];
    const int per = (max(hi - lo, 0) + splits - 1) / splits;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      it.t0[i] = max(it.t0[i], lo + split * per);
      it.t1[i] = max(it.t0[i], min(it.t1[i], lo + (split + 1) * per));
    }
  }
  const bool act0 = it.t0[0] < it.t1[0], act1 = it.t0[1] < it.t1[1];
  const int tb = act0 ? it.t0[0] : it.t0[1];                // tiles of either
  const int te = act1 ? max(it.t1[1], act0 ? it.t1[0] : 0) : act0 ? it.t1[0] : tb;
  const int c_lo = it.c0[0], c_hi = it.rows[1] ? it.c1[1] : it.c1[0];

  const int2 open = open_tiles(a, tl, it.kv, c_lo, c_hi);  // tiles without a mask

  // ---- the rest of the set-up
  // rows of the ring no page ever fills: a weight of 0 must meet a value of 0 there
  if (tl.columns() < kKeys) {
    const int rows = kKeys - tl.columns();
    for (int u = threadIdx.x; u < Sh::kSlots * HALVES * rows * 8; u += kTileThreads) {
      const int tile = u / (rows * 8), at = u - tile * rows * 8;
      *reinterpret_cast<uint4*>(gbase + 2 * Sh::kTile + tile * Sh::kHalf + (tl.columns() * 8 + at) * 16) =
          make_uint4(0, 0, 0, 0);
    }
    fence_proxy_async_smem();
  }
  if (warp == kSoftWarps) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&sh.tmem))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = sh.tmem;

  if (warp < kSoftWarps) {
    // ------------------------------------------------------------------------------------ softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 104;");
    const int i = warp >> 3, hf = warp >> 2 & 1, r = threadIdx.x & 127;
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;  // this warp's 32 lanes of tensor memory
    const uint32_t t_s = tmem + lanes + i * kKeys, t_o = tmem + lanes + 256 + i * 128 + hf * (Sh::kD / 2);
    const int D = a.pool.D, rows_i = i ? it.rows[1] : it.rows[0];
    {  // the rows of q into shared memory, zeros past the rows and past D; every load before the first store
      constexpr int kChunks = 8 * HALVES, kStep = 256 / kChunks, kEach = kRows / kStep;
      const int ch = threadIdx.x % kChunks, row_a = (threadIdx.x & 255) / kChunks;
      const int step_t = kStep / a.G, step_g = kStep - step_t * a.G;
      const int Ra = it.row0 + i * kRows + row_a;
      int tk = Ra / a.G, gk = Ra - tk * a.G;
      uint4 x[kEach];
#pragma unroll
      for (int k = 0; k < kEach; ++k) {
        x[k] = make_uint4(0, 0, 0, 0);
        if (row_a + k * kStep < rows_i && ch * 8 < D)
          x[k] = *reinterpret_cast<const uint4*>(a.q + ((int64_t)(it.lo + tk) * a.q_stride +
                                                        (int64_t)(it.kh * a.G + gk) * D + ch * 8) * 2);
        tk += step_t;
        gk += step_g;
        if (gk >= a.G) {
          gk -= a.G;
          ++tk;
        }
      }
#pragma unroll
      for (int k = 0; k < kEach; ++k) {
        const int row = row_a + k * kStep;
        *reinterpret_cast<uint4*>(gbase + i * Sh::kTile + (ch >> 3) * Sh::kHalf + row * 128 +
                                  (((ch & 7) ^ (row & 7)) << 4)) = x[k];
      }
      fence_proxy_async_smem();
      bar_arrive(q_full);
    }
    // The two threads of a row tell each other their maxima through two buffers in turn: neither can overwrite what the
    // other has yet to read.  They are rounded to bf16 (m need only be near the maximum).
    const uint32_t met = pair_met(i * 4 + (warp & 3));
    const int R = it.row0 + i * kRows + r, tok = R / a.G, g = R - tok * a.G;
    const int c = it.kv - it.len + tok;
    const int t0 = i ? it.t0[1] : it.t0[0], t1 = i ? it.t1[1] : it.t1[0];
    const int cmin = i ? it.c0[1] : it.c0[0], cmax = i ? it.c1[1] : it.c1[0];
    const bool mine = r < rows_i;  // rows past the sequence's take part unmasked, and nothing of theirs is kept
    const int seen_end = a.causal && mine ? min(it.kv, c + 1) : it.kv;
    const int seen_begin = a.window >= 0 && mine ? c - a.window : 0;
    const float sc = a.scale_log2, per_log2 = 1.f / sc;
    const int2 mine_open = open_tiles(a, tl, it.kv, cmin, cmax);
    const bool narrow = tl.columns() < kKeys || tl.gaps();
    uint32_t see_open[2];  // columns that stand for keys
#pragma unroll
    for (int e = 0; e < 2; ++e)
      see_open[e] = tl.gaps() ? __ballot_sync(~0u, tl.place(0, 64 * hf + 32 * e + lane) >= 0)
                              : low_bits(tl.columns() - 64 * hf - 32 * e);
    float m = -INFINITY, l = 0.f, seen = -INFINITY;  // seen: the row's maximum so far
    auto move_to = [&](float m2, bool rescale) {     // the row's sums relative to m2
      const float keep = m == m2 ? 1.f : exp2_fast((m - m2) * sc);
      m = m2;
      l *= keep;
      if (!rescale) return;
#pragma unroll 1
      for (int e = 0; e < Sh::kD / 32; ++e) {
        uint32_t o[16];
        tm_ld16(o, t_o + 16 * e);
        wait_ld(o);
#pragma unroll
        for (int u = 0; u < 16; ++u) o[u] = __float_as_uint(__uint_as_float(o[u]) * keep);
        tm_st16(t_o + 16 * e, o);
      }
    };
    uint32_t scored = 0, swaps = 0;  // parities: score tiles received, exchanges received
    bool ok = true, pending = false;
    auto hear = [&] {  // the other thread's maximum of the last exchange
      ok = warp_wait(met, swaps & 1, &sh.dead);
      seen = fmaxf(seen, __bfloat162float(sh.swap.top[i][swaps & 1][hf ^ 1][r]));
      ++swaps;
      pending = false;
    };
    for (bool careful = false;; careful = true) {
      for (int t = t0; t < t1 && ok; ++t) {
        // columns the row sees: in a masked tile those it may see, else those that stand for keys
        uint32_t see[2] = {see_open[0], see_open[1]};
        const bool masked = !within(mine_open, t), hide = masked || narrow;
        if (masked) {
          const int p0 = tl.first(t);
          if (!tl.gaps()) {
            const int hi = min(seen_end - p0, tl.count(t)) - 64 * hf, lo = seen_begin - p0 - 64 * hf;
#pragma unroll
            for (int e = 0; e < 2; ++e) see[e] = low_bits(hi - 32 * e) & ~low_bits(lo - 32 * e);
          } else {
            int page = 64 * hf / tl.box, row = 64 * hf - page * tl.box;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              uint32_t bits = 0;
#pragma unroll 4
              for (int b = 0; b < 32; ++b) {
                const int pos = p0 + page * tl.bs + row;
                bits |= (uint32_t)(pos >= seen_begin && pos < seen_end) << b;
                if (++row == tl.box) {
                  row = 0;
                  ++page;
                }
              }
              see[e] = bits & see_open[e];
            }
          }
        }
        // m follows what the earlier tiles held
        if (pending) hear();
        // before a row has seen a key there is no maximum to go by: the tile's own, of both threads, comes first
        const bool exact = careful || __any_sync(~0u, seen == -INFINITY);
        const bool grown = m == -INFINITY ? seen > m : (seen - m) * sc > kGrow, move = __any_sync(~0u, grown);
        ok = ok && warp_wait(s_full(i), scored & 1, &sh.dead);
        if (!ok) break;
        ++scored;
        fence_after();
        if (move) move_to(grown ? seen : m, t > t0);
        uint32_t x[2][32];  // the row's scores of keys 64 hf .. 64 hf + 63
        auto cover = [&](int e) {
#pragma unroll
          for (int u = 0; u < 32; ++u) hide_unless(x[e][u], see[e] & (1u << u));
        };
        auto tell = [&](float y) {
          const __nv_bfloat16 own = __float2bfloat16_rn(y);
          sh.swap.top[i][swaps & 1][hf][r] = own;
          __syncwarp();
          if (lane == 0) bar_arrive(met);
          pending = true;
          seen = fmaxf(seen, __bfloat162float(own));
        };
        tm_ld32(x[0], t_s + 64 * hf);
        wait_ld(x[0]);
        tm_ld32(x[1], t_s + 64 * hf + 32);
        if (exact) {
          wait_ld(x[1]);
          if (hide) {
            cover(0);
            cover(1);
          }
          float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int u = 0; u < 32; ++u) top[u & 3] = max3(top[u & 3], x[0][u], x[1][u]);
          const float mine_top = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
          if (careful) {
            // both threads here, then the maximum as it is, in the place of both buffers
            if (lane == 0) bar_arrive(met);
            ok = warp_wait(met, swaps++ & 1, &sh.dead);
            sh.swap.sum[i][hf][r] = mine_top;
            __syncwarp();
            if (lane == 0) bar_arrive(met);
            ok = ok && warp_wait(met, swaps++ & 1, &sh.dead);
            seen = fmaxf(seen, fmaxf(mine_top, sh.swap.sum[i][hf ^ 1][r]));
          } else {
            tell(mine_top);
            hear();
            if (fabsf(seen) * sc > kHuge && seen != -INFINITY) sh.far = 1;
          }
          const bool far = m == -INFINITY ? seen > m : (seen - m) * sc > kGrow;
          if (__any_sync(~0u, far)) move_to(far ? seen : m, t > t0);
        } else if (hide) {
          cover(0);
        }
        const float base = m == -INFINITY ? 0.f : m, off = careful ? 0.f : -base * sc;
        if (careful) {  // scores of any size: their distance from the level is scaled, not the level
#pragma unroll
          for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int u = 0; u < 32; ++u) x[e][u] = __float_as_uint(__uint_as_float(x[e][u]) - base);
        }
        const uint64_t sc2 = pair(sc, sc), off2 = pair(off, off);
        uint64_t sum[2] = {0, 0};
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          if (e && !exact) {
            wait_ld(x[1]);
            if (hide) cover(1);
          }
          uint32_t w[16];
#pragma unroll
          for (int u = 0; u < 16; ++u) {
            float y0, y1;
            unpair(fma2(pair(__uint_as_float(x[e][2 * u]), __uint_as_float(x[e][2 * u + 1])), sc2, off2), y0, y1);
            x[e][2 * u] = __float_as_uint(exp2_fast(y0));
            x[e][2 * u + 1] = __float_as_uint(exp2_fast(y1));
          }
#pragma unroll
          for (int u = 0; u < 16; ++u) {
            const float y0 = __uint_as_float(x[e][2 * u]), y1 = __uint_as_float(x[e][2 * u + 1]);
            sum[u & 1] = add2(sum[u & 1], pair(y0, y1));
            w[u] = pack_bf16x2(y0, y1);
          }
          tm_st16(t_s + 64 * hf + 16 * e, w);  // each half over its own scores
        }
        if (masked) {  // guard the values: see the top of the file
          const int n = 2 * (t - tb + (careful ? te - tb : 0)) + 1, slot = n % Sh::kSlots;
          ok = warp_wait(full(slot), (n / Sh::kSlots) & 1, &sh.dead);
          if (!ok) break;
          uint8_t* const v = gbase + (2 + slot) * Sh::kTile + (threadIdx.x & 255) * 16;
          const int p0 = tl.first(t), row_a = (threadIdx.x & 255) >> 3, filled = min(tl.count(t), it.kv - p0);
          uint4 y[4 * HALVES];
          uint32_t special = 0;
#pragma unroll
          for (int k = 0; k < 4 * HALVES; ++k) y[k] = *reinterpret_cast<const uint4*>(v + k * 4096);
#pragma unroll
          for (int k = 0; k < 4 * HALVES; ++k)
            special |= specials(y[k].x) | specials(y[k].y) | specials(y[k].z) | specials(y[k].w);
          special &= 0x80008000u;
          if (special || filled < kKeys || tl.gaps()) {
#pragma unroll
            for (int k = 0; k < 4 * HALVES; ++k) {
              const int row = row_a + 32 * (k & 3);  // of 128 rows of 64 dims, twice
              bool stands = row < filled;
              if (tl.gaps()) {
                const int place = tl.place(t, row);
                stands = place >= 0 && p0 + place < it.kv;
              }
              if (!stands)
                *reinterpret_cast<uint4*>(v + k * 4096) = make_uint4(0, 0, 0, 0);
              else if ((specials(y[k].x) | specials(y[k].y) | specials(y[k].z) | specials(y[k].w)) & 0x80008000u) {
                *reinterpret_cast<uint4*>(v + k * 4096) =
                    make_uint4(no_special(y[k].x), no_special(y[k].y), no_special(y[k].z), no_special(y[k].w));
                sh.poison = 1;
              }
            }
          }
          // also where nothing was left to replace: the other row tile's warps may have done it a moment ago, and this row
          // tile's product must not read what stood there before
          fence_proxy_async_smem();
        }
        wait_st();
        fence_before();
        __syncwarp();
        if (lane == 0) bar_arrive(p_full(i));
        float y0, y1;
        unpair(add2(sum[0], sum[1]), y0, y1);
        y0 += y1;
        l += y0;
        if (!exact) {  // the largest weight is between a 64th of the sum and the sum
          if (y0 > kSteep) sh.steep = 1;
          tell(m + __log2f(y0) * per_log2);
          if ((seen - m) * sc > kFar || (fabsf(seen) * sc > kHuge && seen != -INFINITY)) sh.far = 1;
        }
      }
      if (ok && t0 < t1) {  // the last product
        ok = warp_wait(s_full(i), scored & 1, &sh.dead);
        ++scored;
        fence_after();
      }
      if (ok && pending) hear();
      if (!ok) wait_st();  // weights on their way
      fence_before();
      __syncthreads();
      fence_after();
      if (!careful && sh.steep) {  // weights of a level left far behind, times large values: past fp32 though O / l is not
        bool over = false;
        for (int e = 0; e < Sh::kD / 64 && ok && t0 < t1; ++e) {
          uint32_t o[32];
          tm_ld32(o, t_o + 32 * e);
          wait_ld(o);
#pragma unroll
          for (int u = 0; u < 32; ++u)
            over |= hf * (Sh::kD / 2) + 32 * e + u < D && !(fabsf(__uint_as_float(o[u])) < INFINITY);
        }
        if (over) sh.far = 1;
        fence_before();
        __syncthreads();
        fence_after();
      }
      if (careful || !sh.far) break;
      m = seen = -INFINITY;
      l = 0.f;
    }
    // ---- result of the row
    if (ok) {
      sh.swap.sum[i][hf][r] = l;
      __syncwarp();
      if (lane == 0) bar_arrive(met);
      ok = warp_wait(met, swaps & 1, &sh.dead);
      l += sh.swap.sum[i][hf ^ 1][r];
    }
    if (!ok) set_status(a.b.status, DCP_ETIMEOUT);
    const float inv = l != 0.f ? 1.f / l : 0.f;
    const int64_t row = (int64_t)(it.lo + tok) * a.Hq + it.kh * a.G + g;
    float* part = part_of(p.part, item - p.whole, p.splits, split, 2 * kRows, D, i * kRows + r);
#pragma unroll 1
    for (int e = 0; e < Sh::kD / 64 && ok; ++e) {
      const int d0 = hf * (Sh::kD / 2) + 32 * e;
      uint32_t o[32];
      if (t0 < t1) {
        tm_ld32(o, t_o + 32 * e);
        wait_ld(o);
      } else {
#pragma unroll
        for (int u = 0; u < 32; ++u) o[u] = 0;
      }
      if (sh.poison && mine) {  // infinities and NaN this row sees in the guarded tiles
        for (int t = t0; t < t1; ++t) {
          if (within(open, t)) continue;
          for (int col = 0; col < kKeys; ++col) {
            const int at = tl.place(t, col), pos = tl.first(t) + at;
            if (at < 0 || !visible(a, it.kv, c, pos)) continue;
            const int blk = table[pos / tl.bs];
            if (blk < 0 || blk >= a.pool.n_blocks) continue;
            const __nv_bfloat16* v = (const __nv_bfloat16*)a.pool.v + blk * a.pool.s_block +
                                     (int64_t)it.kh * a.pool.s_head + (int64_t)(pos % tl.bs) * a.pool.s_row;
#pragma unroll
            for (int u = 0; u < 32; ++u) {
              const float y = d0 + u < D ? __bfloat162float(v[d0 + u]) : 0.f;
              if (!isfinite(y)) o[u] = __float_as_uint(__uint_as_float(o[u]) + y);
            }
          }
        }
      }
      if (!mine) continue;
      if (splits > 1) {
#pragma unroll
        for (int u = 0; u < 32; u += 2)
          if (d0 + u < D)
            *reinterpret_cast<float2*>(part + kPartHead + d0 + u) =
                make_float2(__uint_as_float(o[u]), __uint_as_float(o[u + 1]));
      } else {
#pragma unroll
        for (int u = 0; u < 32; u += 8) {
          if (d0 + u >= D) continue;
          uint4 y;
          uint32_t* w = reinterpret_cast<uint32_t*>(&y);
#pragma unroll
          for (int b = 0; b < 4; ++b)
            w[b] = pack_bf16x2(__uint_as_float(o[u + 2 * b]) * inv, __uint_as_float(o[u + 2 * b + 1]) * inv);
          *reinterpret_cast<uint4*>(a.out + (row * D + d0 + u) * 2) = y;
        }
      }
    }
    if (mine && ok && hf == 0) {
      if (splits > 1) {
        part[0] = m;
        part[1] = l;
      } else if (a.lse) {
        a.lse[row] = row_lse(a, m, l);
      }
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
    if (warp >= kSoftWarps + 2) {
      // ---------------------------------------------------------------------------------- pages
      const bool values = warp == kSoftWarps + 3;
      const CUtensorMap* map = values ? &map_v : &map_k;
      const int n_pages = tl.subs == 1 ? tl.pages : 1;
      const uint32_t bytes = (uint32_t)tl.box * 128 * HALVES;
      const int last_page = it.kv > 0 ? (it.kv - 1) / tl.bs : -1;
      // pages some row of the item sees: these must name a block
      const int see_lo = a.window >= 0 ? max(0, c_lo - a.window) : 0, see_hi = a.causal ? min(it.kv, c_hi + 1) : it.kv;
      auto entry = [&](int t) {  // this lane's page of tile t
        const int pg = (tl.subs == 1 ? t * tl.pages : t / tl.subs) + lane;
        if (t >= te || lane >= n_pages || pg > last_page) return 0;
        const int blk = table[pg];
        if (blk >= 0 && blk < a.pool.n_blocks) return blk;
        if (pg * tl.bs < see_hi && (pg + 1) * tl.bs > see_lo) set_status(a.b.status, DCP_EDEVICE);
        return (int)a.pool.n_blocks;  // outside the tensor map: zeros
      };
      bool ok = true;
      Ring<Sh::kSlots> at{values, 0};
      int issued = 0;
      auto in_flight = [&] {  // copies in flight end by themselves: leave when they have (or have been used)
        const long long start = clock64();
        for (int k = 0; k < (Sh::kSlots + 1) / 2 && k < issued; ++k) {
          at.back();
          at.back();
          while (!bar_try(full(at.slot), at.phase) && !bar_try(empty(at.slot), at.phase) &&
                 clock64() - start < kPatience) {
          }
        }
        issued = 0;
      };
      for (bool careful = false;; careful = true) {
        int next = entry(tb);
        for (int t = tb; t < te && ok; ++t) {
          const int blk = next;
          next = entry(t + 1);
          const int row = tl.subs == 1 ? 0 : t % tl.subs * kKeys;
          const int here = min(n_pages, last_page + 1 - (tl.subs == 1 ? t * tl.pages : t / tl.subs));
          ok = warp_wait(empty(at.slot), at.phase ^ 1, &sh.dead);  // at once in the first round
          if (!ok) break;
          const uint32_t dst = ring + at.slot * Sh::kTile, bar = full(at.slot);
          if (lane == 0) bar_expect(bar, here * bytes);
          __syncwarp();
          for (int pg = 0; pg < here; ++pg) {
            const int b = __shfl_sync(~0u, blk, pg);
#pragma unroll
            for (int e = 0; e < HALVES; ++e)
              tma_page(dst + pg * tl.box * 128 + e * Sh::kHalf, map, 64 * e, row, it.kh, b, bar);
          }
          at.step();
          at.step();
          ++issued;
        }
        if (!ok) in_flight();
        __syncthreads();
        if (!careful && sh.steep) __syncthreads();
        if (careful || !sh.far) break;
      }
      if (sh.dead) in_flight();  // another warp gave up
    } else {
      // ---------------------------------------------------------------------------------- matrix products
      const int i = warp - kSoftWarps;
      const int t0 = i ? it.t0[1] : it.t0[0], t1 = i ? it.t1[1] : it.t1[0];
      const uint32_t t_s = tmem + i * kKeys, t_o = tmem + 256 + i * 128, q = desc_lo(q_smem + i * Sh::kTile, 16);
      bool ok = te > tb ? warp_wait(q_full, 0, &sh.dead) : true;
      const uint32_t lead = elected();
      const bool every_dim = a.pool.D > Sh::kD - 16;
      uint32_t weighed = 0, turns = 0;
      bool waited = false;
      auto in_flight = [&] {  // products in flight end by themselves: leave when they have
        if (waited) return;
        waited = true;
        mma_commit(finished(i), lead);
        const long long start = clock64();
        while (!bar_try(finished(i), 0) && clock64() - start < kPatience) {
        }
      };
      Ring<Sh::kSlots> at{0, 0};  // the next fill to be used: the keys of a tile, then its values
      auto scores = [&](int t) {
        if (t < t0 || t >= t1) return;
        const uint32_t k = desc_lo(ring + at.slot * Sh::kTile, 16);
        if (every_dim) {
#pragma unroll
          for (int e = 0; e < 4 * HALVES; ++e) {
            const uint32_t step = ((e >> 2) * Sh::kHalf + (e & 3) * 32) >> 4;
            mma_ss(t_s, q + step, kDescHi, k + step, kDescHi, p.idesc_qk, e > 0, lead);
          }
        } else {
#pragma unroll 1
          for (int e = 0; 16 * e < a.pool.D; ++e) {
            const uint32_t step = ((e >> 2) * Sh::kHalf + (e & 3) * 32) >> 4;
            mma_ss(t_s, q + step, kDescHi, k + step, kDescHi, p.idesc_qk, e > 0, lead);
          }
        }
        mma_commit(s_full(i), lead);
      };
      for (bool careful = false;; careful = true) {
        if (ok && tb < te) {
          ok = warp_wait(full(at.slot), at.phase, &sh.dead);
          if (ok) {
            fence_after();
            scores(tb);
            mma_commit(empty(at.slot), lead);
            at.step();
          }
        }
        for (int t = tb; t < te && ok; ++t) {
          const uint32_t v = desc_lo(ring + at.slot * Sh::kTile, Sh::kHalf), v_empty = empty(at.slot);
          const bool weigh = t >= t0 && t < t1;
          ok = warp_wait(full(at.slot), at.phase, &sh.dead);
          at.step();
          if (ok && t + 1 < te) ok = warp_wait(full(at.slot), at.phase, &sh.dead);
          // The row tiles take turns, values of a tile and scores of the next at a time: one's softmax runs under the
          // other's products.  (Products in the order of their readiness brought both softmaxes into step.)
          ok = ok && warp_wait(turn(i), (turns++ & 1) ^ (i ^ 1), &sh.dead);
          if (ok && weigh) ok = warp_wait(p_full(i), weighed++ & 1, &sh.dead);
          if (!ok) break;
          fence_after();
          if (weigh) {
#pragma unroll
            for (int k = 0; k < kKeys / 16; ++k)
              mma_ts(t_o, t_s + 64 * (k >> 2) + 8 * (k & 3), v + (k * 2048 >> 4), kDescHi, p.idesc_pv,
                     t > t0 || k > 0, lead);
            if (t + 1 == t1) mma_commit(s_full(i), lead);  // the row tile's O is done
          }
          if (t + 1 < te) scores(t + 1);
          if (lead) bar_arrive(turn(i ^ 1));
          __syncwarp();
          mma_commit(v_empty, lead);
          if (t + 1 < te) {
            mma_commit(empty(at.slot), lead);
            at.step();
          }
        }
        if (!ok) {
          in_flight();
          set_status(a.b.status, DCP_ETIMEOUT);
        }
        fence_before();
        __syncthreads();
        fence_after();
        if (!careful && sh.steep) __syncthreads();
        if (careful || !sh.far) break;
      }
      if (sh.dead) in_flight();  // another warp gave up
    }
    __syncwarp();
  }
  // every warp back to the registers it was launched with
  if (warp < kSoftWarps)
    asm volatile("setmaxnreg.dec.sync.aligned.u32 96;");
  else
    asm volatile("setmaxnreg.inc.sync.aligned.u32 96;");
  fence_before();
  __syncthreads();
  fence_after();
  if (warp == kSoftWarps)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));

  // ---- the item's last split joins the parts
  if (splits > 1 && last_of(p.done + item - p.whole, splits, &sh.last))
    join_parts<__nv_bfloat16>(a, part_of(p.part, item - p.whole, p.splits, 0, 2 * kRows, a.pool.D, 0),
                              part_of(p.part, item - p.whole, p.splits, 1, 2 * kRows, a.pool.D, 0),
                              (int64_t)2 * kRows * (kPartHead + a.pool.D), splits, it.rows[0] + it.rows[1], it.row0,
                              it.lo, it.kh, gbase, Sh::kSmem - Sh::kHead);
}

using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                 const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encode_tiled() {
  static const EncodeTiled fn = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult found;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &found) !=
            cudaSuccess || found != cudaDriverEntryPointSuccess)
      f = nullptr;
    return (EncodeTiled)f;
  }();
  return fn;
}

bool encode(CUtensorMap* map, const Pool& c, void* base, int box) {
  const EncodeTiled f = encode_tiled();
  if (!f) return false;
  const cuuint64_t dims[4] = {(cuuint64_t)c.D, (cuuint64_t)c.bs, (cuuint64_t)c.H, (cuuint64_t)c.n_blocks};
  const cuuint64_t strides[3] = {(cuuint64_t)c.s_row * 2, (cuuint64_t)c.s_head * 2, (cuuint64_t)c.s_block * 2};
  const cuuint32_t boxes[4] = {64, (cuuint32_t)box, 1, 1}, ones[4] = {1, 1, 1, 1};
  auto encoded = [&] {
    return f(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, base, dims, strides, boxes, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
             CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
  };
  if (encoded()) return true;
  // a host thread that has made no CUDA call has no current context, which the driver's encoder asks for and does not
  // make; the runtime does, for the thread's device
  int dev = 0;
  return cudaGetDevice(&dev) == cudaSuccess && cudaSetDevice(dev) == cudaSuccess && encoded();
}

// Tiles of 128 x 128 (or 128 x D) in fp32 from bf16: format bits, N / 8 and M / 16.
uint32_t idesc(int n, bool b_by_rows, bool negate) {
  return (1u << 4) | (1u << 7) | (1u << 10) | (negate ? 1u << 13 : 0u) | (b_by_rows ? 1u << 16 : 0u) |
         ((uint32_t)(n / 8) << 17) | ((uint32_t)(kRows / 16) << 24);
}

LaunchCache g_tile_launch[2];

template <int HALVES>
cudaError_t launch(const TileParams& p, const CUtensorMap& k, const CUtensorMap& v, cudaStream_t s) {
  int blocks;
  const cudaError_t e = launch_setup(g_tile_launch[HALVES - 1], tile_kernel<HALVES>, kTileThreads,
                                     Shape<HALVES>::kSmem, &blocks);
  if (e != cudaSuccess) return e;
  const int64_t items = (int64_t)p.q_tiles * p.a.pool.H * p.a.b.n_seqs;
  const int64_t grid = p.whole + (items - p.whole) * p.splits;
  if (grid > INT32_MAX) return cudaErrorInvalidValue;
  return launch_behind(tile_kernel<HALVES>, dim3((unsigned)grid), kTileThreads, Shape<HALVES>::kSmem, s, p, k, v);
}

}  // namespace

TilePlan plan_tiles(const AttendParams& a, int64_t max_kv) {
  TilePlan t;
  t.q_tiles = (int)(((int64_t)a.b.max_q * a.G + 2 * kRows - 1) / (2 * kRows));
  const int64_t items = (int64_t)t.q_tiles * a.pool.H * a.b.n_seqs;
  const int64_t seen = (int64_t)a.window + 2 * kRows / a.G + 2;  // of an item's rows under a window
  if (a.window >= 0 && max_kv > seen) max_kv = seen;
  const int64_t key_tiles = (max_kv + kKeys - 1) / kKeys;
  // Fewer items than SMs: their keys are split so that the SMs have one part each.  Items of equal work (one sequence
  // without a causal mask) in a few rounds: those of the last, incomplete round are split over the SMs it has.  At least
  // 2 key tiles a part.  (us without / with that split: 976 items of 203 key tiles 2114 / 2008, 200 of 203 tiles 615 /
  // 466, 640 of 47 tiles 412 / 402; it loses where the parts are short beside their join: 200 of 13 tiles 58 / 70, 160 of
  // 47 tiles 165 / 179.  From 16 rounds on a round is too little of the whole.)
  const int64_t sms = sm_count(), rounds = items / sms, left = items % sms;
  const bool tail = rounds > 0 && rounds < 16 && left && a.b.n_seqs == 1 && !a.causal;
  int64_t splits = items < sms ? sms / items : tail ? sms / left : 1;
  if (splits > key_tiles / 2) splits = key_tiles / 2;
  if (splits > kMaxSplits) splits = kMaxSplits;
  t.splits = splits < 1 ? 1 : (int)splits;
  t.whole = t.splits == 1 ? items : rounds * sms;
  const size_t cut = (size_t)(items - t.whole);
  t.bytes = cut * t.splits * 2 * kRows * (kPartHead + a.pool.D) * 4;
  return t;
}

cudaError_t launch_attend_tiles(const AttendParams& a, int64_t max_kv, void* ws, cudaStream_t s) {
  const TilePlan t = plan_tiles(a, max_kv);
  if (t.whole > INT32_MAX) return cudaErrorInvalidValue;
  TileParams p{};
  p.a = a;
  const int bs = a.pool.bs;
  p.tl.bs = bs;
  p.tl.box = bs >= kKeys ? kKeys : (bs + 7) / 8 * 8;
  p.tl.pages = kKeys / p.tl.box;
  p.tl.subs = bs > kKeys ? (bs + kKeys - 1) / kKeys : 1;
  p.tl.span = bs % kKeys == 0 ? kKeys : bs < kKeys ? p.tl.pages * bs : 0;
  p.splits = t.splits;
  p.whole = (int)t.whole;
  p.q_tiles = t.q_tiles;
  p.idesc_qk = idesc(kKeys, false, a.scale < 0.f);
  p.idesc_pv = idesc((a.pool.D + 15) / 16 * 16, true, false);
  p.done = done_counters(ws);
  p.part = (float*)((char*)ws + kScratch);
  CUtensorMap mk, mv;
  if (!encode(&mk, a.pool, a.pool.k, p.tl.box) || !encode(&mv, a.pool, a.pool.v, p.tl.box))
    return cudaErrorInvalidValue;
  return a.pool.D <= 64 ? launch<1>(p, mk, mv, s) : launch<2>(p, mk, mv, s);
}

}  // namespace dcp
