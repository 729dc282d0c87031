// Internal declarations of the serving operators: parameter blocks and launches of the append, attention and page
// kernels.
#pragma once

#include <utility>

#include "dcp_internal.cuh"

namespace dcp {

// What a kernel knows of the ragged batch (dcp_seq_batch) and of a layer's pages (dcp_kv_pool).
struct Batch {
  int32_t n_seqs, total_q, max_q, kv_per_head;
  int64_t table_stride, kv_add;
  const int32_t* q_start;
  const int32_t* tables;
  const int32_t* kv_len;
  int32_t* status;
};

struct Pool {
  char* k;
  char* v;
  int32_t H, D, dtype, bs;
  int64_t n_blocks, s_block, s_head, s_row;  // strides in elements
};

constexpr int32_t kMaxKv = 1 << 30;  // cached positions of a sequence: differences of positions fit 32 bits

struct AppendParams {
  Pool pool;
  Batch b;
  const char* q;
  const char* k;
  const char* v;
  char* q_out;
  int64_t q_stride, kv_stride;  // elements between tokens
  int32_t Hq;
  const int32_t* positions;
  int32_t half_layout, half;    // pairs at (p, p + half) or (2p, 2p + 1); half = number of pairs
  float amplitude;
  uint64_t turns[DCP_ROPE_MAX_PAIRS];
};

struct NormParams {
  AppendParams a;               // its amplitude is not used
  const char* q_weight;         // nullable: ones
  const char* k_weight;
  int32_t weight_bf16, weight_bytes;  // their type
  int32_t weight_heads;         // weights of each head, or one row for all
  int32_t token_span;           // the mean goes over all heads of a token
  int32_t lanes_log2;           // lanes that hold a head
  int32_t tokens, heads;        // of a CTA at a time: tokens, and heads (all, or those of a piece of one token)
  int32_t block;                // tokens whose places are looked up at a time, a multiple of `tokens`
  int32_t rows_bytes;           // of shared memory that they take
  float eps;
  float inv_head, inv_q, inv_k; // 1 / the dims of a head, of all query heads, of all KV heads
  int32_t first[3];             // first pair of each axis, the number of pairs for those that are not there
  float amplitude[3];
};

// Groups of consecutive sequences that share their first positions (dcp_prefix_groups).
struct Groups {
  int32_t n, max_q;             // 0: none; new tokens of a group at most
  const int32_t* start;
  const int32_t* prefix;
};

// How the groups' prefixes are divided: a slot is a piece of one group's prefix, worked on by a CTA for each tile of the
// group's rows and each KV head, which leaves a part for each of its rows.  The slots go to the groups by their lengths.
struct PrefixPlan {
  float* part;                  // [slot][KV head][tile][row][kPartHead + D]
  int2* table;                  // [group] first slot, number of slots
  int32_t slots, tiles, rows, heads;
  int32_t unit, cap;            // keys of a tile; slots of a group at most
};

struct AttendParams {
  Pool pool;
  Batch b;

  const char* q;
  char* out;
  float* lse;
  int64_t q_stride;
  int32_t Hq, G;                // query heads, and those of one KV head
  int32_t causal, window;
  int32_t sink;                 // under a window: positions below it are seen by every row behind them
  float scale;
  Groups groups;                // where sequences share prefixes
  float scale_log2;             // its size in units of log2 (exponentials are powers of two), in kernels; the sign is the
                                // products' (a scale below 0 negates them: maxima then are of what is exponentiated)
};

struct PageParams {
  char* k;
  char* v;
  int32_t L, bs;
  int64_t n_blocks, page_bytes;
  int32_t* status;
};

#ifdef __CUDACC__
// Whether a row at cache position c sees position pos < kv.
__device__ __forceinline__ bool sees(const AttendParams& a, int c, int pos) {
  return (!a.causal || pos <= c) && (a.window < 0 || pos >= c - a.window || pos < a.sink);
}
#endif

cudaError_t launch_append(const AppendParams& p, cudaStream_t s);
cudaError_t launch_norm_append(const NormParams& p, cudaStream_t s);
// The attention's workspace: the counters at its start (kDoneItems of them), from kScratch on the parts.
inline uint32_t* done_counters(void* ws) { return (uint32_t*)((char*)ws + sizeof(Ctrl)); }

// How the attention of few rows (or of an fp32 cache) divides its work, and the bytes its parts take.
struct RowPlan {
  int rows, tiles, splits, span, even;  // rows of a CTA, tiles of them
  size_t bytes;
};
bool attend_by_rows(const AttendParams& p);
RowPlan plan_rows(const AttendParams& p, int64_t max_kv);
RowPlan plan_rest(const AttendParams& p, int64_t max_kv);  // behind a shared prefix
cudaError_t launch_attend_rows(const AttendParams& p, int64_t max_kv, void* ws, cudaStream_t s);
cudaError_t launch_prefix_rows(const AttendParams& p, const PrefixPlan& pre, cudaStream_t s);
cudaError_t launch_rest_rows(const AttendParams& p, const RowPlan& r, const PrefixPlan& pre, void* ws, cudaStream_t s);
int join_parts_room(const AttendParams& p, const RowPlan& r);  // parts of a row that the join's scratch holds

// The same for the tiled attention.
struct TilePlan {
  int q_tiles, splits;
  int64_t whole;  // items that are not split, the first ones
  size_t bytes;
};
cudaError_t launch_prefix_tiles(const AttendParams& p, const PrefixPlan& pre, cudaStream_t s);
TilePlan plan_tiles(const AttendParams& p, int64_t max_kv);
cudaError_t launch_attend_tiles(const AttendParams& p, int64_t max_kv, void* ws, cudaStream_t s);

// Attention of groups that share a prefix: the bytes of parts it needs, and its launches.
size_t shared_bytes(const AttendParams& p, int64_t max_kv, int64_t max_prefix);
cudaError_t launch_shared(const AttendParams& p, int64_t max_kv, int64_t max_prefix, void* ws, cudaStream_t s);

cudaError_t launch_pages_copy(const PageParams& p, const int32_t* src, const int32_t* dst, int32_t n, cudaStream_t s);
cudaError_t launch_pages_fork(const PageParams& p, const int32_t* tables, const int32_t* len, int32_t n_rows,
                              int32_t stride, const int32_t* parent, const int32_t* shared, const int32_t* reserve,
                              int32_t n_children, const int32_t* ref_in, int32_t* child_tables, int32_t* ref_out,
                              int32_t* ws, cudaStream_t s);
cudaError_t launch_pages_free(const PageParams& p, const int32_t* tables, int32_t n_rows, int32_t stride,
                              const int32_t* ref_in, int32_t* tables_out, int32_t* ref_out, cudaStream_t s);
cudaError_t launch_pages_compact(const PageParams& p, const int32_t* tables, int32_t n_rows, int32_t stride,
                                 const int32_t* ref_in, int32_t* tables_out, int32_t* ref_out, int32_t* n_live,
                                 int32_t* ws, cudaStream_t s);

#ifdef __CUDACC__

// Launch with programmatic stream serialization: the kernel's CTAs may take their places while its predecessor on the
// stream drains.  Every kernel launched so waits for its predecessor before it touches global memory and lets its own
// successor come at once (a call of a few microseconds is mostly launch).
template <typename... P, typename... A>
cudaError_t launch_behind(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t s, A&&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<A>(args)...);
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
__device__ __forceinline__ uint64_t mul2(uint64_t x, uint64_t y) {
  uint64_t w;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(w) : "l"(x), "l"(y));
  return w;
}

// Sequence s of the batch: its first row of q and its length, checked.  False (and the status word) where they are
// inconsistent: the caller then leaves the sequence alone.
__device__ __forceinline__ bool seq_rows(const Batch& b, int s, int& lo, int& n) {
  lo = b.q_start[s];
  const int hi = b.q_start[s + 1];
  n = hi - lo;
  if (lo < 0 || hi < lo || hi > b.total_q || n > b.max_q) {
    set_status(b.status, DCP_EDEVICE);
    return false;
  }
  return true;
}

// Cached positions of sequence s as head h sees them, checked against the table row.
__device__ __forceinline__ bool seq_kv(const Batch& b, int bs, int H, int s, int h, int64_t& kv) {
  kv = (int64_t)b.kv_len[b.kv_per_head ? (int64_t)s * H + h : s] + b.kv_add;
  if (kv < 0 || kv > b.table_stride * bs || kv > kMaxKv) {
    set_status(b.status, DCP_EDEVICE);
    return false;
  }
  return true;
}

// Group g of the batch: its first sequence, rows of q and shared positions, checked.
struct GroupRows {
  int g, s, lo, len, prefix;    // g = -1: no group
};
__device__ __forceinline__ bool group_at(const AttendParams& a, int g, GroupRows& of) {
  of.g = g;
  of.s = a.groups.start[g];
  const int end = a.groups.start[g + 1];
  bool sound = of.s >= 0 && end >= of.s && end <= a.b.n_seqs;
  if (sound) {
    of.lo = a.b.q_start[of.s];
    const int hi = a.b.q_start[end];
    of.len = hi - of.lo;
    of.prefix = a.groups.prefix[g];
    sound = of.lo >= 0 && hi >= of.lo && hi <= a.b.total_q && of.len <= a.groups.max_q && of.prefix >= 0 &&
            of.prefix <= a.b.table_stride * a.pool.bs && of.prefix <= kMaxKv;
  }
  if (!sound) set_status(a.b.status, DCP_EDEVICE);
  return sound;
}

// The group of sequence s, whose `len` new tokens begin at row lo of q and end its `kv` positions; `from` is the first
// position that it holds for itself.  False (and the status word) where the group or its prefix is unsound.
__device__ __forceinline__ bool group_of(const AttendParams& a, int s, int lo, int len, int kv, GroupRows& of,
                                         int& from) {
  int g = 0;  // the first group that begins behind s
  for (int n = a.groups.n; n > 0;) {
    const int half = n / 2;
    if (a.groups.start[g + half] <= s) {
      g += half + 1;
      n -= half + 1;
    } else {
      n = half;
    }
  }
  of = GroupRows{-1, 0, 0, 0, 0};
  from = 0;
  if (g == 0 || s >= a.groups.start[g]) return true;  // start[n] ends the last group
  if (!group_at(a, g - 1, of)) return false;
  from = of.prefix;
  if (of.prefix <= kv - len && lo >= of.lo && lo + len <= of.lo + of.len) return true;
  set_status(a.b.status, DCP_EDEVICE);
  return false;
}

#endif

}  // namespace dcp
