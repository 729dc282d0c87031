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

struct AttendParams {
  Pool pool;
  Batch b;
  const char* q;
  char* out;
  float* lse;
  int64_t q_stride;
  int32_t Hq, G;                // query heads, and those of one KV head
  int32_t causal, window;
  float scale;
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

cudaError_t launch_append(const AppendParams& p, cudaStream_t s);
// The attention's workspace: the counters at its start (kDoneItems of them), from kScratch on the parts.
inline uint32_t* done_counters(void* ws) { return (uint32_t*)((char*)ws + sizeof(Ctrl)); }

// How the attention of few rows (or of an fp32 cache) divides its work, and the bytes its parts take.
struct RowPlan {
  int rows, tiles, splits, span, even;  // rows of a CTA, tiles of them
  size_t bytes;
};
bool attend_by_rows(const AttendParams& p);
RowPlan plan_rows(const AttendParams& p, int64_t max_kv);
cudaError_t launch_attend_rows(const AttendParams& p, int64_t max_kv, void* ws, cudaStream_t s);

// The same for the tiled attention.
struct TilePlan {
  int q_tiles, splits;
  int64_t whole;  // items that are not split, the first ones
  size_t bytes;
};
TilePlan plan_tiles(const AttendParams& p, int64_t max_kv);
cudaError_t launch_attend_tiles(const AttendParams& p, int64_t max_kv, void* ws, cudaStream_t s);

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

#endif

}  // namespace dcp
