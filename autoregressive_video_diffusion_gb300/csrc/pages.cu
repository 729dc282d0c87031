// Pages of every layer's pool: copying, forking, packing and freeing.
//
// The bookkeeping (which block goes where) is one CTA's work over the reference counts and tables; it leaves a list
// of (source, destination) blocks in the workspace, which the copy kernel behind it on the stream moves.  The bound is
// HBM: packing 2048 blocks of 32 KB, half of them live, in 40 layers takes 309 us (6.3 TB/s); a fork of 32 children
// that copies 32 pages in 40 layers 23 us, of which the bookkeeping is 4.
#include "serve.cuh"

namespace dcp {

namespace {

constexpr int kPlan = 1024;  // threads of a bookkeeping CTA

// A call's part of the workspace, from kScratch on: [0] number of moves, then (from kHead on) the list of (source,
// destination) pairs.
constexpr int kHead = 64;
int32_t* scratch(int32_t* ws) { return ws + kScratch / 4; }

// Exclusive sum of x over the CTA, *total the whole sum.
__device__ int block_scan(int x, int* s_warp, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  int v = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(~0u, v, o);
    if (lane >= o) v += y;
  }
  __syncthreads();
  if (lane == 31) s_warp[warp] = v;
  __syncthreads();
  int w = lane < warps ? s_warp[lane] : 0;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(~0u, w, o);
    if (lane >= o) w += y;
  }
  *total = __shfl_sync(~0u, w, warps - 1);
  const int before = __shfl_sync(~0u, w, warp ? warp - 1 : 0);
  return v - x + (warp ? before : 0);
}

// ref_out = ref_in by the whole CTA, four counts at a time where the arrays allow it.
__device__ __forceinline__ void copy_counts(const int32_t* ref_in, int32_t* ref_out, int64_t n) {
  if (ref_in == ref_out) return;
  int64_t done = 0;
  if ((((uintptr_t)ref_in | (uintptr_t)ref_out) & 15) == 0) {
    done = n & ~(int64_t)3;
#pragma unroll 4
    for (int64_t b = threadIdx.x; b < n / 4; b += kPlan)
      reinterpret_cast<int4*>(ref_out)[b] = reinterpret_cast<const int4*>(ref_in)[b];
  }
  for (int64_t b = done + threadIdx.x; b < n; b += kPlan) ref_out[b] = ref_in[b];
}

// Moves the listed pages: an item is a piece of one page of one layer and tensor, taken in turn by the CTAs.  Each
// thread has kMoves vectors in flight; nothing that is moved is read again, so it passes the caches by.
constexpr int kMoves = 8;
constexpr int kPiece = kThreads * kMoves * 16;

__global__ void __launch_bounds__(kThreads) move_kernel(PageParams p, const int32_t* src, const int32_t* dst,
                                                        int step, const int32_t* count, int32_t n) {
  allow_dependents();
  wait_for_predecessor();
  const int pieces = (int)((p.page_bytes + kPiece - 1) / kPiece), per_pair = 2 * p.L * pieces;
  const int64_t items = (int64_t)(count ? *count : n) * per_pair;
  for (int64_t it = blockIdx.x; it < items; it += gridDim.x) {
    const int64_t pair = it / per_pair;
    const int rest = (int)(it - pair * per_pair), layer = rest / (2 * pieces), part = rest - layer * 2 * pieces;
    const int64_t a = src[pair * step], b = dst[pair * step];
    if (a < 0 || b < 0 || a >= p.n_blocks || b >= p.n_blocks) {
      if (threadIdx.x == 0) set_status(p.status, DCP_EDEVICE);
      continue;
    }
    char* const base = (part >= pieces ? p.v : p.k) + layer * p.n_blocks * p.page_bytes;
    const int64_t at = (int64_t)(part >= pieces ? part - pieces : part) * kPiece + threadIdx.x * 16;
    const char* from = base + a * p.page_bytes;
    char* to = base + b * p.page_bytes;
    Vec<4> x[kMoves];
#pragma unroll
    for (int k = 0; k < kMoves; ++k)
      if (at + k * kThreads * 16 < p.page_bytes) ld_stream(x[k], from + at + k * kThreads * 16);
#pragma unroll
    for (int k = 0; k < kMoves; ++k)
      if (at + k * kThreads * 16 < p.page_bytes) st_stream(to + at + k * kThreads * 16, x[k]);
  }
}

__global__ void __launch_bounds__(kPlan) fork_kernel(PageParams p, const int32_t* tables, const int32_t* len,
                                                     int32_t n_rows, int32_t stride, const int32_t* parent,
                                                     const int32_t* shared, const int32_t* reserve,
                                                     int32_t n_children, const int32_t* ref_in, int32_t* child,
                                                     int32_t* ref_out, int32_t* ws) {
  allow_dependents();
  wait_for_predecessor();
  __shared__ int s_warp[32];
  __shared__ int s_bad, s_moves;
  int2* moves = (int2*)(ws + kHead);
  int32_t* first = ws + kHead + 2 * (int64_t)n_children * stride;  // fresh blocks before child c
  int32_t* fresh = first + n_children;                             // the lowest free blocks
  if (threadIdx.x == 0) s_bad = s_moves = 0;
  __syncthreads();
  // every child's shared, copied and reserved pages
  int need = 0;
  for (int c0 = 0; c0 < n_children; c0 += kPlan) {
    const int c = c0 + threadIdx.x;
    int want = 0;
    if (c < n_children) {
      const int r = parent[c];
      if (r < 0 || r >= n_rows) {
        s_bad = 1;
      } else {
        const int64_t n = len[r], np = (n + p.bs - 1) / p.bs;
        const int64_t more = reserve ? ((int64_t)reserve[c] + p.bs - 1) / p.bs : 0;
        const int64_t total = max(np, more), ns = shared ? shared[c] : n / p.bs;
        if (n < 0 || total > stride || ns < 0 || ns > np) {
          s_bad = 1;
        } else {
          want = (int)(total - ns);
        }
      }
    }
    int sum;
    const int at = block_scan(want, s_warp, &sum) + need;
    if (c < n_children) first[c] = at;
    need += sum;
  }
  // every page of a parent names a live block
  for (int64_t i = threadIdx.x; i < (int64_t)n_children * stride; i += kPlan) {
    const int c = (int)(i / stride), j = (int)(i - (int64_t)c * stride), r = parent[c];
    if (r < 0 || r >= n_rows || (int64_t)j * p.bs >= len[r]) continue;
    const int b = tables[(int64_t)r * stride + j];
    if (b < 0 || b >= p.n_blocks || ref_in[b] <= 0) s_bad = 1;
  }
  // the lowest free blocks, as many as are needed
  int found = 0;
  for (int64_t b0 = 0; b0 < p.n_blocks && found < need; b0 += kPlan) {
    const int64_t b = b0 + threadIdx.x;
    const int is_free = b < p.n_blocks && ref_in[b] == 0;
    int sum;
    const int at = block_scan(is_free, s_warp, &sum) + found;
    if (is_free && at < need) fresh[at] = (int)b;
    found += sum;
  }
  __syncthreads();
  copy_counts(ref_in, ref_out, p.n_blocks);
  const bool bad = s_bad, full = found < need;
  __syncthreads();
  if (bad || full) {
    for (int64_t i = threadIdx.x; i < (int64_t)n_children * stride; i += kPlan) child[i] = -1;
    if (threadIdx.x == 0) {
      ws[0] = 0;
      set_status(p.status, bad ? DCP_EDEVICE : DCP_ECAPACITY);
    }
    return;
  }
  for (int64_t i = threadIdx.x; i < (int64_t)n_children * stride; i += kPlan) {
    const int c = (int)(i / stride), j = (int)(i % stride), r = parent[c];
    const int64_t n = len[r], np = (n + p.bs - 1) / p.bs;
    const int64_t ns = shared ? shared[c] : n / p.bs;
    const int64_t total = max(np, reserve ? ((int64_t)reserve[c] + p.bs - 1) / p.bs : (int64_t)0);
    int to = -1;
    if (j < ns) {
      to = tables[(int64_t)r * stride + j];
      atomicAdd(ref_out + to, 1);
    } else if (j < total) {
      to = fresh[first[c] + j - ns];
      ref_out[to] = 1;
      if (j < np) moves[atomicAdd(&s_moves, 1)] = make_int2(tables[(int64_t)r * stride + j], to);
    }
    child[i] = to;
  }
  __syncthreads();
  if (threadIdx.x == 0) ws[0] = s_moves;
}

__global__ void __launch_bounds__(kPlan) free_kernel(PageParams p, const int32_t* tables, int64_t n,
                                                     const int32_t* ref_in, int32_t* tables_out, int32_t* ref_out) {
  allow_dependents();
  wait_for_predecessor();
  copy_counts(ref_in, ref_out, p.n_blocks);
  __syncthreads();
  // four entries a thread at a time: their reads, then their counts, in flight together
  for (int64_t i0 = threadIdx.x; i0 < n; i0 += 4 * kPlan) {
    int b[4], left[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int64_t i = i0 + k * kPlan;
      b[k] = i < n ? tables[i] : -1;
      if (i < n) tables_out[i] = -1;
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) left[k] = b[k] >= 0 && b[k] < p.n_blocks ? atomicSub(ref_out + b[k], 1) : 1;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (b[k] >= p.n_blocks || left[k] <= 0) set_status(p.status, DCP_EDEVICE);
      if (left[k] <= 0) atomicAdd(ref_out + b[k], 1);
    }
  }
}

constexpr int kTaken = INT32_MIN;

__global__ void __launch_bounds__(kPlan) compact_kernel(PageParams p, const int32_t* tables, int64_t n,
                                                        const int32_t* ref_in, int32_t* tables_out, int32_t* ref_out,
                                                        int32_t* n_live, int32_t* ws) {
  allow_dependents();
  wait_for_predecessor();
  __shared__ int s_warp[32];
  int2* moves = (int2*)(ws + kHead);
  // where every block goes: itself or its hole; of a free block -1 - itself, or kTaken where a page moves into it
  int32_t* to = ws + kHead + 2 * p.n_blocks;
  int mine = 0, live;
  for (int64_t b = threadIdx.x; b < p.n_blocks; b += kPlan) mine += ref_in[b] > 0;
  block_scan(mine, s_warp, &live);
  int holes = 0, movers = 0;
  for (int64_t b0 = 0; b0 < p.n_blocks; b0 += kPlan) {
    const int64_t b = b0 + threadIdx.x;
    const int r = b < p.n_blocks ? ref_in[b] : 0;
    const int hole = b < live && r <= 0, mover = b >= live && r > 0;
    int sum;
    const int h = block_scan(hole, s_warp, &sum) + holes;
    holes += sum;
    const int m = block_scan(mover, s_warp, &sum) + movers;
    movers += sum;
    if (hole) moves[h].y = (int)b;
    if (mover) moves[m].x = (int)b;
    if (b < p.n_blocks) {
      to[b] = r > 0 ? (int)b : -1 - (int)b;
      ref_out[b] = r;
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < movers; i += kPlan) {
    const int2 m = moves[i];
    to[m.x] = m.y;
    to[m.y] = kTaken;
    ref_out[m.y] = ref_out[m.x];
    ref_out[m.x] = 0;
  }
  __syncthreads();
  for (int64_t i = threadIdx.x; i < n; i += kPlan) {
    const int b = tables[i];
    int now = b < 0 ? -1 : b;
    if (b >= p.n_blocks) {
      set_status(p.status, DCP_EDEVICE);
    } else if (b >= 0) {
      now = to[b];
      if (now < 0) {  // a free block: nothing of the row's stands there
        set_status(p.status, DCP_EDEVICE);
        now = now == kTaken ? -1 : b;
      }
    }
    tables_out[i] = now;
  }
  if (threadIdx.x == 0) {
    ws[0] = movers;
    if (n_live) *n_live = live;
  }
}

// Five CTAs an SM are what fits.  (Copying 682 pages of 32 KB in 40 layers with 3 / 4 / 5 / 6 / 8 / 10 an SM: 558 / 564 /
// 568 / 625 / 548 / 562 us; 5461 pages of 2 KB in 2 layers 54 / 48 / 47 / 54 / 46 / 46.)
cudaError_t move(const PageParams& p, const int32_t* src, const int32_t* dst, int step, const int32_t* count, int32_t n,
                 cudaStream_t s) {
  const int64_t pieces = (p.page_bytes + kPiece - 1) / kPiece, most = (int64_t)sm_count() * 5;
  const int64_t items = (int64_t)n * p.L * 2 * pieces;
  return launch_behind(move_kernel, dim3((unsigned)(count || items > most ? most : items)), kThreads, 0, s, p, src, dst,
                       step, count, n);
}

cudaError_t move_listed(const PageParams& p, int32_t* ws, cudaStream_t s) {
  return move(p, ws + kHead, ws + kHead + 1, 2, ws, 0, s);
}

}  // namespace

cudaError_t launch_pages_copy(const PageParams& p, const int32_t* src, const int32_t* dst, int32_t n, cudaStream_t s) {
  return move(p, src, dst, 1, nullptr, n, s);
}

cudaError_t launch_pages_fork(const PageParams& p, const int32_t* tables, const int32_t* len, int32_t n_rows,
                              int32_t stride, const int32_t* parent, const int32_t* shared, const int32_t* reserve,
                              int32_t n_children, const int32_t* ref_in, int32_t* child_tables, int32_t* ref_out,
                              int32_t* ws, cudaStream_t s) {
  ws = scratch(ws);
  const cudaError_t e = launch_behind(fork_kernel, dim3(1), kPlan, 0, s, p, tables, len, n_rows, stride, parent, shared,
                                      reserve, n_children, ref_in, child_tables, ref_out, ws);
  return e != cudaSuccess ? e : move_listed(p, ws, s);
}

cudaError_t launch_pages_free(const PageParams& p, const int32_t* tables, int32_t n_rows, int32_t stride,
                              const int32_t* ref_in, int32_t* tables_out, int32_t* ref_out, cudaStream_t s) {
  return launch_behind(free_kernel, dim3(1), kPlan, 0, s, p, tables, (int64_t)n_rows * stride, ref_in, tables_out,
                       ref_out);
}

cudaError_t launch_pages_compact(const PageParams& p, const int32_t* tables, int32_t n_rows, int32_t stride,
                                 const int32_t* ref_in, int32_t* tables_out, int32_t* ref_out, int32_t* n_live,
                                 int32_t* ws, cudaStream_t s) {
  ws = scratch(ws);
  const cudaError_t e = launch_behind(compact_kernel, dim3(1), kPlan, 0, s, p, tables, (int64_t)n_rows * stride, ref_in,
                                      tables_out, ref_out, n_live, ws);
  return e != cudaSuccess ? e : move_listed(p, ws, s);
}

}  // namespace dcp
