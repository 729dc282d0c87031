// Attention of sequences that share their first positions: the prefix is read once for all rows of a group, what a sequence
// holds behind it for itself, and a row's result is the sum of both parts.
//
//   out = sum_p e^(m_p - m) o_p / sum_p e^(m_p - m) l_p  over the row's parts p (maximum m_p, sum of weights l_p, of
//   weighted values o_p), m the largest m_p
//
// Two launches.  The first takes the rows of all sequences of a group as one sequence's against the prefix, which hides
// nothing from any of them: few rows in warp-level products, more in tiles on the tensor cores, the prefixes cut by their
// lengths so that every SM has its piece.  The second is the attention of few rows against each sequence's own keys; the CTA
// that joins an item's parts joins those of the prefix with them.
// The bound is HBM: the prefix once, the rest once.  Measured: 32 branches' tokens, 40 query heads over 8 KV heads of 128,
// 24960 shared and 20 .. 700 further positions (162 MB, floor 24 us) 78-81 us, prefix 38 and rest 34 of it, each with some
// 15 us to begin and end (the code is not in the instruction cache when the launches alternate); over 24000 shared positions
// 71 us, one by one 452.  6 groups
// of 1 .. 12 branches with drafts of 1 .. 5 tokens, 32 heads over 8, 500 .. 16000 shared positions: 140 us.
#include <algorithm>

#include "serve.cuh"

namespace dcp {

namespace {

// Sequences of many rows fill the products by themselves: reading the prefix again from the L2 costs them nothing.  Under a
// window the rows see little of it.
bool few_rows(const AttendParams& a) {
  return a.window < 0 && (int64_t)a.b.max_q * a.G <= (a.pool.dtype == DCP_BF16 ? 64 : 128);
}

// What is not read again has to be worth a second launch and the exchange of parts.
// (Measured, us alone / shared, one token a branch: bf16, 40 query heads over 8 KV heads of 128, saving 43 MB 23 / 26, 92 MB
// 32 / 31, 246 MB 55 / 35; over 40 KV heads 31 MB 24 / 24, 82 MB 39 / 37; fp32, 8 heads of 64, 18 MB 25 / 32, 31 MB 38 / 33.)
bool pays(const AttendParams& a, int64_t max_prefix) {
  const double row = 2.0 * a.pool.H * a.pool.D * (a.pool.dtype == DCP_BF16 ? 2 : 4);
  return few_rows(a) && (double)(a.b.n_seqs - a.groups.n) * max_prefix * row >= (a.pool.dtype == DCP_BF16 ? 80e6 : 30e6);
}

struct SharedPlan {
  RowPlan rest;
  PrefixPlan pre;
  bool tiled;
  size_t rest_bytes, part_bytes;
};

constexpr int kPartWidth = 4;  // a part's maximum and sum, before its values

SharedPlan plan_shared(const AttendParams& a, int64_t max_kv, int64_t max_prefix) {
  SharedPlan t{};
  const int64_t rows = (int64_t)a.groups.max_q * a.G;
  const bool half = a.pool.dtype == DCP_BF16;
  // Up to 64 rows of a KV head in warp-level products, more in tiles (40 rows of 8 KV heads over 12000 / 24000 positions,
  // the whole call: 38 / 55 us, in tiles 38 / 61; 60 rows 40 / 56 and 39 / 62).
  t.tiled = half && rows > 64;
  t.pre.rows = t.tiled ? 256 : rows <= 16 ? 16 : half ? 64 : 128;
  t.pre.tiles = (int)((rows + t.pre.rows - 1) / t.pre.rows);
  t.pre.heads = a.pool.H;
  t.rest = plan_rest(a, std::max<int64_t>(max_kv - max_prefix, 1));
  t.rest_bytes = t.rest.bytes;
  if (!t.rest_bytes)  // items in one go leave a part too
    t.rest_bytes = (size_t)t.rest.tiles * a.pool.H * a.b.n_seqs * t.rest.rows * (kPartWidth + a.pool.D) * 4;
  // A piece for each CTA that an SM holds; where there are more groups than that, one for each and as many again to
  // spare for the longer ones, until the rounds of CTAs even out by themselves.
  const int64_t ctas = t.tiled ? sm_count() : 2 * sm_count(), room = ctas / ((int64_t)t.pre.tiles * a.pool.H);
  const int64_t n = a.groups.n;
  t.pre.slots = (int)std::min<int64_t>(65535, std::max(room, n + std::min(n, 2 * room + 1)));
  t.pre.unit = t.tiled ? 128 : half ? 64 : 32;
  t.pre.cap = join_parts_room(a, t.rest) - (t.rest.even ? t.rest.splits : std::max(t.rest.splits, 1));
  t.part_bytes = (size_t)t.pre.slots * t.pre.heads * t.pre.tiles * t.pre.rows * (kPartWidth + a.pool.D) * 4;
  return t;
}

size_t up(size_t x) { return (x + 255) / 256 * 256; }

// The groups of a call that does without them are checked all the same.
__global__ void check_kernel(const __grid_constant__ AttendParams a) {
  allow_dependents();
  wait_for_predecessor();
  for (int g = blockIdx.x * blockDim.x + threadIdx.x; g < a.groups.n; g += gridDim.x * blockDim.x) {
    GroupRows of;
    group_at(a, g, of);
  }
  const int heads = a.b.kv_per_head ? a.pool.H : 1;
  const int64_t n = (int64_t)a.b.n_seqs * heads;
  for (int64_t i = blockIdx.x * blockDim.x + threadIdx.x; i < n; i += gridDim.x * blockDim.x) {
    const int s = (int)(i / heads);
    int lo, len, from;
    int64_t kv;
    GroupRows of;
    if ((seq_rows(a.b, s, lo, len) & seq_kv(a.b, a.pool.bs, a.pool.H, s, (int)(i % heads), kv)) && len)
      group_of(a, s, lo, len, (int)kv, of, from);
  }
}

}  // namespace

size_t shared_bytes(const AttendParams& a, int64_t max_kv, int64_t max_prefix) {
  if (!pays(a, max_prefix)) return attend_by_rows(a) ? plan_rows(a, max_kv).bytes : plan_tiles(a, max_kv).bytes;
  const SharedPlan t = plan_shared(a, max_kv, max_prefix);
  return up(t.rest_bytes) + up(t.part_bytes) + up((size_t)a.groups.n * sizeof(int2));
}

cudaError_t launch_shared(const AttendParams& a, int64_t max_kv, int64_t max_prefix, void* ws, cudaStream_t s) {
  if (!pays(a, max_prefix)) {
    if (few_rows(a)) return launch_rest_rows(a, plan_rows(a, max_kv), PrefixPlan{}, ws, s);
    const cudaError_t e = launch_behind(check_kernel, dim3(8), 256, 0, s, a);
    if (e != cudaSuccess) return e;
    return attend_by_rows(a) ? launch_attend_rows(a, max_kv, ws, s) : launch_attend_tiles(a, max_kv, ws, s);
  }
  SharedPlan t = plan_shared(a, max_kv, max_prefix);
  char* const at = (char*)ws + kScratch + up(t.rest_bytes);
  t.pre.part = (float*)at;
  t.pre.table = (int2*)(at + up(t.part_bytes));
  AttendParams whole = a;  // no row of a group lies before the end of its prefix
  whole.causal = 0;
  const cudaError_t e = t.tiled ? launch_prefix_tiles(whole, t.pre, s) : launch_prefix_rows(whole, t.pre, s);
  return e != cudaSuccess ? e : launch_rest_rows(a, t.rest, t.pre, ws, s);
}

}  // namespace dcp
