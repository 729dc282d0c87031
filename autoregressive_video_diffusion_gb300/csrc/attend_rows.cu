// The attention of few rows and of fp32 caches: how its work is divided, and its plain form (a causal mask, a window).
#include <algorithm>

#include "attend_rows.cuh"

namespace dcp {

namespace {

// Rows of one CTA: all of a KV head's rows where they fit 16, and 16 too where up to 64 meet few keys and the CTAs
// still run in one round: reading the keys again costs nothing then (in a graph, 28 rows of 12 sequences over a few
// keys 8.7 instead of 9.9 us, 40 fp32 rows of 4 sequences 9.4 instead of 12.0; 58 sequences of 28 rows in two rounds
// 15.9 instead of 10.9).  Else 64, and 128 for fp32 (8 warps share the taking apart of a tile).
int rows_a_cta(const AttendParams& a, bool few) {
  const int64_t rows = (int64_t)a.b.max_q * a.G;
  if (rows <= 16) return 16;
  if (few && rows <= 64 && (rows + 15) / 16 * a.pool.H * a.b.n_seqs <= 2 * sm_count()) return 16;
  return a.pool.dtype == DCP_BF16 ? 64 : 128;
}

}  // namespace

cudaError_t launch_rows_plain(const RowParams& p, int rows, cudaStream_t s) { return launch_form<kPlain>(p, rows, s); }

bool attend_by_rows(const AttendParams& a) {
  return a.pool.dtype == DCP_F32 || (int64_t)a.b.max_q * a.G <= 64;
}

RowPlan plan_rows(const AttendParams& a, int64_t max_kv) {
  RowPlan r;
  const int keys = a.pool.dtype == DCP_BF16 ? 64 : 32;
  const int64_t seen = (int64_t)a.window + a.sink + 128 / a.G + 2;  // of a tile's rows under a window
  if (a.window >= 0 && max_kv > seen) max_kv = seen;
  // So few keys that an item in one go is over before parts of it would be joined (11 sequences' tokens over 10 keys in
  // a graph: 6.3 us, against 12.4 in shares of two tiles).
  const bool few = max_kv <= 6 * keys;
  const int per = r.rows = rows_a_cta(a, few);
  r.tiles = (int)(((int64_t)a.b.max_q * a.G + per - 1) / per);
  const int64_t items = (int64_t)r.tiles * a.pool.H * a.b.n_seqs;
  // Items that may differ in length: two CTAs of an SM at a time, each with the same number of key tiles (48 sequences
  // of 200 .. 16000 positions: 324 us, against 354 in pieces of a fixed span; items alike are cut as well by a span,
  // without the sums: one token over 1531 positions 12.3 us, against 14.0).
  r.even = (int64_t)a.b.max_q * a.G <= 16 && items <= (a.sink ? kEvenItemsSink : kEvenItems) &&
           (a.b.n_seqs > 1 || a.b.kv_per_head) && !few;
  if (r.even) {
    r.splits = 2 * (sm_count() < kMaxSms ? sm_count() : kMaxSms);
    r.span = 0;
    r.bytes = (size_t)r.splits * 2 * 16 * (kPartHead + a.pool.D) * 4;
    return r;
  }
  // Two CTAs of an SM at a time: one round of pieces for a few sequences, four rounds of shorter ones where their lengths
  // may differ (8 sequences on) or a causal mask makes tiles of rows differ (128 rows a CTA).  Measured, us with 1 / 2 /
  // 4 / 6 / 8 rounds: fp32, heads of 64, 100 .. 513 new tokens, 3 sequences 262 / 210 / 183 / 187 / 195, 8 sequences 529 /
  // 453 / 373 / 369 / 350, one alone 111 / 128 / 136 / 137 / 137; drafts of 40 rows over 200 .. 16000 keys, 4 sequences
  // 109 / 115 / 134 / 148 / 180, 8 sequences 167 / 160 / 158 / 183 / 195, 48 sequences 574 / 605 / 565 / 586 / 610, 100
  // sequences 1055 / 1055 / 1033 / 982 / 980; 16 sequences alike 122 / 140 / 142 / 165 / 164.  No piece under two tiles (or
  // four, in several rounds), at most kMaxSplits of an item.
  const int64_t slots = 2 * sm_count(), rounds = a.b.n_seqs >= 8 || per == 128 ? 4 : 1;
  int64_t span = (max_kv * items + slots * rounds - 1) / (slots * rounds);
  const int64_t least = (rounds > 1 ? 4 : 2) * keys;
  if (span < least) span = least;
  if (span < (max_kv + kMaxSplits - 1) / kMaxSplits) span = (max_kv + kMaxSplits - 1) / kMaxSplits;
  span = (span + keys - 1) / keys * keys;
  int64_t splits = (max_kv + span - 1) / span;
  if (splits > 65535 / a.b.n_seqs) splits = 65535 / a.b.n_seqs;
  r.splits = splits < 1 || few || items > kDoneItems ? 1 : (int)splits;
  r.span = (int)(span < kMaxKv ? span : kMaxKv);
  r.bytes = r.splits > 1 ? (size_t)items * r.splits * per * (kPartHead + a.pool.D) * 4 : 0;
  return r;
}

// Behind a shared prefix every piece of an item is joined, at some 10 us beside 0.6 us a tile: an item is one CTA's unless
// that leaves CTAs idle or its keys are many.
RowPlan plan_rest(const AttendParams& a, int64_t max_kv) {
  RowPlan r = plan_rows(a, max_kv);
  const int keys = a.pool.dtype == DCP_BF16 ? 64 : 32;
  if (r.splits <= 1 || max_kv > 16 * keys) return r;
  const int64_t items = (int64_t)r.tiles * a.pool.H * a.b.n_seqs;
  r.even = 0;
  const int64_t splits = std::min<int64_t>(2 * sm_count() / items, max_kv / (4 * keys));
  r.splits = items > kDoneItems || splits < 1 ? 1 : (int)splits;
  r.span = (int)((max_kv + r.splits - 1) / r.splits + keys - 1) / keys * keys;
  r.bytes = (size_t)items * r.splits * r.rows * (kPartHead + a.pool.D) * 4;
  return r;
}

namespace {

RowParams row_params(const AttendParams& a, const RowPlan& r, void* ws) {
  RowParams p{};
  p.a = a;
  p.even = r.even;
  p.splits = r.splits;
  p.span = r.span;
  p.row_tiles = r.tiles;
  p.flip = a.scale < 0.f ? 0x80000000u : 0u;
  p.done = done_counters(ws);
  p.part = (float*)((char*)ws + kScratch);
  return p;
}

}  // namespace

int join_parts_room(const AttendParams& a, const RowPlan& r) {
  const bool wide = a.pool.D > 64;
  if (a.pool.dtype == DCP_BF16) {
    if (r.rows == 16) return wide ? Rows<__nv_bfloat16, 128, 1>::kRoom : Rows<__nv_bfloat16, 64, 1>::kRoom;
    return wide ? Rows<__nv_bfloat16, 128, 4>::kRoom : Rows<__nv_bfloat16, 64, 4>::kRoom;
  }
  if (r.rows == 16) return wide ? Rows<float, 128, 1>::kRoom : Rows<float, 64, 1>::kRoom;
  return wide ? Rows<float, 128, 8>::kRoom : Rows<float, 64, 8>::kRoom;
}

cudaError_t launch_prefix_rows(const AttendParams& a, const PrefixPlan& pre, cudaStream_t s) {
  RowParams p = row_params(a, RowPlan{}, nullptr);
  p.pre = pre;
  return launch_rows_prefix(p, pre.rows, s);
}

cudaError_t launch_rest_rows(const AttendParams& a, const RowPlan& r, const PrefixPlan& pre, void* ws, cudaStream_t s) {
  RowParams p = row_params(a, r, ws);
  p.pre = pre;
  return launch_rows_rest(p, r.rows, s);
}

cudaError_t launch_attend_rows(const AttendParams& a, int64_t max_kv, void* ws, cudaStream_t s) {
  const RowPlan r = plan_rows(a, max_kv);
  const RowParams p = row_params(a, r, ws);
  return a.sink ? launch_rows_sink(p, r.rows, s) : launch_rows_plain(p, r.rows, s);
}

}  // namespace dcp
