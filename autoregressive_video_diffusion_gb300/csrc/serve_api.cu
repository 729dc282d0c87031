// Host side of the serving operators: argument checks, the rotary plan and the launches.
// The entry points and their contracts are documented in include/dcp.h.
#include <cfloat>
#include <cmath>
#include <initializer_list>

#include "serve.cuh"

using namespace dcp;

namespace {

// ------------------------------------------------------------------------------------------ frequencies
// A phase of 2^-30 turns at positions up to 2^31 takes theta / (2 pi) to 2^-62, more than a double holds.  So the plan
// computes in unevaluated sums of two doubles (Dekker 1971, Knuth's exact sum; products through fma), about 100 bits.
struct Two {
  double hi, lo;
};

Two quick_sum(double a, double b) {  // |a| >= |b|
  const double s = a + b;
  return {s, b - (s - a)};
}
Two exact_sum(double a, double b) {
  const double s = a + b, t = s - a;
  return {s, (a - (s - t)) + (b - t)};
}
Two exact_product(double a, double b) {
  const double p = a * b;
  return {p, std::fma(a, b, -p)};
}
Two operator+(Two x, Two y) {
  const Two s = exact_sum(x.hi, y.hi), t = exact_sum(x.lo, y.lo);
  const Two u = quick_sum(s.hi, s.lo + t.hi);
  return quick_sum(u.hi, u.lo + t.lo);
}
Two operator-(Two x) { return {-x.hi, -x.lo}; }
Two operator*(Two x, Two y) {
  const Two p = exact_product(x.hi, y.hi);
  return quick_sum(p.hi, p.lo + (x.hi * y.lo + x.lo * y.hi));
}
Two operator/(Two x, Two y) {  // long division in three digits
  const double a = x.hi / y.hi;
  const Two r = x + -(y * Two{a, 0.0});
  const double b = r.hi / y.hi;
  const Two s = r + -(y * Two{b, 0.0});
  return quick_sum(a, b) + Two{s.hi / y.hi, 0.0};
}
constexpr Two kLn2{0x1.62e42fefa39efp-1, 0x1.abc9e3b39803fp-56};
constexpr Two kTwoPi{0x1.921fb54442d18p+2, 0x1.1a62633145c07p-52};

// e^x: x = k ln 2 + 256 r, the Taylor sum of e^r (|r| < 0.0014: ten terms reach 2^-110), squared eight times.
Two exp_two(Two x) {
  const double k = std::nearbyint(x.hi / kLn2.hi);
  Two r = x + -(kLn2 * Two{k, 0.0});
  r = {r.hi / 256, r.lo / 256};
  Two sum{1.0, 0.0};
  for (int n = 10; n; --n) sum = Two{1.0, 0.0} + r * sum / Two{(double)n, 0.0};
  for (int i = 0; i < 8; ++i) sum = sum * sum;
  return {std::ldexp(sum.hi, (int)k), std::ldexp(sum.lo, (int)k)};
}
// ln x: one Newton step from the double's logarithm.
Two log_two(double x) {
  const Two y{std::log(x), 0.0};
  return y + (Two{x, 0.0} * exp_two(-y) + Two{-1.0, 0.0});
}
// x modulo 1 in steps of 2^-64, for 0 <= x.
uint64_t fraction(Two x) {
  const double whole = std::floor(x.hi), scaled = std::ldexp(x.hi - whole, 64), steps = std::floor(scaled);
  // a low part of an eighth and more belongs to a double without a fraction: no phase is left to speak of
  const double low = std::fabs(x.lo) < 0.125 ? std::floor((scaled - steps) + std::ldexp(x.lo, 64)) : 0.0;
  return (uint64_t)steps + (uint64_t)(int64_t)low;
}

// ------------------------------------------------------------------------------------------ checks
bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

int elem_size(int32_t dtype) { return dtype == DCP_BF16 ? 2 : 4; }

dcp_status check_pool(const dcp_kv_pool* c) {
  if (!c || !c->k || !c->v || !aligned(c->k, 16) || !aligned(c->v, 16)) return DCP_EINVAL;
  if (c->dtype != DCP_BF16 && c->dtype != DCP_F32) return DCP_EINVAL;
  const int64_t es = elem_size(c->dtype);
  if (c->H < 1 || c->H > 65535 || c->D < 1 || c->D > 128 || (c->D * es) % 16) return DCP_EINVAL;
  if (c->block_size < 1 || c->n_blocks < 1 || c->n_blocks > INT32_MAX) return DCP_EINVAL;
  // strides below 2^40 bytes: what a tensor map can hold
  for (int64_t s : {c->s_block, c->s_head, c->s_row})
    if (s < 1 || s * es >= (int64_t(1) << 40) || (s * es) % 16) return DCP_EINVAL;
  return DCP_OK;
}

dcp_status check_batch(const dcp_seq_batch* b) {
  if (!b || !b->q_start || !b->tables || !b->kv_len || !b->status) return DCP_EINVAL;
  if (!aligned(b->q_start, 4) || !aligned(b->tables, 4) || !aligned(b->kv_len, 4) || !aligned(b->status, 4))
    return DCP_EINVAL;
  if (b->n_seqs < 1 || b->n_seqs > 65535 || b->total_q < 1 || b->max_q < 1 || b->max_q > b->total_q)
    return DCP_EINVAL;
  if (b->kv_len_per_head != 0 && b->kv_len_per_head != 1) return DCP_EINVAL;
  if (b->max_kv < 0 || b->table_stride < 1 || b->table_stride > INT32_MAX) return DCP_EINVAL;
  if (b->kv_len_add < 0 || b->kv_len_add > INT32_MAX) return DCP_EINVAL;
  return DCP_OK;
}

Pool pool_of(const dcp_kv_pool* c) {
  return Pool{(char*)c->k, (char*)c->v, c->H, c->D, c->dtype, c->block_size, c->n_blocks, c->s_block, c->s_head,
              c->s_row};
}

Batch batch_of(const dcp_seq_batch* b) {
  return Batch{b->n_seqs, b->total_q, b->max_q, b->kv_len_per_head, b->table_stride, b->kv_len_add, b->q_start,
               b->tables, b->kv_len, b->status};
}

bool token_stride_ok(int64_t stride, int64_t heads, int64_t D, int es) {
  return stride >= heads * D && stride <= (int64_t(1) << 40) && (stride * es) % 16 == 0;
}

dcp_status cuda_ok(cudaError_t e) { return e == cudaSuccess ? DCP_OK : DCP_ECUDA; }

// What both appends take: the checks, and everything but the turn.
dcp_status append_of(const dcp_kv_pool* pool, const dcp_seq_batch* batch, const void* q, int64_t q_stride, int32_t Hq,
                     const void* k, const void* v, int64_t kv_stride, const int32_t* positions, void* q_out,
                     AppendParams& p) {
  if (check_pool(pool) != DCP_OK || check_batch(batch) != DCP_OK || batch->kv_len_per_head) return DCP_EINVAL;
  const int es = elem_size(pool->dtype);
  if (!k || !v || !aligned(k, 16) || !aligned(v, 16) || !token_stride_ok(kv_stride, pool->H, pool->D, es))
    return DCP_EINVAL;
  if (!q != !q_out || !aligned(positions, 4)) return DCP_EINVAL;
  if (q) {
    if (Hq < 1 || Hq > 65535 || !aligned(q, 16) || !aligned(q_out, 16) || !token_stride_ok(q_stride, Hq, pool->D, es))
      return DCP_EINVAL;
    if (q == q_out && q_stride != (int64_t)Hq * pool->D) return DCP_EINVAL;
  }
  p.pool = pool_of(pool);
  p.b = batch_of(batch);
  p.q = (const char*)q;
  p.k = (const char*)k;
  p.v = (const char*)v;
  p.q_out = (char*)q_out;
  p.q_stride = q_stride;
  p.kv_stride = kv_stride;
  p.Hq = q ? Hq : 0;
  p.positions = positions;
  return DCP_OK;
}

dcp_status check_attention(const dcp_kv_pool* pool, const dcp_seq_batch* batch, const dcp_attn_config* cfg,
                           int32_t Hq) {
  if (check_pool(pool) != DCP_OK || check_batch(batch) != DCP_OK || !cfg) return DCP_EINVAL;
  if (Hq < 1 || Hq > 65535 || Hq % pool->H) return DCP_EINVAL;
  if (!std::isfinite(cfg->scale) || (cfg->causal != 0 && cfg->causal != 1)) return DCP_EINVAL;
  if (cfg->window < -1 || (cfg->window >= 0 && !cfg->causal)) return DCP_EINVAL;
  if (cfg->sink < 0 || (cfg->sink && cfg->window < 0)) return DCP_EINVAL;
  if ((int64_t)batch->max_q * Hq > kMaxKv) return DCP_EINVAL;
  return DCP_OK;
}

AttendParams attend_of(const dcp_kv_pool* pool, const dcp_seq_batch* batch, const dcp_attn_config* cfg, int32_t Hq) {
  AttendParams p{};
  p.pool = pool_of(pool);
  p.b = batch_of(batch);
  p.Hq = Hq;
  p.G = Hq / pool->H;
  p.causal = cfg->causal;
  p.window = cfg->window < kMaxKv ? cfg->window : kMaxKv;
  p.sink = cfg->sink < kMaxKv ? cfg->sink : kMaxKv;
  p.scale = cfg->scale;
  // one near 0 is held where masked scores of -inf still scale to -inf
  const double mag = std::fabs((double)cfg->scale);
  p.scale_log2 = (float)std::fmin((mag < 1e-30 ? 1e-30 : mag) * 1.4426950408889634, (double)FLT_MAX);
  return p;
}

bool shared_of(const dcp_kv_pool* pool, const dcp_seq_batch* batch, const dcp_prefix_groups* g,
               const dcp_attn_config* cfg, int32_t Hq, AttendParams& p) {
  if (check_attention(pool, batch, cfg, Hq) != DCP_OK || !g) return false;
  if (!g->start || !g->prefix_len || !aligned(g->start, 4) || !aligned(g->prefix_len, 4)) return false;
  if (g->n_groups < 1 || g->n_groups > batch->n_seqs || g->max_q < 1 || g->max_q > batch->total_q || g->max_prefix < 0)
    return false;
  if ((int64_t)g->max_q * Hq > kMaxKv) return false;
  p = attend_of(pool, batch, cfg, Hq);
  p.groups = Groups{g->n_groups, g->max_q, g->start, g->prefix_len};
  return true;
}

dcp_status check_pages(const dcp_page_pool* p) {
  if (!p || !p->k || !p->v || !p->status || !aligned(p->k, 16) || !aligned(p->v, 16) || !aligned(p->status, 4))
    return DCP_EINVAL;
  if (p->L < 1 || p->block_size < 1 || p->n_blocks < 1 || p->n_blocks > INT32_MAX) return DCP_EINVAL;
  if (p->page_bytes < 16 || p->page_bytes % 16 || p->page_bytes > (int64_t(1) << 31)) return DCP_EINVAL;
  return DCP_OK;
}

PageParams pages_of(const dcp_page_pool* p) {
  return PageParams{(char*)p->k, (char*)p->v, p->L, p->block_size, p->n_blocks, p->page_bytes, p->status};
}

bool rows_ok(int32_t n_rows, int32_t stride) {
  return n_rows >= 1 && stride >= 1 && (int64_t)n_rows * stride < (int64_t(1) << 30);
}

bool ws_ok(const void* ws, size_t bytes, size_t need) { return ws && aligned(ws, 256) && need && bytes >= need; }

bool all_words(std::initializer_list<const void*> required, std::initializer_list<const void*> optional) {
  for (const void* p : required)
    if (!p || !aligned(p, 4)) return false;
  for (const void* p : optional)
    if (!aligned(p, 4)) return false;
  return true;
}

}  // namespace

extern "C" {

dcp_status dcp_rope_plan_init(const dcp_rope_config* g, dcp_rope_plan* plan) {
  if (!g || !plan) return DCP_EINVAL;
  if (g->rot_dim < 0 || g->rot_dim > 2 * DCP_ROPE_MAX_PAIRS || (g->rot_dim & 1) || g->reserved != 0)
    return DCP_EINVAL;
  if (g->pair_layout != DCP_ROPE_INTERLEAVED && g->pair_layout != DCP_ROPE_HALF) return DCP_EINVAL;
  if (g->scaling < DCP_ROPE_PLAIN || g->scaling > DCP_ROPE_PARTS) return DCP_EINVAL;
  if (!std::isfinite(g->base) || !(g->base > 0.0) || !std::isfinite(g->amplitude)) return DCP_EINVAL;
  if (g->scaling != DCP_ROPE_PLAIN && (!std::isfinite(g->factor) || !(g->factor > 0.0))) return DCP_EINVAL;
  if (g->scaling == DCP_ROPE_PARTS &&
      (!std::isfinite(g->orig_len) || !(g->orig_len > 0.0) || !std::isfinite(g->beta_fast) ||
       !std::isfinite(g->beta_slow) || !(g->beta_fast > g->beta_slow)))
    return DCP_EINVAL;
  const int rot = g->rot_dim;
  if (g->scaling == DCP_ROPE_BASE && rot > 2) {
    const double base = g->base * std::pow(g->factor, (double)rot / (rot - 2));
    if (!std::isfinite(base) || !(base > 0.0)) return DCP_EINVAL;
  }
  Two log_base = log_two(g->base);
  if (g->scaling == DCP_ROPE_BASE && rot > 2)
    log_base = log_base + log_two(g->factor) * Two{(double)rot, 0.0} / Two{rot - 2.0, 0.0};
  const Two factor{g->factor, 0.0}, one{1.0, 0.0};
  uint64_t turn_of[DCP_ROPE_MAX_PAIRS] = {};
  for (int p = 0; p < rot / 2; ++p) {
    Two theta = exp_two(log_base * Two{-2.0 * p, 0.0} / Two{(double)rot, 0.0});
    if (g->scaling == DCP_ROPE_LINEAR) theta = theta / factor;
    if (g->scaling == DCP_ROPE_PARTS) {
      const double rough = (g->orig_len * theta.hi / kTwoPi.hi - g->beta_slow) / (g->beta_fast - g->beta_slow);
      const Two slow{-g->beta_slow, 0.0};
      Two ramp = rough > 0.5 ? one : Two{0.0, 0.0};
      if (rough > -1.0 && rough < 2.0) {
        const Two r = (theta * Two{g->orig_len, 0.0} / kTwoPi + slow) / (Two{g->beta_fast, 0.0} + slow);
        if (r.hi >= 0.0 && r.hi < 1.0) ramp = r;
      }
      theta = theta * (ramp + (one + -ramp) / factor);
    }
    const Two turns = theta / kTwoPi;
    if (!std::isfinite(turns.hi) || !std::isfinite(turns.lo)) return DCP_EINVAL;
    turn_of[p] = fraction(turns);
  }
  for (int p = 0; p < DCP_ROPE_MAX_PAIRS; ++p) plan->turns[p] = turn_of[p];
  plan->rot_dim = g->rot_dim;
  plan->pair_layout = g->pair_layout;
  plan->amplitude = (float)g->amplitude;
  plan->ready = 1;
  return DCP_OK;
}

dcp_status dcp_rope_axes_init(const dcp_rope_config* cfg, int32_t n_axes, dcp_rope_axes* axes) {
  if (!cfg || !axes || n_axes < 1 || n_axes > DCP_ROPE_MAX_AXES) return DCP_EINVAL;
  dcp_rope_axes out{};
  out.n_axes = n_axes;
  out.pair_layout = cfg[0].pair_layout;
  for (int a = 0; a < n_axes; ++a) {
    dcp_rope_plan plan;
    if (cfg[a].pair_layout != out.pair_layout || dcp_rope_plan_init(&cfg[a], &plan) != DCP_OK) return DCP_EINVAL;
    if (out.rot_dim + plan.rot_dim > 2 * DCP_ROPE_MAX_PAIRS) return DCP_EINVAL;
    out.first[a] = out.rot_dim / 2;
    out.amplitude[a] = plan.amplitude;
    for (int i = 0; i < plan.rot_dim / 2; ++i) out.turns[out.rot_dim / 2 + i] = plan.turns[i];
    out.rot_dim += plan.rot_dim;
  }
  for (int a = n_axes; a < DCP_ROPE_MAX_AXES; ++a) out.first[a] = out.rot_dim / 2;
  out.ready = 1;
  *axes = out;
  return DCP_OK;
}

dcp_status dcp_rope_append(const dcp_kv_pool* pool, const dcp_seq_batch* batch, const dcp_rope_plan* plan,
                           const void* q, int64_t q_stride, int32_t Hq, const void* k, const void* v,
                           int64_t kv_stride, const int32_t* positions, void* q_out, void* stream) {
  AppendParams p{};
  if (append_of(pool, batch, q, q_stride, Hq, k, v, kv_stride, positions, q_out, p) != DCP_OK) return DCP_EINVAL;
  if (!plan || plan->ready != 1 || plan->rot_dim < 0 || plan->rot_dim > pool->D || (plan->rot_dim & 1))
    return DCP_EINVAL;
  p.half_layout = plan->pair_layout == DCP_ROPE_HALF;
  p.half = plan->rot_dim / 2;
  p.amplitude = plan->amplitude;
  for (int i = 0; i < DCP_ROPE_MAX_PAIRS; ++i) p.turns[i] = plan->turns[i];
  return cuda_ok(launch_append(p, (cudaStream_t)stream));
}

dcp_status dcp_norm_rope_append(const dcp_kv_pool* pool, const dcp_seq_batch* batch, const dcp_rope_axes* axes,
                                const dcp_norm_config* norm, const void* q, int64_t q_stride, int32_t Hq, const void* k,
                                const void* v, int64_t kv_stride, const int32_t* positions, void* q_out, void* stream) {
  NormParams n{};
  AppendParams& p = n.a;
  if (append_of(pool, batch, q, q_stride, Hq, k, v, kv_stride, positions, q_out, p) != DCP_OK) return DCP_EINVAL;
  if (!axes || axes->ready != 1 || axes->n_axes < 1 || axes->n_axes > DCP_ROPE_MAX_AXES || axes->rot_dim < 0 ||
      axes->rot_dim > pool->D || (axes->rot_dim & 1))
    return DCP_EINVAL;
  if (axes->n_axes > 1 && !positions) return DCP_EINVAL;
  if (!norm || (norm->span != DCP_NORM_HEAD && norm->span != DCP_NORM_TOKEN) || !std::isfinite(norm->eps) ||
      norm->eps < 0.f)
    return DCP_EINVAL;
  if (norm->weight_dtype != DCP_BF16 && norm->weight_dtype != DCP_F32) return DCP_EINVAL;
  if (norm->weight_per_head != 0 && norm->weight_per_head != 1) return DCP_EINVAL;
  if (!aligned(norm->q_weight, 16) || !aligned(norm->k_weight, 16)) return DCP_EINVAL;
  p.half_layout = axes->pair_layout == DCP_ROPE_HALF;
  p.half = axes->rot_dim / 2;
  for (int i = 0; i < DCP_ROPE_MAX_PAIRS; ++i) p.turns[i] = axes->turns[i];
  n.q_weight = (const char*)norm->q_weight;
  n.k_weight = (const char*)norm->k_weight;
  n.weight_bf16 = norm->weight_dtype == DCP_BF16;
  n.weight_bytes = elem_size(norm->weight_dtype);
  n.weight_heads = norm->weight_per_head;
  n.token_span = norm->span == DCP_NORM_TOKEN;
  n.eps = norm->eps;
  n.inv_head = (float)(1.0 / pool->D);
  n.inv_q = p.Hq ? (float)(1.0 / ((double)p.Hq * pool->D)) : 1.f;
  n.inv_k = (float)(1.0 / ((double)pool->H * pool->D));
  for (int a = 0; a < DCP_ROPE_MAX_AXES; ++a) {
    n.first[a] = axes->first[a];
    n.amplitude[a] = axes->amplitude[a];
  }
  return cuda_ok(launch_norm_append(n, (cudaStream_t)stream));
}

size_t dcp_attention_workspace_size(const dcp_kv_pool* pool, const dcp_seq_batch* batch, const dcp_attn_config* cfg,
                                    int32_t Hq) {
  if (check_attention(pool, batch, cfg, Hq) != DCP_OK) return 0;
  const AttendParams p = attend_of(pool, batch, cfg, Hq);
  const size_t bytes = attend_by_rows(p) ? plan_rows(p, batch->max_kv).bytes : plan_tiles(p, batch->max_kv).bytes;
  return kScratch + (bytes + 255) / 256 * 256;
}

dcp_status dcp_paged_attention(const dcp_kv_pool* pool, const dcp_seq_batch* batch, const dcp_attn_config* cfg,
                               const void* q, int64_t q_stride, int32_t Hq, void* out, float* lse, void* ws,
                               size_t ws_bytes, void* stream) {
  if (!ws_ok(ws, ws_bytes, dcp_attention_workspace_size(pool, batch, cfg, Hq))) return DCP_EINVAL;
  if (!q || !out || !aligned(q, 16) || !aligned(out, 16) || !aligned(lse, 4)) return DCP_EINVAL;
  if (!token_stride_ok(q_stride, Hq, pool->D, elem_size(pool->dtype))) return DCP_EINVAL;
  AttendParams p = attend_of(pool, batch, cfg, Hq);
  p.q = (const char*)q;
  p.out = (char*)out;
  p.lse = lse;
  p.q_stride = q_stride;
  return cuda_ok(attend_by_rows(p) ? launch_attend_rows(p, batch->max_kv, ws, (cudaStream_t)stream)
                                   : launch_attend_tiles(p, batch->max_kv, ws, (cudaStream_t)stream));
}

size_t dcp_shared_attention_workspace_size(const dcp_kv_pool* pool, const dcp_seq_batch* batch,
                                           const dcp_prefix_groups* groups, const dcp_attn_config* cfg, int32_t Hq) {
  AttendParams p;
  if (!shared_of(pool, batch, groups, cfg, Hq, p)) return 0;
  return kScratch + (shared_bytes(p, batch->max_kv, groups->max_prefix) + 255) / 256 * 256;
}

dcp_status dcp_shared_attention(const dcp_kv_pool* pool, const dcp_seq_batch* batch, const dcp_prefix_groups* groups,
                                const dcp_attn_config* cfg, const void* q, int64_t q_stride, int32_t Hq, void* out,
                                float* lse, void* ws, size_t ws_bytes, void* stream) {
  if (!ws_ok(ws, ws_bytes, dcp_shared_attention_workspace_size(pool, batch, groups, cfg, Hq))) return DCP_EINVAL;
  if (!q || !out || !aligned(q, 16) || !aligned(out, 16) || !aligned(lse, 4)) return DCP_EINVAL;
  if (!token_stride_ok(q_stride, Hq, pool->D, elem_size(pool->dtype))) return DCP_EINVAL;
  AttendParams p;
  shared_of(pool, batch, groups, cfg, Hq, p);
  p.q = (const char*)q;
  p.out = (char*)out;
  p.lse = lse;
  p.q_stride = q_stride;
  return cuda_ok(launch_shared(p, batch->max_kv, groups->max_prefix, ws, (cudaStream_t)stream));
}

size_t dcp_pages_workspace_size(const dcp_page_pool* pool, int32_t n_rows, int32_t stride) {
  if (check_pages(pool) != DCP_OK || !rows_ok(n_rows, stride)) return 0;
  // the list of moves and the fresh blocks of a fork, or the list of moves and the map of a packing
  const size_t entries = (size_t)n_rows * stride;
  const size_t fork = 3 * entries + n_rows, pack = 3 * (size_t)pool->n_blocks;
  return (kScratch + 256 + 4 * (fork > pack ? fork : pack) + 255) & ~(size_t)255;
}

dcp_status dcp_pages_copy(const dcp_page_pool* pool, const int32_t* src, const int32_t* dst, int32_t n, void* stream) {
  if (check_pages(pool) != DCP_OK || n < 0 || (n && !all_words({src, dst}, {}))) return DCP_EINVAL;
  if (n == 0) return DCP_OK;
  return cuda_ok(launch_pages_copy(pages_of(pool), src, dst, n, (cudaStream_t)stream));
}

dcp_status dcp_pages_fork(const dcp_page_pool* pool, const int32_t* tables, const int32_t* len, int32_t n_rows,
                          int32_t stride, const int32_t* parent, const int32_t* shared, const int32_t* reserve,
                          int32_t n_children, const int32_t* ref_in, int32_t* child_tables, int32_t* ref_out, void* ws,
                          size_t ws_bytes, void* stream) {
  if (check_pages(pool) != DCP_OK || !rows_ok(n_rows, stride) || !rows_ok(n_children, stride)) return DCP_EINVAL;
  if (!all_words({tables, len, parent, ref_in, child_tables, ref_out}, {shared, reserve})) return DCP_EINVAL;
  if (!ws_ok(ws, ws_bytes, dcp_pages_workspace_size(pool, n_children, stride))) return DCP_EINVAL;
  return cuda_ok(launch_pages_fork(pages_of(pool), tables, len, n_rows, stride, parent, shared, reserve, n_children,
                                   ref_in, child_tables, ref_out, (int32_t*)ws, (cudaStream_t)stream));
}

dcp_status dcp_pages_free(const dcp_page_pool* pool, const int32_t* tables, int32_t n_rows, int32_t stride,
                          const int32_t* ref_in, int32_t* tables_out, int32_t* ref_out, void* stream) {
  if (check_pages(pool) != DCP_OK || !rows_ok(n_rows, stride)) return DCP_EINVAL;
  if (!all_words({tables, ref_in, tables_out, ref_out}, {})) return DCP_EINVAL;
  return cuda_ok(launch_pages_free(pages_of(pool), tables, n_rows, stride, ref_in, tables_out, ref_out,
                                   (cudaStream_t)stream));
}

dcp_status dcp_pages_compact(const dcp_page_pool* pool, const int32_t* tables, int32_t n_rows, int32_t stride,
                             const int32_t* ref_in, int32_t* tables_out, int32_t* ref_out, int32_t* n_live, void* ws,
                             size_t ws_bytes, void* stream) {
  if (check_pages(pool) != DCP_OK || !rows_ok(n_rows, stride)) return DCP_EINVAL;
  if (!all_words({tables, ref_in, tables_out, ref_out}, {n_live})) return DCP_EINVAL;
  if (!ws_ok(ws, ws_bytes, dcp_pages_workspace_size(pool, n_rows, stride))) return DCP_EINVAL;
  return cuda_ok(launch_pages_compact(pages_of(pool), tables, n_rows, stride, ref_in, tables_out, ref_out, n_live,
                                      (int32_t*)ws, (cudaStream_t)stream));
}

uint32_t dcp_abi_norm_struct_size(int32_t which) {
  switch (which) {
    case 0: return sizeof(dcp_rope_axes);
    case 1: return sizeof(dcp_norm_config);
    case 2: return sizeof(dcp_prefix_groups);
    default: return 0;
  }
}

uint32_t dcp_abi_serving_struct_size(int32_t which) {
  switch (which) {
    case 0: return sizeof(dcp_kv_pool);
    case 1: return sizeof(dcp_seq_batch);
    case 2: return sizeof(dcp_rope_config);
    case 3: return sizeof(dcp_rope_plan);
    case 4: return sizeof(dcp_attn_config);
    case 5: return sizeof(dcp_page_pool);
    default: return 0;
  }
}

}  // extern "C"
