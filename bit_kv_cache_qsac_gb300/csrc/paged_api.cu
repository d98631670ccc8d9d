// C ABI of the paged cache (include/qwm_paged.h): argument checks and dispatch.  Nothing here allocates
// device memory; every check is made before the first CUDA call.
#include "paged.cuh"
#include "window_checks.cuh"

namespace {

int log2_of_page(int page) {
  for (int i = 4; i <= 8; i++)
    if (page == 1 << i) return i;
  return -1;
}

qwm_status check_table(const qwm_page_table *t, bool stack) {
  if (!t) return QWM_ERR_ARG;
  if (log2_of_page(t->page) < 0) return QWM_ERR_UNSUPPORTED;
  if (t->batch < 1 || t->width < 1 || !t->table || !t->length) return QWM_ERR_ARG;
  if (t->batch > kPagedMaxBatch || (int64_t)t->width * t->page > kPagedMaxTokens) return QWM_ERR_SHAPE;
  if (!aligned_to(t->table, 4) || !aligned_to(t->length, 8)) return QWM_ERR_ALIGN;
  if (!stack) return QWM_OK;
  if (t->pages < 1 || !t->free_list || !t->free_count) return QWM_ERR_ARG;
  if ((int64_t)t->pages * t->page > ((int64_t)1 << 40)) return QWM_ERR_SHAPE;
  if (!aligned_to(t->free_list, 4) || !aligned_to(t->free_count, 4)) return QWM_ERR_ALIGN;
  return QWM_OK;
}

qwm_status check_pool_shape(const qwm_page_pool *p) {
  if (!p) return QWM_ERR_ARG;
  if ((p->bits != 8 && p->bits != 4) || log2_of_page(p->page) < 0) return QWM_ERR_UNSUPPORTED;
  if (p->pages < 1 || p->kv_heads < 1) return QWM_ERR_ARG;
  if (p->kv_heads > kMaxGridY || (int64_t)p->pages * p->page > ((int64_t)1 << 40)) return QWM_ERR_SHAPE;
  return QWM_OK;
}

qwm_status check_pool(const qwm_page_pool *p) {
  const qwm_status s = check_pool_shape(p);
  if (s != QWM_OK) return s;
  const void *req[] = {p->k_codes, p->v_codes, p->k_step, p->v_step};
  for (const void *x : req) {
    if (!x) return QWM_ERR_ARG;
    if (!aligned16(x)) return QWM_ERR_ALIGN;
  }
  return QWM_OK;
}

// A packed activation: one sequence of n rows.
qwm_status check_packed(const void *p, const qwm_strides *s, int64_t heads, int64_t n, bool written) {
  if (!s) return QWM_ERR_ARG;
  const qwm_strides one = {0, s->head, s->token};
  return check_rows(p, &one, 1, heads, n, written);
}

qwm_status check_norm(const float *weight, int32_t per_head, float eps) {
  if ((per_head != 0 && per_head != 1) || !(eps >= 0.f) || eps > 0x1p100f) return QWM_ERR_ARG;   // (beside a mean square it stays finite)
  return aligned16(weight) ? QWM_OK : QWM_ERR_ALIGN;
}

constexpr int64_t kMaxRows = (int64_t)1 << 30;      // rows of a Key head in a packed batch
constexpr int64_t kMaxAllRows = (int64_t)1 << 36;   // of all heads: items are numbered in 32 bits

// How a call is run and what workspace it takes.  Sequences with up to `few` rows per Key head go to the warp tiles,
// which read the cache once per 8 or 16 rows, others to the tensor-memory tiles, which pay for 256 or 512.
struct Plan {
  bool few_rows, many_rows;
  int few, row_tiles;         // warp tiles of 8 (1) or 16 rows (2) an item
  int shares_few, shares_many;
  size_t part_few, part_many;   // rows of all parts
  size_t bytes;
};

// Both sides of it measured, 40 heads, one sequence, 8 bits (4 bits): 32 rows over 500 / 5,000 / 30,000 tokens take 16 / 36 /
// 136 us (15 / 33 / 116) on warp tiles and 23 / 47 / 149 (23 / 45 / 146) on the others; 64 rows 22 / 59 / 256 (22 / 52 / 215)
// and 23 / 47 / 150 (23 / 45 / 146).
constexpr int kFew = 32;

Plan plan_of(const qwm_ctx *ctx, int group, int64_t max_count) {
  Plan p;
  const int64_t rows = max_count * group;
  p.many_rows = rows > kFew;
  p.few_rows = group <= kFew;
  p.few = kFew;
  // One tile for all rows of a sequence; where longer sequences may stand beside them, for those of one token, which
  // 16-row tiles (one CTA an SM, half of them empty) slow down more than they help more rows.  24 sequences of up to 8,000
  // tokens, 8 bits, with 8-row (16-row) tiles: 1 token each of 32 heads on 8: 60 us (69), on 32: 150 (205); 2 tokens of 4 heads
  // a Key head 54 (71), 5 tokens 117 (118), 8 tokens 149 (139); beside 777 tokens of a prompt 136 (144), 138 (148), 191 (191), 225
  // (208); 40 heads on 5, 1 and 2 tokens: 41 (57) and 67 (61).
  p.row_tiles = (p.many_rows ? group : rows) <= 8 ? 1 : 2;
  p.shares_few = p.few_rows ? paged_decode_shares(p.row_tiles, ctx->num_sms) : 0;
  p.shares_many = p.many_rows ? ctx->num_sms / 2 : 0;
  p.part_few = (size_t)2 * p.shares_few * 8 * p.row_tiles;
  p.part_many = (size_t)2 * p.shares_many * kPagedTileRows;
  // (a place for the cuts of 8-row tiles in any case: what a count takes, smaller ones do not exceed)
  const int cuts_few = p.few_rows ? paged_decode_shares(1, ctx->num_sms) : 0;
  p.bytes = (p.part_few + p.part_many) * (QWM_D + 1) * sizeof(float) + (size_t)(cuts_few + p.shares_many) * sizeof(PagedCut);
  return p;
}

qwm_status check_attend(const qwm_ctx *ctx, const qwm_page_pool *pool, int64_t max_count) {
  if (!ctx || max_count < 0) return QWM_ERR_ARG;
  const qwm_status s = check_pool_shape(pool);
  if (s != QWM_OK) return s;
  if (ctx->cfg.heads % pool->kv_heads != 0 || max_count > kMaxTokens) return QWM_ERR_SHAPE;
  return QWM_OK;
}

}  // namespace

extern "C" {

qwm_status qwm_norm_rope(qwm_ctx *ctx, const qwm_rope_spec *spec, const uint16_t *x, const qwm_strides *xs, int32_t batch,
                         int32_t heads, int64_t n, const int64_t *start, const int64_t *at, const int32_t *pos,
                         const float *weight, int32_t per_head, float eps, uint16_t *out, const qwm_strides *os,
                         qwm_stream stream) {
  if (!ctx || batch < 0 || heads < 0 || n < 0) return QWM_ERR_ARG;
  qwm_status s = spec ? check_rope(spec) : QWM_OK;
  if (s == QWM_OK) s = check_norm(weight, per_head, eps);
  if (s != QWM_OK) return s;
  if (batch > kMaxGridY || heads > kMaxGridY || n > kMaxTokens) return QWM_ERR_SHAPE;
  if ((int64_t)batch * n >= ((int64_t)1 << 34)) return QWM_ERR_SHAPE;
  if (batch == 0 || heads == 0 || n == 0) return QWM_OK;
  if ((s = check_rows(x, xs, batch, heads, n, false)) != QWM_OK) return s;
  if ((s = check_rows(out, os, batch, heads, n, true)) != QWM_OK) return s;
  if ((start && at) || (spec && !start && !at) || (pos && !spec)) return QWM_ERR_ARG;
  if (!aligned_to(start, 8) || !aligned_to(at, 8) || !aligned_to(pos, 4)) return QWM_ERR_ALIGN;
  if (x == out && (xs->batch != os->batch || xs->head != os->head || xs->token != os->token)) return QWM_ERR_ARG;
  DeviceGuard dev(ctx->device);
  if (dev.err != cudaSuccess) return QWM_ERR_CUDA;
  return cuda_status(launch_norm_rope(spec, x, *xs, batch, heads, n, start, at, pos, weight, weight ? per_head : 0, eps, out,
                                      *os, ctx->num_sms, (cudaStream_t)stream));
}

qwm_status qwm_pages_reset(qwm_ctx *ctx, const qwm_page_table *tab, qwm_stream stream) {
  if (!ctx) return QWM_ERR_ARG;
  const qwm_status s = check_table(tab, true);
  if (s != QWM_OK) return s;
  DeviceGuard dev(ctx->device);
  if (dev.err != cudaSuccess) return QWM_ERR_CUDA;
  return cuda_status(launch_pages_reset(*tab, ctx->num_sms, (cudaStream_t)stream));
}

qwm_status qwm_pages_update(qwm_ctx *ctx, const qwm_page_table *tab, const int64_t *keep, const int32_t *count, int64_t n,
                            int32_t *first, int32_t *granted, int64_t *slot, int64_t *at, qwm_stream stream) {
  if (!ctx || n < 0) return QWM_ERR_ARG;
  const qwm_status s = check_table(tab, true);
  if (s != QWM_OK) return s;
  if (n > kMaxTokens) return QWM_ERR_SHAPE;
  if (count ? !first || !granted || (n > 0 && (!slot || !at)) : n > 0) return QWM_ERR_ARG;
  if (!keep && !count) return QWM_OK;
  if (!aligned_to(keep, 8) || !aligned_to(count, 4) || !aligned_to(first, 4) || !aligned_to(granted, 4) ||
      !aligned_to(slot, 8) || !aligned_to(at, 8))
    return QWM_ERR_ALIGN;
  DeviceGuard dev(ctx->device);
  if (dev.err != cudaSuccess) return QWM_ERR_CUDA;
  return cuda_status(launch_pages_update(*tab, log2_of_page(tab->page), keep, count, n, count ? first : nullptr,
                                         count ? granted : nullptr, slot, at, ctx->status, (cudaStream_t)stream));
}

qwm_status qwm_paged_write(qwm_ctx *ctx, const qwm_page_pool *pool, const uint16_t *k, const qwm_strides *ks,
                           const uint16_t *v, const qwm_strides *vs, int64_t n, const int64_t *slot,
                           const qwm_rope_spec *rope, const int64_t *at, const int32_t *pos, int32_t norm, const float *weight,
                           int32_t per_head, float eps, qwm_stream stream) {
  if (!ctx || n < 0) return QWM_ERR_ARG;
  qwm_status s = check_pool(pool);
  if (s == QWM_OK && rope) s = check_rope(rope);
  if (s != QWM_OK) return s;
  if (norm != 0 && norm != 1) return QWM_ERR_ARG;
  if (norm ? (s = check_norm(weight, per_head, eps)) != QWM_OK : weight != nullptr) return norm ? s : QWM_ERR_ARG;
  if (n > kMaxTokens) return QWM_ERR_SHAPE;
  if (n == 0) return QWM_OK;
  if ((s = check_packed(k, ks, pool->kv_heads, n, false)) != QWM_OK) return s;
  if ((s = check_packed(v, vs, pool->kv_heads, n, false)) != QWM_OK) return s;
  if (!slot || (rope ? !at : at || pos)) return QWM_ERR_ARG;
  if (!aligned_to(slot, 8) || !aligned_to(at, 8) || !aligned_to(pos, 4)) return QWM_ERR_ALIGN;
  DeviceGuard dev(ctx->device);
  if (dev.err != cudaSuccess) return QWM_ERR_CUDA;
  return cuda_status(launch_paged_write(*pool, log2_of_page(pool->page), k, *ks, v, *vs, n, slot, rope, at, pos, norm, weight,
                                        weight ? per_head : 0, eps, ctx->num_sms, ctx->status, (cudaStream_t)stream));
}

qwm_status qwm_paged_read(qwm_ctx *ctx, const qwm_page_pool *pool, const int64_t *slot, int64_t n, uint16_t *k_hat,
                          uint16_t *v_hat, qwm_stream stream) {
  if (!ctx || n < 0) return QWM_ERR_ARG;
  const qwm_status s = check_pool(pool);
  if (s != QWM_OK) return s;
  if (n > kMaxTokens) return QWM_ERR_SHAPE;
  if (n == 0 || (!k_hat && !v_hat)) return QWM_OK;
  if (!slot) return QWM_ERR_ARG;
  if (!aligned_to(slot, 8) || !aligned16(k_hat) || !aligned16(v_hat)) return QWM_ERR_ALIGN;
  DeviceGuard dev(ctx->device);
  if (dev.err != cudaSuccess) return QWM_ERR_CUDA;
  return cuda_status(launch_paged_read(*pool, log2_of_page(pool->page), slot, n, k_hat, v_hat, ctx->num_sms, ctx->status,
                                       (cudaStream_t)stream));
}

size_t qwm_paged_attend_workspace(const qwm_ctx *ctx, const qwm_page_pool *pool, int64_t max_count) {
  if (check_attend(ctx, pool, max_count) != QWM_OK || max_count == 0) return 0;
  return plan_of(ctx, ctx->cfg.heads / pool->kv_heads, max_count).bytes;
}

qwm_status qwm_paged_attend(qwm_ctx *ctx, const qwm_page_pool *pool, const qwm_page_table *tab, const uint16_t *q,
                            const qwm_strides *qs, int64_t n, const int32_t *first, const int32_t *count, int64_t max_count,
                            int64_t tpf, int64_t frames, int64_t sink, float softmax_scale, void *out, const qwm_strides *os,
                            int32_t out_f32, float *lse, int32_t merge, void *ws, size_t ws_bytes, qwm_stream stream) {
  qwm_status s = check_attend(ctx, pool, max_count);
  if (s == QWM_OK) s = check_pool(pool);
  if (s == QWM_OK) s = check_table(tab, false);
  if (s != QWM_OK) return s;
  if (n < 0 || tab->page != pool->page || tpf < 1 || frames < 1 || sink < 0) return QWM_ERR_ARG;
  const int H = ctx->cfg.heads, group = H / pool->kv_heads;
  if (n > kMaxTokens || n * group > kMaxRows || n * H > kMaxAllRows || tpf > ((int64_t)1 << 31) || frames > ((int64_t)1 << 31)) return QWM_ERR_SHAPE;
  if (!(softmax_scale > 0.f) || softmax_scale > 0x1p123f) return QWM_ERR_ARG;   // (times 16 log2(e) it stays finite)
  if ((out_f32 != 0 && out_f32 != 1) || (merge != 0 && merge != 1)) return QWM_ERR_ARG;
  if (merge && (!out_f32 || !lse)) return QWM_ERR_ARG;
  if (n == 0 || max_count == 0) return QWM_OK;
  if ((s = check_packed(q, qs, H, n, false)) != QWM_OK) return s;
  if ((s = check_packed(out, os, H, n, true)) != QWM_OK) return s;
  if (!first || !count) return QWM_ERR_ARG;
  if (!aligned_to(first, 4) || !aligned_to(count, 4) || !aligned_to(lse, 4)) return QWM_ERR_ALIGN;
  const Plan p = plan_of(ctx, group, max_count);
  if (!ws || ws_bytes < p.bytes) return QWM_ERR_ARG;
  if (!aligned16(ws)) return QWM_ERR_ALIGN;
  DeviceGuard dev(ctx->device);
  if (dev.err != cudaSuccess) return QWM_ERR_CUDA;
  PagedAttend a;
  a.pool = *pool;
  a.table = tab->table; a.length = tab->length;
  a.batch = tab->batch; a.width = tab->width; a.page_log2 = log2_of_page(tab->page);
  a.q = q; a.qs = *qs; a.n = (int)n;
  a.first = first; a.count = count; a.max_count = (int)max_count;
  a.tpf = tpf; a.frames = frames;
  a.sink = sink < kPagedMaxTokens ? sink : kPagedMaxTokens;   // (no sequence is longer)
  a.scale_log2 = softmax_scale * 1.4426950408889634f;
  a.out = out; a.os = *os; a.out_f32 = out_f32; a.merge = merge; a.lse = lse;
  a.status = ctx->status;
  a.group = group;
  a.few = p.few;
  a.bases = win::kBases;
  // the parts' outputs, their log-sum-exps, the cuts; the few rows' first
  float *part = (float *)ws, *part_lse = part + (p.part_few + p.part_many) * QWM_D;
  PagedCut *cuts = (PagedCut *)(part_lse + p.part_few + p.part_many);
  a.shares = p.shares_few;
  a.part = part;
  a.part_lse = part_lse;
  a.cuts = cuts;
  PagedAttend many = a;
  many.shares = p.shares_many;
  many.part = part + p.part_few * QWM_D;
  many.part_lse = part_lse + p.part_few;
  many.cuts = cuts + p.shares_few;
  const cudaStream_t st = (cudaStream_t)stream;
  cudaError_t e = p.many_rows ? launch_paged_tiles(many, st) : cudaSuccess;
  if (e == cudaSuccess && p.few_rows) e = launch_paged_decode(a, p.row_tiles, p.many_rows, st);
  if (e == cudaSuccess) e = launch_paged_combine(p.few_rows ? &a : nullptr, 8 * p.row_tiles, p.many_rows ? &many : nullptr, st);
  return cuda_status(e);
}

}  // extern "C"
