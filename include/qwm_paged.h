/*
 * qwm_paged.h -- many sequences in one pool of pages, in libqwm.so: norms of Queries and Keys with the
 * rotation in the same pass, page tables and slot maps kept on the device, a paged cache at 8 or 4 bits,
 * and attention of a packed batch over it.
 *
 * The window cache (qwm_window.h) gives every sequence its own slots and takes batches padded to one
 * length.  These calls serve sequences that come, grow and go at different lengths:
 *  - qwm_pages_update shortens, ends and extends sequences: it hands out pages of a shared pool and says
 *    for every row of the step's packed batch which position and slot it has;
 *  - qwm_norm_rope and qwm_paged_write norm and turn Queries and Keys; the latter quantises Keys and
 *    Values into their slots;
 *  - qwm_paged_attend attends with the rows of all sequences at once, whether a sequence has one new
 *    token, a few drafted ones, or a chunk of its prompt, alone or merged into an earlier result;
 *  - qwm_paged_read hands tokens back in bf16 (to be packed by qwm.h once they are history).
 *
 * Conventions as in qwm_window.h, and further:
 *  - A packed batch holds the step's new tokens of all sequences in n rows: Queries, Keys and Values are
 *    [heads][n][128] with the channels contiguous and the other strides given (qwm_strides; `batch` is not
 *    looked at).  Sequence b has rows first[b] .. first[b] + count[b] - 1, sequences in any order and without
 *    rows in common; rows of no sequence are padding and left as they were.
 *  - One page table serves the pools of all layers (the same pages of each).
 *  - Everything that changes from step to step is read on the device, so a captured step can be replayed.
 */
#ifndef QWM_PAGED_H_
#define QWM_PAGED_H_

#include "qwm_window.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------------------------------ norm and rotation */

/* out = x / sqrt(mean(x^2) + eps) * weight per row of 128 channels, then turned by its position, in fp32
 * and rounded to bf16 once.
 *   spec    or NULL for no rotation
 *   x, out  bf16 [batch][heads][n][128] by xs and os; out may be x itself (same strides)
 *   start   device int64 [batch]: position of token 0 of each sequence (a sequence is skipped as by qwm_rope), or
 *   at      device int64 [batch][n]: every token's position; rows with a negative one, or one above 2^62,
 *           are left as they were.  One of the two is given, or neither without a rotation.
 *   pos     device int32 [batch][n][3] (t, y, x) to turn by instead of the grid's, or NULL
 *   weight  fp32 [128], or [heads][128] (per_head == 1), or NULL for ones
 *   eps     >= 0, at most 2^100
 * A row with an infinite or NaN channel becomes what the formula gives in IEEE arithmetic. */
QWM_API qwm_status qwm_norm_rope(qwm_ctx *ctx, const qwm_rope_spec *spec, const uint16_t *x, const qwm_strides *xs,
                                 int32_t batch, int32_t heads, int64_t n, const int64_t *start, const int64_t *at,
                                 const int32_t *pos, const float *weight, int32_t per_head, float eps, uint16_t *out,
                                 const qwm_strides *os, qwm_stream stream);

/* ------------------------------------------------------------------ page tables */

/* The pages of a batch of sequences: a sequence of `length` tokens holds ceil(length / page) of them, entry i
 * of its row of the table being the page of tokens i page .. (i + 1) page - 1; the others are -1.  The free
 * pages are a stack: places 0 .. free_count - 1 of free_list, the top last; the others are -1. */
typedef struct {
  int32_t page;        /* tokens of a page: 16, 32, 64, 128 or 256 */
  int32_t batch;       /* sequences, 1 .. 4096 */
  int32_t width;       /* entries of a row; width * page <= 2^22 */
  int32_t pages;       /* pages of the pool, >= 1; pages * page <= 2^40 */
  int32_t *table;      /* [batch][width] */
  int64_t *length;     /* [batch] */
  int32_t *free_list;  /* [pages] */
  int32_t *free_count; /* [1] */
} qwm_page_table;

/* No sequence has tokens and every page is free, page 0 on top. */
QWM_API qwm_status qwm_pages_reset(qwm_ctx *ctx, const qwm_page_table *tab, qwm_stream stream);

/* First every sequence is shortened to keep[b] tokens (0 or less ends it; more than it has changes nothing), then
 * count[b] new ones are appended (0 or less: none).  New pages are taken from the top of the stack by sequence
 * and place; pages given up return so that they would come out again in the same order.
 * A sequence is refused whole (granted[b] = 0, its length as kept) when its rows pass n, its pages pass the table's
 * width, or it needs pages and there are not enough for it and every sequence before it that needs some and
 * was not refused for another reason.
 *   keep     device int64 [batch], or NULL to shorten none
 *   count    device int32 [batch], or NULL to append nothing (then n is 0 and the four below may be NULL)
 *   first    device int32 [batch]: the sum of the counts before it, refused ones counted (2^31 - 1 at most)
 *   granted  device int32 [batch]: count[b], or 0
 *   slot     device int64 [n]: page * tab.page + place of the row's token, or -1 (padding, refused)
 *   at       device int64 [n]: its position, or -1
 * A length outside 0 .. width * page counts as the nearer end and records QWM_ERR_RANGE. */
QWM_API qwm_status qwm_pages_update(qwm_ctx *ctx, const qwm_page_table *tab, const int64_t *keep, const int32_t *count,
                                    int64_t n, int32_t *first, int32_t *granted, int64_t *slot, int64_t *at,
                                    qwm_stream stream);

/* ------------------------------------------------------------------ the paged cache */

/* One layer's pages: codes and steps as in qwm_window, slot s = (page s / page, place s % page). */
typedef struct {
  int32_t bits;     /* 8 or 4 */
  int32_t page;     /* as qwm_page_table */
  int32_t pages;    /* >= 1 */
  int32_t kv_heads; /* >= 1 */
  uint8_t *k_codes, *v_codes; /* [pages][kv_heads][page][128 * bits / 8] */
  uint8_t *k_step, *v_step;   /* [pages][kv_heads][page][4] */
} qwm_page_pool;

/* Keys normed (weight or norm given), turned (rope given) and rounded to bf16 as qwm_norm_rope does, or as they
 * come; then Keys and Values quantised as by qwm_window_write, token i into slot[i].
 *   k, v    bf16 [kv_heads][n][128] by ks and vs
 *   slot    device int64 [n]: rows with -1 (or any negative one) are skipped, rows beyond the pool too, recording
 *           QWM_ERR_RANGE; otherwise distinct
 *   at, pos as qwm_norm_rope's with batch = 1, when rope is given (rows with a bad position are skipped)
 *   norm    1: divide by the root of the mean square;  0: do not (weight is then NULL)
 *   weight  fp32 [128], [kv_heads][128] (per_head == 1) or NULL */
QWM_API qwm_status qwm_paged_write(qwm_ctx *ctx, const qwm_page_pool *pool, const uint16_t *k, const qwm_strides *ks,
                                   const uint16_t *v, const qwm_strides *vs, int64_t n, const int64_t *slot,
                                   const qwm_rope_spec *rope, const int64_t *at, const int32_t *pos, int32_t norm,
                                   const float *weight, int32_t per_head, float eps, qwm_stream stream);

/* What slots stand for: k_hat, v_hat bf16 [kv_heads][n][128], dense (either may be NULL).  Negative slots read as
 * 0, slots beyond the pool too, recording QWM_ERR_RANGE. */
QWM_API qwm_status qwm_paged_read(qwm_ctx *ctx, const qwm_page_pool *pool, const int64_t *slot, int64_t n,
                                  uint16_t *k_hat, uint16_t *v_hat, qwm_stream stream);

/* ------------------------------------------------------------------ attention */

/* Query row first[b] + i of the packed batch is the token of sequence b at position p = length[b] - count[b] + i
 * (lengths count the new tokens: as qwm_pages_update leaves them), in frame p / tpf.  It sees token j < length[b]
 * when its frame is not later (j / tpf <= p / tpf) and it is recent (p / tpf - j / tpf < frames) or a sink
 * (j < sink).  tpf = 1: causal, a window of `frames` tokens; frames = 2^31: no window.
 * Sequences with count[b] <= 0 have no rows; rows at n and beyond are cut off; a sequence with first[b] < 0 or with
 * fewer tokens than rows is left out; one longer than width * page is left out and QWM_ERR_RANGE recorded.
 * A page outside the pool is read as page 0 and records QWM_ERR_RANGE.
 *   tab        table and length are used
 *   q          bf16 [H][n][128] by qs, H = config.heads, a multiple of kv_heads (grouped as qwm_window_attend's)
 *   max_count  the largest count, or more: what the call's kernels are chosen by.  A sequence with more new
 *              tokens than that is left out and QWM_ERR_RANGE recorded.
 *   softmax_scale, out (bf16 or fp32 [H][n][128] by os), merge  as qwm_window_attend's
 *   lse        fp32 [H][n] dense, or NULL
 *   ws         workspace of qwm_paged_attend_workspace bytes, free again when the call's work on the stream is
 *              done.  Calls (and captured graphs) that may run at the same time need their own.
 * Queries and weights enter the products as in qwm_window_attend: Queries off by at most 2^-25 of their row's largest
 * element, weights in fp16, rounded by at most 2^-11 of their value or 2^-32 of the largest weight of their piece, whichever
 * is more (with out_f32 the largest error beside the cache's own).  Logits, maxima, sums and the output are accumulated in
 * fp32, over pieces of 2^18 keys at most, which are joined. */
QWM_API qwm_status qwm_paged_attend(qwm_ctx *ctx, const qwm_page_pool *pool, const qwm_page_table *tab, const uint16_t *q,
                                    const qwm_strides *qs, int64_t n, const int32_t *first, const int32_t *count,
                                    int64_t max_count, int64_t tpf, int64_t frames, int64_t sink, float softmax_scale,
                                    void *out, const qwm_strides *os, int32_t out_f32, float *lse, int32_t merge, void *ws,
                                    size_t ws_bytes, qwm_stream stream);
/* Bytes for calls of up to max_count new tokens a sequence (0 for a call that would be refused or does nothing). */
QWM_API size_t qwm_paged_attend_workspace(const qwm_ctx *ctx, const qwm_page_pool *pool, int64_t max_count);

#ifdef __cplusplus
}
#endif
#endif /* QWM_PAGED_H_ */
