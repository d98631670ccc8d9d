/*
 * qwm_window.h -- the recent window beside the packed history, in libqwm.so: rotary positions with
 * three axes, a window cache quantised to 8 or 4 bits as it is written, and attention over it with a
 * sliding window and sink tokens.
 *
 * The 2-bit path (qwm.h) packs a chunk once it is complete.  These calls serve what it leaves open:
 *  - the positions of the tokens: qwm_rope turns Queries and Keys by their place in time, height and
 *    width before they are packed or attended;
 *  - the recent tokens: qwm_window_write appends Keys and Values token by token (or frame by frame)
 *    to a ring at 8 or 4 bits, qwm_window_read hands them back in bf16 (to be packed as a chunk once
 *    they leave the window), and qwm_window_attend attends over the ring and the first tokens, alone
 *    or merged into a qwm_attend_merge result over the packed history.
 *
 * Conventions as in qwm.h (device pointers, caller-owned, 16-byte aligned, bf16 as uint16_t bit
 * patterns, asynchronous on the stream, a qwm_status return), and further:
 *  - Activations have shape [batch][heads][tokens][128] with the channels contiguous and the other
 *    three strides given (qwm_strides, in elements, multiples of 8, at most 2^38), so that a projection's
 *    token-major output needs no transposition.  Rows that a call writes must not overlap.
 *  - What changes from step to step is read on the device (start, count, length: one entry per
 *    sequence), so a captured CUDA graph of a step can be replayed with new values in the same
 *    buffers.  A sequence whose start (q_start) is negative or above 2^62, or whose count is 0 or less,
 *    is skipped: its rows are left as they were.  A negative length counts as 0.  With count, rows from count[b] on are padding and left as they were.
 *  - Errors only the device sees (QWM_ERR_RANGE, QWM_ERR_DEVICE_TIMEOUT) go to the context's status
 *    word (qwm_sync_status).
 *  - The calls use no memory of the context but the status word: calls on different streams need
 *    ordering only by their own data.  The context's device must be the one the pointers belong to;
 *    it need not be the current one.
 */
#ifndef QWM_WINDOW_H_
#define QWM_WINDOW_H_

#include "qwm.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element strides of an activation [batch][heads][tokens][128]. */
typedef struct {
  int64_t batch, head, token;
} qwm_strides;

/* ------------------------------------------------------------------ rotary positions */

/* How the two channels of pair i are found among the R rotated channels. */
enum { QWM_ROPE_INTERLEAVED = 0, /* 2 i and 2 i + 1 */
       QWM_ROPE_HALF = 1 };      /* i and i + R / 2 */

/* A rotation, made by qwm_rope_plan (host) and passed to every call that turns by it. */
typedef struct {
  int32_t rot;            /* R, channels turned: 0..R-1; the others pass through */
  int32_t pairing;        /* QWM_ROPE_INTERLEAVED or QWM_ROPE_HALF */
  int32_t grid_h, grid_w; /* token p of a sequence has t = p / (grid_h grid_w), y = p / grid_w % grid_h,
                             x = p % grid_w */
  uint64_t turn[64];      /* pair i: the part of a full turn per unit of position, times 2^64 */
  uint8_t axis[64];       /* pair i: 0 (t), 1 (y) or 2 (x) */
} qwm_rope_spec;

/* Host-only: fill `out`.  Pair j of axis a turns by position_a * theta[a]^(-2 j / axis_dim[a]) radians
 * (shared_freq == 0), or by position_a * theta[a]^(-2 i / R) with i the pair's number over all axes
 * (shared_freq == 1).
 *   axis_dim  channels of the t, y and x sections: even, >= 0, sum R <= 128 (QWM_ROPE_HALF: R a
 *             multiple of 16)
 *   theta     base of each axis with channels: finite, >= 1
 *   inverse   1: turn by the negative angle (undoes the rotation; the gradient of the rotation) */
QWM_API qwm_status qwm_rope_plan(const int32_t axis_dim[3], const double theta[3], int32_t pairing,
                                 int32_t shared_freq, int32_t grid_h, int32_t grid_w, int32_t inverse,
                                 qwm_rope_spec *out);

/* out = x turned by its positions, rounded to bf16 (nearest-even).  An infinite or NaN channel makes its pair
 * what a c - b s and a s + b c are in IEEE arithmetic (c, s: cosine and sine), and no other channel.
 *   x, out  bf16 [batch][heads][n][128] by xs and os; out may be x itself (same strides)
 *   start   device int64 [batch]: position of token 0 of each sequence
 *   pos     device int32 [batch][n][3] (t, y, x) to use instead of the grid's, or NULL
 * Angles are formed as fractions of a turn in 64-bit integers: beside the rounding of the turns per position,
 * at most 2^-65 (so p 2^-65 turns at position p, 2^-26 radians up to 2^36), far positions lose nothing. */
QWM_API qwm_status qwm_rope(qwm_ctx *ctx, const qwm_rope_spec *spec, const uint16_t *x, const qwm_strides *xs,
                            int32_t batch, int32_t heads, int64_t n, const int64_t *start, const int32_t *pos,
                            uint16_t *out, const qwm_strides *os, qwm_stream stream);

/* ------------------------------------------------------------------ the window cache */

/* Slots 0..sink-1 keep the first `sink` tokens of a sequence; token p >= sink lives in slot
 * sink + (p - sink) % ring, so a sequence of `length` tokens holds those and its last `ring` others.
 * Per token and head, groups of 32 channels share a step s; a channel is s times a signed code in
 * -127..127 (8 bits) or -7..7 (4 bits), exact in fp16.
 *   codes: 8 bits: byte c = code + 128; 4 bits: channel 8 j + 2 k + t is nibble k + 4 t (from the low
 *          end) of 32-bit word j = code + 8
 *   step:  one byte, the fp16 bits of s shifted right by 7 (5 exponent and 3 mantissa bits) */
typedef struct {
  int32_t bits;      /* 8 or 4 */
  int32_t batch;     /* sequences, >= 1 */
  int32_t kv_heads;  /* >= 1 */
  int32_t reserved;  /* 0 */
  int64_t sink;      /* >= 0 */
  int64_t ring;      /* >= 1; sink + ring <= 2^30 */
  uint8_t *k_codes, *v_codes; /* [batch][kv_heads][sink + ring][128 * bits / 8] */
  uint8_t *k_step, *v_step;   /* [batch][kv_heads][sink + ring][4] */
} qwm_window;

/* Bytes of one codes array and of one step array of this window; QWM_ERR_* for a bad shape (host-only;
 * the pointers are not looked at). */
QWM_API qwm_status qwm_window_bytes(const qwm_window *win, size_t *codes, size_t *step);

/* Append tokens start[b] .. start[b] + count[b] - 1 of every sequence.  Keys are first turned by `rope`
 * (when given) and rounded to bf16, as qwm_rope would.  s is the smallest step with
 * Q s >= max|x| (Q = 127 or 7) and the code rint(x / s), ties to even, so |x - s code| <= s / 2.  An
 * element beyond 127 * 56 (8 bits) or 7 * 896 (4 bits) is cut to that, a NaN becomes 0, and
 * QWM_ERR_RANGE is recorded.  Of tokens of one call that share a slot the last is kept.
 *   k, v   bf16 [batch][kv_heads][n][128] by ks and vs
 *   start  device int64 [batch];  count  device int32 [batch] (0..n), or NULL for n
 *   rope   or NULL;  pos  device int32 [batch][n][3], or NULL (as qwm_rope) */
QWM_API qwm_status qwm_window_write(qwm_ctx *ctx, const qwm_window *win, const uint16_t *k, const qwm_strides *ks,
                                    const uint16_t *v, const qwm_strides *vs, int64_t n, const int64_t *start,
                                    const int32_t *count, const qwm_rope_spec *rope, const int32_t *pos,
                                    qwm_stream stream);

/* What the cache stands for, for tokens start[b] .. start[b] + count[b] - 1 of sequences that have
 * length[b] tokens: k_hat, v_hat bf16 [batch][kv_heads][n][128], dense, rounded to nearest-even (either
 * may be NULL).  Tokens the cache does not hold (overwritten, or not yet written) read as 0. */
QWM_API qwm_status qwm_window_read(qwm_ctx *ctx, const qwm_window *win, const int64_t *start, const int64_t *length,
                                   const int32_t *count, int64_t n, uint16_t *k_hat, uint16_t *v_hat,
                                   qwm_stream stream);

/* ------------------------------------------------------------------ attention over the window cache */

/* Query row i of sequence b stands at position p = q_start[b] + i, in frame p / tpf.  It sees key j when
 * the cache holds it (j < length[b], and j < sink or j >= length[b] - ring), its frame is not later
 * (j / tpf <= p / tpf), and it is recent (p / tpf - j / tpf < frames) or a sink (j < sink).  tpf = 1 is
 * the causal mask by tokens with a window of `frames` tokens; tpf = the tokens of a frame is
 * block-causal over frames.
 *   q        bf16 [batch][H][nq][128] by qs, H = config.heads, a multiple of kv_heads (Query head h reads
 *            Key head h / (H / kv_heads)); an element beyond the fp16 range records QWM_ERR_RANGE
 *   q_start  device int64 [batch];  length  device int64 [batch];  q_count  device int32 [batch] or NULL
 *   softmax_scale  > 0, at most 2^123, multiplies the logits
 *   out      [batch][H][nq][128] by os: bf16 (out_f32 == 0) or fp32 (out_f32 == 1)
 *   lse      fp32 [batch][H][nq] dense: log2 of the sum over the keys of 2^(softmax_scale log2(e) l), as
 *            qwm_attend_merge's; or NULL
 *   merge    1: out (fp32) and lse hold a result over other keys of the same Queries and become the
 *            result over both;  0: they are written
 *   ws       workspace of qwm_window_attend_workspace bytes (may be NULL when that is 0), free again
 *            when the call's work on the stream is done
 * A row that sees no key gets out = 0 and lse = -inf (merge: stays as it was).  Queries enter the first product
 * off by at most 2^-25 of their row's largest element, whatever its magnitude.  Logits, maxima, sums and the
 * output are accumulated in fp32, over 2^18 keys at most (longer calls are made in parts, which are joined).
 * The weights enter the second product in fp16, rounded by at most 2^-11 of their value or 2^-32 of the
 * largest weight of their part, whichever is more. */
QWM_API qwm_status qwm_window_attend(qwm_ctx *ctx, const qwm_window *win, const uint16_t *q, const qwm_strides *qs,
                                     int64_t nq, const int64_t *q_start, const int64_t *length,
                                     const int32_t *q_count, int64_t tpf, int64_t frames, float softmax_scale,
                                     void *out, const qwm_strides *os, int32_t out_f32, float *lse, int32_t merge,
                                     void *ws, size_t ws_bytes, qwm_stream stream);
QWM_API size_t qwm_window_attend_workspace(const qwm_ctx *ctx, const qwm_window *win, int64_t nq, int64_t tpf,
                                           int64_t frames);

#ifdef __cplusplus
}
#endif
#endif /* QWM_WINDOW_H_ */
