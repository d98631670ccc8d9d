// C ABI of the recent window (include/qwm_window.h): argument checks and dispatch.  Nothing here
// allocates device memory; every check is made before the first CUDA call.
#include <math.h>
#include <string.h>

#include "window.cuh"

namespace {

bool aligned16(const void *p) { return ((uintptr_t)p & 15u) == 0; }
qwm_status cuda_status(cudaError_t e) { return e == cudaSuccess ? QWM_OK : QWM_ERR_CUDA; }

// The context's device current for the duration of a call.
struct DeviceGuard {
  int before = -1;
  cudaError_t err;
  explicit DeviceGuard(int device) {
    err = cudaGetDevice(&before);
    if (err == cudaSuccess && before != device) err = cudaSetDevice(device);
    else before = -1;
  }
  ~DeviceGuard() {
    if (before >= 0) cudaSetDevice(before);
  }
};

constexpr int64_t kMaxTokens = (int64_t)1 << 24;   // tokens of one call and sequence
constexpr int64_t kMaxSlots = (int64_t)1 << 30;    // of a cache and sequence: key numbers are 32 bits in the kernels
constexpr int64_t kMaxGridY = 65535;

// An activation [batch][heads][n][128] by strides; `written`: its rows must not overlap.
qwm_status check_rows(const void *p, const qwm_strides *s, int64_t batch, int64_t heads, int64_t n, bool written) {
  if (!p || !s) return QWM_ERR_ARG;
  if (!aligned16(p)) return QWM_ERR_ALIGN;
  const int64_t st[3] = {s->batch, s->head, s->token}, ex[3] = {batch, heads, n};
  for (int i = 0; i < 3; i++) {
    if (st[i] < 0 || st[i] > ((int64_t)1 << 38)) return QWM_ERR_ARG;
    if (st[i] & 7) return QWM_ERR_ALIGN;
  }
  if (!written) return QWM_OK;
  int64_t need = QWM_D;   // dimensions by ascending stride: each must step over all of the smaller ones
  bool used[3] = {false, false, false};
  for (int k = 0; k < 3; k++) {
    int at = -1;
    for (int i = 0; i < 3; i++)
      if (!used[i] && ex[i] > 1 && (at < 0 || st[i] < st[at])) at = i;
    if (at < 0) break;
    used[at] = true;
    if (st[at] < need) return QWM_ERR_ARG;
    need = st[at] * (ex[at] - 1) + need;
  }
  return QWM_OK;
}

qwm_status check_rope(const qwm_rope_spec *r) {
  if (!r) return QWM_ERR_ARG;
  if (r->pairing != QWM_ROPE_INTERLEAVED && r->pairing != QWM_ROPE_HALF) return QWM_ERR_ARG;
  if (r->rot < 0 || r->rot > QWM_D || (r->rot & 1)) return QWM_ERR_SHAPE;
  if (r->pairing == QWM_ROPE_HALF && (r->rot & 15)) return QWM_ERR_SHAPE;
  if (r->grid_h < 1 || r->grid_w < 1) return QWM_ERR_ARG;
  for (int i = 0; i < r->rot / 2; i++)
    if (r->axis[i] > 2) return QWM_ERR_ARG;
  return QWM_OK;
}

qwm_status check_shape(const qwm_window *w) {
  if (!w) return QWM_ERR_ARG;
  if (w->bits != 8 && w->bits != 4) return QWM_ERR_UNSUPPORTED;
  if (w->batch < 1 || w->kv_heads < 1 || w->reserved != 0 || w->sink < 0 || w->ring < 1) return QWM_ERR_ARG;
  if (w->sink > kMaxSlots || w->ring > kMaxSlots || w->sink + w->ring > kMaxSlots) return QWM_ERR_SHAPE;
  if ((int64_t)w->batch * w->kv_heads > kMaxGridY) return QWM_ERR_SHAPE;
  return QWM_OK;
}

qwm_status check_window(const qwm_window *w) {
  const qwm_status s = check_shape(w);
  if (s != QWM_OK) return s;
  const void *req[] = {w->k_codes, w->v_codes, w->k_step, w->v_step};
  for (const void *p : req) {
    if (!p) return QWM_ERR_ARG;
    if (!aligned16(p)) return QWM_ERR_ALIGN;
  }
  return QWM_OK;
}

// Per-sequence arrays: 8-byte (4-byte) elements at their natural alignment.
bool aligned_to(const void *p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

// theta^(-j / half) / (2 pi) turns in units of 2^-64, rounded once: a double's 53 bits would leave an error of up
// to 2^8 units, which every unit of position multiplies.  One Newton step from the double r of pow(): the
// product r^half theta^j is 1 + d, so the root is r (1 - d / half); the product is taken in pairs of doubles
// (an unevaluated sum hi + lo), each factor in the order that keeps it near 1.
uint64_t turn_of(double theta, int j, int half) {
  const double r = pow(theta, -(double)j / half);
  if (r < 0x1p-64) return 0;   // less than half a unit
  double hi = 1.0, lo = 0.0;
  for (int a = half, b = j; a > 0 || b > 0;) {
    const bool up = b > 0 && (hi < 1.0 || a == 0);
    const double f = up ? theta : r, p = hi * f, e = fma(hi, f, -p) + lo * f;
    up ? b-- : a--;
    hi = p + e;
    lo = e - (hi - p);
  }
  const double rl = -r * ((hi - 1.0) + lo) / half;                                    // the root is r + rl
  const double kTurn = 0x1.45f306dc9c883p-3, kTurnLo = -0x1.6b01ec5417056p-57;        // 1 / (2 pi)
  const double t = r * kTurn, tl = fma(r, kTurn, -t) + (r * kTurnLo + rl * kTurn);
  const double units = t * 0x1p64, whole = floor(units);
  return (uint64_t)whole + (uint64_t)(int64_t)floor((units - whole) + tl * 0x1p64 + 0.5);
}

// The most keys a call's rows can see between them.
int64_t most_keys(const qwm_window &w, int64_t nq, int64_t tpf, int64_t frames) {
  const int64_t span = (nq + tpf - 1) / tpf + 1;   // frames the Queries stand in, at most
  int64_t recent = w.ring;
  if (frames + span < (w.ring + tpf - 1) / tpf) recent = (frames + span) * tpf;
  return w.sink + recent;
}

}  // namespace

extern "C" {

qwm_status qwm_rope_plan(const int32_t axis_dim[3], const double theta[3], int32_t pairing, int32_t shared_freq,
                         int32_t grid_h, int32_t grid_w, int32_t inverse, qwm_rope_spec *out) {
  if (!axis_dim || !theta || !out) return QWM_ERR_ARG;
  if ((shared_freq != 0 && shared_freq != 1) || (inverse != 0 && inverse != 1)) return QWM_ERR_ARG;
  qwm_rope_spec r;
  memset(&r, 0, sizeof(r));
  for (int a = 0; a < 3; a++) {
    if (axis_dim[a] < 0 || axis_dim[a] > QWM_D || (axis_dim[a] & 1)) return QWM_ERR_SHAPE;
    if (axis_dim[a] > 0 && !(theta[a] >= 1.0 && theta[a] <= 1e300)) return QWM_ERR_ARG;
    r.rot += axis_dim[a];
  }
  if (r.rot > QWM_D) return QWM_ERR_SHAPE;
  r.pairing = pairing;
  r.grid_h = grid_h;
  r.grid_w = grid_w;
  int i = 0;
  for (int a = 0; a < 3; a++)
    for (int j = 0; j < axis_dim[a] / 2; j++, i++) {
      const uint64_t t = shared_freq ? turn_of(theta[a], i, r.rot / 2) : turn_of(theta[a], j, axis_dim[a] / 2);
      r.turn[i] = inverse ? 0 - t : t;
      r.axis[i] = (uint8_t)a;
    }
  const qwm_status s = check_rope(&r);
  if (s != QWM_OK) return s;
  *out = r;
  return QWM_OK;
}

qwm_status qwm_rope(qwm_ctx *ctx, const qwm_rope_spec *spec, const uint16_t *x, const qwm_strides *xs, int32_t batch,
                    int32_t heads, int64_t n, const int64_t *start, const int32_t *pos, uint16_t *out,
                    const qwm_strides *os, qwm_stream stream) {
  if (!ctx || batch < 0 || heads < 0 || n < 0) return QWM_ERR_ARG;
  qwm_status s = check_rope(spec);
  if (s != QWM_OK) return s;
  if (batch > kMaxGridY || heads > kMaxGridY || n > kMaxTokens) return QWM_ERR_SHAPE;
  if ((int64_t)batch * n >= ((int64_t)1 << 34)) return QWM_ERR_SHAPE;
  if (batch == 0 || heads == 0 || n == 0) return QWM_OK;
  if ((s = check_rows(x, xs, batch, heads, n, false)) != QWM_OK) return s;
  if ((s = check_rows(out, os, batch, heads, n, true)) != QWM_OK) return s;
  if (!start) return QWM_ERR_ARG;
  if (!aligned_to(start, 8) || (pos && !aligned_to(pos, 4))) return QWM_ERR_ALIGN;
  if (x == out && (xs->batch != os->batch || xs->head != os->head || xs->token != os->token)) return QWM_ERR_ARG;
  DeviceGuard dev(ctx->device);
  if (dev.err != cudaSuccess) return QWM_ERR_CUDA;
  return cuda_status(launch_rope(*spec, x, *xs, batch, heads, n, start, pos, out, *os, ctx->num_sms,
                                 (cudaStream_t)stream));
}

qwm_status qwm_window_bytes(const qwm_window *win, size_t *codes, size_t *step) {
  const qwm_status s = check_shape(win);
  if (s != QWM_OK) return s;
  const size_t rows = (size_t)win->batch * win->kv_heads * (size_t)(win->sink + win->ring);
  if (codes) *codes = rows * QWM_D * win->bits / 8;
  if (step) *step = rows * win::kSteps;
  return QWM_OK;
}

qwm_status qwm_window_write(qwm_ctx *ctx, const qwm_window *win, const uint16_t *k, const qwm_strides *ks,
                            const uint16_t *v, const qwm_strides *vs, int64_t n, const int64_t *start,
                            const int32_t *count, const qwm_rope_spec *rope, const int32_t *pos, qwm_stream stream) {
  if (!ctx || n < 0) return QWM_ERR_ARG;
  qwm_status s = check_window(win);
  if (s == QWM_OK && rope) s = check_rope(rope);
  if (s != QWM_OK) return s;
  if (n > kMaxTokens || win->batch * n >= ((int64_t)1 << 34)) return QWM_ERR_SHAPE;
  if (n == 0) return QWM_OK;
  if ((s = check_rows(k, ks, win->batch, win->kv_heads, n, false)) != QWM_OK) return s;
  if ((s = check_rows(v, vs, win->batch, win->kv_heads, n, false)) != QWM_OK) return s;
  if (!start || (pos && !rope)) return QWM_ERR_ARG;
  if (!aligned_to(start, 8) || !aligned_to(count, 4) || !aligned_to(pos, 4)) return QWM_ERR_ALIGN;
  DeviceGuard dev(ctx->device);
  if (dev.err != cudaSuccess) return QWM_ERR_CUDA;
  return cuda_status(launch_window_write(*win, k, *ks, v, *vs, n, start, count, rope, pos, ctx->num_sms, ctx->status,
                                         (cudaStream_t)stream));
}

qwm_status qwm_window_read(qwm_ctx *ctx, const qwm_window *win, const int64_t *start, const int64_t *length,
                           const int32_t *count, int64_t n, uint16_t *k_hat, uint16_t *v_hat, qwm_stream stream) {
  if (!ctx || n < 0) return QWM_ERR_ARG;
  const qwm_status s = check_window(win);
  if (s != QWM_OK) return s;
  if (n > kMaxTokens || win->batch * n >= ((int64_t)1 << 34)) return QWM_ERR_SHAPE;
  if (n == 0 || (!k_hat && !v_hat)) return QWM_OK;
  if (!start || !length) return QWM_ERR_ARG;
  if (!aligned_to(start, 8) || !aligned_to(length, 8) || !aligned_to(count, 4) || !aligned16(k_hat) || !aligned16(v_hat))
    return QWM_ERR_ALIGN;
  DeviceGuard dev(ctx->device);
  if (dev.err != cudaSuccess) return QWM_ERR_CUDA;
  return cuda_status(launch_window_read(*win, start, length, count, n, k_hat, v_hat, ctx->num_sms, (cudaStream_t)stream));
}

static qwm_status check_attend(const qwm_ctx *ctx, const qwm_window *win, int64_t nq, int64_t tpf, int64_t frames) {
  if (!ctx || nq < 0) return QWM_ERR_ARG;
  const qwm_status s = check_shape(win);
  if (s != QWM_OK) return s;
  if (ctx->cfg.heads % win->kv_heads != 0) return QWM_ERR_SHAPE;
  if (tpf < 1 || frames < 1) return QWM_ERR_ARG;
  if (nq > kMaxTokens || tpf > ((int64_t)1 << 31) || frames > ((int64_t)1 << 31)) return QWM_ERR_SHAPE;
  if ((int64_t)win->batch * ctx->cfg.heads * nq > ((int64_t)1 << 36)) return QWM_ERR_SHAPE;   // Query rows
  return QWM_OK;
}

static WindowPlan plan_of(const qwm_ctx *ctx, const qwm_window *win, int64_t nq, int64_t tpf, int64_t frames) {
  return window_plan(win->batch, win->kv_heads, nq * (ctx->cfg.heads / win->kv_heads), most_keys(*win, nq, tpf, frames),
                     ctx->num_sms);
}

// The parts' outputs and log-sum-exps, when a second kernel joins them.
static size_t workspace_of(const qwm_ctx *ctx, const qwm_window *win, int64_t nq, const WindowPlan &p) {
  return p.joins() ? (size_t)win->batch * ctx->cfg.heads * (size_t)nq * p.splits * (QWM_D + 1) * sizeof(float) : 0;
}

size_t qwm_window_attend_workspace(const qwm_ctx *ctx, const qwm_window *win, int64_t nq, int64_t tpf, int64_t frames) {
  if (check_attend(ctx, win, nq, tpf, frames) != QWM_OK || nq == 0) return 0;
  return workspace_of(ctx, win, nq, plan_of(ctx, win, nq, tpf, frames));
}

qwm_status qwm_window_attend(qwm_ctx *ctx, const qwm_window *win, const uint16_t *q, const qwm_strides *qs, int64_t nq,
                             const int64_t *q_start, const int64_t *length, const int32_t *q_count, int64_t tpf,
                             int64_t frames, float softmax_scale, void *out, const qwm_strides *os, int32_t out_f32,
                             float *lse, int32_t merge, void *ws, size_t ws_bytes, qwm_stream stream) {
  qwm_status s = check_attend(ctx, win, nq, tpf, frames);
  if (s == QWM_OK) s = check_window(win);
  if (s != QWM_OK) return s;
  if (!(softmax_scale > 0.f) || softmax_scale > 0x1p123f) return QWM_ERR_ARG;   // (times 16 log2(e) it stays finite)
  if ((out_f32 != 0 && out_f32 != 1) || (merge != 0 && merge != 1)) return QWM_ERR_ARG;
  if (merge && (!out_f32 || !lse)) return QWM_ERR_ARG;
  if (nq == 0) return QWM_OK;
  const int H = ctx->cfg.heads;
  if ((s = check_rows(q, qs, win->batch, H, nq, false)) != QWM_OK) return s;
  if ((s = check_rows(out, os, win->batch, H, nq, true)) != QWM_OK) return s;
  if (!q_start || !length) return QWM_ERR_ARG;
  if (!aligned_to(q_start, 8) || !aligned_to(length, 8) || !aligned_to(q_count, 4) || !aligned_to(lse, 4))
    return QWM_ERR_ALIGN;
  const WindowPlan p = plan_of(ctx, win, nq, tpf, frames);
  const size_t need = workspace_of(ctx, win, nq, p);
  if (need > 0 && (!ws || ws_bytes < need)) return QWM_ERR_ARG;
  if (need > 0 && !aligned16(ws)) return QWM_ERR_ALIGN;
  DeviceGuard dev(ctx->device);
  if (dev.err != cudaSuccess) return QWM_ERR_CUDA;
  WindowAttend a;
  a.w = *win;
  a.q = q; a.qs = *qs; a.nq = nq;
  a.q_start = q_start; a.length = length; a.q_count = q_count;
  a.tpf = tpf; a.frames = frames;
  a.scale_log2 = softmax_scale * 1.4426950408889634f;
  a.out = out; a.os = *os; a.out_f32 = out_f32; a.merge = merge; a.lse = lse;
  a.status = ctx->status;
  a.H = H; a.group = H / win->kv_heads; a.rows = nq * a.group;
  a.splits = p.splits;
  a.cluster = p.cluster;
  a.bases = win::kBases;
  a.part = p.joins() ? (float *)ws : nullptr;
  a.part_lse = p.joins() ? a.part + (size_t)win->batch * H * (size_t)nq * p.splits * QWM_D : nullptr;
  const cudaStream_t st = (cudaStream_t)stream;
  cudaError_t e = p.tiles ? launch_window_tiles(a, st) : launch_window_decode(a, st);
  if (e == cudaSuccess && p.joins()) e = launch_window_combine(a, st);
  return cuda_status(e);
}

}  // extern "C"
