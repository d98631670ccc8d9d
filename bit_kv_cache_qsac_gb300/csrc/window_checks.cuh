// What the C entry points of the window cache and of the paged cache check, and how they stand on their device.
#pragma once

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

// Per-sequence arrays: 8-byte (4-byte) elements at their natural alignment.
bool aligned_to(const void *p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

}  // namespace
