// The window cache: Keys and Values quantised to 8 or 4 bits as they are written, and read back.
//
// Per (token, head), groups of 32 channels: s = the smallest step with Q s >= max|x|, code = rint(x / s).
// A step has 4 significant bits, so code * s has at most 11 and is exact in fp16, whatever reads it.
// Bound: memory (write: 512 B of bf16 read and 264 or 136 B written per token and head; read: the
// reverse).  16 lanes take one row, 8 channels each; four of them share a step, found by two shuffles.
#include "window.cuh"

namespace {

constexpr int kThreads = 256, kRows = kThreads / 16;

__device__ __forceinline__ bool bf16x2_nonfinite(uint32_t w) {
  return (w & 0x7F80u) == 0x7F80u || (w & 0x7F800000u) == 0x7F800000u;
}

// Eight bf16 channels of a row (4 words) -> this lane's code bytes (8 bits: c0, c1; 4 bits: c0) and the
// group's step byte.  Every lane of the warp takes part.
template <int BITS>
__device__ __forceinline__ void quantise(const uint32_t (&w)[4], uint32_t &c0, uint32_t &c1, uint32_t &step,
                                         bool &bad) {
  constexpr float Q = win::code_max(BITS);
  float f[8], amax = 0.f;
#pragma unroll
  for (int i = 0; i < 4; i++) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
#pragma unroll
  for (int i = 0; i < 8; i++) amax = fmaxf(amax, fabsf(f[i]));   // fmaxf passes over a NaN
  amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
  amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
  constexpr float kTop = Q * (BITS == 8 ? 56.f : 896.f);
  bool out = amax > kTop;
#pragma unroll
  for (int i = 0; i < 4; i++) out |= bf16x2_nonfinite(w[i]);
  if (out) {   // cut to the range, NaN to 0
    bad = true;
#pragma unroll
    for (int i = 0; i < 8; i++) f[i] = isnan(f[i]) ? 0.f : fminf(fmaxf(f[i], -kTop), kTop);
  }
  step = win::step_for<BITS>(amax);
  const float s = win::step_value(step), inv = s > 0.f ? __frcp_rn(s) : 0.f;
  uint32_t c[8];
#pragma unroll
  for (int i = 0; i < 8; i++) c[i] = win::code_of(f[i], inv, BITS == 8 ? 128.f : 8.f);
  if (BITS == 8) {
    c0 = c[0] | (c[1] << 8) | (c[2] << 16) | (c[3] << 24);
    c1 = c[4] | (c[5] << 8) | (c[6] << 16) | (c[7] << 24);
  } else {   // channel 2 k + t in nibble k + 4 t
    c0 = c[0] | (c[2] << 4) | (c[4] << 8) | (c[6] << 12) | (c[1] << 16) | (c[3] << 20) | (c[5] << 24) | (c[7] << 28);
    c1 = 0u;
  }
}

template <int BITS>
__device__ __forceinline__ void store_row(uint8_t *codes, uint8_t *steps, int64_t slot_row, int v, uint32_t c0,
                                          uint32_t c1, uint32_t step) {
  if (BITS == 8) *(uint2 *)(codes + slot_row * win::D + 8 * v) = make_uint2(c0, c1);
  else *(uint32_t *)(codes + slot_row * (win::D / 2) + 4 * v) = c0;
  if ((v & 3) == 0) steps[slot_row * win::kSteps + (v >> 2)] = (uint8_t)step;
}

// TURN: -1 Keys are stored as they come, else the pairing they are turned by.
template <int BITS, int TURN>
__global__ void __launch_bounds__(kThreads)
    window_write_kernel(const __grid_constant__ qwm_rope_spec sp, qwm_window w, const uint16_t *__restrict__ k,
                        qwm_strides ks, const uint16_t *__restrict__ vv, qwm_strides vs, int64_t n,
                        const int64_t *__restrict__ start, const int32_t *__restrict__ count,
                        const int32_t *__restrict__ pos, int heads_per_block, int32_t *status) {
  const int v = threadIdx.x & 15, row = threadIdx.x >> 4;
  const int64_t tok = (int64_t)blockIdx.x * kRows + row;
  const bool in = tok < (int64_t)w.batch * n;
  const int64_t b = in ? tok / n : 0, i = in ? tok - b * n : 0;
  const int64_t s0 = start[b];
  int64_t cnt = count ? (int64_t)count[b] : n;
  cnt = cnt < n ? cnt : n;
  const int64_t p = s0 + i, end = s0 + cnt;
  // of tokens that share a slot the last of the call is kept
  const bool live = in && s0 >= 0 && i < cnt && (p < w.sink || p >= end - w.ring);
  if (!__any_sync(0xffffffffu, live)) return;
  win::RopeVec<TURN == QWM_ROPE_HALF ? QWM_ROPE_HALF : QWM_ROPE_INTERLEAVED> rv;
  if (TURN >= 0) rv.init(sp, v, live ? p : 0, pos ? pos + (b * n + i) * 3 : nullptr);
  const int64_t slots = w.sink + w.ring;
  const int64_t slot = live ? (p < w.sink ? p : w.sink + (p - w.sink) % w.ring) : 0;
  const int h0 = blockIdx.y * heads_per_block;
  const int h1 = h0 + heads_per_block < w.kv_heads ? h0 + heads_per_block : w.kv_heads;
  const uint16_t *kp = k + b * ks.batch + i * ks.token + 8 * v, *vp = vv + b * vs.batch + i * vs.token + 8 * v;
  bool bad = false;
#pragma unroll 2
  for (int h = h0; h < h1; h++) {
    uint4 a = make_uint4(0, 0, 0, 0), c = a;
    if (live) {
      a = *(const uint4 *)(kp + (int64_t)h * ks.head);
      c = *(const uint4 *)(vp + (int64_t)h * vs.head);
    }
    uint32_t kw[4] = {a.x, a.y, a.z, a.w}, vw[4] = {c.x, c.y, c.z, c.w};
    if (TURN >= 0) rv.turn(sp, kw);
    uint32_t c0, c1, step;
    const int64_t slot_row = (b * w.kv_heads + h) * slots + slot;
    quantise<BITS>(kw, c0, c1, step, bad);
    if (live) store_row<BITS>(w.k_codes, w.k_step, slot_row, v, c0, c1, step);
    quantise<BITS>(vw, c0, c1, step, bad);
    if (live) store_row<BITS>(w.v_codes, w.v_step, slot_row, v, c0, c1, step);
  }
  if (bad && live) qwm_dev_error(status, QWM_ERR_RANGE);
}

template <int BITS>
__global__ void __launch_bounds__(kThreads)
    window_read_kernel(qwm_window w, const int64_t *__restrict__ start, const int64_t *__restrict__ length,
                       const int32_t *__restrict__ count, int64_t n, uint16_t *__restrict__ k_hat,
                       uint16_t *__restrict__ v_hat, int heads_per_block, win::Bases bases) {
  const int v = threadIdx.x & 15, row = threadIdx.x >> 4;
  const int64_t tok = (int64_t)blockIdx.x * kRows + row;
  if (tok >= (int64_t)w.batch * n) return;
  const int64_t b = tok / n, i = tok - b * n;
  const int64_t s0 = start[b], len = length[b], p = s0 + i;
  if (s0 < 0 || (count && i >= count[b])) return;
  const bool held = p < len && (p < w.sink || p >= len - w.ring);
  const int64_t slots = w.sink + w.ring;
  const int64_t slot = held ? (p < w.sink ? p : w.sink + (p - w.sink) % w.ring) : 0;
  const int h0 = blockIdx.y * heads_per_block;
  const int h1 = h0 + heads_per_block < w.kv_heads ? h0 + heads_per_block : w.kv_heads;
#pragma unroll 2
  for (int h = h0; h < h1; h++) {
    const int64_t bh = b * w.kv_heads + h, r = bh * slots + slot;
#pragma unroll
    for (int t = 0; t < 2; t++) {
      uint16_t *dst = t ? v_hat : k_hat;
      const uint8_t *codes = t ? w.v_codes : w.k_codes, *steps = t ? w.v_step : w.k_step;
      if (!dst) continue;
      uint32_t o[4] = {0u, 0u, 0u, 0u};
      if (held) {
        uint32_t s2, n2, pr[4];
        win::step_consts<BITS>(steps[r * win::kSteps + (v >> 2)], s2, n2);
        if (BITS == 8) {
          const uint2 x = *(const uint2 *)(codes + r * win::D + 8 * v);
          win::decode8(x.x, s2, n2, bases, pr[0], pr[1]);
          win::decode8(x.y, s2, n2, bases, pr[2], pr[3]);
        } else {
          win::decode4(*(const uint32_t *)(codes + r * (win::D / 2) + 4 * v), s2, n2, bases, pr);
        }
#pragma unroll
        for (int u = 0; u < 4; u++) {
          const float2 f = __half22float2(*(const __half2 *)&pr[u]);
          o[u] = tc::pack_bf16x2(f.x, f.y);
        }
      }
      *(uint4 *)(dst + (bh * n + i) * win::D + 8 * v) = make_uint4(o[0], o[1], o[2], o[3]);
    }
  }
}

int heads_per_block(int64_t tiles, int heads, int num_sms) {
  const int64_t h = tiles * heads / (8 * (int64_t)num_sms);
  return (int)(h < 1 ? 1 : (h > 8 ? 8 : h));
}

template <int BITS>
cudaError_t write_bits(const qwm_window &w, const uint16_t *k, const qwm_strides &ks, const uint16_t *v,
                       const qwm_strides &vs, int64_t n, const int64_t *start, const int32_t *count,
                       const qwm_rope_spec *rope, const int32_t *pos, int num_sms, int32_t *status, cudaStream_t st) {
  const int64_t tiles = ((int64_t)w.batch * n + kRows - 1) / kRows;
  const int hpb = heads_per_block(tiles, w.kv_heads, num_sms);
  const dim3 grid((unsigned)tiles, (unsigned)((w.kv_heads + hpb - 1) / hpb));
  const qwm_rope_spec none = {};
  if (!rope)
    window_write_kernel<BITS, -1><<<grid, kThreads, 0, st>>>(none, w, k, ks, v, vs, n, start, count, pos, hpb, status);
  else if (rope->pairing == QWM_ROPE_INTERLEAVED)
    window_write_kernel<BITS, QWM_ROPE_INTERLEAVED>
        <<<grid, kThreads, 0, st>>>(*rope, w, k, ks, v, vs, n, start, count, pos, hpb, status);
  else
    window_write_kernel<BITS, QWM_ROPE_HALF>
        <<<grid, kThreads, 0, st>>>(*rope, w, k, ks, v, vs, n, start, count, pos, hpb, status);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_window_write(const qwm_window &w, const uint16_t *k, const qwm_strides &ks, const uint16_t *v,
                                const qwm_strides &vs, int64_t n, const int64_t *start, const int32_t *count,
                                const qwm_rope_spec *rope, const int32_t *pos, int num_sms, int32_t *status,
                                cudaStream_t st) {
  return w.bits == 8 ? write_bits<8>(w, k, ks, v, vs, n, start, count, rope, pos, num_sms, status, st)
                     : write_bits<4>(w, k, ks, v, vs, n, start, count, rope, pos, num_sms, status, st);
}

cudaError_t launch_window_read(const qwm_window &w, const int64_t *start, const int64_t *length, const int32_t *count,
                               int64_t n, uint16_t *k_hat, uint16_t *v_hat, int num_sms, cudaStream_t st) {
  const int64_t tiles = ((int64_t)w.batch * n + kRows - 1) / kRows;
  const int hpb = heads_per_block(tiles, w.kv_heads, num_sms);
  const dim3 grid((unsigned)tiles, (unsigned)((w.kv_heads + hpb - 1) / hpb));
  if (w.bits == 8)
    window_read_kernel<8><<<grid, kThreads, 0, st>>>(w, start, length, count, n, k_hat, v_hat, hpb, win::kBases);
  else
    window_read_kernel<4><<<grid, kThreads, 0, st>>>(w, start, length, count, n, k_hat, v_hat, hpb, win::kBases);
  return cudaGetLastError();
}
