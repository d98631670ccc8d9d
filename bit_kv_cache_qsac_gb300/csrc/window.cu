// The window cache: Keys and Values quantised to 8 or 4 bits as they are written, and read back.
//
// Per (token, head), groups of 32 channels: s = the smallest step with Q s >= max|x|, code = rint(x / s).
// A step has 4 significant bits, so code * s has at most 11 and is exact in fp16, whatever reads it.
// Bound: memory (write: 512 B of bf16 read and 264 or 136 B written per token and head; read: the
// reverse).  16 lanes take one row, 8 channels each; four of them share a step, found by two shuffles.
// Measured, 40 heads x 10,800 tokens: written at 4 bits in 47 us, with the Keys turned by three axes in 62 (half
// pairing 68) = 4.5 TB/s; at 8 bits 53, 68 and 72.  Turned and at 4 bits 71% of the issue slots and half of the
// DRAM rate are in use: what remains is the chain of shuffles, step and reciprocal of each row.  Read back in
// 44 us = 6.3 TB/s (4 bits) and 51 = 6.6 (8 bits); 40 heads x 4,680 at 8 bits in 24.8 us = 5.9 TB/s.
#include "window.cuh"

namespace {

constexpr int kThreads = 256, kRows = kThreads / 16, kReadRows = kThreads / 8;

// Eight bf16 channels of a row (4 words) -> this lane's code bytes (8 bits: c0, c1; 4 bits: c0) and the
// group's step byte.  Every lane of the warp takes part.
template <int BITS>
__device__ __forceinline__ void quantise(const uint32_t (&w)[4], uint32_t &c0, uint32_t &c1, uint32_t &step,
                                         bool &bad) {
  constexpr float kTop = win::code_max(BITS) * (BITS == 8 ? 56.f : 896.f);
  uint32_t m = win::max_abs_bf16x2(win::max_abs_bf16x2(w[0], w[1]), win::max_abs_bf16x2(w[2], w[3]));
  m = win::max_abs_bf16x2(m, __shfl_xor_sync(0xffffffffu, m, 1));
  m = win::max_abs_bf16x2(m, __shfl_xor_sync(0xffffffffu, m, 2));
  m = win::max_abs_bf16x2(m, m >> 16);
  float amax = __uint_as_float((m & 0x7FFFu) << 16), f[8], s;
#pragma unroll
  for (int i = 0; i < 4; i++) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
  step = win::normal_step<BITS>(amax, s);
  const bool out = !(amax <= kTop);   // out of range or NaN, somewhere in the group
  if (__any_sync(0xffffffffu, out || win::step_is_small<BITS>(amax))) {
    if (out) {   // cut to the range, NaN to 0
      bad = true;
      amax = 0.f;
#pragma unroll
      for (int i = 0; i < 8; i++) {
        f[i] = isnan(f[i]) ? 0.f : fminf(fmaxf(f[i], -kTop), kTop);
        amax = fmaxf(amax, fabsf(f[i]));
      }
    }
    float a = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    amax = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 2));
    step = win::step_is_small<BITS>(amax) ? win::small_step<BITS>(amax, s) : win::normal_step<BITS>(amax, s);
  }
  float inv;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(s));
  inv = s > 0.f ? inv : 0.f;
  const uint64_t inv2 = win::pair2(inv, inv);
  uint32_t c[8];   // 0x4B400000 + code
#pragma unroll
  for (int i = 0; i < 4; i++) {
    const float2 v = win::split2(win::codes_of(win::pair2(f[2 * i], f[2 * i + 1]), inv2));
    c[2 * i] = __float_as_uint(v.x);
    c[2 * i + 1] = __float_as_uint(v.y);
  }
  if (BITS == 8) {   // low bytes, biased by 128: the sign bit flips
    c0 = __byte_perm(__byte_perm(c[0], c[1], 0x0040), __byte_perm(c[2], c[3], 0x0040), 0x5410) ^ 0x80808080u;
    c1 = __byte_perm(__byte_perm(c[4], c[5], 0x0040), __byte_perm(c[6], c[7], 0x0040), 0x5410) ^ 0x80808080u;
  } else {   // channel 2 k + t in nibble k + 4 t: the sum of (0x4B400000 + code) 16^n, less that of the
             // constants (modulo 2^32) and with 8 added in every nibble
    c0 = ((((((c[7] * 16u + c[5]) * 16u + c[3]) * 16u + c[1]) * 16u + c[6]) * 16u + c[4]) * 16u + c[2]) * 16u + c[0] +
         (0x88888888u - 0x3F400000u);
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

// TURN: -1 Keys are stored as they come, else the pairing they are turned by (WHOLE: all channels).
template <int BITS, int TURN, bool WHOLE>
__global__ void __launch_bounds__(kThreads)
    window_write_kernel(const __grid_constant__ qwm_rope_spec sp, qwm_window w, const uint16_t *__restrict__ k,
                        qwm_strides ks, const uint16_t *__restrict__ vv, qwm_strides vs, int64_t n,
                        const int64_t *__restrict__ start, const int32_t *__restrict__ count,
                        const int32_t *__restrict__ pos, int heads_per_block, int32_t *status) {
  __shared__ win::RopeTable tab;
  const int v = threadIdx.x & 15, row = threadIdx.x >> 4;
  const int64_t tok = (int64_t)blockIdx.x * kRows + row;
  const bool in = tok < (int64_t)w.batch * n;
  const int64_t b = in ? win::quotient(tok, n) : 0, i = in ? tok - b * n : 0;
  const int h0 = blockIdx.y * heads_per_block;
  const int h1 = h0 + heads_per_block < w.kv_heads ? h0 + heads_per_block : w.kv_heads;
  const uint16_t *kp = k + b * ks.batch + i * ks.token + h0 * ks.head + 8 * v;
  const uint16_t *vp = vv + b * vs.batch + i * vs.token + h0 * vs.head + 8 * v;
  uint4 a = *(const uint4 *)kp, c = *(const uint4 *)vp;   // in flight while the angles are formed
  const int64_t s0 = start[b];
  int64_t cnt = count ? (int64_t)count[b] : n;
  cnt = cnt < n ? cnt : n;
  const int64_t p = s0 + i, end = s0 + cnt;
  // of tokens that share a slot the last of the call is kept
  const bool live = in && win::starts(s0) && i < cnt && (p < w.sink || p >= end - w.ring);
  win::RopeVec<TURN == QWM_ROPE_HALF ? QWM_ROPE_HALF : QWM_ROPE_INTERLEAVED, WHOLE> rv;
  if (TURN >= 0) {
    tab.fill(sp);
    rv.init(sp, tab, v, live ? p : 0, pos ? pos + (b * n + i) * 3 : nullptr);
  }
  if (!__any_sync(0xffffffffu, live)) return;
  const bool all = __all_sync(0xffffffffu, live);
  const int64_t slots = w.sink + w.ring;
  const int64_t slot = live ? (p < w.sink ? p : w.sink + win::remainder(p - w.sink, w.ring)) : 0;
  int64_t slot_row = (b * w.kv_heads + h0) * slots + slot;
  bool bad = false;
  for (int h = h0; h < h1; h++) {
    uint32_t kw[4] = {a.x, a.y, a.z, a.w}, vw[4] = {c.x, c.y, c.z, c.w};
    if (h + 1 < h1) {   // the next head's rows
      kp += ks.head;
      vp += vs.head;
      a = *(const uint4 *)kp;
      c = *(const uint4 *)vp;
    }
    if (!all) {   // padding is not looked at
      if (!live) kw[0] = kw[1] = kw[2] = kw[3] = vw[0] = vw[1] = vw[2] = vw[3] = 0u;
    }
    if (TURN >= 0) rv.turn(sp, kw);
    uint32_t c0, c1, step;
    quantise<BITS>(kw, c0, c1, step, bad);
    if (live) store_row<BITS>(w.k_codes, w.k_step, slot_row, v, c0, c1, step);
    quantise<BITS>(vw, c0, c1, step, bad);
    if (live) store_row<BITS>(w.v_codes, w.v_step, slot_row, v, c0, c1, step);
    slot_row += slots;
  }
  if (bad && live) qwm_dev_error(status, QWM_ERR_RANGE);
}

// Eight channels of a cached row -> bf16 (4 words).
template <int BITS>
__device__ __forceinline__ uint4 restore(uint2 x, uint32_t step, const win::Bases &bases) {
  uint32_t pr[4], o[4];
  const win::Step st = win::step_of_byte<BITS>(step);
  if (BITS == 8) {
    win::decode8(x.x, st, bases, pr[0], pr[1]);
    win::decode8(x.y, st, bases, pr[2], pr[3]);
  } else {
    win::decode4(x.x, st, bases, pr);
  }
#pragma unroll
  for (int u = 0; u < 4; u++) {
    if (BITS == 4) pr[u] = win::hmul2(pr[u], 0x4C004C00u);   // times the unit, 16
    const float2 f = __half22float2(*(const __half2 *)&pr[u]);
    o[u] = tc::pack_bf16x2(f.x, f.y);
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

// Eight lanes take a row, vectors v and v + 8 of it each, so that every store instruction writes whole
// 128-byte lines; the loads of a head's Keys and Values are in flight together.
template <int BITS>
__global__ void __launch_bounds__(kThreads)
    window_read_kernel(qwm_window w, const int64_t *__restrict__ start, const int64_t *__restrict__ length,
                       const int32_t *__restrict__ count, int64_t n, uint16_t *__restrict__ k_hat,
                       uint16_t *__restrict__ v_hat, int heads_per_block, win::Bases bases) {
  const int v = threadIdx.x & 7, row = threadIdx.x >> 3;
  const int64_t tok = (int64_t)blockIdx.x * kReadRows + row;
  if (tok >= (int64_t)w.batch * n) return;
  const int64_t b = win::quotient(tok, n), i = tok - b * n;
  const int64_t s0 = start[b], len = win::tokens_of(length[b]), p = s0 + i;
  if (!win::starts(s0) || (count && i >= count[b])) return;
  const bool held = p < len && (p < w.sink || p >= len - w.ring);
  const int64_t slots = w.sink + w.ring;
  const int64_t slot = held ? (p < w.sink ? p : w.sink + win::remainder(p - w.sink, w.ring)) : 0;
  const int h0 = blockIdx.y * heads_per_block;
  const int h1 = h0 + heads_per_block < w.kv_heads ? h0 + heads_per_block : w.kv_heads;
  constexpr int kVec = BITS;   // bytes of a vector's codes
  const int64_t r0 = (b * w.kv_heads + h0) * slots + slot, o0 = ((b * w.kv_heads + h0) * n + i) * win::D + 8 * v;
  const uint8_t *codes[2] = {w.k_codes + r0 * (win::D * BITS / 8) + kVec * v, w.v_codes + r0 * (win::D * BITS / 8) + kVec * v};
  const uint8_t *steps[2] = {w.k_step + r0 * win::kSteps, w.v_step + r0 * win::kSteps};
  uint16_t *dst[2] = {k_hat ? k_hat + o0 : nullptr, v_hat ? v_hat + o0 : nullptr};
#pragma unroll 2
  for (int h = h0; h < h1; h++) {
    uint2 x[2][2];
    uint32_t st[2] = {0u, 0u};
#pragma unroll
    for (int t = 0; t < 2; t++) {
      x[t][0] = x[t][1] = BITS == 8 ? make_uint2(0x80808080u, 0x80808080u) : make_uint2(0x88888888u, 0u);   // codes of 0
      if (held && dst[t]) {
        st[t] = *(const uint32_t *)steps[t];
#pragma unroll
        for (int e = 0; e < 2; e++) {
          const uint8_t *c = codes[t] + 8 * kVec * e;
          if (BITS == 8) x[t][e] = *(const uint2 *)c;
          else x[t][e].x = *(const uint32_t *)c;
        }
      }
      codes[t] += slots * (win::D * BITS / 8);
      steps[t] += slots * win::kSteps;
    }
#pragma unroll
    for (int t = 0; t < 2; t++) {
      if (!dst[t]) continue;
      *(uint4 *)dst[t] = restore<BITS>(x[t][0], (st[t] >> (8 * (v >> 2))) & 0xFFu, bases);
      *(uint4 *)(dst[t] + 64) = restore<BITS>(x[t][1], (st[t] >> (8 * (2 + (v >> 2)))) & 0xFFu, bases);
      dst[t] += n * win::D;
    }
  }
}

template <int BITS>
cudaError_t write_bits(const qwm_window &w, const uint16_t *k, const qwm_strides &ks, const uint16_t *v,
                       const qwm_strides &vs, int64_t n, const int64_t *start, const int32_t *count,
                       const qwm_rope_spec *rope, const int32_t *pos, int num_sms, int32_t *status, cudaStream_t st) {
  const int64_t tiles = ((int64_t)w.batch * n + kRows - 1) / kRows;
  const int hpb = heads_per_block(tiles, w.kv_heads, num_sms, rope ? 9 : 20);
  const dim3 grid((unsigned)tiles, (unsigned)((w.kv_heads + hpb - 1) / hpb));
  const qwm_rope_spec none = {};
  auto kernel = window_write_kernel<BITS, -1, false>;
  if (rope && rope->pairing == QWM_ROPE_INTERLEAVED)
    kernel = rope->rot == win::D ? window_write_kernel<BITS, QWM_ROPE_INTERLEAVED, true>
                                 : window_write_kernel<BITS, QWM_ROPE_INTERLEAVED, false>;
  else if (rope)
    kernel = rope->rot == win::D ? window_write_kernel<BITS, QWM_ROPE_HALF, true>
                                 : window_write_kernel<BITS, QWM_ROPE_HALF, false>;
  kernel<<<grid, kThreads, 0, st>>>(rope ? *rope : none, w, k, ks, v, vs, n, start, count, pos, hpb, status);
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
  const int64_t tiles = ((int64_t)w.batch * n + kReadRows - 1) / kReadRows;
  const int hpb = heads_per_block(tiles, w.kv_heads, num_sms, 40);
  const dim3 grid((unsigned)tiles, (unsigned)((w.kv_heads + hpb - 1) / hpb));
  if (w.bits == 8)
    window_read_kernel<8><<<grid, kThreads, 0, st>>>(w, start, length, count, n, k_hat, v_hat, hpb, win::kBases);
  else
    window_read_kernel<4><<<grid, kThreads, 0, st>>>(w, start, length, count, n, k_hat, v_hat, hpb, win::kBases);
  return cudaGetLastError();
}
