// Norms of Queries and Keys with the rotation in the same pass, and the paged cache: Keys and Values
// quantised into their slots, and read back.
//
//   y = x r w, r = 1 / sqrt(mean(x^2) + eps), then each pair (a, b) of channels becomes (a cos - b sin,
//   a sin + b cos), all in fp32, rounded to bf16 once.
// Bound: memory.  16 lanes take one row, 8 channels each; two heads' sums of squares are reduced together (four
// shuffles and two to hand the roots back instead of eight, and one root a lane instead of two); the angles depend on
// the token alone, so a thread forms those of its channels once and walks over `heads_per_block` heads with them, the
// next two heads' rows in flight.
// Measured, 40 heads x 10,800 tokens, three axes, weights per head: normed and turned in 46 us = 4.8 TB/s of rows read
// and written (72% of the issue slots: the rotation alone takes 37 us, the norm alone 38; with four heads in flight 54, with one
// 57, and with each head's weights fetched from global memory 55); in halves 54 us with shared weights and 69 with weights per
// head: each channel is normed twice, for its own lane and its partner's, and 64 registers do not hold both (80 to 96 bytes
// spilled).  Written at 4 bits 66 us = 4.2 TB/s, at 8 bits 71 (78% of the issue slots; its chain per row is the window cache's,
// and the norm's before it; in halves 73 and 75, normed only 55 and 61, as it comes 46 and 53); read back in 44 us = 6.3 TB/s
// (8 bits 52).  32 x 32 heads x 1 token: 4.2 us.
#include <math.h>

#include "paged.cuh"

namespace {

constexpr int kThreads = 256, kRows = kThreads / 16, kReadRows = kThreads / 8;
constexpr int kUnroll = 2;   // heads whose loads are in flight together

__device__ __forceinline__ float low(uint32_t x) { return __uint_as_float(x << 16); }
__device__ __forceinline__ float high(uint32_t x) { return __uint_as_float(x & 0xFFFF0000u); }

__device__ __forceinline__ uint64_t square_sum(const uint32_t (&w)[4], float f) {
  uint64_t acc = 0ull;
#pragma unroll
  for (int i = 0; i < 4; i++) {
    const uint64_t x = f == 1.f ? win::pair2(low(w[i]), high(w[i])) : win::pair2(low(w[i]) * f, high(w[i]) * f);
    acc = tc::fma2(x, x, acc);
  }
  return acc;
}
// 1 / sqrt(x): the approximation and a Newton step, which leaves about its own rounding.
__device__ __forceinline__ float inverse_root(float x) {
  const float r = rsqrtf(x);
  const float half = 0.5f * x * r;
  return x > 0x1p-120f && x < 0x1p120f ? fmaf(r, fmaf(-half, r, 0.5f), r) : r;
}
// A mean square beyond 2^120, or so small that squares were lost and eps does not cover them.
__device__ __forceinline__ bool out_of_range(float v, float eps) { return !(v <= 0x1p120f) || (v < 0x1p-80f && eps < 0x1p-70f); }

// A row whose squares leave fp32's range: the power of two s that brings it back, and r = 1 / sqrt(mean((x s)^2) +
// eps s^2); r of the row as it is and s = 1 for other rows.  w: this lane's 8 channels; all lanes of the warp take
// part.
__device__ __forceinline__ float2 scale_of_odd_row(const uint32_t (&w)[4], float eps) {
  auto squares = [&](float f) {
    const float2 a = win::split2(square_sum(w, f));
    float v = a.x + a.y;
#pragma unroll
    for (int d = 1; d < 16; d <<= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
    return v;
  };
  float v = squares(1.f), s = 1.f;
  uint32_t m = win::max_abs_bf16x2(win::max_abs_bf16x2(w[0], w[1]), win::max_abs_bf16x2(w[2], w[3])) & 0x7FFF7FFFu;
  m = win::larger_half(m);
#pragma unroll
  for (int d = 1; d < 16; d <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, d));
  // the row's largest channel to about 1 (nothing to be done for infinities, NaN and rows of zeros)
  int e = 127 - (int)(m >> 7);
  e = e < -126 ? -126 : (e > 126 ? 126 : e);
  if (eps > 0.f && e > 50) e = 50;   // (below 2^-50 eps outweighs the squares, or still does)
  const float f = out_of_range(v, eps) && m < 0x7F80u && m > 0u ? __uint_as_float((uint32_t)(127 + e) << 23) : 1.f;
  const float u = squares(f);
  if (f != 1.f) {
    v = u;
    s = f;
  }
  return make_float2(1.f / sqrtf(fmaf(v, 1.f / win::D, eps * s * s)), s);
}

// What the channels of N rows (1 or 2: heads) of this lane's token are multiplied by; -1 for a row whose squares leave
// fp32's range, which is left for later (its code beside the others' would take their registers).  The 16 lanes of a
// token reduce two sums together, each lane ending with one of them, so that a root is formed once a lane.
template <int N>
__device__ __forceinline__ void row_scales(const uint32_t (&w)[N][4], float eps, float (&r)[N]) {
  const int lane = threadIdx.x & 31;
  float v[N];
#pragma unroll
  for (int u = 0; u < N; u++) {
    const float2 a = win::split2(square_sum(w[u], 1.f));
    v[u] = a.x + a.y;
  }
  const bool up = lane & 8;   // two rows: each lane hands on one sum and keeps the other
  const float a = __shfl_xor_sync(0xffffffffu, N == 2 && !up ? v[1 % N] : v[0], 8);
  v[0] = (N == 2 && up ? v[1 % N] : v[0]) + a;
  v[0] += __shfl_xor_sync(0xffffffffu, v[0], 4);
  v[0] += __shfl_xor_sync(0xffffffffu, v[0], 2);
  v[0] += __shfl_xor_sync(0xffffffffu, v[0], 1);
  const float mine = out_of_range(v[0], eps) ? -1.f : inverse_root(fmaf(v[0], 1.f / win::D, eps));
#pragma unroll
  for (int u = 0; u < N; u++) r[u] = N == 1 ? mine : __shfl_sync(0xffffffffu, mine, (lane & 16) | u << 3);   // row u's: lanes of bit 3 = u
}

// Eight channels times r and the weights, and turned (TURN >= 0), rounded to bf16.  g: this
// lane's weights, HALF: and its partner's behind them.  Every lane of the warp takes part.
template <int TURN, typename Rot>
__device__ __forceinline__ void norm_turn(uint32_t (&w)[4], const float *g, float r, const qwm_rope_spec &sp, const Rot &rv) {
  uint64_t y[4], z[4];   // this lane's channels, its partner's
  auto normed = [&](const uint32_t (&x)[4], const float *f, uint64_t (&v)[4]) {
#pragma unroll
    for (int i = 0; i < 4; i++)
      v[i] = tc::mul2(tc::mul2(win::pair2(low(x[i]), high(x[i])), win::pair2(r, r)), win::pair2(f[2 * i], f[2 * i + 1]));
  };
  uint32_t p[4] = {0u, 0u, 0u, 0u};
  if (TURN == QWM_ROPE_HALF) {
    const int from = rv.partner(sp);
#pragma unroll
    for (int i = 0; i < 4; i++) p[i] = __shfl_sync(0xffffffffu, w[i], from);
  }
  normed(w, g, y);
  if (TURN == QWM_ROPE_HALF) normed(p, g + 8, z);
  if (TURN >= 0) rv.turn_normed(y, z);
#pragma unroll
  for (int i = 0; i < 4; i++) w[i] = tc::pack_bf16x2(win::split2(y[i]).x, win::split2(y[i]).y);
}

// The rotation of normed channels: they carry fp32 rounding already, so the products are plain FMAs with the
// cosine's and sine's upper parts.
template <int PAIRING, bool WHOLE>
struct Rotation : win::RopeVec<PAIRING, WHOLE> {
  using Base = win::RopeVec<PAIRING, WHOLE>;
  __device__ __forceinline__ void turn_normed(uint64_t (&y)[4], const uint64_t (&z)[4]) const {
    if (PAIRING == QWM_ROPE_INTERLEAVED) {
#pragma unroll
      for (int i = 0; i < 2; i++) {
        const float2 u = win::split2(y[2 * i]), v = win::split2(y[2 * i + 1]);
        const uint64_t a = win::pair2(u.x, v.x), b = win::pair2(u.y, v.y);
        const float2 c = win::split2(tc::fma2(a, this->ch[i], tc::mul2(b, this->nsh[i])));   // a c - b s
        const float2 d = win::split2(tc::fma2(a, this->sh[i], tc::mul2(b, this->ch[i])));    // a s + b c
        if (WHOLE || 2 * i < this->active) y[2 * i] = win::pair2(c.x, d.x);
        if (WHOLE || 2 * i + 1 < this->active) y[2 * i + 1] = win::pair2(c.y, d.y);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; i++) {
        const uint64_t x = tc::fma2(y[i], this->ch[i % Base::kN], tc::mul2(z[i], this->sh[i % Base::kN]));
        if (WHOLE || this->active) y[i] = x;
      }
    }
  }
};

// The same for a row that row_scales left: its channels times s first (a power of two: exact, or beyond mattering).
template <int TURN, typename Rot>
__device__ __forceinline__ void norm_turn_odd(uint32_t (&w)[4], const float *g, float eps, const qwm_rope_spec &sp, const Rot &rv) {
  const float2 f = scale_of_odd_row(w, eps);
#pragma unroll
  for (int i = 0; i < 4; i++) w[i] = tc::pack_bf16x2(low(w[i]) * f.y, high(w[i]) * f.y);
  norm_turn<TURN>(w, g, f.x, sp, rv);
}

// This lane's weights of a head (HALF: and its partner's), or ones.
template <int TURN, typename Rot>
__device__ __forceinline__ void weights_of(const float *weight, int v, const qwm_rope_spec &sp, const Rot &rv, float (&g)[16]) {
#pragma unroll
  for (int i = 0; i < 16; i++) g[i] = 1.f;
  if (!weight) return;
  auto take = [&](int u, float *to) {
    const float4 a = ((const float4 *)weight)[2 * u], b = ((const float4 *)weight)[2 * u + 1];
    to[0] = a.x; to[1] = a.y; to[2] = a.z; to[3] = a.w;
    to[4] = b.x; to[5] = b.y; to[6] = b.z; to[7] = b.w;
  };
  take(v, g);
  if (TURN == QWM_ROPE_HALF) take(rv.partner(sp) & 15, g + 8);
}

// Each head's own weights of a block's heads in shared memory (512 bytes a head): fetched from where they are, every
// head would wait for its own.  Every thread takes part; a barrier follows.
__device__ __forceinline__ void keep_weights(float *to, const float *weight, int h0, int h1) {
  for (int i = threadIdx.x; i < (h1 - h0) * (win::D / 4); i += kThreads)
    ((float4 *)to)[i] = __ldg((const float4 *)weight + h0 * (win::D / 4) + i);
}

// TURN: -1 no rotation, else the pairing (WHOLE: all channels).
template <int TURN, bool WHOLE>
__global__ void __launch_bounds__(kThreads, 4)
    norm_rope_kernel(const __grid_constant__ qwm_rope_spec sp, const uint16_t *x, qwm_strides xs, int batch, int heads,
                     int64_t n, const int64_t *__restrict__ start, const int64_t *__restrict__ at,
                     const int32_t *__restrict__ pos, const float *__restrict__ weight, int per_head, float eps,
                     uint16_t *out, qwm_strides os, int heads_per_block) {
  __shared__ win::RopeTable tab;
  extern __shared__ __align__(16) float own[];   // per_head: the block's heads' weights
  const int v = threadIdx.x & 15, row = threadIdx.x >> 4;
  const int64_t tok = (int64_t)blockIdx.x * kRows + row;   // over [batch][n]
  const bool in = tok < (int64_t)batch * n;
  const int64_t b = in ? win::quotient(tok, n) : 0, i = in ? tok - b * n : 0;
  const int h0 = blockIdx.y * heads_per_block;
  const int h1 = h0 + heads_per_block < heads ? h0 + heads_per_block : heads;
  const uint16_t *src = x + b * xs.batch + i * xs.token + 8 * v;
  uint16_t *dst = out + b * os.batch + i * os.token + 8 * v;
  uint4 r[kUnroll];
  auto load = [&](int h) {
#pragma unroll
    for (int u = 0; u < kUnroll; u++)
      r[u] = h + u < h1 ? *(const uint4 *)(src + (int64_t)(h + u) * xs.head) : make_uint4(0, 0, 0, 0);
  };
  load(h0);   // in flight while the angles are formed
  if (per_head) keep_weights(own, weight, h0, h1);
  int64_t p = 0;
  bool live = in;
  if (at) {
    p = at[b * n + i];
    live = in && win::starts(p);
  } else if (start) {
    p = start[b];
    live = in && win::starts(p);
    p += i;
  }
  Rotation<TURN == QWM_ROPE_HALF ? QWM_ROPE_HALF : QWM_ROPE_INTERLEAVED, WHOLE> rv;
  if (TURN >= 0) {
    tab.fill(sp);
    rv.init(sp, tab, v, live ? p : 0, pos ? pos + (b * n + i) * 3 : nullptr);
  } else if (per_head) {
    __syncthreads();
  }
  float g[16];
  weights_of<TURN>(weight, v, sp, rv, g);
  uint64_t left = 0ull;   // rows of this token left for later (a block walks over 64 heads at most)
  for (int h = h0; h < h1; h += kUnroll) {
    uint32_t w[kUnroll][4];
#pragma unroll
    for (int u = 0; u < kUnroll; u++) {
      w[u][0] = r[u].x; w[u][1] = r[u].y; w[u][2] = r[u].z; w[u][3] = r[u].w;
    }
    if (h + kUnroll < h1) load(h + kUnroll);   // other rows than the ones written below
    float rs[kUnroll];
    row_scales(w, eps, rs);
    bool some = false;
#pragma unroll
    for (int u = 0; u < kUnroll; u++) some |= rs[u] < 0.f;
    if (__any_sync(0xffffffffu, some)) {
#pragma unroll
      for (int u = 0; u < kUnroll; u++) left |= rs[u] < 0.f ? 1ull << (h + u - h0) : 0ull;
    }
#pragma unroll
    for (int u = 0; u < kUnroll; u++) {
      if (per_head && h + u < h1) weights_of<TURN>(own + (h + u - h0) * win::D, v, sp, rv, g);
      norm_turn<TURN>(w[u], g, rs[u], sp, rv);
      if (live && h + u < h1 && rs[u] >= 0.f)
        *(uint4 *)(dst + (int64_t)(h + u) * os.head) = make_uint4(w[u][0], w[u][1], w[u][2], w[u][3]);
    }
  }
#pragma unroll 1
  for (int h = h0; h < h1 && __any_sync(0xffffffffu, left != 0ull); h++, left >>= 1) {   // (not overwritten so far)
    if (!__any_sync(0xffffffffu, left & 1ull)) continue;
    const uint4 x4 = *(const uint4 *)(src + (int64_t)h * xs.head);
    uint32_t w[4] = {x4.x, x4.y, x4.z, x4.w};
    if (per_head) weights_of<TURN>(own + (h - h0) * win::D, v, sp, rv, g);
    norm_turn_odd<TURN>(w, g, eps, sp, rv);
    if (live && (left & 1ull)) *(uint4 *)(dst + (int64_t)h * os.head) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

template <int BITS, bool NORM, int TURN, bool WHOLE>
__global__ void __launch_bounds__(kThreads)
    paged_write_kernel(const __grid_constant__ qwm_rope_spec sp, qwm_page_pool pool, int page_log2,
                       const uint16_t *__restrict__ k, qwm_strides ks, const uint16_t *__restrict__ vv, qwm_strides vs,
                       int64_t n, const int64_t *__restrict__ slots, const int64_t *__restrict__ at,
                       const int32_t *__restrict__ pos, const float *__restrict__ weight, int per_head, float eps,
                       int heads_per_block, int32_t *status) {
  __shared__ win::RopeTable tab;
  extern __shared__ __align__(16) float own[];   // per_head: the block's heads' weights
  const int v = threadIdx.x & 15, row = threadIdx.x >> 4;
  const int64_t tok = (int64_t)blockIdx.x * kRows + row;
  const bool in = tok < n;
  const int64_t i = in ? tok : 0;
  const int h0 = blockIdx.y * heads_per_block;
  const int h1 = h0 + heads_per_block < pool.kv_heads ? h0 + heads_per_block : pool.kv_heads;
  const uint16_t *kp = k + i * ks.token + h0 * ks.head + 8 * v;
  const uint16_t *vp = vv + i * vs.token + h0 * vs.head + 8 * v;
  uint4 a = *(const uint4 *)kp, c = *(const uint4 *)vp;   // in flight while the angles are formed
  const int64_t slot = in ? slots[i] : -1, p = TURN >= 0 ? at[i] : 0;
  const bool inside = slot < (int64_t)pool.pages << page_log2;
  const bool live = slot >= 0 && inside && (TURN < 0 || win::starts(p));
  if (!inside) qwm_dev_error(status, QWM_ERR_RANGE);
  if (NORM && per_head) keep_weights(own, weight, h0, h1);
  Rotation<TURN == QWM_ROPE_HALF ? QWM_ROPE_HALF : QWM_ROPE_INTERLEAVED, WHOLE> rv;
  if (TURN >= 0) {
    tab.fill(sp);
    rv.init(sp, tab, v, live ? p : 0, pos ? pos + i * 3 : nullptr);
  } else if (NORM && per_head) {
    __syncthreads();
  }
  if (!__any_sync(0xffffffffu, live)) return;
  const bool all = __all_sync(0xffffffffu, live);
  float g[16];
  if (NORM) weights_of<TURN>(weight, v, sp, rv, g);
  const int64_t page = live ? slot >> page_log2 : 0;
  int64_t slot_row = ((page * pool.kv_heads + h0) << page_log2) + (live ? slot & ((1 << page_log2) - 1) : 0);
  bool bad = false;
  uint64_t left = 0ull;   // rows of Keys left for later (a block walks over 64 heads at most)
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
    if (NORM && per_head) weights_of<TURN>(own + (h - h0) * win::D, v, sp, rv, g);
    bool now = live;
    if (NORM) {
      const uint32_t one[1][4] = {{kw[0], kw[1], kw[2], kw[3]}};
      float r[1];
      row_scales(one, eps, r);
      if (__any_sync(0xffffffffu, live && r[0] < 0.f)) {
        left |= live && r[0] < 0.f ? 1ull << (h - h0) : 0ull;
        if (r[0] < 0.f) kw[0] = kw[1] = kw[2] = kw[3] = 0u;
        now = live && r[0] >= 0.f;
      }
      norm_turn<TURN>(kw, g, r[0], sp, rv);
    } else if (TURN >= 0) {
      rv.turn(sp, kw);
    }
    uint32_t c0, c1, step;
    win::quantise<BITS>(kw, c0, c1, step, bad);
    if (now) win::store_row<BITS>(pool.k_codes, pool.k_step, slot_row, v, c0, c1, step);
    win::quantise<BITS>(vw, c0, c1, step, bad);
    if (live) win::store_row<BITS>(pool.v_codes, pool.v_step, slot_row, v, c0, c1, step);
    slot_row += (int64_t)1 << page_log2;
  }
  if (NORM) {   // the rows of Keys that were left
    slot_row -= (int64_t)(h1 - h0) << page_log2;
    kp = k + i * ks.token + h0 * ks.head + 8 * v;
#pragma unroll 1
    for (int h = h0; h < h1 && __any_sync(0xffffffffu, left != 0ull); h++, left >>= 1) {
      const uint4 x = *(const uint4 *)kp;
      uint32_t kw[4] = {x.x, x.y, x.z, x.w}, c0, c1, step;
      if (!(left & 1ull)) kw[0] = kw[1] = kw[2] = kw[3] = 0u;
      if (per_head) weights_of<TURN>(own + (h - h0) * win::D, v, sp, rv, g);
      norm_turn_odd<TURN>(kw, g, eps, sp, rv);
      if (!(left & 1ull)) kw[0] = kw[1] = kw[2] = kw[3] = 0u;   // (no rows of their own: 0 / 0 where eps is 0)
      win::quantise<BITS>(kw, c0, c1, step, bad);
      if (left & 1ull) win::store_row<BITS>(pool.k_codes, pool.k_step, slot_row, v, c0, c1, step);
      kp += ks.head;
      slot_row += (int64_t)1 << page_log2;
    }
  }
  if (bad && live) qwm_dev_error(status, QWM_ERR_RANGE);
}

// Eight lanes take a row, vectors v and v + 8 of it each, so that every store instruction writes whole
// 128-byte lines; the loads of a head's Keys and Values are in flight together.
template <int BITS>
__global__ void __launch_bounds__(kThreads)
    paged_read_kernel(qwm_page_pool pool, int page_log2, const int64_t *__restrict__ slots, int64_t n,
                      uint16_t *__restrict__ k_hat, uint16_t *__restrict__ v_hat, int heads_per_block, int32_t *status,
                      win::Bases bases) {
  const int v = threadIdx.x & 7, row = threadIdx.x >> 3;
  const int64_t i = (int64_t)blockIdx.x * kReadRows + row;
  if (i >= n) return;
  const int64_t slot = slots[i];
  const bool inside = slot < (int64_t)pool.pages << page_log2, held = slot >= 0 && inside;
  if (!inside) qwm_dev_error(status, QWM_ERR_RANGE);
  const int h0 = blockIdx.y * heads_per_block;
  const int h1 = h0 + heads_per_block < pool.kv_heads ? h0 + heads_per_block : pool.kv_heads;
  constexpr int kVec = BITS, kRowBytes = win::D * BITS / 8;   // bytes of a vector's codes, of a row's
  const int64_t page = held ? slot >> page_log2 : 0, o0 = (h0 * n + i) * win::D + 8 * v;
  const int64_t r0 = ((page * pool.kv_heads + h0) << page_log2) + (held ? slot & ((1 << page_log2) - 1) : 0);
  const uint8_t *codes[2] = {pool.k_codes + r0 * kRowBytes + kVec * v, pool.v_codes + r0 * kRowBytes + kVec * v};
  const uint8_t *steps[2] = {pool.k_step + r0 * win::kSteps, pool.v_step + r0 * win::kSteps};
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
      codes[t] += (int64_t)kRowBytes << page_log2;
      steps[t] += (int64_t)win::kSteps << page_log2;
    }
#pragma unroll
    for (int t = 0; t < 2; t++) {
      if (!dst[t]) continue;
      *(uint4 *)dst[t] = win::restore<BITS>(x[t][0], (st[t] >> (8 * (v >> 2))) & 0xFFu, bases);
      *(uint4 *)(dst[t] + 64) = win::restore<BITS>(x[t][1], (st[t] >> (8 * (2 + (v >> 2)))) & 0xFFu, bases);
      dst[t] += n * win::D;
    }
  }
}

template <int BITS, bool NORM>
cudaError_t write_launch(const qwm_page_pool &pool, int page_log2, const uint16_t *k, const qwm_strides &ks, const uint16_t *v,
                         const qwm_strides &vs, int64_t n, const int64_t *slot, const qwm_rope_spec *rope, const int64_t *at,
                         const int32_t *pos, const float *weight, int per_head, float eps, int num_sms, int32_t *status,
                         cudaStream_t st) {
  // (blocks an SM: the chunk above turned, 4 bits, with 5 / 9 / 14 / 20 takes 76 / 68 / 70 / 76 us, in halves 80 / 76 / 80 /
  // 88; not turned with 10 / 20 / 30 / 40: 61 / 57 / 57 / 59)
  const int64_t tiles = (n + kRows - 1) / kRows;
  int hpb = heads_per_block(tiles, pool.kv_heads, num_sms, rope ? 9 : 20);
  hpb = hpb < 64 ? hpb : 64;
  const dim3 grid((unsigned)tiles, (unsigned)((pool.kv_heads + hpb - 1) / hpb));
  const qwm_rope_spec none = {};
  auto kernel = paged_write_kernel<BITS, NORM, -1, false>;
  if (rope && rope->pairing == QWM_ROPE_INTERLEAVED)
    kernel = rope->rot == win::D ? paged_write_kernel<BITS, NORM, QWM_ROPE_INTERLEAVED, true>
                                 : paged_write_kernel<BITS, NORM, QWM_ROPE_INTERLEAVED, false>;
  else if (rope)
    kernel = rope->rot == win::D ? paged_write_kernel<BITS, NORM, QWM_ROPE_HALF, true>
                                 : paged_write_kernel<BITS, NORM, QWM_ROPE_HALF, false>;
  const size_t shared = per_head ? hpb * win::D * sizeof(float) : 0;
  kernel<<<grid, kThreads, shared, st>>>(rope ? *rope : none, pool, page_log2, k, ks, v, vs, n, slot, at, pos, weight, per_head,
                                         eps, hpb, status);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_norm_rope(const qwm_rope_spec *spec, const uint16_t *x, const qwm_strides &xs, int batch, int heads,
                             int64_t n, const int64_t *start, const int64_t *at, const int32_t *pos, const float *weight,
                             int per_head, float eps, uint16_t *out, const qwm_strides &os, int num_sms, cudaStream_t st) {
  // (blocks an SM: the chunk above with 6 / 9 / 12 / 20 takes 51 / 47 / 47 / 51 us, in halves 64 / 58 / 57 / 62)
  const int64_t tiles = ((int64_t)batch * n + kRows - 1) / kRows;
  int hpb = heads_per_block(tiles, heads, num_sms, 12);
  hpb = hpb < 64 ? hpb : 64;
  const dim3 grid((unsigned)tiles, (unsigned)((heads + hpb - 1) / hpb));
  const qwm_rope_spec none = {};
  auto kernel = norm_rope_kernel<-1, false>;
  if (spec && spec->pairing == QWM_ROPE_INTERLEAVED)
    kernel = spec->rot == win::D ? norm_rope_kernel<QWM_ROPE_INTERLEAVED, true> : norm_rope_kernel<QWM_ROPE_INTERLEAVED, false>;
  else if (spec)
    kernel = spec->rot == win::D ? norm_rope_kernel<QWM_ROPE_HALF, true> : norm_rope_kernel<QWM_ROPE_HALF, false>;
  const size_t shared = per_head ? hpb * win::D * sizeof(float) : 0;
  kernel<<<grid, kThreads, shared, st>>>(spec ? *spec : none, x, xs, batch, heads, n, start, at, pos, weight, per_head, eps, out,
                                         os, hpb);
  return cudaGetLastError();
}

cudaError_t launch_paged_write(const qwm_page_pool &pool, int page_log2, const uint16_t *k, const qwm_strides &ks,
                               const uint16_t *v, const qwm_strides &vs, int64_t n, const int64_t *slot,
                               const qwm_rope_spec *rope, const int64_t *at, const int32_t *pos, int norm, const float *weight,
                               int per_head, float eps, int num_sms, int32_t *status, cudaStream_t st) {
  auto launch = pool.bits == 8 ? (norm ? write_launch<8, true> : write_launch<8, false>)
                               : (norm ? write_launch<4, true> : write_launch<4, false>);
  return launch(pool, page_log2, k, ks, v, vs, n, slot, rope, at, pos, weight, per_head, eps, num_sms, status, st);
}

cudaError_t launch_paged_read(const qwm_page_pool &pool, int page_log2, const int64_t *slot, int64_t n, uint16_t *k_hat,
                              uint16_t *v_hat, int num_sms, int32_t *status, cudaStream_t st) {
  // (blocks an SM: the chunk above, 4 bits, with 10 / 20 / 40 / 80 takes 49 / 48 / 47 / 48 us)
  const int64_t tiles = (n + kReadRows - 1) / kReadRows;
  const int hpb = heads_per_block(tiles, pool.kv_heads, num_sms, 40);
  const dim3 grid((unsigned)tiles, (unsigned)((pool.kv_heads + hpb - 1) / hpb));
  auto kernel = pool.bits == 8 ? paged_read_kernel<8> : paged_read_kernel<4>;
  kernel<<<grid, kThreads, 0, st>>>(pool, page_log2, slot, n, k_hat, v_hat, hpb, status, win::kBases);
  return cudaGetLastError();
}
