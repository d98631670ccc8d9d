// Rotary positions with three axes: each pair (a, b) of a row's channels becomes
// (a cos - b sin, a sin + b cos) with the angle of its axis' coordinate and its frequency.
//
// Bound: memory (2 bytes read and 2 written per channel); the angles depend on the token alone, so a
// thread forms those of its 8 channels once and walks over `heads_per_block` heads with them, four heads'
// loads in flight at a time.  Measured: 40 heads x 10,800 tokens in 36.7 us = 6.0 TB/s (0.90 of a copy), 37.3 in halves;
// one token of 16 sequences x 32 heads in 3.4 us (launch, then start -> angle -> product).
#include <math.h>

#include "window.cuh"

namespace {

constexpr int kThreads = 256, kRows = kThreads / 16;
constexpr int kUnroll = 4;   // heads whose loads are in flight together

template <int PAIRING, bool WHOLE>
__global__ void __launch_bounds__(kThreads, 3)
    rope_kernel(const __grid_constant__ qwm_rope_spec sp, const uint16_t *x, qwm_strides xs, int batch,
                int heads, int64_t n, const int64_t *__restrict__ start, const int32_t *__restrict__ pos,
                uint16_t *out, qwm_strides os, int heads_per_block) {
  __shared__ win::RopeTable tab;
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
  const int64_t s0 = start[b];
  const bool live = in && win::starts(s0);
  tab.fill(sp);
  win::RopeVec<PAIRING, WHOLE> rv;
  rv.init(sp, tab, v, live ? s0 + i : 0, pos ? pos + (b * n + i) * 3 : nullptr);
  for (int h = h0; h < h1; h += kUnroll) {
    uint32_t w[kUnroll][4];
#pragma unroll
    for (int u = 0; u < kUnroll; u++) {
      w[u][0] = r[u].x; w[u][1] = r[u].y; w[u][2] = r[u].z; w[u][3] = r[u].w;
    }
    if (h + kUnroll < h1) load(h + kUnroll);   // other rows than the ones written below
#pragma unroll
    for (int u = 0; u < kUnroll; u++) {
      rv.turn(sp, w[u]);
      if (live && h + u < h1)
        *(uint4 *)(dst + (int64_t)(h + u) * os.head) = make_uint4(w[u][0], w[u][1], w[u][2], w[u][3]);
    }
  }
}

}  // namespace

cudaError_t launch_rope(const qwm_rope_spec &spec, const uint16_t *x, const qwm_strides &xs, int batch, int heads,
                        int64_t n, const int64_t *start, const int32_t *pos, uint16_t *out, const qwm_strides &os,
                        int num_sms, cudaStream_t st) {
  const int64_t tiles = ((int64_t)batch * n + kRows - 1) / kRows;
  const int hpb = heads_per_block(tiles, heads, num_sms, 9);
  const dim3 grid((unsigned)tiles, (unsigned)((heads + hpb - 1) / hpb));
  auto kernel = spec.pairing == QWM_ROPE_INTERLEAVED
                    ? (spec.rot == win::D ? rope_kernel<QWM_ROPE_INTERLEAVED, true> : rope_kernel<QWM_ROPE_INTERLEAVED, false>)
                    : (spec.rot == win::D ? rope_kernel<QWM_ROPE_HALF, true> : rope_kernel<QWM_ROPE_HALF, false>);
  kernel<<<grid, kThreads, 0, st>>>(spec, x, xs, batch, heads, n, start, pos, out, os, hpb);
  return cudaGetLastError();
}
