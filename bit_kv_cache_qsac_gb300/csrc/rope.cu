// Rotary positions with three axes: each pair (a, b) of a row's channels becomes
// (a cos - b sin, a sin + b cos) with the angle of its axis' coordinate and its frequency.
//
// Bound: memory (2 bytes read and 2 written per channel); the angles depend on the token alone, so a
// thread forms those of its 8 channels once and walks over `heads_per_block` heads with them.
#include <math.h>

#include "window.cuh"

namespace {

constexpr int kThreads = 256, kRows = kThreads / 16;
constexpr int kUnroll = 4;   // heads whose loads are in flight together

template <int PAIRING>
__global__ void __launch_bounds__(kThreads)
    rope_kernel(const __grid_constant__ qwm_rope_spec sp, const uint16_t *__restrict__ x, qwm_strides xs, int batch,
                int heads, int64_t n, const int64_t *__restrict__ start, const int32_t *__restrict__ pos,
                uint16_t *out, qwm_strides os, int heads_per_block) {
  const int v = threadIdx.x & 15, row = threadIdx.x >> 4;
  const int64_t tok = (int64_t)blockIdx.x * kRows + row;   // over [batch][n]
  const bool in = tok < (int64_t)batch * n;
  const int64_t b = in ? tok / n : 0, i = in ? tok - b * n : 0;
  const int64_t s0 = start[b];
  const bool live = in && s0 >= 0;
  if (!__any_sync(0xffffffffu, live)) return;
  win::RopeVec<PAIRING> rv;
  rv.init(sp, v, live ? s0 + i : 0, pos ? pos + (b * n + i) * 3 : nullptr);
  const int h0 = blockIdx.y * heads_per_block;
  const int h1 = h0 + heads_per_block < heads ? h0 + heads_per_block : heads;
  const uint16_t *src = x + b * xs.batch + i * xs.token + 8 * v;
  uint16_t *dst = out + b * os.batch + i * os.token + 8 * v;
  for (int h = h0; h < h1; h += kUnroll) {
    uint4 r[kUnroll] = {};
#pragma unroll
    for (int u = 0; u < kUnroll; u++)
      if (live && h + u < h1) r[u] = *(const uint4 *)(src + (int64_t)(h + u) * xs.head);
#pragma unroll
    for (int u = 0; u < kUnroll; u++) {
      uint32_t w[4] = {r[u].x, r[u].y, r[u].z, r[u].w};
      if (h + u < h1) rv.turn(sp, w);   // the same for every lane of the block
      if (live && h + u < h1)
        *(uint4 *)(dst + (int64_t)(h + u) * os.head) = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
}

}  // namespace

cudaError_t launch_rope(const qwm_rope_spec &spec, const uint16_t *x, const qwm_strides &xs, int batch, int heads,
                        int64_t n, const int64_t *start, const int32_t *pos, uint16_t *out, const qwm_strides &os,
                        int num_sms, cudaStream_t st) {
  const int64_t tiles = ((int64_t)batch * n + kRows - 1) / kRows;
  // few tokens: one head per block, to fill the SMs; many: up to 8 heads share a token's angles
  int64_t hpb = tiles * heads / (8 * (int64_t)num_sms);
  hpb = hpb < 1 ? 1 : (hpb > 8 ? 8 : hpb);
  const dim3 grid((unsigned)tiles, (unsigned)((heads + hpb - 1) / hpb));
  if (spec.pairing == QWM_ROPE_INTERLEAVED)
    rope_kernel<QWM_ROPE_INTERLEAVED><<<grid, kThreads, 0, st>>>(spec, x, xs, batch, heads, n, start, pos, out, os,
                                                                 (int)hpb);
  else
    rope_kernel<QWM_ROPE_HALF><<<grid, kThreads, 0, st>>>(spec, x, xs, batch, heads, n, start, pos, out, os, (int)hpb);
  return cudaGetLastError();
}
