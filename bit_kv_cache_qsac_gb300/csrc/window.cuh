// Device code shared by the recent-window kernels: rotary angles, the window cache's codes and
// steps, and which keys a Query row sees.
#pragma once

#include <atomic>

#include "../../include/qwm_window.h"
#include "qwm_internal.cuh"
#include "tc.cuh"

namespace win {

constexpr int D = QWM_D;
constexpr int kGroup = 32;              // channels that share a step
constexpr int kSteps = D / kGroup;      // step bytes of a row: one 32-bit word

// Two floats as one operand of the packed fp32 instructions, and back.
__device__ __forceinline__ uint64_t pair2(float lo, float hi) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(lo), "f"(hi));
  return d;
}
__device__ __forceinline__ float2 split2(uint64_t v) {
  float2 f;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(v));
  return f;
}

// The larger magnitude of each half (a NaN stays one); its sign means nothing.
__device__ __forceinline__ uint32_t max_abs_bf16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// ------------------------------------------------------------------ rotary positions

// Cosine and sine of an angle given as pos * turn / 2^64 turns, each as an unevaluated sum hi + lo.
// The product is taken modulo 2^64, i.e. modulo a whole turn, in integers, so that no position loses more
// than the rounding of `turn`, 2^-65 turns per unit of position.
// The remainder to the nearest quarter turn, |x| <= pi/4, goes through the Taylor series of sine and
// cosine with the terms up to x^3 / 6 and x^2 / 2 kept in two floats; hi + lo is within 2^-28 of the value (cosine
// 2^-28.7, sine 2^-30.2 at most in 60 million angles), so a rotated channel is rounded to bf16 as the exact one is but
// for one in some 10^5.
__device__ __forceinline__ void rope_sincos(int64_t pos, uint64_t turn, float &ch, float &cl, float &sh, float &sl) {
  const uint64_t a = (uint64_t)pos * turn;
  const uint32_t quarter = (uint32_t)((a + (1ull << 61)) >> 62);
  const int64_t r = (int64_t)(a - ((uint64_t)quarter << 62));
  const int32_t hi = (int32_t)(r >> 32);
  const float fh = (float)hi;
  const float fl = (float)(hi - (int32_t)fh) + (float)(uint32_t)r * 0x1p-32f;
  // 2 pi 2^-32 as a sum of two floats
  constexpr double kTau = 6.283185307179586476925286766559 * 0x1p-32;
  constexpr float kTauHi = (float)kTau, kTauLo = (float)(kTau - (double)kTauHi);
  const float x = fh * kTauHi;
  const float xl = fmaf(fh, kTauLo, fmaf(fl, kTauHi, fmaf(fh, kTauHi, -x)));
  const float z = x * x, zz = fmaf(x, x, -z);        // x^2 exactly
  const float zl = fmaf(2.f * x, xl, zz);            // z + zl: (x + xl)^2
  float pc = fmaf(z, 1.f / 479001600.f, -1.f / 3628800.f);
  pc = fmaf(pc, z, 1.f / 40320.f);
  pc = fmaf(pc, z, -1.f / 720.f);
  pc = fmaf(pc, z, 1.f / 24.f);
  const float h = 0.5f * z, c0 = 1.f - h;            // zl times -1/2 + z / 12, the slope in z of the terms to z^2
  const float c1 = fmaf(z * z, pc, fmaf(zl, fmaf(z, 1.f / 12.f, -0.5f), (1.f - c0) - h));
  const float c = c0 + c1, cr = c1 - (c - c0);
  float ps = fmaf(z, 1.f / 6227020800.f, -1.f / 39916800.f);
  ps = fmaf(ps, z, 1.f / 362880.f);
  ps = fmaf(ps, z, -1.f / 5040.f);
  ps = fmaf(ps, z, 1.f / 120.f);
  constexpr float kSixth = -1.f / 6.f, kSixthLo = (float)(-1.0 / 6.0 - (double)kSixth);
  const float u = x * kSixth, ul = fmaf(x, kSixthLo, fmaf(x, kSixth, -u));                   // u + ul = -x / 6
  const float q = u * z, ql = fmaf(ul, z, fmaf(u, zz, fmaf(u, z, -q)));                      // q + ql = -x^3 / 6
  const float s0 = x + q, s1 = fmaf(x * z * z, ps, fmaf(xl, c, ql)) + (q - (s0 - x));
  const float s = s0 + s1, sr = s1 - (s - s0);
  const bool swap = quarter & 1u;
  const float sgc = ((quarter + 1u) & 2u) ? -1.f : 1.f, sgs = (quarter & 2u) ? -1.f : 1.f;
  ch = sgc * (swap ? s : c);
  cl = sgc * (swap ? sr : cr);
  sh = sgs * (swap ? c : s);
  sl = sgs * (swap ? cr : sr);
}

// x, but 2^126 of some sign where it is infinite or not a number: the correction of a product with an infinite
// channel is inf - inf, and added as it is would make the infinite result a NaN.  (One instruction; looking
// for such channels with a branch took 2 to 8% of the rotating calls' time, this 1%.)
__device__ __forceinline__ float finite(float x) {
  float d;
  asm("min.xorsign.abs.f32 %0, %1, %2;" : "=f"(d) : "f"(x), "f"(0x1p126f));
  return d;
}

// p x + q y for two channels at a time, with x = xh + xl and y = yh + yl: the error of the rounded product
// q yh is carried (ny = -yh), so each result is within a little over half a unit of fp32.
__device__ __forceinline__ uint64_t rope_pair(uint64_t p, uint64_t q, uint64_t xh, uint64_t xl, uint64_t yh,
                                              uint64_t yl, uint64_t ny) {
  const uint64_t t = tc::mul2(q, yh), e = tc::fma2(q, yh, tc::mul2(q, ny));
  const float2 c = split2(tc::fma2(p, xl, tc::fma2(q, yl, e)));
  return tc::add2(tc::fma2(p, xh, t), pair2(finite(c.x), finite(c.y)));
}

// The coordinate of position p (>= 0) on one axis of the spec's grid.
__device__ __forceinline__ int64_t rope_coord(const qwm_rope_spec &sp, int64_t p, int axis) {
  if (p < ((int64_t)1 << 31)) {
    const uint32_t q = (uint32_t)p, row = q / (uint32_t)sp.grid_w;
    if (axis == 2) return q - row * (uint32_t)sp.grid_w;
    const uint32_t t = row / (uint32_t)sp.grid_h;
    return axis == 0 ? t : row - t * (uint32_t)sp.grid_h;
  }
  const int64_t row = p / sp.grid_w;
  if (axis == 2) return p - row * sp.grid_w;
  const int64_t t = row / sp.grid_h;
  return axis == 0 ? t : row - t * sp.grid_h;
}

// The spec's table in shared memory: lanes read different pairs, which constant memory would serve one
// address at a time.  Every thread of the block takes part.
struct RopeTable {
  uint64_t turn[64];
  uint8_t axis[64];
  __device__ __forceinline__ void fill(const qwm_rope_spec &sp) {
    if (threadIdx.x < 64) {
      turn[threadIdx.x] = sp.turn[threadIdx.x];
      axis[threadIdx.x] = sp.axis[threadIdx.x];
    }
    __syncthreads();
  }
};

// The angles of one token for the 8 channels 8 v .. 8 v + 7 of a row (v = 0..15), two at a time.
// INTERLEAVED: pairs (a, b) inside the vector, out_a = a c - b s, out_b = b c + a s; the packed lanes are
// pairs 2 i and 2 i + 1.  HALF: the vector is the first or the second half of eight pairs and its partner
// is another lane's: out = mine c -+ other s; the packed lanes are channels 2 i and 2 i + 1.
// WHOLE: all 128 channels are turned (every vector is active).
template <int PAIRING, bool WHOLE>
struct RopeVec {
  static constexpr int kN = PAIRING == QWM_ROPE_INTERLEAVED ? 2 : 4;
  uint64_t ch[kN], cl[kN], sh[kN], sl[kN], nch[kN], nsh[kN], nsl[kN];   // HALF: s signed for this half
  int active;   // INTERLEAVED: pairs turned; HALF: 1 first half, 2 second half, 0 neither

  // pos3: (t, y, x) of the token, or NULL to take them from position p and the grid
  __device__ __forceinline__ void init(const qwm_rope_spec &sp, const RopeTable &tab, int v, int64_t p,
                                       const int32_t *pos3) {
    int64_t c[3];
#pragma unroll
    for (int a = 0; a < 3; a++) c[a] = pos3 ? (int64_t)pos3[a] : rope_coord(sp, p, a);
    const int half = sp.rot >> 1;
    int i0, n;   // first pair, pairs turned
    if (PAIRING == QWM_ROPE_INTERLEAVED) {
      i0 = 4 * v;
      n = half - i0 < 0 ? 0 : (half - i0 < 4 ? half - i0 : 4);
      active = n;
    } else {
      active = 8 * v < half ? 1 : (8 * v < sp.rot ? 2 : 0);
      i0 = active == 2 ? 8 * v - half : 8 * v;
      n = active ? 8 : 0;
    }
    // HALF: a lane and its partner turn the same eight pairs; each forms the angles of four
    constexpr int kMine = 4;
    float f[2 * kN][4], g[kMine][4];
#pragma unroll
    for (int k = 0; k < kMine; k++) {
      const int j = k + (PAIRING == QWM_ROPE_HALF && active == 2 ? 4 : 0);
      g[k][0] = 1.f;
      g[k][1] = g[k][2] = g[k][3] = 0.f;
      if (j < n) {
        const int ax = tab.axis[i0 + j];
        rope_sincos(ax == 0 ? c[0] : (ax == 1 ? c[1] : c[2]), tab.turn[i0 + j], g[k][0], g[k][1], g[k][2], g[k][3]);
      }
    }
    if (PAIRING == QWM_ROPE_INTERLEAVED) {
#pragma unroll
      for (int k = 0; k < kMine; k++)
#pragma unroll
        for (int e = 0; e < 4; e++) f[k][e] = g[k][e];
    } else {
      const int other = partner(sp);
#pragma unroll
      for (int k = 0; k < kMine; k++)
#pragma unroll
        for (int e = 0; e < 4; e++) {
          const float o = __shfl_sync(0xffffffffu, g[k][e], other);
          const float a0 = active == 2 ? o : g[k][e], a1 = active == 2 ? g[k][e] : o;
          const float sign = e >= 2 && active == 1 ? -1.f : 1.f;
          f[k][e] = sign * a0;
          f[(k + kMine) % (2 * kN)][e] = sign * a1;
        }
    }
#pragma unroll
    for (int i = 0; i < kN; i++) {
      ch[i] = pair2(f[2 * i][0], f[2 * i + 1][0]);
      cl[i] = pair2(f[2 * i][1], f[2 * i + 1][1]);
      sh[i] = pair2(f[2 * i][2], f[2 * i + 1][2]);
      sl[i] = pair2(f[2 * i][3], f[2 * i + 1][3]);
      nch[i] = pair2(-f[2 * i][0], -f[2 * i + 1][0]);
      nsh[i] = pair2(-f[2 * i][2], -f[2 * i + 1][2]);
      nsl[i] = pair2(-f[2 * i][3], -f[2 * i + 1][3]);
    }
  }
  // HALF: the lane that holds the other half of this lane's pairs (itself where nothing is turned).
  __device__ __forceinline__ int partner(const qwm_rope_spec &sp) const {
    const int lane = threadIdx.x & 31, off = WHOLE ? 8 : sp.rot >> 4;
    return (active == 1 ? lane + off : (active == 2 ? lane - off : lane)) & 31;
  }
  // Turn the 8 bf16 channels in w (4 words).  HALF: every lane of the 16-lane row takes part.
  __device__ __forceinline__ void turn(const qwm_rope_spec &sp, uint32_t (&w)[4]) const {
    auto lo = [](uint32_t x) { return __uint_as_float(x << 16); };
    auto hi = [](uint32_t x) { return __uint_as_float(x & 0xFFFF0000u); };
    if (PAIRING == QWM_ROPE_INTERLEAVED) {
#pragma unroll
      for (int i = 0; i < 2; i++) {
        const uint64_t a = pair2(lo(w[2 * i]), lo(w[2 * i + 1])), b = pair2(hi(w[2 * i]), hi(w[2 * i + 1]));
        const uint64_t x = rope_pair(a, b, ch[i], cl[i], nsh[i], nsl[i], sh[i]);   // a c - b s
        const uint64_t y = rope_pair(a, b, sh[i], sl[i], ch[i], cl[i], nch[i]);    // a s + b c
        if (WHOLE || 2 * i < active) w[2 * i] = tc::pack_bf16x2(split2(x).x, split2(y).x);
        if (WHOLE || 2 * i + 1 < active) w[2 * i + 1] = tc::pack_bf16x2(split2(x).y, split2(y).y);
      }
    } else {
      const int from = partner(sp);
#pragma unroll
      for (int i = 0; i < 4; i++) {
        const uint32_t q = __shfl_sync(0xffffffffu, w[i], from);
        const uint64_t mine = pair2(lo(w[i]), hi(w[i])), other = pair2(lo(q), hi(q));
        const uint64_t x = rope_pair(mine, other, ch[i % kN], cl[i % kN], sh[i % kN], sl[i % kN], nsh[i % kN]);
        if (WHOLE || active) w[i] = tc::pack_bf16x2(split2(x).x, split2(x).y);
      }
    }
  }
};

// ------------------------------------------------------------------ codes and steps

__host__ __device__ constexpr float code_max(int bits) { return bits == 8 ? 127.f : 7.f; }
__host__ __device__ constexpr uint32_t step_max(int bits) { return bits == 8 ? 0xA6u : 0xC6u; }  // 56, 896

__device__ __forceinline__ float step_value(uint32_t b) { return __half2float(__ushort_as_half((uint16_t)(b << 7))); }

// The smallest step with Q s >= amax (amax a bf16 value), at most step_max: its byte, and s itself.
// amax has 8 significant bits and a step 4, so the quotient is a step exactly or at least 2^-11 (relative)
// away from every step: rounding up to 3 mantissa bits after taking 16 units off (the multiplication's
// error is below 2) finds it.  Below 2^-14 (`step_is_small`) steps are multiples of 2^-17.
template <int BITS>
__device__ __forceinline__ bool step_is_small(float amax) {
  return amax * (1.f / code_max(BITS)) < 0x1p-14f * (1.f - 0x1p-20f);
}
template <int BITS>
__device__ __forceinline__ uint32_t small_step(float amax, float &s) {
  const float m = ceilf(amax * (1.f / code_max(BITS)) * 0x1p17f * (1.f - 0x1p-20f));
  s = m * 0x1p-17f;
  return (uint32_t)m;
}
template <int BITS>
__device__ __forceinline__ uint32_t normal_step(float amax, float &s) {
  constexpr uint32_t kTop = (step_max(BITS) << 20) + ((127u - 15u) << 23);
  uint32_t b = (__float_as_uint(amax * (1.f / code_max(BITS))) + (0xFFFFFu - 16u)) & 0xFFF00000u;
  b = b < kTop ? b : kTop;
  s = __uint_as_float(b);
  return (b >> 20) - ((127u - 15u) << 3);
}

// Two codes: rint(x / s) in the low bits of each result's pattern (0x4B400000 + code).  The quotient is
// first rounded to a grid of 2^-11: x has 8 significant bits and s has 4, so a quotient that is not
// halfway between integers is at least 2^-9.9 away from halfway and stays on its side, while one that
// is lands exactly on it (and then ties to even).  The first constant stays in the sum; the second one
// takes it out again while it rounds to integers (both are exact).
__device__ __forceinline__ uint64_t codes_of(uint64_t x2, uint64_t inv2) {
  const uint64_t grid = pair2(0x1.8p12f, 0x1.8p12f), whole = pair2(0x1.8p23f - 0x1.8p12f, 0x1.8p23f - 0x1.8p12f);
  return tc::add2(tc::fma2(x2, inv2, grid), whole);
}

// What the decoders below give is the value over kUnit: at 4 bits a sixteenth, so that every constant of
// every step stays finite in fp16.  Whoever multiplies by decoded values has a scale to fold it into.
template <int BITS>
constexpr float kUnit = BITS == 8 ? 1.f : 16.f;
// Decode constants of a step, in both halves: s / unit and minus that times what a code's fp16 bit pattern
// below stands above the signed code: 1152 (8 bits); 72 (4 bits, pattern from 64) and 1032 (nl: pattern
// from 1024).  (pattern) s - bias s in one fp16 FMA is then exactly code * s: a step has 4 significant bits,
// 9 * s and 129 * s at most 11, and 1152 * 56 and 1032 / 16 * 896 are below 65504; the smallest step, 2^-17,
// over 16 is still on fp16's grid.
struct Step {
  uint32_t s, n, nl;
};
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
template <int BITS>
__device__ __forceinline__ Step step_of(uint32_t s2) {   // two steps as fp16 pairs
  if (BITS == 8) return {s2, hmul2(s2, 0xE480E480u), 0u};
  return {hmul2(s2, 0x2C002C00u), hmul2(s2, 0xC480C480u), hmul2(s2, 0xD408D408u)};   // 1/16, -72/16, -1032/16
}
template <int BITS>
__device__ __forceinline__ Step step_of_byte(uint32_t byte) {
  return step_of<BITS>(byte * 0x00800080u);   // byte << 7 in both halves
}

// fp16 bit patterns that codes are placed into: 0x6400 = 1024 (ulp 1) and 0x5400 = 64 (ulp 1/16), in both
// halves.  They are kernel arguments, not literals: a three-input logic instruction holds one literal,
// so (x & mask) | base is one instruction when `base` is in a register and two when it is not.
struct Bases {
  uint32_t k1024, k64;
};
constexpr Bases kBases = {0x64006400u, 0x54005400u};
template <uint32_t MASK>
__device__ __forceinline__ uint32_t place(uint32_t x, uint32_t base) {   // (x & MASK) | base
  uint32_t d;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(d) : "r"(x), "n"(MASK), "r"(base));
  return d;
}

// 8 bits: four codes (one word) -> fp16 pairs of channels (0, 1) and (2, 3).
__device__ __forceinline__ void decode8(uint32_t x, const Step &st, const Bases &c, uint32_t &p0, uint32_t &p1) {
  p0 = tc::hfma2(__byte_perm(x, c.k1024, 0x5150), st.s, st.n);   // fp16 bits 0x64cc = 1024 + c
  p1 = tc::hfma2(__byte_perm(x, c.k1024, 0x5352), st.s, st.n);
}
// 4 bits: eight codes (one word) -> fp16 pairs of channels (0, 1), (2, 3), (4, 5), (6, 7).  Nibbles at bits
// 4-7 of a half read as 64 + c (0x54c0), those at bits 0-3 as 1024 + c (0x640c).
__device__ __forceinline__ void decode4(uint32_t x, const Step &st, const Bases &c, uint32_t (&p)[4]) {
  const uint32_t y = x >> 8;
  p[0] = tc::hfma2(place<0x000F000Fu>(x, c.k1024), st.s, st.nl);
  p[1] = tc::hfma2(place<0x00F000F0u>(x, c.k64), st.s, st.n);
  p[2] = tc::hfma2(place<0x000F000Fu>(y, c.k1024), st.s, st.nl);
  p[3] = tc::hfma2(place<0x00F000F0u>(y, c.k64), st.s, st.n);
}

// ------------------------------------------------------------------ Queries

// Queries enter the first product in fp16: a bf16 value of 2^-17 to 65504 is exact, smaller ones are rounded to
// multiples of 2^-24.  A row whose largest magnitude is below 1 is first multiplied by a power of two that
// brings it to 2^14 .. 2^15 (2^120 at most), which its logits' scale takes back; so what rounding there is
// stays below 2^-25 of the row's largest element, under the fp32 rounding of its logits.
// The tests of packed magnitudes m (bf16 without signs, in both halves):
__device__ __forceinline__ bool any_from_one(uint32_t m) { return ((m + 0x40804080u) & 0x80008000u) != 0u; }       // 1 or more
__device__ __forceinline__ bool any_beyond_fp16(uint32_t m) { return ((m + 0x38803880u) & 0x80008000u) != 0u; }   // 2^16 or more, or a NaN
// The power of two that a row of largest magnitude `top` (bf16, below 1) is multiplied by, and 2^k.
__device__ __forceinline__ uint32_t row_power(uint32_t top) { return 141u - (top >> 7) < 120u ? 141u - (top >> 7) : 120u; }
__device__ __forceinline__ float power_of_two(int k) { return __uint_as_float((uint32_t)(127 + k) << 23); }
__device__ __forceinline__ uint32_t larger_half(uint32_t m) { return (m & 0xFFFFu) > (m >> 16) ? m & 0xFFFFu : m >> 16; }

// ------------------------------------------------------------------ weights

// The weights 2^(l - m) of the second product are fp16, rounded to 11 bits down to 2^-14 and to multiples of
// 2^-24 below.  So that many small ones beside a large one (a sink) are not lost from the output while the
// sum of the weights, in fp32, has them, m stands 7 below the running maximum: the largest weight is 2^7, at
// most 2^15 while the maximum lags by 8, and the grid is 2^-31 of it.  Output and sum share the factor.
constexpr float kTopWeight = 7.f;

// ------------------------------------------------------------------ which keys a row sees

// a / b of non-negative numbers, in 32 bits where they fit (a 64-bit division takes some 100 instructions).
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
  return ((a | b) >> 32) == 0 ? (int64_t)((uint32_t)a / (uint32_t)b) : a / b;
}
__device__ __forceinline__ int64_t remainder(int64_t a, int64_t b) {
  return ((a | b) >> 32) == 0 ? (int64_t)((uint32_t)a % (uint32_t)b) : a % b;
}

// Positions end here, so that sums of a position, a count and a frame stay inside 64 bits.
constexpr int64_t kMaxPosition = (int64_t)1 << 62;
// A sequence that starts outside 0 .. kMaxPosition is left out.
__device__ __forceinline__ bool starts(int64_t p) { return p >= 0 && p <= kMaxPosition; }
// Tokens of a sequence as the kernels count with them.
__device__ __forceinline__ int64_t tokens_of(int64_t len) { return len > 0 ? len : 0; }

// Sequence and window of an attention call, for one sequence.
struct Seq {
  int64_t len, sink, ring, tpf, frames;
  // first and past-the-last position of the recent keys of frame f (f = -1: none), and sinks seen
  __device__ __forceinline__ int64_t hi(int64_t f) const {
    const int64_t e = (f + 1) * tpf;
    return e < len ? e : len;
  }
  __device__ __forceinline__ int64_t lo(int64_t f) const {
    int64_t l = f + 1 > frames ? (f + 1 - frames) * tpf : 0;
    l = l > len - ring ? l : len - ring;
    return l > sink ? l : sink;
  }
  __device__ __forceinline__ int64_t sinks(int64_t f) const {
    const int64_t e = hi(f);
    return e < sink ? e : sink;
  }
  __device__ __forceinline__ int64_t frame(int64_t p) const {
    return p < 0 ? -1 : (tpf == 1 ? p : quotient(p, tpf));
  }
};

// The keys that the rows of positions p0 .. p1 (p0 <= p1) see between them, numbered 0 .. total - 1: the
// sinks first, then the recent ones.  Key v lives in slot v (v < ns) or sink + (base + v - ns) mod ring.
struct Keys {
  int ns, total;
  int64_t lo;
  uint32_t base;
  __device__ __forceinline__ void init(const Seq &s, int64_t f0, int64_t f1) {
    ns = (int)s.sinks(f1);
    lo = s.lo(f0);
    const int64_t n = s.hi(f1) - lo;
    total = ns + (n > 0 ? (int)n : 0);
    base = (uint32_t)remainder(lo - s.sink, s.ring);   // lo >= sink
  }
  __device__ __forceinline__ uint32_t slot(int v, uint32_t sink, uint32_t ring) const {
    if (v < ns) return (uint32_t)v;
    uint32_t r = base + (uint32_t)(v - ns);
    r = r >= ring ? r - ring : r;
    return sink + r;
  }
};

// The keys of `Keys` that one row sees: 0 .. c0 - 1 and c1 .. c2 - 1.
struct Row {
  int c0, c1, c2;
  __device__ __forceinline__ void init(const Seq &s, const Keys &k, int64_t f) {
    c0 = c1 = c2 = 0;
    if (f < 0) return;
    c0 = (int)s.sinks(f);
    const int64_t l = s.lo(f), h = s.hi(f);
    if (h > l) {
      c1 = k.ns + (int)(l - k.lo);
      c2 = k.ns + (int)(h - k.lo);
    }
  }
  __device__ __forceinline__ bool sees(int v) const { return v < c0 || (v >= c1 && v < c2); }
};

// The keys that every row of frames f0 .. f1 sees: 0 .. e0 - 1 and e1 .. e2 - 1 (both ends of a row's
// recent keys grow with its frame, and where the first and the last row see some, all do).
struct Everyone {
  int e0, e1, e2;
  __device__ __forceinline__ void init(const Seq &s, const Keys &k, int64_t f0, int64_t f1) {
    e0 = (int)s.sinks(f0);
    const int64_t l = s.lo(f1), h = s.hi(f0);
    e1 = e2 = 0;
    if (h > l && h > s.lo(f0) && s.hi(f1) > l) {
      e1 = k.ns + (int)(l - k.lo);
      e2 = k.ns + (int)(h - k.lo);
      if (e1 <= e0) e1 = 0;   // no gap after the sinks
    }
  }
  __device__ __forceinline__ bool see(int v0, int v1) const { return v1 <= e0 || (v0 >= e1 && v1 <= e2); }
};

}  // namespace win

// Allow a kernel its dynamic shared memory, once per device (the attribute stays; setting it again on
// every launch would cost more than the launch).  `done` is the kernel's own; a race sets it twice.
template <typename Kernel>
cudaError_t allow_shared(Kernel kernel, int bytes, std::atomic<uint64_t> &done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (dev < 64 && (done.load(std::memory_order_relaxed) & bit)) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess && dev < 64) done.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

// Heads that a block of the elementwise calls walks over: few enough for about `per_sm` blocks per SM, in
// equal shares.  What a block forms once per token (angles, slots) costs about 2 us of latency, so the
// fewer blocks the better while they still fill the SMs in whole waves: a 720p chunk of 40 heads turns in
// 37 us with 9 blocks per SM (20 heads each), 43 us with 20, 59 us with 45; without angles 20 (writing)
// and 40 (reading back) measure best.
inline int heads_per_block(int64_t tiles, int64_t heads, int num_sms, int per_sm) {
  int64_t parts = ((int64_t)num_sms * per_sm + tiles / 2) / tiles;
  parts = parts < 1 ? 1 : (parts > heads ? heads : parts);
  return (int)((heads + parts - 1) / parts);
}

// Launchers of the recent-window calls (each returns the launch's error).
cudaError_t launch_rope(const qwm_rope_spec &spec, const uint16_t *x, const qwm_strides &xs, int batch, int heads,
                        int64_t n, const int64_t *start, const int32_t *pos, uint16_t *out, const qwm_strides &os,
                        int num_sms, cudaStream_t st);
cudaError_t launch_window_write(const qwm_window &w, const uint16_t *k, const qwm_strides &ks, const uint16_t *v,
                                const qwm_strides &vs, int64_t n, const int64_t *start, const int32_t *count,
                                const qwm_rope_spec *rope, const int32_t *pos, int num_sms, int32_t *status,
                                cudaStream_t st);
cudaError_t launch_window_read(const qwm_window &w, const int64_t *start, const int64_t *length, const int32_t *count,
                               int64_t n, uint16_t *k_hat, uint16_t *v_hat, int num_sms, cudaStream_t st);

// An attention call over the window cache, as its kernels take it.
struct WindowAttend {
  qwm_window w;
  const uint16_t *q;
  qwm_strides qs;
  int64_t nq;
  const int64_t *q_start, *length;
  const int32_t *q_count;
  int64_t tpf, frames;
  float scale_log2;      // softmax_scale * log2(e)
  void *out;
  qwm_strides os;
  int out_f32, merge;
  float *lse;
  int32_t *status;
  int H, group;          // Query heads; Query heads per Key head
  int64_t rows;          // group * nq: Query rows of one Key head, row r = (Query i = r / group, head r % group)
  int splits;            // parts the keys are split into
  int cluster;           // warp tiles: the parts are the CTAs of a cluster
  float *part;           // splits > 1: [batch * kv_heads][splits][rows][128] outputs of the parts,
  float *part_lse;       //             [batch * kv_heads][splits][rows] their log-sum-exps
  win::Bases bases;      // win::kBases
};
// How a call is run: with tensor-memory tiles of 256 Query rows per CTA, or with warp tiles of 8 or 16
// rows; and into how many parts its keys are split.
constexpr int kWindowCluster = 8;   // parts of the warp tiles that are joined inside a thread-block cluster, at most
struct WindowPlan {
  bool tiles;
  int splits;
  bool cluster;   // the parts are a cluster's CTAs; else (splits > 1) a second kernel joins them
  bool joins() const { return splits > 1 && !cluster; }
};
WindowPlan window_plan(int64_t batch, int64_t kv_heads, int64_t rows, int64_t keys, int num_sms);
cudaError_t launch_window_decode(const WindowAttend &a, cudaStream_t st);
cudaError_t launch_window_tiles(const WindowAttend &a, cudaStream_t st);
cudaError_t launch_window_combine(const WindowAttend &a, cudaStream_t st);
