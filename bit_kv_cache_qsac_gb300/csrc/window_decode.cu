// Attention over the window cache for few Query rows (single tokens, drafted tokens, grouped heads),
// and the joining of parts.
//
// A row r of a Key head is (Query r / group, head r % group of the group).  The work is bound by the
// cache's bytes, so the keys are split over `splits` CTAs per Key head and, inside a CTA, over its 8
// warps, 16 keys at a time, straight from global memory into MMA fragments:
//   S^T [16 keys][8 rows] = K [16][128] Q^T        (m16n8k16, fp16 operands, fp32 sums)
//   O^T [128][8 rows]    += V^T [128][16] P^T
// The channels of the first product may come in any order as long as K and Q agree on it, and the rows
// of the second may be any channels, so each thread takes whole 16-byte (8-byte) pieces of a cached row
// and decodes them in registers: one permute and one FMA per pair (two for V, whose pairs run along
// the keys).  Every warp keeps its own running maximum and sum; warps meet in shared memory at the end,
// parts in a second kernel.
#include "window.cuh"

namespace {

constexpr int D = win::D;
constexpr int kWarps = 8, kThreads = 32 * kWarps;
constexpr int kKeys = 16;                  // keys of a warp's step
constexpr float kRescale = 8.f;            // log2 units the maximum may lag behind

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// What a thread holds of 16 cached keys: Key rows g and g + 8, Value rows 2 t, 2 t + 1, 2 t + 8, 2 t + 9.
template <int BITS>
struct Cached {
  uint4 k[2][BITS == 8 ? 2 : 1];
  uint32_t ks[2];
  uint32_t v[4][BITS == 8 ? 4 : 2];
  uint32_t vs[4];
};

// Where a row's output goes, and the final step of every path: write, or merge into what is there.
__device__ __forceinline__ void finish4(const WindowAttend &a, int64_t b, int kvh, int64_t r, int ch, float4 o,
                                        float L) {
  const int64_t i = r / a.group;
  const int h = kvh * a.group + (int)(r - i * a.group);
  const int64_t at = b * a.os.batch + h * a.os.head + i * a.os.token + ch;
  if (a.out_f32) {
    float4 *dst = (float4 *)((float *)a.out + at);
    if (a.merge) {
      const float Lp = a.lse[(b * a.H + h) * a.nq + i], Lm = fmaxf(Lp, L);
      if (Lm == -INFINITY) return;
      const float wp = exp2f(Lp - Lm), wt = exp2f(L - Lm), inv = 1.f / (wp + wt);
      const float4 prev = *dst;
      o.x = fmaf(wt * inv, o.x, wp > 0.f ? wp * inv * prev.x : 0.f);
      o.y = fmaf(wt * inv, o.y, wp > 0.f ? wp * inv * prev.y : 0.f);
      o.z = fmaf(wt * inv, o.z, wp > 0.f ? wp * inv * prev.z : 0.f);
      o.w = fmaf(wt * inv, o.w, wp > 0.f ? wp * inv * prev.w : 0.f);
    }
    *dst = o;
  } else {
    *(uint2 *)((uint16_t *)a.out + at) = make_uint2(tc::pack_bf16x2(o.x, o.y), tc::pack_bf16x2(o.z, o.w));
  }
}
__device__ __forceinline__ void finish_lse(const WindowAttend &a, int64_t b, int kvh, int64_t r, float L) {
  if (!a.lse) return;
  const int64_t i = r / a.group;
  float *p = a.lse + (b * a.H + kvh * a.group + (int)(r - i * a.group)) * a.nq + i;
  if (a.merge) {
    const float Lp = *p, Lm = fmaxf(Lp, L);
    if (Lm == -INFINITY) return;
    L = Lm + log2f(exp2f(Lp - Lm) + exp2f(L - Lm));
  }
  *p = L;
}

template <int BITS, int NT>
__global__ void __launch_bounds__(kThreads, NT == 1 ? 2 : 1) window_decode_kernel(const __grid_constant__ WindowAttend a) {
  __shared__ float osm[kWarps][8][D];
  __shared__ float msm[kWarps][8 * NT], lsm[kWarps][8 * NT];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int64_t b = blockIdx.y / a.w.kv_heads;
  const int kvh = (int)(blockIdx.y - b * a.w.kv_heads);
  const int64_t q0 = a.q_start[b];
  int64_t nq = a.q_count ? (int64_t)a.q_count[b] : a.nq;
  nq = nq < a.nq ? nq : a.nq;
  if (q0 < 0 || nq <= 0) return;
  const win::Seq seq{a.length[b], a.w.sink, a.w.ring, a.tpf, a.frames};
  const int64_t f0 = seq.frame(q0), f1 = seq.frame(q0 + nq - 1);
  win::Keys keys;
  keys.init(seq, f0, f1);
  const uint32_t sink = (uint32_t)a.w.sink, ring = (uint32_t)a.w.ring;
  const int rows = (int)(nq * a.group);

  // ---- the rows this thread masks (columns 2 t, 2 t + 1 of every 8), and what all rows see ----
  win::Row mask[NT][2];
#pragma unroll
  for (int nt = 0; nt < NT; nt++)
#pragma unroll
    for (int e = 0; e < 2; e++) {
      const int r = 8 * nt + 2 * t + e;
      mask[nt][e].init(seq, keys, r < rows ? seq.frame(q0 + r / a.group) : -1);
    }
  win::Everyone every;
  every.init(seq, keys, f0, f1);

  // ---- Queries as the first product's B fragments (row g of every 8), fp16 ----
  uint32_t qf[NT][8][2];
  bool bad = false;
#pragma unroll
  for (int nt = 0; nt < NT; nt++) {
    const int r = 8 * nt + g;
    const int64_t i = r / a.group;
    const uint16_t *qp = a.q + b * a.qs.batch + (kvh * a.group + (r - i * a.group)) * a.qs.head + i * a.qs.token;
#pragma unroll
    for (int ks = 0; ks < 8; ks++) {
      const int ch = BITS == 8 ? 16 * (t + 4 * (ks >> 2)) + 4 * (ks & 3) : 32 * t + 4 * ks;
      const uint2 w = r < rows ? *(const uint2 *)(qp + ch) : make_uint2(0, 0);
      qf[nt][ks][0] = tc::pack_f16x2(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xFFFF0000u));
      qf[nt][ks][1] = tc::pack_f16x2(__uint_as_float(w.y << 16), __uint_as_float(w.y & 0xFFFF0000u));
#pragma unroll
      for (int e = 0; e < 2; e++)
        bad |= (qf[nt][ks][e] & 0x7C00u) == 0x7C00u || (qf[nt][ks][e] & 0x7C000000u) == 0x7C000000u;
    }
  }
  if (bad) qwm_dev_error(a.status, QWM_ERR_RANGE);

  const int64_t head_row = (int64_t)blockIdx.y * (a.w.sink + a.w.ring);
  const uint8_t *kc = a.w.k_codes + head_row * (D * BITS / 8) + 16 * t;
  const uint8_t *vc = a.w.v_codes + head_row * (D * BITS / 8) + (BITS == 8 ? 16 * g : 8 * g);
  const uint8_t *kst = a.w.k_step + head_row * win::kSteps, *vst = a.w.v_step + head_row * win::kSteps + (g >> 1);
  const int steps_all = (keys.total + kKeys - 1) / kKeys;
  const int j0 = (int)((int64_t)steps_all * blockIdx.x / a.splits), j1 = (int)((int64_t)steps_all * (blockIdx.x + 1) / a.splits);

  auto load = [&](int j, Cached<BITS> &c) {
    const int v0 = j * kKeys;
    uint32_t s[6];
    const int dv[6] = {g, g + 8, 2 * t, 2 * t + 1, 2 * t + 8, 2 * t + 9};
    const uint32_t sa = keys.slot(v0, sink, ring);
    if (v0 + kKeys <= keys.total && keys.slot(v0 + kKeys - 1, sink, ring) == sa + kKeys - 1) {
#pragma unroll
      for (int e = 0; e < 6; e++) s[e] = sa + dv[e];
    } else {   // past the sinks, around the ring's end, or the ragged end (its rows masked below)
#pragma unroll
      for (int e = 0; e < 6; e++) s[e] = keys.slot(v0 + dv[e] < keys.total ? v0 + dv[e] : keys.total - 1, sink, ring);
    }
#pragma unroll
    for (int e = 0; e < 2; e++) {
      const uint8_t *p = kc + (uint64_t)s[e] * (D * BITS / 8);
      c.k[e][0] = __ldg((const uint4 *)p);
      if (BITS == 8) c.k[e][BITS == 8 ? 1 : 0] = __ldg((const uint4 *)(p + 64));
      c.ks[e] = __ldg((const uint32_t *)(kst + (uint64_t)s[e] * win::kSteps));
    }
#pragma unroll
    for (int e = 0; e < 4; e++) {
      const uint8_t *p = vc + (uint64_t)s[2 + e] * (D * BITS / 8);
      if (BITS == 8) {
        const uint4 x = __ldg((const uint4 *)p);
        c.v[e][0] = x.x; c.v[e][1] = x.y; c.v[e][BITS == 8 ? 2 : 0] = x.z; c.v[e][BITS == 8 ? 3 : 0] = x.w;
      } else {
        const uint2 x = __ldg((const uint2 *)p);
        c.v[e][0] = x.x; c.v[e][1] = x.y;
      }
      c.vs[e] = __ldg(vst + (uint64_t)s[2 + e] * win::kSteps);
    }
  };

  float o[NT][8][4], m[NT][2], l[NT][2];
#pragma unroll
  for (int nt = 0; nt < NT; nt++) {
#pragma unroll
    for (int i = 0; i < 8; i++)
#pragma unroll
      for (int e = 0; e < 4; e++) o[nt][i][e] = 0.f;
    m[nt][0] = m[nt][1] = -INFINITY;
    l[nt][0] = l[nt][1] = 0.f;
  }

  auto step = [&](int j, const Cached<BITS> &c) {
    const int v0 = j * kKeys;
    float s[NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; nt++) s[nt][0] = s[nt][1] = s[nt][2] = s[nt][3] = 0.f;
    // ---- S^T ----
    if (BITS == 8) {
#pragma unroll
      for (int pc = 0; pc < 2; pc++) {   // pieces t and t + 4: step groups t / 2 and 2 + t / 2
        uint32_t s2[2], n2[2];
#pragma unroll
        for (int e = 0; e < 2; e++) win::step_consts<8>((c.ks[e] >> (8 * (2 * pc + (t >> 1)))) & 0xFFu, s2[e], n2[e]);
        const uint32_t x[2][4] = {{c.k[0][pc % (BITS == 8 ? 2 : 1)].x, c.k[0][pc % (BITS == 8 ? 2 : 1)].y,
                                   c.k[0][pc % (BITS == 8 ? 2 : 1)].z, c.k[0][pc % (BITS == 8 ? 2 : 1)].w},
                                  {c.k[1][pc % (BITS == 8 ? 2 : 1)].x, c.k[1][pc % (BITS == 8 ? 2 : 1)].y,
                                   c.k[1][pc % (BITS == 8 ? 2 : 1)].z, c.k[1][pc % (BITS == 8 ? 2 : 1)].w}};
#pragma unroll
        for (int u = 0; u < 4; u++) {
          uint32_t a0, a1, a2, a3;
          win::decode8(x[0][u], s2[0], n2[0], a0, a2);
          win::decode8(x[1][u], s2[1], n2[1], a1, a3);
#pragma unroll
          for (int nt = 0; nt < NT; nt++) mma16816(s[nt], a0, a1, a2, a3, qf[nt][4 * pc + u][0], qf[nt][4 * pc + u][1]);
        }
      }
    } else {
      uint32_t s2[2], n2[2];
#pragma unroll
      for (int e = 0; e < 2; e++) win::step_consts<4>((c.ks[e] >> (8 * t)) & 0xFFu, s2[e], n2[e]);
      const uint32_t x[2][4] = {{c.k[0][0].x, c.k[0][0].y, c.k[0][0].z, c.k[0][0].w},
                                {c.k[1][0].x, c.k[1][0].y, c.k[1][0].z, c.k[1][0].w}};
#pragma unroll
      for (int u = 0; u < 4; u++) {
        uint32_t p[4], r[4];
        win::decode4(x[0][u], s2[0], n2[0], p);
        win::decode4(x[1][u], s2[1], n2[1], r);
#pragma unroll
        for (int nt = 0; nt < NT; nt++) {
          mma16816(s[nt], p[0], r[0], p[1], r[1], qf[nt][2 * u][0], qf[nt][2 * u][1]);
          mma16816(s[nt], p[2], r[2], p[3], r[3], qf[nt][2 * u + 1][0], qf[nt][2 * u + 1][1]);
        }
      }
    }
    // ---- logits in log2 units, masked; the running maximum; P ----
    const bool full = every.see(v0, v0 + kKeys);
    uint32_t pb[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; nt++) {
#pragma unroll
      for (int e = 0; e < 4; e++) {
        s[nt][e] *= a.scale_log2;
        if (!full && !mask[nt][e & 1].sees(v0 + g + 8 * (e >> 1))) s[nt][e] = -INFINITY;
      }
      const float x0 = fmaxf(s[nt][0], s[nt][2]), x1 = fmaxf(s[nt][1], s[nt][3]);
      if (__any_sync(0xffffffffu, x0 > m[nt][0] + kRescale || x1 > m[nt][1] + kRescale)) {
        float n0 = x0, n1 = x1;
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) {
          n0 = fmaxf(n0, __shfl_xor_sync(0xffffffffu, n0, d));
          n1 = fmaxf(n1, __shfl_xor_sync(0xffffffffu, n1, d));
        }
        n0 = fmaxf(n0, m[nt][0]);
        n1 = fmaxf(n1, m[nt][1]);
        const float w0 = n0 == -INFINITY ? 1.f : tc::ex2_approx(m[nt][0] - n0);
        const float w1 = n1 == -INFINITY ? 1.f : tc::ex2_approx(m[nt][1] - n1);
        l[nt][0] *= w0;
        l[nt][1] *= w1;
#pragma unroll
        for (int i = 0; i < 8; i++) {
          o[nt][i][0] *= w0;
          o[nt][i][1] *= w1;
          o[nt][i][2] *= w0;
          o[nt][i][3] *= w1;
        }
        m[nt][0] = n0;
        m[nt][1] = n1;
      }
      const float m0 = m[nt][0] == -INFINITY ? 0.f : m[nt][0], m1 = m[nt][1] == -INFINITY ? 0.f : m[nt][1];
      const float p0 = tc::ex2_approx(s[nt][0] - m0), p1 = tc::ex2_approx(s[nt][1] - m1);
      const float p2 = tc::ex2_approx(s[nt][2] - m0), p3 = tc::ex2_approx(s[nt][3] - m1);
      l[nt][0] += p0 + p2;
      l[nt][1] += p1 + p3;
      pb[nt][0] = transpose8x8(tc::pack_f16x2(p0, p1));
      pb[nt][1] = transpose8x8(tc::pack_f16x2(p2, p3));
    }
    // ---- O^T: m-tile i holds channels 16 g + 2 i (rows 0-7) and 16 g + 2 i + 1 (rows 8-15) ----
    uint32_t s2[2], n2[2];
#pragma unroll
    for (int e = 0; e < 2; e++) {
      s2[e] = (c.vs[2 * e] << 7) | (c.vs[2 * e + 1] << 23);
      asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(n2[e]) : "r"(s2[e]), "r"(BITS == 8 ? 0xE480E480u : 0xD480D480u));
    }
    if (BITS == 8) {
#pragma unroll
      for (int i = 0; i < 8; i++) {
        const int w = i >> 1;
        const uint32_t sel = (i & 1) ? 0x7632u : 0x5410u;
        const uint32_t x = __byte_perm(c.v[0][w % (BITS == 8 ? 4 : 2)], c.v[1][w % (BITS == 8 ? 4 : 2)], sel);
        const uint32_t y = __byte_perm(c.v[2][w % (BITS == 8 ? 4 : 2)], c.v[3][w % (BITS == 8 ? 4 : 2)], sel);
        const uint32_t a0 = tc::hfma2((x & 0x00FF00FFu) | 0x64006400u, s2[0], n2[0]);
        const uint32_t a1 = tc::hfma2(((x >> 8) & 0x00FF00FFu) | 0x64006400u, s2[0], n2[0]);
        const uint32_t a2 = tc::hfma2((y & 0x00FF00FFu) | 0x64006400u, s2[1], n2[1]);
        const uint32_t a3 = tc::hfma2(((y >> 8) & 0x00FF00FFu) | 0x64006400u, s2[1], n2[1]);
#pragma unroll
        for (int nt = 0; nt < NT; nt++) mma16816(o[nt][i], a0, a1, a2, a3, pb[nt][0], pb[nt][1]);
      }
    } else {
#pragma unroll
      for (int w = 0; w < 2; w++) {
        uint32_t ev[2][4], od[2][4];
#pragma unroll
        for (int e = 0; e < 2; e++) {   // low halves: nibbles 0-3 (even channels), high halves: odd
          win::decode4(__byte_perm(c.v[2 * e][w], c.v[2 * e + 1][w], 0x5410), s2[e], n2[e], ev[e]);
          win::decode4(__byte_perm(c.v[2 * e][w], c.v[2 * e + 1][w], 0x7632), s2[e], n2[e], od[e]);
        }
#pragma unroll
        for (int k = 0; k < 4; k++)
#pragma unroll
          for (int nt = 0; nt < NT; nt++) mma16816(o[nt][4 * w + k], ev[0][k], od[0][k], ev[1][k], od[1][k], pb[nt][0], pb[nt][1]);
      }
    }
  };

  {   // two steps in flight: the next one's loads are issued before this one's products
    Cached<BITS> c0, c1;
    int j = j0 + warp;
    if (j < j1) load(j, c0);
    while (j < j1) {
      if (j + kWarps < j1) load(j + kWarps, c1);
      step(j, c0);
      j += kWarps;
      if (j >= j1) break;
      if (j + kWarps < j1) load(j + kWarps, c0);
      step(j, c1);
      j += kWarps;
    }
  }

  // ---- the warps' parts joined in shared memory ----
#pragma unroll
  for (int nt = 0; nt < NT; nt++) {
#pragma unroll
    for (int e = 0; e < 2; e++) {
      float s = l[nt][e];
#pragma unroll
      for (int d = 4; d < 32; d <<= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
      if (g == 0) {
        msm[warp][8 * nt + 2 * t + e] = m[nt][e];
        lsm[warp][8 * nt + 2 * t + e] = s;
      }
    }
  }
#pragma unroll
  for (int nt = 0; nt < NT; nt++) {
    if (nt) __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; i++) {
      *(float2 *)&osm[warp][2 * t][16 * g + 2 * i] = make_float2(o[nt][i][0], o[nt][i][2]);
      *(float2 *)&osm[warp][2 * t + 1][16 * g + 2 * i] = make_float2(o[nt][i][1], o[nt][i][3]);
    }
    __syncthreads();
    const int r = 8 * nt + warp, ch = 4 * lane;   // warp = row, lane = four channels
    if (r < rows) {
      float M = -INFINITY;
#pragma unroll
      for (int w = 0; w < kWarps; w++) M = fmaxf(M, msm[w][r]);
      float L = 0.f;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kWarps; w++) {
        const float wt = msm[w][r] == -INFINITY ? 0.f : tc::ex2_approx(msm[w][r] - M);
        const float4 x = *(const float4 *)&osm[w][warp][ch];
        L = fmaf(lsm[w][r], wt, L);
        acc.x = fmaf(x.x, wt, acc.x);
        acc.y = fmaf(x.y, wt, acc.y);
        acc.z = fmaf(x.z, wt, acc.z);
        acc.w = fmaf(x.w, wt, acc.w);
      }
      const float inv = L > 0.f ? 1.f / L : 0.f, lse = L > 0.f ? M + log2f(L) : -INFINITY;
      acc = make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
      if (a.splits == 1) {
        finish4(a, b, kvh, r, ch, acc, lse);
        __syncwarp();   // merging lanes have read the earlier log-sum-exp
        if (lane == 0) finish_lse(a, b, kvh, r, lse);
      } else {
        const int64_t pr = ((int64_t)blockIdx.y * a.splits + blockIdx.x) * a.rows + r;
        *(float4 *)(a.part + pr * D + ch) = acc;
        if (lane == 0) a.part_lse[pr] = lse;
      }
    }
  }
}

// Parts of a row joined: the weighted mean of the parts' outputs, each weighted by its share of the
// exponential sum.  One warp per row.
__global__ void __launch_bounds__(256) window_combine_kernel(const __grid_constant__ WindowAttend a) {
  const int lane = threadIdx.x & 31;
  const int64_t item = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int64_t heads = (int64_t)a.w.batch * a.w.kv_heads;
  if (item >= heads * a.rows) return;
  const int64_t y = item / a.rows, r = item - y * a.rows, b = y / a.w.kv_heads;
  const int kvh = (int)(y - b * a.w.kv_heads);
  if (a.q_start[b] < 0 || (a.q_count && r / a.group >= a.q_count[b])) return;
  const float *pl = a.part_lse + y * a.splits * a.rows + r;
  float M = -INFINITY;
  for (int s = 0; s < a.splits; s++) M = fmaxf(M, pl[s * a.rows]);
  float L = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  if (M > -INFINITY) {
    const float *po = a.part + (y * a.splits * a.rows + r) * D + 4 * lane;
#pragma unroll 4
    for (int s = 0; s < a.splits; s++) {
      const float wt = exp2f(pl[s * a.rows] - M);
      const float4 x = *(const float4 *)(po + (int64_t)s * a.rows * D);
      L += wt;
      acc.x = fmaf(x.x, wt, acc.x);
      acc.y = fmaf(x.y, wt, acc.y);
      acc.z = fmaf(x.z, wt, acc.z);
      acc.w = fmaf(x.w, wt, acc.w);
    }
    const float inv = 1.f / L;
    acc = make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
  }
  const float lse = L > 0.f ? M + log2f(L) : -INFINITY;
  finish4(a, b, kvh, r, 4 * lane, acc, lse);
  __syncwarp();
  if (lane == 0) finish_lse(a, b, kvh, r, lse);
}

template <int BITS>
cudaError_t decode_bits(const WindowAttend &a, cudaStream_t st) {
  const dim3 grid((unsigned)a.splits, (unsigned)(a.w.batch * a.w.kv_heads));
  if (a.rows <= 8) window_decode_kernel<BITS, 1><<<grid, kThreads, 0, st>>>(a);
  else window_decode_kernel<BITS, 2><<<grid, kThreads, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_window_decode(const WindowAttend &a, cudaStream_t st) {
  return a.w.bits == 8 ? decode_bits<8>(a, st) : decode_bits<4>(a, st);
}

cudaError_t launch_window_combine(const WindowAttend &a, cudaStream_t st) {
  const int64_t items = (int64_t)a.w.batch * a.w.kv_heads * a.rows;
  window_combine_kernel<<<(unsigned)((items + 7) / 8), 256, 0, st>>>(a);
  return cudaGetLastError();
}
