// Attention of up to 16 Query rows over cached rows on warp MMAs, one warp at a time: the parts that the
// kernels for few rows share (over the window cache, over pages).
//
//   S^T [16 keys][8 rows] = K [16][128] Q^T        (m16n8k16, fp16 operands, fp32 sums)
//   O^T [128][8 rows]    += V^T [128][16] P^T
// The channels of the first product may come in any order as long as K and Q agree on it, the rows of
// the second may be any channels, and the 16 keys may stand in any order as long as P and V agree on it.
// So a thread takes whole 16-byte (8-byte) pieces of a cached row, its four Value rows are neighbours,
// and everything is decoded in registers: one permute and one FMA per pair at 8 bits (half a permute
// more for V, whose pairs run along the keys).
#pragma once

#include "window.cuh"

namespace wt {

constexpr int D = win::D;
constexpr int kWarps = 8;
// Keys of a warp's step: 32 at 4 bits, where instructions count (address and maximum are then shared by
// two MMA rows of keys), 16 at 8 bits, where twice as many would halve the CTAs that fit an SM.
__host__ __device__ constexpr int step_keys(int bits) { return bits == 4 ? 32 : 16; }
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

// Two step bytes (the bytes that `sel` takes from a and b in halves 0 and 1) as a pair of fp16 steps.
__device__ __forceinline__ uint32_t step_pair(uint32_t a, uint32_t b, uint32_t sel) {
  return (__byte_perm(a, b, sel) & 0x00FF00FFu) * 128u;
}

// A warp's ring of shared memory: per stage the Key rows of a step, its Value rows, their steps.
template <int BITS>
struct Ring {
  static constexpr int kKeys = step_keys(BITS);
  static constexpr int kRow = D * BITS / 8;            // bytes of a row
  static constexpr int kV = kKeys * kRow, kKS = 2 * kV, kVS = kKS + 4 * kKeys;
  static constexpr int kStage = kVS + 4 * kKeys;
  static constexpr int kStages = 3;
  static constexpr int kBytes = kWarps * kStages * kStage + 128;
  // 16-byte pieces are permuted within 128 bytes so that a quarter (half) warp's reads of 16 (8) bytes
  // fall into different banks: Key rows are read two neighbours at a time, Value rows four apart
  __device__ static __forceinline__ uint32_t k_at(int row, int piece) {
    if (BITS == 8) return (uint32_t)(row * 128 + ((piece ^ ((row & 1) << 2)) << 4));
    return (uint32_t)(row * 64 + (piece << 4));
  }
  __device__ static __forceinline__ uint32_t v_at(int row, int piece) {
    if (BITS == 8) return (uint32_t)(kV + row * 128 + ((piece ^ (((row >> 2) & 3) << 1)) << 4));
    return (uint32_t)(kV + (row >> 1) * 128 + (((((row & 1) << 2) + piece) ^ (((row >> 2) & 3) << 1)) << 4));
  }
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void *src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}

// One warp's Queries (rows of 8 NT), outputs, maxima and sums.
template <int BITS, int NT>
struct Tile {
  using R = Ring<BITS>;
  static constexpr int kKeys = R::kKeys, kSub = kKeys / 16;   // MMA rows of 16 keys in a step
  uint32_t qf[NT][8][2];   // Queries as the first product's B fragments (row g of every 8): bf16, then fp16
  float sl2[NT][2];        // logit scale of rows 2 t, 2 t + 1 of every 8
  float o[NT][8][4], m[NT][2], mneg[NT][2], l[NT][2];
  int g, t, krow;          // krow: the key of MMA row g; row g + 8 is two further on
  uint32_t ksel, vsel;     // the step byte of the thread's group, of one row or of two
  uint32_t koff, ksoff, vsoff, voff;   // this lane's addresses inside a stage

  __device__ __forceinline__ void place(int lane) {
    g = lane >> 2;
    t = lane & 3;
    krow = 4 * (g >> 1) + (g & 1);
    ksel = BITS == 8 ? (uint32_t)(t >> 1) * 0x1111u : (uint32_t)t * 0x1111u;
    vsel = (uint32_t)(g >> 1) * 0x1111u + 0x4400u;
    koff = R::k_at(krow, t);
    ksoff = R::kKS + 4u * krow;
    vsoff = R::kVS + 16u * t;
    voff = BITS == 8 ? R::v_at(4 * t, g) : R::v_at(4 * t, g >> 1) + 8u * (g & 1);
  }
  // Row g of the nt-th eight rows from qp, or zeros.
  __device__ __forceinline__ void fetch(int nt, const uint16_t *qp, bool there) {
#pragma unroll
    for (int ks = 0; ks < 8; ks++) {
      const int ch = BITS == 8 ? 16 * (t + 4 * (ks >> 2)) + 4 * (ks & 3) : 32 * t + 4 * ks;
      const uint2 w = there ? *(const uint2 *)(qp + ch) : make_uint2(0, 0);
      qf[nt][ks][0] = w.x;
      qf[nt][ks][1] = w.y;
    }
  }
  // The fetched Queries of `rows` live rows made ready, nothing seen yet.
  __device__ __forceinline__ void begin(int rows, float scale_log2, int32_t *status) {
    // ---- the Queries to fp16; each row's logit scale ----
#pragma unroll
    for (int nt = 0; nt < NT; nt++) {
      const bool live = 8 * nt + g < rows;
      uint32_t big = 0u;   // largest magnitudes of this thread's quarter of row g
#pragma unroll
      for (int ks = 0; ks < 8; ks++)
#pragma unroll
        for (int e = 0; e < 2; e++) {
          qf[nt][ks][e] = live ? qf[nt][ks][e] : 0u;
          big = win::max_abs_bf16x2(big, qf[nt][ks][e]);
        }
      big &= 0x7FFF7FFFu;
      if (win::any_beyond_fp16(big)) qwm_dev_error(status, QWM_ERR_RANGE);
      uint32_t whole = __ballot_sync(0xffffffffu, !live || win::any_from_one(big));   // four bits a row
      whole |= whole >> 1;
      whole |= whole >> 2;
      int power = 0;
      if ((whole & 0x11111111u) != 0x11111111u) {   // a row of small Queries
        uint32_t top = win::larger_half(big);
#pragma unroll
        for (int d = 1; d < 4; d <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, d));
        if (top < 0x3F80u) power = (int)win::row_power(top);
      }
      const float up = win::power_of_two(power), back = win::power_of_two(-power);
#pragma unroll
      for (int ks = 0; ks < 8; ks++)
#pragma unroll
        for (int e = 0; e < 2; e++) {
          const uint32_t w = qf[nt][ks][e];
          qf[nt][ks][e] = tc::pack_f16x2(__uint_as_float(w << 16) * up, __uint_as_float(w & 0xFFFF0000u) * up);
        }
#pragma unroll
      for (int e = 0; e < 2; e++)
        sl2[nt][e] = win::logit_scale<BITS>(scale_log2, __shfl_sync(0xffffffffu, back, 4 * (2 * t + e)));
    }

#pragma unroll
    for (int nt = 0; nt < NT; nt++) {
#pragma unroll
      for (int i = 0; i < 8; i++)
#pragma unroll
        for (int e = 0; e < 4; e++) o[nt][i][e] = 0.f;
      m[nt][0] = m[nt][1] = -INFINITY;
      mneg[nt][0] = mneg[nt][1] = 0.f;   // -m, or 0 before any key
      l[nt][0] = l[nt][1] = 0.f;
    }
  }
  // The keys of the stage at shared address st, numbered from v0.  all: every row sees them all; else
  // mask_of(r).sees(v) says whether row r sees key v.
  template <typename MaskOf>
  __device__ __forceinline__ void step(uint32_t st, int v0, bool all, MaskOf mask_of, const win::Bases &bases) {
    // ---- S^T, each 16 keys in two sums ----
    float s[kSub][NT][4];
#pragma unroll
    for (int u16 = 0; u16 < kSub; u16++) {
      float s_[NT][4];
#pragma unroll
      for (int nt = 0; nt < NT; nt++)
#pragma unroll
        for (int e = 0; e < 4; e++) s[u16][nt][e] = s_[nt][e] = 0.f;
      const uint32_t kb = st + koff + (uint32_t)(u16 * 16 * R::kRow), ksb = st + ksoff + 64u * u16;
      const uint32_t kst[2] = {tc::lds32(ksb), tc::lds32(ksb + 8u)};
      if (BITS == 8) {
#pragma unroll
        for (int pc = 0; pc < 2; pc++) {   // pieces t and t + 4: step groups t / 2 and 2 + t / 2
          win::Step ks[2];
#pragma unroll
          for (int e = 0; e < 2; e++) ks[e] = win::step_of<8>(step_pair(kst[e], kst[e], ksel + (pc ? 0x2222u : 0u)));
          const uint32_t ka = kb ^ (pc ? 64u : 0u);
          const uint4 xa = tc::lds128(ka), xb = tc::lds128(ka + 256u);
          const uint32_t x[2][4] = {{xa.x, xa.y, xa.z, xa.w}, {xb.x, xb.y, xb.z, xb.w}};
#pragma unroll
          for (int u = 0; u < 4; u++) {
            uint32_t a0, a1, a2, a3;
            win::decode8(x[0][u], ks[0], bases, a0, a2);
            win::decode8(x[1][u], ks[1], bases, a1, a3);
#pragma unroll
            for (int nt = 0; nt < NT; nt++)
              mma16816((u & 1) ? s_[nt] : s[u16][nt], a0, a1, a2, a3, qf[nt][4 * pc + u][0], qf[nt][4 * pc + u][1]);
          }
        }
      } else {
        win::Step ks[2];
#pragma unroll
        for (int e = 0; e < 2; e++) ks[e] = win::step_of<4>(step_pair(kst[e], kst[e], ksel));
        const uint4 xa = tc::lds128(kb), xb = tc::lds128(kb + 128u);
        const uint32_t x[2][4] = {{xa.x, xa.y, xa.z, xa.w}, {xb.x, xb.y, xb.z, xb.w}};
#pragma unroll
        for (int u = 0; u < 4; u++) {
          uint32_t p[4], r[4];
          win::decode4(x[0][u], ks[0], bases, p);
          win::decode4(x[1][u], ks[1], bases, r);
#pragma unroll
          for (int nt = 0; nt < NT; nt++) {
            mma16816(s[u16][nt], p[0], r[0], p[1], r[1], qf[nt][2 * u][0], qf[nt][2 * u][1]);
            mma16816(s_[nt], p[2], r[2], p[3], r[3], qf[nt][2 * u + 1][0], qf[nt][2 * u + 1][1]);
          }
        }
      }
#pragma unroll
      for (int nt = 0; nt < NT; nt++)
#pragma unroll
        for (int e = 0; e < 4; e++) s[u16][nt][e] += s_[nt][e];
    }
    // ---- masked; the running maximum (log2 units, less kTopWeight); P ----
    if (!all) {   // a few steps of a call: what each of the thread's rows sees is worked out here
#pragma unroll
      for (int nt = 0; nt < NT; nt++)
#pragma unroll
        for (int e = 0; e < 2; e++) {
          const auto mask = mask_of(8 * nt + 2 * t + e);
#pragma unroll
          for (int u16 = 0; u16 < kSub; u16++)
#pragma unroll
            for (int k = 0; k < 2; k++)
              if (!mask.sees(v0 + 16 * u16 + krow + 2 * k)) s[u16][nt][e + 2 * k] = -INFINITY;
        }
    }
    uint32_t pb[kSub][NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; nt++) {
      float x0 = fmaxf(s[0][nt][0], s[0][nt][2]), x1 = fmaxf(s[0][nt][1], s[0][nt][3]);
#pragma unroll
      for (int u16 = 1; u16 < kSub; u16++) {
        x0 = tc::max3(x0, s[u16][nt][0], s[u16][nt][2]);
        x1 = tc::max3(x1, s[u16][nt][1], s[u16][nt][3]);
      }
      x0 = fmaf(x0, sl2[nt][0], -win::kTopWeight);
      x1 = fmaf(x1, sl2[nt][1], -win::kTopWeight);
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
        mneg[nt][0] = n0 == -INFINITY ? 0.f : -n0;
        mneg[nt][1] = n1 == -INFINITY ? 0.f : -n1;
      }
#pragma unroll
      for (int u16 = 0; u16 < kSub; u16++) {
        float p[4];
#pragma unroll
        for (int e = 0; e < 4; e++) p[e] = tc::ex2_approx(fmaf(s[u16][nt][e], sl2[nt][e & 1], mneg[nt][e & 1]));
        l[nt][0] += p[0] + p[2];
        l[nt][1] += p[1] + p[3];
        pb[u16][nt][0] = transpose8x8(tc::pack_f16x2(p[0], p[1]));
        pb[u16][nt][1] = transpose8x8(tc::pack_f16x2(p[2], p[3]));
      }
    }
    // ---- O^T: m-tile i holds channels 16 g + 2 i (rows 0-7) and 16 g + 2 i + 1 (rows 8-15); MMA columns
    // 2 t, 2 t + 1, 2 t + 8, 2 t + 9 are keys 4 t .. 4 t + 3 ----
#pragma unroll
    for (int u16 = 0; u16 < kSub; u16++) {
      const uint32_t vb = st + voff + (uint32_t)(u16 * 16 * R::kRow);
      const uint4 vs = tc::lds128(st + vsoff + 64u * u16);   // the steps of keys 4 t .. 4 t + 3
      const win::Step vt[2] = {win::step_of<BITS>(step_pair(vs.x, vs.y, vsel)), win::step_of<BITS>(step_pair(vs.z, vs.w, vsel))};
      if (BITS == 8) {
        uint4 x[4];
#pragma unroll
        for (int e = 0; e < 4; e++) x[e] = tc::lds128(vb + 128u * e);
#pragma unroll
        for (int w = 0; w < 4; w++) {
          const uint32_t q[4] = {w == 0 ? x[0].x : w == 1 ? x[0].y : w == 2 ? x[0].z : x[0].w,
                                 w == 0 ? x[1].x : w == 1 ? x[1].y : w == 2 ? x[1].z : x[1].w,
                                 w == 0 ? x[2].x : w == 1 ? x[2].y : w == 2 ? x[2].z : x[2].w,
                                 w == 0 ? x[3].x : w == 1 ? x[3].y : w == 2 ? x[3].z : x[3].w};
#pragma unroll
          for (int h = 0; h < 2; h++) {
            const uint32_t sel = h ? 0x7632u : 0x5410u;
            const uint32_t ka = __byte_perm(q[0], q[1], sel), kb = __byte_perm(q[2], q[3], sel);
            const uint32_t a0 = tc::hfma2(win::place<0x00FF00FFu>(ka, bases.k1024), vt[0].s, vt[0].n);
            const uint32_t a1 = tc::hfma2(win::place<0x00FF00FFu>(ka >> 8, bases.k1024), vt[0].s, vt[0].n);
            const uint32_t a2 = tc::hfma2(win::place<0x00FF00FFu>(kb, bases.k1024), vt[1].s, vt[1].n);
            const uint32_t a3 = tc::hfma2(win::place<0x00FF00FFu>(kb >> 8, bases.k1024), vt[1].s, vt[1].n);
#pragma unroll
            for (int nt = 0; nt < NT; nt++) mma16816(o[nt][2 * w + h], a0, a1, a2, a3, pb[u16][nt][0], pb[u16][nt][1]);
          }
        }
      } else {
        uint2 x[4];   // rows 4 t + e: neighbours of one 128-byte line differ in one address bit
#pragma unroll
        for (int e = 0; e < 4; e++) x[e] = tc::lds64((vb ^ (64u * (e & 1))) + 128u * (e >> 1));
#pragma unroll
        for (int w = 0; w < 2; w++) {
          uint32_t ev[2][4], od[2][4];
#pragma unroll
          for (int e = 0; e < 2; e++) {   // low halves: nibbles 0-3 (even channels), high halves: odd
            const uint32_t qa = w ? x[2 * e].y : x[2 * e].x, qb = w ? x[2 * e + 1].y : x[2 * e + 1].x;
            win::decode4(__byte_perm(qa, qb, 0x5410), vt[e], bases, ev[e]);
            win::decode4(__byte_perm(qa, qb, 0x7632), vt[e], bases, od[e]);
          }
#pragma unroll
          for (int k = 0; k < 4; k++)
#pragma unroll
            for (int nt = 0; nt < NT; nt++)
              mma16816(o[nt][4 * w + k], ev[0][k], od[0][k], ev[1][k], od[1][k], pb[u16][nt][0], pb[u16][nt][1]);
        }
      }
    }
  }
  // The warp's sums of row r of its eight, in lanes of g == 0, and its maxima.
  __device__ __forceinline__ void sums(float (&msm)[8 * NT], float (&lsm)[8 * NT]) const {
#pragma unroll
    for (int nt = 0; nt < NT; nt++)
#pragma unroll
      for (int e = 0; e < 2; e++) {
        float s = l[nt][e];
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
        if (g == 0) {
          msm[8 * nt + 2 * t + e] = m[nt][e];
          lsm[8 * nt + 2 * t + e] = s;
        }
      }
  }
  // The outputs of the nt-th eight rows, those of them below `rows`.  Pairs of channels are permuted by the row and the
  // quarter of the row, so that a half warp's stores fall into different banks (in their own order 8 of 16 collide).
  __device__ __forceinline__ void outputs(int nt, int rows, float (*osm)[D]) const {
#pragma unroll
    for (int i = 0; i < 8; i++) {
      const int c = 2 * ((8 * g + i) ^ (2 * t | (g >> 1 & 1)));
      if (8 * nt + 2 * t < rows) *(float2 *)&osm[2 * t][c] = make_float2(o[nt][i][0], o[nt][i][2]);
      if (8 * nt + 2 * t + 1 < rows) *(float2 *)&osm[2 * t + 1][c] = make_float2(o[nt][i][1], o[nt][i][3]);
    }
  }
  // Channels 4 lane .. 4 lane + 3 of row r of eight from there.
  __device__ static __forceinline__ float4 output(const float (*osm)[D], int r, int lane) {
    const float4 x = ((const float4 *)osm[r])[lane ^ (r >> 1)];
    return lane & 8 ? make_float4(x.z, x.w, x.x, x.y) : x;
  }
};

// Four channels of a row from the warps' parts (unnormalised), its maximum M and sum L; osm_of(w): warp w's.
template <int WARPS, int ROWS, typename Osm>
__device__ __forceinline__ float4 join(const float (&msm)[WARPS][ROWS], const float (&lsm)[WARPS][ROWS], int r, Osm osm_of,
                                       float &M, float &L) {
  M = -INFINITY;
#pragma unroll
  for (int w = 0; w < WARPS; w++) M = fmaxf(M, msm[w][r]);
  L = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int w = 0; w < WARPS; w++) {
    const float wt = msm[w][r] == -INFINITY ? 0.f : tc::ex2_approx(msm[w][r] - M);
    const float4 x = osm_of(w);
    L = fmaf(lsm[w][r], wt, L);
    acc.x = fmaf(x.x, wt, acc.x);
    acc.y = fmaf(x.y, wt, acc.y);
    acc.z = fmaf(x.z, wt, acc.z);
    acc.w = fmaf(x.w, wt, acc.w);
  }
  return acc;
}

}  // namespace wt
