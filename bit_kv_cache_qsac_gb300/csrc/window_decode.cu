// Attention over the window cache for few Query rows (single tokens, drafted tokens, grouped heads),
// and the joining of parts.
//
// A row r of a Key head is (Query r / group, head r % group of the group).  The work is bound by the
// cache's bytes, so the keys are split over `splits` CTAs per Key head and, inside a CTA, over its 8
// warps, 16 or 32 keys at a time, copied to a ring of shared memory of the warp's own two steps ahead
// (cp.async; no barrier but the warp's) and multiplied on warp MMAs:
//   S^T [16 keys][8 rows] = K [16][128] Q^T        (m16n8k16, fp16 operands, fp32 sums)
//   O^T [128][8 rows]    += V^T [128][16] P^T
// The channels of the first product may come in any order as long as K and Q agree on it, the rows of
// the second may be any channels, and the 16 keys may stand in any order as long as P and V agree on it.
// So a thread takes whole 16-byte (8-byte) pieces of a cached row, its four Value rows are neighbours,
// and everything is decoded in registers: one permute and one FMA per pair at 8 bits (half a permute
// more for V, whose pairs run along the keys).  Every warp keeps its own running maximum and sum; warps
// meet in shared memory at the end, the parts of a Key head (up to 8) in the shared memory of a
// thread-block cluster, more parts in a second kernel.
// Measured: 16 sequences x 32 heads (8 Key heads) x 4,096 keys at 8 bits in 27 to 28 us = 5.0 TB/s, about 7
// us of it before the first keys arrive and in the join; 40 heads x 39,000 keys at 4 bits in 52 us = 4.1
// TB/s (8 bits: 69 us = 6.0).  At 4 bits neither the issue slots (62%: 316 warp instructions per 16 keys of a
// head, 160 of them placing, unbiasing and scaling codes) nor DRAM (55%) are full: four warps per scheduler
// run load, product, maximum and product one behind the other, and 280 CTAs stand on 304 places.
// 9 to 16 rows take 220 to 234 registers a thread, so one CTA per SM (16 rows of 40 heads over 39,000 keys:
// 90 us at 8 bits, 81 at 4), and 17 to 32 read and decode the cache twice (166 to 170, 140 to 144).
#include "window.cuh"

namespace {

constexpr int D = win::D;
constexpr int kWarps = 8, kThreads = 32 * kWarps;
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

// Where a row's output goes, and the final step of every path: write, or merge into what is there.
__device__ __forceinline__ void finish4(const WindowAttend &a, int64_t b, int kvh, int64_t r, int ch, float4 o,
                                        float L) {
  const int64_t i = win::quotient(r, a.group);
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
  const int64_t i = win::quotient(r, a.group);
  float *p = a.lse + (b * a.H + kvh * a.group + (int)(r - i * a.group)) * a.nq + i;
  if (a.merge) {
    const float Lp = *p, Lm = fmaxf(Lp, L);
    if (Lm == -INFINITY) return;
    L = Lm + log2f(exp2f(Lp - Lm) + exp2f(L - Lm));
  }
  *p = L;
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
__device__ __forceinline__ float4 ld_cluster4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr));
  return v;
}
__device__ __forceinline__ float2 ld_cluster2(uint32_t addr) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr));
  return v;
}

// CLUSTER: the parts of a Key head are the CTAs of a cluster and are joined in it.
template <int BITS, int NT, bool CLUSTER>
__global__ void __launch_bounds__(kThreads, NT == 1 ? 2 : 1) window_decode_kernel(const __grid_constant__ WindowAttend a) {
  using R = Ring<BITS>;
  constexpr int kKeys = R::kKeys, kSub = kKeys / 16;   // MMA rows of 16 keys in a step
  extern __shared__ __align__(16) unsigned char dyn_raw[];
  // stages start on 128-byte boundaries: permuted addresses are reached by flipping bits
  unsigned char *dyn = dyn_raw + ((128u - (tc::smem_u32(dyn_raw) & 127u)) & 127u);
  __shared__ float msm[kWarps][8 * NT], lsm[kWarps][8 * NT];
  __shared__ __align__(16) float part_o[CLUSTER ? 8 * NT : 1][D];
  __shared__ __align__(8) float2 part_ml[CLUSTER ? 8 * NT : 1];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const uint32_t b = blockIdx.y / (uint32_t)a.w.kv_heads;
  const int kvh = (int)(blockIdx.y - b * (uint32_t)a.w.kv_heads);
  if (!CLUSTER) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");   // the joining kernel may line up
  // the sequence's numbers, on their way first: the first copies wait for them
  const int64_t q0 = a.q_start[b], len = win::tokens_of(a.length[b]);
  int64_t nq = a.q_count ? (int64_t)a.q_count[b] : a.nq;
  const int row0 = 8 * NT * (int)blockIdx.z;   // this CTA's block of rows
  // ---- Queries as the first product's B fragments (row g of every 8), bf16 for now; on their way while
  // the rest is worked out, and whatever they are: rows that turn out to be padding are dropped below ----
  uint32_t qf[NT][8][2];
#pragma unroll
  for (int nt = 0; nt < NT; nt++) {
    const int r = row0 + 8 * nt + g, i = (int)((uint32_t)r / (uint32_t)a.group);
    const uint16_t *qp = a.q + b * a.qs.batch + (kvh * a.group + (r - i * a.group)) * a.qs.head + i * a.qs.token;
#pragma unroll
    for (int ks = 0; ks < 8; ks++) {
      const int ch = BITS == 8 ? 16 * (t + 4 * (ks >> 2)) + 4 * (ks & 3) : 32 * t + 4 * ks;
      const uint2 w = r < a.rows ? *(const uint2 *)(qp + ch) : make_uint2(0, 0);
      qf[nt][ks][0] = w.x;
      qf[nt][ks][1] = w.y;
    }
  }
  nq = nq < a.nq ? nq : a.nq;
  if (!win::starts(q0) || nq <= 0 || nq * a.group <= row0) return;   // the whole cluster
  const win::Seq seq{len, a.w.sink, a.w.ring, a.tpf, a.frames};
  const int rows_all = (int)nq * a.group, rows = rows_all - row0 < 8 * NT ? rows_all - row0 : 8 * NT;   // live rows: of all, here
  const int64_t f0 = seq.frame(q0 + (uint32_t)row0 / (uint32_t)a.group);
  const int64_t f1 = seq.frame(q0 + (uint32_t)(row0 + rows - 1) / (uint32_t)a.group);
  win::Keys keys;
  keys.init(seq, f0, f1);
  const uint32_t sink = (uint32_t)a.w.sink, ring = (uint32_t)a.w.ring;
  const int64_t head_row = (int64_t)blockIdx.y * (a.w.sink + a.w.ring);
  const int steps_all = (keys.total + kKeys - 1) / kKeys;
  int j0 = 0, j1 = steps_all;   // (steps_all < 2^28 and splits <= 2^12: the products can pass 32 bits)
  if (a.splits > 1) {
    const uint32_t q = (uint32_t)steps_all / (uint32_t)a.splits, rem = (uint32_t)steps_all - q * (uint32_t)a.splits, k = blockIdx.x;
    j0 = (int)(k * q + (k < rem ? k : rem));
    j1 = j0 + (int)(q + (k < rem ? 1u : 0u));
  }

  // ---- copies of step j's 16 keys into a stage of the warp's ring (one group) ----
  const uint32_t ring0 = tc::smem_u32(dyn) + (uint32_t)(warp * R::kStages * R::kStage);
  constexpr int kPer = R::kRow / 16, kCopies = kKeys * kPer / 32;   // pieces of a row; copies of a lane and tensor
  const uint8_t *kc = a.w.k_codes + head_row * R::kRow + 16 * lane, *vc = a.w.v_codes + head_row * R::kRow + 16 * lane;
  // one step word of Keys or Values per lane (16 keys), or one of each (32 keys)
  const int srow = lane & (kKeys - 1);
  const uint8_t *sc = (kSub == 2 || lane < 16 ? a.w.k_step : a.w.v_step) + (head_row + srow) * win::kSteps;
  const uint8_t *sc2 = a.w.v_step + (head_row + srow) * win::kSteps;
  const uint32_t sdst = (kSub == 2 || lane < 16 ? R::kKS : R::kVS) + 4u * srow;
  const uint32_t kdst = R::k_at(lane / kPer, lane & (kPer - 1));   // k_at(row + 32 / kPer, .) is 512 further on
  // v_at(row + 32 / kPer, .) is 512 further on but for the permutation: one piece bit flips per 4 rows
  const uint32_t vdst = R::v_at(lane / kPer, lane & (kPer - 1));
  auto vdst_of = [&](int i) -> uint32_t { return (vdst ^ (BITS == 8 ? 32u * (i & 3) : 64u * (i & 1))) + 512u * i; };
  auto copy = [&](int j, int stage) {
    if (j < j1) {
      const uint32_t dst = ring0 + (uint32_t)(stage * R::kStage);
      const int v0 = j * kKeys;
      const uint32_t s0 = keys.slot(v0, sink, ring);
      if (v0 + kKeys <= keys.total && keys.slot(v0 + kKeys - 1, sink, ring) == s0 + kKeys - 1) {
        const uint8_t *kp = kc + (uint64_t)s0 * R::kRow, *vp = vc + (uint64_t)s0 * R::kRow;
#pragma unroll
        for (int i = 0; i < kCopies; i++) {
          cp_async16(dst + kdst + 512u * i, kp + 512 * i);
          cp_async16(dst + vdst_of(i), vp + 512 * i);
        }
        cp_async4(dst + sdst, sc + (uint64_t)s0 * win::kSteps);
        if (kSub == 2) cp_async4(dst + R::kVS + 4u * srow, sc2 + (uint64_t)s0 * win::kSteps);
      } else {   // past the sinks, around the ring's end, or the ragged end (masked below): row by row
        auto slot_of = [&](int row) -> int64_t {
          return (int64_t)keys.slot(v0 + row < keys.total ? v0 + row : keys.total - 1, sink, ring) - row;
        };
#pragma unroll
        for (int i = 0; i < kCopies; i++) {
          const int64_t s = slot_of((32 * i + lane) / kPer);
          cp_async16(dst + kdst + 512u * i, kc + s * R::kRow + 512 * i);
          cp_async16(dst + vdst_of(i), vc + s * R::kRow + 512 * i);
        }
        cp_async4(dst + sdst, sc + slot_of(srow) * win::kSteps);
        if (kSub == 2) cp_async4(dst + R::kVS + 4u * srow, sc2 + slot_of(srow) * win::kSteps);
      }
    }
    tc::cp_async_commit();
  };
  copy(j0 + warp, 0);
  copy(j0 + warp + kWarps, 1);

  win::Everyone every;
  every.init(seq, keys, f0, f1);
  // ---- the Queries to fp16; each row's logit scale ----
  float sl2[NT][2];   // of rows 2 t, 2 t + 1 of every 8
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
    if (win::any_beyond_fp16(big)) qwm_dev_error(a.status, QWM_ERR_RANGE);
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
      sl2[nt][e] = a.scale_log2 * __shfl_sync(0xffffffffu, back, 4 * (2 * t + e)) * win::kUnit<BITS>;
  }

  float o[NT][8][4], m[NT][2], mneg[NT][2], l[NT][2];
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
  const int krow = 4 * (g >> 1) + (g & 1);   // the key of MMA row g; row g + 8 is two further on
  // the step byte of the thread's group, of one row or of two
  const uint32_t ksel = BITS == 8 ? (uint32_t)(t >> 1) * 0x1111u : (uint32_t)t * 0x1111u;
  const uint32_t vsel = (uint32_t)(g >> 1) * 0x1111u + 0x4400u;

  // this lane's addresses inside a stage
  const uint32_t koff = R::k_at(krow, t), ksoff = R::kKS + 4u * krow, vsoff = R::kVS + 16u * t;
  const uint32_t voff = BITS == 8 ? R::v_at(4 * t, g) : R::v_at(4 * t, g >> 1) + 8u * (g & 1);

  int stage = 0;
  for (int j = j0 + warp; j < j1; j += kWarps) {
    tc::cp_async_wait<1>();
    __syncwarp();   // the step's copies are there, and the stage before it has been read by every lane
    copy(j + 2 * kWarps, stage == 0 ? 2 : stage - 1);
    const uint32_t st = ring0 + (uint32_t)(stage * R::kStage);
    stage = stage == 2 ? 0 : stage + 1;
    const int v0 = j * kKeys;
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
            win::decode8(x[0][u], ks[0], a.bases, a0, a2);
            win::decode8(x[1][u], ks[1], a.bases, a1, a3);
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
          win::decode4(x[0][u], ks[0], a.bases, p);
          win::decode4(x[1][u], ks[1], a.bases, r);
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
    if (!every.see(v0, v0 + kKeys)) {   // a few steps of a call: what each of the thread's rows sees is worked out here
#pragma unroll
      for (int nt = 0; nt < NT; nt++)
#pragma unroll
        for (int e = 0; e < 2; e++) {
          const int r = 8 * nt + 2 * t + e;
          win::Row mask;
          mask.init(seq, keys, r < rows ? seq.frame(q0 + (uint32_t)(row0 + r) / (uint32_t)a.group) : -1);
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
            const uint32_t a0 = tc::hfma2(win::place<0x00FF00FFu>(ka, a.bases.k1024), vt[0].s, vt[0].n);
            const uint32_t a1 = tc::hfma2(win::place<0x00FF00FFu>(ka >> 8, a.bases.k1024), vt[0].s, vt[0].n);
            const uint32_t a2 = tc::hfma2(win::place<0x00FF00FFu>(kb, a.bases.k1024), vt[1].s, vt[1].n);
            const uint32_t a3 = tc::hfma2(win::place<0x00FF00FFu>(kb >> 8, a.bases.k1024), vt[1].s, vt[1].n);
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
            win::decode4(__byte_perm(qa, qb, 0x5410), vt[e], a.bases, ev[e]);
            win::decode4(__byte_perm(qa, qb, 0x7632), vt[e], a.bases, od[e]);
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
  tc::cp_async_wait<0>();
  __syncthreads();   // the rings are done with: their memory takes the warps' outputs

  // ---- the warps' parts joined in shared memory ----
  float (*osm)[8][D] = (float (*)[8][D])dyn;
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
    if (8 * nt >= rows) break;
    if (nt) __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; i++) {
      if (8 * nt + 2 * t < rows) *(float2 *)&osm[warp][2 * t][16 * g + 2 * i] = make_float2(o[nt][i][0], o[nt][i][2]);
      if (8 * nt + 2 * t + 1 < rows) *(float2 *)&osm[warp][2 * t + 1][16 * g + 2 * i] = make_float2(o[nt][i][1], o[nt][i][3]);
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
      if (CLUSTER) {
        *(float4 *)&part_o[r][ch] = acc;
        if (lane == 0) part_ml[r] = make_float2(M, L);
      } else {
        const float inv = L > 0.f ? win::kUnit<BITS> / L : 0.f, lse = L > 0.f ? M + log2f(L) : -INFINITY;
        acc = make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
        if (a.splits == 1) {
          finish4(a, b, kvh, row0 + r, ch, acc, lse);
          __syncwarp();   // merging lanes have read the earlier log-sum-exp
          if (lane == 0) finish_lse(a, b, kvh, row0 + r, lse);
        } else {
          const int64_t pr = ((int64_t)blockIdx.y * a.splits + blockIdx.x) * a.rows + row0 + r;
          *(float4 *)(a.part + pr * D + ch) = acc;
          if (lane == 0) a.part_lse[pr] = lse;
        }
      }
    }
  }
  if (CLUSTER) {   // CTA k of the cluster joins the parts of rows k, k + splits, ...
    tc::cluster_sync();
    for (int r = (int)blockIdx.x + a.splits * warp; r < rows; r += a.splits * kWarps) {
      const uint32_t ml = tc::smem_u32(&part_ml[r]), po = tc::smem_u32(&part_o[r][4 * lane]);
      float2 p[8];
      float M = -INFINITY;
#pragma unroll
      for (int k = 0; k < 8; k++)
        if (k < a.splits) {
          p[k] = ld_cluster2(tc::mapa(ml, (uint32_t)k));
          M = fmaxf(M, p[k].x);
        }
      float L = 0.f;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int k = 0; k < 8; k++)
        if (k < a.splits) {
          const float wt = p[k].x == -INFINITY ? 0.f : tc::ex2_approx(p[k].x - M);
          const float4 x = ld_cluster4(tc::mapa(po, (uint32_t)k));
          L = fmaf(p[k].y, wt, L);
          acc.x = fmaf(x.x, wt, acc.x);
          acc.y = fmaf(x.y, wt, acc.y);
          acc.z = fmaf(x.z, wt, acc.z);
          acc.w = fmaf(x.w, wt, acc.w);
        }
      const float inv = L > 0.f ? win::kUnit<BITS> / L : 0.f, lse = L > 0.f ? M + log2f(L) : -INFINITY;
      finish4(a, b, kvh, row0 + r, 4 * lane, make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv), lse);
      __syncwarp();
      if (lane == 0) finish_lse(a, b, kvh, row0 + r, lse);
    }
    tc::cluster_sync();   // no CTA leaves while its part is read
  }
}

// Parts of a row joined: the weighted mean of the parts' outputs, each weighted by its share of the
// exponential sum.  One warp per row.
__global__ void __launch_bounds__(256) window_combine_kernel(const __grid_constant__ WindowAttend a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");   // launched while the parts are computed: wait for them
  const int lane = threadIdx.x & 31;
  const int64_t item = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int64_t heads = (int64_t)a.w.batch * a.w.kv_heads;
  if (item >= heads * a.rows) return;
  const int64_t y = win::quotient(item, a.rows), r = item - y * a.rows, b = win::quotient(y, a.w.kv_heads);
  const int kvh = (int)(y - b * a.w.kv_heads);
  if (!win::starts(a.q_start[b]) || (a.q_count && win::quotient(r, a.group) >= a.q_count[b])) return;
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

template <int BITS, int NT, bool CLUSTER>
cudaError_t decode_launch(const WindowAttend &a, cudaStream_t st) {
  auto kernel = window_decode_kernel<BITS, NT, CLUSTER>;
  static std::atomic<uint64_t> allowed{0};
  const cudaError_t e = allow_shared(kernel, Ring<BITS>::kBytes, allowed);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)a.splits, (unsigned)(a.w.batch * a.w.kv_heads), (unsigned)((a.rows + 8 * NT - 1) / (8 * NT)));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = Ring<BITS>::kBytes;
  cfg.stream = st;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = (unsigned)a.splits;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = CLUSTER ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

template <int BITS>
cudaError_t decode_bits(const WindowAttend &a, cudaStream_t st) {
  if (a.rows <= 8) return a.cluster ? decode_launch<BITS, 1, true>(a, st) : decode_launch<BITS, 1, false>(a, st);
  return a.cluster ? decode_launch<BITS, 2, true>(a, st) : decode_launch<BITS, 2, false>(a, st);
}

}  // namespace

cudaError_t launch_window_decode(const WindowAttend &a, cudaStream_t st) {
  return a.w.bits == 8 ? decode_bits<8>(a, st) : decode_bits<4>(a, st);
}

// Launched as a dependent of the parts' kernel, so that its start-up overlaps their work.
cudaError_t launch_window_combine(const WindowAttend &a, cudaStream_t st) {
  const int64_t items = (int64_t)a.w.batch * a.w.kv_heads * a.rows;
  if ((items + 7) / 8 > INT32_MAX) return cudaErrorInvalidValue;   // (its workspace would be terabytes)
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((items + 7) / 8));
  cfg.blockDim = dim3(256);
  cfg.stream = st;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, window_combine_kernel, a);
}
