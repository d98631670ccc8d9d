// Attention over the window cache for many Query rows, on the tensor cores (tcgen05 + TMEM).
//
//   l_ij = scale q_i . k_hat_j over the keys row i sees, o_i = softmax(l_i) V_hat, with k_hat and v_hat
// decoded from the 8- or 4-bit cache inside the kernel.  A cached value is exact in fp16 and so is a
// bf16 Query in the fp16 range, so the logits carry only fp32 rounding; the weights enter the second
// product in fp16.
//
// Work split: a pair of CTAs (a cluster of two, cta_group::2 MMAs) takes one Key head x 512 Query rows
// (row r = Query r / group, head r % group) and one part of the keys those rows see between them; CTA c
// holds rows 256 x + 128 c .. + 127 of its two tiles x = 0, 1.  The B operand of an M = 256 MMA is
// split by N, so CTA c decodes only keys 64 c .. 64 c + 63 of a 128-key tile for Q K^T and only channels
// 64 c .. 64 c + 63 for P V: half of every tile.  Keys are numbered along what the rows see (the sinks,
// then the window), so a tile has no gaps whatever the ring's offset; each producer thread looks its
// rows' slots up.
// Warp roles of each CTA (17 warps):
//   warps 0-3, 4-7  softmax of Query tile 0 / 1: thread = Query row = TMEM lane;
//   warp 8          allocates TMEM; in the even CTA one thread issues every MMA of the pair;
//   warps 9-12      Key producers, warps 13-16 Value producers: codes two tiles ahead in registers,
//                   decoded (one permute and one fp16 FMA per pair at 8 bits) into swizzled stages.
// TMEM (512 columns): S0 | S1 | O0 | O1, P_x over S_x.  MMA order per tile: S0(j), PV1(j-1), S1(j),
// PV0(j); the commit after S_x(j) also certifies PV_x(j-1), so softmax x may then rescale O_x.
// Every wait is bounded (about one second); on expiry QWM_ERR_DEVICE_TIMEOUT is recorded, every role
// stops, outstanding MMAs are drained and TMEM is freed.
#include "window.cuh"

namespace {

constexpr int D = win::D;
constexpr int BM = 128, BN = 128, NQT = 2;
constexpr int kSoftmaxWarps = 8, kMmaWarp = 8, kKWarp0 = 9, kVWarp0 = 13, kProdWarps = 4;
constexpr int kThreads = 32 * (kSoftmaxWarps + 1 + 2 * kProdWarps);
constexpr uint64_t kWaitNs = 1000000000ull;
constexpr float kRescaleThreshold = 8.0f;  // log2 units the maximum may lag behind
constexpr int kStages = 4;
constexpr int kPairRows = 2 * NQT * BM;

// shared-memory map of one CTA (bytes from a 1024-aligned base)
constexpr int kBlk = BM * 128;             // a [128 rows][64 fp16] swizzled block
constexpr int kBlkH = 64 * 128;            // a [64 rows][64 fp16] swizzled block
constexpr int OFF_Q = 0;                   // 2 Query tiles x 2 blocks (channels 0-63, 64-127)
constexpr int OFF_K = OFF_Q + NQT * 2 * kBlk;          // stages x 2 blocks [64 keys][64 ch]
constexpr int OFF_V = OFF_K + kStages * 2 * kBlkH;     // stages x [128 keys][64 ch] (MN-major B)
constexpr int kSmemBytes = OFF_V + kStages * kBlk;
constexpr int kSmemAlloc = kSmemBytes + 1024;

struct Bars {
  uint64_t k_full[kStages], k_empty[kStages], v_full[kStages], v_empty[kStages];
  uint64_t s_full[2], p_ready[2], o_done, drain;
};

__device__ __forceinline__ void fail(int *abort_flag, int32_t *status) {
  *(volatile int *)abort_flag = 1;
  qwm_dev_error(status, QWM_ERR_DEVICE_TIMEOUT);
}
__device__ __forceinline__ uint64_t pk64(uint32_t lo, uint32_t hi) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "r"(lo), "r"(hi));
  return d;
}
__device__ __forceinline__ uint64_t pk64(float lo, float hi) { return pk64(__float_as_uint(lo), __float_as_uint(hi)); }
// The lowest n bits set (n clamped to 0..32).
__device__ __forceinline__ uint32_t low_bits(int n) { return n <= 0 ? 0u : (n >= 32 ? 0xFFFFFFFFu : (1u << n) - 1u); }

// Where one Query row's result goes (splits == 1: out and lse, else the part's workspace).
struct RowOut {
  float *f32 = nullptr;
  uint16_t *bf16 = nullptr;
  float *lse = nullptr;
  int merge = 0;
  __device__ __forceinline__ void init(const WindowAttend &a, int64_t y, int64_t b, int kvh, int split, int64_t r) {
    if (a.splits > 1) {
      const int64_t pr = (y * a.splits + split) * a.rows + r;
      f32 = a.part + pr * D;
      lse = a.part_lse + pr;
      return;
    }
    const int64_t i = r / a.group;
    const int h = kvh * a.group + (int)(r - i * a.group);
    const int64_t at = b * a.os.batch + h * a.os.head + i * a.os.token;
    if (a.out_f32) f32 = (float *)a.out + at;
    else bf16 = (uint16_t *)a.out + at;
    if (a.lse) lse = a.lse + (b * a.H + h) * a.nq + i;
    merge = a.merge;
  }
  // 32 channels from channel c: (keep) out + o inv
  __device__ __forceinline__ void store32(int c, const uint32_t (&o)[32], float inv, float keep) const {
    if (bf16) {
#pragma unroll
      for (int v = 0; v < 4; v++) {
        uint32_t w[4];
#pragma unroll
        for (int u = 0; u < 4; u++)
          w[u] = tc::pack_bf16x2(__uint_as_float(o[8 * v + 2 * u]) * inv, __uint_as_float(o[8 * v + 2 * u + 1]) * inv);
        *(uint4 *)(bf16 + c + 8 * v) = make_uint4(w[0], w[1], w[2], w[3]);
      }
      return;
    }
#pragma unroll
    for (int v = 0; v < 8; v++) {
      float4 *dst = (float4 *)(f32 + c + 4 * v);
      float4 x = make_float4(__uint_as_float(o[4 * v]) * inv, __uint_as_float(o[4 * v + 1]) * inv,
                             __uint_as_float(o[4 * v + 2]) * inv, __uint_as_float(o[4 * v + 3]) * inv);
      if (keep > 0.f) {
        const float4 p = *dst;
        x = make_float4(fmaf(keep, p.x, x.x), fmaf(keep, p.y, x.y), fmaf(keep, p.z, x.z), fmaf(keep, p.w, x.w));
      }
      *dst = x;
    }
  }
};

// A producer thread's share of a 128-key tile: four pieces of 16 channels.
template <int BITS>
struct Pieces {
  uint32_t c[4][BITS / 2];
  uint32_t step;   // one byte per piece
};

// Producer thread of a pair CTA (rank cr): Keys: key rows 64 cr + 16 w + 4 i + lane / 8 (i = 0..3),
// channels 16 (lane % 8); Values: key rows 32 w + 8 i + lane / 4, channels 64 cr + 16 (lane % 4).
template <int BITS, bool VAL>
__device__ __forceinline__ void producer(const WindowAttend &a, unsigned char *sm, Bars &bars, int *abort_flag,
                                         const win::Keys &keys, int64_t y, int j0, int J, int cr, int pr) {
  volatile int *abort_v = abort_flag;
  const int lane = pr & 31, w = pr >> 5;
  const int row0 = VAL ? 32 * w + (lane >> 2) : 16 * w + (lane >> 3);   // row in the block of piece 0
  constexpr int kRowStep = VAL ? 8 : 4;
  const int piece = VAL ? (lane & 3) : (lane & 7);
  const int ch = VAL ? 64 * cr + 16 * piece : 16 * piece;
  const int key0 = VAL ? row0 : 64 * cr + row0;
  const int64_t head_row = y * (a.w.sink + a.w.ring);
  const uint8_t *codes = (VAL ? a.w.v_codes : a.w.k_codes) + head_row * (D * BITS / 8) + ch * BITS / 8;
  const uint8_t *steps = (VAL ? a.w.v_step : a.w.k_step) + head_row * win::kSteps + ch / win::kGroup;
  const uint32_t sink = (uint32_t)a.w.sink, ring = (uint32_t)a.w.ring;
  uint64_t *empty = VAL ? bars.v_empty : bars.k_empty;
  const uint32_t full_base = tc::mapa(tc::smem_u32(VAL ? &bars.v_full[0] : &bars.k_full[0]), 0);
  const uint32_t block0 = tc::smem_u32(sm + (VAL ? OFF_V : OFF_K)) + (VAL ? 0u : (uint32_t)(piece >> 2) * kBlkH);
  constexpr uint32_t kStage = VAL ? (uint32_t)kBlk : 2u * kBlkH;
  const uint32_t chunk = 2u * (uint32_t)(piece & 3);
  // Keys: the upper four lanes of a row store their second chunk first, so that a quarter warp's eight
  // 16-byte stores fall into eight different bank groups
  const uint32_t flip = (!VAL && (piece >> 2)) ? 1u : 0u;

  auto load = [&](int j, Pieces<BITS> &p) {
    p.step = 0u;
#pragma unroll
    for (int i = 0; i < 4; i++) {
      const int v = (j0 + j) * BN + key0 + kRowStep * i;
      if (v < keys.total) {
        const uint64_t s = keys.slot(v, sink, ring);
        if (BITS == 8) {
          const uint4 x = __ldg((const uint4 *)(codes + s * (D * BITS / 8)));
          p.c[i][0] = x.x; p.c[i][1] = x.y; p.c[i][2 % (BITS / 2)] = x.z; p.c[i][3 % (BITS / 2)] = x.w;
        } else {
          const uint2 x = __ldg((const uint2 *)(codes + s * (D * BITS / 8)));
          p.c[i][0] = x.x; p.c[i][1] = x.y;
        }
        p.step |= (uint32_t)__ldg(steps + s * win::kSteps) << (8 * i);
      } else {   // past the last key: a zero row
#pragma unroll
        for (int u = 0; u < BITS / 2; u++) p.c[i][u] = 0u;
      }
    }
  };
  auto store = [&](int stage, const Pieces<BITS> &p) {
    const uint32_t block = block0 + (uint32_t)stage * kStage;
#pragma unroll
    for (int i = 0; i < 4; i++) {
      uint32_t s2, n2, d[8];
      win::step_consts<BITS>((p.step >> (8 * i)) & 0xFFu, s2, n2);
      if (BITS == 8) {
#pragma unroll
        for (int u = 0; u < 4; u++) win::decode8(p.c[i][u % (BITS / 2)], s2, n2, d[2 * u], d[2 * u + 1]);
      } else {
        uint32_t q[4];
        win::decode4(p.c[i][0], s2, n2, q);
        d[0] = q[0]; d[1] = q[1]; d[2] = q[2]; d[3] = q[3];
        win::decode4(p.c[i][1], s2, n2, q);
        d[4] = q[0]; d[5] = q[1]; d[6] = q[2]; d[7] = q[3];
      }
      const uint32_t row = (uint32_t)(row0 + kRowStep * i), rb = block + row * 128u, rx = row & 7u;
      const uint4 lo = make_uint4(d[0], d[1], d[2], d[3]), hi = make_uint4(d[4], d[5], d[6], d[7]);
      tc::sts128(rb + (((chunk + flip) ^ rx) << 4), flip ? hi : lo);
      tc::sts128(rb + (((chunk + 1u - flip) ^ rx) << 4), flip ? lo : hi);
    }
  };

  Pieces<BITS> A, B;
  load(0, A);
  if (J > 1) load(1, B);
  auto step = [&](int j, Pieces<BITS> &cur) -> bool {
    const int s = j % kStages;
    if (j >= kStages && !tc::mbar_wait(&empty[s], (j / kStages - 1) & 1, kWaitNs)) fail(abort_flag, a.status);
    if (__any_sync(0xffffffffu, *abort_v != 0)) return false;  // warp-uniform exit
    store(s, cur);
    tc::fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) tc::mbar_arrive_remote(full_base + 8u * (uint32_t)s);
    if (j + 2 < J) load(j + 2, cur);
    return true;
  };
  for (int j = 0; j < J; j += 2) {
    if (!step(j, A)) break;
    if (j + 1 < J && !step(j + 1, B)) break;
  }
}

template <int BITS>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    window_attend_kernel(const __grid_constant__ WindowAttend a) {
  extern __shared__ __align__(16) unsigned char smem_raw[];
  unsigned char *sm = smem_raw + ((1024u - (tc::smem_u32(smem_raw) & 1023u)) & 1023u);
  __shared__ Bars bars;
  __shared__ uint32_t tmem_base_sh;
  __shared__ int abort_flag;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int64_t y = blockIdx.y, b = y / a.w.kv_heads;
  const int kvh = (int)(y - b * a.w.kv_heads), split = (int)blockIdx.z;
  const int cr = (int)tc::cluster_ctarank();
  volatile int *abort_v = &abort_flag;

  const int64_t q0 = a.q_start[b];
  int64_t nq = a.q_count ? (int64_t)a.q_count[b] : a.nq;
  nq = nq < a.nq ? nq : a.nq;
  const int64_t pair0 = (int64_t)(blockIdx.x >> 1) * kPairRows;
  const int64_t rows = nq * a.group;              // live rows of this Key head
  if (q0 < 0 || pair0 >= rows) return;            // the same in both CTAs
  const win::Seq seq{a.length[b], a.w.sink, a.w.ring, a.tpf, a.frames};
  auto frame_of = [&](int64_t r) { return seq.frame(q0 + r / a.group); };
  const int64_t pair1 = pair0 + kPairRows < rows ? pair0 + kPairRows : rows;
  win::Keys keys;
  keys.init(seq, frame_of(pair0), frame_of(pair1 - 1));
  const int tiles = (keys.total + BN - 1) / BN;
  const int j0 = (int)((int64_t)tiles * split / a.splits);
  const int J = (int)((int64_t)tiles * (split + 1) / a.splits) - j0;
  const int64_t row_base = pair0 + (int64_t)cr * BM;   // this CTA's row 0 of tile 0
  if (J == 0) {   // these rows see no key (in this part)
    for (int e = tid; e < NQT * BM; e += kThreads) {
      const int64_t r = row_base + (int64_t)(e / BM) * 2 * BM + e % BM;
      if (r >= rows) continue;
      RowOut out;
      out.init(a, y, b, kvh, split, r);
      if (out.merge) continue;
      const uint32_t zero[32] = {};
      for (int c = 0; c < D; c += 32) out.store32(c, zero, 0.f, 0.f);
      if (out.lse) *out.lse = -INFINITY;
    }
    return;
  }
  const bool skip1 = pair0 + 2 * BM >= rows;   // the second 256-row tile is empty

  // ---- this CTA's two Query tiles -> shared memory as fp16 ----
  for (int e = tid; e < NQT * BM * (D / 8); e += kThreads) {
    const int row = e / (D / 8), ci = e % (D / 8);
    const int x = row / BM, rr = row % BM;
    const int64_t r = row_base + (int64_t)x * 2 * BM + rr;
    uint4 v = make_uint4(0, 0, 0, 0);
    if (r < rows) {
      const int64_t i = r / a.group;
      v = *(const uint4 *)(a.q + b * a.qs.batch + (kvh * a.group + (r - i * a.group)) * a.qs.head + i * a.qs.token +
                           8 * ci);
    }
    const uint32_t bw[4] = {v.x, v.y, v.z, v.w};
    uint32_t hw[4];
    bool bad = false;
#pragma unroll
    for (int u = 0; u < 4; u++) {
      hw[u] = tc::pack_f16x2(__uint_as_float(bw[u] << 16), __uint_as_float(bw[u] & 0xFFFF0000u));
      bad |= (hw[u] & 0x7C00u) == 0x7C00u || (hw[u] & 0x7C000000u) == 0x7C000000u;
    }
    if (bad) qwm_dev_error(a.status, QWM_ERR_RANGE);
    *(uint4 *)(sm + OFF_Q + (x * 2 + ci / 8) * kBlk + tc::sw128_offset(rr, 8 * (ci % 8))) =
        make_uint4(hw[0], hw[1], hw[2], hw[3]);
  }
  if (tid == 0) {
    for (int i = 0; i < kStages; i++) {
      tc::mbar_init(&bars.k_full[i], 2 * kProdWarps);  // both CTAs' producer warps (even CTA's copy used)
      tc::mbar_init(&bars.v_full[i], 2 * kProdWarps);
      tc::mbar_init(&bars.k_empty[i], 1);
      tc::mbar_init(&bars.v_empty[i], 1);
    }
    for (int i = 0; i < 2; i++) {
      tc::mbar_init(&bars.s_full[i], 1);
      tc::mbar_init(&bars.p_ready[i], 8);              // both CTAs' 4 softmax warps of tile i
    }
    tc::mbar_init(&bars.o_done, 1);
    tc::mbar_init(&bars.drain, 1);
    abort_flag = 0;
    tc::fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    tc::tmem_alloc2(&tmem_base_sh, 512);
    tc::tmem_relinquish2();
  }
  tc::fence_proxy_async_smem();
  tc::fence_before_sync();
  __syncthreads();
  tc::cluster_sync();  // both CTAs' barriers exist before the first arrival from the peer
  tc::fence_after_sync();
  const uint32_t tmem = tmem_base_sh;

  if (warp < kSoftmaxWarps) {
    // ======================= softmax (Query tile x, row = TMEM lane) =======================
    const int x = warp / 4, sub = warp % 4;
    const int Jx = (x == 1 && skip1) ? 0 : J;
    const uint32_t lane_addr = (uint32_t)(32 * sub) << 16;
    const uint32_t tS = tmem + lane_addr + 128u * x, tO = tmem + lane_addr + 256u + 128u * x;
    const uint32_t p_ready0 = tc::mapa(tc::smem_u32(&bars.p_ready[x]), 0);
    const float sl2 = a.scale_log2;
    const uint64_t sc2 = pk64(sl2, sl2);
    const int64_t w0 = row_base + (int64_t)x * 2 * BM + 32 * sub;   // this warp's first row
    const int64_t r = w0 + lane;
    win::Row mine{0, 0, 0};
    win::Everyone every{INT32_MAX, 0, 0};   // a warp without a row masks nothing (its logits are 0)
    if (w0 < rows) {
      mine.init(seq, keys, r < rows ? frame_of(r) : -1);
      every.init(seq, keys, frame_of(w0), frame_of(w0 + 31 < rows ? w0 + 31 : rows - 1));
    }
    float m_used = -INFINITY;
    uint64_t acc0 = 0ull, acc1 = 0ull;
    bool ok = true;
    for (int j = 0; j < Jx; j++) {
      const int v0 = (j0 + j) * BN;
      const bool full = every.see(v0, v0 + BN);
      if (!tc::mbar_wait(&bars.s_full[x], j & 1, kWaitNs)) fail(&abort_flag, a.status);
      if (*abort_v) { ok = false; break; }
      tc::fence_after_sync();
      // one pass over the tile, 32 columns at a time: their maximum, then their exponentials with the
      // running maximum m_used; when it grows by more than 2^8 (rare after the first columns) the sum,
      // O and the P columns already stored for this tile are first rescaled
      uint32_t s[32];
#pragma unroll 1
      for (int cq = 0; cq < 4; cq++) {
        tc::tmem_ld16(tS + 32u * cq, s);
        tc::tmem_ld16(tS + 32u * cq + 16u, s + 16);
        tc::tmem_ld_wait();
        if (!full) {
          const int v = v0 + 32 * cq;
          const uint32_t seen = low_bits(mine.c0 - v) | (low_bits(mine.c2 - v) & ~low_bits(mine.c1 - v));
#pragma unroll
          for (int i = 0; i < 32; i++)
            if (!((seen >> i) & 1u)) s[i] = 0xFF800000u;  // -inf: weight exactly 0
        }
        float mx0 = -INFINITY, mx1 = -INFINITY;
#pragma unroll
        for (int i = 0; i < 32; i += 4) {
          mx0 = tc::max3(mx0, __uint_as_float(s[i]), __uint_as_float(s[i + 1]));
          mx1 = tc::max3(mx1, __uint_as_float(s[i + 2]), __uint_as_float(s[i + 3]));
        }
        const float m_new = fmaxf(m_used, fmaxf(mx0, mx1) * sl2);
        if (__any_sync(0xffffffffu, m_new > m_used + kRescaleThreshold)) {
          const float alpha = m_new == -INFINITY ? 1.f : tc::ex2_approx(m_used - m_new);
          const uint64_t a2 = pk64(alpha, alpha);
          acc0 = tc::fma2(acc0, a2, 0ull);
          acc1 = tc::fma2(acc1, a2, 0ull);
          if (j > 0) {  // O of the earlier tiles (complete: S_x(j) finished after PV_x(j-1))
#pragma unroll 1
            for (int c = 0; c < D; c += 32) {
              uint32_t o[32];
              tc::tmem_ld32(tO + c, o);
              tc::tmem_ld_wait();
#pragma unroll
              for (int i = 0; i < 32; i++) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
              tc::tmem_st32(tO + c, o);
            }
          }
          tc::tmem_st_wait();
#pragma unroll 1
          for (int pc = 0; pc < cq; pc++) {  // P columns of this tile already written
            uint32_t pw[16];
            tc::tmem_ld16(tS + 16u * pc, pw);
            tc::tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 16; i++) {
              const float2 v = __half22float2(*(const __half2 *)&pw[i]);
              pw[i] = tc::pack_f16x2(v.x * alpha, v.y * alpha);
            }
            tc::tmem_st16(tS + 16u * pc, pw);
          }
          m_used = m_new;
        }
        const float mneg = m_used == -INFINITY ? 0.f : -m_used;  // a row that has seen no key yet
        const uint64_t nm2 = pk64(mneg, mneg);
        uint32_t pw[16];
#pragma unroll
        for (int i = 0; i < 16; i++) {  // packed fp32 pairs: S * scale - m, then 2^x
          const uint64_t x2 = tc::fma2(pk64(s[2 * i], s[2 * i + 1]), sc2, nm2);
          const float e0 = tc::ex2_approx(tc::f2lo(x2)), e1 = tc::ex2_approx(tc::f2hi(x2));
          const uint64_t e2 = pk64(e0, e1);
          if (i & 1) acc1 = tc::add2(acc1, e2);
          else acc0 = tc::add2(acc0, e2);
          pw[i] = tc::pack_f16x2(e0, e1);
        }
        tc::tmem_st16(tS + 16u * cq, pw);  // P (fp16 pairs) overlays logits already read
      }
      tc::tmem_st_wait();
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive_remote(p_ready0);
    }
    if (ok && Jx > 0 && !tc::mbar_wait(&bars.o_done, 0, kWaitNs)) fail(&abort_flag, a.status);
    if (ok && Jx > 0 && !*abort_v) {
      tc::fence_after_sync();
      const uint64_t lsum = tc::add2(acc0, acc1);
      const float l = tc::f2lo(lsum) + tc::f2hi(lsum);
      float inv = l > 0.f ? 1.f / l : 0.f, keep = 0.f;
      float L = l > 0.f ? m_used + log2f(l) : -INFINITY;
      bool write = r < rows;
      RowOut out;
      if (write) {
        out.init(a, y, b, kvh, split, r);
        if (out.merge) {  // out = w_prev out + w_this O / l, the weights the parts' shares of the sum
          const float Lp = *out.lse, Lm = fmaxf(Lp, L);
          if (Lm == -INFINITY) {
            write = false;
          } else {
            const float wp = exp2f(Lp - Lm), wt = exp2f(L - Lm), den = wp + wt;
            keep = wp / den;
            inv *= wt / den;
            L = Lm + log2f(den);
          }
        }
        if (write && out.lse) *out.lse = L;
      }
      uint32_t o[32];
#pragma unroll 1
      for (int c = 0; c < D; c += 32) {
        tc::tmem_ld32(tO + c, o);
        tc::tmem_ld_wait();
        if (write) out.store32(c, o, inv, keep);
      }
    }
  } else if (warp == kMmaWarp) {
    // ======================= MMA issue: one thread of the even CTA, for the pair =======================
    if (cr == 0 && lane == 0) {
      const uint32_t idesc = tc::idesc_f16_f32(2 * BM, BN);
      const uint32_t idesc_pv = tc::idesc_f16_f32_bmn(2 * BM, D);
      const uint32_t tS[2] = {tmem, tmem + 128u}, tO[2] = {tmem + 256u, tmem + 384u};
      const uint32_t sQ = tc::smem_u32(sm + OFF_Q), sK = tc::smem_u32(sm + OFF_K), sV = tc::smem_u32(sm + OFF_V);
      constexpr uint16_t kBoth = 3;
      int prev_stage = 0;
      bool ok = true;
      auto qk = [&](int x, int s) {
#pragma unroll
        for (int kk = 0; kk < D / 16; kk++) {
          const uint32_t qo = (uint32_t)((kk / 4) * kBlk + 32 * (kk % 4));
          const uint32_t ko = (uint32_t)((kk / 4) * kBlkH + 32 * (kk % 4));
          tc::mma2_ss(tS[x], tc::desc_sw128(sQ + (x * 2) * kBlk + qo), tc::desc_sw128(sK + s * 2 * kBlkH + ko), idesc,
                      kk > 0);
        }
      };
      auto pv = [&](int x, int s, bool first) {
#pragma unroll
        for (int kk = 0; kk < BN / 16; kk++)
          tc::mma2_ts(tO[x], tS[x] + 8u * kk, tc::desc_sw128_mn(sV + s * kBlk + 2048u * kk, kBlk, 1024), idesc_pv,
                      (!first || kk > 0));
      };
      for (int j = 0; ok && j < J; j++) {
        const int s = j % kStages;
        const uint32_t ph = (uint32_t)(j / kStages) & 1u;
        ok = tc::mbar_wait_cluster(&bars.k_full[s], ph, kWaitNs) && !*abort_v;
        if (!ok) break;
        tc::fence_after_sync();
        qk(0, s);
        tc::mma2_commit(&bars.s_full[0], kBoth);
        if (j > 0 && !skip1) {
          ok = tc::mbar_wait_cluster(&bars.p_ready[1], (j - 1) & 1, kWaitNs) && !*abort_v;
          if (!ok) break;
          tc::fence_after_sync();
          pv(1, prev_stage, j - 1 == 0);
          tc::mma2_commit(&bars.v_empty[prev_stage], kBoth);
        }
        if (!skip1) {
          qk(1, s);
          tc::mma2_commit(&bars.s_full[1], kBoth);
        }
        tc::mma2_commit(&bars.k_empty[s], kBoth);
        ok = tc::mbar_wait_cluster(&bars.v_full[s], ph, kWaitNs) &&
             tc::mbar_wait_cluster(&bars.p_ready[0], j & 1, kWaitNs) && !*abort_v;
        if (!ok) break;
        tc::fence_after_sync();
        pv(0, s, j == 0);
        if (skip1) tc::mma2_commit(&bars.v_empty[s], kBoth);  // no second tile reads this stage
        prev_stage = s;
      }
      if (ok) {
        if (!skip1) {
          ok = tc::mbar_wait_cluster(&bars.p_ready[1], (J - 1) & 1, kWaitNs) && !*abort_v;
          if (ok) {
            tc::fence_after_sync();
            pv(1, prev_stage, J - 1 == 0);
          }
        }
        if (ok) tc::mma2_commit(&bars.o_done, kBoth);
      }
      if (!ok) fail(&abort_flag, a.status);
      tc::mma2_commit(&bars.drain, 1);  // every MMA issued above completes before TMEM is released
      if (!tc::mbar_wait(&bars.drain, 0, kWaitNs)) qwm_dev_error(a.status, QWM_ERR_DEVICE_TIMEOUT);
    }
  } else if (warp < kVWarp0) {
    producer<BITS, false>(a, sm, bars, &abort_flag, keys, y, j0, J, cr, tid - 32 * kKWarp0);
  } else {
    producer<BITS, true>(a, sm, bars, &abort_flag, keys, y, j0, J, cr, tid - 32 * kVWarp0);
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::cluster_sync();  // the peer has finished with this CTA's barriers, shared and tensor memory
  if (warp == kMmaWarp) {
    tc::fence_after_sync();
    tc::tmem_dealloc2(tmem, 512);
  }
}

template <int BITS>
cudaError_t launch_bits(const WindowAttend &a, cudaStream_t st) {
  cudaError_t e = cudaFuncSetAttribute(window_attend_kernel<BITS>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       kSmemAlloc);
  if (e != cudaSuccess) return e;
  const dim3 grid((unsigned)(2 * ((a.rows + kPairRows - 1) / kPairRows)), (unsigned)(a.w.batch * a.w.kv_heads),
                  (unsigned)a.splits);
  window_attend_kernel<BITS><<<grid, kThreads, kSmemAlloc, st>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_window_tiles(const WindowAttend &a, cudaStream_t st) {
  return a.w.bits == 8 ? launch_bits<8>(a, st) : launch_bits<4>(a, st);
}

// Few rows run on warp tiles, which read the cache once per 16 rows at most; more run on tensor-memory
// tiles.  Keys are split until the parts fill the SMs, while a part keeps a few steps of work.
WindowPlan window_plan(int64_t batch, int64_t kv_heads, int64_t rows, int64_t keys, int num_sms) {
  WindowPlan p;
  p.tiles = rows > 16;
  const int64_t items = batch * kv_heads * (p.tiles ? 2 * ((rows + kPairRows - 1) / kPairRows) : 1);
  const int64_t want = (p.tiles ? 1 : (rows <= 8 ? 2 : 1)) * (int64_t)num_sms / items;
  const int64_t most = (keys + 255) / 256;
  int64_t s = want < most ? want : most;
  p.splits = (int)(s < 1 ? 1 : (s > 64 ? 64 : s));
  return p;
}
