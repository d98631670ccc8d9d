// Attention over the window cache for many Query rows, on the tensor cores (tcgen05 + TMEM).
//
//   l_ij = scale q_i . k_hat_j over the keys row i sees, o_i = softmax(l_i) V_hat, with k_hat and v_hat
// decoded from the 8- or 4-bit cache inside the kernel.  A cached value is exact in fp16 and so is a
// bf16 Query, or next to it (see win::row_power), so the logits carry only fp32 rounding; the weights
// enter the second product in fp16, the largest as 2^7 (win::kTopWeight).
//
// Work split: a pair of CTAs (a cluster of two, cta_group::2 MMAs) takes one Key head x 512 Query rows
// (row r = Query r / group, head r % group) and one part of the keys those rows see between them; CTA c
// holds rows 256 x + 128 c .. + 127 of its two tiles x = 0, 1.  The B operand of an M = 256 MMA is
// split by N, so CTA c decodes only keys 32 c .. 32 c + 31 of every 64 for Q K^T and only channels
// 64 c .. 64 c + 63 for P V: half of everything.  Keys are numbered along what the rows see (the sinks,
// then the window), so a tile has no gaps whatever the ring's offset; each producer thread looks its
// rows' slots up.
// Warp roles of each CTA (13 warps, so that a thread may hold 128 registers):
//   warps 0-3, 4-7  softmax of Query tile 0 / 1: thread = Query row = TMEM lane, 64 logits at a time;
//   warps 8-11      producers: codes two stages ahead in registers, decoded (one permute and one fp16
//                   FMA per pair at 8 bits) into swizzled stages;
//   warp 12         allocates TMEM; in the even CTA it issues every MMA of the pair, in the odd one it
//                   passes on to the even one that its producers have filled a stage.
// An item whose rows all fit the first Query tile (a Key head's last one, or any call of up to 256 rows)
// gives both tiles those rows and every other 64 keys each, joined at the end: 1,050 -> 700 cycles per 64 keys.
// TMEM (512 columns): S_x as two buffers of 64 keys, P_x over them, O_x.  Keys arrive in stages of 128
// and are multiplied 64 at a time: as soon as PV_x(t) has been issued its buffer takes S_x(t + 2), so
// the softmax warps find the next step's logits ready and the tensor pipe always holds work: per step
// and tile 8 MMAs of 256 x 64 x 16 (43 cycles each, bound by reading Q from shared memory) and 4 of
// 256 x 128 x 16 (64 cycles).  MMAs execute in issue order, so a buffer is written after the PV that
// read it.
// Measured (device time of calls replayed from a graph; 2 x 2 x 128 operations per row and visible key): 40 heads x
// 4,680 rows over 39,000 keys at 8 bits in 2.26 ms = 1,653 TFLOP/s, 3,600 rows over 43,200 keys at 4 bits in
// 1.92 ms = 1,662 (called one after another 2.47 and 2.02 ms = 1,510 and 1,580); the tensor pipe is active in
// 81% of all cycles, and in 1,200 of about 1,260 per step of the loop.  Around the loop an item spends about
// 15,000 cycles (first loads 7,000, first logits 2,500, output 4,000), which a prompt under a window of 1,024 keys
// feels: 2 x 2,111 tokens x 32 heads in 96 us.  With few rows the tiles' padding costs as much as rows: 33 to 256
// rows of 40 heads over 39,000 keys take 206 to 221 us at 8 bits and 201 to 211 at 4.
// Every wait is bounded (about one second); on expiry QWM_ERR_DEVICE_TIMEOUT is recorded, every role
// stops, outstanding MMAs are drained and TMEM is freed.
#include "window.cuh"

namespace {

constexpr int D = win::D;
constexpr int BM = 128, BN = 128, NQT = 2;  // Query rows of a CTA tile, keys of a stage, CTA tiles
constexpr int BS = 64;                      // keys of a step
constexpr int kSoftmaxWarps = 8, kProdWarp0 = 8, kProdWarps = 4, kMmaWarp = 12;
constexpr int kThreads = 32 * (kSoftmaxWarps + kProdWarps + 1);
constexpr uint64_t kWaitNs = 1000000000ull;
constexpr float kRescaleThreshold = 8.0f;  // log2 units the maximum may lag behind
constexpr int kStages = 4;                  // (a power of two)
constexpr int kPairRows = 2 * NQT * BM;

// shared-memory map of one CTA (bytes from a 1024-aligned base)
constexpr int kBlk = BM * 128;             // a [128 rows][64 fp16] swizzled block
constexpr int kBlkH = 64 * 128;            // a [64 rows][64 fp16] swizzled block
constexpr int OFF_Q = 0;                   // 2 Query tiles x 2 blocks (channels 0-63, 64-127)
constexpr int OFF_K = OFF_Q + NQT * 2 * kBlk;          // stages x 2 blocks [64 keys][64 ch]
constexpr int OFF_V = OFF_K + kStages * 2 * kBlkH;     // stages x [128 keys][64 ch] (MN-major B)
// the power of two that each Query row was multiplied by, 32 bits each.  (As a static array, whichever way it was
// read, a step of the loop took 2,000 cycles instead of 1,260; why is not known.)
constexpr int OFF_POWER = OFF_V + kStages * kBlk;
constexpr int kSmemBytes = OFF_POWER + NQT * BM * 4;
constexpr int kSmemAlloc = kSmemBytes + 1024;

template <bool B>
struct Flag {
  static constexpr bool value = B;
};
struct Bars {
  uint64_t full[kStages], empty[kStages];
  uint64_t s_full[2][2], p_ready[2][2], pv_done[2][2], q_full, o_done, drain;
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
    const int64_t i = win::quotient(r, a.group);
    const int h = kvh * a.group + (int)(r - i * a.group);
    const int64_t at = b * a.os.batch + h * a.os.head + i * a.os.token;
    if (a.out_f32) f32 = (float *)a.out + at;
    else bf16 = (uint16_t *)a.out + at;
    if (a.lse) lse = a.lse + (b * a.H + h) * a.nq + i;
    merge = a.merge;
  }
};

// A producer thread's share of a 128-key stage: four pieces of 16 channels.
template <int BITS>
struct Pieces {
  uint32_t c[4][BITS / 2];
  uint32_t step[4];
};

// One producer thread's side of Keys or Values in CTA cr of a pair.  Keys: rows r = 16 w + 4 i + lane / 4 % 4
// (i = 0..3) of the CTA's half, key 64 (r / 32) + 32 cr + r % 32, channels 16 (lane % 4 + 4 (lane / 16));
// Values: key rows 32 w + 8 i + lane / 4, channels 64 cr + 16 (lane % 4).  A quarter warp's 16-byte stores
// take two rows, one of even and one of odd number, so the swizzle puts them into eight bank groups.
template <int BITS, bool VAL>
struct Producer {
  static constexpr int kRowStep = VAL ? 8 : 4;
  static constexpr uint32_t kStage = VAL ? (uint32_t)kBlk : 2u * kBlkH;
  static constexpr int kRowBytes = D * BITS / 8;
  const uint8_t *codes, *steps;   // of slot key0
  int key0;
  uint32_t dst[2][2];             // shared addresses of the piece's two chunks in even and odd rows i

  __device__ __forceinline__ Producer(const WindowAttend &a, unsigned char *sm, int64_t y, int cr, int w, int lane) {
    const int row0 = VAL ? 32 * w + (lane >> 2) : 16 * w + ((lane >> 2) & 3);
    const int piece = VAL ? (lane & 3) : (lane & 3) + 4 * (lane >> 4);
    const int ch = VAL ? 64 * cr + 16 * piece : 16 * piece;
    key0 = VAL ? row0 : BS * (w >> 1) + 32 * cr + (row0 & 31);
    const int64_t head_row = y * (a.w.sink + a.w.ring) + key0;
    codes = (VAL ? a.w.v_codes : a.w.k_codes) + head_row * kRowBytes + ch * BITS / 8;
    steps = (VAL ? a.w.v_step : a.w.k_step) + head_row * win::kSteps + ch / win::kGroup;
    const uint32_t block = tc::smem_u32(sm + (VAL ? OFF_V : OFF_K)) + (VAL ? 0u : (uint32_t)(piece >> 2) * kBlkH);
#pragma unroll
    for (int i = 0; i < 2; i++)
#pragma unroll
      for (int h = 0; h < 2; h++) {
        const uint32_t row = (uint32_t)(row0 + kRowStep * i), chunk = 2u * (uint32_t)(piece & 3) + h;
        dst[i][h] = block + row * 128u + ((chunk ^ (row & 7u)) << 4);
      }
  }
  __device__ __forceinline__ void load1(const uint8_t *c, const uint8_t *s, Pieces<BITS> &p, int i) const {
    if (BITS == 8) {
      const uint4 x = __ldg((const uint4 *)c);
      p.c[i][0] = x.x; p.c[i][1] = x.y; p.c[i][2 % (BITS / 2)] = x.z; p.c[i][3 % (BITS / 2)] = x.w;
    } else {
      const uint2 x = __ldg((const uint2 *)c);
      p.c[i][0] = x.x; p.c[i][1] = x.y;
    }
    p.step[i] = __ldg(s);
  }
  // The codes of the stage of keys v0 .. v0 + 127; `slot0` >= 0: they lie in consecutive slots from there.
  __device__ __forceinline__ void load(const win::Keys &keys, int v0, int64_t slot0, uint32_t sink, uint32_t ring,
                                       Pieces<BITS> &p) const {
    if (slot0 >= 0) {
      const uint8_t *c = codes + slot0 * kRowBytes, *s = steps + slot0 * win::kSteps;
#pragma unroll
      for (int i = 0; i < 4; i++) load1(c + i * kRowStep * kRowBytes, s + i * kRowStep * win::kSteps, p, i);
    } else {
#pragma unroll
      for (int i = 0; i < 4; i++) {
        const int v = v0 + key0 + kRowStep * i;
        p.step[i] = 0u;   // past the last key: a zero row
#pragma unroll
        for (int u = 0; u < BITS / 2; u++) p.c[i][u] = 0u;
        if (v < keys.total) {
          const int64_t d = (int64_t)keys.slot(v, sink, ring) - key0;
          load1(codes + d * kRowBytes, steps + d * win::kSteps, p, i);
        }
      }
    }
  }
  __device__ __forceinline__ void store(uint32_t stage, const Pieces<BITS> &p, const win::Bases &bases) const {
#pragma unroll
    for (int i = 0; i < 4; i++) {
      uint32_t d[8];
      const win::Step st = win::step_of_byte<BITS>(p.step[i]);
      if (BITS == 8) {
#pragma unroll
        for (int u = 0; u < 4; u++) win::decode8(p.c[i][u % (BITS / 2)], st, bases, d[2 * u], d[2 * u + 1]);
      } else {
        uint32_t q[4];
        win::decode4(p.c[i][0], st, bases, q);
        d[0] = q[0]; d[1] = q[1]; d[2] = q[2]; d[3] = q[3];
        win::decode4(p.c[i][1], st, bases, q);
        d[4] = q[0]; d[5] = q[1]; d[6] = q[2]; d[7] = q[3];
      }
      const uint32_t at = stage * kStage + (uint32_t)(i >> 1) * (2u * kRowStep * 128u);
      tc::sts128(dst[i & 1][0] + at, make_uint4(d[0], d[1], d[2], d[3]));
      tc::sts128(dst[i & 1][1] + at, make_uint4(d[4], d[5], d[6], d[7]));
    }
  }
};

template <int BITS>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    window_attend_kernel(const __grid_constant__ WindowAttend a) {
  extern __shared__ __align__(16) unsigned char smem_raw[];
  unsigned char *sm = smem_raw + ((1024u - (tc::smem_u32(smem_raw) & 1023u)) & 1023u);
  __shared__ Bars bars;
  __shared__ uint32_t tmem_base_sh;
  __shared__ int abort_flag;
  __shared__ float2 half_sums[BM];   // short items: maximum and sum of the second tile's rows
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  // pairs in launch order: every Key head's full items, head by head (its cache stays in L2), then every
  // head's last item, whose second Query tile may be empty: the short ones fill the last wave's gaps
  const int64_t pair = blockIdx.x >> 1, heads = (int64_t)a.w.batch * a.w.kv_heads;
  const int64_t items = (a.rows + kPairRows - 1) / kPairRows, early = heads * (items - 1);
  const int64_t y = pair < early ? win::quotient(pair, items - 1) : pair - early, b = win::quotient(y, a.w.kv_heads);
  const int64_t item = pair < early ? pair - y * (items - 1) : items - 1;
  const int kvh = (int)(y - b * a.w.kv_heads), split = (int)blockIdx.y;
  const int cr = (int)tc::cluster_ctarank();
  volatile int *abort_v = &abort_flag;

  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");   // the joining kernel, if any, may line up
  if (warp == kMmaWarp) {
    if (lane == 0) {
      for (int i = 0; i < kStages; i++) {
        // this CTA's producer warps; in the even CTA also the odd one's last warp, which passes on that its
        // producers are done (a producer's own arrival in the peer would wait for its loads in flight)
        tc::mbar_init(&bars.full[i], kProdWarps + 1 - cr);
        tc::mbar_init(&bars.empty[i], 1);
      }
      for (int i = 0; i < 2; i++) {
        tc::mbar_init(&bars.s_full[i][0], 1);
        tc::mbar_init(&bars.s_full[i][1], 1);
        // both CTAs' 4 softmax warps of tile i; one barrier per buffer, as a warp may finish its next step
        // before another has finished this one
        tc::mbar_init(&bars.p_ready[i][0], 8);
        tc::mbar_init(&bars.p_ready[i][1], 8);
        tc::mbar_init(&bars.pv_done[i][0], 1);
        tc::mbar_init(&bars.pv_done[i][1], 1);
      }
      tc::mbar_init(&bars.q_full, 2 * kSoftmaxWarps);    // both CTAs' softmax warps (even CTA's copy used)
      tc::mbar_init(&bars.o_done, 1);
      tc::mbar_init(&bars.drain, 1);
      abort_flag = 0;
      tc::fence_mbar_init();
    }
    __syncwarp();
    tc::tmem_alloc2(&tmem_base_sh, 512);
    tc::tmem_relinquish2();
    tc::fence_before_sync();
  }
  // Nothing of the peer's is touched before the other half of this barrier, which every way out passes
  // too.  (This half waits for the warp's memory operations, so it stands before the Queries'.)
  tc::cluster_arrive();
  // the sequence's numbers, on their way while the rest is set up
  const int64_t q0 = a.q_start[b], len = win::tokens_of(a.length[b]);
  int64_t nq = a.q_count ? (int64_t)a.q_count[b] : a.nq;
  // ---- this CTA's two Query tiles -> shared memory, by the softmax warps: all rows' copies in flight while
  // the keys are worked out, whatever turns out to be padding.  (Loops stay rolled here and below: a CTA's
  // first pass through its code is paced by instruction fetches.) ----
  const int64_t pair0 = item * kPairRows, row_base = pair0 + (int64_t)cr * BM;   // row_base: this CTA's row 0 of tile 0
  // this thread's piece of row tid / 16 of tile 0; 16 rows on is 2 KB further, the next tile 2 blocks
  const uint32_t q_dst = tc::smem_u32(sm) + OFF_Q + (uint32_t)((tid & 15) / 8) * kBlk +
                         tc::sw128_offset((uint32_t)tid >> 4, 8u * (tid & 7));
  if (warp < kSoftmaxWarps) {
    const int ci = tid & 15, rr0 = tid >> 4;   // 16-byte piece of a row; rows rr0, rr0 + 16, ...
    const uint16_t *qb = a.q + b * a.qs.batch + (int64_t)kvh * a.group * a.qs.head + 8 * ci;
    // 16 rows on: 16 / group Queries and 16 % group heads, a Query more where the heads run over
    const int step_i = 16 / a.group, step_h = 16 - step_i * a.group;
    const int64_t ahead = step_i * a.qs.token + step_h * a.qs.head, wrap = a.qs.token - a.group * a.qs.head;
#pragma unroll 1
    for (int x = 0; x < NQT; x++) {
      const int64_t r = row_base + (int64_t)x * 2 * BM + rr0, i = win::quotient(r, a.group);
      int h = (int)(r - i * a.group), left = a.rows - r < BM ? (int)(a.rows - r) : BM;   // (may be negative)
      const uint16_t *src = qb + h * a.qs.head + i * a.qs.token;
      uint32_t dst = q_dst + (uint32_t)x * 2u * kBlk;
#pragma unroll 2
      for (int k = 0; k < BM / 16; k++) {
        tc::cp_async16_zfill(dst, left > 0 ? src : qb, left > 0 ? 16u : 0u);
        dst += 2048u;
        left -= 16;
        h += step_h;
        src += ahead + (h >= a.group ? wrap : 0);
        h -= h >= a.group ? a.group : 0;
      }
    }
    tc::cp_async_commit();
  }
  auto leave = [&]() {   // without having multiplied anything
    tc::cp_async_wait<0>();
    __syncwarp();
    tc::cluster_wait();
    if (warp == kMmaWarp) {
      tc::fence_after_sync();
      tc::tmem_dealloc2(tmem_base_sh, 512);
    }
  };

  nq = nq < a.nq ? nq : a.nq;
  const int64_t rows = nq * a.group;              // live rows of this Key head
  if (!win::starts(q0) || pair0 >= rows) {        // the same in both CTAs
    leave();
    return;
  }
  const win::Seq seq{len, a.w.sink, a.w.ring, a.tpf, a.frames};
  auto frame_of = [&](int64_t r) { return seq.frame(q0 + win::quotient(r, a.group)); };
  const int64_t pair1 = pair0 + kPairRows < rows ? pair0 + kPairRows : rows;
  win::Keys keys;
  keys.init(seq, frame_of(pair0), frame_of(pair1 - 1));
  const int tiles = (keys.total + BN - 1) / BN;
  // (tiles < 2^24 and splits <= 2^12: the products can pass 32 bits)
  const int j0 = a.splits == 1 ? 0 : (int)win::quotient((int64_t)tiles * split, a.splits);
  const int J = (a.splits == 1 ? tiles : (int)win::quotient((int64_t)tiles * (split + 1), a.splits)) - j0;
  if (J == 0) {   // these rows see no key (in this part): 16 lanes write a row's zeros
    for (int e = tid; e < NQT * BM * 16; e += kThreads) {
      const int64_t r = row_base + (int64_t)(e / 16 / BM) * 2 * BM + e / 16 % BM;
      if (r >= rows) continue;
      RowOut out;
      out.init(a, y, b, kvh, split, r);
      if (out.merge) continue;
      const int c = 8 * (e & 15);
      if (out.bf16) {
        *(uint4 *)(out.bf16 + c) = make_uint4(0, 0, 0, 0);
      } else {
        *(float4 *)(out.f32 + c) = make_float4(0.f, 0.f, 0.f, 0.f);
        *(float4 *)(out.f32 + c + 4) = make_float4(0.f, 0.f, 0.f, 0.f);
      }
      if (out.lse && c == 0) *out.lse = -INFINITY;
    }
    leave();
    return;
  }
  // A short item: its rows fill the first Query tile at most.  Both tiles then take those rows and every
  // other step of 64 keys each, and are joined at the end: two chains of MMA and softmax instead of one.
  const bool brief = pair0 + 2 * BM >= rows;

  const uint32_t powers = tc::smem_u32(sm) + OFF_POWER;
  // ---- the Queries, which have arrived by now: bf16 -> fp16 in place, padding rows 0 ----
  if (warp < kSoftmaxWarps) {
    // this warp's rows: two in each of 16 passes, pass 8 x + k those of tile x from 16 k on
    tc::sts32(powers + 4u * (uint32_t)((lane >> 1) * 16 + (tid >> 5) * 2 + (lane & 1)), 0u);
    tc::cp_async_wait<0>();
    uint32_t top = 0u, small = 0u;   // the largest magnitudes, a NaN above all; passes in which this piece is below 1
#pragma unroll 1
    for (int x = 0; x < NQT; x++) {
      const int64_t r = row_base + (int64_t)x * 2 * BM + (tid >> 4);
      const int left = rows - r < BM ? (int)(rows - r) : BM;
      const uint32_t at = q_dst + (uint32_t)x * 2u * kBlk;
#pragma unroll 4
      for (int k = 0; k < BM / 16; k++) {
        const uint4 v = tc::lds128(at + (uint32_t)k * 2048u);
        const bool live = 16 * k < left;
        const uint32_t w[4] = {live ? v.x : 0u, live ? v.y : 0u, live ? v.z : 0u, live ? v.w : 0u};
        uint32_t hw[4];
#pragma unroll
        for (int u = 0; u < 4; u++) hw[u] = tc::pack_f16x2(__uint_as_float(w[u] << 16), __uint_as_float(w[u] & 0xFFFF0000u));
        tc::sts128(at + (uint32_t)k * 2048u, make_uint4(hw[0], hw[1], hw[2], hw[3]));
        const uint32_t m = win::max_abs_bf16x2(win::max_abs_bf16x2(w[0], w[1]), win::max_abs_bf16x2(w[2], w[3])) & 0x7FFF7FFFu;
        top = win::max_abs_bf16x2(top, m);
        small |= win::any_from_one(m) || !live ? 0u : 1u << (8 * x + k);
      }
    }
    if (win::any_beyond_fp16(top & 0x7FFF7FFFu)) qwm_dev_error(a.status, QWM_ERR_RANGE);
#pragma unroll
    for (int d = 1; d < 16; d <<= 1) small &= __shfl_xor_sync(0xffffffffu, small, d);   // of the whole row
    __syncwarp();
    for (uint32_t again = small | __shfl_xor_sync(0xffffffffu, small, 16); again; again &= again - 1u) {   // fetched once more
      const int pass = __ffs((int)again) - 1, x = pass >> 3, k = pass & 7;
      const bool mine = (small >> pass) & 1u;
      const int64_t r = row_base + (int64_t)x * 2 * BM + 16 * k + (tid >> 4), i = win::quotient(r, a.group);
      uint4 v = make_uint4(0u, 0u, 0u, 0u);
      if (mine) v = *(const uint4 *)(a.q + b * a.qs.batch + (kvh * a.group + (r - i * a.group)) * a.qs.head + i * a.qs.token + 8 * (tid & 15));
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
      uint32_t m = win::max_abs_bf16x2(win::max_abs_bf16x2(w[0], w[1]), win::max_abs_bf16x2(w[2], w[3])) & 0x7FFF7FFFu;
      m = win::larger_half(m);
#pragma unroll
      for (int d = 1; d < 16; d <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, d));
      if (!mine) continue;
      const uint32_t power = win::row_power(m);
      const float up = win::power_of_two((int)power);
      uint32_t hw[4];
#pragma unroll
      for (int u = 0; u < 4; u++) hw[u] = tc::pack_f16x2(__uint_as_float(w[u] << 16) * up, __uint_as_float(w[u] & 0xFFFF0000u) * up);
      tc::sts128(q_dst + (uint32_t)x * 2u * kBlk + (uint32_t)k * 2048u, make_uint4(hw[0], hw[1], hw[2], hw[3]));
      if ((tid & 15) == 0) tc::sts32(powers + 4u * (uint32_t)(pass * 16 + (tid >> 4)), power);
    }
    tc::fence_proxy_async_smem();
  }
  // (once per role, so that the producers' first codes may be on their way before it)
  auto joined = [&]() -> uint32_t {   // both CTAs' barriers exist, and their tensor memory: its address
    __syncwarp();
    tc::cluster_wait();
    tc::fence_after_sync();
    return tmem_base_sh;
  };
  const int key_end = keys.total < (j0 + J) * BN ? keys.total : (j0 + J) * BN;
  const int steps = (key_end - j0 * BN + BS - 1) / BS;   // 2 J, or one less when the last stage is half empty

  if (warp < kSoftmaxWarps) {
    // ======================= softmax (Query tile x, row = TMEM lane) =======================
    const uint32_t tmem = joined();
    if (lane == 0) tc::mbar_arrive_remote(tc::mapa(tc::smem_u32(&bars.q_full), 0));
    asm volatile("bar.sync 1, %0;" ::"n"(32 * kSoftmaxWarps) : "memory");   // the rows' powers
    const int x = warp / 4, sub = warp % 4;
    const uint32_t lane_addr = (uint32_t)(32 * sub) << 16;
    const uint32_t tS0 = tmem + lane_addr + 128u * x, tO = tmem + lane_addr + 256u + 128u * x;
    const uint32_t p_ready0 = tc::mapa(tc::smem_u32(&bars.p_ready[x][0]), 0);
    const int power = (int)tc::lds32(powers + 4u * (uint32_t)((brief ? 0 : x * BM) + 32 * sub + lane));
    const float sl2 = a.scale_log2 * win::power_of_two(-power) * win::kUnit<BITS>;
    const uint64_t sc2 = pk64(sl2, sl2);
    const int64_t w0 = row_base + (brief ? 0 : (int64_t)x * 2 * BM) + 32 * sub;   // this warp's first row
    const int mine_n = brief ? (steps + 1 - x) >> 1 : steps;   // steps of this tile
    const int key_of = j0 * BN + (brief ? x * BS : 0), key_step = brief ? 2 * BS : BS;
    const int64_t r = w0 + lane;
    win::Row mine{0, 0, 0};
    win::Everyone every{INT32_MAX, 0, 0};   // a warp without a row masks nothing (its logits are 0)
    if (w0 < rows) {
      mine.init(seq, keys, r < rows ? frame_of(r) : -1);
      every.init(seq, keys, frame_of(w0), frame_of(w0 + 31 < rows ? w0 + 31 : rows - 1));
    }
    float m_used = -INFINITY;
    uint64_t acc = 0ull;   // the sum of the weights, each step's added as one: 1 / 64 of the additions to a large sum
    bool ok = true;
    for (int t = 0; t < mine_n; t++) {
      const int v0 = key_of + t * key_step;
      const bool full = every.see(v0, v0 + BS);
      const uint32_t tS = tS0 + (uint32_t)(t & 1) * BS;
      if (!__all_sync(0xffffffffu, tc::mbar_try_wait(&bars.s_full[x][t & 1], (t >> 1) & 1))) {
        if (!tc::mbar_wait(&bars.s_full[x][t & 1], (t >> 1) & 1, kWaitNs)) fail(&abort_flag, a.status);
        if (__any_sync(0xffffffffu, *abort_v != 0)) { ok = false; break; }   // the whole warp
      }
      tc::fence_after_sync();
      // the step's logits at once: their maximum, then their exponentials relative to m_used, which stands
      // kTopWeight below the running maximum; when that grows by more than 2^8 (rare after the first step)
      // the sum and O are rescaled
      uint32_t s[BS];
#pragma unroll
      for (int i = 0; i < BS; i += 16) tc::tmem_ld16(tS + (uint32_t)i, s + i);
      tc::tmem_ld_wait();
      if (!full) {
#pragma unroll
        for (int h = 0; h < BS / 32; h++) {
          const int v = v0 + 32 * h;
          const uint32_t seen = low_bits(mine.c0 - v) | (low_bits(mine.c2 - v) & ~low_bits(mine.c1 - v));
#pragma unroll
          for (int i = 0; i < 32; i++)
            if (!((seen >> i) & 1u)) s[32 * h + i] = 0xFF800000u;  // -inf: weight exactly 0
        }
      }
      float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
      for (int i = 0; i < BS; i += 8)
#pragma unroll
        for (int u = 0; u < 4; u++)
          mx[u] = tc::max3(mx[u], __uint_as_float(s[i + 2 * u]), __uint_as_float(s[i + 2 * u + 1]));
      const float m_new = fmaxf(m_used, fmaf(tc::max3(fmaxf(mx[0], mx[1]), mx[2], mx[3]), sl2, -win::kTopWeight));
      if (__any_sync(0xffffffffu, m_new > m_used + kRescaleThreshold)) {
        const float alpha = m_new == -INFINITY ? 1.f : tc::ex2_approx(m_used - m_new);
        const uint64_t a2 = pk64(alpha, alpha);
        acc = tc::fma2(acc, a2, 0ull);
        if (t > 0) {  // O of the earlier steps, once PV_x(t-1) has been added (PV_x(t) waits for this warp)
          if (!tc::mbar_wait(&bars.pv_done[x][(t - 1) & 1], ((t - 1) >> 1) & 1, kWaitNs)) fail(&abort_flag, a.status);
          tc::fence_after_sync();
#pragma unroll 1
          for (int c = 0; c < D; c += 16) {
            uint32_t o[16];
            tc::tmem_ld16(tO + c, o);
            tc::tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 16; i++) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
            tc::tmem_st16(tO + c, o);
          }
        }
        m_used = m_new;
      }
      const float mneg = m_used == -INFINITY ? 0.f : -m_used;  // a row that has seen no key yet
      const uint64_t nm2 = pk64(mneg, mneg);
      uint64_t sum0 = 0ull, sum1 = 0ull;
#pragma unroll
      for (int h = 0; h < BS / 32; h++) {
        uint32_t pw[16];
#pragma unroll
        for (int i = 0; i < 16; i++) {  // packed fp32 pairs: S * scale - m, then 2^x
          const uint64_t x2 = tc::fma2(pk64(s[32 * h + 2 * i], s[32 * h + 2 * i + 1]), sc2, nm2);
          const float e0 = tc::ex2_approx(tc::f2lo(x2)), e1 = tc::ex2_approx(tc::f2hi(x2));
          const uint64_t e2 = pk64(e0, e1);
          if (i & 1) sum1 = h == 0 && i == 1 ? e2 : tc::add2(sum1, e2);
          else sum0 = h == 0 && i == 0 ? e2 : tc::add2(sum0, e2);
          pw[i] = tc::pack_f16x2(e0, e1);
        }
        tc::tmem_st16(tS + 16u * h, pw);  // P (fp16 pairs) over the logits
      }
      acc = tc::add2(acc, tc::add2(sum0, sum1));
      tc::tmem_st_wait();
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive_remote(p_ready0 + 8u * (uint32_t)(t & 1));
    }
    float l = tc::f2lo(acc) + tc::f2hi(acc), share = 1.f, share1 = 0.f;   // what O_0 and O_1 count for
    if (brief) {   // every softmax warp comes here, whatever happened before
      if (x == 1) half_sums[tid & (BM - 1)] = make_float2(m_used, l);
      asm volatile("bar.sync 1, %0;" ::"n"(32 * kSoftmaxWarps) : "memory");
      if (x == 0) {
        const float2 o = half_sums[tid];
        const float m = fmaxf(m_used, o.x);
        share = m_used == -INFINITY ? 0.f : tc::ex2_approx(m_used - m);
        share1 = o.x == -INFINITY ? 0.f : tc::ex2_approx(o.x - m);
        l = fmaf(l, share, o.y * share1);
        m_used = m;
      }
    }
    const bool writer = !(brief && x == 1);
    if (ok && writer && !tc::mbar_wait(&bars.o_done, 0, kWaitNs)) fail(&abort_flag, a.status);
    if (ok && writer && !__any_sync(0xffffffffu, *abort_v != 0)) {
      tc::fence_after_sync();
      float inv = l > 0.f ? win::kUnit<BITS> / l : 0.f, keep = 0.f;
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
      // through shared memory (every operand has been read), so that the stores write whole rows: a
      // 16 KB buffer per warp, 16-byte pieces permuted by the row's low bits against bank conflicts
      const uint32_t buf = tc::smem_u32(sm) + (uint32_t)warp * 16384u, rx = (uint32_t)lane & 7u;
      const bool half = a.splits == 1 && !a.out_f32;   // bf16 rows
      const float w0_out = share * inv, w1_out = share1 * inv;
#pragma unroll 1
      for (int c = 0; c < D; c += 32) {
        uint32_t o[32];
        tc::tmem_ld32(tO + c, o);
        tc::tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 32; i++) o[i] = __float_as_uint(__uint_as_float(o[i]) * w0_out);
        if (brief && steps > 1) {   // (a single step left O_1 unwritten)
          uint32_t o1[32];
          tc::tmem_ld32(tO + 128 + c, o1);
          tc::tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < 32; i++)
            o[i] = __float_as_uint(fmaf(__uint_as_float(o1[i]), w1_out, __uint_as_float(o[i])));
        }
        if (half) {
#pragma unroll
          for (int v = 0; v < 4; v++) {
            uint32_t w[4];
#pragma unroll
            for (int u = 0; u < 4; u++)
              w[u] = tc::pack_bf16x2(__uint_as_float(o[8 * v + 2 * u]), __uint_as_float(o[8 * v + 2 * u + 1]));
            tc::sts128(buf + (uint32_t)lane * 256u + ((((uint32_t)(c / 8 + v)) ^ rx) << 4), make_uint4(w[0], w[1], w[2], w[3]));
          }
        } else {
#pragma unroll
          for (int v = 0; v < 8; v++)
            tc::sts128(buf + (uint32_t)lane * 512u + ((((uint32_t)(c / 4 + v)) ^ rx) << 4),
                       make_uint4(o[4 * v], o[4 * v + 1], o[4 * v + 2], o[4 * v + 3]));
        }
      }
      __syncwarp();
      const uint32_t writes = __ballot_sync(0xffffffffu, write);
      const uint64_t mine_out = half ? (uint64_t)out.bf16 : (uint64_t)out.f32;
      if (half) {
#pragma unroll 8
        for (int i = 0; i < 16; i++) {
          const int rw = 2 * i + (lane >> 4), c = lane & 15;
          uint16_t *dst = (uint16_t *)__shfl_sync(0xffffffffu, mine_out, rw);
          const uint4 v = tc::lds128(buf + (uint32_t)rw * 256u + ((uint32_t)(c ^ (rw & 7)) << 4));
          if ((writes >> rw) & 1u) *(uint4 *)(dst + 8 * c) = v;
        }
      } else {
#pragma unroll 4
        for (int rw = 0; rw < 32; rw++) {
          float *dst = (float *)__shfl_sync(0xffffffffu, mine_out, rw);
          const float k = __shfl_sync(0xffffffffu, keep, rw);
          const uint4 v = tc::lds128(buf + (uint32_t)rw * 512u + ((uint32_t)(lane ^ (rw & 7)) << 4));
          if ((writes >> rw) & 1u) {
            float4 x = make_float4(__uint_as_float(v.x), __uint_as_float(v.y), __uint_as_float(v.z), __uint_as_float(v.w));
            if (k > 0.f) {
              const float4 p = *(const float4 *)(dst + 4 * lane);
              x = make_float4(fmaf(k, p.x, x.x), fmaf(k, p.y, x.y), fmaf(k, p.z, x.z), fmaf(k, p.w, x.w));
            }
            *(float4 *)(dst + 4 * lane) = x;
          }
        }
      }
    }
  } else if (warp == kMmaWarp) {
    // ======================= the last warps: the even CTA's issues the pair's MMAs, the odd one's passes on
    // that its CTA's stages are full =======================
    const uint32_t tmem = joined();
    // The warp's common answer.  Whether someone gave up is looked at only where there is something to
    // wait for: the flag's read behind every barrier cost 12% of a step.
    auto wait = [&](uint64_t *bar, uint32_t parity) -> bool {
      if (__all_sync(0xffffffffu, tc::mbar_try_wait_cluster(bar, parity))) return true;
      return __all_sync(0xffffffffu, tc::mbar_wait_cluster(bar, parity, kWaitNs) && !*abort_v);
    };
    if (cr == 1) {
      const uint32_t full = tc::mapa(tc::smem_u32(&bars.full[0]), 0);
      for (int j = 0; j < J; j++) {
        if (!wait(&bars.full[j & (kStages - 1)], (j / kStages) & 1)) {
          fail(&abort_flag, a.status);
          break;
        }
        if (lane == 0) tc::mbar_arrive_remote(full + 8u * (uint32_t)(j & (kStages - 1)));
      }
    } else {
      constexpr uint32_t idesc = tc::idesc_f16_f32(2 * BM, BS), idesc_pv = tc::idesc_f16_f32_bmn(2 * BM, D);
      constexpr uint16_t kBoth = 3;
      // broadcast, so that everything derived from them is the warp's and not a lane's
      const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0), s0 = __shfl_sync(0xffffffffu, tc::smem_u32(sm), 0);
      const int n = __shfl_sync(0xffffffffu, steps, 0);
      const uint64_t dq = tc::desc_sw128(s0 + OFF_Q), dk = tc::desc_sw128(s0 + OFF_K);
      const uint64_t dv = tc::desc_sw128_mn(s0 + OFF_V, kBlk, 1024);
      bool ok = true;
      // step t of tile x: both tiles take the same 64 keys, or (short items) a half each of stage t.  (The two
      // forms are compiled apart: chosen at every step they cost a tenth of it.)
      auto multiply = [&](auto rows_of_two) {
        constexpr bool two = decltype(rows_of_two)::value;
        const int T = two ? n : (n + 1) >> 1;   // steps of tile 0
        auto stage_of = [&](int t) { return two ? t >> 1 : t; };
        auto half_of = [&](int x, int t) { return two ? t & 1 : x; };
        auto begins = [&](int t) { return !two || !(t & 1); };
        auto ends = [&](int t) { return !two || (t & 1) || t + 1 == n; };
        auto there = [&](int t) { return two || 2 * t + 1 < n; };   // tile 1 has a step t
        auto qk = [&](int x, int t) {
          const uint32_t ko = (uint32_t)(stage_of(t) % kStages) * 2 * kBlkH + (uint32_t)half_of(x, t) * 32 * 128;
          const uint64_t da = dq + (uint64_t)(two ? x * 2 * kBlk / 16 : 0), db = dk + (uint64_t)(ko / 16);
          const uint32_t d = tm + 128u * x + (uint32_t)(t & 1) * BS;
#pragma unroll
          for (int kk = 0; kk < D / 16; kk++)
            tc::mma2_ss_warp(d, da + (uint64_t)(((kk / 4) * kBlk + 32 * (kk % 4)) / 16),
                             db + (uint64_t)(((kk / 4) * kBlkH + 32 * (kk % 4)) / 16), idesc, kk > 0);
          tc::mma2_commit_warp(&bars.s_full[x][t & 1], kBoth);
        };
        auto pv = [&](int x, int t) {
          const uint32_t vo = (uint32_t)(stage_of(t) % kStages) * kBlk + (uint32_t)half_of(x, t) * BS * 128;
          const uint64_t db = dv + (uint64_t)(vo / 16);
          const uint32_t p = tm + 128u * x + (uint32_t)(t & 1) * BS;
#pragma unroll
          for (int kk = 0; kk < BS / 16; kk++)
            tc::mma2_ts_warp(tm + 256u + 128u * x, p + 8u * kk, db + (uint64_t)(2048 * kk / 16), idesc_pv,
                             (t > 0 || kk > 0));
          tc::mma2_commit_warp(&bars.pv_done[x][t & 1], kBoth);
        };
        auto keys_there = [&](int t) {   // the Keys and Values of step t (a stage's first step waits for it)
          return !begins(t) || wait(&bars.full[stage_of(t) % kStages], (stage_of(t) / kStages) & 1);
        };
        for (int t = 0; ok && t < 2 && t < T; t++) {
          ok = keys_there(t);
          if (!ok) break;
          tc::fence_after_sync();
          qk(0, t);
          if (there(t)) qk(1, t);
        }
        for (int t = 0; ok && t < T; t++) {
          ok = wait(&bars.p_ready[0][t & 1], (t >> 1) & 1);
          if (!ok) break;
          tc::fence_after_sync();
          pv(0, t);
          if (t + 2 < T) {
            ok = keys_there(t + 2);
            if (!ok) break;
            tc::fence_after_sync();
            qk(0, t + 2);
          }
          if (there(t)) {
            ok = wait(&bars.p_ready[1][t & 1], (t >> 1) & 1);
            if (!ok) break;
            tc::fence_after_sync();
            pv(1, t);
            if (t + 2 < T && there(t + 2)) qk(1, t + 2);
          }
          if (ends(t)) tc::mma2_commit_warp(&bars.empty[stage_of(t) % kStages], kBoth);   // (S precedes P V)
        }
      };
      ok = wait(&bars.q_full, 0);
      if (__shfl_sync(0xffffffffu, (int)brief, 0)) multiply(Flag<false>{});
      else multiply(Flag<true>{});
      if (ok) tc::mma2_commit_warp(&bars.o_done, kBoth);
      if (!ok) fail(&abort_flag, a.status);
      tc::mma2_commit_warp(&bars.drain, 1);  // every MMA issued above completes before TMEM is released
      if (!tc::mbar_wait(&bars.drain, 0, kWaitNs)) qwm_dev_error(a.status, QWM_ERR_DEVICE_TIMEOUT);
    }
  } else {
    // ======================= producers: Keys, then Values, of every stage =======================
    const int pw = warp - kProdWarp0;
    const Producer<BITS, false> pk(a, sm, y, cr, pw, lane);
    const Producer<BITS, true> pv(a, sm, y, cr, pw, lane);
    const uint32_t sink = (uint32_t)a.w.sink, ring = (uint32_t)a.w.ring;
    Pieces<BITS> k0, v0, k1, v1;
    auto free_again = [&](int j) -> bool {   // the previous contents of stage j's place are consumed
      uint64_t *empty = &bars.empty[j & (kStages - 1)];
      if (j < kStages || __all_sync(0xffffffffu, tc::mbar_try_wait(empty, (j / kStages - 1) & 1))) return true;
      if (!tc::mbar_wait(empty, (j / kStages - 1) & 1, kWaitNs)) fail(&abort_flag, a.status);
      return !__any_sync(0xffffffffu, *abort_v != 0);         // warp-uniform exit
    };
    // stage j is stored and the codes of stage j + 2 fetched in its place; the first round only fetches
    auto stage = [&](int j, Pieces<BITS> &k, Pieces<BITS> &v) -> bool {
      const int s = j & (kStages - 1), next = (j0 + j + 2) * BN;
      const bool store = j >= 0 && j < J, load = j + 2 < J;
      int64_t slot0 = -1;   // that stage's first slot when its slots are consecutive
      if (load) {
        const uint32_t first = keys.slot(next, sink, ring);
        if (next + BN <= keys.total && keys.slot(next + BN - 1, sink, ring) == first + BN - 1) slot0 = first;
      }
      if (store) {
        if (!free_again(j)) return false;
        pk.store((uint32_t)s, k, a.bases);
      }
      if (load) pk.load(keys, next, slot0, sink, ring, k);
      if (store) {
        pv.store((uint32_t)s, v, a.bases);
        tc::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&bars.full[s]);
      }
      if (load) pv.load(keys, next, slot0, sink, ring, v);
      return true;
    };
#pragma unroll 1
    for (int j = -2; j < J; j += 2) {
      if (!stage(j, k0, v0) || !stage(j + 1, k1, v1)) break;
      if (j < 0) joined();
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::cluster_sync();  // the peer has finished with this CTA's barriers, shared and tensor memory
  if (warp == kMmaWarp) {
    tc::fence_after_sync();
    tc::tmem_dealloc2(tmem_base_sh, 512);
  }
}

template <int BITS>
cudaError_t launch_bits(const WindowAttend &a, cudaStream_t st) {
  static std::atomic<uint64_t> allowed{0};
  const cudaError_t e = allow_shared(window_attend_kernel<BITS>, kSmemAlloc, allowed);
  if (e != cudaSuccess) return e;
  const int64_t pairs = (int64_t)a.w.batch * a.w.kv_heads * ((a.rows + kPairRows - 1) / kPairRows);
  if (2 * pairs > INT32_MAX) return cudaErrorInvalidValue;
  const dim3 grid((unsigned)(2 * pairs), (unsigned)a.splits);
  window_attend_kernel<BITS><<<grid, kThreads, kSmemAlloc, st>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_window_tiles(const WindowAttend &a, cudaStream_t st) {
  return a.w.bits == 8 ? launch_bits<8>(a, st) : launch_bits<4>(a, st);
}

// Few rows run on warp tiles, which read the cache once per 16 rows; more than 32 on tensor-memory tiles (at
// 39,000 tokens of 40 heads, 8 bits: 16 rows take 90 us, 32 take 170, 33 to 256 on tensor-memory tiles 206 to 221).
// The keys are split into the number of parts for which whole waves of CTAs end soonest, by what a part
// costs in cycles, as measured: on warp tiles 12 per key (a CTA of 8 warps, whatever the code width) and
// 10,000 for starting and ending, 6,000 more for a second kernel that joins the parts; up to 8 parts may be
// a cluster's CTAs instead, which fill nine tenths of the slots.  On tensor-memory tiles 20 per key, 20,000
// and 7,000; calls that fill the SMs are left whole.
// A part takes 2^18 keys at most, whatever the time: weights below 2^-32 of a part's largest are lost (2^-14 of
// it between them), and its fp32 sums stay within 2^14 additions of products and 2^12 of weights.
constexpr int64_t kPartKeys = (int64_t)1 << 18;
WindowPlan window_plan(int64_t batch, int64_t kv_heads, int64_t rows, int64_t keys, int num_sms) {
  WindowPlan p;
  p.tiles = rows > 32;
  p.splits = 1;
  p.cluster = false;
  const int64_t least = (keys + kPartKeys - 1) / kPartKeys;
  const int64_t heads = batch * kv_heads, most = keys / 256 < 64 ? keys / 256 : 64;   // 256 keys a part at least
  const int64_t work = p.tiles ? heads * ((rows + kPairRows - 1) / kPairRows) : heads * (rows <= 8 ? 1 : (rows + 15) / 16);
  const int64_t slots = p.tiles ? num_sms / 2 : (rows <= 8 ? 2 : 1) * (int64_t)num_sms;
  const int64_t per_key = p.tiles ? 20 : 12, fixed = p.tiles ? 20000 : 10000, join = p.tiles ? 7000 : 6000;
  int64_t best = keys * per_key + fixed;
  for (int64_t s = 2; work < slots && s <= most && work * s <= 4 * slots; s++) {
    const int64_t part = keys * per_key / s + fixed;
    const int64_t joined = (work * s + slots - 1) / slots * part + join;
    if (joined < best) {
      best = joined;
      p.splits = (int)s;
      p.cluster = false;
    }
    if (!p.tiles && s <= kWindowCluster) {
      const int64_t near = slots * 9 / 10, clustered = (work * s + near - 1) / near * part;
      if (clustered < best) {
        best = clustered;
        p.splits = (int)s;
        p.cluster = true;
      }
    }
  }
  if (p.splits < least) {
    p.splits = (int)least;
    p.cluster = false;
  }
  return p;
}
