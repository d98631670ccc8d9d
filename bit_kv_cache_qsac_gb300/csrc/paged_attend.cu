// Attention over a paged cache for sequences with many new rows (chunks of a prompt, frames), on the tensor
// cores (tcgen05 + TMEM).
//
//   l_ij = scale q_i . k_hat_j over the tokens row i sees, o_i = softmax(l_i) V_hat, with k_hat and v_hat
// decoded from the 8- or 4-bit pages inside the kernel (exact in fp16; see window.cuh for Queries and weights).
//
// An item is one Key head of one sequence with 512 of its rows (row r = token r / group, head r % group) and the
// keys those rows see between them.  All items stand in one line (find_cuts) and a CTA pair (a cluster of two,
// cta_group::2 MMAs) takes an equal piece of it: whole items, and parts of those that a cut goes through.  So
// sequences of any lengths, causal items of different lengths and calls of a few items fill all SMs alike.
// CTA c of a pair holds rows 256 x + 128 c .. + 127 of the two Query tiles x = 0, 1.  The B operand of an
// M = 256 MMA is split by N, so CTA c decodes only keys 32 c .. 32 c + 31 of every 64 for Q K^T and only
// channels 64 c .. 64 c + 63 for P V: half of everything.
// Warp roles of each CTA (16 warps):
//   warps 0-3, 4-7  softmax of Query tile 0 / 1: thread = Query row = TMEM lane, 64 logits at a time; between
//                   pieces they write the output and fetch the next Queries;
//   warp 8          allocates TMEM; in the even CTA it issues every MMA of the pair, in the odd one it
//                   passes on to the even one that its producers have filled a stage;
//   warp 12         walks along the share and describes its pieces to the others, one ahead;
//   others          producers (9-11: Keys, 13-15: Values): codes two stages ahead in registers, table entries three,
//                   decoded into swizzled stages; they run ahead into the next piece while the last one is written.
// (No producer shares a scheduler with warp 8, whose instructions would have to be fetched again and again.)
// An item with up to 256 rows gives both tiles those rows and every other 64 keys each, joined at the end.
// TMEM (512 columns): S_x as two buffers of 64 keys, P_x over them, O_x.  Keys arrive in stages of 128, decoded
// in 16 rows of one page at a time; step t issues P V of tile x's keys t, then Q K^T of keys t + 2 into the
// buffer that frees.  Every wait is bounded (about one second); on expiry QWM_ERR_DEVICE_TIMEOUT is
// recorded, every role stops, outstanding MMAs are drained and TMEM is freed.
// Bound: the tensor pipe for long items; what stands around an item's loop for short ones.  Measured: 2,048 tokens over
// 30,000 before them (8 bits, 32 heads on 8): 579 us = 1,795 TFLOP/s; 4,680 over 40,560 (4 bits, 40 heads): 2.17 ms =
// 1,730 TFLOP/s (tensor pipe active in 78.7 and 79.5% of all cycles; under the power cap, after some 50 ms
// of them, 7 to 10% less).  In cycles: 12,000 until the first piece is described (7,500 for the cuts), 6,000 for its
// Queries, 3,300 (bf16) to 7,000 (parts) for writing it.  What was live across the steps decided the rest: pieces read
// from shared memory where they are needed instead of kept in registers gave 751 -> 698 us and 2,557 -> 2,420;
// multiply() written into the kernel's body instead of apart 785 -> 1,200.
#include "paged.cuh"

namespace {

constexpr int D = win::D;
constexpr int BM = 128, BN = 128, NQT = 2;  // Query rows of a CTA tile, keys of a stage, CTA tiles
constexpr int BS = 64;                      // keys of a step
constexpr int kSoftmaxWarps = 8, kProdWarps = 6, kMmaWarp = 8, kPlanWarp = 12;   // producers: 9-11, 13-15
constexpr int kThreads = 32 * 16;
constexpr uint64_t kWaitNs = 1000000000ull;
constexpr float kRescaleThreshold = 8.0f;  // log2 units the maximum may lag behind
constexpr int kStages = 4;                  // (a power of two)
constexpr int kRows = kPagedTileRows;       // rows of an item: 2 NQT BM
static_assert(kRows == 2 * NQT * BM, "");

// What pieces of an item cost, in hundreds of cycles: a stage of 128 keys for two tiles of rows, for one, and starting
// and ending; the least piece (stages) worth its own start, and the shortest share (about an item of one stage: 64 rows
// over 150 tokens take 21 us and 512 over 512 25; twice as long, so that two such items share a CTA pair, 27 and 35).
constexpr int kStageCost = 25, kBriefCost = 14, kStartCost = 110, kLeast = 3, kThin = 100;
constexpr int kMost = kPagedPieceKeys / BN;   // stages of a piece

// shared-memory map of one CTA (bytes from a 1024-aligned base)
constexpr int kBlk = BM * 128;             // a [128 rows][64 fp16] swizzled block
constexpr int kBlkH = 64 * 128;            // a [64 rows][64 fp16] swizzled block
constexpr int OFF_Q = 0;                   // 2 Query tiles x 2 blocks (channels 0-63, 64-127); outputs on their way out
constexpr int OFF_K = OFF_Q + NQT * 2 * kBlk;          // stages x 2 blocks [64 keys][64 ch]
constexpr int OFF_V = OFF_K + kStages * 2 * kBlkH;     // stages x [128 keys][64 ch] (MN-major B)
constexpr int OFF_POWER = OFF_V + kStages * kBlk;      // the power of two each Query row was multiplied by
constexpr int kSmemAlloc = OFF_POWER + NQT * BM * 4 + 1024;

// A piece of an item: stages j0 .. j0 + J - 1 of it (J > 0: a row sees itself), as the planning warp describes it.
struct Piece {
  int b, kvh, first, seq_rows, row0;   // its sequence; packed row of the first token; rows of a Key head; item's first row
  int place;                           // 0: whole item at once; else 1 + its place in the share
  int again, whole;                    // joined with the item's pieces before it there; the last piece of a whole item
  int j0, J, steps;                    // steps of 64 keys
  int brief;                           // 256 rows at most: both tiles take them
  int64_t q0, len;
  pgd::Keys keys;
  int done;                            // no piece: the share ends
};

struct Bars {
  uint64_t full[kStages], empty[kStages];
  uint64_t s_full[2][2], p_ready[2][2], pv_done[2][2], q_full, o_done, drain;
  uint64_t told[2], heard[2];   // a piece's description is there; everyone has read it
};

__shared__ Bars bars;
__shared__ int abort_flag;

__device__ __forceinline__ void fail(int32_t *status) {
  *(volatile int *)&abort_flag = 1;
  qwm_dev_error(status, QWM_ERR_DEVICE_TIMEOUT);
}
__device__ __forceinline__ int aborted() { return *(volatile int *)&abort_flag; }
__device__ __forceinline__ uint64_t pk64(uint32_t lo, uint32_t hi) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "r"(lo), "r"(hi));
  return d;
}
__device__ __forceinline__ uint64_t pk64(float lo, float hi) { return pk64(__float_as_uint(lo), __float_as_uint(hi)); }
// The lowest n bits set (n clamped to 0..32).
__device__ __forceinline__ uint32_t low_bits(int n) { return n <= 0 ? 0u : (n >= 32 ? 0xFFFFFFFFu : (1u << n) - 1u); }
// All softmax warps meet; true when any of them says so.
__device__ __forceinline__ bool softmax_meet(bool p) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbarrier.cta.red.or.pred q, 1, %2, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)p), "n"(32 * kSoftmaxWarps)
      : "memory");
  return r != 0;
}

// The items of a sequence: its Key heads by blocks of 512 rows, of which later ones may see more keys.
struct Work {
  __device__ __forceinline__ static int blocks_of(const PagedAttend &a, const pgd::Seq &q, int ib, pgd::Keys &keys) {
    const int r0 = ib * kRows, r1 = r0 + kRows < q.rows ? r0 + kRows : q.rows;
    keys.init(a, q.s, q.frame(a, r0), q.frame(a, r1 - 1));
    return (keys.total + BN - 1) / BN;
  }
  __device__ __forceinline__ static bool brief(const pgd::Seq &q, int ib) { return ib * kRows + 2 * BM >= q.rows; }
  __device__ __forceinline__ static int each(const pgd::Seq &q, int ib) { return brief(q, ib) ? kBriefCost : kStageCost; }
  __device__ __forceinline__ static int count(const PagedAttend &a, const pgd::Seq &q) {   // blocks of rows
    return q.rows > a.few ? (q.rows + kRows - 1) / kRows : 0;
  }
};

// A block of rows in the line: number f of all, block ib of sequence b, P what the blocks before it cost one Key head.
struct Place {
  int f, b, ib, blocks, each;
  int64_t P;
  __device__ __forceinline__ int64_t cost() const { return kStartCost + (int64_t)blocks * each; }
};
// From block f on, where P stands: the first block that ends behind `target` or has number `index`, or block `end`
// (of which only f and P are told).  starts: the number of each sequence's first block.  (One copy of the code for
// all its uses: what a CTA does once is paced by instruction fetches.)
__device__ __noinline__ Place walk(const PagedAttend &a, const int *starts, int f, int end, int64_t P, int64_t target, int index) {
  Place p;
  p.P = P;
  p.f = f;
  if (f >= end) return p;
  int lo = 0, hi = a.batch;   // starts[lo] <= f < starts[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (starts[mid] <= f) lo = mid;
    else hi = mid;
  }
  p.b = lo;
  pgd::Seq q = pgd::sequence(a, p.b);
#pragma unroll 1
  for (; p.f < end; p.f++) {
    if (p.f >= starts[p.b + 1]) {
      do p.b++;
      while (p.f >= starts[p.b + 1]);
      q = pgd::sequence(a, p.b);
    }
    pgd::Keys keys;
    p.ib = p.f - starts[p.b];
    p.blocks = Work::blocks_of(a, q, p.ib, keys);
    p.each = Work::each(q, p.ib);
    if (p.f == index || p.P + p.cost() > target) break;
    p.P += p.cost();
  }
  return p;
}

// The cuts of share `share` (begin, end) in the line of all items: by sequence, Key head and block of rows.  Found by
// the whole CTA: P, the running sum of the blocks' costs for one Key head, finds first the sequence (whose heads take
// kv_heads equal pieces of the line), then the head and the block.  Up to 512 blocks of rows are one a thread, with P
// in shared memory (5,000 cycles less than the walks); more are neighbours of a thread, walked along for each answer.
// mem: shared memory.  A share without work begins and ends at sequence `batch`.
__device__ __forceinline__ void find_cuts(const PagedAttend &a, int share, unsigned char *mem, PagedCut (&cut)[2]) {
  constexpr int kW = kThreads / 32;
  int *starts = (int *)mem;                                                          // [batch + 1]
  int64_t *sum = (int64_t *)(mem + (kPagedMaxBatch + 2) * (int)sizeof(int));   // [blocks + 1], up to 512 blocks
  __shared__ int64_t sums[kW];
  __shared__ int64_t edge[2][2];   // P at the begin and the end of the cuts' sequences
  __shared__ int where[2];         // the cuts' sequences
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  auto scan = [&](int64_t v, int64_t &total) -> int64_t {   // the sum over the threads before, and over all
    int64_t s = v;
#pragma unroll 1
    for (int d = 1; d < 32; d <<= 1) {
      const int64_t o = __shfl_up_sync(0xffffffffu, s, d);
      if (lane >= d) s += o;
    }
    __syncthreads();
    if (lane == 31) sums[warp] = s;
    __syncthreads();
    int64_t w = lane < kW ? sums[lane] : 0;
#pragma unroll 1
    for (int d = 1; d < kW; d <<= 1) {
      const int64_t o = __shfl_up_sync(0xffffffffu, w, d);
      if (lane >= d) w += o;
    }
    total = __shfl_sync(0xffffffffu, w, kW - 1);
    const int64_t before = __shfl_sync(0xffffffffu, w, warp > 0 ? warp - 1 : 0);
    return (warp > 0 ? before : 0) + s - v;
  };
  if (tid < 2) {
    cut[tid] = PagedCut{a.batch, 0, 0, 0, 0, 0, 0};
    where[tid] = -1;
  }
  int R = 0;   // blocks of rows so far
#pragma unroll 1
  for (int b0 = 0; b0 < a.batch; b0 += kThreads) {
    int64_t total;
    const int n = b0 + tid < a.batch ? Work::count(a, pgd::sequence(a, b0 + tid)) : 0;
    const int64_t before = scan(n, total);
    if (b0 + tid < a.batch) starts[b0 + tid] = R + (int)before;
    R += (int)total;
  }
  if (tid == 0) starts[a.batch] = R;
  __syncthreads();
  const int kv = a.pool.kv_heads;
  int64_t x[2];   // the cuts' places
  auto places = [&](int64_t all) -> bool {   // false: no work (the same for the whole CTA)
    int64_t used = win::quotient(all * kv, kThin);
    used = used < 1 ? 1 : (used < a.shares ? used : a.shares);
    if (share >= used || all == 0) return false;
#pragma unroll 1
    for (int e = 0; e < 2; e++) x[e] = win::quotient(all * kv * (share + e), used);
    return true;
  };
  // cut e, at z of block p's running sums, in Key head kvh
  auto put = [&](int e, const Place &p, int kvh, int64_t z) {
    int item = kvh * (starts[p.b + 1] - starts[p.b]) + p.ib;
    int block = pgd::cut_item(z - p.P, p.blocks, kStartCost, p.each, kLeast);
    if (block == p.blocks && block > 0) {
      item++;
      block = 0;
    }
    cut[e] = PagedCut{p.b, item, block, 0, 0, 0, 0};
  };
  int64_t all;
  if (R <= kThreads) {
    Place p = {};
    int64_t cost = 0;
    if (tid < R) {
      int hi = a.batch;   // starts[p.b] <= tid < starts[hi]
      while (hi - p.b > 1) {
        const int mid = (p.b + hi) >> 1;
        if (starts[mid] <= tid) p.b = mid;
        else hi = mid;
      }
      const pgd::Seq q = pgd::sequence(a, p.b);
      pgd::Keys keys;
      p.ib = tid - starts[p.b];
      p.blocks = Work::blocks_of(a, q, p.ib, keys);
      p.each = Work::each(q, p.ib);
      cost = p.cost();
    }
    p.P = scan(cost, all);
    if (!places(all)) return;
    if (tid < R) sum[tid] = p.P;
    if (tid == 0) sum[R] = all;
#pragma unroll 1
    for (int e = 0; e < 2; e++)
      if (x[e] >= kv * p.P && x[e] < kv * (p.P + cost)) where[e] = p.b;
    __syncthreads();
#pragma unroll 1
    for (int e = 0; e < 2; e++) {
      if (where[e] < 0) continue;   // the line's end
      const int64_t lo = sum[starts[where[e]]], head = sum[starts[where[e] + 1]] - lo, y = x[e] - kv * lo;
      const int kvh = (int)win::quotient(y, head);
      const int64_t z = lo + (y - kvh * head);
      if (z >= p.P && z < p.P + cost) put(e, p, kvh, z);
    }
    return;
  }
  const int per = (R + kThreads - 1) / kThreads, f0 = tid * per < R ? tid * per : R, f1 = f0 + per < R ? f0 + per : R;
  const int64_t mine = walk(a, starts, f0, f1, 0, INT64_MAX, -1).P, before = scan(mine, all);
  if (!places(all)) return;
#pragma unroll 1
  for (int e = 0; e < 2; e++) {
    const int64_t X = win::quotient(x[e], kv);
    if (X >= before && X < before + mine) where[e] = walk(a, starts, f0, f1, before, X, -1).b;
  }
  __syncthreads();
#pragma unroll 1
  for (int e = 0; e < 4; e++) {
    if (where[e >> 1] < 0) continue;   // the line's end
    const int s = starts[where[e >> 1] + (e & 1)];
    if (s >= f0 && s < f1) edge[e >> 1][e & 1] = walk(a, starts, f0, f1, before, INT64_MAX, s).P;
    if (s == R && tid == 0) edge[e >> 1][e & 1] = all;
  }
  __syncthreads();
#pragma unroll 1
  for (int e = 0; e < 2; e++) {
    if (where[e] < 0) continue;
    const int64_t lo = edge[e][0], head = edge[e][1] - lo, y = x[e] - kv * lo;
    const int kvh = (int)win::quotient(y, head);
    const int64_t z = lo + (y - kvh * head);
    if (z >= before && z < before + mine) put(e, walk(a, starts, f0, f1, before, z, -1), kvh, z);
  }
}

// Where one Query row's result goes (a whole item: out and lse, else the part's workspace).
struct RowOut {
  float *f32 = nullptr;
  uint16_t *bf16 = nullptr;
  float *lse = nullptr;
  int merge = 0;
  __device__ __forceinline__ void init(const PagedAttend &a, const volatile Piece &p, int share, int r) {   // r: row of the item
    if (p.place) {
      const int64_t pr = ((int64_t)share * 2 + p.place - 1) * kRows + r;
      f32 = a.part + pr * D;
      lse = a.part_lse + pr;
      merge = p.again;
      return;
    }
    const int i = (int)((uint32_t)(p.row0 + r) / (uint32_t)a.group), h = p.kvh * a.group + (p.row0 + r - i * a.group);
    const int64_t at = h * a.os.head + (int64_t)(p.first + i) * a.os.token;
    if (a.out_f32) f32 = (float *)a.out + at;
    else bf16 = (uint16_t *)a.out + at;
    if (a.lse) lse = a.lse + (int64_t)h * a.n + p.first + i;
    merge = a.merge;
  }
};

// A whole item made in several pieces has its result in its place: the warp's 32 rows from row r0 of the item on, of
// which `live` exist, go to where they belong.
__device__ __noinline__ void hand_over(const PagedAttend &a, const volatile Piece &p, int share, int r0, uint32_t live) {
  const int lane = threadIdx.x & 31;
  __syncwarp();
#pragma unroll 1
  for (int k = 0; k < 32; k++) {
    if (!((live >> k) & 1u)) continue;
    const int64_t pr = ((int64_t)share * 2 + p.place - 1) * kRows + r0 + k;
    const int r = p.row0 + r0 + k, i = (int)((uint32_t)r / (uint32_t)a.group), h = p.kvh * a.group + (r - i * a.group);
    const float L = a.part_lse[pr];
    pgd::finish4(a, p.first + i, h, 4 * lane, *(const float4 *)(a.part + pr * D + 4 * lane), L);
    __syncwarp();   // merging lanes have read the earlier log-sum-exp
    if (lane == 0) pgd::finish_lse(a, p.first + i, h, L);
  }
}

// A producer's unit of a stage: 16 keys (of one page) by 64 channels of Keys or Values, two rows a thread, 16
// channels of each: row lane / 4 and the eighth after it, channels 16 (lane % 4).  A quarter warp's 16-byte
// stores take two rows, one of even and one of odd number, so the swizzle puts them into eight bank groups.
// Of a CTA's 64 Keys by 128 channels and 128 Values by 64 channels, eight units each, a producer has three (or two).
template <int BITS>
struct Codes {
  uint32_t c[2][BITS / 2];
  uint32_t step[2];
};
template <int BITS>
struct Unit {
  static constexpr int kRowBytes = D * BITS / 8;
  static constexpr uint32_t kStage = (uint32_t)kBlk;   // bytes of a stage of either
  int key0, row;                // first key; this thread's row
  uint32_t code_at, step_at;    // bytes from the group's first row to this thread's row and channels
  uint32_t dst[2];              // shared addresses of the row's two chunks

  // Unit u (0..7) of the Values (val) or the Keys of CTA cr.
  __device__ __forceinline__ void place(uint32_t smem, bool val, int u, int cr, int lane) {
    static_assert(2 * kBlkH == kBlk, "");
    row = lane >> 2;
    const int g = val ? u : u >> 1, piece = lane & 3, ch = (val ? 64 * cr : 64 * (u & 1)) + 16 * piece;
    key0 = val ? 16 * g : BS * (g >> 1) + 32 * cr + 16 * (g & 1);
    code_at = (uint32_t)(row * kRowBytes + ch * BITS / 8);
    step_at = (uint32_t)(row * win::kSteps + ch / win::kGroup);
    const uint32_t at = smem + (val ? OFF_V : OFF_K + (uint32_t)(u & 1) * kBlkH) + (uint32_t)(16 * g + row) * 128u;
#pragma unroll
    for (int h = 0; h < 2; h++) dst[h] = at + (((2u * (uint32_t)piece + h) ^ ((uint32_t)row & 7u)) << 4);
  }
  // The table entry of the stage of keys v0 .. v0 + 127.
  __device__ __forceinline__ int look(const PagedAttend &a, const pgd::Keys &keys, const int32_t *table, int v0) const {
    const int v = v0 + key0;
    return v < keys.total ? __ldg(table + (keys.token(v) >> a.page_log2)) : 0;
  }
  // The codes of that stage, from page 0's codes and steps of the piece's Key head; rows past the last key get a step
  // of 0, which makes zeros of whatever codes.
  __device__ __forceinline__ void load(const PagedAttend &a, const pgd::Keys &keys, const uint8_t *codes, const uint8_t *steps, int v0,
                                       int entry, Codes<BITS> &p) const {
    const uint32_t rows = (uint32_t)a.pool.kv_heads << a.page_log2;   // of a page, all heads (at most 2^24)
    const int v = v0 + key0;
    const uint32_t page = (uint32_t)pgd::checked(a, entry), place = (uint32_t)keys.token(v) & ((1u << a.page_log2) - 1u);
    const uint8_t *c = codes + (uint64_t)page * (rows * (uint32_t)kRowBytes) + (place * (uint32_t)kRowBytes + code_at);
    const uint8_t *s = steps + (uint64_t)page * (rows * (uint32_t)win::kSteps) + (place * (uint32_t)win::kSteps + step_at);
#pragma unroll
    for (int k = 0; k < 2; k++) {
      p.step[k] = 0u;
      if (v + row + 8 * k < keys.total) {
        if (BITS == 8) {
          const uint4 x = __ldg((const uint4 *)(c + 8 * k * kRowBytes));
          p.c[k][0] = x.x; p.c[k][1] = x.y; p.c[k][2 % (BITS / 2)] = x.z; p.c[k][3 % (BITS / 2)] = x.w;
        } else {
          const uint2 x = __ldg((const uint2 *)(c + 8 * k * kRowBytes));
          p.c[k][0] = x.x; p.c[k][1] = x.y;
        }
        p.step[k] = __ldg(s + 8 * k * win::kSteps);
      }
    }
  }
  __device__ __forceinline__ void store(uint32_t stage, const Codes<BITS> &p, const win::Bases &bases) const {
#pragma unroll
    for (int k = 0; k < 2; k++) {
      uint32_t d[8];
      const win::Step st = win::step_of_byte<BITS>(p.step[k]);
      if (BITS == 8) {
#pragma unroll
        for (int u = 0; u < 4; u++) win::decode8(p.c[k][u % (BITS / 2)], st, bases, d[2 * u], d[2 * u + 1]);
      } else {
        uint32_t q[4];
        win::decode4(p.c[k][0], st, bases, q);
        d[0] = q[0]; d[1] = q[1]; d[2] = q[2]; d[3] = q[3];
        win::decode4(p.c[k][1], st, bases, q);
        d[4] = q[0]; d[5] = q[1]; d[6] = q[2]; d[7] = q[3];
      }
      const uint32_t at = stage * kStage + (uint32_t)k * 1024u;
      tc::sts128(dst[0] + at, make_uint4(d[0], d[1], d[2], d[3]));
      tc::sts128(dst[1] + at, make_uint4(d[4], d[5], d[6], d[7]));
    }
  }
};

// A wait of the whole warp with one answer (false: someone gave up): every branch goes by a vote, so that the
// warp is never seen to part.  Whether someone gave up is looked at only where there is something to wait for.
__device__ __forceinline__ bool meet(uint64_t *bar, uint32_t parity) {
  if (__all_sync(0xffffffffu, tc::mbar_try_wait_cluster(bar, parity))) return true;
  const uint64_t t0 = tc::globaltimer_ns();
  for (;;) {
    if (__all_sync(0xffffffffu, tc::mbar_try_wait_cluster(bar, parity))) return true;
    if (__any_sync(0xffffffffu, aborted() != 0 || tc::globaltimer_ns() - t0 > kWaitNs)) return false;
  }
}
// A value that all lanes hold, seen to be the warp's.
__device__ __forceinline__ uint32_t uniform(uint32_t v) { return __reduce_max_sync(0xffffffffu, v); }
// One lane's arrival, by predication.
__device__ __forceinline__ void arrive_one(uint32_t cluster_addr) {
  asm volatile(
      "{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\t@q mbarrier.arrive.shared::cluster.b64 _, [%0];\n\t}" ::"r"(cluster_addr)
      : "memory");
}

// The even CTA's MMAs of one piece: n steps, step t of tile x being number c_x + t and in stage g0 + .. of the
// share.  two: both tiles take the same 64 keys a step; else (short items) a half each of stage t.  (Compiled
// apart: chosen at every step they cost a tenth of it.)  False: someone gave up.
template <bool two>
__device__ __noinline__ bool multiply(uint32_t tmem, uint32_t smem, int steps, uint32_t stage0, uint32_t step0, uint32_t step1) {
  constexpr uint32_t idesc = tc::idesc_f16_f32(2 * BM, BS), idesc_pv = tc::idesc_f16_f32_bmn(2 * BM, D);
  constexpr uint16_t kBoth = 3;
  const uint32_t tm = uniform(tmem), s0 = uniform(smem), g0 = uniform(stage0), c0 = uniform(step0), c1 = uniform(step1);
  const int n = (int)uniform((uint32_t)steps);
  // descriptors' lower words: K-major ones with 1 in the place of the stride that they do not use
  const uint32_t dq = ((s0 + OFF_Q) >> 4) | 1u << 16, dk = ((s0 + OFF_K) >> 4) | 1u << 16;
  const uint32_t dv = ((s0 + OFF_V) >> 4) | (uint32_t)(kBlk >> 4) << 16;
  const int T = two ? n : (n + 1) >> 1;   // steps of tile 0
  auto stage_of = [&](int t) -> uint32_t { return g0 + (uint32_t)(two ? t >> 1 : t); };
  auto half_of = [&](int x, int t) { return two ? t & 1 : x; };
  auto begins = [&](int t) { return !two || !(t & 1); };
  auto ends = [&](int t) { return !two || (t & 1) || t + 1 == n; };
  auto there = [&](int t) { return two || 2 * t + 1 < n; };   // tile 1 has a step t
  auto nth = [&](int x, int t) -> uint32_t { return (x ? c1 : c0) + (uint32_t)t; };
  auto qk = [&](int x, int t) {
    const uint32_t ko = (stage_of(t) % kStages) * 2 * kBlkH + (uint32_t)half_of(x, t) * 32 * 128, u = nth(x, t);
    const uint32_t da = dq + (uint32_t)(two ? x * 2 * kBlk / 16 : 0), db = dk + ko / 16;
    const uint32_t d = tm + 128u * x + (u & 1u) * BS;
#pragma unroll
    for (int kk = 0; kk < D / 16; kk++)
      tc::mma2_ss_warp_lo<tc::kDescSw128Hi, tc::kDescSw128Hi>(d, da + (uint32_t)(((kk / 4) * kBlk + 32 * (kk % 4)) / 16),
                                                              db + (uint32_t)(((kk / 4) * kBlkH + 32 * (kk % 4)) / 16), idesc, kk > 0);
    tc::mma2_commit_warp(&bars.s_full[x][u & 1u], kBoth);
  };
  auto pv = [&](int x, int t) {
    const uint32_t vo = (stage_of(t) % kStages) * kBlk + (uint32_t)half_of(x, t) * BS * 128, u = nth(x, t);
    const uint32_t db = dv + vo / 16;
    const uint32_t pp = tm + 128u * x + (u & 1u) * BS;
#pragma unroll
    for (int kk = 0; kk < BS / 16; kk++)
      tc::mma2_ts_warp_lo<tc::kDescSw128Hi>(tm + 256u + 128u * x, pp + 8u * kk, db + (uint32_t)(2048 * kk / 16), idesc_pv,
                                            (t > 0 || kk > 0));
    tc::mma2_commit_warp(&bars.pv_done[x][u & 1u], kBoth);
  };
  auto keys_there = [&](int t) {   // the Keys and Values of step t (a stage's first step waits for it)
    const uint32_t g = stage_of(t);
    return !begins(t) || meet(&bars.full[g % kStages], (g / kStages) & 1u);
  };
  auto weights_there = [&](int x, int t) {
    const uint32_t u = nth(x, t);
    return meet(&bars.p_ready[x][u & 1u], (u >> 1) & 1u);
  };
  for (int t = 0; t < 2 && t < T; t++) {
    if (!keys_there(t)) return false;
    tc::fence_after_sync();
    qk(0, t);
    if (there(t)) qk(1, t);
  }
  for (int t = 0; t < T; t++) {
    if (!weights_there(0, t)) return false;
    tc::fence_after_sync();
    pv(0, t);
    if (t + 2 < T) {
      if (!keys_there(t + 2)) return false;
      tc::fence_after_sync();
      qk(0, t + 2);
    }
    if (there(t)) {
      if (!weights_there(1, t)) return false;
      tc::fence_after_sync();
      pv(1, t);
      if (t + 2 < T && there(t + 2)) qk(1, t + 2);
    }
    if (ends(t)) tc::mma2_commit_warp(&bars.empty[stage_of(t) % kStages], kBoth);   // (S precedes P V)
  }
  return true;
}

template <int BITS>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    paged_attend_kernel(const __grid_constant__ PagedAttend a) {
  extern __shared__ __align__(16) unsigned char smem_raw[];
  unsigned char *sm = smem_raw + ((1024u - (tc::smem_u32(smem_raw) & 1023u)) & 1023u);
  __shared__ PagedCut cut[2];
  __shared__ Piece pieces[2];
  __shared__ uint32_t tmem_base_sh;
  __shared__ float2 half_sums[BM];   // short items: maximum and sum of the second tile's rows
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const int share = (int)(blockIdx.x >> 1), cr = (int)tc::cluster_ctarank();

  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");   // the kernels behind this one may line up
  find_cuts(a, share, sm + OFF_K, cut);
  __syncthreads();
  const PagedCut begin = cut[0], end = cut[1];
  if (begin.b == a.batch || (begin.b == end.b && begin.item == end.item && begin.block == end.block)) {   // both CTAs
    if (tid == 0 && cr == 0) a.cuts[share] = PagedCut{a.batch, 0, 0, 0, 0, 0, 0};
    return;
  }
  if (warp == kMmaWarp) {
    if (lane == 0) {
      for (int i = 0; i < kStages; i++) {
        // this CTA's producer warps; in the even CTA also the odd one's last warp, which passes on that its
        // producers are done (a producer's own arrival in the peer would wait for its loads in flight)
        tc::mbar_init(&bars.full[i], kProdWarps + 1 - cr);
        tc::mbar_init(&bars.empty[i], 1);
      }
      for (int i = 0; i < 2; i++) {
        for (int k = 0; k < 2; k++) {
          tc::mbar_init(&bars.s_full[i][k], 1);
          tc::mbar_init(&bars.p_ready[i][k], 8);   // both CTAs' 4 softmax warps of tile i
          tc::mbar_init(&bars.pv_done[i][k], 1);
        }
        tc::mbar_init(&bars.told[i], 1);
        tc::mbar_init(&bars.heard[i], kSoftmaxWarps + kProdWarps + 1);
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
  auto begun = [&]() {   // both CTAs' barriers exist, and their tensor memory (the planning warp has a piece by then)
    __syncthreads();
    tc::cluster_sync();
    tc::fence_after_sync();
  };
  if (warp != kPlanWarp) begun();
  const uint32_t tmem = tmem_base_sh;

  // The share's piece number i is described in pieces[i & 1] (the whole warp; false: someone gave up), until this
  // warp says that it has read all it needs of it.
  auto hear = [&](int i) -> bool {
    if (__all_sync(0xffffffffu, tc::mbar_try_wait(&bars.told[i & 1], (i >> 1) & 1))) return true;
    if (!tc::mbar_wait(&bars.told[i & 1], (i >> 1) & 1, kWaitNs)) fail(a.status);
    return !__any_sync(0xffffffffu, aborted() != 0);
  };
  auto heard = [&](int i) {
    __syncwarp();
    if (lane == 0) tc::mbar_arrive(&bars.heard[i & 1]);
  };

  const uint32_t powers = tc::smem_u32(sm) + OFF_POWER;
  if (warp < kSoftmaxWarps) {
    // ======================= softmax (Query tile x, row = TMEM lane) =======================
    const int x = warp / 4, sub = warp % 4;
    const uint32_t lane_addr = (uint32_t)(32 * sub) << 16;
    const uint32_t tS0 = tmem + lane_addr + 128u * x, tO = tmem + lane_addr + 256u + 128u * x;
    const uint32_t p_ready0 = tc::mapa(tc::smem_u32(&bars.p_ready[x][0]), 0);
    const uint32_t q_full = tc::mapa(tc::smem_u32(&bars.q_full), 0);
    // this thread's piece of row tid / 16 of tile 0; 16 rows on is 2 KB further, the next tile 2 blocks
    const uint32_t q_dst = tc::smem_u32(sm) + OFF_Q + (uint32_t)((tid & 15) / 8) * kBlk +
                           tc::sw128_offset((uint32_t)tid >> 4, 8u * (tid & 7));
    uint32_t count = 0;   // steps of this tile so far
    for (int pi = 0;; pi++) {
      if (softmax_meet(!hear(pi))) break;
      // (read where they are needed, so that the steps' registers are the logits')
      const volatile Piece &p = pieces[pi & 1];
      if (p.done) break;
      const int key_of = p.j0 * BN + (p.brief ? x * BS : 0), key_step = p.brief ? 2 * BS : BS;
      const int mine_n = p.brief ? (p.steps + 1 - x) >> 1 : p.steps;   // steps of this tile
      pgd::Row mine{0, 0, 0};
      pgd::Everyone every{INT32_MAX, 0, 0};   // a warp without a row masks nothing (its logits are 0)
      {
        // ---- this CTA's two Query tiles -> shared memory, bf16 -> fp16: a tile's rows in flight together.  Both tiles'
        // MMAs of the last piece are done and its outputs have left this memory. ----
        const int rows = p.seq_rows, row_base = p.row0 + cr * BM;   // this CTA's row 0 of tile 0
        const int rr0 = tid >> 4;   // 16-byte piece tid % 16 of rows rr0, rr0 + 16, ...
        const uint16_t *qb = a.q + (int64_t)p.kvh * a.group * a.qs.head + (int64_t)p.first * a.qs.token + 8 * (tid & 15);
        // 16 rows on: 16 / group tokens and 16 % group heads, a token more where the heads run over
        const int step_i = 16 / a.group, step_h = 16 - step_i * a.group;
        const int64_t ahead = step_i * a.qs.token + step_h * a.qs.head, wrap = a.qs.token - a.group * a.qs.head;
        uint32_t top = 0u, small = 0u;   // the largest magnitudes, a NaN above all; passes in which this piece is below 1
#pragma unroll 1
        for (int y = 0; y < (p.brief ? 1 : NQT); y++) {   // (short items take tile 0's place alone)
          const int r = row_base + y * 2 * BM + rr0, i = (int)((uint32_t)r / (uint32_t)a.group);
          int h = r - i * a.group, left = rows - r < BM ? rows - r : BM;   // (may be negative)
          const uint16_t *src = qb + h * a.qs.head + i * a.qs.token;
          uint4 v[BM / 16];
#pragma unroll
          for (int k = 0; k < BM / 16; k++) {
            v[k] = make_uint4(0u, 0u, 0u, 0u);
            if (16 * k < left) v[k] = *(const uint4 *)src;
            h += step_h;
            src += ahead + (h >= a.group ? wrap : 0);
            h -= h >= a.group ? a.group : 0;
          }
          if (y == 0) {   // what this thread's row sees, while they are on their way
            pgd::Seq q;
            q.q0 = p.q0;
            q.s = win::Seq{p.len, a.sink, (int64_t)1 << 62, a.tpf, a.frames};
            const pgd::Keys keys{p.keys.ns, p.keys.skip, p.keys.total};
            const int w0 = row_base + (p.brief ? 0 : x * 2 * BM) + 32 * sub, mr = w0 + lane;   // this warp's first row
            if (w0 < rows) {
              mine.init(q.s, keys, mr < rows ? q.frame(a, mr) : -1);
              every.init(q.s, keys, q.frame(a, w0), q.frame(a, w0 + 31 < rows ? w0 + 31 : rows - 1));
            }
            // this warp's rows: two in each of 16 passes, pass 8 y + k those of tile y from 16 k on
            tc::sts32(powers + 4u * (uint32_t)((lane >> 1) * 16 + warp * 2 + (lane & 1)), 0u);
          }
#pragma unroll
          for (int k = 0; k < BM / 16; k++) {
            const uint32_t w[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
            uint32_t hw[4];
#pragma unroll
            for (int u = 0; u < 4; u++) hw[u] = tc::pack_f16x2(__uint_as_float(w[u] << 16), __uint_as_float(w[u] & 0xFFFF0000u));
            tc::sts128(q_dst + (uint32_t)y * 2u * kBlk + (uint32_t)k * 2048u, make_uint4(hw[0], hw[1], hw[2], hw[3]));
            const uint32_t m = win::max_abs_bf16x2(win::max_abs_bf16x2(w[0], w[1]), win::max_abs_bf16x2(w[2], w[3])) & 0x7FFF7FFFu;
            top = win::max_abs_bf16x2(top, m);
            small |= win::any_from_one(m) || 16 * k >= left ? 0u : 1u << (8 * y + k);
          }
        }
        if (win::any_beyond_fp16(top & 0x7FFF7FFFu)) qwm_dev_error(a.status, QWM_ERR_RANGE);
#pragma unroll
        for (int d = 1; d < 16; d <<= 1) small &= __shfl_xor_sync(0xffffffffu, small, d);   // of the whole row
        __syncwarp();
#pragma unroll 1
        for (uint32_t again = small | __shfl_xor_sync(0xffffffffu, small, 16); again; again &= again - 1u) {   // fetched once more
          const int pass = __ffs((int)again) - 1, y = pass >> 3, k = pass & 7;
          const bool here = (small >> pass) & 1u;
          const int rr = row_base + y * 2 * BM + 16 * k + (tid >> 4), i = (int)((uint32_t)rr / (uint32_t)a.group);
          uint4 v = make_uint4(0u, 0u, 0u, 0u);
          if (here) v = *(const uint4 *)(a.q + (p.kvh * a.group + (rr - i * a.group)) * a.qs.head + (int64_t)(p.first + i) * a.qs.token + 8 * (tid & 15));
          const uint32_t w[4] = {v.x, v.y, v.z, v.w};
          uint32_t m = win::max_abs_bf16x2(win::max_abs_bf16x2(w[0], w[1]), win::max_abs_bf16x2(w[2], w[3])) & 0x7FFF7FFFu;
          m = win::larger_half(m);
#pragma unroll
          for (int d = 1; d < 16; d <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, d));
          if (!here) continue;
          const uint32_t power = win::row_power(m);
          const float up = win::power_of_two((int)power);
          uint32_t hw[4];
#pragma unroll
          for (int u = 0; u < 4; u++) hw[u] = tc::pack_f16x2(__uint_as_float(w[u] << 16) * up, __uint_as_float(w[u] & 0xFFFF0000u) * up);
          tc::sts128(q_dst + (uint32_t)y * 2u * kBlk + (uint32_t)k * 2048u, make_uint4(hw[0], hw[1], hw[2], hw[3]));
          if ((tid & 15) == 0) tc::sts32(powers + 4u * (uint32_t)(pass * 16 + (tid >> 4)), power);
        }
        tc::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive_remote(q_full);
      }
      softmax_meet(false);   // the rows' powers
      const int power = (int)tc::lds32(powers + 4u * (uint32_t)((p.brief ? 0 : x * BM) + 32 * sub + lane));
      const float sl2 = win::logit_scale<BITS>(a.scale_log2, win::power_of_two(-power));
      const uint64_t sc2 = pk64(sl2, sl2);
      float m_used = -INFINITY;
      uint64_t acc = 0ull;   // the sum of the weights, each step's added as one: 1 / 64 of the additions to a large sum
      bool ok = true;
      for (int t = 0; t < mine_n; t++) {
        const uint32_t u = count + (uint32_t)t;
        const int v0 = key_of + t * key_step;
        const bool full = every.see(v0, v0 + BS);
        const uint32_t tS = tS0 + (u & 1u) * BS;
        if (!__all_sync(0xffffffffu, tc::mbar_try_wait(&bars.s_full[x][u & 1u], (u >> 1) & 1u))) {
          if (!tc::mbar_wait(&bars.s_full[x][u & 1u], (u >> 1) & 1u, kWaitNs)) fail(a.status);
          if (__any_sync(0xffffffffu, aborted() != 0)) { ok = false; break; }   // the whole warp
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
          for (int e = 0; e < 4; e++)
            mx[e] = tc::max3(mx[e], __uint_as_float(s[i + 2 * e]), __uint_as_float(s[i + 2 * e + 1]));
        const float m_new = fmaxf(m_used, fmaf(tc::max3(fmaxf(mx[0], mx[1]), mx[2], mx[3]), sl2, -win::kTopWeight));
        if (__any_sync(0xffffffffu, m_new > m_used + kRescaleThreshold)) {
          const float alpha = m_new == -INFINITY ? 1.f : tc::ex2_approx(m_used - m_new);
          const uint64_t a2 = pk64(alpha, alpha);
          acc = tc::fma2(acc, a2, 0ull);
          if (t > 0) {  // O of the earlier steps, once PV_x(t-1) has been added (PV_x(t) waits for this warp)
            const uint32_t b = u - 1u;
            if (!tc::mbar_wait(&bars.pv_done[x][b & 1u], (b >> 1) & 1u, kWaitNs)) fail(a.status);
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
        if (lane == 0) tc::mbar_arrive_remote(p_ready0 + 8u * (u & 1u));
      }
      count += (uint32_t)mine_n;
      float l = tc::f2lo(acc) + tc::f2hi(acc), part0 = 1.f, part1 = 0.f;   // what O_0 and O_1 count for
      if (p.brief) {   // every softmax warp comes here, whatever happened before
        if (x == 1) half_sums[tid & (BM - 1)] = make_float2(m_used, l);
        softmax_meet(false);
        if (x == 0) {
          const float2 o = half_sums[tid];
          const float m = fmaxf(m_used, o.x);
          part0 = m_used == -INFINITY ? 0.f : tc::ex2_approx(m_used - m);
          part1 = o.x == -INFINITY ? 0.f : tc::ex2_approx(o.x - m);
          l = fmaf(l, part0, o.y * part1);
          m_used = m;
        }
      }
      // every MMA of the piece is done: outputs may be read, and the Queries' memory written
      if (ok && !tc::mbar_wait(&bars.o_done, pi & 1, kWaitNs)) fail(a.status);
      ok = !__any_sync(0xffffffffu, !ok || aborted() != 0);
      if (ok && !(p.brief && x == 1)) {
        tc::fence_after_sync();
        float inv = l > 0.f ? win::kUnit<BITS> / l : 0.f, keep = 0.f;
        float L = l > 0.f ? m_used + log2f(l) : -INFINITY;
        const int r = cr * BM + (p.brief ? 0 : x * 2 * BM) + 32 * sub + lane;   // this thread's row of the item
        bool write = p.row0 + r < p.seq_rows;
        RowOut out;
        if (write) {
          out.init(a, p, share, r);
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
        // through the Queries' memory, so that the stores write whole rows: an 8 KB buffer per warp of 256
        // bytes a row (fp32: two halves), 16-byte pieces permuted by the row's low bits against bank conflicts
        const uint32_t buf = tc::smem_u32(sm) + OFF_Q + (uint32_t)warp * 8192u, rx = (uint32_t)lane & 7u;
        const bool half = !p.place && !a.out_f32;   // bf16 rows
        const float w0_out = part0 * inv, w1_out = part1 * inv;
        const uint32_t writes = __ballot_sync(0xffffffffu, write);
        const uint64_t mine_out = half ? (uint64_t)out.bf16 : (uint64_t)out.f32;
#pragma unroll 1
        for (int c = 0; c < D && writes; c += 32) {
          uint32_t o[32];
          tc::tmem_ld32(tO + c, o);
          tc::tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < 32; i++) o[i] = __float_as_uint(__uint_as_float(o[i]) * w0_out);
          if (p.brief && p.steps > 1) {   // (a single step left O_1 unwritten)
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
              for (int e = 0; e < 4; e++)
                w[e] = tc::pack_bf16x2(__uint_as_float(o[8 * v + 2 * e]), __uint_as_float(o[8 * v + 2 * e + 1]));
              tc::sts128(buf + (uint32_t)lane * 256u + ((((uint32_t)(c / 8 + v)) ^ rx) << 4), make_uint4(w[0], w[1], w[2], w[3]));
            }
          } else {
#pragma unroll
            for (int v = 0; v < 8; v++)
              tc::sts128(buf + (uint32_t)lane * 256u + ((((uint32_t)((c & 32) / 4 + v)) ^ rx) << 4),
                         make_uint4(o[4 * v], o[4 * v + 1], o[4 * v + 2], o[4 * v + 3]));
            if (c & 32) {   // 64 channels are there
              __syncwarp();
#pragma unroll 4
              for (int i = 0; i < 16; i++) {
                const int rw = 2 * i + (lane >> 4), e = lane & 15;
                float *dst = (float *)__shfl_sync(0xffffffffu, mine_out, rw) + (c - 32) + 4 * e;
                const float k = __shfl_sync(0xffffffffu, keep, rw);
                const uint4 v = tc::lds128(buf + (uint32_t)rw * 256u + ((uint32_t)(e ^ (rw & 7)) << 4));
                if ((writes >> rw) & 1u) {
                  float4 f = make_float4(__uint_as_float(v.x), __uint_as_float(v.y), __uint_as_float(v.z), __uint_as_float(v.w));
                  if (k > 0.f) {
                    const float4 g = *(const float4 *)dst;
                    f = make_float4(fmaf(k, g.x, f.x), fmaf(k, g.y, f.y), fmaf(k, g.z, f.z), fmaf(k, g.w, f.w));
                  }
                  *(float4 *)dst = f;
                }
              }
              __syncwarp();
            }
          }
        }
        if (p.whole) hand_over(a, p, share, r - lane, __ballot_sync(0xffffffffu, p.row0 + r < p.seq_rows));
        if (half && writes) {
          __syncwarp();
#pragma unroll 8
          for (int i = 0; i < 16; i++) {
            const int rw = 2 * i + (lane >> 4), c = lane & 15;
            uint16_t *dst = (uint16_t *)__shfl_sync(0xffffffffu, mine_out, rw);
            const uint4 v = tc::lds128(buf + (uint32_t)rw * 256u + ((uint32_t)(c ^ (rw & 7)) << 4));
            if ((writes >> rw) & 1u) *(uint4 *)(dst + 8 * c) = v;
          }
        }
      }
      tc::fence_before_sync();
      heard(pi);
      if (softmax_meet(!ok)) break;   // (behind it the Queries' memory and both outputs may be written again)
      tc::fence_after_sync();
    }
  } else if (warp == kMmaWarp) {
    // ======================= the even CTA's issues the pair's MMAs, the odd one's passes on that its CTA's stages
    // are full =======================
    // Everything that MMAs and loops depend on is reduced over the warp, whose lanes hold the same, and a failed
    // wait leaves all loops at once: where the compiler cannot see that the warp stays together, operands pass
    // through a register of each lane, 100 cycles an MMA.
    if (cr == 1) {
      const uint32_t full = tc::mapa(tc::smem_u32(&bars.full[0]), 0);
      uint32_t g = 0;   // stages so far
      for (int pi = 0;; pi++) {
        if (!meet(&bars.told[pi & 1], (uint32_t)(pi >> 1) & 1u)) goto failed;
        const Piece &p = pieces[pi & 1];
        const uint32_t done = uniform((uint32_t)p.done);
        const int J = (int)uniform((uint32_t)p.J);
        arrive_one(tc::smem_u32(&bars.heard[pi & 1]));
        if (done) break;
        for (int j = 0; j < J; j++, g++) {
          if (!meet(&bars.full[g & (kStages - 1)], (g / kStages) & 1u)) goto failed;
          arrive_one(full + 8u * (g & (kStages - 1)));
        }
      }
    } else {
      constexpr uint16_t kBoth = 3;
      const uint32_t tm = uniform(tmem), s0 = uniform(tc::smem_u32(sm));
      uint32_t stages = 0, steps0 = 0, steps1 = 0;   // so far; of tiles 0 and 1
      for (int pi = 0;; pi++) {
        if (!meet(&bars.told[pi & 1], (uint32_t)(pi >> 1) & 1u)) goto failed;
        const Piece &p = pieces[pi & 1];
        const uint32_t J = uniform((uint32_t)p.J), n = uniform((uint32_t)p.steps), brief = uniform((uint32_t)p.brief);
        const uint32_t done = uniform((uint32_t)p.done);
        arrive_one(tc::smem_u32(&bars.heard[pi & 1]));
        if (done) break;
        // (the phase by the piece's number: by a count of its own, the same, the prompt chunk takes 641 us instead of 597)
        if (!meet(&bars.q_full, (uint32_t)pi & 1u)) goto failed;
        tc::fence_after_sync();
        if (brief) {
          if (!multiply<false>(tm, s0, (int)n, stages, steps0, steps1)) goto failed;
          steps0 += (n + 1) >> 1;
          steps1 += n >> 1;
        } else {
          if (!multiply<true>(tm, s0, (int)n, stages, steps0, steps1)) goto failed;
          steps0 += n;
          steps1 += n;
        }
        stages += J;
        tc::mma2_commit_warp(&bars.o_done, kBoth);
      }
    }
    if (false) {
    failed:
      fail(a.status);
    }
    if (cr == 0) {
      tc::mma2_commit_warp(&bars.drain, 1);  // every MMA issued above completes before TMEM is released
      if (!tc::mbar_wait(&bars.drain, 0, kWaitNs)) qwm_dev_error(a.status, QWM_ERR_DEVICE_TIMEOUT);
    }
  } else if (warp == kPlanWarp) {
    // ======================= the pieces of the share =======================
    int b = begin.b, item = begin.item, from = begin.block, block = from, pi = 0;   // from: the share's first of the item
    bool first = true, more = true;
    while (more) {
      Piece p = {};
      p.done = 1;
      for (; b < a.batch; b++, item = from = block = 0) {   // the sequence of the next item
        const pgd::Seq q = pgd::sequence(a, b);
        const int n = Work::count(a, q);
        if (b > end.b || (b == end.b && (item > end.item || (item == end.item && end.block == 0)))) break;
        if (item >= n * a.pool.kv_heads) continue;
        const int kvh = item / n, ib = item - kvh * n;
        const int blocks = Work::blocks_of(a, q, ib, p.keys);
        const bool last = b == end.b && item == end.item;
        const int held = last ? end.block : blocks, block1 = held - block > kMost ? block + kMost : held;
        const bool whole = from == 0 && held == blocks, split = held - from > kMost;
        p.b = b;
        p.kvh = kvh;
        p.first = q.first;
        p.seq_rows = q.rows;
        p.row0 = ib * kRows;
        // (a whole item's pieces meet in the second place: the share's only part there is its last item's)
        p.place = from > 0 ? 1 : (whole && !split ? 0 : 2);
        p.again = block > from;
        p.whole = whole && split && block1 == held;
        p.j0 = block;
        p.J = block1 - block;
        const int to = p.keys.total < block1 * BN ? p.keys.total : block1 * BN;
        p.steps = (to - block * BN + BS - 1) / BS;
        p.brief = Work::brief(q, ib);
        p.q0 = q.q0;
        p.len = q.s.len;
        p.done = 0;
        if (first && lane == 0 && cr == 0)
          a.cuts[share] = PagedCut{b, item, block, q.first, kvh, p.row0, q.rows - p.row0 < kRows ? q.rows - p.row0 : kRows};
        first = false;
        block = block1;
        if (block1 == held) {
          item = last ? INT32_MAX : item + 1;   // (behind the last one everything lies past the end)
          from = block = 0;
        }
        break;
      }
      more = !p.done;
      if (pi == 0) begun();
      if (pi >= 2 && !__all_sync(0xffffffffu, tc::mbar_wait(&bars.heard[pi & 1], ((pi >> 1) - 1) & 1, kWaitNs))) {
        fail(a.status);
        break;
      }
      if (lane == 0) pieces[pi & 1] = p;
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&bars.told[pi & 1]);
      pi++;
    }
    if (first && lane == 0 && cr == 0) a.cuts[share] = PagedCut{a.batch, 0, 0, 0, 0, 0, 0};
  } else {
    // ======================= producers: three of them Keys, three Values =======================
    const int pw = warp - (warp > kPlanWarp ? 10 : 9), units = pw % 3 == 2 ? 2 : 3;   // 9, 10, 11, 13, 14, 15
    Unit<BITS> unit[3];
#pragma unroll
    for (int i = 0; i < 3; i++) unit[i].place(tc::smem_u32(sm), pw >= 3, i < units ? 3 * (pw % 3) + i : 0, cr, lane);
    Codes<BITS> even[3] = {}, odd[3] = {};
    uint32_t g0 = 0;
    bool ok = true;
    for (int pi = 0; ok; pi++) {
      ok = hear(pi);
      if (!ok) break;
      const volatile Piece &vp = pieces[pi & 1];
      if (vp.done) break;
      const int32_t *table = a.table + (int64_t)vp.b * a.width;
      const pgd::Keys keys{vp.keys.ns, vp.keys.skip, vp.keys.total};
      const int j0 = vp.j0, J = vp.J;
      const int64_t head_rows = (int64_t)vp.kvh << a.page_log2;
      const uint8_t *codes = (pw >= 3 ? a.pool.v_codes : a.pool.k_codes) + head_rows * Unit<BITS>::kRowBytes;
      const uint8_t *steps = (pw >= 3 ? a.pool.v_step : a.pool.k_step) + head_rows * win::kSteps;
      heard(pi);
      int entry[3];   // table entries of the next stage to be fetched
#pragma unroll
      for (int i = 0; i < 3; i++) entry[i] = unit[i].look(a, keys, table, j0 * BN);
      auto free_again = [&](uint32_t g) -> bool {   // the previous contents of stage g's place are consumed
        uint64_t *empty = &bars.empty[g & (kStages - 1)];
        if (g < kStages || __all_sync(0xffffffffu, tc::mbar_try_wait(empty, (g / kStages - 1) & 1u))) return true;
        if (!tc::mbar_wait(empty, (g / kStages - 1) & 1u, kWaitNs)) fail(a.status);
        return !__any_sync(0xffffffffu, aborted() != 0);         // warp-uniform exit
      };
      // stage j is stored and the codes of stage j + 2 fetched in its place; the first round only fetches
      auto stage = [&](int j, Codes<BITS> (&c)[3]) -> bool {
        const uint32_t g = g0 + (uint32_t)j, s = g & (kStages - 1);
        const int next = (j0 + j + 2) * BN;
        if (j >= 0 && j < J) {
          if (!free_again(g)) return false;
#pragma unroll
          for (int i = 0; i < 3; i++)
            if (i < units) unit[i].store(s, c[i], a.bases);
          tc::fence_proxy_async_smem();   // (waits for loads in flight, too: they stand behind it)
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(&bars.full[s]);
        }
        if (j + 2 < J) {
#pragma unroll
          for (int i = 0; i < 3; i++)
            if (i < units) unit[i].load(a, keys, codes, steps, next, entry[i], c[i]);
#pragma unroll
          for (int i = 0; i < 3; i++) entry[i] = unit[i].look(a, keys, table, next + BN);
        }
        return true;
      };
#pragma unroll 1
      for (int j = -2; j < J; j += 2)
        if (!stage(j, even) || !stage(j + 1, odd)) {
          ok = false;
          break;
        }
      g0 += (uint32_t)J;
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
cudaError_t launch_bits(const PagedAttend &a, cudaStream_t st) {
  static std::atomic<uint64_t> allowed{0};
  const cudaError_t e = allow_shared(paged_attend_kernel<BITS>, kSmemAlloc, allowed);
  if (e != cudaSuccess) return e;
  paged_attend_kernel<BITS><<<2 * a.shares, kThreads, kSmemAlloc, st>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_paged_tiles(const PagedAttend &a, cudaStream_t st) {
  return a.pool.bits == 8 ? launch_bits<8>(a, st) : launch_bits<4>(a, st);
}
