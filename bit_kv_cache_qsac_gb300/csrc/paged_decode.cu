// Attention over a paged cache on warp tiles, for sequences with few new rows (single tokens, drafted tokens,
// grouped heads), and the joining of parts.
//
// A row r of a Key head is (token r / group, head r % group of the group); an item is one Key head of one
// sequence with up to 8 NT of its rows.  The work is bound by the cache's bytes and sequences differ in
// length, so it is shared out by the key: every CTA takes an equal piece of the line of all items
// (find_cuts).  An item that a cut goes through is computed in parts, which a second kernel joins.
// Inside a CTA an item's keys go to the 8 warps in turn, 16 or 32 at a time, copied to a ring of shared
// memory of the warp's own two steps ahead (cp.async; no barrier but the warp's) and multiplied on warp
// MMAs (warp_tile.cuh).  16 keys from a multiple of 16 lie in one page.  The copies run on into the share's next
// piece while a piece is joined and written.  A share's hold on an item of more than 2^18 keys is several pieces.
// Measured: a token of each of 64 sequences of 125 to 8,000 (8 bits, 8 Key heads): 94 us in all, 5.9 TB/s of its 550 MB; one
// token over 39,000 (4 bits, 40 heads): 60 us, where no unit is full (issue 62%, DRAM 47% of nominal).  Around the
// loops stand 8,000 cycles to the first step (4,000 of them the cuts) and 4,000 to 6,000 a piece (Queries, joining), 9,000 at
// 9 to 16 rows.  16 warps in one CTA an SM: 105 us and 61.5.
#include "paged.cuh"
#include "warp_tile.cuh"

namespace {

constexpr int D = win::D;
using wt::Ring;
constexpr int kWarps = wt::kWarps, kThreads = 32 * kWarps;
template <int BITS>
constexpr int kBlock = kWarps * wt::step_keys(BITS);   // keys that the 8 warps take at once
// What an item costs besides its keys, in blocks; the least piece of an item, and of the line, worth a start.
constexpr int kStart = 4, kLeast = 1, kThin = 4;
template <int BITS>
constexpr int kMost = kPagedPieceKeys / kBlock<BITS>;   // blocks of a piece

// The items of sequence b: blocks of keys of each, and how many (Key heads by blocks of 8 NT rows, all as long).
template <int BITS, int NT>
__device__ __forceinline__ int2 items_of(const PagedAttend &a, int b) {
  const pgd::Seq q = pgd::sequence(a, b);
  if (q.rows == 0 || q.rows > a.few) return make_int2(0, 0);
  pgd::Keys keys;
  keys.init(a, q.s, q.frame(a, 0), q.frame(a, q.rows - 1));
  return make_int2((keys.total + kBlock<BITS> - 1) / kBlock<BITS>, a.pool.kv_heads * ((q.rows + 8 * NT - 1) / (8 * NT)));
}

// The cuts of share `share` (begin, end) in the line of all items, found by the whole CTA.  Fewer shares are used when
// they would be shorter than kThin.  A share without work begins and ends at sequence `batch`.
template <int BITS, int NT>
__device__ __forceinline__ void find_cuts(const PagedAttend &a, int share, PagedCut (&cut)[2]) {
  __shared__ int64_t sums[kWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid < 2) cut[tid] = PagedCut{a.batch, 0, 0, 0, 0, 0, 0};
  int64_t x[2] = {INT64_MAX, INT64_MAX};
  // first the line's length, then the cuts' places; a batch of up to one sequence a thread is looked at once
  const bool once = a.batch <= kThreads;
  int2 w;
  int64_t mine = 0, upto = 0;
  auto scan = [&]() -> int64_t {   // upto: the sum of `mine` over the threads up to this one; the sum over all
    upto = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int64_t o = __shfl_up_sync(0xffffffffu, upto, d);
      if (lane >= d) upto += o;
    }
    __syncthreads();
    if (lane == 31) sums[warp] = upto;
    __syncthreads();
    int64_t total = 0;
#pragma unroll
    for (int k = 0; k < kWarps; k++) {
      const int64_t v = sums[k];
      upto += k < warp ? v : 0;
      total += v;
    }
    return total;
  };
  int64_t all = 0;
#pragma unroll 1
  for (int turn = 0; turn < (once ? 1 : 2); turn++) {
    int64_t base = 0;
#pragma unroll 1
    for (int b0 = 0; b0 < a.batch; b0 += kThreads) {
      w = make_int2(0, 0);
      if (b0 + tid < a.batch) w = items_of<BITS, NT>(a, b0 + tid);
      mine = (int64_t)w.y * (w.x + kStart);
      const int64_t total = scan();
      if (once || (turn == 0 && b0 + kThreads >= a.batch)) {   // the length is known
        all = base + total;
        int64_t used = win::quotient(all, kThin);
        used = used < 1 ? 1 : (used < a.shares ? used : a.shares);
        if (share >= used || all == 0) return;   // (the same for the whole CTA)
        x[0] = win::quotient(all * share, used);
        x[1] = win::quotient(all * (share + 1), used);
      }
      if (once || turn == 1) {
        const int64_t end = base + upto, begin = end - mine;
#pragma unroll 1
        for (int e = 0; e < 2; e++)
          if (x[e] >= begin && x[e] < end) {
            const int64_t y = x[e] - begin;
            int item = (int)win::quotient(y, w.x + kStart);
            int block = pgd::cut_item(y - (int64_t)item * (w.x + kStart), w.x, kStart, 1, kLeast);
            if (block == w.x && block > 0) {
              item++;
              block = 0;
            }
            cut[e] = PagedCut{b0 + tid, item, block, 0, 0, 0, 0};
          }
      }
      base += total;
    }
  }
}

// A piece of an item: blocks `block` .. block1 - 1 of its `blocks`, of which the share holds `from` .. to - 1.
struct Piece {
  int item, from, to, block, block1, blocks, kvh, row0, rows;   // rows: live ones from row0; 0: no piece
  int b, first, seq_rows, q0, len;                    // its sequence
  pgd::Keys keys;
  __device__ __forceinline__ pgd::Seq seq(const PagedAttend &a) const {
    pgd::Seq q;
    q.first = first;
    q.rows = seq_rows;
    q.q0 = q0;
    q.s = win::Seq{len, a.sink, (int64_t)1 << 62, a.tpf, a.frames};
    return q;
  }
};

template <int BITS, int NT>
__global__ void __launch_bounds__(kThreads, NT == 1 ? 2 : 1) paged_decode_kernel(const __grid_constant__ PagedAttend a) {
  using R = Ring<BITS>;
  constexpr int kKeys = R::kKeys, kSub = kKeys / 16;   // MMA rows of 16 keys in a step
  extern __shared__ __align__(16) unsigned char dyn_raw[];
  // stages start on 128-byte boundaries: permuted addresses are reached by flipping bits
  unsigned char *dyn = dyn_raw + ((128u - (tc::smem_u32(dyn_raw) & 127u)) & 127u);
  __shared__ float msm[kWarps][8 * NT], lsm[kWarps][8 * NT];
  __shared__ PagedCut cut[2];
  __shared__ Piece pieces[3];   // the share's pieces number s - 1 (being replaced), s and s + 1
  __shared__ int spare[kWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");   // the joining kernel may line up
  find_cuts<BITS, NT>(a, (int)blockIdx.x, cut);
  __syncthreads();

  // ---- the share's pieces, described by the last warp (which has the fewest steps) one ahead of their use ----
  int nb = cut[0].b, nitem = cut[0].item, nfrom = cut[0].block, nblock = nfrom;   // where the next one begins
  auto plan = [&](Piece &to) {
    Piece p = {};   // (no piece: no rows, and no steps for those who look ahead)
    const PagedCut end = cut[1];
    for (; nb < a.batch; nb++, nitem = nfrom = nblock = 0) {
      if (nb > end.b || (nb == end.b && (nitem > end.item || (nitem == end.item && end.block == 0)))) break;
      const pgd::Seq q = pgd::sequence(a, nb);
      const int tiles = q.rows > a.few ? 0 : (q.rows + 8 * NT - 1) / (8 * NT);
      if (nitem >= a.pool.kv_heads * tiles) continue;
      p.kvh = nitem / tiles;
      p.row0 = (nitem - p.kvh * tiles) * 8 * NT;
      p.rows = q.rows - p.row0 < 8 * NT ? q.rows - p.row0 : 8 * NT;
      p.keys.init(a, q.s, q.frame(a, 0), q.frame(a, q.rows - 1));
      p.blocks = (p.keys.total + kBlock<BITS> - 1) / kBlock<BITS>;
      p.item = nitem;
      p.from = nfrom;
      p.block = nblock;
      const bool last = nb == end.b && nitem == end.item;
      p.to = last ? end.block : p.blocks;
      p.block1 = p.to - p.block > kMost<BITS> ? p.block + kMost<BITS> : p.to;
      p.b = nb;
      p.first = q.first;
      p.seq_rows = q.rows;
      p.q0 = (int)q.q0;
      p.len = (int)q.s.len;
      nblock = p.block1;
      if (p.block1 == p.to) {
        nitem = last ? INT32_MAX : nitem + 1;   // (behind the last one everything lies past the end)
        nfrom = nblock = 0;
      }
      break;
    }
    if (lane == 0) to = p;
  };
  if (warp == kWarps - 1) plan(pieces[0]);
  __syncthreads();
  if (threadIdx.x == 0) {   // where the share begins, for the joining kernel
    const Piece &p = pieces[0];
    a.cuts[blockIdx.x] = p.rows ? PagedCut{p.b, p.item, p.block, p.first, p.kvh, p.row0, p.rows} : PagedCut{a.batch, 0, 0, 0, 0, 0, 0};
  }

  wt::Tile<BITS, NT> tile;
  tile.place(lane);
  auto fetch = [&](const Piece &p) {   // its Queries, bf16 for now
#pragma unroll
    for (int nt = 0; nt < NT; nt++) {
      const int r = p.row0 + 8 * nt + tile.g, i = (int)((uint32_t)r / (uint32_t)a.group);
      tile.fetch(nt, a.q + (p.kvh * a.group + (r - i * a.group)) * a.qs.head + (p.first + i) * a.qs.token, 8 * nt + tile.g < p.rows);
    }
  };
  // ---- copies into the warp's ring, a step (a group) each, across the pieces' borders: up to two steps on their way,
  // into the places behind `stage`, the next to be read; the third place is the one read last ----
  const uint32_t ring0 = tc::smem_u32(dyn) + (uint32_t)(warp * R::kStages * R::kStage);
  constexpr int kPer = R::kRow / 16, kCopies = kKeys * kPer / 32;   // pieces of a row; copies of a lane and tensor
  const uint32_t kdst = R::k_at(lane / kPer, lane & (kPer - 1));   // k_at(row + 32 / kPer, .) is 512 further on
  // v_at(row + 32 / kPer, .) is 512 further on but for the permutation: one piece bit flips per 4 rows
  const uint32_t vdst = R::v_at(lane / kPer, lane & (kPer - 1));
  auto vdst_of = [&](int i) -> uint32_t { return (vdst ^ (BITS == 8 ? 32u * (i & 3) : 64u * (i & 1))) + 512u * i; };
  const uint32_t page_rows = 1u << a.page_log2, head_rows = (uint32_t)a.pool.kv_heads << a.page_log2;   // (all heads': 2^24 at most)
  auto last_step = [&](const Piece &p) -> int {   // steps of an item that the piece ends with
    const int all = (p.keys.total + kKeys - 1) / kKeys;
    return p.block1 * kWarps < all ? p.block1 * kWarps : all;
  };
  int cj, cend;        // the next step to be copied of the piece that copies have come to, and its end
  int entry[kSub];     // the table's entries for that step
  // (what else is needed of the piece is read where it is needed: registers are the products')
  auto look = [&](const volatile Piece &p) {
    if (cj < cend) {
      const int total = p.keys.total, ns = p.keys.ns, skip = p.keys.skip;
      const int32_t *table = a.table + p.b * a.width;   // (4,096 sequences of 2^18 pages at most)
#pragma unroll
      for (int u = 0; u < kSub; u++) {   // each 16 keys; those past the last key repeat its 16
        const int v = cj * kKeys + 16 * u < total ? cj * kKeys + 16 * u : (total - 1) & -16;
        entry[u] = table[(v < ns ? v : v + skip) >> a.page_log2];
      }
    }
  };
  auto turn_to = [&](const Piece &p) {
    cj = p.block * kWarps + warp;
    cend = p.rows ? last_step(p) : 0;
    look(p);
  };
  int stage = 0, flying = 0;
  bool ahead = false;   // copies have come to the piece after the current one
  auto refill = [&](const Piece &now, const Piece &next, bool may_turn) {   // the current piece and the one after it
#pragma unroll 1
    while (flying < 2) {
      if (cj >= cend) {
        if (!may_turn || ahead) break;
        ahead = true;
        turn_to(next);
        if (cj >= cend) break;
      }
      const volatile Piece &p = ahead ? next : now;
      const int total = p.keys.total, ns = p.keys.ns, skip = p.keys.skip;
      const uint32_t chead = (uint32_t)p.kvh << a.page_log2;   // rows of a page before its Key head's
      const int place = stage + flying >= 3 ? stage + flying - 3 : stage + flying;
      const uint32_t dst = ring0 + (uint32_t)(place * R::kStage);
      const int v0 = cj * kKeys;
      const bool whole = v0 + kKeys <= total;
#pragma unroll
      for (int u = 0; u < kSub; u++) {
        // each 16 keys (those past the last key repeat its 16): page, and rows before them in it and its earlier heads
        const int v = whole || v0 + 16 * u < total ? v0 + 16 * u : (total - 1) & -16;
        const uint32_t page = (uint32_t)pgd::checked(a, entry[u]), row0 = chead + ((uint32_t)(v < ns ? v : v + skip) & (page_rows - 1u));
        const uint64_t at = (uint64_t)page * (head_rows * (uint32_t)R::kRow) + (row0 * (uint32_t)R::kRow + 16u * lane);
        const uint64_t step_at = (uint64_t)page * (head_rows * (uint32_t)win::kSteps) + (row0 + (lane & 15u)) * (uint32_t)win::kSteps;
        const uint8_t *kp = a.pool.k_codes + at, *vp = a.pool.v_codes + at, *sp = (lane < 16 ? a.pool.k_step : a.pool.v_step) + step_at;
        const uint32_t sdst = dst + (lane < 16 ? R::kKS : R::kVS) + 4u * ((lane & 15) + 16 * u);
        if (whole) {
#pragma unroll
          for (int i = 0; i < kCopies / kSub; i++) {
            const int c = u * (kCopies / kSub) + i;
            wt::cp_async16(dst + kdst + 512u * c, kp + 512 * i);
            wt::cp_async16(dst + vdst_of(c), vp + 512 * i);
          }
          wt::cp_async4(sdst, sp);   // lanes 0-15: the Keys' step words, 16-31: the Values'
        } else {   // rows past the last one repeat it
          const int follow = total - 1 - v;
#pragma unroll 1
          for (int i = 0; i < kCopies / kSub; i++) {
            const int c = u * (kCopies / kSub) + i, row = (32 * i + lane) / kPer, back = row > follow ? (row - follow) * R::kRow : 0;
            wt::cp_async16(dst + kdst + 512u * c, kp + 512 * i - back);
            wt::cp_async16(dst + vdst_of(c), vp + 512 * i - back);
          }
          wt::cp_async4(sdst, sp - ((lane & 15) > follow ? ((lane & 15) - follow) * win::kSteps : 0));
        }
      }
      tc::cp_async_commit();
      flying++;
      cj += kWarps;
      look(p);
    }
  };
  fetch(pieces[0]);
  turn_to(pieces[0]);
  refill(pieces[0], pieces[0], false);
  if (warp == kWarps - 1) plan(pieces[1]);
  __syncthreads();

  int now = 0;   // the current piece's place
  while (pieces[now].rows) {
    const int then = now == 2 ? 0 : now + 1;
    const Piece &p = pieces[now], &next = pieces[then];
    const int rows = p.rows, row0 = p.row0, jend = last_step(p), jbegin = p.block * kWarps + warp;
    const pgd::Keys keys{p.keys.ns, p.keys.skip, p.keys.total};
    pgd::Everyone every;
    {
      const pgd::Seq q = p.seq(a);
      every.init(q.s, keys, q.frame(a, row0), q.frame(a, row0 + rows - 1));
    }
    tile.begin(rows, a.scale_log2, a.status);
    auto mask_of = [&](int r) {
      const pgd::Seq q = pieces[now].seq(a);
      pgd::Row mask;
      mask.init(q.s, keys, r < rows ? q.frame(a, row0 + r) : -1);
      return mask;
    };
    for (int j = jbegin; j < jend; j += kWarps) {
      if (flying == 2) tc::cp_async_wait<1>();
      else tc::cp_async_wait<0>();
      __syncwarp();   // the step's copies are there, and the stage before it has been read by every lane
      const uint32_t st = ring0 + (uint32_t)(stage * R::kStage);
      stage = stage == 2 ? 0 : stage + 1;
      flying--;
      refill(p, next, true);
      tile.step(st, j * kKeys, every.see(j * kKeys, j * kKeys + kKeys), mask_of, a.bases);
    }
    refill(p, next, true);    // (a warp without a step in the piece has not turned yet; here every one has)
    ahead = false;

    // ---- the warps' parts joined: a warp's outputs go through the stage it has read last, the other two are on
    // their way for the next piece ----
    __syncwarp();
    const int mine = stage == 0 ? 2 : stage - 1;
    float (*osm)[D] = (float (*)[D])(dyn + (size_t)(warp * R::kStages + mine) * R::kStage);
    if (lane == 0) spare[warp] = mine;
    tile.sums(msm[warp], lsm[warp]);
    const bool part = p.from > 0 || p.block1 < p.blocks;
#pragma unroll
    for (int nt = 0; nt < NT; nt++) {
      if (8 * nt < rows) {
        if (nt) __syncthreads();
        tile.outputs(nt, rows, osm);
        if (nt == NT - 1 || 8 * (nt + 1) >= rows) fetch(next);   // the last of them: the registers take the next Queries
        __syncthreads();
        const int r = 8 * nt + warp, ch = 4 * lane;   // warp = row, lane = four channels
        if (r < rows) {
          float M, L;
          float4 acc = wt::join(msm, lsm, r, [&](int w) {
            return tile.output((const float (*)[D])(dyn + (size_t)(w * R::kStages + spare[w]) * R::kStage), warp, lane);
          }, M, L);
          const float inv = L > 0.f ? win::kUnit<BITS> / L : 0.f;
          float lse = L > 0.f ? M + log2f(L) : -INFINITY;
          acc = make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
          // an item's first part in the share's second place, any other in its first (a whole one in the second until
          // its last piece: the share's only part there is its last item's)
          const int64_t pr = ((int64_t)blockIdx.x * 2 + (p.from == 0 ? 1 : 0)) * 8 * NT + r;
          if (p.block > p.from) {   // joined with the pieces before it (of which this lane wrote these channels)
            const float Lp = a.part_lse[pr], Lm = fmaxf(Lp, lse);
            const float wp = Lp == -INFINITY ? 0.f : exp2f(Lp - Lm), wt = lse == -INFINITY ? 0.f : exp2f(lse - Lm), den = wp + wt;
            const float4 prev = *(const float4 *)(a.part + pr * D + ch);
            const float up = den > 0.f ? wp / den : 0.f, ut = den > 0.f ? wt / den : 0.f;
            acc = make_float4(fmaf(prev.x, up, acc.x * ut), fmaf(prev.y, up, acc.y * ut), fmaf(prev.z, up, acc.z * ut), fmaf(prev.w, up, acc.w * ut));
            lse = den > 0.f ? Lm + log2f(den) : -INFINITY;
            __syncwarp();   // every lane has read the earlier log-sum-exp
          }
          if (!part) {
            const int i = (row0 + r) / a.group, h = p.kvh * a.group + (row0 + r - i * a.group);
            pgd::finish4(a, p.first + i, h, ch, acc, lse);
            __syncwarp();   // merging lanes have read the earlier log-sum-exp
            if (lane == 0) pgd::finish_lse(a, p.first + i, h, lse);
          } else {
            *(float4 *)(a.part + pr * D + ch) = acc;
            if (lane == 0) a.part_lse[pr] = lse;
          }
        }
      }
    }
    if (warp == kWarps - 1) plan(pieces[then == 2 ? 0 : then + 1]);   // (it has the fewest rows, too)
    __syncthreads();
    now = then;
  }
  tc::cp_async_wait<0>();
  // launched beside the tile kernel: who waits for this one waits for both
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

// Parts of an item joined: the weighted mean of the parts' outputs, each weighted by its share of the
// exponential sum.  Per share whose beginning cuts an item first, blocks of 8 warps with ROWS rows a warp; the warp
// tiles' blocks (`few_blocks`) come first.  What depends on one another is three loads: the cuts behind this one and
// the one before it (a lane each), the parts' log-sum-exps (a lane each), the parts.
template <int ROWS>
__device__ __forceinline__ void combine(const PagedAttend &a, int at, int part_rows) {
  const int blocks = part_rows / (8 * ROWS), s = at / blocks + 1, lane = threadIdx.x & 31;
  const int r0 = (at % blocks * 8 + (threadIdx.x >> 5)) * ROWS;
  auto same = [&](const PagedCut &x, const PagedCut &y) { return x.b == y.b && x.item == y.item && x.block > 0; };
  const PagedCut c = a.cuts[s];
  const PagedCut near = a.cuts[s - 1 + lane < a.shares ? s - 1 + lane : a.shares - 1];
  if (c.block == 0 || r0 >= c.live) return;
  uint32_t inside = __ballot_sync(0xffffffffu, s - 1 + lane < a.shares && same(near, c));
  if (inside & 1u) return;   // an earlier cut of the item
  // parts: the second place of share s - 1, then the first places of the shares from s on
  int n = 1 + __ffs((int)~(inside >> 1)) - 1;
  if (n == 32)
    while (s - 1 + n < a.shares && same(a.cuts[s - 1 + n], c)) n++;
  auto place = [&](int k, int r) -> int64_t { return ((int64_t)(k == 0 ? 2 * (s - 1) + 1 : 2 * (s - 1 + k))) * part_rows + r; };
  float M[ROWS], mine[ROWS], L[ROWS];
  float4 acc[ROWS], x[2][ROWS];   // the first two parts (there are no fewer) beside the log-sum-exps
#pragma unroll
  for (int k = 0; k < 2; k++) {
#pragma unroll
    for (int i = 0; i < ROWS; i++)
      if (r0 + i < c.live) x[k][i] = __ldcg((const float4 *)(a.part + place(k, r0 + i) * D + 4 * lane));
  }
#pragma unroll
  for (int i = 0; i < ROWS; i++) mine[i] = lane < n && r0 + i < c.live ? a.part_lse[place(lane, r0 + i)] : -INFINITY;
#pragma unroll
  for (int i = 0; i < ROWS; i++) {
    M[i] = mine[i];
    for (int k = 32 + lane; k < n; k += 32) M[i] = fmaxf(M[i], r0 + i < c.live ? a.part_lse[place(k, r0 + i)] : -INFINITY);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) M[i] = fmaxf(M[i], __shfl_xor_sync(0xffffffffu, M[i], d));
    mine[i] = mine[i] == -INFINITY ? 0.f : exp2f(mine[i] - M[i]);   // this lane's part's weight
    L[i] = 0.f;
    acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  auto add = [&](int i, float wt, const float4 &v) {
    L[i] += wt;
    acc[i].x = fmaf(v.x, wt, acc[i].x);
    acc[i].y = fmaf(v.y, wt, acc[i].y);
    acc[i].z = fmaf(v.z, wt, acc[i].z);
    acc[i].w = fmaf(v.w, wt, acc[i].w);
  };
#pragma unroll
  for (int k = 0; k < 2; k++) {
#pragma unroll
    for (int i = 0; i < ROWS; i++) {
      const float wt = __shfl_sync(0xffffffffu, mine[i], k);
      if (r0 + i < c.live) add(i, wt, x[k][i]);
    }
  }
#pragma unroll 4
  for (int k = 2; k < n; k++) {
#pragma unroll
    for (int i = 0; i < ROWS; i++) {
      if (r0 + i >= c.live) break;
      float wt = __shfl_sync(0xffffffffu, mine[i], k & 31);
      if (k >= 32) {
        const float l = a.part_lse[place(k, r0 + i)];
        wt = l == -INFINITY ? 0.f : exp2f(l - M[i]);
      }
      add(i, wt, *(const float4 *)(a.part + place(k, r0 + i) * D + 4 * lane));
    }
  }
#pragma unroll
  for (int i = 0; i < ROWS; i++) {
    if (r0 + i >= c.live) break;
    const float inv = L[i] > 0.f ? 1.f / L[i] : 0.f, lse = L[i] > 0.f ? M[i] + log2f(L[i]) : -INFINITY;
    const int q = (int)((uint32_t)(c.row + r0 + i) / (uint32_t)a.group), h = c.kvh * a.group + (c.row + r0 + i - q * a.group);
    pgd::finish4(a, c.first + q, h, 4 * lane, make_float4(acc[i].x * inv, acc[i].y * inv, acc[i].z * inv, acc[i].w * inv), lse);
    __syncwarp();   // merging lanes have read the earlier log-sum-exp
    if (lane == 0) pgd::finish_lse(a, c.first + q, h, lse);
  }
}

constexpr int kManyRows = 2;   // a warp's rows of the tensor-memory tiles' parts

__global__ void __launch_bounds__(256)
    paged_combine_kernel(const __grid_constant__ PagedAttend few, const __grid_constant__ PagedAttend many, int few_rows,
                         int few_blocks) {
  asm volatile("griddepcontrol.wait;" ::: "memory");   // launched while the parts are computed: wait for them
  if ((int)blockIdx.x < few_blocks) combine<1>(few, (int)blockIdx.x, few_rows);
  else combine<kManyRows>(many, (int)blockIdx.x - few_blocks, kPagedTileRows);
}

template <int BITS, int NT>
cudaError_t decode_launch(const PagedAttend &a, bool beside, cudaStream_t st) {
  auto kernel = paged_decode_kernel<BITS, NT>;
  static std::atomic<uint64_t> allowed{0};
  const cudaError_t e = allow_shared(kernel, Ring<BITS>::kBytes, allowed);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)a.shares);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = Ring<BITS>::kBytes;
  cfg.stream = st;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = beside ? 1 : 0;   // it needs nothing of the tile kernel: its CTAs follow as SMs come free
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

}  // namespace

int paged_decode_shares(int row_tiles, int num_sms) { return (row_tiles == 1 ? 2 : 1) * num_sms; }

cudaError_t launch_paged_decode(const PagedAttend &a, int row_tiles, bool beside, cudaStream_t st) {
  if (row_tiles == 1) return a.pool.bits == 8 ? decode_launch<8, 1>(a, beside, st) : decode_launch<4, 1>(a, beside, st);
  return a.pool.bits == 8 ? decode_launch<8, 2>(a, beside, st) : decode_launch<4, 2>(a, beside, st);
}

// Launched as a dependent of the parts' kernels, so that its start-up overlaps their work.
cudaError_t launch_paged_combine(const PagedAttend *few, int part_rows, const PagedAttend *many, cudaStream_t st) {
  const int few_blocks = few ? (few->shares - 1) * (part_rows / 8) : 0;
  const int many_blocks = many ? (many->shares - 1) * (kPagedTileRows / (8 * kManyRows)) : 0;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(few_blocks + many_blocks));
  cfg.blockDim = dim3(256);
  cfg.stream = st;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, paged_combine_kernel, few ? *few : *many, many ? *many : *few, part_rows, few_blocks);
}
