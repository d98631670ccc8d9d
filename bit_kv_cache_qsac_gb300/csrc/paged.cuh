// Device code shared by the paged kernels: which tokens of a sequence its new rows see and where they
// lie, and how attention work is shared out over the CTAs.
#pragma once

#include "../../include/qwm_paged.h"
#include "window.cuh"

constexpr int kPagedMaxBatch = 4096;              // sequences of a page table
constexpr int64_t kPagedMaxTokens = 1 << 22;      // tokens of a sequence
// Keys of a piece at most.  Products are added to a piece's output 16 keys at a time, each addition off by up to 2^-23 of
// it (the tensor cores truncate), and weights below 2^-32 of its largest are lost.  Longer shares of an item are made in
// several pieces, each joined with those before it in the place of the item's part: 2^22 keys of one sequence held by one
// share came out up to 3.1% small (tiles of 512 rows; 1.5% of 256, 0.4% on warp tiles), in pieces 0.2%.
constexpr int kPagedPieceKeys = 1 << 18;

// An attention call over a paged cache, as its kernels take it.
struct PagedAttend {
  qwm_page_pool pool;
  const int32_t *table;
  const int64_t *length;
  int batch, width, page_log2;
  const uint16_t *q;
  qwm_strides qs;
  int n;                        // rows of the packed batch
  const int32_t *first, *count;
  int max_count;
  int64_t tpf, frames, sink;
  float scale_log2;             // softmax_scale * log2(e)
  void *out;
  qwm_strides os;
  int out_f32, merge;
  float *lse;
  int32_t *status;
  int group;                    // Query heads per Key head; row r of a Key head is (token r / group, head r % group)
  int few;                      // rows of a Key head up to which a sequence goes to the warp tiles
  int shares;                   // shares the work is cut into: CTAs, or CTA pairs
  struct PagedCut *cuts;        // [shares] where each share begins
  float *part;                  // [2 shares][part_rows][128] outputs of the parts of split items,
  float *part_lse;              // [2 shares][part_rows] their log-sum-exps
  win::Bases bases;             // win::kBases
};

// Where a share of the work begins: item `item` of sequence b, at key block `block` (0: not inside an item).
// Its rows: `live` from row `row` of Key head kvh of the sequence whose first token is packed row `first`.
struct PagedCut {
  int b, item, block, first, kvh, row, live;
};

// Warp tiles of 8 (row_tiles 1) or 16 rows (2).  beside: the tile kernel was launched just before it.
cudaError_t launch_paged_decode(const PagedAttend &a, int row_tiles, bool beside, cudaStream_t st);
int paged_decode_shares(int row_tiles, int num_sms);
// Tensor-memory tiles: items of kPagedTileRows rows, a CTA pair a share.
constexpr int kPagedTileRows = 512;
cudaError_t launch_paged_tiles(const PagedAttend &a, cudaStream_t st);
// Joins the parts of either kernel's split items, or both's (null: was not launched), part_rows rows each.
cudaError_t launch_paged_combine(const PagedAttend *few, int part_rows, const PagedAttend *many, cudaStream_t st);

namespace pgd {

// A sequence of an attention call: its rows, and the sequence as the masks see it.
struct Seq {
  int first, rows;     // packed row of its first token; rows of a Key head (0: left out)
  int64_t q0;          // position of its first row
  win::Seq s;
  __device__ __forceinline__ int64_t frame(const PagedAttend &a, int r) const { return s.frame(q0 + (uint32_t)r / (uint32_t)a.group); }
};
__device__ __forceinline__ Seq sequence(const PagedAttend &a, int b) {
  Seq q;
  const int count = a.count[b];
  const int64_t len = a.length[b];
  q.first = a.first[b];
  q.rows = 0;
  q.q0 = len - count;
  // (a window that never ends stands where the window cache has its ring)
  q.s = win::Seq{len, a.sink, (int64_t)1 << 62, a.tpf, a.frames};
  if (count <= 0 || q.first < 0 || q.first >= a.n || len < count) return q;
  if (len > (int64_t)a.width << a.page_log2 || count > a.max_count) {
    qwm_dev_error(a.status, QWM_ERR_RANGE);
    return q;
  }
  q.rows = (count < a.n - q.first ? count : a.n - q.first) * a.group;
  return q;
}

// The tokens that rows of frames f0 .. f1 (f0 <= f1) see between them, numbered in whole pages without the
// pages between the sinks and the window: key v is token v (v < ns) or v + skip.  The numbers of tokens in
// those pages that no row sees are masked like any other.
struct Keys {
  int ns, skip, total;
  __device__ __forceinline__ void init(const PagedAttend &a, const win::Seq &s, int64_t f0, int64_t f1) {
    const int page = 1 << a.page_log2;
    const int sinks = (int)s.sinks(f1), hi = (int)s.hi(f1), end = (sinks + page - 1) & -page;
    const int64_t lo = s.lo(f0);
    ns = INT32_MAX;
    skip = 0;
    total = sinks;
    if (hi > lo) {
      const int begin = (int)lo & -page;
      total = hi;
      if (begin > end) {
        ns = end;
        skip = begin - end;
        total = hi - skip;
      }
    }
  }
  __device__ __forceinline__ int token(int v) const { return v < ns ? v : v + skip; }
  // The number of a token of the window (or, past the last one, the number after it).
  __device__ __forceinline__ int number(int64_t token) const { return ns == INT32_MAX ? (int)token : (int)token - skip; }
};

// The keys that one row sees: 0 .. c0 - 1 and c1 .. c2 - 1.
struct Row {
  int c0, c1, c2;
  __device__ __forceinline__ void init(const win::Seq &s, const Keys &k, int64_t f) {
    c0 = c1 = c2 = 0;
    if (f < 0) return;
    c0 = (int)s.sinks(f);
    const int64_t l = s.lo(f), h = s.hi(f);
    if (h > l) {
      c1 = k.number(l);
      c2 = k.number(h);
    }
  }
  __device__ __forceinline__ bool sees(int v) const { return v < c0 || (v >= c1 && v < c2); }
};

// The keys that every row of frames f0 .. f1 sees: 0 .. e0 - 1 and e1 .. e2 - 1.
struct Everyone {
  int e0, e1, e2;
  __device__ __forceinline__ void init(const win::Seq &s, const Keys &k, int64_t f0, int64_t f1) {
    e0 = (int)s.sinks(f0);
    const int64_t l = s.lo(f1), h = s.hi(f0);
    e1 = e2 = 0;
    if (h > l && h > s.lo(f0) && s.hi(f1) > l) {
      e1 = k.number(l);
      e2 = k.number(h);
      if (e1 <= e0) e1 = 0;   // no gap after the sinks
    }
  }
  __device__ __forceinline__ bool see(int v0, int v1) const { return v1 <= e0 || (v0 >= e1 && v1 <= e2); }
};

// A table entry made safe: one outside the pool is read as page 0.
__device__ __forceinline__ int checked(const PagedAttend &a, int page) {
  if ((uint32_t)page < (uint32_t)a.pool.pages) return page;
  qwm_dev_error(a.status, QWM_ERR_RANGE);
  return 0;
}

// Where a row's output goes, and the final step of every path: write, or merge into what is there.
__device__ __forceinline__ void finish4(const PagedAttend &a, int token, int h, int ch, float4 o, float L) {
  const int64_t at = h * a.os.head + token * a.os.token + ch;
  if (a.out_f32) {
    float4 *dst = (float4 *)((float *)a.out + at);
    if (a.merge) {
      const float Lp = a.lse[(int64_t)h * a.n + token], Lm = fmaxf(Lp, L);
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
__device__ __forceinline__ void finish_lse(const PagedAttend &a, int token, int h, float L) {
  if (!a.lse) return;
  float *p = a.lse + (int64_t)h * a.n + token;
  if (a.merge) {
    const float Lp = *p, Lm = fmaxf(Lp, L);
    if (Lm == -INFINITY) return;
    L = Lm + log2f(exp2f(Lp - Lm) + exp2f(L - Lm));
  }
  *p = L;
}

}  // namespace pgd

// ------------------------------------------------------------------ how the work is shared out
// All items of the sequences an attention kernel takes stand in one line, by sequence, each as long as what its
// keys and its start and end cost.  Share i begins at i / shares of the line; a cut close to an item's border is
// moved there.  Every CTA works out its own two cuts in the same way (find_cuts), so nothing is written down
// beforehand.
namespace pgd {

// An item of `blocks` blocks of keys costs start + blocks * each.  Where place x (counted from the item's begin) cuts
// it: 0, a block at least `least` from both ends, or `blocks` (its end).
__device__ __forceinline__ int cut_item(int64_t x, int blocks, int start, int each, int least) {
  const int block = x < start ? 0 : (int)win::quotient(x - start, each);
  return block < least ? 0 : (blocks - block < least ? blocks : block);
}

}  // namespace pgd

// Launchers of the paged calls (each returns the launch's error).
cudaError_t launch_norm_rope(const qwm_rope_spec *spec, const uint16_t *x, const qwm_strides &xs, int batch, int heads,
                             int64_t n, const int64_t *start, const int64_t *at, const int32_t *pos, const float *weight,
                             int per_head, float eps, uint16_t *out, const qwm_strides &os, int num_sms, cudaStream_t st);
cudaError_t launch_pages_reset(const qwm_page_table &t, int num_sms, cudaStream_t st);
cudaError_t launch_pages_update(const qwm_page_table &t, int page_log2, const int64_t *keep, const int32_t *count, int64_t n,
                                int32_t *first, int32_t *granted, int64_t *slot, int64_t *at, int32_t *status, cudaStream_t st);
cudaError_t launch_paged_write(const qwm_page_pool &pool, int page_log2, const uint16_t *k, const qwm_strides &ks,
                               const uint16_t *v, const qwm_strides &vs, int64_t n, const int64_t *slot,
                               const qwm_rope_spec *rope, const int64_t *at, const int32_t *pos, int norm, const float *weight,
                               int per_head, float eps, int num_sms, int32_t *status, cudaStream_t st);
cudaError_t launch_paged_read(const qwm_page_pool &pool, int page_log2, const int64_t *slot, int64_t n, uint16_t *k_hat,
                              uint16_t *v_hat, int num_sms, int32_t *status, cudaStream_t st);
