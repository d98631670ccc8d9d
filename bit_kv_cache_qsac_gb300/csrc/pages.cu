// Page tables on the device: sequences shortened, ended and extended, with a stack of free pages, and the
// position and slot of every row of a packed batch.
//
// The sequences' requests are scanned three times (rows, pages given up, pages needed); what is granted
// follows from the sums, so that nothing depends on the order in which threads run.  Every CTA of a cluster
// does the scans for itself (4,096 sequences at most, four a thread), and they share the rest: pages pushed,
// pages popped, rows, with a cluster barrier between.  Bound: latency, each of the three being a search in
// shared memory and one or two dependent accesses.  Measured: 64 sequences, a token each, 7.5 us; 256 prompts with 64,100
// rows 11.5 (in one CTA 7.5 and 34).
#include "paged.cuh"

namespace {

constexpr int kThreads = 1024, kCluster = 8, kPer = kPagedMaxBatch / kThreads;

struct Shared {
  int32_t kept[kPagedMaxBatch];        // tokens after shortening
  int32_t first[kPagedMaxBatch];       // packed row of the first new token (clamped to 2^31 - 1)
  int32_t granted[kPagedMaxBatch];
  int32_t dropped[kPagedMaxBatch];     // pages given up by the sequences before this one
  int32_t taken[kPagedMaxBatch];       // pages needed by the sequences before this one (clamped to pages)
  int64_t sums[kThreads / 32];
};

// Sum over the block's earlier threads, and over all.
__device__ __forceinline__ int64_t scan_before(int64_t v, int64_t *sums, int64_t &total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t s = v;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int64_t o = __shfl_up_sync(0xffffffffu, s, d);
    if (lane >= d) s += o;
  }
  __syncthreads();
  if (lane == 31) sums[warp] = s;
  __syncthreads();
  int64_t w = sums[lane];   // 32 warps
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int64_t o = __shfl_up_sync(0xffffffffu, w, d);
    if (lane >= d) w += o;
  }
  total = __shfl_sync(0xffffffffu, w, 31);
  const int64_t before = __shfl_sync(0xffffffffu, w, warp > 0 ? warp - 1 : 0);
  return (warp > 0 ? before : 0) + s - v;
}
// The last sequence whose entry is at most x (entries ascend, the first is 0).
__device__ __forceinline__ int last_at_most(const int32_t *v, int n, int x) {
  int lo = 0, hi = n;   // v[lo] <= x < v[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (v[mid] <= x) lo = mid;
    else hi = mid;
  }
  return lo;
}

__global__ void __launch_bounds__(kThreads) pages_update_kernel(const __grid_constant__ qwm_page_table t, int page_log2,
                                                                const int64_t *__restrict__ keep,
                                                                const int32_t *__restrict__ count, int n, int32_t *first,
                                                                int32_t *granted, int64_t *slot, int64_t *at,
                                                                int32_t *status) {
  extern __shared__ __align__(16) unsigned char raw[];
  Shared &sh = *(Shared *)raw;
  const int tid = threadIdx.x, rank = (int)tc::cluster_ctarank(), worker = rank * kThreads + tid;
  const int workers = kCluster * kThreads;
  const int per = (t.batch + kThreads - 1) / kThreads;   // sequences of a thread, neighbours
  const int64_t most = (int64_t)t.width << page_log2;
  auto pages_of = [&](int64_t tokens) -> int { return (int)((tokens + t.page - 1) >> page_log2); };
  int free0 = *t.free_count;
  free0 = free0 < 0 ? 0 : (free0 < t.pages ? free0 : t.pages);
  // ---- what each sequence asks for ----
  int kept[kPer], drop[kPer];
  int64_t want[kPer], rows = 0, drops = 0;
#pragma unroll
  for (int i = 0; i < kPer; i++) {
    kept[i] = drop[i] = 0;
    want[i] = 0;
    const int b = tid * per + i;
    if (i < per && b < t.batch) {
      int64_t len = t.length[b];
      if (len < 0 || len > most) {
        len = len < 0 ? 0 : most;
        qwm_dev_error(status, QWM_ERR_RANGE);
      }
      const int64_t k = keep ? keep[b] : len, c = count ? count[b] : 0;
      kept[i] = (int)(k < 0 ? 0 : (k < len ? k : len));
      drop[i] = pages_of(len) - pages_of(kept[i]);
      want[i] = c > 0 ? c : 0;
      rows += want[i];
      drops += drop[i];
    }
  }
  int64_t total, row = scan_before(rows, sh.sums, total), dropped_all;
  int64_t gone = scan_before(drops, sh.sums, dropped_all);
  // (a table that was not kept by these calls may give up more than the stack holds)
  const int dropped = (int)(dropped_all < t.pages - free0 ? dropped_all : t.pages - free0);
  const int64_t there = free0 + dropped;
  int64_t needs = 0, need[kPer];
  bool fits[kPer];
#pragma unroll
  for (int i = 0; i < kPer; i++) {
    need[i] = 0;
    fits[i] = false;
    const int b = tid * per + i;
    if (i < per && b < t.batch) {
      fits[i] = row + want[i] <= n && kept[i] + want[i] <= most;
      if (fits[i]) need[i] = pages_of(kept[i] + want[i]) - pages_of(kept[i]);
      sh.first[b] = (int)(row < INT32_MAX ? row : INT32_MAX);
      sh.dropped[b] = (int)(gone < INT32_MAX ? gone : INT32_MAX);
      sh.kept[b] = kept[i];
      row += want[i];
      gone += drop[i];
      needs += need[i];
    }
  }
  int64_t ask = scan_before(needs, sh.sums, total), taken = 0;
#pragma unroll
  for (int i = 0; i < kPer; i++) {
    const int b = tid * per + i;
    if (i < per && b < t.batch) {
      const bool ok = fits[i] && (need[i] == 0 || ask + need[i] <= there);
      sh.granted[b] = ok ? (int)want[i] : 0;
      sh.taken[b] = (int)(ask < there ? ask : there);
      ask += need[i];
      if (ok && need[i] > 0) taken = ask;
    }
  }
  // pages handed out: up to the last sequence that got any
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) {
    const int64_t o = __shfl_xor_sync(0xffffffffu, taken, d);
    taken = o > taken ? o : taken;
  }
  __syncthreads();
  if ((tid & 31) == 0) sh.sums[tid >> 5] = taken;
  __syncthreads();
  taken = sh.sums[tid & 31];
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) {
    const int64_t o = __shfl_xor_sync(0xffffffffu, taken, d);
    taken = o > taken ? o : taken;
  }
  // ---- pages given up, then pages handed out ----
  for (int j = worker; j < dropped; j += workers) {
    const int b = last_at_most(sh.dropped, t.batch, j);
    int32_t *entry = t.table + (int64_t)b * t.width + pages_of(sh.kept[b]) + (j - sh.dropped[b]);
    t.free_list[there - 1 - j] = *entry;
    *entry = -1;
  }
  if (dropped > 0) tc::cluster_sync();
  for (int j = worker; j < (int)taken; j += workers) {
    const int b = last_at_most(sh.taken, t.batch, j);
    int32_t *top = t.free_list + (there - 1 - j);
    t.table[(int64_t)b * t.width + pages_of(sh.kept[b]) + (j - sh.taken[b])] = __ldcg(top);
    *top = -1;
  }
  tc::cluster_sync();   // (every CTA has read the lengths, too)
  // ---- the sequences' new state, and the rows ----
  if (rank == 0) {
#pragma unroll
    for (int i = 0; i < kPer; i++) {
      const int b = tid * per + i;
      if (i < per && b < t.batch) {
        t.length[b] = kept[i] + sh.granted[b];
        if (first) first[b] = sh.first[b];
        if (granted) granted[b] = sh.granted[b];
      }
    }
    if (tid == 0) *t.free_count = (int)(there - taken);
  }
  for (int r = worker; r < n; r += workers) {
    const int b = last_at_most(sh.first, t.batch, r), i = r - sh.first[b];
    int64_t p = -1, s = -1;
    if (i < sh.granted[b]) {
      p = sh.kept[b] + i;
      s = ((int64_t)__ldcg(t.table + (int64_t)b * t.width + (p >> page_log2)) << page_log2) + (p & (t.page - 1));
      s = s < 0 ? -1 : s;
    }
    at[r] = p;
    slot[r] = s;
  }
}

__global__ void pages_reset_kernel(const __grid_constant__ qwm_page_table t) {
  const int64_t i0 = (int64_t)blockIdx.x * blockDim.x + threadIdx.x, step = (int64_t)gridDim.x * blockDim.x;
  for (int64_t i = i0; i < t.pages; i += step) t.free_list[i] = (int)(t.pages - 1 - i);
  for (int64_t i = i0; i < (int64_t)t.batch * t.width; i += step) t.table[i] = -1;
  for (int64_t i = i0; i < t.batch; i += step) t.length[i] = 0;
  if (i0 == 0) *t.free_count = t.pages;
}

}  // namespace

cudaError_t launch_pages_update(const qwm_page_table &t, int page_log2, const int64_t *keep, const int32_t *count, int64_t n,
                                int32_t *first, int32_t *granted, int64_t *slot, int64_t *at, int32_t *status, cudaStream_t st) {
  static std::atomic<uint64_t> allowed{0};
  const cudaError_t e = allow_shared(pages_update_kernel, (int)sizeof(Shared), allowed);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(kCluster);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = sizeof(Shared);
  cfg.stream = st;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = kCluster;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, pages_update_kernel, t, page_log2, keep, count, (int)n, first, granted, slot, at, status);
}

cudaError_t launch_pages_reset(const qwm_page_table &t, int num_sms, cudaStream_t st) {
  pages_reset_kernel<<<2 * num_sms, 256, 0, st>>>(t);
  return cudaGetLastError();
}
