// xlpk_pages_*: forking, reserving, trimming, compacting and copying the pages
// of a paged KV cache on the device (include/xlpk.h has the definitions).
//
// A call is a plan (one CTA: who keeps which page, which free pages are taken)
// and, where bytes move, an apply launch of many CTAs that copies pages and
// rewrites the table; it is set up while the plan runs.  The plan alone reads
// `refs` as they were, so fresh pages never depend on the order in which counts
// change.
//
// Bound (times on the device): small calls by the two launches (8 rows forked: 3.9 us),
// large ones by the bytes copied, each read and written once.  Copies use plain
// 16-byte loads, four in flight a thread and eight CTAs an SM: compacting 54 pages of
// 8.4 MB takes 165 us, of which the bytes are 140 at copy rate; 31 copies of a
// page filled to 40 of 64 positions, in runs of 10 KB, 55 us of 50 (4 to 16 loads
// and 2 to 8 CTAs: the same within 4% for whole pages, 4 to 57% slower for runs).
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <vector>

#include "../../include/xlpk.h"
#include "errors.h"

using namespace xlpk;

namespace {

constexpr int kMaxRows = 1024;
constexpr int kPlanThreads = 1024;   // one thread per table row
constexpr int kCopyThreads = 256;
constexpr int kCopyCtas = 8;         // per SM
constexpr int kCopyUnroll = 4;
constexpr int kSegment = kCopyThreads * kCopyUnroll * 16;   // bytes a CTA copies at a time
constexpr int kTableCols = 8;        // columns of one table block of the fork
constexpr int kListPairs = 480;      // page pairs in one launch's parameters

// ---- plan helpers (one CTA of kPlanThreads)

// Inclusive scan over the block; `total` is the block's sum.
__device__ int block_scan(int v, int* warp_sums, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int x = 1; x < 32; x <<= 1) {
    const int y = __shfl_up_sync(~0u, v, x);
    if (lane >= x) v += y;
  }
  __syncthreads();   // the last call's readers are done with warp_sums
  if (lane == 31) warp_sums[warp] = v;
  __syncthreads();
  if (warp == 0) {
    int s = warp_sums[lane];
    for (int x = 1; x < 32; x <<= 1) {
      const int y = __shfl_up_sync(~0u, s, x);
      if (lane >= x) s += y;
    }
    warp_sums[lane] = s;
  }
  __syncthreads();
  *total = warp_sums[31];
  return v + (warp ? warp_sums[warp - 1] : 0);
}

// Lists free pages with numbers >= *from, in order, until at least `need` (<= 1024) are
// listed or the pool ends: list[0 .. returned), at most need + 1023.  *from moves past
// what was looked at.
__device__ int list_free(const xlpk_page_pool& p, int* from, int* list, int need, int* warp_sums) {
  int have = 0;
  while (have < need && *from < p.n_pages) {
    const int i = *from + static_cast<int>(threadIdx.x);
    const int free_page = i < p.n_pages && p.refs_dev[i] == 0;
    int total;
    const int at = have + block_scan(free_page, warp_sums, &total) - 1;
    if (free_page) list[at] = i;
    have += total;
    *from += kPlanThreads;
  }
  __syncthreads();
  return have;
}

__device__ inline bool in_pool(const xlpk_page_pool& p, int page) { return page >= 0 && page < p.n_pages; }

// ---- fork

struct ForkPlan {       // int32 words in the workspace, rows entries each
  int* count;           // copies, or -1: the call does nothing
  int *children, *heir, *fresh, *full;   // by row (full: the row's full pages before the call)
  int *src, *dst, *filled;               // by copy
};
__host__ __device__ inline ForkPlan fork_plan_at(void* ws, int rows) {
  int* w = static_cast<int*>(ws);
  ForkPlan f;
  f.count = w;
  w += 4;
  f.children = w;
  f.heir = w + rows;
  f.fresh = w + 2 * rows;
  f.full = w + 3 * rows;
  f.src = w + 4 * rows;
  f.dst = w + 5 * rows;
  f.filled = w + 6 * rows;
  return f;
}

__global__ void __launch_bounds__(kPlanThreads) fork_plan_kernel(const xlpk_page_pool p, const int* parents, void* ws) {
  asm volatile("griddepcontrol.launch_dependents;");
  __shared__ int heir[kMaxRows], children[kMaxRows], lens[kMaxRows], list[2 * kPlanThreads], warp_sums[32];
  const ForkPlan f = fork_plan_at(ws, p.rows);
  const int r = threadIdx.x;
  const bool row = r < p.rows;
  if (*p.status_dev != XLPK_OK) {
    if (r == 0) *f.count = -1;
    return;
  }
  const int par = row ? parents[r] : -1, len = row ? p.seq_lens_dev[r] : 0;
  heir[r] = INT32_MAX;
  children[r] = 0;
  lens[r] = len;
  bool bad = par < -1 || par >= p.rows || len < 0 || len > static_cast<long long>(p.cols) * p.page_size;
  if (__syncthreads_or(bad)) {
    if (r == 0) *f.count = -1, *p.status_dev = XLPK_ERR_INVALID_ARG;
    return;
  }
  if (par >= 0) {
    atomicAdd(&children[par], 1);
    atomicMin(&heir[par], par == r ? -1 : r);   // -1: the row itself, before any other
  }
  __syncthreads();
  if (heir[r] < 0) heir[r] = r;
  __syncthreads();
  const int had = par >= 0 ? lens[par] : 0, filled = had % p.page_size;
  const bool needs = par >= 0 && heir[par] != r && filled > 0;
  int src = -1, copies;
  if (needs) src = p.page_table_dev[static_cast<long long>(par) * p.cols + had / p.page_size];
  const int k = block_scan(needs, warp_sums, &copies) - 1;
  bad = needs && !in_pool(p, src);
  const int any_bad = __syncthreads_or(bad);
  int from = 0;
  const int have = list_free(p, &from, list, copies, warp_sums);
  if (any_bad || have < copies) {
    if (r == 0) *f.count = -1, *p.status_dev = any_bad ? XLPK_ERR_INVALID_ARG : XLPK_ERR_OOM;
    return;
  }
  if (row) {
    int fresh = -1;
    if (needs) {
      fresh = list[k];
      p.refs_dev[fresh] = 1;
      f.src[k] = src;
      f.dst[k] = fresh;
      f.filled[k] = filled;
    }
    f.children[r] = children[r];
    f.heir[r] = heir[r];
    f.fresh[r] = fresh;
    f.full[r] = len / p.page_size;
    p.seq_lens_dev[r] = had;
  }
  if (r == 0) *f.count = copies;
}

// Copies bytes [at, at + kSegment) of a run: kCopyUnroll 16-byte loads of every thread are in flight before
// the first store.  `bytes` is a multiple of 16.
__device__ inline void copy_segment(uint8_t* dst, const uint8_t* src, long long at, long long bytes) {
  uint4 v[kCopyUnroll];
#pragma unroll
  for (int i = 0; i < kCopyUnroll; ++i) {
    const long long o = at + (threadIdx.x + i * kCopyThreads) * 16;
    if (o < bytes)
      asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                   : "=r"(v[i].x), "=r"(v[i].y), "=r"(v[i].z), "=r"(v[i].w)
                   : "l"(src + o));
  }
#pragma unroll
  for (int i = 0; i < kCopyUnroll; ++i) {
    const long long o = at + (threadIdx.x + i * kCopyThreads) * 16;
    if (o < bytes) *reinterpret_cast<uint4*>(dst + o) = v[i];
  }
}

__global__ void __launch_bounds__(kCopyThreads) fork_apply_kernel(const xlpk_page_pool p, const int* parents, void* ws,
                                                                  int table_blocks) {
  extern __shared__ int tile[];   // [rows][kTableCols]
  asm volatile("griddepcontrol.wait;" ::: "memory");   // the plan
  const ForkPlan f = fork_plan_at(ws, p.rows);
  const int copies = *f.count;
  if (copies < 0) return;
  if (static_cast<int>(blockIdx.x) < table_blocks) {
    // all rows of a few columns, read whole before any is written: rows trade places
    const int c0 = blockIdx.x * kTableCols, nc = min(kTableCols, p.cols - c0);
    for (int i = threadIdx.x; i < p.rows * nc; i += kCopyThreads)
      tile[i] = p.page_table_dev[static_cast<long long>(i / nc) * p.cols + c0 + i % nc];
    __syncthreads();
    for (int i = threadIdx.x; i < p.rows * nc; i += kCopyThreads) {
      const int r = i / nc, c = i % nc, col = c0 + c, par = parents[r];
      int e = -1;
      if (par >= 0) {
        const bool heir = f.heir[par] == r;
        if (col < f.full[par] || heir)
          e = tile[par * nc + c];
        else if (col == f.full[par])
          e = f.fresh[r];
      }
      p.page_table_dev[static_cast<long long>(r) * p.cols + col] = e;
      const int old = tile[i];
      if (in_pool(p, old)) {
        const int held = col < f.full[r] ? f.children[r] : f.children[r] > 0;
        if (held != 1) atomicAdd(p.refs_dev + old, held - 1);
      }
    }
    return;
  }
  const long long head = static_cast<long long>(p.page_size) * p.row_bytes, page = head * p.n_kv_heads;
  const long long segs = (head + kSegment - 1) / kSegment, per_copy = p.n_layers * 2ll * p.n_kv_heads * segs;
  for (long long u = blockIdx.x - table_blocks; u < copies * per_copy; u += gridDim.x - table_blocks) {
    const int k = static_cast<int>(u / per_copy);
    const long long w = u - k * per_copy, run = w / segs, plane = run / p.n_kv_heads;   // K and V of each layer
    uint8_t* pool = static_cast<uint8_t*>(plane & 1 ? p.v_dev : p.k_dev) + (plane >> 1) * p.n_pages * page +
                    (run - plane * p.n_kv_heads) * head;
    copy_segment(pool + f.dst[k] * page, pool + f.src[k] * page, (w - run * segs) * kSegment,
                 static_cast<long long>(f.filled[k]) * p.row_bytes);
  }
}

// ---- reserve

__global__ void __launch_bounds__(kPlanThreads) reserve_kernel(const xlpk_page_pool p, const int* want_dev) {
  __shared__ int list[2 * kPlanThreads], warp_sums[32];
  const int r = threadIdx.x;
  const bool row = r < p.rows;
  if (*p.status_dev != XLPK_OK) return;
  const long long cap = static_cast<long long>(p.cols) * p.page_size;
  const int len = row ? p.seq_lens_dev[r] : 0, want = row ? want_dev[r] : 0;
  const int bad = __syncthreads_or(len < 0 || len > cap), full = __syncthreads_or(want > cap);
  if (bad || full) {
    if (r == 0) *p.status_dev = bad ? XLPK_ERR_INVALID_ARG : XLPK_ERR_KV_FULL;
    return;
  }
  int* mine = p.page_table_dev + static_cast<long long>(r) * p.cols;
  const int end = want > len ? (want - 1) / p.page_size + 1 : 0;
  int col = len / p.page_size, lack = 0;
  for (int j = col; j < end; ++j) lack += !in_pool(p, mine[j]);
  int total, free_pages = 0;
  const int last = block_scan(lack, warp_sums, &total);   // this row takes ranks [last - lack, last)
  if (total == 0) return;
  for (int i = r; i < p.n_pages; i += kPlanThreads) free_pages += p.refs_dev[i] == 0;
  int all_free;
  block_scan(free_pages, warp_sums, &all_free);
  if (all_free < total) {
    if (r == 0) *p.status_dev = XLPK_ERR_OOM;
    return;
  }
  int rank = last - lack, from = 0;
  for (int base = 0; base < total;) {
    const int have = list_free(p, &from, list, min(total - base, kPlanThreads), warp_sums);
    while (rank < last && rank < base + have) {
      while (in_pool(p, mine[col])) ++col;
      mine[col++] = list[rank - base];
      p.refs_dev[list[rank - base]] = 1;
      ++rank;
    }
    base += have;
    __syncthreads();   // the list is taken before the next stretch overwrites it
  }
}

// ---- trim

__global__ void __launch_bounds__(kCopyThreads) trim_kernel(const xlpk_page_pool p, int window, int sinks) {
  const long long cap = static_cast<long long>(p.cols) * p.page_size;
  // Every CTA looks at all lengths and comes to the same answer; the first says it.  (It may do so while
  // others still read the status: one that some of a CTA's threads see set stops all of them, none early,
  // so that no thread's lengths go unlooked at.)
  const bool stopped = *p.status_dev != XLPK_OK;
  bool bad = false;
  for (int r = threadIdx.x; r < p.rows; r += kCopyThreads) bad |= p.seq_lens_dev[r] < 0 || p.seq_lens_dev[r] > cap;
  if (__syncthreads_or(stopped)) return;
  if (__syncthreads_or(bad)) {
    if (blockIdx.x == 0 && threadIdx.x == 0) *p.status_dev = XLPK_ERR_INVALID_ARG;
    return;
  }
  const long long n = static_cast<long long>(p.rows) * p.cols, step = static_cast<long long>(gridDim.x) * kCopyThreads;
  for (long long i = blockIdx.x * static_cast<long long>(kCopyThreads) + threadIdx.x; i < n; i += step) {
    const int r = static_cast<int>(i / p.cols);
    const long long j = i - static_cast<long long>(r) * p.cols;
    const int e = p.page_table_dev[i];
    if (in_pool(p, e) && (j + 1) * p.page_size <= static_cast<long long>(p.seq_lens_dev[r]) - window &&
        j * p.page_size >= sinks) {
      p.page_table_dev[i] = -1;
      atomicSub(p.refs_dev + e, 1);
    }
  }
}

// ---- compact

struct CompactPlan {
  int* count;          // moves, or -1
  int *dst, *src;      // n_pages / 2 + 1 entries
  int* remap;          // n_pages entries
};
__host__ __device__ inline CompactPlan compact_plan_at(void* ws, int n_pages) {
  int* w = static_cast<int*>(ws);
  return {w, w + 4, w + 4 + (n_pages / 2 + 1), w + 4 + 2 * (n_pages / 2 + 1)};
}

__global__ void __launch_bounds__(kPlanThreads) compact_plan_kernel(const xlpk_page_pool p, int* remap_dev, void* ws) {
  asm volatile("griddepcontrol.launch_dependents;");
  __shared__ int warp_sums[32];
  const CompactPlan c = compact_plan_at(ws, p.n_pages);
  int* remap = remap_dev ? remap_dev : c.remap;
  if (*p.status_dev != XLPK_OK) {   // nothing moves: every live page keeps its number
    for (int i = threadIdx.x; i < p.n_pages; i += kPlanThreads) remap[i] = p.refs_dev[i] > 0 ? i : -1;
    if (threadIdx.x == 0) *c.count = -1;
    return;
  }
  int mine = 0, live;
  for (int i = threadIdx.x; i < p.n_pages; i += kPlanThreads) mine += p.refs_dev[i] > 0;
  block_scan(mine, warp_sums, &live);
  int holes = 0, highs = 0;
  for (int i0 = 0; i0 < p.n_pages; i0 += kPlanThreads) {
    const int i = i0 + threadIdx.x;
    const bool used = i < p.n_pages && p.refs_dev[i] > 0;
    const int hole = i < live && !used, high = i >= live && used;
    int total;
    const int both = block_scan(hole | high << 16, warp_sums, &total);
    if (hole) c.dst[holes + (both & 0xffff) - 1] = i;
    if (high) c.src[highs + (both >> 16) - 1] = i;
    if (i < p.n_pages) remap[i] = used ? i : -1;
    holes += total & 0xffff;
    highs += total >> 16;
  }
  __syncthreads();
  for (int k = threadIdx.x; k < highs; k += kPlanThreads) {   // as many holes as high pages
    const int s = c.src[k], d = c.dst[k];
    remap[s] = d;
    p.refs_dev[d] = p.refs_dev[s];
    p.refs_dev[s] = 0;
  }
  if (threadIdx.x == 0) *c.count = highs;
}

__device__ inline void copy_pages(const xlpk_page_pool& p, int n, const int* src, const int* dst, int block, int blocks) {
  const long long page = static_cast<long long>(p.page_size) * p.row_bytes * p.n_kv_heads;
  const long long segs = (page + kSegment - 1) / kSegment, per_page = segs * p.n_layers * 2;
  for (long long u = block; u < n * per_page; u += blocks) {
    const int k = static_cast<int>(u / per_page);
    const long long w = u - k * per_page, plane = w / segs;
    uint8_t* pool = static_cast<uint8_t*>(plane & 1 ? p.v_dev : p.k_dev) + (plane >> 1) * p.n_pages * page;
    copy_segment(pool + dst[k] * page, pool + src[k] * page, (w - plane * segs) * kSegment, page);
  }
}

__global__ void __launch_bounds__(kCopyThreads) compact_apply_kernel(const xlpk_page_pool p, const int* remap_dev,
                                                                     void* ws, int table_blocks) {
  asm volatile("griddepcontrol.wait;" ::: "memory");   // the plan
  const CompactPlan c = compact_plan_at(ws, p.n_pages);
  const int n = *c.count;
  if (n < 0) return;
  const int* remap = remap_dev ? remap_dev : c.remap;
  if (static_cast<int>(blockIdx.x) < table_blocks) {
    const long long all = static_cast<long long>(p.rows) * p.cols, step = static_cast<long long>(table_blocks) * kCopyThreads;
    for (long long i = blockIdx.x * static_cast<long long>(kCopyThreads) + threadIdx.x; i < all; i += step) {
      const int e = p.page_table_dev[i];
      if (in_pool(p, e)) p.page_table_dev[i] = remap[e];
    }
    return;
  }
  copy_pages(p, n, c.src, c.dst, blockIdx.x - table_blocks, gridDim.x - table_blocks);
}

// ---- copy

struct PagePairs {
  int n;
  int src[kListPairs], dst[kListPairs];
};

__global__ void __launch_bounds__(kCopyThreads) copy_kernel(const xlpk_page_pool p, const __grid_constant__ PagePairs l) {
  if (*p.status_dev != XLPK_OK) return;
  copy_pages(p, l.n, l.src, l.dst, blockIdx.x, gridDim.x);
}

// ---- host

xlpk_status check_pool(const xlpk_page_pool* p) {
  if (!p) return refuse(XLPK_ERR_INVALID_ARG, "xlpk_pages: no pool");
  if (p->n_layers < 1 || p->n_pages < 1 || p->n_kv_heads < 1 || p->page_size < 1 || p->rows < 1 || p->cols < 1 ||
      p->row_bytes < 16 || p->row_bytes % 16)
    return refuse(XLPK_ERR_INVALID_ARG, "xlpk_pages: a size is not positive, or row_bytes not a multiple of 16");
  if (p->rows > kMaxRows) return refuse(XLPK_ERR_UNSUPPORTED, "xlpk_pages: more than 1024 rows");
  // (indexes run past their end by up to a CTA's threads)
  if (p->n_pages > 1 << 30 || p->cols > 1 << 30) return refuse(XLPK_ERR_UNSUPPORTED, "xlpk_pages: more than 2^30 pages or columns");
  if (static_cast<int64_t>(p->cols) * p->page_size > INT32_MAX)
    return refuse(XLPK_ERR_UNSUPPORTED, "xlpk_pages: a table row of 2^31 positions or more");
  if (!p->k_dev || !p->v_dev || !p->page_table_dev || !p->seq_lens_dev || !p->refs_dev || !p->status_dev)
    return refuse(XLPK_ERR_INVALID_ARG, "xlpk_pages: a pointer is missing");
  if (!aligned(p->k_dev, 16) || !aligned(p->v_dev, 16) || !aligned(p->page_table_dev, 4) || !aligned(p->seq_lens_dev, 4) ||
      !aligned(p->refs_dev, 4) || !aligned(p->status_dev, 4))
    return refuse(XLPK_ERR_INVALID_ARG, "xlpk_pages: a pointer is not aligned");
  return XLPK_OK;
}

// A launch that may be set up while the one before it runs; the kernel waits for its end.
template <class... K, class... A>
xlpk_status launch_after(void (*kernel)(K...), int blocks, int smem, cudaStream_t st, A... args) {
  cudaLaunchConfig_t c{};
  c.gridDim = dim3(blocks);
  c.blockDim = dim3(kCopyThreads);
  c.dynamicSmemBytes = smem;
  c.stream = st;
  cudaLaunchAttribute early{};
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  c.attrs = &early;
  c.numAttrs = 1;
  XLPK_CUDA(cudaLaunchKernelEx(&c, kernel, static_cast<K>(args)...));
  return XLPK_OK;
}

xlpk_status check_workspace(const xlpk_page_pool* p, const void* ws, int64_t bytes) {
  if (!ws || !aligned(ws, 16) || bytes < xlpk_pages_workspace(p))
    return refuse(XLPK_ERR_INVALID_ARG, "xlpk_pages: workspace missing, unaligned or too small");
  return XLPK_OK;
}

}  // namespace

#define XLPK_TRY(call)                     \
  do {                                     \
    const xlpk_status st_ = (call);        \
    if (st_ != XLPK_OK) return st_;        \
  } while (0)

extern "C" {

int64_t xlpk_pages_workspace(const xlpk_page_pool* p) {
  if (!p || p->rows < 1 || p->n_pages < 1) return 0;
  const int64_t fork = 4 + 7ll * p->rows, compact = 4 + 2ll * (p->n_pages / 2 + 1) + p->n_pages;
  return std::max(fork, compact) * 4;
}

xlpk_status xlpk_pages_fork(const xlpk_page_pool* p, const int32_t* parents_dev, void* ws, int64_t ws_bytes, void* stream) {
  XLPK_TRY(check_pool(p));
  XLPK_TRY(check_workspace(p, ws, ws_bytes));
  if (!parents_dev || !aligned(parents_dev, 4)) return refuse(XLPK_ERR_INVALID_ARG, "xlpk_pages_fork: parents");
  int sms = 0;
  XLPK_TRY(current_sms(&sms));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  fork_plan_kernel<<<1, kPlanThreads, 0, st>>>(*p, parents_dev, ws);
  XLPK_CUDA(cudaGetLastError());
  const int table_blocks = (p->cols + kTableCols - 1) / kTableCols;
  return launch_after(fork_apply_kernel, table_blocks + sms * kCopyCtas, p->rows * kTableCols * 4, st, *p, parents_dev, ws,
                      table_blocks);
}

xlpk_status xlpk_pages_reserve(const xlpk_page_pool* p, const int32_t* want_dev, void* stream) {
  XLPK_TRY(check_pool(p));
  if (!want_dev || !aligned(want_dev, 4)) return refuse(XLPK_ERR_INVALID_ARG, "xlpk_pages_reserve: want");
  int sms = 0;
  XLPK_TRY(current_sms(&sms));
  reserve_kernel<<<1, kPlanThreads, 0, static_cast<cudaStream_t>(stream)>>>(*p, want_dev);
  XLPK_CUDA(cudaGetLastError());
  return XLPK_OK;
}

xlpk_status xlpk_pages_trim(const xlpk_page_pool* p, int32_t window, int32_t sinks, void* stream) {
  XLPK_TRY(check_pool(p));
  if (window < 0 || sinks < 0) return refuse(XLPK_ERR_INVALID_ARG, "xlpk_pages_trim: window or sinks is negative");
  int sms = 0;
  XLPK_TRY(current_sms(&sms));
  if (window == 0) return XLPK_OK;
  const long long n = static_cast<long long>(p->rows) * p->cols;
  const int blocks = static_cast<int>(std::min<long long>(sms * 4, (n + kCopyThreads - 1) / kCopyThreads));
  trim_kernel<<<blocks, kCopyThreads, 0, static_cast<cudaStream_t>(stream)>>>(*p, window, sinks);
  XLPK_CUDA(cudaGetLastError());
  return XLPK_OK;
}

xlpk_status xlpk_pages_compact(const xlpk_page_pool* p, int32_t* remap_dev, void* ws, int64_t ws_bytes, void* stream) {
  XLPK_TRY(check_pool(p));
  XLPK_TRY(check_workspace(p, ws, ws_bytes));
  if (!aligned(remap_dev, 4)) return refuse(XLPK_ERR_INVALID_ARG, "xlpk_pages_compact: remap");
  int sms = 0;
  XLPK_TRY(current_sms(&sms));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  compact_plan_kernel<<<1, kPlanThreads, 0, st>>>(*p, remap_dev, ws);
  XLPK_CUDA(cudaGetLastError());
  const long long n = static_cast<long long>(p->rows) * p->cols;
  const int table_blocks = static_cast<int>(std::min<long long>(sms, (n + kCopyThreads - 1) / kCopyThreads));
  return launch_after(compact_apply_kernel, table_blocks + sms * kCopyCtas, 0, st, *p, remap_dev, ws, table_blocks);
}

xlpk_status xlpk_pages_copy(const xlpk_page_pool* p, const int32_t* src, const int32_t* dst, int32_t n, void* stream) {
  XLPK_TRY(check_pool(p));
  if (n < 0 || (n > 0 && (!src || !dst))) return refuse(XLPK_ERR_INVALID_ARG, "xlpk_pages_copy: the page lists");
  try {
    std::vector<uint8_t> role(static_cast<size_t>(p->n_pages), 0);   // 1: source, 2: destination
    for (int32_t i = 0; i < n; ++i) {
      if (src[i] < 0 || src[i] >= p->n_pages || dst[i] < 0 || dst[i] >= p->n_pages)
        return refuse(XLPK_ERR_INVALID_ARG, "xlpk_pages_copy: a page outside the pool");
      role[src[i]] |= 1;
    }
    for (int32_t i = 0; i < n; ++i) {
      if (role[dst[i]]) return refuse(XLPK_ERR_INVALID_ARG, "xlpk_pages_copy: a destination named twice, or also a source");
      role[dst[i]] = 2;
    }
  } catch (...) {
    return refuse(XLPK_ERR_OOM, "xlpk_pages_copy: host memory");
  }
  int sms = 0;
  XLPK_TRY(current_sms(&sms));
  for (int32_t i = 0; i < n; i += kListPairs) {
    PagePairs l;
    l.n = std::min(kListPairs, n - i);
    std::copy_n(src + i, l.n, l.src);
    std::copy_n(dst + i, l.n, l.dst);
    copy_kernel<<<sms * kCopyCtas, kCopyThreads, 0, static_cast<cudaStream_t>(stream)>>>(*p, l);
  }
  XLPK_CUDA(cudaGetLastError());
  return XLPK_OK;
}

}  // extern "C"
