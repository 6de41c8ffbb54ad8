// Which row owns which page, and the copies that follow from it (include/paged_cache.h documents
// the contract): freeing, extending and forking rows, compacting the live pages, copying pages.
//
// A call is at most two kernels.  The first decides: one cluster of CTAs scans the page counts
// and the items in order, so that the k-th fresh page goes to the k-th demand without atomics
// whose order could change the result; its CTAs exchange their totals through distributed shared
// memory.  The second moves: every SM copies runs of contiguous bytes, as many as the first one
// listed.  The first is bound by the latency of its dependent steps (a handful of cluster
// barriers and L2 round trips), the second by HBM.
#include <cooperative_groups.h>

#include "../../include/paged_cache.h"
#include "common.cuh"
#include "internal.h"

namespace cg = cooperative_groups;

namespace pa {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kPlanCluster = 8;            // portable cluster size
constexpr int kSmallPages = 8192;          // up to here one CTA plans alone
constexpr int kMaxPages = 1 << 24;
constexpr int kCopyThreads = 256;
constexpr int kCopyChunk = 16384;          // bytes of one copy unit

struct Pools {
  void* p[PAGED_CACHE_MAX_POOLS];
};

// ---- scans over the cluster ------------------------------------------------------------------
// Sums saturate at kManyPages, far above any pool's page count, so that absurd demands cannot
// wrap around into served ones (summands are at most kMaxPages + 1, so a saturated exclusive
// prefix is still above every page count).
constexpr int kManyPages = 1 << 29;
__device__ __forceinline__ int add_pages(int a, int b) { return min(a + b, kManyPages); }

// Prefix sum over the CTA; returns this thread's exclusive prefix, *total the sum.
__device__ __forceinline__ int block_scan(int x, int* warp_sums, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int v = x;
#pragma unroll
  for (int d = 1; d < 32; d *= 2) {
    const int y = __shfl_up_sync(0xffffffffu, v, d);
    if (lane >= d) v = add_pages(v, y);
  }
  if (lane == 31) warp_sums[warp] = v;
  __syncthreads();
  if (warp == 0) {
    int w = warp_sums[lane];
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
      const int y = __shfl_up_sync(0xffffffffu, w, d);
      if (lane >= d) w = add_pages(w, y);
    }
    warp_sums[lane] = w;
  }
  __syncthreads();
  const int before = warp > 0 ? warp_sums[warp - 1] : 0;
  *total = warp_sums[31];
  __syncthreads();
  return before + v - x;
}

// The page counts [0, P) are split over the CTAs in segments of whole 4096-page steps: thread t
// of a step holds pages 4 t .. 4 t + 3, so loads coalesce and the order of (step, thread, page)
// is the order of page ids.
struct Segment {
  int first, last, steps;
};
__device__ __forceinline__ Segment page_segment(int P, int rank, int size) {
  const int all = (P + 4095) / 4096;
  const int each = (all + size - 1) / size;
  Segment s;
  s.first = min(P, rank * each * 4096);
  s.last = min(P, (rank + 1) * each * 4096);
  s.steps = (s.last - s.first + 4095) / 4096;
  return s;
}
// Counts of pages p .. p + 3 (aligned loads; 1, that is not free, past the end).
__device__ __forceinline__ int4 load_refs(const int* refs, int p, int last, bool aligned) {
  int4 r = make_int4(1, 1, 1, 1);
  if (aligned && p + 3 < last) return *reinterpret_cast<const int4*>(refs + p);
  if (p < last) r.x = refs[p];
  if (p + 1 < last) r.y = refs[p + 1];
  if (p + 2 < last) r.z = refs[p + 2];
  if (p + 3 < last) r.w = refs[p + 3];
  return r;
}
__device__ __forceinline__ int free_of(const int4& r) {
  return (r.x == 0) + (r.y == 0) + (r.z == 0) + (r.w == 0);
}

// Free pages of the CTA's segment per (step, warp), turned into exclusive prefixes within the
// segment; returns the segment's total.
__device__ int scan_segment(const int* refs, const Segment& s, bool aligned, int* step_warp,
                            int* warp_sums) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int i = 0; i < s.steps; ++i) {
    const int4 r = load_refs(refs, s.first + i * 4096 + 4 * threadIdx.x, s.last, aligned);
    const int n = __reduce_add_sync(0xffffffffu, free_of(r));
    if (lane == 0) step_warp[i * 32 + warp] = n;
  }
  __syncthreads();
  int carry = 0;
  for (int i0 = 0; i0 < s.steps * 32; i0 += kPlanThreads) {
    const int i = i0 + threadIdx.x;
    const int x = i < s.steps * 32 ? step_warp[i] : 0;
    int total;
    const int before = block_scan(x, warp_sums, &total);
    if (i < s.steps * 32) step_warp[i] = carry + before;
    carry += total;
  }
  __syncthreads();
  return carry;
}
// Free pages of this thread's warp before the thread.
__device__ __forceinline__ int free_before_in_warp(int mine) {
  const int lane = threadIdx.x & 31;
  int v = mine;
#pragma unroll
  for (int d = 1; d < 32; d *= 2) {
    const int y = __shfl_up_sync(0xffffffffu, v, d);
    if (lane >= d) v += y;
  }
  return v - mine;
}

// Sums of one int per CTA over the cluster: the CTAs before this one, and all.
struct Totals {
  int before, all;
};
__device__ __forceinline__ Totals cluster_totals(cg::cluster_group& cl, int* slot) {
  Totals t{0, 0};
  const int rank = cl.block_rank(), size = cl.num_blocks();
  for (int r = 0; r < size; ++r) {
    const int x = *cl.map_shared_rank(slot, r);
    if (r < rank) t.before = add_pages(t.before, x);
    t.all = add_pages(t.all, x);
  }
  return t;
}

// ---- extend and fork: who gets which fresh page ------------------------------------------------
struct PlanArgs {
  const int* rows;         // extend: rows; fork: children
  const int* parents;      // fork
  const int* new_tokens;   // extend
  int n;
  int* tables;
  int* lens;
  int* refs;
  int R, C, ps, P;
  uint32_t* status;
  int* off;                // workspace [n]: first fresh page of the item among all demands
  int* need;               // workspace [n]: pages; -1: the item is left out
  int* len;                // workspace [n]: the row's (parent's) length before the call
  int* page;               // workspace [n], fork: the fresh page of the item, -1 none
};

template <bool kFork>
__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const PlanArgs a) {
  extern __shared__ int step_warp[];
  __shared__ int warp_sums[32];
  __shared__ int total_free, total_need;
  cg::cluster_group cl = cg::this_cluster();
  const int rank = cl.block_rank(), size = cl.num_blocks();
  const int tid = threadIdx.x;
  if (rank == 0 && tid < 4) a.status[tid] = 0;
  // this CTA's items, in order
  const int each = (a.n + size - 1) / size;
  const int i0 = min(a.n, rank * each), i1 = min(a.n, i0 + each);
  uint32_t bits = 0;
  for (int i = i0 + tid; i < i1; i += kPlanThreads) {
    const int row = a.rows[i];
    int need = -1, L = 0;
    if (row >= 0 && row < a.R) {
      if (kFork) {
        const int parent = a.parents[i];
        if (parent >= 0 && parent < a.R && parent != row && a.lens[row] == 0) {
          L = a.lens[parent];
          if (L >= 0 && (L + a.ps - 1LL) / a.ps <= a.C) need = L % a.ps > 0;
        }
      } else {
        L = a.lens[row];
        const int more = a.new_tokens[i];
        if (L >= 0 && more >= 0) {
          const long long have = (L + a.ps - 1LL) / a.ps;
          const long long want = (static_cast<long long>(L) + more + a.ps - 1) / a.ps;
          if (want <= a.C) need = static_cast<int>(want - have);
        }
      }
    }
    if (need < 0) bits |= kErrMetadata;
    a.need[i] = need;
    a.len[i] = L;
    if (kFork) a.page[i] = -1;
  }
  // Free pages of the segment, while the items' lengths are on their way.
  const Segment seg = page_segment(a.P, rank, size);
  const bool aligned = (reinterpret_cast<uintptr_t>(a.refs) & 15) == 0;
  const int my_free = scan_segment(a.refs, seg, aligned, step_warp, warp_sums);
  cl.sync();
  // A row listed more than once belongs to its first item: the lengths of the listed rows hold
  // the smallest i - n for a moment (every length has been read).
  for (int i = i0 + tid; i < i1; i += kPlanThreads)
    if (a.need[i] >= 0) atomicMin(a.lens + a.rows[i], i - a.n);
  cl.sync();
  int carry = 0;
  for (int b = i0; b < i1; b += kPlanThreads) {
    const int i = b + tid;
    int need = i < i1 ? a.need[i] : -1;
    if (need >= 0 && atomicAdd(a.lens + a.rows[i], 0) != i - a.n) {
      need = a.need[i] = -1;
      bits |= kErrMetadata;
    }
    int total;
    const int before = block_scan(min(max(need, 0), kMaxPages + 1), warp_sums, &total);
    if (i < i1) a.off[i] = add_pages(carry, before);
    carry = add_pages(carry, total);
  }
  if (tid == 0) {
    total_free = my_free;
    total_need = carry;
  }
  cl.sync();
  const Totals free = cluster_totals(cl, &total_free), demand = cluster_totals(cl, &total_need);
  for (int i = i0 + tid; i < i1; i += kPlanThreads) {
    const int need = a.need[i];
    const int off = add_pages(a.off[i], demand.before);
    a.off[i] = off;
    if (need < 0) continue;
    const bool served = need == 0 || static_cast<long long>(off) + need <= free.all;
    const int L = a.len[i];
    if (!served) {
      bits |= kErrCapacity;
      a.need[i] = -1;
    }
    a.lens[a.rows[i]] = kFork ? (served ? L : 0) : (served ? L + a.new_tokens[i] : L);
  }
  if (bits) report_error(a.status, bits);
  cl.sync();
  // The k-th free page goes to the item whose demands [off, off + need) hold k.
  const int warp = tid >> 5;
  for (int s = 0; s < seg.steps; ++s) {
    const int p0 = seg.first + s * 4096 + 4 * tid;
    const int4 r = load_refs(a.refs, p0, seg.last, aligned);
    int k = free.before + step_warp[s * 32 + warp] + free_before_in_warp(free_of(r));
    const int c[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (c[j] != 0) continue;
      const int rank_k = k++;
      if (rank_k >= demand.all) continue;
      int lo = 0, hi = a.n;                    // last item with off <= k and a demand
      while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (a.off[mid] <= rank_k) lo = mid; else hi = mid;
      }
      // items without a demand share their successor's offset: the last one found owns k
      const int need = a.need[lo];
      if (need < 0 || rank_k - a.off[lo] >= need) continue;
      const int row = a.rows[lo], have = kFork ? a.len[lo] / a.ps : (a.len[lo] + a.ps - 1) / a.ps;
      a.tables[static_cast<long long>(row) * a.C + have + rank_k - a.off[lo]] = p0 + j;
      a.refs[p0 + j] = 1;
      if (kFork) a.page[lo] = p0 + j;
    }
  }
  grid_launch_dependents();
}

// ---- copies ----------------------------------------------------------------------------------
__device__ __forceinline__ uint4 ld_stream(const uint4* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

// One CTA copies n16 16-byte words.
__device__ __forceinline__ void copy_words(uint4* __restrict__ dst, const uint4* __restrict__ src,
                                           int n16) {
  int i = threadIdx.x;
  for (; i + 3 * kCopyThreads < n16; i += 4 * kCopyThreads) {
    const uint4 a = ld_stream(src + i), b = ld_stream(src + i + kCopyThreads);
    const uint4 c = ld_stream(src + i + 2 * kCopyThreads), d = ld_stream(src + i + 3 * kCopyThreads);
    dst[i] = a;
    dst[i + kCopyThreads] = b;
    dst[i + 2 * kCopyThreads] = c;
    dst[i + 3 * kCopyThreads] = d;
  }
  for (; i < n16; i += kCopyThreads) dst[i] = ld_stream(src + i);
}

struct CopyArgs {
  Pools src, dst;
  int pools;                 // pointers per side
  const int *src_pages, *dst_pages;
  int n;                     // pairs, or
  const int* n_dev;          // their number on the device
  int src_num_pages, dst_num_pages;
  long long page_bytes;
  int chunks;                // of kCopyChunk bytes per page
  uint32_t* status;
  // compact: table entries to rename
  const int *tables, *lens, *to;
  int* tables_out;
  int R, C, ps, P;
};

template <bool kCompact>
__global__ void __launch_bounds__(kCopyThreads) copy_kernel(const __grid_constant__ CopyArgs a) {
  if (kCompact) grid_dependency_wait();
  const int n = kCompact ? *a.n_dev : a.n;
  const long long units = static_cast<long long>(n) * a.pools * a.chunks;
  for (long long u = blockIdx.x; u < units; u += gridDim.x) {
    const int chunk = static_cast<int>(u % a.chunks);
    const long long w = u / a.chunks;
    const int pool = static_cast<int>(w % a.pools);
    const int i = static_cast<int>(w / a.pools);
    const int s = a.src_pages[i], d = a.dst_pages[i];
    if (s < 0 || s >= a.src_num_pages || d < 0 || d >= a.dst_num_pages) {
      if (threadIdx.x == 0) report_error(a.status, kErrMetadata);
      continue;
    }
    if (s == d && a.src.p[pool] == a.dst.p[pool]) continue;
    const long long at = static_cast<long long>(chunk) * kCopyChunk;
    const int bytes = static_cast<int>(min(static_cast<long long>(kCopyChunk), a.page_bytes - at));
    copy_words(reinterpret_cast<uint4*>(static_cast<uint8_t*>(a.dst.p[pool]) + d * a.page_bytes + at),
               reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(a.src.p[pool]) +
                                              s * a.page_bytes + at),
               bytes / 16);
  }
  if (kCompact) {
    const long long entries = static_cast<long long>(a.R) * a.C;
    for (long long e = blockIdx.x * static_cast<long long>(kCopyThreads) + threadIdx.x; e < entries;
         e += static_cast<long long>(gridDim.x) * kCopyThreads) {
      const int row = static_cast<int>(e / a.C), j = static_cast<int>(e - static_cast<long long>(row) * a.C);
      const int L = a.lens[row];
      int p = a.tables[e];
      const int old = p;
      if (j < (L + a.ps - 1LL) / a.ps) {
        if (p >= 0 && p < a.P) p = a.to[p];
        else report_error(a.status, kErrMetadata);
      }
      if (j == 0 && (L + a.ps - 1LL) / a.ps > a.C) report_error(a.status, kErrMetadata);
      if (p != old || a.tables_out != a.tables) a.tables_out[e] = p;
    }
  }
}

// ---- fork: shared pages and the copied tail ------------------------------------------------------
struct ForkArgs {
  Pools pools;
  int npools, segs;          // runs of tail bytes per pool: one per head, K and V
  long long page_bytes, seg_bytes, token_bytes;
  const int *children, *parents, *need, *len, *page;
  int n;
  int* tables;
  int* refs;
  int C, ps, P;
  int table_units;           // CTAs per item for the table row
  uint32_t* status;
};

__global__ void __launch_bounds__(kCopyThreads) fork_kernel(const __grid_constant__ ForkArgs a) {
  grid_dependency_wait();
  const int per_item = a.npools + a.table_units;
  const long long units = static_cast<long long>(a.n) * per_item;
  for (long long u = blockIdx.x; u < units; u += gridDim.x) {
    const int i = static_cast<int>(u / per_item), w = static_cast<int>(u - static_cast<long long>(i) * per_item);
    if (a.need[i] < 0) continue;
    const int L = a.len[i], full = L / a.ps;
    const long long from = static_cast<long long>(a.parents[i]) * a.C;
    if (w < a.npools) {
      const int d = a.page[i];
      if (d < 0) continue;
      const int s = a.tables[from + full];
      if (s < 0 || s >= a.P) {
        if (threadIdx.x == 0) report_error(a.status, kErrMetadata);
        continue;
      }
      const int words = static_cast<int>((L - full * a.ps) * a.token_bytes / 16);
      uint8_t* base = static_cast<uint8_t*>(a.pools.p[w]);
      for (int x = threadIdx.x; x < words * a.segs; x += kCopyThreads) {
        const int seg = x / words, at = x - seg * words;
        const long long o = seg * a.seg_bytes + at * 16LL;
        *reinterpret_cast<uint4*>(base + d * a.page_bytes + o) =
            ld_stream(reinterpret_cast<const uint4*>(base + s * a.page_bytes + o));
      }
    } else {
      const long long to = static_cast<long long>(a.children[i]) * a.C;
      for (int j = (w - a.npools) * kCopyThreads + threadIdx.x; j < full;
           j += a.table_units * kCopyThreads) {
        const int p = a.tables[from + j];
        a.tables[to + j] = p;
        if (p >= 0 && p < a.P) atomicAdd(a.refs + p, 1);
        else report_error(a.status, kErrMetadata);
      }
    }
  }
}

// ---- free ------------------------------------------------------------------------------------
__global__ void __launch_bounds__(kCopyThreads)
free_kernel(const int* rows, int n, const int* tables, int* lens, int* refs, int R, int C, int ps,
            int P, uint32_t* status) {
  __shared__ int len;
  const int row = rows[blockIdx.x];
  if (row < 0 || row >= R) {
    if (threadIdx.x == 0) report_error(status, kErrMetadata);
    return;
  }
  if (threadIdx.x == 0) len = atomicExch(lens + row, 0);
  __syncthreads();
  const long long pages = (len + ps - 1LL) / ps;
  if (threadIdx.x == 0 && (len < 0 || pages > C)) report_error(status, kErrMetadata);
  const int* t = tables + static_cast<long long>(row) * C;
  for (int j = threadIdx.x; j < min(pages, static_cast<long long>(C)); j += kCopyThreads) {
    const int p = t[j];
    bool bad = p < 0 || p >= P;
    if (!bad && atomicSub(refs + p, 1) <= 0) {
      atomicAdd(refs + p, 1);
      bad = true;
    }
    if (bad) report_error(status, kErrMetadata);
  }
}

// ---- compact: which page moves where -------------------------------------------------------------
struct CompactArgs {
  const int* refs;
  int* refs_out;
  int* num_live;
  int P;
  int *src, *dst, *to, *moves;   // workspace: move lists, new id of every page, their number
  uint32_t* status;
};

__global__ void __launch_bounds__(kPlanThreads) compact_kernel(const CompactArgs a) {
  extern __shared__ int step_warp[];
  __shared__ int warp_sums[32];
  __shared__ int total_free, total_holes;
  cg::cluster_group cl = cg::this_cluster();
  const int rank = cl.block_rank(), size = cl.num_blocks();
  const int tid = threadIdx.x, warp = tid >> 5;
  if (rank == 0 && tid < 4) a.status[tid] = 0;
  const Segment seg = page_segment(a.P, rank, size);
  const bool aligned = (reinterpret_cast<uintptr_t>(a.refs) & 15) == 0;
  const int my_free = scan_segment(a.refs, seg, aligned, step_warp, warp_sums);
  if (tid == 0) {
    total_free = my_free;
    total_holes = 0;
  }
  cl.sync();
  const Totals free = cluster_totals(cl, &total_free);
  const int live = a.P - free.all;
  // holes of this CTA: free pages below `live`
  int holes = 0;
  for (int s = 0; s < seg.steps; ++s) {
    const int p0 = seg.first + s * 4096 + 4 * tid;
    const int4 r = load_refs(a.refs, p0, seg.last, aligned);
    const int c[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) holes += c[j] == 0 && p0 + j < live;
  }
  holes = __reduce_add_sync(0xffffffffu, holes);
  if ((tid & 31) == 0 && holes) atomicAdd(&total_holes, holes);
  cl.sync();
  const int H = cluster_totals(cl, &total_holes).all;   // holes below, and live pages above
  for (int s = 0; s < seg.steps; ++s) {
    const int p0 = seg.first + s * 4096 + 4 * tid;
    const int4 r = load_refs(a.refs, p0, seg.last, aligned);
    int f = free.before + step_warp[s * 32 + warp] + free_before_in_warp(free_of(r));
    const int c[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int p = p0 + j;
      if (p >= seg.last) continue;
      if (c[j] == 0) {
        if (p < live) a.dst[f] = p;
        ++f;
      } else if (p >= live) {
        a.src[p - f - (live - H)] = p;       // p - f live pages lie before p, live - H below `live`
      }
    }
  }
  if (rank == 0 && tid == 0) {
    *a.moves = H;
    *a.num_live = live;
  }
  cl.sync();
  // new ids and counts (every count has been read)
  const int i0 = rank * kPlanThreads + tid, stride = size * kPlanThreads;
  for (int p = i0; p < a.P; p += stride) a.to[p] = p;
  if (a.refs_out != a.refs)
    for (int p = i0; p < a.P; p += stride) a.refs_out[p] = a.refs[p];
  cl.sync();
  for (int k = i0; k < H; k += stride) {
    const int s = a.src[k], d = a.dst[k];
    a.to[s] = d;
    a.refs_out[d] = a.refs[s];
    a.refs_out[s] = 0;
  }
  grid_launch_dependents();
}

// ---- host --------------------------------------------------------------------------------------
struct Take {
  size_t off = 0;
  size_t ints(long long n) {
    const size_t at = off;
    off = align_up(off + sizeof(int) * static_cast<size_t>(n > 0 ? n : 1), 256);
    return at;
  }
};
int* at(void* ws, size_t off) { return reinterpret_cast<int*>(static_cast<uint8_t*>(ws) + off); }

struct PlanLayout {
  size_t status, off, need, len, page, total;
  explicit PlanLayout(int n) {
    Take t;
    status = t.ints(4);
    off = t.ints(n);
    need = t.ints(n);
    len = t.ints(n);
    page = t.ints(n);
    total = t.off;
  }
};
struct CompactLayout {
  size_t status, moves, src, dst, to, total;
  explicit CompactLayout(int P) {
    Take t;
    status = t.ints(4);
    moves = t.ints(1);
    src = t.ints(P);
    dst = t.ints(P);
    to = t.ints(P);
    total = t.off;
  }
};

bool cache_params_ok(const paged_cache_params* p) {
  return p && p->rows >= 0 && p->max_pages_per_request > 0 && p->page_size >= 8 &&
         p->page_size <= 128 && p->page_size % 8 == 0 && p->num_pages > 0 &&
         p->num_pages <= kMaxPages;
}
bool pools_ok(const paged_cache_pools* p) {
  if (!p || !p->pools_host || p->num_layers <= 0 || p->num_layers > PAGED_CACHE_MAX_POOLS)
    return false;
  const int count = p->num_layers * (p->combined_cache ? 1 : 2);
  if (count > PAGED_CACHE_MAX_POOLS || p->num_pages <= 0 || p->num_pages > kMaxPages) return false;
  if (p->num_kv_heads <= 0 || p->num_kv_heads > 65535 || p->head_dim <= 0 || p->head_dim > 512 ||
      p->head_dim % 8)
    return false;
  if (p->page_size < 8 || p->page_size > 128 || p->page_size % 8) return false;
  for (int i = 0; i < count; ++i)
    if (!p->pools_host[i] || (reinterpret_cast<uintptr_t>(p->pools_host[i]) & 15)) return false;
  return true;
}
int pool_count(const paged_cache_pools* p) { return p->num_layers * (p->combined_cache ? 1 : 2); }
long long seg_bytes(const paged_cache_pools* p) { return 2LL * p->page_size * p->head_dim; }
long long page_bytes(const paged_cache_pools* p) {
  return (p->combined_cache ? 2 : 1) * p->num_kv_heads * seg_bytes(p);
}
bool same_geometry(const paged_cache_pools* a, const paged_cache_pools* b) {
  return a->num_layers == b->num_layers && a->num_kv_heads == b->num_kv_heads &&
         a->page_size == b->page_size && a->head_dim == b->head_dim &&
         (a->combined_cache != 0) == (b->combined_cache != 0);
}
bool overlap(const void* a, long long na, const void* b, long long nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + static_cast<uintptr_t>(nb) && y < x + static_cast<uintptr_t>(na);
}
int cuda_status(cudaError_t e) { return e == cudaSuccess ? PAGED_ATTN_OK : PAGED_ATTN_ERR_CUDA; }

// Launch one of the planning kernels as a single cluster (one CTA for small pools).
template <typename Args>
cudaError_t launch_plan(void (*kernel)(Args), const Args& a, int P, std::atomic<uint64_t>& ready,
                        cudaStream_t st) {
  const int size = P <= kSmallPages ? 1 : kPlanCluster;
  const int each = ceil_div(ceil_div(P, 4096), size);
  const size_t smem = static_cast<size_t>(each) * 32 * sizeof(int);
  if (!kernel_smem_ready(kernel, kMaxPages / kPlanCluster / 128 * static_cast<int>(sizeof(int)),
                         ready))
    return cudaErrorUnknown;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = size;
  cfg.blockDim = kPlanThreads;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = size;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  count_launches(1);
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

}  // namespace
}  // namespace pa

using namespace pa;

extern "C" {

int paged_cache_free_run(const paged_cache_params* p, const int32_t* rows, int n,
                         const int32_t* tables, int32_t* lens, int32_t* refs, uint32_t* status,
                         void* stream) {
  if (!cache_params_ok(p) || n < 0) return PAGED_ATTN_ERR_INVALID_ARGUMENT;
  if (n == 0) return PAGED_ATTN_OK;
  if (!rows || !tables || !lens || !refs) return PAGED_ATTN_ERR_INVALID_ARGUMENT;
  free_kernel<<<n, kCopyThreads, 0, static_cast<cudaStream_t>(stream)>>>(
      rows, n, tables, lens, refs, p->rows, p->max_pages_per_request, p->page_size, p->num_pages,
      status);
  count_launches(1);
  return cuda_status(cudaGetLastError());
}

size_t paged_cache_extend_workspace_size(int n) { return n < 0 ? 0 : PlanLayout(n).total; }
size_t paged_cache_fork_workspace_size(int n) { return n < 0 ? 0 : PlanLayout(n).total; }
size_t paged_cache_compact_workspace_size(int num_pages) {
  return num_pages <= 0 || num_pages > kMaxPages ? 0 : CompactLayout(num_pages).total;
}

int paged_cache_extend_run(const paged_cache_params* p, const int32_t* rows,
                           const int32_t* new_tokens, int n, int32_t* tables, int32_t* lens,
                           int32_t* refs, void* ws, size_t ws_bytes, void* stream) {
  if (!cache_params_ok(p) || n < 0) return PAGED_ATTN_ERR_INVALID_ARGUMENT;
  if (n > 0 && (!rows || !new_tokens || !tables || !lens || !refs))
    return PAGED_ATTN_ERR_INVALID_ARGUMENT;
  const PlanLayout l(n);
  if (!ws || ws_bytes < l.total) return PAGED_ATTN_ERR_WORKSPACE;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (n == 0) return cuda_status(cudaMemsetAsync(ws, 0, 4 * sizeof(uint32_t), st));
  PlanArgs a{};
  a.rows = rows; a.new_tokens = new_tokens; a.n = n;
  a.tables = tables; a.lens = lens; a.refs = refs;
  a.R = p->rows; a.C = p->max_pages_per_request; a.ps = p->page_size; a.P = p->num_pages;
  a.status = reinterpret_cast<uint32_t*>(at(ws, l.status));
  a.off = at(ws, l.off); a.need = at(ws, l.need); a.len = at(ws, l.len);
  static std::atomic<uint64_t> ready{0};
  return cuda_status(launch_plan(plan_kernel<false>, a, a.P, ready, st));
}

int paged_cache_fork_run(const paged_cache_params* p, const paged_cache_pools* pools,
                         const int32_t* parents, const int32_t* children, int n, int32_t* tables,
                         int32_t* lens, int32_t* refs, void* ws, size_t ws_bytes, void* stream) {
  if (!cache_params_ok(p) || !pools_ok(pools) || n < 0) return PAGED_ATTN_ERR_INVALID_ARGUMENT;
  if (pools->num_pages != p->num_pages || pools->page_size != p->page_size)
    return PAGED_ATTN_ERR_INVALID_ARGUMENT;
  if (n > 0 && (!parents || !children || !tables || !lens || !refs))
    return PAGED_ATTN_ERR_INVALID_ARGUMENT;
  const PlanLayout l(n);
  if (!ws || ws_bytes < l.total) return PAGED_ATTN_ERR_WORKSPACE;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (n == 0) return cuda_status(cudaMemsetAsync(ws, 0, 4 * sizeof(uint32_t), st));
  PlanArgs a{};
  a.rows = children; a.parents = parents; a.n = n;
  a.tables = tables; a.lens = lens; a.refs = refs;
  a.R = p->rows; a.C = p->max_pages_per_request; a.ps = p->page_size; a.P = p->num_pages;
  a.status = reinterpret_cast<uint32_t*>(at(ws, l.status));
  a.off = at(ws, l.off); a.need = at(ws, l.need); a.len = at(ws, l.len); a.page = at(ws, l.page);
  static std::atomic<uint64_t> ready{0};
  cudaError_t e = launch_plan(plan_kernel<true>, a, a.P, ready, st);
  if (e != cudaSuccess) return PAGED_ATTN_ERR_CUDA;
  ForkArgs f{};
  f.npools = pool_count(pools);
  for (int i = 0; i < f.npools; ++i) f.pools.p[i] = pools->pools_host[i];
  f.segs = (pools->combined_cache ? 2 : 1) * pools->num_kv_heads;
  f.page_bytes = page_bytes(pools);
  f.seg_bytes = seg_bytes(pools);
  f.token_bytes = 2LL * pools->head_dim;
  f.children = children; f.parents = parents; f.need = a.need; f.len = a.len; f.page = a.page;
  f.n = n;
  f.tables = tables; f.refs = refs;
  f.C = a.C; f.ps = a.ps; f.P = a.P;
  f.table_units = ceil_div(a.C, 4 * kCopyThreads);
  f.status = a.status;
  const int sms = current_sm_count();
  if (sms <= 0) return PAGED_ATTN_ERR_CUDA;
  const long long units = static_cast<long long>(n) * (f.npools + f.table_units);
  const long long most = 8LL * sms;
  count_launches(1);
  return cuda_status(launch_after_previous(fork_kernel, static_cast<int>(units < most ? units : most),
                                           kCopyThreads, 0, st, f));
}

int paged_cache_compact_run(const paged_cache_params* p, const paged_cache_pools* pools,
                            const int32_t* tables, const int32_t* lens, const int32_t* refs,
                            int32_t* tables_out, int32_t* refs_out, int32_t* num_live, void* ws,
                            size_t ws_bytes, void* stream) {
  if (!cache_params_ok(p) || !pools_ok(pools)) return PAGED_ATTN_ERR_INVALID_ARGUMENT;
  if (pools->num_pages != p->num_pages || pools->page_size != p->page_size)
    return PAGED_ATTN_ERR_INVALID_ARGUMENT;
  if (!refs || !refs_out || !num_live) return PAGED_ATTN_ERR_INVALID_ARGUMENT;
  if (p->rows > 0 && (!tables || !tables_out || !lens)) return PAGED_ATTN_ERR_INVALID_ARGUMENT;
  const long long tb = 4LL * p->rows * p->max_pages_per_request, rb = 4LL * p->num_pages;
  if (p->rows > 0 && tables != tables_out && overlap(tables, tb, tables_out, tb))
    return PAGED_ATTN_ERR_INVALID_ARGUMENT;
  if (refs != refs_out && overlap(refs, rb, refs_out, rb)) return PAGED_ATTN_ERR_INVALID_ARGUMENT;
  const CompactLayout l(p->num_pages);
  if (!ws || ws_bytes < l.total) return PAGED_ATTN_ERR_WORKSPACE;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  CompactArgs a{};
  a.refs = refs; a.refs_out = refs_out; a.num_live = num_live; a.P = p->num_pages;
  a.src = at(ws, l.src); a.dst = at(ws, l.dst); a.to = at(ws, l.to); a.moves = at(ws, l.moves);
  a.status = reinterpret_cast<uint32_t*>(at(ws, l.status));
  static std::atomic<uint64_t> ready{0};
  cudaError_t e = launch_plan(compact_kernel, a, a.P, ready, st);
  if (e != cudaSuccess) return PAGED_ATTN_ERR_CUDA;
  CopyArgs c{};
  c.pools = pool_count(pools);
  for (int i = 0; i < c.pools; ++i) c.src.p[i] = c.dst.p[i] = pools->pools_host[i];
  c.src_pages = a.src; c.dst_pages = a.dst; c.n_dev = a.moves;
  c.src_num_pages = c.dst_num_pages = p->num_pages;
  c.page_bytes = page_bytes(pools);
  c.chunks = static_cast<int>(ceil_div_ll(c.page_bytes, kCopyChunk));
  c.status = a.status;
  c.tables = tables; c.lens = lens; c.to = a.to; c.tables_out = tables_out;
  c.R = p->rows; c.C = p->max_pages_per_request; c.ps = p->page_size; c.P = p->num_pages;
  const int sms = current_sm_count();
  if (sms <= 0) return PAGED_ATTN_ERR_CUDA;
  count_launches(1);
  return cuda_status(launch_after_previous(copy_kernel<true>, 8 * sms, kCopyThreads, 0, st, c));
}

int paged_cache_copy_run(const paged_cache_pools* src, const paged_cache_pools* dst,
                         const int32_t* src_pages, const int32_t* dst_pages, int n,
                         uint32_t* status, void* stream) {
  if (!pools_ok(src) || !pools_ok(dst) || !same_geometry(src, dst) || n < 0)
    return PAGED_ATTN_ERR_INVALID_ARGUMENT;
  if (n == 0) return PAGED_ATTN_OK;
  if (!src_pages || !dst_pages) return PAGED_ATTN_ERR_INVALID_ARGUMENT;
  CopyArgs c{};
  c.pools = pool_count(src);
  for (int i = 0; i < c.pools; ++i) {
    c.src.p[i] = src->pools_host[i];
    c.dst.p[i] = dst->pools_host[i];
  }
  c.src_pages = src_pages; c.dst_pages = dst_pages; c.n = n;
  c.src_num_pages = src->num_pages;
  c.dst_num_pages = dst->num_pages;
  c.page_bytes = page_bytes(src);
  c.chunks = static_cast<int>(ceil_div_ll(c.page_bytes, kCopyChunk));
  c.status = status;
  const int sms = current_sm_count();
  if (sms <= 0) return PAGED_ATTN_ERR_CUDA;
  const long long units = static_cast<long long>(n) * c.pools * c.chunks;
  const long long most = 8LL * sms;
  copy_kernel<false><<<static_cast<int>(units < most ? units : most), kCopyThreads, 0,
                       static_cast<cudaStream_t>(stream)>>>(c);
  count_launches(1);
  return cuda_status(cudaGetLastError());
}

}  // extern "C"
