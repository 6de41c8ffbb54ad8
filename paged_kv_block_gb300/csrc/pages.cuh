// What the page kernels share (cache.cu, evict.cu): finding the free pages in order, the pools of
// every layer, where findings are reported, and the checks and launches of their entry points.
#pragma once

#include <climits>

#include <cooperative_groups.h>

#include "../../include/paged_cache.h"
#include "common.cuh"
#include "internal.h"

namespace pa {

namespace cg = cooperative_groups;

constexpr int kPlanThreads = 1024;         // of a planning CTA, or
constexpr int kFewThreads = 256;           // where the pool and the list are small
constexpr int kPlanCluster = 8;            // portable cluster size
constexpr int kThreadPages = 8;            // pages that a thread counts at a time
constexpr int kMaxPages = 1 << 24;
constexpr int kPerThread = 4;              // items that a thread of the planning CTA holds
constexpr int kMaxItems = kPerThread * kPlanThreads;
// Shared memory of a planning kernel at most: items, the hash table of their rows, page counts.
constexpr int kMaxSteps = kMaxPages / (kPlanThreads * kThreadPages);
constexpr int kPlanSmem = (9 * kMaxItems + kMaxSteps / kPlanCluster * 33 + kMaxSteps) * 4;
static_assert(kPlanSmem <= 226 * 1024, "shared memory of the planning kernels");
constexpr long long kMaxGrid = 1LL << 30;

struct Pools {
  void* p[PAGED_CACHE_MAX_POOLS];
};

// Where a call reports: the word of its workspace and the caller's own (either may be null).
struct Status {
  uint32_t *ws, *own;
};
__device__ __forceinline__ void report(const Status& s, uint32_t bits) {
  report_error(s.ws, bits);
  report_error(s.own, bits);
}

// ---- free pages in order, over a cluster -------------------------------------------------------
// Sums saturate at kManyPages, far above any pool's page count, so that absurd demands cannot
// wrap around into served ones (summands are at most kMaxPages + 1, so a saturated exclusive
// prefix is still above every page count).
constexpr int kManyPages = 1 << 29;
__device__ __forceinline__ int add_pages(int a, int b) { return min(a + b, kManyPages); }

__device__ __forceinline__ int warp_inclusive(int v) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int d = 1; d < 32; d *= 2) {
    const int y = __shfl_up_sync(0xffffffffu, v, d);
    if (lane >= d) v = add_pages(v, y);
  }
  return v;
}
// Prefix sum over the CTA; returns this thread's exclusive prefix, *total the sum.
__device__ __forceinline__ int block_scan(int x, int* warp_sums, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int v = warp_inclusive(x);
  if (lane == 31) warp_sums[warp] = v;
  __syncthreads();
  // every warp scans the warps' sums itself
  const int w = warp_inclusive(lane < static_cast<int>(blockDim.x >> 5) ? warp_sums[lane] : 0);
  const int before = __shfl_sync(0xffffffffu, w, (warp + 31) & 31);
  *total = __shfl_sync(0xffffffffu, w, 31);
  __syncthreads();
  return (warp > 0 ? before : 0) + v - x;
}

// The two halves of a cluster barrier that orders no memory.
__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
}
// A barrier over the cluster, with its memory; a plain one where the cluster is one CTA.
__device__ __forceinline__ void sync_cluster(cg::cluster_group& cl) {
  if (cl.num_blocks() == 1) __syncthreads();
  else cl.sync();
}

// The page counts [0, P) are cut into steps of 8 pages per thread; step g belongs to CTA g % size,
// and thread t of it holds pages 8 t .. 8 t + 7, so loads coalesce and the order of (step, thread,
// page) is the order of page ids.  The CTAs interleave so that a demand met by the lowest pages
// is still handed out by all of them.
// What bounds this is instructions, not bytes (every warp of a CTA issues through four schedulers):
// hence 32-byte loads, one mask per thread and step, and one CTA of 256 threads for small pools.
struct FreePages {
  const int* refs;
  int P, rank, size, steps, own;     // steps in all, steps of this CTA
  bool aligned;
  uint32_t kept;                     // the thread's masks of its first 4 steps
  int* warp_before;                  // shared [own, 32]: free pages of the step before a warp
  int* step_total;                   // shared [own]
  int* step_before;                  // shared [steps]: free pages before a step
  int total;                         // free pages

  static __host__ __device__ int steps_of(int P, int threads) {
    return (P + threads * kThreadPages - 1) / (threads * kThreadPages);
  }
  static __host__ size_t shared_ints(int P, int size, int threads) {
    const int steps = steps_of(P, threads);
    return static_cast<size_t>((steps + size - 1) / size) * 33 + steps;
  }

  __device__ __forceinline__ int first_page(int j) const {
    return ((j * size + rank) * static_cast<int>(blockDim.x) + static_cast<int>(threadIdx.x)) *
           kThreadPages;
  }
  // Counts of the thread's pages of its j-th step (1, that is not free, past the end).
  __device__ __forceinline__ void load(int j, uint32_t (&r)[kThreadPages]) const {
    const int p = first_page(j);
    if (j < own && aligned && p + kThreadPages <= P) {
      asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                   : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]),
                     "=r"(r[6]), "=r"(r[7])
                   : "l"(refs + p)
                   : "memory");
    } else {
#pragma unroll
      for (int b = 0; b < kThreadPages; ++b)
        r[b] = j < own && p + b < P ? static_cast<uint32_t>(refs[p + b]) : 1u;
    }
  }
  static __device__ __forceinline__ uint32_t mask_of(const uint32_t (&r)[kThreadPages]) {
    uint32_t m = 0;
#pragma unroll
    for (int b = 0; b < kThreadPages; ++b) m |= r[b] == 0 ? 1u << b : 0u;
    return m;
  }
  // Which of them were free at count().
  __device__ __forceinline__ uint32_t mask(int j) const {
    if (j < 4) return (kept >> (8 * j)) & 255u;
    uint32_t r[kThreadPages];
    load(j, r);
    return mask_of(r);
  }

  // Count the CTA's own steps (before the cluster barrier); `meanwhile` runs while the first loads
  // are on their way.
  template <typename F>
  __device__ void count(const int* counts, int num_pages, int cta, int ctas, int* shared,
                        const F& meanwhile) {
    refs = counts;
    P = num_pages;
    rank = cta;
    size = ctas;
    steps = steps_of(P, blockDim.x);
    own = (steps - rank + size - 1) / size;
    aligned = (reinterpret_cast<uintptr_t>(refs) & 31) == 0;
    kept = 0;
    const int room = (steps + size - 1) / size;
    warp_before = shared;
    step_total = warp_before + room * 32;
    step_before = step_total + room;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int warps = blockDim.x >> 5;
    for (int j0 = 0; j0 < own; j0 += 4) {
      uint32_t r[4][kThreadPages];                     // four steps' loads in flight
#pragma unroll
      for (int u = 0; u < 4; ++u) load(j0 + u, r[u]);
      if (j0 == 0) meanwhile();
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        if (j0 + u >= own) break;
        const uint32_t m = mask_of(r[u]);
        if (j0 == 0) kept |= m << (8 * u);
        const int n = __reduce_add_sync(0xffffffffu, __popc(m));
        if (lane == 0) warp_before[(j0 + u) * 32 + warp] = n;
      }
    }
    __syncthreads();
    for (int j = warp; j < own; j += warps) {
      const int n = lane < warps ? warp_before[j * 32 + lane] : 0, v = warp_inclusive(n);
      warp_before[j * 32 + lane] = v - n;
      if (lane == 31) step_total[j] = v;
    }
  }
  // Put the steps of all CTAs in order (after the cluster barrier).
  __device__ void order(cg::cluster_group& cl) {
    const int lane = threadIdx.x & 31;
    int carry = 0;
    for (int g0 = 0; g0 < steps; g0 += 32) {           // every warp for itself
      const int g = g0 + lane;
      const int n = g < steps ? *cl.map_shared_rank(step_total + g / size, g % size) : 0;
      const int v = warp_inclusive(n);
      if (threadIdx.x < 32 && g < steps) step_before[g] = carry + v - n;
      carry += __shfl_sync(0xffffffffu, v, 31);
    }
    total = carry;
    __syncthreads();
  }
  // Calls f(page, is_free, free pages before it, free pages among the warp's 32) for the pages
  // of the j-th step with a page per lane: neighbouring lanes hold neighbouring pages and, where
  // those are free, neighbouring ranks, so that what f stores by either coalesces.  Whole warps.
  template <typename F>
  __device__ __forceinline__ void each(int j, const F& f) const {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t m = mask(j);
    int before = step_before[j * size + rank] + warp_before[j * 32 + warp];
    int p = ((j * size + rank) * static_cast<int>(blockDim.x) + warp * 32) * kThreadPages + lane;
#pragma unroll
    for (int g = 0; g < kThreadPages; ++g) {           // 32 pages: the masks of 4 lanes
      const uint32_t theirs = __shfl_sync(0xffffffffu, m, 4 * g + (lane >> 3));
      const bool is_free = theirs >> (lane & 7) & 1u;
      const uint32_t all = __ballot_sync(0xffffffffu, is_free);
      f(p, is_free, before + __popc(all & ((1u << lane) - 1u)), __popc(all));
      before += __popc(all);
      p += 32;
    }
  }
};

__device__ __forceinline__ uint4 ld_stream(const uint4* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
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
inline int* at(void* ws, size_t off) {
  return reinterpret_cast<int*>(static_cast<uint8_t*>(ws) + off);
}

inline bool cache_params_ok(const paged_cache_params* p) {
  return p && p->rows >= 0 && p->max_pages_per_request > 0 && p->page_size >= 8 &&
         p->page_size <= 128 && p->page_size % 8 == 0 && p->num_pages > 0 &&
         p->num_pages <= kMaxPages && (reinterpret_cast<uintptr_t>(p->status_dev) & 3) == 0;
}
inline int pool_count(const paged_cache_pools* p) {
  return p->num_layers * (p->combined_cache ? 1 : 2);
}
inline long long seg_bytes(const paged_cache_pools* p) {
  return 2LL * p->page_size * p->head_dim;
}
inline long long page_bytes(const paged_cache_pools* p) {
  return (p->combined_cache ? 2 : 1) * p->num_kv_heads * seg_bytes(p);
}
inline bool pools_ok(const paged_cache_pools* p) {
  if (!p || !p->pools_host || p->num_layers <= 0 || p->num_layers > PAGED_CACHE_MAX_POOLS)
    return false;
  const int count = p->num_layers * (p->combined_cache ? 1 : 2);
  if (count > PAGED_CACHE_MAX_POOLS || p->num_pages <= 0 || p->num_pages > kMaxPages) return false;
  if (p->num_kv_heads <= 0 || p->num_kv_heads > 65535 || p->head_dim <= 0 || p->head_dim > 512 ||
      p->head_dim % 8)
    return false;
  if (p->page_size < 8 || p->page_size > 128 || p->page_size % 8) return false;
  if (page_bytes(p) >= 1LL << 31) return false;
  for (int i = 0; i < count; ++i)
    if (!p->pools_host[i] || (reinterpret_cast<uintptr_t>(p->pools_host[i]) & 15)) return false;
  return true;
}
inline int cuda_status(cudaError_t e) {
  return e == cudaSuccess ? PAGED_ATTN_OK : PAGED_ATTN_ERR_CUDA;
}
inline bool aligned_to(const void* p, uintptr_t bytes) {
  return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0;
}
// int32 arrays at 4-byte addresses (NULL is one).
template <typename... P>
inline bool ints_aligned(const P*... p) {
  return (... && aligned_to(p, 4));
}

// Launch one of the planning kernels as a single cluster; `ints` of shared memory besides the
// page counts'.  Small pools and lists: one CTA of 256 threads (its 4 steps of pages stay in
// registers, an item list fits its threads); else CTAs of 1024, one per step, up to the portable
// cluster size.
inline bool plan_is_small(int P, int few_steps, int items) {
  return P <= few_steps * kFewThreads * kThreadPages && items <= kPerThread * kFewThreads;
}
template <typename Args>
inline cudaError_t launch_plan(void (*kernel)(Args), const Args& a, int P, int few_steps,
                               int items, size_t ints, std::atomic<uint64_t>& ready,
                               cudaStream_t st) {
  const bool few = plan_is_small(P, few_steps, items);
  const int threads = few ? kFewThreads : kPlanThreads;
  int size = 1;
  while (size < kPlanCluster && size < FreePages::steps_of(P, threads) && !few) size *= 2;
  const size_t smem = (FreePages::shared_ints(P, size, threads) + ints) * sizeof(int);
  if (smem > 47 * 1024 && !kernel_smem_ready(kernel, kPlanSmem, ready)) return cudaErrorUnknown;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = size;
  cfg.blockDim = threads;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = size;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  count_launches(1);
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

}  // namespace pa
