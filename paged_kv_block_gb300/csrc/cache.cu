// Which row owns which page, and the copies that follow from it (include/paged_cache.h documents
// the contract): freeing, extending and forking rows, compacting the live pages, copying pages.
//
// A call is at most two kernels.  The first decides: one cluster of CTAs scans the page counts
// and the items in order, so that the k-th fresh page goes to the k-th demand without atomics
// whose order could change the result; its CTAs exchange their totals through distributed shared
// memory.  The second moves: every SM copies runs of contiguous bytes, as many as the first one
// listed.  The first is bound by the latency of its dependent steps (a handful of cluster
// barriers and L2 round trips), the second by HBM.
#include <type_traits>

#include "pages.cuh"

namespace pa {
namespace {

constexpr int kCopyThreads = 256;
constexpr int kCopyChunk = 16384;          // bytes of one copy unit
constexpr int kCopyCtas = 24;              // CTAs per SM where they walk the units (copy_kernel)
// A fork of so little is done by the planning CTA itself, unit after unit: one launch less.  One
// child and its free, by the planning CTA / by a second kernel, in a graph and as calls:
//   2 units (a pool and the table row), 64 KB pages    8.4 /  8.7 us    11.1 / 13.2 us
//   3 units, 16 KB pages                               8.2    8.2       11.0   12.9
//   3 units, 32 KB pages                               9.4    8.8       11.1   12.8
//   3 units, 64 KB pages                              10.4    9.3       11.4   13.5
//   5 units, 8 KB pages                                9.4    7.8       11.0   13.7
//   9                                                 11.5    7.3       12.0   13.7
//   15                                                15.8    8.4       16.4   13.8
// so it stops where a graph, which saves no launch, would lose more than 0.6 us (units times the
// page count as bytes).
constexpr int kOwnUnits = 3;
constexpr int kOwnBytes = 1 << 17;

// ---- fork: shared pages and the copied tail ---------------------------------------------------
struct ForkArgs {
  Pools pools;
  int npools, segs;          // runs of tail bytes per pool: one per head, K and V
  int page_bytes, seg_bytes, token_bytes;
  const int4* items;         // of the planning kernel (PlanArgs::forks)
  const int* page;           // the fresh page of the item, -1 none
  int n;
  int* tables;
  int* refs;
  int C, ps, P;
  int table_units;           // CTAs per item for the table row
  Status status;
};

// One unit of a fork, by a whole CTA: the tail of an item in one pool, or part of its table row.
// It starts with a round trip to L2 for its item and then has four 16-byte words per thread in
// flight: forking 256 children in 8 layers takes 28.6 us in a graph with its frees (28.0 before
// plan_kernel looked at the parents' last pages, 0.6 us for one more dependent read); with one word
// in flight 4 us more; two pools per CTA changed nothing, half a pool per CTA (more round trips)
// cost 5 us, CTAs of 512 threads 3.  The copies then run at 8 to 9 TB/s of L2.
__device__ __forceinline__ void fork_unit(const ForkArgs& a, long long u) {
  const int tid = threadIdx.x, threads = blockDim.x;
  const int per_item = a.npools + a.table_units;
  const int i = static_cast<int>(u / per_item);
  const int w = static_cast<int>(u - static_cast<long long>(i) * per_item);
  const int4 item = a.items[i];
  const int L = item.x, s = item.y, d = a.page[i], parent = item.z;
  if (L < 0) return;
  const int full = L / a.ps;
  const long long from = static_cast<long long>(parent) * a.C;
  if (w < a.npools) {
    if (d < 0) return;
    const int words = (L - full * a.ps) * a.token_bytes / 16, all = words * a.segs;
    uint8_t* base = static_cast<uint8_t*>(a.pools.p[w]);
    const uint8_t* src = base + static_cast<long long>(s) * a.page_bytes;
    uint8_t* dst = base + static_cast<long long>(d) * a.page_bytes;
    // word x of the tail lies in run x / words; the next one of the thread is `threads` further on
    const int runs = threads / words, rest = threads - runs * words;
    int seg = tid / words, at = tid - seg * words;
    for (int x0 = tid; x0 < all; x0 += 4 * threads) {
      uint4 v[4];
      int o[4];
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        o[b] = seg * a.seg_bytes + at * 16;
        if (x0 + b * threads < all) v[b] = ld_stream(reinterpret_cast<const uint4*>(src + o[b]));
        seg += runs;
        at += rest;
        if (at >= words) {
          at -= words;
          ++seg;
        }
      }
#pragma unroll
      for (int b = 0; b < 4; ++b)
        if (x0 + b * threads < all) *reinterpret_cast<uint4*>(dst + o[b]) = v[b];
    }
  } else {
    const long long to = static_cast<long long>(item.w) * a.C;
    for (int j = (w - a.npools) * threads + tid; j < full; j += a.table_units * threads) {
      const int p = a.tables[from + j];
      a.tables[to + j] = p;
      if (p >= 0 && p < a.P) atomicAdd(a.refs + p, 1);
      else report(a.status, kErrMetadata);
    }
  }
}

__global__ void __launch_bounds__(kCopyThreads) fork_kernel(const __grid_constant__ ForkArgs a) {
  grid_dependency_wait();
  grid_launch_dependents();
  const long long units = static_cast<long long>(a.n) * (a.npools + a.table_units);
  for (long long u = blockIdx.x; u < units; u += gridDim.x) fork_unit(a, u);
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
  unsigned long long by_ps;  // ceil(2^64 / ps)
  int hash;                // entries of the table of rows seen, a power of two >= 2 n
  Status status;
  int4* forks;             // workspace [n], fork: the parent's length before the call (-1: left
                           // out), its partly filled page (in the pool), the parent, the child
  int* page;               // workspace [n], fork: the fresh page of the item, -1 none
};
struct ForkPlanArgs : PlanArgs {
  int units;               // units that the (only) CTA does itself; 0: a second kernel does them
  ForkArgs fork;
};
template <bool kFork>
using PlanArgsOf = std::conditional_t<kFork, ForkPlanArgs, PlanArgs>;
struct Item {
  int off;                 // first fresh page of the item among all demands
  int need;                // pages (0: none, or left out)
  int have;                // pages of the row before the call
  int row;
};

// x / page_size, exact for every 32-bit x (x * page_size < 2^64).
__device__ __forceinline__ int over_page(unsigned x, unsigned long long by_ps) {
  return static_cast<int>(__umul64hi(x, by_ps));
}

// CTA 0 looks after the items, all CTAs after the pages.  Latency bounds this kernel where there is
// little to do: the chain is rows -> lengths -> scan -> barrier -> tables, with the counts read
// beside it (6 us for one item in 1,024 pages; a round trip to L2 alone is half a microsecond);
// instructions and barriers of eight SMs where there is much: 13 us for 128 items that get 33,000
// of 262,144 pages, 45 when every page searched for its item and neighbouring lanes stored to
// distant words.
template <bool kFork>
__global__ void __launch_bounds__(kPlanThreads)
plan_kernel(const __grid_constant__ PlanArgsOf<kFork> a) {
  extern __shared__ __align__(16) int shared[];
  __shared__ int warp_sums[32];
  __shared__ int total_need;
  cg::cluster_group cl = cg::this_cluster();
  const int rank = cl.block_rank(), size = cl.num_blocks();
  const int tid = threadIdx.x, threads = blockDim.x;
  Item* items = reinterpret_cast<Item*>(shared);
  int* keys = reinterpret_cast<int*>(items + a.n);             // CTA 0: rows seen, their first item
  Item* mine = reinterpret_cast<Item*>(keys);                  // later: the CTA's copy of the items
  int* item_of = keys + 2 * a.hash;                            // fork: the item of the k-th demand
  int* pages_shared = item_of + (kFork ? a.n : 0);
  // CTA 0: rows, lengths, and the new tokens or (fork) the child's length, then the parent's last
  // page if it is partly filled (else 0)
  int row[kPerThread], L[kPerThread], other[kPerThread];
  uint32_t bits = 0;
  grid_dependency_wait();
  grid_launch_dependents();
  if (rank == 0) {
    if (tid < 4) a.status.ws[tid] = 0;
    for (int i = tid; i < a.hash; i += threads) {
      keys[i] = -1;
      keys[a.hash + i] = a.n;
    }
#pragma unroll
    for (int j = 0; j < kPerThread; ++j) {
      const int i = j * threads + tid;
      if (j * threads >= a.n) break;
      row[j] = i < a.n ? a.rows[i] : -1;
      other[j] = i < a.n ? (kFork ? a.parents[i] : a.new_tokens[i]) : -1;
    }
#pragma unroll
    for (int j = 0; j < kPerThread; ++j) {
      if (j * threads >= a.n) break;
      const int parent = other[j];
      const bool known = row[j] >= 0 && row[j] < a.R &&
                         (!kFork || (parent >= 0 && parent < a.R && parent != row[j]));
      L[j] = -1;
      if (!known) continue;
      L[j] = a.lens[kFork ? parent : row[j]];
      if (kFork) other[j] = a.lens[row[j]];
    }
  }
  // The counts are read while the lengths are on their way, and the parents' last pages after them.
  // Before an item gets a page its parent's last one has to lie in the pool: else the child's would
  // be live without ever having been written.
  FreePages pages;
  pages.count(a.refs, a.P, rank, size, pages_shared, [&] {
    if (!kFork || rank != 0) return;
#pragma unroll
    for (int j = 0; j < kPerThread; ++j) {
      const int i = j * threads + tid;
      if (j * threads >= a.n) break;
      if (L[j] < 0 || other[j] != 0) {                 // left out
        L[j] = -1;
        continue;
      }
      const int full = over_page(L[j], a.by_ps);
      if (full < a.C && full * a.ps < L[j])
        other[j] = a.tables[static_cast<long long>(a.parents[i]) * a.C + full];
    }
  });
  if (rank == 0) {
    int* first = keys + a.hash;
    int need[kPerThread], at[kPerThread], pages_of[kPerThread];
#pragma unroll
    for (int j = 0; j < kPerThread; ++j) {
      if (j * threads >= a.n) break;
      need[j] = -1;
      at[j] = pages_of[j] = 0;
      if (L[j] < 0 || other[j] < 0 || (kFork && other[j] >= a.P)) continue;
      if (!kFork && L[j] > INT_MAX - other[j]) continue;
      const int full = over_page(L[j], a.by_ps), have = over_page(L[j] + a.ps - 1u, a.by_ps);
      const int want = kFork ? have : over_page(L[j] + other[j] + a.ps - 1u, a.by_ps);
      if (want <= a.C) need[j] = kFork ? have - full : want - have;
      pages_of[j] = kFork ? full : have;
    }
    // A row listed more than once belongs to its first item that is in order.
#pragma unroll
    for (int j = 0; j < kPerThread; ++j) {
      if (j * threads >= a.n) break;
      if (need[j] < 0) continue;
      int h = static_cast<int>((static_cast<unsigned>(row[j]) * 2654435769u) >> 8) & (a.hash - 1);
      while (true) {                           // ends: at most half the table is used
        const int key = atomicCAS(keys + h, -1, row[j]);
        if (key == -1 || key == row[j]) break;
        h = (h + 1) & (a.hash - 1);
      }
      atomicMin(first + h, j * threads + tid);
      at[j] = h;
    }
    __syncthreads();
    int carry = 0;
#pragma unroll
    for (int j = 0; j < kPerThread; ++j) {
      const int i = j * threads + tid;
      if (j * threads >= a.n) break;
      if (need[j] >= 0 && first[at[j]] != i) need[j] = -1;
      if (need[j] < 0 && i < a.n) bits |= kErrMetadata;
      const int pages_needed = min(max(need[j], 0), kMaxPages + 1);
      int sum;
      const int before = add_pages(carry, block_scan(pages_needed, warp_sums, &sum));
      carry = add_pages(carry, sum);
      if (i < a.n)
        items[i] = {before, pages_needed, pages_of[j], need[j] < 0 ? -1 : row[j]};
    }
    if (tid == 0) total_need = carry;
  }
  sync_cluster(cl);
  pages.order(cl);
  const int demand = *cl.map_shared_rank(&total_need, 0);
  const Item* from = cl.map_shared_rank(items, 0);
  if (rank == 0) {
#pragma unroll
    for (int j = 0; j < kPerThread; ++j) {
      const int i = j * threads + tid;
      if (j * threads >= a.n) break;
      if (i >= a.n) continue;
      const Item it = items[i];
      const bool served = it.row >= 0 && (it.need == 0 || it.off + it.need <= pages.total);
      if (it.row >= 0 && !served) bits |= kErrCapacity;
      if (served) a.lens[it.row] = kFork ? L[j] : L[j] + other[j];
      if (kFork) {
        a.forks[i] = make_int4(served ? L[j] : -1, other[j], a.parents[i], row[j]);
        if (it.need == 0 || !served) a.page[i] = -1;
      }
    }
    if (bits) report(a.status, bits);
  }
  if (demand > 0) {
    for (int i = tid; i < a.n; i += threads) {
      const Item x = from[i];
      mine[i] = x;
      if (kFork && x.need > 0) item_of[x.off] = i;             // a fork demands one page at most
    }
    __syncthreads();
  }
  // From here on no CTA reads another's shared memory; none may end before all have come here.
  if (size > 1) cluster_arrive();
  if (demand > 0) {
    // The item whose demand holds the k-th fresh page: the last one with off <= k (items without
    // a demand share their successor's offset).
    const auto owner = [&](int k, int lo) {
      int hi = a.n;
      while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (mine[mid].off <= k) lo = mid; else hi = mid;
      }
      return lo;
    };
    // Served items come before the first whose demand the free pages do not hold.
    const int handed = demand <= pages.total ? demand : mine[owner(pages.total, 0)].off;
    int which = 0;
    Item it{0, 0, 0, -1};                              // of the warp's last pages
    for (int j = 0; j < pages.own; ++j) {
      if (pages.step_before[j * size + rank] >= handed) break;
      pages.each(j, [&](int p, bool is_free, int k, int count) {
        const int first = __shfl_sync(0xffffffffu, k, 0), last = min(first + count, handed) - 1;
        if (last < first) return;
        int w = which;
        Item own = it;
        if (kFork) {
          w = item_of[min(k, last)];
          own = mine[w];
        } else if (first < it.off || last >= it.off + it.need) {
          // The warp's fresh pages mostly go to the item of its last ones; here each lane looks
          // for its own.
          w = owner(min(k, last), which);
          own = mine[w];
          which = __shfl_sync(0xffffffffu, w, 31);
          it = mine[which];
        }
        if (!is_free || k > last) return;
        a.tables[static_cast<long long>(own.row) * a.C + own.have + (k - own.off)] = p;
        a.refs[p] = 1;
        if (kFork) a.page[w] = p;
      });
    }
  }
  if constexpr (kFork) {
    if (a.units > 0) {                     // a small fork: no second launch
      __syncthreads();
      for (int u = 0; u < a.units; ++u) fork_unit(a.fork, u);
    }
  }
  if (size > 1) cluster_wait();
}

// ---- copies ----------------------------------------------------------------------------------
// One CTA copies n16 16-byte words.
__device__ __forceinline__ void copy_words(uint4* __restrict__ dst, const uint4* __restrict__ src,
                                           int n16) {
  int i = threadIdx.x;
  for (; i + 3 * kCopyThreads < n16; i += 4 * kCopyThreads) {
    const uint4 a = ld_stream(src + i), b = ld_stream(src + i + kCopyThreads);
    const uint4 c = ld_stream(src + i + 2 * kCopyThreads);
    const uint4 d = ld_stream(src + i + 3 * kCopyThreads);
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
  Status status;
  // compact: table entries to rename
  const int *tables, *lens, *to, *num_live;
  int* tables_out;
  int R, C, ps, P;
};

// A unit is up to kCopyChunk bytes of one page of one pool.  Where the host knows the number of
// pairs there is a CTA per unit; else (compact) four times the CTAs that fit walk the units, each
// reading the next unit's page ids before it copies the present one.
// HBM bounds it.  Measured (64 KB pages): copying 1,201 pages of 8 layers, 630 MB, takes 187 us
// with a CTA per unit, 99% of the rate of a plain copy, and 201 us with 6 resident CTAs per SM that
// walk the units; moving 1,500 pages of 4 layers 127 us a call with 24 CTAs per SM, 134 with 6, and
// the same 134 with a ring of bulk copies through shared memory, so there is none.  Units of 8 KB
// cost 244 us (the CTAs' launches), of 32 KB 190 us.
template <bool kCompact>
__global__ void __launch_bounds__(kCopyThreads) copy_kernel(const __grid_constant__ CopyArgs a) {
  grid_dependency_wait();
  grid_launch_dependents();
  const int n = kCompact ? *a.n_dev : a.n;
  const long long units = static_cast<long long>(n) * a.pools * a.chunks;
  const int per_pair = a.pools * a.chunks;
  const auto pair_of = [&](long long u) { return static_cast<int>(u / per_pair); };
  long long u = blockIdx.x;
  int s = 0, d = 0;
  if (u < units) {
    s = a.src_pages[kCompact ? n - 1 - pair_of(u) : pair_of(u)];
    d = a.dst_pages[pair_of(u)];
  }
  for (; u < units; u += gridDim.x) {
    const int from = s, to = d;
    const long long next = u + gridDim.x;
    if (next < units) {
      s = a.src_pages[kCompact ? n - 1 - pair_of(next) : pair_of(next)];
      d = a.dst_pages[pair_of(next)];
    }
    if (from < 0 || from >= a.src_num_pages || to < 0 || to >= a.dst_num_pages) {
      if (threadIdx.x == 0) report(a.status, kErrMetadata);
      continue;
    }
    const int w = static_cast<int>(u - static_cast<long long>(pair_of(u)) * per_pair);
    const int pool = w / a.chunks, chunk = w - pool * a.chunks;
    if (from == to && a.src.p[pool] == a.dst.p[pool]) continue;
    const long long at = static_cast<long long>(chunk) * kCopyChunk;
    const int bytes = static_cast<int>(min(static_cast<long long>(kCopyChunk), a.page_bytes - at));
    copy_words(
        reinterpret_cast<uint4*>(static_cast<uint8_t*>(a.dst.p[pool]) + to * a.page_bytes + at),
        reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(a.src.p[pool]) +
                                       from * a.page_bytes + at),
        bytes / 16);
  }
  if (kCompact) {
    const int live = *a.num_live;
    const long long entries = static_cast<long long>(a.R) * a.C;
    for (long long e = blockIdx.x * static_cast<long long>(kCopyThreads) + threadIdx.x; e < entries;
         e += static_cast<long long>(gridDim.x) * kCopyThreads) {
      const int row = static_cast<int>(e / a.C);
      const int j = static_cast<int>(e - static_cast<long long>(row) * a.C);
      const int L = a.lens[row];
      int p = a.tables[e];
      const int old = p;
      if (j < (L + a.ps - 1LL) / a.ps) {
        if (p < 0 || p >= a.P) report(a.status, kErrMetadata);
        else if (p >= live) p = a.to[p];
      }
      if (j == 0 && (L + a.ps - 1LL) / a.ps > a.C) report(a.status, kErrMetadata);
      if (p != old || a.tables_out != a.tables) a.tables_out[e] = p;
    }
  }
}

// ---- free ------------------------------------------------------------------------------------
// A CTA per row.  The exchange makes a row that is listed twice free once; three dependent round
// trips to L2 (row, length, pages) and the atomics bound it: 4 us for a row, 5 for 128 rows of 256
// pages.
__global__ void __launch_bounds__(kCopyThreads)
free_kernel(const int* rows, int n, const int* tables, int* lens, int* refs, int R, int C, int ps,
            int P, uint32_t* status) {
  __shared__ int len;
  grid_dependency_wait();
  grid_launch_dependents();
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

// ---- compact: which page moves where ----------------------------------------------------------
struct CompactArgs {
  const int* refs;
  int* refs_out;
  int* num_live;
  int P;
  int *src, *dst, *to, *moves;   // workspace: move lists, new ids of pages >= live, their number
  Status status;
};

// Latency-bound like plan_kernel: 5 us for 256 pages, 8 for 6,007.
__global__ void __launch_bounds__(kPlanThreads) compact_kernel(const CompactArgs a) {
  extern __shared__ __align__(16) int shared[];
  cg::cluster_group cl = cg::this_cluster();
  const int rank = cl.block_rank(), size = cl.num_blocks();
  const int tid = threadIdx.x, threads = blockDim.x;
  grid_dependency_wait();
  grid_launch_dependents();
  if (rank == 0 && tid < 4) a.status.ws[tid] = 0;
  FreePages pages;
  pages.count(a.refs, a.P, rank, size, shared, [] {});
  if (a.refs_out != a.refs) {              // what moves is set right below, after the barriers
    constexpr int kBatch = 8;
    const int stride = size * threads;
    for (int p0 = rank * threads + tid; p0 < a.P; p0 += kBatch * stride) {
      int r[kBatch];
#pragma unroll
      for (int u = 0; u < kBatch; ++u)
        if (p0 + u * stride < a.P) r[u] = a.refs[p0 + u * stride];
#pragma unroll
      for (int u = 0; u < kBatch; ++u)
        if (p0 + u * stride < a.P) a.refs_out[p0 + u * stride] = r[u];
    }
  }
  sync_cluster(cl);
  pages.order(cl);
  const int live = a.P - pages.total;
  if (rank == 0 && tid == 0) {
    *a.num_live = live;
    if (live == a.P) *a.moves = 0;
  }
  // f free and p - f live pages lie before page p.  The f-th hole is p; of the live pages that
  // move, live - 1 - (p - f) come after p, which numbers them without knowing how many they are.
  for (int j = 0; j < pages.own; ++j) {
    pages.each(j, [&](int p, bool is_free, int f, int) {
      if (p >= a.P) return;
      if (p == live) *a.moves = f;                  // holes below `live` = live pages from it on
      if (is_free) {
        if (p < live) a.dst[f] = p;
        else a.to[p] = p;
      } else if (p >= live) {
        a.src[live - 1 - (p - f)] = p;
      }
    });
  }
  sync_cluster(cl);                        // also: every CTA has read the others' step totals
  const int moves = *a.moves;
  for (int k = rank * threads + tid; k < moves; k += size * threads) {
    const int s = a.src[moves - 1 - k], d = a.dst[k];
    a.to[s] = d;
    a.refs_out[d] = a.refs[s];
    a.refs_out[s] = 0;
  }
}

// ---- host --------------------------------------------------------------------------------------
struct PlanLayout {
  size_t status, forks, page, total;
  explicit PlanLayout(int n) {
    Take t;
    status = t.ints(4);
    forks = t.ints(4LL * n);
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

bool same_geometry(const paged_cache_pools* a, const paged_cache_pools* b) {
  return a->num_layers == b->num_layers && a->num_kv_heads == b->num_kv_heads &&
         a->page_size == b->page_size && a->head_dim == b->head_dim &&
         (a->combined_cache != 0) == (b->combined_cache != 0);
}
bool overlap(const void* a, long long na, const void* b, long long nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + static_cast<uintptr_t>(nb) && y < x + static_cast<uintptr_t>(na);
}
template <bool kFork>
cudaError_t launch_items(PlanArgsOf<kFork> a, cudaStream_t st) {
  static std::atomic<uint64_t> ready{0};
  a.hash = 2;
  while (a.hash < 2 * a.n) a.hash *= 2;
  a.by_ps = ~0ull / static_cast<unsigned>(a.ps) + 1;       // ceil(2^64 / ps): ps is even
  return launch_plan(plan_kernel<kFork>, a, a.P, 4, a.n,
                     (kFork ? 5 : 4) * static_cast<size_t>(a.n) + 2 * a.hash, ready, st);
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
  if (!rows || !tables || !lens || !refs || !ints_aligned(rows, tables, lens, refs, status))
    return PAGED_ATTN_ERR_INVALID_ARGUMENT;
  count_launches(1);
  return cuda_status(launch_after_previous(
      free_kernel, n, kCopyThreads, 0, static_cast<cudaStream_t>(stream), rows, n, tables, lens,
      refs, p->rows, p->max_pages_per_request, p->page_size, p->num_pages, status));
}

size_t paged_cache_extend_workspace_size(int n) {
  return n < 0 || n > kMaxItems ? 0 : PlanLayout(0).total;      // the status word
}
size_t paged_cache_fork_workspace_size(int n) {
  return n < 0 || n > kMaxItems ? 0 : PlanLayout(n).total;
}
size_t paged_cache_compact_workspace_size(int num_pages) {
  return num_pages <= 0 || num_pages > kMaxPages ? 0 : CompactLayout(num_pages).total;
}

int paged_cache_extend_run(const paged_cache_params* p, const int32_t* rows,
                           const int32_t* new_tokens, int n, int32_t* tables, int32_t* lens,
                           int32_t* refs, void* ws, size_t ws_bytes, void* stream) {
  if (!cache_params_ok(p) || n < 0 || n > kMaxItems) return PAGED_ATTN_ERR_INVALID_ARGUMENT;
  if (n > 0 && (!rows || !new_tokens || !tables || !lens || !refs))
    return PAGED_ATTN_ERR_INVALID_ARGUMENT;
  if (!ints_aligned(rows, new_tokens, tables, lens, refs) || !aligned_to(ws, 16))
    return PAGED_ATTN_ERR_INVALID_ARGUMENT;
  const PlanLayout l(0);
  if (!ws || ws_bytes < l.total) return PAGED_ATTN_ERR_WORKSPACE;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (n == 0) return cuda_status(cudaMemsetAsync(ws, 0, 4 * sizeof(uint32_t), st));
  PlanArgs a{};
  a.rows = rows; a.new_tokens = new_tokens; a.n = n;
  a.tables = tables; a.lens = lens; a.refs = refs;
  a.R = p->rows; a.C = p->max_pages_per_request; a.ps = p->page_size; a.P = p->num_pages;
  a.status = {reinterpret_cast<uint32_t*>(at(ws, l.status)), p->status_dev};
  return cuda_status(launch_items<false>(a, st));
}

int paged_cache_fork_run(const paged_cache_params* p, const paged_cache_pools* pools,
                         const int32_t* parents, const int32_t* children, int n, int32_t* tables,
                         int32_t* lens, int32_t* refs, void* ws, size_t ws_bytes, void* stream) {
  if (!cache_params_ok(p) || !pools_ok(pools) || n < 0 || n > kMaxItems)
    return PAGED_ATTN_ERR_INVALID_ARGUMENT;
  if (pools->num_pages != p->num_pages || pools->page_size != p->page_size)
    return PAGED_ATTN_ERR_INVALID_ARGUMENT;
  if (n > 0 && (!parents || !children || !tables || !lens || !refs))
    return PAGED_ATTN_ERR_INVALID_ARGUMENT;
  if (!ints_aligned(parents, children, tables, lens, refs) || !aligned_to(ws, 16))
    return PAGED_ATTN_ERR_INVALID_ARGUMENT;
  const PlanLayout l(n);
  if (!ws || ws_bytes < l.total) return PAGED_ATTN_ERR_WORKSPACE;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (n == 0) return cuda_status(cudaMemsetAsync(ws, 0, 4 * sizeof(uint32_t), st));
  ForkPlanArgs a{};
  a.rows = children; a.parents = parents; a.n = n;
  a.tables = tables; a.lens = lens; a.refs = refs;
  a.R = p->rows; a.C = p->max_pages_per_request; a.ps = p->page_size; a.P = p->num_pages;
  a.status = {reinterpret_cast<uint32_t*>(at(ws, l.status)), p->status_dev};
  a.forks = reinterpret_cast<int4*>(at(ws, l.forks)); a.page = at(ws, l.page);
  ForkArgs& f = a.fork;
  f.npools = pool_count(pools);
  for (int i = 0; i < f.npools; ++i) f.pools.p[i] = pools->pools_host[i];
  f.segs = (pools->combined_cache ? 2 : 1) * pools->num_kv_heads;
  f.page_bytes = static_cast<int>(page_bytes(pools));
  f.seg_bytes = static_cast<int>(seg_bytes(pools));
  f.token_bytes = 2 * pools->head_dim;
  f.items = a.forks; f.page = a.page;
  f.n = n;
  f.tables = tables; f.refs = refs;
  f.C = a.C; f.ps = a.ps; f.P = a.P;
  f.table_units = ceil_div(a.C, 4 * kCopyThreads);
  f.status = a.status;
  const long long units = static_cast<long long>(n) * (f.npools + f.table_units);
  // A few small pages: the planning CTA copies them itself.
  if (plan_is_small(a.P, 4, n) && units <= kOwnUnits && units * f.page_bytes <= kOwnBytes)
    a.units = static_cast<int>(units);
  if (launch_items<true>(a, st) != cudaSuccess) return PAGED_ATTN_ERR_CUDA;
  if (a.units > 0) return PAGED_ATTN_OK;
  count_launches(1);
  return cuda_status(launch_after_previous(fork_kernel,
                                           static_cast<int>(units < kMaxGrid ? units : kMaxGrid),
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
  if (!ints_aligned(tables, lens, refs, tables_out, refs_out, num_live) || !aligned_to(ws, 16))
    return PAGED_ATTN_ERR_INVALID_ARGUMENT;
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
  a.status = {reinterpret_cast<uint32_t*>(at(ws, l.status)), p->status_dev};
  static std::atomic<uint64_t> ready{0};
  if (launch_plan(compact_kernel, a, a.P, 1, 0, 0, ready, st) != cudaSuccess)
    return PAGED_ATTN_ERR_CUDA;
  CopyArgs c{};
  c.pools = pool_count(pools);
  for (int i = 0; i < c.pools; ++i) c.src.p[i] = c.dst.p[i] = pools->pools_host[i];
  c.src_pages = a.src; c.dst_pages = a.dst; c.n_dev = a.moves;
  c.src_num_pages = c.dst_num_pages = p->num_pages;
  c.page_bytes = page_bytes(pools);
  c.chunks = static_cast<int>(ceil_div_ll(c.page_bytes, kCopyChunk));
  c.status = a.status;
  c.tables = tables; c.lens = lens; c.to = a.to; c.num_live = num_live; c.tables_out = tables_out;
  c.R = p->rows; c.C = p->max_pages_per_request; c.ps = p->page_size; c.P = p->num_pages;
  const int sms = current_sm_count();
  if (sms <= 0) return PAGED_ATTN_ERR_CUDA;
  // at most half the pages can move; the table's entries want threads too
  const long long units = (p->num_pages / 2LL) * c.pools * c.chunks;
  const long long renames = ceil_div_ll(static_cast<long long>(c.R) * c.C, kCopyThreads);
  long long ctas = units > renames ? units : renames;
  if (ctas > kCopyCtas * sms) ctas = kCopyCtas * sms;
  count_launches(1);
  return cuda_status(launch_after_previous(copy_kernel<true>, static_cast<int>(ctas > 0 ? ctas : 1),
                                           kCopyThreads, 0, st, c));
}

int paged_cache_copy_run(const paged_cache_pools* src, const paged_cache_pools* dst,
                         const int32_t* src_pages, const int32_t* dst_pages, int n,
                         uint32_t* status, void* stream) {
  if (!pools_ok(src) || !pools_ok(dst) || !same_geometry(src, dst) || n < 0)
    return PAGED_ATTN_ERR_INVALID_ARGUMENT;
  if (n == 0) return PAGED_ATTN_OK;
  if (!src_pages || !dst_pages || !ints_aligned(src_pages, dst_pages, status))
    return PAGED_ATTN_ERR_INVALID_ARGUMENT;
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
  c.status = {nullptr, status};
  const long long units = static_cast<long long>(n) * c.pools * c.chunks;
  const long long most = kMaxGrid;
  count_launches(1);
  return cuda_status(launch_after_previous(copy_kernel<false>,
                                           static_cast<int>(units < most ? units : most),
                                           kCopyThreads, 0, static_cast<cudaStream_t>(stream), c));
}

}  // extern "C"
