// Decode attention for requests that share a prefix (include/paged_attn.h documents the contract):
// the plan and the final merge.  The prefix of a group is attended once for all of its rows (query,
// head) by the tensor-core kernel, its keys split over CTAs; what each request has of its own by
// tail_kernel, or the split-KV decode kernel where it has many rows; all leave normalised fp32
// partials with their log-sum-exp.
#include <climits>

#include "common.cuh"
#include "internal.h"

namespace pa {
namespace {

constexpr int kThreads = 1024;             // of the planning CTA, or
constexpr int kFewThreads = 256;           // for so many groups and requests
constexpr int kD = 128;
constexpr float kLn2 = 0.6931471805599453f;
// SM time in microseconds of a step of 256 rows (128, where a group has no more) and 128 keys, and
// of 128 keys of a tail, as measured: the SMs are shared out by them.
constexpr float kStepCost = 2.0f, kHalfStepCost = 1.2f, kTailCost = 2.1f;
constexpr float kTileCost = 4.0f;          // of a part of a prefix besides its steps
constexpr int kPartChoices = 32;           // lengths of parts that are weighed up, one per lane
constexpr int kOrdered = 1024;             // groups that are ordered by the lengths of their parts

// Two sums in one 64-bit word: the upper and the lower half.
__device__ __forceinline__ long long pack(long long upper, int lower) {
  return upper << 32 | static_cast<unsigned>(lower);
}
__device__ __forceinline__ int upper_of(long long x) { return static_cast<int>(x >> 32); }
__device__ __forceinline__ int lower_of(long long x) { return static_cast<int>(x); }
// Exclusive prefix sum over the CTA.
__device__ __forceinline__ long long block_scan(long long x, long long* warp_sums,
                                                long long* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const auto inclusive = [&](long long v) {
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
      const long long y = __shfl_up_sync(0xffffffffu, v, d);
      if (lane >= d) v += y;
    }
    return v;
  };
  const long long v = inclusive(x);
  if (lane == 31) warp_sums[warp] = v;
  __syncthreads();
  const long long w = inclusive(lane < static_cast<int>(blockDim.x >> 5) ? warp_sums[lane] : 0);
  const long long before = __shfl_sync(0xffffffffu, w, (warp + 31) & 31);
  *total = __shfl_sync(0xffffffffu, w, 31);
  __syncthreads();
  return (warp > 0 ? before : 0) + v - x;
}

__device__ __forceinline__ int ceil_tiles(int keys) { return (keys + kKvTile - 1) / kKvTile; }

// One CTA.  Groups: the prefix that may be shared (no longer than what every query of every member
// sees, so that no mask is needed in it; members of length 0, such as a batch is padded with, see
// nothing and have no say), tiles of up to 256 rows, and equal key parts.  Requests:
// what is left, split as decode splits it.  The kernels of the two run side by side, a prefix CTA
// or two tail CTAs on an SM, so the prefixes are cut into parts for their share of the SMs: 64
// requests with tails of some 300 keys behind 8,192 common ones took 64 us with parts for all SMs,
// one kernel after the other.  Latency bounds this kernel: the lengths stay in shared memory (up
// to kHeld requests), tiles and items are counted in one scan.
constexpr int kHeld = 8192;
__global__ void __launch_bounds__(kThreads)
shared_plan_kernel(const __grid_constant__ SharedLaunch a) {
  // Shared memory: lengths, shared keys and first splits of the requests, and the groups' offsets,
  // or, where those are too many, the arrays in global memory.
  extern __shared__ int held[];
  __shared__ long long sums[32];
  __shared__ float costs[3][32];
  __shared__ float items_at[kPartChoices];
  __shared__ int chosen[2], sizes[kOrdered], order[kOrdered];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int threads = blockDim.x, warps = threads >> 5;
  const bool hold = a.B <= kHeld, hold_groups = a.groups <= kOrdered;
  int* prefix = hold ? held + a.B : a.prefix_of;
  int* split_at = hold ? held + 2 * a.B : a.split_offset;
  int* first_of = held + (hold ? 3 * a.B + 1 : 0);
  grid_dependency_wait();
  grid_launch_dependents();
  if (tid < 4) a.status[tid] = 0;
  if (tid == 0) *a.work_counter = 0;
  const auto length_of = [&](int b) { return min(max(a.lens[b], 0), a.max_len); };
  bool bad = false;
  for (int g = tid; g <= a.groups; g += threads) {
    const int at = a.group_indptr[g];
    bad |= at < 0 || at > a.B || (g > 0 && a.group_indptr[g - 1] > at);
    if (hold_groups) first_of[g] = at;
  }
  for (int b = tid; b < a.B; b += threads) {
    if (hold) held[b] = length_of(b);
    prefix[b] = 0;
  }
  bad = __syncthreads_or(bad);
  if (bad && tid == 0) report_error(a.status, kErrMetadata);
  const int groups = bad ? 0 : a.groups;
  const auto start = [&](int g) { return hold_groups ? first_of[g] : a.group_indptr[g]; };
  const auto length = [&](int b) { return hold ? held[b] : length_of(b); };
  // the first item of a tail starts at the prefix, the others at multiples of their unit from here
  const auto tail_base = [&](int p) { return p / a.item_unit * a.item_unit; };
  const auto tail_units = [&](int b) {
    const int keys = length(b) - tail_base(prefix[b]);
    return keys > 0 ? (keys + a.item_unit - 1) / a.item_unit : 0;
  };
  // a warp per group
  const int tile_tokens = 2 * (kMTileRows / a.G);
  for (int g = warp; g < groups; g += warps) {
    const int first = start(g), last = start(g + 1);
    int n = a.prefix_lens[g], members = 0;
    if (last - first < 2) continue;
    for (int b = first + lane; b < last; b += 32) {
      if (length(b) == 0) continue;
      n = min(n, a.causal ? length(b) - a.SQ + 1 : length(b));     // what all queries of b see
      ++members;
    }
    n = __reduce_min_sync(0xffffffffu, n);
    if (n <= 0 || __reduce_add_sync(0xffffffffu, members) < 2) continue;
    for (int b = first + lane; b < last; b += 32) prefix[b] = n;
  }
  __syncthreads();
  // a thread per group and per request: steps of 128 keys of all tiles, and of all tails
  const auto row_tiles = [&](int g) {
    const int first = start(g), last = start(g + 1);
    if (last <= first || prefix[first] == 0) return 0;
    return ((last - first) * a.SQ + tile_tokens - 1) / tile_tokens;
  };
  const auto step_cost = [&](int g) {
    const int tokens = (start(g + 1) - start(g)) * a.SQ;
    return 2 * tokens <= tile_tokens ? kHalfStepCost : kStepCost;
  };
  float steps = 0.f, cost = 0.f, tails = 0.f;    // of the tiles; units of the tails
  for (int g = tid; g < groups; g += threads) {
    const int rows = row_tiles(g);
    if (rows == 0) continue;
    const float n = static_cast<float>(rows) * ceil_tiles(prefix[start(g)]);
    steps += n;
    cost += n * step_cost(g);
  }
  for (int b = tid; b < a.B; b += threads) tails += static_cast<float>(tail_units(b));
#pragma unroll
  for (int d = 16; d > 0; d /= 2) {
    steps += __shfl_xor_sync(0xffffffffu, steps, d);
    cost += __shfl_xor_sync(0xffffffffu, cost, d);
    tails += __shfl_xor_sync(0xffffffffu, tails, d);
  }
  if (lane == 0) {
    costs[0][warp] = steps;
    costs[1][warp] = cost;
    costs[2][warp] = tails;
  }
  if (tid < kPartChoices) items_at[tid] = 0.f;
  __syncthreads();
  // Keys (in tiles) of a part: a choice per lane.  Few long parts leave CTAs idle at the end, many
  // short ones pay kTileCost more often and write more partials.
  const int choice = 1 << (lane / 2) | (lane & 1 ? 1 << (lane / 2) >> 1 : 0);   // 1 1 2 3 4 6 8 ..
  for (int g = warp; g < groups; g += warps) {
    const int rows = row_tiles(g);
    if (rows > 0)
      atomicAdd(&items_at[lane],           // (exact below 2^24)
                static_cast<float>(rows) *
                    ((ceil_tiles(prefix[start(g)]) + choice - 1) / choice));
  }
  __syncthreads();
  if (warp == 0) {
    float x = lane < warps ? costs[0][lane] : 0.f, y = lane < warps ? costs[1][lane] : 0.f;
    float z = lane < warps ? costs[2][lane] : 0.f;
#pragma unroll
    for (int d = 16; d > 0; d /= 2) {
      x += __shfl_xor_sync(0xffffffffu, x, d);
      y += __shfl_xor_sync(0xffffffffu, y, d);
      z += __shfl_xor_sync(0xffffffffu, z, d);
    }
    x *= a.Hkv;
    y *= a.Hkv;
    z *= a.Hkv;
    // the prefixes' share of the SMs, and the time that a choice takes on it
    const float each = x > 0.f ? y / x : 0.f, count = items_at[lane] * a.Hkv;
    const float work = y + count * kTileCost;
    const float share = work / (work + kTailCost * z * a.item_unit / kKvTile + 1e-6f);
    const int ctas = max(static_cast<int>(a.sms * share + 0.5f), 1);
    const float longest = choice * each + kTileCost;
    float time = count <= ctas ? longest : work / ctas + 0.5f * longest;
    if (count > a.tile_capacity || choice > kPartTiles) time = 3.4e38f;    // (kPartTiles fits)
    const uint32_t best = __reduce_min_sync(0xffffffffu, __float_as_uint(time));
    const int pick = __ffs(__ballot_sync(0xffffffffu, __float_as_uint(time) == best)) - 1;
    if (lane == pick) {
      chosen[0] = choice;
      *a.max_ctas = ctas;
    }
    const float aim = static_cast<float>(a.items_per_sm * a.sms);
    if (lane == 0) chosen[1] = max(static_cast<int>(ceilf(z / aim)), 1);
  }
  __syncthreads();
  const int part = chosen[0], chunk = chosen[1];   // in tiles of 128 keys, in units of the tails
  const auto splits_of = [&](int b) {      // of the tail of request b
    return length(b) > prefix[b] ? (tail_units(b) + chunk - 1) / chunk : 0;
  };
  // Groups with the longest parts first, where they are few enough to be ordered by counting.
  const bool ordered = groups <= threads && groups <= kOrdered;
  if (ordered) {
    const auto size_of = [&](int g) {
      if (row_tiles(g) == 0) return 0;
      const int keys = ceil_tiles(prefix[start(g)]), n = (keys + part - 1) / part;
      return (keys + n - 1) / n;
    };
    if (tid < groups) sizes[tid] = size_of(tid);
    __syncthreads();
    if (tid < groups) {
      int rank = 0;
      const int mine = sizes[tid];
      for (int g = 0; g < groups; ++g) rank += sizes[g] > mine || (sizes[g] == mine && g < tid);
      order[rank] = tid;
    }
    __syncthreads();
  }
  // tiles before each group, items before each request
  int tiles = 0, items = 0;
  for (int x0 = 0; x0 < max(groups, a.B); x0 += threads) {
    const int x = x0 + tid, g = x < groups && ordered ? order[x] : x;
    int rows = 0, splits = 0;
    if (x < groups) rows = row_tiles(g);
    if (rows > 0) splits = (ceil_tiles(prefix[start(g)]) + part - 1) / part;
    const int n = x < a.B ? splits_of(x) : 0;
    long long total;
    const long long before =
        block_scan(pack(static_cast<long long>(rows) * splits * a.Hkv, n), sums, &total);
    if (rows > 0)                          // the group's first request keeps it for all of them
      a.refs[start(g)] = {tiles + upper_of(before), splits, rows, 0};
    if (x < a.B) split_at[x] = items + lower_of(before);
    tiles += upper_of(total);
    items += lower_of(total);
  }
  // (cannot be: the capacities are these sums' bounds)
  const bool fits = tiles <= a.tile_capacity &&
                    static_cast<long long>(items) * a.Hkv <= a.item_capacity;
  if (!fits) {
    tiles = items = 0;
    if (tid == 0) report_error(a.status, kErrCapacity);
    __syncthreads();
    for (int b = tid; b < a.B; b += threads) split_at[b] = 0;
  }
  if (tid == 0) {
    *a.n_tiles = tiles;
    a.split_offset[a.B] = items;
  }
  __syncthreads();
  for (int b = tid; b < a.B; b += threads) {
    if (hold) {
      a.prefix_of[b] = prefix[b];
      a.split_offset[b] = split_at[b];
    }
    // requests outside every group, or in one that shares nothing
    if (prefix[b] == 0 || !fits) a.refs[b] = {0, 0, 0, 0};
  }
  for (int g = warp; fits && g < groups; g += warps) {
    const int rows = row_tiles(g);
    if (rows == 0) continue;
    const int first = start(g), last = start(g + 1);
    const int keys = ceil_tiles(prefix[first]);
    const PrefixRef ref = a.refs[first];
    __syncwarp();
    int reader = last;                     // the first member that has the prefix
    for (int b = first + lane; b < last; b += 32) {
      const bool empty = length(b) == 0;
      if (!empty) reader = min(reader, b);
      a.refs[b] = {ref.base, empty ? 0 : ref.splits, ref.row_tiles, (b - first) * a.SQ};
    }
    reader = __reduce_min_sync(0xffffffffu, reader);
    const int tokens = (last - first) * a.SQ, count = rows * ref.splits * a.Hkv;
    for (int k = lane; k < count; k += 32) {
      const int s = k % ref.splits, r = k / ref.splits % rows, h = k / ref.splits / rows;
      TileRec t;
      t.b = reader;
      t.g = h;
      t.tok0 = r * tile_tokens;
      t.ntok = min(tile_tokens, tokens - t.tok0);
      t.kv_begin = static_cast<int>(static_cast<long long>(s) * keys / ref.splits);
      t.kv_end = static_cast<int>(static_cast<long long>(s + 1) * keys / ref.splits);
      t.q_row0 = first * a.SQ + t.tok0;
      t.pad = ref.base + k;
      a.tiles[ref.base + k] = t;
    }
  }
  // a thread per request and KV head
  for (int x = tid; items > 0 && x < a.B * a.Hkv; x += threads) {
    const int b = x / a.Hkv, h = x - b * a.Hkv, n = splits_of(b);
    const int L = length(b), p = prefix[b];
    SplitItem* to = a.items + static_cast<long long>(split_at[b]) * a.Hkv + h * n;
    for (int s = 0; s < n; ++s) {
      SplitItem it;
      it.b = b;
      it.g = h;
      it.kv_begin = s == 0 ? p : tail_base(p) + s * chunk * a.item_unit;
      it.kv_end = s == n - 1 ? L : tail_base(p) + (s + 1) * chunk * a.item_unit;
      to[s] = it;
    }
  }
}

// What a request has of its own, for up to 16 rows (query, head) of a KV head: a warp per item, 16
// keys at a time through warp MMAs, S = Q K^T and O += P V.  Tails are short, so what CTA barriers
// and a combine of warps cost per item counts (16,000 cycles for an item of 170 keys on the decode
// kernel, a third of them its keys); here every warp has a ring of its own, three steps deep, that
// its lanes fill by asynchronous copies, with the next item's steps where its own are all under
// way, and the warps of an SM (eight) share nothing.  Rows that are no key of the item are zeros in
// the ring.  Operands come from shared memory 16 bytes a lane, 16-byte words swapped by row:
//   K   the contraction runs over columns in any order, so a lane takes 16 bytes of its key's row
//       as its operands of two MMAs;
//   V   a lane takes 16 bytes, columns 8 g .. 8 g + 7, of the four keys of its operand; a register
//       pairs two keys at one column, and column 8 n + j is column n of output tile j.
// 160 MB of tails of 170 keys, 16 rows, take 42 us cold and by themselves; 58 us on the decode
// kernel, 66 us with loads from HBM straight into the operands (too few in flight), 43 us with TMA
// boxes of 16 rows.
constexpr int kTailThreads = 128, kTailStages = 3;
constexpr int kStepKeys = 16, kStepHalf = kStepKeys * 128, kStepBytes = 4 * kStepHalf;
constexpr int kTailSmem = kTailThreads / 32 * kTailStages * kStepBytes + 1024;

template <bool kRowMask>
__global__ void __launch_bounds__(kTailThreads, 2)
tail_kernel(const __grid_constant__ SharedLaunch a) {
  extern __shared__ uint8_t raw[];
  const int lane = threadIdx.x & 31, gr = lane >> 2, tq = lane & 3;
  uint8_t* ring = smem_align<1024>(raw) + (threadIdx.x >> 5) * kTailStages * kStepBytes;
  // (__ldcg: behind the prefixes, whose kernel has waited for the plan, this one has not)
  if (!a.behind_prefix) grid_dependency_wait();
  const int items = launch_aborted(a.status) ? 0 : a.Hkv * __ldcg(a.split_offset + a.B);
  const auto claim = [&] {
    int x = 0;
    if (lane == 0) x = atomicAdd(a.work_counter, 1);
    return __shfl_sync(0xffffffffu, x, 0);
  };
  const int M = a.SQ * a.G, ps = a.ps;
  const unsigned long long by_ps = ~0ull / static_cast<unsigned>(ps) + 1;    // ceil(2^64 / ps)
  // Copies of a step: 8 times two rows of K, and of V, 16 bytes a lane.
  const int copy_row = lane >> 4, copy_chunk = lane & 15;
  const uint32_t copy_to = smem_u32(ring) + (copy_chunk >> 3) * kStepHalf + copy_row * 128;
  int issued = 0, used = 0;                // steps, over all items
  // The item whose steps are being issued, which may be the one after the one that is computed: its
  // id is claimed, its record and the place of its pages are read in the steps before, so that no
  // item starts with those round trips (5 us).
  int to_h = 0, to_first = 0, to_begin = 0, to_end = 0, to_step = 0, to_steps = 0;
  int ahead[2] = {-1, -1};                 // pages of the next step's keys 0 .. 7 and 8 .. 15
  const int* to_pages = nullptr;
  const auto look_ahead = [&] {
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      const int key = to_first + to_step * kStepKeys + 8 * p;
      ahead[p] = -1;
      if (to_step < to_steps && key < to_end && key + 8 > to_begin) {
        ahead[p] = __ldg(to_pages + __umul64hi(static_cast<unsigned>(key), by_ps));
        if (ahead[p] < 0) ahead[p] = INT_MAX;                // no page of the pool
      }
    }
  };
  const auto issue_from = [&](const int4& rec, int indptr) {
    to_h = rec.y;
    to_begin = rec.z;
    to_end = rec.w;
    to_first = to_begin / kStepKeys * kStepKeys;
    to_steps = (to_end - to_first + kStepKeys - 1) / kStepKeys;
    to_step = 0;
    to_pages = a.kv_indices + indptr;
    look_ahead();
  };
  const auto issue = [&] {                 // the next step of that item
    const int key0 = to_first + to_step * kStepKeys;
    const uint32_t to = copy_to + issued % kTailStages * kStepBytes;
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      const int key8 = key0 + 8 * p, page = ahead[p];
      const bool in = page >= 0 && page < a.num_pages;
      if (page >= a.num_pages) report_error(a.status, kErrMetadata);
      const int slot =
          key8 - static_cast<int>(__umul64hi(static_cast<unsigned>(key8), by_ps)) * ps;
      // (in bounds also where nothing is copied)
      const long long row = in ? static_cast<long long>(page) * a.page_rows + to_h * ps + slot : 0;
      const __nv_bfloat16* k = a.k + row * kD + copy_row * kD + copy_chunk * 8;
      const __nv_bfloat16* v = a.v + (in ? a.v_head_off * static_cast<long long>(kD) : 0) +
                               row * kD + copy_row * kD + copy_chunk * 8;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = 8 * p + 2 * i + copy_row, key = key0 + r;
        const uint32_t bytes = in && key >= to_begin && key < to_end ? 16u : 0u;
        const uint32_t at = to + (8 * p + 2 * i) * 128 + (((copy_chunk & 7) ^ (r & 7)) << 4);
        cp_async16(at, k + (bytes ? i * 2 * kD : 0), bytes);
        cp_async16(at + 2 * kStepHalf, v + (bytes ? i * 2 * kD : 0), bytes);
      }
    }
    cp_async_commit();
    ++issued;
    ++to_step;
    look_ahead();
  };
  int item = claim();
  int4 it = make_int4(0, 0, 0, 0);
  if (item < items) {
    it = __ldcg(reinterpret_cast<const int4*>(a.items + item));
    issue_from(it, a.kv_indptr[it.x]);
    while (issued < kTailStages && to_step < to_steps) issue();
  }
  while (item < items) {
    const int b = it.x, h = it.y, begin = it.z, end = it.w;
    const int L = kRowMask ? a.lens[b] : 0;
    const int first = begin / kStepKeys * kStepKeys;
    const int steps = (end - first + kStepKeys - 1) / kStepKeys;
    int next = items, next_indptr = 0, claimed = 0;
    int4 next_it = make_int4(0, 0, 0, 0);
    bool onward = false;                   // the steps being issued are the next item's
    if (lane == 0) claimed = atomicAdd(a.work_counter, 1);
    // rows gr and gr + 8 of Q, and how far they see
    uint4 qa[4], qb[4];
    int high[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int m = gr + 8 * r, i = m / a.G;
      const uint4* src = reinterpret_cast<const uint4*>(
          a.q + ((static_cast<long long>(b) * a.SQ + i) * a.Hq + h * a.G + m - i * a.G) * kD +
          tq * 8);
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const uint4 v = m < M ? __ldg(src + x * 4) : make_uint4(0u, 0u, 0u, 0u);
        if (r == 0) qa[x] = v; else qb[x] = v;
      }
      high[r] = kRowMask && m < M ? min(end, L - a.SQ + i + 1) : end;
    }
    float o[16][4];
#pragma unroll
    for (int j = 0; j < 16; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;
    float top[2] = {-INFINITY, -INFINITY}, sum[2] = {0.f, 0.f};
    for (int step = 0; step < steps; ++step, ++used) {
      const int slot = used % kTailStages;
      // this step's group has landed when at most the later ones are pending
      const int later = issued - used - 1;
      if (later >= 2) cp_async_wait<2>();
      else if (later == 1) cp_async_wait<1>();
      else cp_async_wait<0>();
      __syncwarp();
      if (step == 0) {
        next = __shfl_sync(0xffffffffu, claimed, 0);
        if (next < items) next_it = __ldcg(reinterpret_cast<const int4*>(a.items + next));
      } else if (step == 1 && next < items) {
        next_indptr = a.kv_indptr[next_it.x];
      }
      const uint8_t* st = ring + slot * kStepBytes;
      const int key0 = first + step * kStepKeys;
      // scores of rows gr, gr + 8 and keys 8 n + 2 tq, + 1
      float s[2][4];
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          // key gr + 8 n, columns 32 i + 8 tq ..
          const uint4 k = *reinterpret_cast<const uint4*>(
              st + (i >> 1) * kStepHalf + (gr + 8 * n) * 128 + ((((i & 1) * 4 + tq) ^ gr) << 4));
          const uint32_t a0[4] = {qa[i].x, qb[i].x, qa[i].y, qb[i].y};
          const uint32_t a1[4] = {qa[i].z, qb[i].z, qa[i].w, qb[i].w};
          mma_16816(s[n], a0, k.x, k.y);
          mma_16816(s[n], a1, k.z, k.w);
        }
      }
      float best[2] = {-INFINITY, -INFINITY};
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int r = e >> 1, key = key0 + 8 * n + 2 * tq + (e & 1);
          s[n][e] = key >= begin && key < high[r] ? s[n][e] * a.scale_log2 : -INFINITY;
          best[r] = fmaxf(best[r], s[n][e]);
        }
      // The maximum in use moves only when it is exceeded by more than 8 (powers of two), so O is
      // rarely rescaled; the quotient at the end does not depend on it.
      float fade[2] = {1.f, 1.f};
      bool moved = false;
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        best[r] = fmaxf(best[r], __shfl_xor_sync(0xffffffffu, best[r], 1));
        best[r] = fmaxf(best[r], __shfl_xor_sync(0xffffffffu, best[r], 2));
        if (best[r] > top[r] + 8.f) {
          fade[r] = top[r] == -INFINITY ? 0.f : fast_exp2(top[r] - best[r]);
          top[r] = best[r];
          moved = true;
        }
      }
      const float shift[2] = {top[0] == -INFINITY ? 0.f : top[0],
                              top[1] == -INFINITY ? 0.f : top[1]};
      // P in bf16, as everywhere in this library: its rounding (2^-8 of a probability at most) is
      // averaged over the keys; the sums are of the unrounded ones
      uint32_t p[4];
      float add[2] = {0.f, 0.f};
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const float p0 = fast_exp2(s[n][2 * r] - shift[r]);
          const float p1 = fast_exp2(s[n][2 * r + 1] - shift[r]);
          add[r] += p0 + p1;
          p[2 * n + r] = pack_bf16(p0, p1);
        }
      sum[0] = sum[0] * fade[0] + add[0];
      sum[1] = sum[1] * fade[1] + add[1];
      if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          o[j][0] *= fade[0];
          o[j][1] *= fade[0];
          o[j][2] *= fade[1];
          o[j][3] *= fade[1];
        }
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        uint4 v[4];                        // keys 2 tq, + 1, + 8, + 9; columns 64 i + 8 gr ..
#pragma unroll
        for (int n = 0; n < 4; ++n) {
          const int row = 2 * tq + (n & 1) + (n & 2) * 4;
          v[n] = *reinterpret_cast<const uint4*>(st + (2 + i) * kStepHalf + row * 128 +
                                                 ((gr ^ (row & 7)) << 4));
        }
        const auto word = [](const uint4& x, int w) {
          return w == 0 ? x.x : (w == 1 ? x.y : (w == 2 ? x.z : x.w));
        };
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int sel = j & 1 ? 0x7632 : 0x5410;
          mma_16816(o[8 * i + j], p,
                    __byte_perm(word(v[0], j / 2), word(v[1], j / 2), sel),
                    __byte_perm(word(v[2], j / 2), word(v[3], j / 2), sel));
        }
      }
      __syncwarp();                        // every lane has read the step
      // the ring is full again, with steps of the next item where this one's are all issued
      const int most = used + 1 + kTailStages;
      while (issued < most && to_step < to_steps) issue();
      if (!onward && to_step >= to_steps && next < items) {
        if (step == 0) next_indptr = a.kv_indptr[next_it.x];
        issue_from(next_it, next_indptr);
        onward = true;
        while (issued < most && to_step < to_steps) issue();
      }
    }
    // this lane's columns 64 i + 16 tq .. + 15 of rows gr and gr + 8
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      sum[r] += __shfl_xor_sync(0xffffffffu, sum[r], 1);
      sum[r] += __shfl_xor_sync(0xffffffffu, sum[r], 2);
      const int m = gr + 8 * r;
      if (m >= M) continue;
      const long long to = static_cast<long long>(item) * M + m;
      const float inv = sum[r] > 0.f ? 1.f / sum[r] : 0.f;
      float* out = a.tail_o + to * kD + tq * 16;
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
          for (int j = 0; j < 8; j += 4)
            *reinterpret_cast<float4*>(out + i * 64 + e * 8 + j) = make_float4(
                o[8 * i + j][2 * r + e] * inv, o[8 * i + j + 1][2 * r + e] * inv,
                o[8 * i + j + 2][2 * r + e] * inv, o[8 * i + j + 3][2 * r + e] * inv);
      if (tq == 0)
        a.tail_lse[to] = sum[r] > 0.f ? (top[r] + fast_log2(sum[r])) * kLn2 : -INFINITY;
    }
    item = next;
    it = next_it;
  }
  if (a.behind_prefix) grid_dependency_wait();
}

// A warp per (query row, head), a lane per 4 columns: weights of the partials from their
// log-sum-exps, a lane per partial, then their sum.  (Four rows per warp, for more loads in flight,
// took half as many warps per SM and 3 us longer.)
constexpr int kMergeThreads = 256;
__global__ void __launch_bounds__(kMergeThreads)
shared_merge_kernel(const __grid_constant__ SharedLaunch a) {
  const int lane = threadIdx.x & 31;
  const long long x =
      static_cast<long long>(blockIdx.x) * (kMergeThreads / 32) + (threadIdx.x >> 5);
  grid_dependency_wait();
  grid_launch_dependents();
  if (x >= static_cast<long long>(a.B) * a.SQ * a.Hq) return;
  const int row = static_cast<int>(x / a.Hq);
  const int head = static_cast<int>(x - static_cast<long long>(row) * a.Hq);
  const int b = row / a.SQ, i = row - b * a.SQ, h = head / a.G, e = head - h * a.G;
  const PrefixRef ref = a.refs[b];
  // partial s of the prefix, then of the tail
  const int TM = kMTileRows / a.G, token = ref.token + i;
  const int in_tile = token % (2 * TM);
  const long long pre0 =
      (ref.base + (static_cast<long long>(h) * ref.row_tiles + token / (2 * TM)) * ref.splits) *
          (2 * kMTileRows) +
      in_tile / TM * kMTileRows + in_tile % TM * a.G + e;
  const int at = a.split_offset[b], tails = a.split_offset[b + 1] - at;
  const int M = a.SQ * a.G;
  const long long tail0 =
      (static_cast<long long>(at) * a.Hkv + static_cast<long long>(h) * tails) * M + i * a.G + e;
  // Two runs of partials, each at a stride of its own.
  const long long step[2] = {2 * kMTileRows, M};
  const long long row0[2] = {pre0, tail0};
  const int count[2] = {ref.splits, tails};
  const float* lses[2] = {a.pre_lse + row0[0], a.tail_lse + row0[1]};
  const float4* outs[2] = {reinterpret_cast<const float4*>(a.pre_o + row0[0] * kD) + lane,
                           reinterpret_cast<const float4*>(a.tail_o + row0[1] * kD) + lane};
  float top = -INFINITY, first[2];         // first: of the first 32 partials, a lane each
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    first[r] = lane < count[r] ? __ldcg(lses[r] + lane * step[r]) : -INFINITY;
    top = fmaxf(top, first[r]);
    for (int s = lane + 32; s < count[r]; s += 32) top = fmaxf(top, __ldcg(lses[r] + s * step[r]));
  }
#pragma unroll
  for (int d = 16; d > 0; d /= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
  const float shift = top == -INFINITY ? 0.f : top;
  float total = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    const float4* o = outs[r];
    const long long stride = step[r] * (kD / 4);
    for (int s0 = 0; s0 < count[r]; s0 += 32) {
      const int s = s0 + lane;
      const float l = s0 == 0        ? first[r]
                      : s < count[r] ? __ldcg(lses[r] + s * step[r])
                                     : -INFINITY;
      const float w = __expf(l - shift);
      total += w;
      const int n = min(32, count[r] - s0);
      int j = 0;
      for (; j + 4 <= n; j += 4) {
        float4 v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = __ldcg(o + e * stride);
        o += 4 * stride;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float f = __shfl_sync(0xffffffffu, w, j + e);
          acc.x += f * v[e].x;
          acc.y += f * v[e].y;
          acc.z += f * v[e].z;
          acc.w += f * v[e].w;
        }
      }
      for (; j < n; ++j, o += stride) {
        const float4 v = __ldcg(o);
        const float f = __shfl_sync(0xffffffffu, w, j);
        acc.x += f * v.x;
        acc.y += f * v.y;
        acc.z += f * v.z;
        acc.w += f * v.w;
      }
    }
  }
#pragma unroll
  for (int d = 16; d > 0; d /= 2) total += __shfl_xor_sync(0xffffffffu, total, d);
  const float sc = total > 0.f ? a.out_scale / total : 0.f;
  store_out4(a.out, x * kD + lane * 4,
             make_float4(acc.x * sc, acc.y * sc, acc.z * sc, acc.w * sc), a.out_dtype);
  if (a.lse && lane == 0) a.lse[x] = total > 0.f ? shift + __logf(total) : -INFINITY;
}

}  // namespace

int launch_shared_plan(const SharedLaunch& a, cudaStream_t st) {
  count_launches(1);
  const int threads = a.B * a.Hkv <= 2 * kFewThreads && a.groups < kFewThreads
                          ? kFewThreads
                          : kThreads;
  const size_t smem = sizeof(int) * ((a.B <= kHeld ? 3 * static_cast<size_t>(a.B) + 1 : 0) +
                                     (a.groups <= kOrdered ? a.groups + 1 : 0));
  static std::atomic<uint64_t> ready{0};
  constexpr int most = 4 * (3 * kHeld + 1 + kOrdered + 1);
  if (smem > 38 * 1024 && !kernel_smem_ready(shared_plan_kernel, most, ready)) return -1;
  return launch_after_previous(shared_plan_kernel, dim3(1), dim3(threads), smem, st, a) ==
                 cudaSuccess
             ? 0
             : -1;
}

int launch_shared_tail(const SharedLaunch& a, cudaStream_t st) {
  const bool rowmask = a.causal && a.SQ > 1;
  const auto kernel = rowmask ? tail_kernel<true> : tail_kernel<false>;
  static std::atomic<uint64_t> ready[2];
  const int sms = current_sm_count();
  if (sms <= 0 || !kernel_smem_ready(kernel, kTailSmem, ready[rowmask])) return -1;
  const int most = ceil_div(a.item_capacity, kTailThreads / 32);
  count_launches(1);
  return launch_after_previous(kernel, dim3(most < 2 * sms ? most : 2 * sms), dim3(kTailThreads),
                               kTailSmem, st, a) == cudaSuccess
             ? 0
             : -1;
}

int launch_shared_merge(const SharedLaunch& a, cudaStream_t st) {
  const long long rows = static_cast<long long>(a.B) * a.SQ * a.Hq;
  const long long ctas = ceil_div_ll(rows, kMergeThreads / 32);
  if (ctas > INT_MAX) return -1;
  count_launches(1);
  return launch_after_previous(shared_merge_kernel, dim3(static_cast<unsigned>(ctas)),
                               dim3(kMergeThreads), 0, st, a) == cudaSuccess
             ? 0
             : -1;
}

}  // namespace pa
