// Attention weight per cached token (include/paged_cache.h documents the contract): for every key
// of a request the sum over its queries, and over the query heads of the key's KV head, of
// exp(scale q.k - lse), with the log-sum-exp that the attention call returned.  No maximum and no
// second pass are needed, and no value row is read.
#include <climits>
#include <cmath>

#include "pages.cuh"

namespace pa {
namespace {

constexpr float kLog2e = 1.4426950408889634f;

struct WeightsArgs {
  const __nv_bfloat16* q;                  // [total, Hq, D]
  const float* lse;                        // [total, Hq]
  const __nv_bfloat16* k;                  // K pool, or the combined cache
  const int* qo_indptr;                    // packed queries, or null: SQ per request
  const int* kv_indptr;                    // CSR table, or null: pages is [B, C]
  const int* pages;
  const int* lens;
  float* w;                                // [B, Hkv, W]
  uint32_t* status;
  int B, Hq, Hkv, G, W, C, SQ, total, last, causal, ps, P;
  int chunk;                               // narrow: keys of a unit
  int more_than, at_most;                  // rows (query, head) of the requests looked after
  int beside;                              // narrow: the launch before this one is the same call's
  unsigned long long by_ps;                // ceil(2^64 / ps)
  long long page_rows;                     // rows of D columns per page
  float scale_log2, decay;
};

// What a request's part of a call is.
struct Request {
  int keys;                                // tokens that have a weight to write
  int row0, n;                             // first counted query row, and how many
  int first_pos;                           // its position
  int old;                                 // tokens before the call's queries
  const int* pages;
  bool bad;
};
__device__ __forceinline__ Request request_of(const WeightsArgs& a, int b) {
  Request r;
  const int L = a.lens[b];
  int q0 = a.qo_indptr ? a.qo_indptr[b] : b * a.SQ;
  int q1 = a.qo_indptr ? a.qo_indptr[b + 1] : q0 + a.SQ;
  r.bad = q0 < 0 || q1 < q0 || q1 > a.total || L < 0;
  if (r.bad) q0 = q1 = 0;
  const int nq = q1 - q0;
  r.n = a.last > 0 && a.last < nq ? a.last : nq;
  r.row0 = q1 - r.n;
  r.first_pos = L - r.n;
  r.old = max(L - nq, 0);
  int entries = a.C;
  r.pages = a.pages + static_cast<long long>(b) * a.C;
  if (a.kv_indptr) {
    const int p0 = a.kv_indptr[b], p1 = a.kv_indptr[b + 1];
    entries = p0 >= 0 && p1 > p0 ? p1 - p0 : 0;
    r.pages = a.pages + p0;
  }
  const long long room = static_cast<long long>(entries) * a.ps;
  r.keys = min(max(L, 0), a.W);
  if (r.keys > room) r.keys = static_cast<int>(room);
  if (nq == 0) r.keys = 0;                 // nothing is asked of the request
  else r.bad |= r.keys < L;
  const long long rows = static_cast<long long>(r.n) * a.G;
  if (rows <= a.more_than || rows > a.at_most) r.keys = 0;     // another launch's
  return r;
}
// Row of a head of KV head h in lse, and of D columns in q.
__device__ __forceinline__ long long head_row(const WeightsArgs& a, int row, int h, int head) {
  return static_cast<long long>(row) * a.Hq + h * a.G + head;
}
__device__ __forceinline__ int over(int x, unsigned long long by_ps) {
  return static_cast<int>(__umul64hi(static_cast<unsigned>(x), by_ps));
}

// ---- few rows: decode --------------------------------------------------------------------------
// Bound by reading K.  A warp takes 16 keys at a time as the A operand of warp MMAs, the request's
// rows (query, head) as the B operand, 8 NT of them.  The contraction runs over columns in any
// order, so a lane loads 16 bytes of its key's row and takes them as its operands of two MMAs:
// K comes from HBM straight into registers, without shared memory or barriers, and the loads of
// all the SM's warps are in flight together.  The scores of a key then lie in the four lanes of a
// quad.
// A unit is a.chunk keys of a request and KV head, 128 at a time (32 per warp); the pages of the
// next 128 are looked up while the present ones are on their way.
// 690 MB of keys (64 requests, 8 KV heads): 128 us, 79% of the copy rate.  Rings in shared memory,
// a warp each, took longer: filled by the lanes' asynchronous copies 212 us, by bulk copies of 16
// rows, 12 warps per SM, 175 us, of 32 rows, 8 warps, 149 us (what a step needs beside its keys
// then stands in the way of fewer warps).
constexpr int kHeavyRows = 32;             // with more, a request is taken as a prompt
constexpr int kNarrowThreads = 128;
constexpr int kNarrowKeys = 128;

template <int D, int NT>
__global__ void __launch_bounds__(kNarrowThreads, NT == 1 && D == 128 ? 6 : 1)
narrow_kernel(const __grid_constant__ WeightsArgs a) {
  constexpr int kBlocks = D / 32;          // 32 columns: two MMAs
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int gr = lane >> 2, tq = lane & 3;
  // (beside: wide_kernel starts this one when it has waited itself, and writes other requests)
  if (!a.beside) grid_dependency_wait();
  grid_launch_dependents();
  const int pairs = a.B * a.Hkv;
  const int chunks = (a.W + a.chunk - 1) / a.chunk;
  for (long long u = blockIdx.x; u < static_cast<long long>(pairs) * chunks; u += gridDim.x) {
    const int c = static_cast<int>(u / pairs);
    const int bh = static_cast<int>(u - static_cast<long long>(c) * pairs);
    const int b = bh / a.Hkv, h = bh - b * a.Hkv;
    const Request r = request_of(a, b);
    if (r.bad && c == 0 && h == 0 && threadIdx.x == 0) report_error(a.status, kErrMetadata);
    const int begin = c * a.chunk + warp * 32;
    if (begin >= r.keys) continue;
    const int end = min(r.keys, (c + 1) * a.chunk);
    float* w = a.w + static_cast<long long>(bh) * a.W;
    // this lane's rows of the two 16-key steps from key0 on, keys gr and gr + 8 of each; -1: none
    const auto find = [&](int key0, int (&row)[4]) {
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const int key = key0 + 8 * x + gr;
        row[x] = -1;
        if (key < end) {
          const int p = over(key, a.by_ps), page = __ldg(r.pages + p);
          if (page >= 0 && page < a.P)
            row[x] = static_cast<int>(page * a.page_rows) + h * a.ps + (key - p * a.ps);
          else
            report_error(a.status, kErrMetadata);
        }
      }
    };
    const int rows = r.n * a.G;
    for (int r0 = 0; r0 < rows; r0 += 8 * NT) {
      // columns of this lane in the scores: rows r0 + 8 nt + 2 tq and + 1
      float shift[NT][2];
      int limit[NT][2];                    // the last key that the row sees
      uint4 q[NT][kBlocks];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int x = r0 + nt * 8 + tq * 2 + e, t = x / a.G;
          shift[nt][e] = 0.f;
          limit[nt][e] = -1;
          if (x < rows) {
            const float l = __ldg(a.lse + head_row(a, r.row0 + t, h, x - t * a.G));
            shift[nt][e] = -l * kLog2e;
            if (l != -INFINITY) limit[nt][e] = a.causal ? r.first_pos + t : 0x7fffffff;
          }
        }
        const int x = r0 + nt * 8 + gr, t = x / a.G;
        const uint4* src = reinterpret_cast<const uint4*>(
            a.q + head_row(a, r.row0 + t, h, x - t * a.G) * D + tq * 8);
#pragma unroll
        for (int i = 0; i < kBlocks; ++i)
          q[nt][i] = x < rows ? __ldg(src + i * 4) : make_uint4(0u, 0u, 0u, 0u);
      }
      int next[4];
      find(begin, next);
      for (int key0 = begin; key0 < end; key0 += kNarrowKeys) {
        int row[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) row[x] = next[x];
        float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          uint4 ka[kBlocks], kb[kBlocks];
          const __nv_bfloat16* pa = a.k + static_cast<long long>(row[2 * s]) * D + tq * 8;
          const __nv_bfloat16* pb = a.k + static_cast<long long>(row[2 * s + 1]) * D + tq * 8;
#pragma unroll
          for (int i = 0; i < kBlocks; ++i) {
            ka[i] = kb[i] = make_uint4(0u, 0u, 0u, 0u);
            if (row[2 * s] >= 0) ka[i] = ld_stream(reinterpret_cast<const uint4*>(pa + i * 32));
            if (row[2 * s + 1] >= 0) kb[i] = ld_stream(reinterpret_cast<const uint4*>(pb + i * 32));
          }
          if (s == 0) find(key0 + kNarrowKeys, next);
          const int key = key0 + 16 * s + gr;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            float d[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int i = 0; i < kBlocks; ++i) {
              const uint32_t a0[4] = {ka[i].x, kb[i].x, ka[i].y, kb[i].y};
              const uint32_t a1[4] = {ka[i].z, kb[i].z, ka[i].w, kb[i].w};
              mma_16816(d, a0, q[nt][i].x, q[nt][i].y);
              mma_16816(d, a1, q[nt][i].z, q[nt][i].w);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float p = fast_exp2(fmaf(d[e], a.scale_log2, shift[nt][e & 1]));
              if (key + 8 * (e >> 1) <= limit[nt][e & 1]) sum[2 * s + (e >> 1)] += p;
            }
          }
        }
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          sum[x] += __shfl_xor_sync(0xffffffffu, sum[x], 1);
          sum[x] += __shfl_xor_sync(0xffffffffu, sum[x], 2);
        }
        // lane tq of the quad writes key key0 + 8 tq + gr
        const float mine = tq == 0 ? sum[0] : (tq == 1 ? sum[1] : (tq == 2 ? sum[2] : sum[3]));
        const int live = tq == 0 ? row[0] : (tq == 1 ? row[1] : (tq == 2 ? row[2] : row[3]));
        const int key = key0 + 8 * tq + gr;
        if (live >= 0) {
          float before = 0.f;
          if (r0 > 0) before = w[key];
          else if (key < r.old && a.decay != 0.f) before = a.decay * w[key];
          w[key] = before + mine;
        }
      }
    }
  }
  if (a.beside) grid_dependency_wait();
}

// ---- many rows: prompts ------------------------------------------------------------------------
// S = Q K^T on the 5th-generation tensor cores: the keys of a unit stay in shared memory while the
// request's queries stream past them, 128 rows (TMEM lanes) at a time.  A thread owns a row, whose
// shift -lse log2 e it keeps in a register, and 64 keys, whose sums over its rows it keeps in 64
// registers until the unit ends and the lanes are summed.  Persistent, one CTA per SM; a unit is a
// (request, KV head, key tile).  Roles (640 threads):
//   warps 0-15  exponentials and sums
//   warp  16    TMA producer of K and of Q (a ring of 64-column stages)
//   warp  17    TMEM owner and MMA issuer
//   warp  19    unit descriptions, page ids among them
// kPair: tiles of 256 keys; the four warpgroups take every query tile, 64 keys each.  Else tiles of
// 128 keys, and two pairs of warpgroups take query tiles in turn.
// The queries come from L2 once per key tile, so tiles of 256 keys halve that traffic (3.4 GB a
// call for four prompts of up to 8,192 tokens, 32 heads: 4.9 TB/s); tiles of 128 make more and
// smaller units and leave room for the next unit's K at D = 256.  Those four prompts take 690 us,
// 1.24 PFLOP/s: the tensor pipe is active 62% of the time and 60% of the issue slots are taken,
// neither full; which of the waits between them costs the rest is not known.
constexpr int kGroups = 4;                 // warpgroups of exponentials
constexpr int kOwn = 64;                   // keys of a thread
constexpr int kSumWarps = 4 * kGroups;
constexpr int kWideThreads = 32 * kSumWarps + 128;
constexpr int kRows = 128;                 // of a query tile
constexpr int kBlockBytes = kRows * 128;   // 128 rows of 64 columns
constexpr int kUnits = 4;                  // units described ahead
constexpr int kListed = 512;               // requests with units that the schedule keeps at hand
// Registers after set-up (launch: 640 x 96): 512 x 104 + 128 x 64 = 640 x 96.
constexpr int kSumRegs = 104;
constexpr int kControlRegs = 64;
static_assert(32 * kSumWarps * kSumRegs + 128 * kControlRegs <= kWideThreads * 96, "registers");

template <int D, bool kPair>
struct Wide {
  static constexpr int kKeys = kPair ? 256 : 128;
  static constexpr int kBlocks = D / 64;                        // of 64 columns
  static constexpr int kKBuffers = D == 256 && kPair ? 1 : 2;
  static constexpr int kSBuffers = 512 / kKeys;                 // score buffers
  static constexpr int kQStages = D == 128 && !kPair ? 8 : 5;
  static constexpr int kKBytes = kKeys * 128;                   // of a block
};
struct Unit {
  int tiles;               // query tiles; -1: no more units
  int h;
  int key0, keys;          // first key, live keys of the tile
  int old;                 // keys below it have an older weight
  int row0, tokens;        // query rows from row0 on, whole tokens
  int pos0;                // position of the first one; INT_MAX: every row sees every key
  long long w;             // offset of the tile's weights
  int pages[32];           // of each piece; -1: outside the pool or past the live keys
};
struct WideCtrl {
  Unit units[kUnits];
  alignas(16) float sums[2][kSumWarps][kOwn];    // by unit parity: each warp's sums of its keys
  uint64_t unit_full[kUnits], unit_empty[kUnits];
  uint64_t s_full[4], s_empty[4];
  uint64_t k_full[2], k_empty[2];
  uint64_t q_full[8], q_empty[8];
  uint32_t tmem;
  int abort_flag;
  int tiles_begun, looked;               // beats of the MMA warp, and of the units' warp
  int2 listed[kListed];                  // requests with units, their key tiles
};
// A wait for a ring entry of the units may last as long as another role's whole unit (0.1 s are
// 13 million rows of queries), or its look through a large batch.  Its limit is one of progress:
// the clock starts anew whenever the beat of the role waited for moves.
__device__ __forceinline__ bool unit_wait_warp(uint64_t* bar, uint32_t parity,
                                               const volatile int* beat, uint32_t* status,
                                               volatile int* abort) {
  bool ok = mbar_test(bar, parity);
  if (!ok) {
    long long t0 = clock64();
    int seen = *beat;
    while (!*abort && !(ok = mbar_test(bar, parity))) {
      const int now = *beat;
      if (now != seen) {
        seen = now;
        t0 = clock64();
      } else if (clock64() - t0 > kWaitCycles) {
        *abort = 1;
        report_error(status, kErrTimeout);
      }
    }
  }
  return __all_sync(0xffffffffu, ok);
}
template <int D, bool kPair>
constexpr int wide_smem() {
  using X = Wide<D, kPair>;
  return X::kKBuffers * X::kBlocks * X::kKBytes + X::kQStages * kBlockBytes +
         static_cast<int>(sizeof(WideCtrl)) + 1024;
}

// Exponentials of 16 scores, added to the sums of their keys.  kMask: only keys j <= limit count.
template <bool kMask>
__device__ __forceinline__ void add_weights(float (&sums)[kOwn], const uint32_t (&r)[16], int j0,
                                            float scale, float shift, int limit) {
#pragma unroll
  for (int j = 0; j < 16; j += 2) {
    float y0, y1;
    ffma2_bcast(y0, y1, __uint_as_float(r[j]), __uint_as_float(r[j + 1]), scale, shift);
    y0 = fast_exp2(y0);
    y1 = fast_exp2(y1);
    if (kMask) {
      y0 = j0 + j <= limit ? y0 : 0.f;
      y1 = j0 + j + 1 <= limit ? y1 : 0.f;
    }
    fadd2(sums[j0 + j], sums[j0 + j + 1], y0, y1);
  }
}
// A thread's scores of a row; `done` is called when they have left TMEM.
template <bool kMask, typename F>
__device__ __forceinline__ void add_row(float (&sums)[kOwn], uint32_t column, float scale,
                                        float shift, int limit, const F& done) {
#pragma unroll
  for (int q = 0; q < kOwn / 16; ++q) {
    uint32_t r[16];
    tmem_ld16(column + q * 16, r);
    tmem_ld_wait();
    if (q == kOwn / 16 - 1) done();
    add_weights<kMask>(sums, r, q * 16, scale, shift, limit);
  }
}

// Sums over a warp's rows: at each step a lane gives away half of its keys, until lane l has those
// of keys 2 l and 2 l + 1.
template <int kHalf, int kLane>
__device__ __forceinline__ void sum_lanes(float (&sums)[kOwn], int lane) {
  const bool upper = lane & kLane;
#pragma unroll
  for (int j = 0; j < kHalf; ++j) {
    const float give = upper ? sums[j] : sums[j + kHalf];
    const float keep = upper ? sums[j + kHalf] : sums[j];
    sums[j] = keep + __shfl_xor_sync(0xffffffffu, give, kLane);
  }
  if constexpr (kLane > 1) sum_lanes<kHalf / 2, kLane / 2>(sums, lane);
}

template <int D, bool kPair>
__global__ void __launch_bounds__(kWideThreads, 1)
wide_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
            const __grid_constant__ WeightsArgs a) {
  using X = Wide<D, kPair>;
  constexpr int kKeys = X::kKeys, kBlocks = X::kBlocks, kKBytes = X::kKBytes;
  constexpr int kKBuffers = X::kKBuffers, kSBuffers = X::kSBuffers, kStages = X::kQStages;
  extern __shared__ uint8_t raw[];
  uint8_t* k_s = smem_align<1024>(raw);
  uint8_t* q_s = k_s + kKBuffers * kBlocks * kKBytes;
  WideCtrl* ctl = reinterpret_cast<WideCtrl*>(q_s + kStages * kBlockBytes);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int TM = kRows / a.G;
  if (a.more_than > 0) {
    // The host could not rule out requests with that many rows.  Without any (packed single tokens)
    // the other launch, which looks at every request, must not wait for this one's set-up.
    grid_dependency_wait();
    bool some = false;
    for (int b = threadIdx.x; b < a.B; b += kWideThreads) {
      const long long n = static_cast<long long>(a.qo_indptr[b + 1]) - a.qo_indptr[b];
      some |= (a.last > 0 && a.last < n ? a.last : n) * a.G > a.more_than;
    }
    if (!__syncthreads_or(some)) return;
  }
  if (threadIdx.x == 0) {
    for (int i = 0; i < kUnits; ++i) {
      mbar_init(&ctl->unit_full[i], 1);
      mbar_init(&ctl->unit_empty[i], 2 + kSumWarps);
    }
    for (int i = 0; i < kSBuffers; ++i) {
      mbar_init(&ctl->s_full[i], 1);
      mbar_init(&ctl->s_empty[i], kPair ? kSumWarps : kSumWarps / 2);
    }
    for (int i = 0; i < kKBuffers; ++i) {
      mbar_init(&ctl->k_full[i], 1);
      mbar_init(&ctl->k_empty[i], 1);
    }
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&ctl->q_full[i], 1);
      mbar_init(&ctl->q_empty[i], 1);
    }
    ctl->abort_flag = ctl->tiles_begun = ctl->looked = 0;
    fence_mbar_init();
  }
  // rows of a query tile that no box writes: zero scores
  const int spare = (kRows - TM * a.G) * 8;
  for (int i = threadIdx.x; i < kStages * spare; i += kWideThreads)
    reinterpret_cast<uint4*>(q_s + i / spare * kBlockBytes + TM * a.G * 128)[i % spare] =
        make_uint4(0u, 0u, 0u, 0u);
  fence_proxy_async_smem();
  if (warp == kSumWarps + 1) {
    tmem_alloc(&ctl->tmem, 512);
    tmem_relinquish();
  }
  grid_dependency_wait();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  grid_launch_dependents();
  const uint32_t tmem = ctl->tmem;
  volatile int* abort_flag = &ctl->abort_flag;
  // A role's view of the units: entry s of the ring, given back by release().
  const auto next_unit = [&](int s) {
    return unit_wait_warp(&ctl->unit_full[s % kUnits], (s / kUnits) & 1, &ctl->looked, a.status,
                          abort_flag);
  };
  const auto entry_free = [&](int s) {
    return s < kUnits || unit_wait_warp(&ctl->unit_empty[s % kUnits], ((s / kUnits) - 1) & 1,
                                        &ctl->tiles_begun, a.status, abort_flag);
  };
  const auto release = [&](int s) {
    __syncwarp();
    if (lane == 0) mbar_arrive(&ctl->unit_empty[s % kUnits]);
  };

  if (warp >= kSumWarps) {
  regs_decrease<kControlRegs>();
  if (warp == kSumWarps + 3) {
    // =============================== units ==============================================
    // Units in order of the key tiles left to the request's end: a tile's queries are about as many
    // under the causal mask, so long units come first whatever the lengths.  The CTAs take them in
    // turns that reverse from round to round.  (In order of the tiles' indexes, with requests of
    // 8,192 down to 2,048 tokens, the busiest CTA had 1.25 times the mean, so 1.12.)
    // Requests with units and their tiles are listed (batches with idle rows or single tokens,
    // which another launch takes, have few); where the list overflows, tiles are counted anew.
    const int R = page_piece_rows(a.ps, kRows), pieces = kKeys / R, grid = gridDim.x;
    const auto tiles_of = [&](const Request& r) { return (r.keys + kKeys - 1) / kKeys; };
    volatile int* looked = &ctl->looked;
    int most = 0, listed = 0, beat = 0;
    for (int b0 = 0; b0 < a.B; b0 += 4 * 32) {
      int n[4];
#pragma unroll
      for (int g = 0; g < 4; ++g) {        // (four requests' loads on their way together)
        const int b = b0 + 32 * g + lane;
        n[g] = 0;
        if (b >= a.B) continue;
        const Request r = request_of(a, b);
        n[g] = tiles_of(r);
        if (r.bad && blockIdx.x == 0) report_error(a.status, kErrMetadata);
      }
      *looked = ++beat;
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        most = max(most, n[g]);
        const uint32_t some = __ballot_sync(0xffffffffu, n[g] > 0);
        const int at = listed + __popc(some & ((1u << lane) - 1u));
        if (n[g] > 0 && at < kListed) ctl->listed[at] = make_int2(b0 + 32 * g + lane, n[g]);
        listed += __popc(some);
      }
    }
    __syncwarp();
    most = __reduce_max_sync(0xffffffffu, most);
    const bool complete = listed <= kListed;
    const int candidates = complete ? listed : a.B;
    int s = 0;
    long long before = 0, round = 0, mine = blockIdx.x;      // units before; this CTA's next one
    bool ok = true;
    for (int left = most; ok && left > 0; --left) {
      for (int x0 = 0; ok && x0 < candidates; x0 += 32) {
        *looked = ++beat;
        int2 mine_of = make_int2(x0 + lane, 0);              // request and tiles
        if (x0 + lane >= candidates) mine_of.x = 0;
        else if (complete) mine_of = ctl->listed[x0 + lane];
        else mine_of.y = tiles_of(request_of(a, mine_of.x));
        const uint32_t live = __ballot_sync(0xffffffffu, mine_of.y >= left);
        const long long after = before + static_cast<long long>(__popc(live)) * a.Hkv;
        while (mine < after) {
          const int which = static_cast<int>(mine - before) / a.Hkv;
          const int h = static_cast<int>(mine - before) - which * a.Hkv;
          const int at = __fns(live, 0, which + 1);
          const int b = __shfl_sync(0xffffffffu, mine_of.x, at);
          const Request r = request_of(a, b);
          const int key0 = (__shfl_sync(0xffffffffu, mine_of.y, at) - left) * kKeys;
          const int keys = min(kKeys, r.keys - key0);
          int page = -1;
          const int key = key0 + lane * R;
          if (lane < pieces && key < key0 + keys) {
            page = __ldg(r.pages + over(key, a.by_ps));
            if (page < 0 || page >= a.P) {
              report_error(a.status, kErrMetadata);
              page = -1;
            }
          }
          const int slot = s % kUnits;
          if (!entry_free(s)) {
            ok = false;
            break;
          }
          Unit* out = &ctl->units[slot];
          out->pages[lane] = page;
          if (lane == 0) {
            // from the first token on that sees a key of the tile
            const int t0 = a.causal ? min(max(key0 - r.first_pos, 0), r.n) : 0;
            out->tiles = (r.n - t0 + TM - 1) / TM;
            out->h = h;
            out->key0 = key0;
            out->keys = keys;
            out->old = r.old;
            out->row0 = r.row0 + t0;
            out->tokens = r.n - t0;
            out->pos0 = a.causal ? r.first_pos + t0 : INT_MAX;
            out->w = (static_cast<long long>(b) * a.Hkv + h) * a.W + key0;
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&ctl->unit_full[slot]);
          ++s;
          ++round;
          mine = round * grid + (round & 1 ? grid - 1 - blockIdx.x : blockIdx.x);
        }
        before = after;
      }
    }
    const int slot = s % kUnits;
    if (ok && entry_free(s) && lane == 0) {
      ctl->units[slot].tiles = -1;
      mbar_arrive(&ctl->unit_full[slot]);
    }
  } else if (warp == kSumWarps) {
    // =============================== copies =============================================
    if (lane == 0) {
      tma_prefetch_desc(&qmap);
      tma_prefetch_desc(&kmap);
    }
    const int R = page_piece_rows(a.ps, kRows), boxes = kKeys / R * kBlocks;
    const uint32_t q_box = static_cast<uint32_t>(TM * a.G) * 128u;
    int units = 0, qs = 0;                 // K tiles, Q stages
    bool ok = true;
    for (int s = 0; ok && next_unit(s); ++s) {
      const Unit& x = ctl->units[s % kUnits];
      const int tiles = x.tiles, h = x.h, key0 = x.key0, row0 = x.row0;
      if (tiles <= 0) {
        release(s);
        if (tiles < 0) break;
        continue;
      }
      const int kb = units % kKBuffers;
      if (units >= kKBuffers && !mbar_wait_warp<true>(&ctl->k_empty[kb],
                                                      (units / kKBuffers - 1) & 1, a.status,
                                                      abort_flag))
        break;
      uint32_t live = 0;
      for (int i = lane; i < boxes; i += 32) live += x.pages[i / kBlocks] >= 0;
      live = __reduce_add_sync(0xffffffffu, live);
      if (lane == 0) mbar_arrive_expect_tx(&ctl->k_full[kb], live * R * 128u);
      __syncwarp();
      for (int i = lane; i < boxes; i += 32) {
        const int piece = i / kBlocks, col = i % kBlocks, page = x.pages[piece];
        if (page < 0) continue;
        const int key = key0 + piece * R;
        const int row = static_cast<int>(page * a.page_rows) + h * a.ps + key % a.ps;
        tma_load_2d(k_s + (kb * kBlocks + col) * kKBytes + piece * R * 128, &kmap,
                    &ctl->k_full[kb], col * 64, row);
      }
      ++units;
      release(s);
      for (int i = 0; ok && i < tiles * kBlocks; ++i, ++qs) {
        const int stage = qs % kStages;
        if (qs >= kStages && !mbar_wait_fast_warp(&ctl->q_empty[stage], ((qs / kStages) - 1) & 1,
                                                  a.status, abort_flag)) {
          ok = false;
          break;
        }
        if (lane == 0) {
          mbar_arrive_expect_tx(&ctl->q_full[stage], q_box);
          tma_load_3d(q_s + stage * kBlockBytes, &qmap, &ctl->q_full[stage], i % kBlocks * 64,
                      h * a.G, row0 + i / kBlocks * TM);
        }
      }
    }
    if (*abort_flag) {                     // no copy may land after the CTA has ended
      for (int i = max(0, units - kKBuffers); i < units; ++i)
        drain_wait(&ctl->k_full[i % kKBuffers], (i / kKBuffers) & 1);
      for (int i = max(0, qs - kStages); i < qs; ++i)
        drain_wait(&ctl->q_full[i % kStages], (i / kStages) & 1);
    }
  } else if (warp == kSumWarps + 1) {
    // =============================== MMAs ===============================================
    constexpr uint32_t idesc_all = idesc_bf16(kRows, kKeys, false, false);
    constexpr uint32_t idesc_half = idesc_bf16(kRows, 128, false, false);
    const uint64_t k_desc = sdesc_sw128(smem_u32(k_s), 16, 1024);
    const uint64_t q_desc = sdesc_sw128(smem_u32(q_s), 16, 1024);
    int units = 0, qs = 0, it = 0;
    bool ok = true;
    for (int s = 0; ok && next_unit(s); ++s) {
      const int tiles = ctl->units[s % kUnits].tiles, keys = ctl->units[s % kUnits].keys;
      release(s);
      if (tiles < 0) break;
      if (tiles == 0) continue;
      const uint32_t idesc = keys > 128 ? idesc_all : idesc_half;
      const int kb = units % kKBuffers;
      if (!mbar_wait_fast_warp(&ctl->k_full[kb], (units / kKBuffers) & 1, a.status, abort_flag))
        break;
      ++units;
      for (int i = 0; ok && i < tiles; ++i, ++it) {
        const int buf = it % kSBuffers;
        if (lane == 0) *const_cast<volatile int*>(&ctl->tiles_begun) = it;
        if (it >= kSBuffers && !mbar_wait_fast_warp(&ctl->s_empty[buf], ((it / kSBuffers) - 1) & 1,
                                                    a.status, abort_flag)) {
          ok = false;
          break;
        }
        for (int c = 0; c < kBlocks; ++c, ++qs) {
          const int stage = qs % kStages;
          if (!mbar_wait_fast_warp(&ctl->q_full[stage], (qs / kStages) & 1, a.status,
                                   abort_flag)) {
            ok = false;
            break;
          }
          if (lane == 0) {
            tc_fence_after();
            const uint64_t kd = k_desc + ((kb * kBlocks + c) * kKBytes >> 4);
            const uint64_t qd = q_desc + (stage * kBlockBytes >> 4);
#pragma unroll
            for (int k = 0; k < 4; ++k)
              mma_ss(tmem + buf * kKeys, qd + (k * 32 >> 4), kd + (k * 32 >> 4), idesc,
                     c > 0 || k > 0);
            mma_commit(&ctl->q_empty[stage]);
            if (c == kBlocks - 1) mma_commit(&ctl->s_full[buf]);
            if (c == kBlocks - 1 && i == tiles - 1) mma_commit(&ctl->k_empty[kb]);
          }
          __syncwarp();
        }
      }
    }
  }
  } else {
    regs_increase<kSumRegs>();
    // =============================== exponentials and sums ==============================
    const int group = warp >> 2, m = threadIdx.x & 127;      // this thread's row
    // its group's keys, from `first` on, and which of the query tiles it takes
    const int first = (kPair ? group : group & 1) * kOwn, turn = kPair ? 0 : group >> 1;
    const uint32_t column0 = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + first;
    const float scale = a.scale_log2;
    const int R = page_piece_rows(a.ps, kRows);
    const int token = m / a.G;                               // of the row, in its tile
    const long long lse_at = static_cast<long long>(token) * a.Hq + m - token * a.G;
    const long long lse_step = static_cast<long long>(TM) * a.Hq;
    int it = 0;
    for (int s = 0;; ++s) {
      bool ok = next_unit(s);
      const Unit& x = ctl->units[s % kUnits];
      const int tiles = ok ? x.tiles : 0;
      const int key0 = x.key0 + first, tokens = x.tokens, pos0 = x.pos0;
      // the first half of a group that takes turn 0 writes its keys
      const int k = first + m;
      const bool writes = ok && tiles >= 0 && turn == 0 && m < kOwn && k < x.keys &&
                          x.pages[k / R] >= 0;
      const bool had = writes && key0 + m < x.old && a.decay != 0.f;
      const bool idle = kPair && x.keys <= first;            // no live key of this group
      float* w = a.w + x.w + k;
      const float* lse = a.lse + head_row(a, x.row0, x.h, 0) + lse_at;
      if (ok) release(s);
      const float before = had ? *w : 0.f;                   // on its way during the sums
      float sums[kOwn];
#pragma unroll
      for (int j = 0; j < kOwn; ++j) sums[j] = 0.f;
      const auto load = [&](int i) {
        return token < TM && i * TM + token < tokens ? __ldg(lse + i * lse_step) : -INFINITY;
      };
      constexpr int kStep = kPair ? 1 : 2;
      const int i0 = turn;
      float next = ok && i0 < tiles ? load(i0) : 0.f;
      for (int i = i0; ok && i < tiles; i += kStep) {
        const int t = it + i, buf = t % kSBuffers;
        const float l = next;
        if (i + kStep < tiles) next = load(i + kStep);
        // keys up to `limit` of this thread's count
        const int limit = l == -INFINITY  ? -1
                          : pos0 == INT_MAX ? INT_MAX
                                            : pos0 + i * TM + token - key0;
        const float shift = -l * kLog2e;
        ok = mbar_wait_fast_warp(&ctl->s_full[buf], (t / kSBuffers) & 1, a.status, abort_flag);
        if (!ok) break;
        tc_fence_after();
        const uint32_t column = column0 + buf * kKeys;
        const auto done = [&] {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&ctl->s_empty[buf]);
        };
        if (idle || __all_sync(0xffffffffu, limit < 0)) done();
        else if (__all_sync(0xffffffffu, limit >= kOwn - 1))
          add_row<false>(sums, column, scale, shift, limit, done);
        else
          add_row<true>(sums, column, scale, shift, limit, done);
      }
      it += tiles;
      sum_lanes<kOwn / 2, 16>(sums, lane);
      reinterpret_cast<float2*>(ctl->sums[s & 1][warp])[lane] = make_float2(sums[0], sums[1]);
      // Every warp comes here whatever its waits said and also after the last unit, so that those
      // that meet here leave together.
      const bool leave = !ok || tiles < 0;
      if (kPair ? named_bar_or(1 + group, 128, leave) : named_bar_or(1 + (group & 1), 256, leave))
        break;
      if (writes) {
        float sum = 0.f;
#pragma unroll
        for (int t = 0; t < (kPair ? 1 : 2); ++t)
#pragma unroll
          for (int g = 0; g < 4; ++g) sum += ctl->sums[s & 1][(group + 2 * t) * 4 + g][m];
        *w = (had ? a.decay * before : 0.f) + sum;
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kSumWarps + 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int D, bool kPair>
int launch_wide(const WeightsArgs& a, cudaStream_t st) {
  constexpr int smem = wide_smem<D, kPair>();
  static_assert(smem <= 227 * 1024, "shared memory");
  const int sms = current_sm_count();
  static std::atomic<uint64_t> ready{0};
  constexpr auto kernel = wide_kernel<D, kPair>;
  if (sms <= 0 || !kernel_smem_ready(kernel, smem, ready)) return PAGED_ATTN_ERR_CUDA;
  CUtensorMap qmap, kmap;
  if (!encode_q_map(&qmap, a.q, a.total, a.Hq, D, a.G, kRows / a.G) ||
      !encode_rows_map(&kmap, a.k, a.page_rows * a.P, D, page_piece_rows(a.ps, kRows)))
    return PAGED_ATTN_ERR_CUDA;
  const long long units =
      static_cast<long long>(a.B) * a.Hkv * ceil_div(a.W, Wide<D, kPair>::kKeys);
  count_launches(1);
  return cuda_status(launch_after_previous(kernel, static_cast<int>(units < sms ? units : sms),
                                           kWideThreads, smem, st, qmap, kmap, a));
}

// All of the SM's memory as L1, where the loads in flight lie: behind a kernel with much shared
// memory (attention's) the SMs would keep its division, and narrow_kernel take 1.6 times as long.
template <typename Kernel>
bool all_l1(Kernel* kernel, std::atomic<uint64_t>& done) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return false;
  const uint64_t bit = dev >= 0 && dev < 64 ? (uint64_t{1} << dev) : 0;
  if (bit != 0 && (done.load(std::memory_order_acquire) & bit) != 0) return true;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout,
                           cudaSharedmemCarveoutMaxL1) != cudaSuccess)
    return false;
  if (bit != 0) done.fetch_or(bit, std::memory_order_acq_rel);
  return true;
}

template <int D, int NT>
int launch_narrow(WeightsArgs a, cudaStream_t st) {
  const int sms = current_sm_count();
  if (sms <= 0) return PAGED_ATTN_ERR_CUDA;
  // long units where there are many: what a unit reads of its request counts once per unit
  const long long steps = static_cast<long long>(a.B) * a.Hkv * ceil_div(a.W, kNarrowKeys);
  const long long most = 16LL * sms;
  a.chunk = kNarrowKeys * (steps >= 8 * most ? 4 : (steps >= 4 * most ? 2 : 1));
  const long long units = static_cast<long long>(a.B) * a.Hkv * ceil_div(a.W, a.chunk);
  count_launches(1);
  static std::atomic<uint64_t> ready{0};
  if (!all_l1(narrow_kernel<D, NT>, ready)) return PAGED_ATTN_ERR_CUDA;
  return cuda_status(launch_after_previous(narrow_kernel<D, NT>,
                                           static_cast<int>(units < most ? units : most),
                                           kNarrowThreads, 0, st, a));
}

bool params_ok(const paged_weights_params* p) {
  if (!p || p->batch < 0 || p->total_q < 0 || p->seq_len_q < 0 || p->last_queries < 0)
    return false;
  if (p->num_kv_heads <= 0 || p->num_qo_heads <= 0 || p->num_qo_heads % p->num_kv_heads)
    return false;
  if (p->num_qo_heads / p->num_kv_heads > 64) return false;
  if (p->head_dim != 128 && p->head_dim != 256) return false;
  if (p->page_size < 8 || p->page_size > 128 || p->page_size % 8) return false;
  if (p->num_pages <= 0 || p->num_pages > kMaxPages || p->width <= 0) return false;
  if (p->mask_type != PAGED_ATTN_MASK_DENSE && p->mask_type != PAGED_ATTN_MASK_CAUSAL) return false;
  if (!std::isfinite(p->decay) || !std::isfinite(p->sm_scale)) return false;
  const long long rows = static_cast<long long>(p->num_pages) * (p->combined_cache ? 2 : 1) *
                         p->num_kv_heads * p->page_size;
  return rows < (1LL << 31);
}

}  // namespace
}  // namespace pa

using namespace pa;

extern "C" {

int paged_weights_run(const paged_weights_params* p, const void* q, const float* lse,
                      const void* k_cache, const int32_t* qo_indptr, const int32_t* kv_indptr,
                      const int32_t* pages, const int32_t* lens, float* weights, uint32_t* status,
                      void* stream) {
  if (!params_ok(p)) return PAGED_ATTN_ERR_INVALID_ARGUMENT;
  if (p->batch == 0) return PAGED_ATTN_OK;
  if (!qo_indptr && static_cast<long long>(p->batch) * p->seq_len_q != p->total_q)
    return PAGED_ATTN_ERR_INVALID_ARGUMENT;
  if (!kv_indptr && p->max_pages_per_request <= 0) return PAGED_ATTN_ERR_INVALID_ARGUMENT;
  if (p->total_q == 0) return PAGED_ATTN_OK;             // no query looks at anything
  if (!q || !lse || !k_cache || !pages || !lens || !weights)
    return PAGED_ATTN_ERR_INVALID_ARGUMENT;
  if (!aligned_to(q, 16) || !aligned_to(k_cache, 16) ||
      !ints_aligned(lse, qo_indptr, kv_indptr, pages, lens, weights, status))
    return PAGED_ATTN_ERR_INVALID_ARGUMENT;
  WeightsArgs a{};
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.lse = lse;
  a.k = static_cast<const __nv_bfloat16*>(k_cache);
  a.qo_indptr = qo_indptr; a.kv_indptr = kv_indptr; a.pages = pages; a.lens = lens;
  a.w = weights; a.status = status;
  a.B = p->batch; a.Hq = p->num_qo_heads; a.Hkv = p->num_kv_heads; a.G = a.Hq / a.Hkv;
  a.W = p->width; a.C = p->max_pages_per_request; a.SQ = p->seq_len_q; a.total = p->total_q;
  a.last = p->last_queries; a.causal = p->mask_type == PAGED_ATTN_MASK_CAUSAL;
  a.ps = p->page_size; a.P = p->num_pages;
  a.by_ps = ~0ull / static_cast<unsigned>(a.ps) + 1;
  a.page_rows = static_cast<long long>(p->combined_cache ? 2 : 1) * a.Hkv * a.ps;
  const float scale =
      p->sm_scale > 0.f ? p->sm_scale : 1.0f / std::sqrt(static_cast<float>(p->head_dim));
  a.scale_log2 = scale * kLog2e;
  a.decay = p->decay;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  a.more_than = 0;
  a.at_most = INT_MAX;
  long long rows = ceil_div(p->total_q, p->batch);         // of a request, on average
  if (a.last > 0 && a.last < rows) rows = a.last;
  rows *= a.G;
  if (rows > 16) {
    // Tiles of 256 keys wherever they make a unit per SM by the weights' width (the lengths are on
    // the device); else 128: two prompts' 512 queries of 2 heads, D = 128, 46 us against 62.  16
    // prompts' last 32 queries of 2 KV heads, D = 256: 40 us against 47, their last 8 23 against
    // 27, 128 85 against 121.  A width far above the lengths takes the 256 where 128 were better:
    // two prompts of 512 tokens, 8 heads, 17.3 us in rows of 576 weights, 20.3 in rows of 32,768.
    const bool pair = static_cast<long long>(a.B) * a.Hkv * ceil_div(a.W, 256) >=
                      current_sm_count();
    if (p->head_dim == 128)
      return pair ? launch_wide<128, true>(a, st) : launch_wide<128, false>(a, st);
    return pair ? launch_wide<256, true>(a, st) : launch_wide<256, false>(a, st);
  }
  // Few rows on average, but some request may have many (a prompt among single tokens, or in a
  // batch whose other rows sit the call out): a launch for each kind.  511 single tokens and one of
  // 1,000, 2,000 keys each, 8 KV heads: 510 us; 3,650 as few rows, 618 as many.  63 and a prompt of
  // 64, 4,000 keys: 104 us; 214 and 156.  511 idle rows and a prompt of 512: 48 us, 1,840 as few
  // rows; 63 and one of 9: 25 and 30.  Packed single tokens pay 2 us for the launch that finds no
  // prompt (64 of up to 8,192 keys 136 us, 134 without it; 9 of up to 700 15.5 and 13.4).
  const long long total = p->total_q, most = a.last > 0 && a.last < total ? a.last : total;
  const bool mixed = qo_indptr && most * a.G > kHeavyRows;
  if (mixed) {
    WeightsArgs heavy = a;
    heavy.more_than = kHeavyRows;
    const int rc = p->head_dim == 128 ? launch_wide<128, false>(heavy, st)
                                      : launch_wide<256, false>(heavy, st);
    if (rc != PAGED_ATTN_OK) return rc;
    a.at_most = kHeavyRows;
    a.beside = 1;
  }
  if (p->head_dim == 128)
    return rows <= 8 ? launch_narrow<128, 1>(a, st) : launch_narrow<128, 2>(a, st);
  return rows <= 8 ? launch_narrow<256, 1>(a, st) : launch_narrow<256, 2>(a, st);
}

}  // extern "C"
