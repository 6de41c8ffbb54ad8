// Rotary positions, and appending rotated keys and values to the paged cache
// (include/paged_cache.h documents the contract).
//
// Both are one pass over rows of D columns: a row (token, head) is read once, the first R
// columns are rotated pair by pair in fp32, and the row is written once, in place, to another
// tensor or to its slot in a page.  What bounds a large call is HBM, what bounds a small one is
// the chain of dependent loads before the first row can be written (position or request,
// length, page id), so a CTA resolves its tokens and their sines first and then streams rows.
//
// Angles.  A table entry is the frequency in turns per position as a 0.64 fixed-point fraction;
// position x entry modulo 2^64 is the exact fraction of a turn for every int32 position (the
// integer turns fall off the top), so the angle carries no error that grows with the position.
// The nearest quarter turn is taken off in integers and the rest, at most an eighth of a turn,
// is rounded to fp32 once (relative 2^-24) before its sine and cosine.
#include <cfloat>
#include <cmath>
#include <type_traits>

#include "../../include/paged_cache.h"
#include "common.cuh"
#include "internal.h"

namespace pa {
namespace {

// Threads of a CTA: 128, but 64 where rows are staged and the slots of its tokens fill no more than
// half of those (6 heads of 80 columns: 15.9 us with 128 threads, 17.2 with 64, for 32,749 tokens).
// Small CTAs with one wide token or a few narrow ones keep loads, sines and stores of many tokens
// overlapped: staging 17,408 tokens of 32 + 8 + 8 bf16 heads (append) takes 65.9 us with 64 threads
// and 12 KB each, 66.6 with 128 and 24 KB; registers for 16 of the 64-thread CTAs per SM instead of
// 12 make it 67.2.
constexpr int kMaxThreads = 128;
constexpr int kFewThreads = 64;
constexpr int kStageGoal = 12288;        // bytes of rows that a CTA stages where it may choose
constexpr int kMaxStaged = 196608;       // and at most
constexpr int kStagedCtas = 5;           // per SM, of 128 threads: bounds their registers
constexpr int kInSharedCtas = 7;         // the same where the rows are rotated in shared memory
constexpr int kTileTokens = 8;           // per SM: from here on a CTA takes several tokens
constexpr int kStagedTokens = 4;         // per SM: from here on rows are staged

struct RopeArgs {
  const void *q, *k, *v;
  void *qo, *ko, *vo;                    // ko, vo: outputs, or the cache's K and V pools
  long long q_ts, q_hs, k_ts, k_hs, v_ts;
  long long qo_ts, qo_hs, ko_ts, ko_hs;
  const int* positions;
  const unsigned long long* table;
  int T, Hq, Hkv, D, n;                  // n = R / 2 column pairs
  int slots;                             // of a row
  int inverse, q_in_place, k_in_place;
  float m;
  int tile;                              // tokens per CTA
  int chunk;                             // heads per CTA
  int staged_bytes;                      // shared memory of staged rows
  // append
  const int *qo_indptr, *kv_indptr, *pages, *lens;
  int B, SQ, C, ps, num_pages;
  long long page_elems;                  // elements of a page of the K (or V) pool
  uint32_t* status;
};

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename T>
__device__ __forceinline__ T from_f(float x);
template <>
__device__ __forceinline__ float from_f<float>(float x) { return x; }
template <>
__device__ __forceinline__ __half from_f<__half>(float x) { return __float2half_rn(x); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float x) {
  return __float2bfloat16_rn(x);
}

// V elements as one access of V * sizeof(T) bytes (at most 16, or two of 16).
template <typename T, int V>
struct alignas(sizeof(T) * V <= 16 ? sizeof(T) * V : 16) Vec {
  T e[V];
};

template <typename T, int V>
__device__ __forceinline__ void unpack(const Vec<T, V>& x, float (&f)[V]) {
#pragma unroll
  for (int i = 0; i < V; ++i) f[i] = to_f(x.e[i]);
}
// Rounded to nearest-even; two 16-bit values per conversion.
template <typename T, int V>
__device__ __forceinline__ Vec<T, V> pack(const float (&f)[V]) {
  Vec<T, V> x;
  if constexpr (sizeof(T) == 2 && V % 2 == 0) {
#pragma unroll
    for (int i = 0; i < V; i += 2) {
      if constexpr (std::is_same<T, __half>::value)
        *reinterpret_cast<__half2*>(&x.e[i]) = __floats2half2_rn(f[i], f[i + 1]);
      else
        *reinterpret_cast<__nv_bfloat162*>(&x.e[i]) = __floats2bfloat162_rn(f[i], f[i + 1]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) x.e[i] = from_f<T>(f[i]);
  }
  return x;
}

// V elements of TIn, as values of TOut, unchanged where the types agree.
template <typename TIn, typename TOut, int V>
__device__ __forceinline__ Vec<TOut, V> convert(const Vec<TIn, V>& x) {
  if constexpr (std::is_same<TIn, TOut>::value) {
    return x;
  } else {
    float f[V];
    unpack(x, f);
    return pack<TOut>(f);
  }
}

// (cos, sin) of p * f, times m; the sine's sign carries the direction.
__device__ __forceinline__ float2 turn_of(int p, unsigned long long f, float m, float sign) {
  const unsigned long long a = static_cast<unsigned long long>(static_cast<long long>(p)) * f;
  const unsigned quarter = static_cast<unsigned>((a + (1ull << 61)) >> 62) & 3u;
  // The rest in units of 2^-64 turns, at most 2^61 of them.  All its bits count where the angle is
  // small: its upper 32 alone leave a slow pair's sine off by 1e-5 to 4e-3 at position 1.
  const auto rest = static_cast<long long>(a - (static_cast<unsigned long long>(quarter) << 62));
  float s, c;
  sincospif(__ll2float_rn(rest) * 1.0842021724855044e-19f, &s, &c);      // 2^-63: half turns
  const float cc = (quarter & 1u) ? -s : c, ss = (quarter & 1u) ? c : s;
  const float k = (quarter & 2u) ? -m : m;
  return make_float2(cc * k, ss * k * sign);
}

// a c + b s with the roundings fixed (one product rounded, the other fused into the sum), so that
// every access width gives the same bits.
__device__ __forceinline__ float turned(float a, float c, float b, float s) {
  return __fmaf_rn(a, c, __fmul_rn(b, s));
}

// Bytes (a multiple of 16) from 16-byte aligned global to shared memory, counted on an mbarrier.
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes,
                                          uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
      ::"r"(smem_u32(dst)), "l"(src), "r"(bytes), "r"(smem_u32(bar))
      : "memory");
}

// What a thread holds of one slot between its load and its store.  A slot is V column pairs (half:
// V columns of each half) or V columns (interleaved; the last one may hold columns past the
// rotated ones too.  V = 1 is one pair element by element, for rows whose alignment allows no
// wider access); the slots from `rot` on copy V columns each, from column `first`.
template <typename TIn, int V, bool kHalf>
struct Slot {
  static constexpr bool kTwo = kHalf || V == 1;
  static constexpr int kPairs = kTwo ? V : V / 2;
  Vec<TIn, V> a, b;
  static __host__ __device__ int rotated_slots(int n) { return (n + kPairs - 1) / kPairs; }
  static __host__ __device__ int first_copied(int n) {
    return kTwo ? 2 * n : rotated_slots(n) * V;
  }
  __device__ __forceinline__ void load(const TIn* x, int n, int s, int rot, int first) {
    if (s < rot) {
      a = *reinterpret_cast<const Vec<TIn, V>*>(x + (!kHalf && V == 1 ? 2 * s : s * V));
      if constexpr (kTwo)
        b = *reinterpret_cast<const Vec<TIn, V>*>(x + (kHalf ? n + s * V : 2 * s + 1));
    } else {
      a = *reinterpret_cast<const Vec<TIn, V>*>(x + first + (s - rot) * V);
    }
  }
  // cs: (cos, sin) of the slot's pairs; `rotated` columns of the row are kept as they lie in `a`
  // (already results: mode 2) where TIn is not TOut.
  template <typename TOut>
  __device__ __forceinline__ void store(TOut* y, const float2 (&cs)[kPairs], int n, int s, int rot,
                                        int first, bool rotate, int results) const {
    if (s >= rot) {
      const int at = first + (s - rot) * V;
      Vec<TOut, V> c = convert<TIn, TOut, V>(a);
      if constexpr (sizeof(TIn) == sizeof(TOut) && !std::is_same<TIn, TOut>::value) {
#pragma unroll
        for (int i = 0; i < V; ++i)
          if (at + i < results) c.e[i] = reinterpret_cast<const TOut*>(&a)[i];
      }
      *reinterpret_cast<Vec<TOut, V>*>(y + at) = c;
      return;
    }
    Vec<TOut, V> c = convert<TIn, TOut, V>(a), d;
    if constexpr (kTwo) {
      d = convert<TIn, TOut, V>(b);
      if (rotate) {
        float u[V], w[V], y1[V], y2[V];
        unpack(a, u);
        unpack(b, w);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          y1[i] = turned(u[i], cs[i].x, -w[i], cs[i].y);
          y2[i] = turned(w[i], cs[i].x, u[i], cs[i].y);
        }
        c = pack<TOut>(y1);
        d = pack<TOut>(y2);
      }
      *reinterpret_cast<Vec<TOut, V>*>(y + (kHalf ? s * V : 2 * s)) = c;
      *reinterpret_cast<Vec<TOut, V>*>(y + (kHalf ? n + s * V : 2 * s + 1)) = d;
    } else {
      if (rotate) {
        float u[V], y1[V];
        unpack(a, u);
#pragma unroll
        for (int i = 0; i < V; i += 2) {
          y1[i] = turned(u[i], cs[i / 2].x, -u[i + 1], cs[i / 2].y);
          y1[i + 1] = turned(u[i + 1], cs[i / 2].x, u[i], cs[i / 2].y);
        }
        const Vec<TOut, V> r = pack<TOut>(y1);
#pragma unroll
        for (int i = 0; i < V; ++i)            // a column past the rotated ones keeps its bits
          if (s * kPairs + i / 2 < n) c.e[i] = r.e[i];
      }
      *reinterpret_cast<Vec<TOut, V>*>(y + s * V) = c;
    }
  }
};

struct TokenSlot {
  long long off;        // element offset of (page, head 0, slot) in a pool; -1: not written
  int request;          // -1: no request owns the token
  int position;
};

// The request that owns row t of the packed rows (-1: none), by a warp: the last b with
// offsets[b] <= t, each round trip narrowing the choice to a 32nd.
__device__ __forceinline__ int request_of(const int* offsets, int B, int t) {
  const int lane = threadIdx.x & 31;
  int lo = 0, hi = B;
  while (true) {
    const int step = (hi - lo + 31) / 32, at = lo + lane * step;
    const unsigned after = __ballot_sync(0xffffffffu, at >= hi || offsets[at] > t);
    const int c = after == 0 ? 32 : __ffs(after) - 1;       // probes not after t
    if (c == 0) return -1;
    lo += (c - 1) * step;
    hi = min(hi, lo + step);
    if (step == 1) break;
  }
  return t < offsets[lo + 1] ? lo : -1;
}

// How a CTA gets at its rows.
constexpr int kDirect = 0;    // straight from global memory, a few rows in flight per thread
constexpr int kStaged = 1;    // brought to shared memory by bulk copies: tens of KB in flight per
                              // SM whatever the registers allow (16-byte aligned, adjacent heads)
constexpr int kOnePiece = 2;  // the same where the rows of q, k and v and the tokens are one run in
                              // memory (slices of one projection): one copy per CTA
constexpr int kInShared = 3;  // staged, and rotated there element by element: half layout whose
                              // halves do not both start on a 16-byte access

template <typename TIn, typename TOut, int V, bool kHalf, bool kAppend, int kMode>
__global__ void __launch_bounds__(kMaxThreads, kMode == kDirect      ? 1
                                                         : kMode == kInShared ? kInSharedCtas
                                                                              : kStagedCtas)
rope_kernel(const RopeArgs a) {
  using Held = Slot<TIn, V, kHalf>;
  // Rows in flight per thread: 64 bytes of loads.
  constexpr int kBytes = V * static_cast<int>(sizeof(TIn)) * (Held::kTwo ? 2 : 1);
  constexpr int kBatch = kMode != kDirect || kBytes >= 64 ? 1 : (64 / kBytes > 8 ? 8 : 64 / kBytes);
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint64_t arrived;
  __shared__ int gave_up;
  float2* cs = reinterpret_cast<float2*>(smem + a.staged_bytes);    // [tile, n]
  TokenSlot* tok = reinterpret_cast<TokenSlot*>(cs + static_cast<size_t>(a.tile) * a.n);
  const int tid = threadIdx.x, threads = blockDim.x;
  const int t0 = blockIdx.x * a.tile;
  const int nt = min(a.tile, a.T - t0);
  const int rot = kMode == kInShared ? 0 : Held::rotated_slots(a.n);
  const int first = kMode == kInShared ? 0 : Held::first_copied(a.n);
  const int heads = a.Hq + a.Hkv * (kAppend ? 2 : 1);
  const int h_begin = blockIdx.y * a.chunk, h_end = min(heads, h_begin + a.chunk);
  // A thread keeps one slot of one token, and so its sines, and walks the heads; consecutive
  // threads hold consecutive slots, then tokens.  `groups` threads share the heads of a slot.
  const int slots = min(a.slots, threads), units = a.tile * slots, groups = threads / units;
  const int group = tid / units, unit = tid - group * units;
  const int t = unit / slots, s = blockIdx.z * threads + unit - t * slots;
  const bool active = group < groups && t < nt && s < a.slots;
  const long long token = t0 + t;
  grid_dependency_wait();
  grid_launch_dependents();
  // Staged rows: [tile, heads, D] in one piece, else tensor by tensor [tile, its heads of the
  // chunk, D], so that a tensor whose tokens are adjacent comes in one copy too.  (Few large
  // copies: 12 heads of 32,749 tokens take 38.8 us in one copy per CTA, 42.9 in three or more.)
  TIn* const rows = reinterpret_cast<TIn*>(smem);
  const int k_begin = a.Hq, v_begin = a.Hq + a.Hkv;
  const int q_rows = max(0, min(h_end, k_begin) - h_begin);
  const int k_rows = max(0, min(h_end, v_begin) - max(h_begin, k_begin));
  const int v_rows = h_end - h_begin - q_rows - k_rows;
  // Where row (t, head h of the chunk) would lie if every tensor were laid out as q, k or v is.
  struct Staged {
    TIn *q, *k, *v;
  };
  const auto staged = [&](int t) {
    if constexpr (kMode == kOnePiece) {
      TIn* const p = rows + t * heads * a.D;
      return Staged{p, p, p};
    }
    return Staged{rows + t * q_rows * a.D,
                  rows + (a.tile * q_rows + t * k_rows - q_rows) * a.D,
                  rows + (a.tile * (q_rows + k_rows) + t * v_rows - q_rows - k_rows) * a.D};
  };
  if constexpr (kMode != kDirect) {
    if (tid < 32) {
      if (tid == 0) {
        gave_up = 0;
        mbar_init(&arrived, 1);
        fence_mbar_init();
        fence_proxy_async_smem();
        mbar_arrive_expect_tx(&arrived,
                              nt * (h_end - h_begin) * a.D * static_cast<int>(sizeof(TIn)));
      }
      __syncwarp();
      // n rows of one tensor (of `all`, from its head h on) for every token of the tile
      const auto bring = [&](const void* x, long long ts, int h, int n, int all, TIn* to) {
        if (n == 0) return;
        const TIn* from = static_cast<const TIn*>(x) + t0 * ts + static_cast<long long>(h) * a.D;
        const bool adjacent = n == all && ts == static_cast<long long>(n) * a.D;
        const int copies = adjacent ? 1 : nt;
        const int bytes = (adjacent ? nt : 1) * n * a.D * static_cast<int>(sizeof(TIn));
        for (int i = tid; i < copies; i += 32)
          bulk_load(to + i * n * a.D, from + i * ts, bytes, &arrived);
      };
      if constexpr (kMode == kOnePiece) {
        bring(a.q, a.q_ts, 0, heads, heads, rows);
      } else {
        const int tile = a.tile * a.D;
        bring(a.q, a.q_ts, h_begin, q_rows, a.Hq, rows);
        bring(a.k, a.k_ts, max(h_begin, k_begin) - k_begin, k_rows, a.Hkv, rows + tile * q_rows);
        if (kAppend)
          bring(a.v, a.v_ts, max(h_begin, v_begin) - v_begin, v_rows, a.Hkv,
                rows + tile * (q_rows + k_rows));
      }
    }
  }
  Held x[kBatch];
  const Staged mine = staged(t);
  auto load = [&](int h0) {
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int h = h0 + u * groups;
      if (h >= h_end) break;
      const TIn* p;
      if (kMode != kDirect)
        p = (kMode == kOnePiece || h < k_begin ? mine.q : h < v_begin ? mine.k : mine.v) +
            (h - h_begin) * a.D;
      else if (h < a.Hq)
        p = static_cast<const TIn*>(a.q) + token * a.q_ts + h * a.q_hs;
      else if (!kAppend || h < a.Hq + a.Hkv)
        p = static_cast<const TIn*>(a.k) + token * a.k_ts + (h - a.Hq) * a.k_hs;
      else
        p = static_cast<const TIn*>(a.v) + token * a.v_ts +
            static_cast<long long>(h - a.Hq - a.Hkv) * a.D;
      x[u].load(p, a.n, s, rot, first);
    }
  };
  // The first rows are on their way while positions, pages and sines are found.
  if (kMode == kDirect && active) load(h_begin + group);
  // The chain to the first store of an append is request -> length -> page; what does not depend on
  // it is fetched beside it: the thread's first table entry before, the page while sines are
  // taken (17,408 tokens of 48 heads: 67.1 us without either, 65.9 with both; 32,749 of 12:
  // 41.3 and 38.8).
  const unsigned long long entry = kAppend && tid < a.tile * a.n ? a.table[tid % a.n] : 0;
  TokenSlot found{-1, -1, 0};                                       // of token tid (tile <= 16)
  int page = -1, slot = 0;
  if constexpr (kAppend) {
    if (a.qo_indptr != nullptr) {
      for (int t = tid >> 5; t < nt; t += threads >> 5) {
        const int b = request_of(a.qo_indptr, a.B, t0 + t);
        if ((tid & 31) == 0) tok[t].request = b;
      }
      __syncthreads();
    }
    if (tid < nt) {
      const int b = a.qo_indptr != nullptr ? tok[tid].request : (t0 + tid) / a.SQ;
      found.request = b;
      if (b >= 0) {
        const int end = a.qo_indptr != nullptr ? a.qo_indptr[b + 1] : (b + 1) * a.SQ;
        long long first = static_cast<long long>(b) * a.C;
        int count = a.C;
        if (a.kv_indptr != nullptr) {
          first = a.kv_indptr[b];
          count = a.kv_indptr[b + 1] - a.kv_indptr[b];
        }
        const int p = a.lens[b] - (end - (t0 + tid)), j = p / a.ps;
        found.position = p;
        slot = p - j * a.ps;
        if (p >= 0 && j < count) page = a.pages[first + j];
      }
      tok[tid].position = found.position;
    }
    __syncthreads();
  }
  for (int i = tid; i < nt * a.n; i += threads) {
    const int j = i / a.n, pair = i - j * a.n;
    const int p = kAppend ? tok[j].position : a.positions[t0 + j];
    cs[i] = turn_of(p, kAppend && i == tid ? entry : a.table[pair], a.m, a.inverse ? -1.f : 1.f);
  }
  if constexpr (kAppend) {
    if (tid < nt) {
      if (page >= 0 && page < a.num_pages)
        found.off = page * a.page_elems + static_cast<long long>(slot) * a.D;
      else if (found.request >= 0)
        report_error(a.status, kErrMetadata);
      tok[tid] = found;
    }
  }
  __syncthreads();
  if constexpr (kMode != kDirect) {
    const bool ok = mbar_wait(&arrived, 0, a.status, &gave_up);
    if (!ok) drain_wait(&arrived, 0);
    if (kMode == kInShared ? __syncthreads_or(!ok) != 0 : !ok) return;
  }
  if constexpr (kMode == kInShared) {
    // One pair of one token per thread, over the heads to rotate: q and k.
    const int rotated = min(h_end, a.Hq + a.Hkv) - h_begin;
    const int pairs = nt * a.n, share = max(1, threads / pairs);
    for (int i = tid; i < pairs * share; i += threads) {
      const int g = i / pairs, j = i - g * pairs, at = j / a.n, pair = j - at * a.n;
      const float2 turn = cs[j];
      const Staged of = staged(at);
      for (int h = g; h < rotated; h += share) {
        TIn* x = (h_begin + h < k_begin ? of.q : of.k) + h * a.D + pair;
        const float u = to_f(x[0]), w = to_f(x[a.n]);
        const float y1 = turned(u, turn.x, -w, turn.y), y2 = turned(w, turn.x, u, turn.y);
        if constexpr (sizeof(TIn) == sizeof(TOut)) {   // the results, rounded once
          reinterpret_cast<TOut*>(x)[0] = from_f<TOut>(y1);
          reinterpret_cast<TOut*>(x)[a.n] = from_f<TOut>(y2);
        } else {                                       // fp32 rows: rounded as they leave
          x[0] = y1;
          x[a.n] = y2;
        }
      }
    }
    __syncthreads();
  }
  if (!active) return;
  if constexpr (kMode != kDirect) load(h_begin + group);
  float2 turn[Held::kPairs];
#pragma unroll
  for (int i = 0; i < Held::kPairs; ++i) {
    const int pair = s * Held::kPairs + i;
    turn[i] = s < rot && pair < a.n ? cs[t * a.n + pair] : make_float2(0.f, 0.f);
  }
  bool write_q = a.Hq > 0, write_k = true;
  TOut *q_to, *k_to, *v_to = nullptr;
  long long k_step;
  if constexpr (kAppend) {
    write_q = tok[t].request >= 0;
    write_k = tok[t].off >= 0;
    k_to = static_cast<TOut*>(a.ko) + tok[t].off;
    v_to = static_cast<TOut*>(a.vo) + tok[t].off;
    k_step = static_cast<long long>(a.ps) * a.D;
  } else {
    // in place, what only copies stays where it is
    const bool moves = kMode == kInShared ? s * V < 2 * a.n : s < rot;
    write_q = moves || !a.q_in_place;
    write_k = moves || !a.k_in_place;
    k_to = static_cast<TOut*>(a.ko) + token * a.ko_ts;
    k_step = a.ko_hs;
  }
  q_to = static_cast<TOut*>(a.qo) + token * a.qo_ts;
  const int results = kMode == kInShared ? 2 * a.n : 0;
  for (int h0 = h_begin + group; h0 < h_end;) {
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int h = h0 + u * groups;
      if (h >= h_end) break;
      if (h < a.Hq) {
        if (write_q) x[u].store(q_to + h * a.qo_hs, turn, a.n, s, rot, first, true, results);
      } else if (write_k) {
        const int j = h - a.Hq;
        if (!kAppend || j < a.Hkv)
          x[u].store(k_to + j * k_step, turn, a.n, s, rot, first, true, results);
        else
          x[u].store(v_to + (j - a.Hkv) * k_step, turn, a.n, s, rot, first, false, 0);
      }
    }
    h0 += kBatch * groups;
    load(h0);
  }
}

template <typename TIn, typename TOut, int V, bool kHalf, bool kAppend, int kMode>
cudaError_t launch_mode(RopeArgs a, cudaStream_t st) {
  using Held = Slot<TIn, V, kHalf>;
  const int sms = current_sm_count();
  if (sms <= 0) return cudaErrorUnknown;
  // Slots of a row: those that rotate, and unless every output is its input the ones that copy.
  const bool copies = !(a.q_in_place && (a.Hkv == 0 || a.k_in_place));
  if (kMode == kInShared)
    a.slots = copies ? a.D / V : ceil_div(2 * a.n, V);
  else
    a.slots = Held::rotated_slots(a.n) + (copies ? (a.D - Held::first_copied(a.n)) / V : 0);
  const int heads = a.Hq + a.Hkv * (kAppend ? 2 : 1);
  const long long token_bytes = static_cast<long long>(heads) * a.D * sizeof(TIn);
  const long long goal = token_bytes < kStageGoal ? kStageGoal / token_bytes : 1;
  const bool few = (kMode == kStaged || kMode == kOnePiece) && goal * a.slots <= kFewThreads / 2;
  const int threads = few ? kFewThreads : kMaxThreads;
  const int slots = a.slots < threads ? a.slots : threads;
  // Tokens per CTA: one while there are few; else the most that keep 7 of 8 threads busy (the
  // slots of the tile's tokens, times the groups that share the heads), or that keep the most
  // busy.  12,627 tokens of 8 + 2 + 2 heads with 32 of 128 columns rotated (14 slots) take 47 us
  // one by one, 22 by four.
  a.tile = 1;
  if (a.T >= kTileTokens * sms) {
    const long long most = kMode == kDirect ? 4 : goal < 16 ? goal : 16;
    int best = 0;
    for (int tile = 1; tile <= most && tile * slots <= threads; ++tile) {
      int busy = threads / (tile * slots) * (tile * slots);
      if (busy * 8 >= threads * 7) busy = threads;
      if (busy >= best) {
        best = busy;
        a.tile = tile;
      }
    }
  }
  // Few tokens: their heads are shared out over more CTAs, down to one round of a CTA's groups.
  const int tiles = ceil_div(a.T, a.tile), groups = threads / (a.tile * slots);
  int chunks = kMode != kOnePiece && tiles < 2 * sms ? 2 * sms / tiles : 1;
  if (chunks > ceil_div(heads, groups)) chunks = ceil_div(heads, groups);
  a.chunk = ceil_div(heads, chunks);
  chunks = ceil_div(heads, a.chunk);
  const size_t rows = static_cast<size_t>(a.tile) * a.chunk;
  a.staged_bytes =
      kMode == kDirect ? 0 : static_cast<int>(align_up(rows * a.D * sizeof(TIn), 128));
  const size_t smem = a.staged_bytes +
                      static_cast<size_t>(a.tile) * (a.n * sizeof(float2) + sizeof(TokenSlot));
  void (*const kernel)(RopeArgs) = rope_kernel<TIn, TOut, V, kHalf, kAppend, kMode>;
  if (smem > 47 * 1024) {                  // the default limit holds the static part too
    static std::atomic<uint64_t> ready{0};
    if (!kernel_smem_ready(kernel, kMaxStaged + 16384, ready)) return cudaErrorUnknown;
  }
  count_launches(1);
  return launch_after_previous(kernel, dim3(tiles, chunks, ceil_div(a.slots, threads)),
                               dim3(threads), smem, st, a);
}

// may_stage: alignment and strides allow bulk copies and 16-byte accesses.
template <typename TIn, typename TOut, int V, bool kHalf, bool kAppend>
cudaError_t launch_v(const RopeArgs& a, bool may_stage, cudaStream_t st) {
  if constexpr (V * sizeof(TIn) == 16) {
    const int sms = current_sm_count();
    const bool skips = a.q_in_place && (a.Hkv == 0 || a.k_in_place) && a.D > 2 * a.n;
    if constexpr (kHalf) {
      if (a.n % V != 0) return launch_mode<TIn, TOut, V, kHalf, kAppend, kInShared>(a, st);
    }
    // In place, direct reads skip the columns that do not rotate; copies would bring them.
    if (may_stage && !skips && a.T >= kStagedTokens * sms) {
      const long long heads = a.Hq + a.Hkv * (kAppend ? 2 : 1);
      const TIn *q = static_cast<const TIn*>(a.q), *k = static_cast<const TIn*>(a.k),
                *v = static_cast<const TIn*>(a.v);
      const bool k_follows = a.Hkv == 0 || (k == q + a.Hq * a.D && a.k_ts == a.q_ts);
      const bool v_follows = !kAppend || (v == k + a.Hkv * a.D && a.v_ts == a.q_ts);
      if (a.Hq > 0 && a.q_ts == heads * a.D && k_follows && v_follows)
        return launch_mode<TIn, TOut, V, kHalf, kAppend, kOnePiece>(a, st);
      return launch_mode<TIn, TOut, V, kHalf, kAppend, kStaged>(a, st);
    }
  }
  return launch_mode<TIn, TOut, V, kHalf, kAppend, kDirect>(a, st);
}

template <typename TIn, typename TOut, bool kAppend>
cudaError_t launch_typed(const RopeArgs& a, int v, bool half, bool may_stage, cudaStream_t st) {
  const auto run = [&](auto width) {
    constexpr int V = decltype(width)::value;
    return half ? launch_v<TIn, TOut, V, true, kAppend>(a, may_stage, st)
                : launch_v<TIn, TOut, V, false, kAppend>(a, may_stage, st);
  };
  if constexpr (sizeof(TIn) == 2) {
    if (v >= 8) return run(std::integral_constant<int, 8>());
  }
  if (v >= 4) return run(std::integral_constant<int, 4>());
  if (v >= 2) return run(std::integral_constant<int, 2>());
  return run(std::integral_constant<int, 1>());
}

bool layout_ok(int R, int D, int layout, float m, bool may_be_zero) {
  if (R < 0 || R > D || R % 2 || (R == 0 && !may_be_zero)) return false;
  return (layout == PAGED_ROPE_HALF || layout == PAGED_ROPE_INTERLEAVED) && std::isfinite(m);
}

size_t size_of(int dtype) { return dtype == PAGED_ATTN_DTYPE_FP32 ? 4 : 2; }

bool aligned_to(const void* p, size_t bytes) {
  return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0;
}

// The largest power of two of elements per access that the columns, the pointers and the strides
// allow.  In the half layout both halves have to start on an access, unless the rows are
// rotated in shared memory.
struct Width {
  int v;
  explicit Width(size_t elem) : v(elem == 4 ? 4 : 8) {}
  void pointer(const void* p, size_t elem) {
    while (v > 1 && !aligned_to(p, v * elem)) v /= 2;
  }
  void stride(long long s) {
    while (v > 1 && s % v != 0) v /= 2;
  }
  void halves(int n, bool in_shared) {
    if (!in_shared)
      while (v > 1 && n % v != 0) v /= 2;
  }
};

// Whether T x H rows of D elements lie apart: the rows of one dimension fit in a step of the other.
bool rows_apart(long long T, long long H, long long D, long long ts, long long hs) {
  if (ts < 0) ts = -ts;
  if (hs < 0) hs = -hs;
  if (H == 1) return T == 1 || ts >= D;
  if (T == 1) return hs >= D;
  return (hs >= D && (ts - D) / (H - 1) >= hs) || (ts >= D && (hs - D) / (T - 1) >= ts);
}

bool dtype_ok(int t) { return t >= PAGED_ATTN_DTYPE_BF16 && t <= PAGED_ATTN_DTYPE_FP32; }

bool rope_params_ok(const paged_rope_params* p) {
  if (!p || p->num_tokens < 0 || p->num_qo_heads <= 0 || p->num_kv_heads < 0) return false;
  if (p->head_dim <= 0 || p->head_dim > 512 || p->head_dim % 8 || !dtype_ok(p->dtype)) return false;
  if (!layout_ok(p->rotary_dim, p->head_dim, p->layout, p->attention_factor, false)) return false;
  if (static_cast<long long>(p->num_qo_heads) + p->num_kv_heads > 65535) return false;
  return true;
}

bool append_params_ok(const paged_append_params* p, bool packed) {
  if (!p || p->batch < 0 || p->num_qo_heads < 0 || p->num_kv_heads <= 0) return false;
  if (p->head_dim <= 0 || p->head_dim > 512 || p->head_dim % 8 || !dtype_ok(p->in_dtype))
    return false;
  if (p->page_size < 8 || p->page_size > 128 || p->page_size % 8 || p->num_pages <= 0) return false;
  if (!layout_ok(p->rotary_dim, p->head_dim, p->layout, p->attention_factor, true)) return false;
  if (static_cast<long long>(p->num_qo_heads) + 2LL * p->num_kv_heads > 65535) return false;
  if (packed) return p->total_q >= 0;
  return p->seq_len_q >= 0 && static_cast<long long>(p->batch) * p->seq_len_q < (1LL << 31);
}

int cuda_status(cudaError_t e) { return e == cudaSuccess ? PAGED_ATTN_OK : PAGED_ATTN_ERR_CUDA; }

}  // namespace
}  // namespace pa

using namespace pa;

extern "C" {

int paged_rope_frequencies(const paged_rope_scaling* s, double* freqs, float* factor) {
  if (!s || !freqs || !factor) return PAGED_ATTN_ERR_INVALID_ARGUMENT;
  const int R = s->rotary_dim, kind = s->kind;
  if (R < 2 || R > 512 || R % 2 || !(s->base > 1) || !std::isfinite(s->base))
    return PAGED_ATTN_ERR_INVALID_ARGUMENT;
  if (kind < PAGED_ROPE_SCALE_NONE || kind > PAGED_ROPE_SCALE_WAVELENGTH)
    return PAGED_ATTN_ERR_INVALID_ARGUMENT;
  const bool scaled = kind != PAGED_ROPE_SCALE_NONE;
  if (scaled && (!(s->factor > 0) || !std::isfinite(s->factor)))
    return PAGED_ATTN_ERR_INVALID_ARGUMENT;
  const bool ramped = kind == PAGED_ROPE_SCALE_YARN || kind == PAGED_ROPE_SCALE_WAVELENGTH;
  double low = s->low, high = s->high;
  if (ramped) {
    if (!(s->original_max_position > 0) || !std::isfinite(s->original_max_position))
      return PAGED_ATTN_ERR_INVALID_ARGUMENT;
    if (low == 0 && high == 0) {
      low = 1;
      high = kind == PAGED_ROPE_SCALE_YARN ? 32 : 4;
    }
    if (!(low > 0) || !(high > low) || !std::isfinite(high))
      return PAGED_ATTN_ERR_INVALID_ARGUMENT;
  }
  const double two_pi = 6.283185307179586476925, L = s->original_max_position;
  double base = s->base;
  if (kind == PAGED_ROPE_SCALE_NTK && R > 2)
    base *= std::pow(s->factor, static_cast<double>(R) / (R - 2));
  double d0 = 0, d1 = 0;
  if (kind == PAGED_ROPE_SCALE_YARN) {
    const double per_log = R / (2 * std::log(s->base));
    d0 = std::fmax(std::floor(per_log * std::log(L / (two_pi * high))), 0.0);
    d1 = std::fmin(std::ceil(per_log * std::log(L / (two_pi * low))), R - 1.0);
  }
  for (int i = 0; i < R / 2; ++i) {
    double f = std::pow(base, -2.0 * i / R);
    if (kind == PAGED_ROPE_SCALE_LINEAR) {
      f /= s->factor;
    } else if (kind == PAGED_ROPE_SCALE_YARN) {
      const double g = std::fmin(std::fmax((i - d0) / std::fmax(d1 - d0, 1e-3), 0.0), 1.0);
      f = f * (1 - g) + f / s->factor * g;
    } else if (kind == PAGED_ROPE_SCALE_WAVELENGTH) {
      const double c =
          std::fmin(std::fmax((L * f / two_pi - low) / (high - low), 0.0), 1.0);
      f = (1 - c) * f / s->factor + c * f;
    }
    freqs[i] = f;
  }
  *factor = kind == PAGED_ROPE_SCALE_YARN && s->factor > 1
                ? static_cast<float>(0.1 * std::log(s->factor) + 1.0)
                : 1.0f;
  return PAGED_ATTN_OK;
}

int paged_rope_table(const double* freqs, int n, uint64_t* table) {
  if (!freqs || !table || n < 0) return PAGED_ATTN_ERR_INVALID_ARGUMENT;
  for (int i = 0; i < n; ++i)
    if (!(std::fabs(freqs[i]) <= 1048576.0)) return PAGED_ATTN_ERR_INVALID_ARGUMENT;
  // 1 / (2 pi) as the sum of two doubles: f / (2 pi) is then exact to about 2^-106 relative,
  // and its fraction to 2^-64, while f * (1 / (2 pi)) alone would be off by 2^-53.
  const double hi = 0.15915494309189535, lo = -9.839338337591243e-18;
  for (int i = 0; i < n; ++i) {
    const double f = std::fabs(freqs[i]);          // a negative one: minus the entry
    double a = f * hi;
    double b = std::fma(f, hi, -a) + f * lo;       // f / (2 pi) = a + b
    a -= std::floor(a);                            // exact: whole turns do not count
    double c = std::floor(std::ldexp(a, 32));      // the first 32 bits, exact
    const double rest = std::ldexp(std::ldexp(a, 32) - c, 32) + std::ldexp(b, 64);
    // rest in units of 2^-64: below 2^32 in magnitude, plus |b| 2^64 < 2^31
    const long long low_bits = static_cast<long long>(std::nearbyint(rest));
    const uint64_t turn = (static_cast<uint64_t>(c) << 32) + static_cast<uint64_t>(low_bits);
    table[i] = freqs[i] < 0 ? 0 - turn : turn;
  }
  return PAGED_ATTN_OK;
}

int paged_rope_run(const paged_rope_params* p, const void* q, const void* k,
                   const int32_t* positions, const uint64_t* table, void* q_out, void* k_out,
                   uint32_t* status, void* stream) {
  if (!rope_params_ok(p)) return PAGED_ATTN_ERR_INVALID_ARGUMENT;
  const bool has_k = p->num_kv_heads > 0;
  if (!q || !q_out || !positions || !table || has_k != (k != nullptr) ||
      has_k != (k_out != nullptr))
    return PAGED_ATTN_ERR_INVALID_ARGUMENT;
  if (!aligned_to(positions, 4) || !aligned_to(table, 8) || !aligned_to(status, 4))
    return PAGED_ATTN_ERR_INVALID_ARGUMENT;
  RopeArgs a{};
  a.q = q; a.k = k; a.qo = q_out; a.ko = k_out;
  a.status = status;
  const long long D = p->head_dim;
  auto strides = [&](long long ts, long long hs, int heads, long long* to_ts, long long* to_hs) {
    const bool packed = ts == 0 && hs == 0;
    *to_ts = packed ? heads * D : ts;
    *to_hs = packed ? D : hs;
  };
  strides(p->q_token_stride, p->q_head_stride, p->num_qo_heads, &a.q_ts, &a.q_hs);
  strides(p->k_token_stride, p->k_head_stride, p->num_kv_heads, &a.k_ts, &a.k_hs);
  strides(p->q_out_token_stride, p->q_out_head_stride, p->num_qo_heads, &a.qo_ts, &a.qo_hs);
  strides(p->k_out_token_stride, p->k_out_head_stride, p->num_kv_heads, &a.ko_ts, &a.ko_hs);
  a.q_in_place = q == q_out;
  a.k_in_place = has_k && k == k_out;
  if ((a.q_in_place && (a.q_ts != a.qo_ts || a.q_hs != a.qo_hs)) ||
      (a.k_in_place && (a.k_ts != a.ko_ts || a.k_hs != a.ko_hs)))
    return PAGED_ATTN_ERR_INVALID_ARGUMENT;
  if (p->num_tokens > 0 &&
      (!rows_apart(p->num_tokens, p->num_qo_heads, D, a.qo_ts, a.qo_hs) ||
       (has_k && !rows_apart(p->num_tokens, p->num_kv_heads, D, a.ko_ts, a.ko_hs))))
    return PAGED_ATTN_ERR_INVALID_ARGUMENT;
  const size_t e = size_of(p->dtype);
  if (!aligned_to(q, e) || !aligned_to(q_out, e) || !aligned_to(k, e) || !aligned_to(k_out, e))
    return PAGED_ATTN_ERR_INVALID_ARGUMENT;
  if (p->num_tokens == 0) return PAGED_ATTN_OK;
  const bool half = p->layout == PAGED_ROPE_HALF;
  a.T = p->num_tokens; a.Hq = p->num_qo_heads; a.Hkv = p->num_kv_heads;
  a.D = p->head_dim; a.n = p->rotary_dim / 2;
  Width w(e);
  for (const void* t : {q, k, static_cast<const void*>(q_out), static_cast<const void*>(k_out)})
    w.pointer(t, e);
  for (long long s : {a.q_ts, a.q_hs, a.qo_ts, a.qo_hs}) w.stride(s);
  if (has_k)
    for (long long s : {a.k_ts, a.k_hs, a.ko_ts, a.ko_hs}) w.stride(s);
  const bool may_stage = w.v * e == 16 && a.q_hs == D && (!has_k || a.k_hs == D) &&
                         (a.Hq + a.Hkv) * D * static_cast<long long>(e) <= kMaxStaged;
  if (half) w.halves(a.n, may_stage);
  a.positions = positions;
  a.table = reinterpret_cast<const unsigned long long*>(table);
  a.inverse = p->inverse != 0;
  a.m = p->attention_factor;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  switch (p->dtype) {
    case PAGED_ATTN_DTYPE_BF16:
      return cuda_status(
          launch_typed<__nv_bfloat16, __nv_bfloat16, false>(a, w.v, half, may_stage, st));
    case PAGED_ATTN_DTYPE_FP16:
      return cuda_status(launch_typed<__half, __half, false>(a, w.v, half, may_stage, st));
    default:
      return cuda_status(launch_typed<float, float, false>(a, w.v, half, may_stage, st));
  }
}

int paged_append_run(const paged_append_params* p, const void* q, const void* k, const void* v,
                     const int32_t* qo_indptr, const int32_t* kv_indptr, const int32_t* pages,
                     const int32_t* lens, const uint64_t* table, void* q_out, void* k_cache,
                     void* v_cache, uint32_t* status, void* stream) {
  const bool packed = qo_indptr != nullptr;
  if (!append_params_ok(p, packed)) return PAGED_ATTN_ERR_INVALID_ARGUMENT;
  const bool has_q = p->num_qo_heads > 0;
  // without requests there are no lengths and no pages, and empty arrays have no address
  if (!k || !v || (p->batch > 0 && (!pages || !lens)) || !k_cache || has_q != (q != nullptr) ||
      has_q != (q_out != nullptr) || (p->combined_cache != 0) == (v_cache != nullptr))
    return PAGED_ATTN_ERR_INVALID_ARGUMENT;
  if (p->rotary_dim > 0 && !table) return PAGED_ATTN_ERR_INVALID_ARGUMENT;
  if (!aligned_to(table, 8)) return PAGED_ATTN_ERR_INVALID_ARGUMENT;
  for (const void* i : {static_cast<const void*>(qo_indptr), static_cast<const void*>(kv_indptr),
                        static_cast<const void*>(pages), static_cast<const void*>(lens),
                        static_cast<const void*>(status)})
    if (!aligned_to(i, 4)) return PAGED_ATTN_ERR_INVALID_ARGUMENT;
  if (p->batch > 0 && !kv_indptr && p->max_pages_per_request <= 0)
    return PAGED_ATTN_ERR_INVALID_ARGUMENT;
  const size_t e = size_of(p->in_dtype);
  if (!aligned_to(q, e) || !aligned_to(k, e) || !aligned_to(v, e) || !aligned_to(q_out, 16) ||
      !aligned_to(k_cache, 16) || !aligned_to(v_cache, 16))
    return PAGED_ATTN_ERR_INVALID_ARGUMENT;
  RopeArgs a{};
  a.T = packed ? p->total_q : p->batch * p->seq_len_q;
  if (a.T == 0 || p->batch == 0) return PAGED_ATTN_OK;
  const long long D = p->head_dim;
  a.q = q; a.k = k; a.v = v; a.qo = q_out; a.ko = k_cache;
  a.Hq = p->num_qo_heads; a.Hkv = p->num_kv_heads; a.D = p->head_dim; a.n = p->rotary_dim / 2;
  a.q_ts = p->q_token_stride ? p->q_token_stride : a.Hq * D;
  a.k_ts = p->k_token_stride ? p->k_token_stride : a.Hkv * D;
  a.v_ts = p->v_token_stride ? p->v_token_stride : a.Hkv * D;
  a.q_hs = a.k_hs = a.qo_hs = D;
  a.qo_ts = a.Hq * D;
  const long long head_page = static_cast<long long>(p->page_size) * D;
  a.page_elems = (p->combined_cache ? 2 : 1) * a.Hkv * head_page;
  a.vo = p->combined_cache ? static_cast<__nv_bfloat16*>(k_cache) + a.Hkv * head_page : v_cache;
  a.table = reinterpret_cast<const unsigned long long*>(table);
  a.m = p->attention_factor;
  a.qo_indptr = qo_indptr; a.kv_indptr = kv_indptr; a.pages = pages; a.lens = lens;
  a.B = p->batch; a.SQ = p->seq_len_q; a.C = p->max_pages_per_request; a.ps = p->page_size;
  a.num_pages = p->num_pages;
  a.status = status;
  const bool half = p->layout == PAGED_ROPE_HALF;
  Width w(e);
  for (const void* t : {q, k, v}) w.pointer(t, e);
  for (long long s : {a.q_ts, a.k_ts, a.v_ts}) w.stride(s);
  const bool may_stage = w.v * e == 16 &&
                         (a.Hq + 2LL * a.Hkv) * D * static_cast<long long>(e) <= kMaxStaged;
  if (half) w.halves(a.n, may_stage);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  switch (p->in_dtype) {
    case PAGED_ATTN_DTYPE_BF16:
      return cuda_status(
          launch_typed<__nv_bfloat16, __nv_bfloat16, true>(a, w.v, half, may_stage, st));
    case PAGED_ATTN_DTYPE_FP16:
      return cuda_status(launch_typed<__half, __nv_bfloat16, true>(a, w.v, half, may_stage, st));
    default:
      return cuda_status(launch_typed<float, __nv_bfloat16, true>(a, w.v, half, may_stage, st));
  }
}

}  // extern "C"
