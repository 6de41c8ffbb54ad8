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

constexpr int kThreads = 128;
constexpr int kMaxStaged = 196608;       // bytes of the rows that one CTA stages at most
constexpr int kStageGoal = 24576;        // bytes of rows that a CTA stages where it may choose
constexpr int kStagedCtas = 6;

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
  int staged_bytes;                      // shared memory of staged rows (a request: may be staged)
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
  const int rest = static_cast<int>((a - (static_cast<unsigned long long>(quarter) << 62)) >> 32);
  float s, c;                              // rest in units of 2^-32 turns, |rest| <= 2^29
  sincospif(static_cast<float>(rest) * 4.656612873077393e-10f, &s, &c);
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
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          smem_u32(dst)),
      "l"(src), "r"(bytes), "r"(smem_u32(bar))
      : "memory");
}

// What a thread holds of one slot between its load and its store.  A slot is V columns pairs (half:
// V of each half) or V columns (interleaved; V = 1 is one pair, element by element, for rows whose
// alignment allows no wider access); the slots behind the rotated ones copy V columns each.
template <typename TIn, int V, bool kHalf>
struct Slot {
  static constexpr bool kTwo = kHalf || V == 1;
  Vec<TIn, V> a, b;
  __device__ __forceinline__ void load(const TIn* x, int n, int s, int rot, int first) {
    if (s < rot) {
      a = *reinterpret_cast<const Vec<TIn, V>*>(x + (!kHalf && V == 1 ? 2 * s : s * V));
      if constexpr (kTwo) b = *reinterpret_cast<const Vec<TIn, V>*>(x + (kHalf ? n + s * V : 2 * s + 1));
    } else {
      a = *reinterpret_cast<const Vec<TIn, V>*>(x + first + (s - rot) * V);
    }
  }
  // (cos, sin) of the slot's pairs
  static constexpr int kPairs = kTwo ? V : V / 2;
  template <typename TOut>
  __device__ __forceinline__ void store(TOut* y, const float2 (&cs)[kPairs], int n, int s, int rot,
                                        int first, bool rotate) const {
    if (s >= rot) {
      *reinterpret_cast<Vec<TOut, V>*>(y + first + (s - rot) * V) = convert<TIn, TOut, V>(a);
      return;
    }
    Vec<TOut, V> c, d;
    if (!rotate) {
      c = convert<TIn, TOut, V>(a);
      if constexpr (kTwo) d = convert<TIn, TOut, V>(b);
    } else {
      float u[V], y1[V];
      unpack(a, u);
      if constexpr (kTwo) {
        float w[V], y2[V];
        unpack(b, w);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          y1[i] = turned(u[i], cs[i].x, -w[i], cs[i].y);
          y2[i] = turned(w[i], cs[i].x, u[i], cs[i].y);
        }
        d = pack<TOut>(y2);
      } else {
#pragma unroll
        for (int i = 0; i < V; i += 2) {
          y1[i] = turned(u[i], cs[i / 2].x, -u[i + 1], cs[i / 2].y);
          y1[i + 1] = turned(u[i + 1], cs[i / 2].x, u[i], cs[i / 2].y);
        }
      }
      c = pack<TOut>(y1);
    }
    if constexpr (kTwo) {
      *reinterpret_cast<Vec<TOut, V>*>(y + (kHalf ? s * V : 2 * s)) = c;
      *reinterpret_cast<Vec<TOut, V>*>(y + (kHalf ? n + s * V : 2 * s + 1)) = d;
    } else {
      *reinterpret_cast<Vec<TOut, V>*>(y + s * V) = c;
    }
  }
};

struct TokenSlot {
  long long off;        // element offset of (page, head 0, slot) in a pool; -1: not written
  int request;          // -1: no request owns the token
  int position;
};

// kStaged: the tile's rows are brought to shared memory by bulk copies, which keeps tens of KB in
// flight per SM whatever the registers allow.  It needs 16-byte aligned tokens with adjacent heads.
template <typename TIn, typename TOut, int V, bool kHalf, bool kAppend, bool kStaged>
__global__ void __launch_bounds__(kThreads, kStaged ? kStagedCtas : 1) rope_kernel(const RopeArgs a) {
  using Held = Slot<TIn, V, kHalf>;
  // Rows in flight per thread: 64 bytes of loads.
  constexpr int kBytes = V * static_cast<int>(sizeof(TIn)) * (Held::kTwo ? 2 : 1);
  constexpr int kBatch = kStaged || kBytes >= 64 ? 1 : (64 / kBytes > 8 ? 8 : 64 / kBytes);
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint64_t arrived;
  __shared__ int gave_up;
  float2* cs = reinterpret_cast<float2*>(smem + a.staged_bytes);    // [tile, n]
  TokenSlot* tok = reinterpret_cast<TokenSlot*>(cs + static_cast<size_t>(a.tile) * a.n);
  const int tid = threadIdx.x;
  const int t0 = blockIdx.x * a.tile;
  const int nt = min(a.tile, a.T - t0);
  const int rot = kHalf ? a.n / V : (V == 1 ? a.n : 2 * a.n / V), first = 2 * a.n;
  const int heads = a.Hq + a.Hkv * (kAppend ? 2 : 1);
  // A thread keeps one slot of one token, and so its sines, and walks the heads; consecutive
  // threads hold consecutive slots, then tokens.  `groups` threads share the heads of a slot.
  const int slots = min(a.slots, kThreads), units = a.tile * slots, groups = kThreads / units;
  const int group = tid / units, unit = tid - group * units;
  const int t = unit / slots, s = blockIdx.y * kThreads + unit - t * slots;
  const bool active = group < groups && t < nt && s < a.slots;
  const long long token = t0 + t;
  grid_dependency_wait();
  grid_launch_dependents();
  const int q_row = a.Hq * a.D, k_row = a.Hkv * a.D;                // staged: elements of a token
  if constexpr (kStaged) {
    if (tid < 32) {
      if (tid == 0) {
        gave_up = 0;
        mbar_init(&arrived, 1);
        fence_mbar_init();
        fence_proxy_async_smem();
        mbar_arrive_expect_tx(&arrived, nt * heads * a.D * static_cast<int>(sizeof(TIn)));
      }
      __syncwarp();
      TIn* to = reinterpret_cast<TIn*>(smem);
      for (int i = tid; i < nt * (kAppend ? 3 : 2); i += 32) {
        const int which = i / nt, j = i - which * nt;
        const long long at = t0 + j;
        TIn* dst = to + j * heads * a.D;
        if (which == 0 && a.Hq > 0)
          bulk_load(dst, static_cast<const TIn*>(a.q) + at * a.q_ts, q_row * sizeof(TIn), &arrived);
        else if (which == 1 && a.Hkv > 0)
          bulk_load(dst + q_row, static_cast<const TIn*>(a.k) + at * a.k_ts, k_row * sizeof(TIn),
                    &arrived);
        else if (which == 2)
          bulk_load(dst + q_row + k_row, static_cast<const TIn*>(a.v) + at * a.v_ts,
                    k_row * sizeof(TIn), &arrived);
      }
    }
  }
  Held x[kBatch];
  auto load = [&](int h0) {
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int h = h0 + u * groups;
      if (h >= heads) break;
      const TIn* p;
      if (kStaged)
        p = reinterpret_cast<const TIn*>(smem) + (t * heads + h) * a.D;
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
  if (!kStaged && active) load(group);
  if constexpr (kAppend) {
    if (a.qo_indptr != nullptr) {
      for (int t = tid; t < nt; t += kThreads) tok[t].request = -1;
      __syncthreads();
      for (int b = tid; b < a.B; b += kThreads) {
        const int lo = max(a.qo_indptr[b], t0), hi = min(a.qo_indptr[b + 1], t0 + nt);
        for (int t = lo; t < hi; ++t) tok[t - t0].request = b;
      }
      __syncthreads();
    }
    for (int t = tid; t < nt; t += kThreads) {
      const int b = a.qo_indptr != nullptr ? tok[t].request : (t0 + t) / a.SQ;
      TokenSlot found{-1, b, 0};
      if (b >= 0) {
        const int end = a.qo_indptr != nullptr ? a.qo_indptr[b + 1] : (b + 1) * a.SQ;
        const int p = a.lens[b] - (end - (t0 + t));
        long long first = static_cast<long long>(b) * a.C;
        int count = a.C;
        if (a.kv_indptr != nullptr) {
          first = a.kv_indptr[b];
          count = a.kv_indptr[b + 1] - a.kv_indptr[b];
        }
        found.position = p;
        const int j = p / a.ps;
        const int page = p >= 0 && j < count ? a.pages[first + j] : -1;
        if (page >= 0 && page < a.num_pages)
          found.off = page * a.page_elems + static_cast<long long>(p - j * a.ps) * a.D;
        else
          report_error(a.status, kErrMetadata);
      }
      tok[t] = found;
    }
    __syncthreads();
  }
  for (int i = tid; i < nt * a.n; i += kThreads) {
    const int j = i / a.n, pair = i - j * a.n;
    const int p = kAppend ? tok[j].position : a.positions[t0 + j];
    cs[i] = turn_of(p, a.table[pair], a.m, a.inverse ? -1.f : 1.f);
  }
  __syncthreads();
  if constexpr (kStaged) {
    if (!mbar_wait(&arrived, 0, a.status, &gave_up)) {
      drain_wait(&arrived, 0);
      return;
    }
  }
  if (!active) return;
  if constexpr (kStaged) load(group);
  float2 turn[Held::kPairs];
#pragma unroll
  for (int i = 0; i < Held::kPairs; ++i)
    turn[i] = s < rot ? cs[t * a.n + s * Held::kPairs + i] : make_float2(0.f, 0.f);
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
    write_q = !(a.q_in_place && s >= rot);
    write_k = !(a.k_in_place && s >= rot);
    k_to = static_cast<TOut*>(a.ko) + token * a.ko_ts;
    k_step = a.ko_hs;
  }
  q_to = static_cast<TOut*>(a.qo) + token * a.qo_ts;
  for (int h0 = group; h0 < heads;) {
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int h = h0 + u * groups;
      if (h >= heads) break;
      if (h < a.Hq) {
        if (write_q) x[u].store(q_to + h * a.qo_hs, turn, a.n, s, rot, first, true);
      } else if (write_k) {
        const int j = h - a.Hq;
        if (!kAppend || j < a.Hkv)
          x[u].store(k_to + j * k_step, turn, a.n, s, rot, first, true);
        else
          x[u].store(v_to + (j - a.Hkv) * k_step, turn, a.n, s, rot, first, false);
      }
    }
    h0 += kBatch * groups;
    load(h0);
  }
}

template <typename TIn, typename TOut, int V, bool kHalf, bool kAppend>
cudaError_t launch_kernel(const RopeArgs& a, dim3 grid, size_t smem, bool staged, cudaStream_t st) {
  count_launches(1);
  if constexpr (V * sizeof(TIn) == 16) {
    if (staged) {
      static std::atomic<uint64_t> ready{0};
      void (*const kernel)(RopeArgs) = rope_kernel<TIn, TOut, V, kHalf, kAppend, true>;
      if (!kernel_smem_ready(kernel, kMaxStaged + 16384, ready)) return cudaErrorUnknown;
      return launch_after_previous(kernel, grid, dim3(kThreads), smem, st, a);
    }
  }
  return launch_after_previous(rope_kernel<TIn, TOut, V, kHalf, kAppend, false>, grid,
                               dim3(kThreads), smem, st, a);
}

template <typename TIn, typename TOut, int V, bool kAppend>
cudaError_t launch_v(RopeArgs a, bool half, cudaStream_t st) {
  const int sms = current_sm_count();
  if (sms <= 0) return cudaErrorUnknown;
  const bool copies = !(a.q_in_place && (a.Hkv == 0 || a.k_in_place));  // columns past the rotated
  const int rot = half ? a.n / V : (V == 1 ? a.n : 2 * a.n / V);
  a.slots = rot + (copies ? (a.D - 2 * a.n) / V : 0);
  const int slots = a.slots < kThreads ? a.slots : kThreads;
  const long long token_bytes =
      static_cast<long long>(a.Hq + a.Hkv * (kAppend ? 2 : 1)) * a.D * sizeof(TIn);
  const bool staged = a.staged_bytes != 0 && V * sizeof(TIn) == 16 && a.T >= 16 * sms &&
                      (copies || a.D == 2 * a.n) && token_bytes <= kMaxStaged;
  // Tokens per CTA: one while there are few; else as many as keep most threads busy (the slots of
  // the tile's tokens, times the groups that share the heads, within the CTA).
  a.tile = 1;
  if (a.T >= 16 * sms) {
    int best = 0;
    for (int tile = 1; tile <= (staged ? 16 : 4) && tile * slots <= kThreads; tile *= 2) {
      if (staged && tile > 1 && tile * token_bytes > kStageGoal) break;
      const int busy = kThreads / (tile * slots) * (tile * slots);
      if (busy >= best) {
        best = busy;
        a.tile = tile;
      }
    }
  }
  a.staged_bytes = staged ? static_cast<int>(align_up(a.tile * token_bytes, 128)) : 0;
  const size_t smem = a.staged_bytes +
                      static_cast<size_t>(a.tile) * (a.n * sizeof(float2) + sizeof(TokenSlot));
  const dim3 grid(ceil_div(a.T, a.tile), ceil_div(a.slots, kThreads));
  return half ? launch_kernel<TIn, TOut, V, true, kAppend>(a, grid, smem, staged, st)
              : launch_kernel<TIn, TOut, V, false, kAppend>(a, grid, smem, staged, st);
}

template <typename TIn, typename TOut, bool kAppend>
cudaError_t launch_typed(const RopeArgs& a, int v, bool half, cudaStream_t st) {
  if constexpr (sizeof(TIn) == 2) {
    if (v >= 8) return launch_v<TIn, TOut, 8, kAppend>(a, half, st);
  }
  if (v >= 4) return launch_v<TIn, TOut, 4, kAppend>(a, half, st);
  if (v >= 2) return launch_v<TIn, TOut, 2, kAppend>(a, half, st);
  return launch_v<TIn, TOut, 1, kAppend>(a, half, st);
}

bool layout_ok(int R, int D, int layout, float m, bool may_be_zero) {
  if (R < 0 || R > D || R % 2 || (R == 0 && !may_be_zero)) return false;
  return (layout == PAGED_ROPE_HALF || layout == PAGED_ROPE_INTERLEAVED) && std::isfinite(m);
}

size_t size_of(int dtype) { return dtype == PAGED_ATTN_DTYPE_FP32 ? 4 : 2; }

bool aligned_to(const void* p, size_t bytes) {
  return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0;
}

// The largest power of two of elements per access that the columns, the pointers and the
// strides allow: in the half layout both halves have to start on an access.
struct Width {
  int v;
  Width(int R, bool half, size_t elem) : v(elem == 4 ? 4 : 8) {
    while (v > 1 && (half ? (R / 2) % v : R % v) != 0) v /= 2;
  }
  void pointer(const void* p, size_t elem) {
    while (v > 1 && !aligned_to(p, v * elem)) v /= 2;
  }
  void stride(long long s) {
    while (v > 1 && s % v != 0) v /= 2;
  }
};

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
                   void* stream) {
  if (!rope_params_ok(p)) return PAGED_ATTN_ERR_INVALID_ARGUMENT;
  const bool has_k = p->num_kv_heads > 0;
  if (!q || !q_out || !positions || !table || has_k != (k != nullptr) ||
      has_k != (k_out != nullptr))
    return PAGED_ATTN_ERR_INVALID_ARGUMENT;
  RopeArgs a{};
  a.q = q; a.k = k; a.qo = q_out; a.ko = k_out;
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
  if (a.q_in_place && (a.q_ts != a.qo_ts || a.q_hs != a.qo_hs)) return PAGED_ATTN_ERR_INVALID_ARGUMENT;
  if (a.k_in_place && (a.k_ts != a.ko_ts || a.k_hs != a.ko_hs)) return PAGED_ATTN_ERR_INVALID_ARGUMENT;
  const size_t e = size_of(p->dtype);
  if (!aligned_to(q, e) || !aligned_to(q_out, e) || !aligned_to(k, e) || !aligned_to(k_out, e))
    return PAGED_ATTN_ERR_INVALID_ARGUMENT;
  if (p->num_tokens == 0) return PAGED_ATTN_OK;
  const bool half = p->layout == PAGED_ROPE_HALF;
  Width w(p->rotary_dim, half, e);
  for (const void* t : {q, k, static_cast<const void*>(q_out), static_cast<const void*>(k_out)})
    w.pointer(t, e);
  for (long long s : {a.q_ts, a.q_hs, a.qo_ts, a.qo_hs}) w.stride(s);
  if (has_k)
    for (long long s : {a.k_ts, a.k_hs, a.ko_ts, a.ko_hs}) w.stride(s);
  a.staged_bytes = aligned_to(q, 16) && aligned_to(k, 16) && a.q_hs == D && a.q_ts * e % 16 == 0 &&
                   (!has_k || (a.k_hs == D && a.k_ts * e % 16 == 0));
  a.positions = positions;
  a.table = reinterpret_cast<const unsigned long long*>(table);
  a.T = p->num_tokens; a.Hq = p->num_qo_heads; a.Hkv = p->num_kv_heads;
  a.D = p->head_dim; a.n = p->rotary_dim / 2;
  a.inverse = p->inverse != 0;
  a.m = p->attention_factor;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  switch (p->dtype) {
    case PAGED_ATTN_DTYPE_BF16:
      return cuda_status(launch_typed<__nv_bfloat16, __nv_bfloat16, false>(a, w.v, half, st));
    case PAGED_ATTN_DTYPE_FP16:
      return cuda_status(launch_typed<__half, __half, false>(a, w.v, half, st));
    default:
      return cuda_status(launch_typed<float, float, false>(a, w.v, half, st));
  }
}

int paged_append_run(const paged_append_params* p, const void* q, const void* k, const void* v,
                     const int32_t* qo_indptr, const int32_t* kv_indptr, const int32_t* pages,
                     const int32_t* lens, const uint64_t* table, void* q_out, void* k_cache,
                     void* v_cache, uint32_t* status, void* stream) {
  const bool packed = qo_indptr != nullptr;
  if (!append_params_ok(p, packed)) return PAGED_ATTN_ERR_INVALID_ARGUMENT;
  const bool has_q = p->num_qo_heads > 0;
  if (!k || !v || !pages || !lens || !k_cache || has_q != (q != nullptr) ||
      has_q != (q_out != nullptr) || (p->combined_cache != 0) == (v_cache != nullptr))
    return PAGED_ATTN_ERR_INVALID_ARGUMENT;
  if (p->rotary_dim > 0 && !table) return PAGED_ATTN_ERR_INVALID_ARGUMENT;
  if (!kv_indptr && p->max_pages_per_request <= 0) return PAGED_ATTN_ERR_INVALID_ARGUMENT;
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
  a.staged_bytes = aligned_to(q, 16) && aligned_to(k, 16) && aligned_to(v, 16) &&
                   a.q_ts * e % 16 == 0 && a.k_ts * e % 16 == 0 && a.v_ts * e % 16 == 0;
  const bool half = p->layout == PAGED_ROPE_HALF;
  Width w(p->rotary_dim, half, e);
  for (const void* t : {q, k, v}) w.pointer(t, e);
  for (long long s : {a.q_ts, a.k_ts, a.v_ts}) w.stride(s);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  switch (p->in_dtype) {
    case PAGED_ATTN_DTYPE_BF16:
      return cuda_status(launch_typed<__nv_bfloat16, __nv_bfloat16, true>(a, w.v, half, st));
    case PAGED_ATTN_DTYPE_FP16:
      return cuda_status(launch_typed<__half, __nv_bfloat16, true>(a, w.v, half, st));
    default:
      return cuda_status(launch_typed<float, __nv_bfloat16, true>(a, w.v, half, st));
  }
}

}  // extern "C"
