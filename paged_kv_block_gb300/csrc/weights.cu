// Attention weight per cached token (include/paged_cache.h documents the contract): for every key
// of a request the sum over its queries, and over the query heads of the key's KV head, of
// exp(scale q.k - lse), with the log-sum-exp that the attention call returned.  No maximum and no
// second pass are needed, and no value row is read.
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
  r.bad |= r.keys < L;
  if (nq == 0) r.keys = 0;                 // nothing is asked of the request
  return r;
}
// Row of a head of KV head h in lse, and of D columns in q.
__device__ __forceinline__ long long head_row(const WeightsArgs& a, int row, int h, int head) {
  return static_cast<long long>(row) * a.Hq + h * a.G + head;
}
__device__ __forceinline__ int over(int x, unsigned long long by_ps) {
  return static_cast<int>(__umul64hi(static_cast<unsigned>(x), by_ps));
}

// ---- few rows: decode ----------------------------------------------------------------------------
// Bound by reading K.  A warp takes 16 keys at a time as the A operand of warp MMAs, the request's
// rows (query, head) as the B operand, 8 NT of them.  The contraction runs over columns in any
// order, so a lane loads 16 bytes of its key's row and takes them as its operands of two MMAs:
// K comes from HBM straight into registers, without shared memory or barriers, and the loads of
// all the SM's warps are in flight together.  The scores of a key then lie in the four lanes of a
// quad.
constexpr int kNarrowThreads = 128;
constexpr int kNarrowChunk = 128;          // keys of a unit: 32 per warp

template <int D, int NT>
__global__ void __launch_bounds__(kNarrowThreads)
narrow_kernel(const __grid_constant__ WeightsArgs a) {
  constexpr int kBlocks = D / 32;          // 32 columns: two MMAs
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int gr = lane >> 2, tq = lane & 3;
  grid_dependency_wait();
  grid_launch_dependents();
  const int pairs = a.B * a.Hkv;
  const int chunks = (a.W + kNarrowChunk - 1) / kNarrowChunk;
  for (long long u = blockIdx.x; u < static_cast<long long>(pairs) * chunks; u += gridDim.x) {
    const int c = static_cast<int>(u / pairs);
    const int bh = static_cast<int>(u - static_cast<long long>(c) * pairs);
    const int b = bh / a.Hkv, h = bh - b * a.Hkv;
    const Request r = request_of(a, b);
    if (r.bad && c == 0 && h == 0 && threadIdx.x == 0) report_error(a.status, kErrMetadata);
    const int key0 = c * kNarrowChunk + warp * 32;
    if (key0 >= r.keys) continue;
    float* w = a.w + static_cast<long long>(bh) * a.W;
    // this lane's rows of the two 16-key steps: keys key0 + 16 s + gr and + 8
    const __nv_bfloat16* row[4];
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const int key = key0 + 8 * x + gr;
      row[x] = nullptr;
      if (key < r.keys) {
        const int p = over(key, a.by_ps), page = __ldg(r.pages + p);
        if (page >= 0 && page < a.P)
          row[x] = a.k + (page * a.page_rows + h * a.ps + (key - p * a.ps)) * D + tq * 8;
        else
          report_error(a.status, kErrMetadata);
      }
    }
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
      float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        uint4 ka[kBlocks], kb[kBlocks];
#pragma unroll
        for (int i = 0; i < kBlocks; ++i) {
          ka[i] = kb[i] = make_uint4(0u, 0u, 0u, 0u);
          if (row[2 * s]) ka[i] = ld_stream(reinterpret_cast<const uint4*>(row[2 * s] + i * 32));
          if (row[2 * s + 1])
            kb[i] = ld_stream(reinterpret_cast<const uint4*>(row[2 * s + 1] + i * 32));
        }
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
      const __nv_bfloat16* live =
          tq == 0 ? row[0] : (tq == 1 ? row[1] : (tq == 2 ? row[2] : row[3]));
      const int key = key0 + 8 * tq + gr;
      if (live) {
        float before = 0.f;
        if (r0 > 0) before = w[key];
        else if (key < r.old && a.decay != 0.f) before = a.decay * w[key];
        w[key] = before + mine;
      }
    }
  }
}

template <int D, int NT>
cudaError_t launch_narrow(const WeightsArgs& a, cudaStream_t st) {
  const int sms = current_sm_count();
  if (sms <= 0) return cudaErrorUnknown;
  const long long units = static_cast<long long>(a.B) * a.Hkv * ceil_div(a.W, kNarrowChunk);
  const long long most = 16LL * sms;
  count_launches(1);
  return launch_after_previous(narrow_kernel<D, NT>, static_cast<int>(units < most ? units : most),
                               kNarrowThreads, 0, st, a);
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
  long long rows = ceil_div(p->total_q, p->batch);         // of a request, on average
  if (a.last > 0 && a.last < rows) rows = a.last;
  rows *= a.G;
  if (p->head_dim == 128)
    return cuda_status(rows <= 8 ? launch_narrow<128, 1>(a, st)
                                 : (rows <= 16 ? launch_narrow<128, 2>(a, st)
                                               : launch_narrow<128, 4>(a, st)));
  return cuda_status(rows <= 8 ? launch_narrow<256, 1>(a, st) : launch_narrow<256, 2>(a, st));
}

}  // extern "C"
