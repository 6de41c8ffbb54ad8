// Keeping a row within a budget of tokens (include/paged_cache.h documents the contract): the
// tokens to keep are selected by the attention weight that they received, and the rows are cut
// back to them.
#include "pages.cuh"

namespace pa {
namespace {

// ---- select ------------------------------------------------------------------------------------
// A list is the weights of one (layer, row, KV head).  Its tokens get 32-bit keys whose unsigned
// order is the order of preference.  The smallest key that is kept, T, is bracketed between keys of
// which at least and fewer than the wanted number of tokens follow.  The first bracket comes from a
// sample of 32 keys of every warp; it is cut at pivots by interpolation between its counts until
// exactly the wanted number of tokens follow or one key is left.  Keys stay in registers, kOwn a
// thread (32; 8 where there are CTAs to spare and time is latency): a step costs two instructions a
// key and a barrier.  What a bracket of few keys holds goes to shared memory: cheap steps there.
// A last pass writes the indices in order, those of key T until their number is reached.
// Instructions bound it: the issue slots are 70% full, some 3,000 instructions a warp, of which its
// keys ask for about 1,000; the rest is the sample and what every warp does at each step.  For
// 2,048 lists of up to 8,192 tokens histograms of the keys' digits took 143 us (half of the tokens
// may have the same weight, and then shared-memory atomics queue up), plain bisection 112 us,
// interpolation between the least and the greatest key 64 us, this 56 us; one warp alone in the
// last steps 58 us, four pivots at a time there 60 us (what every warp does beside the counting
// doubles).  Where no warp has 32 open keys, or T lies outside the sample, a second sample and the
// ends of the list's range cost 2 us of them, and save up to half: 384 lists of 796 tokens, 301 of
// them kept anyway, 18.6 us against 39.  Lists of more than 32,768 tokens that get no cluster are
// read from memory at every step.
constexpr uint32_t kMustKeep = 0xffffffffu;
constexpr int kSelectCluster = 8;
constexpr int kSelectThreads = 1024;
constexpr int kLeft = 2048;                // keys of the bracket that go to shared memory

struct SelectArgs {
  const int* rows;
  int n, R, N, Hkv, W, K, sink, recent;
  const float* weights;                    // [N, R, Hkv, W]
  const int* lens;
  int* kept;                               // [N, n, Hkv, K]
  uint32_t* status;
};

// Keys order floats, -0.0 as 0.0 and NaN below everything.
__device__ __forceinline__ uint32_t weight_key(float x) {
  if (x != x) return 0u;
  const uint32_t u = __float_as_uint(x + 0.f);
  return (u >> 31) ? ~u : (u | 0x80000000u);
}

// What the warps and CTAs of a list exchange, in shared memory; two buffers used in turn, so that a
// barrier orders each.  The CTAs of a list take the same turns: the sample, for which some may need
// a second attempt, has buffers of its own.
struct SelectShared {
  uint32_t warps[2][2][32], sample[2][2][32];
  uint32_t cta[2][2][kSelectCluster];
  alignas(16) uint32_t left[kLeft];        // the last keys of the bracket, and how many
  uint32_t lefts;
};

// The tokens [begin, begin + count) of a list, this CTA's share of it.
template <bool kHeld, int kOwn>
__device__ __forceinline__ void select_list(const SelectArgs& a, SelectShared& sh, const float* w,
                                            int L, int begin, int count, int* out) {
  cg::cluster_group cl = cg::this_cluster();
  const int rank = cl.block_rank(), size = cl.num_blocks();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  // Warp v goes through tokens from v * run on, a lane each, 32 at a time.
  const int run = kHeld ? 32 * kOwn : ((count + warps - 1) / warps + 31) / 32 * 32;
  const int first = min(warp * run, count), last = min(first + run, count);
  const int kept_from = L - a.recent;
  const auto make_key = [&](int t, float x) {
    const int j = begin + t;
    return j < a.sink || j >= kept_from ? kMustKeep : weight_key(x);
  };
  // few warps have tokens that are kept whatever their weight
  const bool ends = begin + first < a.sink || begin + last > kept_from;
  uint32_t held[kOwn];                     // keys past the end are 0, below every pivot
  if (kHeld) {
    const float* mine = w + begin + first + lane;
    const int mine_left = last - first - lane;
    float x[kOwn];                         // all loads on their way together
#pragma unroll
    for (int e = 0; e < kOwn; ++e) x[e] = e * 32 < mine_left ? __ldcs(mine + e * 32) : NAN;
#pragma unroll
    for (int e = 0; e < kOwn; ++e) held[e] = weight_key(x[e]);
    if (ends) {
#pragma unroll
      for (int e = 0; e < kOwn; ++e)
        if (e * 32 < mine_left) held[e] = make_key(first + e * 32 + lane, x[e]);
    }
  }
  const auto load_key = [&](int t) { return t < last ? make_key(t, w[begin + t]) : 0u; };
  int turn = 0;
  const auto min_of = [](uint32_t v) { return __reduce_min_sync(0xffffffffu, v); };
  const auto max_of = [](uint32_t v) { return __reduce_max_sync(0xffffffffu, v); };
  const auto sum = [](uint32_t v) { return __reduce_add_sync(0xffffffffu, v); };
  // Both values, which the CTA's threads agree on, over the CTAs of the list.
  const auto over_cluster = [&](uint32_t& x, uint32_t& y, const auto& op_x, const auto& op_y,
                                uint32_t zero_x, uint32_t zero_y) {
    if (warp == 0 && lane < size) {
      *cl.map_shared_rank(&sh.cta[turn][0][rank], lane) = x;
      *cl.map_shared_rank(&sh.cta[turn][1][rank], lane) = y;
    }
    cl.sync();
    x = op_x(lane < size ? sh.cta[turn][0][lane] : zero_x);
    y = op_y(lane < size ? sh.cta[turn][1][lane] : zero_y);
  };
  const auto own_count = [&](uint32_t pivot) {               // of this thread; pivot > 0
    uint32_t p[4] = {0, 0, 0, 0};
    if (kHeld) {
      // key >= pivot is the carry of key + (2^32 - pivot)
#pragma unroll
      for (int e = 0; e < kOwn; ++e)
        asm("{\n\t.reg .u32 t;\n\tadd.cc.u32 t, %1, %2;\n\taddc.u32 %0, %0, 0;\n\t}"
            : "+r"(p[e & 3])
            : "r"(held[e]), "r"(0u - pivot));
    } else {
      for (int t0 = first; t0 < last; t0 += 32) p[0] += load_key(t0 + lane) >= pivot;
    }
    return (p[0] + p[1]) + (p[2] + p[3]);
  };
  // Over all threads of the list.
  const auto sum_all = [&](uint32_t& x, uint32_t& y) {
    x = sum(x);
    y = sum(y);
    if (lane == 0) {
      sh.warps[turn][0][warp] = x;
      sh.warps[turn][1][warp] = y;
    }
    __syncthreads();
    x = sum(lane < warps ? sh.warps[turn][0][lane] : 0u);
    y = sum(lane < warps ? sh.warps[turn][1][lane] : 0u);
    if (size > 1) over_cluster(x, y, sum, sum, 0u, 0u);
    turn ^= 1;
  };
  const auto sum_one = [&](uint32_t x) {
    x = sum(x);
    if (lane == 0) sh.warps[turn][0][warp] = x;
    __syncthreads();
    x = sum(lane < warps ? sh.warps[turn][0][lane] : 0u);
    if (size > 1) {
      if (warp == 0 && lane < size) *cl.map_shared_rank(&sh.cta[turn][0][rank], lane) = x;
      cl.sync();
      x = sum(lane < size ? sh.cta[turn][0][lane] : 0u);
    }
    turn ^= 1;
    return static_cast<int>(x);
  };
  // from_low tokens have keys >= low, at least K; above of them keys >= high, fewer than K (K where
  // it ends early).
  uint32_t low = 0u, high = kMustKeep;
  int from_low = L, above = a.sink + a.recent;
  bool done = above == a.K;                // nothing else is kept
  // The sample: every warp with 32 keys, all of them open, takes the one at the wanted place in
  // their order (where no warp has, every one of 32 from all over the list); of up to 8 warps' keys
  // the least and the greatest, of more those some two deviations about the median, are the first
  // two pivots.
  uint32_t from = kMustKeep, to = 0u;
  bool tied = false;                       // T may be `from`, the key of many tokens
  if (threadIdx.x == 0) sh.lefts = 0;      // (the barriers below order it)
  for (int again = 0; !done && again < 2; ++again) {
    const int open = L - above;
    uint32_t key = 0u;
    int same = 0;
    if (again > 0 || (last - first >= 32 && !ends)) {
      const uint32_t mine =
          again > 0 ? weight_key(w[a.sink + static_cast<int>(static_cast<long long>(threadIdx.x) *
                                                             open / static_cast<int>(blockDim.x))])
                    : (kHeld ? held[0] : load_key(first + lane));
      uint32_t not_less = 0;
#pragma unroll 8
      for (int j = 0; j < 32; ++j) not_less += __shfl_sync(0xffffffffu, mine, j) >= mine;
      const uint32_t place = static_cast<uint32_t>(32LL * (a.K - above) / open);
      key = max_of(not_less > place ? mine : 0u);
      same = __popc(__ballot_sync(0xffffffffu, mine == key));
    }
    if (lane == 0) {
      sh.sample[again][0][warp] = key;
      sh.sample[again][1][warp] = same;
    }
    __syncthreads();
    const uint32_t x = lane < warps ? sh.sample[again][0][lane] : 0u;
    const int n = __popc(__ballot_sync(0xffffffffu, x != 0u));
    if (n == 0 && again == 0) continue;
    if (n <= 8) {
      from = min_of(x != 0u ? x : kMustKeep);
      to = max_of(x);
    } else {
      int more = 0;                        // of the others
      for (int j = 0; j < warps; ++j) {
        const uint32_t y = __shfl_sync(0xffffffffu, x, j);
        more += y > x || (y == x && j < lane);
      }
      const int spread = static_cast<int>(sqrtf(static_cast<float>(n))) + 1;
      from = max_of(x != 0u && more == min(n - 1, n / 2 + spread) ? x : 0u);
      to = max_of(x != 0u && more == max(0, (n - 1) / 2 - spread) ? x : 0u);
    }
    // (half of the warps say so)
    tied = size == 1 && 2 * __popc(__ballot_sync(0xffffffffu,
                                                 lane < warps && x == from &&
                                                     sh.sample[again][1][lane] >= 4u)) >= n;
    break;
  }
  if (!done && size > 1) over_cluster(from, to, min_of, max_of, kMustKeep, 0u);
  turn ^= 1;
  from = min(max(from, 1u), kMustKeep - 2);
  to = min(max(to, from), kMustKeep - 2) + 1;
  // Then the root of count - K.  An end that stays while the other one moves twice in a row loses
  // half of its weight; every fourth pivot is the middle.
  float f_low = 1.f, f_high = 1.f;
  int moved = 0;
  uint32_t own_low = 0, own_high = 0;      // of this thread, once the end has moved
  const auto cut_at = [&](uint32_t pivot, int c, uint32_t own) {
    if (c == a.K) {                        // exactly the keys from here on are kept
      high = pivot;
      above = c;
      done = true;
    } else if (c > a.K) {
      low = pivot;
      from_low = c;
      own_low = own;
      f_low = static_cast<float>(c - a.K) + 0.5f;
      if (moved > 0) f_high *= 0.5f;
      moved = 1;
    } else {
      high = pivot;
      above = c;
      own_high = own;
      f_high = static_cast<float>(a.K - c) - 0.5f;
      if (moved < 0) f_low *= 0.5f;
      moved = -1;
    }
  };
  int step = 0;
  const auto next_pivot = [&] {
    ++step;
    const uint32_t width = high - low;
    uint32_t d = width / 2;
    if (low == from && (step == 5 || (step == 1 && tied))) d = 1;     // that key alone?
    else if ((step & 3) != 0)
      d = static_cast<uint32_t>(static_cast<float>(width) * __fdividef(f_low, f_low + f_high));
    return low + min(max(d, 1u), width - 1);
  };
  if (!done) {
    const uint32_t own_from = own_count(from), own_to = own_count(to);
    uint32_t x = own_from, y = own_to;
    sum_all(x, y);
    cut_at(from, x, own_from);             // x >= y: the second one lies inside the bracket, too
    if (!done && to < high) cut_at(to, y, own_to);
  }
  if (!done && (low == 0u || high == kMustKeep)) {
    // T is not inside the sample: the least and the greatest open key are the ends.
    uint32_t least = kMustKeep, most = 0u;
    const auto range = [&](uint32_t k, bool live) {
      if (!live || k == kMustKeep) return;
      least = min(least, k);
      most = max(most, k);
    };
    if (kHeld) {
#pragma unroll
      for (int e = 0; e < kOwn; ++e) range(held[e], first + e * 32 + lane < last);
    } else {
      for (int t0 = first; t0 < last; t0 += 32) range(load_key(t0 + lane), t0 + lane < last);
    }
    least = min_of(least);
    most = max_of(most);
    if (lane == 0) {
      sh.warps[turn][0][warp] = least;
      sh.warps[turn][1][warp] = most;
    }
    __syncthreads();
    least = min_of(lane < warps ? sh.warps[turn][0][lane] : kMustKeep);
    most = max_of(lane < warps ? sh.warps[turn][1][lane] : 0u);
    if (size > 1) over_cluster(least, most, min_of, max_of, kMustKeep, 0u);
    turn ^= 1;
    if (low == 0u && least > 0u) {         // (0: a NaN, which the end at 0 serves)
      low = least;
      own_low = own_count(low);
    }
    if (low == least) f_low = static_cast<float>(from_low - a.K) + 0.5f;
    if (high == kMustKeep) {
      high = most + 1;
      own_high = own_count(high);
      f_high = static_cast<float>(a.K - above) - 0.5f;
    }
  }
  moved = 0;
  bool few = false;                        // the bracket's keys, `left`, are in shared memory
  int left = 0, beyond = 0;                // and `beyond` tokens have greater ones
  while (!done && high - low > 1) {
    if (kHeld && size == 1 && !few && low > 0u &&
        from_low - above <= min(kLeft, 8 * static_cast<int>(blockDim.x))) {
      // (in no order that matters)
      const uint32_t own = own_low - own_high, width = high - low;
      const int upto = warp_inclusive(static_cast<int>(own));
      int base = 0;
      if (lane == 31) base = atomicAdd(&sh.lefts, static_cast<uint32_t>(upto));
      uint32_t* put = sh.left + __shfl_sync(0xffffffffu, base, 31) + upto - own;
#pragma unroll
      for (int e = 0; e < kOwn; ++e)
        if (held[e] - low < width) *put++ = held[e];
      few = true;
      left = from_low - above;
      beyond = above;
      for (int x = left + threadIdx.x; x < (left + 3) / 4 * 4; x += blockDim.x) sh.left[x] = 0u;
      __syncthreads();
    }
    const uint32_t pivot = next_pivot();
    if (few) {
      uint32_t c[2] = {0, 0};
      for (int x = threadIdx.x * 4; x < left; x += blockDim.x * 4) {
        const uint4 k = *reinterpret_cast<const uint4*>(sh.left + x);
        c[0] += k.x >= pivot;
        c[1] += k.y >= pivot;
        c[0] += k.z >= pivot;
        c[1] += k.w >= pivot;
      }
      cut_at(pivot, beyond + sum_one(c[0] + c[1]), 0u);
    } else {
      const uint32_t own = own_count(pivot);
      cut_at(pivot, sum_one(own), own);
    }
  }
  // Kept: the keys >= high and, while they last, the first K - above tokens with key low.  Where
  // there is nothing to choose among those, the keys from one cut on.
  const int need = a.K - above;
  const bool choose = need > 0 && need < from_low - above;
  const uint32_t cut = need > 0 ? low : high;
  uint32_t gt = 0, eq = 0;                 // tokens from the cut on (choose: above it), and at it
  const auto tally = [&](uint32_t k, bool live) {
    if (!live) return;
    gt += choose ? k > cut : k >= cut;
    eq += k == cut;
  };
  if (kHeld && cut > 0 && !choose) {
#pragma unroll
    for (int e = 0; e < kOwn; ++e) gt += held[e] >= cut;
  } else if (kHeld) {
#pragma unroll
    for (int e = 0; e < kOwn; ++e) tally(held[e], first + e * 32 + lane < last);
  } else {
    for (int t0 = first; t0 < last; t0 += 32) tally(load_key(t0 + lane), t0 + lane < last);
  }
  gt = sum(gt);
  eq = sum(eq);
  if (lane == 0) {
    sh.warps[turn][0][warp] = gt;
    sh.warps[turn][1][warp] = eq;
  }
  __syncthreads();
  const int g = lane < warps ? sh.warps[turn][0][lane] : 0;
  const int q = lane < warps ? sh.warps[turn][1][lane] : 0;
  const int gs = warp_inclusive(g), qs = warp_inclusive(q);
  int gt_before = __shfl_sync(0xffffffffu, gs - g, warp);
  int eq_before = __shfl_sync(0xffffffffu, qs - q, warp);
  if (size > 1) {
    const int all_gt = __shfl_sync(0xffffffffu, gs, 31), all_eq = __shfl_sync(0xffffffffu, qs, 31);
    if (warp == 0 && lane < size) {
      *cl.map_shared_rank(&sh.cta[turn][0][rank], lane) = all_gt;
      *cl.map_shared_rank(&sh.cta[turn][1][rank], lane) = all_eq;
    }
    cl.sync();
    for (int r = 0; r < rank; ++r) {
      gt_before += sh.cta[turn][0][r];
      eq_before += sh.cta[turn][1][r];
    }
  }
  const uint32_t below = (1u << lane) - 1u;
  if (kHeld && cut > 0 && !choose) {
    int* to = out + gt_before;
    const int token = begin + first + lane;
#pragma unroll
    for (int e = 0; e < kOwn; ++e) {
      const bool keep = held[e] >= cut;
      const uint32_t m = __ballot_sync(0xffffffffu, keep);
      if (keep) to[__popc(m & below)] = token + e * 32;
      to += __popc(m);
    }
    return;
  }
  for (int t0 = first, e = 0; t0 < last; t0 += 32, ++e) {
    uint32_t k;
    if (kHeld) {
      k = held[0];
#pragma unroll
      for (int x = 1; x < kOwn; ++x) k = e == x ? held[x] : k;
    } else {
      k = load_key(t0 + lane);
    }
    const bool in = t0 + lane < last;
    const uint32_t gm = __ballot_sync(0xffffffffu, in && (choose ? k > cut : k >= cut));
    const uint32_t qm = __ballot_sync(0xffffffffu, choose && in && k == cut);
    const int rank_eq = choose ? eq_before + __popc(qm & below) : 0;
    const bool is_eq = choose && k == cut;
    if (in && (is_eq ? rank_eq < need : k >= cut))
      out[gt_before + __popc(gm & below) + min(rank_eq, need)] = begin + t0 + lane;
    gt_before += __popc(gm);
    eq_before += __popc(qm);
  }
}

// Short lists: every token is ranked by comparing it with all.  1,568 lists of 20 tokens take 6 us;
// 35 us through the search, whose sample they are too short for.
constexpr int kShort = 256;
__device__ __forceinline__ void select_short(const SelectArgs& a, SelectShared& sh, const float* w,
                                             int L, int* out) {
  const int tid = threadIdx.x, lane = tid & 31, threads = blockDim.x;
  const int all = (L + 31) / 32 * 32;
  for (int j = tid; j < all; j += threads)
    sh.left[j] = j >= L ? 0u : (j < a.sink || j >= L - a.recent ? kMustKeep : weight_key(w[j]));
  __syncthreads();
  for (int j = tid; j < all; j += threads) {
    const uint32_t mine = sh.left[j];
    int before = 0;                        // tokens that are preferred to this one
    for (int x = 0; x < L; x += 4) {       // (those past the end follow in any order)
      const uint4 k = *reinterpret_cast<const uint4*>(sh.left + x);
      before += (k.x > mine || (k.x == mine && x < j)) +
                (k.y > mine || (k.y == mine && x + 1 < j)) +
                (k.z > mine || (k.z == mine && x + 2 < j)) +
                (k.w > mine || (k.w == mine && x + 3 < j));
    }
    const uint32_t kept = __ballot_sync(0xffffffffu, j < L && before < a.K);
    if (lane == 0) sh.warps[0][0][j / 32] = kept;
  }
  __syncthreads();
  for (int j = tid; j < all; j += threads) {
    const uint32_t kept = sh.warps[0][0][j / 32];
    int at = __popc(kept & ((1u << lane) - 1u));
    for (int x = 0; x < j / 32; ++x) at += __popc(sh.warps[0][0][x]);
    if (kept >> lane & 1u) out[at] = j;
  }
}

template <int kOwn>
__global__ void __launch_bounds__(kSelectThreads)
select_kernel(const __grid_constant__ SelectArgs a) {
  __shared__ SelectShared sh;
  cg::cluster_group cl = cg::this_cluster();
  const int rank = cl.block_rank(), size = cl.num_blocks();
  const int tid = threadIdx.x, threads = blockDim.x;
  grid_dependency_wait();
  grid_launch_dependents();
  const int list = blockIdx.x / size;      // ((layer, item), head)
  const int h = list % a.Hkv, li = list / a.Hkv, i = li % a.n, layer = li / a.n;
  const int row = a.rows[i];
  int* out = a.kept + static_cast<long long>(list) * a.K;
  const bool known = row >= 0 && row < a.R;
  const int L = known ? a.lens[row] : -1;
  if (L < 0 || L > a.W) {                  // left out: no list
    if (rank == 0 && tid == 0) report_error(a.status, kErrMetadata);
    for (int j = rank * threads + tid; j < a.K; j += size * threads) out[j] = -1;
    return;
  }
  if (L <= a.K) {                          // everything is kept
    for (int j = rank * threads + tid; j < a.K; j += size * threads) out[j] = j < L ? j : -1;
    return;
  }
  const float* w = a.weights + ((static_cast<long long>(layer) * a.R + row) * a.Hkv + h) * a.W;
  if (L <= kShort) {
    if (rank == 0) select_short(a, sh, w, L, out);
    return;
  }
  if (size > 1) cl.sync();                 // every CTA's shared memory is there
  const int per = ((L + size - 1) / size + 31) / 32 * 32;
  const int begin = min(rank * per, L), count = min(per, L - begin);
  if (per <= threads * kOwn) select_list<true, kOwn>(a, sh, w, L, begin, count, out);
  else select_list<false, kOwn>(a, sh, w, L, begin, count, out);
}

// ---- evict -------------------------------------------------------------------------------------
// Three kernels.  The first looks at every item: is it in order, and which of the pages that it
// will write are shared and so need a fresh one.  The second hands out the fresh pages in order
// (FreePages) and writes the new tables and lengths.  The third moves the tokens and gives the
// pages back that the rows no longer name.
constexpr int kThreads = 256;

struct EvictArgs {
  Pools pools;
  int npools, segs;          // runs of tokens per page and pool: one per head, K and V
  int per_layer;             // pools of a layer
  long long page_bytes;
  int seg_bytes, token_bytes;
  const int* rows;
  int n;
  const int* kept;           // [N, n, Hkv, K]
  int N, Hkv, K;
  int first_page;            // pages before it keep their contents: sink / ps
  int need_pages;            // Kp = ceil(K / ps)
  float* weights;            // [N, R, Hkv, W] or null
  int W;
  int* tables;
  int* lens;
  int* refs;
  int R, C, ps, P;
  unsigned long long by_ps;  // ceil(2^64 / ps)
  int4* items;               // workspace [n]: row, length (-1: left out), fresh pages needed
  int* old;                  // workspace [n, Kp]: the row's first pages before the call
  int* slots;                // workspace [n, Kp]: table columns of the pages to replace
  int shift, slices;         // move: words of a token per unit (log2), units per token
  Status status;
};

__device__ __forceinline__ int page_of(int token, unsigned long long by_ps) {
  return static_cast<int>(__umul64hi(static_cast<unsigned>(token), by_ps));
}

__global__ void __launch_bounds__(kThreads) look_kernel(const __grid_constant__ EvictArgs a) {
  __shared__ int warp_sums[32];
  const int tid = threadIdx.x, i = blockIdx.x;
  grid_dependency_wait();
  grid_launch_dependents();
  const int row = a.rows[i];
  int L = row >= 0 && row < a.R ? a.lens[row] : -1;
  bool bad = L < 0;
  for (int k = tid; k < i; k += kThreads) bad |= a.rows[k] == row;
  const int pages = bad ? 0 : static_cast<int>((L + a.ps - 1LL) / a.ps);
  bad |= pages > a.C;
  const bool cut = L > a.K;
  if (cut && !bad) {
    if (a.weights) bad |= L > a.W;
    const int lists = a.N * a.Hkv;
    for (int k = tid; k < lists; k += kThreads) {
      const int layer = k / a.Hkv, h = k - layer * a.Hkv;
      const int* list =
          a.kept + ((static_cast<long long>(layer) * a.n + i) * a.Hkv + h) * a.K;
      const int last = list[a.K - 1];
      bad |= list[0] < 0 || last < a.K - 1 || last >= L;
    }
    const int* t = a.tables + static_cast<long long>(row) * a.C;
    if (pages <= a.C)
      for (int p = tid; p < pages; p += kThreads) bad |= t[p] < 0 || t[p] >= a.P;
  }
  bad = __syncthreads_or(bad);
  int need = 0;
  if (cut && !bad) {
    const int* t = a.tables + static_cast<long long>(row) * a.C;
    const long long at = static_cast<long long>(i) * a.need_pages;
    for (int p0 = 0; p0 < a.need_pages; p0 += kThreads) {
      const int p = p0 + tid;
      bool shared = false;
      if (p < a.need_pages) {
        const int page = t[p];
        a.old[at + p] = page;
        shared = p >= a.first_page && a.refs[page] > 1;
      }
      int sum;
      const int rank = need + block_scan(shared, warp_sums, &sum);
      if (shared) a.slots[at + rank] = p;
      need += sum;
    }
  }
  if (tid == 0) a.items[i] = make_int4(row, bad ? -1 : L, need, 0);
}

// One cluster.  Every CTA sums the items' demands for itself; without any (rows whose pages are
// their own) nobody looks at the pages.
__global__ void __launch_bounds__(kPlanThreads)
evict_plan_kernel(const __grid_constant__ EvictArgs a) {
  extern __shared__ __align__(16) int shared[];
  __shared__ int warp_sums[32];
  cg::cluster_group cl = cg::this_cluster();
  const int rank = cl.block_rank(), size = cl.num_blocks();
  const int tid = threadIdx.x, threads = blockDim.x;
  int* off = shared;                       // [n] first fresh page of the item among all demands
  grid_dependency_wait();
  grid_launch_dependents();
  if (rank == 0 && tid < 4) a.status.ws[tid] = 0;
  int need[kPerThread], before[kPerThread], demand = 0;
#pragma unroll
  for (int j = 0; j < kPerThread; ++j) {
    const int i = j * threads + tid;
    if (j * threads >= a.n) break;
    need[j] = i < a.n ? a.items[i].z : 0;
    int sum;
    before[j] = add_pages(demand, block_scan(need[j], warp_sums, &sum));
    demand = add_pages(demand, sum);
    if (i < a.n) off[i] = before[j];
  }
  FreePages pages;
  pages.total = 0;
  if (demand > 0) {
    pages.count(a.refs, a.P, rank, size, off + a.n, [] {});
    sync_cluster(cl);
    pages.order(cl);
    if (size > 1) cluster_arrive();
  }
  uint32_t bits = 0;
  if (rank == 0) {
#pragma unroll
    for (int j = 0; j < kPerThread; ++j) {
      const int i = j * threads + tid;
      if (j * threads >= a.n) break;
      if (i >= a.n) continue;
      const int4 it = a.items[i];
      if (it.y < 0) bits |= kErrMetadata;
      if (it.y <= a.K) continue;
      if (need[j] == 0 || before[j] + need[j] <= pages.total) {
        a.lens[it.x] = a.K;
      } else {
        bits |= kErrCapacity;
        a.items[i].y = -1;
      }
    }
    __syncthreads();                       // the word is cleared
    if (bits) report(a.status, bits);
  }
  if (demand == 0) return;
  __syncthreads();
  const auto owner = [&](int k) {          // the last item with off <= k
    int lo = 0, hi = a.n;
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (off[mid] <= k) lo = mid; else hi = mid;
    }
    return lo;
  };
  const int handed = demand <= pages.total ? demand : off[owner(pages.total)];
  for (int j = 0; j < pages.own; ++j) {
    if (pages.step_before[j * size + rank] >= handed) break;
    pages.each(j, [&](int p, bool is_free, int k, int) {
      if (!is_free || k >= handed) return;
      const int i = owner(k);
      const int slot = a.slots[static_cast<long long>(i) * a.need_pages + (k - off[i])];
      a.tables[static_cast<long long>(a.items[i].x) * a.C + slot] = p;
      a.refs[p] = 1;
    });
  }
  if (size > 1) cluster_wait();
}

__device__ __forceinline__ uint4 ld_words(const uint8_t* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p)
               : "memory");
  return v;
}

// A unit is the tokens of one (item, pool, head), or a slice of their columns where that makes
// more CTAs.  Lists are ascending, so token kept[j] lies at or behind slot j: a CTA that goes
// through the slots in order, loads a tile of tokens, waits for all of its threads and then stores
// it overwrites nothing that is still to be read.  16 words of 16 bytes per thread are in flight.
constexpr int kWords = 16;
__global__ void __launch_bounds__(kThreads, 2) move_kernel(const __grid_constant__ EvictArgs a) {
  extern __shared__ __align__(16) long long offsets[];       // [2][source, target][tile]
  const int tid = threadIdx.x;
  const int tile = (kWords * kThreads) >> a.shift;           // tokens
  grid_dependency_wait();
  grid_launch_dependents();
  const int per_pool = a.segs * a.slices, data = a.npools * per_pool;
  const int lists = a.weights ? a.N * a.Hkv : 0;
  const int per_item = data + lists + 1;
  const long long units = static_cast<long long>(a.n) * per_item;
  for (long long u = blockIdx.x; u < units; u += gridDim.x) {
    const int i = static_cast<int>(u / per_item);
    const int w = static_cast<int>(u - static_cast<long long>(i) * per_item);
    const int4 item = a.items[i];
    const int L = item.y;
    if (L <= a.K) continue;
    const int* now = a.tables + static_cast<long long>(item.x) * a.C;
    const int* old = a.old + static_cast<long long>(i) * a.need_pages;
    if (w == data + lists) {               // pages that the row no longer names
      const int pages = static_cast<int>((L + a.ps - 1LL) / a.ps);
      bool bad = false;
      for (int p = a.first_page + tid; p < pages; p += kThreads) {
        int page;
        if (p < a.need_pages) {
          page = old[p];
          if (page == now[p]) continue;
        } else {
          page = now[p];
        }
        if (atomicSub(a.refs + page, 1) <= 0) {
          atomicAdd(a.refs + page, 1);
          bad = true;
        }
      }
      if (bad) report(a.status, kErrMetadata);
      continue;
    }
    if (w >= data) {                       // the weights of one layer and head
      const int layer = (w - data) / a.Hkv, h = (w - data) - layer * a.Hkv;
      const int* list = a.kept + ((static_cast<long long>(layer) * a.n + i) * a.Hkv + h) * a.K;
      float* x = a.weights + ((static_cast<long long>(layer) * a.R + item.x) * a.Hkv + h) * a.W;
      for (int j0 = 0; j0 < a.K; j0 += kWords * kThreads) {
        float v[kWords];
        uint32_t have = 0;
#pragma unroll
        for (int b = 0; b < kWords; ++b) {
          const int j = j0 + b * kThreads + tid;
          if (j >= a.K) break;
          const int t = list[j];
          if (t < j || t >= L) continue;
          v[b] = x[t];
          have |= 1u << b;
        }
        __syncthreads();
#pragma unroll
        for (int b = 0; b < kWords; ++b)
          if (have >> b & 1u) x[j0 + b * kThreads + tid] = v[b];
        __syncthreads();
      }
      continue;
    }
    const int pool = w / per_pool, seg = (w - pool * per_pool) / a.slices;
    const int slice = w % a.slices;
    const int layer = pool / a.per_layer, h = seg % a.Hkv;
    const int* list = a.kept + ((static_cast<long long>(layer) * a.n + i) * a.Hkv + h) * a.K;
    uint8_t* base = static_cast<uint8_t*>(a.pools.p[pool]) +
                    static_cast<long long>(seg) * a.seg_bytes;
    const int words = a.token_bytes / 16;
    int buf = 0;
    bool bad = false;
    for (int j0 = 0; j0 < a.K; j0 += tile, buf ^= 1) {
      long long* from = offsets + buf * 2 * tile;
      long long* to = from + tile;
      for (int x = tid; x < tile; x += kThreads) {
        const int j = j0 + x;
        long long s = -1, d = 0;
        if (j < a.K) {
          const int t = list[j], q = page_of(j, a.by_ps);
          if (t < j || t >= L || (q < a.first_page && t != j)) {
            bad = true;
          } else {
            const int p = page_of(t, a.by_ps);
            const int source = p < a.need_pages ? old[p] : now[p], target = now[q];
            s = source * a.page_bytes + static_cast<long long>(t - p * a.ps) * a.token_bytes;
            d = target * a.page_bytes + static_cast<long long>(j - q * a.ps) * a.token_bytes;
            if (s == d) s = -1;            // it stays where it is
          }
        }
        from[x] = s;
        to[x] = d;
      }
      __syncthreads();
      uint4 v[kWords];
#pragma unroll
      for (int b = 0; b < kWords; ++b) {
        const int x = b * kThreads + tid, t = x >> a.shift;
        const int word = (slice << a.shift) + (x & ((1 << a.shift) - 1));
        if (word < words && from[t] >= 0) v[b] = ld_words(base + from[t] + word * 16);
      }
      __syncthreads();                     // the whole tile is read
#pragma unroll
      for (int b = 0; b < kWords; ++b) {
        const int x = b * kThreads + tid, t = x >> a.shift;
        const int word = (slice << a.shift) + (x & ((1 << a.shift) - 1));
        if (word < words && from[t] >= 0)
          *reinterpret_cast<uint4*>(base + to[t] + word * 16) = v[b];
      }
    }
    if (bad) report(a.status, kErrMetadata);
    __syncthreads();                       // the next unit writes the offsets anew
  }
}

struct EvictLayout {
  size_t status, items, old, slots, total;
  EvictLayout(int n, int pages) {
    Take t;
    status = t.ints(4);
    items = t.ints(4LL * n);
    old = t.ints(static_cast<long long>(n) * pages);
    slots = t.ints(static_cast<long long>(n) * pages);
    total = t.off;
  }
};

bool page_size_ok(int ps) { return ps >= 8 && ps <= 128 && ps % 8 == 0; }

}  // namespace
}  // namespace pa

using namespace pa;

extern "C" {

int paged_cache_select_run(const paged_cache_select_params* p, const int32_t* rows, int n,
                           const float* weights, const int32_t* lens, int32_t* kept,
                           uint32_t* status, void* stream) {
  if (!p || n < 0 || p->num_layers <= 0 || p->rows < 0 || p->num_kv_heads <= 0 || p->width <= 0 ||
      p->keep <= 0 || p->sink < 0 || p->recent < 0 || p->recent > p->keep - p->sink)
    return PAGED_ATTN_ERR_INVALID_ARGUMENT;
  if (n == 0) return PAGED_ATTN_OK;
  if (!rows || !weights || !lens || !kept || !ints_aligned(rows, weights, lens, kept, status))
    return PAGED_ATTN_ERR_INVALID_ARGUMENT;
  const long long lists = static_cast<long long>(p->num_layers) * n * p->num_kv_heads;
  if (lists * kSelectCluster > kMaxGrid) return PAGED_ATTN_ERR_INVALID_ARGUMENT;
  const int sms = current_sm_count();
  if (sms <= 0) return PAGED_ATTN_ERR_CUDA;
  SelectArgs a{};
  a.rows = rows; a.n = n; a.R = p->rows; a.N = p->num_layers; a.Hkv = p->num_kv_heads;
  a.W = p->width; a.K = p->keep; a.sink = p->sink; a.recent = p->recent;
  a.weights = weights; a.lens = lens; a.kept = kept; a.status = status;
  // A cluster where there are few lists and long ones; threads for all of a list's keys.
  int size = 1;
  while (size < kSelectCluster && lists * size * 2 <= sms && p->width / size > 8192) size *= 2;
  const int per = ceil_div(p->width, size);
  const bool few = lists * size <= 2 * sms && per <= 8 * kSelectThreads;
  int threads = (ceil_div(per, few ? 8 : 32) + 31) / 32 * 32;
  threads = threads < 64 ? 64 : (threads > kSelectThreads ? kSelectThreads : threads);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = static_cast<unsigned>(lists * size);
  cfg.blockDim = threads;
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = size;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  count_launches(1);
  return cuda_status(few ? cudaLaunchKernelEx(&cfg, select_kernel<8>, a)
                         : cudaLaunchKernelEx(&cfg, select_kernel<32>, a));
}

size_t paged_cache_evict_workspace_size(int n, int keep, int page_size) {
  if (n < 0 || n > kMaxItems || keep <= 0 || !page_size_ok(page_size)) return 0;
  return EvictLayout(n, (keep - 1) / page_size + 1).total;
}

int paged_cache_evict_run(const paged_cache_params* p, const paged_cache_pools* pools,
                          const int32_t* rows, int n, const int32_t* kept, int keep, int sink,
                          float* weights, int weights_width, int32_t* tables, int32_t* lens,
                          int32_t* refs, void* ws, size_t ws_bytes, void* stream) {
  if (!cache_params_ok(p) || !pools_ok(pools) || n < 0 || n > kMaxItems || keep <= 0 || sink < 0 ||
      sink > keep)
    return PAGED_ATTN_ERR_INVALID_ARGUMENT;
  if (pools->num_pages != p->num_pages || pools->page_size != p->page_size)
    return PAGED_ATTN_ERR_INVALID_ARGUMENT;
  if (n > 0 && (!rows || !kept || !tables || !lens || !refs))
    return PAGED_ATTN_ERR_INVALID_ARGUMENT;
  if (weights && weights_width <= 0) return PAGED_ATTN_ERR_INVALID_ARGUMENT;
  if (!ints_aligned(rows, kept, weights, tables, lens, refs) || !aligned_to(ws, 16))
    return PAGED_ATTN_ERR_INVALID_ARGUMENT;
  EvictArgs a{};
  a.need_pages = (keep - 1) / p->page_size + 1;
  const EvictLayout l(n, a.need_pages);
  if (!ws || ws_bytes < l.total) return PAGED_ATTN_ERR_WORKSPACE;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (n == 0) return cuda_status(cudaMemsetAsync(ws, 0, 4 * sizeof(uint32_t), st));
  const int sms = current_sm_count();
  if (sms <= 0) return PAGED_ATTN_ERR_CUDA;
  a.npools = pool_count(pools);
  for (int i = 0; i < a.npools; ++i) a.pools.p[i] = pools->pools_host[i];
  a.per_layer = pools->combined_cache ? 1 : 2;
  a.segs = (pools->combined_cache ? 2 : 1) * pools->num_kv_heads;
  a.page_bytes = page_bytes(pools);
  a.seg_bytes = static_cast<int>(seg_bytes(pools));
  a.token_bytes = 2 * pools->head_dim;
  a.rows = rows; a.n = n; a.kept = kept;
  a.N = pools->num_layers; a.Hkv = pools->num_kv_heads; a.K = keep;
  a.first_page = sink / p->page_size;
  a.weights = weights; a.W = weights_width;
  a.tables = tables; a.lens = lens; a.refs = refs;
  a.R = p->rows; a.C = p->max_pages_per_request; a.ps = p->page_size; a.P = p->num_pages;
  a.by_ps = ~0ull / static_cast<unsigned>(a.ps) + 1;         // ceil(2^64 / ps): ps is even
  a.items = reinterpret_cast<int4*>(at(ws, l.items));
  a.old = at(ws, l.old);
  a.slots = at(ws, l.slots);
  a.status = {reinterpret_cast<uint32_t*>(at(ws, l.status)), p->status_dev};
  // Slices of a token's columns: whole tokens where there are CTAs enough, never under 32 bytes.
  const int words = pools->head_dim / 8;
  int shift = 1;
  while ((1 << shift) < words) ++shift;
  const long long runs = static_cast<long long>(n) * a.npools * a.segs;
  while (shift > 1 && runs * ceil_div(words, 1 << shift) < 2LL * sms) --shift;
  a.shift = shift;
  a.slices = ceil_div(words, 1 << shift);
  count_launches(1);
  cudaError_t e = launch_after_previous(look_kernel, n, kThreads, 0, st, a);
  if (e != cudaSuccess) return PAGED_ATTN_ERR_CUDA;
  static std::atomic<uint64_t> ready{0};
  e = launch_plan(evict_plan_kernel, a, a.P, 4, n, n, ready, st);
  if (e != cudaSuccess) return PAGED_ATTN_ERR_CUDA;
  const long long units =
      n * (static_cast<long long>(a.npools) * a.segs * a.slices +
           (weights ? static_cast<long long>(a.N) * a.Hkv : 0) + 1);
  const int tile = (kWords * kThreads) >> shift;
  static std::atomic<uint64_t> move_ready{0};
  if (!kernel_smem_ready(move_kernel, 4 * 8 * ((kWords * kThreads) >> 1), move_ready))
    return PAGED_ATTN_ERR_CUDA;
  count_launches(1);
  return cuda_status(launch_after_previous(move_kernel,
                                           static_cast<int>(units < kMaxGrid ? units : kMaxGrid),
                                           kThreads, 4 * 8 * tile, st, a));
}

}  // extern "C"
