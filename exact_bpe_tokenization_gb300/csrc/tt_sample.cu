// tt_sample.cu - drawing token IDs from rows of logits (include/toktier.h).
//
// Every sum is of whole numbers, so it is exact and any split of a row gives
// the same ID.  A cluster of blocks holds a row in shared memory: it is read
// once, and the passes over it (the maximum; the weights' sum; for rows that
// need them, histograms) cost no memory traffic.
//
// What top-k and top-p keep is a prefix of the tokens in the order of their
// weights.  Sorting a row for it would cost far more than reading it, and the
// prefix is nearly always short, so a list of the heaviest tokens is made
// first: the row's maxima over 128 groups of threads are known from the first
// pass, and the tokens at or above the q-th largest of them are at least q and
// rarely twice as many.  If the prefix ends within the list (its count, or
// its sum against the row's, says so), one block ranks the list by counting.
// Else (a top-k above 96, a flat row) the end is found by histograms of the
// weights' bits over the cluster, 16 bins an octave and then finer, until few
// enough tokens share a bin to be ranked.
#include <algorithm>

#include "tt_ops.cuh"

using namespace tt::ops;

namespace {

typedef unsigned long long u64;

constexpr int THREADS = 512;
constexpr int WARPS = THREADS / 32;
constexpr int HELD = 88 * 1024;                   // bytes of a row a block holds: two blocks an SM
constexpr int GROUPS = 128;                       // groups of threads a row's maxima are taken over
constexpr int LIST = 512;                         // tokens one block ranks
constexpr int BIN_LIST = 256;                     // tokens of a bin that are ranked and not divided further
constexpr int SHIFT = 19;                         // first histogram: 16 bins an octave
constexpr int BINS = (40 << (23 - SHIFT)) + 1;    // weights 1 .. 2^40
constexpr int FINER = 9;                          // bits a further histogram resolves
constexpr float ONE = 1099511627776.f;            // 2^40, the largest weight
constexpr uint32_t KEY_ONE = 0x3F800000u;         // the bits of weight 1

struct SampleArgs {
  int64_t n_vocab, stride;
  const float *uniform, *temperature;
  const int32_t *top_k;
  const float *top_p, *min_p;
  int32_t *ids;
  float *logprobs;
  int32_t *status;
  int cluster_log2, held;
};

// rint(e * 2^40) of an e in [0, 1]: whole above 2^23, below it rounded by the
// addition
__device__ __forceinline__ float weight_of(float e) {
  const float x = e * ONE;
  return x >= 8388608.f ? x : (x + 8388608.f) - 8388608.f;
}

// A sum of rint(e * 2^40) without a conversion: adding 96 leaves e rounded to
// 2^-17 in the low bits, and adding 1.5 * 2^-17 to what that cut off leaves the
// rest, rounded to 2^-40.  Both counts stay below 2^31 for 256 terms.
struct Sum {
  int hi = 0, lo = 0;
  __device__ __forceinline__ void add(float e) {
    const float a = __fadd_rn(e, 96.f), h = __fadd_rn(a, -96.f);
    const float b = __fadd_rn(__fadd_rn(e, -h), 1.5f / 131072.f);
    hi += __float_as_int(a) - 0x42C00000;
    lo += __float_as_int(b) - 0x37400000;
  }
  __device__ __forceinline__ u64 value() const { return ((u64)hi << 23) + (u64)(long long)lo; }
};

__device__ __forceinline__ u64 warp_sum(u64 v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
  return v;
}

struct Shared {
  float group_max[GROUPS];          // this block's part, then (in all_max) the row's
  float all_max[GROUPS];
  float nth_max;
  u64 seg[WARPS];                   // sums over the warps' parts of the row
  u64 sum, list_sum;                // the block's, and its list's
  u64 scan[WARPS];
  uint32_t scan_n[WARPS];
  int n_list;
  int index;                        // a token found in the row (the first block's counts)
  int bin;                          // where a prefix ends
  uint32_t bin_n, bin_before;
  u64 bin_sum_before;
  u64 cut_key;
  u64 list[LIST];                   // bits of the weight << 32 | ~ID: larger first
  u64 red_sum[BINS];                // a histogram over the row
  uint32_t red_n[BINS];
  uint32_t n[BINS], low[BINS], high[BINS];   // and this block's
};

__device__ __forceinline__ u64 list_key(float w, int j) { return (u64)__float_as_uint(w) << 32 | (uint32_t)~j; }
__device__ __forceinline__ float key_weight(u64 k) { return __uint_as_float((uint32_t)(k >> 32)); }

// One row, as a block of its cluster sees it.
template <class T> struct Row {
  static constexpr int E = RowParts<T>::E;
  const uint4 *body;
  uint4 *s_row;
  int held, lo, hi;                 // the warp's vectors of the block's
  int first;                        // index of the block's vector 0's first element
  int lone;                         // a single element of this thread's, or -1
  bool lone_first;                  // which comes before the vectors, or behind them
  float x_lone;
  float m, c;
  bool infinite;                    // the maximum is +inf

  __device__ __forceinline__ uint4 vec(int v) const { return v < held ? s_row[v] : __ldg(body + v); }

  // 2^((l - M) c); 0 for NaN and -inf
  __device__ __forceinline__ void powers(const uint4 &r, float e[E]) const {
    vec_f32(r, e, T{});
    if (infinite) {
#pragma unroll
      for (int i = 0; i < E; ++i) e[i] = e[i] == INF ? 1.f : 0.f;
      return;
    }
#pragma unroll
    for (int i = 0; i < E; i += 2) {
      const float2 z = sub_mul2(make_float2(e[i], e[i + 1]), m, c);
      e[i] = ex2(fmaxf(z.x, -200.f));
      e[i + 1] = ex2(fmaxf(z.y, -200.f));
    }
  }
  __device__ __forceinline__ float power(float l) const {
    if (infinite) return l == INF ? 1.f : 0.f;
    return ex2(fmaxf((l - m) * c, -200.f));
  }
  __device__ __forceinline__ int index(int v, int i) const { return first + v * E + i; }

  // f(e, index) of the warp's elements, lane by lane
  template <class F> __device__ __forceinline__ void each(F f) const {
    for (int v = lo + (threadIdx.x & 31); v < hi; v += 32) {
      float e[E];
      powers(vec(v), e);
#pragma unroll
      for (int i = 0; i < E; ++i) f(e[i], index(v, i));
    }
    if (lone >= 0) f(power(x_lone), lone);
  }

  // The first of the warp's elements, by index, at which the running sum of
  // val(e, index) passes r (it does); its value in `own`.
  template <class F> __device__ int find(F val, u64 r, u64 &own) const {
    const int lane = threadIdx.x & 31;
    u64 before = 0;
    auto lone_step = [&](int &found) {
      const u64 mine = lone >= 0 ? val(power(x_lone), lone) : 0;
      return step(mine, before, r, found, own);
    };
    int found = -1;
    const bool any_lone = __any_sync(~0u, lone >= 0), at_first = __any_sync(~0u, lone >= 0 && lone_first);
    if (any_lone && at_first && lone_step(found)) {
      own = __shfl_sync(~0u, own, found);
      return __shfl_sync(~0u, lone, found);
    }
    for (int v0 = lo; v0 < hi; v0 += 32) {
      const int v = v0 + lane;
      u64 val8[E], mine = 0;
      if (v < hi) {
        float e[E];
        powers(vec(v), e);
#pragma unroll
        for (int i = 0; i < E; ++i) mine += val8[i] = val(e[i], index(v, i));
      }
      u64 start = before;
      if (step(mine, before, r, found, own)) {
        // the lane whose vector passes r walks through it
        start = start_of(mine, start);
        int at = 0;
        u64 w = 0;
        if (lane == found) {
          bool past = false;
#pragma unroll
          for (int i = 0; i < E; ++i) {
            start += val8[i];
            if (!past && start > r) {
              past = true;
              at = index(v, i);
              w = val8[i];
            }
          }
        }
        own = __shfl_sync(~0u, w, found);
        return __shfl_sync(~0u, at, found);
      }
    }
    if (any_lone && !at_first && lone_step(found)) {
      own = __shfl_sync(~0u, own, found);
      return __shfl_sync(~0u, lone, found);
    }
    return -1;
  }
  // sum of the lanes before this one, from `base`
  static __device__ __forceinline__ u64 start_of(u64 mine, u64 base) {
    u64 x = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const u64 y = __shfl_up_sync(~0u, x, o);
      if ((threadIdx.x & 31) >= o) x += y;
    }
    return base + x - mine;
  }
  // whether the running sum passes r at a lane; else it is carried on
  static __device__ __forceinline__ bool step(u64 mine, u64 &before, u64 r, int &found, u64 &own) {
    const u64 start = start_of(mine, before);
    const uint32_t past = __ballot_sync(~0u, start + mine > r);
    own = mine;
    found = __ffs(past) - 1;
    before = __shfl_sync(~0u, start + mine, 31);
    return past != 0;
  }
};

template <class T>
__global__ void __launch_bounds__(THREADS, 2) k_sample(SampleArgs a, const T *__restrict__ logits) {
  constexpr int E = RowParts<T>::E, U = 4;
  extern __shared__ uint4 s_row[];
  __shared__ Shared s;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int C = 1 << a.cluster_log2, rank = C > 1 ? (int)cluster_rank() : 0;
  const int64_t row = blockIdx.x >> a.cluster_log2;
  const int V = (int)a.n_vocab;
  auto sync_row = [&]() {
    if (C > 1) cluster_sync(); else __syncthreads();
  };
  auto at = [&](auto *p, int r) { return C > 1 ? of_block(p, r) : p; };
  auto arrive = [&]() { if (C > 1) cluster_arrive(); };   // blocks stay until all have read from them
  auto leave = [&]() { if (C > 1) cluster_wait(); };

  const float u = a.uniform[row], temp = a.temperature ? a.temperature[row] : 1.f;
  const float top_p = a.top_p ? a.top_p[row] : 1.f, min_p = a.min_p ? a.min_p[row] : 0.f;
  const int top_k = a.top_k ? a.top_k[row] : 0;

  // ---- the row into shared memory, and the groups' maxima.  A warp takes
  // consecutive vectors, so that warps and blocks lie in the order of the IDs.
  Row<T> x;
  {
    const T *l = logits + row * a.stride;
    const RowParts<T> part(l, V);
    const int each = (part.vecs + C - 1) >> a.cluster_log2, first = min(part.vecs, rank * each);
    const int n = min(part.vecs - first, each), slab = (n + WARPS - 1) / WARPS;
    x.body = reinterpret_cast<const uint4 *>(l + part.lead) + first;
    x.s_row = s_row;
    x.held = a.held;
    x.first = part.lead + first * E;
    x.lo = min(n, warp * slab);
    x.hi = min(n, x.lo + slab);
    x.lone_first = rank == 0 && warp == 0 && lane < part.lead;
    x.lone = x.lone_first ? lane : rank == C - 1 && warp == WARPS - 1 && lane < part.rest ? V - part.rest + lane : -1;
    // (a thread has at most one: with both in one warp, C and WARPS would be 1)
    x.x_lone = x.lone >= 0 ? to_f32(l[x.lone]) : -INF;
  }
  float m = fmaxf(x.x_lone, -INF);
  for (int v0 = x.lo + lane; v0 < x.hi; v0 += 32 * U) {
    uint4 r[U];
#pragma unroll
    for (int i = 0; i < U; ++i)
      if (v0 + 32 * i < x.hi) r[i] = __ldg(x.body + v0 + 32 * i);
#pragma unroll
    for (int i = 0; i < U; ++i)
      if (v0 + 32 * i < x.hi) {
        if (v0 + 32 * i < x.held) s_row[v0 + 32 * i] = r[i];
        float v[E];
        vec_f32(r[i], v, T{});
#pragma unroll
        for (int k = 0; k < E; ++k) m = fmaxf(m, v[k]);
      }
  }
  const int group_lanes = 4 * C, block_groups = GROUPS >> a.cluster_log2;
  for (int o = 1; o < group_lanes; o <<= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, o));
  if (tid % group_lanes == 0) s.group_max[tid / group_lanes] = m;
  if (tid == 0) s.n_list = 0;
  sync_row();
  if (tid < GROUPS) s.all_max[tid] = at(s.group_max, tid / block_groups)[tid % block_groups];
  __syncthreads();
  m = warp_all(fmaxf(fmaxf(s.all_max[lane], s.all_max[lane + 32]), fmaxf(s.all_max[lane + 64], s.all_max[lane + 96])), OpMax());
  const bool valid = u >= 0 && u < 1 && temp >= 0 && temp < INF && top_p >= 0 && top_p <= 1 && min_p >= 0 && min_p <= 1;
  if (!valid || m == -INF) {
    arrive();
    if (rank == 0 && tid == 0) {
      a.ids[row] = -1;
      if (a.logprobs) a.logprobs[row] = -INF;
      if (!valid) op_status(a.status, TT_ERR_INVALID_ARG);
    }
    leave();
    return;
  }
  x.m = m;
  x.c = fminf(1.44269504f / temp, 3.402823466e38f);
  x.infinite = m == INF;
  const int k = temp == 0 ? 1 : top_k > 0 ? min(top_k, V) : V;
  const float least_w = fmaxf(min_p * ONE, 1.f);              // min-p, and weight 0 is never drawn
  auto write = [&](int id, u64 w, u64 total) {
    a.ids[row] = id;
    if (a.logprobs) {
      // the smaller of the share and its complement, whole until then
      const u64 rest = total - w;
      a.logprobs[row] = rest < w ? log1pf(-__fdiv_rn((float)rest, (float)total)) : logf(__fdiv_rn((float)w, (float)total));
    }
  };

  // ---- the lowest ID of the largest weight
  if (k == 1) {
    int best = INT32_MAX;
    x.each([&](float e, int j) {
      if (weight_of(e) == ONE) best = min(best, j);
    });
    best = __reduce_min_sync(~0u, best);
    if (lane == 0) s.scan_n[warp] = best;
    __syncthreads();
    if (tid == 0) {
      for (int w = 1; w < WARPS; ++w) best = min(best, (int)s.scan_n[w]);
      s.index = best;
    }
    sync_row();
    if (rank == 0 && tid == 0) {
      for (int r = 1; r < C; ++r) best = min(best, *at(&s.index, r));
      write(best, 1, 1);
    }
    arrive();
    leave();
    return;
  }

  // ---- sums, and the list of the heaviest tokens
  const bool all = k == V && top_p == 1.f;                    // nothing but min-p cuts
  float list_w = least_w;                                     // the list holds all weights from here on
  if (!all) {
    const int q = min(k, GROUPS * 3 / 4);
    // four threads rank a group's maximum
    const float own = s.all_max[tid >> 2];
    int above = 0;
    for (int i = tid & 3; i < GROUPS; i += 4) above += s.all_max[i] > own || (s.all_max[i] == own && i < (tid >> 2));
    above += __shfl_xor_sync(~0u, above, 1);
    above += __shfl_xor_sync(~0u, above, 2);
    if ((tid & 3) == 0 && above == q - 1) s.nth_max = own;
    __syncthreads();
    list_w = fmaxf(list_w, weight_of(x.power(s.nth_max)));
  }
  auto push = [&](float w, int j) {
    const int n = atomicAdd(&s.n_list, 1);
    if (n < LIST) s.list[n] = list_key(w, j);
  };
  u64 sum = 0;
  if (min_p == 0.f) {
    const float near_e = all ? 2.f : list_w * (0.99999f / ONE);
    for (int v = x.lo + lane; v < x.hi; v += 32) {
      float e[E];
      x.powers(x.vec(v), e);
      Sum t;
      float top = e[0];
#pragma unroll
      for (int i = 0; i < E; ++i) {
        t.add(e[i]);
        top = fmaxf(top, e[i]);
      }
      sum += t.value();
      if (top >= near_e) {
#pragma unroll
        for (int i = 0; i < E; ++i)
          if (weight_of(e[i]) >= list_w) push(weight_of(e[i]), x.index(v, i));
      }
    }
    if (x.lone >= 0) {
      const float w = weight_of(x.power(x.x_lone));
      sum += (u64)w;
      if (!all && w >= list_w) push(w, x.lone);
    }
  } else {
    x.each([&](float e, int j) {
      const float w = weight_of(e);
      if (w >= least_w) {
        sum += (u64)w;
        if (!all && w >= list_w) push(w, j);
      }
    });
  }
  sum = warp_sum(sum);
  if (lane == 0) s.seg[warp] = sum;
  __syncthreads();
  auto block_totals = [&]() {                                 // s.seg summed, by warp 0
    if (warp == 0) {
      const u64 t = warp_sum(lane < WARPS ? s.seg[lane] : 0);
      u64 l = 0;
      for (int i = lane; i < min(s.n_list, LIST); i += 32) l += (u64)key_weight(s.list[i]);
      l = warp_sum(l);
      if (lane == 0) {
        s.sum = t;
        s.list_sum = l;
      }
    }
  };
  block_totals();
  sync_row();
  u64 total = 0, list_sum = 0;
  int n_list = 0;
  for (int r = 0; r < C; ++r) {
    total += *at(&s.sum, r);
    list_sum += *at(&s.list_sum, r);
    n_list += *at(&s.n_list, r);
  }
  auto share = [&](u64 t) { return (u64)fmax(ceil((double)top_p * (double)t), 1.0); };

  // ---- the draw among all elements: the block, the warp, the element
  auto draw_row = [&](auto val, u64 drawn_total) {
    const u64 r = (u64)floor((double)u * (double)drawn_total);
    u64 before = 0;
    for (int b = 0; b < rank; ++b) before += *at(&s.sum, b);
    arrive();
    if (before <= r && r < before + s.sum) {
      for (int w = 0; w < warp; ++w) before += s.seg[w];
      if (before <= r && r < before + s.seg[warp]) {
        u64 own;
        const int j = x.find(val, r - before, own);
        if (lane == 0) write(j, own, drawn_total);
      }
    }
    leave();
  };
  if (all) {
    draw_row([&](float e, int) {
      const float w = weight_of(e);
      return w >= least_w ? (u64)w : 0ull;
    }, total);
    return;
  }

  // ---- the prefix ends within the list: one block ranks it
  const bool whole = list_w == least_w;                       // the list is all there is
  if (n_list <= LIST && (whole || (k < V ? k <= n_list : share(total) <= list_sum))) {
    if (rank != 0) {
      arrive();
      leave();
      return;
    }
    int n = s.n_list;
    for (int r = 1; r < C; ++r) {
      const int more = *at(&s.n_list, r);
      for (int i = tid; i < more; i += THREADS) s.list[n + i] = at(s.list, r)[i];
      n += more;
    }
    arrive();
    __syncthreads();
    // the rank and the sum before it of each token; 1, 2, 4 or 8 threads a token
    int per_log2 = 0;
    while (per_log2 < 3 && (n << (per_log2 + 1)) <= THREADS) ++per_log2;
    const int per = 1 << per_log2, i = tid >> per_log2;
    const u64 own = i < n ? s.list[i] : 0;
    int before_n = 0;
    u64 before = 0;
    for (int o = tid & (per - 1); o < n; o += per) {
      const u64 y = s.list[o];
      if (y > own) {
        ++before_n;
        before += (u64)key_weight(y);
      }
    }
    for (int o = 1; o < per; o <<= 1) {
      before_n += __shfl_xor_sync(~0u, before_n, o);
      before += __shfl_xor_sync(~0u, before, o);
    }
    const u64 w = (u64)key_weight(own);
    const bool first = (tid & (per - 1)) == 0 && i < n;
    // top-k's sum, then what top-p leaves of it
    u64 kept_sum = k < V ? (first && before_n < k ? w : 0) : 0;
    if (k < V) kept_sum = block_all(kept_sum, OpSum(), s.scan); else kept_sum = total;
    const u64 least = share(kept_sum);
    const bool keep = i < n && before_n < k && (top_p == 1.f || before < least);
    kept_sum = block_all(first && keep ? w : 0ull, OpSum(), s.scan);
    __syncthreads();
    if (first) s.red_sum[i] = keep ? w : 0;                   // i < LIST <= BINS
    __syncthreads();
    const u64 r = (u64)floor((double)u * (double)kept_sum);
    u64 low = 0;                                              // kept weights of lower IDs
    for (int o = tid & (per - 1); o < n; o += per)
      if ((uint32_t)s.list[o] > (uint32_t)own) low += s.red_sum[o];
    for (int o = 1; o < per; o <<= 1) low += __shfl_xor_sync(~0u, low, o);
    if (first && keep && low <= r && r < low + w) write((int)~(uint32_t)own, w, kept_sum);
    leave();
    return;
  }

  // ---- the prefix's end by histograms of the weights' bits
  uint32_t hist_base = 0;
  int hist_shift = -1;
  auto histogram = [&](uint32_t base, int shift, int bins) {
    hist_base = base;
    hist_shift = shift;
    for (int b = tid; b < bins; b += THREADS) s.n[b] = s.low[b] = s.high[b] = 0;
    __syncthreads();
    x.each([&](float e, int) {
      const float w = weight_of(e);
      const uint32_t key = __float_as_uint(w);
      const uint32_t b = (key - base) >> shift;
      if (w >= least_w && key >= base && b < (uint32_t)bins) {
        const uint32_t low = key & ((1u << shift) - 1);
        atomicAdd(&s.n[b], 1u);
        atomicAdd(&s.low[b], low & 1023u);
        atomicAdd(&s.high[b], low >> 10);
      }
    });
    sync_row();
    // each block adds up its share of the bins over the row
    const int share_bins = (bins + C - 1) >> a.cluster_log2;
    for (int i = tid; i < share_bins; i += THREADS) {
      const int b = rank * share_bins + i;
      if (b < bins) {
        u64 n = 0, low = 0;
        for (int r = 0; r < C; ++r) {
          n += at(s.n, r)[b];
          low += at(s.low, r)[b] + ((u64)at(s.high, r)[b] << 10);
        }
        // weights are mantissa << (exponent - 23); whole, so nothing is lost
        const uint32_t key = base + ((uint32_t)b << shift);
        const int ex = (int)(key >> 23) - 150;
        const u64 mant = n * ((key & 0x7FFFFFu) | 0x800000u) + low;
        s.red_n[b] = (uint32_t)n;
        s.red_sum[b] = ex >= 0 ? mant << ex : mant >> -ex;
      }
    }
    sync_row();
    for (int b = tid; b < bins; b += THREADS) {
      const int r = b / share_bins;
      if (r != rank) {
        s.red_n[b] = at(s.red_n, r)[b];
        s.red_sum[b] = at(s.red_sum, r)[b];
      }
    }
    sync_row();                                               // (and no block runs ahead)
  };
  // the bin, from the heaviest down, where the count (by_n) or the sum reaches `want`
  auto locate = [&](int bins, bool by_n, u64 want, uint32_t before_n, u64 before_sum) {
    constexpr int PER = (BINS + THREADS - 1) / THREADS;
    uint32_t n[PER], own_n = 0;
    u64 w[PER], own_w = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int b = bins - 1 - (tid * PER + i);
      n[i] = b >= 0 ? s.red_n[b] : 0;
      w[i] = b >= 0 ? s.red_sum[b] : 0;
      own_n += n[i];
      own_w += w[i];
    }
    uint32_t pn = own_n;
    u64 pw = own_w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t yn = __shfl_up_sync(~0u, pn, o);
      const u64 yw = __shfl_up_sync(~0u, pw, o);
      if (lane >= o) pn += yn, pw += yw;
    }
    __syncthreads();
    if (lane == 31) s.scan_n[warp] = pn, s.scan[warp] = pw;
    __syncthreads();
    pn += before_n - own_n;
    pw += before_sum - own_w;
    for (int i = 0; i < warp; ++i) pn += s.scan_n[i], pw += s.scan[i];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const bool crosses = by_n ? pn < want && pn + n[i] >= want : pw < want && pw + w[i] >= want;
      if (crosses) {
        s.bin = bins - 1 - (tid * PER + i);
        s.bin_n = n[i];
        s.bin_before = pn;
        s.bin_sum_before = pw;
      }
      pn += n[i];
      pw += w[i];
    }
    __syncthreads();
  };
  // the last token (as a list key) of the shortest prefix with `want` tokens
  // (by_n) or a sum of `want`, and the prefix's sum
  auto prefix_end = [&](bool by_n, u64 want, u64 &end_key, u64 &prefix_sum) {
    uint32_t base = KEY_ONE, before_n = 0;
    int shift = SHIFT, bins = BINS;
    u64 before_sum = 0;
    for (;;) {
      if (hist_base != base || hist_shift != shift) histogram(base, shift, bins);
      locate(bins, by_n, want, before_n, before_sum);
      base += (uint32_t)s.bin << shift;
      before_n = s.bin_before;
      before_sum = s.bin_sum_before;
      const uint32_t n_bin = s.bin_n;
      __syncthreads();
      if (n_bin <= BIN_LIST) {
        // rank the bin's tokens in the first block
        if (tid == 0) s.n_list = 0;
        __syncthreads();
        x.each([&](float e, int j) {
          const float w = weight_of(e);
          const uint32_t key = __float_as_uint(w);
          if (w >= least_w && key >= base && (key - base) >> shift == 0) push(w, j);
        });
        sync_row();
        if (rank == 0) {
          int n = s.n_list;
          for (int r = 1; r < C; ++r) {
            const int more = *at(&s.n_list, r);
            for (int i = tid; i < more; i += THREADS) s.list[n + i] = at(s.list, r)[i];
            n += more;
          }
          __syncthreads();
          const int i = tid >> 1;
          const u64 own = i < n ? s.list[i] : 0;
          u64 rank_n = 0, sum_to = 0;
          for (int o = tid & 1; o < n; o += 2) {
            const u64 y = s.list[o];
            if (y >= own) {
              ++rank_n;
              sum_to += (u64)key_weight(y);
            }
          }
          rank_n += __shfl_xor_sync(~0u, rank_n, 1) + before_n;
          sum_to += __shfl_xor_sync(~0u, sum_to, 1) + before_sum;
          const u64 w = (u64)key_weight(own);
          if ((tid & 1) == 0 && i < n && (by_n ? rank_n == want : sum_to >= want && sum_to - w < want)) {
            s.cut_key = own;
            s.bin_sum_before = sum_to;
          }
        }
        sync_row();
        end_key = *at(&s.cut_key, 0);
        prefix_sum = *at(&s.bin_sum_before, 0);
        sync_row();
        return;
      }
      if (shift == 0) {
        // tokens of one weight: the prefix ends at one of them by its place
        const float one = __uint_as_float(base);
        const u64 w = (u64)one, some = by_n ? want - before_n : (want - before_sum + w - 1) / w;
        u64 c = 0;
        x.each([&](float e, int) { c += weight_of(e) == one; });
        c = warp_sum(c);
        if (lane == 0) s.seg[warp] = c;
        __syncthreads();
        block_totals();
        sync_row();
        u64 before = 0;
        for (int b = 0; b < rank; ++b) before += *at(&s.sum, b);
        if (before < some && some <= before + s.sum) {
          for (int i = 0; i < warp; ++i) before += s.seg[i];
          if (before < some && some <= before + s.seg[warp]) {
            u64 own;
            const int j = x.find([&](float e, int) { return weight_of(e) == one ? 1ull : 0ull; }, some - 1 - before, own);
            if (lane == 0) *at(&s.index, 0) = j;
          }
        }
        sync_row();
        end_key = list_key(one, *at(&s.index, 0));
        prefix_sum = before_sum + some * w;
        sync_row();
        return;
      }
      const int finer = max(0, shift - FINER);
      bins = 1 << (shift - finer);
      shift = finer;
    }
  };
  u64 end_key = 0;                                            // keeps everything
  if (k < V) {
    // fewer than k tokens may be left by min-p
    if (hist_shift != SHIFT) histogram(KEY_ONE, SHIFT, BINS);
    u64 n = 0;
    for (int b = tid; b < BINS; b += THREADS) n += s.red_n[b];
    n = block_all(n, OpSum(), s.scan);
    if (n > (u64)k) prefix_end(true, k, end_key, total);
  }
  const u64 least = share(total);
  if (top_p < 1.f && least < total) prefix_end(false, least, end_key, total);
  // what is kept, by the warps' parts
  auto val = [&](float e, int j) {
    const float w = weight_of(e);
    return w >= least_w && list_key(w, j) >= end_key ? (u64)w : 0ull;
  };
  sum = 0;
  x.each([&](float e, int j) { sum += val(e, j); });
  sum = warp_sum(sum);
  __syncthreads();
  if (lane == 0) s.seg[warp] = sum;
  __syncthreads();
  block_totals();
  sync_row();
  draw_row(val, total);
}

}  // namespace

extern "C" tt_status tt_sample(const void *d_logits, int32_t type, int64_t n_rows, int64_t n_vocab,
                               int64_t logits_stride, const float *d_uniform, const float *d_temperature,
                               const int32_t *d_top_k, const float *d_top_p, const float *d_min_p,
                               int32_t *d_out_ids, float *d_out_logprobs, int32_t *d_status, tt_stream_t stream) {
  if (!type_ok(type) || n_rows < 0 || !vocab_ok(n_vocab) || logits_stride < n_vocab || !optional_ok(d_temperature, 4) ||
      !optional_ok(d_top_k, 4) || !optional_ok(d_top_p, 4) || !optional_ok(d_min_p, 4) ||
      !optional_ok(d_out_logprobs, 4) || !optional_ok(d_status, 4))
    return TT_ERR_INVALID_ARG;
  if (n_rows > TT_MAX_IDS) return TT_ERR_CAPACITY;
  if (n_rows == 0) return TT_OK;
  if (!array_ok(d_logits, type_size(type)) || !array_ok(d_uniform, 4) || !array_ok(d_out_ids, 4)) return TT_ERR_INVALID_ARG;
  SampleArgs a{n_vocab, logits_stride, d_uniform, d_temperature, d_top_k, d_top_p, d_min_p,
               d_out_ids, d_out_logprobs, d_status, 0, 0};
  // blocks a row: up to 16,384 elements each
  while (a.cluster_log2 < 3 && (n_vocab >> a.cluster_log2) > 16384) ++a.cluster_log2;
  with_type(type, [&](auto t) {
    using T = decltype(t);
    const int64_t vecs = (n_vocab * (int64_t)sizeof(T) + 15) / 16;
    a.held = (int)std::min<int64_t>((vecs + (1 << a.cluster_log2) - 1) >> a.cluster_log2, HELD / 16);
    const size_t shared = (size_t)a.held * 16;
    auto k = k_sample<T>;
    if (shared + sizeof(Shared) > 48 * 1024) cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, HELD);
    launch_cluster(k, (unsigned)(n_rows << a.cluster_log2), THREADS, shared, 1u << a.cluster_log2, stream, a, (const T *)d_logits);
  });
  return launched("tt_sample");
}
