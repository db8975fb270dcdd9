// tt_sample.cu - drawing token IDs from rows of logits (include/toktier.h).
//
// Every sum is of whole numbers, so it is exact and any split of a row gives
// the same ID.  A cluster of blocks reads a row once and holds it in shared
// memory (or L2, where it is larger); the passes over it cost instructions.
//
// What top-k and top-p keep is a prefix of the tokens in the order of their
// weights.  Sorting a row for it would cost far more than reading it, and the
// prefix is nearly always short, so a list of the heaviest tokens is made
// first: the row's maxima over 128 groups of threads are known from the first
// pass, and the tokens at or above the q-th largest of them are at least q and
// rarely twice as many.  If the prefix ends within the list (its count, or
// its sum against the row's, says so), one block sorts the list.  For the other
// rows (a top-k above 96, flat rows) a histogram of the weights' bits over the
// cluster, 64 bins an octave, says between which bins the prefix ends, and the
// few tokens there are sorted; bins that hold too many are divided further.
// Where all rows run at once, a kernel does both; of more rows, a second kernel
// does those that the first one left, since the registers, shared memory and
// cluster size of the histograms would slow the lists down by half.
//
// 256 x 100256 bfloat16, whose bytes need 7.6 us, take 31 us with a temperature
// alone (a pass that reads and one that sums, over one or two rows an SM), 37
// with a top-k of 50 and top-p, 147 with a top-k of 1000 and 204 where every row
// is flat (calls back to back, their inputs not in L2).  A mixture, of which a
// quarter goes to the histograms, takes 81: 37 for the lists' kernel and 52 for
// theirs, each alone.  Of a row's time in the latter, parts that were timed are 3 of
// reading, 10 of the first histogram (an atomic in shared memory for each token of
// the row, which twice the warps do not speed up), 4 to find the bins, and 20 for
// the finer ones and the last tokens, passes and cluster barriers in turn.
#include <algorithm>

#include "tt_ops.cuh"

using namespace tt::ops;

namespace {

typedef unsigned long long u64;

constexpr int THREADS = 512;
constexpr int WARPS = THREADS / 32;
constexpr int HELD = 96 * 1024;                   // bytes of a row a block holds, two blocks an SM,
constexpr int HELD_BINS = 160 * 1024;             // and in the second kernel, one an SM
constexpr int PENDING = -2, CLAIMED = -3;         // in the place of an ID that the second kernel writes
constexpr int GROUPS = 128;                       // groups of threads a row's maxima are taken over
constexpr int MOST_LISTED = GROUPS * 3 / 4;       // the largest top-k that a list is made for
constexpr int LIST = THREADS;                     // tokens one block sorts
constexpr int LONG_LIST = 1792;                   // tokens worth a list of their own for the later passes
constexpr int RANGE = 1024;                       // tokens of a range that are ranked and not divided further, by
constexpr int RANGE_FEW = 512;                    // clusters of 4 or 8 blocks, and by fewer
constexpr int SHIFT = 17;                         // first histogram: 64 bins an octave
constexpr int BINS = (40 << (23 - SHIFT)) + 1;    // weights 1 .. 2^40
constexpr int FINER_BINS = 640;                   // of a range
constexpr float ONE = 1099511627776.f;            // 2^40, the largest weight
constexpr uint32_t KEY_ONE = 0x3F800000u;         // the bits of weight 1
constexpr float LARGEST = 3.402823466e38f;
constexpr float NEVER = 2.f;                      // above every power

// the larger, or NaN if there is one
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

struct SampleArgs {
  int64_t n_vocab, stride;
  const float *uniform, *temperature;
  const int32_t *top_k;
  const float *top_p, *min_p;
  int32_t *ids;
  float *logprobs;
  int32_t *status;
  int cluster_log2, held;
  int64_t n_rows;
};

// rint(e * 2^40) of an e in [0, 1]: whole above 2^23, below it rounded by the
// addition.  Its bits (the key) order weights.
__device__ __forceinline__ float weight_of(float e) {
  const float x = e * ONE;
  return x >= 8388608.f ? x : (x + 8388608.f) - 8388608.f;
}
__device__ __forceinline__ uint32_t key_of(float e) { return __float_as_uint(weight_of(e)); }

// The least e whose key is at least `key`: passes over a row compare powers,
// which they have, and not weights, which cost four instructions more.  Below
// 2^23, half a unit under the weight; a tie goes to an even one.
__device__ __forceinline__ float least_power(uint32_t key) {
  const float w = ceilf(__uint_as_float(key));
  if (w > 8388608.f) return w * (1.f / ONE);
  const float half = w - 0.5f;
  return (((int)w & 1) ? __uint_as_float(__float_as_uint(half) + 1) : half) * (1.f / ONE);
}

// A sum of rint(e * 2^40) without a conversion: adding 96 leaves e rounded to
// 2^-17 in the low bits, and adding 1.5 * 2^-17 to what that cut off leaves the
// rest, rounded to 2^-40.  Both counts stay below 2^31 for 256 terms.  Two
// terms at a time; the added constants' bits come off at the end.
struct Sum {
  uint32_t hi = 0, lo = 0;
  __device__ __forceinline__ void add2(float e0, float e1) {
    uint32_t a0, a1, b0, b1;
    asm("{ .reg .b64 e, a, h, b, k; mov.b64 e, {%4, %5}; mov.b64 k, {%6, %6}; add.rn.f32x2 a, e, k;\n\t"
        "mov.b64 k, {%7, %7}; add.rn.f32x2 h, a, k; mov.b64 k, {%8, %8}; fma.rn.f32x2 b, h, k, e;\n\t"
        "mov.b64 k, {%9, %9}; add.rn.f32x2 b, b, k; mov.b64 {%0, %1}, a; mov.b64 {%2, %3}, b; }"
        : "=r"(a0), "=r"(a1), "=r"(b0), "=r"(b1)
        : "f"(e0), "f"(e1), "f"(96.f), "f"(-96.f), "f"(-1.f), "f"(1.5f / 131072.f));
    hi += a0 + a1;
    lo += b0 + b1;
  }
  template <int TERMS> __device__ __forceinline__ u64 value() const {
    return ((u64)(hi - TERMS * 0x42C00000u) << 23) + (u64)(long long)(int)(lo - TERMS * 0x37400000u);
  }
};

// the same of one term
__device__ __forceinline__ u64 whole(float e) {
  Sum t;
  t.add2(e, 0.f);
  return t.value<2>();
}

// A token in a list: its key above its complemented ID, so that larger means
// earlier; or with the halves exchanged, for the order of IDs.
__device__ __forceinline__ u64 list_key(uint32_t key, int j) { return (u64)key << 32 | (uint32_t)~j; }
__device__ __forceinline__ int list_id(u64 k) { return (int)~(uint32_t)k; }
__device__ __forceinline__ u64 key_whole(uint32_t key) { return whole(__uint_as_float(key) * (1.f / ONE)); }
__device__ __forceinline__ u64 list_whole(u64 k) { return key_whole((uint32_t)(k >> 32)); }

__device__ __forceinline__ u64 warp_sum(u64 v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
  return v;
}
// the sum of the lanes before this one
__device__ __forceinline__ u64 sum_of_lanes_before(u64 v) {
  const int lane = threadIdx.x & 31;
  u64 x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const u64 y = __shfl_up_sync(~0u, x, o);
    if (lane >= o) x += y;
  }
  return x - v;
}

// floor or ceil of f * t, exactly, for an f in [0, 1]
__device__ __forceinline__ u64 times(float f, u64 t, bool up) {
  if (f == 1.f) return t;
  const uint32_t b = __float_as_uint(f), e = max(b >> 23, 1u);
  const u64 m = (b & 0x7FFFFFu) | (b >> 23 ? 0x800000u : 0u);
  const int shift = 150 - (int)e;                 // 24 .. 149
  const u64 lo = m * t, hi = __umul64hi(m, t);
  u64 q, cut;
  if (shift < 64) {
    q = hi << (64 - shift) | lo >> shift;
    cut = lo << (64 - shift);
  } else {
    q = shift < 128 ? hi >> (shift - 64) : 0;
    cut = lo | (shift >= 128 ? hi : shift > 64 ? hi << (128 - shift) : 0);
  }
  return q + (up && cut ? 1 : 0);
}

struct Shared {
  float4 all_max[GROUPS / 4];       // maxima over the row's groups
  float nth_max;
  uint32_t lowest;                  // complement of an ID
  int n_kept, n_list;
  u64 seg[WARPS];                   // sums over the warps' parts of the row
  u64 sums[8], list_sums[8];        // of the row's blocks, and of their lists
  int n_lists[8];
  u64 total, least, draw;           // of a sorted list: the kept sum, top-p's share, the draw's place
  u64 scan[WARPS];
  u64 list[LIST];
  u64 sorted[LIST];                 // the blocks' lists
};

struct SharedBins : Shared {
  u64 range[RANGE];                 // the block's tokens of a range
  u64 all_range[RANGE], sorted_range[RANGE];      // the row's
  u64 scan2[WARPS];
  uint32_t scan_n[WARPS];
  int n_long;
  int bin[2];                       // the lowest and the highest bin where a prefix may end
  uint32_t bin_before, bin_to;      // tokens above the highest, and down to the lowest
  u64 cut_key, cut_sum;             // where a prefix ends, and its sum
  uint32_t part_low[WARPS], part_high[WARPS];
  uint32_t red_n[BINS];             // a histogram over the row: counts
  union {
    uint32_t counts[BINS];          // this block's
    struct {
      u64 red_sum[FINER_BINS];      // and sums
      uint32_t n[3 * FINER_BINS];   // this block's: counts and the sums of the mantissas' low and high bits
    };
    u64 long_list[LONG_LIST];       // the block's tokens among which the prefix ends
  };
};

extern __shared__ uint4 s_row[];              // the held part of the block's vectors

// One row, as a thread of a block of its cluster sees it.
template <class T> struct Row {
  static constexpr int E = RowParts<T>::E;
  const uint4 *body;
  int n, slab;                      // the block's vectors, and how many a warp takes
  int held, lo, hi;                 // the warp's
  int first;                        // index of the block's vector 0's first element
  int lone;                         // a single element of this thread's, or -1
  bool lone_first;                  // which comes before the vectors, or behind them
  float x_lone;
  float m, c;
  bool odd, infinite;               // a NaN or +inf among the elements; +inf the largest

  __device__ __forceinline__ uint4 vec(int v) const { return v < held ? s_row[v] : __ldg(body + v); }

  // 2^((l - M) c); 0 for NaN and -inf.  With an infinite M, 1 for +inf alone
  // (M and c are then the largest floats, so that its power is infinite).
  __device__ __forceinline__ float mended(float e) const { return infinite ? (e == INF ? 1.f : 0.f) : e == e ? e : 0.f; }
  __device__ __forceinline__ void powers(const uint4 &r, float e[E]) const {
    vec_f32(r, e, T{});
#pragma unroll
    for (int i = 0; i < E; i += 2) {
      const float2 z = sub_mul2(make_float2(e[i], e[i + 1]), m, c);
      e[i] = ex2(z.x);
      e[i + 1] = ex2(z.y);
    }
    if (odd) {
#pragma unroll
      for (int i = 0; i < E; ++i) e[i] = mended(e[i]);
    }
  }
  __device__ __forceinline__ float power(float l) const { return mended(ex2((l - m) * c)); }
  __device__ __forceinline__ int index(int v, int i) const { return first + v * E + i; }
};

// What a pass does with powers in [from, to).
enum Act { NOTHING, PUSH, PUSH_RANGE, PUSH_LONG, COUNT_BINS, SUM_BINS, LOWEST_ID, COUNT };
// Which weights it adds: all (those below 1 are 0), or from `sum_from` on.
enum Sums { NONE, ALL, FROM };

struct Pass {
  float sum_from;                   // adds the weights of powers from here on
  float from, to;
  uint32_t base;                    // of the bins' keys
  int shift, bins;
};

template <int ACT, class S> __device__ __forceinline__ void act_on(S &s, const Pass &p, float e, int j, u64 &sum) {
  if constexpr (ACT == COUNT_BINS) {
    const uint32_t b = (key_of(e) - p.base) >> p.shift;       // (keys below the base come out above the bins)
    if (e >= p.from && b < (uint32_t)p.bins) atomicAdd(&s.counts[b], 1u);
    return;
  }
  if (!(e >= p.from && e < p.to)) return;
  if constexpr (ACT == PUSH) {
    if (*(volatile int *)&s.n_list > LIST) return;            // too many already
    const int n = atomicAdd(&s.n_list, 1);
    if (n < LIST) s.list[n] = list_key(key_of(e), j);
  } else if constexpr (ACT == PUSH_RANGE) {
    s.range[atomicAdd(&s.n_list, 1)] = list_key(key_of(e), j);
  } else if constexpr (ACT == PUSH_LONG) {
    s.long_list[atomicAdd(&s.n_long, 1)] = list_key(key_of(e), j);
  } else if constexpr (ACT == SUM_BINS) {
    const uint32_t key = key_of(e), b = (key - p.base) >> p.shift, low = key & ((1u << p.shift) - 1);
    atomicAdd(&s.n[b], 1u);
    atomicAdd(&s.n[FINER_BINS + b], low & 1023u);
    atomicAdd(&s.n[2 * FINER_BINS + b], low >> 10);
  } else if constexpr (ACT == LOWEST_ID) {
    sum = max(sum, (u64)(uint32_t)~j);
  } else if constexpr (ACT == COUNT) {
    ++sum;
  }
}

// One pass over the warp's part of the row: this thread's sum (with COUNT a
// count, with LOWEST_ID the complement of the lowest ID).
template <int ACT, int SUM, class T, class S> __device__ __forceinline__ u64 pass(const Row<T> &x, S &s, const Pass p) {
  constexpr int E = Row<T>::E;
  u64 sum = 0;
  int v = x.lo + (threadIdx.x & 31);
  uint4 next = v < x.hi ? x.vec(v) : make_uint4(0, 0, 0, 0);  // (a vector ahead: it may come from L2)
  for (; v < x.hi; v += 32) {
    float e[E];
    const uint4 now = next;
    if (v + 32 < x.hi) next = x.vec(v + 32);
    x.powers(now, e);
    float top = e[0];
    if (ACT != NOTHING || SUM == FROM) {
#pragma unroll
      for (int i = 1; i < E; ++i) top = fmaxf(top, e[i]);
    }
    if constexpr (ACT == COUNT_BINS) {
      float least = e[0];
#pragma unroll
      for (int i = 1; i < E; ++i) least = fminf(least, e[i]);
      if (least == top) {                                     // rows of one value would meet at one counter
        const uint32_t b = (key_of(top) - p.base) >> p.shift;
        if (top >= p.from && b < (uint32_t)p.bins) atomicAdd(&s.counts[b], (uint32_t)E);
        if (SUM != NONE && top >= p.sum_from) sum += E * whole(top);
        continue;
      }
    }
    if (SUM == ALL || (SUM == FROM && top >= p.sum_from)) {
      Sum t;
#pragma unroll
      for (int i = 0; i < E; i += 2) {
        if (SUM == ALL) t.add2(e[i], e[i + 1]);
        else t.add2(e[i] >= p.sum_from ? e[i] : 0.f, e[i + 1] >= p.sum_from ? e[i + 1] : 0.f);
      }
      sum += t.template value<E>();
    }
    if (ACT != NOTHING && top >= p.from) {
#pragma unroll
      for (int i = 0; i < E; ++i) act_on<ACT>(s, p, e[i], x.index(v, i), sum);
    }
  }
  if (x.lone >= 0) {
    const float e = x.power(x.x_lone);
    if (SUM != NONE && e >= p.sum_from) sum += whole(e);
    if (ACT != NOTHING) act_on<ACT>(s, p, e, x.lone, sum);
  }
  return sum;
}

// What is kept: powers from `above` on, and of those from `from` on the ones
// not behind `end` in the list order.  With `count`, each of [from, above) is 1.
struct Keep {
  float from, above;
  u64 end;
  bool count;
  __device__ __forceinline__ u64 value(float e, int j) const {
    if (count) return e >= from && e < above;
    return e >= above || (e >= from && list_key(key_of(e), j) >= end) ? whole(e) : 0;
  }
};

// The first of the warp's elements, by index, at which the running sum of the
// kept values passes r (it does); its value in `own`.
template <class T> __device__ __forceinline__ int find(const Row<T> x, const Keep keep, u64 r, u64 &own) {
  constexpr int E = Row<T>::E;
  const int lane = threadIdx.x & 31;
  const bool any_lone = __any_sync(~0u, x.lone >= 0), at_first = __any_sync(~0u, x.lone >= 0 && x.lone_first);
  u64 before = 0;
  // step -1: single elements ahead of the vectors; the last step: those behind
  const int steps = (x.hi - x.lo + 31) / 32;
  for (int i0 = any_lone && at_first ? -1 : 0; i0 < steps + (any_lone && !at_first ? 1 : 0); ++i0) {
    const bool lones = i0 < 0 || i0 == steps;
    const int v = x.lo + i0 * 32 + lane;
    u64 val[E], mine = 0;
#pragma unroll
    for (int i = 0; i < E; ++i) val[i] = 0;
    if (lones) {
      if (x.lone >= 0) mine = val[0] = keep.value(x.power(x.x_lone), x.lone);
    } else if (v < x.hi) {
      float e[E];
      x.powers(x.vec(v), e);
#pragma unroll
      for (int i = 0; i < E; ++i) mine += val[i] = keep.value(e[i], x.index(v, i));
    }
    // the warp's sum in parts of 22 bits, each in one instruction
    const u64 sum = (u64)__reduce_add_sync(~0u, (uint32_t)mine & 0x3FFFFFu) +
                    ((u64)__reduce_add_sync(~0u, (uint32_t)(mine >> 22)) << 22);
    if (before + sum <= r) {
      before += sum;
      continue;
    }
    // the lane whose elements pass r walks through them
    u64 start = before + sum_of_lanes_before(mine);
    const bool here = start <= r && r < start + mine;
    int at = -1;
    own = 0;
    if (here) {
#pragma unroll
      for (int i = 0; i < E; ++i) {
        start += val[i];
        if (at < 0 && start > r) {
          at = lones ? x.lone : x.index(v, i);
          own = val[i];
        }
      }
    }
    const int lane_of = __ffs(__ballot_sync(~0u, here)) - 1;
    own = __shfl_sync(~0u, own, lane_of);
    return __shfl_sync(~0u, at, lane_of);
  }
  return -1;
}

// The sum over the threads before this one.
__device__ __forceinline__ u64 sum_before(Shared &s, u64 own) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  u64 before = sum_of_lanes_before(own);
  __syncthreads();
  if (lane == 31) s.scan[warp] = before + own;
  __syncthreads();
  for (int w = 0; w < warp; ++w) before += s.scan[w];
  return before;
}

// A falling sort of one value a thread; n of them, all different, are not 0 and
// the first n threads'.  Up to half a block by counting what is above each, with
// 2 to 8 threads a value; else a bitonic sort.
__device__ __noinline__ u64 sort(Shared &s, u64 key, int n) {
  const int tid = threadIdx.x;
  if (n <= THREADS / 2) {
    __syncthreads();
    if (tid < n) s.sorted[tid] = key;
    __syncthreads();
    int log2 = 1;
    while (log2 < 3 && (n << (log2 + 1)) <= THREADS) ++log2;
    const int per = 1 << log2, i = tid >> log2;
    const u64 own = i < n ? s.sorted[i] : 0;
    int above = 0;
    for (int o = tid & (per - 1); o < n; o += per) above += s.sorted[o] > own;
    for (int o = 1; o < per; o <<= 1) above += __shfl_xor_sync(~0u, above, o);
    __syncthreads();
    if (i < n && (tid & (per - 1)) == 0) s.sorted[above] = own;
    __syncthreads();
    return tid < n ? s.sorted[tid] : 0;
  }
  for (int size = 2; size < 2 * n; size <<= 1)
    for (int step = size >> 1; step; step >>= 1) {
      u64 other;
      if (step >= 32) {
        __syncthreads();
        s.sorted[tid] = key;
        __syncthreads();
        other = s.sorted[tid ^ step];
      } else {
        other = __shfl_xor_sync(~0u, key, step);
      }
      const bool larger = ((tid & step) == 0) == ((tid & size) == 0);
      key = (key > other) == larger ? key : other;
    }
  return key;
}

// Where a prefix of `want` tokens, or with a sum of `want`, ends in the
// histogram over the row, from the heaviest bin down.
//   BY_COUNT  the bin where the count reaches it
//   BY_SUM    the bin where the sum does
//   BETWEEN   the bins between which the sum does, from counts alone: a bin's
//             sum is its count times weights it bounds, added from above, or
//             from below and taken from the row's sum
enum Locate { BY_COUNT, BY_SUM, BETWEEN };
template <Locate L> struct How { static constexpr Locate value = L; };

template <Locate HOW, int PER>                    // PER bins a thread
__device__ __noinline__ void locate(SharedBins &s, int bins, u64 want, uint32_t before_n, u64 above, u64 row_sum) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int b0 = bins - 1 - tid * PER;                        // this thread's first, falling
  // a bin's sum is at least and at most ...: it holds whole weights, from its
  // base on and below the next one's
  auto base_of = [&](int b) {
    const uint32_t key = KEY_ONE + ((uint32_t)b << SHIFT);
    const int ex = (int)(key >> 23) - 150;
    const u64 mant = (key & 0x7FFFFFu) | 0x800000u;
    return ex >= 0 ? mant << ex : mant >> -ex;
  };
  uint32_t n[PER], mine = 0;
  u64 least[PER], most[PER], low = 0, high = 0;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int b = b0 - i;
    n[i] = b >= 0 ? s.red_n[b] : 0;
    if (HOW == BY_COUNT) {
      least[i] = n[i];
    } else if (HOW == BY_SUM) {
      least[i] = b >= 0 ? s.red_sum[b] : 0;
    } else {
      least[i] = n[i] * base_of(b);
      most[i] = b == BINS - 1 ? least[i] : n[i] * base_of(b + 1);
    }
    if (HOW != BETWEEN) most[i] = least[i];
    mine += n[i];
    low += least[i];
    high += most[i];
  }
  uint32_t pn = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(~0u, pn, o);
    if (lane >= o) pn += y;
  }
  u64 pl = sum_of_lanes_before(low), ph = HOW == BETWEEN ? sum_of_lanes_before(high) : pl;
  __syncthreads();
  if (lane == 31) {
    s.scan_n[warp] = pn;
    s.scan[warp] = pl + low;
    s.scan2[warp] = ph + high;
  }
  __syncthreads();
  pn = before_n + pn - mine;
  u64 all_l = 0, all_h = 0;
#pragma unroll
  for (int w = 0; w < WARPS; ++w) {
    if (w < warp) pn += s.scan_n[w], pl += s.scan[w], ph += s.scan2[w];
    if (HOW == BETWEEN) all_l += s.scan[w], all_h += s.scan2[w];
  }
  if (HOW == BY_COUNT) pl = ph = pn;
  if (HOW == BY_SUM) pl += above, ph += above;
  const long long t = (long long)want;
  // a sum is at least what is known from above, or the row's less what may be below; at most ...
  auto at_least = [&](u64 l, u64 h) { return HOW == BETWEEN ? max((long long)l, (long long)(row_sum + h - all_h)) : (long long)l; };
  auto at_most = [&](u64 l, u64 h) { return HOW == BETWEEN ? min((long long)h, (long long)(row_sum + l - all_l)) : (long long)h; };
  // it ends in one thread's bins
  if ((at_most(pl, ph) < t && at_most(pl + low, ph + high) >= t) || (at_least(pl, ph) < t && at_least(pl + low, ph + high) >= t)) {
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const u64 l = least[i], h = most[i];
      if (at_most(pl, ph) < t && at_most(pl + l, ph + h) >= t) {
        s.bin[1] = b0 - i;
        s.bin_before = pn;
      }
      if (at_least(pl, ph) < t && at_least(pl + l, ph + h) >= t) {
        s.bin[0] = b0 - i;
        s.bin_to = pn + n[i];
      }
      pn += n[i];
      pl += l;
      ph += h;
    }
  }
  __syncthreads();
}

// A block of a row's cluster: what both kernels do first, and how blocks tell
// each other sums.
template <class T, class S> struct Block {
  S &s;
  const SampleArgs &a;
  const int tid, lane, warp, C, rank;
  Row<T> x;
  float u, temp, top_p, min_p;
  int k;                            // 1 .. V
  uint32_t least_key;               // min-p; and weight 0 is never drawn
  float least_e, row_max;
  u64 before_block;

  __device__ __forceinline__ Block(S &s, const SampleArgs &a)
      : s(s), a(a), tid(threadIdx.x), lane(threadIdx.x & 31), warp(threadIdx.x >> 5), C(1 << a.cluster_log2),
        rank(a.cluster_log2 ? (int)cluster_rank() : 0) {}
  __device__ __forceinline__ void arrive() const { if (C > 1) cluster_arrive(); }
  __device__ __forceinline__ void leave() const { if (C > 1) cluster_wait(); }
  __device__ __forceinline__ void sync_row() const {
    if (C > 1) cluster_sync(); else __syncthreads();
  }
  template <class P> __device__ __forceinline__ P *at(P *p, int r) const { return C > 1 ? of_block(p, r) : p; }

  // the row's parameters; whether they are what the header allows
  // (adding 0 takes a zero's sign off and changes nothing else: a negative one
  // would turn 1 / T around, and times() reads a factor's bits)
  __device__ __forceinline__ bool parameters(int64_t row) {
    u = a.uniform[row] + 0.f;
    temp = a.temperature ? a.temperature[row] + 0.f : 1.f;
    top_p = a.top_p ? a.top_p[row] + 0.f : 1.f;
    min_p = a.min_p ? a.min_p[row] + 0.f : 0.f;
    const int V = (int)a.n_vocab, top_k = a.top_k ? a.top_k[row] : 0;
    k = temp == 0 ? 1 : top_k > 0 ? min(top_k, V) : V;
    least_key = __float_as_uint(fmaxf(min_p * ONE, 1.f));
    least_e = least_power(least_key);
    return u >= 0 && u < 1 && temp >= 0 && temp < INF && top_p >= 0 && top_p <= 1 && min_p >= 0 && min_p <= 1;
  }

  // The row into shared memory, and its maxima over groups of threads.  A warp
  // takes consecutive vectors, so that warps and blocks lie in the order of the
  // IDs.  What blocks tell each other is written to all of them ahead of a
  // barrier, so that nothing has to be fetched behind it.  Between begun() and
  // sync_row(): the blocks have begun, and the last row's words are read.
  template <class B> __device__ __forceinline__ void load(const T *__restrict__ logits, int64_t row, B begun) {
    constexpr int E = RowParts<T>::E, U = 4;
    const int V = (int)a.n_vocab;
    const T *l = logits + row * a.stride;
    const RowParts<T> part(l, V);
    const int each = (part.vecs + C - 1) >> a.cluster_log2, first = min(part.vecs, rank * each);
    x.n = min(part.vecs - first, each);
    x.slab = (x.n + WARPS - 1) / WARPS;
    x.body = reinterpret_cast<const uint4 *>(l + part.lead) + first;
    x.held = a.held;
    x.first = part.lead + first * E;
    x.lo = min(x.n, warp * x.slab);
    x.hi = min(x.n, x.lo + x.slab);
    x.lone_first = rank == 0 && warp == 0 && lane < part.lead;
    x.lone = x.lone_first ? lane : rank == C - 1 && warp == WARPS - 1 && lane < part.rest ? V - part.rest + lane : -1;
    x.x_lone = x.lone >= 0 ? to_f32(l[x.lone]) : -INF;
    float m = fmaxf(x.x_lone, -INF);
    bool nan = x.x_lone != x.x_lone;
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
          float top = v[0];
#pragma unroll
          for (int j = 1; j < E; ++j) top = max_nan(top, v[j]);
          if (top != top) {                       // a NaN: the others' maximum
            nan = true;
#pragma unroll
            for (int j = 0; j < E; ++j) m = fmaxf(m, v[j]);
          } else {
            m = fmaxf(m, top);
          }
        }
    }
    const int group_lanes = 4 * C;
    for (int o = 1; o < group_lanes; o <<= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, o));
    begun();
    const float y = __shfl_sync(~0u, m, lane < 8 ? (lane >> a.cluster_log2) * group_lanes : 0);
    if (lane < 8)
      reinterpret_cast<float *>(at(s.all_max, lane & (C - 1)))[((rank * WARPS + warp) << (3 - a.cluster_log2)) +
                                                               (lane >> a.cluster_log2)] = y;
    if (tid == 0) {
      s.n_list = 0;
      s.lowest = 0;
    }
    if (C < 8 && tid >= C && tid < 8) s.sums[tid] = s.list_sums[tid] = s.n_lists[tid] = 0;
    sync_row();
    static_assert(GROUPS == 128, "a float4 a lane");
    const float4 four = s.all_max[lane];
    m = warp_all(fmaxf(fmaxf(four.x, four.y), fmaxf(four.z, four.w)), OpMax());
    row_max = m;
    x.infinite = m == INF;
    x.odd = nan || x.infinite;
    x.m = fminf(m, LARGEST);
    x.c = x.infinite ? LARGEST : fminf(1.44269504f / temp, LARGEST);
  }

  __device__ __forceinline__ u64 share(u64 t) const { return max(times(top_p, t, true), 1ull); }
  __device__ __forceinline__ u64 place(u64 t) const { return times(u, t, false); }
  __device__ __forceinline__ void write(int64_t row, int id, u64 w, u64 total) const {
    a.ids[row] = id;
    if (a.logprobs) {
      // the smaller of the share and its complement, whole until then
      const u64 rest = total - w;
      a.logprobs[row] = rest < w ? log1pf(-__fdiv_rn((float)rest, (float)total)) : logf(__fdiv_rn((float)w, (float)total));
    }
  }
  __device__ __forceinline__ void none(int64_t row, int id) const {       // for the second kernel, or nothing to draw
    if (rank == 0 && tid == 0) {
      a.ids[row] = id;
      if (a.logprobs) a.logprobs[row] = -INF;
    }
  }
  __device__ __forceinline__ void block_totals() const {      // s.seg summed, for all blocks; by warp 0
    if (warp == 0) {
      const u64 t = warp_sum(lane < WARPS ? s.seg[lane] : 0);
      if (lane < C) at(s.sums, lane)[rank] = t;
    }
  }
  __device__ __forceinline__ void push_sums(u64 t) const {    // a sum over the row, known behind the next barrier
    t = warp_sum(t);
    if (lane == 0) s.seg[warp] = t;
    __syncthreads();
    block_totals();
  }
  // the row's sum, in every thread, and that of the blocks before this one
  __device__ __forceinline__ u64 row_total() {
    u64 t = before_block = 0;
#pragma unroll
    for (int r = 0; r < 8; ++r) {
      const u64 y = s.sums[r];
      t += y;
      before_block += r < rank ? y : 0;
    }
    return t;
  }
  // token i of the blocks' lists one behind another; 0 behind the last
  __device__ __forceinline__ u64 listed(u64 *list, int i) const {
    int r = 0;
#pragma unroll
    for (int k = 0; k < 7; ++k)
      if (r == k && r < C - 1 && i >= s.n_lists[k]) i -= s.n_lists[k], r = k + 1;
    return i < s.n_lists[r] ? at(list, r)[i] : 0;
  }
  __device__ __forceinline__ int all_listed() const {
    int n = 0;
#pragma unroll
    for (int r = 0; r < 8; ++r) n += r < C ? s.n_lists[r] : 0;
    return n;
  }
  // The draw among what is kept, whose sums by the warps' parts are in s.seg:
  // that warp's vectors are divided among all warps, then a warp finds the
  // element.  Called by the block that holds the drawn place r of the block.
  __device__ __forceinline__ void draw(int64_t row, const Keep &keep, u64 r, u64 total) {
    constexpr int E = RowParts<T>::E;
    int part = 0;
    while (r >= s.seg[part]) r -= s.seg[part++];
    Row<T> y = x;
    const int lo = min(x.n, part * x.slab), hi = min(x.n, lo + x.slab), each = (hi - lo + WARPS - 1) / WARPS;
    y.lo = min(hi, lo + warp * each);
    y.hi = min(hi, y.lo + each);
    if (part != (x.lone_first ? 0 : WARPS - 1)) y.lone = -1;  // single elements stay with the first and the last
    u64 sum = 0;
    for (int v = y.lo + lane; v < y.hi; v += 32) {
      float e[E];
      y.powers(y.vec(v), e);
#pragma unroll
      for (int i = 0; i < E; ++i) sum += keep.value(e[i], y.index(v, i));
    }
    if (y.lone >= 0) sum += keep.value(y.power(y.x_lone), y.lone);
    sum = warp_sum(sum);
    __syncthreads();
    if (lane == 0) s.seg[warp] = sum;
    __syncthreads();
    u64 before = 0;
    for (int w = 0; w < warp; ++w) before += s.seg[w];
    if (before <= r && r < before + sum) {
      u64 own;
      const int j = find(y, keep, r - before, own);
      if (lane == 0) write(row, j, own, total);
    }
  }
};

// One row by its heaviest tokens: whether that did.  Where it did not, all
// blocks return together.
template <class T, class S> __device__ __forceinline__ bool sample_by_list(Block<T, S> &b, const SampleArgs &a, int64_t row) {
  S &s = b.s;
  const int tid = b.tid, lane = b.lane, warp = b.warp, C = b.C, rank = b.rank, V = (int)a.n_vocab, k = b.k;
  const float top_p = b.top_p;

  // ---- the lowest ID of the largest weight
  if (k == 1) {
    const u64 mine = pass<LOWEST_ID, NONE>(b.x, s, Pass{NEVER, least_power(__float_as_uint(ONE)), NEVER, 0, 0, 0});
    const uint32_t warps = __reduce_max_sync(~0u, (uint32_t)mine);
    if (lane == 0) atomicMax(&s.lowest, warps);
    __syncthreads();
    if (tid == 0) b.at(s.n_lists, 0)[rank] = (int)s.lowest;
    b.sync_row();
    if (rank == 0 && warp == 0) {
      const uint32_t rows = __reduce_max_sync(~0u, lane < C ? (uint32_t)s.n_lists[lane] : 0u);
      if (lane == 0) b.write(row, (int)~rows, 1, 1);
    }
    return true;
  }

  // ---- the row's sum, and the list of its heaviest tokens
  const bool all = k == V && top_p == 1.f;                    // nothing but min-p cuts
  uint32_t list_from = b.least_key;                           // the list holds all keys from here on
  if (!all) {
    const int q = min(k, MOST_LISTED);
    // four threads count what is above a group's maximum, and what equals it
    const float own = reinterpret_cast<const float *>(s.all_max)[tid >> 2];
    int above = 0, from = 0;
#pragma unroll
    for (int i = 0; i < GROUPS / 16; ++i) {
      const float4 y = s.all_max[i * 4 + (tid & 3)];
      above += (y.x > own) + (y.y > own) + (y.z > own) + (y.w > own);
      from += (y.x >= own) + (y.y >= own) + (y.z >= own) + (y.w >= own);
    }
    above += __shfl_xor_sync(~0u, above, 1);
    above += __shfl_xor_sync(~0u, above, 2);
    from += __shfl_xor_sync(~0u, from, 1);
    from += __shfl_xor_sync(~0u, from, 2);
    if (above < q && q <= from) s.nth_max = own;              // the same value whoever writes it
    __syncthreads();
    list_from = max(list_from, key_of(b.x.power(s.nth_max)));
  }
  const Pass p{b.least_e, all ? NEVER : least_power(list_from), INF, 0, 0, 0};
  b.push_sums(b.least_key == KEY_ONE ? pass<PUSH, ALL>(b.x, s, p) : pass<PUSH, FROM>(b.x, s, p));
  if (warp == 1 && !all) {
    u64 l = 0;
    const int n = s.n_list;
    for (int i = lane; i < min(n, LIST); i += 32) l += list_whole(s.list[i]);
    l = warp_sum(l);
    if (lane < C) {
      b.at(s.list_sums, lane)[rank] = l;
      b.at(s.n_lists, lane)[rank] = n;
    }
  }
  b.sync_row();
  const u64 total = b.row_total();
  if (all) {
    const u64 r = b.place(total) - b.before_block;
    if (r < s.sums[rank]) b.draw(row, Keep{b.least_e, b.least_e, 0, false}, r, total);
    return true;
  }
  u64 list_sum = 0;
  int n_list = 0;
#pragma unroll
  for (int r = 0; r < 8; ++r) {
    list_sum += s.list_sums[r];
    n_list += s.n_lists[r];
  }

  // ---- if the prefix ends within the list, one block sorts it
  const bool all_listed = list_from == b.least_key;           // the list is all there is
  if (n_list > LIST || !(all_listed || (k < V ? k <= n_list : b.share(total) <= list_sum))) return false;
  if (rank != 0) {
    b.arrive();
    b.leave();
    return true;
  }
  const int n = n_list;
  u64 key = b.listed(s.list, tid);
  b.arrive();
  const int kept_n = min(k, n);
  key = sort(s, key, n);
  u64 w = list_whole(key), before = sum_before(s, w);
  if (k < V) {                                                // top-k's sum, then what top-p leaves of it
    if (tid == kept_n - 1) s.least = top_p < 1.f ? b.share(before + w) : before + w;
    __syncthreads();
  }
  const u64 least = top_p < 1.f ? (k < V ? s.least : b.share(total)) : ~0ull;
  const bool keep = tid < kept_n && before < least;
  if (keep && (tid == kept_n - 1 || before + w >= least)) {
    s.n_kept = tid + 1;
    s.total = before + w;
    s.draw = b.place(before + w);
  }
  __syncthreads();
  key = sort(s, keep ? key << 32 | key >> 32 : 0, s.n_kept);  // by ID
  w = key_whole((uint32_t)key);
  before = sum_before(s, w);
  if (before <= s.draw && s.draw < before + w) b.write(row, (int)~(uint32_t)(key >> 32), w, s.total);
  b.leave();
  return true;
}

template <class T>
__global__ void __launch_bounds__(THREADS, 2) k_sample(const SampleArgs a, const T *__restrict__ logits) {
  __shared__ Shared s;
  Block<T, Shared> b(s, a);
  const int64_t row = blockIdx.x >> a.cluster_log2;
  let_next_start();
  b.arrive();
  const bool valid = b.parameters(row);
  if (valid && b.k < (int)a.n_vocab && b.k > MOST_LISTED) {   // more than a list holds
    b.none(row, PENDING);
    b.leave();
    return;
  }
  b.load(logits, row, [&]() { b.leave(); });
  if (!valid || b.row_max == -INF) {
    b.none(row, -1);
    if (!valid && b.rank == 0 && b.tid == 0) op_status(a.status, TT_ERR_INVALID_ARG);
    return;
  }
  if (!sample_by_list(b, a, row)) b.none(row, PENDING);
}

// One row that the list could not do: all blocks of the cluster.
template <class T>
__device__ __forceinline__ void sample_by_bins(Block<T, SharedBins> &b, const SampleArgs &a, int64_t row) {
  constexpr int E = RowParts<T>::E;
  SharedBins &s = b.s;
  const int tid = b.tid, lane = b.lane, warp = b.warp, C = b.C, rank = b.rank, V = (int)a.n_vocab, k = b.k;
  const float top_p = b.top_p;
  u64 end_key = 0, total = 0;                                 // keeps everything
  bool listed = false;                                        // s.long_list holds what may be kept
  bool parts_known = false;                                   // s.seg has the sums of what lies above s.range
  // ---- the prefix's end by histograms of the weights' bits
  int hist = 0;                                             // 1: s.red_n holds the first histogram
  auto add_bins = [&](int bins, bool sums, uint32_t base, int shift) {
    // each block adds up its share of the bins over the row
    const int share_bins = (bins + C - 1) >> a.cluster_log2;
    for (int i = rank * share_bins + tid; i < min(bins, (rank + 1) * share_bins); i += THREADS) {
      u64 n = 0, low = 0;
#pragma unroll
      for (int r = 0; r < 8; ++r)
        if (r < C) {
          n += sums ? b.at(s.n, r)[i] : b.at(s.counts, r)[i];
          if (sums) low += b.at(s.n, r)[FINER_BINS + i] + ((u64)b.at(s.n, r)[2 * FINER_BINS + i] << 10);
        }
      // weights are mantissa << (exponent - 23); whole, so nothing is lost
      const uint32_t key = base + ((uint32_t)i << shift);
      const int ex = (int)(key >> 23) - 150;
      const u64 mant = n * ((key & 0x7FFFFFu) | 0x800000u) + low, w = ex >= 0 ? mant << ex : mant >> -ex;
      for (int r = 0; r < C; ++r) {
        b.at(s.red_n, r)[i] = (uint32_t)n;
        if (sums) b.at(s.red_sum, r)[i] = w;
      }
    }
    b.sync_row();
  };
  // (with `sum`, the row's sum: read between the two barriers, since a block that
  // is ahead tells new ones behind the second)
  auto count_bins = [&](uint32_t base, int shift, int bins, bool sum) {
    for (int i = tid; i < bins; i += THREADS) s.counts[i] = 0;
    __syncthreads();
    if (sum) b.push_sums(pass<COUNT_BINS, FROM>(b.x, s, Pass{b.least_e, b.least_e, INF, base, shift, bins}));
    else pass<COUNT_BINS, NONE>(b.x, s, Pass{NEVER, b.least_e, INF, base, shift, bins});
    b.sync_row();
    const u64 all = sum ? b.row_total() : 0;
    add_bins(bins, false, base, shift);
    return all;
  };
  constexpr int PER = (BINS + THREADS - 1) / THREADS, PER_FINER = (FINER_BINS + THREADS - 1) / THREADS;
  auto first_bins = [&](auto how, u64 want, u64 row_sum) {
    if (!hist) count_bins(KEY_ONE, SHIFT, BINS, false);
    hist = 1;
    locate<decltype(how)::value, PER>(s, BINS, want, 0, 0, row_sum);
  };
  // a list of its own for what the prefix ends in, where that is short
  auto list_if_few = [&]() {
    if (s.bin_to > LONG_LIST) return;
    const uint32_t from = max(b.least_key, KEY_ONE + ((uint32_t)s.bin[0] << SHIFT));
    if (tid == 0) s.n_long = 0;
    __syncthreads();
    pass<PUSH_LONG, NONE>(b.x, s, Pass{NEVER, least_power(from), INF, 0, 0, 0});
    __syncthreads();
    listed = true;
  };
  // The last token (as a list key) of the shortest prefix with `want` tokens
  // (by_n) or a sum of `want`, and the prefix's sum; behind first_bins.
  auto prefix_end = [&](bool by_n, u64 want) {
    parts_known = false;
    uint32_t base = KEY_ONE + ((uint32_t)s.bin[0] << SHIFT), end = KEY_ONE + ((uint32_t)(s.bin[1] + 1) << SHIFT);
    uint32_t before_n = s.bin_before, n_range = s.bin_to - s.bin_before;
    for (;;) {
      const float from_e = fmaxf(b.least_e, least_power(base)), above_e = fmaxf(b.least_e, least_power(end));
      __syncthreads();
      if (n_range <= (C >= 4 ? RANGE : RANGE_FEW)) {
        // The tokens that are left, in every block; each finds the places of its
        // share, by as many threads as there are, for all of them.
        if (tid == 0) s.n_list = 0;
        __syncthreads();
        u64 above = 0;
        if (listed) {
          for (int i = tid; i < s.n_long; i += THREADS) {
            const u64 key = s.long_list[i];
            const float e = __uint_as_float((uint32_t)(key >> 32)) * (1.f / ONE);
            if (e >= above_e) above += whole(e);
            else if (e >= from_e) s.range[atomicAdd(&s.n_list, 1)] = key;
          }
        } else {
          above = pass<PUSH_RANGE, FROM>(b.x, s, Pass{above_e, from_e, above_e, 0, 0, 0});
        }
        b.push_sums(above);
        if (tid < C) b.at(s.n_lists, tid)[rank] = s.n_list;
        b.sync_row();
        const u64 sum_above = b.row_total();
        const int n = b.all_listed();
        for (int i = tid; i < n; i += THREADS) s.all_range[i] = b.listed(s.range, i);
        __syncthreads();
        const int each = (n + C - 1) >> a.cluster_log2;
        int log2 = 0;
        while (log2 < 5 && (each << (log2 + 1)) <= THREADS) ++log2;
        const int per = 1 << log2;
        for (int i0 = 0; i0 < each; i0 += THREADS >> log2) {
          const int i = rank * each + i0 + (tid >> log2);
          const bool there = i0 + (tid >> log2) < each && i < n;
          const u64 own = there ? s.all_range[i] : 0;
          int above = 0;
#pragma unroll 4
          for (int o = tid & (per - 1); o < n; o += per) above += s.all_range[o] > own;
          for (int o = 1; o < per; o <<= 1) above += __shfl_xor_sync(~0u, above, o);
          if (there && (tid & (per - 1)) == 0)
            for (int r = 0; r < C; ++r) b.at(s.sorted_range, r)[above] = own;
        }
        b.sync_row();
        static_assert(RANGE == 2 * THREADS, "two tokens a thread");
        u64 key[2], w[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          key[i] = 2 * tid + i < n ? s.sorted_range[2 * tid + i] : 0;
          w[i] = list_whole(key[i]);
        }
        u64 sum_to = sum_above + sum_before(s, w[0] + w[1]);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          sum_to += w[i];
          if (2 * tid + i < n && (by_n ? before_n + 2 * tid + i + 1 == want : sum_to >= want && sum_to - w[i] < want)) {
            s.cut_key = key[i];
            s.cut_sum = sum_to;
          }
        }
        __syncthreads();
        end_key = s.cut_key;
        total = s.cut_sum;
        parts_known = true;
        return;
      }
      if (end - base == 1) {
        // tokens of one weight: the prefix ends at one of them by its place
        const u64 w = key_whole(base);
        b.push_sums(pass<NOTHING, FROM>(b.x, s, Pass{above_e, NEVER, NEVER, 0, 0, 0}));
        b.sync_row();
        const u64 above = b.row_total(), some = by_n ? want - before_n : (want - above + w - 1) / w;
        total = above + some * w;
        b.sync_row();                                         // (the sums are read)
        b.push_sums(pass<COUNT, NONE>(b.x, s, Pass{NEVER, from_e, above_e, 0, 0, 0}));
        b.sync_row();
        b.row_total();
        u64 before = b.before_block;
        if (before < some && some <= before + s.sums[rank]) {
          for (int i = 0; i < warp; ++i) before += s.seg[i];
          if (before < some && some <= before + s.seg[warp]) {
            u64 own;
            const int j = find(b.x, Keep{from_e, above_e, 0, true}, some - 1 - before, own);
            if (lane < C) *b.at(&s.cut_key, lane) = list_key(base, j);
          }
        }
        b.sync_row();
        end_key = s.cut_key;
        return;
      }
      // finer bins of what is left, as many as fit; none spans an octave
      listed = false;                                       // (they lie over the list)
      hist = 0;
      int shift = 0;
      while ((end - (base >> shift << shift) + (1u << shift) - 1) >> shift > FINER_BINS) ++shift;
      base = base >> shift << shift;
      const int bins = (int)((end - base + (1u << shift) - 1) >> shift);
      if (by_n) {
        count_bins(base, shift, bins, false);
        locate<BY_COUNT, PER_FINER>(s, bins, want, before_n, 0, 0);
        before_n = s.bin_before;
      } else {
        for (int i = tid; i < 3 * FINER_BINS; i += THREADS) s.n[i] = 0;
        __syncthreads();
        const float bins_e = fmaxf(b.least_e, least_power(base + ((uint32_t)bins << shift)));
        b.push_sums(pass<SUM_BINS, FROM>(b.x, s, Pass{bins_e, fmaxf(b.least_e, least_power(base)), bins_e, base, shift, bins}));
        b.sync_row();
        const u64 above = b.row_total();                    // (before the barrier in add_bins, as in count_bins)
        add_bins(bins, true, base, shift);
        locate<BY_SUM, PER_FINER>(s, bins, want, 0, above, 0);
      }
      n_range = s.red_n[s.bin[0]];
      base += (uint32_t)s.bin[0] << shift;
      end = base + (1u << shift);
    }
  };
  // the first histogram, and the row's sum where it is wanted
  const u64 row_sum = total = count_bins(KEY_ONE, SHIFT, BINS, top_p < 1.f);
  hist = 1;
  if (k < V) {
    // fewer than k tokens may be left by min-p
    uint32_t n = 0;
    for (int i = tid; i < BINS; i += THREADS) n += s.red_n[i];
    n = block_all(n, OpSum(), s.scan_n);
    if (n > (uint32_t)k) {
      first_bins(How<BY_COUNT>{}, k, 0);
      list_if_few();
      prefix_end(true, k);
    }
  }
  if (top_p < 1.f) {
    const u64 least = b.share(total);
    if (least < total) {
      first_bins(How<BETWEEN>{}, least, row_sum);
      if (end_key == 0) list_if_few();
      prefix_end(false, least);
    }
  }

  // ---- the draw: what is kept by the warps' parts of the row, then the
  // block, the part and the element that holds the drawn place
  const uint32_t end_w = max(b.least_key, (uint32_t)(end_key >> 32));
  const Keep keep{least_power(end_w), least_power(end_w + 1), end_key, false};
  auto part_of = [&](u64 key) {
    const int j = list_id(key), v = (j - b.x.first) / E;
    return j < b.x.first ? 0 : v >= b.x.n ? WARPS - 1 : v / b.x.slab;
  };
  {
    if (listed) {
      if (tid < WARPS) s.part_low[tid] = s.part_high[tid] = 0;
      __syncthreads();
      for (int i = tid; i < s.n_long; i += THREADS) {
        const u64 key = s.long_list[i];
        if (key >= end_key) {                                 // 2^21 * LONG_LIST is below 2^32
          const u64 w = list_whole(key);
          const int part = part_of(key);
          atomicAdd(&s.part_low[part], (uint32_t)w & 0x1FFFFFu);
          atomicAdd(&s.part_high[part], (uint32_t)(w >> 21));
        }
      }
      __syncthreads();
      if (tid < WARPS) s.seg[tid] = s.part_low[tid] + ((u64)s.part_high[tid] << 21);
      __syncthreads();
      b.block_totals();
    } else if (parts_known) {
      // the sums of what lies above the sorted tokens, and those
      for (int i = tid; i < s.n_list; i += THREADS) {
        const u64 key = s.range[i];
        if (key >= end_key) atomicAdd(&s.seg[part_of(key)], list_whole(key));
      }
      __syncthreads();
      b.block_totals();
    } else {
      u64 sum = pass<NOTHING, FROM>(b.x, s, Pass{keep.above, NEVER, NEVER, 0, 0, 0});
      // those of the last weight, in the list's order
      if (keep.from < keep.above) {
        for (int v = b.x.lo + lane; v < b.x.hi; v += 32) {
          float e[E];
          b.x.powers(b.x.vec(v), e);
#pragma unroll
          for (int i = 0; i < E; ++i)
            if (e[i] < keep.above) sum += keep.value(e[i], b.x.index(v, i));
        }
        if (b.x.lone >= 0 && b.x.power(b.x.x_lone) < keep.above) sum += keep.value(b.x.power(b.x.x_lone), b.x.lone);
      }
      b.push_sums(sum);
    }
    b.sync_row();
    total = b.row_total();
  }
  const u64 r = b.place(total) - b.before_block;
  if (r >= s.sums[rank]) return;
  if (listed) {
    int part = 0;
    u64 at_r = r;
    while (at_r >= s.seg[part]) at_r -= s.seg[part++];
    if (tid == 0) s.n_list = 0;
    __syncthreads();
    for (int i = tid; i < s.n_long; i += THREADS) {
      const u64 key = s.long_list[i];
      if (key >= end_key && part_of(key) == part) {
        const int n = atomicAdd(&s.n_list, 1);
        if (n < LIST) s.list[n] = key << 32 | key >> 32;
      }
    }
    __syncthreads();
    const int n = s.n_list;
    if (n <= LIST) {
      const u64 key = sort(s, tid < n ? s.list[tid] : 0, n), w = key_whole((uint32_t)key);
      const u64 before = sum_before(s, w);
      if (before <= at_r && at_r < before + w) b.write(row, (int)~(uint32_t)(key >> 32), w, total);
      return;
    }
  }
  b.draw(row, keep, r, total);
}

// Rows that run at once: both in one launch, a cluster a row.
template <class T>
__global__ void __launch_bounds__(THREADS, 1) k_sample_few(const SampleArgs a, const T *__restrict__ logits) {
  __shared__ SharedBins s;
  Block<T, SharedBins> b(s, a);
  const int64_t row = blockIdx.x >> a.cluster_log2;
  b.arrive();
  const bool valid = b.parameters(row);
  b.load(logits, row, [&]() { b.leave(); });
  if (!valid || b.row_max == -INF) {
    b.none(row, -1);
    if (!valid && b.rank == 0 && b.tid == 0) op_status(a.status, TT_ERR_INVALID_ARG);
    return;
  }
  if (!(b.k < (int)a.n_vocab && b.k > MOST_LISTED)) {
    if (sample_by_list(b, a, row)) return;
    b.sync_row();                                             // (the sums are read)
  }
  sample_by_bins<T>(b, a, row);
}

// The rows that the first kernel left.  A cluster claims one at a time, so that
// they spread over the clusters wherever they lie; each begins to look at a
// place of its own and goes round once.
template <class T>
__global__ void __launch_bounds__(THREADS, 1) k_sample_bins(const SampleArgs a, const T *__restrict__ logits) {
  __shared__ SharedBins s;
  __shared__ int64_t s_row_of_cluster;
  Block<T, SharedBins> b(s, a);
  const int64_t clusters = gridDim.x >> a.cluster_log2, cluster = blockIdx.x >> a.cluster_log2;
  const int64_t begin = a.n_rows * cluster / clusters;
  int64_t looked = 0;                                         // rows from `begin` on that are claimed or done
  wait_for_last();
  b.sync_row();                                               // all blocks have begun
  for (;;) {
    if (b.rank == 0 && b.warp == 0) {
      int64_t row = -1;
      while (row < 0 && looked < a.n_rows) {
        // 256 rows at a time, eight a lane
        int mine = 8;
#pragma unroll
        for (int i = 7; i >= 0; --i) {
          const int64_t n = looked + i * 32 + b.lane, r = begin + n - (begin + n >= a.n_rows ? a.n_rows : 0);
          if (n < a.n_rows && *(volatile int32_t *)(a.ids + r) == PENDING) mine = i;
        }
        const int first = __reduce_min_sync(~0u, mine * 32 + b.lane);
        if (first >= 256) {
          looked += 256;
          continue;
        }
        looked += first + 1;
        const int64_t n = looked - 1, r = begin + n - (begin + n >= a.n_rows ? a.n_rows : 0);
        int32_t old = 0;
        if (b.lane == 0) old = atomicCAS(a.ids + r, PENDING, CLAIMED);
        if (__shfl_sync(~0u, old, 0) == PENDING) row = r;
      }
      if (b.lane < b.C) *b.at(&s_row_of_cluster, b.lane) = row;
    }
    b.sync_row();                                             // the row is known, and all are done with the last one
    const int64_t row = s_row_of_cluster;
    if (row < 0) return;
    b.parameters(row);
    b.load(logits, row, [] {});
    if (b.row_max == -INF) {                                  // nothing to draw
      if (b.rank == 0 && b.tid == 0) a.ids[row] = -1;
    } else {
      sample_by_bins<T>(b, a, row);
    }
  }
}

template <class T> struct Lists {};
template <class T> struct Bins {};
template <class T> struct Few {};

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
               d_out_ids, d_out_logprobs, d_status, 0, 0, n_rows};
  // Blocks a row: as many as run at once for all rows, of at least 8,192
  // elements.  Clusters of 8, 4, 2 and 1 blocks fit 15, 36, 76 and 152 times at
  // one block an SM, and 32, 72, 152 and 304 times at two.
  auto spread = [&](const int64_t at_once[4]) {
    int log2 = 0;
    while (log2 < 3 && (n_vocab >> (log2 + 1)) >= 8192 && n_rows <= at_once[log2 + 1]) ++log2;
    return log2;
  };
  static const int64_t one_an_sm[4] = {152, 76, 36, 15}, two_an_sm[4] = {304, 152, 72, 32};
  with_type(type, [&](auto t) {
    using T = decltype(t);
    const int64_t vecs = (n_vocab * (int64_t)sizeof(T) + 15) / 16;
    auto launch = [&](auto tag, auto k, int64_t clusters, int most, bool chained) {
      a.held = (int)std::min<int64_t>((vecs + (1 << a.cluster_log2) - 1) >> a.cluster_log2, most / 16);
      if (allow_shared<decltype(tag)>(k, most)) return;       // (the error is kept)
      launch_cluster(k, dim3((unsigned)(clusters << a.cluster_log2)), THREADS, (size_t)a.held * 16, 1u << a.cluster_log2, chained,
                     stream, a, (const T *)d_logits);
    };
    if (!d_top_k && !d_top_p) {                               // a list, or no cut, always does
      a.cluster_log2 = spread(two_an_sm);
      launch(Lists<T>{}, k_sample<T>, n_rows, HELD, false);
      return;
    }
    // Rows that run at once, and whose parts are held to four fifths at least,
    // in one launch.  us for it and for two kernels, rows of bfloat16, with a
    // top-k of 50 and top-p, a top-k of 1000 and top-p, and a mixture of all:
    //     8 x 100256    10   12     28   30     28   40
    //    32 x 100256    11   16     31   72     31   42
    //    76 x 100256    14   15     39   63     49   58
    //   152 x 100256    19   21     53   98     75   64
    //    76 x  32768    11   12      -    -     29   42
    //   152 x   4352     8   10      -    -     25   37
    // With less held it loses: 76 x 200255 floats 25 and 26, 94 and 103 us, 37 of
    // them 25 and 23, 95 and 55.  So do rows that come in turn: 200 x 100256 take
    // 36 and 28, 76 and 72 us.  Other mixtures, by which row is the slowest: 37 x
    // 100256 70 and 54 us, 64 of them 56 and 77, 80 of them 89 and 79; 37 to 120 of
    // 20000 to 50257 IDs 40 to 60 and 50 to 62.
    a.cluster_log2 = spread(one_an_sm);
    if (n_rows <= one_an_sm[0] && (vecs >> a.cluster_log2) * 16 <= HELD_BINS / 4 * 5) {
      launch(Few<T>{}, k_sample_few<T>, n_rows, HELD_BINS, false);
      return;
    }
    a.cluster_log2 = spread(two_an_sm);
    launch(Lists<T>{}, k_sample<T>, n_rows, HELD, false);
    // One block an SM; as a rule a quarter of the rows is left.  us of a call on a
    // mixture, its input not in L2, for 8, 4, 2 and 1 blocks a row:
    //        100256 bfloat16          200255 float
    //    37    (in one launch)        67   79  113  164
    //    64                           74   87  119  171
    //    80                           91  103  134  185
    //   120                          117  107  137  186
    //   153   91   70   83   99      160  147  174  226
    //   200  117   99   89  107      202  191  191  245
    //   256  128  101   91  107      222  201  195  251
    //   300  142  109   93  109      238  214  199  253
    //   400  180  132  124  117      342  295  304  310
    //   512  213  144  132  127      424  350  339  378
    // The rule takes the best of them up to 72 rows and from 200 to 288.  Between, 8
    // blocks would save up to a third and 4 a sixth; above 288, 2 would save up to a
    // fifth.  Rows of 20,000 to 50,257 IDs, 153 to 512 of them, are within a tenth.
    a.cluster_log2 = n_vocab < 16384 ? 0 : n_rows <= 72 ? 3 : n_rows <= 288 ? 1 : 0;
    launch(Bins<T>{}, k_sample_bins<T>, std::min<int64_t>(n_rows, 144 >> a.cluster_log2), HELD_BINS, true);
  });
  return launched("tt_sample");
}
