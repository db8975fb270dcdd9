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
constexpr int HELD = 74 * 1024;                   // bytes of a row a block holds: two blocks an SM
constexpr int GROUPS = 128;                       // groups of threads a row's maxima are taken over
constexpr int LIST = 512;                         // tokens one block ranks
constexpr int LONG_LIST = 1792;                   // tokens worth a list of their own for the later passes
constexpr int BIN_LIST = 512;                     // tokens of a range that are ranked and not divided further
constexpr int SHIFT = 17;                         // first histogram: 64 bins an octave
constexpr int BINS = (40 << (23 - SHIFT)) + 1;    // weights 1 .. 2^40
constexpr int FINER_BINS = 640;                   // of a range
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

// The least e whose weight's bits are at least `key`: passes over a row compare
// powers, which they have, and not weights, which cost four instructions more.
// Below 2^23, half a unit under the weight; a tie goes to an even one.
__device__ __forceinline__ float least_power(uint32_t key) {
  const float w = ceilf(__uint_as_float(key));
  if (w > 8388608.f) return w * (1.f / ONE);
  const float half = w - 0.5f;
  return (((int)w & 1) ? __uint_as_float(__float_as_uint(half) + 1) : half) * (1.f / ONE);
}

// A sum of rint(e * 2^40) without a conversion: adding 96 leaves e rounded to
// 2^-17 in the low bits, and adding 1.5 * 2^-17 to what that cut off leaves the
// rest, rounded to 2^-40.  Both counts stay below 2^31 for 256 terms.  Two
// terms at a time.
struct Sum {
  int hi = 0, lo = 0;
  __device__ __forceinline__ void add2(float e0, float e1) {
    float a0, a1, b0, b1;
    asm("{ .reg .b64 e, a, h, b, k; mov.b64 e, {%4, %5}; mov.b64 k, {%6, %6}; add.rn.f32x2 a, e, k;\n\t"
        "mov.b64 k, {%7, %7}; add.rn.f32x2 h, a, k; mov.b64 k, {%8, %8}; fma.rn.f32x2 b, h, k, e;\n\t"
        "mov.b64 k, {%9, %9}; add.rn.f32x2 b, b, k; mov.b64 {%0, %1}, a; mov.b64 {%2, %3}, b; }"
        : "=f"(a0), "=f"(a1), "=f"(b0), "=f"(b1)
        : "f"(e0), "f"(e1), "f"(96.f), "f"(-96.f), "f"(-1.f), "f"(1.5f / 131072.f));
    hi += __float_as_int(a0) - 0x42C00000;
    hi += __float_as_int(a1) - 0x42C00000;
    lo += __float_as_int(b0) - 0x37400000;
    lo += __float_as_int(b1) - 0x37400000;
  }
  __device__ __forceinline__ u64 value() const { return ((u64)hi << 23) + (u64)(long long)lo; }
};

// the same of one term
__device__ __forceinline__ u64 whole(float e) {
  Sum t;
  t.add2(e, 0.f);
  return t.value();
}

__device__ __forceinline__ u64 warp_sum(u64 v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
  return v;
}

// floor or ceil of f * t, exactly, for an f in [0, 1]: 64-bit floats would
// round, and are slow here (4 us for one product and its conversions)
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

template <int N> struct Most { static constexpr int value = N; };

struct Shared {
  float4 all_max[GROUPS / 4];       // maxima over the row's groups
  float nth_max;
  u64 seg[WARPS];                   // sums over the warps' parts of the row
  u64 sums[8], list_sums[8];        // of the row's blocks, and of their lists
  int n_lists[8];
  u64 total, least, draw;           // of a ranked list: the kept sum, top-p's share, the draw's place
  u64 scan[WARPS], scan2[WARPS];
  uint32_t scan_n[WARPS];
  int n_list, n_long;
  int index;                        // a token found in the row (the first block's counts)
  int bin[2];                       // the lowest and the highest bin where a prefix may end
  uint32_t bin_before, bin_to;      // tokens above the highest, and down to the lowest
  u64 cut_key, cut_sum;             // where a prefix ends, and its sum
  u64 list[LIST];                   // bits of the weight << 32 | ~ID: larger first
  uint32_t red_n[BINS];             // a histogram over the row: counts
  ulonglong2 few[BIN_LIST];         // a bin's tokens and their weights
  uint32_t n_few, part_low[WARPS], part_high[WARPS];
  union {
    uint32_t counts[BINS];          // this block's
    struct {
      u64 red_sum[FINER_BINS];      // and sums
      uint32_t n[3 * FINER_BINS];   // this block's: counts and the sums of the mantissas' low and high bits
    };
    ulonglong2 ranked[LIST];        // the blocks' lists: tokens and their weights
    u64 long_list[LONG_LIST];       // the block's tokens among which the prefix ends
  };
};

__device__ __forceinline__ u64 list_key(float w, int j) { return (u64)__float_as_uint(w) << 32 | (uint32_t)~j; }
__device__ __forceinline__ u64 key_weight(u64 k) { return whole(__uint_as_float((uint32_t)(k >> 32)) * (1.f / ONE)); }

// One row, as a block of its cluster sees it.
template <class T> struct Row {
  static constexpr int E = RowParts<T>::E;
  const uint4 *body;
  uint4 *s_row;
  int n, slab;                      // the block's vectors, and how many a warp takes
  int held, lo, hi;                 // the warp's
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

  // the sum of the weights that keep(e, index) keeps, of this thread's elements
  template <class F> __device__ __forceinline__ u64 sum_if(F keep) const {
    u64 sum = 0;
    for (int v = lo + (threadIdx.x & 31); v < hi; v += 32) {
      float e[E];
      powers(vec(v), e);
      Sum t;
#pragma unroll
      for (int i = 0; i < E; i += 2)
        t.add2(keep(e[i], index(v, i)) ? e[i] : 0.f, keep(e[i + 1], index(v, i + 1)) ? e[i + 1] : 0.f);
      sum += t.value();
    }
    if (lone >= 0) {
      const float e = power(x_lone);
      if (keep(e, lone)) sum += whole(e);
    }
    return sum;
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
      // the warp's sum in parts of 22 bits, each in one instruction
      const u64 sum = (u64)__reduce_add_sync(~0u, (uint32_t)mine & 0x3FFFFFu) +
                      ((u64)__reduce_add_sync(~0u, (uint32_t)(mine >> 22)) << 22);
      if (before + sum <= r) {
        before += sum;
        continue;
      }
      // the lane whose vector passes r walks through it
      const u64 start0 = start_of(mine, before);
      step(mine, before, r, found, own);
      int at = 0;
      u64 w = 0, start = start0;
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

  arrive();
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
    x.n = n;
    x.slab = slab;
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
  const int group_lanes = 4 * C;
  for (int o = 1; o < group_lanes; o <<= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, o));
  // What blocks tell each other is written to all of them ahead of a barrier,
  // so that nothing has to be fetched behind it.
  leave();                                                    // all blocks have begun
  {
    const float y = __shfl_sync(~0u, m, lane < 8 ? (lane >> a.cluster_log2) * group_lanes : 0);
    if (lane < 8)
      reinterpret_cast<float *>(at(s.all_max, lane & (C - 1)))[((rank * WARPS + warp) << (3 - a.cluster_log2)) +
                                                               (lane >> a.cluster_log2)] = y;
  }
  if (tid == 0) s.n_list = 0;
  if (C < 8 && tid >= C && tid < 8) s.sums[tid] = s.list_sums[tid] = s.n_lists[tid] = 0;
  sync_row();
  static_assert(GROUPS == 128, "a float4 a lane");
  const float4 four = s.all_max[lane];
  m = warp_all(fmaxf(fmaxf(four.x, four.y), fmaxf(four.z, four.w)), OpMax());
  const bool valid = u >= 0 && u < 1 && temp >= 0 && temp < INF && top_p >= 0 && top_p <= 1 && min_p >= 0 && min_p <= 1;
  if (!valid || m == -INF) {
    if (rank == 0 && tid == 0) {
      a.ids[row] = -1;
      if (a.logprobs) a.logprobs[row] = -INF;
      if (!valid) op_status(a.status, TT_ERR_INVALID_ARG);
    }
    return;
  }
  x.m = m;
  x.c = fminf(1.44269504f / temp, 3.402823466e38f);
  x.infinite = m == INF;
  const int k = temp == 0 ? 1 : top_k > 0 ? min(top_k, V) : V;
  const float least_w = fmaxf(min_p * ONE, 1.f);              // min-p, and weight 0 is never drawn
  const uint32_t least_key = __float_as_uint(least_w);
  const float least_e = least_power(least_key);
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
    if (warp == 0) {
      best = __reduce_min_sync(~0u, lane < WARPS ? (int)s.scan_n[lane] : INT32_MAX);
      if (lane == 0) at(s.n_lists, 0)[rank] = best;
    }
    sync_row();
    if (rank == 0 && warp == 0) {
      best = __reduce_min_sync(~0u, lane < C ? s.n_lists[lane] : INT32_MAX);
      if (lane == 0) write(best, 1, 1);
    }
    return;
  }

  // ---- sums, and the list of the heaviest tokens
  const bool all = k == V && top_p == 1.f;                    // nothing but min-p cuts
  const bool many = k < V && k > GROUPS * 3 / 4;              // more than the first list holds
  float list_w = least_w;                                     // the list holds all weights from here on
  if (!all && !many) {
    const int q = min(k, GROUPS * 3 / 4);
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
    list_w = fmaxf(list_w, weight_of(x.power(s.nth_max)));
  }
  auto push = [&](float w, int j) {
    const int n = atomicAdd(&s.n_list, 1);
    if (n < LIST) s.list[n] = list_key(w, j);
  };
  auto block_totals = [&]() {                                 // s.seg summed, for all blocks; by warp 0
    if (warp == 0) {
      const u64 t = warp_sum(lane < WARPS ? s.seg[lane] : 0);
      if (lane < C) at(s.sums, lane)[rank] = t;
    }
  };
  auto push_sums = [&](u64 t) {                               // a sum over the row, known behind the next barrier
    t = warp_sum(t);
    if (lane == 0) s.seg[warp] = t;
    __syncthreads();
    block_totals();
  };
  if (!many) {
    u64 sum = 0;
    const float near_e = all ? 2.f : least_power(__float_as_uint(list_w));
    if (min_p == 0.f) {
      for (int v = x.lo + lane; v < x.hi; v += 32) {
        float e[E];
        x.powers(x.vec(v), e);
        Sum t;
        float top = e[0];
#pragma unroll
        for (int i = 0; i < E; i += 2) {
          t.add2(e[i], e[i + 1]);
          top = fmaxf(top, fmaxf(e[i], e[i + 1]));
        }
        sum += t.value();
        if (top >= near_e) {
#pragma unroll
          for (int i = 0; i < E; ++i)
            if (e[i] >= near_e) push(weight_of(e[i]), x.index(v, i));
        }
      }
      if (x.lone >= 0) {
        const float e = x.power(x.x_lone);
        sum += whole(e);
        if (e >= near_e) push(weight_of(e), x.lone);
      }
    } else {
      sum = x.sum_if([&](float e, int j) {
        if (e >= near_e) push(weight_of(e), j);
        return e >= least_e;
      });
    }
    push_sums(sum);
    if (warp == 1 && !all) {
      u64 l = 0;
      const int n = s.n_list;
      for (int i = lane; i < min(n, LIST); i += 32) l += key_weight(s.list[i]);
      l = warp_sum(l);
      if (lane < C) {
        at(s.list_sums, lane)[rank] = l;
        at(s.n_lists, lane)[rank] = n;
      }
    }
    sync_row();
  }

  // ---- what the row's sums say
  auto share = [&](u64 t) { return max(times(top_p, t, true), 1ull); };
  auto place = [&](u64 t) { return times(u, t, false); };
  // of the row's blocks, in every thread: their sum, and that of the ones before this
  auto row_total = [&](u64 &before) {
    u64 t = before = 0;
#pragma unroll
    for (int r = 0; r < 8; ++r) {
      const u64 y = s.sums[r];
      t += y;
      before += r < rank ? y : 0;
    }
    return t;
  };
  u64 before_block = 0, total = many ? 0 : row_total(before_block);

  // ---- the draw among all elements: the block, the warp, the element
  auto draw_row = [&](auto keep) {
    const u64 r = place(total);
    u64 before = before_block;
    if (r < before || r >= before + s.sums[rank]) return;
    int part = 0;
    while (r >= before + s.seg[part]) before += s.seg[part++];
    // that warp's vectors, divided among all warps
    const int lo = min(x.n, part * x.slab), hi = min(x.n, lo + x.slab), each = (hi - lo + WARPS - 1) / WARPS;
    x.lo = min(hi, lo + warp * each);
    x.hi = min(hi, x.lo + each);
    if (part != (x.lone_first ? 0 : WARPS - 1)) x.lone = -1;  // single elements stay with the first and the last
    const u64 sum = warp_sum(x.sum_if(keep));
    __syncthreads();
    if (lane == 0) s.seg[warp] = sum;
    __syncthreads();
    for (int w = 0; w < warp; ++w) before += s.seg[w];
    if (before <= r && r < before + sum) {
      u64 own;
      const int j = x.find([&](float e, int i) { return keep(e, i) ? whole(e) : 0ull; }, r - before, own);
      if (lane == 0) write(j, own, total);
    }
  };
  if (all) {
    draw_row([&](float e, int) { return e >= least_e; });
    return;
  }
  u64 list_sum = 0;
  int n_list = 0;
#pragma unroll
  for (int r = 0; r < 8; ++r) {
    list_sum += s.list_sums[r];
    n_list += s.n_lists[r];
  }

  // the blocks' lists side by side in the first, a warp a block; the others have gone on
  auto gather = [&](ulonglong2 *into) {
    int to = 0;
    for (int r = 0; r < C; ++r) {
      const int n = s.n_lists[r];
      if (warp == r)
        for (int i = lane; i < n; i += 32) {
          const u64 key = at(s.list, r)[i];
          into[to + i] = make_ulonglong2(key, key_weight(key));
        }
      to += n;
    }
    return to;
  };

  // ---- the prefix ends within the list: one block ranks it
  const bool all_listed = list_w == least_w;                  // the list is all there is
  if (!many && n_list <= LIST && (all_listed || (k < V ? k <= n_list : share(total) <= list_sum))) {
    if (rank != 0) {
      arrive();
      leave();
      return;
    }
    const int n = gather(s.ranked), kept_n = min(k, n);
    arrive();
    __syncthreads();
    // the rank of each token and the sum before it; 1, 2, 4 or 8 threads a token
    int per_log2 = 0;
    while (per_log2 < 3 && (n << (per_log2 + 1)) <= THREADS) ++per_log2;
    const int per = 1 << per_log2, i = tid >> per_log2, part = tid & (per - 1);
    const ulonglong2 own = i < n ? s.ranked[i] : make_ulonglong2(0, 0);
    int before_n = 0;
    u64 before = 0;
    for (int o = part; o < n; o += per) {
      const ulonglong2 y = s.ranked[o];
      if (y.x > own.x) {
        ++before_n;
        before += y.y;
      }
    }
    for (int o = 1; o < per; o <<= 1) {
      before_n += __shfl_xor_sync(~0u, before_n, o);
      before += __shfl_xor_sync(~0u, before, o);
    }
    const bool one = part == 0 && i < n;
    if (k < V) {                                              // top-k's sum, then what top-p leaves of it
      if (one && before_n == kept_n - 1) s.least = top_p < 1.f ? share(before + own.y) : before + own.y;
      __syncthreads();
    }
    const u64 least = top_p < 1.f ? (k < V ? s.least : share(total)) : ~0ull;
    const bool keep = before_n < kept_n && before < least;
    if (one && keep) {
      s.list[before_n] = own.x;                               // in their order
      if (before_n == kept_n - 1 || before + own.y >= least) {
        s.index = before_n + 1;
        s.total = before + own.y;
        s.draw = place(before + own.y);
      }
    }
    __syncthreads();
    const int n_kept = s.index;
    u64 low = 0;                                              // kept weights of lower IDs
    if (i < n && keep)
      for (int o = part; o < n_kept; o += per) {
        const u64 y = s.list[o];
        if ((uint32_t)y > (uint32_t)own.x) low += key_weight(y);
      }
    for (int o = 1; o < per; o <<= 1) low += __shfl_xor_sync(~0u, low, o);
    if (one && keep && low <= s.draw && s.draw < low + own.y) write((int)~(uint32_t)own.x, own.y, s.total);
    leave();
    return;
  }

  // ---- the prefix's end by histograms of the weights' bits
  auto key_of = [&](float e) { return __float_as_uint(weight_of(e)); };
  auto key_whole = [&](uint32_t key) { return key_weight((u64)key << 32); };
  uint32_t hist_base = 0;
  int hist_shift = -1;
  // counts of the keys from `base` on, in bins of 2^shift
  auto count_bins = [&](uint32_t base, int shift, int bins) {
    hist_base = base;
    hist_shift = shift;
    for (int b = tid; b < bins; b += THREADS) s.counts[b] = 0;
    __syncthreads();
    x.each([&](float e, int) {
      const uint32_t b = (key_of(e) - base) >> shift;         // (keys below the base come out above the bins)
      if (e >= least_e && b < (uint32_t)bins) atomicAdd(&s.counts[b], 1u);
    });
    sync_row();
    // each block adds up its share of the bins over the row
    const int share_bins = (bins + C - 1) >> a.cluster_log2;
    for (int i = tid; i < share_bins; i += THREADS) {
      const int b = rank * share_bins + i;
      if (b < bins) {
        uint32_t n = 0;
#pragma unroll
        for (int r = 0; r < 8; ++r)
          if (r < C) n += at(s.counts, r)[b];
#pragma unroll
        for (int r = 0; r < 8; ++r)
          if (r < C) at(s.red_n, r)[b] = n;
      }
    }
    sync_row();
  };
  // The same with the bins' sums (a mantissa's low and high bits counted
  // apart), and the sum of what lies above the bins.
  auto sum_bins = [&](uint32_t base, int shift, int bins) {
    hist_shift = -1;
    for (int b = tid; b < 3 * FINER_BINS; b += THREADS) s.n[b] = 0;
    __syncthreads();
    const float from_e = fmaxf(least_e, least_power(base)), above_e = fmaxf(least_e, least_power(base + ((uint32_t)bins << shift)));
    const u64 above = x.sum_if([&](float e, int) {
      if (e >= from_e && e < above_e) {
        const uint32_t key = key_of(e), b = (key - base) >> shift, low = key & ((1u << shift) - 1);
        atomicAdd(&s.n[b], 1u);
        atomicAdd(&s.n[FINER_BINS + b], low & 1023u);
        atomicAdd(&s.n[2 * FINER_BINS + b], low >> 10);
      }
      return e >= above_e;
    });
    push_sums(above);
    sync_row();
    const int share_bins = (bins + C - 1) >> a.cluster_log2;
    for (int i = tid; i < share_bins; i += THREADS) {
      const int b = rank * share_bins + i;
      if (b < bins) {
        u64 n = 0, low = 0;
#pragma unroll
        for (int r = 0; r < 8; ++r)
          if (r < C) {
            n += at(s.n, r)[b];
            low += at(s.n, r)[FINER_BINS + b] + ((u64)at(s.n, r)[2 * FINER_BINS + b] << 10);
          }
        // weights are mantissa << (exponent - 23); whole, so nothing is lost
        const uint32_t key = base + ((uint32_t)b << shift);
        const int ex = (int)(key >> 23) - 150;
        const u64 mant = n * ((key & 0x7FFFFFu) | 0x800000u) + low, w = ex >= 0 ? mant << ex : mant >> -ex;
#pragma unroll
        for (int r = 0; r < 8; ++r)
          if (r < C) {
            at(s.red_n, r)[b] = (uint32_t)n;
            at(s.red_sum, r)[b] = w;
          }
      }
    }
    sync_row();
  };
  // From the heaviest bin down, f(bin, count, count before, sum, sum before) of
  // this thread's bins; what goes into the sums, val(bin, which) for two sums.
  auto scan_bins = [&](auto most, int bins, auto val, auto f) {
    constexpr int PER = (decltype(most)::value + THREADS - 1) / THREADS;
    uint32_t n[PER], own_n = 0;
    u64 w[PER][2], own_w[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int b = bins - 1 - (tid * PER + i);
      n[i] = b >= 0 ? s.red_n[b] : 0;
      own_n += n[i];
#pragma unroll
      for (int c = 0; c < 2; ++c) own_w[c] += w[i][c] = b >= 0 ? val(b, c) : 0;
    }
    uint32_t pn = own_n;
    u64 pw[2] = {own_w[0], own_w[1]};
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t yn = __shfl_up_sync(~0u, pn, o);
      const u64 y0 = __shfl_up_sync(~0u, pw[0], o), y1 = __shfl_up_sync(~0u, pw[1], o);
      if (lane >= o) pn += yn, pw[0] += y0, pw[1] += y1;
    }
    __syncthreads();
    if (lane == 31) s.scan_n[warp] = pn, s.scan[warp] = pw[0], s.scan2[warp] = pw[1];
    __syncthreads();
    pn -= own_n;
    pw[0] -= own_w[0];
    pw[1] -= own_w[1];
    u64 all_w[2] = {0, 0};
    for (int i = 0; i < WARPS; ++i) {
      if (i < warp) pn += s.scan_n[i], pw[0] += s.scan[i], pw[1] += s.scan2[i];
      all_w[0] += s.scan[i];
      all_w[1] += s.scan2[i];
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int b = bins - 1 - (tid * PER + i);
      if (b >= 0) f(b, n[i], pn, w[i], pw, all_w);
      pn += n[i];
      pw[0] += w[i][0];
      pw[1] += w[i][1];
    }
    __syncthreads();
  };
  // In the first histogram, the bin where the count reaches `want`; or the bins
  // between which the sum does: a bin's sum is its count times weights it
  // bounds, added from above, or from below and taken from the row's sum.
  u64 row_sum = total;
  auto first_bins = [&](bool by_n, u64 want) {
    if (hist_base != KEY_ONE || hist_shift != SHIFT) count_bins(KEY_ONE, SHIFT, BINS);
    if (by_n) {
      scan_bins(Most<BINS>{}, BINS, [](int, int) { return 0ull; }, [&](int b, uint32_t n, uint32_t pn, const u64 *, const u64 *, const u64 *) {
        if (pn < want && pn + n >= want) {
          s.bin[0] = s.bin[1] = b;
          s.bin_before = pn;
          s.bin_to = pn + n;
        }
      });
    } else {
      scan_bins(
          Most<BINS>{}, BINS,
          [&](int b, int c) {
            // a bin holds weights of whole numbers: from its base on, below the next one's
            const uint32_t key = KEY_ONE + ((uint32_t)b << SHIFT);
            const u64 low = key_whole(key), next = key_whole(key + (1u << SHIFT));
            return s.red_n[b] * (c == 0 ? low : b == BINS - 1 ? low : max(low, next));
          },
          [&](int b, uint32_t n, uint32_t pn, const u64 *w, const u64 *pw, const u64 *all_w) {
            auto least_sum = [&](u64 l, u64 h) { return max((long long)l, (long long)(row_sum + h - all_w[1])); };
            auto most_sum = [&](u64 l, u64 h) { return min((long long)h, (long long)(row_sum + l - all_w[0])); };
            const long long t = (long long)want;
            if (most_sum(pw[0], pw[1]) < t && most_sum(pw[0] + w[0], pw[1] + w[1]) >= t) {
              s.bin[1] = b;
              s.bin_before = pn;
            }
            if (least_sum(pw[0], pw[1]) < t && least_sum(pw[0] + w[0], pw[1] + w[1]) >= t) {
              s.bin[0] = b;
              s.bin_to = pn + n;
            }
          });
    }
  };

  // A row's heaviest tokens, from a key on, as lists of the blocks' own: the
  // later passes go over these where they are few.
  bool listed = false;
  auto make_list = [&](uint32_t least_in) {
    if (tid == 0) s.n_long = 0;
    __syncthreads();
    const float from_e = least_power(least_in);
    x.each([&](float e, int j) {
      if (e >= from_e) s.long_list[atomicAdd(&s.n_long, 1)] = list_key(weight_of(e), j);
    });
    __syncthreads();
    listed = true;
  };
  // the sum of the weights that f(power, ID) keeps, of this thread's share of the block
  auto sum_keys = [&](auto f) {
    if (!listed) return x.sum_if(f);
    u64 sum = 0;
    for (int i = tid; i < s.n_long; i += THREADS) {
      const u64 key = s.long_list[i];
      const float e = __uint_as_float((uint32_t)(key >> 32)) * (1.f / ONE);
      if (f(e, (int)~(uint32_t)key)) sum += whole(e);
    }
    return sum;
  };

  // the last token (as a list key) of the shortest prefix with `want` tokens
  // (by_n) or a sum of `want`, and the prefix's sum; behind first_bins
  bool parts_known = false;                                   // s.seg has the sums of what lies above s.list
  auto prefix_end = [&](bool by_n, u64 want, u64 &end_key, u64 &prefix_sum) {
    parts_known = false;
    uint32_t base = KEY_ONE, before_n = 0;
    int shift = SHIFT;
    uint32_t end = base + ((uint32_t)(s.bin[1] + 1) << shift);
    base += (uint32_t)s.bin[0] << shift;
    uint32_t n_range = s.bin_to - s.bin_before;
    if (by_n) before_n = s.bin_before;
    for (;;) {
      __syncthreads();
      if (n_range <= BIN_LIST) {
        // the tokens that are left, ranked in the first block
        if (tid == 0) s.n_list = 0;
        __syncthreads();
        const float from_e = fmaxf(least_e, least_power(base)), above_e = fmaxf(least_e, least_power(end));
        const u64 above = sum_keys([&](float e, int j) {
          if (e >= from_e && e < above_e) push(weight_of(e), j);
          return e >= above_e;
        });
        push_sums(above);
        if (tid == 0) at(s.n_lists, 0)[rank] = s.n_list;
        sync_row();
        if (rank == 0) {
          const int n = gather(s.few), two = n <= THREADS / 2, i = tid >> two;
          u64 unused;
          const u64 before_sum = row_total(unused);
          __syncthreads();
          const ulonglong2 own = i < n ? s.few[i] : make_ulonglong2(0, 0);
          u64 rank_n = 0, sum_to = 0;
          for (int o = tid & two; o < n; o += 1 + two) {
            const ulonglong2 y = s.few[o];
            if (y.x >= own.x) {
              ++rank_n;
              sum_to += y.y;
            }
          }
          if (two) {
            rank_n += __shfl_xor_sync(~0u, rank_n, 1);
            sum_to += __shfl_xor_sync(~0u, sum_to, 1);
          }
          rank_n += before_n;
          sum_to += before_sum;
          if ((tid & two) == 0 && i < n && (by_n ? rank_n == want : sum_to >= want && sum_to - own.y < want)) {
            for (int r = 0; r < C; ++r) {
              *at(&s.cut_key, r) = own.x;
              *at(&s.cut_sum, r) = sum_to;
            }
          }
        }
        sync_row();
        end_key = s.cut_key;
        prefix_sum = s.cut_sum;
        parts_known = true;
        return;
      }
      if (end - base == 1) {
        // tokens of one weight: the prefix ends at one of them by its place
        const u64 w = key_whole(base);
        const float own_e = least_power(base), above_e = least_power(base + 1);
        push_sums(x.sum_if([&](float e, int) { return e >= above_e; }));
        sync_row();
        u64 before;
        const u64 above = row_total(before), some = by_n ? want - before_n : (want - above + w - 1) / w;
        prefix_sum = above + some * w;
        u64 c = 0;
        x.each([&](float e, int) { c += e >= own_e && e < above_e; });
        sync_row();                                           // (the sums are read)
        push_sums(c);
        sync_row();
        row_total(before);
        if (before < some && some <= before + s.sums[rank]) {
          for (int i = 0; i < warp; ++i) before += s.seg[i];
          if (before < some && some <= before + s.seg[warp]) {
            u64 own;
            const int j = x.find([&](float e, int) { return e >= own_e && e < above_e ? 1ull : 0ull; }, some - 1 - before, own);
            if (lane < C) *at(&s.cut_key, lane) = list_key(__uint_as_float(base), j);
          }
        }
        sync_row();
        end_key = s.cut_key;
        return;
      }
      // finer bins of what is left, as many as fit; none spans an octave
      listed = false;                                         // (they lie over the list)
      for (shift = 0; (end - (base >> shift << shift) + (1u << shift) - 1) >> shift > FINER_BINS;) ++shift;
      base = base >> shift << shift;
      const int bins = (int)((end - base + (1u << shift) - 1) >> shift);
      if (by_n) {
        count_bins(base, shift, bins);
        const uint32_t from = before_n;
        scan_bins(Most<FINER_BINS>{}, bins, [](int, int) { return 0ull; }, [&](int b, uint32_t n, uint32_t pn, const u64 *, const u64 *, const u64 *) {
          pn += from;
          if (pn < want && pn + n >= want) {
            s.bin[0] = b;
            s.bin_before = pn;
          }
        });
        before_n = s.bin_before;
      } else {
        sum_bins(base, shift, bins);
        u64 unused;
        const u64 above = row_total(unused);
        scan_bins(Most<FINER_BINS>{}, bins, [&](int b, int c) { return c == 0 ? s.red_sum[b] : 0; },
                  [&](int b, uint32_t, uint32_t, const u64 *w, const u64 *pw, const u64 *) {
                    if (above + pw[0] < want && above + pw[0] + w[0] >= want) s.bin[0] = b;
                  });
      }
      n_range = s.red_n[s.bin[0]];
      base += (uint32_t)s.bin[0] << shift;
      end = base + (1u << shift);
    }
  };
  u64 end_key = 0;                                            // keeps everything
  auto list_if_few = [&]() {
    const uint32_t n = s.bin_to, from = KEY_ONE + ((uint32_t)s.bin[0] << SHIFT);
    if (n <= LONG_LIST) make_list(max(least_key, from));
  };
  if (k < V) {
    // fewer than k tokens may be left by min-p
    count_bins(KEY_ONE, SHIFT, BINS);
    uint32_t n = 0;
    for (int b = tid; b < BINS; b += THREADS) n += s.red_n[b];
    n = block_all(n, OpSum(), s.scan_n);
    const bool cuts = n > (uint32_t)k;
    if (many && (!cuts || top_p < 1.f)) {
      push_sums(x.sum_if([&](float e, int) { return e >= least_e; }));
      sync_row();
      row_sum = total = row_total(before_block);
      sync_row();
    }
    if (cuts) {
      first_bins(true, k);
      list_if_few();
      prefix_end(true, k, end_key, total);
    }
  }
  if (top_p < 1.f) {
    const u64 least = share(total);
    if (least < total) {
      first_bins(false, least);
      if (end_key == 0) list_if_few();
      prefix_end(false, least, end_key, total);
    }
  }
  // what is kept, by the warps' parts of the row
  const uint32_t end_w = max(least_key, (uint32_t)(end_key >> 32));
  const float from_e = least_power(end_w), above_e = least_power(end_w + 1);
  auto keep = [&](float e, int j) { return e >= above_e || (e >= from_e && list_key(weight_of(e), j) >= end_key); };
  auto part_of = [&](u64 key) {
    const int j = (int)~(uint32_t)key, v = (j - x.first) / E;
    return j < x.first ? 0 : v >= x.n ? WARPS - 1 : v / x.slab;
  };
  if (listed) {
    if (tid < WARPS) s.part_low[tid] = s.part_high[tid] = 0;
    if (tid == 0) s.n_few = 0;
    __syncthreads();
    for (int i = tid; i < s.n_long; i += THREADS) {
      const u64 key = s.long_list[i];
      if (key >= end_key) {                                   // 2^21 * LONG_LIST is below 2^32
        const u64 w = key_weight(key);
        const int part = part_of(key);
        atomicAdd(&s.part_low[part], (uint32_t)w & 0x1FFFFFu);
        atomicAdd(&s.part_high[part], (uint32_t)(w >> 21));
      }
    }
    __syncthreads();
    if (tid < WARPS) s.seg[tid] = s.part_low[tid] + ((u64)s.part_high[tid] << 21);
    __syncthreads();
    block_totals();
  } else if (parts_known) {
    // the sums of what lies above the ranked tokens, and those
    for (int i = tid; i < s.n_list; i += THREADS) {
      const u64 key = s.list[i];
      if (key >= end_key) atomicAdd(&s.seg[part_of(key)], key_weight(key));
    }
    __syncthreads();
    block_totals();
  } else {
    push_sums(x.sum_if(keep));
  }
  sync_row();
  total = row_total(before_block);
  if (!listed) {
    draw_row(keep);
    return;
  }
  // the part of the row that holds the drawn token, and its listed tokens by ID
  const u64 r = place(total);
  if (r < before_block || r >= before_block + s.sums[rank]) return;
  int part = 0;
  while (r >= before_block + s.seg[part]) before_block += s.seg[part++];
  for (int i = tid; i < s.n_long; i += THREADS) {
    const u64 key = s.long_list[i];
    if (key >= end_key && part_of(key) == part) {
      const uint32_t n = atomicAdd(&s.n_few, 1u);
      if (n < BIN_LIST) s.few[n] = make_ulonglong2(key, key_weight(key));
    }
  }
  __syncthreads();
  const int n_few = s.n_few;
  if (n_few <= THREADS / 2) {
    const int i = tid >> 1;
    const ulonglong2 own = i < n_few ? s.few[i] : make_ulonglong2(0, 0);
    u64 low = 0;
    for (int o = tid & 1; o < n_few; o += 2) {
      const ulonglong2 y = s.few[o];
      if ((uint32_t)y.x > (uint32_t)own.x) low += y.y;
    }
    low += __shfl_xor_sync(~0u, low, 1) + before_block;
    if ((tid & 1) == 0 && i < n_few && low <= r && r < low + own.y) write((int)~(uint32_t)own.x, own.y, total);
  } else if (warp == part) {
    u64 own;
    const int j = x.find([&](float e, int i) { return keep(e, i) ? whole(e) : 0ull; }, r - before_block, own);
    if (lane == 0) write(j, own, total);
  }
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
  // Blocks a row: as many as run at once for all rows (clusters of 8, 4 and 2
  // fit 32, 72 and 152 times, two blocks an SM), of at least 8,192 elements
  const int64_t at_once[4] = {INT64_MAX, 152, 72, 32};
  while (a.cluster_log2 < 3 && (n_vocab >> (a.cluster_log2 + 1)) >= 8192 && n_rows <= at_once[a.cluster_log2 + 1]) ++a.cluster_log2;
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
