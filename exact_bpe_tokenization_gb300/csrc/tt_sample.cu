// tt_sample.cu - drawing token IDs from rows of logits (include/toktier.h).
#include "tt_ops.cuh"

using namespace tt::ops;

namespace {

struct SampleArgs {
  int64_t n_vocab, stride;
  const float *uniform, *temperature;
  const int32_t *top_k;
  const float *top_p, *min_p;
  int32_t *ids;
  float *logprobs;
  int32_t *status;
};

constexpr float WEIGHT_ONE = 1099511627776.f;   // 2^40, the largest weight
constexpr int THREADS = 512;
constexpr int WARPS = THREADS / 32;

// The weight of a logit: a whole number below 2^41 that a float holds
// exactly, so its bits order weights and its value converts without loss.
__device__ __forceinline__ float weight(float l, float m, float c) {
  if (!(l > -INF)) return 0.f;                     // -inf and NaN
  const float y = l == m ? 0.f : (m - l) * c;
  return rintf(exp2f(-y) * WEIGHT_ONE);
}

// What is kept: weights above `thr`, and those equal to it at IDs below `ties`.
struct Kept {
  float thr;
  int64_t ties;
  __device__ bool operator()(float w, int64_t j) const { return w > thr || (w == thr && j < ties); }
};

// a block a row; thresholds found by bisection over the weights' bits
template <class T>
__global__ void __launch_bounds__(THREADS) k_sample(SampleArgs a, const T *__restrict__ logits) {
  __shared__ float fbox[WARPS];
  __shared__ unsigned long long ubox[WARPS];
  typedef unsigned long long u64;
  const int64_t row = blockIdx.x;
  const T *l = logits + row * a.stride;
  const int V = (int)a.n_vocab, tid = threadIdx.x;
  const float u = a.uniform[row], t = a.temperature ? a.temperature[row] : 1.f;
  const float top_p = a.top_p ? a.top_p[row] : 1.f, min_p = a.min_p ? a.min_p[row] : 0.f;
  const int top_k = a.top_k ? a.top_k[row] : 0;
  const bool valid = u >= 0 && u < 1 && t >= 0 && t < INF && top_p >= 0 && top_p <= 1 && min_p >= 0 && min_p <= 1;
  float m = -INF;
  for (int j = tid; j < V; j += THREADS) m = fmaxf(m, to_f32(l[j]));
  m = block_all(m, OpMax(), fbox);
  if (!valid || m == -INF) {
    if (tid == 0) {
      a.ids[row] = -1;
      if (a.logprobs) a.logprobs[row] = -INF;
      if (!valid) op_status(a.status, TT_ERR_INVALID_ARG);
    }
    return;
  }
  const float c = fminf(1.44269504f / t, 3.402823466e38f);
  const int64_t k = t == 0 ? 1 : top_k > 0 ? top_k : V;
  Kept kept{fmaxf(min_p * WEIGHT_ONE, 1.f), V};

  // number (or sum of weights) of the kept tokens with weight >= x
  auto count = [&](float x, bool equal_only, int64_t below) {
    u64 s = 0;
    for (int j = tid; j < V; j += THREADS) {
      const float w = weight(to_f32(l[j]), m, c);
      if (kept(w, j) && (equal_only ? w == x && j < below : w >= x)) ++s;
    }
    return block_all(s, OpSum(), ubox);
  };
  auto sum = [&](float x) {
    u64 s = 0;
    for (int j = tid; j < V; j += THREADS) {
      const float w = weight(to_f32(l[j]), m, c);
      if (kept(w, j) && w >= x) s += (u64)w;
    }
    return block_all(s, OpSum(), ubox);
  };
  // the largest weight x with f(x) >= want (f falls with x, f(0) >= want)
  auto find = [&](auto f, u64 want) {
    uint32_t lo = 0, hi = __float_as_uint(WEIGHT_ONE) + 1;
    while (hi - lo > 1) {
      const uint32_t mid = (lo + hi) >> 1;
      if (f(__uint_as_float(mid)) >= want) lo = mid; else hi = mid;
    }
    return __uint_as_float(lo);
  };
  // keep only the first `some` of the kept tokens of weight x, and those above
  auto cut = [&](float x, u64 some) {
    int64_t lo = 0, hi = V;                       // count below lo < some <= count below hi
    while (hi - lo > 1) {
      const int64_t mid = (lo + hi) >> 1;
      if (count(x, true, mid) >= some) hi = mid; else lo = mid;
    }
    kept = Kept{x, hi};
  };

  if (count(0.f, false, 0) > (u64)k) {
    const float x = find([&](float y) { return count(y, false, 0); }, (u64)k);
    const u64 equal = count(x, true, V);
    cut(x, (u64)k - (count(x, false, 0) - equal));
  }
  u64 total = sum(0.f);
  const u64 least = (u64)fmax(ceil((double)top_p * (double)total), 1.0);
  if (least < total) {
    const float x = find(sum, least);
    const u64 above = sum(x) - count(x, true, V) * (u64)x;
    cut(x, (least - above + (u64)x - 1) / (u64)x);
    total = sum(0.f);
  }
  // the warp whose part of the row holds the drawn token, then the token
  const u64 r = (u64)floor((double)u * (double)total);
  const int part = (V + WARPS - 1) / WARPS, warp = tid >> 5, lane = tid & 31;
  const int lo = min(V, warp * part), hi = min(V, lo + part);
  u64 s = 0;
  for (int j = lo + lane; j < hi; j += 32) {
    const float w = weight(to_f32(l[j]), m, c);
    if (kept(w, j)) s += (u64)w;
  }
  s = warp_all(s, OpSum());
  __syncthreads();
  if (lane == 0) ubox[warp] = s;
  __syncthreads();
  u64 before = 0;
  for (int i = 0; i < warp; ++i) before += ubox[i];
  if (!(before <= r && r < before + s)) return;
  for (int base = lo; base < hi; base += 32) {
    const int j = base + lane;
    const float w = j < hi ? weight(to_f32(l[j]), m, c) : 0.f;
    const u64 own = j < hi && kept(w, j) ? (u64)w : 0;
    u64 x = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const u64 y = __shfl_up_sync(~0u, x, o);
      if (lane >= o) x += y;
    }
    const uint32_t past = __ballot_sync(~0u, before + x > r);
    if (past) {
      if (lane == __ffs(past) - 1) {
        a.ids[row] = j;
        if (a.logprobs) a.logprobs[row] = logf((float)((double)own / (double)total));
      }
      return;
    }
    before += __shfl_sync(~0u, x, 31);
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
  const SampleArgs a{n_vocab, logits_stride, d_uniform, d_temperature, d_top_k, d_top_p, d_min_p,
                     d_out_ids, d_out_logprobs, d_status};
  with_type(type, [&](auto t) {
    using T = decltype(t);
    k_sample<T><<<(unsigned)n_rows, THREADS, 0, stream>>>(a, (const T *)d_logits);
  });
  return launched("tt_sample");
}
