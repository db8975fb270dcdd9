// tt_loss.cu - next-token loss of rows of logits and its gradient
// (include/toktier.h).
//
//   lse = M + log(sum_j exp(l_j - M)),  loss = lse - l_t,
//   dl_j = g * (exp(l_j - lse) - (j == t))
//
// Bound by memory: each logit has to be read and each gradient written once.
// The gradient needs lse, which needs the whole row, so a row is read, kept in
// shared memory, and turned into gradients from there: a cluster of blocks
// holds a row (two blocks an SM, so that one reads or writes while the other
// computes).  What does not fit (rows above 832 KB) is read again, from L2.
#include <algorithm>

#include "tt_ops.cuh"

using namespace tt::ops;

namespace {

constexpr int THREADS = 512;
constexpr int WARPS = THREADS / 32;
constexpr int HELD = 104 * 1024;                 // bytes of a row a block holds: two blocks an SM
constexpr float LOG2E = 1.44269504f;
constexpr float LOWEST = -3.402823466e38f;

struct LossArgs {
  int64_t n_vocab, logits_stride, dlogits_stride;
  const int32_t *targets;
  float *loss, *lse_out;
  const float *lse_in, *row_grads;
  int32_t *status;
  int cluster, held;                             // blocks a row, vectors a block can hold
};

// A running maximum and the sum of exp(l - maximum).  The maximum stays within
// the finite floats, so that a difference is NaN only where a logit is: +inf
// adds +inf to the sum, -inf nothing.
struct Running {
  float m = LOWEST, s = 0;
  template <int E> __device__ __forceinline__ void add(const float (&v)[E]) {
    float vm = v[0];
#pragma unroll
    for (int i = 1; i < E; ++i) vm = fmaxf(vm, v[i]);
    if (vm > m) {
      vm = fminf(vm, -LOWEST);
      s *= ex2((m - vm) * LOG2E);
      m = vm;
    }
#pragma unroll
    for (int i = 0; i < E; i += 2) {
      const float2 y = sub_mul2(make_float2(v[i], v[i + 1]), m, LOG2E);
      s += ex2(y.x);
      s += ex2(y.y);
    }
  }
  __device__ __forceinline__ void join(float om, float os) {
    const float nm = fmaxf(m, om);
    s = s * ex2((m - nm) * LOG2E) + os * ex2((om - nm) * LOG2E);
    m = nm;
  }
};

// GRAD: 0 the loss alone, 1 with its gradient, 2 the gradient from lse
constexpr int UC = 2, AHEAD = 6;                // vectors a group of copies, groups ahead

// a thread's first vector behind the held ones
__device__ __forceinline__ int first_of(int tid, int held) { return tid + (held - tid + THREADS - 1) / THREADS * THREADS; }

template <class T, int GRAD>
__global__ void __launch_bounds__(THREADS, 2) k_loss(LossArgs a, const T *logits, T *dlogits) {
  constexpr int E = RowParts<T>::E, U = 4;
  extern __shared__ uint4 s_row[];
  __shared__ float2 s_warp[WARPS], s_block;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = a.cluster > 1 ? (int)cluster_rank() : 0;
  const int64_t row = blockIdx.x / a.cluster;
  const T *l = logits + row * a.logits_stride;
  const RowParts<T> part(l, (int)a.n_vocab);
  const int each = (part.vecs + a.cluster - 1) / a.cluster, first = min(part.vecs, rank * each);
  const int n = min(part.vecs - first, each);
  const uint4 *body = reinterpret_cast<const uint4 *>(l + part.lead) + first;
  const int lone = rank == 0 ? part.scalar(tid) : -1;
  const float x = lone >= 0 ? to_f32(l[lone]) : -INF;
  const int32_t t = a.targets[row];
  const bool there = (uint32_t)t < (uint32_t)a.n_vocab;
  if (!there && t >= 0 && rank == 0 && tid == 0) op_status(a.status, TT_ERR_INVALID_ARG);

  float lse;
  if (GRAD == 2) {
    lse = a.lse_in[row];
  } else {
    // read by one thread, before any block can write to the row
    const float lt = there && rank == 0 && tid == 0 ? to_f32(l[t]) : 0.f;
    Running run;
    if (GRAD) {
      // what is held comes by copies that run ahead; a thread reads its own
      const int n_held = min(n, a.held);
      auto fetch = [&](int v0) {
#pragma unroll
        for (int u = 0; u < UC; ++u)
          if (v0 + u * THREADS < n_held) copy_async(s_row + v0 + u * THREADS, body + v0 + u * THREADS);
        copy_group();
      };
#pragma unroll
      for (int d = 0; d < AHEAD; ++d) fetch(tid + d * UC * THREADS);
      for (int v0 = tid; v0 < n_held; v0 += UC * THREADS) {
        copy_wait<AHEAD - 1>();
        fetch(v0 + AHEAD * UC * THREADS);
#pragma unroll
        for (int u = 0; u < UC; ++u)
          if (v0 + u * THREADS < n_held) {
            float v[E];
            vec_f32(s_row[v0 + u * THREADS], v, T{});
            run.add(v);
          }
      }
    }
    for (int v0 = GRAD ? first_of(tid, a.held) : tid; v0 < n; v0 += U * THREADS) {
      uint4 r[U];
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (v0 + u * THREADS < n) r[u] = __ldcs(body + v0 + u * THREADS);
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (v0 + u * THREADS < n) {
          float v[E];
          vec_f32(r[u], v, T{});
          run.add(v);
        }
    }
    if (lone >= 0) {
      const float v[2] = {x, -INF};
      run.add(v);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) run.join(__shfl_xor_sync(~0u, run.m, o), __shfl_xor_sync(~0u, run.s, o));
    if (lane == 0) s_warp[warp] = make_float2(run.m, run.s);
    __syncthreads();
    run = Running();
    for (int w = 0; w < WARPS; ++w) run.join(s_warp[w].x, s_warp[w].y);
    if (a.cluster > 1) {
      if (tid == 0) s_block = make_float2(run.m, run.s);
      cluster_sync();
      run = Running();
      for (int b = 0; b < a.cluster; ++b) {
        const float2 o = *of_block(&s_block, b);
        run.join(o.x, o.y);
      }
      cluster_arrive();                          // blocks stay until all have read
    }
    lse = run.m + logf(run.s);
    if (rank == 0 && tid == 0) {
      if (a.lse_out) a.lse_out[row] = lse;
      a.loss[row] = !there ? 0.f : lse == -INF ? INF : lse - lt;
    }
  }
  if (GRAD) {
    T *d = dlogits + row * a.dlogits_stride;
    const bool none = !there || lse == -INF;
    const float g = none ? 0.f : a.row_grads ? a.row_grads[row] : 1.f;
    const bool same = ((reinterpret_cast<uintptr_t>(d) ^ reinterpret_cast<uintptr_t>(l)) & 15) == 0;
    // the target among this block's vectors: its vector, and its place there
    const int at = t - part.lead - first * E, tv = there && at >= 0 ? at / E : -1;
    for (int v0 = tid; v0 < n; v0 += U * THREADS) {
      uint4 r[U];
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (v0 + u * THREADS < n)
          r[u] = GRAD == 1 && v0 + u * THREADS < a.held ? s_row[v0 + u * THREADS] : __ldcs(body + v0 + u * THREADS);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int vi = v0 + u * THREADS;
        if (vi < n) {
          float v[E];
          vec_f32(r[u], v, T{});
#pragma unroll
          for (int i = 0; i < E; i += 2) {
            const float2 y = sub_mul2(make_float2(v[i], v[i + 1]), lse, LOG2E);
            v[i] = ex2(y.x);
            v[i + 1] = ex2(y.y);
          }
          if (vi == tv) {
#pragma unroll
            for (int i = 0; i < E; ++i) v[i] -= i == at % E ? 1.f : 0.f;
          }
#pragma unroll
          for (int i = 0; i < E; ++i) v[i] = none ? 0.f : v[i] * g;
          T *to = d + part.lead + (int64_t)(first + vi) * E;
          if (same) {
            __stcs(reinterpret_cast<uint4 *>(to), f32_vec(v, T{}));
          } else {
#pragma unroll
            for (int i = 0; i < E; ++i) to[i] = from_f32<T>(v[i]);
          }
        }
      }
    }
    if (lone >= 0) d[lone] = from_f32<T>(none ? 0.f : (ex2((x - lse) * LOG2E) - (lone == t ? 1.f : 0.f)) * g);
  }
  if (GRAD != 2 && a.cluster > 1) cluster_wait();
}

template <class T, int GRAD> struct Tag {};

template <class T, int GRAD>
void run_rows(LossArgs a, int64_t n_rows, const void *logits, void *dlogits, tt_stream_t stream) {
  const int64_t bytes = a.n_vocab * (int64_t)sizeof(T);
  a.cluster = (int)std::min<int64_t>(8, (bytes + HELD - 1) / HELD);
  // few rows: spread each over more blocks, down to 16 KB a block
  while (a.cluster <= 4 && n_rows * a.cluster * 2 <= 2 * 152 && bytes >= a.cluster * 2 * 16384) a.cluster *= 2;
  const int64_t each = ((bytes + 15) / 16 + a.cluster - 1) / a.cluster;
  a.held = GRAD == 1 ? (int)std::min<int64_t>(each, HELD / 16) : 0;
  auto k = k_loss<T, GRAD>;
  const size_t shared = (size_t)a.held * 16;
  if (GRAD == 1 && allow_shared<Tag<T, GRAD>>(k, HELD)) return;     // (the error is kept)
  launch_cluster(k, dim3((unsigned)(n_rows * a.cluster)), THREADS, shared, a.cluster, false, stream, a, (const T *)logits, (T *)dlogits);
}

tt_status run_loss(const void *d_logits, int32_t type, int64_t n_rows, const LossArgs &a, void *d_dlogits,
                   tt_stream_t stream, const char *what) {
  if (!type_ok(type) || n_rows < 0 || !vocab_ok(a.n_vocab) || a.logits_stride < a.n_vocab ||
      (d_dlogits && a.dlogits_stride < a.n_vocab) || !optional_ok(a.status, 4) || !optional_ok(a.row_grads, 4) ||
      !optional_ok(a.lse_out, 4) || !optional_ok(a.lse_in, 4) || !optional_ok(a.loss, 4) ||
      !optional_ok(d_dlogits, type_size(type)) || (d_dlogits == d_logits && d_logits && a.dlogits_stride != a.logits_stride))
    return TT_ERR_INVALID_ARG;
  if (n_rows > TT_MAX_IDS) return TT_ERR_CAPACITY;
  if (n_rows == 0) return TT_OK;
  if (!array_ok(d_logits, type_size(type)) || !array_ok(a.targets, 4)) return TT_ERR_INVALID_ARG;
  if (!a.lse_in && !a.loss) return TT_ERR_INVALID_ARG;
  with_type(type, [&](auto t) {
    using T = decltype(t);
    if (a.lse_in) run_rows<T, 2>(a, n_rows, d_logits, d_dlogits, stream);
    else if (d_dlogits) run_rows<T, 1>(a, n_rows, d_logits, d_dlogits, stream);
    else run_rows<T, 0>(a, n_rows, d_logits, nullptr, stream);
  });
  return launched(what);
}

}  // namespace

extern "C" tt_status tt_token_loss(const void *d_logits, int32_t type, int64_t n_rows, int64_t n_vocab,
                                   int64_t logits_stride, const int32_t *d_targets, float *d_loss, float *d_lse,
                                   const float *d_row_grads, void *d_dlogits, int64_t dlogits_stride,
                                   int32_t *d_status, tt_stream_t stream) {
  const LossArgs a{n_vocab, logits_stride, dlogits_stride, d_targets, d_loss, d_lse, nullptr, d_row_grads, d_status, 1, 0};
  return run_loss(d_logits, type, n_rows, a, d_dlogits, stream, "tt_token_loss");
}

extern "C" tt_status tt_token_loss_grad(const void *d_logits, int32_t type, int64_t n_rows, int64_t n_vocab,
                                        int64_t logits_stride, const int32_t *d_targets, const float *d_lse,
                                        const float *d_row_grads, void *d_dlogits, int64_t dlogits_stride,
                                        int32_t *d_status, tt_stream_t stream) {
  if (n_rows > 0 && n_rows <= TT_MAX_IDS && (!d_lse || !d_dlogits)) return TT_ERR_INVALID_ARG;
  const LossArgs a{n_vocab, logits_stride, dlogits_stride, d_targets, nullptr, nullptr, d_lse, d_row_grads, d_status, 1, 0};
  return run_loss(d_logits, type, n_rows, a, d_dlogits, stream, "tt_token_loss_grad");
}
