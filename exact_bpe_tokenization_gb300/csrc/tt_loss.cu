// tt_loss.cu - next-token loss of rows of logits and its gradient
// (include/toktier.h).
//
//   lse = M + log(S),  S = sum_j exp(l_j - M),  loss = (M - l_t) + log(S),
//   dl_j = g * (exp(l_j - lse) - (j == t))
//
// lse is rounded to 32 bits, by up to 2^-24 of itself, which every probability
// taken from it is off by: 5e-7 at lse = 15.  That is the gradient's error, so that
// it has the same bits whether it comes with the loss or from lse later, as long
// as lse stays below FAR; above, log(S) would soon be lost in it (a row of the
// type's lowest value would get probabilities of 1), and the gradient that comes
// with the loss is exp(l_j - M) / S instead.  The loss never goes through lse.
//
// Bound by memory: each logit has to be read and each gradient written once.
// The gradient needs lse, which needs the whole row, so a row is read, kept in
// shared memory, and turned into gradients from there: a cluster of blocks
// holds a row (two blocks an SM, so that one reads or writes while the other
// computes).  What does not fit (rows above 832 KB) is read again, from L2.
//
// With gradients 4096 x 100256 bfloat16 take 287 us (1.64 GB, 84% of the measured
// copy bandwidth) and 1023 x 200255 floats 291 us (83%); in place 306 us either,
// the loss alone 129 and 137, and the gradient from lse 240 us, the time of a copy
// of as many bytes.  A block reads, waits
// for its cluster, and writes; its neighbour on the SM fills the wait, and not
// all of it.  Rows of that size need clusters of 8, which leave a few SMs of
// each group of them idle, but hold the row: with 4 blocks a row, half of it
// comes from L2 a second time, and 323 us became 370 when that was tried.
//
// Gradients whose rows lie otherwise against 16 bytes than the logits' are written
// an element at a time: rows of 100,257 cut from 100,352 bfloat16 take 286 us into
// gradients of the same stride and 817 into contiguous ones.
#include <algorithm>

#include "tt_rows.cuh"

using namespace tt::ops;

namespace {

constexpr int HELD = 104 * 1024;                 // bytes of a row a block holds: two blocks an SM
constexpr float FAR = 128.f;                     // |lse| from where a probability would be off by 2^-18

struct LossArgs {
  int64_t n_vocab, logits_stride, dlogits_stride;
  const int32_t *targets;
  float *loss, *lse_out;
  const float *lse_in, *row_grads;
  int32_t *status;
  int cluster, held;                             // blocks a row, vectors a block can hold
};

// GRAD: 0 the loss alone, 1 with its gradient, 2 the gradient from lse
constexpr int U = 4;                             // vectors a thread takes at a time
constexpr int UC = 4, AHEAD = 4;                 // vectors a group of copies, groups ahead

template <class T, int GRAD, int THREADS>
__global__ void __launch_bounds__(THREADS, 1024 / THREADS) k_loss(LossArgs a, const T *logits, T *dlogits) {
  constexpr int E = RowParts<T>::E, WARPS = THREADS / 32;
  extern __shared__ uint4 s_row[];
  __shared__ float2 s_warp[WARPS], s_blocks[8];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = a.cluster > 1 ? (int)cluster_rank() : 0;
  if (GRAD != 2 && a.cluster > 1) cluster_arrive();
  const int64_t row = blockIdx.x / a.cluster;
  const T *l = logits + row * a.logits_stride;
  const RowParts<T> part(l, (int)a.n_vocab);
  const int each = (part.vecs + a.cluster - 1) / a.cluster, first = min(part.vecs, rank * each);
  const int n = min(part.vecs - first, each), n_held = GRAD == 1 ? min(n, a.held) : 0;
  const uint4 *body = reinterpret_cast<const uint4 *>(l + part.lead) + first;
  // what is held comes by copies that run ahead; a thread reads its own
  auto fetch = [&](int v0) {
    if (v0 - tid + UC * THREADS <= n_held) {
#pragma unroll
      for (int u = 0; u < UC; ++u) copy_async(s_row + v0 + u * THREADS, body + v0 + u * THREADS);
    } else {
#pragma unroll
      for (int u = 0; u < UC; ++u)
        if (v0 + u * THREADS < n_held) copy_async(s_row + v0 + u * THREADS, body + v0 + u * THREADS);
    }
    copy_group();
  };
  if (GRAD == 1) {
#pragma unroll
    for (int d = 0; d < AHEAD; ++d) fetch(tid + d * UC * THREADS);
  }
  const int lone = rank == 0 ? part.scalar(tid) : -1;
  const float x = lone >= 0 ? to_f32(l[lone]) : -INF;
  const int32_t t = a.targets[row];
  const float g_row = GRAD && a.row_grads ? a.row_grads[row] : 1.f;        // (here, so that it is there behind the barrier)
  const bool there = (uint32_t)t < (uint32_t)a.n_vocab;
  if (!there && t >= 0 && rank == 0 && tid == 0) op_status(a.status, TT_ERR_INVALID_ARG);

  float lse, from, inverse = 1.f;                // probabilities are exp(l - from) * inverse
  if (GRAD == 2) {
    lse = from = a.lse_in[row];
  } else {
    // read by one thread, before any block can write to the row
    const float lt = there && rank == 0 && tid == 0 ? to_f32(l[t]) : 0.f;
    Running<false> run;
    if (GRAD == 1)
      groups<THREADS>(0, n_held, UC, [&](int v0, auto whole) {
        copy_wait<AHEAD - 1>();
        fetch(v0 + AHEAD * UC * THREADS);
#pragma unroll
        for (int u = 0; u < UC; ++u)
          if (whole.value || v0 + u * THREADS < n_held) run.add(s_row[v0 + u * THREADS], T{});
      });
    groups<THREADS>(n_held, n, U, [&](int v0, auto whole) {
      uint4 r[U];
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (whole.value || v0 + u * THREADS < n) r[u] = __ldcs(body + v0 + u * THREADS);
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (whole.value || v0 + u * THREADS < n) run.add(r[u], T{});
    });
    if (lone >= 0) run.add(x);
    run.total();
#pragma unroll
    for (int o = 16; o; o >>= 1) run.join(__shfl_xor_sync(~0u, run.m, o), __shfl_xor_sync(~0u, run.s, o));
    if (lane == 0) s_warp[warp] = make_float2(run.m, run.s);
    __syncthreads();
    run.m = LOWEST;
    run.s = 0;
    for (int w = 0; w < WARPS; ++w) run.join(s_warp[w].x, s_warp[w].y);
    if (a.cluster > 1) {
      // written to all blocks ahead of the barrier, so that nothing has to be fetched behind it
      cluster_wait();                            // all blocks have begun
      if (tid < a.cluster) *of_block(&s_blocks[rank], tid) = make_float2(run.m, run.s);
      cluster_sync();
      run.m = LOWEST;
      run.s = 0;
      for (int b = 0; b < a.cluster; ++b) run.join(s_blocks[b].x, s_blocks[b].y);
    }
    const float log_s = logf(run.s);
    lse = from = run.m + log_s;
    if (fabsf(lse) >= FAR && fabsf(lse) < INF) {
      from = run.m;
      inverse = __fdividef(1.f, run.s);         // of 1 .. 2^20
    }
    if (rank == 0 && tid == 0) {
      if (a.lse_out) a.lse_out[row] = lse;
      a.loss[row] = !there ? 0.f : lse == -INF ? INF : (run.m - lt) + log_s;
    }
  }
  if (GRAD) {
    T *d = dlogits + row * a.dlogits_stride;
    const bool none = !there || lse == -INF;
    const float g = none ? 0.f : g_row, g_inverse = g * inverse;
    const bool same = ((reinterpret_cast<uintptr_t>(d) ^ reinterpret_cast<uintptr_t>(l)) & 15) == 0;
    T *out = d + part.lead + (int64_t)first * E;
    // the thread that has the target among its vectors writes it once more behind them
    const int at = t - part.lead - first * E;
    const bool held = at / E < n_held, mine = there && at >= 0 && at / E < n && (at / E - (held ? 0 : n_held)) % THREADS == tid;
    const float xt = mine ? to_f32(l[t]) : 0.f;
    auto write = [&](uint4 r, int vi) {
      float v[E];
      vec_f32(r, v, T{});
#pragma unroll
      for (int i = 0; i < E; i += 2) {
        float2 y = sub_mul2(make_float2(v[i], v[i + 1]), from, LOG2E);
        y.x = ex2(y.x);
        y.y = ex2(y.y);
        y = mul2(y, g_inverse);
        v[i] = y.x;
        v[i + 1] = y.y;
      }
      if (none)
#pragma unroll
        for (int i = 0; i < E; ++i) v[i] = 0;
      T *to = out + (int64_t)vi * E;
      if (same) {
        __stcs(reinterpret_cast<uint4 *>(to), f32_vec(v, T{}));
      } else {
#pragma unroll
        for (int i = 0; i < E; ++i) to[i] = from_f32<T>(v[i]);
      }
    };
    groups<THREADS>(0, n_held, U, [&](int v0, auto whole) {
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (whole.value || v0 + u * THREADS < n_held) write(s_row[v0 + u * THREADS], v0 + u * THREADS);
    });
    groups<THREADS>(n_held, n, U, [&](int v0, auto whole) {
      uint4 r[U];
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (whole.value || v0 + u * THREADS < n) r[u] = __ldcs(body + v0 + u * THREADS);
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (whole.value || v0 + u * THREADS < n) write(r[u], v0 + u * THREADS);
    });
    if (mine) d[t] = from_f32<T>(none ? 0.f : (ex2((xt - from) * LOG2E) * inverse - 1.f) * g);
    if (lone >= 0) d[lone] = from_f32<T>(none ? 0.f : (ex2((x - from) * LOG2E) * inverse - (lone == t ? 1.f : 0.f)) * g);
  }
}

template <class T, int GRAD, int THREADS> struct Tag {};

template <class T, int GRAD, int THREADS>
void run_rows_by(LossArgs a, int64_t n_rows, const void *logits, void *dlogits, tt_stream_t stream) {
  const int64_t bytes = a.n_vocab * (int64_t)sizeof(T);
  a.cluster = (int)std::min<int64_t>(8, (bytes + HELD - 1) / HELD);
  // few rows: spread each over more blocks, down to 16 KB a block (1 x 100256
  // bfloat16 7.8 us to 4.9, 16 rows 8.1 to 5.9, 64 rows 8.2 both ways; four blocks
  // an SM instead of two make those 9.0)
  while (a.cluster <= 4 && n_rows * a.cluster * 2 <= 2 * 152 && bytes >= a.cluster * 2 * 16384) a.cluster *= 2;
  const int64_t each = ((bytes + 15) / 16 + a.cluster - 1) / a.cluster;
  a.held = GRAD == 1 ? (int)std::min<int64_t>(each, HELD / 16) : 0;
  auto k = k_loss<T, GRAD, THREADS>;
  const size_t shared = (size_t)a.held * 16;
  if (GRAD == 1 && allow_shared<Tag<T, GRAD, THREADS>>(k, HELD)) return;     // (the error is kept)
  launch_cluster(k, dim3((unsigned)(n_rows * a.cluster)), THREADS, shared, a.cluster, false, stream, a, (const T *)logits, (T *)dlogits);
}

// A short row is little work behind a block's start, its barrier and its end, so
// that small blocks, of which more share an SM, are faster.  Rows and gradients
// in bfloat16, us for 32, 128, 256, 512 threads, when this was chosen:
//   32768 x   257     23    79   161   378
//   32768 x  1024     33    85   166   387
//   32768 x  4096     88   119   193   406
//   32768 x  8192    182   165   236   451
//    4096 x 16384     70    47    48    78
//    4096 x 24000    120    70    62    88
//    4096 x 50257    426   174   139   139
//    4096 x 100256   855   359   291   290
// (32-bit rows, and fewer of them, divide at about the same bytes.)
template <class T, int GRAD> void run_rows(const LossArgs &a, int64_t n_rows, const void *logits, void *dlogits, tt_stream_t stream) {
  const int64_t bytes = a.n_vocab * (int64_t)sizeof(T);
  if (bytes <= 4096) run_rows_by<T, GRAD, 32>(a, n_rows, logits, dlogits, stream);
  else if (bytes <= 32768) run_rows_by<T, GRAD, 128>(a, n_rows, logits, dlogits, stream);
  else run_rows_by<T, GRAD, 256>(a, n_rows, logits, dlogits, stream);
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
