// tt_distill.cu - distillation from a teacher's top logits: the Kullback-Leibler
// divergence of each row of logits from them, and its gradient (include/toktier.h).
//
//   q = softmax of the row's teacher logits over the temperature T
//   lse = M / T + log(S),  S = sum_j exp((l_j - M) / T)
//   loss = sum_k q_k (log q_k - (l_id(k) - M) / T + log(S))
//   dl_j = g / T (exp((l_j - M) / T) / S - sum of q_k over the k with id(k) = j)
//
// Bound by memory, like the next-token loss: a row is read once into the shared
// memory of a cluster of blocks, summed on the way with a running maximum, and
// turned into gradients from there.  The teacher's entries (at most 1024) stay beside
// it: each block has their shares q, and the logits of those that lie in its part of
// the row.  The gradient of the whole part is written first, without q, and each thread
// then writes the entries' places among those that it wrote once more: lists say which
// those are.  (By the threads that had the entries, behind a barrier, 4096 x 100256 bf16
// with 64 entries took 326 us; 302 so.)
//
// With gradients 4096 x 100256 bfloat16 and 64 entries take 302 us (1.64 GB, 80% of the
// measured copy bandwidth; the next-token loss 288) and 1023 x 200255 floats and 37 entries
// 303; the loss alone 140 us (86%), the gradient from lse 255.  What it takes beyond the
// next-token loss is some 1500 cycles a block between reading and writing: the entries'
// shares, their logits and two more sums over the warps.
#include <algorithm>

#include "tt_rows.cuh"

using namespace tt::ops;

namespace {

constexpr int SPACE = 112 * 1024;                // bytes of shared memory of a block: two blocks an SM
constexpr int HELD = 104 * 1024;                 // the most of them for a row
constexpr int U = 4;                             // vectors a thread takes at a time
constexpr int UC = 4, AHEAD = 4;                 // vectors a group of copies, groups ahead

struct DistillArgs {
  int64_t n_vocab, logits_stride, dlogits_stride, ids_stride, values_stride;
  const int32_t *ids;
  const void *values;
  int32_t values_type;
  int k;                                         // entries a row
  float inv_t, c;                                // 1 / T and log2(e) / T
  float *loss, *lse_out;
  const float *lse_in, *row_grads;
  int32_t *status;
  int cluster, held;                             // blocks a row, vectors a block can hold
};

__device__ __forceinline__ float value_of(const DistillArgs &a, int64_t row, int i) {
  const int64_t at = row * a.values_stride + i;
  if (a.values_type == TT_F32) return reinterpret_cast<const float *>(a.values)[at];
  if (a.values_type == TT_F16) return to_f32(reinterpret_cast<const __half *>(a.values)[at]);
  return to_f32(reinterpret_cast<const __nv_bfloat16 *>(a.values)[at]);
}

// The maximum and sum of a warp's, or of n entries of an array: the maximum first, so
// that no sum waits for another.  (Joined in turn, what stands between reading a row and
// writing its gradient took twice as long.)
__device__ __forceinline__ float warp_top(float m) {
  float top;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(top) : "f"(m));
  return top;
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
  return v;
}
__device__ __forceinline__ float2 warp_join(const Running<true> &r) {
  const float top = warp_top(r.m);
  return make_float2(top, warp_sum(r.s * ex2((r.m - top) * r.c)));
}
template <int N> __device__ __forceinline__ float2 join_all(const float2 *p, int n, float c) {
  float top = LOWEST, s = 0;
#pragma unroll
  for (int i = 0; i < N; ++i)
    if (i < n) top = fmaxf(top, p[i].x);
#pragma unroll
  for (int i = 0; i < N; ++i)
    if (i < n) s += p[i].y * ex2((p[i].x - top) * c);
  return make_float2(top, s);
}

// GRAD: 0 the loss alone, 1 with its gradient, 2 the gradient from lse
// Threads an SM that registers are kept for: without the gradient, and for short rows, more
// blocks hide each other's ends (4096 x 100256 bf16 without gradient, k 64: 158 us with
// 1024 threads, 146 with 1280, 140 with 1536; 32768 x 4352 with it 211, 202, 202; long
// rows with it are held two blocks an SM, whatever the registers).
template <class T, int GRAD, int THREADS>
__global__ void __launch_bounds__(THREADS, (GRAD && THREADS == 256 ? 1024 : 1536) / THREADS) k_distill(DistillArgs a, const T *logits, T *dlogits) {
  constexpr int E = RowParts<T>::E, WARPS = THREADS / 32;
  extern __shared__ uint4 s_row[];
  int32_t *s_id = reinterpret_cast<int32_t *>(s_row + a.held);              // [k] the entries' IDs, -1: none
  float *s_q = reinterpret_cast<float *>(s_id + a.k), *s_x = s_q + a.k;     // [k] shares and logits
  int32_t *s_next = reinterpret_cast<int32_t *>(s_x + a.k);                 // [k] with the gradient: the next one in a thread's list
  __shared__ float2 s_warp[2][WARPS];
  __shared__ float2 s_blocks[8], s_terms[8 * WARPS];                        // what blocks tell all others, and warps the first block
  __shared__ int32_t s_list[THREADS];
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
  const float g_row = GRAD && a.row_grads ? a.row_grads[row] : 1.f;

  // The teacher's entries, and the maximum and sum of their softmax.  A thread's first
  // entry is on its way while the row is summed.
  Running<true> teacher, run;
  teacher.c = run.c = a.c;
  const int32_t *ids = a.ids + row * a.ids_stride;
  const int lo = part.lead + first * E, hi = lo + n * E;                    // this block's part of the row
  auto in_part = [&](int id) { return (id >= lo && id < hi) || (rank == 0 && (id < part.lead || id >= part.lead + part.vecs * E)); };
  float x0 = 0;
  const int id0 = tid < a.k ? ids[tid] : -1;
  const float value0 = tid < a.k ? value_of(a, row, tid) : 0.f;
  auto take = [&](int i, int id, float value) {
    if (id >= a.n_vocab) {
      if (rank == 0) op_status(a.status, TT_ERR_INVALID_ARG);
      id = -1;
    }
    s_id[i] = max(id, -1);
    s_q[i] = value;
    if (id >= 0) teacher.add(value);
  };
  if (GRAD) s_list[tid] = -1;
  if (GRAD != 2) {
    if (GRAD == 1)
      groups<THREADS>(0, n_held, UC, [&](int v0, auto whole) {
        copy_wait<AHEAD - 1>();
        fetch(v0 + AHEAD * UC * THREADS);
#pragma unroll
        for (int u = 0; u < UC; ++u)
          if (whole.value || v0 + u * THREADS < n_held) run.add(s_row[v0 + u * THREADS], T{});
      });
    auto sum = [&](int from, int to) {
      groups<THREADS>(from, to, U, [&](int v0, auto whole) {
        uint4 r[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (whole.value || v0 + u * THREADS < to) r[u] = __ldcs(body + v0 + u * THREADS);
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (whole.value || v0 + u * THREADS < to) run.add(r[u], T{});
      });
    };
    if (GRAD == 0) {
      // the logit of the thread's first entry is asked for when its ID is there, halfway
      const int half = n / 2 / (U * THREADS) * (U * THREADS);
      sum(0, half);
      if (tid < a.k && id0 >= 0 && id0 < a.n_vocab && in_part(id0)) x0 = to_f32(l[id0]);
      sum(half, n);
    } else {
      sum(n_held, n);
    }
    if (lone >= 0) run.add(x);
  }
  if (tid < a.k) take(tid, id0, value0);
  for (int i = tid + THREADS; i < a.k; i += THREADS) take(i, ids[i], value_of(a, row, i));
  run.total();
  teacher.total();
  float2 mine = warp_join(run), theirs = warp_join(teacher);
  if (lane == 0) {
    s_warp[0][warp] = mine;
    s_warp[1][warp] = theirs;
  }
  __syncthreads();                               // (a thread's copies are there, and so are all others')
  mine = join_all<WARPS>(s_warp[0], WARPS, a.c);
  theirs = join_all<WARPS>(s_warp[1], WARPS, a.c);
  const bool none = theirs.y == 0;               // nothing that the teacher gives any weight to

  // The shares of the entries in this block's part of the row, which each of them lies in
  // one block's of, and their terms of the loss, against this block's maximum.  The
  // logits are read before any block can write to the row, from what is held if they are.
  const float log_mass = logf(theirs.y), one = __fdividef(1.f, theirs.y);
  float2 terms = make_float2(0, 0);              // the loss's, and the shares
  for (int i = tid; i < a.k; i += THREADS) {
    const int id = s_id[i];
    if (id < 0) continue;
    const float above = s_q[i] - theirs.x, q = ex2(above * a.c) * one;
    s_q[i] = q;
    if (!in_part(id)) continue;
    const float xi = GRAD == 0 && i == tid                             ? x0
                     : id >= lo && (id - lo) / E < n_held ? to_f32(reinterpret_cast<const T *>(s_row)[id - lo])
                                                          : to_f32(l[id]);
    s_x[i] = xi;
    if (GRAD) {
      // the entry goes to the thread that will write its place in the gradient
      const int v = (id - lo) / E;
      const int owner = id >= lo && id < hi ? (v < n_held ? v : v - n_held) % THREADS : id < part.lead ? id : 16 + id - part.lead - part.vecs * E;
      s_next[i] = atomicExch(&s_list[owner], i);
    }
    if (GRAD != 2 && q != 0) {
      terms.x += q * (above * a.inv_t - log_mass - (xi - mine.x) * a.inv_t);
      terms.y += q;
    }
  }
  float lse, from, log_s = 0, inverse = 1.f;     // probabilities are 2^(c (l - from)) * inverse
  if (GRAD == 2) {
    lse = a.lse_in[row];
    from = 0;
    __syncthreads();                             // the lists are complete
  } else {
    if (warp * 32 < a.k) terms = make_float2(warp_sum(terms.x), warp_sum(terms.y));
    if (a.cluster > 1) {
      cluster_wait();                            // all blocks have begun
      if (tid < a.cluster) *of_block(&s_blocks[rank], tid) = mine;
      if (lane == 0) *of_block(&s_terms[rank * WARPS + warp], 0) = terms;
      cluster_arrive();
      cluster_wait();
    } else {
      if (tid == 0) s_blocks[0] = mine;
      if (lane == 0) s_terms[warp] = terms;
      __syncthreads();
    }
    const float2 all = join_all<8>(s_blocks, a.cluster, a.c);
    log_s = logf(all.y);
    from = all.x;
    inverse = __fdividef(1.f, all.y);            // of 1 .. 2^20
    lse = all.y == 0 ? -INF : all.x * a.inv_t + log_s;
  }
  // the row's loss, by the warp that is likely to have least to do
  auto report = [&]() {
    float loss = 0;
    for (int i = lane; i < a.cluster * WARPS; i += 32) {
      const float2 t = s_terms[i];
      if (t.y != 0) loss += t.x + t.y * ((from - s_blocks[i / WARPS].x) * a.inv_t);
    }
    loss = warp_sum(loss);
    if (lane == 0) {
      if (a.lse_out) a.lse_out[row] = lse;
      a.loss[row] = none ? 0.f : lse == -INF ? INF : loss + log_s;
    }
  };
  if (GRAD == 0 && rank == 0 && warp == WARPS - 1) report();
  if (GRAD) {
    T *d = dlogits + row * a.dlogits_stride;
    const bool zero = none || lse == -INF;
    const float g = zero ? 0.f : g_row * a.inv_t, shift = GRAD == 2 ? lse * LOG2E : 0.f, factor = g * inverse;
    // 2^(c (l - from)), or from lse 2^(c l - lse log2(e))
    auto power = [&](float v) { return GRAD == 2 ? ex2(fmaf(v, a.c, -shift)) : ex2((v - from) * a.c); };
    const bool same = ((reinterpret_cast<uintptr_t>(d) ^ reinterpret_cast<uintptr_t>(l)) & 15) == 0;
    T *out = d + part.lead + (int64_t)first * E;
    auto write = [&](uint4 r, int vi) {
      float v[E];
      vec_f32(r, v, T{});
#pragma unroll
      for (int i = 0; i < E; i += 2) {
        float2 y;
        if (GRAD == 2) {
          y = make_float2(power(v[i]), power(v[i + 1]));
        } else {
          y = sub_mul2(make_float2(v[i], v[i + 1]), from, a.c);
          y = make_float2(ex2(y.x), ex2(y.y));
        }
        y = mul2(y, factor);
        v[i] = y.x;
        v[i + 1] = y.y;
      }
      if (zero)
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
    if (lone >= 0) d[lone] = from_f32<T>(zero ? 0.f : power(x) * factor);
    if (GRAD == 1 && rank == 0 && warp == WARPS - 1) report();
    if (zero) return;
    // The entries whose places this thread has written (the exchange above lies behind
    // all that is read here).  All of an ID's are in the same list, and nearly always it
    // is one; if not, their shares are added up in the entries' order, once.
    for (int i = s_list[tid]; i >= 0; i = s_next[i]) {
      const int id = s_id[i];
      if (id < 0) continue;                      // done
      float q = s_q[i];
      bool twice = false;
      for (int e = s_next[i]; e >= 0 && !twice; e = s_next[e]) twice = s_id[e] == id;
      if (twice) {
        q = 0;
        for (int e = 0; e < a.k; ++e)
          if (s_id[e] == id) {
            q += s_q[e];
            s_id[e] = -1;
          }
      }
      d[id] = from_f32<T>((power(s_x[i]) * inverse - q) * g);
    }
  }
}

template <class T, int GRAD, int THREADS> struct Tag {};

template <class T, int GRAD, int THREADS>
void run_rows_by(DistillArgs a, int64_t n_rows, const void *logits, void *dlogits, tt_stream_t stream) {
  const int64_t bytes = a.n_vocab * (int64_t)sizeof(T);
  // the same blocks a row, and the same order of its sums, with the gradient and without
  const int extra = a.k * 16;
  const int held = std::min(HELD, SPACE - extra) / (16 * THREADS) * (16 * THREADS);
  a.cluster = (int)std::min<int64_t>(8, (bytes + held - 1) / held);
  // few rows: spread each over more blocks, down to 16 KB a block, as for the next-token loss
  while (a.cluster <= 4 && n_rows * a.cluster * 2 <= 2 * 152 && bytes >= a.cluster * 2 * 16384) a.cluster *= 2;
  const int64_t each = ((bytes + 15) / 16 + a.cluster - 1) / a.cluster;
  a.held = GRAD == 1 ? (int)std::min<int64_t>(each, held / 16) : 0;
  auto k = k_distill<T, GRAD, THREADS>;
  if (allow_shared<Tag<T, GRAD, THREADS>>(k, SPACE)) return;                // (the error is kept)
  launch_cluster(k, dim3((unsigned)(n_rows * a.cluster)), THREADS, (size_t)a.held * 16 + extra, a.cluster, false, stream, a,
                 (const T *)logits, (T *)dlogits);
}

// block sizes by the row's bytes, as for the next-token loss (tt_loss.cu has the table)
template <class T, int GRAD> void run_rows(const DistillArgs &a, int64_t n_rows, const void *logits, void *dlogits, tt_stream_t stream) {
  const int64_t bytes = a.n_vocab * (int64_t)sizeof(T);
  if (bytes <= 4096) run_rows_by<T, GRAD, 32>(a, n_rows, logits, dlogits, stream);
  else if (bytes <= 32768) run_rows_by<T, GRAD, 128>(a, n_rows, logits, dlogits, stream);
  else run_rows_by<T, GRAD, 256>(a, n_rows, logits, dlogits, stream);
}

tt_status run_distill(const void *d_logits, int32_t type, int64_t n_rows, int64_t k, float temperature, DistillArgs a, void *d_dlogits,
                      tt_stream_t stream, const char *what) {
  if (!type_ok(type) || !type_ok(a.values_type) || n_rows < 0 || !vocab_ok(a.n_vocab) || a.logits_stride < a.n_vocab ||
      (d_dlogits && a.dlogits_stride < a.n_vocab) || k < 1 || k > TT_MAX_TEACHER || a.ids_stride < k || a.values_stride < k ||
      !(temperature >= 0x1p-64f && temperature <= 0x1p64f) || !optional_ok(a.status, 4) || !optional_ok(a.row_grads, 4) ||
      !optional_ok(a.lse_out, 4) || !optional_ok(a.lse_in, 4) || !optional_ok(a.loss, 4) ||
      !optional_ok(d_dlogits, type_size(type)) || (d_dlogits == d_logits && d_logits && a.dlogits_stride != a.logits_stride))
    return TT_ERR_INVALID_ARG;
  if (n_rows > TT_MAX_IDS) return TT_ERR_CAPACITY;
  if (n_rows == 0) return TT_OK;
  if (!array_ok(d_logits, type_size(type)) || !array_ok(a.ids, 4) || !array_ok(a.values, type_size(a.values_type))) return TT_ERR_INVALID_ARG;
  if (!a.lse_in && !a.loss) return TT_ERR_INVALID_ARG;
  a.k = (int)k;
  a.inv_t = 1.f / temperature;
  a.c = (float)(1.4426950408889634 / temperature);
  with_type(type, [&](auto t) {
    using T = decltype(t);
    if (a.lse_in) run_rows<T, 2>(a, n_rows, d_logits, d_dlogits, stream);
    else if (d_dlogits) run_rows<T, 1>(a, n_rows, d_logits, d_dlogits, stream);
    else run_rows<T, 0>(a, n_rows, d_logits, nullptr, stream);
  });
  return launched(what);
}

}  // namespace

extern "C" tt_status tt_distill_loss(const void *d_logits, int32_t type, int64_t n_rows, int64_t n_vocab, int64_t logits_stride,
                                     const int32_t *d_teacher_ids, int64_t ids_stride, const void *d_teacher_logits,
                                     int32_t teacher_type, int64_t teacher_stride, int64_t k, float temperature, float *d_loss,
                                     float *d_lse, const float *d_row_grads, void *d_dlogits, int64_t dlogits_stride,
                                     int32_t *d_status, tt_stream_t stream) {
  const DistillArgs a{n_vocab, logits_stride, dlogits_stride, ids_stride, teacher_stride, d_teacher_ids, d_teacher_logits, teacher_type,
                      0, 0, 0, d_loss, d_lse, nullptr, d_row_grads, d_status, 1, 0};
  return run_distill(d_logits, type, n_rows, k, temperature, a, d_dlogits, stream, "tt_distill_loss");
}

extern "C" tt_status tt_distill_loss_grad(const void *d_logits, int32_t type, int64_t n_rows, int64_t n_vocab, int64_t logits_stride,
                                          const int32_t *d_teacher_ids, int64_t ids_stride, const void *d_teacher_logits,
                                          int32_t teacher_type, int64_t teacher_stride, int64_t k, float temperature,
                                          const float *d_lse, const float *d_row_grads, void *d_dlogits, int64_t dlogits_stride,
                                          int32_t *d_status, tt_stream_t stream) {
  if (n_rows > 0 && n_rows <= TT_MAX_IDS && (!d_lse || !d_dlogits)) return TT_ERR_INVALID_ARG;
  const DistillArgs a{n_vocab, logits_stride, dlogits_stride, ids_stride, teacher_stride, d_teacher_ids, d_teacher_logits, teacher_type,
                      0, 0, 0, nullptr, nullptr, d_lse, d_row_grads, d_status, 1, 0};
  return run_distill(d_logits, type, n_rows, k, temperature, a, d_dlogits, stream, "tt_distill_loss_grad");
}
