// tt_loss.cu - next-token loss of rows of logits and its gradient
// (include/toktier.h).
#include "tt_ops.cuh"

using namespace tt::ops;

namespace {

struct LossArgs {
  int64_t n_vocab, logits_stride, dlogits_stride;
  const int32_t *targets;
  float *loss, *lse_out;
  const float *lse_in, *row_grads;
  int32_t *status;
};

// a block a row: the maximum, the sum of exp(l - M), then the gradient
template <class T>
__global__ void __launch_bounds__(512) k_loss(LossArgs a, const T *logits, T *dlogits) {
  __shared__ float box[16];
  const int64_t row = blockIdx.x;
  const T *l = logits + row * a.logits_stride;
  const int32_t t = a.targets[row];
  const bool there = (uint32_t)t < (uint32_t)a.n_vocab;
  if (!there && t >= 0 && threadIdx.x == 0) op_status(a.status, TT_ERR_INVALID_ARG);
  const float lt = there ? to_f32(l[t]) : 0.f;
  float lse;
  if (a.lse_in) {
    lse = a.lse_in[row];
  } else {
    float m = -INF, s = 0;
    bool nan = false;
    for (int64_t j = threadIdx.x; j < a.n_vocab; j += 512) {
      const float x = to_f32(l[j]);
      nan |= x != x;
      m = fmaxf(m, x);
    }
    m = block_all(m, OpMax(), box);
    nan = __syncthreads_or(nan);
    const float ref = fabsf(m) == INF ? 0.f : m;
    for (int64_t j = threadIdx.x; j < a.n_vocab; j += 512) s += expf(to_f32(l[j]) - ref);
    s = block_all(s, OpSum(), box);
    lse = nan ? NAN : fabsf(m) == INF ? m : m + logf(s);
    if (threadIdx.x == 0) {
      if (a.lse_out) a.lse_out[row] = lse;
      a.loss[row] = !there ? 0.f : lse == -INF ? INF : lse - lt;
    }
  }
  if (!dlogits) return;
  __syncthreads();
  T *d = dlogits + row * a.dlogits_stride;
  const float g = a.row_grads ? a.row_grads[row] : 1.f;
  const bool none = !there || lse == -INF;
  for (int64_t j = threadIdx.x; j < a.n_vocab; j += 512)
    d[j] = from_f32<T>(none ? 0.f : g * (expf(to_f32(l[j]) - lse) - (j == t ? 1.f : 0.f)));
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
    k_loss<T><<<(unsigned)n_rows, 512, 0, stream>>>(a, (const T *)d_logits, (T *)d_dlogits);
  });
  return launched(what);
}

}  // namespace

extern "C" tt_status tt_token_loss(const void *d_logits, int32_t type, int64_t n_rows, int64_t n_vocab,
                                   int64_t logits_stride, const int32_t *d_targets, float *d_loss, float *d_lse,
                                   const float *d_row_grads, void *d_dlogits, int64_t dlogits_stride,
                                   int32_t *d_status, tt_stream_t stream) {
  const LossArgs a{n_vocab, logits_stride, dlogits_stride, d_targets, d_loss, d_lse, nullptr, d_row_grads, d_status};
  return run_loss(d_logits, type, n_rows, a, d_dlogits, stream, "tt_token_loss");
}

extern "C" tt_status tt_token_loss_grad(const void *d_logits, int32_t type, int64_t n_rows, int64_t n_vocab,
                                        int64_t logits_stride, const int32_t *d_targets, const float *d_lse,
                                        const float *d_row_grads, void *d_dlogits, int64_t dlogits_stride,
                                        int32_t *d_status, tt_stream_t stream) {
  if (n_rows > 0 && n_rows <= TT_MAX_IDS && (!d_lse || !d_dlogits)) return TT_ERR_INVALID_ARG;
  const LossArgs a{n_vocab, logits_stride, dlogits_stride, d_targets, nullptr, nullptr, d_lse, d_row_grads, d_status};
  return run_loss(d_logits, type, n_rows, a, d_dlogits, stream, "tt_token_loss_grad");
}
