// The arithmetic of csrc/tt_plan.h for the host tests.
#include "../exact_bpe_tokenization_gb300/csrc/tt_plan.h"

using namespace tt::linear;

extern "C" {

// out: rows of a chunk, parts of dhidden's and of dweight's contraction, bytes of scratch
void plan_host(int64_t n, int64_t vocab, int64_t dim, int32_t type, int pack_h, int pack_w, int dh, int dw, int dw_f32, int64_t *out) {
  const Plan p = plan_of(n, vocab, dim, type, pack_h, pack_w, dh, dw, dw_f32);
  out[0] = p.chunk;
  out[1] = p.split_h;
  out[2] = p.split_w;
  out[3] = p.bytes;
}

// the first of n looks at the clock at which a wait has run out, or n
int plan_host_patience(const uint64_t *looks, int n) {
  Patience p(looks[0]);
  for (int i = 1; i < n; ++i)
    if (p.over(looks[i])) return i;
  return n;
}

int plan_host_splits(int planned, int64_t k) { return splits_of(planned, k); }

}
