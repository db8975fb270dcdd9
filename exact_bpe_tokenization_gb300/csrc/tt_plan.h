// tt_plan.h - how a call of tt_linear_loss is cut up: tiles of its products, parts of
// their contractions, chunks of rows, and what lies where in the workspace; and when a
// wait within a kernel has run out.  Arithmetic alone, which tests compile without CUDA.
#pragma once
#include <stdint.h>

#include <algorithm>

#include "../../include/toktier.h"

namespace tt {
namespace gemm {

constexpr int TILE = 256, HALF = 128, KB = 64;            // rows and columns of a tile, a block's part, contraction a stage
constexpr int SMS = 152;

// How long a wait within a kernel has taken, from looks at a clock that goes on while the
// kernel does not run (a context switched out, a debugger, a machine put to sleep): a gap
// between two looks counts for a quarter of a second at most, so that a wait of which nobody
// looked for minutes has not run out.
constexpr uint64_t PATIENCE = 4000000000ull, GAP = PATIENCE / 16;  // nanoseconds
#ifdef __CUDACC__
#define TT_BOTH __host__ __device__ __forceinline__
#else
#define TT_BOTH inline
#endif
struct Patience {
  uint64_t last, waited;
  TT_BOTH explicit Patience(uint64_t now) : last(now), waited(0) {}
  TT_BOTH bool over(uint64_t now) {
    const uint64_t gap = now - last;
    waited += gap < GAP ? gap : GAP;
    last = now;
    return waited > PATIENCE;
  }
};

inline int64_t up(int64_t x, int64_t to) { return (x + to - 1) / to * to; }

inline int pairs_of(int a, int b) { return a == 3 ? 6 : a + b - 1; }

// Parts to cut a contraction into, so that every pair of SMs has as much to do: the
// least of the rounds of tiles, each of its blocks and a tile's start and end, and the
// traffic of the parts (times in blocks of 64, 0.27 us).  What it chooses, against one part and
// the best other number tried of 2, 3, 4 and 8, in us of a call from lse: dhidden of 1023 x 20001 x
// 640 bf16 59 (123; 65 with 4), of 1023 x 200255 x 641 fp16 507 (1154; 542 with 4), of 2047 x
// 4352 x 1024 floats 155 (196; 150 with 2), of 300 x 20001 x 640 floats 148 (586; 160 with 8);
// dweight of the same 60, 531, 149 and 145, which are one part's (94, 985, 159, 171 with 2).
//   The tensor cores cut off the
// sums at each step: operands of several parts, which are 32-bit values, are summed over
// no more than 2048 at a time (dhidden of 100,000 tokens was off by 1.4e-5 of its size in one
// sum, 7e-6 with 8192, 2.4e-6 so; plain 32-bit sums 2e-6).
constexpr int64_t LONGEST = 2048;
inline int choose_splits(int64_t m, int64_t n, int64_t k, int pairs) {
  const int64_t tiles = ((m + TILE - 1) / TILE) * ((n + TILE - 1) / TILE), blocks = (k + KB - 1) / KB;
  const int64_t least_splits = pairs == 6 ? (k + LONGEST - 1) / LONGEST : 1;
  const int64_t most = std::max<int64_t>(least_splits, std::min<int64_t>(std::min<int64_t>(32, blocks), blocks * pairs / 4));
  int best = (int)least_splits;
  double least = 1e300;
  for (int64_t s = least_splits; s <= most; ++s) {
    const int64_t rounds = (tiles * s + SMS / 2 - 1) / (SMS / 2);
    double cost = (double)rounds * ((double)((blocks + s - 1) / s) * pairs + 4);
    if (s > 1) cost += 12 + (double)s * m * n * 8 / 6.8e12 / 0.27e-6;
    if (cost < least * 0.99) {
      least = cost;
      best = (int)s;
    }
  }
  return best;
}

// The parts of a contraction of k that was planned for a longer one (the last chunk of
// rows is shorter): each has one block at least, since a tile without any would leave
// with what its tensor memory held before.
inline int splits_of(int planned, int64_t k) { return (int)std::min<int64_t>(planned, (k + KB - 1) / KB); }

}  // namespace gemm

namespace linear {

using namespace tt::gemm;

constexpr int64_t MAX_WIDTH = 1 << 16;
// Bytes of G at a time.  Fewer and larger chunks read and write the 32-bit sums of dweight
// less often: 16400 x 100256 x 2048 bf16 takes 12.5 ms with 1 GB, 12.1 with 2, 11.9 with 4.
constexpr int64_t KEPT = 2ll << 30;
constexpr int64_t PARTIALS = 1ll << 28;                    // bytes of maxima and sums at a time
constexpr int FEW = 64, FEW_16 = 4;                        // rows that have kernels of their own

// What a row's G is made from: G = exp(l - from) * mul - g (j == t); t < 0: zeros.
struct RowInfo { float from, mul, g; int t; };

// what lies where in the workspace, in bytes, and how the rows are cut into chunks
struct Plan {
  int64_t chunk, width, g_stride;                          // rows; columns of packed operands and of G
  int split_h, split_w;
  int64_t words;                                           // one, and one a tile row
  int64_t hidden, weight, part, rows, word, info, scaled, g, acc, sums, bytes;
};

inline bool is_few(int64_t n, int32_t type) { return n <= (type == TT_F32 ? FEW : FEW_16); }
// Parts of G, and of hidden's scaled copy.  Rounded to 16 bits once each, the gradients of few
// rows are off by up to the whole of such a rounding, where those of many rows average it;
// up to 64 rows a second part of both is nearly free.
inline int g_parts(int64_t n, int32_t type) { return type == TT_F32 || is_few(n, type) ? 3 : n <= FEW ? 2 : 1; }
inline int scaled_parts(int64_t n, int32_t type) { return type == TT_F16 && !is_few(n, type) ? 1 : g_parts(n, type); }
// tokens a block of k_few_hidden takes: two blocks an SM, whole stages, 128 at least (64 x 4352
// x 64 with all gradients, from a graph: 45 us with 256, 39 with 128)
inline int64_t few_each(int64_t vocab, int64_t dim) {
  const int64_t splits = std::max<int64_t>(1, std::min<int64_t>(2 * SMS / ((dim + 127) / 128), (vocab + 127) / 128));
  return up((vocab + splits - 1) / splits, 64);
}

inline Plan plan_of(int64_t n, int64_t vocab, int64_t dim, int32_t type, bool pack_h, bool pack_w, bool dh, bool dw, bool dw_f32) {
  Plan p{};
  if (is_few(n, type)) pack_h = pack_w = false;
  const int parts = type == TT_F32 ? 3 : 1;
  const bool grad = dh || dw;
  n = std::max<int64_t>(n, 1);
  p.width = up(dim, 64);                                   // whole 128-byte lines: a box's rows are one each
  p.g_stride = up(vocab, 64);
  const int64_t halves = (vocab + HALF - 1) / HALF;
  int64_t most = PARTIALS / (halves * 8);
  const int of_g = g_parts(n, type), of_h = scaled_parts(n, type);
  if (grad) most = std::min(most, KEPT / (p.g_stride * 2 * of_g));
  // Copies of hidden, whether or not this call needs them: the chunk comes from the sizes
  // alone, so that no call needs more than the one with copies and with both gradients,
  // which is the one that tt_linear_loss_workspace knows.
  most = std::min(most, KEPT / (p.width * 2 * parts));
  most = std::max<int64_t>(most / TILE * TILE, TILE);
  const int64_t chunks = (n + most - 1) / most;
  p.chunk = std::min(n, up((n + chunks - 1) / chunks, TILE));
  const int pairs = parts == 1 ? of_g : 6;
  p.split_h = is_few(n, type) ? (int)((vocab + few_each(vocab, dim) - 1) / few_each(vocab, dim)) : choose_splits(p.chunk, dim, vocab, pairs);
  p.split_w = choose_splits(vocab, dim, p.chunk, pairs_of(of_g, of_h));
  int64_t at = 0;
  auto take = [&](int64_t bytes) {
    const int64_t here = at;
    at += up(bytes, 256);
    return here;
  };
  p.hidden = take(pack_h ? p.chunk * p.width * 2 * parts : 0);
  p.weight = take(pack_w ? vocab * p.width * 2 * parts : 0);
  p.part = take(halves * 8 * p.chunk);
  p.rows = take(4 * 3 * p.chunk);                          // target_logit, target_power, row_scale
  p.words = 1 + (p.chunk + TILE - 1) / TILE;
  p.word = take(4 * p.words);
  if (grad) {
    p.info = take(sizeof(RowInfo) * p.chunk);
    p.scaled = take(dw ? p.chunk * p.width * 2 * of_h : 0);
    p.g = take(p.g_stride * 2 * of_g * p.chunk);
    p.acc = take(dw && !dw_f32 && p.chunk < n ? vocab * p.width * 4 : 0);
    int64_t sums = 0;
    if (dh && (p.split_h > 1 || is_few(n, type))) sums = std::max(sums, p.split_h * p.chunk * p.width * 4);
    if (dw && p.split_w > 1) sums = std::max(sums, p.split_w * vocab * p.width * 4);
    p.sums = take(sums);
  }
  p.bytes = std::max<int64_t>(at, 256);
  return p;
}

}  // namespace linear
}  // namespace tt
