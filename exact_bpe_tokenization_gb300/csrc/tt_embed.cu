// tt_embed.cu - token embedding and its gradient (include/toktier.h).
#include <algorithm>

#include "tt_ops.cuh"

using namespace tt::ops;

namespace {

// ============================================================ tt_embed
// out[i] = scale * table[ids[i]]: no arithmetic to speak of, bound by the
// bytes of the rows read and written.
//
// Threads take groups of eight elements.  A warp takes four groups a lane at a
// time, so that four loads are in flight before the first store: of one row
// (WIDE), whose address is then worked out once, or of several rows.  Blocks take
// rows in their order and do not loop: 304,824 rows of 4096 bf16 take 423 us
// (97% of the measured copy bandwidth), and 458 us by 16 blocks an SM that go on
// to later rows, whose stores are further apart.
struct EmbedArgs {
  const int32_t *ids;
  const int64_t *n_ids;
  int64_t max_ids, n_vocab, dim, table_stride, out_stride;
  float scale;
  int lanes_log2;    // lanes that share a row
  int32_t *status;
};

template <class TI, class TO> __device__ __forceinline__ void store_scaled(TO *to, const Raw8<TI> &r, float scale) {
  float f[8];
  raw_f32(r, f);
#pragma unroll
  for (int k = 0; k < 8; k += 2) {
    const float2 y = mul2(make_float2(f[k], f[k + 1]), scale);
    f[k] = y.x;
    f[k + 1] = y.y;
  }
  store8(to, f);
}

template <class TI, class TO, bool WIDE>
__global__ void __launch_bounds__(256) k_embed(EmbedArgs a, const TI *__restrict__ table, TO *__restrict__ out) {
  constexpr int R = 4;
  const int64_t n = a.n_ids ? max((int64_t)0, min(*a.n_ids, a.max_ids)) : a.max_ids;
  const int units = (int)(a.dim >> 3), lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (WIDE) {
    const int unit = blockIdx.y * 32 * R + lane;
    const bool whole = (int)(blockIdx.y + 1) * 32 * R <= units;
    const int64_t row = (int64_t)blockIdx.x * 8 + warp;
    if (row >= n) return;
    const int32_t id = __ldg(a.ids + row);
    TO *to = out + row * a.out_stride + unit * 8;
    const bool there = (uint32_t)id < (uint32_t)a.n_vocab;
    const float scale = there ? a.scale : 0.f;    // an infinite one leaves padding zero, too
    Raw8<TI> v[R];
    if (there) {
      const TI *from = table + id * a.table_stride + unit * 8;
#pragma unroll
      for (int j = 0; j < R; ++j)
        if (whole || unit + j * 32 < units) load_raw(from + j * 256, v[j]);
    } else {
#pragma unroll
      for (int j = 0; j < R; ++j) v[j] = Raw8<TI>{};
      if (id >= 0 && unit == 0) op_status(a.status, TT_ERR_INVALID_ARG);
    }
#pragma unroll
    for (int j = 0; j < R; ++j)
      if (whole || unit + j * 32 < units) store_scaled(to + j * 256, v[j], scale);
  } else {
    const int rows_per_warp = 32 >> a.lanes_log2, unit = lane & ((1 << a.lanes_log2) - 1);
    const int64_t rows_per_block = 8 * rows_per_warp * R;
    for (int64_t row0 = blockIdx.x * rows_per_block + warp * rows_per_warp * R + (lane >> a.lanes_log2); row0 < n;
         row0 += gridDim.x * rows_per_block) {
      Raw8<TI> v[R];
      float scale[R];
#pragma unroll
      for (int j = 0; j < R; ++j) {
        const int64_t row = row0 + j * rows_per_warp;
        if (row < n && unit < units) {
          const int32_t id = __ldg(a.ids + row);
          const bool there = (uint32_t)id < (uint32_t)a.n_vocab;
          scale[j] = there ? a.scale : 0.f;
          if (there) {
            load_raw(table + id * a.table_stride + unit * 8, v[j]);
          } else {
            v[j] = Raw8<TI>{};
            if (id >= 0 && unit == 0) op_status(a.status, TT_ERR_INVALID_ARG);
          }
        }
      }
#pragma unroll
      for (int j = 0; j < R; ++j) {
        const int64_t row = row0 + j * rows_per_warp;
        if (row < n && unit < units) store_scaled(out + row * a.out_stride + unit * 8, v[j], scale[j]);
      }
    }
  }
}

// Rows that are not whole 16-byte groups: a warp a row, its lanes side by side,
// eight loads ahead of the stores: 200,000 rows of 641 floats take 160 us (6.4
// TB/s), of 641 bfloat16, at 64 bytes a warp's load, 106 us (4.8 TB/s).
template <class TI, class TO>
__global__ void __launch_bounds__(256) k_embed_any(EmbedArgs a, const TI *__restrict__ table, TO *__restrict__ out) {
  constexpr int R = 8;
  const int64_t n = a.n_ids ? max((int64_t)0, min(*a.n_ids, a.max_ids)) : a.max_ids;
  const int lane = threadIdx.x & 31, dim = (int)a.dim;
  const int64_t row = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (row >= n) return;
  const int32_t id = __ldg(a.ids + row);
  const bool there = (uint32_t)id < (uint32_t)a.n_vocab;
  if (!there && id >= 0 && lane == 0) op_status(a.status, TT_ERR_INVALID_ARG);
  const TI *src = table + (there ? id : 0) * a.table_stride;
  TO *dst = out + row * a.out_stride;
  int c = lane;
  for (; c - lane + 32 * R <= dim; c += 32 * R) {
    float v[R];
#pragma unroll
    for (int j = 0; j < R; ++j) v[j] = there ? to_f32(__ldg(src + c + j * 32)) * a.scale : 0.f;
#pragma unroll
    for (int j = 0; j < R; ++j) dst[c + j * 32] = from_f32<TO>(v[j]);
  }
  float v[R];
#pragma unroll
  for (int j = 0; j < R; ++j) v[j] = there && c + j * 32 < dim ? to_f32(__ldg(src + c + j * 32)) * a.scale : 0.f;
#pragma unroll
  for (int j = 0; j < R; ++j)
    if (c + j * 32 < dim) dst[c + j * 32] = from_f32<TO>(v[j]);
}

// ============================================================ tt_embed_grad
// Tokens sorted by ID with their order kept (two passes of a radix sort), then
// each row's terms summed in that order.  The kernels are chained: each starts
// while the one before ends.
//
// A pass needs, for each tile of tokens and digit, how many tokens of the digit
// stand before the tile.  The first pass's counts are a kernel of their own;
// the second's are added up by the first pass as it places tokens in tiles.
// With up to SUM_TILES tiles each block adds the earlier tiles' counts itself
// (they come from L2); with more, a kernel scans them.  Whole calls, 64 columns
// into 100,256 rows, the one and the other: 8 tiles 23.4 and 25.8 us, 20 tiles
// 26.4 and 26.2, 30 tiles 31.9 and 29.9.
//
// The sums are bound by memory, the sort by the latency of its kernels: 304,824
// tokens of 2048 bfloat16 into 100,256 float rows take 374 us (2.07 GB, 81% of
// the measured copy bandwidth), some 330 of them the sums, and 367 us added to
// what the rows hold (1.82 GB, since absent rows are left alone); 16,400 tokens
// of 1024 floats into 4,352 rows take 42 us, of which the bytes need 13.
constexpr int SORT_THREADS = 512;
constexpr int SORT_WARPS = SORT_THREADS / 32;
constexpr int MAX_BINS = 1 << 11;
constexpr int SUM_TILES = 20;

struct SortArgs {
  const int64_t *n_ids;
  int64_t max_ids;
  int32_t n_vocab;
  int bits[2];              // of the two digits, low first
  int tiles;
  uint32_t *hist[2];        // [tiles][bins]: counts, or scanned
  uint32_t *total[2];       // [bins], where scanned
  int32_t *status;
  int32_t *cut_count;       // cleared for the sums
  // a table that is cleared meanwhile, in three parts: its rows, in 16-bit
  // words, and how many of them a block takes
  uint16_t *clear;
  int64_t clear_rows, clear_words, clear_stride, clear_each;
  unsigned clear_blocks;    // of each part
};

// zeros, 16 bytes a store; thread t of `group`
__device__ __forceinline__ void fill_zero(uint16_t *p, int64_t n, int t, int group) {
  const int64_t lead = min(n, (int64_t)((16 - (reinterpret_cast<uintptr_t>(p) & 15)) & 15) / 2);
  const int64_t vecs = (n - lead) / 8, done = lead + vecs * 8;
  if (t < lead) p[t] = 0;
  uint4 *q = reinterpret_cast<uint4 *>(p + lead);
  for (int64_t i = t; i < vecs; i += group) __stcs(q + i, make_uint4(0, 0, 0, 0));
  for (int64_t i = done + t; i < n; i += group) p[i] = 0;
  for (int64_t i = group + t; i < lead; i += group) p[i] = 0;
}

__device__ __forceinline__ void clear_part(const SortArgs &a, int part) {
  const int64_t r = ((int64_t)part * a.clear_blocks + blockIdx.x - a.tiles) * a.clear_each;
  const int64_t rows = min(a.clear_each, a.clear_rows - r);
  uint16_t *p = a.clear + r * a.clear_stride;
  if (rows <= 0) return;
  if (a.clear_stride == a.clear_words) {
    fill_zero(p, rows * a.clear_words, threadIdx.x, SORT_THREADS);
  } else {
    for (int64_t i = threadIdx.x >> 5; i < rows; i += SORT_WARPS) fill_zero(p + i * a.clear_stride, a.clear_words, threadIdx.x & 31, 32);
  }
}

__device__ __forceinline__ int64_t count_of(const int64_t *n_ids, int64_t max_ids) {
  return n_ids ? max((int64_t)0, min(*n_ids, max_ids)) : max_ids;
}

// the key of an ID: padding sorts behind every row
__device__ __forceinline__ uint32_t key_of(int32_t id, int32_t n_vocab) {
  return (uint32_t)id < (uint32_t)n_vocab ? (uint32_t)id : (uint32_t)n_vocab;
}

// the first digit's counts; and the second's cleared
template <int KEYS>
__global__ void __launch_bounds__(SORT_THREADS) k_sort_count(SortArgs a, const int32_t *__restrict__ ids) {
  __shared__ uint32_t count[MAX_BINS];
  let_next_start();
  if ((int)blockIdx.x >= a.tiles) return clear_part(a, 0);
  const int64_t n = count_of(a.n_ids, a.max_ids), base = (int64_t)blockIdx.x * (SORT_THREADS * KEYS);
  const int bins = 1 << a.bits[0];
  int32_t id[KEYS];
#pragma unroll
  for (int k = 0; k < KEYS; ++k) {
    const int64_t i = base + k * SORT_THREADS + threadIdx.x;
    id[k] = i < n ? ids[i] : -1;
  }
  for (int i = threadIdx.x; i < bins; i += SORT_THREADS) count[i] = 0;
  for (int i = threadIdx.x; i < 1 << a.bits[1]; i += SORT_THREADS) a.hist[1][((int64_t)blockIdx.x << a.bits[1]) + i] = 0;
  if (blockIdx.x == 0 && threadIdx.x < 2) a.cut_count[threadIdx.x] = 0;
  __syncthreads();
#pragma unroll
  for (int k = 0; k < KEYS; ++k) {
    const int64_t i = base + k * SORT_THREADS + threadIdx.x;
    if (i < n) {
      if (id[k] >= a.n_vocab) op_status(a.status, TT_ERR_INVALID_ARG);
      atomicAdd(&count[key_of(id[k], a.n_vocab) & (bins - 1)], 1u);
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < bins; i += SORT_THREADS) a.hist[0][((int64_t)blockIdx.x << a.bits[0]) + i] = count[i];
}

// counts -> how many in earlier tiles; a block 32 digits, its warps parts of the tiles
__global__ void __launch_bounds__(1024) k_sort_scan(SortArgs a, int pass) {
  __shared__ uint32_t part[32][33];
  wait_for_last();
  let_next_start();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, d = blockIdx.x * 32 + lane, bins = 1 << a.bits[pass];
  const int each = (a.tiles + 31) / 32, lo = min(a.tiles, warp * each), hi = min(a.tiles, lo + each);
  uint32_t *h = a.hist[pass] + d;
  uint32_t sum = 0;
  if (d < bins)
#pragma unroll 8
    for (int t = lo; t < hi; ++t) sum += h[(int64_t)t << a.bits[pass]];
  part[warp][lane] = sum;
  __syncthreads();
  uint32_t before = 0, all = 0;
  for (int w = 0; w < 32; ++w) {
    before += w < warp ? part[w][lane] : 0;
    all += part[w][lane];
  }
  if (d < bins) {
#pragma unroll 4
    for (int t = lo; t < hi; ++t) {
      const uint32_t c = h[(int64_t)t << a.bits[pass]];
      h[(int64_t)t << a.bits[pass]] = before;
      before += c;
    }
    if (warp == 0) a.total[pass][d] = all;
  }
}

// The second pass reads what the kernel before writes while this one may be there
// already: keys and pos are plain pointers, read behind wait_for_last(), since
// const and __restrict__ would allow loads that take memory as constant from the
// kernel's start on.  ids, the caller's, are.
template <int PASS, int KEYS>
__global__ void __launch_bounds__(SORT_THREADS)
k_sort_place(SortArgs a, const int32_t *__restrict__ ids, const int32_t *keys, const int32_t *pos, int32_t *keys_out,
             int32_t *pos_out) {
  extern __shared__ uint32_t sm[];                         // base[bins], then uint16 seen[SORT_WARPS][bins]
  __shared__ uint32_t box[SORT_WARPS];
  if ((int)blockIdx.x >= a.tiles) {
    let_next_start();
    return clear_part(a, 1 + PASS);
  }
  const int bins = 1 << a.bits[PASS], shift = PASS ? a.bits[0] : 0;
  uint32_t *base = sm;
  uint16_t *seen = reinterpret_cast<uint16_t *>(sm + bins);
  const int64_t tile = (int64_t)blockIdx.x * (SORT_THREADS * KEYS);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int i = threadIdx.x; i < bins * SORT_WARPS / 2; i += SORT_THREADS) reinterpret_cast<uint32_t *>(seen)[i] = 0;
  if (PASS || a.tiles > SUM_TILES) wait_for_last();
  const int64_t n = count_of(a.n_ids, a.max_ids);
  // a warp's keys are KEYS consecutive groups of 32
  const int64_t first = tile + warp * (32 * KEYS) + lane;
  uint32_t key[KEYS];
  int32_t at[KEYS];
#pragma unroll
  for (int k = 0; k < KEYS; ++k) {
    const int64_t i = first + k * 32;
    key[k] = i < n ? (PASS ? (uint32_t)keys[i] : key_of(ids[i], a.n_vocab)) : 0;
    at[k] = PASS ? (i < n ? pos[i] : 0) : (int32_t)i;
  }
  if (!PASS && a.tiles <= SUM_TILES) wait_for_last();
  let_next_start();
  // four digits a thread: their tokens in earlier tiles and in all
  uint32_t t[4] = {0, 0, 0, 0}, before[4] = {0, 0, 0, 0}, x = 0;
  const int d0 = threadIdx.x * 4;
  if (d0 < bins) {
    if (a.tiles <= SUM_TILES) {
      if (bins >= 4) {
        const uint4 *h = reinterpret_cast<const uint4 *>(a.hist[PASS] + d0);
#pragma unroll 8
        for (int i = 0; i < a.tiles; ++i) {
          const uint4 c = h[(int64_t)i << (a.bits[PASS] - 2)];
          t[0] += c.x, t[1] += c.y, t[2] += c.z, t[3] += c.w;
          if (i < (int)blockIdx.x) before[0] += c.x, before[1] += c.y, before[2] += c.z, before[3] += c.w;
        }
      } else {
        for (int i = 0; i < a.tiles; ++i)
          for (int k = 0; k < bins; ++k) {
            const uint32_t c = a.hist[PASS][i * bins + k];
            t[k & 3] += c;
            before[k & 3] += i < (int)blockIdx.x ? c : 0;
          }
      }
    } else {
      for (int k = 0; k < 4; ++k)
        if (d0 + k < bins) {
          t[k] = a.total[PASS][d0 + k];
          before[k] = a.hist[PASS][((int64_t)blockIdx.x << a.bits[PASS]) + d0 + k];
        }
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) x += t[k];
  }
  // where each digit begins: exclusive scan of the totals
  const uint32_t own = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(~0u, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) box[warp] = x;
  __syncthreads();
  x -= own;
  for (int w = 0; w < warp; ++w) x += box[w];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if (d0 + k < bins) base[d0 + k] = x + before[k];
    x += t[k];
  }
  // rank of each key among its warp's keys of the same digit
  uint32_t rank[KEYS];
#pragma unroll
  for (int k = 0; k < KEYS; ++k) {
    const bool there = first + k * 32 < n;
    const uint32_t d = there ? (key[k] >> shift) & (bins - 1) : 0xFFFFu;
    const uint32_t same = __match_any_sync(~0u, d);
    const int lead = __ffs(same) - 1;
    uint32_t s = 0;
    if (there && lane == lead) {
      s = seen[warp * bins + d];
      seen[warp * bins + d] = (uint16_t)(s + __popc(same));
    }
    rank[k] = __shfl_sync(~0u, s, lead) + __popc(same & ((1u << lane) - 1));
    __syncwarp();
  }
  __syncthreads();
  for (int d = threadIdx.x; d < bins; d += SORT_THREADS) {
    uint32_t sum = 0;
    for (int w = 0; w < SORT_WARPS; ++w) {
      const uint32_t c = seen[w * bins + d];
      seen[w * bins + d] = (uint16_t)sum;
      sum += c;
    }
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < KEYS; ++k) {
    if (first + k * 32 < n) {
      const uint32_t d = (key[k] >> shift) & (bins - 1);
      const uint32_t to = base[d] + seen[warp * bins + d] + rank[k];
      keys_out[to] = (int32_t)key[k];
      pos_out[to] = at[k];
      if (!PASS) atomicAdd(&a.hist[1][((int64_t)(to / (SORT_THREADS * KEYS)) << a.bits[1]) + (key[k] >> a.bits[0])], 1u);
    }
  }
}

// The sums.  Rows and sorted tokens are one list of items, the tokens of a row
// before the row's end: token i stands at place i + key[i], the end of row r
// behind the tokens of rows 0 .. r.  The list is cut into equal parts, one for
// a worker (a group of threads that covers up to 2048 columns); a token costs
// a row read and a row's end a row written, so the parts cost the same however
// the tokens are spread: absent rows, rows of one token and rows of a tenth of
// all tokens.  A row that ends where it began is written at once; one that is
// cut leaves its pieces in the workspace, and k_grad_join adds them in order.
// Where rows without tokens cost nothing (they keep what they hold, or are many
// and the sort's kernels clear them beside their own work), tokens alone are
// the items.
struct GradArgs {
  const int64_t *n_ids;
  int64_t max_ids, n_vocab, dim, dout_stride, dtable_stride;
  float scale;
  int accumulate;
  int tokens_only;               // rows are no items
  const int32_t *keys, *pos;     // sorted
  int items, workers;            // items a worker, workers a block
  int group, cols;               // threads a worker, columns of its tile
  int64_t carry_stride;          // dim rounded up to whole float4
  float *heads, *tails;          // [workers in all][carry_stride]
  int whole;                     // rows of at most so many tokens are not cut
  int32_t *row_first;            // [n_vocab]: the worker where a cut row begins
  int32_t *cut_count;
  int2 *cut;                     // the worker where a cut row ends, and the row
  int64_t pieces;                // room in `cut`
};

// how many of 0 .. n-1, from the first on, satisfy `pred` (a prefix does): a
// 33-ary search by a warp
template <class P> __device__ __forceinline__ int64_t warp_search(int64_t n, P pred) {
  const int lane = threadIdx.x & 31;
  int64_t lo = 0, hi = n;        // lo - 1 does, hi does not
  while (lo < hi) {
    const int64_t step = (hi - lo + 31) / 32, i = lo + lane * step;
    const int c = __popc(__ballot_sync(~0u, i < hi && pred(i)));       // probes 0 .. c-1 do
    if (c < 32) hi = min(hi, lo + c * step);
    if (c > 0) lo = lo + (c - 1) * step + 1;
  }
  return lo;
}

// the number of tokens that stand before `place`
__device__ __forceinline__ int64_t tokens_before(const int32_t *keys, int64_t n, int64_t place) {
  return warp_search(n, [&](int64_t i) { return i + keys[i] < place; });
}

// A thread's columns: eight side by side, or four 32 apart (a warp's 128).  How
// its parts of AHEAD rows are kept in flight: what ends a row is much code, and a
// batch in registers has a copy of it for each of its rows, which soon cost more
// instruction fetches than the sums; parts that wait in shared memory, where
// nobody else reads, go through one copy.  us for 100,256 rows of (columns,
// tokens, type of dout; a batch, copied to shared memory, a batch put there):
//   256  200,000 bfloat16   86   72   77     1024 60,000 bfloat16 106   87   97
//   256  200,000 float      84  102   89     1024 60,000 float    140  160  142
//   641  200,000 bfloat16  262    -  163      641 200,000 float   293  193  176
// The float batch in registers is a tight fit: 64 of them, and 16 to 28 bytes
// spilled, with which these were measured.
enum Ahead { IN_REGISTERS, COPIED, STAGED };
constexpr int SUM_THREADS = 256;                  // at most
template <class T, int COLS> struct Cols;
template <class T> struct Cols<T, 8> {
  typedef uint4 Part;
  static constexpr Ahead HOW = sizeof(T) == 4 ? IN_REGISTERS : COPIED;
  static constexpr int AHEAD = 16 / sizeof(T), PARTS = sizeof(T) / 2;
  // (`left`: columns from the thread's first on)
  static __device__ __forceinline__ void load(Part raw[PARTS], const T *row, int) {
#pragma unroll
    for (int j = 0; j < PARTS; ++j) raw[j] = __ldg(reinterpret_cast<const uint4 *>(row) + j);
  }
  static __device__ __forceinline__ void f32(const Part raw[PARTS], float v[8]) {
    Raw8<T> r;
#pragma unroll
    for (int j = 0; j < PARTS; ++j) r.w[j] = raw[j];
    raw_f32(r, v);
  }
  static __device__ __forceinline__ void store(T *row, int, float v[8], bool accumulate) {
    if (accumulate) {
      float o[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) o[j] = to_f32(row[j]);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] += o[j];
    }
    store8(row, v);
  }
};
template <class T> struct Cols<T, 4> {
  typedef T Part;
  static constexpr Ahead HOW = STAGED;
  static constexpr int AHEAD = 8, PARTS = 4;
  static __device__ __forceinline__ void load(Part raw[4], const T *row, int left) {
#pragma unroll
    for (int j = 0; j < 4; ++j) raw[j] = j * 32 < left ? row[j * 32] : from_f32<T>(0.f);
  }
  static __device__ __forceinline__ void f32(const Part raw[4], float v[4]) {
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = to_f32(raw[j]);
  }
  static __device__ __forceinline__ void store(T *row, int left, float v[4], bool accumulate) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (j * 32 < left) row[j * 32] = from_f32<T>(accumulate ? to_f32(row[j * 32]) + v[j] : v[j]);
  }
};
template <class In> constexpr int slot_bytes() {  // a block's
  return In::HOW == IN_REGISTERS ? 0 : In::AHEAD * In::PARTS * (int)sizeof(typename In::Part) * SUM_THREADS;
}

constexpr int HALO = 64;
constexpr int LONG_ROW = 6;                       // pieces, at least, of a row that a block joins

template <class TI, class TO, int COLS>
__global__ void __launch_bounds__(SUM_THREADS, 4) k_grad_sum(GradArgs a, const TI *__restrict__ dout, TO *__restrict__ dtable) {
  typedef Cols<TI, COLS> In;
  // the threads' parts ahead; then keys, and places in dout, HALO more on both sides
  extern __shared__ uint4 s_ahead[];
  int32_t *const s_tok = reinterpret_cast<int32_t *>(s_ahead) + slot_bytes<In>() / 4;
  __shared__ int64_t s_at[2];
  wait_for_last();
  let_next_start();
  const int64_t n = count_of(a.n_ids, a.max_ids);
  const int block_items = a.items * a.workers;
  const int64_t d0 = (int64_t)blockIdx.x * block_items;
  // tokens of the block's places; padding stands behind every row
  int64_t i0 = min(n, d0), i1 = min(n, d0 + block_items);
  if (!a.tokens_only) {
    if (threadIdx.x < 64) {
      const int64_t at = tokens_before(a.keys, n, d0 + (threadIdx.x >> 5) * block_items);
      if ((threadIdx.x & 31) == 0) s_at[threadIdx.x >> 5] = at;
    }
    __syncthreads();
    i0 = s_at[0];
    i1 = s_at[1];
  }
  const int n_tok = (int)(i1 - i0);
  int32_t *s_key = s_tok + HALO, *s_pos = s_key + block_items + HALO;
  for (int i = (int)threadIdx.x - HALO; i < n_tok + HALO; i += blockDim.x) {
    const bool there = i0 + i >= 0 && i0 + i < n;
    s_key[i] = there ? a.keys[i0 + i] : i < 0 ? -1 : INT32_MAX;
    if (there && i >= 0) s_pos[i] = a.pos[i0 + i];
  }
  __syncthreads();
  const int sub = threadIdx.x / a.group, t = threadIdx.x - sub * a.group;
  const int dim = (int)a.dim, n_vocab = (int)a.n_vocab;
  const int c = (int)blockIdx.y * a.cols + (COLS == 8 ? t * 8 : t / 32 * 128 + t % 32);
  if (sub >= a.workers) return;
  const bool mine = c < dim;                    // threads past the columns still fill
  // the first of [lo, hi) whose key is at least k
  auto first_of = [&](int lo, int hi, int k) {
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (s_key[mid] < k) lo = mid + 1; else hi = mid;
    }
    return lo;
  };
  // The cut at the block's place p: the tokens of the block before it, and the
  // rows.  One inside a row of at most a.whole tokens moves behind that row.
  auto cut_at = [&](int p, int &i, int &r) {
    int lo = p == block_items ? n_tok : 0, hi = min(p, n_tok);
    if (a.tokens_only) lo = hi;
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (i0 + mid + s_key[mid] < d0 + p) lo = mid + 1; else hi = mid;
    }
    i = lo;
    r = a.tokens_only ? min(n_vocab, s_key[lo]) : (int)min(a.n_vocab, d0 + p - i0 - lo);
    if (s_key[lo - 1] == r && r < n_vocab) {
      const int begin = first_of(lo - a.whole, lo, r), end = first_of(lo, lo + a.whole, r + 1);
      if (end - begin <= a.whole && s_key[begin - 1] < r) {       // else it is longer
        i = end;
        r = a.tokens_only ? min(n_vocab, s_key[end]) : r + 1;
      }
    }
  };
  int i, end, r, r_end;
  cut_at(sub * a.items, i, r);
  cut_at((sub + 1) * a.items, end, r_end);
  while (end > i && s_key[end - 1] >= n_vocab) --end;
  const int w = (int)blockIdx.x * a.workers + sub;
  bool head = s_key[i - 1] == r && r < n_vocab, any = false;
  const bool side_by_side = !a.tokens_only && gridDim.y == 1 && a.dtable_stride == a.dim;
  float acc[COLS];
#pragma unroll
  for (int j = 0; j < COLS; ++j) acc[j] = 0;
  auto keep = [&](float *to) {                    // a piece of a cut row
    float *p = to + (int64_t)w * a.carry_stride + c;
    if (COLS == 8) {
      if (mine) {
        reinterpret_cast<float4 *>(p)[0] = make_float4(acc[0], acc[1], acc[2], acc[3]);
        reinterpret_cast<float4 *>(p)[1] = make_float4(acc[4 % COLS], acc[5 % COLS], acc[6 % COLS], acc[7 % COLS]);
      }
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (c + j * 32 < dim) p[j * 32] = acc[j];
    }
  };
  auto finish_to = [&](int k) {               // rows r .. k-1 end here
    if (head) {
      keep(a.heads);
      if (t == 0 && blockIdx.y == 0) {
        // rows of many pieces are listed from the other end
        const int64_t far = i0 + i - (int64_t)LONG_ROW * a.items;
        if (far >= 0 && a.keys[far] == r) a.cut[a.pieces - 1 - atomicAdd(a.cut_count + 1, 1)] = make_int2(w, r);
        else a.cut[atomicAdd(a.cut_count, 1)] = make_int2(w, r);
      }
    } else if (any) {
      float v[COLS];
#pragma unroll
      for (int j = 0; j < COLS; ++j) v[j] = acc[j] * a.scale;
      if (mine) Cols<TO, COLS>::store(dtable + (int64_t)r * a.dtable_stride + c, dim - c, v, a.accumulate);
    }
    if (head || any) ++r;
    head = any = false;
#pragma unroll
    for (int j = 0; j < COLS; ++j) acc[j] = 0;
    if (side_by_side) {
      constexpr int WORDS = sizeof(TO) / 2;
      if (r < k) fill_zero(reinterpret_cast<uint16_t *>(dtable + (int64_t)r * a.dim), (int64_t)(k - r) * a.dim * WORDS, t, a.group);
    } else if (!a.tokens_only && mine) {
      for (; r < k; ++r) {
        float v[COLS] = {};
        Cols<TO, COLS>::store(dtable + (int64_t)r * a.dtable_stride + c, dim - c, v, false);
      }
    }
    r = k;
  };
  auto *const slots = reinterpret_cast<typename In::Part *>(s_ahead) + threadIdx.x;
  auto from = [&](int at) { return dout + (int64_t)s_pos[at] * a.dout_stride + c; };
  auto add = [&](int32_t k, const typename In::Part raw[In::PARTS]) {
    if (r < k) finish_to(k);
    float f[COLS];
    In::f32(raw, f);
#pragma unroll
    for (int j = 0; j < COLS; ++j) acc[j] += f[j];
    any = true;
  };
  auto add_slot = [&](int slot) {
    typename In::Part raw[In::PARTS];
#pragma unroll
    for (int j = 0; j < In::PARTS; ++j) raw[j] = slots[(slot * In::PARTS + j) * SUM_THREADS];
    add(s_key[i], raw);
  };
  if constexpr (In::HOW == IN_REGISTERS) {
    for (; i < end; i += In::AHEAD) {
      typename In::Part raw[In::AHEAD][In::PARTS];
#pragma unroll
      for (int b = 0; b < In::AHEAD; ++b)
        if (mine && i + b < end) In::load(raw[b], from(i + b), dim - c);
#pragma unroll
      for (int b = 0; b < In::AHEAD; ++b)
        if (i + b < end) add(s_key[i + b], raw[b]);
    }
  } else if constexpr (In::HOW == COPIED) {
    auto fetch = [&](int at, int slot) {
      if (mine && at < end) {
        const uint4 *row = reinterpret_cast<const uint4 *>(from(at));
#pragma unroll
        for (int j = 0; j < In::PARTS; ++j) copy_async(slots + (slot * In::PARTS + j) * SUM_THREADS, row + j);
      }
      copy_group();
    };
#pragma unroll
    for (int b = 0; b < In::AHEAD - 1; ++b) fetch(i + b, b);
#pragma unroll 1
    for (int slot = 0; i < end; ++i) {
      copy_wait<In::AHEAD - 2>();
      fetch(i + In::AHEAD - 1, slot ? slot - 1 : In::AHEAD - 1);        // into what was added last
      add_slot(slot);
      slot = slot + 1 < In::AHEAD ? slot + 1 : 0;
    }
    copy_wait<0>();
  } else {
    while (i < end) {
      typename In::Part raw[In::AHEAD][In::PARTS];
#pragma unroll
      for (int b = 0; b < In::AHEAD; ++b) In::load(raw[b], from(min(i + b, end - 1)), dim - c);
#pragma unroll
      for (int b = 0; b < In::AHEAD; ++b)
#pragma unroll
        for (int j = 0; j < In::PARTS; ++j) slots[(b * In::PARTS + j) * SUM_THREADS] = raw[b][j];
#pragma unroll 1
      for (int b = 0; b < In::AHEAD && i < end; ++b, ++i) add_slot(b);
    }
  }
  if (r < r_end) finish_to(r_end);
  if (any) {
    keep(a.tails);
    if (!head && t == 0 && blockIdx.y == 0) a.row_first[r] = w;
  }
}

// The rows that were cut: the tails of the workers before, then the last
// worker's head, 128 columns at a time.  A warp takes rows of few pieces; a
// block those of many, in 32 runs side by side.
template <class TO>
__device__ __forceinline__ float4 join_pieces(const GradArgs &a, int64_t c, int64_t lo, int64_t hi) {
  float4 s = make_float4(0, 0, 0, 0);
  if (c < a.dim) {
#pragma unroll 8
    for (int64_t k = lo; k < hi; ++k) {
      const float4 x = *reinterpret_cast<const float4 *>(a.tails + k * a.carry_stride + c);
      s.x += x.x; s.y += x.y; s.z += x.z; s.w += x.w;
    }
  }
  return s;
}
template <class TO>
__device__ __forceinline__ void join_store(const GradArgs &a, TO *dtable, int2 at, int64_t c, float4 s) {
  if (c >= a.dim) return;
  const float4 h = *reinterpret_cast<const float4 *>(a.heads + at.x * a.carry_stride + c);
  const float v[4] = {(s.x + h.x) * a.scale, (s.y + h.y) * a.scale, (s.z + h.z) * a.scale, (s.w + h.w) * a.scale};
  TO *p = dtable + at.y * a.dtable_stride + c;
  for (int j = 0; j < 4; ++j)
    if (c + j < a.dim) p[j] = from_f32<TO>(a.accumulate ? to_f32(p[j]) + v[j] : v[j]);
}

template <class TO>
__global__ void __launch_bounds__(1024) k_grad_join(GradArgs a, TO *__restrict__ dtable) {
  __shared__ float4 part[32][32];
  wait_for_last();
  const int few = a.cut_count[0], many = a.cut_count[1], chunks = (int)((a.dim + 127) / 128);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int64_t job = blockIdx.x; job < (int64_t)many * chunks; job += gridDim.x) {
    const int2 at = a.cut[a.pieces - 1 - job / chunks];
    const int64_t w = at.x, c = (job % chunks) * 128 + lane * 4, first = a.row_first[at.y];
    const int64_t each = (w - first + 31) / 32, lo = min(w, first + warp * each);
    float4 s = join_pieces<TO>(a, c, lo, min(w, lo + each));
    __syncthreads();
    part[warp][lane] = s;
    __syncthreads();
    if (warp == 0) {
#pragma unroll 8
      for (int k = 1; k < 32; ++k) {
        const float4 x = part[k][lane];
        s.x += x.x; s.y += x.y; s.z += x.z; s.w += x.w;
      }
      join_store(a, dtable, at, c, s);
    }
  }
  for (int64_t job = (int64_t)(gridDim.x - 1 - blockIdx.x) * 32 + warp; job < (int64_t)few * chunks; job += (int64_t)gridDim.x * 32) {
    const int2 at = a.cut[job / chunks];
    const int64_t c = (job % chunks) * 128 + lane * 4;
    join_store(a, dtable, at, c, join_pieces<TO>(a, c, a.row_first[at.y], at.x));
  }
}

// ------------------------------------------------------------ host side
bool grad_sizes_ok(int64_t max_ids, int64_t n_vocab, int64_t dim) {
  return max_ids >= 0 && max_ids <= TT_MAX_IDS && vocab_ok(n_vocab) && dim >= 1 && dim <= MAX_DIM;
}

template <int PASS, int KEYS> struct Place {};
template <class TI, class TO, int COLS> struct Sum {};
template <int N> struct Per { static constexpr int value = N; };

struct GradPlan {
  int tiles = 0, per_thread = 0, bits[2] = {0, 0};       // tokens a thread in the sort: fewer make short calls shorter
  int col_tiles[2], cols[2], group[2], workers[2];       // [1]: eight columns a thread, [0]: four
  int items[2][2];                                       // [..][1]: tokens only
  int64_t blocks[2][2];
  int64_t keys[2], pos[2], hist[2], total[2], pieces, row_first, cut_count, cut, heads, tails, carry_stride, bytes;   // offsets into the workspace
};


constexpr int BLOCK_ITEMS = 4096;                 // at most, in shared memory

GradPlan grad_plan(int64_t max_ids, int64_t n_vocab, int64_t dim) {
  GradPlan p;
  int bits = 1;
  while ((n_vocab >> bits) != 0) ++bits;          // keys are 0 .. n_vocab
  p.bits[0] = (bits + 1) / 2;
  p.bits[1] = bits - p.bits[0];
  // tokens a thread of the sort: 2, 4 and 8 take 23, 27 and 34 us for 8,191 tokens
  // (of 64 columns), 37, 40 and 46 for 130,000, 43, 41 and 48 for 200,000, 194,
  // 182 and 178 for 2,000,000
  p.per_thread = max_ids <= 1 << 17 ? 2 : max_ids <= 1 << 20 ? 4 : 8;
  p.tiles = (int)((max_ids + SORT_THREADS * p.per_thread - 1) / (SORT_THREADS * p.per_thread));
  int64_t pieces = 0;
  for (int v = 0; v < 2; ++v) {
    const int per = v ? 8 : 4;
    const int64_t threads = (dim + per - 1) / per;
    p.col_tiles[v] = (int)((threads + 255) / 256);
    int need = (int)((threads + p.col_tiles[v] - 1) / p.col_tiles[v]);
    if (!v) need = std::max(need, (int)std::min<int64_t>(dim, 32));      // its columns are 32 apart
    if (need > 128) {
      p.group[v] = (need + 31) / 32 * 32;
      p.workers[v] = 1;
    } else {
      p.group[v] = 1;
      while (p.group[v] < need) p.group[v] *= 2;
      p.workers[v] = 256 / p.group[v];
    }
    p.cols[v] = p.group[v] * per;
    p.col_tiles[v] = (int)((dim + p.cols[v] - 1) / p.cols[v]);
    // Four rounds of the blocks that run at once, or fewer for short calls, but
    // whole rounds: one block more costs a round.  Few enough pieces.
    const int64_t at_once = std::max<int64_t>(1, 152 * (1024 / (p.group[v] * p.workers[v])) / p.col_tiles[v]);
    for (int tokens_only = 0; tokens_only < 2; ++tokens_only) {
      const int64_t places = tokens_only ? std::max<int64_t>(max_ids, 1) : n_vocab + max_ids;
      const int64_t rounds = std::max<int64_t>(1, std::min<int64_t>(4, places / (16 * p.workers[v] * at_once)));
      const int64_t blocks = std::min(rounds * at_once, std::max<int64_t>(1, std::max<int64_t>(8192, (1 << 21) / dim) / p.workers[v]));
      int64_t items = (places + blocks * p.workers[v] - 1) / (blocks * p.workers[v]);
      items = std::min<int64_t>(BLOCK_ITEMS / p.workers[v], std::max<int64_t>(16, items));
      p.items[v][tokens_only] = (int)items;
      p.blocks[v][tokens_only] = (places + items * p.workers[v] - 1) / (items * p.workers[v]);
      pieces = std::max(pieces, p.blocks[v][tokens_only] * p.workers[v]);
    }
  }
  int64_t at = 0;
  auto take = [&](int64_t bytes) {
    const int64_t o = at;
    at += (bytes + 255) / 256 * 256;
    return o;
  };
  for (int i = 0; i < 2; ++i) {
    p.keys[i] = take(4 * max_ids);
    p.pos[i] = take(4 * max_ids);
  }
  for (int i = 0; i < 2; ++i) {
    p.hist[i] = take(4 * ((int64_t)p.tiles << p.bits[i]));
    p.total[i] = take(4 * MAX_BINS);
  }
  p.pieces = pieces;
  p.carry_stride = (dim + 3) / 4 * 4;
  p.row_first = p.cut_count = p.cut = p.heads = p.tails = 0;
  if (max_ids > 0) {
    p.row_first = take(4 * n_vocab);
    p.cut_count = take(8);
    p.cut = take(8 * pieces);
    p.heads = take(4 * pieces * p.carry_stride);
    p.tails = take(4 * pieces * p.carry_stride);
  }
  p.bytes = at;
  return p;
}

}  // namespace

extern "C" tt_status tt_embed(const int32_t *d_ids, int64_t max_ids, const int64_t *d_n_ids, const void *d_table,
                              int32_t table_type, int64_t n_vocab, int64_t dim, int64_t table_stride, float scale,
                              void *d_out, int32_t out_type, int64_t out_stride, int32_t *d_status,
                              tt_stream_t stream) {
  if (!type_ok(table_type) || !type_ok(out_type) || !vocab_ok(n_vocab) || dim < 1 || dim > MAX_DIM || max_ids < 0 ||
      table_stride < dim || out_stride < dim || !optional_ok(d_n_ids, 8) || !optional_ok(d_status, 4))
    return TT_ERR_INVALID_ARG;
  if (max_ids > TT_MAX_IDS) return TT_ERR_CAPACITY;
  if (max_ids == 0) return TT_OK;
  if (!array_ok(d_ids, 4) || !array_ok(d_table, type_size(table_type)) || !array_ok(d_out, type_size(out_type)))
    return TT_ERR_INVALID_ARG;
  EmbedArgs a{d_ids, d_n_ids, max_ids, n_vocab, dim, table_stride, out_stride, scale, 0, d_status};
  const bool vec = rows_vector(d_table, table_stride, dim) && rows_vector(d_out, out_stride, dim);
  with_type(table_type, [&](auto ti) {
    with_type(out_type, [&](auto to) {
      using TI = decltype(ti);
      using TO = decltype(to);
      if (vec) {
        const int64_t units = dim / 8;
        while (a.lanes_log2 < 5 && (1 << a.lanes_log2) < units) ++a.lanes_log2;
        if (a.lanes_log2 == 5) {
          const dim3 grid((unsigned)((max_ids + 7) / 8), (unsigned)((units + 127) / 128));
          k_embed<TI, TO, true><<<grid, 256, 0, stream>>>(a, (const TI *)d_table, (TO *)d_out);
        } else {
          const int64_t rows = 8 * (32 >> a.lanes_log2) * 4;
          k_embed<TI, TO, false><<<(unsigned)((max_ids + rows - 1) / rows), 256, 0, stream>>>(a, (const TI *)d_table, (TO *)d_out);
        }
      } else {
        k_embed_any<TI, TO><<<(unsigned)((max_ids + 7) / 8), 256, 0, stream>>>(a, (const TI *)d_table, (TO *)d_out);
      }
    });
  });
  return launched("tt_embed");
}

extern "C" int64_t tt_embed_grad_workspace(int64_t max_ids, int64_t n_vocab, int64_t dim) {
  return grad_sizes_ok(max_ids, n_vocab, dim) ? grad_plan(max_ids, n_vocab, dim).bytes : -1;
}

extern "C" tt_status tt_embed_grad(const int32_t *d_ids, int64_t max_ids, const int64_t *d_n_ids, const void *d_dout,
                                   int32_t dout_type, int64_t dim, int64_t dout_stride, float scale, void *d_dtable,
                                   int32_t dtable_type, int64_t n_vocab, int64_t dtable_stride, int32_t accumulate,
                                   void *d_workspace, int64_t workspace_bytes, int32_t *d_status, tt_stream_t stream) {
  if (!type_ok(dout_type) || !type_ok(dtable_type) || max_ids < 0 || dout_stride < dim || dtable_stride < dim ||
      !optional_ok(d_n_ids, 8) || !optional_ok(d_status, 4) || !array_ok(d_dtable, type_size(dtable_type)))
    return TT_ERR_INVALID_ARG;
  if (max_ids > TT_MAX_IDS) return TT_ERR_CAPACITY;
  if (!grad_sizes_ok(max_ids, n_vocab, dim)) return TT_ERR_INVALID_ARG;
  if (max_ids > 0 && (!array_ok(d_ids, 4) || !array_ok(d_dout, type_size(dout_type)))) return TT_ERR_INVALID_ARG;
  const GradPlan p = grad_plan(max_ids, n_vocab, dim);
  if (!array_ok(d_workspace, 16)) return TT_ERR_INVALID_ARG;
  if (workspace_bytes < p.bytes) return TT_ERR_CAPACITY;
  if (max_ids == 0 && accumulate) return TT_OK;
  char *ws = (char *)d_workspace;
  // Rows that are mostly absent are cleared by blocks beside the sort's; with more
  // tokens, rows written twice cost what that saves.  us cleared there and written
  // by the sums, for a token count of 1/32, 1/8, 1/4, 1/2 and all of the rows':
  //    200256 x  641 bfloat16            61  73    79  87    99 101   128 126   181 177
  //    100256 x 1024 bfloat16 -> float   81  82    82  92    95 101   109 113   138 134
  //    200256 x 2048 bfloat16           129 153   158 175   185 191   224 224   298 292
  //   1048576 x  128 bfloat16 -> float  107 120   115 134   131 152   174 179   228 224
  //    100256 x   64 float               39  34    41  38    46  42    46  46    56  50
  // (The last, a table of 26 MB, would rather not.)
  const bool clear = !accumulate && max_ids > 0 && max_ids <= n_vocab / 4;
  const int tokens_only = accumulate || clear;
  int32_t *keys[2] = {(int32_t *)(ws + p.keys[0]), (int32_t *)(ws + p.keys[1])};
  int32_t *pos[2] = {(int32_t *)(ws + p.pos[0]), (int32_t *)(ws + p.pos[1])};
  if (max_ids > 0) {
    SortArgs s{d_n_ids, max_ids, (int32_t)n_vocab, {p.bits[0], p.bits[1]}, p.tiles,
                     {(uint32_t *)(ws + p.hist[0]), (uint32_t *)(ws + p.hist[1])},
                     {(uint32_t *)(ws + p.total[0]), (uint32_t *)(ws + p.total[1])}, d_status, (int32_t *)(ws + p.cut_count),
               (uint16_t *)d_dtable, n_vocab, 0, 0, 0, 0};
    if (clear) {
      const int64_t words = (int64_t)type_size(dtable_type) / 2;
      s.clear_words = dim * words;
      s.clear_stride = dtable_stride * words;
      s.clear_each = std::max<int64_t>(1, 65536 / s.clear_words);
      s.clear_blocks = (unsigned)((n_vocab + 3 * s.clear_each - 1) / (3 * s.clear_each));
    }
    auto run = [&](auto per) {
      constexpr int KEYS = decltype(per)::value;
      const auto shared = [](int bits) { return ((size_t)4 << bits) + ((size_t)2 * SORT_WARPS << bits); };
      if (allow_shared<Place<0, KEYS>>(k_sort_place<0, KEYS>, (int)shared(11)) ||
          allow_shared<Place<1, KEYS>>(k_sort_place<1, KEYS>, (int)shared(11)))
        return;                                               // (the error is kept)
      k_sort_count<KEYS><<<p.tiles + s.clear_blocks, SORT_THREADS, 0, stream>>>(s, d_ids);
      for (int pass = 0; pass < 2; ++pass) {
        if (p.tiles > SUM_TILES)
          launch_cluster(k_sort_scan, dim3(((1u << p.bits[pass]) + 31) / 32), 1024, 0, 1, true, stream, s, pass);
        launch_cluster(pass ? k_sort_place<1, KEYS> : k_sort_place<0, KEYS>, dim3(p.tiles + s.clear_blocks), SORT_THREADS, shared(p.bits[pass]), 1, true,
                       stream, s, d_ids, keys[0], pos[0], keys[pass], pos[pass]);
      }
    };
    if (p.per_thread == 2) run(Per<2>{});
    else if (p.per_thread == 4) run(Per<4>{});
    else run(Per<8>{});
  }
  const int v = rows_vector(d_dout, dout_stride, dim) && rows_vector(d_dtable, dtable_stride, dim);
  const GradArgs a{d_n_ids, max_ids, n_vocab, dim, dout_stride, dtable_stride, scale, accumulate != 0, tokens_only, keys[1], pos[1],
                   p.items[v][tokens_only], p.workers[v], p.group[v], p.cols[v], p.carry_stride,
                   (float *)(ws + p.heads), (float *)(ws + p.tails), std::min(std::max(p.items[v][tokens_only], 16), HALO - 1),
                   (int32_t *)(ws + p.row_first), (int32_t *)(ws + p.cut_count), (int2 *)(ws + p.cut), p.pieces};
  with_type(dout_type, [&](auto ti) {
    with_type(dtable_type, [&](auto to) {
      using TI = decltype(ti);
      using TO = decltype(to);
      const dim3 grid((unsigned)p.blocks[v][tokens_only], (unsigned)p.col_tiles[v]);
      const unsigned threads = (unsigned)(p.group[v] * p.workers[v]);
      auto run = [&](auto cols) {
        constexpr int COLS = decltype(cols)::value;
        auto sum = k_grad_sum<TI, TO, COLS>;
        const auto shared = [](int64_t items) { return slot_bytes<Cols<TI, COLS>>() + 4 * (4 * HALO + 2 * (size_t)items); };
        if (allow_shared<Sum<TI, TO, COLS>>(sum, (int)shared(BLOCK_ITEMS))) return;        // (the error is kept)
        launch_cluster(sum, grid, threads, shared(p.items[v][tokens_only] * p.workers[v]), 1, max_ids > 0, stream, a,
                       (const TI *)d_dout, (TO *)d_dtable);
      };
      if (v) run(Per<8>{}); else run(Per<4>{});
      if (max_ids > 0)
        launch_cluster(k_grad_join<TO>, dim3((unsigned)std::min<int64_t>(152 * 2, p.blocks[v][tokens_only] * p.workers[v])), 1024, 0, 1, true, stream, a,
                       (TO *)d_dtable);
    });
  });
  return launched("tt_embed_grad");
}
