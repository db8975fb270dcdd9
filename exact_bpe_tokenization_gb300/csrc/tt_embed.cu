// tt_embed.cu - token embedding and its gradient (include/toktier.h).
#include "tt_ops.cuh"

using namespace tt::ops;

namespace {

// ============================================================ tt_embed
// out[i] = scale * table[ids[i]]: no arithmetic to speak of, bound by the
// bytes of the rows read and written.
//
// Threads take groups of eight elements.  A warp takes four groups a lane at a
// time, of one row where the row has them (unit_step 32), else of several rows
// (row_step), so that four loads are in flight before the first store.
struct EmbedArgs {
  const int32_t *ids;
  const int64_t *n_ids;
  int64_t max_ids, n_vocab, dim, table_stride, out_stride;
  float scale;
  int lanes_log2;    // lanes that share a row
  int32_t *status;
};

template <class TI, class TO>
__global__ void __launch_bounds__(256) k_embed(EmbedArgs a, const TI *__restrict__ table, TO *__restrict__ out) {
  constexpr int R = 4;
  const int64_t n = a.n_ids ? max((int64_t)0, min(*a.n_ids, a.max_ids)) : a.max_ids;
  const int units = (int)(a.dim >> 3);
  const int lane = threadIdx.x & 31, rows_per_warp = 32 >> a.lanes_log2;
  const bool wide = a.lanes_log2 == 5;
  const int row_step = wide ? 0 : rows_per_warp, unit_step = wide ? 32 : 0;
  const int unit0 = (lane & ((1 << a.lanes_log2) - 1)) + (wide ? (int)blockIdx.y * 32 * R : 0);
  const int64_t rows_per_block = 8 * (wide ? 1 : rows_per_warp * R);
  for (int64_t row0 = blockIdx.x * rows_per_block + (threadIdx.x >> 5) * (wide ? 1 : rows_per_warp * R) + (lane >> a.lanes_log2);
       row0 < n; row0 += gridDim.x * rows_per_block) {
    float v[R][8];
#pragma unroll
    for (int j = 0; j < R; ++j) {
      const int64_t row = row0 + j * row_step;
      const int unit = unit0 + j * unit_step;
      if (row < n && unit < units) {
        const int32_t id = __ldg(a.ids + row);
        if ((uint32_t)id < (uint32_t)a.n_vocab) {
          load8(table + id * a.table_stride + unit * 8, v[j]);
        } else {
#pragma unroll
          for (int k = 0; k < 8; ++k) v[j][k] = 0;
          if (id >= 0 && unit == 0) op_status(a.status, TT_ERR_INVALID_ARG);
        }
      }
    }
#pragma unroll
    for (int j = 0; j < R; ++j) {
      const int64_t row = row0 + j * row_step;
      const int unit = unit0 + j * unit_step;
      if (row < n && unit < units) {
#pragma unroll
        for (int k = 0; k < 8; ++k) v[j][k] *= a.scale;
        store8(out + row * a.out_stride + unit * 8, v[j]);
      }
    }
  }
}

// rows that are not whole 16-byte groups: a warp a row, an element a lane
template <class TI, class TO>
__global__ void __launch_bounds__(256) k_embed_any(EmbedArgs a, const TI *__restrict__ table, TO *__restrict__ out) {
  const int64_t n = a.n_ids ? max((int64_t)0, min(*a.n_ids, a.max_ids)) : a.max_ids;
  const int lane = threadIdx.x & 31;
  for (int64_t row = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); row < n; row += (int64_t)gridDim.x * 8) {
    const int32_t id = __ldg(a.ids + row);
    const bool there = (uint32_t)id < (uint32_t)a.n_vocab;
    if (!there && id >= 0 && lane == 0 && blockIdx.y == 0) op_status(a.status, TT_ERR_INVALID_ARG);
    const TI *src = table + (there ? id : 0) * a.table_stride;
    TO *dst = out + row * a.out_stride;
    for (int64_t c = lane; c < a.dim; c += 32) dst[c] = from_f32<TO>(there ? to_f32(src[c]) * a.scale : 0.f);
  }
}

// ============================================================ tt_embed_grad
// Tokens sorted by ID with their order kept (two passes of a radix sort), then
// each row's terms summed in that order.
constexpr int SORT_THREADS = 512;
constexpr int SORT_KEYS = 8;                             // keys a thread
constexpr int SORT_TILE = SORT_THREADS * SORT_KEYS;
constexpr int MAX_BINS = 1 << 11;

struct SortArgs {
  const int64_t *n_ids;
  int64_t max_ids;
  int32_t n_vocab;
  int shift, bins;          // this pass's digit: (key >> shift) & (bins - 1)
  int tiles;
  uint32_t *hist;           // [bins][tiles]
  uint32_t *total;          // [bins]
  int32_t *status;
};

__device__ __forceinline__ int64_t count_of(const int64_t *n_ids, int64_t max_ids) {
  return n_ids ? max((int64_t)0, min(*n_ids, max_ids)) : max_ids;
}

// the key of an ID: padding sorts behind every row
__device__ __forceinline__ uint32_t key_of(int32_t id, int32_t n_vocab) {
  return (uint32_t)id < (uint32_t)n_vocab ? (uint32_t)id : (uint32_t)n_vocab;
}

// keys: of the IDs in the first pass, sorted by the low digit in the second
template <bool FIRST>
__global__ void __launch_bounds__(SORT_THREADS) k_sort_count(SortArgs a, const int32_t *__restrict__ keys) {
  __shared__ uint32_t count[MAX_BINS];
  const int64_t n = count_of(a.n_ids, a.max_ids), base = (int64_t)blockIdx.x * SORT_TILE;
  for (int i = threadIdx.x; i < a.bins; i += SORT_THREADS) count[i] = 0;
  __syncthreads();
#pragma unroll
  for (int k = 0; k < SORT_KEYS; ++k) {
    const int64_t i = base + k * SORT_THREADS + threadIdx.x;
    if (i < n) {
      const int32_t id = keys[i];
      if (FIRST && id >= a.n_vocab) op_status(a.status, TT_ERR_INVALID_ARG);
      const uint32_t key = FIRST ? key_of(id, a.n_vocab) : (uint32_t)id;
      atomicAdd(&count[(key >> a.shift) & (a.bins - 1)], 1u);
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < a.bins; i += SORT_THREADS) a.hist[(int64_t)i * a.tiles + blockIdx.x] = count[i];
}

// one block a digit: exclusive scan of its counts over the tiles
__global__ void __launch_bounds__(256) k_sort_scan(SortArgs a) {
  __shared__ uint32_t box[8];
  uint32_t *h = a.hist + (int64_t)blockIdx.x * a.tiles;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t before = 0;
  for (int base = 0; base < a.tiles; base += 256) {
    const int i = base + threadIdx.x;
    const uint32_t own = i < a.tiles ? h[i] : 0;
    uint32_t x = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_up_sync(~0u, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) box[warp] = x;
    __syncthreads();
    uint32_t add = 0, all = 0;
    for (int w = 0; w < 8; ++w) {
      add += w < warp ? box[w] : 0;
      all += box[w];
    }
    if (i < a.tiles) h[i] = before + add + x - own;
    before += all;
    __syncthreads();
  }
  if (threadIdx.x == 0) a.total[blockIdx.x] = before;
}

template <bool FIRST>
__global__ void __launch_bounds__(SORT_THREADS)
k_sort_place(SortArgs a, const int32_t *__restrict__ keys, const int32_t *__restrict__ pos, int32_t *__restrict__ keys_out,
             int32_t *__restrict__ pos_out) {
  constexpr int WARPS = SORT_THREADS / 32;
  extern __shared__ uint32_t sm[];                         // base[bins], then uint16 seen[WARPS][bins]
  __shared__ uint32_t box[WARPS];
  uint32_t *base = sm;
  uint16_t *seen = reinterpret_cast<uint16_t *>(sm + a.bins);
  const int64_t n = count_of(a.n_ids, a.max_ids), tile = (int64_t)blockIdx.x * SORT_TILE;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (tile >= n) return;
  for (int i = threadIdx.x; i < a.bins * WARPS / 2; i += SORT_THREADS) reinterpret_cast<uint32_t *>(seen)[i] = 0;
  // where each digit begins: exclusive scan of the totals, four a thread
  uint32_t t[4], x = 0;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int d = threadIdx.x * 4 + k;
    t[k] = d < a.bins ? a.total[d] : 0;
    x += t[k];
  }
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
    const int d = threadIdx.x * 4 + k;
    if (d < a.bins) base[d] = x + a.hist[(int64_t)d * a.tiles + blockIdx.x];
    x += t[k];
  }
  // rank of each key among its warp's keys of the same digit; a warp's keys
  // are SORT_KEYS consecutive groups of 32
  uint32_t key[SORT_KEYS], rank[SORT_KEYS];
#pragma unroll
  for (int k = 0; k < SORT_KEYS; ++k) {
    const int64_t i = tile + warp * (32 * SORT_KEYS) + k * 32 + lane;
    const bool there = i < n;
    key[k] = there ? (FIRST ? key_of(keys[i], a.n_vocab) : (uint32_t)keys[i]) : 0;
    const uint32_t d = there ? (key[k] >> a.shift) & (a.bins - 1) : 0xFFFFu;
    const uint32_t same = __match_any_sync(~0u, d);
    const int lead = __ffs(same) - 1;
    uint32_t s = 0;
    if (there && lane == lead) {
      s = seen[warp * a.bins + d];
      seen[warp * a.bins + d] = (uint16_t)(s + __popc(same));
    }
    rank[k] = __shfl_sync(~0u, s, lead) + __popc(same & ((1u << lane) - 1));
    __syncwarp();
  }
  __syncthreads();
  for (int d = threadIdx.x; d < a.bins; d += SORT_THREADS) {
    uint32_t before = 0;
    for (int w = 0; w < WARPS; ++w) {
      const uint32_t c = seen[w * a.bins + d];
      seen[w * a.bins + d] = (uint16_t)before;
      before += c;
    }
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < SORT_KEYS; ++k) {
    const int64_t i = tile + warp * (32 * SORT_KEYS) + k * 32 + lane;
    if (i < n) {
      const uint32_t d = (key[k] >> a.shift) & (a.bins - 1);
      const uint32_t to = base[d] + seen[warp * a.bins + d] + rank[k];
      keys_out[to] = (int32_t)key[k];
      pos_out[to] = FIRST ? (int32_t)i : pos[i];
    }
  }
}

struct GradArgs {
  const int64_t *n_ids;
  int64_t max_ids, n_vocab, dim, dout_stride, dtable_stride;
  float scale;
  int accumulate;
  const int32_t *keys, *pos;     // sorted
};

__device__ __forceinline__ int64_t lower_bound(const int32_t *keys, int64_t n, int32_t v) {
  int64_t lo = 0, hi = n;
  while (lo < hi) {
    const int64_t mid = (lo + hi) >> 1;
    if (keys[mid] < v) lo = mid + 1; else hi = mid;
  }
  return lo;
}

// a block a row of the table
template <class TI, class TO>
__global__ void __launch_bounds__(256) k_grad_rows(GradArgs a, const TI *__restrict__ dout, TO *__restrict__ dtable) {
  const int64_t n = count_of(a.n_ids, a.max_ids);
  const int32_t v = blockIdx.x;
  const int64_t lo = lower_bound(a.keys, n, v), hi = lower_bound(a.keys, n, v + 1);
  for (int64_t c = threadIdx.x; c < a.dim; c += 256) {
    float s = 0;
    for (int64_t i = lo; i < hi; ++i) s += to_f32(dout[a.pos[i] * a.dout_stride + c]);
    TO *p = dtable + v * a.dtable_stride + c;
    s *= a.scale;
    *p = from_f32<TO>(a.accumulate ? to_f32(*p) + s : s);
  }
}

// ------------------------------------------------------------ host side
bool grad_sizes_ok(int64_t max_ids, int64_t n_vocab, int64_t dim) {
  return max_ids >= 0 && max_ids <= TT_MAX_IDS && vocab_ok(n_vocab) && dim >= 1 && dim <= INT32_MAX;
}

struct GradPlan {
  int tiles = 0, bits[2] = {0, 0};
  int64_t keys[2], pos[2], hist, total, bytes;   // offsets into the workspace
};

GradPlan grad_plan(int64_t max_ids, int64_t n_vocab) {
  GradPlan p;
  int bits = 1;
  while ((n_vocab >> bits) != 0) ++bits;          // keys are 0 .. n_vocab
  p.bits[0] = (bits + 1) / 2;
  p.bits[1] = bits - p.bits[0];
  p.tiles = (int)((max_ids + SORT_TILE - 1) / SORT_TILE);
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
  p.hist = take(4 * ((int64_t)p.tiles << p.bits[0]));
  p.total = take(4 * MAX_BINS);
  p.bytes = at;
  return p;
}

}  // namespace

extern "C" tt_status tt_embed(const int32_t *d_ids, int64_t max_ids, const int64_t *d_n_ids, const void *d_table,
                              int32_t table_type, int64_t n_vocab, int64_t dim, int64_t table_stride, float scale,
                              void *d_out, int32_t out_type, int64_t out_stride, int32_t *d_status,
                              tt_stream_t stream) {
  if (!type_ok(table_type) || !type_ok(out_type) || !vocab_ok(n_vocab) || dim < 1 || dim > INT32_MAX || max_ids < 0 ||
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
        const int64_t rows = 8 * (a.lanes_log2 == 5 ? 1 : (32 >> a.lanes_log2) * 4);
        const dim3 grid((unsigned)((max_ids + rows - 1) / rows), a.lanes_log2 == 5 ? (unsigned)((units + 127) / 128) : 1);
        k_embed<TI, TO><<<grid, 256, 0, stream>>>(a, (const TI *)d_table, (TO *)d_out);
      } else {
        k_embed_any<TI, TO><<<(unsigned)((max_ids + 7) / 8), 256, 0, stream>>>(a, (const TI *)d_table, (TO *)d_out);
      }
    });
  });
  return launched("tt_embed");
}

extern "C" int64_t tt_embed_grad_workspace(int64_t max_ids, int64_t n_vocab, int64_t dim) {
  return grad_sizes_ok(max_ids, n_vocab, dim) ? grad_plan(max_ids, n_vocab).bytes : -1;
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
  const GradPlan p = grad_plan(max_ids, n_vocab);
  if (!array_ok(d_workspace, 16)) return TT_ERR_INVALID_ARG;
  if (workspace_bytes < p.bytes) return TT_ERR_CAPACITY;
  char *ws = (char *)d_workspace;
  int32_t *keys[2] = {(int32_t *)(ws + p.keys[0]), (int32_t *)(ws + p.keys[1])};
  int32_t *pos[2] = {(int32_t *)(ws + p.pos[0]), (int32_t *)(ws + p.pos[1])};
  if (max_ids > 0) {
    SortArgs s{d_n_ids, max_ids, (int32_t)n_vocab, 0, 1 << p.bits[0], p.tiles, (uint32_t *)(ws + p.hist),
               (uint32_t *)(ws + p.total), d_status};
    const auto shared = [](int bins) { return (size_t)bins * 4 + (size_t)bins * 2 * (SORT_THREADS / 32); };
    {
      cudaFuncSetAttribute(k_sort_place<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)shared(MAX_BINS));
      cudaFuncSetAttribute(k_sort_place<false>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)shared(MAX_BINS));
    }
    k_sort_count<true><<<p.tiles, SORT_THREADS, 0, stream>>>(s, d_ids);
    k_sort_scan<<<s.bins, 256, 0, stream>>>(s);
    k_sort_place<true><<<p.tiles, SORT_THREADS, shared(s.bins), stream>>>(s, d_ids, nullptr, keys[0], pos[0]);
    s.shift = p.bits[0];
    s.bins = 1 << p.bits[1];
    k_sort_count<false><<<p.tiles, SORT_THREADS, 0, stream>>>(s, keys[0]);
    k_sort_scan<<<s.bins, 256, 0, stream>>>(s);
    k_sort_place<false><<<p.tiles, SORT_THREADS, shared(s.bins), stream>>>(s, keys[0], pos[0], keys[1], pos[1]);
  }
  const GradArgs a{d_n_ids, max_ids, n_vocab, dim, dout_stride, dtable_stride, scale, accumulate != 0, keys[1], pos[1]};
  with_type(dout_type, [&](auto ti) {
    with_type(dtable_type, [&](auto to) {
      using TI = decltype(ti);
      using TO = decltype(to);
      k_grad_rows<TI, TO><<<(unsigned)n_vocab, 256, 0, stream>>>(a, (const TI *)d_dout, (TO *)d_dtable);
    });
  });
  return launched("tt_embed_grad");
}
