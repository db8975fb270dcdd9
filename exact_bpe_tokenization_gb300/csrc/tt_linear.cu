// tt_linear.cu - next-token loss of hidden states through the head's weight, and
// its gradients, without the matrix of logits (include/toktier.h).
//
//   l = H W^T,  lse_i = M + log(S),  S = sum_j exp(l_ij - M),  loss_i = (M - l_it) + log(S)
//   G_ij = g_i (exp(l_ij - lse_i) - (j == t_i)),  dH = G W,  dW = G^T H
//
// The products run on the tensor cores (tt_gemm.cuh), and what would be the logits
// never leaves them.  Three products are the least; each of them is bound by the tensor
// cores under the power limit (4096 x 100256 x 2048 bf16: 850, 860 and 897 us alone, 1.95
// to 1.87 PFLOP/s; the measured peak is 1.92).
//   The loss alone: one product, whose epilogue keeps a maximum and a sum of each row and
// 128 tokens; k_finish joins them.
//   With gradients, from bfloat16 and float: the first product's epilogue writes powers
// exp(l - l_t) in the operands' type, which has a float's range, and sums them.  S = exp(loss)
// is known behind it, so G = (powers - S (j == t)) g / S needs no second product: the factor
// g / S is a row's of dhidden, and goes into a copy of hidden for dweight (rounded there, a
// second time beside G: dweight is off by 2.1e-3 to 2.4e-3 of its size with many rows, 1.7e-3
// being its own rounding; up to 64 rows both keep a second part).  Rows of a loss beyond 41
// have G made anew.  2.76 to 3.19 ms for the sizes above, by the card and its clocks, of which
// the products are 2.61 alone; 2.95 to 3.08 from an lse, where all of G is made anew.
//   From 16-bit floats, which lack the range, the first product runs twice, for lse and for G.
// G is the one place where less than 32 bits stands between the logits and the gradients
// (float: three bfloat16 parts, whose products are added in 32 bits; what is left out is
// below 2^-24).  A chunk of rows of it is kept at a time.  dhidden's long sums are cut into
// parts that k_join adds; dweight's over chunks are kept in 32 bits.
//   Few rows are bound by reading the weight, and have kernels of their own below: 1 x 100256
// x 2048 bf16 takes 70 to 74 us with k_finish (411 MB, 6.1 TB/s in the product).
#include "tt_gemm.cuh"
#include "tt_rows.cuh"

using namespace tt::ops;
using namespace tt::gemm;
using namespace tt::linear;

namespace tt {
namespace gemm {

CUresult encode_map(CUtensorMap *map, bool bf16, const Matrix &m, uint32_t box_rows) {
  static std::atomic<void *> entry{nullptr};
  void *f = entry.load(std::memory_order_acquire);
  if (!f) {
    cudaDriverEntryPointQueryResult found;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &found) != cudaSuccess ||
        found != cudaDriverEntryPointSuccess)
      return CUDA_ERROR_NOT_FOUND;
    entry.store(f, std::memory_order_release);
  }
  const cuuint64_t dims[3] = {(cuuint64_t)m.cols, (cuuint64_t)m.rows, (cuuint64_t)m.parts};
  const cuuint64_t strides[2] = {(cuuint64_t)m.stride * 2, (cuuint64_t)m.part_stride * 2};
  const cuuint32_t box[3] = {KB, box_rows, 1}, steps[3] = {1, 1, 1};
  return reinterpret_cast<decltype(&cuTensorMapEncodeTiled)>(f)(
      map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<void *>(m.p), dims, strides, box, steps,
      CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
}

}  // namespace gemm
}  // namespace tt

namespace {

constexpr int F16_UP = 14;                                 // G in 16 bits: the largest |g| is brought to 2^13 .. 2^14

// ------------------------------------------------------------ epilogues
// 64 columns of a warp's rows to a matrix in PARTS parts of type E (each the rest of those
// before): a TMA store of 32 rows, from the warp's own memory.
template <class E, int PARTS>
__device__ __forceinline__ void put_box(const CUtensorMap *map, int row, int col, uint32_t own, float v[64], bool inside) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int p = 0; p < PARTS; ++p) {
    if (lane == 0) stores_read();
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 8; ++i) own_write(own_chunk(own, lane, i), f32_vec(v + 8 * i, E{}));
    fence_copies();
    __syncwarp();
    if (lane == 0 && inside) store_box(map, col, row, p, own);
    if (p < PARTS - 1) {
#pragma unroll
      for (int i = 0; i < 64; ++i) v[i] -= to_f32(from_f32<E>(v[i]));
    }
  }
}

// a running maximum and sum, with 64 values of columns of which n are there (the others
// become -inf); in several chains, since a warp has one other to wait with
__device__ __forceinline__ void cut64(float v[64], int n) {
  if (n < 64)
#pragma unroll
    for (int i = 0; i < 64; ++i) v[i] = i < n ? v[i] : -INF;
}
__device__ __forceinline__ void add64(const float v[64], float &m, float2 s[2]) {
  float top[4] = {v[0], v[1], v[2], v[3]};
#pragma unroll
  for (int i = 4; i < 64; i += 4)
#pragma unroll
    for (int j = 0; j < 4; ++j) top[j] = fmaxf(top[j], v[i + j]);
  top[0] = fminf(fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])), -LOWEST);
  if (top[0] > m) {
    const float by = ex2((m - top[0]) * LOG2E);
    s[0] = mul2(s[0], by);
    s[1] = mul2(s[1], by);
    m = top[0];
  }
#pragma unroll
  for (int i = 0; i < 64; i += 4)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const float2 y = sub_mul2(make_float2(v[i + 2 * j], v[i + 2 * j + 1]), m, LOG2E);
      s[j] = add2(s[j], make_float2(ex2(y.x), ex2(y.y)));
    }
}
__device__ __forceinline__ float total(const float2 s[2]) { return (s[0].x + s[0].y) + (s[1].x + s[1].y); }

// The maximum and sum of each row and 128 columns, and the target's logit.  The
// maximum stays within the finite floats, so that a difference is NaN only where a
// logit is.
struct StatsEpi {
  int n_rows, n_cols;
  const int32_t *targets;
  float2 *part;                                            // [column halves][n_rows]
  float *target_logit;                                     // [n_rows]
  __device__ __forceinline__ int begin(int row) const { return row < n_rows ? targets[row] : -1; }
  template <class Load, class Release>
  __device__ __forceinline__ void operator()(int row, int col, int, uint32_t, int t, Load load, Release release) const {
    const bool mine = row < n_rows;
    float m = LOWEST;
    float2 s[2] = {{0, 0}, {0, 0}};
    for (int c = 0; c < HALF; c += 64) {
      float v[64];
      load(c, v);
      if (c) release();
      const int n = n_cols - col - c;                      // columns that are there
      cut64(v, n);
      if ((uint32_t)(t - col - c) < 64u)
#pragma unroll
        for (int i = 0; i < 64; ++i)
          if (i == t - col - c && i < n) target_logit[row] = v[i];
      add64(v, m, s);
    }
    if (mine && col < n_cols) part[(int64_t)(col / HALF) * n_rows + row] = make_float2(m, total(s));
  }
  __device__ __forceinline__ void end() const {}
};

// The same in one pass with what G is made from: powers exp(l - c), c the target's
// logit, of which k_finish knows the sum, the row's exp(loss), later.  They are
// written in the operands' type, whose range is a float's: precise for any loss that
// is not absurd, and k_finish finds the rows for which they are not.  Where a sum
// leaves the safe range, the columns are read once more with a maximum.
template <class E, int PARTS> struct PowersEpi {
  CUtensorMap map;
  int n_rows, n_cols;
  const int32_t *targets;
  const float *from;                                       // [n_rows] c
  float2 *part;                                            // [column halves][n_rows]
  float *target_power;                                     // [n_rows]
  struct Row { int t; float c; };
  __device__ __forceinline__ Row begin(int row) const { return row < n_rows ? Row{targets[row], from[row]} : Row{-1, 0}; }
  template <class Load, class Release>
  __device__ __forceinline__ void operator()(int row, int col, int, uint32_t own, Row r, Load load, Release release) const {
    const bool mine = row < n_rows;
    const int t = r.t;
    const bool there = (uint32_t)t < (uint32_t)n_cols;
    const float c0 = r.c;
    float2 s[2] = {{0, 0}, {0, 0}}, p;
    for (int c = 0; c < HALF; c += 64) {
      float v[64];
      load(c, v);
      cut64(v, n_cols - col - c);
#pragma unroll
      for (int i = 0; i < 64; i += 2) {
        const float2 y = sub_mul2(make_float2(v[i], v[i + 1]), c0, LOG2E);
        v[i] = ex2(y.x);
        v[i + 1] = ex2(y.y);
        s[i / 2 & 1] = add2(s[i / 2 & 1], make_float2(v[i], v[i + 1]));
      }
      if (c) {
        p = make_float2(c0, total(s));
        const bool safe = p.y > 0x1p-100f && p.y < 0x1p100f;
        if (__any_sync(~0u, mine && !safe)) {
          float m = LOWEST;
          float2 again[2] = {{0, 0}, {0, 0}};
          for (int d = 0; d < HALF; d += 64) {
            float w[64];
            load(d, w);
            cut64(w, n_cols - col - d);
            add64(w, m, again);
          }
          if (!safe) p = make_float2(m, total(again));
        }
        release();
      }
      if (there && (uint32_t)(t - col - c) < 64u)
#pragma unroll
        for (int i = 0; i < 64; ++i)
          if (i == t - col - c) target_power[row] = v[i];
      if (!there)
#pragma unroll
        for (int i = 0; i < 64; ++i) v[i] = 0;
      put_box<E, PARTS>(&map, row & ~31, col + c, own, v, (row & ~31) < n_rows && col + c < n_cols);
    }
    if (mine && col < n_cols) part[(int64_t)(col / HALF) * n_rows + row] = p;
  }
  __device__ __forceinline__ void end() const { stores_done(); }
};

__device__ __forceinline__ float f16_up(const uint32_t *g_max) {
  // 2^(F16_UP - e) for a largest |g| of [2^(e-1), 2^e): what G is multiplied by
  const float g = __uint_as_float(*g_max);
  return g > 0 ? exp2f((float)min(max(F16_UP - 1 - ilogbf(g), -100), 100)) : 1.f;
}

// G, in the operands' type or in bfloat16 parts.  16-bit floats lack the range for
// a mean's 1 / n: there G is scaled by a power of two that brings the largest |g| to 2^13 ..
// 2^14, and the gradients' epilogue takes it back.
template <class E, int PARTS> struct GradEpi {
  CUtensorMap map;
  int n_rows, n_cols;
  const RowInfo *info;
  const uint32_t *g_max;                                   // or NULL
  __device__ __forceinline__ RowInfo begin(int row) const {
    RowInfo r = {0, 0, 0, -1};
    if (row < n_rows) r = info[row];
    if (g_max) {
      const float up = f16_up(g_max);
      r.mul *= up;
      r.g *= up;
    }
    return r;
  }
  template <class Load, class Release>
  __device__ __forceinline__ void operator()(int row, int col, int, uint32_t own, RowInfo r, Load load, Release release) const {
    for (int c = 0; c < HALF; c += 64) {
      float v[64];
      load(c, v);
      if (c) release();
#pragma unroll
      for (int i = 0; i < 64; i += 2) {
        float2 y = sub_mul2(make_float2(v[i], v[i + 1]), r.from, LOG2E);
        y = mul2(make_float2(ex2(y.x), ex2(y.y)), r.mul);
        v[i] = y.x;
        v[i + 1] = y.y;
      }
      if (r.t >= 0 && (uint32_t)(r.t - col - c) < 64u)
#pragma unroll
        for (int i = 0; i < 64; ++i)
          if (i == r.t - col - c) v[i] -= r.g;
      if (r.t < 0)
#pragma unroll
        for (int i = 0; i < 64; ++i) v[i] = 0;
      put_box<E, PARTS>(&map, row & ~31, col + c, own, v, (row & ~31) < n_rows && col + c < n_cols);
    }
  }
  __device__ __forceinline__ void end() const { stores_done(); }
};

// Where a gradient goes: dst = sums * scale * the row's (+ src), T the type of dst.
struct Target {
  int64_t n_rows, n_cols;
  void *dst;
  int64_t dst_stride;
  const void *src;                                         // or NULL
  int64_t src_stride;
  int32_t src_type;
  const uint32_t *g_max;                                   // 16-bit floats: what scaled G, or NULL
  const float *row_scale;                                  // or NULL; 0: a row of zeros, whatever the sums
  int vec;                                                 // rows of dst and src lie on 16-byte boundaries
  __device__ __forceinline__ float scale() const { return g_max ? 1.f / f16_up(g_max) : 1.f; }
  __device__ __forceinline__ float scaled(float x, int64_t row, float by) const {
    if (row_scale) {
      const float r = row_scale[row];
      return r == 0 ? 0.f : x * r * by;
    }
    return x * by;
  }
};

// eight elements by plain loads: what chained kernels read may have been written by the
// kernel before, so that none of it is declared constant
template <class T> __device__ __forceinline__ void plain8(const T *p, float v[8]) {
  Raw8<T> r;
#pragma unroll
  for (int i = 0; i < (int)(sizeof(T) / 2); ++i) r.w[i] = reinterpret_cast<const uint4 *>(p)[i];
  raw_f32(r, v);
}
template <class S> __device__ __forceinline__ void add8(const void *src, int64_t at, float v[8], int n, bool vec) {
  const S *p = reinterpret_cast<const S *>(src) + at;
  if (vec) {
    float w[8];
    plain8(p, w);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] += w[i];
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) v[i] += to_f32(p[i]);
  }
}

// n of eight columns of a row
template <class T> __device__ __forceinline__ void put8(const Target &o, int64_t row, int64_t col, float v[8], int n, float scale) {
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = o.scaled(v[i], row, scale);
  T *to = reinterpret_cast<T *>(o.dst) + row * o.dst_stride + col;
  const bool vec = o.vec && n == 8;
  if (o.src) {
    const int64_t at = row * o.src_stride + col;
    if (o.src_type == TT_F32) add8<float>(o.src, at, v, n, vec);
    else if (o.src_type == TT_F16) add8<__half>(o.src, at, v, n, vec);
    else add8<__nv_bfloat16>(o.src, at, v, n, vec);
  }
  if (vec) {
    store8(to, v);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) to[i] = from_f32<T>(v[i]);
  }
}

// Sums to a matrix of any alignment: through the warp's own memory, so that a warp
// writes whole lines of a few rows at a time.
template <class T> struct OutEpi {
  Target o;
  int64_t split_rows;                                      // rows between the parts of a split contraction
  __device__ __forceinline__ float begin(int) const { return o.scale(); }
  template <class Load, class Release>
  __device__ __forceinline__ void operator()(int row, int col, int split, uint32_t own, float scale, Load load, Release release) const {
    const int lane = threadIdx.x & 31, row0 = row & ~31;
    Target to = o;
    to.dst = reinterpret_cast<T *>(o.dst) + split * split_rows * o.dst_stride;
    for (int c = 0; c < HALF; c += 64) {
      float v[64];
      load(c, v);
      if (c) release();
#pragma unroll
      for (int h = 0; h < 64; h += 32) {
        const int n = (int)min((int64_t)32, o.n_cols - col - c - h), rows = (int)min((int64_t)32, o.n_rows - row0);
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 8; ++i) own_write(own_chunk(own, lane, i), f32_vec(v + h + 4 * i, float{}));
        __syncwarp();
        if (n <= 0 || rows <= 0) continue;
        const int64_t to_col = col + c + h;
        if (o.vec) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int r = i * 8 + lane / 4, k = lane % 4 * 8;
            if (r >= rows || k >= n) continue;
            float w[8];
            vec_f32(own_read(own_chunk(own, r, k / 4)), w, float{});
            vec_f32(own_read(own_chunk(own, r, k / 4 + 1)), w + 4, float{});
            put8<T>(to, row0 + r, to_col + k, w, min(8, n - k), scale);
          }
        } else if (lane < n) {
          T *q = reinterpret_cast<T *>(to.dst) + row0 * o.dst_stride + to_col + lane;
          if (rows == 32 && !o.src && !o.row_scale) {
            // the common case, in few instructions an element (with the general one's 1023 x
            // 200255 x 641 fp16's dweight took 311 us)
#pragma unroll
            for (int r = 0; r < 32; ++r) {
              *q = from_f32<T>(own_float(own_chunk(own, r, lane / 4) + (lane & 3) * 4) * scale);
              q += o.dst_stride;
            }
          } else if (rows == 32 && !o.src) {
#pragma unroll 8
            for (int r = 0; r < 32; ++r) {
              *q = from_f32<T>(o.scaled(own_float(own_chunk(own, r, lane / 4) + (lane & 3) * 4), row0 + r, scale));
              q += o.dst_stride;
            }
          } else {
            for (int r = 0; r < rows; ++r) {
              const int64_t at = row0 + r;
              float x = o.scaled(own_float(own_chunk(own, r, lane / 4) + (lane & 3) * 4), at, scale);
              if (o.src) {
                const int64_t from = at * o.src_stride + to_col + lane;
                x += o.src_type == TT_F32 ? reinterpret_cast<const float *>(o.src)[from]
                     : o.src_type == TT_F16 ? to_f32(reinterpret_cast<const __half *>(o.src)[from])
                                            : to_f32(reinterpret_cast<const __nv_bfloat16 *>(o.src)[from]);
              }
              *q = from_f32<T>(x);
              q += o.dst_stride;
            }
          }
        }
      }
    }
  }
  __device__ __forceinline__ void end() const {}
};

// The parts of a split contraction, [split][n_rows][stride] floats, stride a multiple of
// 8: eight columns by SHARE threads, which have some of the parts each.
template <class T, int SHARE> __global__ void __launch_bounds__(256) k_join(const float *part, int splits, int64_t stride, Target o) {
  let_next_start();
  wait_for_last();
  constexpr int EACH = 256 / SHARE;
  const int64_t per = (o.n_cols + 7) / 8, total = o.n_rows * per;
  const float scale = o.scale();
  const int share = threadIdx.x % SHARE;
  const int64_t step = o.n_rows * stride / 4;
  for (int64_t i0 = (int64_t)blockIdx.x * EACH; i0 < total; i0 += (int64_t)gridDim.x * EACH) {
    const int64_t i = min(i0 + threadIdx.x / SHARE, total - 1), row = i / per, col = (i - row * per) * 8;
    float v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    const float4 *p = reinterpret_cast<const float4 *>(part + row * stride + col);
#pragma unroll 4
    for (int s = share; s < splits; s += SHARE) {
      const float4 a = p[s * step], b = p[s * step + 1];
      v[0] += a.x, v[1] += a.y, v[2] += a.z, v[3] += a.w;
      v[4] += b.x, v[5] += b.y, v[6] += b.z, v[7] += b.w;
    }
#pragma unroll
    for (int o = SHARE / 2; o; o /= 2)
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] += __shfl_xor_sync(~0u, v[j], o);
    if (share == 0 && i0 + threadIdx.x / SHARE < total) put8<T>(o, row, col, v, (int)min((int64_t)8, o.n_cols - col), scale);
  }
}

// ------------------------------------------------------------ rows
// n of eight elements
template <class T> __device__ __forceinline__ void take8(const T *p, float v[8], int n, bool vec) {
  if (vec && n == 8) {
    plain8(p, v);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < n ? to_f32(p[i]) : 0.f;
  }
}
// eight elements as TMA reads them, in parts of type E
template <class E> __device__ __forceinline__ void pack8(uint16_t *to, int64_t part_stride, float v[8], int parts) {
  *reinterpret_cast<uint4 *>(to) = f32_vec(v, E{});
  for (int p = 1; p < parts; ++p) {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] -= to_f32(from_f32<E>(v[j]));
    *reinterpret_cast<uint4 *>(to + p * part_stride) = f32_vec(v, E{});
  }
}
template <class T> using Element = typename std::conditional<sizeof(T) == 2, T, __nv_bfloat16>::type;

// A matrix as TMA can read it: rows of whole 16-byte groups.
struct Pack {
  const void *x;                                           // NULL: it can as it is
  int64_t rows, stride;
  int vec;
  uint16_t *out;                                           // [parts][rows][width]
};
struct BeginArgs {
  Pack hidden, weight;
  int dim, width, n_vocab;
  const void *h, *w;                                       // hidden and weight, whose targets' logits go to:
  int64_t n_rows, h_stride, w_stride;
  int h_vec, w_vec;
  const int32_t *targets;
  float *target_logit;                                     // [n_rows], or NULL: not wanted here
  int32_t *words;                                          // and words to be cleared
  int64_t n_words;
};

template <class T> __device__ __forceinline__ void pack_group(const Pack &p, int64_t i, int dim, int width) {
  const int per = width / 8;
  const int64_t row = i / per;
  const int col = (int)(i - row * per) * 8;
  float v[8];
  take8((const T *)p.x + row * p.stride + col, v, min(8, dim - col), p.vec);
  pack8<Element<T>>(p.out + row * width + col, p.rows * width, v, sizeof(T) == 2 ? 1 : 3);
}

// What a chunk of rows begins with: operands laid out, the targets' logits (a warp a row, 0 for
// padding), words cleared.
template <class T> __global__ void __launch_bounds__(256) k_begin(BeginArgs a) {
  let_next_start();
  wait_for_last();
  const int64_t id = blockIdx.x * 256ll + threadIdx.x, step = gridDim.x * 256ll;
  const int lane = threadIdx.x & 31;
  for (int64_t i = id; i < a.n_words; i += step) a.words[i] = 0;
  if (a.target_logit)
    for (int64_t row = id / 32; row < a.n_rows; row += step / 32) {
      const int32_t t = a.targets[row];
      float sum = 0;
      if ((uint32_t)t < (uint32_t)a.n_vocab) {
        const T *h = (const T *)a.h + row * a.h_stride, *w = (const T *)a.w + t * a.w_stride;
#pragma unroll 2
        for (int c = lane * 8; c < a.dim; c += 256) {
          float x[8], y[8];
          take8(h + c, x, min(8, a.dim - c), a.h_vec);
          take8(w + c, y, min(8, a.dim - c), a.w_vec);
#pragma unroll
          for (int i = 0; i < 8; ++i) sum = fmaf(x[i], y[i], sum);
        }
      }
      sum = warp_all(sum, OpSum{});
      if (lane == 0) a.target_logit[row] = sum;
    }
  if (a.hidden.x)
    for (int64_t i = id; i < a.hidden.rows * (a.width / 8); i += step) pack_group<T>(a.hidden, i, a.dim, a.width);
  if (a.weight.x)
    for (int64_t i = id; i < a.weight.rows * (a.width / 8); i += step) pack_group<T>(a.weight, i, a.dim, a.width);
}

struct RowArgs {
  int n_rows, n_parts, n_vocab, dim;                       // rows of the chunk, whose arrays the pointers point to
  float2 *part;
  const float *row_grads, *lse_in;
  const int32_t *targets;
  float *loss, *lse;
  float *target_logit, *target_power;                      // the latter NULL: no powers
  RowInfo *info;                                           // or NULL: no gradients
  float *row_scale;
  uint32_t *g_max;                                         // or NULL
  int32_t *only, *status;
  const void *hidden;
  int64_t hidden_stride;
  int hidden_vec;
  uint16_t *scaled;                                        // hidden by its scale, [scaled_parts][n_rows][width], or NULL
  int scaled_parts;
  int width;
  uint16_t *g;
  int64_t g_stride, g_part;
  int parts;                                               // of G
};

// What G and hidden's scaled copy are made from.  With powers: G is left without the
// row's factor g / S (S their sum), which dhidden's rows and the copy of hidden for
// dweight get.  Rows of a loss beyond 41, whose powers leave what is safe, ask for G to
// be made anew from their maximum and sum, with all of their 256.
// Returned is the scale of hidden's copy (none: a row of zeros).
__device__ __forceinline__ float row_info(const RowArgs &a, int row, bool there, float m, float s, float lse, float loss, bool &none) {
  const float g = a.row_grads ? a.row_grads[row] : 1.f;
  const int t = a.targets[row];
  RowInfo r = {m, __fdividef(1.f, s) * g, g, there && lse != -INF ? t : -1};
  float row_scale = 1, hidden_scale = 1;
  if (a.target_power && r.t >= 0) {
    if (loss <= 41.f) {
      const float c = a.target_logit[row];
      s *= ex2((m - c) * LOG2E);
      r = RowInfo{c, 1.f, s, t};
      row_scale = hidden_scale = g / s;
      float x = a.target_power[row] - s;                   // the target's place in G
      __nv_bfloat16 *to = reinterpret_cast<__nv_bfloat16 *>(a.g) + row * a.g_stride + t;
      // The row's largest term by far: what G's rounding does to it in a single part, the
      // row's factor takes back, which costs the others no more than their own roundings
      // (dhidden's error 2.4e-3 -> 1.7e-3 of its size, the rounding of the result; dweight's of
      // 512 rows 2.9e-3 -> 2.3e-3).
      const float whole = __bfloat162float(__float2bfloat16_rn(x)), back = x / whole;
      if (a.parts == 1 && fabsf(back - 1.f) < 0.01f) row_scale = hidden_scale = row_scale * back;
      for (int p = 0; p < a.parts; ++p) {
        to[p * a.g_part] = __float2bfloat16_rn(x);
        x -= __bfloat162float(__float2bfloat16_rn(x));
      }
    } else {
      r = RowInfo{m, __fdividef(1.f, s), 1.f, t};
      row_scale = hidden_scale = g;
      a.only[0] = a.only[1 + row / TILE] = 1;
    }
  } else if (r.t < 0) {
    row_scale = 0;                                         // (G's zeros would not do: weight may hold NaN)
  }
  a.info[row] = r;
  a.row_scale[row] = row_scale;
  if (a.g_max && r.t >= 0 && fabsf(g) < INF) atomicMax(a.g_max, __float_as_uint(fabsf(g)));
  none = r.t < 0;
  return hidden_scale;
}

// The loss of a row.  With powers against c, the target's 32-bit logit, what is there is S
// and the target's own power, of the same product's logits: their ratio is the loss's power,
// and neither c nor what the tensor cores cut off every logit of the row stands in it.  (As
// (m - c) + log(S) it was off by what they cut off the logits alone: 8e-4 at logits of 300, so
// that a confident row's loss was below zero.)  S is a sum of powers, the target's among
// them, and no rounding brings a sum of such terms below one of them: no loss is negative.
__device__ __forceinline__ float row_loss(const RowArgs &a, int row, float m, float s, float log_s) {
  const float c = a.target_logit[row];
  if (a.target_power) {
    const float p = a.target_power[row];
    // (1 but for what the sums of c and of the product cut off; infinities and NaN go on below)
    if (p > 0x1p-16f && p < 0x1p16f) return m == c ? log1pf((s - p) / p) : (m - c) + (log_s - logf(p));
  }
  return (m - c) + log_s;
}

// R rows a block: the parts of a row are joined by 256 / R threads (or its lse is the
// caller's), and then hidden's rows copied by their scale for dweight (padding rows as
// zeros, whatever they hold).
template <class T, int R> __global__ void __launch_bounds__(256) k_finish(RowArgs a) {
  constexpr int EACH = 256 / R;
  __shared__ float2 box[256];
  __shared__ float s_scale[R];
  __shared__ int s_none[R];
  let_next_start();
  wait_for_last();
  const int r = threadIdx.x % R, j = threadIdx.x / R, row = blockIdx.x * R + r;
  float m = LOWEST, s = 0;
  if (a.lse_in) {
    if (row < a.n_rows) m = a.lse_in[row];
    s = 1;
  } else {
    auto join = [&](float2 p) {
      const float nm = fmaxf(m, p.x);
      s = s * ex2((m - nm) * LOG2E) + p.y * ex2((p.x - nm) * LOG2E);
      m = nm;
    };
    if (row < a.n_rows) {
      const float2 *p = a.part + row;
      int i = j;
      for (; i + 7 * EACH < a.n_parts; i += 8 * EACH) {
        float2 q[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) q[u] = p[(int64_t)(i + u * EACH) * a.n_rows];
        float top = q[0].x, sum = 0;
#pragma unroll
        for (int u = 1; u < 8; ++u) top = fmaxf(top, q[u].x);
        top = fmaxf(top, LOWEST);
#pragma unroll
        for (int u = 0; u < 8; ++u) sum += q[u].y * ex2((q[u].x - top) * LOG2E);
        join(make_float2(top, sum));
      }
      for (; i < a.n_parts; i += EACH) join(p[(int64_t)i * a.n_rows]);
    }
    box[threadIdx.x] = make_float2(m, s);
    for (int k = EACH / 2; k; k /= 2) {
      __syncthreads();
      if (j < k) {
        join(box[threadIdx.x + k * R]);
        box[threadIdx.x] = make_float2(m, s);
      }
    }
  }
  if (j == 0 && row < a.n_rows) {
    const float log_s = logf(s), lse = m + log_s;
    const int32_t t = a.targets[row];
    const bool there = (uint32_t)t < (uint32_t)a.n_vocab;
    if (!there && t >= 0) op_status(a.status, TT_ERR_INVALID_ARG);
    float loss = 0;
    if (!a.lse_in) {
      loss = !there ? 0.f : lse == -INF ? INF : row_loss(a, row, m, s, log_s);
      if (a.lse) a.lse[row] = lse;
      a.loss[row] = loss;
    }
    if (a.info) {
      bool none;
      s_scale[r] = row_info(a, row, there, m, s, lse, loss, none);
      s_none[r] = none;
    }
  }
  if (!a.scaled) return;
  __syncthreads();
  const int per = a.width / 8, rows = min(R, a.n_rows - blockIdx.x * R);
  for (int i = threadIdx.x; i < rows * per; i += 256) {
    const int k = i / per, c = (i - k * per) * 8;
    const int64_t at = blockIdx.x * R + k;
    float v[8];
    take8((const T *)a.hidden + at * a.hidden_stride + c, v, min(8, a.dim - c), a.hidden_vec);
    const float scale = s_scale[k];
    const bool none = s_none[k];
#pragma unroll
    for (int u = 0; u < 8; ++u) v[u] = none ? 0.f : v[u] * scale;
    uint16_t *to = a.scaled + at * a.width + c;
    if (a.scaled_parts == 3) pack8<__nv_bfloat16>(to, (int64_t)a.n_rows * a.width, v, 3);
    else pack8<Element<T>>(to, (int64_t)a.n_rows * a.width, v, a.scaled_parts);
  }
}

// ------------------------------------------------------------ few rows
// Up to 64 rows of 32-bit values: laying out the weight in parts and multiplying 256 rows,
// six times, would cost several times what reading it once costs (1 x 200256 x 2096: 1490
// us for the loss; the weight alone is 247).  Here the weight goes by asynchronous copies
// into shared memory, where ordinary 32-bit products, two at a time, take it from: 254 to 269 us
// for 1 row, 258 to 272 for 4, 266 to 276 for 8, 404 for 16, 667 for 32, 1186 for 64 (the latter bound by the
// products: 60% of their rate), where the tensor cores take 1510 to 1530 for any number up to 256.
// A warp has eight rows, or the two or four that there are; warps that are left over divide
// the contraction.
// Up to four rows of 16-bit values take the same way, for their precision: the tensor cores
// cut off their sums at each step, and a single token's loss may be a small difference of
// large logits (of 1e-4, off by a fiftieth of itself; 3.5e-4 so).  1 x 100256 x 2048 bf16: 70 to
// 74 us, 82 by the tensor cores; 4 rows 82 to 86 and 82; 8 rows would take 129.

// What a kernel for up to ROWS rows copies at a time, and how far ahead: few rows are little
// work a stage, so that larger ones pay.  With 128 bytes a token and four stages instead of 256
// and three, the loss of 1 and 4 x 100256 x 2048 bf16 takes 78 and 87 us instead of 73 and 84, of 1, 4 and
// 8 x 200256 x 2096 floats 277, 279 and 296 instead of 264, 266 and 272.
template <int ROWS> struct FewShape {
  static constexpr int EACH = ROWS < 8 ? ROWS : 8;         // rows a warp
  static constexpr int GROUPS = ROWS / EACH, SHARES = 8 / GROUPS;
  static constexpr int BYTES = ROWS <= 8 ? 256 : 128, LINE = BYTES + 16;  // of a row of the operands, and as it lies in shared memory
  static constexpr int STAGES = ROWS <= 8 ? 3 : 4;
  static constexpr int TOKENS = ROWS <= 8 ? 64 : 32;       // of k_few_hidden
  static constexpr int SHARED_LOGITS = STAGES * (128 + ROWS) * LINE;
  template <class T> static constexpr int shared_hidden() {
    const int a = STAGES * TOKENS * (128 * (int)sizeof(T) + ROWS * 4), b = SHARES * ROWS * 128 * 4;
    return a > b ? a : b;
  }
};

__device__ __forceinline__ float2 fma2(float2 x, float2 y, float2 z) {
  float2 r;
  asm("{ .reg .b64 a, b, c; mov.b64 a, {%2, %3}; mov.b64 b, {%4, %5}; mov.b64 c, {%6, %7}; fma.rn.f32x2 a, a, b, c; mov.b64 {%0, %1}, a; }"
      : "=f"(r.x), "=f"(r.y)
      : "f"(x.x), "f"(x.y), "f"(y.x), "f"(y.y), "f"(z.x), "f"(z.y));
  return r;
}
// 16 bytes of elements of which n are there (the others become zeros) from any address
template <class T> __device__ __forceinline__ void copy16(uint8_t *to, const T *from, int n, bool vec) {
  constexpr int E = 16 / sizeof(T);
  const uint32_t at = saddr(to);
  if (vec) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(at), "l"(from), "r"(max(0, min(E, n)) * (int)sizeof(T)) : "memory");
  } else if (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < E; ++i)
      asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(at + 4 * i), "l"(from + (i < n ? i : 0)), "r"(i < n ? 4 : 0) : "memory");
  } else {
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < n ? to_f32(from[i]) : 0.f;
    *reinterpret_cast<uint4 *>(to) = f32_vec(v, Element<T>{});
  }
}

// The logits of 128 tokens a block, and what becomes of them: MODE 0 maxima and sums,
// 1 powers and their sums, 2 G (see the epilogues above).
template <class T, int ROWS, int MODE>
__global__ void __launch_bounds__(256, 2) k_few_logits(RowArgs a, const T *weight, int64_t weight_stride, bool vec_w) {
  using S = FewShape<ROWS>;
  constexpr int EACH = S::EACH, GROUPS = S::GROUPS, SHARES = S::SHARES, LINE = S::LINE, STAGES = S::STAGES, STAGE = (128 + ROWS) * LINE;
  constexpr int E = 16 / sizeof(T), STEP = S::BYTES / sizeof(T), CHUNKS = S::BYTES / 16, PASS = 256 / CHUNKS;
  extern __shared__ uint4 s_few[];
  uint8_t *bytes = reinterpret_cast<uint8_t *>(s_few);
  float *stages = reinterpret_cast<float *>(s_few);
  let_next_start();
  wait_for_last();
  if (MODE == 2 && a.only && !a.only[0]) return;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, group = warp % GROUPS, share = warp / GROUPS;
  const int col0 = blockIdx.x * 128, steps = (a.dim + STEP - 1) / STEP;
  const T *hidden = (const T *)a.hidden;
  // a thread copies 16 bytes of every PASS-th row: its places are found once
  constexpr int OF_W = 128 / PASS, COPIES = OF_W + (ROWS + PASS - 1) / PASS;
  const int k0 = tid % CHUNKS * E;
  const T *from[COPIES];
  int left[COPIES];                                        // of the contraction behind its first
#pragma unroll
  for (int q = 0; q < COPIES; ++q) {
    const bool w = q < OF_W;
    const int r = tid / CHUNKS + PASS * (w ? q : q - OF_W);
    const bool there = w ? col0 + r < a.n_vocab : r < a.n_rows;
    left[q] = there ? a.dim - k0 : 0;
    from[q] = w ? weight : hidden;
    if (left[q] > 0) from[q] += w ? (col0 + r) * weight_stride + k0 : r * a.hidden_stride + k0;
  }
  auto fetch = [&](int step) {
    if (step < steps) {
      uint8_t *to = bytes + step % STAGES * STAGE + tid / CHUNKS * LINE + tid % CHUNKS * 16;
#pragma unroll
      for (int q = 0; q < COPIES; ++q) {
        if (q >= OF_W && ROWS < PASS && tid / CHUNKS >= ROWS) break;
        const int n = left[q] - step * STEP;
        copy16(to + (q < OF_W ? PASS * q : 128 + PASS * (q - OF_W)) * LINE, n > 0 ? from[q] + step * STEP : from[q], n, q < OF_W ? vec_w : a.hidden_vec);
      }
    }
    copy_group();
  };
#pragma unroll
  for (int i = 0; i < STAGES - 1; ++i) fetch(i);
  float2 acc[EACH][4];
#pragma unroll
  for (int m = 0; m < EACH; ++m)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[m][j] = make_float2(0, 0);
  for (int step = 0; step < steps; ++step) {
    copy_wait<STAGES - 2>();
    __syncthreads();
    fetch(step + STAGES - 1);
    const uint8_t *w = bytes + step % STAGES * STAGE, *h = w + (128 + group * EACH) * LINE;
#pragma unroll 1
    for (int k = share * (CHUNKS / SHARES); k < (share + 1) * (CHUNKS / SHARES); ++k) {
      float x[4][E];
#pragma unroll
      for (int j = 0; j < 4; ++j) vec_f32(*reinterpret_cast<const uint4 *>(w + (lane + 32 * j) * LINE + k * 16), x[j], T{});
#pragma unroll
      for (int m = 0; m < EACH; ++m) {
        float y[E];
        vec_f32(*reinterpret_cast<const uint4 *>(h + m * LINE + k * 16), y, T{});
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int e = 0; e < E; e += 2) acc[m][j] = fma2(make_float2(x[j][e], x[j][e + 1]), make_float2(y[e], y[e + 1]), acc[m][j]);
      }
    }
  }
  // the shares' sums side by side: [share][row][128]
  copy_wait<0>();
  __syncthreads();
#pragma unroll
  for (int m = 0; m < EACH; ++m)
#pragma unroll
    for (int j = 0; j < 4; ++j) stages[(share * ROWS + group * EACH + m) * 128 + lane + 32 * j] = acc[m][j].x + acc[m][j].y;
  __syncthreads();
  const int col = col0 + lane * 4;
  for (int row = warp; row < a.n_rows; row += 8) {
    float v[4] = {0, 0, 0, 0};
#pragma unroll
    for (int k = 0; k < SHARES; ++k) {
      const float4 x = *reinterpret_cast<const float4 *>(stages + (k * ROWS + row) * 128 + lane * 4);
      v[0] += x.x, v[1] += x.y, v[2] += x.z, v[3] += x.w;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (col + i >= a.n_vocab) v[i] = -INF;
    const int t = a.targets[row];
    auto stats = [&]() {
      float m = fmaxf(fmaxf(v[0], v[1]), fmaxf(v[2], v[3])), e = 0;
      m = fminf(fmaxf(warp_all(m, OpMax{}), LOWEST), -LOWEST);
#pragma unroll
      for (int i = 0; i < 4; ++i) e += ex2((v[i] - m) * LOG2E);
      return make_float2(m, warp_all(e, OpSum{}));
    };
    if (MODE == 0) {
      if ((uint32_t)(t - col) < 4u && t < a.n_vocab)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (i == t - col) a.target_logit[row] = v[i];
      const float2 p = stats();
      if (lane == 0) a.part[(int64_t)blockIdx.x * a.n_rows + row] = p;
      continue;
    }
    float g[4];
    if (MODE == 1) {
      const float c = a.target_logit[row];
#pragma unroll
      for (int i = 0; i < 4; ++i) g[i] = ex2((v[i] - c) * LOG2E);
      float2 p = make_float2(c, warp_all((g[0] + g[1]) + (g[2] + g[3]), OpSum{}));
      if (!(p.y > 0x1p-100f && p.y < 0x1p100f)) p = stats();
      if (lane == 0) a.part[(int64_t)blockIdx.x * a.n_rows + row] = p;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (t >= 0 && col + i == t && t < a.n_vocab) a.target_power[row] = g[i];
      if ((uint32_t)t >= (uint32_t)a.n_vocab)
#pragma unroll
        for (int i = 0; i < 4; ++i) g[i] = 0;
    } else {
      const RowInfo r = a.info[row];
#pragma unroll
      for (int i = 0; i < 4; ++i) g[i] = r.t < 0 ? 0.f : ex2((v[i] - r.from) * LOG2E) * r.mul - (col + i == r.t ? r.g : 0.f);
    }
    if (col >= a.g_stride) continue;
    uint16_t *to = a.g + row * a.g_stride + col;
#pragma unroll
    for (int p = 0; p < 3; ++p) {
      *reinterpret_cast<uint2 *>(to + p * a.g_part) = make_uint2(f32_two<__nv_bfloat16>(g[0], g[1]), f32_two<__nv_bfloat16>(g[2], g[3]));
#pragma unroll
      for (int i = 0; i < 4; ++i) g[i] -= __bfloat162float(__float2bfloat16_rn(g[i]));
    }
  }
}

// dhidden's sums over a share of the tokens, by 128 columns a block: [share][n_rows][width]
template <class T, int ROWS>
__global__ void __launch_bounds__(256, 2) k_few_hidden(RowArgs a, const T *weight, int64_t weight_stride, bool vec_w, int each, float *sums) {
  using S = FewShape<ROWS>;
  constexpr int EACH = S::EACH, GROUPS = S::GROUPS, SHARES = S::SHARES, STAGES = S::STAGES, TOKENS = S::TOKENS;
  constexpr int E = 16 / sizeof(T), ROW = 128 * sizeof(T), STAGE = TOKENS * (ROW + ROWS * 4);
  extern __shared__ uint4 s_few[];
  uint8_t *bytes = reinterpret_cast<uint8_t *>(s_few);
  float *stages = reinterpret_cast<float *>(s_few);
  let_next_start();
  wait_for_last();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, group = warp % GROUPS, share = warp / GROUPS;
  const int col0 = blockIdx.x * 128, first = blockIdx.y * each, last = min(a.n_vocab, first + each), steps = (last - first + TOKENS - 1) / TOKENS;
  // a stage: TOKENS tokens' 128 columns, and G of the rows and those tokens, [token][row]
  auto fetch = [&](int step) {
    if (step < steps) {
      uint8_t *to = bytes + step % STAGES * STAGE;
#pragma unroll
      for (int q = 0; q < TOKENS * ROW / 16 / 256; ++q) {
        const int i = tid + 256 * q, r = i / (ROW / 16), c = i % (ROW / 16) * E, token = first + step * TOKENS + r;
        const int n = token < last ? a.dim - col0 - c : 0;
        copy16(to + i * 16, n > 0 ? weight + token * weight_stride + col0 + c : weight, n, vec_w);
      }
    }
    copy_group();
  };
  const int g_row = tid / (TOKENS / 8), g_at = tid % (TOKENS / 8) * 8;  // eight tokens of a row's G
  uint4 part[3];
  auto ask = [&](int step) {
    const int token = first + step * TOKENS + g_at;
#pragma unroll
    for (int p = 0; p < 3; ++p) {
      part[p] = make_uint4(0, 0, 0, 0);
      if (step < steps && g_row < min(ROWS, a.n_rows) && token < last) part[p] = *reinterpret_cast<const uint4 *>(a.g + p * a.g_part + g_row * a.g_stride + token);
    }
  };
  auto give = [&](int step) {
    if (step >= steps || g_row >= ROWS) return;
    float *to = reinterpret_cast<float *>(bytes + step % STAGES * STAGE + TOKENS * ROW) + g_row;
    float v[8], w[8], x[8];
    vec_f32(part[0], v, __nv_bfloat16{});
    vec_f32(part[1], w, __nv_bfloat16{});
    vec_f32(part[2], x, __nv_bfloat16{});
    const int left = last - first - step * TOKENS - g_at;
#pragma unroll
    for (int i = 0; i < 8; ++i) to[(g_at + i) * ROWS] = i < left ? v[i] + (w[i] + x[i]) : 0.f;
  };
#pragma unroll
  for (int i = 0; i < STAGES - 1; ++i) fetch(i);
  ask(0);
  float2 acc[EACH][2];
#pragma unroll
  for (int m = 0; m < EACH; ++m) acc[m][0] = acc[m][1] = make_float2(0, 0);
  for (int step = 0; step < steps; ++step) {
    give(step);
    ask(step + 1);
    copy_wait<STAGES - 2>();
    __syncthreads();
    fetch(step + STAGES - 1);
    const uint8_t *w = bytes + step % STAGES * STAGE;
    const float *g = reinterpret_cast<const float *>(w + TOKENS * ROW) + group * EACH;
#pragma unroll 4
    for (int j = share; j < TOKENS; j += SHARES) {
      float x[4];
      if (sizeof(T) == 4) {
        vec_f32(*reinterpret_cast<const uint4 *>(w + j * ROW + lane * 16), x, float{});
      } else {
        const uint2 two = *reinterpret_cast<const uint2 *>(w + j * ROW + lane * 8);
        two_f32(two.x, x, Element<T>{});
        two_f32(two.y, x + 2, Element<T>{});
      }
      float y[EACH];
      if (EACH == 2) {
        const float2 two = *reinterpret_cast<const float2 *>(g + j * ROWS);
        y[0] = two.x, y[1] = two.y;
      } else {
#pragma unroll
        for (int m = 0; m < EACH; m += 4) vec_f32(*reinterpret_cast<const uint4 *>(g + j * ROWS + m), y + m, float{});
      }
#pragma unroll
      for (int m = 0; m < EACH; ++m) {
        acc[m][0] = fma2(make_float2(x[0], x[1]), make_float2(y[m], y[m]), acc[m][0]);
        acc[m][1] = fma2(make_float2(x[2], x[3]), make_float2(y[m], y[m]), acc[m][1]);
      }
    }
  }
  copy_wait<0>();
  __syncthreads();
#pragma unroll
  for (int m = 0; m < EACH; ++m)
    *reinterpret_cast<float4 *>(stages + (share * ROWS + group * EACH + m) * 128 + lane * 4) =
        make_float4(acc[m][0].x, acc[m][0].y, acc[m][1].x, acc[m][1].y);
  __syncthreads();
  const int col = col0 + lane * 4;
  for (int row = warp; row < a.n_rows; row += 8) {
    float v[4] = {0, 0, 0, 0};
#pragma unroll
    for (int k = 0; k < SHARES; ++k) {
      const float4 x = *reinterpret_cast<const float4 *>(stages + (k * ROWS + row) * 128 + lane * 4);
      v[0] += x.x, v[1] += x.y, v[2] += x.z, v[3] += x.w;
    }
    if (col < a.width) *reinterpret_cast<float4 *>(sums + ((int64_t)blockIdx.y * a.n_rows + row) * a.width + col) = make_float4(v[0], v[1], v[2], v[3]);
  }
}

// ------------------------------------------------------------ host
struct Call {
  const void *hidden, *weight;
  int32_t type;
  int64_t n, vocab, dim, hidden_stride, weight_stride;
  const int32_t *targets;
  float *loss, *lse;
  const float *lse_in, *row_grads;
  void *dhidden, *dweight;
  int64_t dhidden_stride;
  int32_t dweight_type;
  int64_t dweight_stride;
  int accumulate;
  int32_t *status;
};

// rows lie on 16-byte boundaries
inline int vec_of(const void *p, int64_t stride, int32_t type) {
  return aligned(p, 16) && stride * (int64_t)type_size(type) % 16 == 0;
}
inline bool rows_tma(const void *p, int64_t stride) { return aligned(p, 16) && stride % 8 == 0; }
inline bool needs_pack(int32_t type, const void *p, int64_t stride) { return type == TT_F32 || !rows_tma(p, stride); }

// Few columns are few threads, which wait for one part after the other: four share them
// (64 x 64 in 23 parts: 9 us, and 5 with four; 2047 x 1024 in 2 parts: 8, and 13 with four).
template <class T> void join(const float *part, int splits, int64_t stride, const Target &o, cudaStream_t stream) {
  const int64_t groups = o.n_rows * ((o.n_cols + 7) / 8);
  auto run = [&](auto k, int share) {
    const unsigned blocks = (unsigned)std::min<int64_t>((groups * share + 255) / 256, SMS * 16);
    launch_cluster(k, dim3(blocks), 256, 0, 1, true, stream, part, splits, stride, o);
  };
  if (splits >= 8 && groups < SMS * 256) run(k_join<T, 4>, 4);
  else run(k_join<T, 1>, 1);
}

// a gradient: the product a * b^T (their contraction lies across b's rows), to o
template <bool A_MN>
bool product(bool bf16, const Matrix &a, const Matrix &b, int splits, float *sums, int64_t width, int32_t type, const Target &o,
             int32_t *status, cudaStream_t stream) {
  splits = splits_of(splits, b.rows);
  if (splits > 1) {
    const Target part{o.n_rows, o.n_cols, sums, width, nullptr, 0, TT_F32, nullptr, nullptr, 1};
    if (!run_gemm<A_MN, true>(bf16, a, b, splits, 8, OutEpi<float>{part, o.n_rows}, status, stream)) return false;
    with_type(type, [&](auto t) { join<decltype(t)>(sums, splits, width, o, stream); });
    return true;
  }
  bool ok = true;
  with_type(type, [&](auto t) { ok = run_gemm<A_MN, true>(bf16, a, b, 1, 8, OutEpi<decltype(t)>{o, 0}, status, stream); });
  return ok;
}

template <class T, int ROWS, int MODE> struct FewTag {};
// f(number of rows that there is a kernel for)
template <class T, class F> void with_rows(int n, F f) {
  if (n <= 2) f(std::integral_constant<int, 2>{});
  else if (sizeof(T) == 2 || n <= 4) f(std::integral_constant<int, 4>{});
  else if (n <= 8) f(std::integral_constant<int, 8>{});
  else if (n <= 16) f(std::integral_constant<int, 16>{});
  else if (n <= 32) f(std::integral_constant<int, 32>{});
  else f(std::integral_constant<int, 64>{});
}
template <class T, int MODE> bool few_logits(const Call &c, const RowArgs &r, cudaStream_t stream) {
  bool ok = true;
  auto run = [&](auto rows) {
    constexpr int ROWS = sizeof(T) == 2 && decltype(rows)::value > 4 ? 4 : decltype(rows)::value;
    const int shared = FewShape<ROWS>::SHARED_LOGITS;
    auto k = k_few_logits<T, ROWS, MODE>;
    if (!(ok = !allow_shared<FewTag<T, ROWS, MODE>>(k, shared))) return;
    launch_cluster(k, dim3(r.n_parts), 256, shared, 1, true, stream, r, (const T *)c.weight, c.weight_stride,
                   vec_of(c.weight, c.weight_stride, c.type) != 0);
  };
  with_rows<T>(r.n_rows, run);
  return ok;
}
template <class T> bool few_hidden(const Call &c, const RowArgs &r, const Plan &p, float *sums, const Target &o, cudaStream_t stream) {
  bool ok = true;
  auto run = [&](auto rows) {
    constexpr int ROWS = sizeof(T) == 2 && decltype(rows)::value > 4 ? 4 : decltype(rows)::value;
    const int shared = FewShape<ROWS>::template shared_hidden<T>();
    auto k = k_few_hidden<T, ROWS>;
    if (!(ok = !allow_shared<FewTag<T, ROWS, 3>>(k, shared))) return;
    launch_cluster(k, dim3((unsigned)((c.dim + 127) / 128), (unsigned)p.split_h), 256, shared, 1, true, stream, r,
                   (const T *)c.weight, c.weight_stride, vec_of(c.weight, c.weight_stride, c.type) != 0, (int)few_each(c.vocab, c.dim), sums);
  };
  with_rows<T>(r.n_rows, run);
  if (ok) join<T>(sums, p.split_h, p.width, o, stream);
  return ok;
}

// the product of hidden and weight into powers, or into G, in as many parts as g has
template <class E, int PARTS> bool powers_to(const Matrix &h, const Matrix &w, const Matrix &g, const RowArgs &r, cudaStream_t stream) {
  PowersEpi<E, PARTS> e{{}, r.n_rows, r.n_vocab, r.targets, r.target_logit, r.part, r.target_power};
  if (encode_map(&e.map, true, g, 32) != CUDA_SUCCESS) return false;
  return run_gemm<false, false>(true, h, w, 1, 16, e, r.status, stream);
}
bool make_powers(const Matrix &h, const Matrix &w, const Matrix &g, const RowArgs &r, cudaStream_t stream) {
  using B = __nv_bfloat16;
  return g.parts == 1 ? powers_to<B, 1>(h, w, g, r, stream) : g.parts == 2 ? powers_to<B, 2>(h, w, g, r, stream) : powers_to<B, 3>(h, w, g, r, stream);
}
template <class E, int PARTS> bool g_to(const Matrix &h, const Matrix &w, const Matrix &g, const RowArgs &r, cudaStream_t stream) {
  const bool bf16 = !std::is_same<E, __half>::value;
  GradEpi<E, PARTS> e{{}, r.n_rows, r.n_vocab, r.info, r.g_max};
  if (encode_map(&e.map, bf16, g, 32) != CUDA_SUCCESS) return false;
  return run_gemm<false, false>(bf16, h, w, 1, 16, e, r.status, stream, r.only);
}
bool make_g(bool bf16, const Matrix &h, const Matrix &w, const Matrix &g, const RowArgs &r, cudaStream_t stream) {
  using B = __nv_bfloat16;
  if (!bf16) return g.parts == 1 ? g_to<__half, 1>(h, w, g, r, stream) : g_to<__half, 2>(h, w, g, r, stream);
  return g.parts == 1 ? g_to<B, 1>(h, w, g, r, stream) : g.parts == 2 ? g_to<B, 2>(h, w, g, r, stream) : g_to<B, 3>(h, w, g, r, stream);
}

// Rows a block of k_finish: a row alone has more threads for its parts, several read whole
// lines of them.  For 100,256 tokens (784 parts), in us, the loss alone / with hidden's copy of
// 2048, by 1, 4 and 8 rows a block: 300 rows 6/8, 6/10, 6/13; 512 rows 6.5/8.0, 6.5/9.4,
// 6.8/12.6; 1024 rows 10.7/13.4, 6.5/10.3, 7.0/13.1; 2048 rows 15/20, 7.2/11.3, 7.4/13.9; 4096
// rows 28/35, 11.7/18.9, 9.0/16.4.
template <class T> void finish(const RowArgs &r, cudaStream_t stream) {
  const int n = r.n_rows;
  if (n >= 4096) launch_cluster(k_finish<T, 8>, dim3((n + 7) / 8), 256, 0, 1, true, stream, r);
  else if (n >= 512) launch_cluster(k_finish<T, 4>, dim3((n + 3) / 4), 256, 0, 1, true, stream, r);
  else launch_cluster(k_finish<T, 1>, dim3(n), 256, 0, 1, true, stream, r);
}

bool run_chunks(const Call &c, const Plan &p, uint8_t *ws, cudaStream_t stream) {
  const int parts = c.type == TT_F32 ? 3 : 1;
  const size_t size = type_size(c.type);
  const bool bf16 = c.type != TT_F16, grad = c.dhidden || c.dweight, few = is_few(c.n, c.type);
  const int of_g = g_parts(c.n, c.type), of_h = scaled_parts(c.n, c.type);
  // a 16-bit float has no range for powers: the product runs twice, for lse and for G
  const bool powers = grad && !c.lse_in && (c.type != TT_F16 || few);
  Matrix w{c.weight, c.vocab, c.dim, c.weight_stride, parts, 8};
  const bool pack_h = !few && needs_pack(c.type, c.hidden, c.hidden_stride), pack_w = !few && needs_pack(c.type, c.weight, c.weight_stride);
  if (pack_w) w = Matrix{ws + p.weight, c.vocab, c.dim, p.width, parts, c.vocab * p.width};
  RowArgs r{};
  r.n_parts = (int)((c.vocab + HALF - 1) / HALF);
  r.n_vocab = (int)c.vocab;
  r.dim = (int)c.dim;
  r.part = (float2 *)(ws + p.part);
  r.target_logit = (float *)(ws + p.rows);
  r.row_scale = r.target_logit + 2 * p.chunk;
  r.status = c.status;
  r.hidden_stride = c.hidden_stride;
  r.hidden_vec = vec_of(c.hidden, c.hidden_stride, c.type);
  r.width = (int)p.width;
  r.parts = of_g;
  r.scaled_parts = of_h;
  r.g_stride = p.g_stride;
  r.g_part = p.chunk * p.g_stride;
  if (grad) {
    r.info = (RowInfo *)(ws + p.info);
    r.g = (uint16_t *)(ws + p.g);
    if (c.dweight) r.scaled = (uint16_t *)(ws + p.scaled);
    if (c.type == TT_F16 && !few) r.g_max = (uint32_t *)(ws + p.word);
    if (powers) {
      r.target_power = r.target_logit + p.chunk;
      r.only = (int32_t *)(ws + p.word);
    }
  }
  BeginArgs begin{};
  begin.dim = (int)c.dim;
  begin.width = (int)p.width;
  begin.n_vocab = (int)c.vocab;
  begin.w = c.weight;
  begin.h_stride = c.hidden_stride;
  begin.w_stride = c.weight_stride;
  begin.h_vec = r.hidden_vec;
  begin.w_vec = vec_of(c.weight, c.weight_stride, c.type);
  if (powers) begin.target_logit = r.target_logit;
  if (r.g_max || r.only) {
    begin.words = (int32_t *)(ws + p.word);
    begin.n_words = p.words;
  }
  for (int64_t row0 = 0; row0 < c.n; row0 += p.chunk) {
    const int n = (int)std::min(p.chunk, c.n - row0);
    r.n_rows = n;
    r.hidden = (const uint8_t *)c.hidden + row0 * c.hidden_stride * size;
    r.targets = c.targets + row0;
    r.row_grads = c.row_grads ? c.row_grads + row0 : nullptr;
    r.lse_in = c.lse_in ? c.lse_in + row0 : nullptr;
    r.loss = c.loss ? c.loss + row0 : nullptr;
    r.lse = c.lse ? c.lse + row0 : nullptr;
    const Matrix g{r.g, n, c.vocab, p.g_stride, of_g, r.g_part};
    Matrix hc{r.hidden, n, c.dim, c.hidden_stride, parts, 8};
    if (pack_h) hc = Matrix{ws + p.hidden, n, c.dim, p.width, parts, n * p.width};
    begin.hidden = Pack{pack_h ? r.hidden : nullptr, n, c.hidden_stride, r.hidden_vec, (uint16_t *)(ws + p.hidden)};
    begin.weight = Pack{pack_w && row0 == 0 ? c.weight : nullptr, c.vocab, c.weight_stride, begin.w_vec, (uint16_t *)(ws + p.weight)};
    begin.h = r.hidden;
    begin.n_rows = n;
    begin.targets = r.targets;
    const int64_t units = std::max(std::max(begin.hidden.x ? n * (p.width / 8) : 0, begin.weight.x ? c.vocab * (p.width / 8) : 0),
                                   std::max<int64_t>(powers ? n * 32ll : 0, begin.n_words));
    if (units)
      with_type(c.type, [&](auto t) {
        launch_cluster(k_begin<decltype(t)>, dim3((unsigned)std::min<int64_t>((units + 255) / 256, SMS * 16)), 256, 0, 1, true, stream, begin);
      });
    bool ok = true;
    if (few) {
      if (!c.lse_in)
        with_type(c.type, [&](auto t) { ok = powers ? few_logits<decltype(t), 1>(c, r, stream) : few_logits<decltype(t), 0>(c, r, stream); });
    } else if (powers) {
      ok = make_powers(hc, w, g, r, stream);
    } else if (!c.lse_in) {
      const StatsEpi e{n, (int)c.vocab, r.targets, r.part, r.target_logit};
      ok = run_gemm<false, false>(bf16, hc, w, 1, 16, e, c.status, stream);
    }
    if (!ok) return false;
    with_type(c.type, [&](auto t) {
      using T = decltype(t);
      finish<T>(r, stream);
      if (grad) ok = few ? few_logits<T, 2>(c, r, stream) : make_g(bf16, hc, w, g, r, stream);
    });
    if (!ok) return false;
    if (!grad) continue;
    float *sums = (float *)(ws + p.sums);
    if (c.dhidden) {
      const Target o{n, c.dim, (uint8_t *)c.dhidden + row0 * c.dhidden_stride * size, c.dhidden_stride, nullptr, 0, TT_F32, r.g_max,
                     r.row_scale, vec_of(c.dhidden, c.dhidden_stride, c.type)};
      if (few) with_type(c.type, [&](auto t) { ok = few_hidden<decltype(t)>(c, r, p, sums, o, stream); });
      else ok = product<false>(bf16, g, w, p.split_h, sums, p.width, c.type, o, c.status, stream);
      if (!ok) return false;
    }
    if (c.dweight) {
      // the sums of several chunks stay in 32 bits until the last
      const bool first = row0 == 0, last = row0 + n == c.n, own = c.dweight_type == TT_F32;
      const int vec = vec_of(c.dweight, c.dweight_stride, c.dweight_type);
      Target o{c.vocab, c.dim, c.dweight, c.dweight_stride, nullptr, 0, TT_F32, r.g_max, nullptr, vec};
      int32_t type = c.dweight_type;
      if (!last && !own) {
        o.dst = ws + p.acc;
        o.dst_stride = p.width;
        type = TT_F32;
      }
      if (first ? c.accumulate : own) {
        o.src = c.dweight;
        o.src_stride = c.dweight_stride;
        o.src_type = c.dweight_type;
      } else if (!first) {
        o.src = ws + p.acc;
        o.src_stride = p.width;
      }
      const Matrix scaled{r.scaled, n, c.dim, p.width, of_h, n * p.width};
      if (!product<true>(bf16 || few, g, scaled, p.split_w, sums, p.width, type, o, c.status, stream)) return false;
    }
  }
  if (c.n == 0 && c.dweight && !c.accumulate) {
    const Target o{c.vocab, c.dim, c.dweight, c.dweight_stride, nullptr, 0, TT_F32, nullptr, nullptr,
                   vec_of(c.dweight, c.dweight_stride, c.dweight_type)};
    with_type(c.dweight_type, [&](auto t) { join<decltype(t)>(nullptr, 0, up(c.dim, 8), o, stream); });
  }
  return true;
}

tt_status run_linear(const Call &c, void *d_workspace, int64_t workspace_bytes, cudaStream_t stream, const char *what) {
  if (!type_ok(c.type) || c.n < 0 || !vocab_ok(c.vocab) || c.dim < 1 || c.dim > MAX_WIDTH || c.hidden_stride < c.dim ||
      c.weight_stride < c.dim || !optional_ok(c.hidden, type_size(c.type)) || !optional_ok(c.targets, 4) || !optional_ok(c.loss, 4) ||
      !optional_ok(c.lse, 4) || !optional_ok(c.lse_in, 4) || !optional_ok(c.row_grads, 4) || !optional_ok(c.status, 4) ||
      !array_ok(c.weight, type_size(c.type)))
    return TT_ERR_INVALID_ARG;
  if (c.dhidden && (c.dhidden_stride < c.dim || !array_ok(c.dhidden, type_size(c.type)))) return TT_ERR_INVALID_ARG;
  if (c.dweight && (c.dweight_stride < c.dim || (c.dweight_type != TT_F32 && c.dweight_type != c.type) ||
                    !array_ok(c.dweight, type_size(c.dweight_type))))
    return TT_ERR_INVALID_ARG;
  if (c.n > TT_MAX_IDS) return TT_ERR_CAPACITY;
  if (c.n > 0 && (!c.hidden || !c.targets || !(c.lse_in || c.loss))) return TT_ERR_INVALID_ARG;
  if (c.n == 0 && !c.dweight) return TT_OK;
  const Plan p = plan_of(c.n, c.vocab, c.dim, c.type, needs_pack(c.type, c.hidden, c.hidden_stride),
                         needs_pack(c.type, c.weight, c.weight_stride), c.dhidden, c.dweight, c.dweight_type == TT_F32);
  if (!d_workspace || !aligned(d_workspace, 256)) return TT_ERR_INVALID_ARG;
  if (workspace_bytes < p.bytes) return TT_ERR_CAPACITY;
  if (!run_chunks(c, p, (uint8_t *)d_workspace, stream)) {
    const tt_status st = launched(what);
    return st == TT_OK ? TT_ERR_CUDA : st;
  }
  return launched(what);
}

}  // namespace

extern "C" tt_status tt_linear_loss(const void *d_hidden, const void *d_weight, int32_t type, int64_t n_rows, int64_t n_vocab,
                                    int64_t dim, int64_t hidden_stride, int64_t weight_stride, const int32_t *d_targets,
                                    float *d_loss, float *d_lse, const float *d_row_grads, void *d_dhidden, int64_t dhidden_stride,
                                    void *d_dweight, int32_t dweight_type, int64_t dweight_stride, int32_t accumulate,
                                    void *d_workspace, int64_t workspace_bytes, int32_t *d_status, tt_stream_t stream) {
  const Call c{d_hidden, d_weight, type, n_rows, n_vocab, dim, hidden_stride, weight_stride, d_targets, d_loss, d_lse, nullptr,
               d_row_grads, d_dhidden, d_dweight, dhidden_stride, dweight_type, dweight_stride, accumulate, d_status};
  return run_linear(c, d_workspace, workspace_bytes, stream, "tt_linear_loss");
}

extern "C" tt_status tt_linear_loss_grad(const void *d_hidden, const void *d_weight, int32_t type, int64_t n_rows, int64_t n_vocab,
                                         int64_t dim, int64_t hidden_stride, int64_t weight_stride, const int32_t *d_targets,
                                         const float *d_lse, const float *d_row_grads, void *d_dhidden, int64_t dhidden_stride,
                                         void *d_dweight, int32_t dweight_type, int64_t dweight_stride, int32_t accumulate,
                                         void *d_workspace, int64_t workspace_bytes, int32_t *d_status, tt_stream_t stream) {
  if (n_rows > 0 && (!d_lse || (!d_dhidden && !d_dweight))) return TT_ERR_INVALID_ARG;
  const Call c{d_hidden, d_weight, type, n_rows, n_vocab, dim, hidden_stride, weight_stride, d_targets, nullptr, nullptr, d_lse,
               d_row_grads, d_dhidden, d_dweight, dhidden_stride, dweight_type, dweight_stride, accumulate, d_status};
  return run_linear(c, d_workspace, workspace_bytes, stream, "tt_linear_loss_grad");
}

extern "C" int64_t tt_linear_loss_workspace(int64_t n_rows, int64_t n_vocab, int64_t dim, int32_t type, int32_t aligned_rows,
                                            int32_t dweight_type, int32_t want_grad) {
  if (!type_ok(type) || n_rows < 0 || n_rows > TT_MAX_IDS || !vocab_ok(n_vocab) || dim < 1 || dim > MAX_WIDTH ||
      (want_grad && dweight_type != TT_F32 && dweight_type != type))
    return -1;
  const bool pack = type == TT_F32 || !aligned_rows;
  return plan_of(n_rows, n_vocab, dim, type, pack, pack, want_grad != 0, want_grad != 0, dweight_type == TT_F32).bytes;
}
