// tt_ops.cuh - what the operators around token IDs share: element types,
// 16-byte vector loads and stores, argument checks and block reductions.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>
#include <stdio.h>

#include <atomic>

#include "../../include/toktier.h"

namespace tt {
namespace ops {

constexpr int64_t MAX_VOCAB = 1 << 20;
constexpr int64_t MAX_DIM = 1 << 24;
constexpr float INF = __builtin_huge_valf();

// ------------------------------------------------------------ elements
__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
template <class T> __device__ __forceinline__ T from_f32(float x);
template <> __device__ __forceinline__ float from_f32<float>(float x) { return x; }
template <> __device__ __forceinline__ __half from_f32<__half>(float x) { return __float2half_rn(x); }
template <> __device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

// eight elements as they lie in memory, and as floats
template <class T> struct Raw8 { uint4 w[sizeof(T) / 2]; };
template <class T> __device__ __forceinline__ void load_raw(const T *p, Raw8<T> &r) {
#pragma unroll
  for (int i = 0; i < (int)(sizeof(T) / 2); ++i) r.w[i] = __ldg(reinterpret_cast<const uint4 *>(p) + i);
}
__device__ __forceinline__ void two_f32(uint32_t w, float *v, __half) {
  const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w));
  v[0] = f.x;
  v[1] = f.y;
}
__device__ __forceinline__ void two_f32(uint32_t w, float *v, __nv_bfloat16) {
  v[0] = __uint_as_float(w << 16);
  v[1] = __uint_as_float(w & 0xFFFF0000u);
}
template <class T> __device__ __forceinline__ void raw_f32(const Raw8<T> &r, float v[8]) {
  const uint32_t w[4] = {r.w[0].x, r.w[0].y, r.w[0].z, r.w[0].w};
#pragma unroll
  for (int i = 0; i < 4; ++i) two_f32(w[i], v + 2 * i, T{});
}
__device__ __forceinline__ void raw_f32(const Raw8<float> &r, float v[8]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    v[4 * i] = __uint_as_float(r.w[i].x);
    v[4 * i + 1] = __uint_as_float(r.w[i].y);
    v[4 * i + 2] = __uint_as_float(r.w[i].z);
    v[4 * i + 3] = __uint_as_float(r.w[i].w);
  }
}

// eight elements to a 16-byte aligned address, marked as not to be read soon
__device__ __forceinline__ void store8(float *p, const float v[8]) {
  __stcs(reinterpret_cast<float4 *>(p), make_float4(v[0], v[1], v[2], v[3]));
  __stcs(reinterpret_cast<float4 *>(p) + 1, make_float4(v[4], v[5], v[6], v[7]));
}
__device__ __forceinline__ void op_status(int32_t *st, int code) {
  if (st) atomicCAS(st, TT_OK, code);
}

// ------------------------------------------------------------ checks
inline size_t type_size(int32_t t) { return t == TT_F32 ? 4 : 2; }
inline bool type_ok(int32_t t) { return t == TT_F32 || t == TT_F16 || t == TT_BF16; }
inline bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
inline bool array_ok(const void *p, size_t elem) { return p && aligned(p, elem); }
inline bool optional_ok(const void *p, size_t elem) { return !p || aligned(p, elem); }
inline bool vocab_ok(int64_t n_vocab) { return n_vocab >= 1 && n_vocab <= MAX_VOCAB; }
// rows of whole 16-byte groups of eight elements
inline bool rows_vector(const void *p, int64_t stride, int64_t dim) {
  return aligned(p, 16) && stride % 8 == 0 && dim % 8 == 0;
}

inline tt_status launched(const char *what) {
  const cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess) return TT_OK;
  fprintf(stderr, "toktier: %s failed: %s\n", what, cudaGetErrorString(e));
  return TT_ERR_CUDA;
}

// Let a kernel use so much dynamic shared memory, once a device (Tag: the
// kernel's own type); true if that failed.
template <class Tag, class K> inline bool allow_shared(K kernel, int bytes) {
  static std::atomic<uint64_t> done{0};
  int dev = 0;
  cudaGetDevice(&dev);
  const uint64_t bit = 1ull << (dev & 63);
  if (done.load(std::memory_order_relaxed) & bit) return false;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess) return true;
  done.fetch_or(bit, std::memory_order_relaxed);
  return false;
}

// call f(T{}) with the element type of a tt_dtype
template <class F> void with_type(int32_t t, F f) {
  if (t == TT_F32) f(float{});
  else if (t == TT_F16) f(__half{});
  else f(__nv_bfloat16{});
}

// ------------------------------------------------------------ block reductions
struct OpMax { template <class V> __device__ V operator()(V a, V b) const { return a > b ? a : b; } };
struct OpSum { template <class V> __device__ V operator()(V a, V b) const { return a + b; } };

template <class V, class Op> __device__ __forceinline__ V warp_all(V v, Op op) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v = op(v, __shfl_xor_sync(~0u, v, o));
  return v;
}

// every thread gets the reduction over the block; `box` holds one V per warp
template <class V, class Op> __device__ V block_all(V v, Op op, V *box) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, n = blockDim.x >> 5;
  v = warp_all(v, op);
  __syncthreads();
  if (lane == 0) box[warp] = v;
  __syncthreads();
  v = box[0];
  for (int i = 1; i < n; ++i) v = op(v, box[i]);
  return v;
}

// ------------------------------------------------------------ clusters
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// whole warps arrive and wait
__device__ __forceinline__ void cluster_arrive() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  __syncwarp();
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_sync() {
  cluster_arrive();
  cluster_wait();
}
// the same variable of another block of the cluster
template <class V> __device__ __forceinline__ V *of_block(V *p, uint32_t rank) {
  uint64_t a;
  asm volatile("mapa.u64 %0, %1, %2;" : "=l"(a) : "l"(reinterpret_cast<uint64_t>(p)), "r"(rank));
  return reinterpret_cast<V *>(a);
}

// 16 bytes from global to shared memory behind the thread's back; groups of
// copies end in order
__device__ __forceinline__ void copy_async(uint4 *to, const uint4 *from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((uint32_t)__cvta_generic_to_shared(to)), "l"(from) : "memory");
}
__device__ __forceinline__ void copy_group() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void copy_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// 2^x, results below the normal range as zero
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// (x - y) * z of two values at once
__device__ __forceinline__ float2 sub_mul2(float2 x, float y, float z) {
  float2 r;
  asm("{ .reg .b64 a, b, c; mov.b64 a, {%2, %3}; mov.b64 b, {%4, %4}; mov.b64 c, {%5, %5};\n\t"
      "add.rn.f32x2 a, a, b; mul.rn.f32x2 a, a, c; mov.b64 {%0, %1}, a; }"
      : "=f"(r.x), "=f"(r.y)
      : "f"(x.x), "f"(x.y), "f"(-y), "f"(z));
  return r;
}

// two sums, or products with the same factor, at once
__device__ __forceinline__ float2 add2(float2 x, float2 y) {
  float2 r;
  asm("{ .reg .b64 a, b; mov.b64 a, {%2, %3}; mov.b64 b, {%4, %5}; add.rn.f32x2 a, a, b; mov.b64 {%0, %1}, a; }"
      : "=f"(r.x), "=f"(r.y)
      : "f"(x.x), "f"(x.y), "f"(y.x), "f"(y.y));
  return r;
}
__device__ __forceinline__ float2 mul2(float2 x, float z) {
  float2 r;
  asm("{ .reg .b64 a, b; mov.b64 a, {%2, %3}; mov.b64 b, {%4, %4}; mul.rn.f32x2 a, a, b; mov.b64 {%0, %1}, a; }"
      : "=f"(r.x), "=f"(r.y)
      : "f"(x.x), "f"(x.y), "f"(z));
  return r;
}

// the largest of a 16-byte vector's elements that are not NaN (NaN if all are)
__device__ __forceinline__ float vec_max(uint4 r, float) {
  return fmaxf(fmaxf(__uint_as_float(r.x), __uint_as_float(r.y)), fmaxf(__uint_as_float(r.z), __uint_as_float(r.w)));
}
template <class T2> __device__ __forceinline__ T2 as_two(uint32_t w) { return *reinterpret_cast<T2 *>(&w); }
__device__ __forceinline__ float vec_max(uint4 r, __half) {
  const __half2 m = __hmax2(__hmax2(as_two<__half2>(r.x), as_two<__half2>(r.y)), __hmax2(as_two<__half2>(r.z), as_two<__half2>(r.w)));
  return fmaxf(__low2float(m), __high2float(m));
}
__device__ __forceinline__ float vec_max(uint4 r, __nv_bfloat16) {
  const __nv_bfloat162 m = __hmax2(__hmax2(as_two<__nv_bfloat162>(r.x), as_two<__nv_bfloat162>(r.y)),
                                   __hmax2(as_two<__nv_bfloat162>(r.z), as_two<__nv_bfloat162>(r.w)));
  return fmaxf(__low2float(m), __high2float(m));
}

// A row of elements as a scalar lead up to the first 16-byte boundary, whole
// 16-byte vectors, and a scalar rest.
template <class T> struct RowParts {
  static constexpr int E = 16 / sizeof(T);
  int lead, vecs, rest;
  __device__ __forceinline__ RowParts(const T *p, int n) {
    lead = min(n, (int)((16 - (reinterpret_cast<uintptr_t>(p) & 15)) & 15) / (int)sizeof(T));
    vecs = (n - lead) / E;
    rest = n - lead - vecs * E;
  }
  // the scalar element of a thread of the block's first warp (at most seven lie
  // ahead of the vectors and seven behind them), or -1
  __device__ __forceinline__ int scalar(int tid) const {
    return tid < lead ? tid : tid >= 16 && tid < 16 + rest ? lead + vecs * E + tid - 16 : -1;
  }
};

__device__ __forceinline__ void vec_f32(uint4 r, float v[4], float) {
  v[0] = __uint_as_float(r.x);
  v[1] = __uint_as_float(r.y);
  v[2] = __uint_as_float(r.z);
  v[3] = __uint_as_float(r.w);
}
template <class T> __device__ __forceinline__ void vec_f32(uint4 r, float v[8], T) {
  two_f32(r.x, v, T{});
  two_f32(r.y, v + 2, T{});
  two_f32(r.z, v + 4, T{});
  two_f32(r.w, v + 6, T{});
}
__device__ __forceinline__ uint4 f32_vec(const float v[4], float) {
  return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
}
template <class T> __device__ __forceinline__ uint32_t f32_two(float a, float b);
template <> __device__ __forceinline__ uint32_t f32_two<__half>(float a, float b) {
  __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<uint32_t *>(&h);
}
template <> __device__ __forceinline__ uint32_t f32_two<__nv_bfloat16>(float a, float b) {
  __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<uint32_t *>(&h);
}
template <class T> __device__ __forceinline__ uint4 f32_vec(const float v[8], T) {
  return make_uint4(f32_two<T>(v[0], v[1]), f32_two<T>(v[2], v[3]), f32_two<T>(v[4], v[5]), f32_two<T>(v[6], v[7]));
}

template <class T> __device__ __forceinline__ void store8(T *p, const float v[8]) {
  __stcs(reinterpret_cast<uint4 *>(p), f32_vec(v, T{}));
}

// A kernel launched with launch_chained may start when the blocks of the one
// before have all called let_next_start() or ended; what it does before
// wait_for_last() must not depend on that kernel.
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_last() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// launch on clusters of `cluster` blocks along x
template <class... P, class... A>
inline void launch_cluster(void (*f)(P...), dim3 grid, unsigned threads, size_t shared, unsigned cluster, bool chained,
                           cudaStream_t stream, A... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = shared;
  cfg.stream = stream;
  cudaLaunchAttribute at[2]{};
  if (cluster > 1) {
    at[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
    at[cfg.numAttrs].val.clusterDim.x = cluster;
    at[cfg.numAttrs].val.clusterDim.y = at[cfg.numAttrs].val.clusterDim.z = 1;
    ++cfg.numAttrs;
  }
  if (chained) {
    at[cfg.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[cfg.numAttrs].val.programmaticStreamSerializationAllowed = 1;
    ++cfg.numAttrs;
  }
  cfg.attrs = at;
  cudaLaunchKernelEx(&cfg, f, static_cast<P>(args)...);
}

}  // namespace ops
}  // namespace tt
