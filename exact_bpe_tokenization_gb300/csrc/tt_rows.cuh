// tt_rows.cuh - what the losses over rows of logits share: the running maximum and
// sum of a softmax, and the walk over a row's vectors.
#pragma once
#include "tt_ops.cuh"

namespace tt {
namespace ops {

constexpr float LOG2E = 1.44269504f;
constexpr float LOWEST = -3.402823466e38f;

// A running maximum and the sum of exp(l - maximum), or with SCALED of powers of
// another base, 2^(c (l - maximum)).  The maximum stays within
// the finite floats, so that a difference is NaN only where a logit is: +inf
// adds +inf to the sum, -inf nothing.
template <bool SCALED> struct Running {
  float c = LOG2E;                               // SCALED: times another factor
  float m = LOWEST;
  float2 s2 = make_float2(0, 0);                 // the sum in two halves
  float s;                                       // and whole, from total() on
  __device__ __forceinline__ float factor() const { return SCALED ? c : LOG2E; }
  template <class T> __device__ __forceinline__ void add(uint4 r, T) {
    constexpr int E = 16 / sizeof(T);
    const float vm = vec_max(r, T{});
    if (vm > m) raise(vm);
    float v[E];
    vec_f32(r, v, T{});
#pragma unroll
    for (int i = 0; i < E; i += 2) {
      const float2 y = sub_mul2(make_float2(v[i], v[i + 1]), m, factor());
      s2 = add2(s2, make_float2(ex2(y.x), ex2(y.y)));
    }
  }
  __device__ __forceinline__ void add(float x) {
    if (x > m) raise(x);
    s2.x += ex2((x - m) * factor());
  }
  __device__ __forceinline__ void raise(float vm) {
    vm = fminf(vm, -LOWEST);
    s2 = mul2(s2, ex2((m - vm) * factor()));
    m = vm;
  }
  __device__ __forceinline__ void total() { s = s2.x + s2.y; }
  __device__ __forceinline__ void join(float om, float os) {
    const float nm = fmaxf(m, om);
    s = s * ex2((m - nm) * factor()) + os * ex2((om - nm) * factor());
    m = nm;
  }
};

// f(vector, whether all of the group's are there) for groups of `per` vectors
// a thread between lo and hi: the tests of whole groups are left out.
template <bool WHOLE> struct Whole { static constexpr bool value = WHOLE; };
template <int THREADS, class F> __device__ __forceinline__ void groups(int lo, int hi, int per, F f) {
  for (; lo + per * THREADS <= hi; lo += per * THREADS) f(lo + (int)threadIdx.x, Whole<true>{});
  if (lo < hi) f(lo + (int)threadIdx.x, Whole<false>{});
}

}  // namespace ops
}  // namespace tt
