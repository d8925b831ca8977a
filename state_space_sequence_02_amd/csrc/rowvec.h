// Row-vector access of the kernels around the SSD (conv1d, selective scan,
// norm): V consecutive elements of a row as float32 registers, 16 bytes at a
// time where V * sizeof(T) is 16, one element where V is 1 (rows whose length
// or stride is no multiple of 16 bytes).  Also the activations they share.
#pragma once

#include "common.h"

namespace m2 {

// Elements of one 16-byte access.
template <typename T>
constexpr int vec_of() { return 16 / (int)sizeof(T); }

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(bf16 v) { return bf2f(v); }
template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ bf16 from_f32<bf16>(float v) { return f2bf(v); }

template <typename T, int V>
struct RowVec {
  typedef T type __attribute__((ext_vector_type(V)));
};
template <typename T>
struct RowVec<T, 1> {
  typedef T type;
};

template <typename T, int V>
using raw_t = typename RowVec<T, V>::type;

// Element e of a loaded vector.  Rows that wait for their turn stay in their
// own type: as float32, bfloat16 rows would hold twice the registers.
template <typename T, int V>
__device__ __forceinline__ float elem(const raw_t<T, V>& r, int e) {
  if constexpr (V == 1)
    return to_f32(r);
  else
    return to_f32(r[e]);
}

template <typename T, int V>
__device__ __forceinline__ void load_row(const T* p, float (&v)[V]) {
  const raw_t<T, V> r = *(const raw_t<T, V>*)p;
#pragma unroll
  for (int e = 0; e < V; ++e) v[e] = elem<T, V>(r, e);
}

template <typename T, int V>
__device__ __forceinline__ void store_row(T* p, const float (&v)[V]) {
  if constexpr (V == 1) {
    *p = from_f32<T>(v[0]);
  } else {
    raw_t<T, V> r;
#pragma unroll
    for (int e = 0; e < V; ++e) r[e] = from_f32<T>(v[e]);
    *(raw_t<T, V>*)p = r;
  }
}

// 1 / (1 + exp(-v)).  exp2 overflows to infinity far below zero, whose
// reciprocal is the right zero.
__device__ __forceinline__ float sigmoid_f32(float v) {
  return __builtin_amdgcn_rcpf(1.f + fast_exp2(-kLog2e * v));
}

// softplus(v) = max(v, 0) + log(1 + e), e = exp(-|v|).  The logarithm is
// 2 atanh(s) with s = e / (2 + e) <= 1/3, summed as an odd series: relative
// accuracy is kept where e is small (time steps of 1e-3 sit near v = -7),
// where forming 1 + e first would lose it.  The terms left out are below
// s^18 / 19 < 2^-32 of the value.
__device__ __forceinline__ float softplus_f32(float v) {
  const float e = fast_exp2(-kLog2e * __builtin_fabsf(v));
  const float s = e * __builtin_amdgcn_rcpf(2.f + e);
  const float q = s * s;
  float p = 1.f / 17;
  p = __builtin_fmaf(p, q, 1.f / 15);
  p = __builtin_fmaf(p, q, 1.f / 13);
  p = __builtin_fmaf(p, q, 1.f / 11);
  p = __builtin_fmaf(p, q, 1.f / 9);
  p = __builtin_fmaf(p, q, 1.f / 7);
  p = __builtin_fmaf(p, q, 1.f / 5);
  p = __builtin_fmaf(p, q, 1.f / 3);
  p = __builtin_fmaf(p, q, 1.f);
  return __builtin_fmaxf(v, 0.f) + 2.f * s * p;
}

}  // namespace m2
