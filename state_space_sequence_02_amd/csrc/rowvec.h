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

// Lanes of a row of 16 rotated by CTRL - 0x120, or another DPP control.
template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
  return __builtin_bit_cast(
      float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xf, 0xf, true));
}

// v + the same of the lane whose number differs in bit 5 (4): the two halves
// of a register pair that is exchanged with itself.
__device__ __forceinline__ float add_xor32(float v) {
  const unsigned u = __builtin_bit_cast(unsigned, v);
  const auto s = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  const unsigned x = s[0], y = s[1];  // a bit cast of s[1] itself reads s[0]
  return __builtin_bit_cast(float, x) + __builtin_bit_cast(float, y);
}
__device__ __forceinline__ float add_xor16(float v) {
  const unsigned u = __builtin_bit_cast(unsigned, v);
  const auto s = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  const unsigned x = s[0], y = s[1];
  return __builtin_bit_cast(float, x) + __builtin_bit_cast(float, y);
}

// Sum over LANES = 32 or 64 neighbouring lanes, in each of them: rotations
// inside the rows of 16, then the exchanges between rows.
template <int LANES>
__device__ __forceinline__ float lanes_sum(float v) {
  v += dpp<0x121>(v);
  v += dpp<0x122>(v);
  v += dpp<0x124>(v);
  v += dpp<0x128>(v);
  v = add_xor16(v);
  if constexpr (LANES == 64) v = add_xor32(v);
  return v;
}

// Element of a row whose address is the same for the wavefront, at this lane's
// offset in bytes: one instruction with a scalar address and a 32-bit offset.
template <typename T>
__device__ __forceinline__ const T& lane_at(const T* row, unsigned bytes) {
  return *(const T*)((const char*)row + bytes);
}
template <typename T>
__device__ __forceinline__ T& lane_at(T* row, unsigned bytes) {
  return *(T*)((char*)row + bytes);
}

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

constexpr float kLn2 = 0.693147180559945309417f;

// 1 / (1 + exp(-v)).  exp2 overflows to infinity far below zero, whose
// reciprocal is the right zero.
__device__ __forceinline__ float sigmoid_f32(float v) {
  return __builtin_amdgcn_rcpf(1.f + fast_exp2(-kLog2e * v));
}

// softplus(v) = max(v, 0) + log(1 + e), e = exp(-|v|).  x = 1 + e rounded
// loses what is small in e (time steps of 1e-3 sit near v = -7); e - (x - 1)
// is exactly what was lost, and log(x) + that is the logarithm to second
// order in it.  Measured over [-15, 20]: within 18 steps of 2^-24 relative,
// most of it the exponent's own rounding, 1.44 |v| of them.
__device__ __forceinline__ float softplus_f32(float v) {
  const float e = fast_exp2(-kLog2e * __builtin_fabsf(v));
  const float x = 1.f + e;
  const float lost = e - (x - 1.f);
  return __builtin_fmaxf(v, 0.f) + __builtin_fmaf(__builtin_amdgcn_logf(x), kLn2, lost);
}

}  // namespace m2
