// The sum of one workgroup's 64 columns of parts (partial_sums.hip), for
// kernels that do it beside other work.
#pragma once

#include "common.h"

namespace m2 {

constexpr int kSumWaves = 16;
constexpr int kSumLoads = 8;  // rows in flight per wavefront

struct SumOuts {
  float* p[3];
  int64_t end[3];
};

// Workgroup `block` of 64 * kSumWaves threads; red: LDS of its own.
__device__ __forceinline__ void sum_columns(const float* __restrict__ part, int64_t P, int64_t M,
                                            const SumOuts& out, int64_t block,
                                            float (*red)[64]) {
  const int lane = lane_id(), wave = wave_id();
  const int64_t m = block * 64 + lane;
  float s = 0.f;
  if (m < M) {
    int64_t p = wave;
    for (; p + (kSumLoads - 1) * kSumWaves < P; p += kSumLoads * kSumWaves) {
      float v[kSumLoads];
#pragma unroll
      for (int i = 0; i < kSumLoads; ++i) v[i] = part[(p + i * kSumWaves) * M + m];
#pragma unroll
      for (int n = kSumLoads / 2; n >= 1; n /= 2)
#pragma unroll
        for (int i = 0; i < n; ++i) v[i] += v[i + n];
      s += v[0];
    }
    for (; p < P; p += kSumWaves) s += part[p * M + m];
  }
  red[wave][lane] = s;
  __syncthreads();
  if (wave || m >= M) return;
  s = red[0][lane];
#pragma unroll
  for (int o = 1; o < kSumWaves; ++o) s += red[o][lane];
  const int i = m < out.end[0] ? 0 : m < out.end[1] ? 1 : 2;
  if (out.p[i]) out.p[i][m - (i ? out.end[i - 1] : 0)] = s;
}

inline SumOuts sum_outs(const int64_t ends[3], float* const outs[3]) {
  SumOuts o;
  for (int i = 0; i < 3; ++i) {
    o.p[i] = outs[i];
    o.end[i] = ends[i];
  }
  return o;
}

}  // namespace m2
