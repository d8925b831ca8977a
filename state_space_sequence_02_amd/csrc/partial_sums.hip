// partial_sums: the last step of every gradient that is a sum over tokens.
// The kernels before it leave rows of float32 parts [P][M], one row for each
// of their workgroups; here out[m] = sum_p part[p][m], in a fixed order, so
// a gradient has the same bits each time (no atomics).  Columns go to up to
// three outputs: [0, end0) to the first, [end0, end1) to the second and
// [end1, end2) to the third; an output that is NULL is not written.  A
// workgroup sums 64 columns, each of its 16 wavefronts every sixteenth row.
#include "common.h"
#include "launch.h"

namespace m2 {

namespace {

constexpr int kSumWaves = 16;
constexpr int kSumLoads = 8;  // rows in flight per wavefront

struct Outs {
  float* p[3];
  int64_t end[3];
};

__global__ void __launch_bounds__(64 * kSumWaves) partial_sums_kernel(
    const float* __restrict__ part, int64_t P, int64_t M, Outs out) {
  __shared__ float red[kSumWaves][64];
  const int lane = lane_id(), wave = wave_id();
  const int64_t m = (int64_t)blockIdx.x * 64 + lane;
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

}  // namespace

hipError_t launch_partial_sums(const float* part, int64_t P, int64_t M, const int64_t ends[3],
                               float* const outs[3], hipStream_t s) {
  Outs o;
  for (int i = 0; i < 3; ++i) {
    o.p[i] = outs[i];
    o.end[i] = ends[i];
  }
  partial_sums_kernel<<<(unsigned)((M + 63) / 64), 64 * kSumWaves, 0, s>>>(part, P, M, o);
  return hipGetLastError();
}

}  // namespace m2
