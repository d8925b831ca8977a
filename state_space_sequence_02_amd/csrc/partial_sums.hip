// partial_sums: the last step of every gradient that is a sum over tokens.
// The kernels before it leave rows of float32 parts [P][M], one row for each
// of their workgroups; here out[m] = sum_p part[p][m], in a fixed order, so
// a gradient has the same bits each time (no atomics).  Columns go to up to
// three outputs: [0, end0) to the first, [end0, end1) to the second and
// [end1, end2) to the third; an output that is NULL is not written.  A
// workgroup sums 64 columns, each of its 16 wavefronts every sixteenth row.
#include "launch.h"
#include "partial_sums.h"

namespace m2 {

namespace {

__global__ void __launch_bounds__(64 * kSumWaves) partial_sums_kernel(
    const float* __restrict__ part, int64_t P, int64_t M, SumOuts out) {
  __shared__ float red[kSumWaves][64];
  sum_columns(part, P, M, out, blockIdx.x, red);
}

}  // namespace

hipError_t launch_partial_sums(const float* part, int64_t P, int64_t M, const int64_t ends[3],
                               float* const outs[3], hipStream_t s) {
  partial_sums_kernel<<<(unsigned)((M + 63) / 64), 64 * kSumWaves, 0, s>>>(part, P, M,
                                                                           sum_outs(ends, outs));
  return hipGetLastError();
}

}  // namespace m2
