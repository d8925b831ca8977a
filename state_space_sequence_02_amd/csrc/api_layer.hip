// C ABI of the operators around the SSD (conv1d, selective_scan, norm):
// argument checks on the host and stream-ordered launches.  Declarations and
// the contract of every entry point are in include/mamba2_ssd.h.
#include <math.h>
#include <stdint.h>

#include "launch.h"
#include "mamba2_ssd.h"
#include "status.h"

namespace {

using m2::fail;
using m2::hip_status;
using m2::maybe;
using m2::need;
using m2::need_workspace;
using m2::ok;
using m2::round256;

// Bounds that keep every index inside 64 bits and every grid inside the
// launch limits (2^32 threads along x, 65535 workgroups along y).
constexpr int64_t kMaxBatch = 65535;
constexpr int64_t kMaxTokens = (int64_t)1 << 30;    // batch * seqlen, and rows of a norm
constexpr int64_t kMaxChannels = (int64_t)1 << 20;
constexpr int64_t kMaxStride = (int64_t)1 << 24;    // elements between tokens
constexpr int64_t kMaxUnits = (int64_t)1 << 31;     // channels * batch * ceil(seqlen / 8)
constexpr int64_t kMaxRows = (int64_t)1 << 26;      // batch * channels of a scan
constexpr int64_t kMaxGroups = ((int64_t)1 << 24) - 1;  // workgroups of 256 along x
constexpr int64_t kMaxSums = (int64_t)1 << 30;

int check_dtype(int32_t dtype) {
  if (dtype != MAMBA2_DTYPE_F32 && dtype != MAMBA2_DTYPE_BF16)
    return fail(MAMBA2_ERR_DTYPE, "unknown dtype code %d", (int)dtype);
  return MAMBA2_OK;
}

// A token stride: 0 stands for rows without gaps.
int check_stride(int64_t* stride, int64_t least, const char* name) {
  if (*stride == 0) *stride = least;
  if (*stride < least)
    return fail(MAMBA2_ERR_SHAPE, "%s (%lld) is shorter than a row (%lld)", name,
                (long long)*stride, (long long)least);
  if (*stride > kMaxStride)
    return fail(MAMBA2_ERR_UNSUPPORTED, "%s (%lld) is beyond %lld", name, (long long)*stride,
                (long long)kMaxStride);
  return MAMBA2_OK;
}

int check_tokens(int64_t batch, int64_t seqlen, int64_t channels) {
  if (batch < 1 || seqlen < 1 || channels < 1)
    return fail(MAMBA2_ERR_SHAPE, "sizes must be >= 1 (batch=%lld seqlen=%lld channels=%lld)",
                (long long)batch, (long long)seqlen, (long long)channels);
  if (batch > kMaxBatch || seqlen > kMaxTokens || channels > kMaxChannels ||
      batch * seqlen > kMaxTokens)
    return fail(MAMBA2_ERR_UNSUPPORTED, "sizes beyond the supported range");
  return MAMBA2_OK;
}

int validate(const mamba2_conv_dims* p, m2::ConvDims* d) {
  if (!p) return fail(MAMBA2_ERR_NULL, "dims is NULL");
  CHECK(check_dtype(p->dtype));
  CHECK(check_tokens(p->batch, p->seqlen, p->channels));
  if (p->width < 2 || p->width > 4)
    return fail(MAMBA2_ERR_UNSUPPORTED, "width must be 2, 3 or 4 (got %lld)", (long long)p->width);
  if (p->activation != MAMBA2_ACT_NONE && p->activation != MAMBA2_ACT_SILU)
    return fail(MAMBA2_ERR_UNSUPPORTED, "unknown activation code %d", (int)p->activation);
  int64_t sum = 0;
  for (int i = 0; i < 3; ++i) {
    if (p->part[i] < (i == 0 ? 1 : 0) || p->part[i] > p->channels ||
        (i && p->part[i] && !p->part[i - 1]))
      return fail(MAMBA2_ERR_SHAPE, "part[%d] is %lld of %lld channels", i, (long long)p->part[i],
                  (long long)p->channels);
    sum += p->part[i];
  }
  if (sum != p->channels)
    return fail(MAMBA2_ERR_SHAPE, "the parts hold %lld of %lld channels", (long long)sum,
                (long long)p->channels);
  d->B = p->batch;
  d->L = p->seqlen;
  d->C = p->channels;
  d->W = p->width;
  for (int i = 0; i < 3; ++i) d->part[i] = p->part[i];
  d->xs = p->x_stride;
  d->dxs = p->dx_stride;
  CHECK(check_stride(&d->xs, d->C, "x_stride"));
  CHECK(check_stride(&d->dxs, d->C, "dx_stride"));
  d->bf16 = p->dtype == MAMBA2_DTYPE_BF16;
  d->silu = p->activation == MAMBA2_ACT_SILU;
  if (d->B * ((d->L + 7) / 8) > kMaxUnits / d->C)
    return fail(MAMBA2_ERR_UNSUPPORTED, "problem too large for one call");
  return MAMBA2_OK;
}

int need_parts(const m2::ConvDims& d, const void* p0, const void* p1, const void* p2,
               const char* const names[3]) {
  const void* p[3] = {p0, p1, p2};
  for (int i = 0; i < 3; ++i)
    if (d.part[i]) CHECK(need(p[i], names[i]));
  return MAMBA2_OK;
}

int validate(const mamba2_scan_dims* p, m2::ScanDims* d) {
  if (!p) return fail(MAMBA2_ERR_NULL, "dims is NULL");
  CHECK(check_dtype(p->dtype));
  CHECK(check_tokens(p->batch, p->seqlen, p->channels));
  if (p->dstate < 1 || p->ngroups < 1)
    return fail(MAMBA2_ERR_SHAPE, "sizes must be >= 1 (dstate=%lld ngroups=%lld)",
                (long long)p->dstate, (long long)p->ngroups);
  if (p->channels % p->ngroups != 0)
    return fail(MAMBA2_ERR_SHAPE, "channels (%lld) is not a multiple of ngroups (%lld)",
                (long long)p->channels, (long long)p->ngroups);
  if (p->dstate > MAMBA2_SCAN_MAX_STATE)
    return fail(MAMBA2_ERR_UNSUPPORTED, "dstate must be at most %d (got %lld)",
                MAMBA2_SCAN_MAX_STATE, (long long)p->dstate);
  if (p->softplus != 0 && p->softplus != 1)
    return fail(MAMBA2_ERR_SHAPE, "softplus must be 0 or 1 (got %d)", (int)p->softplus);
  d->B = p->batch;
  d->L = p->seqlen;
  d->D = p->channels;
  d->N = p->dstate;
  d->G = p->ngroups;
  d->zs = p->z_stride;
  d->bs = p->b_stride;
  d->cs = p->c_stride;
  d->dzs = p->dz_stride;
  CHECK(check_stride(&d->zs, d->D, "z_stride"));
  CHECK(check_stride(&d->bs, d->G * d->N, "b_stride"));
  CHECK(check_stride(&d->cs, d->G * d->N, "c_stride"));
  CHECK(check_stride(&d->dzs, d->D, "dz_stride"));
  d->bf16 = p->dtype == MAMBA2_DTYPE_BF16;
  d->softplus = p->softplus != 0;
  // the backward's workgroups (at least 16 tokens of 64 channels of a group)
  // and its [B, L, G, states] sums, whose states are padded to a power of two
  const int64_t tiles = d->G * ((d->D / d->G + 63) / 64);
  const int64_t padded = d->N < 2 ? 4 : 2 * d->N;
  if (d->B * d->D > kMaxRows || (d->L + 15) / 16 > kMaxGroups / tiles ||
      d->B * d->L > kMaxSums / (d->G * padded))
    return fail(MAMBA2_ERR_UNSUPPORTED, "problem too large for one call");
  return MAMBA2_OK;
}

int validate(const mamba2_norm_dims* p, m2::NormDims* d) {
  if (!p) return fail(MAMBA2_ERR_NULL, "dims is NULL");
  CHECK(check_dtype(p->dtype));
  if (p->rows < 1 || p->channels < 1 || p->ngroups < 1)
    return fail(MAMBA2_ERR_SHAPE, "sizes must be >= 1 (rows=%lld channels=%lld ngroups=%lld)",
                (long long)p->rows, (long long)p->channels, (long long)p->ngroups);
  if (p->channels % p->ngroups != 0)
    return fail(MAMBA2_ERR_SHAPE, "channels (%lld) is not a multiple of ngroups (%lld)",
                (long long)p->channels, (long long)p->ngroups);
  if (p->rows > kMaxTokens || p->channels > kMaxChannels)
    return fail(MAMBA2_ERR_UNSUPPORTED, "sizes beyond the supported range");
  if (p->channels / p->ngroups > m2::kNormMaxGroup)
    return fail(MAMBA2_ERR_UNSUPPORTED, "a group must have at most %lld channels (got %lld)",
                (long long)m2::kNormMaxGroup, (long long)(p->channels / p->ngroups));
  if (p->kind != MAMBA2_NORM_RMS && p->kind != MAMBA2_NORM_LAYER)
    return fail(MAMBA2_ERR_UNSUPPORTED, "unknown norm code %d", (int)p->kind);
  if (!(p->eps >= 0.f) || isinf(p->eps))
    return fail(MAMBA2_ERR_SHAPE, "eps must be finite and >= 0 (got %g)", (double)p->eps);
  if (p->reserved != 0) return fail(MAMBA2_ERR_SHAPE, "dims.reserved must be 0");
  d->R = p->rows;
  d->D = p->channels;
  d->G = p->ngroups;
  d->xs = p->x_stride;
  d->zs = p->z_stride;
  d->dzs = p->dz_stride;
  CHECK(check_stride(&d->xs, d->D, "x_stride"));
  CHECK(check_stride(&d->zs, d->D, "z_stride"));
  CHECK(check_stride(&d->dzs, d->D, "dz_stride"));
  d->eps = p->eps;
  d->bf16 = p->dtype == MAMBA2_DTYPE_BF16;
  d->layer = p->kind == MAMBA2_NORM_LAYER;
  return MAMBA2_OK;
}

// Never 0 for valid sizes: 0 says that they are not.
size_t at_least_256(size_t n) { return n < 256 ? 256 : round256(n); }

}  // namespace

extern "C" {

int mamba2_conv1d_forward(const mamba2_conv_dims* dims, const void* x, const float* weight,
                          const float* bias, const void* init_state, const int32_t* lengths,
                          void* y0, void* y1, void* y2, void* final_state, void* stream) {
  m2::ConvDims d;
  CHECK(validate(dims, &d));
  CHECK(need(x, "x"));
  CHECK(need(weight, "weight"));
  CHECK(maybe(bias, "bias"));
  CHECK(maybe(init_state, "init_state"));
  CHECK(maybe(lengths, "lengths"));
  static const char* const names[3] = {"y0", "y1", "y2"};
  CHECK(need_parts(d, y0, y1, y2, names));
  CHECK(maybe(final_state, "final_state"));
  void* const y[3] = {y0, y1, y2};
  return hip_status(m2::launch_conv1d(d, x, weight, bias, init_state, lengths, y, final_state,
                                      (hipStream_t)stream),
                    "conv1d launch");
}

size_t mamba2_conv1d_backward_workspace_bytes(const mamba2_conv_dims* dims) {
  m2::ConvDims d;
  if (validate(dims, &d) != MAMBA2_OK) return 0;
  return at_least_256(m2::conv1d_part_bytes(d));
}

int mamba2_conv1d_backward(const mamba2_conv_dims* dims, const void* x, const float* weight,
                           const float* bias, const void* init_state, const int32_t* lengths,
                           const void* dy0, const void* dy1, const void* dy2, const void* dfinal,
                           void* dx, float* dweight, float* dbias, void* dinit, void* workspace,
                           size_t workspace_bytes, void* stream) {
  m2::ConvDims d;
  CHECK(validate(dims, &d));
  CHECK(need(x, "x"));
  CHECK(need(weight, "weight"));
  CHECK(maybe(bias, "bias"));
  CHECK(maybe(init_state, "init_state"));
  CHECK(maybe(lengths, "lengths"));
  static const char* const names[3] = {"dy0", "dy1", "dy2"};
  CHECK(need_parts(d, dy0, dy1, dy2, names));
  CHECK(maybe(dfinal, "dfinal"));
  CHECK(need(dx, "dx"));
  CHECK(need(dweight, "dweight"));
  CHECK(maybe(dbias, "dbias"));
  CHECK(maybe(dinit, "dinit"));
  CHECK(need_workspace(workspace, workspace_bytes, at_least_256(m2::conv1d_part_bytes(d))));
  void* const dy[3] = {(void*)dy0, (void*)dy1, (void*)dy2};
  return hip_status(m2::launch_conv1d_backward(d, x, weight, bias, init_state, lengths, dy, dfinal,
                                               dx, dinit, dweight, dbias, (float*)workspace,
                                               (hipStream_t)stream),
                    "conv1d backward launch");
}

int mamba2_conv1d_step(const mamba2_conv_dims* dims, const void* x, const float* weight,
                       const float* bias, void* state, void* y0, void* y1, void* y2,
                       void* stream) {
  m2::ConvDims d;
  CHECK(validate(dims, &d));
  if (d.L != 1)
    return fail(MAMBA2_ERR_SHAPE, "conv1d_step advances one token: seqlen must be 1 (got %lld)",
                (long long)d.L);
  CHECK(need(x, "x"));
  CHECK(need(weight, "weight"));
  CHECK(maybe(bias, "bias"));
  CHECK(need(state, "state"));
  static const char* const names[3] = {"y0", "y1", "y2"};
  CHECK(need_parts(d, y0, y1, y2, names));
  void* const y[3] = {y0, y1, y2};
  return hip_status(m2::launch_conv1d_step(d, x, weight, bias, state, y, (hipStream_t)stream),
                    "conv1d_step launch");
}

size_t mamba2_selective_scan_workspace_bytes(const mamba2_scan_dims* dims) {
  m2::ScanDims d;
  if (validate(dims, &d) != MAMBA2_OK) return 0;
  return at_least_256(m2::scan_forward_bytes(d));
}

int mamba2_selective_scan_forward(const mamba2_scan_dims* dims, const void* u, const void* dt,
                                  const float* A, const void* B, const void* C, const float* D,
                                  const void* z, const float* dt_bias, const float* init_state,
                                  const int32_t* lengths, void* y, float* final_state,
                                  void* workspace, size_t workspace_bytes, void* stream) {
  m2::ScanDims d;
  CHECK(validate(dims, &d));
  CHECK(need(u, "u"));
  CHECK(need(dt, "dt"));
  CHECK(need(A, "A"));
  CHECK(need(B, "B"));
  CHECK(need(C, "C"));
  CHECK(maybe(D, "D"));
  CHECK(maybe(z, "z"));
  CHECK(maybe(dt_bias, "dt_bias"));
  CHECK(maybe(init_state, "init_state"));
  CHECK(maybe(lengths, "lengths"));
  CHECK(need(y, "y"));
  CHECK(maybe(final_state, "final_state"));
  CHECK(need_workspace(workspace, workspace_bytes, at_least_256(m2::scan_forward_bytes(d))));
  return hip_status(m2::launch_selective_scan(d, u, dt, A, B, C, D, z, dt_bias, init_state,
                                              lengths, y, final_state, workspace,
                                              (hipStream_t)stream),
                    "selective_scan launch");
}

size_t mamba2_selective_scan_backward_workspace_bytes(const mamba2_scan_dims* dims) {
  m2::ScanDims d;
  if (validate(dims, &d) != MAMBA2_OK) return 0;
  return at_least_256(m2::scan_backward_bytes(d));
}

int mamba2_selective_scan_backward(const mamba2_scan_dims* dims, const void* u, const void* dt,
                                   const float* A, const void* B, const void* C, const float* D,
                                   const void* z, const float* dt_bias, const float* init_state,
                                   const int32_t* lengths, const void* dy, const float* dfinal,
                                   void* du, void* ddt, float* dA, void* dB, void* dC, float* dD,
                                   void* dz, float* ddt_bias, float* dinit, void* workspace,
                                   size_t workspace_bytes, void* stream) {
  m2::ScanDims d;
  CHECK(validate(dims, &d));
  CHECK(need(u, "u"));
  CHECK(need(dt, "dt"));
  CHECK(need(A, "A"));
  CHECK(need(B, "B"));
  CHECK(need(C, "C"));
  CHECK(maybe(D, "D"));
  CHECK(maybe(z, "z"));
  CHECK(maybe(dt_bias, "dt_bias"));
  CHECK(maybe(init_state, "init_state"));
  CHECK(maybe(lengths, "lengths"));
  CHECK(need(dy, "dy"));
  CHECK(maybe(dfinal, "dfinal"));
  CHECK(need(du, "du"));
  CHECK(need(ddt, "ddt"));
  CHECK(need(dA, "dA"));
  CHECK(need(dB, "dB"));
  CHECK(need(dC, "dC"));
  CHECK(maybe(dD, "dD"));
  if (z) CHECK(need(dz, "dz"));
  CHECK(maybe(ddt_bias, "ddt_bias"));
  CHECK(maybe(dinit, "dinit"));
  CHECK(need_workspace(workspace, workspace_bytes, at_least_256(m2::scan_backward_bytes(d))));
  return hip_status(
      m2::launch_selective_scan_backward(d, u, dt, A, B, C, D, z, dt_bias, init_state, lengths, dy,
                                         dfinal, du, ddt, dA, dB, dC, dD, z ? dz : nullptr,
                                         ddt_bias, dinit, workspace, (hipStream_t)stream),
      "selective_scan backward launch");
}

int mamba2_selective_scan_step(const mamba2_scan_dims* dims, const void* u, const void* dt,
                               const float* A, const void* B, const void* C, const float* D,
                               const void* z, const float* dt_bias, float* state, void* y,
                               void* stream) {
  m2::ScanDims d;
  CHECK(validate(dims, &d));
  if (d.L != 1)
    return fail(MAMBA2_ERR_SHAPE,
                "selective_scan_step advances one token: seqlen must be 1 (got %lld)",
                (long long)d.L);
  CHECK(need(u, "u"));
  CHECK(need(dt, "dt"));
  CHECK(need(A, "A"));
  CHECK(need(B, "B"));
  CHECK(need(C, "C"));
  CHECK(maybe(D, "D"));
  CHECK(maybe(z, "z"));
  CHECK(maybe(dt_bias, "dt_bias"));
  CHECK(need(state, "state"));
  CHECK(need(y, "y"));
  return hip_status(m2::launch_selective_scan_step(d, u, dt, A, B, C, D, z, dt_bias, state, y,
                                                   (hipStream_t)stream),
                    "selective_scan_step launch");
}

int mamba2_norm_forward(const mamba2_norm_dims* dims, const void* x, const void* z,
                        const float* weight, const float* bias, void* y, void* stream) {
  m2::NormDims d;
  CHECK(validate(dims, &d));
  CHECK(need(x, "x"));
  CHECK(maybe(z, "z"));
  CHECK(need(weight, "weight"));
  CHECK(maybe(bias, "bias"));
  CHECK(need(y, "y"));
  return hip_status(m2::launch_norm(d, x, z, weight, bias, y, (hipStream_t)stream), "norm launch");
}

size_t mamba2_norm_backward_workspace_bytes(const mamba2_norm_dims* dims) {
  m2::NormDims d;
  if (validate(dims, &d) != MAMBA2_OK) return 0;
  return at_least_256(m2::norm_part_bytes(d));
}

int mamba2_norm_backward(const mamba2_norm_dims* dims, const void* x, const void* z,
                         const float* weight, const void* dy, void* dx, void* dz, float* dweight,
                         float* dbias, void* workspace, size_t workspace_bytes, void* stream) {
  m2::NormDims d;
  CHECK(validate(dims, &d));
  CHECK(need(x, "x"));
  CHECK(maybe(z, "z"));
  CHECK(need(weight, "weight"));
  CHECK(need(dy, "dy"));
  CHECK(need(dx, "dx"));
  if (z) CHECK(need(dz, "dz"));
  CHECK(need(dweight, "dweight"));
  CHECK(maybe(dbias, "dbias"));
  CHECK(need_workspace(workspace, workspace_bytes, at_least_256(m2::norm_part_bytes(d))));
  return hip_status(m2::launch_norm_backward(d, x, z, weight, dy, dx, z ? dz : nullptr, dweight,
                                             dbias, (float*)workspace, (hipStream_t)stream),
                    "norm backward launch");
}

}  // extern "C"
