// C ABI of the operators of an attention layer (rotary, attention,
// attention_step): argument checks on the host and stream-ordered launches.
// Declarations and the contract of every entry point are in
// include/mamba2_ssd.h.
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
using m2::round256;

constexpr int64_t kMaxBatch = 65535;
constexpr int64_t kMaxTokens = (int64_t)1 << 28;       // rows of one side
constexpr int64_t kMaxHeads = 1024;
constexpr int64_t kMaxStride = (int64_t)1 << 24;       // elements between tokens
constexpr int64_t kMaxTileStride = (int64_t)1 << 22;   // of attention: a tile within 2^30 bytes
constexpr int64_t kMaxRows = ((int64_t)1 << 31) - 256;  // rows of q times heads of a group, tile included
constexpr int64_t kMaxBlocks = ((int64_t)1 << 23) - 1;  // workgroups of 512 along x

int check_dtype(int32_t dtype) {
  if (dtype != MAMBA2_DTYPE_F32 && dtype != MAMBA2_DTYPE_BF16)
    return fail(MAMBA2_ERR_DTYPE, "unknown dtype code %d", (int)dtype);
  return MAMBA2_OK;
}

int check_flag(int32_t v, const char* name) {
  if (v != 0 && v != 1) return fail(MAMBA2_ERR_SHAPE, "%s must be 0 or 1 (got %d)", name, (int)v);
  return MAMBA2_OK;
}

// A token stride: 0 stands for rows without gaps.  `step` elements are 16 bytes
// where the kernels read rows that way, else 1.
int check_stride(int64_t* stride, int64_t least, int64_t step, const char* name) {
  if (*stride == 0) *stride = least;
  if (*stride < least)
    return fail(MAMBA2_ERR_SHAPE, "%s (%lld) is shorter than a row (%lld)", name,
                (long long)*stride, (long long)least);
  const int64_t most = step > 1 ? kMaxTileStride : kMaxStride;
  if (*stride > most)
    return fail(MAMBA2_ERR_UNSUPPORTED, "%s (%lld) is beyond %lld", name, (long long)*stride,
                (long long)most);
  if (*stride % step)
    return fail(MAMBA2_ERR_UNSUPPORTED, "%s (%lld) is no multiple of %lld elements (16 bytes)",
                name, (long long)*stride, (long long)step);
  return MAMBA2_OK;
}

int check_heads(int64_t heads, int64_t groups, int64_t dim) {
  if (heads < 1 || groups < 1 || dim < 1)
    return fail(MAMBA2_ERR_SHAPE, "sizes must be >= 1 (nheads=%lld ngroups=%lld headdim=%lld)",
                (long long)heads, (long long)groups, (long long)dim);
  if (heads % groups != 0)
    return fail(MAMBA2_ERR_SHAPE, "nheads (%lld) is not a multiple of ngroups (%lld)",
                (long long)heads, (long long)groups);
  if (heads > kMaxHeads)
    return fail(MAMBA2_ERR_UNSUPPORTED, "nheads must be at most %lld (got %lld)",
                (long long)kMaxHeads, (long long)heads);
  if (dim > m2::kAttentionMaxHead || dim % 8)
    return fail(MAMBA2_ERR_UNSUPPORTED,
                "headdim must be a multiple of 8 and at most %lld (got %lld)",
                (long long)m2::kAttentionMaxHead, (long long)dim);
  return MAMBA2_OK;
}

int check_scale(float scale) {
  if (!(scale > 0.f) || isinf(scale))
    return fail(MAMBA2_ERR_SHAPE, "scale must be finite and > 0 (got %g)", (double)scale);
  return MAMBA2_OK;
}

// Attention's exponentials are base 2: the scale with log2(e) is a float32 factor.
int check_attention_scale(float scale) {
  CHECK(check_scale(scale));
  if (isinf(scale * 1.44269504088896340736f))
    return fail(MAMBA2_ERR_UNSUPPORTED, "scale times log2(e) is beyond float32 (scale %g)",
                (double)scale);
  return MAMBA2_OK;
}

int validate(const mamba2_rotary_dims* p, m2::RotaryDims* d) {
  if (!p) return fail(MAMBA2_ERR_NULL, "dims is NULL");
  CHECK(check_dtype(p->dtype));
  if (p->batch < 1 || p->seqlen < 1 || p->nheads < 1 || p->headdim < 1 || p->ngroups < 0)
    return fail(MAMBA2_ERR_SHAPE,
                "sizes must be >= 1 (batch=%lld seqlen=%lld nheads=%lld headdim=%lld) and ngroups "
                ">= 0 (%lld)",
                (long long)p->batch, (long long)p->seqlen, (long long)p->nheads,
                (long long)p->headdim, (long long)p->ngroups);
  if (p->batch > kMaxBatch || p->seqlen > kMaxTokens || p->batch * p->seqlen > kMaxTokens ||
      p->nheads > kMaxHeads || p->ngroups > kMaxHeads)
    return fail(MAMBA2_ERR_UNSUPPORTED, "sizes beyond the supported range");
  if (p->headdim > 1024)
    return fail(MAMBA2_ERR_UNSUPPORTED, "headdim must be at most 1024 (got %lld)",
                (long long)p->headdim);
  if (p->rotary < 2 || p->rotary % 2 || p->rotary > p->headdim)
    return fail(MAMBA2_ERR_SHAPE, "rotary (%lld) must be even and from 2 to headdim (%lld)",
                (long long)p->rotary, (long long)p->headdim);
  if (p->layout != MAMBA2_ROTARY_HALF && p->layout != MAMBA2_ROTARY_INTERLEAVED)
    return fail(MAMBA2_ERR_UNSUPPORTED, "unknown rotary layout code %d", (int)p->layout);
  if (!(p->scale > 0.f) || isinf(p->scale)) return check_scale(p->scale);
  if (p->reserved != 0) return fail(MAMBA2_ERR_SHAPE, "dims.reserved must be 0");
  d->B = p->batch;
  d->L = p->seqlen;
  d->H = p->nheads;
  d->G = p->ngroups;
  d->D = p->headdim;
  d->R = p->rotary;
  d->qs = p->q_stride;
  d->ks = p->k_stride;
  d->yqs = p->yq_stride;
  d->yks = p->yk_stride;
  CHECK(check_stride(&d->qs, d->H * d->D, 1, "q_stride"));
  CHECK(check_stride(&d->ks, d->G * d->D, 1, "k_stride"));
  CHECK(check_stride(&d->yqs, d->H * d->D, 1, "yq_stride"));
  CHECK(check_stride(&d->yks, d->G * d->D, 1, "yk_stride"));
  d->scale = p->scale;
  d->bf16 = p->dtype == MAMBA2_DTYPE_BF16;
  d->half = p->layout == MAMBA2_ROTARY_HALF;
  return MAMBA2_OK;
}

int validate(const mamba2_attention_dims* p, m2::AttentionDims* d) {
  if (!p) return fail(MAMBA2_ERR_NULL, "dims is NULL");
  CHECK(check_dtype(p->dtype));
  if (p->batch < 1 || p->q_len < 1 || p->k_len < 1)
    return fail(MAMBA2_ERR_SHAPE, "sizes must be >= 1 (batch=%lld q_len=%lld k_len=%lld)",
                (long long)p->batch, (long long)p->q_len, (long long)p->k_len);
  CHECK(check_heads(p->nheads, p->ngroups, p->headdim));
  CHECK(check_flag(p->causal, "causal"));
  CHECK(check_flag(p->q_packed, "q_packed"));
  CHECK(check_flag(p->k_packed, "k_packed"));
  CHECK(check_attention_scale(p->scale));
  if (p->reserved != 0) return fail(MAMBA2_ERR_SHAPE, "dims.reserved must be 0");
  if (p->batch > kMaxBatch || p->q_len > kMaxTokens || p->k_len > kMaxTokens)
    return fail(MAMBA2_ERR_UNSUPPORTED, "sizes beyond the supported range");
  d->B = p->batch;
  d->Lq = p->q_len;
  d->Lk = p->k_len;
  d->H = p->nheads;
  d->G = p->ngroups;
  d->D = p->headdim;
  d->qpacked = p->q_packed != 0;
  d->kpacked = p->k_packed != 0;
  d->causal = p->causal != 0;
  d->scale = p->scale;
  d->bf16 = p->dtype == MAMBA2_DTYPE_BF16;
  d->qs = p->q_stride;
  d->ks = p->k_stride;
  d->vs = p->v_stride;
  d->dqs = p->dq_stride;
  d->dks = p->dk_stride;
  d->dvs = p->dv_stride;
  const int64_t step = d->bf16 ? 8 : 4;
  CHECK(check_stride(&d->qs, d->H * d->D, step, "q_stride"));
  CHECK(check_stride(&d->ks, d->G * d->D, step, "k_stride"));
  CHECK(check_stride(&d->vs, d->G * d->D, step, "v_stride"));
  CHECK(check_stride(&d->dqs, d->H * d->D, step, "dq_stride"));
  CHECK(check_stride(&d->dks, d->G * d->D, step, "dk_stride"));
  CHECK(check_stride(&d->dvs, d->G * d->D, step, "dv_stride"));
  if (d->q_rows() > kMaxTokens || d->k_rows() > kMaxTokens ||
      d->q_rows() > kMaxRows / (d->H / d->G) || m2::attention_blocks(*d) > kMaxBlocks ||
      m2::attention_key_blocks(*d) > kMaxBlocks)
    return fail(MAMBA2_ERR_UNSUPPORTED, "problem too large for one call");
  return MAMBA2_OK;
}

int validate(const mamba2_attention_step_dims* p, m2::AttentionStepDims* d) {
  if (!p) return fail(MAMBA2_ERR_NULL, "dims is NULL");
  CHECK(check_dtype(p->dtype));
  if (p->batch < 1 || p->rows < 1 || p->prefix < 0)
    return fail(MAMBA2_ERR_SHAPE, "sizes must be >= 1 (batch=%lld rows=%lld) and prefix >= 0 (%lld)",
                (long long)p->batch, (long long)p->rows, (long long)p->prefix);
  CHECK(check_heads(p->nheads, p->ngroups, p->headdim));
  CHECK(check_attention_scale(p->scale));
  if (p->batch > kMaxBatch || p->rows > kMaxTokens || p->prefix > kMaxTokens)
    return fail(MAMBA2_ERR_UNSUPPORTED, "sizes beyond the supported range");
  d->B = p->batch;
  d->rows = p->rows;
  d->prefix = p->prefix;
  d->H = p->nheads;
  d->G = p->ngroups;
  d->D = p->headdim;
  d->scale = p->scale;
  d->bf16 = p->dtype == MAMBA2_DTYPE_BF16;
  d->qs = p->q_stride;
  d->ks = p->k_stride;
  d->vs = p->v_stride;
  const int64_t step = d->bf16 ? 8 : 4;
  CHECK(check_stride(&d->qs, d->H * d->D, step, "q_stride"));
  CHECK(check_stride(&d->ks, d->G * d->D, step, "k_stride"));
  CHECK(check_stride(&d->vs, d->G * d->D, step, "v_stride"));
  if (m2::attention_step_blocks(*d) > kMaxBlocks ||
      m2::attention_blocks(m2::attention_step_prefix(*d)) > kMaxBlocks)
    return fail(MAMBA2_ERR_UNSUPPORTED, "problem too large for one call");
  return MAMBA2_OK;
}

// Never 0 for valid sizes: 0 says that they are not.
size_t at_least_256(size_t n) { return n < 256 ? 256 : round256(n); }

int rotary(const mamba2_rotary_dims* dims, const void* q, const void* k, const float* inv_freq,
           const int32_t* positions, void* yq, void* yk, bool back, const char* const names[4],
           void* stream) {
  m2::RotaryDims d;
  CHECK(validate(dims, &d));
  CHECK(need(q, names[0]));
  if (d.G) CHECK(need(k, names[1]));
  CHECK(need(inv_freq, "inv_freq"));
  CHECK(maybe(positions, "positions"));
  CHECK(need(yq, names[2]));
  if (d.G) CHECK(need(yk, names[3]));
  return hip_status(
      m2::launch_rotary(d, q, k, inv_freq, positions, yq, yk, back, (hipStream_t)stream),
      "rotary launch");
}

int need_seqs(const m2::AttentionDims& d, const int32_t* q_seqs, const int32_t* k_seqs) {
  CHECK(d.qpacked ? need(q_seqs, "q_seqs") : maybe(q_seqs, "q_seqs"));
  CHECK(d.kpacked ? need(k_seqs, "k_seqs") : maybe(k_seqs, "k_seqs"));
  return MAMBA2_OK;
}

}  // namespace

extern "C" {

int mamba2_rotary_forward(const mamba2_rotary_dims* dims, const void* q, const void* k,
                          const float* inv_freq, const int32_t* positions, void* yq, void* yk,
                          void* stream) {
  static const char* const names[4] = {"q", "k", "yq", "yk"};
  return rotary(dims, q, k, inv_freq, positions, yq, yk, false, names, stream);
}

int mamba2_rotary_backward(const mamba2_rotary_dims* dims, const void* dyq, const void* dyk,
                           const float* inv_freq, const int32_t* positions, void* dq, void* dk,
                           void* stream) {
  static const char* const names[4] = {"dyq", "dyk", "dq", "dk"};
  return rotary(dims, dyq, dyk, inv_freq, positions, dq, dk, true, names, stream);
}

size_t mamba2_attention_workspace_bytes(const mamba2_attention_dims* dims) {
  m2::AttentionDims d;
  if (validate(dims, &d) != MAMBA2_OK) return 0;
  return at_least_256(m2::attention_forward_bytes(d));
}

int mamba2_attention_forward(const mamba2_attention_dims* dims, const void* q, const void* k,
                             const void* v, const int32_t* q_seqs, const int32_t* k_seqs, void* o,
                             float* lse, void* workspace, size_t workspace_bytes, void* stream) {
  m2::AttentionDims d;
  CHECK(validate(dims, &d));
  CHECK(need(q, "q"));
  CHECK(need(k, "k"));
  CHECK(need(v, "v"));
  CHECK(need_seqs(d, q_seqs, k_seqs));
  CHECK(need(o, "o"));
  CHECK(need(lse, "lse"));
  CHECK(need_workspace(workspace, workspace_bytes, at_least_256(m2::attention_forward_bytes(d))));
  return hip_status(
      m2::launch_attention(d, q, k, v, q_seqs, k_seqs, o, lse, workspace, (hipStream_t)stream),
      "attention launch");
}

size_t mamba2_attention_backward_workspace_bytes(const mamba2_attention_dims* dims) {
  m2::AttentionDims d;
  if (validate(dims, &d) != MAMBA2_OK) return 0;
  return at_least_256(m2::attention_backward_bytes(d));
}

int mamba2_attention_backward(const mamba2_attention_dims* dims, const void* q, const void* k,
                              const void* v, const int32_t* q_seqs, const int32_t* k_seqs,
                              const void* o, const float* lse, const void* dout, void* dq,
                              void* dk, void* dv, void* workspace, size_t workspace_bytes,
                              void* stream) {
  m2::AttentionDims d;
  CHECK(validate(dims, &d));
  CHECK(need(q, "q"));
  CHECK(need(k, "k"));
  CHECK(need(v, "v"));
  CHECK(need_seqs(d, q_seqs, k_seqs));
  CHECK(need(o, "o"));
  CHECK(need(lse, "lse"));
  CHECK(need(dout, "dout"));
  CHECK(need(dq, "dq"));
  CHECK(need(dk, "dk"));
  CHECK(need(dv, "dv"));
  CHECK(need_workspace(workspace, workspace_bytes, at_least_256(m2::attention_backward_bytes(d))));
  return hip_status(m2::launch_attention_backward(d, q, k, v, q_seqs, k_seqs, o, lse, dout, dq, dk,
                                                  dv, workspace, (hipStream_t)stream),
                    "attention backward launch");
}

size_t mamba2_attention_step_workspace_bytes(const mamba2_attention_step_dims* dims) {
  m2::AttentionStepDims d;
  if (validate(dims, &d) != MAMBA2_OK) return 0;
  return at_least_256(m2::attention_step_bytes(d));
}

int mamba2_attention_step(const mamba2_attention_step_dims* dims, const void* q, const void* k,
                          const void* v, void* k_cache, void* v_cache, const int32_t* lengths,
                          const void* k_prefix, const void* v_prefix, void* o, void* workspace,
                          size_t workspace_bytes, void* stream) {
  m2::AttentionStepDims d;
  CHECK(validate(dims, &d));
  CHECK(need(q, "q"));
  CHECK(need(k, "k"));
  CHECK(need(v, "v"));
  CHECK(need(k_cache, "k_cache"));
  CHECK(need(v_cache, "v_cache"));
  CHECK(need(lengths, "lengths"));
  if (d.prefix) CHECK(need(k_prefix, "k_prefix"));
  if (d.prefix) CHECK(need(v_prefix, "v_prefix"));
  CHECK(need(o, "o"));
  CHECK(need_workspace(workspace, workspace_bytes, at_least_256(m2::attention_step_bytes(d))));
  return hip_status(m2::launch_attention_step(d, q, k, v, k_cache, v_cache, lengths, k_prefix,
                                              v_prefix, o, workspace, (hipStream_t)stream),
                    "attention_step launch");
}

}  // extern "C"
