// Host-side launchers of the SSD kernels.  Sizes are validated by the C ABI
// layer before any of these is called; each launcher only enqueues.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace m2 {

struct Dims {
  int64_t B, L, H, P, N, G, Q, nc;
  bool bf16;
};

hipError_t launch_chunk_cumsum(const Dims& d, const void* dt, const float* A, float* dA_cs,
                               float* dt_T, hipStream_t s);
hipError_t launch_chunk_state(const Dims& d, const void* x, const void* B, const float* dA_cs,
                              const float* dt_T, float* states, hipStream_t s);
hipError_t launch_state_passing(const Dims& d, float* states, const float* dA_cs,
                                const float* init, float* final_state, hipStream_t s);
hipError_t launch_chunk_scan(const Dims& d, const void* x, const void* B, const void* C,
                             const float* dA_cs, const float* dt_T, const float* states,
                             const float* D, void* y, hipStream_t s);

// Fused-forward variants: state_passing that leaves the chunk-start states as
// bfloat16 in a separate buffer (the float32 per-chunk states are read once),
// and the grouped chunk_scan that consumes them.
hipError_t launch_state_passing_bf16(const Dims& d, const float* states, const float* dA_cs,
                                     const float* init, void* hst, float* final_state,
                                     hipStream_t s);
bool grouped_scan_supported(const Dims& d);
bool grouped_state_supported(const Dims& d);
hipError_t launch_chunk_state_grouped(const Dims& d, const void* x, const void* B,
                                      const float* dA_cs, const float* dt_T, float* states,
                                      hipStream_t s);
// State size 512 runs as two passes over column halves and needs `part`, a
// bfloat16 [B, L, H, P] scratch of grouped_scan_part_bytes(d) (else NULL).
size_t grouped_scan_part_bytes(const Dims& d);
hipError_t launch_chunk_scan_grouped(const Dims& d, const void* x, const void* B, const void* C,
                                     const float* dA_cs, const float* dt_T, const void* hst,
                                     const float* D, void* y, void* part, hipStream_t s);

// Backward pass (bfloat16, P = 64, N in {64, 128, 256}, Q in {64, 128, 256}).
bool backward_supported(const Dims& d);
// E[B,nc,H,P,N] f32: per-chunk adjoint states sum_i 2^cs_i dy_i C_i^T.
hipError_t launch_chunk_state_adjoint(const Dims& d, const void* dy, const void* C,
                                      const float* dA_cs, const float* dt_T, float* states,
                                      hipStream_t s);
// Reverse jump over E: gst[B,nc,H,P,N] bf16 (gradient at each chunk's end),
// dh0 (nullable), dots[B,H,nc,wph] (parts of 2^cs_last <g_c, h_c>).
int64_t state_reverse_waves_per_head(const Dims& d);
hipError_t launch_state_passing_reverse(const Dims& d, const float* E, const float* dA_cs,
                                        const float* dfinal, const void* hst, void* gst,
                                        float* dh0, float* dots, hipStream_t s);
// dB, dC, and th[B,nc,H,N/64,Q]: per state-column tile parts of
// 2^cs_i dy_i . (h_c C_i), the carried-state term of y_i weighted by dy_i.
// wsum: [B,nc,G] blocks of Q(Q+16)/2 bf16 (the group's summed W triangle);
// rsum [B,H,nc,Q] f32: the rectangle sums of the log-decay gradient.
hipError_t launch_chunk_bwd_dbdc(const Dims& d, const void* x, const void* dy, const void* B,
                                 const void* C, const float* dA_cs, const float* dt_T,
                                 const void* hst, const void* gst, void* wsum, float* rsum,
                                 void* dB, void* dC, float* th, hipStream_t s);
hipError_t launch_chunk_bwd_dx(const Dims& d, const void* x, const void* dy, const void* B,
                               const void* C, const float* dA_cs, const float* dt_T,
                               const void* gst, const float* dots, int wph, const float* th,
                               const float* rsum, const float* A, const float* D, void* dx,
                               void* ddt, float* dA_part, float* dD_part, const float* dus,
                               hipStream_t s);
// Above N = 256 (backward_state_term_separate): the state term of dU before
// its row decay, dus[B,L,H,P] f32 = B g^T per (chunk, head), which
// launch_chunk_bwd_dx then reads (dus non-NULL) instead of forming it.
bool backward_state_term_separate(const Dims& d);
hipError_t launch_chunk_bwd_dus(const Dims& d, const void* B, const void* gst, float* dus,
                                hipStream_t s);
hipError_t launch_bwd_param_sums(const Dims& d, const float* dA_part, const float* dD_part,
                                 float* dA, float* dD, hipStream_t s);

// Backward pass for the sizes backward_supported() rejects (chunk_bwd_generic.hip):
// float32 arithmetic on the vector ALU, any size the forward accepts with
// Q <= 256.  hs: the float32 chunk-start states [B,nc,H,P,N] (from
// chunk_state + state_passing); E: [B,nc,H,P,N] float32 scratch (left holding
// the gradient at every chunk end); the scratch below in float32 elements.
struct GenericBwdSizes {
  size_t vg, thp, xup, ghp, cb, part;
};
GenericBwdSizes generic_backward_sizes(const Dims& d);
struct GenericBwdScratch {
  float *vg, *thp, *xup, *ghp, *cb, *dA_part, *dD_part;
};
hipError_t launch_backward_generic(const Dims& d, const void* x, const void* dy, const void* B,
                                   const void* C, const float* dA_cs, const float* dt_T,
                                   float* hs, float* E, const float* dfinal, float* dinit,
                                   const float* A, const float* D, void* dx, void* ddt, void* dB,
                                   void* dC, const GenericBwdScratch& w, hipStream_t s);

// fwd_pass_state as one kernel (bfloat16, P = 64, N in {64, 128, 256},
// Q in {64, 128, 256}): chunk-start states to hst (bf16 [B,nc,H,P,N]) and the
// final state, from the weights w_T = 2^(cs_last - cs_j) dt_j [B,H,nc,Q].
// fwd_pass_state over spans of chunks (state_span.hip): span_chunks gives the
// span length K (0 = this path does not apply to these sizes).  span_states
// [B, ng, H, P, N] float32 and span_decay [B, H, ng] are scratch
// (ng = ceil(nc / K)); hst receives the bfloat16 chunk-start states.  `mid`
// (may be null) is recorded after the span-end kernel.
int span_chunks(const Dims& d);
size_t span_states_bytes(const Dims& d, int K);
// replay = false stops after the jump across spans (span_states then hold
// every span's start state, for span_scan).
hipError_t launch_fwd_pass_state_span(const Dims& d, int K, const void* x, const void* B,
                                      const float* dA_cs, const float* dt_T, const float* init,
                                      float* span_states, float* span_decay, void* hst,
                                      float* final_state, hipStream_t s, hipEvent_t mid,
                                      bool replay);

// span_scan (span_scan.hip): the replay of each span fused with compute_out,
// from the span start states the jump leaves in span_states; y only.
// span_scan_heads gives the heads per workgroup (0 = not covered: the replay
// and the grouped chunk_scan run instead).
int span_scan_heads(const Dims& d, int K);
// The forward's span length where span_scan runs (0 = span_chunks decides).
int span_scan_chunks(const Dims& d);
hipError_t launch_span_scan(const Dims& d, int K, int R, const void* x, const void* B,
                            const void* C, const float* dA_cs, const float* dt_T,
                            const float* span_states, const float* D, void* y, hipStream_t s);

bool fused_state_supported(const Dims& d);
hipError_t launch_chunk_weights(const Dims& d, const float* dA_cs, const float* dt_T, float* w_T,
                                hipStream_t s);
hipError_t launch_fwd_pass_state(const Dims& d, const void* x, const void* B, const float* dA_cs,
                                 const float* w_T, const float* init, void* hst,
                                 float* final_state, hipStream_t s);

// One-token recurrent step, in place on the float32 state [B,H,P,N];
// x, y [B,H,P], dt [B,H], B, C [B,G,N].
hipError_t launch_decode_step(const Dims& d, const void* x, const void* dt, const float* A,
                              const void* B, const void* C, const float* D, float* state,
                              void* y, hipStream_t s);

// The operators around the SSD (conv1d.hip, selective_scan.hip, norm.hip).
// Token strides are in elements; batches follow each other at L token strides.
struct ConvDims {
  int64_t B, L, C, W, part[3], xs, dxs;
  bool bf16, silu;
};
hipError_t launch_conv1d(const ConvDims& d, const void* x, const float* w, const float* bias,
                         const void* init, const int32_t* lengths, void* const* y,
                         void* final_state, hipStream_t s);
size_t conv1d_part_bytes(const ConvDims& d);
hipError_t launch_conv1d_backward(const ConvDims& d, const void* x, const float* w,
                                  const float* bias, const void* init, const int32_t* lengths,
                                  void* const* dy, const void* dfinal, void* dx, void* dinit,
                                  float* dw, float* dbias, float* part, hipStream_t s);
hipError_t launch_conv1d_step(const ConvDims& d, const void* x, const float* w, const float* bias,
                              void* state, void* const* y, hipStream_t s);

struct NormDims {
  int64_t R, D, G, xs, zs, dzs;
  float eps;
  bool bf16, layer;
};
// Longest group of channels one workgroup holds in registers.
constexpr int64_t kNormMaxGroup = 8192;
hipError_t launch_norm(const NormDims& d, const void* x, const void* z, const float* w,
                       const float* bias, void* y, hipStream_t s);
size_t norm_part_bytes(const NormDims& d);
hipError_t launch_norm_backward(const NormDims& d, const void* x, const void* z, const float* w,
                                const void* dy, void* dx, void* dz, float* dw, float* dbias,
                                float* part, hipStream_t s);

struct ScanDims {
  int64_t B, L, D, N, G, zs, bs, cs, dzs;
  bool bf16, softplus;
};
// Chunks of the sequence that run in parallel and the tokens of each.
struct ScanSplit {
  int64_t chunks, len;
};
size_t scan_forward_bytes(const ScanDims& d);
hipError_t launch_selective_scan(const ScanDims& d, const void* u, const void* dt, const float* A,
                                 const void* B, const void* C, const float* D, const void* z,
                                 const float* dt_bias, const float* init, const int32_t* lengths,
                                 void* y, float* final_state, void* ws, hipStream_t s);
size_t scan_backward_bytes(const ScanDims& d);
hipError_t launch_selective_scan_backward(
    const ScanDims& d, const void* u, const void* dt, const float* A, const void* B, const void* C,
    const float* D, const void* z, const float* dt_bias, const float* init, const int32_t* lengths,
    const void* dy, const float* dfinal, void* du, void* ddt, float* dA, void* dB, void* dC,
    float* dD, void* dz, float* ddt_bias, float* dinit, void* ws, hipStream_t s);
hipError_t launch_selective_scan_step(const ScanDims& d, const void* u, const void* dt,
                                      const float* A, const void* B, const void* C, const float* D,
                                      const void* z, const float* dt_bias, float* state, void* y,
                                      hipStream_t s);

// The operators of an attention layer (rotary.hip, attention*.hip).  Strides as above.
struct RotaryDims {
  int64_t B, L, H, G, D, R, qs, ks, yqs, yks;
  float scale;
  bool bf16, half;
};
hipError_t launch_rotary(const RotaryDims& d, const void* q, const void* k, const float* inv_freq,
                         const int32_t* positions, void* yq, void* yk, bool back, hipStream_t s);

struct AttentionDims {
  int64_t B, Lq, Lk, H, G, D, qs, ks, vs, dqs, dks, dvs;
  float scale;
  bool causal, qpacked, kpacked, bf16;
  int64_t q_rows() const { return qpacked ? Lq : B * Lq; }
  int64_t k_rows() const { return kpacked ? Lk : B * Lk; }
};
// Largest head; workgroups along x of the largest launch.
constexpr int64_t kAttentionMaxHead = 128;
int64_t attention_blocks(const AttentionDims& d);
int64_t attention_key_blocks(const AttentionDims& d);
size_t attention_forward_bytes(const AttentionDims& d);
hipError_t launch_attention(const AttentionDims& d, const void* q, const void* k, const void* v,
                            const int32_t* q_seqs, const int32_t* k_seqs, void* o, float* lse,
                            void* ws, hipStream_t s);
// The forward in attention_parts(d) ranges of the keys: normalised float32
// outputs [parts][rows of q][H][D] and their log2 sums [parts][rows of q][H];
// and their join (lse may be NULL).
int attention_parts(const AttentionDims& d);
hipError_t launch_attention_parts(const AttentionDims& d, const void* q, const void* k,
                                  const void* v, float* part_o, float* part_lse, hipStream_t s);
hipError_t launch_attention_join(const float* part_o, const float* part_lse, void* o, float* lse,
                                 int64_t rows, int64_t D, int parts, bool bf16, hipStream_t s);
size_t attention_backward_bytes(const AttentionDims& d);
hipError_t launch_attention_backward(const AttentionDims& d, const void* q, const void* k,
                                     const void* v, const int32_t* q_seqs, const int32_t* k_seqs,
                                     const void* o, const float* lse, const void* dout, void* dq,
                                     void* dk, void* dv, void* ws, hipStream_t s);

struct AttentionStepDims {
  int64_t B, rows, prefix, H, G, D, qs, ks, vs;
  float scale;
  bool bf16;
};
int64_t attention_step_blocks(const AttentionStepDims& d);
// The prefix as a prompt's keys: the batch's tokens are its rows.
AttentionDims attention_step_prefix(const AttentionStepDims& d);
size_t attention_step_bytes(const AttentionStepDims& d);
hipError_t launch_attention_step(const AttentionStepDims& d, const void* q, const void* k,
                                 const void* v, void* k_cache, void* v_cache,
                                 const int32_t* lengths, const void* k_prefix,
                                 const void* v_prefix, void* o, void* ws, hipStream_t s);

// out[m] = sum over rows p of part[p][m], columns [0, ends[0]), [ends[0],
// ends[1]) and [ends[1], ends[2]) going to outs[0..2] (NULL: not written).
hipError_t launch_partial_sums(const float* part, int64_t P, int64_t M, const int64_t ends[3],
                               float* const outs[3], hipStream_t s);

}  // namespace m2
