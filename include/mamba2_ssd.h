/*
 * mamba2_ssd.h - C ABI of the MI355X (gfx950) chunked Mamba-2 SSD forward pass.
 *
 * The method (pages: devotd.net news item on the Mamba-2 CUDA Tile
 * forward-pass kernels, sections 1-2; disconfirmai.com "Jane Street ML
 * Engineers Map Mamba-2 Recurrent State Computation to Tensor Cores with
 * cuTile", abstract and body) evaluates the recurrence
 *
 *     h_t = exp(dt_t * A) * h_{t-1} + dt_t * x_t (outer) B_t      state [P, N]
 *     y_t = h_t . C_t + D * x_t
 *
 * chunk by chunk: an in-chunk log-space cumulative sum of dt*A
 * (chunk_cumsum), per-chunk B X^T contractions and the decayed jump that
 * carries the state across chunks in order (fwd_pass_state, exposed here as
 * chunk_state + state_passing), and the fused output stage (compute_out,
 * exposed as chunk_scan): carried-state term C.h, the causally masked,
 * decay-weighted C B^T interaction times X, and the D skip.
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 * Sizes: B = batch, L = seqlen, H = nheads, P = headdim, N = dstate,
 *        G = ngroups (H % G == 0; head h reads B/C group h / (H/G)),
 *        Q = chunk_size, nc = ceil(L / Q).
 * Layouts (contiguous, row-major, innermost last):
 *        x, y          [B, L, H, P]
 *        dt            [B, L, H]
 *        A, D          [H]                 float32
 *        B, C          [B, L, G, N]
 *        init/final    [B, H, P, N]        float32
 *        dA_cs, dt_T   [B, H, nc, Q]       float32 (time contiguous)
 *        states        [B, nc, H, P, N]    float32
 * dtype: MAMBA2_DTYPE_F32  - every tensor is float32;
 *        MAMBA2_DTYPE_BF16 - x, dt, B, C and y are bfloat16; A, D, the
 *                            cumsum outputs, states and the initial/final
 *                            state are float32.
 * Positions past L inside the last chunk are treated as zero input (dt = 0,
 * x = 0), following the zero-padded tile loads of the pages' chunk_cumsum
 * figure; y is written only for t < L.
 * Memory: every pointer is device memory owned by the caller.  The library
 * never allocates or frees and keeps no pointer after a call returns.  Every
 * pointer must be 16-byte aligned (MAMBA2_ERR_ALIGN otherwise).
 * Streams: `stream` is a hipStream_t (NULL = default stream).  Every call
 * only enqueues work on that stream; there is no device synchronisation
 * inside.  Stages given the same stream run in call order.
 * Errors: every int-returning call returns a mamba2_status.  Arguments are
 * checked on the host before anything is enqueued; on a failed check nothing
 * is launched and no output is touched.  MAMBA2_ERR_HIP reports a launch
 * failure, with the HIP error text in mamba2_last_error().  No C++ exception
 * crosses this interface.  Calls are thread-safe: the library keeps no
 * mutable global state except the calling thread's last-error message.
 * Preconditions that are not checked (checking would cost a pass over the
 * data): A <= 0, dt >= 0 and every input finite - the decay regime the
 * method describes (decay rate times time interval).
 * Supported sizes: Q in {16, 32, 64, 128, 256} for float32 and
 * {64, 128, 256} for bfloat16; bfloat16 also needs P and N multiples of 16
 * with P <= 128 and N <= 512 (the MFMA tile is 16 wide; larger states do not
 * fit one workgroup's registers and LDS).  The fastest kernels (shared B/C
 * operands across the heads of a group, spans of chunks) cover bfloat16
 * with P = 64 and N in {64, 128, 256, 512}; other supported sizes run
 * per-head kernels.  Other sizes give MAMBA2_ERR_UNSUPPORTED.
 */
#ifndef MAMBA2_SSD_H_
#define MAMBA2_SSD_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  MAMBA2_OK = 0,
  MAMBA2_ERR_NULL = 1,        /* a required pointer is NULL */
  MAMBA2_ERR_SHAPE = 2,       /* non-positive size, H % G != 0, overflow */
  MAMBA2_ERR_DTYPE = 3,       /* unknown dtype code */
  MAMBA2_ERR_UNSUPPORTED = 4, /* valid but not implemented size */
  MAMBA2_ERR_ALIGN = 5,       /* a pointer is not 16-byte aligned */
  MAMBA2_ERR_WORKSPACE = 6,   /* workspace missing or too small */
  MAMBA2_ERR_HIP = 7          /* a HIP launch failed */
} mamba2_status;

typedef enum { MAMBA2_DTYPE_F32 = 0, MAMBA2_DTYPE_BF16 = 1 } mamba2_dtype;

typedef struct {
  int64_t batch;      /* B  >= 1 */
  int64_t seqlen;     /* L  >= 1 */
  int64_t nheads;     /* H  >= 1 */
  int64_t headdim;    /* P  >= 1 */
  int64_t dstate;     /* N  >= 1 */
  int64_t ngroups;    /* G  >= 1, divides H */
  int64_t chunk_size; /* Q */
  int32_t dtype;      /* mamba2_dtype */
  int32_t reserved;   /* must be 0 */
} mamba2_dims;

/* Checks `dims` alone (host only, touches no device).  Returns MAMBA2_OK when
 * every entry point supports these sizes. */
int mamba2_validate(const mamba2_dims* dims);

/*
 * chunk_cumsum (devotd.net page, section 2 and its code figure): for every
 * batch b, head h and chunk c, the inclusive cumulative sum of A[h]*dt along
 * the chunk's time steps, multiplied by log2(e) so consumers use base-2
 * exponentials:
 *     dA_cs[b,h,c,i] = log2(e) * sum_{j<=i} A[h] * dt[b, c*Q+j, h]
 *     dt_T[b,h,c,i]  = dt[b, c*Q+i, h]        (0 past L)
 * Inputs dt (dtype of dims), A (float32).  Outputs float32 [B,H,nc,Q],
 * fully overwritten.  The sum is evaluated as a tree (wavefront scan).
 */
int mamba2_chunk_cumsum(const mamba2_dims* dims, const void* dt, const float* A,
                        float* dA_cs, float* dt_T, void* stream);

/*
 * chunk_state (first half of fwd_pass_state; disconfirmai.com page, body:
 * the jump formula's B X^T product with rows pre-scaled by exponentials): the
 * state each chunk reaches from a zero start,
 *     states[b,c,h,p,n] = sum_{j in chunk} 2^(cs[Q-1] - cs[j]) * dt_j
 *                                          * x[b,cQ+j,h,p] * B[b,cQ+j,g,n]
 * with cs = dA_cs[b,h,c,:], dt_j = dt_T[b,h,c,j].  Inputs x, B (dtype of
 * dims), dA_cs and dt_T from mamba2_chunk_cumsum.  Output states float32
 * [B,nc,H,P,N], fully overwritten.
 */
int mamba2_chunk_state(const mamba2_dims* dims, const void* x, const void* B,
                       const float* dA_cs, const float* dt_T, float* states,
                       void* stream);

/*
 * state_passing (second half of fwd_pass_state; devotd.net page, section 2:
 * the state at each chunk start and after the last chunk, chunks in order,
 * independent parts of the state in parallel).  In place over `states`:
 *     run = init_state (zeros if NULL)
 *     for c in 0..nc-1:  S = states[b,c,h];  states[b,c,h] = run;
 *                        run = 2^(dA_cs[b,h,c,Q-1]) * run + S
 *     final_state = run                   (not written if NULL)
 * On entry states holds chunk_state's per-chunk states; on return it holds
 * the state at the start of every chunk.  All float32.
 */
int mamba2_state_passing(const mamba2_dims* dims, float* states, const float* dA_cs,
                         const float* init_state, float* final_state, void* stream);

/*
 * chunk_scan = compute_out (devotd.net page, section 2; disconfirmai.com
 * page, abstract): outputs of every chunk from its start state, fused so the
 * Q x Q interaction matrix never reaches memory.  For token i of chunk c,
 * head h, group g:
 *     y[i,p] = 2^cs[i] * sum_n C[i,n] h[p,n]
 *            + sum_{j<=i} (sum_n C[i,n] B[j,n]) 2^(cs[i]-cs[j]) dt_j x[j,p]
 *            + D[h] x[i,p]
 * with h = states[b,c,h] (chunk-start states from mamba2_state_passing),
 * cs = dA_cs[b,h,c,:], dt = dt_T[b,h,c,:].  D may be NULL (no skip term).
 * Output y (dtype of dims) [B,L,H,P]; rows t >= L are not written.
 */
int mamba2_chunk_scan(const mamba2_dims* dims, const void* x, const void* B,
                      const void* C, const float* dA_cs, const float* dt_T,
                      const float* states, const float* D, void* y, void* stream);

/* Bytes of device workspace mamba2_ssd_forward needs for `dims` (0 if the
 * dims are invalid).  Host only. */
size_t mamba2_ssd_workspace_bytes(const mamba2_dims* dims);

/*
 * The whole forward pass: chunk_cumsum -> fwd_pass_state -> chunk_scan on
 * `stream`, intermediates in the caller's workspace (at least
 * mamba2_ssd_workspace_bytes(dims) bytes, 256-byte aligned; contents on
 * return are unspecified).  init_state and D may be NULL; final_state may
 * be NULL (not written).  Outputs y [B,L,H,P] (dtype of dims) and
 * final_state [B,H,P,N] float32.  fwd_pass_state runs as chunk_state ->
 * state_passing, or, for bfloat16 with headdim 64, dstate 64/128/256/512
 * and enough (batch, head, span) work to fill the device, over spans of 8
 * (or 4) chunks (devotd.net news item, section 2: the same jump across
 * chunks, taken span by span): the state after each span from a zero start,
 * the jump across spans, then each span replayed from its start state.  At
 * dstate 256 and 512 the replay writes bfloat16 chunk-start states for
 * chunk_scan; at dstate 64 and 128, with an even number of heads per group,
 * one kernel replays each span and forms its outputs in the same pass, so
 * the chunk-start states stay on chip.  At dstate 512 the output stage runs
 * over two halves of the state columns and the first hands its partial y to
 * the second in bfloat16 (one more rounding of that partial).  All forms
 * give the same result up to rounding.
 */
int mamba2_ssd_forward(const mamba2_dims* dims, const void* x, const void* dt,
                       const float* A, const void* B, const void* C, const float* D,
                       const float* init_state, void* y, float* final_state,
                       void* workspace, size_t workspace_bytes, void* stream);

/*
 * mamba2_ssd_forward for callers that cannot allocate device memory (code
 * under HIP graph capture, tight serving loops, harnesses that forbid
 * hipMalloc): the same kernels, with the workspace taken from a static
 * device array of MAMBA2_NOALLOC_SCRATCH_BYTES that the library holds on
 * each GPU it runs on until the process ends.  The caller passes inputs and
 * outputs only; the call allocates and frees nothing.  Sizes whose
 * mamba2_ssd_workspace_bytes exceed the array are rejected with
 * MAMBA2_ERR_WORKSPACE before any launch.  The array's address on the
 * current device is looked up once per device (hipGetSymbolAddress) and
 * kept; the current device must be the one the pointers and the stream
 * belong to.  Every call on one GPU shares that GPU's array and it keeps the
 * last call's contents (no part needs clearing: each piece is written
 * before it is read within a call), so calls that overlap on one GPU - on
 * different streams, or from different threads - race and give wrong
 * results: order them on one stream or otherwise.  Other rules as for
 * mamba2_ssd_forward.
 */
#define MAMBA2_NOALLOC_SCRATCH_BYTES ((size_t)128 << 20)

int mamba2_ssd_forward_noalloc(const mamba2_dims* dims, const void* x, const void* dt,
                               const float* A, const void* B, const void* C, const float* D,
                               const float* init_state, void* y, float* final_state,
                               void* stream);

/*
 * Same as mamba2_ssd_forward, then waits for the work to finish and writes
 * the device time of each stage in milliseconds to stage_ms[0..3]
 * (chunk_cumsum, chunk_state, state_passing, chunk_scan; on the span path
 * the second and third are the span-end kernel and the jump across spans
 * plus the replay), measured with HIP events recorded on `stream` between
 * the launches.  For measurement only:
 * it creates and destroys five events and blocks the calling thread.
 */
int mamba2_ssd_forward_profile(const mamba2_dims* dims, const void* x, const void* dt,
                               const float* A, const void* B, const void* C, const float* D,
                               const float* init_state, void* y, float* final_state,
                               void* workspace, size_t workspace_bytes, void* stream,
                               float* stage_ms);

/*
 * fwd_pass_state as one kernel, the pages' own second kernel (devotd.net news
 * item, section 2: the state at every chunk start and after the last chunk,
 * chunk order kept while independent parts of the state run in parallel;
 * disconfirmai.com, body: the jump formula with exponentially pre-scaled rows
 * of X): per state tile, walks the chunks in order with the running state in
 * float32 MFMA accumulators, so the per-chunk states never reach memory.
 * Inputs: x, B, dA_cs, dt_T (from mamba2_chunk_cumsum), init_state (NULL =
 * zeros).  Outputs: w_T [B,H,nc,Q] float32, the contraction weights
 * 2^(cs[Q-1] - cs[j]) * dt_j (written first, then read by the kernel);
 * chunk_start_states [B,nc,H,P,N] bfloat16 (round to nearest even);
 * final_state [B,H,P,N] float32.  Supported: bfloat16 with headdim 64,
 * dstate 64, 128 or 256 and chunk_size 64, 128 or 256 (UNSUPPORTED
 * otherwise).  The default forward (chunk_state + state_passing) is faster on
 * this chip; this path is the one-kernel form for callers that want it.
 */
int mamba2_fwd_pass_state(const mamba2_dims* dims, const void* x, const void* B,
                          const float* dA_cs, const float* dt_T, const float* init_state,
                          float* w_T, void* chunk_start_states, float* final_state,
                          void* stream);

/*
 * The whole forward through the one-kernel fwd_pass_state: chunk_cumsum ->
 * weights -> fwd_pass_state -> chunk_scan.  Same arguments, results (up to
 * rounding order) and workspace as mamba2_ssd_forward (at least
 * mamba2_ssd_workspace_bytes(dims)); final_state is required.  Sizes as for
 * mamba2_fwd_pass_state.
 */
int mamba2_ssd_forward_fused(const mamba2_dims* dims, const void* x, const void* dt,
                             const float* A, const void* B, const void* C, const float* D,
                             const float* init_state, void* y, float* final_state,
                             void* workspace, size_t workspace_bytes, void* stream);

/*
 * Recurrent single-token step: the constant-memory inference mode of the same
 * recurrence (pages: devotd.net news item, section 1 - a fixed-size hidden
 * state updated as tokens are processed; disconfirmai.com, abstract - the
 * recurrent state).  For one new token of every (batch, head), in place:
 *     state[b,h] = exp(dt[b,h] * A[h]) * state[b,h] + dt[b,h] * x[b,h] (outer) B[b,g]
 *     y[b,h]     = state[b,h] . C[b,g] + D[h] * x[b,h]          (g = h / (H/G))
 * i.e. one token of the forward pass, reading the state after the update.
 * dims: seqlen must be 1 (MAMBA2_ERR_SHAPE otherwise); chunk_size is not
 *       used but must be a supported value, as for every dims.
 * Layouts: x, y [B, H, P] (the forward's [B, L, H, P] with L = 1);
 *          dt [B, H]; B, C [B, G, N]; A, D [H] float32 (D may be NULL);
 *          state [B, H, P, N] float32, read and overwritten.
 * dtype as for the forward: bfloat16 makes x, dt, B, C and y bfloat16.
 * Every pointer 16-byte aligned, as everywhere (a per-token view sliced out
 * of a [B, L, ...] tensor usually is not: copy it).
 * Bound by HBM on the state (read once, written once).
 */
int mamba2_decode_step(const mamba2_dims* dims, const void* x, const void* dt, const float* A,
                       const void* B, const void* C, const float* D, float* state, void* y,
                       void* stream);

/*
 * Backward pass: gradients of a scalar loss through mamba2_ssd_forward.  The
 * pages publish no backward pass (disconfirmai.com, lead paragraph: the
 * forward speedups rest on one that is not yet published); this is the exact
 * derivative of the forward's chunked form (devotd.net news item, section 2),
 * for the loss whose gradients with respect to y and final_state are dy and
 * dfinal:
 *     dx, ddt, dB, dC   same layouts and dtype as x, dt, B, C
 *     dA [H], dD [H]    float32 (dD written only when D is non-NULL; it is
 *                       required then)
 *     dinit [B,H,P,N]   float32, may be NULL (not written); it is the
 *                       gradient with respect to init_state (whether or not
 *                       init_state is NULL, which means a zero start)
 * Inputs are the forward's (x, dt, A, B, C, D, init_state; D and init_state
 * may be NULL), dy [B,L,H,P] (dtype of dims) and dfinal [B,H,P,N] float32
 * (NULL = zero).  The forward quantities the gradients need are recomputed
 * inside (nothing from an earlier forward call is read).
 * Supported: every size the forward accepts.  bfloat16 with headdim 64 and
 * dstate 64, 128 or 256 with chunk_size 64, 128 or 256, or dstate 512 with
 * chunk_size 256, runs MFMA kernels; every other size (float32, other head
 * sizes, dstate 512 with shorter chunks and the other multiples of 16) runs
 * a generic path of float32 vector-ALU kernels without MFMA: exact to
 * float32 rounding, and much slower.  Workspace: at least
 * mamba2_ssd_backward_workspace_bytes(dims), 256-byte aligned, contents on
 * return unspecified.  Pointer, stream and error rules as for the forward.
 */
size_t mamba2_ssd_backward_workspace_bytes(const mamba2_dims* dims);

int mamba2_ssd_backward(const mamba2_dims* dims, const void* x, const void* dt, const float* A,
                        const void* B, const void* C, const float* D, const float* init_state,
                        const void* dy, const float* dfinal, void* dx, void* ddt, float* dA,
                        void* dB, void* dC, float* dD, float* dinit, void* workspace,
                        size_t workspace_bytes, void* stream);

/*
 * Same as mamba2_ssd_backward, then waits and writes the device time of each
 * of its eight stages in milliseconds to stage_ms[0..7]: chunk_cumsum,
 * chunk_state, state_passing (the recomputed forward states), adjoint
 * chunk_state, reverse state_passing, dB/dC kernel, dx kernel (at dstate 512
 * with the kernel forming dx's state term before it), dA/dD sums.
 * On the generic path stage 0 holds the whole pass and the others read 0.
 * For measurement only (creates events, blocks).
 */
int mamba2_ssd_backward_profile(const mamba2_dims* dims, const void* x, const void* dt,
                                const float* A, const void* B, const void* C, const float* D,
                                const float* init_state, const void* dy, const float* dfinal,
                                void* dx, void* ddt, float* dA, void* dB, void* dC, float* dD,
                                float* dinit, void* workspace, size_t workspace_bytes,
                                void* stream, float* stage_ms);

/*
 * The operators around the SSD
 * ----------------------------
 * What a layer built on the SSD computes next to it: the short causal
 * convolution that makes x, B and C (conv1d), the same recurrence with a
 * decay for each (channel, state) (selective_scan), and the norm of its
 * input or gated output (norm).  The conventions above hold, with these
 * additions:
 * Strides: where dims has a <name>_stride, token t of batch b of that tensor
 *        starts at element (b * L + t) * <name>_stride of it (row r of a norm
 *        at r * <name>_stride): a tensor may be a column range of a wider
 *        one.  0 means rows without gaps; a stride is at least a row (a row
 *        that stands for several tokens is refused) and at most 2^24.  The
 *        base pointer is 16-byte aligned; rows need not be (rows and sizes
 *        that are multiples of 16 bytes run faster).  Everything else is
 *        contiguous.
 * Sizes: batch <= 65535; batch * L, and the rows of a norm, <= 2^30; channels
 *        <= 2^20; each operator's further bounds stand at it.  Beyond them
 *        a call returns MAMBA2_ERR_UNSUPPORTED.
 * lengths: int32 [B] or NULL (every sequence has L tokens): sequence b has
 *        lengths[b] tokens, values outside 0 .. L are taken as the nearer
 *        bound.  What stands in the inputs behind them is not read; outputs
 *        and gradients there are written as zeros, also where the sequence's
 *        own are not finite, and sums over tokens take nothing from there.
 *        A final state is the state after the sequence's own last token (the
 *        initial state where it has none).
 * Outputs do not overlap inputs, but final_state may be init_state.
 * Gradients that are sums over tokens are formed from per-workgroup float32
 * parts in a fixed order: the same call gives the same bits.
 */
typedef enum { MAMBA2_ACT_NONE = 0, MAMBA2_ACT_SILU = 1 } mamba2_activation;
typedef enum { MAMBA2_NORM_RMS = 0, MAMBA2_NORM_LAYER = 1 } mamba2_norm_kind;

typedef struct {
  int64_t batch;      /* B >= 1 */
  int64_t seqlen;     /* L >= 1 */
  int64_t channels;   /* C >= 1 */
  int64_t width;      /* W: 2, 3 or 4 taps */
  int64_t part[3];    /* channels of the outputs y0, y1, y2; they add up to C, unused ones are 0 */
  int64_t x_stride;   /* elements between tokens of x; 0: C */
  int64_t dx_stride;  /* the same of dx (backward) */
  int32_t dtype;      /* mamba2_dtype */
  int32_t activation; /* mamba2_activation */
} mamba2_conv_dims;

/*
 * conv1d: a causal depthwise convolution over the tokens, per channel c
 *     p[t]  = bias + sum_k weight[c, k] * x[t - (W-1) + k],  k = 0 .. W-1
 *     y[t]  = p[t] * sigmoid(p[t])   (MAMBA2_ACT_SILU)   or   p[t]
 * where x[-j] is row W-1-j of init_state (zeros if NULL).
 *     x             [B, L, C]       rows of x_stride
 *     y0, y1, y2    [B, L, part[i]] contiguous: channels in order, so one
 *                   call makes the x, B and C that mamba2_ssd_forward takes
 *     weight        [C, W] float32; bias [C] float32 or NULL
 *     init_state    [B, W-1, C] or NULL; final_state the same or NULL (not
 *                   written): the last W-1 rows of [init_state; x]
 * x, y and the states have the type of dims.  Sums are float32.  Supported:
 * C * B * ceil(L / 8) <= 2^31.
 */
int mamba2_conv1d_forward(const mamba2_conv_dims* dims, const void* x, const float* weight,
                          const float* bias, const void* init_state, const int32_t* lengths,
                          void* y0, void* y1, void* y2, void* final_state, void* stream);

/*
 * Gradients of conv1d for the loss whose gradients with respect to y0, y1,
 * y2 and final_state are dy0, dy1, dy2 and dfinal (NULL = zero):
 *     dx [B, L, C] rows of dx_stride, dinit [B, W-1, C] (may be NULL: not
 *     written), type of dims; dweight [C, W] and dbias [C] float32 (dbias
 *     may be NULL).
 * The convolution is recomputed; workspace at least
 * mamba2_conv1d_backward_workspace_bytes(dims) (0: dims invalid), 256-byte
 * aligned.
 */
size_t mamba2_conv1d_backward_workspace_bytes(const mamba2_conv_dims* dims);

int mamba2_conv1d_backward(const mamba2_conv_dims* dims, const void* x, const float* weight,
                           const float* bias, const void* init_state, const int32_t* lengths,
                           const void* dy0, const void* dy1, const void* dy2, const void* dfinal,
                           void* dx, float* dweight, float* dbias, void* dinit, void* workspace,
                           size_t workspace_bytes, void* stream);

/*
 * One token of conv1d for every sequence: seqlen must be 1, x [B, C] with
 * rows of x_stride, y0, y1, y2 [B, part[i]]; state [B, W-1, C] (the last
 * rows of x) is read and moved on by one row in place.
 */
int mamba2_conv1d_step(const mamba2_conv_dims* dims, const void* x, const float* weight,
                       const float* bias, void* state, void* y0, void* y1, void* y2,
                       void* stream);

#define MAMBA2_SCAN_MAX_STATE 64

typedef struct {
  int64_t batch;      /* B >= 1 */
  int64_t seqlen;     /* L >= 1 */
  int64_t channels;   /* D >= 1 */
  int64_t dstate;     /* N: 1 .. MAMBA2_SCAN_MAX_STATE */
  int64_t ngroups;    /* G, divides D: channel c reads B/C group c / (D/G) */
  int64_t z_stride;   /* elements between tokens of z; 0: D */
  int64_t b_stride;   /* the same of B and of C; 0: G * N */
  int64_t c_stride;
  int64_t dz_stride;  /* the same of dz (backward) */
  int32_t dtype;      /* mamba2_dtype */
  int32_t softplus;   /* 1: the time step is softplus(dt + dt_bias); 0: dt + dt_bias */
} mamba2_scan_dims;

/*
 * selective_scan: the recurrence of the SSD with a decay of its own for each
 * (channel, state).  For token t, channel c, group g = c / (D/G):
 *     d    = softplus(dt[t, c] + dt_bias[c])
 *     h[n] = exp(d * A[c, n]) * h[n] + d * u[t, c] * B[t, g, n]
 *     s    = sum_n C[t, g, n] * h[n] + D[c] * u[t, c]
 *     y    = s * z[t, c] * sigmoid(z[t, c])        (or s, z NULL)
 *     u, dt, y      [B, L, D]; z [B, L, D] rows of z_stride, or NULL
 *     B, C          [B, L, G, N] rows of b_stride and c_stride
 *     A             [D, N] float32, <= 0; D, dt_bias [D] float32 or NULL
 *     init_state, final_state [B, D, N] float32 or NULL
 * u, dt, B, C, z and y have the type of dims; the recurrence is float32.
 * Supported: B * D <= 2^26; ceil(L / 16) * G * ceil(D / G / 64) < 2^24 (the
 * backward's workgroups: 64 channels of one group each, so many small groups
 * count in full); B * L * G * N <= 2^29 (N = 1 counts as 2).
 * Workspace at least mamba2_selective_scan_workspace_bytes(dims) (0: dims invalid),
 * 256-byte aligned.
 */
size_t mamba2_selective_scan_workspace_bytes(const mamba2_scan_dims* dims);

int mamba2_selective_scan_forward(const mamba2_scan_dims* dims, const void* u, const void* dt,
                                  const float* A, const void* B, const void* C, const float* D,
                                  const void* z, const float* dt_bias, const float* init_state,
                                  const int32_t* lengths, void* y, float* final_state,
                                  void* workspace, size_t workspace_bytes, void* stream);

/*
 * Gradients of selective_scan from dy [B, L, D] and dfinal [B, D, N] float32
 * (NULL = zero):
 *     du, ddt [B, L, D]; dz [B, L, D] rows of dz_stride (required exactly
 *     when z is given); dB, dC [B, L, G, N]: type of dims
 *     dA [D, N]; dD, ddt_bias [D] and dinit [B, D, N] (each may be NULL: not
 *     written): float32
 * ddt is the gradient with respect to dt as passed (before bias and
 * softplus); dB and dC are summed over the channels of a group.  The states
 * are recomputed; workspace at least
 * mamba2_selective_scan_backward_workspace_bytes(dims) (0: dims invalid),
 * 256-byte aligned.
 */
size_t mamba2_selective_scan_backward_workspace_bytes(const mamba2_scan_dims* dims);

int mamba2_selective_scan_backward(const mamba2_scan_dims* dims, const void* u, const void* dt,
                                   const float* A, const void* B, const void* C, const float* D,
                                   const void* z, const float* dt_bias, const float* init_state,
                                   const int32_t* lengths, const void* dy, const float* dfinal,
                                   void* du, void* ddt, float* dA, void* dB, void* dC, float* dD,
                                   void* dz, float* ddt_bias, float* dinit, void* workspace,
                                   size_t workspace_bytes, void* stream);

/*
 * One token of selective_scan for every sequence: seqlen must be 1; u, dt, z,
 * y [B, D], B, C [B, G, N] (strides as above); state [B, D, N] float32, read
 * and overwritten.  Bound by HBM on the state.
 */
int mamba2_selective_scan_step(const mamba2_scan_dims* dims, const void* u, const void* dt,
                               const float* A, const void* B, const void* C, const float* D,
                               const void* z, const float* dt_bias, float* state, void* y,
                               void* stream);

typedef struct {
  int64_t rows;      /* R >= 1 */
  int64_t channels;  /* D >= 1 */
  int64_t ngroups;   /* groups of D/G channels that are normalised apart; D/G <= 8192 */
  int64_t x_stride;  /* elements between rows of x; 0: D */
  int64_t z_stride;  /* the same of z, and of dz (backward) */
  int64_t dz_stride;
  float eps;         /* >= 0 */
  int32_t kind;      /* mamba2_norm_kind */
  int32_t dtype;     /* mamba2_dtype */
  int32_t reserved;  /* must be 0 */
} mamba2_norm_dims;

/*
 * norm: per row and group, of v = x * z * sigmoid(z) (v = x where z is NULL),
 *     RMS:   y = v / sqrt(mean(v^2) + eps) * weight + bias
 *     layer: y = (v - mean(v)) / sqrt(mean((v - mean(v))^2) + eps) * weight + bias
 *     x, z, y [R, D] of the type of dims (x and z strided); weight [D]
 *     float32; bias [D] float32 or NULL.  Statistics are float32.
 */
int mamba2_norm_forward(const mamba2_norm_dims* dims, const void* x, const void* z,
                        const float* weight, const float* bias, void* y, void* stream);

/*
 * Gradients of norm from dy [R, D]: dx [R, D], dz [R, D] (rows of dz_stride;
 * required exactly when z is given), dweight [D] and dbias [D] float32
 * (dbias may be NULL: not written).  The statistics are recomputed; workspace
 * at least mamba2_norm_backward_workspace_bytes(dims) (0: dims invalid),
 * 256-byte aligned.
 */
size_t mamba2_norm_backward_workspace_bytes(const mamba2_norm_dims* dims);

int mamba2_norm_backward(const mamba2_norm_dims* dims, const void* x, const void* z,
                         const float* weight, const void* dy, void* dx, void* dz, float* dweight,
                         float* dbias, void* workspace, size_t workspace_bytes, void* stream);

/*
 * The operators of an attention layer
 * -----------------------------------
 * What a layer of softmax attention between SSD layers computes: positions
 * (rotary), attention over prompts with its gradients (attention) and one
 * token of every sequence against a cache (attention_step).  The conventions
 * above hold, those of the operators around the SSD included (strides of
 * tokens, outputs that overlap no input unless it is said here, fixed order
 * of sums).  H query heads read G groups of keys and values: head h reads
 * group h / (H/G).  The values of a sequence's own tokens are finite.
 */
typedef enum { MAMBA2_ROTARY_HALF = 0, MAMBA2_ROTARY_INTERLEAVED = 1 } mamba2_rotary_layout;

typedef struct {
  int64_t batch;     /* B >= 1; B * L <= 2^28 */
  int64_t seqlen;    /* L >= 1 */
  int64_t nheads;    /* H: 1 .. 1024 */
  int64_t ngroups;   /* G: 0 .. 1024; 0: no k */
  int64_t headdim;   /* D <= 1024 */
  int64_t rotary;    /* R: the first R elements of a head are turned; even, 2 .. D */
  int64_t q_stride;  /* elements between tokens of q; 0: H * D */
  int64_t k_stride;  /* the same of k; 0: G * D */
  int64_t yq_stride; /* of yq */
  int64_t yk_stride; /* of yk */
  float scale;       /* > 0: factor of the turned elements */
  int32_t layout;    /* mamba2_rotary_layout */
  int32_t dtype;     /* mamba2_dtype */
  int32_t reserved;  /* must be 0 */
} mamba2_rotary_dims;

/*
 * rotary: pair i (0 .. R/2 - 1) of every head of token t, turned by the angle
 * a = position(t) * inv_freq[i]:
 *     (x1, x2) -> scale * (x1 cos a - x2 sin a, x1 sin a + x2 cos a)
 * The pair is elements (i, i + R/2) (MAMBA2_ROTARY_HALF) or (2i, 2i + 1)
 * (MAMBA2_ROTARY_INTERLEAVED); elements R .. D - 1 are copied as they are.
 *     q, yq     [B, L, H, D] rows of q_stride and yq_stride
 *     k, yk     [B, L, G, D] rows of k_stride and yk_stride (G = 0: not used)
 *     inv_freq  [R/2] float32
 *     positions [B, L] int32, or NULL: token t of a sequence is at t
 * q, k, yq, yk have the type of dims.  Angles are exact to float32 at any
 * position (formed in float64).  yq may be q and yk may be k, with equal
 * strides.  Packed sequences are one batch with their positions.
 * rotary_backward: the gradients dq, dk from those of yq, yk (the same turn
 * the other way; the strides are those of dyq, dyk and dq, dk).
 */
int mamba2_rotary_forward(const mamba2_rotary_dims* dims, const void* q, const void* k,
                          const float* inv_freq, const int32_t* positions, void* yq, void* yk,
                          void* stream);

int mamba2_rotary_backward(const mamba2_rotary_dims* dims, const void* dyq, const void* dyk,
                           const float* inv_freq, const int32_t* positions, void* dq, void* dk,
                           void* stream);

typedef struct {
  int64_t batch;    /* B: 1 .. 65535 sequences */
  int64_t q_len;    /* rows of q for each sequence (padded), or for all together (packed); >= 1 */
  int64_t k_len;    /* the same of k and v */
  int64_t nheads;   /* H: 1 .. 1024 */
  int64_t ngroups;  /* G, divides H */
  int64_t headdim;  /* D: a multiple of 8, at most 128 */
  int64_t q_stride; /* elements between tokens of q; 0: H * D */
  int64_t k_stride; /* the same of k and of v; 0: G * D */
  int64_t v_stride;
  int64_t dq_stride; /* of dq, dk, dv (backward) */
  int64_t dk_stride;
  int64_t dv_stride;
  float scale;      /* > 0; scale * log2(e) is a float32 too */
  int32_t causal;   /* 0 or 1 */
  int32_t q_packed; /* 0 or 1: how the sequences lie in q */
  int32_t k_packed; /* the same of k and v */
  int32_t dtype;    /* mamba2_dtype */
  int32_t reserved; /* must be 0 */
} mamba2_attention_dims;

/*
 * attention: softmax attention of B sequences.  Query i of a sequence with nq
 * queries and nk keys sees the keys j < nk, with causal only j <= i + nk - nq
 * (the last query sees all: a prompt's piece on top of earlier keys).  Per
 * head, with s_j = scale * q_i . k_j over the keys that it sees,
 *     o_i = sum_j exp(s_j - lse_i) v_j,    lse_i = log sum_j exp(s_j)
 * A query that sees no key has o = 0 and lse = -infinity.
 * Scores are float32 (q_i . k_j, and times scale * log2(e)): one above its range
 * makes the query's o and lse NaN (and gradients of its sequence), one below it
 * is a weight of 0; a query all of whose scores are below it has NaN too, or
 * counts as one that sees no key.
 *     q, o  [B, q_len, H, D]  (packed: [q_len, H, D]); q rows of q_stride
 *     k, v  [B, k_len, G, D]  (packed: [k_len, G, D]); rows of k_stride, v_stride
 *     lse   [B, q_len, H] float32 (packed: [q_len, H])
 *     q_seqs, k_seqs  int32.  Padded: [B] lengths (nq, nk), or NULL (all full);
 *           values outside 0 .. len are taken as the nearer bound.  Packed:
 *           [B + 1] starts, not decreasing, taken the same way: sequence b is
 *           rows starts[b] .. starts[b + 1] - 1.
 * q, k, v and o have the type of dims.  What stands behind a sequence's
 * tokens, or in packed rows of no sequence, is not used (it may hold
 * anything); o there is 0, lse -infinity and gradients are zeros.
 * Strides are multiples of 16 bytes and at most 2^22.  Statistics and sums are float32; with
 * bfloat16 the weights are rounded to it before the product with v.
 * Supported: rows of q and of k <= 2^28; rows of q * H / G < 2^31 - 256;
 * workgroups (G times the tiles of 128 rows of q * H / G, or of k; packed: and
 * B + 2) < 2^23.
 * Workspace at least mamba2_attention_workspace_bytes(dims) (0: dims
 * invalid), 256-byte aligned.
 */
size_t mamba2_attention_workspace_bytes(const mamba2_attention_dims* dims);

int mamba2_attention_forward(const mamba2_attention_dims* dims, const void* q, const void* k,
                             const void* v, const int32_t* q_seqs, const int32_t* k_seqs, void* o,
                             float* lse, void* workspace, size_t workspace_bytes, void* stream);

/*
 * Gradients of attention from dout, the gradient of o (lse has none): dq, dk,
 * dv as q, k, v with rows of dq_stride, dk_stride, dv_stride.  o and lse are
 * what the forward wrote for the same inputs; o and dout are without gaps.
 * dk and dv are sums over the heads of a group.  Workspace at least
 * mamba2_attention_backward_workspace_bytes(dims), 256-byte aligned.
 */
size_t mamba2_attention_backward_workspace_bytes(const mamba2_attention_dims* dims);

int mamba2_attention_backward(const mamba2_attention_dims* dims, const void* q, const void* k,
                              const void* v, const int32_t* q_seqs, const int32_t* k_seqs,
                              const void* o, const float* lse, const void* dout, void* dq,
                              void* dk, void* dv, void* workspace, size_t workspace_bytes,
                              void* stream);

typedef struct {
  int64_t batch;    /* B: 1 .. 65535 */
  int64_t rows;     /* rows of a sequence's cache, 1 .. 2^28 */
  int64_t prefix;   /* rows of the shared prefix, 0 .. 2^28; 0: none */
  int64_t nheads;   /* H, G, D as for attention */
  int64_t ngroups;
  int64_t headdim;
  int64_t q_stride; /* elements between sequences of q; 0: H * D */
  int64_t k_stride; /* the same of k and of v; 0: G * D */
  int64_t v_stride;
  float scale;      /* as for attention */
  int32_t dtype;    /* mamba2_dtype */
} mamba2_attention_step_dims;

/*
 * One token of every sequence.  Sequence b has n = lengths[b] tokens in its
 * cache (values outside 0 .. rows are taken as the nearer bound); the token
 * sees the prefix, those n and itself, and its key and value are written to
 * row n of the cache.  A cache with n = rows stays as it is (the token is
 * seen all the same).  lengths is not changed: it belongs to all layers.
 *     q, o  [B, H, D], k, v [B, G, D]; q, k, v rows of their strides
 *     k_cache, v_cache    [B, rows, G, D]; rows behind n are not read
 *     k_prefix, v_prefix  [prefix, G, D]: the first tokens of every sequence
 *     lengths             [B] int32
 * Types and strides as for attention.  Workspace at least
 * mamba2_attention_step_workspace_bytes(dims) (0: dims invalid), 256-byte
 * aligned.  Bound by HBM on the caches; the prefix is read once for all.
 * Supported: B * G * ceil(H / G / 32) and G * ceil(B * H / G / 128) < 2^23.
 */
size_t mamba2_attention_step_workspace_bytes(const mamba2_attention_step_dims* dims);

int mamba2_attention_step(const mamba2_attention_step_dims* dims, const void* q, const void* k,
                          const void* v, void* k_cache, void* v_cache, const int32_t* lengths,
                          const void* k_prefix, const void* v_prefix, void* o, void* workspace,
                          size_t workspace_bytes, void* stream);

/* Static description of a status code. */
const char* mamba2_status_string(int status);

/* Detail of the calling thread's most recent failure ("" if none). */
const char* mamba2_last_error(void);

#ifdef __cplusplus
}
#endif

#endif /* MAMBA2_SSD_H_ */
