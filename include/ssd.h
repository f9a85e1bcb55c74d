/*
 * ssd.h - C ABI of the MI355X (gfx950) Mamba-2 SSD layer core.
 *
 * The operation is the multi-head selective state-space transform with a
 * scalar-times-identity transition per head:
 *
 *     a_t = exp(dt_t * A_h)
 *     h_t = a_t * h_{t-1} + (dt_t * x_t) B_t^T          (state: headdim x dstate per head)
 *     y_t = h_t C_t + D_h * x_t
 *
 * (the recurrence of the "Mamba-2" wiki note, section "Question"; the
 * discretised decay of "Mamba-2: State Space Models and Linear-Time
 * Sequence Modeling Without Attention", section "State Space Models: The
 * Core Abstraction", where the continuous system also carries the D x
 * term; the dt-scaled input of that page's multi-head block, section
 * "Architecture: Multi-Head SSM"; one decay scalar per head, "Transformers
 * are SSMs" paper card, section "How It Works").  B and C are shared by the
 * heads of a group: head h reads group h / (nheads / ngroups).
 *
 * Two modes compute it ("Mamba-2" wiki note, section "Algorithmic Lesson";
 * mohakchugh blog, section "Why This Matters for Hardware"):
 *   ssd_forward - the chunked (dual) mode over a whole sequence: quadratic,
 *                 matmul-shaped work inside chunks of chunk_size tokens and
 *                 the recurrent state passed between chunks (mohakchugh blog,
 *                 section "Block Decomposition"; ql.gl, "The Core of SSD").
 *                 It runs the four stage kernels below in order.
 *   ssd_step    - the recurrent mode: one token per call, O(1) in the
 *                 sequence length (crackai.dev paper card, "Why It Matters").
 *
 * For comparison the library also runs the layer SSD replaces, the Mamba-1
 * selective scan with a diagonal transition per channel
 * (ssd_selective_scan, at the end of this header).
 *
 * Conventions for every call:
 *   - All tensor pointers are DEVICE pointers (current HIP device) to dense,
 *     row-major arrays in the layouts given per call.  The caller owns every
 *     buffer, including the workspace; the library allocates nothing, keeps
 *     no mutable global state and is safe to call from several threads
 *     (except ssd_forward_noalloc, whose static scratch is shared: see there).
 *   - "T" is the storage type of x, B, C, y and of the chunk-entry states:
 *     dtype SSD_F32 (float) or SSD_BF16 (bfloat16, 2 bytes).  dt, A, D,
 *     initial/final/step states and the fp32 workspace arrays are float.
 *     Arithmetic accumulates in fp32; bf16 operands of the matrix-core
 *     products are rounded to nearest even.
 *   - dt must already be positive (softplus applied by the caller) and A
 *     negative (or zero); neither is clamped.
 *   - Work is enqueued on `stream` (a hipStream_t; NULL = the default
 *     stream) and the call returns without synchronising.  SSD_OK means
 *     "enqueued"; completion is the stream's business.
 *   - Arguments are validated on the host before anything is enqueued: an
 *     error status means no device memory was read or written.  A launch
 *     failure reported by the runtime returns SSD_ERR_HIP.  No C++
 *     exception crosses this interface.
 *   - Shape limits: 0 <= batch <= 65535; seqlen >= 0; 1 <= nheads <= 65535
 *     with nheads * headdim <= 2^20; headdim in {16, 32, 64, 128}; dstate a
 *     multiple of 16 in [16, 256]; ngroups >= 1 dividing nheads, with
 *     ngroups * dstate <= 2^20; chunk_size
 *     a multiple of 16 in [16, 256].  seqlen need not be a multiple of
 *     chunk_size: the last chunk is then shorter.
 *   - Outputs must not overlap inputs (the step state is the one in/out
 *     argument); overlap is reported as SSD_ERR_ALIAS.
 *   - Non-finite inputs: in the recurrence a NaN or Inf in x at token t of
 *     head h reaches y only from token t on (in that head and head-dimension
 *     column).  The chunked forwards reach it from the first token of t's
 *     32-token block within its chunk (the block's masked scores are zero
 *     and zero times NaN is NaN on the matrix cores), up to 31 tokens
 *     earlier, still only in that column of that head.  Non-finite dt, B or
 *     C values reach y from their own token on.
 */
#ifndef SSD_MI355X_H
#define SSD_MI355X_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { SSD_F32 = 0, SSD_BF16 = 1 } ssd_dtype;

typedef enum {
    SSD_OK = 0,
    SSD_ERR_NULL = -1,      /* a required pointer is NULL */
    SSD_ERR_SHAPE = -2,     /* a size is out of the supported range */
    SSD_ERR_DTYPE = -3,     /* dtype is not SSD_F32 or SSD_BF16 */
    SSD_ERR_WORKSPACE = -4, /* workspace smaller than ssd_forward_workspace_bytes */
    SSD_ERR_HIP = -5,       /* the HIP runtime reported an error at launch */
    SSD_ERR_ALIAS = -6,     /* an output overlaps an input */
    SSD_ERR_SCRATCH = -7    /* ssd_forward_noalloc: one batch row needs more than the static scratch */
} ssd_status;

/* Human-readable text of a status code (static storage; never NULL). */
const char* ssd_status_string(int status);

/* Version of this interface: 100 * major + minor. */
int ssd_abi_version(void);

/* Number of chunks ceil(seqlen / chunk_size) (0 for seqlen 0); -1 on bad sizes. */
int64_t ssd_num_chunks(int64_t seqlen, int64_t chunk_size);

/* ---------------------------------------------------------------------------------------------
 * Chunked (dual) mode.
 * ------------------------------------------------------------------------------------------- */

/* Bytes of device workspace ssd_forward needs for these sizes: at least 256
 * for valid sizes, 0 when the sizes or dtype are invalid.
 * Layout (each part 256-byte aligned, nc = number of chunks):
 *   dA_cs      float (batch, nheads, nc, chunk_size)
 *   dt_chunked float (batch, nheads, nc, chunk_size)
 *   chunk_states float (batch, nc, nheads, headdim, dstate)
 *   entry_states T   (batch, nc, nheads, headdim, dstate)          */
size_t ssd_forward_workspace_bytes(int64_t batch, int64_t seqlen, int64_t nheads, int64_t headdim,
                                   int64_t dstate, int64_t chunk_size, int dtype);

/* y, final_states = SSD(x, dt, A, B, C, D, init_states) in chunks of chunk_size.
 *   x            T     (batch, seqlen, nheads, headdim)
 *   dt           float (batch, seqlen, nheads)
 *   A, D         float (nheads)
 *   B, C         T     (batch, seqlen, ngroups, dstate)
 *   init_states  float (batch, nheads, headdim, dstate), the state before
 *                token 0 (h_{-1}); NULL means zeros
 *   y            T     (batch, seqlen, nheads, headdim), written
 *   final_states float (batch, nheads, headdim, dstate), written: the state
 *                after the last token (equal to init_states when seqlen = 0)
 *   workspace    device buffer of at least ssd_forward_workspace_bytes()
 * Runs ssd_dA_cumsum, ssd_chunk_state, ssd_state_passing, ssd_chunk_scan. */
int ssd_forward(const void* x, const float* dt, const float* A, const void* B, const void* C,
                const float* D, const float* init_states, void* y, float* final_states,
                int64_t batch, int64_t seqlen, int64_t nheads, int64_t headdim, int64_t dstate,
                int64_t ngroups, int64_t chunk_size, int dtype, void* workspace,
                size_t workspace_bytes, void* stream);

/* ssd_forward for callers that cannot allocate device memory (code under HIP graph capture, tight
 * serving loops, harnesses that forbid hipMalloc): the same arguments, results and errors, with no
 * workspace argument.  The workspace is a static scratch array in the library's device code
 * (ssd_forward_noalloc_scratch_bytes() = 64 MiB), one copy per GPU, held from the library's load
 * until the process ends; the call allocates nothing.  Batch rows are independent, so the forward
 * runs on slices of batch rows whose workspace (ssd_forward_workspace_bytes of the slice) fits the
 * scratch, one slice after another on `stream`; the results equal ssd_forward's bit for bit.
 * Returns SSD_ERR_SCRATCH, before any device work, when one batch row's workspace exceeds the
 * scratch (for example 65536 tokens x 80 heads of 64 x 256 states).  Every call on a GPU shares
 * that GPU's scratch: calls that overlap in time on one GPU (on different streams, or from
 * different threads without ordering) race and give wrong results.  Nothing in the scratch needs
 * to start at zero: every byte a call reads was written by the same call. */
size_t ssd_forward_noalloc_scratch_bytes(void);
int ssd_forward_noalloc(const void* x, const float* dt, const float* A, const void* B, const void* C,
                        const float* D, const float* init_states, void* y, float* final_states, int64_t batch,
                        int64_t seqlen, int64_t nheads, int64_t headdim, int64_t dstate, int64_t ngroups,
                        int64_t chunk_size, int dtype, void* stream);

/* Gradients of ssd_forward (the training pass) for dL/dy = dy and dL/d(final_states) = dfinal
 * (NULL = 0), by the adjoint of the recurrence: the adjoint state runs backwards in time as an SSD
 * of its own (dy as input, C in the role of B), computed with the same stage kernels on
 * time-reversed and role-swapped arrays; the log-decay gradient is the suffix sum over tokens of
 * dy.(y - D x) - (dt x).(dL/d(dt x)), summed within each chunk from its end (bf16 inputs: the mean
 * of the sums from both ends), where the gradient is the inner product of the adjoint and forward
 * states at the chunk boundary (so rounding does not accumulate across chunks).  Arguments as for
 * ssd_forward, plus
 *   dy T (batch, seqlen, nheads, headdim); dfinal float (batch, nheads, headdim, dstate) or NULL
 *   dx T like x; ddt float like dt; dA, dD float (nheads); dB, dC T like B, C;
 *   dinit float (batch, nheads, headdim, dstate): the gradient of the initial state (written
 *     also when init_states is NULL)
 *   workspace of at least ssd_backward_workspace_bytes() bytes
 * dstate must be one of 16, 32, 64, 128, 256 and nheads * dstate <= 2^20.  The decay gradients
 * cancel too much for bf16 operands: fp32 inputs take the fp32 matrix cores for the recompute, the
 * adjoint states and the readouts; with bf16 inputs each fp32 operand there is carried as a pair of
 * bf16 values (hi + lo, the fp32 value to 2^-18) and multiplied on the bf16 matrix cores with fp32
 * sums; dx, dB, dC are rounded to bf16 once. */
size_t ssd_backward_workspace_bytes(int64_t batch, int64_t seqlen, int64_t nheads, int64_t headdim, int64_t dstate,
                                    int64_t ngroups, int64_t chunk_size, int dtype);
int ssd_backward(const void* x, const float* dt, const float* A, const void* B, const void* C, const float* D,
                 const float* init_states, const void* dy, const float* dfinal, void* dx, float* ddt, float* dA,
                 void* dB, void* dC, float* dD, float* dinit, int64_t batch, int64_t seqlen, int64_t nheads,
                 int64_t headdim, int64_t dstate, int64_t ngroups, int64_t chunk_size, int dtype, void* workspace,
                 size_t workspace_bytes, void* stream);

/* The same forward as one pass over the sequence per (batch, head), the state kept on chip (the
 * chunk-ordered walk of the mohakchugh blog's block-decomposition outline, section "Block
 * Decomposition: The Hardware-Aware Algorithm"): a workgroup per (batch, head, slice of the head dimension) steps through the tokens
 * in blocks of 32, so no chunk size and no workspace.  Arguments, layouts, results and errors as for ssd_forward (y and
 * final_states to the same tolerance; the sums run in another order), plus SSD_ERR_SHAPE when
 * headdim x (dstate rounded up to 32, 64, 128 or 256) exceeds 16384 (headdim 128 with dstate > 128).
 * The sequential walk leaves little parallelism on a large GPU: ssd_forward is the fast path. */
int ssd_forward_fused(const void* x, const float* dt, const float* A, const void* B, const void* C, const float* D,
                      const float* init_states, void* y, float* final_states, int64_t batch, int64_t seqlen,
                      int64_t nheads, int64_t headdim, int64_t dstate, int64_t ngroups, int dtype, void* stream);

/* Packed variable-length batch: nseq sequences stored back to back on one token axis of
 * total_tokens tokens, sequence k being tokens cu_seqlens[k] .. cu_seqlens[k+1]-1 (the padding-free
 * variable-length batches of the ql.gl page, section "Mamba-2 Changes More Than the Algorithm").
 * Every sequence starts from a zero state: the recurrence is reset at each sequence start, so y
 * equals running ssd_forward on every sequence alone.  Chunks of chunk_size tokens are laid over the
 * packed axis (a chunk may hold parts of several sequences).
 *   x T (total_tokens, nheads, headdim); dt float (total_tokens, nheads); A, D float (nheads)
 *   B, C T (total_tokens, ngroups, dstate)
 *   cu_seqlens int32 (nseq + 1), DEVICE memory, non-decreasing from 0 to total_tokens (empty
 *     sequences allowed).  Its content is not checked on the host; other content yields
 *     unspecified values but no access outside the buffers.
 *   y T (total_tokens, nheads, headdim), written
 *   final_states float (nseq, nheads, headdim, dstate), written: each sequence's state after its
 *     last token (zeros for an empty sequence)
 *   workspace of at least ssd_forward_varlen_workspace_bytes() bytes:
 *     dA_cs, dt_chunked float (nheads, nc, chunk_size); chunk states float (nc, nheads, headdim,
 *     dstate); entry states T (same shape); int32 per-token sequence starts (total_tokens) and
 *     int32 x 4 per-chunk boundary records (nc)
 * Limits as for ssd_forward with batch 1; 0 <= nseq <= 2^24 (nseq 0 only with no tokens). */
size_t ssd_forward_varlen_workspace_bytes(int64_t total_tokens, int64_t nheads, int64_t headdim, int64_t dstate,
                                          int64_t chunk_size, int dtype);
int ssd_forward_varlen(const void* x, const float* dt, const float* A, const void* B, const void* C, const float* D,
                       const int32_t* cu_seqlens, int64_t nseq, void* y, float* final_states, int64_t total_tokens,
                       int64_t nheads, int64_t headdim, int64_t dstate, int64_t ngroups, int64_t chunk_size, int dtype,
                       void* workspace, size_t workspace_bytes, void* stream);

/* Stage 1 (segment decays).  For every chunk c and position l inside it:
 *   dA_cs[b,h,c,l]      = sum_{j = cQ .. cQ+l} dt[b,j,h] * A[h]
 *   dt_chunked[b,h,c,l] = dt[b, cQ+l, h]
 * so that exp(dA_cs[l] - dA_cs[s]) is the decay product prod_{j=s+1..l} a_j
 * of the matrix-mixer entries ("Mamba-2" wiki note, "Matrix Mixer View").
 * Positions past seqlen in a short last chunk get dt 0 (the sum stays flat).
 *   dt float (batch, seqlen, nheads); A float (nheads)
 *   dA_cs, dt_chunked float (batch, nheads, nc, chunk_size), written */
int ssd_dA_cumsum(const float* dt, const float* A, float* dA_cs, float* dt_chunked, int64_t batch,
                  int64_t seqlen, int64_t nheads, int64_t chunk_size, void* stream);

/* Stage 2 (chunk states).  The state each chunk reaches from a zero state,
 * the rank-dstate factor of the off-diagonal blocks of the mixing matrix
 * ("Mamba-2" wiki note, "Structured Semiseparable Matrices"):
 *   chunk_states[b,c,h,p,n] = sum_l x[b,cQ+l,h,p] * dt_l * exp(dA_cs[Q-1] - dA_cs[l]) * B[b,cQ+l,g(h),n]
 *   x T (batch, seqlen, nheads, headdim); B T (batch, seqlen, ngroups, dstate)
 *   dt_chunked, dA_cs float (batch, nheads, nc, chunk_size) as written by stage 1
 *   chunk_states float (batch, nc, nheads, headdim, dstate), written */
int ssd_chunk_state(const void* x, const void* B, const float* dt_chunked, const float* dA_cs,
                    float* chunk_states, int64_t batch, int64_t seqlen, int64_t nheads,
                    int64_t headdim, int64_t dstate, int64_t ngroups, int64_t chunk_size, int dtype,
                    void* stream);

/* Stage 3 (state passing).  The recurrence between chunks (ql.gl, "The Core
 * of SSD"; mohakchugh blog, "Block Decomposition"), sequential over chunks:
 *   S = init (or 0); for c: entry_states[b,c] = S; S = exp(dA_cs[b,h,c,Q-1]) * S + chunk_states[b,c]
 *   final_states = S
 *   chunk_states float (batch, nc, nheads, headdim, dstate); dA_cs float (batch, nheads, nc, chunk_size)
 *   init_states float (batch, nheads, headdim, dstate) or NULL (zeros)
 *   entry_states T (batch, nc, nheads, headdim, dstate), written (rounded to T)
 *   final_states float (batch, nheads, headdim, dstate), written */
int ssd_state_passing(const float* chunk_states, const float* dA_cs, const float* init_states,
                      void* entry_states, float* final_states, int64_t batch, int64_t seqlen,
                      int64_t nheads, int64_t headdim, int64_t dstate, int64_t chunk_size,
                      int dtype, void* stream);

/* Stage 4 (chunk scan).  The output of every chunk: the masked quadratic
 * (attention-like) form inside the chunk plus the entering state read out
 * by C, plus the skip term (mohakchugh blog, "Block Decomposition" and "The
 * Tensor Core Connection"):
 *   y[l,p] = sum_{s<=l} (C_l . B_s) exp(dA_cs[l] - dA_cs[s]) dt_s x[s,p]
 *          + exp(dA_cs[l]) * sum_n C_l[n] entry_states[c,p,n] + D[h] x[l,p]
 *   x, y T (batch, seqlen, nheads, headdim); B, C T (batch, seqlen, ngroups, dstate)
 *   dt_chunked, dA_cs float (batch, nheads, nc, chunk_size); entry_states T (batch, nc, nheads, headdim, dstate)
 *   D float (nheads) */
int ssd_chunk_scan(const void* x, const void* B, const void* C, const float* dt_chunked,
                   const float* dA_cs, const void* entry_states, const float* D, void* y,
                   int64_t batch, int64_t seqlen, int64_t nheads, int64_t headdim, int64_t dstate,
                   int64_t ngroups, int64_t chunk_size, int dtype, void* stream);

/* ---------------------------------------------------------------------------------------------
 * Recurrent mode.
 * ------------------------------------------------------------------------------------------- */

/* One token: a = exp(dt*A); state = a*state + (dt*x) B^T; y = state C + D x.
 *   state float (batch, nheads, headdim, dstate), read and written IN PLACE
 *   x T (batch, nheads, headdim); dt float (batch, nheads); A, D float (nheads)
 *   B, C T (batch, ngroups, dstate); y T (batch, nheads, headdim), written */
int ssd_step(float* state, const void* x, const float* dt, const float* A, const void* B,
             const void* C, const float* D, void* y, int64_t batch, int64_t nheads,
             int64_t headdim, int64_t dstate, int64_t ngroups, int dtype, void* stream);

/* ---------------------------------------------------------------------------------------------
 * The Mamba-1 selective scan (mohakchugh blog, section "Mamba-1: Selective State Spaces"): each
 * channel d of the input has its own diagonal transition, one decay per state entry, and B, C
 * are per token, shared by all channels:
 *
 *     h_t[d, n] = exp(delta_t[d] A[d, n]) h_{t-1}[d, n] + (delta_t[d] x_t[d]) B_t[n]
 *     y_t[d]    = sum_n C_t[n] h_t[d, n] + D[d] x_t[d]
 *
 * The input enters as delta * B * x, as in ssd_forward.  It runs as a sequential scan on the
 * vector units (one kernel); there is no workspace.
 *   x T (batch, seqlen, dim); delta float (batch, seqlen, dim), positive
 *   A float (dim, dstate), negative or zero; D float (dim)
 *   B, C T (batch, seqlen, dstate)
 *   init_states float (batch, dim, dstate) or NULL (zeros)
 *   y T (batch, seqlen, dim), written; final_states float (batch, dim, dstate), written
 * Shape limits: 0 <= batch <= 65535; 0 <= seqlen < 2^31; dim a multiple of 8 in [8, 2^20];
 * dstate in {4, 8, 16, 32, 64}.  x, delta and y must be 16-byte aligned; with seqlen 0 the
 * token arrays (x, delta, B, C, y) may be NULL and final_states receives the initial state.  Errors as above
 * (SSD_ERR_SHAPE for a bad size or alignment, SSD_ERR_ALIAS when an output overlaps an input
 * or the other output). */
int ssd_selective_scan(const void* x, const float* delta, const float* A, const void* B, const void* C,
                       const float* D, const float* init_states, void* y, float* final_states, int64_t batch,
                       int64_t seqlen, int64_t dim, int64_t dstate, int dtype, void* stream);

/* ---------------------------------------------------------------------------------------------
 * The gated delta rule: the other recurrence of linear-recurrent sequence layers.  Like the SSD layer
 * a head keeps a headdim x dstate state that decays by one scalar per token, but a token first takes out
 * what the state already answers for its key, then writes its value (beta in [0, 1] says how much):
 *
 *     S' = exp(g_t) S_{t-1}
 *     e_t = v_t - S' k_t                  (what the state does not yet answer for k_t)
 *     S_t = S' + beta_t e_t k_t^T
 *     y_t = S_t q_t
 *
 * v takes the place of x, k of B, q of C in the calls above: k and q are shared by the heads of a group
 * (head h reads group h / (nheads / ngroups)).  Conventions, limits and errors are those at the top of
 * this header, and:
 *   - g is the log decay, <= 0 (dt * A in the SSD layer's terms); it is not clamped, except that
 *     every g below -1000 acts as -1000 (exp is 0 in fp32 from -104 on), so -inf is a reset.
 *   - k is used as given.  The recurrence is stable for beta |k|^2 < 2: callers scale k to at most unit
 *     length.  q carries any scale the caller wants on y.
 *   - 0 <= batch <= 65535; nseq <= 2^24; (tokens / 32 + rows) * nheads < 2^24 and rows * nheads * headdim < 2^29,
 *     rows being batch or nseq (for ssd_delta_step batch * nheads < 2^24).  There is no chunk size.
 *   - With bf16 inputs the final states and the fp32 gradients keep fp32's accuracy (about 1e-5 of their
 *     norm, up to 3e-5 where all keys of a row are alike): every fp32 operand of a matrix-core product
 *     that reaches them is carried as a pair of bf16 values.  For dg that is each head's own norm, however
 *     strong its decay (a few times more in a head of a few dozen tokens whose final state has a gradient), unless what
 *     it is summed from cancels, as where one unit key is written again and again with beta 1.
 *   - The bf16 outputs are a little further off than their own rounding (1.7e-3 of the norm): y 2.4e-3, because the
 *     state and the scores are rounded to bf16 where they lead to y only, dk and dq 1.8e-3, dv 1.7e-3.  The roundings go
 *     with the terms of a sum: where these cancel, as with like keys, more of the sum is lost (y 4e-3 to 9e-3, dk and
 *     dq 2.5e-3 to 3e-3).  With fp32 inputs everything is fp32.
 *   - Non-finite inputs: the sums run over blocks of 32 tokens in which a later token's values carry a
 *     weight of zero, so a NaN or Inf at a token can reach the outputs of earlier tokens of the same
 *     32-token block of its sequence (and all later ones), never another sequence, batch row or group.
 *     ssd_delta_backward sums over chunks of 64: beside the gradients that depend on the token, all of its chunk's.
 * ------------------------------------------------------------------------------------------- */

/* y, final_states of the gated delta rule over whole sequences.
 *   v T (batch, seqlen, nheads, headdim); g, beta float (batch, seqlen, nheads)
 *   k, q T (batch, seqlen, ngroups, dstate)
 *   init_states float (batch, nheads, headdim, dstate) or NULL (zeros)
 *   y T like v, written; final_states float (batch, nheads, headdim, dstate), written: the state after the
 *     last token (the initial one when seqlen = 0)
 *   workspace of at least ssd_delta_forward_workspace_bytes() bytes (0 = the sizes or dtype are refused): 6.5 KB
 *     (fp32 8.5) for every 32 tokens of a row and head; 0.27 GB at 4 x 4096 tokens and 80 heads in bf16 */
size_t ssd_delta_forward_workspace_bytes(int64_t batch, int64_t seqlen, int64_t nheads, int64_t headdim,
                                         int64_t dstate, int64_t ngroups, int dtype);
int ssd_delta_forward(const void* v, const float* g, const float* beta, const void* k, const void* q,
                      const float* init_states, void* y, float* final_states, int64_t batch, int64_t seqlen,
                      int64_t nheads, int64_t headdim, int64_t dstate, int64_t ngroups, int dtype, void* workspace,
                      size_t workspace_bytes, void* stream);

/* The same for a packed variable-length batch, laid out as for ssd_forward_varlen: sequence i is tokens
 * cu_seqlens[i] .. cu_seqlens[i + 1] - 1 of one token axis.
 *   v, y T (total_tokens, nheads, headdim); g, beta float (total_tokens, nheads); k, q T (total_tokens, ngroups, dstate)
 *   cu_seqlens int32 (nseq + 1), DEVICE memory, non-decreasing from 0 to total_tokens (empty sequences
 *     allowed); content not checked, other content yields unspecified values but no access outside the buffers
 *   init_states float (nseq, nheads, headdim, dstate) or NULL (zeros): a sequence may continue from a state
 *   final_states float (nseq, nheads, headdim, dstate), written */
size_t ssd_delta_forward_varlen_workspace_bytes(int64_t total_tokens, int64_t nseq, int64_t nheads, int64_t headdim,
                                                int64_t dstate, int64_t ngroups, int dtype);
int ssd_delta_forward_varlen(const void* v, const float* g, const float* beta, const void* k, const void* q,
                             const int32_t* cu_seqlens, int64_t nseq, const float* init_states, void* y,
                             float* final_states, int64_t total_tokens, int64_t nheads, int64_t headdim,
                             int64_t dstate, int64_t ngroups, int dtype, void* workspace, size_t workspace_bytes,
                             void* stream);

/* Gradients of ssd_delta_forward for dL/dy = dy and dL/d(final_states) = dfinal (NULL = 0), by the adjoint of the
 * recurrence in the same blocks; y and the states are recomputed.
 *   dy T like v; dfinal float (batch, nheads, headdim, dstate) or NULL
 *   dv T like v; dg, dbeta float like g; dk, dq T like k (summed over a group's heads, in a fixed order);
 *   dinit float (batch, nheads, headdim, dstate), written also when init_states is NULL
 *   workspace of at least ssd_delta_backward_workspace_bytes() bytes: for bf16 inputs 2.1 GB at 4 x 4096 tokens, 80
 *     heads of 64 x 128; 12.4 GB at 65536 tokens, 80 heads of 64 x 256 (mostly the states kept every 64 tokens)
 * dg at the first token is 0 without an initial state (nothing decays into it), and 0 at every token with g below -104
 * (exp(g) is below fp32's range: nothing of the state passes). */
size_t ssd_delta_backward_workspace_bytes(int64_t batch, int64_t seqlen, int64_t nheads, int64_t headdim,
                                          int64_t dstate, int64_t ngroups, int dtype);
int ssd_delta_backward(const void* v, const float* g, const float* beta, const void* k, const void* q,
                       const float* init_states, const void* dy, const float* dfinal, void* dv, float* dg,
                       float* dbeta, void* dk, void* dq, float* dinit, int64_t batch, int64_t seqlen, int64_t nheads,
                       int64_t headdim, int64_t dstate, int64_t ngroups, int dtype, void* workspace,
                       size_t workspace_bytes, void* stream);

/* One token, the state advanced IN PLACE.
 *   state float (batch, nheads, headdim, dstate); v T (batch, nheads, headdim); g, beta float (batch, nheads)
 *   k, q T (batch, ngroups, dstate); y T (batch, nheads, headdim), written */
int ssd_delta_step(float* state, const void* v, const float* g, const float* beta, const void* k, const void* q,
                   void* y, int64_t batch, int64_t nheads, int64_t headdim, int64_t dstate, int64_t ngroups,
                   int dtype, void* stream);

/* ---------------------------------------------------------------------------------------------
 * Linear attention with a decay for each head: the recurrence with a constant decay, a query per head, and keys and
 * values that may be shared by the heads of a group (retention; grouped queries).
 *
 *     S_t = exp(g_h) S_{t-1} + v_t k_t^T      (state: headdim x dstate per head, as above)
 *     y_t = S_t q_t
 *
 * q is a head's own; head h reads k and v of group h / (nheads / ngroups), ngroups = nheads where nothing is shared.
 * Conventions and errors are those at the top of this header, and:
 *   - g float (nheads) is the log decay, <= 0 and constant in time; it is not clamped, except that every g below
 *     -1000 acts as -1000, so -inf leaves each token alone. A power of the decay below 2^-126 (exp(-87)) is 0. g = 0
 *     is plain causal linear attention. A NaN makes all of its head's results NaN. No scale is applied to q.
 *   - headdim and dstate are multiples of 16 in [16, 256]; nheads * headdim and nheads * dstate <= 2^20; 0 <= batch <=
 *     65535, nseq <= 2^24, tokens < 2^31. There is no chunk size. Grids limit the sizes too (SSD_ERR_SHAPE): (rows + their
 *     segments) * nheads * the 64-column slices of the wider of headdim and dstate < 2^24, rows * nheads * headdim * dstate
 *     < 2^34, tokens * ngroups * the wider < 2^34; for ssd_linear_step batch * nheads * headdim < 2^28.
 *   - Final states, dinit and dg keep fp32's accuracy with bf16 inputs too: what leads to them is carried as three bf16
 *     values. States and dinit are off by 5e-7 of their norm, dg by 1e-6 of the 2-norm of what its tokens add to it (more of dg
 *     itself where that cancels). A state is rounded three times with every chunk of 32 tokens, with fp32 inputs with every
 *     token; where it hardly decays n roundings add up to 2^-24 sqrt(n / 6) of its norm. Measured: states 4e-7 after 2048
 *     tokens, 1.6e-6 after 65536, with fp32 inputs 8e-7 and 4.7e-6; dg 3.3e-6 after 65536.
 *   - bf16 outputs are a little further off than their own rounding (1.7e-3 of the norm), because the scores and, where they are
 *     read, the states are rounded to bf16 on the way: 2.4e-3, at most 2.6e-3. With fp32 inputs everything is fp32: outputs
 *     are off by 1e-6 of their norm and by what their states are.
 *   - Sums are made in a fixed order: the same call gives the same bits.
 *   - Non-finite inputs: tokens are summed in chunks of 32 (of their sequence or of a segment of it) in which later
 *     tokens have a weight of zero, so a NaN or Inf at a token can reach the outputs of earlier tokens of its chunk and
 *     all later ones (where the decay has left nothing of it, it need not), of the heads that read it, never another
 *     sequence, batch row or group. dk's and dv's chunks go from the end: there it can reach later tokens of the
 *     chunk and all earlier ones. What arrives of an Inf is an Inf or a NaN: with bf16 inputs a NaN in the states, as an Inf
 *     less its bf16 value is, and where it meets a weight or an element of zero.
 * ------------------------------------------------------------------------------------------- */

/* y, final_states over whole sequences.
 *   v T (batch, seqlen, ngroups, headdim); g float (nheads); k T (batch, seqlen, ngroups, dstate)
 *   q T (batch, seqlen, nheads, dstate)
 *   init_states float (batch, nheads, headdim, dstate) or NULL (zeros)
 *   y T (batch, seqlen, nheads, headdim), written; final_states float (batch, nheads, headdim, dstate), written: the state
 *     after the last token (the initial one when seqlen = 0)
 *   workspace of at least ssd_linear_forward_workspace_bytes() bytes (0 = the sizes or dtype are refused): the states
 *     between segments where rows are cut into segments, else 256 */
size_t ssd_linear_forward_workspace_bytes(int64_t batch, int64_t seqlen, int64_t nheads, int64_t headdim,
                                          int64_t dstate, int64_t ngroups, int dtype);
int ssd_linear_forward(const void* v, const float* g, const void* k, const void* q, const float* init_states, void* y,
                       float* final_states, int64_t batch, int64_t seqlen, int64_t nheads, int64_t headdim,
                       int64_t dstate, int64_t ngroups, int dtype, void* workspace, size_t workspace_bytes, void* stream);

/* The same for a packed variable-length batch: sequence i is tokens cu_seqlens[i] .. cu_seqlens[i + 1] - 1 of one token
 * axis; a sequence may continue from a state.
 *   v T (total_tokens, ngroups, headdim); k T (total_tokens, ngroups, dstate); q T (total_tokens, nheads, dstate)
 *   cu_seqlens int32 (nseq + 1), DEVICE memory, non-decreasing from 0 to at most total_tokens (empty sequences
 *     allowed); content not checked, other content yields unspecified values but no access outside the buffers. Tokens
 *     behind cu_seqlens[nseq] are no sequence's: their y is left as it was
 *   init_states float (nseq, nheads, headdim, dstate) or NULL (zeros)
 *   y T (total_tokens, nheads, headdim), written; final_states float (nseq, nheads, headdim, dstate), written */
size_t ssd_linear_forward_varlen_workspace_bytes(int64_t total_tokens, int64_t nseq, int64_t nheads, int64_t headdim,
                                                 int64_t dstate, int64_t ngroups, int dtype);
int ssd_linear_forward_varlen(const void* v, const float* g, const void* k, const void* q, const int32_t* cu_seqlens,
                              int64_t nseq, const float* init_states, void* y, float* final_states,
                              int64_t total_tokens, int64_t nheads, int64_t headdim, int64_t dstate, int64_t ngroups,
                              int dtype, void* workspace, size_t workspace_bytes, void* stream);

/* Gradients of ssd_linear_forward for dL/dy = dy and dL/d(final_states) = dfinal (NULL = 0).
 *   dy T like y; dfinal float (batch, nheads, headdim, dstate) or NULL
 *   dv, dk T like v, k: summed over the heads of a group, in their order, and rounded once; dq T like q
 *   dg float (nheads): summed over tokens and batch rows, 0 where g is below -87.3 (and without rows)
 *   dinit float (batch, nheads, headdim, dstate), written also when init_states is NULL
 *   workspace of at least ssd_linear_backward_workspace_bytes() bytes: with shared keys and values an fp32 copy of every
 *     head's dk and dv, else the states between segments and a few sums */
size_t ssd_linear_backward_workspace_bytes(int64_t batch, int64_t seqlen, int64_t nheads, int64_t headdim,
                                           int64_t dstate, int64_t ngroups, int dtype);
int ssd_linear_backward(const void* v, const float* g, const void* k, const void* q, const float* init_states,
                        const void* dy, const float* dfinal, void* dv, float* dg, void* dk, void* dq, float* dinit,
                        int64_t batch, int64_t seqlen, int64_t nheads, int64_t headdim, int64_t dstate,
                        int64_t ngroups, int dtype, void* workspace, size_t workspace_bytes, void* stream);

/* One token, the states advanced IN PLACE.
 *   state float (nslots, nheads, headdim, dstate); v T (batch, ngroups, headdim); k T (batch, ngroups, dstate)
 *   q T (batch, nheads, dstate); y T (batch, nheads, headdim), written
 *   slots int32 (batch), DEVICE memory, or NULL (then nslots = batch, row i's state is state[i]): row i's state is
 *     state[slots[i]]. A row whose slot is out of range (padding: -1) touches no state and gets y = 0, and so
 *     does a row whose slot an earlier row has. States that no row names are left as they were. */
int ssd_linear_step(float* state, const int32_t* slots, int64_t nslots, const void* v, const float* g, const void* k,
                    const void* q, void* y, int64_t batch, int64_t nheads, int64_t headdim, int64_t dstate,
                    int64_t ngroups, int dtype, void* stream);

/* ---------------------------------------------------------------------------------------------
 * Pools of states. A server keeps the states of ssd_step, ssd_delta_step or ssd_linear_step in slots of a pool, one
 * sequence a slot: copying, forking, reordering, compacting and freeing them is one map of slots,
 *
 *     states[l, i] = source[l, src[i]]   where 0 <= src[i] < nsource
 *     states[l, i] = 0                   where src[i] = -1 (freed)
 *     states[l, i] stays                 for any other src[i]
 *
 * for every layer l. With source NULL it works IN PLACE: every slot takes what src[i] held before the call, whatever
 * the map (beams reordered, one prompt forked to many, live slots moved together), and src[i] = i leaves a slot alone.
 *   states float (nlayers, nslots, slot_floats), read (in place) and written
 *   source float (nlayers, nsource, slot_floats) or NULL (then nsource = nslots): for instance the final states of a prefill
 *   src int32 (nslots), DEVICE memory; any content is safe
 * No workspace. 0 <= nlayers <= 65535; 0 <= nslots <= 65535, in place at most 2048, since all that moves is held at once;
 * nsource <= 2^24; slot_floats (nheads * headdim * dstate) a multiple of 4, at most 2^32. The values are copied as they are, NaN
 * included. A larger pool moves through a buffer of as many states as move, in two calls: into the buffer with source = the
 * pool, and back with source = the buffer (-2 for the slots that stay). ssd_step and ssd_delta_step take no slots: they
 * advance the first `batch` states of a layer, which a pool that is kept compact has its live ones in. */
int ssd_state_move(float* states, const float* source, const int32_t* src, int64_t nlayers, int64_t nslots,
                   int64_t nsource, int64_t slot_floats, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* SSD_MI355X_H */
