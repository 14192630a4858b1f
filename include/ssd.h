/*
 * libssd -- Mamba-2 SSD (state space duality) chunked selective-scan forward
 * for AMD MI355X (gfx950).  C ABI; no HIP or torch types appear here.
 *
 * The operation
 * -------------
 * For every sequence b, head h (B/C group g = floor(h*G/H)) and token t:
 *
 *     h_t[p][n] = exp(dt[b,t,h] * A[h]) * h_{t-1}[p][n] + dt[b,t,h] * x[b,t,h,p] * B[b,t,g,n]
 *     y[b,t,h,p] = sum_n C[b,t,g,n] * h_t[p][n] + D[h] * x[b,t,h,p]
 *
 * with h_{-1} = init_state[b,h] (zero when absent).  This is the selective
 * SSM with one scalar decay per head that the Mamba-2 SSD layer evaluates
 * ("Transformers are SSMs" article, cloud.tencent.com.cn, section
 * "核心创新——SSD"; the page's formula image is lost and the recurrence above
 * is the reading used, with y read after the state update).
 *
 * It is evaluated by the block decomposition of section "SSD算法" of that
 * article: the sequence is cut into chunks of `chunk_size` tokens; inside a
 * chunk the output is computed in the attention-like quadratic form from a
 * zero state (orange part), each chunk's final state from a zero start is a
 * batched matrix product (green), a short scan over chunks turns those into
 * every chunk's true initial state (yellow), and each chunk's output gains
 * the contribution of that initial state (blue).  Section
 * "深入解析分块与状态传递机制" describes the same four steps.  The result equals
 * the recurrence up to floating-point rounding for every chunk size.
 *
 * Multi-step verify ("3天把Llama训成Mamba" article, blog.csdn.net, section
 * "推测解码"): started from a cached state, one call returns every output,
 * the state after the last token (final_state) and the state after a
 * per-sequence accepted index (state_out), the only extra state the
 * speculative-decoding verifier keeps.
 *
 * Conventions common to every entry point
 * ---------------------------------------
 * - All tensor pointers are DEVICE pointers, owned by the caller, dense and
 *   row-major in the shapes given below (last dimension fastest).  The
 *   library never allocates, frees or synchronises device memory.
 * - Work is enqueued asynchronously on `hip_stream` (a hipStream_t passed as
 *   void*; NULL = the default stream) in stream order.
 * - Every argument check runs on the host before the first launch: a return
 *   other than SSD_OK means nothing was enqueued and no output was touched.
 * - Device-side values are preconditions, not checked (checking would need
 *   a synchronisation): dt finite and >= 0, A finite and <= 0, state_out_idx
 *   in [-1, seqlen-1].  Violations give unspecified values but never an
 *   out-of-bounds access (indices are clamped).
 * - ssd_last_error() holds a description of the last non-OK return on the
 *   calling thread.
 */
#ifndef SSD_H
#define SSD_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define SSD_ABI_VERSION 8

/* Element type of x, B, C and y.  dt, A, D and every state are always fp32. */
typedef enum {
    SSD_DTYPE_F32 = 0,
    SSD_DTYPE_BF16 = 1
} ssd_dtype;

typedef enum {
    SSD_OK = 0,
    SSD_ERR_NULL = 1,        /* a required pointer is NULL                          */
    SSD_ERR_SHAPE = 2,       /* a size is negative, or ngroups does not divide nheads */
    SSD_ERR_CHUNK = 3,       /* chunk_size not in {8, 16, 32, 64, 128, 256}          */
    SSD_ERR_ALIGN = 4,       /* a tensor pointer is not 16-byte aligned              */
    SSD_ERR_WORKSPACE = 5,   /* workspace NULL or smaller than the call's path needs */
    SSD_ERR_ALIAS = 6,       /* an output overlaps an input, another output or the workspace */
    SSD_ERR_ARGS = 7,        /* state_out without state_out_idx or vice versa, an unknown
                                dtype or path, or marks missing for n_marks > 0      */
    SSD_ERR_HIP = 8,         /* a kernel launch failed; outputs are unspecified      */
    SSD_ERR_UNSUPPORTED = 9  /* headdim not in {16,32,64,128}, dstate not in {16,32,64,128,256},
                                fp32 with headdim*dstate > 16384, or a requested path
                                that does not take the call                          */
} ssd_status;

/* Problem sizes.  batch and seqlen may be 0. */
typedef struct {
    int64_t batch;    /* b: independent sequences                     */
    int64_t seqlen;   /* T: tokens per sequence                       */
    int64_t nheads;   /* H: heads (one scalar decay A[h] each)         */
    int64_t headdim;  /* P: channels per head                         */
    int64_t dstate;   /* N: state size per channel                    */
    int64_t ngroups;  /* G: B/C groups; head h reads group h*G/H      */
} ssd_shape;

/* How a call is computed.  Every path gives the same results up to
 * floating-point rounding; the automatic choice depends only on the shape,
 * chunk_size and dtype (ssd_select_path).
 *   SSD_PATH_ONE_CHUNK       at most 32 tokens in one chunk (the multi-step
 *                            verify, a decode step): one kernel reads the
 *                            initial state once and writes y, final_state
 *                            and state_out.  Needs headdim a multiple of
 *                            1024 / dstate.
 *   SSD_PATH_SINGLE_PASS     bf16, dstate 64 or 128, headdim 32, 64 or 128,
 *                            at least 64 items (an item is a (b, h) pair, or
 *                            a 64-channel half of a head of headdim 128):
 *                            one kernel walks each item's sequence in
 *                            128-token blocks with the state in registers
 *                            (the state passing of section
 *                            "深入解析分块与状态传递机制" of the "Transformers
 *                            are SSMs" article, carried inside the kernel).
 *                            When there are fewer items than workgroups, an
 *                            item's blocks are split into ranges; a range
 *                            not starting at token 0 first recomputes the
 *                            state it starts from, so no workgroup ever
 *                            waits for another.  Its internal block length
 *                            does not depend on chunk_size.
 *   SSD_PATH_CHUNK_PARALLEL  any call: the four steps of the block
 *                            decomposition as separate kernels, with the
 *                            intermediates in the workspace.
 * No path uses the workspace except SSD_PATH_CHUNK_PARALLEL. */
typedef enum {
    SSD_PATH_AUTO = 0,
    SSD_PATH_ONE_CHUNK = 1,
    SSD_PATH_SINGLE_PASS = 2,
    SSD_PATH_CHUNK_PARALLEL = 3
} ssd_path;

/* The path ssd_chunk_scan_fwd takes for this problem; SSD_PATH_AUTO (0) when
 * batch or seqlen is 0 (no kernel but a state copy runs), -1 when the
 * arguments are invalid (ssd_last_error() says why). */
int ssd_select_path(const ssd_shape *shape, int chunk_size, ssd_dtype dtype);

/* The workspace of SSD_PATH_CHUNK_PARALLEL: byte offsets from the workspace
 * pointer of the intermediates that path leaves there, exposed so that the
 * individual steps can be checked.
 *   cumsum   fp32 [batch, nheads, nchunks, chunk_size]: the chunk-local
 *            cumulative log-decay A[h] * sum_{k<=i} dt[b, c*Q+k, h]; tokens
 *            past seqlen count as dt = 0.
 *   ct       fp32, same layout: cs * log2(e) - log2(dt) (+inf past seqlen),
 *            so that dt_j exp(cs_i - cs_j) = exp2(cs_i log2(e) - ct_j).
 *   dt_decay fp32, same layout: dt_i * exp(cs_e - cs_i), e = the last token
 *            (within seqlen) of the 32-token block holding i.
 *   states   dtype [batch, nchunks, nheads, headdim, dstate]: entry c is the
 *            state chunk c reaches from a zero initial state (accumulated in
 *            fp32, rounded to nearest even to dtype once).
 *   prev     dtype, same layout: entry c is the state entering chunk c,
 *            rounded to nearest even to dtype; entry 0 is written only when
 *            init_state is given (otherwise it is never read).
 *   hj       fp32 [batch, nheads, headdim, dstate]: the state entering the
 *            chunk that holds state_out_idx[b] (written only with state_out).
 * Every region a kernel reads was written earlier in the same call: the
 * contents on entry never matter. */
typedef struct {
    size_t cumsum_offset;
    size_t ct_offset;
    size_t dt_decay_offset;
    size_t states_offset;
    size_t prev_offset;
    size_t hj_offset;
    size_t total_bytes;   /* bytes SSD_PATH_CHUNK_PARALLEL needs (0 when batch or seqlen is 0) */
    int64_t nchunks;
} ssd_workspace_layout;

/* Bytes of device workspace ssd_chunk_scan_fwd needs for this problem: the
 * layout's total_bytes when the call takes SSD_PATH_CHUNK_PARALLEL, else 0
 * (then workspace may be NULL).  0 also when the arguments are invalid
 * (ssd_last_error() says why). */
size_t ssd_workspace_bytes(const ssd_shape *shape, int chunk_size, ssd_dtype dtype);

/* Fills *out with the workspace layout of SSD_PATH_CHUNK_PARALLEL for this
 * problem (also for problems that take another path automatically). */
ssd_status ssd_get_workspace_layout(const ssd_shape *shape, int chunk_size, ssd_dtype dtype,
                                    ssd_workspace_layout *out);

/* The SSD chunked-scan forward.
 *
 *   x             [b,T,H,P]  dtype      input channels
 *   dt            [b,T,H]    fp32       step sizes, already positive (no
 *                                       softplus, bias or clamp is applied)
 *   A             [H]        fp32       per-head decay rate (<= 0)
 *   B, C          [b,T,G,N]  dtype      input / output projections of the state
 *   D             [H]        fp32       skip weight; NULL = no skip term
 *   init_state    [b,H,P,N]  fp32       state before token 0; NULL = zeros
 *   chunk_size    Q in {8,16,32,64,128,256}; any T >= 0 (the last chunk may
 *                 be partial).  Results do not depend on Q beyond rounding.
 *   y             [b,T,H,P]  dtype      outputs, fully overwritten (rounded
 *                                       to nearest even from fp32 for bf16)
 *   final_state   [b,H,P,N]  fp32       state after token T-1; NULL = not returned
 *   state_out_idx [b]        int32      accepted index j_b per sequence; NULL = none
 *   state_out     [b,H,P,N]  fp32       state after token j_b (0-based,
 *                                       inclusive; j_b = -1 gives init_state);
 *                                       non-NULL exactly when state_out_idx is
 *   shape, dtype             sizes and element type as above
 *   workspace     device scratch of at least ssd_workspace_bytes(...) bytes,
 *                 16-byte aligned; contents on entry are ignored; may be
 *                 NULL when ssd_workspace_bytes(...) is 0
 *   hip_stream    hipStream_t as void*, NULL for the default stream
 *
 * Outputs must not overlap inputs, each other or the workspace, with one
 * exception: final_state may be init_state itself (same pointer), updating
 * the state in place (a decode step, a verifier keeping its cache).  An
 * in-place call on SSD_PATH_SINGLE_PASS runs every item whole on one
 * workgroup (no ranges), since a range's recomputation reads init_state.
 * Errors: see ssd_status; checks are host-side and happen before any launch. */
ssd_status ssd_chunk_scan_fwd(const void *x, const float *dt, const float *A,
                              const void *B, const void *C, const float *D,
                              const float *init_state, int chunk_size,
                              void *y, float *final_state,
                              const int32_t *state_out_idx, float *state_out,
                              const ssd_shape *shape, ssd_dtype dtype,
                              void *workspace, size_t workspace_bytes, void *hip_stream);

/* Same as ssd_chunk_scan_fwd with two additions.
 *   path    SSD_PATH_AUTO, or the path to take (SSD_ERR_UNSUPPORTED when it
 *           does not take the call; calls of zero tokens or sequences only
 *           copy states whatever the path).  The workspace must then hold the
 *           bytes that path needs: the layout's total_bytes for
 *           SSD_PATH_CHUNK_PARALLEL, none for the others.
 *   marks   caller-created HIP events (hipEvent_t as void*) recorded on
 *           hip_stream around the kernels, so that a caller can time each
 *           kernel in place: marks[0] before the first kernel, marks[k]
 *           after the k-th kernel launched (k = 1 .. n_marks-1).  Marks
 *           beyond the kernels launched are not recorded.  n_marks may be 0
 *           (marks NULL).
 * On SSD_OK, *n_kernels (if non-NULL) is the number of kernels launched and
 * kernel_names[k-1] (if kernel_names is non-NULL and k < n_marks) names the
 * kernel that marks[k] ends. */
ssd_status ssd_chunk_scan_fwd_ex(const void *x, const float *dt, const float *A,
                                 const void *B, const void *C, const float *D,
                                 const float *init_state, int chunk_size,
                                 void *y, float *final_state,
                                 const int32_t *state_out_idx, float *state_out,
                                 const ssd_shape *shape, ssd_dtype dtype,
                                 void *workspace, size_t workspace_bytes, void *hip_stream,
                                 int path, void *const *marks, int n_marks, int *n_kernels,
                                 const char **kernel_names);

/* Bytes of the library's static device scratch (64 MiB), the workspace of
 * ssd_chunk_scan_fwd_noalloc. */
#define SSD_NOALLOC_SCRATCH_BYTES (64u << 20)

/* ssd_chunk_scan_fwd without a workspace argument, for callers that cannot
 * allocate device memory (code under HIP graph capture, tight serving loops,
 * harnesses that forbid allocation).  A call that needs a workspace (the
 * chunk-parallel path, ssd_workspace_bytes(...) > 0) uses a static array of
 * SSD_NOALLOC_SCRATCH_BYTES in the library's device code instead; every GPU
 * holds its own copy until the process ends, and its device address is
 * looked up once per GPU on the first such call there.  Neither this entry
 * point nor anything it calls allocates or frees memory.
 *   - Calls needing more than SSD_NOALLOC_SCRATCH_BYTES return
 *     SSD_ERR_WORKSPACE before anything is enqueued.
 *   - hip_stream must belong to the current device (else SSD_ERR_ARGS).
 *   - All calls on one GPU share its scratch: calls that may overlap in time
 *     on one GPU (on different streams, or from several threads without
 *     ordering) race and give unspecified results.  Calls in one stream's
 *     order are safe.  The scratch keeps the last call's intermediates;
 *     nothing in a call depends on what it held before.
 * Arguments, results and every other error are as for ssd_chunk_scan_fwd. */
ssd_status ssd_chunk_scan_fwd_noalloc(const void *x, const float *dt, const float *A,
                                      const void *B, const void *C, const float *D,
                                      const float *init_state, int chunk_size,
                                      void *y, float *final_state,
                                      const int32_t *state_out_idx, float *state_out,
                                      const ssd_shape *shape, ssd_dtype dtype, void *hip_stream);

/* Sequence sharding (context parallelism): the step a GPU runs on its shard
 * once it knows the state entering the shard.
 *
 * "Transformers are SSMs" article (cloud.tencent.com.cn), section
 * "序列并行的两种形式": with the sequence split over GPUs, each GPU computes
 * its shard's outputs and final state on its own and only states pass between
 * GPUs.  A shard run with ssd_chunk_scan_fwd from a zero initial state gives
 * y0, F (its final_state) and, with an accepted index, h0_j (its state_out).
 * The recurrence is linear in its initial state, so from the true entering
 * state h_in the shard's results are
 *     y_t   = y0_t + exp(cs_t) * sum_n C[b,t,g,n] * h_in[b,h,p,n]
 *     final = F + exp(cs_{T-1}) * h_in
 *     h_j   = h0_j + exp(cs_j) * h_in          (j = -1: h0_j + h_in)
 * with cs_t = A[h] * sum_{k<=t} dt[b,k,h] over the shard's own tokens.  This
 * call applies them in place; the exchange of states between GPUs is the
 * caller's.
 *
 *   y             [b,T,H,P]  dtype  in/out: y0 on entry, y on return (rounded
 *                                   to nearest even from fp32 for bf16)
 *   dt, A, C      as passed to ssd_chunk_scan_fwd for the shard
 *   h_in          [b,H,P,N]  fp32   state entering the shard (required)
 *   shard_final   [b,H,P,N]  fp32   F; required when final_state is given
 *   final_state   [b,H,P,N]  fp32   out: F + exp(cs_{T-1}) h_in; NULL = not
 *                                   returned; may be shard_final itself
 *   state_out_idx [b]        int32  the accepted index j_b within the shard
 *                                   (as given to the shard's forward); NULL = none
 *   state_out     [b,H,P,N]  fp32   in/out: h0_j on entry, h_j on return;
 *                                   non-NULL exactly when state_out_idx is
 * h_in rounds once to dtype before its product with C (fp32 accumulation).
 * Outputs must not overlap the inputs or each other (final_state ==
 * shard_final excepted).  Same shape limits, alignment rules and errors as
 * ssd_chunk_scan_fwd, and SSD_ERR_UNSUPPORTED unless 64*nheads*headdim and
 * 64*ngroups*dstate elements of dtype, and seqlen*nheads*4 bytes, stay below
 * 2^31 bytes (32-bit offsets within a 64-token block and within dt); no
 * workspace; T = 0 gives final = F + h_in. */
ssd_status ssd_state_correction(void *y, const float *dt, const float *A, const void *C,
                                const float *h_in, const float *shard_final, float *final_state,
                                const int32_t *state_out_idx, float *state_out,
                                const ssd_shape *shape, ssd_dtype dtype, void *hip_stream);

/* ---------------------------------------------------------------------------
 * The operators around the scan in its layer and in its verify loop: the short
 * causal convolution before it, the selective scan with one decay per channel
 * and state index, the gated delta rule, the gated RMS norm after it, the norms
 * and residual stream between blocks, and the verification of drafted tokens
 * that yields the accepted index.  Conventions as above (device
 * pointers, stream order, host-side checks before any launch, no allocation),
 * except that inputs named with a stride below need not be dense: strides are
 * in elements, >= 0 (0 repeats a row), and of no account along a dimension of
 * size 1 or less.  The innermost dimension is always contiguous.  Pointers
 * need the alignment of one element unless said otherwise, and any strides and
 * sizes within the limits are taken.  hip_stream belongs to the current device.
 * These entry points were added to ABI version 8; nothing in it changed.
 * -------------------------------------------------------------------------*/

/* Sizes of ssd_causal_conv_fwd.  batch and seqlen may be 0. */
typedef struct {
    int64_t batch;           /* b: independent sequences                          */
    int64_t seqlen;          /* T: tokens per sequence                            */
    int64_t channels[3];     /* channels of the outputs, in x's order; the first
                                is > 0, the others may be 0 (no such output)      */
    int64_t width;           /* W: taps, 2, 3 or 4                                */
    int64_t x_batch_stride;
    int64_t x_token_stride;
} ssd_conv_shape;

/* Activation codes of ssd_causal_conv_fwd (NONE, SILU) and of
 * ssd_residual_norm_fwd's gate (all). */
typedef enum {
    SSD_ACT_NONE = 0,
    SSD_ACT_SILU = 1,    /* v * sigmoid(v)                               */
    SSD_ACT_SIGMOID = 2  /* 1 / (1 + exp(-v)); of a gate only            */
} ssd_activation;

/* Depthwise causal convolution over tokens, with Ch = the sum of channels:
 *
 *     o[b,t,c] = act(bias[c] + sum_{k<W} weight[c,k] * x[b, t-(W-1)+k, c])
 *
 * where the W-1 tokens before token 0 are init_state (zeros when absent).
 * The outputs are x's channels in up to three dense tensors, so that a
 * projection's rows [... | x | B | C | ...] turn into the dense x, B and C
 * that ssd_chunk_scan_fwd reads (views [b,T,H,P] and [b,T,G,N]).
 *
 *   x             [b,T,Ch]     dtype  strided (a slice of a projection's rows)
 *   weight        [Ch,W]       fp32   the last tap meets the current token
 *   bias          [Ch]         fp32   NULL = none
 *   init_state    [b,W-1,Ch]   dtype  the inputs before token 0, oldest first;
 *                                     NULL = zeros
 *   out0..out2    [b,T,channels[i]]   dtype; NULL exactly where channels[i] is 0
 *                                     (sums in fp32, rounded once)
 *   final_state   [b,W-1,Ch]   dtype  the last W-1 inputs (reaching back into
 *                                     init_state when T < W-1); NULL = not
 *                                     returned; may be init_state itself
 *   state_out_idx [b]          int32  accepted index j_b in [-1, T-1]; NULL = none
 *   state_out     [b,W-1,Ch]   dtype  the W-1 inputs ending at token j_b (-1:
 *                                     init_state); non-NULL exactly when
 *                                     state_out_idx is
 * With a padded batch, j_b = length - 1 gives each sequence's own state.
 * One kernel, no workspace.  batch <= 65535, T < 2^31, Ch <= 2^20. */
ssd_status ssd_causal_conv_fwd(const void *x, const float *weight, const float *bias,
                               const void *init_state, int activation,
                               void *out0, void *out1, void *out2, void *final_state,
                               const int32_t *state_out_idx, void *state_out,
                               const ssd_conv_shape *shape, ssd_dtype dtype, void *hip_stream);

/* Sizes of ssd_selective_scan_fwd.  batch and seqlen may be 0. */
typedef struct {
    int64_t batch;      /* b                                                    */
    int64_t seqlen;     /* T                                                    */
    int64_t channels;   /* Dm: channels, a multiple of ngroups                  */
    int64_t dstate;     /* N: 8, 16, 32 or 64                                   */
    int64_t ngroups;    /* G: B/C groups; channel d reads group d*G/Dm          */
    int64_t u_batch_stride, u_token_stride;
    int64_t delta_batch_stride, delta_token_stride;
    int64_t z_batch_stride, z_token_stride;
    int64_t B_batch_stride, B_token_stride;
    int64_t C_batch_stride, C_token_stride;
} ssd_selective_shape;

/* The selective scan with one decay per channel and state index:
 *
 *     s[b,t,d]   = delta + delta_bias[d], through softplus when delta_softplus
 *     h_t[d][n]  = exp(s * A[d][n]) * h_{t-1}[d][n] + s * u[b,t,d] * B[b,t,g,n]
 *     y[b,t,d]   = (sum_n C[b,t,g,n] * h_t[d][n] + D[d] * u[b,t,d]) * silu(z[b,t,d])
 *
 * with h_{-1} = init_state (zeros when absent); silu(z) is left out without z.
 *
 *   u, delta      [b,T,Dm]    dtype  strided
 *   A             [Dm,N]      fp32   (<= 0; values > 0 are computed as given)
 *   B, C          [b,T,G,N]   dtype  strided by batch and token; a token's G*N
 *                                    values are contiguous
 *   D             [Dm]        fp32   NULL = no skip term
 *   z             [b,T,Dm]    dtype  strided; NULL = no gate
 *   delta_bias    [Dm]        fp32   NULL = none
 *   init_state    [b,Dm,N]    fp32   NULL = zeros
 *   y             [b,T,Dm]    dtype  dense, rounded once from fp32
 *   final_state   [b,Dm,N]    fp32   NULL = not returned; may be init_state itself
 *   state_out_idx [b]         int32  accepted index j_b in [-1, T-1]; NULL = none
 *   state_out     [b,Dm,N]    fp32   the state after token j_b (-1: init_state);
 *                                    non-NULL exactly when state_out_idx is
 *   workspace     16-byte aligned, ssd_selective_scan_workspace_bytes(...) bytes,
 *                 contents on entry ignored; may be NULL when that is 0
 * A and every state are 16-byte aligned.  Calls of few sequences and channels
 * share a long sequence out over the GPU (this needs the workspace); the choice
 * depends on the sizes alone.  batch and ngroups <= 65535, T < 2^31, Dm <= 2^20. */
ssd_status ssd_selective_scan_fwd(const void *u, const void *delta, const float *A,
                                  const void *B, const void *C, const float *D,
                                  const void *z, const float *delta_bias, int delta_softplus,
                                  const float *init_state, void *y, float *final_state,
                                  const int32_t *state_out_idx, float *state_out,
                                  const ssd_selective_shape *shape, ssd_dtype dtype,
                                  void *workspace, size_t workspace_bytes, void *hip_stream);

/* Bytes of workspace ssd_selective_scan_fwd needs; 0 also when the arguments
 * are invalid (ssd_last_error() says why). */
size_t ssd_selective_scan_workspace_bytes(const ssd_selective_shape *shape, ssd_dtype dtype);

/* Sizes of ssd_gated_norm_fwd.  batch and seqlen may be 0. */
typedef struct {
    int64_t batch, seqlen;  /* b, T: one row per token                           */
    int64_t dim;            /* elements per row, a multiple of ngroups           */
    int64_t ngroups;        /* each row is normalised in ngroups equal parts     */
    int64_t x_batch_stride, x_token_stride;
    int64_t z_batch_stride, z_token_stride;
} ssd_norm_shape;

/* RMS norm with a gate, the step between the scan and the output projection:
 *
 *     norm_before_gate == 0:  v = x * silu(z);  out = v / rms(v) * weight
 *     norm_before_gate != 0:  out = x / rms(x) * weight * silu(z)
 *
 * with rms(v) = sqrt(mean(v^2) + eps) over each of the row's ngroups parts
 * (statistics in fp32).  Without z: out = x / rms(x) * weight.
 *
 *   x       [b,T,dim]  dtype  strided
 *   z       [b,T,dim]  dtype  strided; NULL = no gate
 *   weight  [dim]      fp32   NULL = ones
 *   out     [b,T,dim]  dtype  dense; may be x or z itself where that is dense
 *   eps     >= 0 and finite (with 0 a part of zeros gives NaN)
 * One kernel, no workspace.  dim <= 2^20, b*T < 2^31. */
ssd_status ssd_gated_norm_fwd(const void *x, const void *z, const float *weight, void *out,
                              float eps, int norm_before_gate,
                              const ssd_norm_shape *shape, ssd_dtype dtype, void *hip_stream);

/* Sizes of ssd_verify_drafts.  batch and drafts may be 0. */
typedef struct {
    int64_t batch;       /* b: sequences                                         */
    int64_t drafts;      /* K: drafted tokens per sequence (at most)             */
    int64_t vocab;       /* V: probabilities per row                             */
    int64_t target_batch_stride, target_row_stride;
    int64_t draft_batch_stride, draft_row_stride;
} ssd_verify_shape;

/* Verification of drafted tokens against the target's probabilities, by the
 * rejection rule that leaves the target's distribution unchanged.  For each
 * sequence with m = draft_lens[b] drafts (K without draft_lens):
 *
 *     n    = the first i < m with  u_i * q_i(tok_i) >= p_i(tok_i)   (m if none)
 *     r(v) = max(p_n(v) - q_n(v), 0)  for n < m;   p_m(v)  for n = m
 *     next = the smallest v with  r(0) + ... + r(v) > u_K * sum(r)
 *
 * u_i = uniforms[b,i] and u_K = uniforms[b,K] lie in [0,1).  A row need not
 * sum to 1: the last line normalises by r's own sum.  Products and sums are in
 * fp64 in a fixed order, so equal inputs give equal tokens.  Without
 * draft_probs every q_i is 1 at tok_i and 0 elsewhere (looked-up drafts).
 * Where rounding left r without mass, p_n takes its place; a row without mass
 * gives V-1; NaN and negative probabilities count as 0.
 *
 *   target_probs  [b,K+1,V]  dtype  strided; row i judges draft i
 *   draft_probs   [b,K,V]    dtype  strided; NULL = as above
 *   draft_tokens  [b,K]      int32  a token outside [0,V) is never accepted
 *                                   (and takes nothing from p without
 *                                   draft_probs); may be NULL when K is 0
 *   draft_lens    [b]        int32  clamped to [0,K]; NULL = K
 *   uniforms      [b,K+1]    fp32
 *   n_accepted    [b]        int32  n: also the state_out_idx of a scan over
 *                                   [last token, drafts], whose index 0 is the
 *                                   last token that was already accepted
 *   next_token    [b]        int32
 *   tokens        [b,K+1]    int32  the n accepted drafts, next, then -1; NULL =
 *                                   not returned
 *   workspace     16-byte aligned, ssd_verify_workspace_bytes(...) bytes,
 *                 contents on entry ignored; may be NULL when that is 0
 * batch <= 65535, K <= 2^20, V < 2^31. */
ssd_status ssd_verify_drafts(const void *target_probs, const void *draft_probs,
                             const int32_t *draft_tokens, const int32_t *draft_lens,
                             const float *uniforms, int32_t *n_accepted, int32_t *next_token,
                             int32_t *tokens, const ssd_verify_shape *shape, ssd_dtype dtype,
                             void *workspace, size_t workspace_bytes, void *hip_stream);

/* Bytes of workspace ssd_verify_drafts needs; 0 also when the arguments are
 * invalid (ssd_last_error() says why). */
size_t ssd_verify_workspace_bytes(const ssd_verify_shape *shape, ssd_dtype dtype);

/* Sizes of ssd_gated_delta_fwd.  batch and seqlen may be 0. */
typedef struct {
    int64_t batch;     /* b: independent sequences                              */
    int64_t seqlen;    /* T: tokens per sequence                                */
    int64_t nheads;    /* H: heads, a multiple of ngroups                       */
    int64_t headdim;   /* P: values per head, a multiple of 16 up to 256        */
    int64_t dstate;    /* N: size of a key, a multiple of 16 up to 256          */
    int64_t ngroups;   /* G: query/key groups; head h reads group h*G/H         */
    int64_t q_batch_stride, q_token_stride;
    int64_t k_batch_stride, k_token_stride;
    int64_t v_batch_stride, v_token_stride;
    int64_t g_batch_stride, g_token_stride;
    int64_t beta_batch_stride, beta_token_stride;
} ssd_delta_shape;

/* The gated delta rule: a matrix state that forgets by exp(g) and replaces what
 * it holds under a key by beta's share, instead of adding to it as the SSD scan
 * does.  For every sequence, head h (group gr = h*G/H) and token t:
 *
 *     r_t = v[b,t,h,:] - exp(g[b,t,h]) * S_{t-1} k_t           k_t = k[b,t,gr,:]
 *     S_t = exp(g[b,t,h]) * S_{t-1} + beta[b,t,h] * r_t k_t'
 *     y[b,t,h,:] = scale * S_t q_t                             q_t = q[b,t,gr,:]
 *
 * with S_{-1} = init_state (zeros when absent).  With qk_l2norm, q_t and k_t are
 * divided by sqrt(sum of their squares + 1e-6) first.
 *
 *   q, k          [b,T,G,N]  dtype  strided by batch and token; a token's G*N
 *                                   values are contiguous
 *   v             [b,T,H,P]  dtype  strided like them
 *   g             [b,T,H]    fp32   log decays, <= 0 down to -inf (which empties
 *                                   the state; greater ones are computed as given
 *                                   while sums over 32 tokens stay below 80),
 *                                   strided by batch and token; NULL = 0 (no decay)
 *   beta          [b,T,H]    fp32   strided like g
 *   init_state    [b,H,P,N]  fp32   NULL = zeros
 *   y             [b,T,H,P]  dtype  dense, rounded once from fp32
 *   final_state   [b,H,P,N]  fp32   NULL = not returned; may be init_state itself
 *   state_out_idx [b]        int32  accepted index j_b in [-1, T-1]; NULL = none
 *   state_out     [b,H,P,N]  fp32   the state after token j_b (-1: init_state);
 *                                   non-NULL exactly when state_out_idx is
 *   workspace     16-byte aligned, ssd_gated_delta_workspace_bytes(...) bytes,
 *                 contents on entry ignored; may be NULL when that is 0
 * States are fp32 throughout and 16-byte aligned.  Values but those of g are
 * finite, and so are in fp32 the squares of q's and k's norms and the states that
 * the rule makes, padding tokens included: a chunk's products read all of its
 * tokens.  Keys of norm above sqrt(2 / beta) make the rule itself grow.  A few
 * tokens run token by token, prompts in chunks (this needs the workspace); the
 * choice depends on the sizes and dtype alone.  With a
 * padded batch, j_b = length - 1 gives each sequence's own state.
 * batch, nheads <= 65535, T < 2^31, batch * nheads * ceil(P / 32) < 2^24,
 * batch * nheads * ceil(T / 32) < 2^26. */
ssd_status ssd_gated_delta_fwd(const void *q, const void *k, const void *v, const float *g,
                               const float *beta, float scale, int qk_l2norm,
                               const float *init_state, void *y, float *final_state,
                               const int32_t *state_out_idx, float *state_out,
                               const ssd_delta_shape *shape, ssd_dtype dtype,
                               void *workspace, size_t workspace_bytes, void *hip_stream);

/* Bytes of workspace ssd_gated_delta_fwd needs; 0 also when the arguments are
 * invalid (ssd_last_error() says why). */
size_t ssd_gated_delta_workspace_bytes(const ssd_delta_shape *shape, ssd_dtype dtype);

/* Sizes of ssd_residual_norm_fwd.  batch and seqlen may be 0. */
typedef struct {
    int64_t batch, seqlen;  /* b, T: one row per token                           */
    int64_t dim;            /* elements per row                                  */
    int64_t x_batch_stride, x_token_stride;
    int64_t residual_batch_stride, residual_token_stride;
    int64_t gate_batch_stride, gate_token_stride;  /* token stride 0: one gate per sequence */
} ssd_residual_norm_shape;

/* What stands between two blocks: the norm after a block, its gate and scale,
 * the residual stream, and the norm before the next block:
 *
 *     n   = post_norm ? x / rms(x) * post_weight : x
 *     h   = residual_scale * residual + branch_scale * layer_scale * act(gate) * n
 *     out = h / rms(h) * weight
 *
 * with rms(v) = sqrt(mean(v^2) + eps) over the row; everything in fp32, h
 * rounded once where it is stored (out comes from h before that rounding).
 * What is absent is left out.
 *
 *   x            [b,T,dim]  dtype         the block's output, strided
 *   residual     [b,T,dim]  stream_dtype  strided; NULL = none (h is the branch)
 *   gate         [b,T,dim]  dtype         strided; NULL = none
 *   gate_activation         SSD_ACT_*     of the gate
 *   post_weight  [dim]      fp32          NULL = ones; only with post_norm
 *   layer_scale  [dim]      fp32          NULL = ones
 *   weight       [dim]      fp32          NULL = ones
 *   out          [b,T,dim]  dtype         dense; may be x itself where that is dense
 *   residual_out [b,T,dim]  stream_dtype  h, dense; NULL = not returned; may be
 *                                         residual itself where that is dense
 *   eps                     >= 0 and finite (with 0 a row of zeros gives NaN)
 * stream_dtype is dtype or fp32.  One kernel, no workspace.  dim <= 2^20,
 * b*T < 2^31. */
ssd_status ssd_residual_norm_fwd(const void *x, const void *residual, const void *gate,
                                 int gate_activation, int post_norm, const float *post_weight,
                                 const float *layer_scale, float residual_scale,
                                 float branch_scale, const float *weight, float eps, void *out,
                                 void *residual_out, const ssd_residual_norm_shape *shape,
                                 ssd_dtype dtype, ssd_dtype stream_dtype, void *hip_stream);

/* Static description of a status code. */
const char *ssd_status_string(ssd_status status);

/* Detail for the last non-OK return on the calling thread ("" if none). */
const char *ssd_last_error(void);

/* SSD_ABI_VERSION of the built library. */
int ssd_abi_version(void);

#ifdef __cplusplus
}
#endif

#endif /* SSD_H */
