// Internal interface between the host orchestrator (ssd_api.hip) and the
// kernels.  Not installed; the public boundary is include/ssd.h.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace ssd {

enum class Elem { F32, BF16 };

// Everything a kernel needs, passed by value.  Pointers are device pointers
// with the layouts documented in include/ssd.h; `cs` and `states` point into
// the caller's workspace.
struct Params {
    const void *x;            // [b,T,H,P]  T_elem
    const float *dt;          // [b,T,H]
    const float *A;           // [H]
    const void *B;            // [b,T,G,N]  T_elem
    const void *C;            // [b,T,G,N]  T_elem
    const float *D;           // [H] or null
    const float *init_state;  // [b,H,P,N] or null
    const int32_t *state_out_idx;  // [b] or null
    void *y;                  // [b,T,H,P]  T_elem
    float *final_state;       // [b,H,P,N] or null
    float *state_out;         // [b,H,P,N] or null
    float *cs;                // workspace [b,H,nc,Q]: chunk-local cumulative log-decay
    float *ct;                // workspace [b,H,nc,Q]: cs * log2(e) - log2(dt) (+inf past the end)
    float *dte;               // workspace [b,H,nc,Q]: dt_i * exp(cs_e - cs_i), e = last token of i's 32-token block
    void *states;             // workspace [b,nc,H,P,N] T_elem: chunk states S_c (from a zero start),
                              // rounded once to the input type
    void *prev;               // workspace [b,nc,H,P,N] T_elem: state entering each chunk (chunk 0 only with init_state)
    float *hj;                // workspace [b,H,P,N] fp32: state entering the chunk of state_out_idx[b]
    const float *shard_final; // [b,H,P,N] fp32: a shard's final state from a zero start (state correction only)
    int64_t batch, seqlen;
    int nheads, headdim, dstate, ngroups, chunk, nchunks;
    int heads_per_group;
    int no_split;             // single pass: run every item whole on one workgroup (in-place calls)
};

// Each launcher enqueues one kernel on `stream` and returns hipGetLastError().
hipError_t launch_chunk_cumsum(const Params &p, hipStream_t stream);
hipError_t launch_chunk_state(const Params &p, Elem e, hipStream_t stream);
// Head-batched bf16 chunk states; returns hipErrorNotSupported when the shape
// does not fit its LDS budget or wave split (the caller then uses launch_chunk_state).
hipError_t launch_chunk_state_heads(const Params &p, hipStream_t stream);
hipError_t launch_state_pass(const Params &p, Elem e, hipStream_t stream);
hipError_t launch_chunk_output(const Params &p, Elem e, hipStream_t stream);
// Head-batched bf16 chunk outputs; returns hipErrorNotSupported when the
// shape does not fit its LDS budget (the caller then uses launch_chunk_output).
hipError_t launch_chunk_output_heads(const Params &p, hipStream_t stream);
hipError_t launch_state_at_index(const Params &p, Elem e, hipStream_t stream);
// Single-pass bf16 forward: one kernel for the whole call (its own
// chunk-local tables from dt and A; y, final_state and state_out written
// directly; the workspace is not used).  A grid of two workgroups per
// compute unit in which one workgroup at a time runs an item ((b, h), or a
// 64-channel half of a head of headdim 128), or a range of its blocks, in
// order with the state in registers.  chunk_scan_fused_takes says whether
// it takes a call; launch_chunk_scan_fused returns hipErrorNotSupported for
// calls it does not take.
constexpr int64_t kFusedMinItems = 64;
bool chunk_scan_fused_takes(const Params &p);
hipError_t launch_chunk_scan_fused(const Params &p, hipStream_t stream);
// Whole forward of a one-chunk call of at most 32 tokens in one kernel (y,
// final_state, state_out; the workspace is not used).  one_chunk_takes says
// whether it takes a call; launch_one_chunk returns hipErrorNotSupported for
// calls it does not take.
bool one_chunk_takes(const Params &p);
hipError_t launch_one_chunk(const Params &p, Elem e, hipStream_t stream);
hipError_t launch_empty_sequence(const Params &p, hipStream_t stream);
// Sequence-shard correction: y += exp(cs_t) C_t . init_state over the whole
// shard (cs from the shard's first token), final_state = shard_final +
// exp(cs_{T-1}) init_state, state_out += exp(cs_j) init_state.  Reads
// init_state (the state entering the shard), dt, A, C, shard_final and
// state_out_idx; updates y and state_out in place.
hipError_t launch_state_correction(const Params &p, Elem e, hipStream_t stream);

// ------------------------------------------------- operators around the scan
// Short causal convolution (ssd_causal_conv_fwd); pointers and strides as in
// include/ssd.h.
struct ConvParams {
    const void *x;             // [b,T,Ch] strided
    const float *weight;       // [Ch,W]
    const float *bias;         // [Ch] or null
    const void *init_state;    // [b,W-1,Ch] or null
    void *out[3];              // [b,T,channels[i]]
    void *final_state;         // [b,W-1,Ch] or null
    const int32_t *state_out_idx;
    void *state_out;           // [b,W-1,Ch] or null
    int64_t batch, seqlen;
    int64_t x_bs, x_ts;        // batch and token stride
    int channels[3], total;    // outputs' channels and their sum
    int width;
    int silu;
};
hipError_t launch_causal_conv(const ConvParams &p, Elem e, hipStream_t stream);

// Selective scan with one decay per channel and state index
// (ssd_selective_scan_fwd).
struct SelectiveParams {
    const void *u, *delta, *B, *C, *z;  // strided; z may be null
    const float *A;                     // [D,N]
    const float *D, *delta_bias;        // [D] or null
    const float *init_state;            // [b,D,N] or null
    void *y;                            // [b,T,D]
    float *final_state;                 // [b,D,N] or null
    const int32_t *state_out_idx;
    float *state_out;                   // [b,D,N] or null
    int64_t batch, seqlen;
    int64_t u_bs, u_ts, delta_bs, delta_ts, z_bs, z_ts, B_bs, B_ts, C_bs, C_ts;
    int channels, dstate, ngroups;
    int group_channels;                 // channels / ngroups
    int softplus;
    // Token ranges (selective_ranges): with more than one, the workspace holds
    // each range's final state [ranges][b,D,N] (the last slot: a copy of
    // init_state) and sum of steps [ranges][b,D].
    int ranges;
    int64_t range_len;                  // a multiple of the kernel's tile
    float *range_state, *range_steps;
};
// Chooses ranges and range_len from the sizes.
void selective_ranges(SelectiveParams &p);
hipError_t launch_selective_scan(const SelectiveParams &p, Elem e, hipStream_t stream);

// Gated RMS norm (ssd_gated_norm_fwd).
struct NormParams {
    const void *x, *z;         // [b,T,dim] strided; z may be null
    const float *weight;       // [dim] or null
    void *out;                 // [b,T,dim]
    int64_t rows, seqlen;      // rows = b * T
    int64_t x_bs, x_ts, z_bs, z_ts;
    int dim, ngroups, group_dim;
    float eps;
    int norm_before_gate;
};
hipError_t launch_gated_norm(const NormParams &p, Elem e, hipStream_t stream);

// Gated delta rule (ssd_gated_delta_fwd).
struct DeltaParams {
    const void *q, *k, *v;      // strided
    const float *g, *beta;      // strided; g may be null
    const float *init_state;    // [b,H,P,N] or null
    void *y;                    // [b,T,H,P]
    float *final_state;         // [b,H,P,N] or null
    const int32_t *state_out_idx;
    float *state_out;           // [b,H,P,N] or null
    int64_t batch, seqlen;
    int64_t q_bs, q_ts, k_bs, k_ts, v_bs, v_ts, g_bs, g_ts, beta_bs, beta_ts;
    int nheads, headdim, dstate, ngroups, heads_per_group;
    float scale;
    int l2norm;
    // Chunked form only, in the workspace: delta_pack_bytes per (b, chunk, h) and
    // delta_at_bytes per (b, h).
    int64_t nchunks;
    int prepare_heads;  // heads of a group per wave of the preparation
    char *pack;
    float *at_tables;
    // Ranges of chunks (delta_ranges); with more than one, the workspace holds
    // [ranges - 1][b,H,P,N] states, [ranges - 2][b,H,N,N] maps and a copy of
    // init_state.
    int ranges;
    int64_t range_chunks;
    float *range_state, *range_map, *range_init;
};
// Chooses ranges and range_chunks from the sizes.
void delta_ranges(DeltaParams &p, Elem e);
constexpr int kDeltaChunk = 32;  // tokens of a chunk
// Token by token (any number of them), and in chunks with the workspace.
hipError_t launch_delta_tokens(const DeltaParams &p, Elem e, hipStream_t stream);
hipError_t launch_delta_chunks(const DeltaParams &p, Elem e, hipStream_t stream);
size_t delta_pack_bytes(Elem e);
size_t delta_at_bytes();

// Norms before and after a block (ssd_residual_norm_fwd).
struct ResidualNormParams {
    const void *x, *residual, *gate;  // strided; residual and gate may be null
    const float *post_weight, *layer_scale, *weight;  // [dim] or null
    void *out;                        // [b,T,dim]
    void *residual_out;               // [b,T,dim] or null
    int64_t rows, seqlen;             // rows = b * T
    int64_t x_bs, x_ts, r_bs, r_ts, gate_bs, gate_ts;
    int dim;
    int activation, post_norm;
    float residual_scale, branch_scale, eps;
};
hipError_t launch_residual_norm(const ResidualNormParams &p, Elem e, Elem stream_elem, hipStream_t stream);

// Verification of drafted tokens (ssd_verify_drafts).
struct VerifyParams {
    const void *target, *draft;  // strided; draft may be null
    const int32_t *tok;          // [b,K] or null when K is 0
    const int32_t *lens;         // [b] or null
    const float *u;              // [b,K+1]
    int32_t *n_accepted, *next_token, *tokens;  // tokens may be null
    int64_t batch, vocab;
    int64_t t_bs, t_rs, d_bs, d_rs;
    int drafts;
    // Segments of a row summed by the first of two launches (verify_segments);
    // 1: one launch.
    int segments;
    int64_t segment;             // elements per segment
    double *sums;                // [b,segments] in the workspace
};
// Chooses segments and segment from the sizes.
void verify_segments(VerifyParams &p);
hipError_t launch_verify_drafts(const VerifyParams &p, Elem e, hipStream_t stream);

}  // namespace ssd
