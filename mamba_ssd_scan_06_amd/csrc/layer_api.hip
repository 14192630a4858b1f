// Host side of the operators around the scan: argument checks and launches of
// ssd_causal_conv_fwd, ssd_selective_scan_fwd, ssd_gated_norm_fwd and
// ssd_verify_drafts.  The public contract is include/ssd.h.
#include <math.h>

#include "host_common.hpp"
#include "kernels.hpp"
#include "ssd.h"

namespace {

using ssd::extent3;
using ssd::fail;
using ssd::overlaps;
using ssd::product;
using ssd::Range;
using ssd::range;

constexpr int64_t kMaxBatch = 65535;             // a grid dimension
constexpr int64_t kMaxTokens = (int64_t)1 << 31;  // token indices fit 32 bits
constexpr int64_t kMaxWide = (int64_t)1 << 20;    // channels, norm dims

size_t elem_size(ssd_dtype dtype) { return dtype == SSD_DTYPE_BF16 ? 2 : 4; }
ssd::Elem elem(ssd_dtype dtype) { return dtype == SSD_DTYPE_BF16 ? ssd::Elem::BF16 : ssd::Elem::F32; }

ssd_status check_dtype(ssd_dtype dtype) {
    if (dtype != SSD_DTYPE_F32 && dtype != SSD_DTYPE_BF16) return fail(SSD_ERR_ARGS, "unknown dtype %d", (int)dtype);
    return SSD_OK;
}

struct Ptr {
    const char *name;
    const void *p;
    size_t align;
};

template <int K>
ssd_status check_align(const Ptr (&ptrs)[K]) {
    for (const Ptr &q : ptrs)
        if ((uintptr_t)q.p % q.align != 0) return fail(SSD_ERR_ALIGN, "%s is not %zu-byte aligned", q.name, q.align);
    return SSD_OK;
}

// An output that may be one of the inputs itself (an in-place update).
struct InPlace {
    int out, in;
};

// No output may overlap an input or another output, except the allowed pairs
// of identical pointers.
template <int NO, int NI, int NA>
ssd_status check_alias(const Range (&outs)[NO], const Range (&ins)[NI], const InPlace (&allowed)[NA]) {
    for (int i = 0; i < NO; ++i) {
        for (int k = 0; k < NI; ++k) {
            bool same = false;
            for (const InPlace &a : allowed)
                same = same || (a.out == i && a.in == k && outs[i].lo == ins[k].lo && outs[i].hi == ins[k].hi);
            if (!same && overlaps(outs[i], ins[k]))
                return fail(SSD_ERR_ALIAS, "%s overlaps %s", outs[i].name, ins[k].name);
        }
        for (int k = i + 1; k < NO; ++k)
            if (overlaps(outs[i], outs[k])) return fail(SSD_ERR_ALIAS, "%s overlaps %s", outs[i].name, outs[k].name);
    }
    return SSD_OK;
}

// A stride of a dimension without a second index is never used: 0 keeps it
// out of the offsets.
int64_t used_stride(int64_t n, int64_t stride) { return n > 1 ? stride : 0; }

ssd_status launched(const char *what, hipError_t r) {
    if (r != hipSuccess) return fail(SSD_ERR_HIP, "%s launch failed: %s", what, hipGetErrorString(r));
    return SSD_OK;
}

ssd_status check_selective(const ssd_selective_shape *s, ssd_dtype dtype) {
    if (!s) return fail(SSD_ERR_NULL, "shape is NULL");
    ssd_status st = check_dtype(dtype);
    if (st != SSD_OK) return st;
    if (s->batch < 0 || s->seqlen < 0) return fail(SSD_ERR_SHAPE, "batch and seqlen must be >= 0");
    if (s->channels <= 0 || s->dstate <= 0 || s->ngroups <= 0)
        return fail(SSD_ERR_SHAPE, "channels, dstate and ngroups must be > 0");
    if (s->channels % s->ngroups != 0)
        return fail(SSD_ERR_SHAPE, "ngroups (%lld) must divide channels (%lld)", (long long)s->ngroups,
                    (long long)s->channels);
    if (s->dstate != 8 && s->dstate != 16 && s->dstate != 32 && s->dstate != 64)
        return fail(SSD_ERR_UNSUPPORTED, "dstate %lld not in {8, 16, 32, 64}", (long long)s->dstate);
    if (s->batch > kMaxBatch || s->seqlen >= kMaxTokens || s->channels > kMaxWide || s->ngroups > kMaxBatch)
        return fail(SSD_ERR_UNSUPPORTED, "problem too large (batch and ngroups <= 65535, seqlen < 2^31, "
                                         "channels <= 2^20)");
    return SSD_OK;
}

ssd::SelectiveParams selective_params(const ssd_selective_shape *s) {
    ssd::SelectiveParams p = {};
    p.batch = s->batch;
    p.seqlen = s->seqlen;
    p.channels = (int)s->channels;
    p.dstate = (int)s->dstate;
    p.ngroups = (int)s->ngroups;
    p.group_channels = (int)(s->channels / s->ngroups);
    p.u_bs = used_stride(s->batch, s->u_batch_stride);
    p.u_ts = used_stride(s->seqlen, s->u_token_stride);
    p.delta_bs = used_stride(s->batch, s->delta_batch_stride);
    p.delta_ts = used_stride(s->seqlen, s->delta_token_stride);
    p.z_bs = used_stride(s->batch, s->z_batch_stride);
    p.z_ts = used_stride(s->seqlen, s->z_token_stride);
    p.B_bs = used_stride(s->batch, s->B_batch_stride);
    p.B_ts = used_stride(s->seqlen, s->B_token_stride);
    p.C_bs = used_stride(s->batch, s->C_batch_stride);
    p.C_ts = used_stride(s->seqlen, s->C_token_stride);
    return p;
}

// Byte offsets of the range states and sums of steps in the workspace.
struct SelectiveWorkspace {
    size_t steps_off, total;
};
SelectiveWorkspace selective_workspace(const ssd::SelectiveParams &p) {
    if (p.ranges <= 1) return {0, 0};
    const size_t n = (size_t)p.ranges * p.batch * p.channels;
    const size_t states = (n * p.dstate * sizeof(float) + 255) / 256 * 256;
    return {states, states + n * sizeof(float)};
}

ssd_status check_verify(const ssd_verify_shape *s, ssd_dtype dtype) {
    if (!s) return fail(SSD_ERR_NULL, "shape is NULL");
    ssd_status st = check_dtype(dtype);
    if (st != SSD_OK) return st;
    if (s->batch < 0 || s->drafts < 0) return fail(SSD_ERR_SHAPE, "batch and drafts must be >= 0");
    if (s->vocab <= 0) return fail(SSD_ERR_SHAPE, "vocab must be > 0");
    if (s->batch > kMaxBatch || s->drafts > kMaxWide || s->vocab >= ((int64_t)1 << 31))
        return fail(SSD_ERR_UNSUPPORTED, "problem too large (batch <= 65535, drafts <= 2^20, vocab < 2^31)");
    return SSD_OK;
}

ssd::VerifyParams verify_params(const ssd_verify_shape *s) {
    ssd::VerifyParams p = {};
    p.batch = s->batch;
    p.vocab = s->vocab;
    p.t_bs = used_stride(s->batch, s->target_batch_stride);
    p.t_rs = used_stride(s->drafts + 1, s->target_row_stride);
    p.d_bs = used_stride(s->batch, s->draft_batch_stride);
    p.d_rs = used_stride(s->drafts, s->draft_row_stride);
    p.drafts = (int)s->drafts;
    ssd::verify_segments(p);
    return p;
}

size_t verify_workspace(const ssd::VerifyParams &p) {
    return p.segments > 1 ? (size_t)p.batch * p.segments * sizeof(double) : 0;
}

}  // namespace

extern "C" {

ssd_status ssd_causal_conv_fwd(const void *x, const float *weight, const float *bias, const void *init_state,
                               int activation, void *out0, void *out1, void *out2, void *final_state,
                               const int32_t *state_out_idx, void *state_out, const ssd_conv_shape *s,
                               ssd_dtype dtype, void *hip_stream) {
    if (!s) return fail(SSD_ERR_NULL, "shape is NULL");
    ssd_status st = check_dtype(dtype);
    if (st != SSD_OK) return st;
    if (activation != SSD_ACT_NONE && activation != SSD_ACT_SILU)
        return fail(SSD_ERR_ARGS, "unknown activation %d", activation);
    if (s->batch < 0 || s->seqlen < 0) return fail(SSD_ERR_SHAPE, "batch and seqlen must be >= 0");
    if (s->channels[0] <= 0 || s->channels[1] < 0 || s->channels[2] < 0)
        return fail(SSD_ERR_SHAPE, "channels[0] must be > 0, channels[1] and channels[2] >= 0");
    if (s->width < 2 || s->width > 4)
        return fail(SSD_ERR_UNSUPPORTED, "width %lld not in {2, 3, 4}", (long long)s->width);
    const int64_t b = s->batch, T = s->seqlen, held = s->width - 1;
    if (s->channels[0] > kMaxWide || s->channels[1] > kMaxWide || s->channels[2] > kMaxWide)
        return fail(SSD_ERR_UNSUPPORTED, "more than 2^20 channels");
    const int64_t Ch = s->channels[0] + s->channels[1] + s->channels[2];
    if (b > kMaxBatch || T >= kMaxTokens || Ch > kMaxWide)
        return fail(SSD_ERR_UNSUPPORTED, "problem too large (batch <= 65535, seqlen < 2^31, 2^20 channels)");
    const int64_t x_n = extent3(b, s->x_batch_stride, T, s->x_token_stride, Ch), out_n = product(b, T, Ch),
                  st_n = product(b, held, Ch);
    if (x_n < 0 || out_n < 0 || st_n < 0) return fail(SSD_ERR_SHAPE, "a stride is negative or the problem too large");
    if ((state_out == nullptr) != (state_out_idx == nullptr))
        return fail(SSD_ERR_ARGS, "state_out and state_out_idx must be given together");
    void *const outs[] = {out0, out1, out2};
    if (b > 0 && !weight) return fail(SSD_ERR_NULL, "weight is required");
    if (b > 0 && T > 0) {
        if (!x) return fail(SSD_ERR_NULL, "x is required");
        for (int i = 0; i < 3; ++i)
            if ((outs[i] == nullptr) != (s->channels[i] == 0))
                return fail(SSD_ERR_NULL, "out%d must be given exactly when channels[%d] is not 0", i, i);
    }
    const size_t e = elem_size(dtype);
    const Ptr ptrs[] = {{"x", x, e}, {"weight", weight, 4}, {"bias", bias, 4}, {"init_state", init_state, e},
                        {"out0", out0, e}, {"out1", out1, e}, {"out2", out2, e}, {"final_state", final_state, e},
                        {"state_out_idx", state_out_idx, 4}, {"state_out", state_out, e}};
    if ((st = check_align(ptrs)) != SSD_OK) return st;
    const Range o[] = {range("out0", out0, e * b * T * s->channels[0]), range("out1", out1, e * b * T * s->channels[1]),
                       range("out2", out2, e * b * T * s->channels[2]), range("final_state", final_state, e * st_n),
                       range("state_out", state_out, e * st_n)};
    const Range in[] = {range("x", x, e * x_n), range("weight", weight, 4 * Ch * s->width),
                        range("bias", bias, 4 * Ch), range("init_state", init_state, e * st_n),
                        range("state_out_idx", state_out_idx, 4 * b)};
    const InPlace allowed[] = {{3, 3}};  // final_state == init_state
    if ((st = check_alias(o, in, allowed)) != SSD_OK) return st;
    if (b == 0 || (T == 0 && !final_state && !state_out)) return SSD_OK;  // nothing to enqueue

    ssd::ConvParams p = {};
    p.x = x;
    p.weight = weight;
    p.bias = bias;
    p.init_state = init_state;
    for (int i = 0; i < 3; ++i) {
        p.out[i] = outs[i];
        p.channels[i] = (int)s->channels[i];
    }
    p.final_state = final_state;
    p.state_out_idx = state_out_idx;
    p.state_out = state_out;
    p.batch = b;
    p.seqlen = T;
    p.x_bs = used_stride(b, s->x_batch_stride);
    p.x_ts = used_stride(T, s->x_token_stride);
    p.total = (int)Ch;
    p.width = (int)s->width;
    p.silu = activation == SSD_ACT_SILU;
    (void)hipGetLastError();  // start from a clean error state
    return launched("causal_conv", ssd::launch_causal_conv(p, elem(dtype), static_cast<hipStream_t>(hip_stream)));
}

size_t ssd_selective_scan_workspace_bytes(const ssd_selective_shape *shape, ssd_dtype dtype) {
    if (check_selective(shape, dtype) != SSD_OK) return 0;
    ssd::SelectiveParams p = selective_params(shape);
    ssd::selective_ranges(p);
    return selective_workspace(p).total;
}

ssd_status ssd_selective_scan_fwd(const void *u, const void *delta, const float *A, const void *B, const void *C,
                                  const float *D, const void *z, const float *delta_bias, int delta_softplus,
                                  const float *init_state, void *y, float *final_state,
                                  const int32_t *state_out_idx, float *state_out, const ssd_selective_shape *s,
                                  ssd_dtype dtype, void *workspace, size_t workspace_bytes, void *hip_stream) {
    ssd_status st = check_selective(s, dtype);
    if (st != SSD_OK) return st;
    const int64_t b = s->batch, T = s->seqlen, Dm = s->channels, N = s->dstate, GN = s->ngroups * N;
    const int64_t u_n = extent3(b, s->u_batch_stride, T, s->u_token_stride, Dm),
                  dl_n = extent3(b, s->delta_batch_stride, T, s->delta_token_stride, Dm),
                  z_n = z ? extent3(b, s->z_batch_stride, T, s->z_token_stride, Dm) : 0,
                  B_n = extent3(b, s->B_batch_stride, T, s->B_token_stride, GN),
                  C_n = extent3(b, s->C_batch_stride, T, s->C_token_stride, GN), y_n = product(b, T, Dm),
                  st_n = product(b, Dm, N);
    if (u_n < 0 || dl_n < 0 || z_n < 0 || B_n < 0 || C_n < 0 || y_n < 0 || st_n < 0)
        return fail(SSD_ERR_SHAPE, "a stride is negative or the problem too large");
    if ((state_out == nullptr) != (state_out_idx == nullptr))
        return fail(SSD_ERR_ARGS, "state_out and state_out_idx must be given together");
    if (b > 0 && T > 0 && (!u || !delta || !A || !B || !C || !y))
        return fail(SSD_ERR_NULL, "u, delta, A, B, C and y are required");
    ssd::SelectiveParams p = selective_params(s);
    ssd::selective_ranges(p);
    const SelectiveWorkspace ws = selective_workspace(p);
    const size_t ws_need = ws.total;
    if (ws_need > 0 && !workspace) return fail(SSD_ERR_WORKSPACE, "workspace is NULL");
    if (workspace_bytes < ws_need)
        return fail(SSD_ERR_WORKSPACE, "workspace has %zu bytes, needs %zu", workspace_bytes, ws_need);
    const size_t e = elem_size(dtype);
    const Ptr ptrs[] = {{"u", u, e}, {"delta", delta, e}, {"A", A, 16}, {"B", B, e}, {"C", C, e}, {"D", D, 4},
                        {"z", z, e}, {"delta_bias", delta_bias, 4}, {"init_state", init_state, 16}, {"y", y, e},
                        {"final_state", final_state, 16}, {"state_out_idx", state_out_idx, 4},
                        {"state_out", state_out, 16}, {"workspace", workspace, 16}};
    if ((st = check_align(ptrs)) != SSD_OK) return st;
    const Range o[] = {range("y", y, e * y_n), range("final_state", final_state, 4 * st_n),
                       range("state_out", state_out, 4 * st_n), range("workspace", workspace, ws_need)};
    const Range in[] = {range("u", u, e * u_n), range("delta", delta, e * dl_n), range("A", A, 4 * Dm * N),
                        range("B", B, e * B_n), range("C", C, e * C_n), range("D", D, 4 * Dm),
                        range("z", z, e * z_n), range("delta_bias", delta_bias, 4 * Dm),
                        range("init_state", init_state, 4 * st_n), range("state_out_idx", state_out_idx, 4 * b)};
    const InPlace allowed[] = {{1, 8}};  // final_state == init_state
    if ((st = check_alias(o, in, allowed)) != SSD_OK) return st;
    if (b == 0 || (T == 0 && !final_state && !state_out)) return SSD_OK;  // nothing to enqueue

    p.u = u;
    p.delta = delta;
    p.A = A;
    p.B = B;
    p.C = C;
    p.D = D;
    p.z = z;
    p.delta_bias = delta_bias;
    p.softplus = delta_softplus != 0;
    if (ws_need > 0) {
        p.range_state = static_cast<float *>(workspace);
        p.range_steps = reinterpret_cast<float *>(static_cast<char *>(workspace) + ws.steps_off);
    }
    p.init_state = init_state;
    p.y = y;
    p.final_state = final_state;
    p.state_out_idx = state_out_idx;
    p.state_out = state_out;
    (void)hipGetLastError();  // start from a clean error state
    return launched("selective_scan", ssd::launch_selective_scan(p, elem(dtype), static_cast<hipStream_t>(hip_stream)));
}

ssd_status ssd_gated_norm_fwd(const void *x, const void *z, const float *weight, void *out, float eps,
                              int norm_before_gate, const ssd_norm_shape *s, ssd_dtype dtype, void *hip_stream) {
    if (!s) return fail(SSD_ERR_NULL, "shape is NULL");
    ssd_status st = check_dtype(dtype);
    if (st != SSD_OK) return st;
    if (s->batch < 0 || s->seqlen < 0) return fail(SSD_ERR_SHAPE, "batch and seqlen must be >= 0");
    if (s->dim <= 0 || s->ngroups <= 0 || s->dim % s->ngroups != 0)
        return fail(SSD_ERR_SHAPE, "dim (%lld) must be a positive multiple of ngroups (%lld)", (long long)s->dim,
                    (long long)s->ngroups);
    const int64_t rows = product(s->batch, s->seqlen);
    if (s->dim > kMaxWide || rows < 0 || rows >= kMaxTokens)
        return fail(SSD_ERR_UNSUPPORTED, "problem too large (dim <= 2^20, batch * seqlen < 2^31)");
    if (!(eps >= 0.0f) || isinf(eps)) return fail(SSD_ERR_ARGS, "eps must be finite and >= 0");
    const int64_t x_n = extent3(s->batch, s->x_batch_stride, s->seqlen, s->x_token_stride, s->dim),
                  z_n = z ? extent3(s->batch, s->z_batch_stride, s->seqlen, s->z_token_stride, s->dim) : 0,
                  out_n = product(rows, s->dim);
    if (x_n < 0 || z_n < 0 || out_n < 0) return fail(SSD_ERR_SHAPE, "a stride is negative or the problem too large");
    if (rows > 0 && (!x || !out)) return fail(SSD_ERR_NULL, "x and out are required");
    const size_t e = elem_size(dtype);
    const Ptr ptrs[] = {{"x", x, e}, {"z", z, e}, {"weight", weight, 4}, {"out", out, e}};
    if ((st = check_align(ptrs)) != SSD_OK) return st;
    // In place only where out's rows are the input's own.
    auto dense = [&](int64_t bs, int64_t ts) {
        return (s->seqlen == 1 || ts == s->dim) && (s->batch == 1 || bs == s->seqlen * s->dim);
    };
    const Range o[] = {range("out", out, e * out_n)};
    const Range in[] = {range("x", x, e * x_n), range("z", z, e * z_n), range("weight", weight, 4 * s->dim)};
    const InPlace allowed[] = {{dense(s->x_batch_stride, s->x_token_stride) ? 0 : -1, 0},
                               {dense(s->z_batch_stride, s->z_token_stride) ? 0 : -1, 1}};
    if ((st = check_alias(o, in, allowed)) != SSD_OK) return st;
    if (rows == 0) return SSD_OK;  // nothing to enqueue

    ssd::NormParams p = {};
    p.x = x;
    p.z = z;
    p.weight = weight;
    p.out = out;
    p.rows = rows;
    p.seqlen = s->seqlen;
    p.x_bs = used_stride(s->batch, s->x_batch_stride);
    p.x_ts = used_stride(s->seqlen, s->x_token_stride);
    p.z_bs = used_stride(s->batch, s->z_batch_stride);
    p.z_ts = used_stride(s->seqlen, s->z_token_stride);
    p.dim = (int)s->dim;
    p.ngroups = (int)s->ngroups;
    p.group_dim = (int)(s->dim / s->ngroups);
    p.eps = eps;
    p.norm_before_gate = norm_before_gate != 0;
    (void)hipGetLastError();  // start from a clean error state
    return launched("gated_norm", ssd::launch_gated_norm(p, elem(dtype), static_cast<hipStream_t>(hip_stream)));
}

size_t ssd_verify_workspace_bytes(const ssd_verify_shape *shape, ssd_dtype dtype) {
    if (check_verify(shape, dtype) != SSD_OK) return 0;
    return verify_workspace(verify_params(shape));
}

ssd_status ssd_verify_drafts(const void *target_probs, const void *draft_probs, const int32_t *draft_tokens,
                             const int32_t *draft_lens, const float *uniforms, int32_t *n_accepted,
                             int32_t *next_token, int32_t *tokens, const ssd_verify_shape *s, ssd_dtype dtype,
                             void *workspace, size_t workspace_bytes, void *hip_stream) {
    ssd_status st = check_verify(s, dtype);
    if (st != SSD_OK) return st;
    const int64_t b = s->batch, K = s->drafts, V = s->vocab;
    const int64_t t_n = extent3(b, s->target_batch_stride, K + 1, s->target_row_stride, V),
                  d_n = draft_probs ? extent3(b, s->draft_batch_stride, K, s->draft_row_stride, V) : 0;
    if (t_n < 0 || d_n < 0) return fail(SSD_ERR_SHAPE, "a stride is negative or the problem too large");
    if (b > 0 && (!target_probs || !uniforms || !n_accepted || !next_token))
        return fail(SSD_ERR_NULL, "target_probs, uniforms, n_accepted and next_token are required");
    if (b > 0 && K > 0 && !draft_tokens) return fail(SSD_ERR_NULL, "draft_tokens is required");
    ssd::VerifyParams p = verify_params(s);
    const size_t ws_need = verify_workspace(p);
    if (ws_need > 0 && !workspace) return fail(SSD_ERR_WORKSPACE, "workspace is NULL");
    if (workspace_bytes < ws_need)
        return fail(SSD_ERR_WORKSPACE, "workspace has %zu bytes, needs %zu", workspace_bytes, ws_need);
    const size_t e = elem_size(dtype);
    const Ptr ptrs[] = {{"target_probs", target_probs, e}, {"draft_probs", draft_probs, e},
                        {"draft_tokens", draft_tokens, 4}, {"draft_lens", draft_lens, 4}, {"uniforms", uniforms, 4},
                        {"n_accepted", n_accepted, 4}, {"next_token", next_token, 4}, {"tokens", tokens, 4},
                        {"workspace", workspace, 16}};
    if ((st = check_align(ptrs)) != SSD_OK) return st;
    const Range o[] = {range("n_accepted", n_accepted, 4 * b), range("next_token", next_token, 4 * b),
                       range("tokens", tokens, 4 * b * (K + 1)), range("workspace", workspace, ws_need)};
    const Range in[] = {range("target_probs", target_probs, e * t_n), range("draft_probs", draft_probs, e * d_n),
                        range("draft_tokens", draft_tokens, 4 * b * K), range("draft_lens", draft_lens, 4 * b),
                        range("uniforms", uniforms, 4 * b * (K + 1))};
    const InPlace allowed[] = {{-1, -1}};
    if ((st = check_alias(o, in, allowed)) != SSD_OK) return st;
    if (b == 0) return SSD_OK;  // nothing to enqueue

    p.target = target_probs;
    p.draft = K > 0 ? draft_probs : nullptr;
    p.tok = draft_tokens;
    p.lens = draft_lens;
    p.u = uniforms;
    p.n_accepted = n_accepted;
    p.next_token = next_token;
    p.tokens = tokens;
    p.sums = static_cast<double *>(workspace);
    (void)hipGetLastError();  // start from a clean error state
    return launched("verify_drafts", ssd::launch_verify_drafts(p, elem(dtype), static_cast<hipStream_t>(hip_stream)));
}

}  // extern "C"
