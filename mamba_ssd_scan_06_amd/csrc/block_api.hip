// Host side of the gated delta rule and of the norms between blocks: argument
// checks and launches of ssd_gated_delta_fwd and ssd_residual_norm_fwd.  The
// public contract is include/ssd.h.
#include <math.h>

#include "host_common.hpp"
#include "kernels.hpp"
#include "ssd.h"

namespace {

using namespace ssd::host;
using ssd::extent3;
using ssd::fail;
using ssd::product;
using ssd::Range;
using ssd::range;

// Calls of more tokens run in chunks.  N and P 128, 32 heads, token by token and in
// chunks: bf16, 16 tokens of 1, 8 and 64 sequences 13.8 / 12.9, 17.9 / 19.1 and 108 /
// 82 us (118 / 114 with an accepted state), 12 tokens 11.6 / 12.7, 15.6 / 18.9 and 90 /
// 81 (100 / 112), 24 tokens 19.0 / 13.2, 24.0 / 19.4 and 143 / 85 (153 / 118); fp32,
// whose chunks cost twice as much, 24 tokens 17.8 / 19.3, 23.6 / 30.9 and 136 / 178 (150
// / 215), 32 tokens 22.4 / 20.0, 30.4 / 32.0 and 171 / 185.
int64_t delta_tokens(ssd_dtype dtype) { return dtype == SSD_DTYPE_BF16 ? 16 : 24; }

ssd_status check_delta(const ssd_delta_shape *s, ssd_dtype dtype) {
    if (!s) return fail(SSD_ERR_NULL, "shape is NULL");
    ssd_status st = check_dtype(dtype);
    if (st != SSD_OK) return st;
    if (s->batch < 0 || s->seqlen < 0) return fail(SSD_ERR_SHAPE, "batch and seqlen must be >= 0");
    if (s->nheads <= 0 || s->headdim <= 0 || s->dstate <= 0 || s->ngroups <= 0)
        return fail(SSD_ERR_SHAPE, "nheads, headdim, dstate and ngroups must be > 0");
    if (s->nheads % s->ngroups != 0)
        return fail(SSD_ERR_SHAPE, "ngroups (%lld) must divide nheads (%lld)", (long long)s->ngroups,
                    (long long)s->nheads);
    if (s->headdim % 16 != 0 || s->headdim > 256 || s->dstate % 16 != 0 || s->dstate > 256)
        return fail(SSD_ERR_UNSUPPORTED, "headdim %lld and dstate %lld must be multiples of 16 up to 256",
                    (long long)s->headdim, (long long)s->dstate);
    if (s->batch > kMaxBatch || s->nheads > kMaxBatch || s->seqlen >= kMaxTokens ||
        s->batch * s->nheads * ((s->headdim + 31) / 32) >= ((int64_t)1 << 24))
        return fail(SSD_ERR_UNSUPPORTED, "problem too large (batch and nheads <= 65535, seqlen < 2^31, "
                                         "batch * nheads * ceil(headdim / 32) < 2^24)");
    // The chunks' waves are one launch of fewer than 2^32 threads.
    if (s->batch * s->nheads * ((s->seqlen + ssd::kDeltaChunk - 1) / ssd::kDeltaChunk) >= ((int64_t)1 << 26))
        return fail(SSD_ERR_UNSUPPORTED, "problem too large (batch * nheads * ceil(seqlen / 32) < 2^26)");
    return SSD_OK;
}

ssd::DeltaParams delta_params(const ssd_delta_shape *s, ssd_dtype dtype) {
    ssd::DeltaParams p = {};
    p.batch = s->batch;
    p.seqlen = s->seqlen;
    p.nheads = (int)s->nheads;
    p.headdim = (int)s->headdim;
    p.dstate = (int)s->dstate;
    p.ngroups = (int)s->ngroups;
    p.heads_per_group = (int)(s->nheads / s->ngroups);
    p.q_bs = used_stride(s->batch, s->q_batch_stride);
    p.q_ts = used_stride(s->seqlen, s->q_token_stride);
    p.k_bs = used_stride(s->batch, s->k_batch_stride);
    p.k_ts = used_stride(s->seqlen, s->k_token_stride);
    p.v_bs = used_stride(s->batch, s->v_batch_stride);
    p.v_ts = used_stride(s->seqlen, s->v_token_stride);
    p.g_bs = used_stride(s->batch, s->g_batch_stride);
    p.g_ts = used_stride(s->seqlen, s->g_token_stride);
    p.beta_bs = used_stride(s->batch, s->beta_batch_stride);
    p.beta_ts = used_stride(s->seqlen, s->beta_token_stride);
    p.nchunks = s->seqlen > delta_tokens(dtype) ? (s->seqlen + ssd::kDeltaChunk - 1) / ssd::kDeltaChunk : 0;
    ssd::delta_ranges(p, elem(dtype));
    return p;
}

// Byte offsets behind the chunks' packs: the accepted index's tables, the ranges'
// states, maps and copy of init_state.
struct DeltaWorkspace {
    size_t at_off, state_off, map_off, init_off, total;
};
DeltaWorkspace delta_workspace(const ssd::DeltaParams &p, ssd_dtype dtype) {
    if (p.nchunks == 0) return {};
    auto up = [](size_t n) { return (n + 255) / 256 * 256; };
    const size_t bh = (size_t)p.batch * p.nheads, state = bh * p.headdim * p.dstate * sizeof(float),
                 map = bh * p.dstate * p.dstate * sizeof(float), more = p.ranges > 1 ? p.ranges - 1 : 0;
    DeltaWorkspace w = {};
    w.at_off = up(bh * p.nchunks * ssd::delta_pack_bytes(elem(dtype)));
    w.state_off = w.at_off + up(bh * ssd::delta_at_bytes());
    w.map_off = w.state_off + up(more * state);
    w.init_off = w.map_off + up(more > 0 ? (more - 1) * map : 0);
    w.total = w.init_off + (more > 0 ? state : 0);
    return w;
}

}  // namespace

extern "C" {

size_t ssd_gated_delta_workspace_bytes(const ssd_delta_shape *shape, ssd_dtype dtype) {
    if (check_delta(shape, dtype) != SSD_OK) return 0;
    return delta_workspace(delta_params(shape, dtype), dtype).total;
}

ssd_status ssd_gated_delta_fwd(const void *q, const void *k, const void *v, const float *g, const float *beta,
                               float scale, int qk_l2norm, const float *init_state, void *y, float *final_state,
                               const int32_t *state_out_idx, float *state_out, const ssd_delta_shape *s,
                               ssd_dtype dtype, void *workspace, size_t workspace_bytes, void *hip_stream) {
    ssd_status st = check_delta(s, dtype);
    if (st != SSD_OK) return st;
    const int64_t b = s->batch, T = s->seqlen, H = s->nheads, P = s->headdim, N = s->dstate, GN = s->ngroups * N;
    const int64_t q_n = extent3(b, s->q_batch_stride, T, s->q_token_stride, GN),
                  k_n = extent3(b, s->k_batch_stride, T, s->k_token_stride, GN),
                  v_n = extent3(b, s->v_batch_stride, T, s->v_token_stride, H * P),
                  g_n = g ? extent3(b, s->g_batch_stride, T, s->g_token_stride, H) : 0,
                  beta_n = extent3(b, s->beta_batch_stride, T, s->beta_token_stride, H), y_n = product(b, T, H * P),
                  st_n = product(b, H, P, N);
    if (q_n < 0 || k_n < 0 || v_n < 0 || g_n < 0 || beta_n < 0 || y_n < 0 || st_n < 0)
        return fail(SSD_ERR_SHAPE, "a stride is negative or the problem too large");
    if ((state_out == nullptr) != (state_out_idx == nullptr))
        return fail(SSD_ERR_ARGS, "state_out and state_out_idx must be given together");
    if (!isfinite(scale)) return fail(SSD_ERR_ARGS, "scale must be finite");
    if (b > 0 && T > 0 && (!q || !k || !v || !beta || !y))
        return fail(SSD_ERR_NULL, "q, k, v, beta and y are required");
    ssd::DeltaParams p = delta_params(s, dtype);
    const DeltaWorkspace ws = delta_workspace(p, dtype);
    const size_t ws_need = ws.total;
    if (ws_need > 0 && !workspace) return fail(SSD_ERR_WORKSPACE, "workspace is NULL");
    if (workspace_bytes < ws_need)
        return fail(SSD_ERR_WORKSPACE, "workspace has %zu bytes, needs %zu", workspace_bytes, ws_need);
    const size_t e = elem_size(dtype);
    const Ptr ptrs[] = {{"q", q, e}, {"k", k, e}, {"v", v, e}, {"g", g, 4}, {"beta", beta, 4},
                        {"init_state", init_state, 16}, {"y", y, e}, {"final_state", final_state, 16},
                        {"state_out_idx", state_out_idx, 4}, {"state_out", state_out, 16},
                        {"workspace", workspace, 16}};
    if ((st = check_align(ptrs)) != SSD_OK) return st;
    const Range o[] = {range("y", y, e * y_n), range("final_state", final_state, 4 * st_n),
                       range("state_out", state_out, 4 * st_n), range("workspace", workspace, ws_need)};
    const Range in[] = {range("q", q, e * q_n), range("k", k, e * k_n), range("v", v, e * v_n),
                        range("g", g, 4 * g_n), range("beta", beta, 4 * beta_n),
                        range("init_state", init_state, 4 * st_n), range("state_out_idx", state_out_idx, 4 * b)};
    const InPlace allowed[] = {{1, 5}};  // final_state == init_state
    if ((st = check_alias(o, in, allowed)) != SSD_OK) return st;
    if (b == 0 || (T == 0 && !final_state && !state_out)) return SSD_OK;  // nothing to enqueue

    p.q = q;
    p.k = k;
    p.v = v;
    p.g = g;
    p.beta = beta;
    p.scale = scale;
    p.l2norm = qk_l2norm != 0;
    p.init_state = init_state;
    p.y = y;
    p.final_state = final_state;
    p.state_out_idx = state_out_idx;
    p.state_out = state_out;
    (void)hipGetLastError();  // start from a clean error state
    const hipStream_t stream = static_cast<hipStream_t>(hip_stream);
    if (p.nchunks == 0) return launched("gated_delta", ssd::launch_delta_tokens(p, elem(dtype), stream));
    p.pack = static_cast<char *>(workspace);
    p.at_tables = reinterpret_cast<float *>(p.pack + ws.at_off);
    p.range_state = reinterpret_cast<float *>(p.pack + ws.state_off);
    p.range_map = reinterpret_cast<float *>(p.pack + ws.map_off);
    p.range_init = reinterpret_cast<float *>(p.pack + ws.init_off);
    return launched("gated_delta", ssd::launch_delta_chunks(p, elem(dtype), stream));
}

ssd_status ssd_residual_norm_fwd(const void *x, const void *residual, const void *gate, int gate_activation,
                                 int post_norm, const float *post_weight, const float *layer_scale,
                                 float residual_scale, float branch_scale, const float *weight, float eps, void *out,
                                 void *residual_out, const ssd_residual_norm_shape *s, ssd_dtype dtype,
                                 ssd_dtype stream_dtype, void *hip_stream) {
    if (!s) return fail(SSD_ERR_NULL, "shape is NULL");
    ssd_status st = check_dtype(dtype);
    if (st != SSD_OK) return st;
    if ((st = check_dtype(stream_dtype)) != SSD_OK) return st;
    if (stream_dtype != dtype && stream_dtype != SSD_DTYPE_F32)
        return fail(SSD_ERR_UNSUPPORTED, "stream_dtype must be dtype or fp32");
    if (gate_activation != SSD_ACT_NONE && gate_activation != SSD_ACT_SILU && gate_activation != SSD_ACT_SIGMOID)
        return fail(SSD_ERR_ARGS, "unknown activation %d", gate_activation);
    if (s->batch < 0 || s->seqlen < 0) return fail(SSD_ERR_SHAPE, "batch and seqlen must be >= 0");
    if (s->dim <= 0) return fail(SSD_ERR_SHAPE, "dim must be > 0");
    const int64_t rows = product(s->batch, s->seqlen);
    if (s->dim > kMaxWide || rows < 0 || rows >= kMaxTokens)
        return fail(SSD_ERR_UNSUPPORTED, "problem too large (dim <= 2^20, batch * seqlen < 2^31)");
    if (!(eps >= 0.0f) || isinf(eps)) return fail(SSD_ERR_ARGS, "eps must be finite and >= 0");
    if (!isfinite(residual_scale) || !isfinite(branch_scale))
        return fail(SSD_ERR_ARGS, "residual_scale and branch_scale must be finite");
    if (post_weight && !post_norm) return fail(SSD_ERR_ARGS, "post_weight needs post_norm");
    const int64_t x_n = extent3(s->batch, s->x_batch_stride, s->seqlen, s->x_token_stride, s->dim),
                  r_n = residual ? extent3(s->batch, s->residual_batch_stride, s->seqlen, s->residual_token_stride,
                                           s->dim) : 0,
                  gate_n = gate ? extent3(s->batch, s->gate_batch_stride, s->seqlen, s->gate_token_stride, s->dim) : 0,
                  out_n = product(rows, s->dim);
    if (x_n < 0 || r_n < 0 || gate_n < 0 || out_n < 0)
        return fail(SSD_ERR_SHAPE, "a stride is negative or the problem too large");
    if (rows > 0 && (!x || !out)) return fail(SSD_ERR_NULL, "x and out are required");
    const size_t e = elem_size(dtype), se = elem_size(stream_dtype);
    const Ptr ptrs[] = {{"x", x, e}, {"residual", residual, se}, {"gate", gate, e}, {"post_weight", post_weight, 4},
                        {"layer_scale", layer_scale, 4}, {"weight", weight, 4}, {"out", out, e},
                        {"residual_out", residual_out, se}};
    if ((st = check_align(ptrs)) != SSD_OK) return st;
    // In place only where an output's rows are the input's own.
    auto dense = [&](int64_t bs, int64_t ts) {
        return (s->seqlen == 1 || ts == s->dim) && (s->batch == 1 || bs == s->seqlen * s->dim);
    };
    const Range o[] = {range("out", out, e * out_n), range("residual_out", residual_out, se * out_n)};
    const Range in[] = {range("x", x, e * x_n), range("residual", residual, se * r_n), range("gate", gate, e * gate_n),
                        range("post_weight", post_weight, 4 * s->dim), range("layer_scale", layer_scale, 4 * s->dim),
                        range("weight", weight, 4 * s->dim)};
    const InPlace allowed[] = {{dense(s->x_batch_stride, s->x_token_stride) ? 0 : -1, 0},
                               {dense(s->residual_batch_stride, s->residual_token_stride) ? 1 : -1, 1}};
    if ((st = check_alias(o, in, allowed)) != SSD_OK) return st;
    if (rows == 0) return SSD_OK;  // nothing to enqueue

    ssd::ResidualNormParams p = {};
    p.x = x;
    p.residual = residual;
    p.gate = gate;
    p.post_weight = post_weight;
    p.layer_scale = layer_scale;
    p.weight = weight;
    p.out = out;
    p.residual_out = residual_out;
    p.rows = rows;
    p.seqlen = s->seqlen;
    p.x_bs = used_stride(s->batch, s->x_batch_stride);
    p.x_ts = used_stride(s->seqlen, s->x_token_stride);
    p.r_bs = used_stride(s->batch, s->residual_batch_stride);
    p.r_ts = used_stride(s->seqlen, s->residual_token_stride);
    p.gate_bs = used_stride(s->batch, s->gate_batch_stride);
    p.gate_ts = used_stride(s->seqlen, s->gate_token_stride);
    p.dim = (int)s->dim;
    p.activation = gate_activation;
    p.post_norm = post_norm != 0;
    p.residual_scale = residual_scale;
    p.branch_scale = branch_scale;
    p.eps = eps;
    (void)hipGetLastError();  // start from a clean error state
    return launched("residual_norm", ssd::launch_residual_norm(p, elem(dtype), elem(stream_dtype),
                                                               static_cast<hipStream_t>(hip_stream)));
}

}  // extern "C"
