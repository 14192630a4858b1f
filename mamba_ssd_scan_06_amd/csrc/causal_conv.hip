// Depthwise causal convolution over tokens with the layer's activation and the
// split into the scan's inputs:
//     o[t][c] = act(bias[c] + sum_k weight[c][k] x[t-(W-1)+k][c])
//
// Every input is needed by W outputs of its own channel only, so the work is
// one read and one write per element: memory bound.  A thread owns 16 bytes of
// adjacent channels (fewer at the end of an output) and walks a run of tokens
// with the last W-1 inputs in registers; a run re-reads W-1 rows of the run
// before it.  Eight tokens' loads are in flight per thread (8 x 2048 tokens of
// 5376 bf16 channels: 78-85 us, 4.3 TB/s; one token of 64 sequences 5 us, the
// latency of one round of loads).  Products and sums are in fp32, rounded once
// on store; the states are raw inputs and never rounded.
#include "device_common.hpp"
#include "kernels.hpp"

namespace ssd {
namespace {

constexpr int kThreads = 256;
constexpr int kBatchLoads = 8;  // tokens loaded together

// Grid of a launch: threads are numbered channels first, then runs of tokens.
struct ConvGrid {
    int vecs[3];      // vectors of VEC channels per output
    unsigned vecs_all;
    unsigned work;    // vecs_all * runs
    int run;          // tokens per run
};

// One thread's run: channels c0 .. c0 + valid - 1 of x, from channel co of an
// output with `width` channels.  WHOLE: all VEC of them.
template <typename T, int W, bool WHOLE>
__device__ __forceinline__ void conv_run(const ConvParams &p, unsigned run, int run_len, int c0, int valid, T *out,
                                         int width) {
    constexpr int VEC = 16 / sizeof(T);
    const int64_t b = blockIdx.z, T_len = p.seqlen;
    const T *x = reinterpret_cast<const T *>(p.x) + b * p.x_bs + c0;
    const int64_t held = (b * (W - 1)) * p.total + c0;
    const int64_t t0 = (int64_t)run * run_len, t1 = min(t0 + run_len, T_len);
    auto load = [&](const auto *from) {
        if constexpr (WHOLE) return load_words(from);
        else return load_first(from, valid);
    };
    auto store = [&](T *to, const u32x4 &v) {
        if constexpr (WHOLE) store_words(to, v);
        else store_first(to, v, valid);
    };

    // All of a thread's loads before its first store: the weights, the W-1
    // inputs before the run (hist[k] is token t0 - (W-1) + k) and the states'
    // rows.  A single token is bound by the latency of this one round.
    float w[W][VEC], bias[VEC];
    if constexpr (WHOLE) {
        constexpr int WV = VEC * W / 4;
        u32x4 wv[WV];
#pragma unroll
        for (int k = 0; k < WV; ++k) wv[k] = load_words(p.weight + (int64_t)c0 * W + 4 * k);
#pragma unroll
        for (int i = 0; i < VEC; ++i)
#pragma unroll
            for (int k = 0; k < W; ++k) w[k][i] = word_f32(wv[(i * W + k) / 4], (i * W + k) % 4, float());
    } else {
#pragma unroll
        for (int i = 0; i < VEC; ++i)
#pragma unroll
            for (int k = 0; k < W; ++k) w[k][i] = p.weight[(int64_t)(c0 + min(i, valid - 1)) * W + k];
    }
#pragma unroll
    for (int i = 0; i < VEC; ++i) bias[i] = p.bias ? p.bias[c0 + (WHOLE ? i : min(i, valid - 1))] : 0.0f;
    u32x4 hist[W - 1];
#pragma unroll
    for (int k = 0; k < W - 1; ++k) hist[k] = u32x4{0u, 0u, 0u, 0u};
    if (run > 0) {  // t0 >= run_len >= W - 1
#pragma unroll
        for (int k = 0; k < W - 1; ++k) hist[k] = load(x + (t0 - (W - 1) + k) * p.x_ts);
    } else if (p.init_state) {
#pragma unroll
        for (int k = 0; k < W - 1; ++k)
            hist[k] = load(reinterpret_cast<const T *>(p.init_state) + held + (int64_t)k * p.total);
    }
    // Both states come from run 0's threads, which have read init_state by
    // the time they store: final_state may be the same memory.
    if (run == 0 && (p.state_out || p.final_state)) {
        u32x4 at[W - 1], fin[W - 1];
        // The W-1 inputs ending at token `last`, the first `before` of them held
        // from before token 0 (uniform conditions, constant indices).
        auto inputs = [&](u32x4 (&v)[W - 1], int64_t last) {
            const int before = (int)max((int64_t)(W - 2) - last, (int64_t)0);
            static_for<W>([&](auto c) {
                if (before != c) return;
#pragma unroll
                for (int k = 0; k < W - 1; ++k)
                    v[k] = k < c ? hist[(k + W - 1 - c) % (W - 1)] : load(x + (last - (W - 2) + k) * p.x_ts);
            });
        };
        auto keep = [&](void *to, const u32x4 (&v)[W - 1]) {
#pragma unroll
            for (int k = 0; k < W - 1; ++k) store(reinterpret_cast<T *>(to) + held + (int64_t)k * p.total, v[k]);
        };
        if (p.state_out) {
            const int64_t j = p.state_out_idx[b];
            inputs(at, j < -1 ? -1 : (j > T_len - 1 ? T_len - 1 : j));
        }
        if (p.final_state) inputs(fin, T_len - 1);
        if (p.state_out) keep(p.state_out, at);
        if (p.final_state) keep(p.final_state, fin);
    }

    // last[k]: the inputs of tokens t - (W-1) + k in fp32.
    float last[W - 1][VEC];
#pragma unroll
    for (int k = 0; k < W - 1; ++k)
#pragma unroll
        for (int i = 0; i < VEC; ++i) last[k][i] = word_f32(hist[k], i, T());
    auto token = [&](const u32x4 &v) {
        float r[VEC];
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            const float cur = word_f32(v, i, T());
            float acc = bias[i];
#pragma unroll
            for (int k = 0; k < W - 1; ++k) acc = fmaf(w[k][i], last[k][i], acc);
            acc = fmaf(w[W - 1][i], cur, acc);
#pragma unroll
            for (int k = 0; k + 1 < W - 1; ++k) last[k][i] = last[k + 1][i];
            last[W - 2][i] = cur;
            r[i] = p.silu ? silu<T>(acc) : acc;
        }
        return to_words(r, T());
    };
    out += b * T_len * width;
    wait_vmcnt<0>();  // weights and history: the loop then waits for its own loads one by one
    int64_t t = t0;
    for (; t + kBatchLoads <= t1; t += kBatchLoads) {
        u32x4 v[kBatchLoads];
#pragma unroll
        for (int q = 0; q < kBatchLoads; ++q) v[q] = load(x + (t + q) * p.x_ts);
#pragma unroll
        for (int q = 0; q < kBatchLoads; ++q) store(out + (t + q) * width, token(v[q]));
    }
    for (; t < t1; ++t) store(out + t * width, token(load(x + t * p.x_ts)));
}

template <typename T, int W>
__global__ __launch_bounds__(kThreads) void causal_conv_kernel(ConvParams p, ConvGrid gr) {
    constexpr int VEC = 16 / sizeof(T);
    const unsigned id = blockIdx.x * kThreads + threadIdx.x;
    if (id >= gr.work) return;
    const unsigned run = id / gr.vecs_all;
    int cv = (int)(id - run * gr.vecs_all);
    // The output this vector of channels belongs to, its first channel there
    // (co) and overall (c0).
    int o = 0, base = 0;
    if (cv >= gr.vecs[0]) {
        cv -= gr.vecs[0];
        base = p.channels[0];
        o = 1;
        if (cv >= gr.vecs[1]) {
            cv -= gr.vecs[1];
            base += p.channels[1];
            o = 2;
        }
    }
    const int width = o == 0 ? p.channels[0] : o == 1 ? p.channels[1] : p.channels[2];
    const int co = cv * VEC, valid = min(VEC, width - co);
    T *out = reinterpret_cast<T *>(o == 0 ? p.out[0] : o == 1 ? p.out[1] : p.out[2]) + co;
    if (valid == VEC) conv_run<T, W, true>(p, run, gr.run, base + co, valid, out, width);
    else conv_run<T, W, false>(p, run, gr.run, base + co, valid, out, width);
}

template <typename T, int W>
hipError_t run(const ConvParams &p, hipStream_t stream) {
    constexpr int VEC = 16 / sizeof(T);
    ConvGrid gr;
    int64_t vecs = 0;
    for (int i = 0; i < 3; ++i) {
        gr.vecs[i] = (p.channels[i] + VEC - 1) / VEC;
        vecs += gr.vecs[i];
    }
    gr.vecs_all = (unsigned)vecs;
    // Long runs re-read fewer rows; short ones give more threads.  From 32
    // tokens down to 8 until the GPU has eight waves per compute unit; and
    // longer ones where thread numbers would pass 31 bits.
    int64_t len = 32;
    while (len > kBatchLoads && vecs * ((p.seqlen + len - 1) / len) * p.batch < 8 * 256 * 64) len /= 2;
    while (vecs * ((p.seqlen + len - 1) / len) >= ((int64_t)1 << 31) - kThreads) len *= 2;
    gr.run = (int)len;
    const int64_t runs = std::max<int64_t>((p.seqlen + len - 1) / len, 1);
    gr.work = (unsigned)(vecs * runs);
    const dim3 grid((gr.work + kThreads - 1) / kThreads, 1, (unsigned)p.batch);
    causal_conv_kernel<T, W><<<grid, kThreads, 0, stream>>>(p, gr);
    return hipGetLastError();
}

template <typename T>
hipError_t by_width(const ConvParams &p, hipStream_t stream) {
    switch (p.width) {
        case 2: return run<T, 2>(p, stream);
        case 3: return run<T, 3>(p, stream);
        default: return run<T, 4>(p, stream);
    }
}

}  // namespace

hipError_t launch_causal_conv(const ConvParams &p, Elem e, hipStream_t stream) {
    return e == Elem::BF16 ? by_width<bf16>(p, stream) : by_width<float>(p, stream);
}

}  // namespace ssd
