// Depthwise causal convolution over tokens with the layer's activation and the
// split into the scan's inputs:
//     o[t][c] = act(bias[c] + sum_k weight[c][k] x[t-(W-1)+k][c])
// A thread owns VEC adjacent channels and walks a run of tokens with the last
// W-1 inputs in registers, so each input is read once (plus W-1 rows per run).
// Products and sums are in fp32, rounded once on store; the states are raw
// inputs and never rounded.
#include "device_common.hpp"
#include "kernels.hpp"

namespace ssd {
namespace {

constexpr int kThreads = 256;
constexpr int kRun = 32;  // tokens per run


template <typename T, int W, int VEC>
__global__ __launch_bounds__(kThreads) void causal_conv_kernel(ConvParams p) {
    using P = Pack<T, VEC>;
    const int c0 = (blockIdx.x * kThreads + threadIdx.x) * VEC;
    if (c0 >= p.total) return;
    const int64_t b = blockIdx.z, T_len = p.seqlen;
    const T *x = reinterpret_cast<const T *>(p.x) + b * p.x_bs + c0;
    const int64_t held = (b * (W - 1)) * p.total + c0;
    // The output this vector of channels belongs to.
    int o = 0, co = c0, width = p.channels[0];
    if (co >= width) {
        co -= width;
        o = 1;
        width = p.channels[1];
        if (co >= width) {
            co -= width;
            o = 2;
            width = p.channels[2];
        }
    }
    T *out = reinterpret_cast<T *>(o == 0 ? p.out[0] : o == 1 ? p.out[1] : p.out[2]) + b * T_len * width + co;

    P init[W - 1];
#pragma unroll
    for (int k = 0; k < W - 1; ++k) {
#pragma unroll
        for (int i = 0; i < VEC; ++i) init[k].v[i] = from_f32<T>(0.0f);
        if (p.init_state && blockIdx.y == 0)
            init[k] = *reinterpret_cast<const P *>(reinterpret_cast<const T *>(p.init_state) + held +
                                                   (int64_t)k * p.total);
    }
    // Input of token t, which may be one held from before token 0 (t >= 1 - W).
    // Only run 0 asks for those.
    auto input = [&](int64_t t) {
        if (t >= 0) return *reinterpret_cast<const P *>(x + t * p.x_ts);
        P r = init[0];
#pragma unroll
        for (int k = 1; k < W - 1; ++k)
            if (t + (W - 1) == k) r = init[k];
        return r;
    };
    // Both states come from run 0's threads, which have read init_state by
    // now: final_state may be the same memory.
    if (blockIdx.y == 0) {
        if (p.state_out) {
            int64_t j = p.state_out_idx[b];
            j = j < -1 ? -1 : (j > T_len - 1 ? T_len - 1 : j);
#pragma unroll
            for (int k = 0; k < W - 1; ++k)
                *reinterpret_cast<P *>(reinterpret_cast<T *>(p.state_out) + held + (int64_t)k * p.total) =
                    input(j - (W - 2) + k);
        }
        if (p.final_state) {
#pragma unroll
            for (int k = 0; k < W - 1; ++k)
                *reinterpret_cast<P *>(reinterpret_cast<T *>(p.final_state) + held + (int64_t)k * p.total) =
                    input(T_len - (W - 1) + k);
        }
    }

    float w[W][VEC], bias[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
        bias[i] = p.bias ? p.bias[c0 + i] : 0.0f;
#pragma unroll
        for (int k = 0; k < W; ++k) w[k][i] = p.weight[(int64_t)(c0 + i) * W + k];
    }
    for (int64_t t0 = (int64_t)blockIdx.y * kRun; t0 < T_len; t0 += (int64_t)gridDim.y * kRun) {
        const int64_t t1 = t0 + kRun < T_len ? t0 + kRun : T_len;
        float hist[W - 1][VEC];
#pragma unroll
        for (int k = 0; k < W - 1; ++k) {
            const P v = input(t0 - (W - 1) + k);
#pragma unroll
            for (int i = 0; i < VEC; ++i) hist[k][i] = to_f32(v.v[i]);
        }
        for (int64_t t = t0; t < t1; ++t) {
            const P v = *reinterpret_cast<const P *>(x + t * p.x_ts);
            P r;
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                const float cur = to_f32(v.v[i]);
                float acc = bias[i];
#pragma unroll
                for (int k = 0; k < W - 1; ++k) acc = fmaf(w[k][i], hist[k][i], acc);
                acc = fmaf(w[W - 1][i], cur, acc);
#pragma unroll
                for (int k = 0; k + 1 < W - 1; ++k) hist[k][i] = hist[k + 1][i];
                hist[W - 2][i] = cur;
                r.v[i] = from_f32<T>(p.silu ? silu(acc) : acc);
            }
            *reinterpret_cast<P *>(out + t * width) = r;
        }
    }
}

template <typename T, int W, int VEC>
hipError_t run(const ConvParams &p, hipStream_t stream) {
    const int64_t runs = (p.seqlen + kRun - 1) / kRun;
    const unsigned gy = (unsigned)std::min<int64_t>(std::max<int64_t>(runs, 1), 65535);
    const unsigned gx = (unsigned)((p.total / VEC + kThreads - 1) / kThreads);
    causal_conv_kernel<T, W, VEC><<<dim3(gx, gy, (unsigned)p.batch), kThreads, 0, stream>>>(p);
    return hipGetLastError();
}

template <typename T>
hipError_t by_width(const ConvParams &p, hipStream_t stream) {
    switch (p.width) {
        case 2: return run<T, 2, 1>(p, stream);
        case 3: return run<T, 3, 1>(p, stream);
        default: return run<T, 4, 1>(p, stream);
    }
}

}  // namespace

hipError_t launch_causal_conv(const ConvParams &p, Elem e, hipStream_t stream) {
    return e == Elem::BF16 ? by_width<bf16>(p, stream) : by_width<float>(p, stream);
}

}  // namespace ssd
